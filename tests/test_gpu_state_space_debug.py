"""The bounds-checked build of the state-space layer over strided inputs, states, masks and every direction: the same bits
as the release build, and no check fails."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_gpu_state_space import DT, FORMS, W, _conv_case, _dev, _ssm_case, _t   # noqa: F401

pytestmark = pytest.mark.gpu


def _both(W, run):   # noqa: F811
    import torch
    want = run()
    prev = W.use_build("debug")
    try:
        W.device_status()
        got = run()
        assert W.device_status() == W.OK
    finally:
        W.use_build(prev)
    for n in want:
        a, b = (t[n].view(torch.uint8) if t[n].dtype == torch.float8_e4m3fn else t[n] for t in (got, want))
        assert torch.equal(a, b), n


@pytest.mark.parametrize("dtype,algo", FORMS)
@pytest.mark.parametrize("B,T,H,G,N", ((2, 301, 4, 2, 64), (1, 790, 3, 1, 128)))
def test_scan(W, dtype, algo, B, T, H, G, N):   # noqa: F811
    """Slices of wider rows, initial states and their gradients; the second shape is cut into runs."""
    import torch
    rng = np.random.default_rng(1000 + T)
    dev, _ = _ssm_case(rng, dtype, B, T, H, G, N)
    wide = torch.randn(B, T, H + 5, device="cuda").to(_t(dtype))
    dev["dt"] = wide[..., 3:3 + H]
    dy, ds = torch.randn(B, T, H, 64, device="cuda").to(_t(dtype)), torch.randn(B, H, 64, N, device="cuda")

    def run():
        y, s, ws = W.ssm_forward(**dev, algo=algo)
        y2, s2, _ = W.ssm_forward(**dev, algo=algo, need_workspace=False)
        return {"y": y, "s": s, "y2": y2, "s2": s2, **W.ssm_backward(dy=dy, workspace=ws, dsT=ds, algo=algo, **dev)}
    _both(W, run)


@pytest.mark.parametrize("dtype", DT)
def test_steps(W, dtype):   # noqa: F811
    import torch
    rng = np.random.default_rng(1010)
    dev, _ = _ssm_case(rng, dtype, 5, 3, 4, 2, 128, reset=None)
    x, _, k, _, _ = _conv_case(rng, dtype, 5, 9, 72, 4, None, True, True)
    active = torch.tensor([1, 0, 1, 1, 0], dtype=torch.uint8, device="cuda")

    def run():
        state, conv = dev["s0"].clone(), k["s0"][0].clone()
        y = W.ssm_step(dev["x"][:, 1], dev["dt"][:, 1], dev["A"], dev["b"][:, 1], dev["c"][:, 1], state, dev["D"], dev["dt_bias"], active)
        u = W.conv_step(x[:, 3], k["weight"][0], conv, k["bias"][0], active)
        return {"y": y, "state": state, "u": u, "conv": conv}
    _both(W, run)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("taps,T", ((4, 2), (2, 33), (4, 200)))
def test_convolution(W, dtype, taps, T):   # noqa: F811
    rng = np.random.default_rng(1020 + T)
    x, _, k, reset, _ = _conv_case(rng, dtype, 3, T, 200, taps, "some", True, True)
    dy, _ = _dev(rng.standard_normal((3, T, 200)), dtype)
    ds, _ = _dev(rng.standard_normal((3, taps - 1, 200)), dtype)

    def run():
        y, s = W.conv_forward(x, k["weight"][0], k["bias"][0], k["s0"][0], reset)
        return {"y": y, "s": s, **W.conv_backward(x, k["weight"][0], dy, k["bias"][0], k["s0"][0], reset, ds)}
    _both(W, run)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("rows,D,groups", ((3001, 384, 3), (5, 16384, 1)))
def test_norm(W, dtype, rows, D, groups):   # noqa: F811
    import torch
    x, z, d = (torch.randn(rows, D, device="cuda").to(_t(dtype)) for _ in range(3))
    w = torch.randn(D, device="cuda")

    def run():
        f = W.rms_forward(x, w, 1e-5, residual=z, groups=groups)
        r = {"h": f["h"], "out": f["out"], "gated": W.rms_forward(x, w, 1e-5, gate=z, groups=groups)["out"]}
        for block in (128, -1):
            r.update({f"{n}{block}": t for n, t in W.rms_forward(x, w, 1e-5, groups=groups, quant_block=block).items()})
        r.update(W.rms_backward(x, w, d, 1e-5, groups=groups, gate=z))
        r.update({"h" + n: t for n, t in W.rms_backward(f["h"], w, d, 1e-5, groups=groups, dh=z).items()})
        return r
    _both(W, run)
