"""The state-space layer on memory full of NaN: every output, workspace and scratch that the binding allocates is filled with
0xFF bytes before the call, and the results are the same bits as on other memory (nothing unwritten is read or returned)."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_gpu_state_space import DT, FORMS, W, _conv_case, _dev, _ssm_case, _t   # noqa: F401

pytestmark = pytest.mark.gpu


def _compare(monkeypatch, run):
    import torch
    want = run()
    assert all(t.float().isfinite().all() for t in want.values())
    real = torch.Tensor.new_empty
    count = [0]

    def poisoned(self, *a, **k):
        t = real(self, *a, **k)
        if t.is_cuda and t.numel() > 0:
            t.view(-1).view(torch.uint8).fill_(0xFF)
            count[0] += 1
        return t
    monkeypatch.setattr(torch.Tensor, "new_empty", poisoned)
    got = run()
    assert count[0] > 0
    for n in want:
        a, b = (t[n].view(torch.uint8) if t[n].dtype == torch.float8_e4m3fn else t[n] for t in (got, want))
        assert torch.equal(a, b), n


@pytest.mark.parametrize("dtype,algo", FORMS)
@pytest.mark.parametrize("B,T,H,G,N", ((2, 1, 2, 1, 64), (2, 129, 6, 3, 128), (1, 791, 4, 2, 64), (1, 300, 12, 1, 128)))
def test_scan(W, monkeypatch, dtype, algo, B, T, H, G, N):   # noqa: F811
    import torch
    rng = np.random.default_rng(1100 + T)
    dev, _ = _ssm_case(rng, dtype, B, T, H, G, N)
    dy, ds = torch.randn(B, T, H, 64, device="cuda").to(_t(dtype)), torch.randn(B, H, 64, N, device="cuda")

    def run():
        y, s, ws = W.ssm_forward(**dev, algo=algo)
        return {"y": y, "s": s, **W.ssm_backward(dy=dy, workspace=ws, dsT=ds, algo=algo, **dev)}
    _compare(monkeypatch, run)


@pytest.mark.parametrize("dtype", DT)
def test_convolution_and_norm(W, monkeypatch, dtype):   # noqa: F811
    import torch
    rng = np.random.default_rng(1110)
    x, _, k, reset, _ = _conv_case(rng, dtype, 3, 77, 200, 4, "some", True, True)
    dy, _ = _dev(rng.standard_normal((3, 77, 200)), dtype)
    h, z, d = (torch.randn(700, 1152, device="cuda").to(_t(dtype)) for _ in range(3))
    w = torch.randn(1152, device="cuda")

    def run():
        y, s = W.conv_forward(x, k["weight"][0], k["bias"][0], k["s0"][0], reset)
        r = {"y": y, "s": s, **W.conv_backward(x, k["weight"][0], dy, k["bias"][0], k["s0"][0], reset)}
        for groups, block in ((1, 128), (3, -1)):
            r.update({f"{n}{block}": t for n, t in W.rms_forward(h, w, 1e-5, residual=z, groups=groups, quant_block=block).items()})
        r.update({"n" + n: t for n, t in W.rms_backward(h, w, d, 1e-5, gate=z, groups=3).items()})
        return r
    _compare(monkeypatch, run)
