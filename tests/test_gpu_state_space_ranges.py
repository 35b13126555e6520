"""The selective scan where single tokens, or parameters, leave the ordinary range: a step that clears the state among
ordinary ones, and what is not a number in a parameter.  Tolerances as in test_gpu_state_space.py."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import state_space as S
from tests.test_gpu_state_space import FORMS, FP32, W, _close, _close_chunked, _dev, _f64, _sizes, _ssm_case   # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,algo", FORMS)
@pytest.mark.parametrize("step", (60.0, 200.0, 1e4, 6e4, 1e13, 1e18, 1e30))
def test_one_step_clears_the_state(W, dtype, algo, step):   # noqa: F811
    """A step of any size at a token with x = 0 decays the state and nothing else: the ordinary decays behind it keep their
    weights, in every output.  (dx at that token itself is as large as the step, so it is looked at apart.)"""
    if dtype == "f16" and step > 200:
        pytest.skip("dx at the token, a few times the step, leaves this type")
    rng = np.random.default_rng(500)
    B, T, H, G, N = 2, 300, 4, 2, 64
    dev, ref = _ssm_case(rng, dtype, B, T, H, G, N, reset=None, A_scale=0.25)
    big = np.zeros((B, T), bool)
    big[0, [3, 40, 41, 127, 200]] = True
    big[1, [0, 128, 255, 299]] = True
    for b, t in np.argwhere(big):
        dev["x"][b, t] = 0
        ref["x"][b, t] = 0
        dev["dt"][b, t] = step
    ref["dt"] = _f64(dev["dt"])
    y, s, ws = W.ssm_forward(**dev, algo=algo)
    yo, so = S.ssm_forward(**ref)
    dy, dy64 = _dev(rng.standard_normal(ref["x"].shape), dtype)
    ds, ds64 = _dev(rng.standard_normal(so.shape).astype(np.float32))
    g = W.ssm_backward(dy=dy, workspace=ws, dsT=ds, algo=algo, **dev)
    go = S.ssm_backward(dy=dy64, dsT=ds64, **ref)
    _close(s, so, "f32", FP32, "s_out")
    for n in ("dA", "dD", "ddt_bias", "ds0"):
        _close(g[n], go[n], "f32", FP32, n)
    got = {"y": y, **g}
    want = {"y": yo, **go}
    # dL/da at a token is formed as a difference of sums over the paths of up to 128 tokens (128 terms each, every one rounded
    # to 2^-53, and none larger than 2^10 of the largest ddt's terms, whose softplus' derivative is at least 2^-10 here): where
    # a decay leaves next to nothing, ddt is off by up to 128 * 128 * 2^-53 * 2^10 = 2^-29 of that, and not of its own size.
    size = {"y": np.abs(_sizes(ref, True)), **{n: np.abs(v) for n, v in _sizes(ref, True, dy64, ds64).items()}}
    size["ddt"] = np.maximum(size["ddt"], 2.0 ** -20 * size["ddt"].max((0, 1)))   # (times 2^-8: 2^-28)
    for n in ("y", "dx", "ddt", "db", "dc"):
        for part in (~big, big) if n == "dx" else (np.ones_like(big),):
            if algo == "chunked":
                _close_chunked(got[n][part], want[n][part], size[n][part], n)
            else:
                _close(got[n][part], want[n][part], dtype, FP32, n)


@pytest.mark.parametrize("dtype,algo", FORMS)
@pytest.mark.parametrize("name", ("A", "dt_bias", "D"))
def test_what_is_not_a_number_in_a_parameter_shows(W, dtype, algo, name):   # noqa: F811
    """A NaN in one head's parameter reaches that head's outputs and gradients, and no other head's (db and dc are the group's)."""
    import torch
    rng = np.random.default_rng(510)
    dev, _ = _ssm_case(rng, dtype, 2, 150, 4, 4, 64, reset=None)
    dy = torch.randn(2, 150, 4, 64, device="cuda").to(dev["x"].dtype)

    def run():
        y, s, ws = W.ssm_forward(**dev, algo=algo)
        return {"y": y, "s": s, **W.ssm_backward(dy=dy, workspace=ws, algo=algo, **dev)}
    want = run()
    dev[name] = dev[name].clone()
    dev[name][1] = float("nan")
    got = run()
    other = [0, 2, 3]
    dims = {"y": 2, "s": 1, "dx": 2, "ddt": 2, "db": 2, "dc": 2, "ds0": 1, "dA": 0, "dD": 0, "ddt_bias": 0}
    for n, t in got.items():
        a, b = t.movedim(dims[n], 0), want[n].movedim(dims[n], 0)
        assert torch.equal(a[other], b[other]), n
    reached = {"A": ("y", "s", "dA", "ddt_bias"), "dt_bias": ("y", "s", "dA", "ddt_bias"), "D": ("y", "dx")}[name]
    for n in reached:
        assert got[n].movedim(dims[n], 0)[1].isnan().any(), n
    if name == "A":
        assert got["y"][:, 1:, 1].isnan().all() and got["s"][:, 1].isnan().all()


@pytest.mark.parametrize("dtype", ("f32", "bf16", "f16"))
def test_runs_whose_decay_leaves_the_range(W, dtype):   # noqa: F811
    """Token order, a row cut into runs, decays of e^3 per token: over a run of 35 the product is e^105, no fp32 number, but what
    it multiplies is zero until the last tokens (and, for the gradients, behind the first)."""
    import torch
    rng = np.random.default_rng(520)
    B, T, H, N = 1, 140, 2, 64
    dev, ref = _ssm_case(rng, dtype, B, T, H, 1, N, reset=None, state=False, params=False, strided=False)
    assert W.lib().wkv7_ssm_workspace_bytes(W.make_desc(B, T, H, dev["x"].dtype, "scan", N=N), W.Ssm(1, None, None, None, 0, 0, 0, 0, 0)) \
        > 4 * B * H * 3 * 64 * N                                    # the row is cut into runs
    dev["dt"].fill_(1.0)
    dev["A"].fill_(3.0)
    ref["dt"], ref["A"] = np.ones((B, T, H)), np.full(H, 3.0)
    dev["x"][:, : T - 2] = 0
    ref["x"] = _f64(dev["x"])
    y, s, ws = W.ssm_forward(**dev, softplus=False, algo="scan")
    yo, so = S.ssm_forward(**ref, softplus=False)
    _close(s, so, "f32", FP32, "s_out")
    _close(y, yo, dtype, FP32, "y")
    dy = torch.zeros_like(dev["x"])
    dy[:, :2] = torch.randn(B, 2, H, 64, device="cuda").to(dy.dtype)
    g = W.ssm_backward(dy=dy, workspace=ws, softplus=False, algo="scan", **dev)
    go = S.ssm_backward(dy=_f64(dy), softplus=False, **ref)
    for n in ("ds0", "dx", "db", "dc", "ddt", "dA"):
        _close(g[n], go[n], "f32" if n in ("ds0", "dA") else dtype, FP32, n)


@pytest.mark.parametrize("dtype", ("f32", "bf16", "f16"))
def test_token_order_backward_without_a_workspace(W, dtype):   # noqa: F811
    """Token order walks forward again: no workspace and the same bits; the chunked form refuses."""
    import torch
    rng = np.random.default_rng(530)
    dev, _ = _ssm_case(rng, dtype, 2, 200, 4, 2, 64)
    dy = torch.randn(2, 200, 4, 64, device="cuda").to(dev["x"].dtype)
    _, _, ws = W.ssm_forward(**dev, algo="scan")
    want = W.ssm_backward(dy=dy, workspace=ws, algo="scan", **dev)
    got = W.ssm_backward(dy=dy, workspace=None, algo="scan", **dev)
    assert all(torch.equal(got[n], want[n]) for n in want)
    if dtype == "bf16":
        for algo in ("auto", "chunked"):
            with pytest.raises(ValueError, match="workspace"):
                W.ssm_backward(dy=dy, workspace=None, algo=algo, **dev)
