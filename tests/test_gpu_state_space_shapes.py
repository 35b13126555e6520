"""The state-space layer at sizes whose loops turn more than once: rows of the scan cut into runs that remember, the
convolution's long runs of tokens, and the norm's CTAs with several slices.  The scan against the fp64 oracle; the other two,
too large for it, against the same formulas in fp64 torch.  Tolerances as in test_gpu_state_space.py."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_gpu_state_space import DT, FORMS, FP32, W, _ssm_case, _ssm_check, _t   # noqa: F401

pytestmark = pytest.mark.gpu


def _close64(got, ref, dtype, what):
    """As _close, on the device: the largest error beyond the half step of storing, relative to the reference's RMS."""
    import torch
    assert got.shape == ref.shape and bool(got.isfinite().all()), what
    got = got.double()
    d = (got - ref).abs()
    if dtype != "f32":
        top = torch.maximum(got.abs(), ref.abs())
        step = torch.ldexp(torch.ones_like(top), torch.floor(torch.log2(top.clamp(min=1e-300))).int() - (7 if dtype == "bf16" else 10) - 1)
        d = (d - torch.where(top > 0, step, torch.zeros_like(step))).clamp(min=0)
    err = (d.max() / ref.square().mean().sqrt()).item()
    assert err <= FP32, (what, err)


# ------------------------------------------------------------------ scan
@pytest.mark.parametrize("dtype,algo", FORMS)
@pytest.mark.parametrize("reset", (None, "one"))
@pytest.mark.parametrize("H,T,N", ((2, 900, 64), (1, 1021, 128), (3, 769, 128)))
def test_cut_rows_remember(W, monkeypatch, dtype, algo, reset, H, T, N):   # noqa: F811
    """A row cut into runs whose decays leave a good part of the state from end to end, so that s0 reaches the last token and
    dsT the first; or with one reset in a run in the middle.

    The fp32 tolerance counts 512 operations in a chain.  In token order a state that is remembered for T tokens is the end
    of 3 T of them (a decay, its product, a sum), so there the same formula takes 3 T: 3 T * 2^-24 * 3."""
    import torch
    from tests import test_gpu_state_space as base
    if algo == "scan":
        monkeypatch.setattr(base, "FP32", 3 * T * 2.0 ** -24 * 3)
    rng = np.random.default_rng(600 + T)
    dev, ref = _ssm_case(rng, dtype, 1, T, H, 1, N, reset=None, A_scale=1e-3)
    states = 4 * H * (-(-T // 128) + 1) * 64 * N
    desc = W.make_desc(1, T, H, _t(dtype), algo, N=N)
    assert W.lib().wkv7_ssm_workspace_bytes(desc, W.Ssm(1, None, None, None, 1, 0, 0, 0, 0)) >= states + 3 * 4 * H * 64 * N   # three runs at least
    if reset:
        ref["reset"] = np.zeros((1, T), np.uint8)
        ref["reset"][0, T // 2 + 5] = 1
        dev["reset"] = torch.from_numpy(ref["reset"]).cuda()
    else:   # what is left at the end of what the row starts from
        step = np.logaddexp(0.0, ref["dt"] + ref["dt_bias"])
        assert np.exp((step * ref["A"]).sum(1)).min() > 0.05
    _ssm_check(W, rng, dtype, algo, dev, ref)


# ------------------------------------------------------------------ convolution
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("taps,T,run,state", ((4, 1203, 64, True), (3, 1203, 64, False), (2, 1200, 64, True), (4, 1201, 64, False), (4, 603, 32, True),
                                              (3, 301, 16, True)))
def test_conv_long_runs(W, dtype, taps, T, run, state):   # noqa: F811
    """Enough rows and channels for runs of 64, 32 and 16 tokens (the backward's; the forward's are half as long): several batches of
    four in a run, with resets inside, at the ends and just behind the ends of batches and runs, and a ragged last run."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(700 + T + taps)
    B, D = 8, 2048
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    x, dy = r(B, T, D + 8).to(_t(dtype))[..., 8:], r(B, T, D).to(_t(dtype))
    w, bias = r(D, taps), r(D)
    s0, dsT = (r(B, taps - 1, D).to(_t(dtype)) for _ in range(2)) if state else (None, None)
    desc = W.make_desc(B, T, 0, _t(dtype))
    assert W.lib().wkv7_conv_scratch_bytes(desc, W.Conv(D, taps, 1, None, None, 0)) == 4 * B * -(-T // run) * (taps + 1) * D
    reset = (torch.rand(B, T, generator=g, device="cuda") < 0.01).to(torch.uint8)
    reset[1] = 0                                           # a row without any
    for t in (3, 4, 5, 31, 32, 63, 64, 65, 67, 127, 130, 200, 201, T - 1):
        reset[t % B, t] = 1
    y, s_out = W.conv_forward(x, w, bias, s0, reset)
    got = W.conv_backward(x, w, dy, bias, s0, reset, dsT)
    # the formulas in fp64: the taps that no reset cuts off
    x64, w64, b64 = (v.double().requires_grad_(True) for v in (x, w, bias))
    past = (torch.zeros(B, taps - 1, D, device="cuda", dtype=torch.float64) if s0 is None else s0.double()).requires_grad_(True)
    full = torch.cat([past, x64], 1)
    seg = torch.cat([torch.zeros(B, taps - 1, device="cuda", dtype=torch.int64), reset.long().cumsum(1)], 1)
    u = b64 + 0.0 * x64
    for j in range(taps):
        at = taps - 1 - j
        u = u + full[:, at:at + T] * w64[:, taps - 1 - j] * (seg[:, at:at + T] == seg[:, taps - 1:]).double()[..., None]
    y64 = torch.nn.functional.silu(u)
    s64 = full[:, T:] * (seg[:, T:] == seg[:, -1:]).double()[..., None]
    _close64(y, y64.detach(), dtype, "y")
    assert torch.equal(s_out.double(), s64.detach())
    loss = (y64 * dy.double()).sum() + ((s64 * dsT.double()).sum() if state else 0.0)
    loss.backward()
    _close64(got["dx"], x64.grad, dtype, "dx")
    _close64(got["ds0"], past.grad, dtype, "ds0")
    _close64(got["dweight"], w64.grad, "f32", "dweight")
    _close64(got["dbias"], b64.grad, "f32", "dbias")


# ------------------------------------------------------------------ norm
# rows, channels, slices per row: more slices than the forward has CTAs (2368) and more rows than one wave of the backward's,
# with one, two and four vectors per thread, several slices per CTA, and a ragged end
NORMS = ((5003, 2048, 1), (100003, 64, 1), (2501, 12288, 1), (2500, 16384, 1), (2503, 6144, 3), (20011, 192, 3))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kind", ("residual", "gate"))
@pytest.mark.parametrize("rows,D,groups", NORMS)
def test_rms_many_rows(W, dtype, kind, rows, D, groups):   # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(800 + D)
    x, z, dout, dh = (torch.randn(rows, D, generator=g, device="cuda").to(_t(dtype)) for _ in range(4))
    w = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
    f = W.rms_forward(x, w, 1e-5, groups=groups, **{kind: z})
    if kind == "residual":
        assert torch.equal(f["h"], (x.float() + z.float()).to(x.dtype))
        got = W.rms_backward(f["h"], w, dout, 1e-5, groups=groups, dh=dh)
        h = f["h"].double()
    else:
        got = W.rms_backward(x, w, dout, 1e-5, groups=groups, gate=z)
        s = torch.sigmoid(z.double())
        h = x.double() * z.double() * s
    v = h.view(rows, groups, -1)
    rstd = (v.square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    xh = (v * rstd).view(rows, D)
    _close64(f["out"], xh * w.double(), dtype, "out")
    d64 = dout.double()
    _close64(got["dweight"], (d64 * xh).sum(0), "f32", "dweight")
    q = (d64 * w.double()).view_as(v)
    dv = (rstd * (q - xh.view_as(v) * (q * xh.view_as(v)).mean(-1, keepdim=True))).view(rows, D)
    if kind == "residual":
        _close64(got["dx"], dv + dh.double(), dtype, "dx")
    else:
        _close64(got["dx"], dv * z.double() * s, dtype, "dx")
        _close64(got["dgate"], dv * x.double() * s * (1.0 + z.double() * (1.0 - s)), dtype, "dgate")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("block,rows,D,groups", ((128, 5003, 2048, 1), (-1, 5003, 2048, 1), (128, 40009, 128, 1), (-1, 100003, 64, 1), (128, 2501, 12288, 1),
                                                 (-1, 2501, 16384, 1), (128, 5003, 768, 2), (-1, 20011, 192, 3)))
def test_rms_e4m3_many_rows(W, dtype, block, rows, D, groups):   # noqa: F811
    """Half a step of e4m3 per code (2^-4 of the value, 2^-10 of the scale below its normal range) and the scale's largest value
    over 448, for every slice, with the sum stored beside it."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(900 + D)
    x, r = (torch.randn(rows, D, generator=g, device="cuda").to(_t(dtype)) for _ in range(2))
    w = 1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")
    f = W.rms_forward(x, w, 1e-5, residual=r, groups=groups, quant_block=block)
    assert torch.equal(f["h"], (x.float() + r.float()).to(x.dtype))
    v = f["h"].double().view(rows, groups, -1)
    ref = ((v * (v.square().mean(-1, keepdim=True) + 1e-5).rsqrt()).view(rows, D) * w.double()).view(rows, -1, 128 if block > 0 else D // groups)
    scale = f["scale"].double().view(rows, -1, 1)
    assert ((scale - ref.abs().amax(2, keepdim=True) / 448.0).abs() <= 1e-5 * scale).all()
    code = f["q"].float().double().view_as(ref) * scale
    assert ((code - ref).abs() <= torch.maximum(ref.abs() * 2.0 ** -4, scale * 2.0 ** -10) * (1.0 + 1e-4)).all()
