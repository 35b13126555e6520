"""The state-space layer's entry points without a GPU: every bad argument is refused before anything is launched,
sizes are counted, empty calls succeed, and the binding refuses what the C ABI cannot see."""
from __future__ import annotations

import ctypes
import math

import pytest

FAKE = 0x10000       # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    from linear_recurrent_lm_b200 import build
    build.build_all()
    from linear_recurrent_lm_b200 import wkv7
    return wkv7


def _desc(L, dtype="bfloat16", **over):
    import torch
    k = dict(B=2, T=16, H=4, N=64, algo="auto", flags=0)
    k.update(over)
    return L.make_desc(k["B"], k["T"], k["H"], getattr(torch, dtype), k["algo"], N=k["N"], flags=k["flags"])


def _conv(L, desc, cv, **over):
    p = dict(x=FAKE, s0=None, reset=None, y=FAKE, s_out=None)
    p.update(over)
    return L.lib().wkv7_conv_forward(desc, cv, p["x"], p["s0"], p["reset"], p["y"], p["s_out"], None)


def test_conv_refusals(L):
    ok = lambda **k: L.Conv(*[{**dict(D=16, W=4, silu=1, weight=FAKE, bias=None, x_ld=0), **k}[n] for n, _ in L.Conv._fields_])   # noqa: E731
    d = _desc(L)
    assert _conv(L, None, ok()) == L.ERR_NULL and _conv(L, d, None) == L.ERR_NULL
    for k in (dict(W=1), dict(W=5), dict(D=12)):
        assert _conv(L, d, ok(**k)) == L.ERR_UNSUPPORTED
    assert _conv(L, d, ok(D=-8)) == L.ERR_SHAPE
    assert _conv(L, d, ok(weight=None)) == L.ERR_NULL and _conv(L, d, ok(weight=FAKE + 4)) == L.ERR_ALIGN
    assert _conv(L, d, ok(bias=FAKE + 8)) == L.ERR_ALIGN
    assert _conv(L, d, ok(x_ld=8)) == L.ERR_SHAPE and _conv(L, d, ok(x_ld=20)) == L.ERR_ALIGN
    assert _conv(L, d, ok(), x=None) == L.ERR_NULL and _conv(L, d, ok(), y=FAKE + 8) == L.ERR_ALIGN
    assert _conv(L, d, ok(), s0=FAKE, s_out=FAKE) == L.ERR_UNSUPPORTED
    assert _conv(L, _desc(L, flags=L.FLAG_LOG_DECAY), ok()) == L.ERR_UNSUPPORTED
    bad = _desc(L)
    bad.dtype = 7
    assert _conv(L, bad, ok()) == L.ERR_DTYPE
    assert _conv(L, _desc(L, T=-1), ok()) == L.ERR_SHAPE and _conv(L, _desc(L, T=1 << 62), ok()) == L.ERR_SHAPE
    assert _conv(L, _desc(L, B=0), ok(), x=None, y=None) == L.OK
    lib = L.lib()
    assert lib.wkv7_conv_scratch_bytes(d, ok(weight=None)) > 0 and lib.wkv7_conv_scratch_bytes(d, ok(W=9)) == 0
    back = lambda desc, cv, dx=FAKE, dw=FAKE, sc=FAKE: lib.wkv7_conv_backward(desc, cv, FAKE, None, None, FAKE, None, dx, dw, None, None, sc, None)   # noqa: E731
    assert back(d, ok(), sc=None) == L.ERR_WORKSPACE and back(d, ok(), dx=None) == L.ERR_NULL and back(d, ok(), dw=FAKE + 4) == L.ERR_ALIGN
    assert lib.wkv7_conv_backward(d, ok(), FAKE, None, None, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, None) == L.ERR_UNSUPPORTED   # ds0 is dsT
    step = lambda desc, cv, st=FAKE: lib.wkv7_conv_step(desc, cv, FAKE, st, None, FAKE, None)   # noqa: E731
    assert step(d, ok()) == L.ERR_UNSUPPORTED                      # T must be 1
    assert step(_desc(L, T=1), ok(), None) == L.ERR_NULL


def _ssm_struct(L, **k):
    return L.Ssm(*[{**dict(G=1, A=FAKE, D=None, dt_bias=None, softplus=1, x_ld=0, dt_ld=0, b_ld=0, c_ld=0), **k}[n] for n, _ in L.Ssm._fields_])


def _ssm(L, desc, sp, **over):
    p = dict(x=FAKE, dt=FAKE, b=FAKE, c=FAKE, s0=None, reset=None, y=FAKE, s_out=None, ws=None)
    p.update(over)
    return L.lib().wkv7_ssm_forward(desc, sp, *(p[n] for n in ("x", "dt", "b", "c", "s0", "reset", "y", "s_out", "ws")), None)


def test_ssm_refusals(L):
    sp = lambda **k: _ssm_struct(L, **k)   # noqa: E731
    d = _desc(L)
    assert _ssm(L, None, sp()) == L.ERR_NULL and _ssm(L, d, None) == L.ERR_NULL
    for k in (dict(N=96), dict(algo="chunked_fused"), dict(algo="chunked_split"), dict(flags=4), dict(flags=8)):
        assert _ssm(L, _desc(L, **k), sp()) == L.ERR_UNSUPPORTED, k
    for t in ("float32", "float16"):
        assert _ssm(L, _desc(L, dtype=t, algo="chunked"), sp()) == L.ERR_UNSUPPORTED
    for g in (0, 3, -1):
        assert _ssm(L, d, sp(G=g)) == L.ERR_UNSUPPORTED
    assert _ssm(L, d, sp(A=None)) == L.ERR_NULL and _ssm(L, d, sp(D=FAKE + 2)) == L.ERR_ALIGN
    for k in (dict(x_ld=255), dict(dt_ld=3), dict(b_ld=63), dict(c_ld=-64)):
        assert _ssm(L, d, sp(**k)) == L.ERR_SHAPE, k
    assert _ssm(L, d, sp(x_ld=260)) == L.ERR_ALIGN and _ssm(L, d, sp(b_ld=68)) == L.ERR_ALIGN
    for n in ("x", "dt", "b", "c", "y"):
        assert _ssm(L, d, sp(), **{n: None}) == L.ERR_NULL
        assert _ssm(L, d, sp(), **{n: FAKE + (1 if n == "dt" else 8)}) == L.ERR_ALIGN
    assert _ssm(L, d, sp(), ws=FAKE + 4) == L.ERR_ALIGN and _ssm(L, d, sp(), s0=FAKE + 8) == L.ERR_ALIGN
    for k in (dict(B=-1), dict(T=-2), dict(B=1 << 20, H=1 << 20), dict(T=1 << 50)):
        assert _ssm(L, _desc(L, **k), sp()) == L.ERR_SHAPE, k
    assert _ssm(L, _desc(L, B=0), sp(), x=None, dt=None, b=None, c=None, y=None) == L.OK
    lib = L.lib()
    # a state before every 128th token and the last one
    assert lib.wkv7_ssm_workspace_bytes(_desc(L, T=129), sp(A=None)) == 2 * 4 * 3 * 64 * 64 * 4
    assert lib.wkv7_ssm_workspace_bytes(_desc(L, T=0), sp()) == 0 and lib.wkv7_ssm_workspace_bytes(_desc(L, N=32), sp()) == 0
    assert lib.wkv7_ssm_scratch_bytes(d, sp()) > 0
    back = lambda desc, ws=FAKE, sc=FAKE, dx=FAKE, ddt=FAKE, dA=None: lib.wkv7_ssm_backward(   # noqa: E731
        desc, sp(), FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, ws, dx, ddt, FAKE, FAKE, dA, None, None, None, sc, None)
    assert back(d, ws=None) == L.ERR_WORKSPACE and back(d, sc=None) == L.ERR_WORKSPACE and back(d, dx=None) == L.ERR_NULL
    assert back(d, ddt=FAKE + 2) == L.ERR_ALIGN and back(d, dA=FAKE + 4) == L.ERR_ALIGN
    assert _ssm(L, d, sp(), s0=FAKE, s_out=FAKE) == L.ERR_UNSUPPORTED
    assert lib.wkv7_ssm_backward(d, sp(), FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None, None, FAKE,
                                 FAKE, None) == L.ERR_UNSUPPORTED                     # ds0 is dsT
    step = lambda desc, st=FAKE: lib.wkv7_ssm_step(desc, sp(), FAKE, FAKE, FAKE, FAKE, st, None, FAKE, None)   # noqa: E731
    assert step(d) == L.ERR_UNSUPPORTED and step(_desc(L, T=1), None) == L.ERR_NULL


def test_rms_refusals(L):
    rn = lambda **k: L.Rms(*[{**dict(D=256, groups=1, weight=FAKE, eps=1e-5, gate=0, quant_block=0), **k}[n] for n, _ in L.Rms._fields_])   # noqa: E731
    d = _desc(L)
    lib = L.lib()
    f = lambda desc, r, x=FAKE, other=None, h=None, out=FAKE, scale=None: lib.wkv7_rms_forward(desc, r, x, other, h, out, scale, None)   # noqa: E731
    assert f(None, rn()) == L.ERR_NULL and f(d, None) == L.ERR_NULL
    for k in (dict(groups=0), dict(groups=3), dict(D=260, groups=1), dict(D=12), dict(D=16392), dict(eps=0.0), dict(eps=-1.0),
              dict(eps=math.nan), dict(eps=math.inf), dict(quant_block=64), dict(D=320, quant_block=128), dict(D=256, groups=4, quant_block=128)):
        assert f(d, rn(**k)) == L.ERR_UNSUPPORTED, k
    assert f(d, rn(D=-8)) == L.ERR_SHAPE
    assert f(d, rn(weight=None)) == L.ERR_NULL and f(d, rn(weight=FAKE + 8)) == L.ERR_ALIGN
    assert f(d, rn(), x=None) == L.ERR_NULL and f(d, rn(), out=FAKE + 4) == L.ERR_ALIGN
    assert f(d, rn(), other=FAKE) == L.ERR_NULL                       # the sum has nowhere to go
    assert f(d, rn(), h=FAKE) == L.ERR_UNSUPPORTED and f(d, rn(gate=1), other=FAKE, h=FAKE) == L.ERR_UNSUPPORTED
    assert f(d, rn(gate=1)) == L.ERR_NULL
    assert f(d, rn(quant_block=128)) == L.ERR_NULL and f(d, rn(quant_block=-1), scale=FAKE + 4) == L.ERR_ALIGN
    assert f(_desc(L, T=0), rn(), x=None, out=None) == L.OK
    b = lambda r, x=FAKE, other=None, dout=FAKE, dh=None, dx=FAKE, dother=None, dw=FAKE, sc=FAKE: lib.wkv7_rms_backward(   # noqa: E731
        d, r, x, other, dout, dh, dx, dother, dw, sc, None)
    assert b(rn(quant_block=128)) == L.ERR_UNSUPPORTED and b(rn(), other=FAKE) == L.ERR_UNSUPPORTED
    assert b(rn(gate=1), other=FAKE, dother=FAKE, dh=FAKE) == L.ERR_UNSUPPORTED and b(rn(gate=1), other=FAKE) == L.ERR_NULL
    assert b(rn(), sc=None) == L.ERR_WORKSPACE and b(rn(), dx=None) == L.ERR_NULL
    assert lib.wkv7_rms_scratch_bytes(d, rn(weight=None)) >= 256 * 4 and lib.wkv7_rms_scratch_bytes(d, rn(D=12)) == 0


def test_binding_refuses_host_tensors_and_strides(L):
    """A host tensor never reaches the library; `_rows` takes slices of wider token rows and nothing else."""
    import torch
    x = torch.zeros(2, 8, 16, dtype=torch.bfloat16)
    for call in (lambda: L.conv_forward(x, torch.zeros(16, 4)), lambda: L.rms_forward(x, torch.ones(16), 1e-5),
                 lambda: L.ssm_forward(x[..., None, :], x, x, x, x)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    wide = torch.zeros(2, 8, 40)
    rows = lambda t, lead=2: L._rows(t, "x", t.shape, lead, t)[1]   # noqa: E731
    assert rows(wide) == 0 and rows(wide[..., 8:24]) == 40 and rows(wide[:1, :, :16]) == 40 and rows(wide[:, :1, :16]) == 320
    assert rows(wide[:, 3, :16], 1) == 320 and rows(wide[..., :32].unflatten(-1, (4, 8))) == 40 and rows(wide[:1, :1, :8]) == 0
    assert rows(wide[:, ::2]) == 80                                        # every second token of both rows
    for bad in (wide[:, :, ::2], wide[:, :4], wide.transpose(0, 1), wide[:, :1, :16].expand(2, 8, 16),
                wide[..., :32].unflatten(-1, (4, 8)).transpose(2, 3)):
        with pytest.raises(ValueError, match="dense"):
            rows(bad)
    with pytest.raises(ValueError, match="must be"):
        L._dense(x, "s0", (2, 8, 16), torch.float32, x)
    with pytest.raises(ValueError, match="contiguous"):
        L._dense(wide[..., ::2], "s0", (2, 8, 20), torch.float32, wide)


def test_valid_calls_need_a_gpu(L):
    import torch
    if torch.cuda.is_available():
        pytest.skip("host has a GPU")
    assert _ssm(L, _desc(L), _ssm_struct(L)) == L.ERR_CUDA
    assert _conv(L, _desc(L), L.Conv(16, 4, 1, FAKE, None, 0)) == L.ERR_CUDA
    assert L.lib().wkv7_rms_forward(_desc(L), L.Rms(256, 1, FAKE, 1e-5, 0, 0), FAKE, None, None, FAKE, None, None) == L.ERR_CUDA


def test_binding_checks_every_gradient_it_is_given(L):
    """An entry of ``grads`` is written whether or not it was asked for, so a wrong one is refused either way.  (The functions
    under their device check, with host tensors: they refuse before they reach the library.)"""
    import torch
    z = torch.zeros
    x, w = z(2, 8, 16), z(16, 4)
    for bad, name in ((z(2, 3, 8), "ds0"), (z(16, 2), "dweight"), (z(16, dtype=torch.float64), "dbias"), (z(2, 8, 8), "dx")):
        with pytest.raises(ValueError, match=name):
            L.conv_backward.__wrapped__(x, w, x, grads={name: bad}, want_params=False, want_ds0=False)
    xs, bc, A, ws = z(1, 8, 2, 64), z(1, 8, 1, 64), z(2), z(1 << 18, dtype=torch.uint8)
    for bad, name in ((z(1, 2, 64, 32), "ds0"), (z(1), "dD"), (z(3), "ddt_bias"), (z(2, dtype=torch.float64), "dA"), (z(1, 8, 1, 32), "db")):
        with pytest.raises(ValueError, match=name):
            L.ssm_backward.__wrapped__(xs, z(1, 8, 2), A, bc, bc, xs, ws, grads={name: bad}, want_ds0=False)
    for bad, name in ((z(8), "dweight"), (z(2, 8, 8), "dgate")):
        with pytest.raises(ValueError, match=name):
            L.rms_backward.__wrapped__(x, z(16), x, 1e-5, grads={name: bad}, want_params=False)


def test_workspace_of_the_backward(L):
    """CHUNKED (AUTO for bf16, whatever the length) refuses a missing workspace; token order, which reads none, does not."""
    import torch
    sp = _ssm_struct(L)
    back = lambda **k: L.lib().wkv7_ssm_backward(_desc(L, **k), sp, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, None, FAKE, FAKE, FAKE, FAKE,   # noqa: E731
                                                 None, None, None, None, FAKE, None)
    for k in (dict(), dict(T=4), dict(algo="chunked")):
        assert back(**k) == L.ERR_WORKSPACE, k
    if not torch.cuda.is_available():      # (these pass the checks, and would be launched)
        for k in (dict(algo="scan"), dict(dtype="float32"), dict(dtype="float16")):
            assert back(**k) == L.ERR_CUDA, k
