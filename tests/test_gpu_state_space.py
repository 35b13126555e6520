"""GPU parity of the state-space layer (short convolution, selective scan, RMS norm) against the fp64 oracle: every
direction and dtype, lengths around the tile and chunk borders, resets in every position, carried states, slices of
wider tensors, other streams, captured graphs, and the whole layer run as it is used.

Tolerances, all relative to the reference's RMS and beyond the half step that storing in a 16-bit type costs:
* fp32 arithmetic (every kernel but the chunked scan): an output is a chain of at most a few hundred fp32
  operations on terms of at most some tens of RMS, each off by 2^-24: 512 * 2^-24 * 3 = 9e-5, taken as 1e-4;
* chunked scan, 16-bit outputs: at most two factors of each term of an output's sum are rounded to bf16 (2^-9 each at
  most), so an element is off by no more than 2^-8 of the sum of its terms' absolute values, which the oracle gives on
  the absolute values of the inputs; and as the roundings are independent (1.7e-3 of a value on average, three of them
  with the output's own), all elements together by 1.7e-3 * sqrt(3) = 3e-3 of the output's norm: 4e-3;
* chunked scan, fp32 outputs (states, parameter gradients): operands split in three bf16 parts: as fp32 arithmetic.
"""
from __future__ import annotations

import numpy as np
import pytest

from oracle import state_space as S
from tests.metrics import err_rms, err_rms_excess

pytestmark = pytest.mark.gpu

FP32, CHUNKED, CHUNKED_NORM = 1e-4, 2.0 ** -8, 4e-3
DT = ("f32", "bf16", "f16")


@pytest.fixture(scope="module")
def W():
    import torch
    from linear_recurrent_lm_b200 import wkv7
    torch.cuda.set_device(0)
    return wkv7


def _t(dtype):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]


def _dev(a, dtype=None):
    """A device tensor of ``a`` (rounded to ``dtype``) and the same values in fp64."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    if dtype is not None:
        t = t.to(_t(dtype))
    return t, t.double().cpu().numpy() if t.is_floating_point() else a


def _f64(t):
    return t.detach().double().cpu().numpy()


def _close(got, ref, dtype, tol, what=""):
    got = _f64(got)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    err = err_rms(got, ref) if dtype == "f32" else err_rms_excess(got, ref, dtype)
    assert err <= tol, (what, err)


def _close_chunked(got, ref, size, what=""):
    """bf16 outputs of the chunked scan: ``size`` holds the sums of the absolute terms of each element."""
    got = _f64(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    half = np.abs(ref) * 2.0 ** -8 + 1e-30                     # storing the result: half a step of bf16
    worst = np.max((np.abs(got - ref) - half) / (size + 1e-30))
    assert worst <= CHUNKED, (what, worst)
    norm = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-30)
    assert norm <= CHUNKED_NORM, (what, norm)


# ------------------------------------------------------------------ convolution
def _conv_case(rng, dtype, B, T, D, taps, reset="some", state=True, strided=False):
    import torch
    wide = rng.standard_normal((B, T, D + 24))
    x, x64 = _dev(wide, dtype)
    x, x64 = (x[..., 16:16 + D], x64[..., 16:16 + D]) if strided else (x[..., :D].contiguous(), x64[..., :D])
    k = {"weight": _dev(rng.standard_normal((D, taps)).astype(np.float32)), "bias": _dev(rng.standard_normal(D).astype(np.float32)),
         "s0": _dev(rng.standard_normal((B, taps - 1, D)), dtype) if state else (None, None)}
    r = np.zeros((B, T), np.uint8)
    if reset == "all":
        r[:] = 1
    elif reset == "some":
        r[rng.random((B, T)) < 0.15] = 1
        r[0, T - 1] = 1
    rd = None if reset is None else torch.from_numpy(r).cuda()
    return x, x64, k, rd, None if reset is None else r


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("taps", (2, 3, 4))
@pytest.mark.parametrize("T", (1, 2, 3, 5, 64, 131))
def test_conv_forward_backward(W, dtype, taps, T):
    rng = np.random.default_rng(100 + 10 * taps + T)
    for B, D, reset, state, strided, silu in ((2, 24, "some", True, True, True), (1, 8, None, False, False, False),
                                              (3, 136, "all", True, False, True), (2, 40, "some", False, True, False)):
        x, x64, k, rd, r = _conv_case(rng, dtype, B, T, D, taps, reset, state, strided)
        y, s = W.conv_forward(x, k["weight"][0], k["bias"][0], k["s0"][0], rd, silu=silu)
        yo, so = S.conv_forward(x64, k["weight"][1], k["bias"][1], k["s0"][1], r, silu)
        _close(y, yo, dtype, FP32, "y")
        assert np.array_equal(_f64(s), so)                       # copies of inputs, or zero
        dy, dy64 = _dev(rng.standard_normal((B, T, D)), dtype)
        ds, ds64 = _dev(rng.standard_normal((B, taps - 1, D)), dtype) if state else (None, None)
        g = W.conv_backward(x, k["weight"][0], dy, k["bias"][0], k["s0"][0], rd, ds, silu=silu)
        go = S.conv_backward(x64, k["weight"][1], dy64, k["bias"][1], k["s0"][1], r, ds64, silu)
        for n in ("dx", "ds0"):
            _close(g[n], go[n], dtype, FP32, n)
        for n in ("dweight", "dbias"):
            _close(g[n], go[n], "f32", FP32, n)


@pytest.mark.parametrize("dtype", DT)
def test_conv_steps_equal_the_forward(W, dtype):
    """Decode token by token from a carried state gives the forward's outputs bit for bit; idle rows keep theirs."""
    import torch
    rng = np.random.default_rng(120)
    for taps in (2, 3, 4):
        x, _, k, _, _ = _conv_case(rng, dtype, 5, 9, 72, taps, None, True, True)
        y, s = W.conv_forward(x, k["weight"][0], k["bias"][0], k["s0"][0])
        state = k["s0"][0].clone()
        for t in range(9):
            assert torch.equal(W.conv_step(x[:, t], k["weight"][0], state, k["bias"][0]), y[:, t])
        assert torch.equal(state, s)
        active = torch.tensor([1, 0, 1, 0, 0], dtype=torch.uint8, device="cuda")
        z = W.conv_step(x[:, 0], k["weight"][0], state, k["bias"][0], active)
        idle = active == 0
        assert torch.equal(state[idle], s[idle]) and not z[idle].any() and not torch.equal(state[~idle], s[~idle])


def test_conv_split_equals_one_call(W):
    import torch
    rng = np.random.default_rng(121)
    x, _, k, rd, _ = _conv_case(rng, "bf16", 2, 50, 64, 4, "some", True, False)
    y, s = W.conv_forward(x, k["weight"][0], k["bias"][0], k["s0"][0], rd)
    for cut in (1, 2, 17, 49):
        ya, sa = W.conv_forward(x[:, :cut].contiguous(), k["weight"][0], k["bias"][0], k["s0"][0], rd[:, :cut].contiguous())
        yb, sb = W.conv_forward(x[:, cut:].contiguous(), k["weight"][0], k["bias"][0], sa, rd[:, cut:].contiguous())
        assert torch.equal(torch.cat([ya, yb], 1), y) and torch.equal(sb, s)


# ------------------------------------------------------------------ selective scan
def _ssm_case(rng, dtype, B, T, H, G, N, reset="some", state=True, strided=True, params=True, dt_scale=1.0, A_scale=1.0):
    import torch
    width = H * 64 + 2 * G * N
    wide, wide64 = _dev(rng.standard_normal((B, T, width + 8)), dtype)
    dev, ref = {}, {}
    at = 0
    for n, shape in (("x", (H, 64)), ("b", (G, N)), ("c", (G, N))):
        size = shape[0] * shape[1]
        v = wide[..., at:at + size].unflatten(-1, shape)
        dev[n] = v if strided else v.contiguous()
        ref[n] = wide64[..., at:at + size].reshape(B, T, *shape)
        at += size
    dev["dt"], ref["dt"] = _dev(dt_scale * rng.standard_normal((B, T, H)), dtype)
    for n, v in (("A", -A_scale * rng.uniform(0.05, 4.0, H)), ("D", rng.standard_normal(H)), ("dt_bias", rng.uniform(-3.0, 0.5, H))):
        dev[n], ref[n] = _dev(v.astype(np.float32)) if n == "A" or params else (None, None)
    dev["s0"], ref["s0"] = _dev(rng.standard_normal((B, H, 64, N)).astype(np.float32)) if state else (None, None)
    r = None
    if reset is not None:
        r = np.zeros((B, T), np.uint8)
        if reset == "all":
            r[:] = 1
        else:
            r[rng.random((B, T)) < 0.03] = 1
            r[0, T // 2] = 1
            r[B - 1, 0] = 1
    dev["reset"], ref["reset"] = None if r is None else torch.from_numpy(r).cuda(), r
    return dev, ref


def _sizes(ref, softplus, dy=None, dsT=None):
    """Sums of the absolute terms of the outputs: the oracle on absolute values."""
    a = {n: v if n in ("dt", "A", "dt_bias", "reset") or v is None else np.abs(v) for n, v in ref.items()}
    if not softplus:
        step = ref["dt"] + (0.0 if ref["dt_bias"] is None else ref["dt_bias"])   # may be negative: keep its size in the terms
        scale = np.where(step < 0, -1.0, 1.0)
        a["x"] = a["x"] * scale[..., None]
    if dy is None:
        return S.ssm_forward(**a, softplus=softplus)[0]
    return S.ssm_backward(dy=np.abs(dy), dsT=None if dsT is None else np.abs(dsT), softplus=softplus, sizes=True, **a)


def _ssm_check(W, rng, dtype, algo, dev, ref, softplus=True):
    chunked = algo == "chunked"
    y, s, ws = W.ssm_forward(**dev, softplus=softplus, algo=algo)
    yo, so = S.ssm_forward(**ref, softplus=softplus)
    if chunked:
        _close_chunked(y, yo, np.abs(_sizes(ref, softplus)), "y")
    else:
        _close(y, yo, dtype, FP32, "y")
    _close(s, so, "f32", FP32, "s_out")
    dy, dy64 = _dev(rng.standard_normal(ref["x"].shape), dtype)
    ds, ds64 = _dev(rng.standard_normal(so.shape).astype(np.float32)) if ref["s0"] is not None else (None, None)
    g = W.ssm_backward(dy=dy, workspace=ws, dsT=ds, softplus=softplus, algo=algo, **dev)
    go = S.ssm_backward(dy=dy64, dsT=ds64, softplus=softplus, **ref)
    size = _sizes(ref, softplus, dy64, ds64) if chunked else None
    assert set(g) == {"dx", "ddt", "db", "dc", "dA", "ds0"} | ({"dD", "ddt_bias"} if dev["D"] is not None else set())
    for n in g:
        fp32 = n in ("dA", "dD", "ddt_bias", "ds0")
        if chunked and not fp32:
            _close_chunked(g[n], go[n], np.abs(size[n]), n)
        else:
            _close(g[n], go[n], "f32" if fp32 else dtype, FP32, n)


FORMS = [("f32", "scan"), ("bf16", "scan"), ("f16", "scan"), ("bf16", "chunked")]


@pytest.mark.parametrize("dtype,algo", FORMS)
@pytest.mark.parametrize("T", (1, 15, 16, 17, 127, 128, 129, 300))
def test_ssm_forward_backward(W, dtype, algo, T):
    rng = np.random.default_rng(200 + T)
    B, H, G, N = (2, 4, 2, 64) if T % 2 else (1, 3, 1, 128)
    dev, ref = _ssm_case(rng, dtype, B, T, H, G, N)
    _ssm_check(W, rng, dtype, algo, dev, ref)


@pytest.mark.parametrize("dtype,algo", FORMS)
@pytest.mark.parametrize("case", ("no_state", "every_token_reset", "no_parameters", "linear_dt", "long_memory", "no_memory", "one_head"))
def test_ssm_edges(W, dtype, algo, case):
    rng = np.random.default_rng(230)
    kw = dict(B=2, T=150, H=4, G=1, N=128, strided=False)
    kw.update({"no_state": dict(state=False, reset=None), "every_token_reset": dict(reset="all"), "no_parameters": dict(params=False),
               "linear_dt": dict(dt_scale=0.2), "long_memory": dict(A_scale=1e-3, reset=None), "no_memory": dict(dt_scale=20.0, A_scale=20.0),
               "one_head": dict(B=1, H=1, N=64)}[case])
    dev, ref = _ssm_case(rng, dtype, **kw)
    if case == "linear_dt":      # d = dt + bias of either sign: decays above one
        dev["dt_bias"], ref["dt_bias"] = _dev(np.full(4, 0.01, np.float32))
        dev["A"], ref["A"] = _dev(np.array([-0.1, 0.05, 0.0, -1.0], np.float32))
    _ssm_check(W, rng, dtype, algo, dev, ref, softplus=case != "linear_dt")


@pytest.mark.parametrize("shape", ((2, 1000, 40, 2, 64), (1, 2500, 6, 1, 128), (3, 700, 64, 1, 128)))
def test_ssm_chunked_equals_scan_on_larger_shapes(W, shape):
    """More heads than SMs, long rows of few heads: the two forms against each other, all outputs."""
    import torch
    B, T, H, G, N = shape
    rng = np.random.default_rng(240)
    dev, _ = _ssm_case(rng, "bf16", B, T, H, G, N)
    dy = torch.randn(B, T, H, 64, device="cuda").bfloat16()
    ds = torch.randn(B, H, 64, N, device="cuda")
    r = {}
    for algo in ("scan", "chunked"):
        y, s, ws = W.ssm_forward(**dev, algo=algo)
        r[algo] = {"y": y, "s_out": s, **W.ssm_backward(dy=dy, workspace=ws, dsT=ds, algo=algo, **dev)}
        y2, s2, _ = W.ssm_forward(**dev, algo=algo, need_workspace=False)
        _near(y2, y, "y without a workspace")
        _close(s2, _f64(s), "f32", FP32, "s_out without a workspace")
    for n, t in r["chunked"].items():
        if t.dtype == torch.float32:
            _close(t, _f64(r["scan"][n]), "f32", FP32, n)
        else:
            _near(t, r["scan"][n], n)


def _near(got, want, what=""):
    """bf16 results of two forms of the scan, each stored once more than _close_chunked counts."""
    norm = ((got.double() - want.double()).norm() / want.double().norm()).item()
    assert norm <= CHUNKED_NORM, (what, norm)


@pytest.mark.parametrize("dtype,algo", FORMS)
def test_ssm_split_equals_one_call(W, dtype, algo):
    """Two chained calls, forward and backward, against the single one, cut inside and at the border of a chunk."""
    import torch
    rng = np.random.default_rng(250)
    dev, ref = _ssm_case(rng, dtype, 2, 290, 4, 2, 64, strided=False)
    dy, _ = _dev(rng.standard_normal((2, 290, 4, 64)), dtype)
    ds, _ = _dev(rng.standard_normal((2, 4, 64, 64)).astype(np.float32))
    y, s, ws = W.ssm_forward(**dev, algo=algo)
    g = W.ssm_backward(dy=dy, workspace=ws, dsT=ds, algo=algo, **dev)
    def same(a, b, n):   # both are stored: each is off by up to half a step, so they may differ by a whole one
        if algo == "chunked":
            return _near(a, b, n)
        if dtype == "f32":
            return _close(a, _f64(b), dtype, FP32, n)
        b = _f64(b)
        step = 2.0 * np.maximum(np.abs(b), np.abs(_f64(a))) * 2.0 ** (-8 if dtype == "bf16" else -11)
        worst = np.max(np.maximum(np.abs(_f64(a) - b) - step, 0.0)) / np.sqrt(np.mean(b * b))
        assert worst <= FP32, (n, worst)
    for cut in (128, 77):
        part = lambda a, z: {n: (v[:, a:z].contiguous() if n in ("x", "dt", "b", "c", "reset") else v) for n, v in dev.items()}   # noqa: E731
        first, second = part(0, cut), part(cut, 290)
        ya, sa, wa = W.ssm_forward(**first, algo=algo)
        second["s0"] = sa
        yb, sb, wb = W.ssm_forward(**second, algo=algo)
        same(torch.cat([ya, yb], 1), y, "y")
        _close(sb, _f64(s), "f32", FP32, "s")
        gb = W.ssm_backward(dy=dy[:, cut:].contiguous(), workspace=wb, dsT=ds, algo=algo, **second)
        ga = W.ssm_backward(dy=dy[:, :cut].contiguous(), workspace=wa, dsT=gb["ds0"], algo=algo, **first)
        for n in ("dx", "ddt", "db", "dc"):
            same(torch.cat([ga[n], gb[n]], 1), g[n], n)
        _close(ga["ds0"], _f64(g["ds0"]), "f32", FP32, "ds0")
        for n in ("dA", "dD", "ddt_bias"):
            _close(ga[n] + gb[n], _f64(g[n]), "f32", FP32, n)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("N,G", ((64, 1), (128, 2)))
def test_ssm_steps_follow_the_forward(W, dtype, N, G):
    import torch
    rng = np.random.default_rng(260)
    B, T, H = 5, 6, 4
    dev, ref = _ssm_case(rng, dtype, B, T, H, G, N, reset=None)
    yo, so = S.ssm_forward(**ref)
    state = dev["s0"].clone()
    args = [dev[n] for n in ("A", "D", "dt_bias")]
    for t in range(T):
        y = W.ssm_step(dev["x"][:, t], dev["dt"][:, t], args[0], dev["b"][:, t], dev["c"][:, t], state, args[1], args[2])
        _close(y, yo[:, t], dtype, FP32, t)
    _close(state, so, "f32", FP32, "state")
    keep = state.clone()
    active = torch.tensor([0, 1, 1, 0, 1], dtype=torch.bool, device="cuda")
    y = W.ssm_step(dev["x"][:, 0], dev["dt"][:, 0], args[0], dev["b"][:, 0], dev["c"][:, 0], state, args[1], args[2], active)
    assert torch.equal(state[~active], keep[~active]) and not y[~active].any()
    assert not torch.equal(state[active], keep[active])


def test_ssm_backward_takes_either_workspace(W):
    """The states that one form's forward leaves serve the other form's backward."""
    import torch
    rng = np.random.default_rng(252)
    dev, _ = _ssm_case(rng, "bf16", 2, 300, 4, 1, 64)
    dy = torch.randn(2, 300, 4, 64, device="cuda").bfloat16()
    ws = {a: W.ssm_forward(**dev, algo=a)[2] for a in ("scan", "chunked")}
    assert ws["scan"].numel() != ws["chunked"].numel()        # room for runs of tokens, or for none
    want = W.ssm_backward(dy=dy, workspace=ws["scan"], algo="scan", **dev)
    for back, forward in (("scan", "chunked"), ("chunked", "scan")):
        g = W.ssm_backward(dy=dy, workspace=ws[forward], algo=back, **dev)
        for n, t in g.items():
            if t.dtype == torch.float32:
                _close(t, _f64(want[n]), "f32", FP32, n)
            else:
                _near(t, want[n], n)
    with pytest.raises(ValueError, match="workspace"):
        W.ssm_backward(dy=dy, workspace=ws["scan"][:64], algo="scan", **dev)


@pytest.mark.parametrize("dtype,algo", FORMS)
def test_ssm_masked_steps(W, dtype, algo):
    """dt = -inf, or the type's lowest value, is a step of zero: the token adds nothing, the state passes, ddt is zero."""
    import torch
    rng = np.random.default_rng(253)
    dev, ref = _ssm_case(rng, dtype, 2, 150, 4, 2, 64)
    dev["dt"][:, 100:] = -float("inf")
    dev["dt"][1, 40:60] = torch.finfo(_t(dtype)).min
    ref["dt"] = _f64(dev["dt"])
    with np.errstate(over="ignore"):
        _ssm_check(W, rng, dtype, algo, dev, ref)
    dy = torch.ones(2, 150, 4, 64, device="cuda", dtype=_t(dtype))
    _, _, ws = W.ssm_forward(**dev, algo=algo)
    g = W.ssm_backward(dy=dy, workspace=ws, algo=algo, **dev)
    for n in ("ddt", "db"):
        assert not g[n][:, 100:].any() and not g[n][1, 40:60].any(), n


@pytest.mark.parametrize("dtype,algo", FORMS)
def test_ssm_decays_beyond_the_exponents_range(W, dtype, algo):
    """d A overflows fp32: nothing is remembered, and nothing is NaN."""
    rng = np.random.default_rng(255)
    dev, ref = _ssm_case(rng, dtype, 2, 140, 4, 1, 64)
    dev["dt_bias"], ref["dt_bias"] = _dev(np.full(4, 100.0, np.float32))
    dev["A"], ref["A"] = _dev(np.array([-3e38, -1e37, -1e30, -3e38], np.float32))
    _ssm_check(W, rng, dtype, algo, dev, ref)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", (90, 700))
def test_ssm_scan_keeps_what_is_not_finite_in_its_segment(W, dtype, T):
    """In token order a NaN or infinity before a reset changes nothing after it, and no gradient crosses back."""
    import torch
    rng = np.random.default_rng(254)
    dev, _ = _ssm_case(rng, dtype, 2, T, 4, 2, 64, reset=None, strided=False)
    cut = T // 2 + 3
    dev["reset"] = torch.zeros(2, T, dtype=torch.uint8, device="cuda")
    dev["reset"][:, cut] = 1
    dy = torch.randn(2, T, 4, 64, device="cuda").to(_t(dtype))
    ds = torch.randn(2, 4, 64, 64, device="cuda")
    y, s, ws = W.ssm_forward(**dev, algo="scan")
    g = W.ssm_backward(dy=dy, workspace=ws, dsT=ds, algo="scan", **dev)
    bad = {n: v.clone() if v is not None else None for n, v in dev.items()}
    bad["x"][0, cut - 2, 1, 3] = float("nan")
    bad["b"][0, 5, 0, 7] = float("inf")
    bad["c"][1, 9, 1, 0] = float("nan")
    bad["s0"][1, 2, 0, 0] = float("inf")
    y2, s2, ws = W.ssm_forward(**bad, algo="scan")
    g2 = W.ssm_backward(dy=dy, workspace=ws, dsT=ds, algo="scan", **bad)
    assert torch.equal(y2[:, cut:], y[:, cut:]) and torch.equal(s2, s) and not y2[:, :cut].isfinite().all()
    for n in ("dx", "ddt", "db", "dc"):
        assert torch.equal(g2[n][:, cut:], g[n][:, cut:]), n
    late = dy.clone()
    late[0, cut + 1] = float("nan")
    _, _, ws = W.ssm_forward(**dev, algo="scan")
    g2 = W.ssm_backward(dy=late, workspace=ws, dsT=ds, algo="scan", **dev)
    for n in ("dx", "ddt", "db", "dc"):
        assert torch.equal(g2[n][:, :cut], g[n][:, :cut]), n
    assert torch.equal(g2["ds0"], g["ds0"])


@pytest.mark.parametrize("dtype", DT)
def test_conv_keeps_what_is_not_finite_in_its_window(W, dtype):
    import torch
    rng = np.random.default_rng(122)
    x, _, k, _, _ = _conv_case(rng, dtype, 2, 40, 24, 4, None, True, False)
    w, bias, s0 = (k[n][0] for n in ("weight", "bias", "s0"))
    r = torch.zeros(2, 40, dtype=torch.uint8, device="cuda")
    r[:, 21] = 1
    dy = torch.randn(2, 40, 24, device="cuda").to(_t(dtype))
    y, _ = W.conv_forward(x, w, bias, s0, r)
    g = W.conv_backward(x, w, dy, bias, s0, r)
    bad = x.clone()
    bad[0, 20, 5], bad[1, 10, 7] = float("nan"), float("inf")
    y2, _ = W.conv_forward(bad, w, bias, s0, r)
    g2 = W.conv_backward(bad, w, dy, bias, s0, r)
    touched = torch.zeros(2, 40, 24, dtype=torch.bool, device="cuda")      # outputs whose taps see the value
    touched[0, 20, 5] = touched[1, 10:14, 7] = True
    assert torch.equal(y2[~touched], y[~touched]) and not y2[0, 20, 5].isfinite()
    back = torch.zeros_like(touched)                                        # inputs of those outputs
    back[0, 17:21, 5] = back[1, 7:14, 7] = True
    assert torch.equal(g2["dx"][~back], g["dx"][~back])


@pytest.mark.parametrize("algo", ("scan", "chunked"))
def test_ssm_repeats_bit_for_bit(W, algo):
    import torch
    rng = np.random.default_rng(270)
    dev, _ = _ssm_case(rng, "bf16", 2, 400, 8, 2, 128)
    dy = torch.randn(2, 400, 8, 64, device="cuda").bfloat16()
    runs = []
    for _ in range(3):
        y, s, ws = W.ssm_forward(**dev, algo=algo)
        runs.append({"y": y, "s": s, **W.ssm_backward(dy=dy, workspace=ws, algo=algo, **dev)})
    for r in runs[1:]:
        assert all(torch.equal(r[n], runs[0][n]) for n in r)


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("kind", ("plain", "residual", "gate"))
@pytest.mark.parametrize("rows,D,groups", ((1, 8, 1), (5, 64, 8), (300, 520, 1), (3, 2048, 1), (7, 4096, 2), (2, 16384, 1), (257, 192, 3),
                                             (9, 2560, 1), (5, 15360, 3), (3, 12288, 1), (700, 1288, 1)))
def test_rms_forward_backward(W, dtype, kind, rows, D, groups):
    rng = np.random.default_rng(300 + D)
    eps = 1e-5
    x, x64 = _dev(rng.standard_normal((rows, D)), dtype)
    z, z64 = (None, None) if kind == "plain" else _dev(rng.standard_normal((rows, D)), dtype)
    w, w64 = _dev((1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32))
    f = W.rms_forward(x, w, eps, groups=groups, **({} if z is None else {kind: z}))
    h, h64 = x, x64
    if kind == "residual":
        h = f["h"]
        h64 = _f64(h)
        # one rounding of the sum, relative to each value (not to the RMS, which values here exceed five times over)
        import torch
        assert torch.equal(h, (x.float() + z.float()).to(h.dtype))
    gate64 = z64 if kind == "gate" else None
    _close(f["out"], S.rms_forward(h64, w64, eps, gate64, groups), dtype, FP32, "out")
    dout, dout64 = _dev(rng.standard_normal((rows, D)), dtype)
    dh, dh64 = _dev(rng.standard_normal((rows, D)), dtype) if kind == "residual" else (None, None)
    g = W.rms_backward(h, w, dout, eps, groups=groups, gate=z if kind == "gate" else None, dh=dh)
    go = S.rms_backward(h64, w64, dout64, eps, gate64, dh64, groups)
    for n in ("dx",) + (("dgate",) if kind == "gate" else ()):
        _close(g[n], go[n], dtype, FP32, n)
    _close(g["dweight"], go["dweight"], "f32", FP32, "dweight")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("block,D,groups", ((128, 128, 1), (128, 2048, 1), (128, 768, 2), (128, 16384, 1), (-1, 8, 1), (-1, 520, 1), (-1, 512, 8),
                                            (128, 2560, 1), (-1, 2568, 1), (128, 10240, 2)))
def test_rms_e4m3(W, dtype, block, D, groups):
    """Codes times scale against the norm: half a step of e4m3 (2^-4 of the value, and 2^-10 of the scale below its
    normal range), the scale exactly the largest value over 448."""
    import torch
    rng = np.random.default_rng(320 + D)
    x, _ = _dev(rng.standard_normal((37, D)) * np.exp(rng.standard_normal((37, 1))), dtype)
    x[3] = 0
    x[5, : D // groups] = 0
    r, _ = _dev(rng.standard_normal((37, D)), dtype)
    r[3] = 0
    r[5, : D // groups] = 0
    w, w64 = _dev((1.0 + 0.2 * rng.standard_normal(D)).astype(np.float32))
    f = W.rms_forward(x, w, 1e-5, residual=r, groups=groups, quant_block=block)
    assert f["q"].dtype == torch.float8_e4m3fn
    ref = S.rms_forward(_f64(f["h"]), w64, 1e-5, None, groups)
    per = 128 if block > 0 else D // groups
    ref = ref.reshape(37, -1, per)
    scale = _f64(f["scale"]).reshape(37, -1, 1)
    top = np.abs(ref).max(2, keepdims=True)
    assert np.all(np.abs(scale - np.where(top > 0, top / 448.0, 1.0)) <= 1e-5 * scale)
    got = f["q"].float().double().cpu().numpy().reshape(ref.shape) * scale
    assert np.all(np.abs(got - ref) <= np.maximum(np.abs(ref) * 2.0 ** -4, scale * 2.0 ** -10) * (1.0 + 1e-4))
    zero = top[..., 0] == 0
    assert zero.any() and not got[zero].any()


def test_rms_e4m3_shows_what_is_not_finite(W):
    """A NaN or infinity in a slice gives NaN codes in its blocks and leaves the others alone."""
    import torch
    x = torch.randn(4, 256, device="cuda").bfloat16()
    w = torch.ones(256, device="cuda")
    good = W.rms_forward(x, w, 1e-5, quant_block=128)
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    f = W.rms_forward(x, w, 1e-5, quant_block=128)
    assert f["q"][1].float().isnan().all() and f["scale"][1].isnan().all()
    assert f["q"][2, 200].float().isnan()
    for i in (0, 3):
        assert torch.equal(f["q"][i].view(torch.uint8), good["q"][i].view(torch.uint8)) and torch.equal(f["scale"][i], good["scale"][i])


def test_rms_in_place_sum(W):
    import torch
    x, r = (torch.randn(33, 1024, device="cuda").bfloat16() for _ in range(2))
    w = torch.randn(1024, device="cuda")
    a = W.rms_forward(x, w, 1e-5, residual=r)
    keep = r.clone()
    b = W.rms_forward(x, w, 1e-5, residual=r, h=r)
    assert b["h"].data_ptr() == r.data_ptr() and torch.equal(r, a["h"]) and torch.equal(b["out"], a["out"])
    assert not torch.equal(r, keep)


# ------------------------------------------------------------------ around the kernels
def test_empty_calls(W):
    import torch
    z = lambda *s, d=torch.bfloat16: torch.zeros(*s, device="cuda", dtype=d)   # noqa: E731
    f = torch.float32
    s0 = torch.randn(2, 3, 64, 64, device="cuda")
    A = -torch.ones(3, device="cuda")
    args = (z(2, 0, 3, 64), z(2, 0, 3), A, z(2, 0, 1, 64), z(2, 0, 1, 64))
    y, s, ws = W.ssm_forward(*args, s0=s0)
    assert y.shape == (2, 0, 3, 64) and torch.equal(s, s0)
    g = W.ssm_backward(*args, z(2, 0, 3, 64), ws, D=A, dt_bias=A, dsT=s0)
    assert torch.equal(g["ds0"], s0) and not g["dA"].any() and not g["dD"].any() and not g["ddt_bias"].any()
    w = z(16, 4, d=f)
    c0 = torch.randn(2, 3, 16, device="cuda").bfloat16()
    y, s = W.conv_forward(z(2, 0, 16), w, s0=c0)
    assert torch.equal(s, c0)
    g = W.conv_backward(z(2, 0, 16), w, z(2, 0, 16), s0=c0, dsT=c0)
    assert torch.equal(g["ds0"], c0) and not g["dweight"].any() and not g["dbias"].any()
    assert not W.conv_forward(z(2, 0, 16), w)[1].any()
    assert W.rms_forward(z(0, 64), z(64, d=f), 1e-5)["out"].shape == (0, 64)
    assert not W.rms_backward(z(0, 64), z(64, d=f), z(0, 64), 1e-5)["dweight"].any()
    assert W.conv_step(z(0, 16), w, z(0, 3, 16)).shape == (0, 16)
    assert W.ssm_step(z(0, 3, 64), z(0, 3), A, z(0, 1, 64), z(0, 1, 64), z(0, 3, 64, 64, d=f)).shape == (0, 3, 64)


def _layer(W, p, x, res, reset=None, conv0=None, ssm0=None, algo="auto"):
    """Norm (with the residual) -> projection -> convolution -> scan -> gated norm -> projection."""
    import torch
    H, G, N = 4, 1, 64
    n = W.rms_forward(x, p["w_in"], 1e-5, residual=res)
    z, xbc, dt = torch.split(n["out"] @ p["proj"], [H * 64, H * 64 + 2 * G * N, 8], -1)
    z, dt = z.contiguous(), dt[..., :H]
    u, conv1 = W.conv_forward(xbc, p["filter"], p["conv_bias"], conv0, reset)
    xs, b, c = u[..., :256].unflatten(-1, (H, 64)), u[..., 256:320].unflatten(-1, (G, N)), u[..., 320:].unflatten(-1, (G, N))
    y, ssm1, ws = W.ssm_forward(xs, dt, p["A"], b, c, p["D"], p["dt_bias"], ssm0, reset, algo=algo)
    o = W.rms_forward(y.flatten(2), p["w_out"], 1e-5, gate=z)
    saved = dict(n=n, z=z, xbc=xbc, dt=dt, xs=xs, b=b, c=c, y=y, ws=ws, o=o["out"])
    return o["out"] @ p["back"], n["h"], conv1, ssm1, saved


def _layer_params():
    import torch
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")   # noqa: E731
    return dict(w_in=1 + 0.1 * r(128), proj=(r(128, 648) / 11.3).bfloat16(), filter=r(384, 4) / 2, conv_bias=0.1 * r(384),
                A=-torch.linspace(0.2, 4.0, 4, device="cuda"), D=r(4), dt_bias=r(4) - 2, w_out=1 + 0.1 * r(256),
                back=(r(256, 128) / 16).bfloat16())


@pytest.mark.parametrize("algo", ("scan", "auto"))
def test_layer_prompt_then_tokens(W, algo):
    """A prompt through the layer, then single tokens from its states, against the whole row in one call."""
    import torch
    p = _layer_params()
    g = torch.Generator(device="cuda").manual_seed(6)
    x, res = (torch.randn(3, 140, 128, generator=g, device="cuda").bfloat16() for _ in range(2))
    whole, *_ = _layer(W, p, x, res, algo=algo)
    out, _, conv, ssm, _ = _layer(W, p, x[:, :133].contiguous(), res[:, :133].contiguous(), algo=algo)
    assert err_rms(_f64(out), _f64(whole[:, :133])) <= 0.1    # the same kernels; bf16 between them, chunk borders apart
    for t in range(133, 140):
        n = W.rms_forward(x[:, t].contiguous(), p["w_in"], 1e-5, residual=res[:, t].contiguous())
        z, xbc, dt = torch.split(n["out"] @ p["proj"], [256, 384, 8], -1)
        u = W.conv_step(xbc, p["filter"], conv, p["conv_bias"])
        y = W.ssm_step(u[:, :256].unflatten(-1, (4, 64)), dt[:, :4], p["A"], u[:, 256:320].unflatten(-1, (1, 64)),
                       u[:, 320:].unflatten(-1, (1, 64)), ssm, p["D"], p["dt_bias"])
        o = W.rms_forward(y.flatten(1), p["w_out"], 1e-5, gate=z.contiguous())["out"] @ p["back"]
        # a few bf16 roundings (2^-9 each, up to 5 RMS) between the two ways to the same token
        assert err_rms(_f64(o), _f64(whole[:, t])) <= 0.1, t


@pytest.mark.parametrize("algo", ("scan", "auto"))
def test_layer_gradients(W, algo):
    """The kernels' backward passes chained through the layer against reverse mode over the same formulas in fp64 torch."""
    import torch
    p = _layer_params()
    g = torch.Generator(device="cuda").manual_seed(7)
    B, T, H, G, N = 2, 70, 4, 1, 64
    x, res, dout = (torch.randn(B, T, 128, generator=g, device="cuda").bfloat16() for _ in range(3))
    reset = torch.zeros(B, T, dtype=torch.uint8, device="cuda")
    reset[0, 31] = 1
    out, h, _, _, s = _layer(W, p, x, res, reset, algo=algo)
    do = (dout.float() @ p["back"].float().T).bfloat16()
    g2 = W.rms_backward(s["y"].flatten(2), p["w_out"], do, 1e-5, gate=s["z"])
    gs = W.ssm_backward(s["xs"], s["dt"], p["A"], s["b"], s["c"], g2["dx"].unflatten(-1, (H, 64)), s["ws"], p["D"], p["dt_bias"],
                        None, reset, algo=algo)
    du = torch.cat([gs["dx"].flatten(2), gs["db"].flatten(2), gs["dc"].flatten(2)], -1)
    gc = W.conv_backward(s["xbc"], p["filter"], du, p["conv_bias"], None, reset)
    dn = torch.cat([g2["dgate"], gc["dx"], gs["ddt"], torch.zeros(B, T, 4, device="cuda", dtype=torch.bfloat16)], -1)
    g1 = W.rms_backward(h, p["w_in"], (dn.float() @ p["proj"].float().T).bfloat16(), 1e-5)
    # the formulas in fp64
    q = {n: v.double().requires_grad_(True) for n, v in p.items()}
    X = (x.float() + res.float()).bfloat16().double().requires_grad_(True)
    norm = lambda v, w: v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-5) * w   # noqa: E731
    z, xbc, dt = torch.split(norm(X, q["w_in"]) @ q["proj"], [256, 384, 8], -1)
    cuts = reset.long().cumsum(1)
    taps = []
    for j in range(4):
        same = torch.zeros(B, T, device="cuda", dtype=torch.float64)
        same[:, j:] = (cuts[:, j:] == cuts[:, :T - j]).double()
        taps.append(torch.nn.functional.pad(xbc, (0, 0, j, 0))[:, :T] * same[..., None] * q["filter"][:, 3 - j])
    u = torch.nn.functional.silu(sum(taps) + q["conv_bias"])
    xs, b, c = u[..., :256].unflatten(-1, (H, 64)), u[..., 256:320], u[..., 320:]
    d = torch.nn.functional.softplus(dt[..., :H] + q["dt_bias"])
    lam = (d * q["A"]).cumsum(1)
    keep = (cuts[:, :, None] == cuts[:, None]) & torch.ones(T, T, dtype=torch.bool, device="cuda").tril()
    m = torch.exp((lam[:, :, None] - lam[:, None]).masked_fill(~keep[..., None], -torch.inf)) * (c @ b.mT)[..., None]
    y = torch.einsum("btsh,bsh,bshp->bthp", m, d, xs) + q["D"][:, None] * xs
    o = norm(y.flatten(2) * torch.nn.functional.silu(z), q["w_out"]) @ q["back"]
    (o * dout.double()).sum().backward()
    # chained bf16 tensors between the kernels: cosine, as the framework holds its composed layers
    pairs = [("dx", g1["dx"], X.grad), ("w_in", g1["dweight"], q["w_in"].grad), ("filter", gc["dweight"], q["filter"].grad),
             ("conv_bias", gc["dbias"], q["conv_bias"].grad), ("A", gs["dA"], q["A"].grad), ("D", gs["dD"], q["D"].grad),
             ("dt_bias", gs["ddt_bias"], q["dt_bias"].grad), ("w_out", g2["dweight"], q["w_out"].grad)]
    for n, got, ref in pairs:
        cos = torch.nn.functional.cosine_similarity(got.double().flatten(), ref.flatten(), 0).item()
        assert cos >= 0.999, (n, cos)


def test_other_stream_and_graph(W):
    """The layer on a stream of its own, and captured once and replayed on new inputs, gives the same bits as eager."""
    import torch
    p = _layer_params()
    x, res = (torch.randn(2, 200, 128, device="cuda").bfloat16() for _ in range(2))
    want = [t.clone() for t in _layer(W, p, x, res)[:4]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = _layer(W, p, x, res)[:4]
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = W.rms_forward(x, p["w_in"], 1e-5, residual=res, stream=side)
    side.synchronize()
    assert torch.equal(y["h"], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _layer(W, p, x, res)[:4]
    x2 = torch.randn_like(x)
    want2 = [t.clone() for t in _layer(W, p, x2, res)[:4]]
    for src, ref in ((x2, want2), (x.clone(), want)):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_two_graphs_share_no_scratch(W):
    """A forward-and-backward captured twice on different inputs: both replayed, in either order, on two streams."""
    import torch
    rng = np.random.default_rng(280)
    cases = []
    for i in range(2):
        dev, _ = _ssm_case(rng, "bf16", 1, 260, 4, 1, 64)
        dy = torch.randn(1, 260, 4, 64, device="cuda").bfloat16()

        def run(dev=dev, dy=dy):
            y, s, ws = W.ssm_forward(**dev)
            return {"y": y, "s": s, **W.ssm_backward(dy=dy, workspace=ws, **dev)}
        ref = {n: t.clone() for n, t in run().items()}
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        cases.append((graph, out, ref, run))   # a graph reads its inputs where they were: they stay alive
    streams = [torch.cuda.Stream() for _ in range(2)]
    for order in ((0, 1), (1, 0)):
        for i in order:
            with torch.cuda.stream(streams[i]):
                cases[i][0].replay()
        torch.cuda.synchronize()
        for _, out, ref, _ in cases:
            assert all(torch.equal(out[n], ref[n]) for n in ref)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T", (40, 400))
def test_token_order_in_a_graph(W, dtype, T):
    """The token-order backward's scans run beside one another: captured and replayed back to back with another call
    behind them on the stream, they give the eager bits every time."""
    import torch
    rng = np.random.default_rng(285)
    dev, _ = _ssm_case(rng, dtype, 2, T, 6, 2, 128, strided=False)
    dy = torch.randn(2, T, 6, 64, device="cuda").to(_t(dtype))

    def run():
        y, s, ws = W.ssm_forward(**dev, algo="scan")
        g = W.ssm_backward(dy=dy, workspace=ws, algo="scan", **dev)
        y2, _, _ = W.ssm_forward(g["dx"], dev["dt"], dev["A"], g["db"], g["dc"], algo="scan")   # reads what came before
        return {"y": y, "s": s, "y2": y2, **g}
    ref = {n: t.clone() for n, t in run().items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(3):
        for _ in range(10):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], ref[n]) for n in ref)
        again = run()
        assert all(torch.equal(again[n], ref[n]) for n in ref)


def test_finite_check_reports(W):
    import torch
    x = torch.randn(4, 256, device="cuda").bfloat16()
    w = torch.ones(256, device="cuda")
    W.device_status()
    W.rms_forward(x, w, 1e-5, flags=W.FLAG_CHECK_FINITE)
    assert W.device_status() == W.OK
    x[1, 1] = float("nan")
    W.rms_forward(x, w, 1e-5, flags=W.FLAG_CHECK_FINITE)
    assert W.device_status() == W.ERR_NONFINITE
    W.rms_forward(x, w, 1e-5, quant_block=128, flags=W.FLAG_CHECK_FINITE)
    assert W.device_status() == W.ERR_NONFINITE
    xs = torch.randn(1, 5, 16, device="cuda").bfloat16()
    xs[0, 2, 3] = float("inf")
    W.conv_forward(xs, torch.ones(16, 4, device="cuda"), flags=W.FLAG_CHECK_FINITE)
    assert W.device_status() == W.ERR_NONFINITE
    assert W.device_status() == W.OK


def test_debug_build_agrees(W):
    """The bounds-checked build gives the same bits and reports no failed check."""
    import torch
    rng = np.random.default_rng(290)
    dev, _ = _ssm_case(rng, "bf16", 2, 150, 4, 2, 64)
    dy = torch.randn(2, 150, 4, 64, device="cuda").bfloat16()
    p = _layer_params()
    x, res = (torch.randn(2, 37, 128, device="cuda").bfloat16() for _ in range(2))

    def run():
        y, s, ws = W.ssm_forward(**dev)
        out = {"y": y, "s": s, **W.ssm_backward(dy=dy, workspace=ws, **dev)}
        o, h, c1, s1, saved = _layer(W, p, x, res, algo="scan")
        out.update(o=o, h=h, c1=c1, s1=s1)
        xbc = saved["xbc"]
        out.update({"c" + n: t for n, t in W.conv_backward(xbc, p["filter"], torch.ones_like(xbc), p["conv_bias"]).items()})
        out.update({"n" + n: t for n, t in W.rms_backward(h, p["w_in"], x, 1e-5).items()})
        return out
    want = run()
    prev = W.use_build("debug")
    try:
        W.device_status()
        got = run()
        assert W.device_status() == W.OK
    finally:
        W.use_build(prev)
    for n in want:
        assert torch.equal(got[n], want[n]), n
