"""Token tensors of more than 2^31 elements: the last tokens, behind a reset, equal a call on them alone."""
from __future__ import annotations

import pytest

from tests.test_gpu_state_space import FP32, W   # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free():
    import torch
    yield
    torch.cuda.empty_cache()


def _normal(*shape):
    import torch
    t = torch.empty(*shape, device="cuda", dtype=torch.bfloat16)
    return t.normal_()


def test_convolution(W):   # noqa: F811
    import torch
    T, D, tail = 940_007, 2304, 1000
    assert T * D > 1 << 31
    x, dy = _normal(1, T, D), _normal(1, T, D)
    w, bias = torch.randn(D, 4, device="cuda"), torch.randn(D, device="cuda")
    reset = torch.zeros(1, T, dtype=torch.uint8, device="cuda")
    reset[0, T - tail] = 1
    y, s = W.conv_forward(x, w, bias, None, reset)
    y2, s2 = W.conv_forward(x[:, T - tail:], w, bias)
    assert torch.equal(y[:, T - tail:], y2) and torch.equal(s, s2)
    del y
    g = W.conv_backward(x, w, dy, bias, None, reset)
    g2 = W.conv_backward(x[:, T - tail:], w, dy[:, T - tail:].contiguous(), bias)
    assert torch.equal(g["dx"][:, T - tail:], g2["dx"])


@pytest.mark.parametrize("groups,D", ((1, 2048), (8, 1024)))
def test_norm(W, groups, D):   # noqa: F811
    import torch
    rows, tail = (1 << 31) // D + 1003, 777
    x, z = _normal(rows, D), _normal(rows, D)
    w = torch.randn(D, device="cuda")
    f = W.rms_forward(x, w, 1e-5, residual=z, groups=groups, quant_block=128)
    f2 = W.rms_forward(x[-tail:], w, 1e-5, residual=z[-tail:], groups=groups, quant_block=128)
    for n in ("h", "scale"):
        assert torch.equal(f[n][-tail:], f2[n]), n
    assert torch.equal(f["q"][-tail:].view(torch.uint8), f2["q"].view(torch.uint8))
    del f
    g = W.rms_backward(x, w, z, 1e-5, groups=groups)
    g2 = W.rms_backward(x[-tail:], w, z[-tail:], 1e-5, groups=groups)
    assert torch.equal(g["dx"][-tail:], g2["dx"]) and g["dweight"].isfinite().all()


@pytest.mark.parametrize("algo", ("scan", "chunked"))
def test_scan(W, algo):   # noqa: F811
    """Chunks of the tail start where those of the whole row do, so the chunked form gives the same bits but for the order of the
    sums over heads (db and dc: an fp32 sum in another order, then each rounded: a step of 2^-7 of the value and 32 * 2^-24 of
    the largest).  Token order cuts the tail alone into runs that the whole row does not have there: the states are the same
    sums, rounded in another order (a chain of at most 301 tokens of three roundings each: 903 * 2^-24 of what they are made of,
    taken as the fp32 tolerance, 1e-4 of the RMS), and y is each time rounded from them."""
    import torch
    T, H, N = 128 * 8203 + 45, 32, 64
    tail = 128 * 2 + 45
    assert T * H * 64 > 1 << 31
    x, dy = _normal(1, T, H, 64), _normal(1, T, H, 64)
    b, c, dt = _normal(1, T, 1, N), _normal(1, T, 1, N), _normal(1, T, H)
    A, D, bias = -torch.linspace(0.05, 4.0, H, device="cuda"), torch.randn(H, device="cuda"), torch.randn(H, device="cuda") - 3
    reset = torch.zeros(1, T, dtype=torch.uint8, device="cuda")
    reset[0, T - tail] = 1
    end = lambda t: t[:, T - tail:].contiguous()   # noqa: E731
    y, s, ws = W.ssm_forward(x, dt, A, b, c, D, bias, None, reset, algo=algo)
    y2, s2, ws2 = W.ssm_forward(end(x), end(dt), A, end(b), end(c), D, bias, algo=algo)
    if algo == "chunked":
        assert bool((end(y) == y2).all()) and bool((s == s2).all())
    else:
        for a, r, step in ((end(y).float(), y2.float(), 2.0 ** -7), (s, s2, 0.0)):
            assert bool(((a - r).abs() <= step * r.abs() + FP32 * r.square().mean().sqrt()).all())
    del y
    if algo == "scan":   # its backward's fp64 parts per head would be 34 GB
        return
    g = W.ssm_backward(x, dt, A, b, c, dy, ws, D, bias, None, reset, algo=algo, want_ds0=False)
    g2 = W.ssm_backward(end(x), end(dt), A, end(b), end(c), end(dy), ws2, D, bias, algo=algo, want_ds0=False)
    assert bool((end(g["dx"]) == g2["dx"]).all()) and bool((end(g["ddt"]) == g2["ddt"]).all())
    for n in ("db", "dc"):
        a, r = end(g[n]).float(), g2[n].float()
        assert ((a - r).abs() <= 2.0 ** -7 * r.abs() + 32 * 2.0 ** -24 * r.abs().max()).all(), n
    assert all(t.isfinite().all() for t in g.values())
