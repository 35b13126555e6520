"""Pins of the state-space layer's oracle: closed forms, splits, and fp64 central differences on every input."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import state_space as S


def _ssm_case(rng, B=2, T=9, H=4, G=2, P=3, N=5, reset=True):
    r = np.zeros((B, T), np.uint8)
    if reset:
        r[0, 4] = 1
        r[1, 0] = 1
    return dict(x=rng.standard_normal((B, T, H, P)), dt=rng.standard_normal((B, T, H)), A=-rng.uniform(0.2, 2.0, H),
                b=rng.standard_normal((B, T, G, N)), c=rng.standard_normal((B, T, G, N)), D=rng.standard_normal(H),
                dt_bias=rng.standard_normal(H), s0=rng.standard_normal((B, H, P, N)), reset=r)


def _differences(f, inputs, names, grads, rng, count=6, h=1e-5):
    """Central differences of f at ``count`` places of every named input against its gradient."""
    for n in names:
        flat = inputs[n].reshape(-1)
        for i in rng.choice(flat.size, min(count, flat.size), replace=False):
            keep = flat[i]
            flat[i] = keep + h
            up = f()
            flat[i] = keep - h
            down = f()
            flat[i] = keep
            got = grads["d" + n].reshape(-1)[i]
            assert abs((up - down) / (2 * h) - got) <= 1e-6 * max(1.0, abs(got)), (n, i)


def test_scan_closed_forms():
    rng = np.random.default_rng(0)
    k = _ssm_case(rng, reset=False)
    # A = 0, no softplus, dt = 1, D = 0: y is causal linear attention with shared keys and queries per group
    one = np.ones_like(k["dt"])
    y, s = S.ssm_forward(k["x"], one, np.zeros(4), k["b"], k["c"], softplus=False)
    bh, ch = np.repeat(k["b"], 2, 2), np.repeat(k["c"], 2, 2)
    m = np.einsum("bthn,bshn->bhts", ch, bh) * np.tril(np.ones((9, 9)))
    assert np.allclose(y, np.einsum("bhts,bshp->bthp", m, k["x"]), atol=1e-12)
    assert np.allclose(s, np.einsum("bthp,bthn->bhpn", k["x"], bh), atol=1e-12)
    # x = 0: the state decays by exp(A sum dt), the output reads it
    d = np.abs(k["dt"])
    _, s = S.ssm_forward(0 * k["x"], d, k["A"], k["b"], k["c"], s0=k["s0"], softplus=False)
    assert np.allclose(s, k["s0"] * np.exp(k["A"] * d.sum(1))[..., None, None], atol=1e-12)
    # softplus: log(1 + e^v)
    assert np.isclose(S._steps(np.zeros(1), None, True)[0][0], np.log(2.0))


def test_scan_reset_and_split():
    rng = np.random.default_rng(1)
    k = _ssm_case(rng)
    y, s = S.ssm_forward(**k)
    tail = {n: (v[:1, 4:] if n in ("x", "dt", "b", "c") else v) for n, v in k.items() if n not in ("s0", "reset")}
    y1, s1 = S.ssm_forward(**tail)                       # a reset is a fresh zero-state call
    assert np.allclose(y[:1, 4:], y1) and np.allclose(s[:1], s1)
    cut = lambda a, z: {n: (v[:, a:z] if n in ("x", "dt", "b", "c", "reset") else v) for n, v in k.items()}   # noqa: E731
    ya, sa = S.ssm_forward(**cut(0, 5))
    yb, sb = S.ssm_forward(**{**cut(5, 9), "s0": sa})
    assert np.allclose(np.concatenate([ya, yb], 1), y) and np.allclose(sb, s)


@pytest.mark.parametrize("softplus", (True, False))
def test_scan_gradients_by_differences(softplus):
    rng = np.random.default_rng(2)
    k = _ssm_case(rng)
    dy, dsT = rng.standard_normal(k["x"].shape), rng.standard_normal(k["s0"].shape)

    def loss():
        y, s = S.ssm_forward(**k, softplus=softplus)
        return (y * dy).sum() + (s * dsT).sum()
    args = {n: v for n, v in k.items()}
    g = S.ssm_backward(dy=dy, dsT=dsT, softplus=softplus, **args)
    _differences(loss, k, ("x", "dt", "A", "b", "c", "D", "dt_bias", "s0"), g, rng)


@pytest.mark.parametrize("W", (2, 3, 4))
@pytest.mark.parametrize("T", (1, 2, 7))
def test_conv_by_convolution_and_differences(W, T):
    rng = np.random.default_rng(3 + W + T)
    B, D = 2, 5
    k = dict(x=rng.standard_normal((B, T, D)), weight=rng.standard_normal((D, W)), bias=rng.standard_normal(D),
             s0=rng.standard_normal((B, W - 1, D)), reset=np.zeros((B, T), np.uint8))
    y, s = S.conv_forward(**{**k, "reset": None}, silu=False)
    full = np.concatenate([k["s0"], k["x"]], 1)
    for d in range(D):
        for b in range(B):
            assert np.allclose(y[b, :, d], np.convolve(full[b, :, d], k["weight"][d, ::-1], "valid") + k["bias"][d])
    assert np.array_equal(s, full[:, T:])
    if T > 2:
        k["reset"][0, 3] = k["reset"][0, T - 1] = 1
        ya, _ = S.conv_forward(k["x"][:1, 3:], k["weight"], k["bias"], None, k["reset"][:1, 3:])
        assert np.allclose(S.conv_forward(**k)[0][:1, 3:], ya)      # a reset is a fresh start
        assert not S.conv_forward(**k)[1][0, :-1].any()
    dy, dsT = rng.standard_normal((B, T, D)), rng.standard_normal((B, W - 1, D))

    def loss():
        y, s = S.conv_forward(**k)
        return (y * dy).sum() + (s * dsT).sum()
    _differences(loss, k, ("x", "weight", "bias", "s0"), S.conv_backward(dy=dy, dsT=dsT, **k), rng)


@pytest.mark.parametrize("groups", (1, 3))
@pytest.mark.parametrize("gated", (False, True))
def test_norm_closed_form_and_differences(groups, gated):
    rng = np.random.default_rng(9)
    k = dict(x=rng.standard_normal((4, 12)), weight=rng.standard_normal(12), gate=rng.standard_normal((4, 12)) if gated else None)
    assert np.allclose(S.rms_forward(3.0 * np.ones((2, 12)), np.ones(12), 0.0, groups=groups), 1.0)
    assert np.allclose(S.rms_forward(7.0 * k["x"], k["weight"], 0.0, groups=groups), S.rms_forward(k["x"], k["weight"], 0.0, groups=groups))
    dout = rng.standard_normal((4, 12))
    g = S.rms_backward(k["x"], k["weight"], dout, 1e-3, k["gate"], groups=groups)
    loss = lambda: (S.rms_forward(k["x"], k["weight"], 1e-3, k["gate"], groups) * dout).sum()   # noqa: E731
    _differences(loss, k, ("x", "weight") + (("gate",) if gated else ()), g, rng)
    if not gated:
        dh = rng.standard_normal((4, 12))
        assert np.allclose(S.rms_backward(k["x"], k["weight"], dout, 1e-3, dh=dh, groups=groups)["dx"], g["dx"] + dh)
