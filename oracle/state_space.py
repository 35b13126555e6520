"""fp64 oracle of the state-space layer: the short causal convolution, the selective scan and the RMS norm, token by
token from their definitions, with hand-derived reverse modes.  Test infrastructure only; shares no code with the
CUDA path."""
from __future__ import annotations

import numpy as np


def _f64(*xs):
    return [None if x is None else np.asarray(x, np.float64) for x in xs]


def sigmoid(v):
    return 1.0 / (1.0 + np.exp(-v))


def _window(x, s0, reset, t, W):
    """The W inputs that token t's taps see, oldest first, zero where there is none or a reset cuts it off."""
    B, T, D = x.shape
    win = np.zeros((B, W, D))
    alive = np.ones(B, bool)
    for j in range(W):          # tap j reads token t - j
        if j > 0 and reset is not None and t - j + 1 >= 0:
            alive &= reset[:, t - j + 1] == 0
        i = t - j
        row = x[:, i] if i >= 0 else (s0[:, W - 1 + i] if s0 is not None else np.zeros((B, D)))
        win[:, W - 1 - j] = np.where(alive[:, None], row, 0.0)
    return win


def conv_state(x, s0, reset, W):
    """The last W - 1 inputs after the row, oldest first (zero before the last reset)."""
    B, T, D = x.shape
    out = np.zeros((B, W - 1, D))
    alive = np.ones(B, bool)
    for j in range(1, W):       # x_{T-j}
        i = T - j
        row = x[:, i] if i >= 0 else (s0[:, W - 1 + i] if s0 is not None else np.zeros((B, D)))
        out[:, W - 1 - j] = np.where(alive[:, None], row, 0.0)
        if reset is not None and i >= 0:
            alive &= reset[:, i] == 0
    return out


def conv_forward(x, weight, bias=None, s0=None, reset=None, silu=True):
    x, weight, bias, s0 = _f64(x, weight, bias, s0)
    B, T, D = x.shape
    W = weight.shape[1]
    y = np.zeros((B, T, D))
    for t in range(T):
        u = np.einsum("bwd,dw->bd", _window(x, s0, reset, t, W), weight) + (0.0 if bias is None else bias)
        y[:, t] = u * sigmoid(u) if silu else u
    return y, conv_state(x, s0, reset, W)


def conv_backward(x, weight, dy, bias=None, s0=None, reset=None, dsT=None, silu=True):
    x, weight, dy, bias, s0, dsT = _f64(x, weight, dy, bias, s0, dsT)
    B, T, D = x.shape
    W = weight.shape[1]
    dfull = np.zeros((B, W - 1 + T, D))          # gradients of s0, then of x
    dw, db = np.zeros((D, W)), np.zeros(D)
    for t in range(T):
        win = _window(x, s0, reset, t, W)
        u = np.einsum("bwd,dw->bd", win, weight) + (0.0 if bias is None else bias)
        s = sigmoid(u)
        g = dy[:, t] * (s * (1.0 + u * (1.0 - s)) if silu else 1.0)
        db += g.sum(0)
        dw += np.einsum("bd,bwd->dw", g, win)
        alive = np.ones(B, bool)
        for j in range(W):
            if j > 0 and reset is not None and t - j + 1 >= 0:
                alive &= reset[:, t - j + 1] == 0
            dfull[:, W - 1 + t - j] += np.where(alive[:, None], g * weight[:, W - 1 - j], 0.0)
    if dsT is not None:
        alive = np.ones(B, bool)
        for j in range(1, W):
            i = T - j
            dfull[:, W - 1 + i] += np.where(alive[:, None], dsT[:, W - 1 - j], 0.0)
            if reset is not None and i >= 0:
                alive &= reset[:, i] == 0
    return {"dx": dfull[:, W - 1:], "ds0": dfull[:, :W - 1], "dweight": dw, "dbias": db}


def _steps(dt, dt_bias, softplus):
    raw = dt + (0.0 if dt_bias is None else dt_bias)
    return (np.logaddexp(0.0, raw), sigmoid(raw)) if softplus else (raw, np.ones_like(raw))


def ssm_forward(x, dt, A, b, c, D=None, dt_bias=None, s0=None, reset=None, softplus=True, keep=False):
    """y [B,T,H,P], final state [B,H,P,N] (and every state when ``keep``)."""
    x, dt, A, b, c, D, dt_bias, s0 = _f64(x, dt, A, b, c, D, dt_bias, s0)
    B, T, H, P = x.shape
    hg = H // b.shape[2]
    b, c = np.repeat(b, hg, 2), np.repeat(c, hg, 2)
    d, _ = _steps(dt, dt_bias, softplus)
    S = np.zeros((B, H, P, b.shape[-1])) if s0 is None else s0.copy()
    y, states = np.zeros((B, T, H, P)), [S]
    for t in range(T):
        if reset is not None:
            S = np.where((reset[:, t] != 0)[:, None, None, None], 0.0, S)
        S = np.exp(d[:, t] * A)[:, :, None, None] * S + (d[:, t, :, None] * x[:, t])[..., None] * b[:, t, :, None]
        y[:, t] = np.einsum("bhpn,bhn->bhp", S, c[:, t]) + (0.0 if D is None else D[:, None] * x[:, t])
        if keep:
            states.append(S)
    return (y, S, states) if keep else (y, S)


def ssm_backward(x, dt, A, b, c, dy, D=None, dt_bias=None, s0=None, reset=None, dsT=None, softplus=True, sizes=False):
    """``sizes``: with every input but dt and A non-negative, the sums of the absolute terms behind each gradient."""
    _, _, states = ssm_forward(x, dt, A, b, c, D, dt_bias, s0, reset, softplus, keep=True)
    x, dt, A, b, c, dy, D, dt_bias, dsT = _f64(x, dt, A, b, c, dy, D, dt_bias, dsT)
    B, T, H, P = x.shape
    G, N = b.shape[2], b.shape[3]
    hg = H // G
    bh, ch = np.repeat(b, hg, 2), np.repeat(c, hg, 2)
    d, sg = _steps(dt, dt_bias, softplus)
    dS = np.zeros((B, H, P, N)) if dsT is None else dsT.copy()
    g = {"dx": np.zeros_like(x), "ddt": np.zeros_like(dt), "db": np.zeros_like(b), "dc": np.zeros_like(c),
         "dA": np.zeros(H), "dD": np.zeros(H), "ddt_bias": np.zeros(H)}
    for t in range(T - 1, -1, -1):
        before = states[t]
        if reset is not None:
            before = np.where((reset[:, t] != 0)[:, None, None, None], 0.0, before)
        dS = dS + dy[:, t, :, :, None] * ch[:, t, :, None]
        g["dc"][:, t] = np.einsum("bhpn,bhp->bhn", states[t + 1], dy[:, t]).reshape(B, G, hg, N).sum(2)
        du = np.einsum("bhpn,bhn->bhp", dS, bh[:, t])
        g["db"][:, t] = np.einsum("bhpn,bhp->bhn", dS, d[:, t, :, None] * x[:, t]).reshape(B, G, hg, N).sum(2)
        f = np.exp(d[:, t] * A)
        da = f * np.einsum("bhpn,bhpn->bh", before, dS)
        g["dx"][:, t] = d[:, t, :, None] * du + (0.0 if D is None else D[:, None] * dy[:, t])
        ddt = ((np.abs(A) if sizes else A) * da + np.einsum("bhp,bhp->bh", x[:, t], du)) * sg[:, t]
        g["ddt"][:, t] = ddt
        g["dA"] += (d[:, t] * da).sum(0)
        g["ddt_bias"] += ddt.sum(0)
        g["dD"] += np.einsum("bhp,bhp->h", x[:, t], dy[:, t])
        dS = f[:, :, None, None] * dS
        if reset is not None:
            dS = np.where((reset[:, t] != 0)[:, None, None, None], 0.0, dS)
    g["ds0"] = dS
    return g


def rms_forward(x, weight, eps, gate=None, groups=1):
    """out for h = x (a residual's sum is formed, and rounded to its storage, by the caller) or x silu(gate)."""
    x, weight, gate = _f64(x, weight, gate)
    h = x if gate is None else x * gate * sigmoid(gate)
    v = h.reshape(*h.shape[:-1], groups, -1)
    return (v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)).reshape(h.shape) * weight


def rms_backward(x, weight, dout, eps, gate=None, dh=None, groups=1):
    x, weight, dout, gate, dh = _f64(x, weight, dout, gate, dh)
    D = x.shape[-1]
    s = None if gate is None else sigmoid(gate)
    h = x if gate is None else x * gate * s
    v = h.reshape(-1, groups, D // groups)
    r = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    q = (dout * weight).reshape(v.shape)
    dv = r * q - v * r ** 3 * (q * v).mean(-1, keepdims=True)
    dv = dv.reshape(x.shape)
    g = {"dweight": (dout.reshape(-1, D) * (v * r).reshape(-1, D)).sum(0)}
    if gate is None:
        g["dx"] = dv if dh is None else dv + dh
    else:
        g["dx"] = dv * gate * s
        g["dgate"] = dv * x * s * (1.0 + gate * (1.0 - s))
    return g
