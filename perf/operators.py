"""What the state-space operators cost: the cases, their plain forms in elementary torch operations, the
library's calls, the work of one pass, and the same results from the definitions in 64 bits.

``own`` is false for the plain forms and true for the library's kernels.  Operators: the short causal
convolution (``conv``), the selective state-space scan (``ssm``) and the RMS norm (``rms``), each in the
directions that a layer uses: forward (prompts), training (forward and backward) and single tokens.
"""
from __future__ import annotations

import math

import torch

own = False

P = 64                      # channels of a head
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
CHUNK = 64                  # tokens of a chunk of the plain scan
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a layer's convolution on a packed training batch: 32 heads of 64 and one 128-wide b and c
        dict(name="conv_forward_packed", op="conv", mode="forward", dtype="bf16", B=8, T=4096, D=2304, W=4, silu=True,
             reset=True, state=False),
        # its training step at the 184M-model layer shape: 12 heads of 64, b and c of 64
        dict(name="conv_train_layer", op="conv", mode="train", dtype="bf16", B=2, T=512, D=896, W=4, silu=True,
             reset=True, state=True),
        # batched decode, one token per row
        dict(name="conv_step_decode", op="conv", mode="step", dtype="bf16", B=256, T=1, D=2304, W=4, silu=True,
             reset=False, state=True),
        # prompt of the 1.5B-model layer on a carried state
        dict(name="ssm_forward_prefill", op="ssm", mode="forward", dtype="bf16", B=1, T=1024, H=32, G=1, N=128,
             reset=False, state=True),
        # one long prompt over few heads, odd length
        dict(name="ssm_forward_long_odd", op="ssm", mode="forward", dtype="bf16", B=1, T=8001, H=24, G=2, N=64,
             reset=False, state=True),
        # packed training batch of documents, forward and backward
        dict(name="ssm_train_packed", op="ssm", mode="train", dtype="bf16", B=8, T=4096, H=32, G=1, N=128,
             reset=True, state=False),
        # the 184M-model layer shape in fp32
        dict(name="ssm_train_layer_f32", op="ssm", mode="train", dtype="f32", B=2, T=512, H=12, G=1, N=64,
             reset=True, state=True),
        # fp16, ragged, two groups
        dict(name="ssm_train_odd_f16", op="ssm", mode="train", dtype="f16", B=3, T=777, H=6, G=2, N=64,
             reset=True, state=True),
        # batched decode, all states resident
        dict(name="ssm_step_decode", op="ssm", mode="step", dtype="bf16", B=256, T=1, H=32, G=1, N=128,
             reset=False, state=True),
        # the norm before the projection of a packed batch, with the residual's addition and 8-bit output
        dict(name="rms_residual_e4m3", op="rms", mode="forward", dtype="bf16", rows=32768, D=2048, groups=1,
             kind="residual", block=128),
        # the gated norm after the scan, trained
        dict(name="rms_gate_train", op="rms", mode="train", dtype="bf16", rows=8192, D=2048, groups=1, kind="gate",
             block=0),
        # the norm of a decode step, 8-bit output
        dict(name="rms_decode_e4m3", op="rms", mode="forward", dtype="bf16", rows=256, D=2048, groups=1,
             kind="residual", block=128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("conv", "ssm", "ssm", "rms"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "rms":
        groups = rng.choice((1, 1, 1, 2, 8))
        block = rng.choice((0, 0, 128, -1))
        # a slice of a row: whole 128-channel blocks where the output is in 8 bits, else any multiple of 8
        per = 128 * _log_int(rng, 1, 16) if block == 128 else 8 * _log_int(rng, 1, 512 // groups)
        mode = "forward" if block else rng.choice(("forward", "train"))
        rows = min(_log_int(rng, 1, 32768), max(1, 32768 * 2048 // (per * groups)))
        return dict(op="rms", mode=mode, dtype=dtype, rows=rows, D=per * groups, groups=groups,
                    kind=rng.choice(("plain", "residual", "gate")), block=block)
    mode = rng.choice(("forward", "train", "train", "step"))
    T = 1 if mode == "step" else _log_int(rng, 1, 6000)
    B = _log_int(rng, 1, 256 if mode == "step" else 8)
    reset = mode != "step" and rng.random() < 0.5
    state = mode == "step" or rng.random() < 0.5
    if op == "conv":
        D = 8 * _log_int(rng, 1, 512)
        return dict(op="conv", mode=mode, dtype=dtype, B=B, T=min(T, max(1, 4096 * 8 * 2304 // (B * D))), D=D,
                    W=rng.choice((2, 3, 4, 4)), silu=rng.random() < 0.8, reset=reset, state=state)
    G = rng.choice((1, 1, 2, 4))
    H = G * _log_int(rng, 1, 32 // G)
    N = rng.choice((64, 128))
    cap = (256 * 32 if mode == "step" else 1 << 19) // (B * H)   # token-heads of a drawn case
    return dict(op="ssm", mode=mode, dtype=dtype, B=B, T=min(T, max(1, cap)), H=H, G=G, N=N, reset=reset, state=state)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    s = {"case": case}
    train = case["mode"] == "train"
    if case["op"] == "rms":
        n, D = case["rows"], case["D"]
        s["x"] = normal(n, D, dtype=dt)
        s["other"] = None if case["kind"] == "plain" else normal(n, D, dtype=dt)
        s["weight"] = 1.0 + normal(D, std=0.1)
        if train:
            s["dy"] = normal(n, D, dtype=dt)
            s["dh"] = normal(n, D, dtype=dt) if case["kind"] == "residual" else None
        return s
    B, T = case["B"], case["T"]
    if case["reset"]:   # documents of geometric length, mean 512 (shorter rows: an eighth of the row)
        s["reset"] = (torch.rand(B, T, generator=g, device="cuda") < 1.0 / min(512, max(2, T // 8))).to(torch.uint8)
    else:
        s["reset"] = None
    if case["op"] == "conv":
        D, W = case["D"], case["W"]
        s["x"] = normal(B, T, D, dtype=dt)
        s["weight"] = uniform(-1.0, 1.0, D, W) / math.sqrt(W)
        s["bias"] = normal(D, std=0.1)
        s["s0"] = normal(B, W - 1, D, dtype=dt) if case["state"] else None
        s["active"] = (torch.rand(B, generator=g, device="cuda") < 0.9).to(torch.uint8) if case["mode"] == "step" else None
        if train:
            s["dy"] = normal(B, T, D, dtype=dt)
            s["dsT"] = normal(B, W - 1, D, dtype=dt) if case["state"] else None
        return s
    H, G, N = case["H"], case["G"], case["N"]
    # x, b and c lie side by side in the convolution's output, whose activation is silu
    xbc = torch.nn.functional.silu(normal(B, T, H * P + 2 * G * N)).to(dt)
    s["x"] = xbc[..., :H * P].unflatten(-1, (H, P))
    s["b"] = xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N))
    s["c"] = xbc[..., H * P + G * N:].unflatten(-1, (G, N))
    s["dt"] = normal(B, T, H, dtype=dt)
    s["A"] = -uniform(1.0, 16.0, H)
    s["D"] = 1.0 + normal(H, std=0.1)
    dt0 = torch.exp(uniform(math.log(1e-3), math.log(1e-1), H))
    s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))          # softplus(dt_bias) = dt0
    s["s0"] = normal(B, H, P, N, std=0.1) if case["state"] else None
    s["active"] = (torch.rand(B, generator=g, device="cuda") < 0.9).to(torch.uint8) if case["mode"] == "step" else None
    if case["mode"] == "step":
        s["x"], s["b"], s["c"], s["dt"] = (s[n][:, 0].contiguous() for n in ("x", "b", "c", "dt"))
    if train:
        s["dy"] = normal(B, T, H, P, dtype=dt)
        s["dsT"] = normal(B, H, P, N, std=0.1) if case["state"] else None
    return s


# ------------------------------------------------------------------ plain forms (32 bits)
def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _softplus(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp(min=0.0)


def _plain_conv(x, weight, bias, s0, reset, silu):
    """(y, s_out) in 32 bits: the W - 1 inputs before the row, then W shifted products."""
    B, T, D = x.shape
    W = weight.shape[1]
    past = torch.zeros(B, W - 1, D, device=x.device) if s0 is None else s0.float()
    full = torch.cat([past, x.float()], 1)                       # [B, T + W - 1, D]
    seg = torch.zeros(B, T + W - 1, dtype=torch.int32, device=x.device)
    if reset is not None:
        seg[:, W - 1:] = torch.cumsum((reset != 0).to(torch.int32), 1)
    taps = full.unfold(1, W, 1)                                  # [B, T, D, W]: x_{t-W+1} .. x_t
    same = seg.unfold(1, W, 1)
    same = (same == same[..., -1:]).to(taps.dtype)
    u = (taps * same[:, :, None] * weight).sum(-1) + bias
    y = _silu(u) if silu else u
    s_out = full[:, T:] * (seg[:, T:] == seg[:, -1:]).to(full.dtype)[..., None]
    return y, s_out


def _plain_ssm(x, dt, A, b, c, D, dt_bias, s0, reset):
    """(y, s_out) in 32 bits (the running sums of the decays in 64), chunk by chunk of CHUNK tokens, all chunks at once."""
    B, T, H, _ = x.shape
    G, N = b.shape[2], b.shape[3]
    x, b, c = x.float(), b.float(), c.float()
    step = _softplus(dt.float() + dt_bias)
    y_d = D[:, None] * x
    pad = -T % CHUNK
    n = (T + pad) // CHUNK
    rst = torch.zeros(B, T, dtype=torch.int64, device=x.device) if reset is None else (reset != 0).to(torch.int64)
    if pad:
        x, b, c, step = (torch.cat([t, t.new_zeros(B, pad, *t.shape[2:])], 1) for t in (x, b, c, step))
        rst = torch.cat([rst, rst.new_zeros(B, pad)], 1)
    u = (x * step[..., None]).view(B, n, CHUNK, G, H // G, P)
    b, c = b.view(B, n, CHUNK, G, N), c.view(B, n, CHUNK, G, N)
    log = (step.double() * A.double()).view(B, n, CHUNK, G, H // G)
    lam = torch.cumsum(log, 2)                                    # within the chunk, this token's decay included
    seg = torch.cumsum(rst.view(B, n, CHUNK), 2)
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=x.device).tril()
    keep = (seg[:, :, :, None] == seg[:, :, None, :]) & tri                       # [B, n, t, s]
    diff = lam[:, :, :, None] - lam[:, :, None, :]                                 # [B, n, t, s, G, h]
    diff = diff.masked_fill(~keep[..., None, None], -math.inf).float()
    gram = torch.einsum("bntgk,bnsgk->bntsg", c, b)
    y = torch.einsum("bntsgh,bnsghp->bntghp", torch.exp(diff) * gram[..., None], u)
    # states that the chunks leave, from zero
    to_end = (lam[:, :, -1:] - lam).masked_fill((seg != seg[:, :, -1:])[..., None, None], -math.inf).float()
    local = torch.einsum("bnsghp,bnsgk->bnghpk", u * torch.exp(to_end)[..., None], b)
    # state entering chunk i: sum over j < i of the decays of the chunks between, then the initial state
    total = torch.cumsum(lam[:, :, -1], 1)                                         # [B, n, G, h], inclusive
    cuts = torch.cumsum(seg[:, :, -1], 1)                                          # resets so far, inclusive
    total = torch.cat([torch.zeros_like(total[:, :1]), total], 1)                  # [B, n + 1, ...]: before chunk i
    cuts = torch.cat([torch.zeros_like(cuts[:, :1]), cuts], 1)
    i, j = torch.arange(n + 1, device=x.device), torch.arange(n, device=x.device)
    ok = (j[None, :] < i[:, None]) & (cuts[:, :, None] == cuts[:, None, 1:])       # [B, n + 1, n]
    between = (total[:, :, None] - total[:, None, 1:]).masked_fill(~ok[..., None, None], -math.inf).float()
    S = torch.einsum("bijgh,bjghpk->bighpk", torch.exp(between), local)
    if s0 is not None:
        from0 = total.masked_fill((cuts != 0)[..., None, None], -math.inf).float()
        S = S + torch.exp(from0)[..., None, None] * s0.view(B, 1, G, H // G, P, N)
    reach = lam.masked_fill((seg != 0)[..., None, None], -math.inf).float()
    y = y + torch.exp(reach)[..., None] * torch.einsum("bntgk,bnghpk->bntghp", c, S[:, :n])
    y = y.reshape(B, n * CHUNK, H, P)[:, :T] + y_d
    return y, S[:, n].reshape(B, H, P, N)


def _plain_rms(x, other, weight, kind, groups, dt):
    """(out, h) in 32 bits."""
    h = x.float()
    if kind == "residual":   # the stored sum is what is normalised (and what a backward pass reads)
        h = h + other.float()
        h = h + (h.to(dt).float() - h).detach()
    elif kind == "gate":
        h = h * _silu(other.float())
    v = h.unflatten(-1, (groups, -1))
    out = (v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)).flatten(-2) * weight
    return out, h


def _quantise(out, block, groups):
    """e4m3 codes and one scale per block of channels (-1: per normalised slice); a block of zeros keeps the scale 1."""
    v = out.unflatten(-1, (-1, block if block > 0 else out.shape[-1] // groups))
    top = v.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    return (v / scale).flatten(-2).to(torch.float8_e4m3fn), scale[..., 0]


def _grad(outputs, grads, inputs):
    """Gradients of the plain form by the chain rule over its own elementary steps."""
    return torch.autograd.grad([o for o, g in zip(outputs, grads) if g is not None],
                               inputs, [g.float() for g in grads if g is not None])


def _leaf(t):
    return None if t is None else t.detach().float().requires_grad_(True)


def _run_plain(s):
    case = s["case"]
    dt = DTYPES[case["dtype"]]
    op, mode = case["op"], case["mode"]
    if op == "rms":
        if mode == "forward":
            out, h = _plain_rms(s["x"], s["other"], s["weight"], case["kind"], case["groups"], dt)
            r = {"h": h.to(dt)} if case["kind"] == "residual" else {}
            if case["block"]:
                r["q"], r["scale"] = _quantise(out, case["block"], case["groups"])
            else:
                r["out"] = out.to(dt)
            return r
        x, other, w = _leaf(s["x"]), _leaf(s["other"]), _leaf(s["weight"])
        out, h = _plain_rms(x, other, w, case["kind"], case["groups"], dt)
        g = _grad((out, h), (s["dy"], s["dh"]), (x, w) + ((other,) if case["kind"] == "gate" else ()))
        r = {"out": out.detach().to(dt), "dx": g[0].to(dt), "dweight": g[1]}
        if case["kind"] == "gate":
            r["dgate"] = g[2].to(dt)
        return r
    if op == "conv":
        if mode == "step":
            on = s["active"].bool()
            y, s_out = _plain_conv(s["x"], s["weight"], s["bias"], s["s0"], None, case["silu"])
            s["s0"].copy_(torch.where(on[:, None, None], s_out.to(dt), s["s0"]))   # the resident state
            return {"y": torch.where(on[:, None, None], y, torch.zeros_like(y)).to(dt), "state": s["s0"]}
        if mode == "forward":
            y, s_out = _plain_conv(s["x"], s["weight"], s["bias"], s["s0"], s["reset"], case["silu"])
            return {"y": y.to(dt), "s_out": s_out.to(dt)}
        x, w, bias, s0 = (_leaf(s[n]) for n in ("x", "weight", "bias", "s0"))
        y, s_out = _plain_conv(x, w, bias, s0, s["reset"], case["silu"])
        g = _grad((y, s_out), (s["dy"], s["dsT"]), (x, w, bias) + (() if s0 is None else (s0,)))
        r = {"y": y.detach().to(dt), "s_out": s_out.detach().to(dt), "dx": g[0].to(dt), "dweight": g[1], "dbias": g[2]}
        if s0 is not None:
            r["ds0"] = g[3].to(dt)
        return r
    if mode == "step":
        G, hg = case["G"], case["H"] // case["G"]
        on = s["active"].bool()[:, None, None, None]
        step = _softplus(s["dt"].float() + s["dt_bias"])[..., None, None]
        x = s["x"].float()
        b, c = (s[n].float().repeat_interleave(hg, 1)[:, :, None] for n in ("b", "c"))
        S = torch.exp(step * s["A"][:, None, None]) * s["s0"] + step * x[..., None] * b
        y = (S * c).sum(-1) + s["D"][:, None] * x
        s["s0"].copy_(torch.where(on, S, s["s0"]))                                  # the resident state
        return {"y": torch.where(on[..., 0], y, torch.zeros_like(y)).to(dt), "state": s["s0"]}
    if mode == "forward":
        y, s_out = _plain_ssm(s["x"], s["dt"], s["A"], s["b"], s["c"], s["D"], s["dt_bias"], s["s0"], s["reset"])
        return {"y": y.to(dt), "s_out": s_out}
    names = ("x", "dt", "A", "b", "c", "D", "dt_bias") + (("s0",) if s["s0"] is not None else ())
    leaf = {n: _leaf(s[n]) for n in names}
    y, s_out = _plain_ssm(leaf["x"], leaf["dt"], leaf["A"], leaf["b"], leaf["c"], leaf["D"], leaf["dt_bias"], leaf.get("s0"),
                          s["reset"])
    g = dict(zip(names, _grad((y, s_out), (s["dy"], s["dsT"]), [leaf[n] for n in names])))
    r = {"y": y.detach().to(dt), "s_out": s_out.detach()}
    r.update({"d" + n: g[n].to(dt) for n in ("x", "dt", "b", "c")})
    r.update({"d" + n: g[n] for n in names if n in ("A", "D", "dt_bias", "s0")})
    return r


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    from linear_recurrent_lm_b200 import wkv7
    case = s["case"]
    op, mode = case["op"], case["mode"]
    if op == "rms":
        kw = {case["kind"]: s["other"]} if s["other"] is not None else {}
        f = wkv7.rms_forward(s["x"], s["weight"], EPS, groups=case["groups"], quant_block=case["block"], **kw)
        if mode == "forward":
            names = ("h",) * (case["kind"] == "residual") + (("q", "scale") if case["block"] else ("out",))
            return {n: f[n] for n in names}
        if case["kind"] == "residual":   # the backward reads the sum that the forward stored
            g = wkv7.rms_backward(f["h"], s["weight"], s["dy"], EPS, groups=case["groups"], dh=s["dh"])
        else:
            g = wkv7.rms_backward(s["x"], s["weight"], s["dy"], EPS, groups=case["groups"], **kw)
        return {"out": f["out"], **{n: g[n] for n in ("dx", "dweight", "dgate") if n in g}}
    if op == "conv":
        if mode == "step":
            y = wkv7.conv_step(s["x"][:, 0], s["weight"], s["s0"], s["bias"], s["active"], silu=case["silu"])
            return {"y": y[:, None], "state": s["s0"]}
        y, s_out = wkv7.conv_forward(s["x"], s["weight"], s["bias"], s["s0"], s["reset"], silu=case["silu"])
        if mode == "forward":
            return {"y": y, "s_out": s_out}
        g = wkv7.conv_backward(s["x"], s["weight"], s["dy"], s["bias"], s["s0"], s["reset"], s["dsT"], silu=case["silu"],
                               want_ds0=s["s0"] is not None)
        return {"y": y, "s_out": s_out, **{n: g[n] for n in ("dx", "dweight", "dbias", "ds0") if g.get(n) is not None}}
    args = [s[n] for n in ("x", "dt", "A", "b", "c")]
    if mode == "step":
        y = wkv7.ssm_step(*args, s["s0"], s["D"], s["dt_bias"], s["active"], softplus=True)
        return {"y": y, "state": s["s0"]}
    y, s_out, ws = wkv7.ssm_forward(*args, s["D"], s["dt_bias"], s["s0"], s["reset"], softplus=True)
    if mode == "forward":
        return {"y": y, "s_out": s_out}
    g = wkv7.ssm_backward(*args, s["dy"], ws, s["D"], s["dt_bias"], s["s0"], s["reset"], s["dsT"], softplus=True,
                          want_ds0=s["s0"] is not None)
    return {"y": y, "s_out": s_out, **{n: t for n, t in g.items() if t is not None}}


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ------------------------------------------------------------------ work
def work(case):
    e = BYTES[case["dtype"]]
    op, train = case["op"], case["mode"] == "train"
    if op == "rms":
        n, D = case["rows"] * case["D"], case["D"]
        two = case["kind"] != "plain"
        if train:   # x (and the other) and dy in, out, dx (and dgate) out; dh in
            t = 4 + (2 if case["kind"] == "gate" else 0) + (2 if case["kind"] == "residual" else 0)
            return {"bytes": t * n * e + 8 * D, "flops": 20 * n}
        out = n * (1 if case["block"] else e) + (4 * n / (case["block"] if case["block"] > 0 else D // case["groups"]) if case["block"] else 0)
        return {"bytes": n * e * (1 + two + (case["kind"] == "residual")) + out + 4 * D, "flops": 8 * n}
    B, T = case["B"], case["T"]
    if op == "conv":
        D, W = case["D"], case["W"]
        state = B * (W - 1) * D * e
        if case["mode"] == "step":
            return {"bytes": 2 * B * D * e + 2 * state + 4 * D * (W + 1), "flops": B * D * (2 * W + 6)}
        n = B * T * D
        per = 4 if train else 2
        return {"bytes": per * n * e + state * (2 if train else 1) + 4 * D * (W + 1) * (2 if train else 1),
                "flops": n * (2 * W + 6) * (3 if train else 1)}
    H, G, N = case["H"], case["G"], case["N"]
    th = B * T * H
    state = 4 * B * H * P * N
    tok = e * (th * (P + 1) + 2 * B * T * G * N)          # x, dt, b, c once
    if case["mode"] == "step":
        return {"bytes": tok + e * th * P + 2 * state, "flops": th * P * N * 5}
    if train:   # inputs, dy; y, the four gradients; the end state
        return {"bytes": 2 * tok + 2 * e * th * P + state * (1 + (3 if case["state"] else 0)), "flops": th * P * N * 16}
    return {"bytes": tok + e * th * P + state * (1 + case["state"]), "flops": th * P * N * 5}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    """What ``run`` returns for these inputs, from the definitions in 64 bits: the convolution tap by tap, the
    scan as one dense lower-triangular matrix per row and head, gradients by reverse mode on those."""
    s = prepare(case, seed)
    d = {n: t.double() if torch.is_tensor(t) and t.is_floating_point() else t for n, t in s.items()}
    op, mode = case["op"], case["mode"]
    with torch.enable_grad():
        if op == "rms":
            return _exact_rms(case, d)
        if op == "conv":
            return _exact_conv(case, d)
        return _exact_ssm_step(case, d) if mode == "step" else _exact_ssm(case, d)


def _exact_rms(case, d):
    train = case["mode"] == "train"
    x, w, z = (t.requires_grad_(train) if t is not None else None for t in (d["x"], d["weight"], d["other"]))
    h = x * z * torch.sigmoid(z) if case["kind"] == "gate" else x
    if case["kind"] == "residual":   # the sum as it is stored, in the inputs' type
        h = x + z
        h = h + ((x + z).detach().to(DTYPES[case["dtype"]]).double() - h.detach())
    parts = []
    per = case["D"] // case["groups"]
    for i in range(case["groups"]):
        v = h[:, i * per:(i + 1) * per]
        parts.append(v / torch.sqrt(v.pow(2).sum(1, keepdim=True) / per + EPS) * w[i * per:(i + 1) * per])
    out = torch.cat(parts, 1)
    if not train:
        r = {"h": h} if case["kind"] == "residual" else {}
        if case["block"]:
            v = out.reshape(case["rows"], -1, case["block"] if case["block"] > 0 else per)
            top = v.abs().max(2).values
            r["scale"] = torch.where(top > 0, top / E4M3_MAX, 1.0)
            r["q"] = (v / r["scale"][..., None]).reshape(out.shape)
        else:
            r["out"] = out
        return r
    loss = (out * d["dy"]).sum() + ((h * d["dh"]).sum() if d["dh"] is not None else 0.0)
    loss.backward()
    r = {"out": out.detach(), "dx": x.grad, "dweight": w.grad}
    if case["kind"] == "gate":
        r["dgate"] = z.grad
    return r


def _exact_conv(case, d):
    B, T, D, W = case["B"], case["T"], case["D"], case["W"]
    train = case["mode"] == "train"
    x, w, bias, s0 = (t.requires_grad_(train) if t is not None else None for t in (d["x"], d["weight"], d["bias"], d["s0"]))
    past = torch.zeros(B, W - 1, D, device=x.device, dtype=torch.float64) if s0 is None else s0
    rst = torch.zeros(B, T, dtype=torch.bool, device=x.device) if d["reset"] is None else d["reset"].bool()
    u = bias + w[:, W - 1] * x
    alive = torch.ones(B, T, 1, dtype=torch.float64, device=x.device)   # no reset between the tap and the token
    keep = []                                                           # the state after the row, newest first
    live = torch.ones(B, 1, dtype=torch.float64, device=x.device)
    for j in range(1, W):
        cut = torch.ones(B, T, dtype=torch.bool, device=x.device)       # reset at token t - j + 1 (none before the row)
        if j - 1 < T:
            cut[:, j - 1:] = ~rst[:, :T - j + 1]
        alive = alive * cut[..., None]
        tap = torch.cat([past[:, max(0, W - 1 - j):W - 1 - j + min(j, T)], x[:, :max(0, T - j)]], 1)
        u = u + w[:, W - 1 - j] * alive * tap
    for j in range(1, W):
        keep.append((x[:, T - j] if T - j >= 0 else past[:, W - 1 + T - j]) * live)
        if T - j >= 0:
            live = live * (~rst[:, T - j])[:, None]
    y = u * torch.sigmoid(u) if case["silu"] else u
    s_out = torch.stack(keep[::-1], 1)
    if case["mode"] == "step":
        on = d["active"].bool()[:, None, None]
        return {"y": torch.where(on, y, 0.0), "state": torch.where(on, s_out, past)}
    if not train:
        return {"y": y, "s_out": s_out}
    loss = (y * d["dy"]).sum() + ((s_out * d["dsT"]).sum() if d["dsT"] is not None else 0.0)
    loss.backward()
    r = {"y": y.detach(), "s_out": s_out.detach(), "dx": x.grad, "dweight": w.grad, "dbias": bias.grad}
    if s0 is not None:
        r["ds0"] = s0.grad
    return r


def _exact_ssm_step(case, d):
    hg = case["H"] // case["G"]
    on = d["active"].bool()[:, None, None, None]
    y, new = [], []
    for h in range(case["H"]):
        step = torch.log1p(torch.exp(d["dt"][:, h] + d["dt_bias"][h]))[:, None, None]
        S = torch.exp(step * d["A"][h]) * d["s0"][:, h] + step * d["x"][:, h, :, None] * d["b"][:, h // hg, None, :]
        y.append(torch.einsum("bpk,bk->bp", S, d["c"][:, h // hg]) + d["D"][h] * d["x"][:, h])
        new.append(S)
    y, S = torch.stack(y, 1), torch.stack(new, 1)
    return {"y": torch.where(on[..., 0], y, 0.0), "state": torch.where(on, S, d["s0"])}


def _exact_ssm(case, d):
    B, T, H, hg = case["B"], case["T"], case["H"], case["H"] // case["G"]
    train = case["mode"] == "train"
    names = [n for n in ("x", "dt", "A", "b", "c", "D", "dt_bias", "s0") if d.get(n) is not None]
    y = torch.zeros_like(d["x"])
    s_out = torch.zeros(B, H, P, case["N"], device=y.device, dtype=torch.float64)
    grads = {n: torch.zeros_like(d[n]) for n in names}
    late = torch.ones(T, T, dtype=torch.bool, device=y.device).triu(1)
    for i in range(B):
        cuts = torch.zeros(T, dtype=torch.int64, device=y.device) if d["reset"] is None else d["reset"][i].bool().cumsum(0)
        off = late | (cuts[:, None] != cuts[None, :])
        for h in range(H):
            at = {"x": (i, slice(None), h), "dt": (i, slice(None), h), "A": h, "b": (i, slice(None), h // hg),
                  "c": (i, slice(None), h // hg), "D": h, "dt_bias": h, "s0": (i, h)}
            v = {n: d[n][at[n]].detach().requires_grad_(train) for n in names}
            step = torch.log1p(torch.exp(v["dt"] + v["dt_bias"]))
            lam = torch.cumsum(step * v["A"], 0)
            m = torch.exp((lam[:, None] - lam[None, :]).masked_fill(off, -math.inf)) * step * (v["c"] @ v["b"].T)
            yh = m @ v["x"] + v["D"] * v["x"]
            last = (torch.exp((lam[-1] - lam).masked_fill(off[-1], -math.inf)) * step)[:, None] * v["x"]
            S = last.T @ v["b"]
            if "s0" in v:
                S = S + torch.exp(lam[-1]) * (cuts[-1] == 0) * v["s0"]
                yh = yh + (torch.exp(lam) * (cuts == 0))[:, None] * (v["c"] @ v["s0"].T)
            y[i, :, h], s_out[i, h] = yh.detach(), S.detach()
            if train:
                loss = (yh * d["dy"][i, :, h]).sum() + ((S * d["dsT"][i, h]).sum() if d["dsT"] is not None else 0.0)
                for n, g in zip(names, torch.autograd.grad(loss, [v[n] for n in names])):
                    grads[n][at[n]] += g
    r = {"y": y, "s_out": s_out}
    if train:
        r.update({"d" + n: g for n, g in grads.items()})
    return r
