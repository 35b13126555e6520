"""Python binding of libwkv7 (the C ABI in include/wkv7.h).

Argument marshalling only: every step of the WKV-7 path runs in the CUDA
kernels of ``libwkv7.so``.  PyTorch provides device memory and the current
stream.  The same entry points as the C ABI:

* ``forward(r, w, k, v, a, b, s0=None, reset=None, ...)``  -> (y, s_out, workspace)
* ``backward(r, w, k, v, a, b, dy, workspace, s0=None, reset=None, dsT=None, ...)``
  -> dict(dr, dw, dk, dv, da, db, ds0)
* ``step(r, w, k, v, a, b, state, active=None, ...)`` -> y   (state updated in place)
* ``gdn_map(q, k, g, beta, H, ...)`` -> dict(r, x, kw, a, b)   (gated-DeltaNet inputs -> WKV-7 inputs)
* ``state_compose(S, P, U, ...)`` -> S P + U (or S P^T + U) per (b, h)   (context parallelism)
* the state-space layer: ``conv_forward`` / ``conv_backward`` / ``conv_step`` (short causal convolution),
  ``ssm_forward`` / ``ssm_backward`` / ``ssm_step`` (selective scan), ``rms_forward`` / ``rms_backward`` (RMS norm with
  the residual's addition or a gate, e4m3 output)
* ``workspace_bytes(B, T, H, dtype)``
* ``device_status(clear=True)`` -> OK, ERR_TIMEOUT, ERR_BOUNDS or ERR_NONFINITE (synchronises the device)
* ``use_build("release" | "debug")``: route every call through ``libwkv7.so`` (default) or its
  bounds-checked twin ``libwkv7_debug.so`` (same ABI; ``WKV7_BUILD=debug`` in the environment
  selects it at import)

Tensors of the WKV-7 entry points are [B,T,H,N] (token inputs), [B,H,N,N] fp32 (states), [B,T] uint8
(reset), [B] uint8 (active), all on one CUDA device and contiguous.  The head size N is 64; the
token-order forward and the decode step also take N = 128 (the gated-delta-rule map's heads).  If the
library is missing, importing this module raises: there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Dict, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATHS = {"release": os.path.join(_HERE, "libwkv7.so"), "debug": os.path.join(_HERE, "libwkv7_debug.so")}
LIB_PATH = LIB_PATHS["release"]

(OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_ALIGN, ERR_WORKSPACE, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT,
 ERR_SCRATCH_LIMIT, ERR_NONFINITE, ERR_BOUNDS) = range(12)
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024   # WKV7_NOALLOC_SCRATCH_BYTES
FLAG_TEST_WAIT_TIMEOUT = 0x80000000        # WKV7_FLAG_TEST_WAIT_TIMEOUT (test hook, T <= 16)
FLAG_CHECK_FINITE = 0x1                    # WKV7_FLAG_CHECK_FINITE: scan outputs for NaN / Inf
FLAG_LOG_DECAY = 0x2                       # WKV7_FLAG_LOG_DECAY: w holds x, decay = exp(-exp(x))
FLAG_EPILOGUE_GRADS = 0x4                  # WKV7_FLAG_EPILOGUE_GRADS: dy is the epilogue's fp32 block
DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ALGO_CODE = {"auto": 0, "scan": 1, "chunked": 2, "chunked_fused": 3, "chunked_split": 4}
N_HEAD = 64
HEAD_SIZES = (64, 128)
CHUNK = 16


class Desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("algo", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Epilogue(ctypes.Structure):
    """wkv7_epilogue_t: fp32 [H,64] GroupNorm weight and bias, bonus weights, and eps."""
    _fields_ = [("ln_w", ctypes.c_void_p), ("ln_b", ctypes.c_void_p), ("r_k", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class Gdn(ctypes.Structure):
    """wkv7_gdn_t: key heads, the L2-normalisation guard and the scale taken into r."""
    _fields_ = [("Hk", ctypes.c_int64), ("eps", ctypes.c_float), ("r_scale", ctypes.c_float)]


class Conv(ctypes.Structure):
    """wkv7_conv_t: channels, taps, silu, fp32 filter [D,W] and bias [D], token stride of x."""
    _fields_ = [("D", ctypes.c_int64), ("W", ctypes.c_int32), ("silu", ctypes.c_int32), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("x_ld", ctypes.c_int64)]


class Ssm(ctypes.Structure):
    """wkv7_ssm_t: groups, fp32 [H] decay rates, skip weights and dt bias, softplus, token strides."""
    _fields_ = [("G", ctypes.c_int64), ("A", ctypes.c_void_p), ("D", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("softplus", ctypes.c_int32), ("x_ld", ctypes.c_int64), ("dt_ld", ctypes.c_int64),
                ("b_ld", ctypes.c_int64), ("c_ld", ctypes.c_int64)]


class Rms(ctypes.Structure):
    """wkv7_rms_t: channels, slices of a row, fp32 weight [D], eps, how the second input enters, 8-bit blocks."""
    _fields_ = [("D", ctypes.c_int64), ("groups", ctypes.c_int64), ("weight", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("gate", ctypes.c_int32), ("quant_block", ctypes.c_int32)]


class WKV7Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {lib().wkv7_status_string(status).decode()} (status {status})")
        self.status = status


_loaded: Dict[str, ctypes.CDLL] = {}
_active = os.environ.get("WKV7_BUILD", "release")
if _active not in LIB_PATHS:
    raise ValueError(f"WKV7_BUILD must be one of {sorted(LIB_PATHS)}, got {_active!r}")


def _load(variant: str) -> ctypes.CDLL:
    path = LIB_PATHS[variant]
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m linear_recurrent_lm_b200.build` "
                          "(or __graft_entry__.build()); the WKV-7 path has no CPU fallback")
    L = ctypes.CDLL(path)
    vp = ctypes.c_void_p
    dp = ctypes.POINTER(Desc)
    L.wkv7_version.restype = ctypes.c_int
    L.wkv7_status_string.restype = ctypes.c_char_p
    L.wkv7_status_string.argtypes = [ctypes.c_int]
    L.wkv7_workspace_bytes.restype = ctypes.c_size_t
    L.wkv7_workspace_bytes.argtypes = [dp]
    L.wkv7_forward.restype = ctypes.c_int
    L.wkv7_forward.argtypes = [dp] + [vp] * 12
    L.wkv7_backward.restype = ctypes.c_int
    L.wkv7_backward.argtypes = [dp] + [vp] * 19
    L.wkv7_step.restype = ctypes.c_int
    L.wkv7_step.argtypes = [dp] + [vp] * 10
    L.wkv7_train_step_noalloc.restype = ctypes.c_int
    L.wkv7_train_step_noalloc.argtypes = [dp] + [vp] * 20
    L.wkv7_get_device_status.restype = ctypes.c_int
    L.wkv7_get_device_status.argtypes = [ctypes.c_int]
    L.wkv7_debug_checks.restype = ctypes.c_int
    L.wkv7_debug_checks.argtypes = []
    ep = ctypes.POINTER(Epilogue)
    L.wkv7_epilogue_forward.restype = ctypes.c_int
    L.wkv7_epilogue_forward.argtypes = [dp, ep] + [vp] * 7
    L.wkv7_forward_epilogue.restype = ctypes.c_int
    L.wkv7_forward_epilogue.argtypes = [dp, ep] + [vp] * 14
    L.wkv7_epilogue_backward.restype = ctypes.c_int
    L.wkv7_epilogue_backward.argtypes = [dp, ep] + [vp] * 12
    L.wkv7_state_compose.restype = ctypes.c_int
    L.wkv7_state_compose.argtypes = [dp, vp, vp, vp, vp, ctypes.c_int, vp]
    L.wkv7_gdn_map.restype = ctypes.c_int
    L.wkv7_gdn_map.argtypes = [dp, ctypes.POINTER(Gdn)] + [vp] * 10
    for op, struct, calls in (("conv", Conv, (("forward", 6), ("backward", 11), ("step", 5))),
                              ("ssm", Ssm, (("forward", 10), ("backward", 19), ("step", 8))),
                              ("rms", Rms, (("forward", 6), ("backward", 9)))):
        sp = ctypes.POINTER(struct)
        for call, n in calls:
            f = getattr(L, f"wkv7_{op}_{call}")
            f.restype = ctypes.c_int
            f.argtypes = [dp, sp] + [vp] * n
        for size in ("scratch",) + (("workspace",) if op == "ssm" else ()):
            f = getattr(L, f"wkv7_{op}_{size}_bytes")
            f.restype = ctypes.c_size_t
            f.argtypes = [dp, sp]
    return L


def lib() -> ctypes.CDLL:
    """The library every call goes through (raises if it has not been built)."""
    if _active not in _loaded:
        _loaded[_active] = _load(_active)
    return _loaded[_active]


def use_build(variant: str) -> str:
    """Route every later call through ``variant`` ("release" or "debug"); return the previous one.

    The two builds are separate CUDA modules: each has its own device status word, which
    ``device_status`` reads from the build in use."""
    global _active
    if variant not in LIB_PATHS:
        raise ValueError(f"unknown build {variant!r}; expected one of {sorted(LIB_PATHS)}")
    prev = _active
    _active = variant
    try:
        lib()
    except ImportError:
        _active = prev
        raise
    return prev


def active_build() -> str:
    return _active


lib()   # fail at import time if the CUDA library is absent


def make_desc(B: int, T: int, H: int, dtype, algo: str = "auto", N: int = N_HEAD, flags: int = 0) -> Desc:
    code = DTYPE_CODE[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return Desc(int(B), int(T), int(H), int(N), code, ALGO_CODE[algo] if isinstance(algo, str) else int(algo), int(flags))


def workspace_bytes(B: int, T: int, H: int, dtype=torch.bfloat16, N: int = N_HEAD) -> int:
    return int(lib().wkv7_workspace_bytes(ctypes.byref(make_desc(B, T, H, dtype, N=N))))


def device_status(clear: bool = True) -> int:
    """The device status word of the current device (synchronises it): OK, ERR_TIMEOUT, ERR_BOUNDS or
    ERR_NONFINITE (in that order of precedence)."""
    return int(lib().wkv7_get_device_status(1 if clear else 0))


def _ptr(x: Optional[torch.Tensor]):
    """Device address of a contiguous CUDA tensor (the C ABI takes device pointers only)."""
    if x is None:
        return None
    if not x.is_cuda:
        raise ValueError(f"WKV-7 tensors must be on a CUDA device, got a {x.device} tensor of shape {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"WKV-7 tensors must be contiguous, got strides {x.stride()} for shape {tuple(x.shape)}")
    return ctypes.c_void_p(x.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != OK:
        raise WKV7Error(status, where)


def _token_shape(x: torch.Tensor, sizes=(N_HEAD,)):
    if x.dim() != 4 or x.shape[-1] not in sizes:
        raise ValueError(f"expected [B,T,H,N] with N in {sizes}, got {tuple(x.shape)}")
    return tuple(int(s) for s in x.shape[:3])


def _flags(flags: int, log_decay: bool) -> int:
    return int(flags) | (FLAG_LOG_DECAY if log_decay else 0)


def forward(r, w, k, v, a, b, s0=None, reset=None, *, y=None, s_out=None, workspace=None,
            need_workspace: bool = True, want_state: bool = True, algo: str = "auto", stream=None, flags: int = 0,
            log_decay: bool = False):
    """WKV-7 forward over [B,T,H,N] inputs (N = 64, or 128 with the token-order scan).  Returns (y,
    s_out, workspace).  With ``log_decay`` the ``w`` tensor holds x and the decay is exp(-exp(x))."""
    B, T, H = _token_shape(r, HEAD_SIZES)
    N = int(r.shape[-1])
    dev = r.device
    if y is None:
        y = torch.empty_like(r)
    if s_out is None and want_state:
        s_out = torch.empty((B, H, N, N), device=dev, dtype=torch.float32)
    if workspace is None and need_workspace:
        workspace = torch.empty(max(workspace_bytes(B, T, H, r.dtype, N), 16), device=dev, dtype=torch.uint8)
    d = make_desc(B, T, H, r.dtype, algo, N=N, flags=_flags(flags, log_decay))
    st = lib().wkv7_forward(ctypes.byref(d), *(_ptr(x) for x in (r, w, k, v, a, b, s0, reset, y, s_out, workspace)),
                            _stream(stream))
    _check(st, "wkv7_forward")
    return y, s_out, workspace


def backward(r, w, k, v, a, b, dy, workspace, s0=None, reset=None, dsT=None, *, grads=None,
             want_ds0: bool = True, algo: str = "auto", stream=None, flags: int = 0,
             log_decay: bool = False) -> Dict[str, torch.Tensor]:
    """WKV-7 backward from the checkpoints written by ``forward``.  With ``log_decay`` (as in the
    forward) ``w`` holds x and the "dw" entry receives dL/dx.  ``dy`` may be the fp32 block
    [4,B,T,H,64] that ``epilogue_backward`` returns as "eg" (dy, then the epilogue's parts of dr, dk,
    dv, which are added in)."""
    if dy.dim() == 5:
        if dy.dtype != torch.float32 or tuple(dy.shape) != (4,) + tuple(r.shape):
            raise ValueError(f"the epilogue's gradient block must be fp32 [4,B,T,H,64], got {tuple(dy.shape)}")
        flags = int(flags) | FLAG_EPILOGUE_GRADS
    B, T, H = _token_shape(r)
    g = dict(grads) if grads is not None else {}
    for n in ("dr", "dw", "dk", "dv", "da", "db"):
        if g.get(n) is None:
            g[n] = torch.empty_like(r)
    if g.get("ds0") is None and want_ds0:
        g["ds0"] = torch.empty((B, H, N_HEAD, N_HEAD), device=r.device, dtype=torch.float32)
    d = make_desc(B, T, H, r.dtype, algo, flags=_flags(flags, log_decay))
    st = lib().wkv7_backward(ctypes.byref(d), *(_ptr(x) for x in (r, w, k, v, a, b, s0, reset, dy, dsT, workspace)),
                             *(_ptr(g[n]) for n in ("dr", "dw", "dk", "dv", "da", "db")), _ptr(g.get("ds0")),
                             _stream(stream))
    _check(st, "wkv7_backward")
    return g


def step(r, w, k, v, a, b, state, active=None, *, y=None, stream=None, flags: int = 0, log_decay: bool = False):
    """One decode token on ``state`` [B,H,N,N] (in place).  Inputs [B,H,N], N = 64 or 128.  Returns y."""
    if r.dim() != 3 or r.shape[-1] not in HEAD_SIZES:
        raise ValueError(f"expected [B,H,N] with N in {HEAD_SIZES}, got {tuple(r.shape)}")
    B, H = int(r.shape[0]), int(r.shape[1])
    if y is None:
        y = torch.empty_like(r)
    d = make_desc(B, 1, H, r.dtype, N=int(r.shape[-1]), flags=_flags(flags, log_decay))
    st = lib().wkv7_step(ctypes.byref(d), *(_ptr(x) for x in (r, w, k, v, a, b, state, active, y)), _stream(stream))
    _check(st, "wkv7_step")
    return y


def train_step_noalloc(r, w, k, v, a, b, dy, s0=None, reset=None, dsT=None, *, y=None, s_out=None, grads=None,
                       want_ds0: bool = True, algo: str = "auto", stream=None, log_decay: bool = False):
    """Forward + backward with the library's fixed scratch instead of a workspace (nothing is
    allocated by the library; outputs not given are allocated here by torch).  For callers that
    cannot allocate device memory themselves: pass every output.  Returns (y, s_out, grads)."""
    B, T, H = _token_shape(r)
    if y is None:
        y = torch.empty_like(r)
    if s_out is None:
        s_out = torch.empty((B, H, N_HEAD, N_HEAD), device=r.device, dtype=torch.float32)
    g = dict(grads) if grads is not None else {}
    for n in ("dr", "dw", "dk", "dv", "da", "db"):
        if g.get(n) is None:
            g[n] = torch.empty_like(r)
    if g.get("ds0") is None and want_ds0:
        g["ds0"] = torch.empty((B, H, N_HEAD, N_HEAD), device=r.device, dtype=torch.float32)
    flags = FLAG_EPILOGUE_GRADS if dy.dim() == 5 else 0   # the epilogue's fp32 block (see backward)
    d = make_desc(B, T, H, r.dtype, algo, flags=_flags(flags, log_decay))
    st = lib().wkv7_train_step_noalloc(ctypes.byref(d), *(_ptr(x) for x in (r, w, k, v, a, b, s0, reset, y, s_out, dy, dsT)),
                                       *(_ptr(g[n]) for n in ("dr", "dw", "dk", "dv", "da", "db")), _ptr(g.get("ds0")),
                                       _stream(stream))
    _check(st, "wkv7_train_step_noalloc")
    return y, s_out, g


def _epi(ln_w, ln_b, r_k, eps) -> Epilogue:
    for t in (ln_w, ln_b, r_k):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError("epilogue parameters must be contiguous fp32 CUDA tensors [H,64]")
    return Epilogue(ln_w.data_ptr(), ln_b.data_ptr(), r_k.data_ptr(), float(eps))


def epilogue_forward(y, r, k, v, g, ln_w, ln_b, r_k, eps: float, *, out=None, stream=None, flags: int = 0):
    """The WKV epilogue: out = (GroupNorm_h(y) ln_w + ln_b + (sum r k r_k) v) g, per (b,t,h).  Token
    tensors [B,T,H,64]; ln_w, ln_b, r_k fp32 [H,64]."""
    B, T, H = _token_shape(y)
    if out is None:
        out = torch.empty_like(y)
    d = make_desc(B, T, H, y.dtype, flags=flags)
    ep = _epi(ln_w, ln_b, r_k, eps)
    st = lib().wkv7_epilogue_forward(ctypes.byref(d), ctypes.byref(ep), *(_ptr(x) for x in (y, r, k, v, g, out)),
                                     _stream(stream))
    _check(st, "wkv7_epilogue_forward")
    return out


def epilogue_backward(y, r, k, v, g, dout, ln_w, ln_b, r_k, eps: float, *, grads=None, want_params: bool = True,
                      stream=None, flags: int = 0) -> Dict[str, torch.Tensor]:
    """Reverse mode of ``epilogue_forward``: dict of "eg" (fp32 [4,B,T,H,64]: dy, then the bonus parts
    of dr, dk, dv -- pass it to ``backward`` as its dy), "dg" [B,T,H,64], and (zeroed here, then summed
    over b and t) dln_w, dln_b, dr_k [H,64]."""
    B, T, H = _token_shape(y)
    g_ = dict(grads) if grads is not None else {}
    if g_.get("eg") is None:
        g_["eg"] = torch.empty((4,) + tuple(y.shape), device=y.device, dtype=torch.float32)
    if g_.get("dg") is None:
        g_["dg"] = torch.empty_like(y)
    if want_params:
        for n in ("dln_w", "dln_b", "dr_k"):
            g_[n] = torch.zeros((H, N_HEAD), device=y.device, dtype=torch.float32)
    d = make_desc(B, T, H, y.dtype, flags=flags)
    ep = _epi(ln_w, ln_b, r_k, eps)
    st = lib().wkv7_epilogue_backward(ctypes.byref(d), ctypes.byref(ep), *(_ptr(x) for x in (y, r, k, v, g, dout)),
                                      _ptr(g_["eg"]), _ptr(g_["dg"]),
                                      *(_ptr(g_.get(n)) for n in ("dln_w", "dln_b", "dr_k")), _stream(stream))
    _check(st, "wkv7_epilogue_backward")
    return g_


def forward_epilogue(r, w, k, v, a, b, g, ln_w, ln_b, r_k, eps: float, s0=None, reset=None, *, out=None, y=None,
                     want_y: bool = True, s_out=None, workspace=None, need_workspace: bool = True,
                     want_state: bool = True, algo: str = "auto", stream=None, flags: int = 0,
                     log_decay: bool = False):
    """The forward with the WKV epilogue: out = epilogue(y) (fused into the recurrence's kernel in the
    fused chunked form).  Returns (out, y or None, s_out, workspace)."""
    B, T, H = _token_shape(r)
    dev = r.device
    if out is None:
        out = torch.empty_like(r)
    if y is None and want_y:
        y = torch.empty_like(r)
    if s_out is None and want_state:
        s_out = torch.empty((B, H, N_HEAD, N_HEAD), device=dev, dtype=torch.float32)
    if workspace is None and need_workspace:
        workspace = torch.empty(max(workspace_bytes(B, T, H, r.dtype), 16), device=dev, dtype=torch.uint8)
    d = make_desc(B, T, H, r.dtype, algo, flags=_flags(flags, log_decay))
    ep = _epi(ln_w, ln_b, r_k, eps)
    st = lib().wkv7_forward_epilogue(ctypes.byref(d), ctypes.byref(ep),
                                     *(_ptr(x) for x in (r, w, k, v, a, b, s0, reset, g, y, out, s_out, workspace)),
                                     _stream(stream))
    _check(st, "wkv7_forward_epilogue")
    return out, y, s_out, workspace


def gdn_map(q, k, g, beta, H: int, eps: float = 1e-6, r_scale: Optional[float] = None, *, out=None, stream=None,
            flags: int = 0) -> Dict[str, torch.Tensor]:
    """The gated-DeltaNet front end (wkv7_gdn_map): q, k [B,T,Hk,N] and fp32 g, beta [B,T,H] ->
    dict of r, x, kw, a, b [B,T,H,N] for ``forward`` / ``step`` with ``log_decay=True`` and GDN's
    own v.  ``r_scale`` defaults to 1/sqrt(N)."""
    B, T, Hk = _token_shape(q, HEAD_SIZES)
    N = int(q.shape[-1])
    if tuple(k.shape) != tuple(q.shape) or k.dtype != q.dtype:
        raise ValueError(f"q and k must match, got {tuple(q.shape)} {q.dtype} and {tuple(k.shape)} {k.dtype}")
    for n, t in (("g", g), ("beta", beta)):
        if t.dtype != torch.float32 or tuple(t.shape) != (B, T, H):
            raise ValueError(f"{n} must be fp32 [B,T,H] = {(B, T, H)}, got {tuple(t.shape)} {t.dtype}")
    o = dict(out) if out is not None else {}
    for n in ("r", "x", "kw", "a", "b"):
        if o.get(n) is None:
            o[n] = torch.empty((B, T, H, N), device=q.device, dtype=q.dtype)
    d = make_desc(B, T, H, q.dtype, N=N, flags=flags)
    gd = Gdn(int(Hk), float(eps), float(N ** -0.5 if r_scale is None else r_scale))
    st = lib().wkv7_gdn_map(ctypes.byref(d), ctypes.byref(gd), *(_ptr(x) for x in (q, k, g, beta)),
                            *(_ptr(o[n]) for n in ("r", "x", "kw", "a", "b")), _stream(stream))
    _check(st, "wkv7_gdn_map")
    return o


def state_compose(S, P, U, *, out=None, transpose: bool = False, stream=None, flags: int = 0) -> torch.Tensor:
    """wkv7_state_compose: out = S P + U (S P^T + U with ``transpose``) per (b, h) unit, all fp32
    [B,H,N,N]; S or U may be None (zero).  ``out`` may be U itself."""
    ref = next(t for t in (S, P, U, out) if t is not None)
    if ref.dim() != 4 or ref.shape[-1] != ref.shape[-2] or ref.shape[-1] not in HEAD_SIZES:
        raise ValueError(f"expected fp32 states [B,H,N,N] with N in {HEAD_SIZES}, got {tuple(ref.shape)}")
    for t in (S, P, U, out):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != tuple(ref.shape)):
            raise ValueError(f"states must all be fp32 {tuple(ref.shape)}, got {tuple(t.shape)} {t.dtype}")
    B, H, N = int(ref.shape[0]), int(ref.shape[1]), int(ref.shape[-1])
    if out is None:
        out = torch.empty_like(ref)
    d = make_desc(B, 1, H, torch.float32, N=N, flags=flags)
    st = lib().wkv7_state_compose(ctypes.byref(d), _ptr(S), _ptr(P), _ptr(U), _ptr(out), 1 if transpose else 0,
                                  _stream(stream))
    _check(st, "wkv7_state_compose")
    return out


# ------------------------------------------------------------------ state-space layer
# Calls of single tokens last a few microseconds on the GPU, so the checks here are kept short.
def _on_device(f):
    """Run ``f`` on its first tensor's device and on ``stream`` (default: that device's current stream); what it
    allocates belongs to that stream."""
    @functools.wraps(f)
    def call(x, *args, stream=None, **kw):
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise ValueError(f"{f.__name__}: tensors must be on a CUDA device")
        if stream is not None:
            if stream.device != x.device:
                raise ValueError(f"{f.__name__}: the stream is on {stream.device}, the tensors on {x.device}")
            with torch.cuda.stream(stream):
                return f(x, *args, **kw)
        if x.get_device() != torch._C._cuda_getDevice():
            with torch.cuda.device(x.device):
                return f(x, *args, **kw)
        return f(x, *args, **kw)
    return call


def _dense(t: Optional[torch.Tensor], name: str, shape, dtype, like: torch.Tensor):
    """Address of a contiguous tensor of the given shape and dtype on ``like``'s device (None stays None)."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, got strides {t.stride()} for shape {tuple(t.shape)}")
    return t.data_ptr()


def _rows(t: torch.Tensor, name: str, shape, lead: int, like: torch.Tensor):
    """(address, token stride) of token rows [B,T,..] (``lead`` = 2) or [B,..] (``lead`` = 1) whose rows are dense;
    the rows themselves may be slices of wider ones.  The stride is 0 where it is the row's size."""
    if t.shape != shape or t.dtype != like.dtype:
        raise ValueError(f"{name} must be {like.dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")
    if t.is_contiguous():
        return t.data_ptr(), 0
    st, width = t.stride(), 1
    ok = True
    for i in range(t.dim() - 1, lead - 1, -1):
        ok = ok and (shape[i] == 1 or st[i] == width)
        width *= shape[i]
    ld, n = None, 1
    for i in range(lead - 1, -1, -1):
        if shape[i] != 1:
            ld = st[i] // n if ld is None else ld
            ok = ok and st[i] == ld * n
        n *= shape[i]
    if not ok or (ld is not None and ld < width):
        raise ValueError(f"{name}: only the distance between tokens may differ from a dense tensor's, got strides {st} for "
                         f"shape {tuple(shape)}")
    return t.data_ptr(), ld or 0


def _mask(t: Optional[torch.Tensor], name: str, shape, like: torch.Tensor):
    if t is None:
        return None
    return _dense(t.view(torch.uint8) if t.dtype == torch.bool else t, name, shape, torch.uint8, like)


def _out(t: Optional[torch.Tensor], name: str, shape, dtype, like: torch.Tensor):
    if t is None:
        if shape == like.shape:   # half the time of new_empty
            return torch.empty_like(like, dtype=dtype, memory_format=torch.contiguous_format)
        return like.new_empty(shape, dtype=dtype)
    _dense(t, name, shape, dtype, like)
    return t


def _wanted(g: Dict[str, torch.Tensor], name: str, want: bool, shape, dtype, like: torch.Tensor):
    """An optional gradient in ``g``: made where it is wanted, and what the caller put there is written, so it is checked."""
    if want or g.get(name) is not None:
        g[name] = _out(g.get(name), name, shape, dtype, like)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _scratch(n: int, like: torch.Tensor):
    return like.new_empty(max(n, 16), dtype=torch.uint8)


def _now(like: torch.Tensor):
    """The current stream of ``like``'s device, which is the current device."""
    return torch._C._cuda_getCurrentRawStream(like.get_device())


def _code(dtype) -> int:
    code = DTYPE_CODE.get(dtype)
    if code is None:
        raise ValueError(f"expected one of {list(DTYPE_CODE)}, got {dtype}")
    return code


def _conv_args(x, weight, bias, silu, lead, flags):
    shape = x.shape
    if len(shape) != lead + 1 or weight.dim() != 2:
        raise ValueError(f"expected x [B,{'T,' if lead == 2 else ''}D] and weight [D,W], got {tuple(shape)} and {tuple(weight.shape)}")
    B, T, D, W = shape[0], shape[1] if lead == 2 else 1, shape[-1], weight.shape[1]
    px, ld = _rows(x, "x", shape, lead, x)
    cv = Conv(D, W, 1 if silu else 0, _dense(weight, "weight", (D, W), torch.float32, x), _dense(bias, "bias", (D,), torch.float32, x), ld)
    return Desc(B, T, 0, N_HEAD, _code(x.dtype), 0, flags), cv, px, (B, T, D, W)


@_on_device
def conv_forward(x, weight, bias=None, s0=None, reset=None, *, silu: bool = True, y=None, s_out=None,
                 want_state: bool = True, flags: int = 0):
    """Short causal convolution per channel: u_t = bias + sum_j weight[:, W-1-j] x_{t-j}, y = silu(u) (or u).

    x [B,T,D] (token rows may be slices of wider ones), weight fp32 [D,W] with W = 2..4, bias fp32 [D]; s0 [B,W-1,D]
    holds the inputs before the row (oldest first), reset [B,T] cuts the taps before a token.  Returns (y, s_out)."""
    d, cv, px, (B, T, D, W) = _conv_args(x, weight, bias, silu, 2, flags)
    y = _out(y, "y", (B, T, D), x.dtype, x)
    if s_out is not None or want_state:
        s_out = _out(s_out, "s_out", (B, W - 1, D), x.dtype, x)
    st = lib().wkv7_conv_forward(d, cv, px, _dense(s0, "s0", (B, W - 1, D), x.dtype, x), _mask(reset, "reset", (B, T), x),
                                 y.data_ptr(), _addr(s_out), _now(x))
    _check(st, "wkv7_conv_forward")
    return y, s_out


@_on_device
def conv_backward(x, weight, dy, bias=None, s0=None, reset=None, dsT=None, *, silu: bool = True, grads=None,
                  want_params: bool = True, want_ds0: bool = True, flags: int = 0) -> Dict[str, torch.Tensor]:
    """Reverse mode of ``conv_forward`` from dy [B,T,D] and dsT (gradient of s_out, or None): dict of dx, and, where
    wanted, fp32 dweight [D,W], dbias [D] and ds0 [B,W-1,D]."""
    d, cv, px, (B, T, D, W) = _conv_args(x, weight, bias, silu, 2, flags)
    g = dict(grads) if grads is not None else {}
    g["dx"] = _out(g.get("dx"), "dx", (B, T, D), x.dtype, x)
    _wanted(g, "dweight", want_params, (D, W), torch.float32, x)
    _wanted(g, "dbias", want_params, (D,), torch.float32, x)
    _wanted(g, "ds0", want_ds0, (B, W - 1, D), x.dtype, x)
    params = g.get("dweight") is not None or g.get("dbias") is not None
    tmp = _scratch(lib().wkv7_conv_scratch_bytes(d, cv), x) if params else None
    st = lib().wkv7_conv_backward(d, cv, px, _dense(s0, "s0", (B, W - 1, D), x.dtype, x), _mask(reset, "reset", (B, T), x),
                                  _dense(dy, "dy", (B, T, D), x.dtype, x), _dense(dsT, "dsT", (B, W - 1, D), x.dtype, x),
                                  g["dx"].data_ptr(), _addr(g.get("dweight")), _addr(g.get("dbias")), _addr(g.get("ds0")),
                                  _addr(tmp), _now(x))
    _check(st, "wkv7_conv_backward")
    return g


@_on_device
def conv_step(x, weight, state, bias=None, active=None, *, silu: bool = True, y=None, flags: int = 0):
    """One decode token of the convolution: x [B,D], state [B,W-1,D] shifted in place.  Returns y [B,D]."""
    d, cv, px, (B, _, D, W) = _conv_args(x, weight, bias, silu, 1, flags)
    y = _out(y, "y", (B, D), x.dtype, x)
    st = lib().wkv7_conv_step(d, cv, px, _dense(state, "state", (B, W - 1, D), x.dtype, x), _mask(active, "active", (B,), x),
                              y.data_ptr(), _now(x))
    _check(st, "wkv7_conv_step")
    return y


def _ssm_args(x, dt, A, b, c, D, dt_bias, softplus, lead, algo, flags):
    if x.dim() != lead + 2 or b.dim() != lead + 2 or x.shape[-1] != N_HEAD:
        raise ValueError(f"expected x [B,{'T,' if lead == 2 else ''}H,{N_HEAD}] and b, c [B,{'T,' if lead == 2 else ''}G,N], got "
                         f"{tuple(x.shape)} and {tuple(b.shape)}")
    lead_shape = tuple(x.shape[:lead])
    B, T, H = lead_shape[0], lead_shape[1] if lead == 2 else 1, x.shape[lead]
    G, N = b.shape[lead], b.shape[-1]
    px, x_ld = _rows(x, "x", lead_shape + (H, N_HEAD), lead, x)
    pt, t_ld = _rows(dt, "dt", lead_shape + (H,), lead, x)
    pb, b_ld = _rows(b, "b", lead_shape + (G, N), lead, x)
    pc, c_ld = _rows(c, "c", lead_shape + (G, N), lead, x)
    sp = Ssm(G, *(_dense(t, n, (H,), torch.float32, x) for t, n in ((A, "A"), (D, "D"), (dt_bias, "dt_bias"))),
             1 if softplus else 0, x_ld, t_ld, b_ld, c_ld)
    return Desc(B, T, H, N, _code(x.dtype), ALGO_CODE[algo], flags), sp, (px, pt, pb, pc), (B, T, H, G, N)


@_on_device
def ssm_forward(x, dt, A, b, c, D=None, dt_bias=None, s0=None, reset=None, *, softplus: bool = True, y=None, s_out=None,
                workspace=None, need_workspace: bool = True, want_state: bool = True, algo: str = "auto", flags: int = 0):
    """Selective state space scan: d = softplus(dt + dt_bias), S_t = exp(d A) S_{t-1} + d x_t b_t^T, y_t = S_t c_t + D x_t.

    x [B,T,H,64], dt [B,T,H], b, c [B,T,G,N] (H / G consecutive heads share a group; N = 64 or 128; token rows may be
    slices of wider ones), A, D, dt_bias fp32 [H], s0 fp32 [B,H,64,N], reset [B,T].  algo "auto" is "chunked" (tensor
    cores) for bf16 rows of more than 16 tokens and "scan" (token order) else; under "chunked" a NaN or infinity in a token may reach every output of
    its 128-token chunk, so fill padding with finite values.  Returns (y, s_out, workspace)."""
    d, sp, ptrs, (B, T, H, G, N) = _ssm_args(x, dt, A, b, c, D, dt_bias, softplus, 2, algo, flags)
    y = _out(y, "y", (B, T, H, N_HEAD), x.dtype, x)
    if s_out is not None or want_state:
        s_out = _out(s_out, "s_out", (B, H, N_HEAD, N), torch.float32, x)
    need = int(lib().wkv7_ssm_workspace_bytes(d, sp)) if workspace is not None or need_workspace else 0
    if workspace is None and need_workspace:
        workspace = _scratch(need, x)
    elif workspace is not None and workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"the workspace must hold {need} bytes")
    st = lib().wkv7_ssm_forward(d, sp, *ptrs, _dense(s0, "s0", (B, H, N_HEAD, N), torch.float32, x),
                                _mask(reset, "reset", (B, T), x), y.data_ptr(), _addr(s_out),
                                None if workspace is None else _dense(workspace, "workspace", workspace.shape, workspace.dtype, x),
                                _now(x))
    _check(st, "wkv7_ssm_forward")
    return y, s_out, workspace


@_on_device
def ssm_backward(x, dt, A, b, c, dy, workspace, D=None, dt_bias=None, s0=None, reset=None, dsT=None, *,
                 softplus: bool = True, grads=None, want_ds0: bool = True, algo: str = "auto",
                 flags: int = 0) -> Dict[str, torch.Tensor]:
    """Reverse mode of ``ssm_forward`` from its workspace, dy [B,T,H,64] and dsT (gradient of s_out, or None): dict of
    dx, ddt, db, dc, fp32 dA, dD, ddt_bias (the last two where D and dt_bias are given) and, where wanted, ds0.  Token order
    ("scan", which "auto" is for fp32 and fp16) reads no workspace: None will do."""
    d, sp, ptrs, (B, T, H, G, N) = _ssm_args(x, dt, A, b, c, D, dt_bias, softplus, 2, algo, flags)
    g = dict(grads) if grads is not None else {}
    shapes = {"dx": (B, T, H, N_HEAD), "ddt": (B, T, H), "db": (B, T, G, N), "dc": (B, T, G, N)}
    for n, shape in shapes.items():
        g[n] = _out(g.get(n), n, shape, x.dtype, x)
    for n, on in (("dA", True), ("dD", D is not None), ("ddt_bias", dt_bias is not None)):
        _wanted(g, n, on, (H,), torch.float32, x)
    _wanted(g, "ds0", want_ds0, (B, H, N_HEAD, N), torch.float32, x)
    need = 4 * B * H * (-(-T // 128) + 1) * N_HEAD * N if T else 0   # the states alone, whichever form wrote them
    reads = x.dtype == torch.bfloat16 and algo != "scan"   # token order walks forward again
    if reads if workspace is None else workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"the backward needs the forward's workspace of at least {need} bytes")
    tmp = _scratch(lib().wkv7_ssm_scratch_bytes(d, sp), x)
    st = lib().wkv7_ssm_backward(d, sp, *ptrs, _dense(s0, "s0", (B, H, N_HEAD, N), torch.float32, x),
                                 _mask(reset, "reset", (B, T), x), _dense(dy, "dy", (B, T, H, N_HEAD), x.dtype, x),
                                 _dense(dsT, "dsT", (B, H, N_HEAD, N), torch.float32, x),
                                 None if workspace is None else _dense(workspace, "workspace", workspace.shape, workspace.dtype, x),
                                 *(_addr(g.get(n)) for n in ("dx", "ddt", "db", "dc", "dA", "dD", "ddt_bias", "ds0")),
                                 tmp.data_ptr(), _now(x))
    _check(st, "wkv7_ssm_backward")
    return g


@_on_device
def ssm_step(x, dt, A, b, c, state, D=None, dt_bias=None, active=None, *, softplus: bool = True, y=None, flags: int = 0):
    """One decode token of the scan: x [B,H,64], dt [B,H], b, c [B,G,N], state fp32 [B,H,64,N] in place.  Returns y."""
    d, sp, ptrs, (B, _, H, G, N) = _ssm_args(x, dt, A, b, c, D, dt_bias, softplus, 1, "auto", flags)
    y = _out(y, "y", (B, H, N_HEAD), x.dtype, x)
    st = lib().wkv7_ssm_step(d, sp, *ptrs, _dense(state, "state", (B, H, N_HEAD, N), torch.float32, x),
                             _mask(active, "active", (B,), x), y.data_ptr(), _now(x))
    _check(st, "wkv7_ssm_step")
    return y


def _rms_args(x, weight, eps, groups, gate, quant_block, flags):
    if x.dim() < 1:
        raise ValueError("x must have a channel dimension")
    D = x.shape[-1]
    rows = x.numel() // D if D > 0 else 0
    rn = Rms(D, groups, _dense(weight, "weight", (D,), torch.float32, x), eps, 1 if gate else 0, quant_block)
    return Desc(rows, 1, 0, N_HEAD, _code(x.dtype), 0, flags), rn, rows


@_on_device
def rms_forward(x, weight, eps: float, *, residual=None, gate=None, groups: int = 1, quant_block: int = 0, h=None, out=None,
                scale=None, flags: int = 0) -> Dict[str, torch.Tensor]:
    """RMS norm over ``groups`` equal slices of the last dimension: out = h / sqrt(mean(h^2) + eps) * weight with
    h = x, x + residual (stored, and returned as "h") or x * silu(gate).

    quant_block = 0: dict with "out" in x's dtype.  128: e4m3 "q" and one fp32 "scale" per 128 channels; -1: one scale
    per slice (value = q * scale)."""
    if residual is not None and gate is not None:
        raise ValueError("rms_forward takes a residual or a gate, not both")
    other = residual if residual is not None else gate
    d, rn, _ = _rms_args(x, weight, eps, groups, gate is not None, quant_block, flags)
    D = x.shape[-1]
    px = _dense(x, "x", x.shape, x.dtype, x)
    r = {}
    if residual is not None:
        r["h"] = _out(h, "h", x.shape, x.dtype, x)
    elif h is not None:
        raise ValueError("h is an output of the residual's addition only")
    if quant_block:
        r["q"] = _out(out, "out", x.shape, torch.float8_e4m3fn, x)
        r["scale"] = _out(scale, "scale", tuple(x.shape[:-1]) + ((D // 128) if quant_block > 0 else int(groups),), torch.float32, x)
    else:
        r["out"] = _out(out, "out", x.shape, x.dtype, x)
    st = lib().wkv7_rms_forward(d, rn, px, _dense(other, "residual or gate", x.shape, x.dtype, x), _addr(r.get("h")),
                                (r["q"] if quant_block else r["out"]).data_ptr(), _addr(r.get("scale")), _now(x))
    _check(st, "wkv7_rms_forward")
    return r


@_on_device
def rms_backward(x, weight, dout, eps: float, *, gate=None, dh=None, groups: int = 1, grads=None, want_params: bool = True,
                 flags: int = 0) -> Dict[str, torch.Tensor]:
    """Reverse mode of ``rms_forward`` (without 8-bit output): dict of dx, fp32 dweight and, with a gate, dgate.  After a
    residual's addition x is the stored sum "h"; dx is then the gradient of both summands, and ``dh``, the gradient
    that reaches the sum directly, is added in."""
    d, rn, _ = _rms_args(x, weight, eps, groups, gate is not None, 0, flags)
    g = dict(grads) if grads is not None else {}
    px = _dense(x, "x", x.shape, x.dtype, x)
    g["dx"] = _out(g.get("dx"), "dx", x.shape, x.dtype, x)
    _wanted(g, "dgate", gate is not None, x.shape, x.dtype, x)
    _wanted(g, "dweight", want_params, (x.shape[-1],), torch.float32, x)
    tmp = _scratch(lib().wkv7_rms_scratch_bytes(d, rn), x) if g.get("dweight") is not None else None
    st = lib().wkv7_rms_backward(d, rn, px, _dense(gate, "gate", x.shape, x.dtype, x),
                                 _dense(dout, "dout", x.shape, x.dtype, x), _dense(dh, "dh", x.shape, x.dtype, x),
                                 g["dx"].data_ptr(), _addr(g.get("dgate")), _addr(g.get("dweight")), _addr(tmp), _now(x))
    _check(st, "wkv7_rms_backward")
    return g
