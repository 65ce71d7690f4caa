"""ctypes binding of libboost_block.so (argument marshalling only).

Every function here checks the torch tensors it is given (dtype, device,
contiguity, shape), passes raw pointers and sizes to the C ABI declared in
``include/boost_block.h`` and ``include/boost_ops.h`` and raises ``BoostError`` on a non-OK status. No
arithmetic of the block happens in Python; there is no CPU fallback: if the
library is missing, ``lib()`` raises.
"""

from __future__ import annotations

import array
import ctypes
import functools
import operator
import os

import torch

from . import build as _build

_LIB = None

BOOST_OK = 0
STATUS_NAMES = {
    0: "BOOST_OK", 1: "BOOST_ERR_INVALID_ARG", 2: "BOOST_ERR_UNSUPPORTED_SHAPE",
    3: "BOOST_ERR_ALIGNMENT", 4: "BOOST_ERR_WORKSPACE", 5: "BOOST_ERR_CUDA",
    6: "BOOST_ERR_TIMEOUT", 7: "BOOST_ERR_DEVICE_CHECK",
}
ACT = {"identity": 0, "silu": 1}

EXPORTS = (
    "boost_block_workspace_bytes", "boost_block_ws_init", "boost_block_fwd", "boost_block_bwd",
    "boost_rmsnorm_stats", "boost_block_layout", "boost_block_check", "boost_status_string",
    "boost_swiglu_fwd", "boost_swiglu_bwd", "boost_add", "boost_debug_wait_timeout",
    "boost_block_ws_layout", "boost_profile_enable", "boost_profile_kernel_count",
    "boost_profile_read", "boost_rmsnorm_rstd_noalloc", "boost_block_bwd_swiglu",
    "boost_profile_read_kernels", "boost_block_fwd_swiglu", "boost_block_fwd_btp",
    "boost_block_up", "boost_debug_count_writes", "boost_debug_count_log",
    "boost_profile_only", "boost_block_fwd_residual", "boost_block_bwd_residual",
    "boost_rope", "boost_dropout", "boost_fp8_scale_bytes", "boost_fp8_quantize",
    "boost_fp8_matmul_workspace_bytes", "boost_fp8_matmul",
    "boost_attention_workspace_bytes", "boost_attention", "boost_attention_bwd",
    "boost_norm_quantize", "boost_grad_clip_workspace_bytes", "boost_grad_clip",
)


class BoostError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        name = STATUS_NAMES.get(status, str(status))
        msg = lib().boost_status_string(status).decode() if _LIB is not None else name
        super().__init__(f"{what}: {name} ({msg})")


class Desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d", ctypes.c_int64), ("r", ctypes.c_int64),
                ("k", ctypes.c_int64), ("n", ctypes.c_int64), ("S", ctypes.c_int32),
                ("eps", ctypes.c_float), ("act", ctypes.c_int32), ("has_norm", ctypes.c_int32)]


ROPE_MAX_DIM = 512
FP8_FORMATS = {"e4m3": (0, torch.float8_e4m3fn), "e5m2": (1, torch.float8_e5m2)}
FP8_CODE = {dtype: code for code, dtype in FP8_FORMATS.values()}


class RopeDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64)] + \
        [(f, ctypes.c_int32) for f in ("hq", "hk", "dim", "rot", "axes", "interleaved", "inverse",
                                       "pos64")] + \
        [(f, ctypes.c_int64) for f in ("q_ts", "q_hs", "k_ts", "k_hs", "qo_ts", "qo_hs", "ko_ts",
                                       "ko_hs", "pos_at", "pos_as")] + \
        [("axis", ctypes.c_uint8 * (ROPE_MAX_DIM // 2))]


class Fp8QuantDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("G", "rows", "cols", "ldx", "gstride")] + \
        [("fmt", ctypes.c_int32), ("block_rows", ctypes.c_int32)]


class Fp8MatmulDesc(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int64) for f in ("G", "M", "N", "K", "a_pitch", "b_pitch")] + \
        [(f, ctypes.c_int32) for f in ("a_fmt", "b_fmt", "act")]


ATTENTION_MAX_DIM = 128


class AttentionDesc(ctypes.Structure):
    _fields_ = [("Tq", ctypes.c_int64), ("Tk", ctypes.c_int64)] + \
        [(f, ctypes.c_int32) for f in ("hq", "hk", "dim", "sequences", "causal")] + \
        [("scale", ctypes.c_float)] + \
        [(f"{x}_{y}", ctypes.c_int64) for x in ("q", "k", "v", "o", "do", "dq", "dk", "dv")
         for y in ("ts", "hs")]


class Grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("wide", ctypes.c_int32)]


def lib_path() -> str:
    return _build.LIB


def lib():
    """Load the library once; raise if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m rank_bottleneck_online_gb300.build`")
    L = ctypes.CDLL(path)
    vp, sz, i64, u32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int64, ctypes.c_uint32
    dp = ctypes.POINTER(Desc)
    L.boost_block_workspace_bytes.argtypes = [dp]
    L.boost_block_workspace_bytes.restype = sz
    L.boost_block_ws_init.argtypes = [vp, sz, vp]
    L.boost_block_fwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.boost_block_fwd_swiglu.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.boost_block_fwd_btp.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.boost_block_up.argtypes = [dp, vp, vp, vp, vp, vp, sz, vp]
    L.boost_debug_count_writes.argtypes = [vp, i64]
    L.boost_debug_count_log.argtypes = [ctypes.POINTER(i64), i64]
    L.boost_debug_count_log.restype = i64
    L.boost_block_bwd.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.boost_block_fwd_residual.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.boost_block_bwd_residual.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                           sz, vp]
    L.boost_rmsnorm_stats.argtypes = [dp, vp, vp, vp, vp]
    L.boost_block_layout.argtypes = [dp, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                     ctypes.POINTER(i64)]
    L.boost_block_check.argtypes = [vp, vp]
    L.boost_rope.argtypes = [ctypes.POINTER(RopeDesc), vp, vp, vp, vp, vp, vp, vp]
    L.boost_dropout.argtypes = [i64, vp, vp, vp, ctypes.c_double, ctypes.c_uint64,
                                ctypes.c_uint64, vp, vp]
    L.boost_fp8_scale_bytes.argtypes = [i64, i64]
    L.boost_fp8_scale_bytes.restype = sz
    L.boost_fp8_quantize.argtypes = [ctypes.POINTER(Fp8QuantDesc)] + [vp] * 7
    L.boost_fp8_matmul_workspace_bytes.argtypes = [ctypes.POINTER(Fp8MatmulDesc)]
    L.boost_fp8_matmul_workspace_bytes.restype = sz
    L.boost_fp8_matmul.argtypes = [ctypes.POINTER(Fp8MatmulDesc)] + [vp] * 7 + [sz, vp]
    ap = ctypes.POINTER(AttentionDesc)
    L.boost_attention_workspace_bytes.argtypes = [ap]
    L.boost_attention_workspace_bytes.restype = sz
    L.boost_attention.argtypes = [ap] + [vp] * 8 + [sz, vp]
    L.boost_attention_bwd.argtypes = [ap] + [vp] * 12 + [sz, vp]
    L.boost_norm_quantize.argtypes = [i64, i64, ctypes.c_int32, ctypes.c_float] + [vp] * 8
    L.boost_grad_clip_workspace_bytes.argtypes = []
    L.boost_grad_clip_workspace_bytes.restype = sz
    L.boost_grad_clip.argtypes = [i64, vp, ctypes.c_double, vp, vp, sz, vp]
    L.boost_status_string.argtypes = [ctypes.c_int]
    L.boost_status_string.restype = ctypes.c_char_p
    L.boost_swiglu_fwd.argtypes = [i64, i64, vp, vp, vp, vp]
    L.boost_swiglu_bwd.argtypes = [i64, i64, vp, vp, vp, vp, vp, vp]
    L.boost_add.argtypes = [i64, vp, vp, vp, vp]
    L.boost_debug_wait_timeout.argtypes = [vp, sz, u32, vp]
    szp = ctypes.POINTER(sz)
    L.boost_block_ws_layout.argtypes = [dp, szp, szp, szp, szp]
    L.boost_rmsnorm_rstd_noalloc.argtypes = [dp, vp, vp, vp]
    L.boost_block_bwd_swiglu.argtypes = [dp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.boost_profile_enable.argtypes = [ctypes.c_int]
    L.boost_profile_only.argtypes = [ctypes.c_int]
    L.boost_profile_kernel_count.argtypes = []
    dbl = ctypes.POINTER(ctypes.c_double)
    L.boost_profile_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_char_p),
                                     ctypes.POINTER(i64), dbl, dbl, dbl]
    L.boost_profile_read_kernels.argtypes = [ctypes.c_int, ctypes.POINTER(i64)]
    for name in EXPORTS:
        if name not in ("boost_block_workspace_bytes", "boost_status_string",
                        "boost_debug_count_log", "boost_fp8_scale_bytes",
                        "boost_fp8_matmul_workspace_bytes", "boost_attention_workspace_bytes",
                        "boost_grad_clip_workspace_bytes"):
            getattr(L, name).restype = ctypes.c_int
    _LIB = L
    return L


def _check(status: int, what: str):
    if status != BOOST_OK:
        raise BoostError(status, what)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype, shape=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def make_desc(T, d, r, k, n, *, S=1, eps=1e-5, act="silu", has_norm=True) -> Desc:
    return Desc(int(T), int(d), int(r), int(k), int(n), int(S), float(eps),
                ACT[act] if isinstance(act, str) else int(act), 1 if has_norm else 0)


def workspace_bytes(desc: Desc) -> int:
    return int(lib().boost_block_workspace_bytes(ctypes.byref(desc)))


class Workspace:
    """Caller-owned device workspace (torch memory), error word cleared on creation."""

    def __init__(self, nbytes: int, device=None, stream=None):
        self.nbytes = max(int(nbytes), 256)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8,
                               device=device or torch.device("cuda"))
        _check(lib().boost_block_ws_init(_ptr(self.buf), self.nbytes, _stream(stream)),
               "boost_block_ws_init")

    @property
    def ptr(self):
        return _ptr(self.buf)

    def ensure(self, nbytes: int):
        if nbytes > self.nbytes:
            self.__init__(nbytes, self.buf.device)
        return self


def layout(desc: Desc):
    """Shard offsets [S+1], group column offsets [k+1], exchange element count (host)."""
    S = desc.S if desc.has_norm else 1
    so = (ctypes.c_int64 * (S + 1))()
    go = (ctypes.c_int64 * (desc.k + 1))()
    ex = ctypes.c_int64(0)
    _check(lib().boost_block_layout(ctypes.byref(desc), so, go, ctypes.byref(ex)),
           "boost_block_layout")
    return list(so), list(go), ex.value


def ws_layout(desc: Desc):
    """Byte offsets of a, dzs, A' and rstd inside a workspace for ``desc``."""
    o = [ctypes.c_size_t(0) for _ in range(4)]
    _check(lib().boost_block_ws_layout(ctypes.byref(desc), *(ctypes.byref(v) for v in o)),
           "boost_block_ws_layout")
    return {"a": o[0].value, "dzs": o[1].value, "Ap": o[2].value, "rstd": o[3].value}


def ws_view(ws: "Workspace", offset: int, shape, dtype):
    """A torch view of workspace bytes (for tests and inspection)."""
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.tensor([], dtype=dtype).element_size()
    return ws.buf[offset:offset + nbytes].view(dtype).view(*shape)


def rmsnorm_stats(desc: Desc, x, ssq=None, rstd=None, stream=None):
    _need(x, "x", torch.bfloat16, (desc.T, desc.d))
    if ssq is None:
        ssq = torch.empty(desc.S, desc.T, dtype=torch.float32, device=x.device)
    if rstd is None:
        rstd = torch.empty(desc.T, dtype=torch.float32, device=x.device)
    _check(lib().boost_rmsnorm_stats(ctypes.byref(desc), _ptr(x), _ptr(ssq), _ptr(rstd),
                                     _stream(stream)), "boost_rmsnorm_stats")
    return ssq, rstd


def rmsnorm_rstd_noalloc(desc: Desc, x, rstd=None, stream=None):
    """Row scales through the allocation-free entry point (for callers that cannot
    allocate device memory; the partials use the library's fixed device array)."""
    _need(x, "x", torch.bfloat16, (desc.T, desc.d))
    if rstd is None:
        rstd = torch.empty(desc.T, dtype=torch.float32, device=x.device)
    _need(rstd, "rstd", torch.float32, (desc.T,))
    _check(lib().boost_rmsnorm_rstd_noalloc(ctypes.byref(desc), _ptr(x), _ptr(rstd),
                                            _stream(stream)), "boost_rmsnorm_rstd_noalloc")
    return rstd


def block_fwd(desc: Desc, x, gamma, A, B, ws: Workspace, *, y=None, rstd=None, stream=None,
              residual=None):
    """y [k,T,n] (and the row scale into ``rstd`` if given). With ``residual`` [T,n]
    (k == 1): y = residual + block(x), added in the up-projection's epilogue."""
    bf = torch.bfloat16
    _need(x, "x", bf, (desc.T, desc.d))
    _need(A, "A", bf, (desc.d, desc.k * desc.r))
    _need(B, "B", bf, (desc.k, desc.r, desc.n))
    if desc.has_norm:
        _need(gamma, "gamma", bf, (desc.d,))
    if y is None:
        y = torch.empty(desc.k, desc.T, desc.n, dtype=bf, device=x.device)
    _need(y, "y", bf, (desc.k, desc.T, desc.n))
    if rstd is not None:
        _need(rstd, "rstd", torch.float32, (desc.T,))
    if residual is not None:
        _need(residual, "residual", bf, (desc.T, desc.n))
        _check(lib().boost_block_fwd_residual(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(A),
                                              _ptr(B), _ptr(residual), _ptr(y), _ptr(rstd),
                                              ws.ptr, ws.nbytes, _stream(stream)),
               "boost_block_fwd_residual")
        return y
    _check(lib().boost_block_fwd(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(A), _ptr(B),
                                 _ptr(y), _ptr(rstd), ws.ptr, ws.nbytes, _stream(stream)),
           "boost_block_fwd")
    return y


def block_fwd_swiglu(desc: Desc, x, gamma, A, B, ws: Workspace, *, y=None, h=None, rstd=None,
                     stream=None):
    """Gate/up block (k == 2) forward with the SwiGLU forward fused in: returns
    (y [2,T,n] = gate, up; h [T,n] = silu(gate) * up)."""
    bf = torch.bfloat16
    if desc.k != 2:
        raise ValueError("block_fwd_swiglu needs k == 2 (gate and up groups)")
    _need(x, "x", bf, (desc.T, desc.d))
    _need(A, "A", bf, (desc.d, desc.k * desc.r))
    _need(B, "B", bf, (desc.k, desc.r, desc.n))
    if desc.has_norm:
        _need(gamma, "gamma", bf, (desc.d,))
    if y is None:
        y = torch.empty(desc.k, desc.T, desc.n, dtype=bf, device=x.device)
    if h is None:
        h = torch.empty(desc.T, desc.n, dtype=bf, device=x.device)
    _need(y, "y", bf, (desc.k, desc.T, desc.n))
    _need(h, "h", bf, (desc.T, desc.n))
    if rstd is not None:
        _need(rstd, "rstd", torch.float32, (desc.T,))
    _check(lib().boost_block_fwd_swiglu(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(A),
                                        _ptr(B), _ptr(y), _ptr(h), _ptr(rstd), ws.ptr, ws.nbytes,
                                        _stream(stream)),
           "boost_block_fwd_swiglu")
    return y, h


def block_up(desc: Desc, a, B, ws: Workspace, *, y=None, h=None, stream=None):
    """The up-projection alone from a given bottleneck activation a [T, k*r]; with h
    (k == 2) also h = silu(y[0]) * y[1]. Returns y (and h)."""
    bf = torch.bfloat16
    _need(a, "a", bf, (desc.T, desc.k * desc.r))
    _need(B, "B", bf, (desc.k, desc.r, desc.n))
    if y is None:
        y = torch.empty(desc.k, desc.T, desc.n, dtype=bf, device=a.device)
    _need(y, "y", bf, (desc.k, desc.T, desc.n))
    if h is not None:
        _need(h, "h", bf, (desc.T, desc.n))
    _check(lib().boost_block_up(ctypes.byref(desc), _ptr(a), _ptr(B), _ptr(y), _ptr(h), ws.ptr,
                                ws.nbytes, _stream(stream)), "boost_block_up")
    return y if h is None else (y, h)


def btp_payload_elems(desc: Desc) -> int:
    """fp32 values of the emulated exchange payload: S*T*k*r partial products, then
    (normed blocks) S*T sums of squares."""
    return desc.S * desc.T * (desc.k * desc.r + (1 if desc.has_norm else 0))


def block_fwd_btp(desc: Desc, x, gamma, A, B, ws: Workspace, *, y=None, rstd=None,
                  payload=None, stream=None):
    """Forward with the down-projection as the emulated bottleneck-aware TP exchange.
    Returns (y [k,T,n], zpart [S,T,k*r], ssq [S,T] or None), the last two views of the
    payload buffer."""
    bf = torch.bfloat16
    _need(x, "x", bf, (desc.T, desc.d))
    _need(A, "A", bf, (desc.d, desc.k * desc.r))
    _need(B, "B", bf, (desc.k, desc.r, desc.n))
    if desc.has_norm:
        _need(gamma, "gamma", bf, (desc.d,))
    if y is None:
        y = torch.empty(desc.k, desc.T, desc.n, dtype=bf, device=x.device)
    _need(y, "y", bf, (desc.k, desc.T, desc.n))
    n_pay = btp_payload_elems(desc)
    if payload is None:
        payload = torch.empty(n_pay, dtype=torch.float32, device=x.device)
    _need(payload, "payload", torch.float32, (n_pay,))
    if rstd is not None:
        _need(rstd, "rstd", torch.float32, (desc.T,))
    _check(lib().boost_block_fwd_btp(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(A), _ptr(B),
                                     _ptr(y), _ptr(rstd), _ptr(payload), ws.ptr, ws.nbytes,
                                     _stream(stream)),
           "boost_block_fwd_btp")
    S, T, kr = desc.S, desc.T, desc.k * desc.r
    zpart = payload[:S * T * kr].view(S, T, kr)
    ssq = payload[S * T * kr:].view(S, T) if desc.has_norm else None
    return y, zpart, ssq


def block_bwd(desc: Desc, x, gamma, A, B, dy, ws: Workspace, *, rstd=None, dx=None,
              dgamma=None, dA=None, dB=None, stream=None, dx_residual=None):
    """Returns (dx, dgamma or None, dA, dB). With ``dx_residual`` [T,d]: dx =
    dx_residual + the block's input gradient, added in the dx epilogue."""
    bf = torch.bfloat16
    _need(x, "x", bf, (desc.T, desc.d))
    _need(A, "A", bf, (desc.d, desc.k * desc.r))
    _need(B, "B", bf, (desc.k, desc.r, desc.n))
    _need(dy, "dy", bf, (desc.k, desc.T, desc.n))
    dev = x.device
    if dx is None:
        dx = torch.empty(desc.T, desc.d, dtype=bf, device=dev)
    if dA is None:
        dA = torch.empty(desc.d, desc.k * desc.r, dtype=bf, device=dev)
    if dB is None:
        dB = torch.empty(desc.k, desc.r, desc.n, dtype=bf, device=dev)
    if desc.has_norm:
        _need(gamma, "gamma", bf, (desc.d,))
        if dgamma is None:
            dgamma = torch.empty(desc.d, dtype=bf, device=dev)
    if rstd is not None:
        _need(rstd, "rstd", torch.float32, (desc.T,))
    if dx_residual is not None:
        _need(dx_residual, "dx_residual", bf, (desc.T, desc.d))
        _check(lib().boost_block_bwd_residual(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(A),
                                              _ptr(B), _ptr(rstd), _ptr(dy), _ptr(dx_residual),
                                              _ptr(dx), _ptr(dgamma), _ptr(dA), _ptr(dB),
                                              ws.ptr, ws.nbytes, _stream(stream)),
               "boost_block_bwd_residual")
        return dx, dgamma, dA, dB
    _check(lib().boost_block_bwd(ctypes.byref(desc), _ptr(x), _ptr(gamma), _ptr(A), _ptr(B),
                                 _ptr(rstd), _ptr(dy), _ptr(dx), _ptr(dgamma), _ptr(dA),
                                 _ptr(dB), ws.ptr, ws.nbytes, _stream(stream)),
           "boost_block_bwd")
    return dx, dgamma, dA, dB


def block_bwd_swiglu(desc: Desc, h, A, B, dy, gate, up, ws: Workspace, *, dgate=None,
                     dup=None, dA=None, dB=None, stream=None):
    """Backward of a no-norm block whose input is h = silu(gate)*up: (dgate, dup, dA, dB)."""
    bf = torch.bfloat16
    _need(h, "h", bf, (desc.T, desc.d))
    _need(A, "A", bf, (desc.d, desc.k * desc.r))
    _need(B, "B", bf, (desc.k, desc.r, desc.n))
    _need(dy, "dy", bf, (desc.k, desc.T, desc.n))
    _need(gate, "gate", bf, (desc.T, desc.d))
    _need(up, "up", bf, (desc.T, desc.d))
    dev = h.device
    if dgate is None:
        dgate = torch.empty(desc.T, desc.d, dtype=bf, device=dev)
    if dup is None:
        dup = torch.empty(desc.T, desc.d, dtype=bf, device=dev)
    if dA is None:
        dA = torch.empty(desc.d, desc.k * desc.r, dtype=bf, device=dev)
    if dB is None:
        dB = torch.empty(desc.k, desc.r, desc.n, dtype=bf, device=dev)
    _check(lib().boost_block_bwd_swiglu(ctypes.byref(desc), _ptr(h), _ptr(A), _ptr(B), _ptr(dy),
                                        _ptr(gate), _ptr(up), _ptr(dgate), _ptr(dup), _ptr(dA),
                                        _ptr(dB), ws.ptr, ws.nbytes, _stream(stream)),
           "boost_block_bwd_swiglu")
    return dgate, dup, dA, dB


def swiglu_fwd(gate, up, h=None, stream=None):
    bf = torch.bfloat16
    _need(gate, "gate", bf)
    _need(up, "up", bf, gate.shape)
    T, n = gate.shape
    if h is None:
        h = torch.empty_like(gate)
    _check(lib().boost_swiglu_fwd(T, n, _ptr(gate), _ptr(up), _ptr(h), _stream(stream)),
           "boost_swiglu_fwd")
    return h


def swiglu_bwd(gate, up, dh, dgate=None, dup=None, stream=None):
    bf = torch.bfloat16
    _need(gate, "gate", bf)
    _need(up, "up", bf, gate.shape)
    _need(dh, "dh", bf, gate.shape)
    T, n = gate.shape
    if dgate is None:
        dgate = torch.empty_like(gate)
    if dup is None:
        dup = torch.empty_like(gate)
    _check(lib().boost_swiglu_bwd(T, n, _ptr(gate), _ptr(up), _ptr(dh), _ptr(dgate), _ptr(dup),
                                  _stream(stream)), "boost_swiglu_bwd")
    return dgate, dup


def add(a, b, out=None, stream=None):
    bf = torch.bfloat16
    _need(a, "a", bf)
    _need(b, "b", bf, a.shape)
    if out is None:
        out = torch.empty_like(a)
    _check(lib().boost_add(a.numel(), _ptr(a), _ptr(b), _ptr(out), _stream(stream)), "boost_add")
    return out


# ---------------------------------------------------- operators around the block
#
# Small calls are bound by this code, so it checks a tensor in one pass and leaves the
# words to _refuse; pointers and the stream go to ctypes as plain integers.

def _refuse(t, name, dtype, shape, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on the current CUDA device {device}, not {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _take(t, name, dtype, shape, device):
    """Address of a contiguous tensor of this type and shape on the current device (the
    stream and the workspace are its)."""
    if (t is None or t.dtype is not dtype or t.get_device() != device or not t.is_contiguous()
            or t.shape != shape):
        _refuse(t, name, dtype, shape, device)
    return t.data_ptr()


# The current device and its current stream straight from torch's bookkeeping where it offers
# them (0.2 us a call instead of 1.5), by the public functions otherwise.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda device: torch.cuda.current_stream(device).cuda_stream)


def _raw_stream(stream, device):
    return _current_raw_stream(device) if stream is None else stream.cuda_stream


def _on(t, name, dtype, device):
    """Address of a tensor of this type on the current device, whatever its strides (the call's
    plan has checked those)."""
    if t.dtype is not dtype or t.get_device() != device:
        _refuse(t.contiguous(), name, dtype, t.shape, device)
    return t.data_ptr()


def _head_strides(shape, stride, name, T, dim):
    """Token and head strides of a [T, heads, dim] tensor whose values are adjacent."""
    if len(shape) != 3 or shape[0] != T or shape[2] != dim:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [T={T}, heads, dim={dim}]")
    if stride[2] != 1 and dim > 1:
        raise ValueError(f"{name} must have adjacent values, not a stride of {stride[2]}")
    # the stride of a single token or head says nothing: a plain one in its place
    heads = shape[1]
    return stride[0] if T > 1 else heads * dim, stride[1] if heads > 1 else dim


@functools.lru_cache(maxsize=512)
def _rope_plan(q, k, q_out, k_out, positions, pos64, pos_at, freq, interleaved, inverse, sections,
               pair_axis):
    """The descriptor of a call whose tensors have these (shape, stride) pairs."""
    T, hq, dim = q[0] if len(q[0]) == 3 else (None, None, None)
    if T is None:
        raise ValueError("q must be [T, heads, dim]")
    strides = [_head_strides(*q, "q", T, dim)]
    strides.append(_head_strides(*k, "k", T, dim) if k else (0, 0))
    strides.append(_head_strides(*q_out, "q_out", T, dim))
    strides.append(_head_strides(*k_out, "k_out", T, dim) if k_out else (0, 0))
    if q_out[0] != q[0] or (k and k_out[0] != k[0]):
        raise ValueError("an output has another shape than its input")
    shape, step = positions
    if len(shape) not in (1, 2) or shape[-1] != T:
        raise ValueError(f"positions has shape {tuple(shape)}, expected [T] or [axes, T]")
    axes = 1 if len(shape) == 1 else shape[0]
    # the stride of a single token or axis says nothing: a plain one in its place
    pos_as = step[0] if axes > 1 else T
    if (T > 1 and step[-1] != 1) or pos_as < T:
        raise ValueError("positions must be contiguous, or columns of a contiguous table")
    if len(freq) != 1:
        raise ValueError("inv_freq must be a vector")
    pairs = freq[0]
    if 2 * pairs > ROPE_MAX_DIM:
        raise BoostError(2, "boost_rope")
    D = RopeDesc(T, hq, k[0][1] if k else 0, dim, 2 * pairs, axes, interleaved, inverse, pos64,
                 *(v for pair in strides for v in pair), pos_at, pos_as)
    if pair_axis is not None:
        if sections is not None:
            raise ValueError("sections and pair_axis exclude each other")
        if len(pair_axis) != pairs or not all(0 <= a < axes for a in pair_axis):
            raise ValueError(f"pair_axis must give one of {axes} axes for each of {pairs} pairs")
        D.axis[:pairs] = pair_axis
    elif sections is not None:
        if len(sections) != axes or min(sections) < 0 or sum(sections) != pairs:
            raise ValueError(f"sections must share {pairs} pairs among {axes} axes")
        D.axis[:pairs] = [a for a, n in enumerate(sections) for _ in range(n)]
    return D


def rope(q, k, positions, inv_freq, *, sections=None, pair_axis=None, interleaved=False,
         inverse=False, q_out=None, k_out=None, stream=None):
    """Rotary positions of q [T, hq, dim] and k [T, hk, dim] (k may be None): returns
    (q_out, k_out). ``inverse`` takes the gradients of the rotated q and k back.

    positions: [T] or [axes, T], int32 or int64. inv_freq: float64 [rot / 2], radians per
    position, below 2^64 in magnitude; the first rot values of each head turn. ``sections``: how many pairs turn with
    each axis, in order (default: all with the first); ``pair_axis``: the axis of each pair
    instead. q, k and the outputs take any token and head strides (multiples of 8), so slices
    of a packed projection and [heads, T, dim] tensors seen as [T, heads, dim] are fine, and
    q_out may be q (in place). positions may be a slice of a vector or columns of a table
    [axes, any]; frequencies are contiguous."""
    bf, device = torch.bfloat16, _device()
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=bf, device=q.device)
    ks = kos = kp = kop = None
    if k is not None:
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=bf, device=k.device)
        ks, kos = (k.shape, k.stride()), (k_out.shape, k_out.stride())
        kp, kop = _on(k, "k", bf, device), _on(k_out, "k_out", bf, device)
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos64 = positions.dtype is torch.int64
    if not pos64 and positions.dtype is not torch.int32:
        raise TypeError(f"positions must be int32 or int64, got {positions.dtype}")
    # the call takes an aligned address and where the positions begin behind it
    pp = _on(positions, "positions", positions.dtype, device)
    behind = pp & 15
    if behind & (7 if pos64 else 3):
        raise BoostError(3, "boost_rope")
    D = _rope_plan((q.shape, q.stride()), ks, (q_out.shape, q_out.stride()), kos,
                   (positions.shape, positions.stride()), pos64, behind >> (3 if pos64 else 2),
                   inv_freq.shape, bool(interleaved), bool(inverse),
                   None if sections is None else tuple(sections),
                   None if pair_axis is None else tuple(pair_axis))
    _check(lib().boost_rope(
        D, _on(q, "q", bf, device), kp,
        pp - behind,
        _take(inv_freq, "inv_freq", torch.float64, inv_freq.shape, device),
        _on(q_out, "q_out", bf, device), kop, _raw_stream(stream, device)), "boost_rope")
    return q_out, k_out


def dropout_add(x, p, seed, offset=0, *, residual=None, out=None, counter=None, stream=None):
    """residual + dropout(x): the element at flat index e is kept by a pure function of (e,
    seed, offset), so no mask is stored (``boost_dropout``). ``counter``: an int64 tensor of
    one value, added to the offset when the kernel runs, for replayed graphs."""
    bf, shape, device = torch.bfloat16, x.shape, _device()
    xp = _take(x, "x", bf, shape, device)
    if out is None:
        out = torch.empty(shape, dtype=bf, device=x.device)
    op = _take(out, "out", bf, shape, device)
    rp = None if residual is None else _take(residual, "residual", bf, shape, device)
    cp = None
    if counter is not None:
        if counter.numel() != 1:
            raise ValueError("counter must hold one value")
        cp = _take(counter, "counter", torch.int64, counter.shape, device)
    if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
        raise ValueError("seed and offset must be unsigned 64-bit values")
    _check(lib().boost_dropout(x.numel(), xp, rp, op, p, seed, offset, cp,
                               _raw_stream(stream, device)), "boost_dropout")
    return out


def dropout_bwd(dout, p, seed, offset=0, *, dx=None, counter=None, stream=None):
    """Gradient of x of ``dropout_add`` with the same p, seed and offset (the residual's
    gradient is dout itself)."""
    return dropout_add(dout, p, seed, offset, out=dx, counter=counter, stream=stream)


def fp8_scale_bytes(rows, K) -> int:
    """Bytes of the scales of one [rows, K] operand (``boost_fp8_scale_bytes``)."""
    return -(-rows // 128) * -(-K // 512) * 512


def _operand_out(given, name, shape, planes, dtype, device_of, device):
    """The (values, scales) tensors of a quantised operand and their addresses."""
    if given is None:
        q = torch.empty(shape, dtype=dtype, device=device_of)
        sf = torch.empty(planes, dtype=torch.uint8, device=device_of)
        return (q, sf), q.data_ptr(), sf.data_ptr()
    return (given, _take(given[0], name, dtype, shape, device),
            _take(given[1], f"{name} scales", torch.uint8, planes, device))


@functools.lru_cache(maxsize=512)
def _fp8_quant_plan(dims, strides, fmt, block_rows):
    """(descriptor, type, values' and scales' shapes by rows, by columns) of a matrix or
    matrices with these dimensions and strides."""
    code, dtype = FP8_FORMATS[fmt]
    if len(dims) not in (2, 3) or (dims[-1] > 1 and strides[-1] != 1):
        raise ValueError("x must be [rows, cols] or [G, rows, cols] with adjacent columns")
    lead = tuple(dims[:-2])
    G, (rows, cols) = (lead[0] if lead else 1), dims[-2:]
    # the stride of a single row or matrix says nothing: a plain one in its place
    D = Fp8QuantDesc(G, rows, cols, strides[-2] if rows > 1 else cols,
                     strides[0] if G > 1 else 0, code, block_rows)

    def shapes(r, K):
        return lead + (r, -(-K // 16) * 16), lead + (fp8_scale_bytes(r, K),)

    return D, dtype, shapes(rows, cols), shapes(cols, rows)


def fp8_quantize(x, *, fmt="e4m3", block_rows=1, way="rows", gamma=None, rows_out=None,
                 cols_out=None, stream=None):
    """8-bit operands of x [rows, cols] or [G, rows, cols] (any row and matrix strides that
    are multiples of 8): ((q, scales) or None, (qt, scales) or None).

    way "rows": q [.., rows, pitch] contracts the columns; "columns": qt [.., cols, pitch]
    contracts the rows; "both": one reading of x gives both. pitch is the contracted length
    rounded up to 16. ``block_rows`` 128 shares a scale among 128 x 128 values, so that q and
    qt hold the same values. ``gamma`` [rows]: x is replaced by bf16(gamma[row] x).
    ``rows_out``, ``cols_out``: (q, scales) tensors to write into."""
    if fmt not in FP8_FORMATS or way not in ("rows", "columns", "both"):
        raise ValueError("fmt is 'e4m3' or 'e5m2', way 'rows', 'columns' or 'both'")
    device = _device()
    xp = _on(x, "x", torch.bfloat16, device)
    D, dtype, of_rows, of_cols = _fp8_quant_plan(x.shape, x.stride(), fmt, block_rows)
    gp = None if gamma is None else _take(gamma, "gamma", torch.bfloat16, (D.rows,), device)
    by_rows = by_cols = q = sf = qt = sft = None
    if way != "columns":
        by_rows, q, sf = _operand_out(rows_out, "rows_out", *of_rows, dtype, x.device, device)
    elif rows_out is not None:
        raise ValueError("rows_out given, but way is 'columns'")
    if way != "rows":
        by_cols, qt, sft = _operand_out(cols_out, "cols_out", *of_cols, dtype, x.device, device)
    elif cols_out is not None:
        raise ValueError("cols_out given, but way is 'rows'")
    _check(lib().boost_fp8_quantize(D, xp, gp, q, sf, qt, sft, _raw_stream(stream, device)),
           "boost_fp8_quantize")
    return by_rows, by_cols


def fp8_matmul_workspace_bytes(M, N, K, G=1) -> int:
    pitch = -(-K // 16) * 16
    return int(lib().boost_fp8_matmul_workspace_bytes(
        Fp8MatmulDesc(G, M, N, K, pitch, pitch, 0, 0, 0)))


@functools.lru_cache(maxsize=512)
def _fp8_matmul_plan(da, db, a_dtype, b_dtype, K, act):
    """(descriptor, shapes of a's and b's scales, of the result, of a row scale)."""
    lead = tuple(da[:-2])
    if len(da) not in (2, 3) or len(db) != len(da) or tuple(db[:-2]) != lead:
        raise ValueError("operands must be [M, pitch] and [N, pitch], or [G, ...] of them")
    if a_dtype not in FP8_CODE or b_dtype not in FP8_CODE:
        raise TypeError(f"operands must be float8_e4m3fn or float8_e5m2, got {a_dtype}, {b_dtype}")
    M, N = da[-2], db[-2]
    D = Fp8MatmulDesc(lead[0] if lead else 1, M, N, K, da[-1], db[-1], FP8_CODE[a_dtype],
                      FP8_CODE[b_dtype], ACT[act])
    return (D, lead + (fp8_scale_bytes(M, K),), lead + (fp8_scale_bytes(N, K),), lead + (M, N),
            (M,))


def fp8_matmul(a, a_scales, b, b_scales, K, ws: Workspace, *, row_scale=None, act="identity",
               out=None, stream=None):
    """act(row_scale * (A @ B^T)) [M, N] in bf16 of 8-bit operands A [M, pitch], B [N, pitch]
    with their scales (``fp8_quantize``), K values contracted; [G, ...] operands give the G
    products [G, M, N]. row_scale: float32 [M]."""
    device = _device()
    da, db, ta, tb, wb = a.shape, b.shape, a.dtype, b.dtype, ws.buf
    D, a_planes, b_planes, shape, rows = _fp8_matmul_plan(da, db, ta, tb, K, act)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=a.device)
    _check(lib().boost_fp8_matmul(
        D, _take(a, "a", ta, da, device),
        _take(a_scales, "a_scales", torch.uint8, a_planes, device),
        _take(b, "b", tb, db, device),
        _take(b_scales, "b_scales", torch.uint8, b_planes, device),
        None if row_scale is None else _take(row_scale, "row_scale", torch.float32, rows, device),
        _take(out, "out", torch.bfloat16, shape, device), _on(wb, "ws", torch.uint8, device),
        ws.nbytes, _raw_stream(stream, device)), "boost_fp8_matmul")
    return out


# ------------------------------------------------------------------------ attention
def attention_workspace_bytes(Tq, Tk, hq, hk, dim, sequences=1) -> int:
    """Bytes of a workspace for ``attention`` and ``attention_bwd`` at these sizes."""
    return int(lib().boost_attention_workspace_bytes(
        AttentionDesc(Tq, Tk, hq, hk, dim, sequences, 0, 1.0)))


@functools.lru_cache(maxsize=512)
def _attention_plan(q, k, v, out, grads, causal, scale, starts):
    """The descriptor of a call whose tensors have these (shape, stride) pairs; grads: those of
    dout, dq, dk, dv; starts: the shapes of q_starts and k_starts."""
    if len(q[0]) != 3 or len(k[0]) != 3:
        raise ValueError("q, k and v must be [T, heads, dim]")
    Tq, hq, dim = q[0]
    Tk, hk = k[0][:2]
    like_q, like_k = (Tq, hq, dim), (Tk, hk, dim)
    named = [("q", q, like_q), ("k", k, like_k), ("v", v, like_k), ("out", out, like_q)]
    if grads:
        named += list(zip(("dout", "dq", "dk", "dv"), grads, (like_q, like_q, like_k, like_k)))
    strides = []
    for name, (shape, stride), want in named:
        if tuple(shape) != want:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected {want}")
        strides += _head_strides(shape, stride, name, want[0], dim)
    given = [s for s in starts if s is not None]
    if any(len(s) != 1 or s[0] < 2 or s != given[0] for s in given):
        raise ValueError("q_starts and k_starts are vectors of one length, sequences + 1")
    sequences = given[0][0] - 1 if given else 1
    if sequences > 1 and len(given) != 2:
        raise ValueError("several sequences need both q_starts and k_starts")
    return AttentionDesc(Tq, Tk, hq, hk, dim, sequences, causal,
                         dim ** -0.5 if scale is None else scale, *strides)


def _of(t):
    return t.shape, t.stride()


def _number(scale):
    """A plan is kept by its arguments' values: a tensor's would be kept by the tensor."""
    return None if scale is None else float(scale)


def _starts(t, name, device):
    return None if t is None else _take(t, name, torch.int32, t.shape, device)


def attention(q, k, v, ws: Workspace, *, causal=True, scale=None, q_starts=None, k_starts=None,
              out=None, lse=None, stream=None):
    """softmax(scale q k^T) v of q [Tq, hq, dim], k and v [Tk, hk, dim] (hq a multiple of hk, dim
    a multiple of 8 up to 128, scale dim^-1/2 where none is given): returns (out [Tq, hq, dim],
    lse [hq, Tq] float32, the logarithms of the rows' sums, which the backward takes).

    q_starts, k_starts: int32 [sequences + 1] on the device, where the packed sequences begin;
    one sequence of all rows without them. causal: a sequence's last query sees all its keys, each
    one before one key less, so new tokens may follow a context; a query that sees none gives 0
    (lse -inf). Rows behind the last sequence are left as they were. q, k, v and out take any
    token and head strides that are multiples of 8."""
    bf, device = torch.bfloat16, _device()
    if out is None:
        out = torch.empty(q.shape, dtype=bf, device=q.device)
    D = _attention_plan(_of(q), _of(k), _of(v), _of(out), None, bool(causal), _number(scale),
                        (None if q_starts is None else q_starts.shape,
                         None if k_starts is None else k_starts.shape))
    if lse is None:
        lse = torch.empty((D.hq, D.Tq), dtype=torch.float32, device=q.device)
    _check(lib().boost_attention(
        D, _on(q, "q", bf, device), _on(k, "k", bf, device), _on(v, "v", bf, device),
        _starts(q_starts, "q_starts", device), _starts(k_starts, "k_starts", device),
        _on(out, "out", bf, device), _take(lse, "lse", torch.float32, (D.hq, D.Tq), device),
        _on(ws.buf, "ws", torch.uint8, device), ws.nbytes, _raw_stream(stream, device)),
        "boost_attention")
    return out, lse


def attention_bwd(q, k, v, out, lse, dout, ws: Workspace, *, causal=True, scale=None,
                  q_starts=None, k_starts=None, dq=None, dk=None, dv=None, stream=None):
    """Gradients (dq, dk, dv) of ``attention`` from its out and lse and the gradient of out; the
    other arguments are the forward's. Every sum is taken in a fixed order."""
    bf, device = torch.bfloat16, _device()
    if dq is None:
        dq = torch.empty(q.shape, dtype=bf, device=q.device)
    if dk is None:
        dk = torch.empty(k.shape, dtype=bf, device=q.device)
    if dv is None:
        dv = torch.empty(v.shape, dtype=bf, device=q.device)
    D = _attention_plan(_of(q), _of(k), _of(v), _of(out), (_of(dout), _of(dq), _of(dk), _of(dv)),
                        bool(causal), _number(scale),
                        (None if q_starts is None else q_starts.shape,
                         None if k_starts is None else k_starts.shape))
    _check(lib().boost_attention_bwd(
        D, _on(q, "q", bf, device), _on(k, "k", bf, device), _on(v, "v", bf, device),
        _on(out, "out", bf, device), _take(lse, "lse", torch.float32, (D.hq, D.Tq), device),
        _on(dout, "dout", bf, device), _starts(q_starts, "q_starts", device),
        _starts(k_starts, "k_starts", device), _on(dq, "dq", bf, device),
        _on(dk, "dk", bf, device), _on(dv, "dv", bf, device),
        _on(ws.buf, "ws", torch.uint8, device), ws.nbytes, _raw_stream(stream, device)),
        "boost_attention_bwd")
    return dq, dk, dv


# ------------------------------------------------------- norm with an 8-bit output
def norm_quantize(x, *, residual=None, gamma=None, eps=1e-5, fmt="e4m3", h=None, rstd=None,
                  rows_out=None, stream=None):
    """h = x + residual [T, d], rstd [T] = (mean h^2 + eps)^-1/2 and the 8-bit operand of h, or of
    bf16(gamma h): returns (h, rstd, (q, scales)) with (q, scales) as ``fp8_quantize`` gives it by
    rows. The norm's value is q's times rstd, the product's ``row_scale``. Without a residual h is
    x itself, unless a tensor to copy it into is given; with one, h may be x or the residual."""
    if fmt not in FP8_FORMATS:
        raise ValueError("fmt is 'e4m3' or 'e5m2'")
    bf, device = torch.bfloat16, _device()
    if x.dim() != 2:
        raise ValueError("x must be [T, d]")
    shape = T, d = x.shape
    code, dtype = FP8_FORMATS[fmt]
    xp = _take(x, "x", bf, shape, device)
    rp = None if residual is None else _take(residual, "residual", bf, shape, device)
    gp = None if gamma is None else _take(gamma, "gamma", bf, (d,), device)
    if h is None and residual is not None:
        h = torch.empty(shape, dtype=bf, device=x.device)
    hp = None if h is None else _take(h, "h", bf, shape, device)
    if rstd is None:
        rstd = torch.empty((T,), dtype=torch.float32, device=x.device)
    by_rows, q, sf = _operand_out(rows_out, "rows_out", (T, -(-d // 16) * 16),
                                  (fp8_scale_bytes(T, d),), dtype, x.device, device)
    _check(lib().boost_norm_quantize(
        T, d, code, eps, xp, rp, gp, hp, _take(rstd, "rstd", torch.float32, (T,), device), q, sf,
        _raw_stream(stream, device)), "boost_norm_quantize")
    return x if h is None else h, rstd, by_rows


# ------------------------------------------------------------- gradient clipping
_dtype_of = operator.attrgetter("dtype")


def grad_clip_workspace_bytes() -> int:
    return int(lib().boost_grad_clip_workspace_bytes())


def grad_clip(grads, max_norm, ws: Workspace, *, outs=None, norm=None, stream=None):
    """The norm over all gradients (float32 [1], on the device), and each scaled in place by
    min(1, max_norm / (norm + 1e-6)), or into ``outs``, each of its gradient's type and number of
    values. max_norm None: the norm alone. Gradients are contiguous, bfloat16 or float32, of any
    number, sizes and shapes, at addresses that are multiples of 16 bytes."""
    device = _device()
    grads = list(grads)
    outs = grads if outs is None else list(outs)
    if len(outs) != len(grads):
        raise ValueError(f"{len(outs)} outs for {len(grads)} gradients")
    if norm is None:
        norm = torch.empty((1,), dtype=torch.float32, device=ws.buf.device)
    # (a model has hundreds: whole lists at a time, and the words for what is wrong afterwards)
    n, bf, wide, T = len(grads), torch.bfloat16, torch.float32, torch.Tensor
    types, sizes = list(map(_dtype_of, grads)), list(map(T.numel, grads))
    fine = ({bf, wide}.issuperset(types) and all(map(T.is_contiguous, grads))
            and {device}.issuperset(map(T.get_device, grads)))
    if outs is not grads:
        fine = (fine and list(map(_dtype_of, outs)) == types and list(map(T.numel, outs)) == sizes
                and all(map(T.is_contiguous, outs))
                and {device}.issuperset(map(T.get_device, outs)))
    if not fine:
        for i, (g, o) in enumerate(zip(grads, outs)):
            if g.dtype is not bf and g.dtype is not wide:
                raise TypeError(f"gradient {i} must be bfloat16 or float32, got {g.dtype}")
            _take(g, f"gradient {i}", g.dtype, g.shape, device)
            _take(o, f"out {i}", g.dtype, g.shape, device)
    at = list(map(T.data_ptr, grads))
    to = [0] * n if max_norm is None else at if outs is grads else list(map(T.data_ptr, outs))
    # the table of Grad entries: four words each
    words = [0] * (4 * n)
    words[0::4], words[1::4], words[2::4], words[3::4] = at, to, sizes, [d is wide for d in types]
    table = array.array("q", words)
    _check(lib().boost_grad_clip(
        n, table.buffer_info()[0], float("inf") if max_norm is None else max_norm,
        _take(norm, "norm", wide, (1,), device), _on(ws.buf, "ws", torch.uint8, device), ws.nbytes,
        _raw_stream(stream, device)), "boost_grad_clip")
    return norm


def check(ws: Workspace, stream=None):
    """Synchronise and raise if a kernel recorded a device-side error."""
    _check(lib().boost_block_check(ws.ptr, _stream(stream)), "boost_block_check")


def profile_enable(on: bool):
    _check(lib().boost_profile_enable(1 if on else 0), "boost_profile_enable")


def profile_only(name=None):
    """Time only the named kernel's operations (None: every kernel)."""
    L = lib()
    idx = -1
    if name is not None:
        names = {}
        for i in range(L.boost_profile_kernel_count()):
            nm = ctypes.c_char_p()
            _check(L.boost_profile_read(i, ctypes.byref(nm), None, None, None, None),
                   "boost_profile_read")
            names[nm.value.decode()] = i
        if name not in names:
            raise KeyError(name)
        idx = names[name]
    _check(L.boost_profile_only(idx), "boost_profile_only")


def profile_kernels():
    """{kernel name: kernels launched} for kernels that ran (an operation split over
    concurrent launches counts each of them)."""
    L = lib()
    out = {}
    for i in range(L.boost_profile_kernel_count()):
        name = ctypes.c_char_p()
        n = ctypes.c_int64(0)
        _check(L.boost_profile_read(i, ctypes.byref(name), None, None, None, None),
               "boost_profile_read")
        _check(L.boost_profile_read_kernels(i, ctypes.byref(n)), "boost_profile_read_kernels")
        if n.value:
            out[name.value.decode()] = n.value
    return out


def profile_read():
    """{kernel name: (launches, total_ms, total_flops, total_bytes)} for kernels that ran."""
    L = lib()
    out = {}
    for i in range(L.boost_profile_kernel_count()):
        name = ctypes.c_char_p()
        n = ctypes.c_int64(0)
        ms, fl, by = ctypes.c_double(0), ctypes.c_double(0), ctypes.c_double(0)
        _check(L.boost_profile_read(i, ctypes.byref(name), ctypes.byref(n), ctypes.byref(ms),
                                    ctypes.byref(fl), ctypes.byref(by)), "boost_profile_read")
        if n.value:
            out[name.value.decode()] = (n.value, ms.value, fl.value, by.value)
    return out


def debug_count_writes(counts=None):
    """Start (with a zeroed int32 CUDA tensor) or stop (None) write counting."""
    if counts is None:
        _check(lib().boost_debug_count_writes(None, 0), "boost_debug_count_writes")
        return
    if counts.dtype != torch.int32 or not counts.is_cuda or not counts.is_contiguous():
        raise TypeError("counts must be a contiguous int32 CUDA tensor")
    _check(lib().boost_debug_count_writes(_ptr(counts), counts.numel()),
           "boost_debug_count_writes")


def debug_count_log():
    """[(offset, M, N, ld, planes, splits, plane_stride, split_stride)] of the recorded
    GEMM operations; raises if the count buffer ran out."""
    L = lib()
    n = L.boost_debug_count_log(None, 0)
    if n < 0:
        raise RuntimeError("write-count buffer too small")
    buf = (ctypes.c_int64 * (8 * max(n, 1)))()
    L.boost_debug_count_log(buf, n)
    return [tuple(buf[8 * i:8 * i + 8]) for i in range(n)]


def debug_wait_timeout(ws: Workspace, limit_us: int, stream=None):
    _check(lib().boost_debug_wait_timeout(ws.ptr, ws.nbytes, int(limit_us), _stream(stream)),
           "boost_debug_wait_timeout")
