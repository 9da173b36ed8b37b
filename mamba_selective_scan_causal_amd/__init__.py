"""MI355X-native Mamba-1 (S6) block core: Python binding of libmss.

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libmss.so`` (built in-tree by ``build.py``); PyTorch supplies
device memory and the current stream.  There is no fallback: if the library
is missing or a call fails, an exception is raised.

Layouts (fp32, contiguous, on the current CUDA/HIP device):
  x, z, delta, u, y : (batch*seq_len, D)     B, C : (batch*seq_len, N)
  A_log : (D, N)   D_vec, b_conv : (D,)   w_conv : (D, K)
  h0, h_last : (batch, D, N)   h_cache : (batch, seq_len, D, N)
Single-token step: x, z, delta, y : (batch, D); B, C : (batch, N);
  conv_state : (batch, K-1, D) oldest first; h : (batch, D, N).

The gated linear recurrence (``gated_scan``, ``gated_scan_backward``,
``gated_step``) and the norms before and after a block (``add_norm``,
``gated_norm`` and their backward passes) take activations in float32,
bfloat16 or float16, row-strided where that is handy; see each function.  So do
the two ends of a model, the embedding (``embedding``) and the head with its
loss (``head_loss``), with their backward passes; ``grad_norm`` and
``clip_grads`` take lists of gradients of any of these types.

A call given ``stream=`` allocates what it returns, and its workspace, as that
stream's own memory.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from operator import index as _index

from . import inputs  # noqa: F401  (seeded synthetic inputs; no method arithmetic)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmss.so")

ZOH = 0
EULER = 1
_DISC = {"zoh": ZOH, "euler": EULER, ZOH: ZOH, EULER: EULER}

MSS_OK = 0


class MssError(RuntimeError):
    def __init__(self, fn, status, msg, hip_error=0):
        super().__init__(f"{fn} failed: status {status} ({msg})"
                         + (f", hipError {hip_error}" if hip_error else ""))
        self.status = status
        self.hip_error = hip_error


class Dims(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("seq_len", ctypes.c_int64),
                ("d_inner", ctypes.c_int64), ("d_state", ctypes.c_int64),
                ("d_conv", ctypes.c_int64)]


FLAG_EXACT = 1          # no time split: the plain sequential recurrence
FLAG_CKPT8 = 2          # state checkpoints every 8 steps (forward h_cache / backward h_ckpt)


def make_dims(batch, seq_len, d_inner, d_state, d_conv=1, exact=False, ckpt8=False) -> Dims:
    flags = (FLAG_EXACT if exact else 0) | (FLAG_CKPT8 if ckpt8 else 0)
    return Dims(ctypes.sizeof(Dims), flags, batch, seq_len, d_inner, d_state, d_conv)


class Strides(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("x", ctypes.c_int64), ("z", ctypes.c_int64), ("delta", ctypes.c_int64),
                ("B", ctypes.c_int64), ("C", ctypes.c_int64), ("y", ctypes.c_int64)]


def make_strides(x, z, delta, B, C, y) -> Strides:
    return Strides(ctypes.sizeof(Strides), 0, x, z, delta, B, C, y)


class SsdDims(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("seq_len", ctypes.c_int64),
                ("n_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("d_state", ctypes.c_int64), ("n_groups", ctypes.c_int64)]


def make_ssd_dims(batch, seq_len, n_heads, head_dim, d_state, n_groups=1, exact=False) -> SsdDims:
    return SsdDims(ctypes.sizeof(SsdDims), FLAG_EXACT if exact else 0, batch, seq_len, n_heads,
                   head_dim, d_state, n_groups)


class GatedDims(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("seq_len", ctypes.c_int64),
                ("d_inner", ctypes.c_int64), ("gate_scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class GatedStrides(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                *((n, ctypes.c_int64) for n in ("x", "r", "i", "z", "y", "dx", "dr", "di", "dz"))]


class NormDims(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("res_dtype", ctypes.c_int32),
                ("kind", ctypes.c_int32), ("order", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("width", ctypes.c_int64), ("groups", ctypes.c_int64),
                ("eps", ctypes.c_float), ("alpha", ctypes.c_float)]


class NormStrides(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                *((n, ctypes.c_int64) for n in ("x", "z", "residual", "s", "y", "ds", "dx", "dz",
                                                "dresidual"))]


class EmbedDims(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("id_bytes", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("width", ctypes.c_int64),
                ("scale", ctypes.c_float), ("reserved2", ctypes.c_int32)]


class EmbedStrides(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("weight", ctypes.c_int64), ("y", ctypes.c_int64)]


class HeadDims(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("id_bytes", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("width", ctypes.c_int64),
                ("logit_scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class HeadStrides(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                *((n, ctypes.c_int64) for n in ("x", "weight", "dx", "dweight"))]


class ListTensor(ctypes.Structure):      # mss_tensor; struct format PPqii
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


EXPORTS = ("mss_conv1d_silu", "mss_selective_scan", "mss_mamba1_core", "mss_selective_step",
           "mss_selective_scan_strided", "mss_mamba1_core_strided",
           "mss_workspace_bytes", "mss_selective_scan_backward", "mss_conv1d_silu_backward",
           "mss_ssd_scan", "mss_time_split", "mss_ssd_time_split",
           "mss_selective_scan_backward_noalloc",
           "mss_gated_workspace_bytes", "mss_gated_scan", "mss_gated_scan_backward",
           "mss_gated_step", "mss_norm_workspace_bytes", "mss_add_norm", "mss_add_norm_backward",
           "mss_gated_norm", "mss_gated_norm_backward",
           "mss_embedding", "mss_embedding_backward", "mss_embed_workspace_bytes",
           "mss_head_workspace_bytes", "mss_head_loss", "mss_head_loss_backward",
           "mss_clip_workspace_bytes", "mss_grad_norm", "mss_clip_grads",
           "mss_strerror", "mss_version", "mss_last_hip_error")

OP_SELECTIVE_SCAN_BACKWARD = 1
OP_CONV1D_SILU_BACKWARD = 2
OP_SELECTIVE_SCAN = 3
OP_GATED_SCAN = 4
OP_GATED_SCAN_BACKWARD = 5
OP_ADD_NORM_BACKWARD = 6
OP_GATED_NORM_BACKWARD = 7
OP_HEAD_LOSS = 8
OP_HEAD_LOSS_BACKWARD = 9
EMBED_ACCUMULATE = 1                  # MSS_EMBED_ACCUMULATE
GATED_CKPT_STEPS = 64                 # MSS_GATED_CKPT_STEPS
MAX_WIDTH = 1 << 28                   # MSS_MAX_WIDTH
NOALLOC_SCRATCH_BYTES = 256 << 20     # MSS_NOALLOC_SCRATCH_BYTES
MSS_ESCRATCH = -6

_lib = None


def lib():
    """The loaded libmss (ctypes).  Raises if the HIP library is not built."""
    global _lib
    if _lib is None:
        # torch ships its own HIP runtime (soname libamdhip64.so.7, file name
        # libamdhip64.so).  Loaded first, it also serves libmss's dependency;
        # loading libmss first would bring in a second runtime from the ROCm
        # install, which does not see torch's device memory.
        import torch  # noqa: F401
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m mamba_selective_scan_causal_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i = ctypes.c_void_p, ctypes.c_int
        dp = ctypes.POINTER(Dims)
        L.mss_conv1d_silu.argtypes = [dp, p, p, p, p, p]
        L.mss_selective_scan.argtypes = [dp, i, p, p, p, p, p, p, p, p, p, p, p, p]
        L.mss_mamba1_core.argtypes = [dp, i, p, p, p, p, p, p, p, p, p, p, p, p, p, p]
        L.mss_selective_step.argtypes = [dp, i, p, p, p, p, p, p, p, p, p, p, p, p, p]
        sp = ctypes.POINTER(Strides)
        L.mss_selective_scan_strided.argtypes = [dp, sp, i] + [p] * 12
        L.mss_mamba1_core_strided.argtypes = [dp, sp, i] + [p] * 14
        sz = ctypes.c_size_t
        L.mss_workspace_bytes.argtypes = [dp, i, ctypes.POINTER(sz)]
        L.mss_selective_scan_backward.argtypes = [dp, i] + [p] * 19 + [sz, p]
        L.mss_selective_scan_backward_noalloc.argtypes = [dp, i] + [p] * 18
        L.mss_conv1d_silu_backward.argtypes = [dp] + [p] * 8 + [sz, p]
        L.mss_ssd_scan.argtypes = [ctypes.POINTER(SsdDims), i] + [p] * 11
        L.mss_time_split.argtypes = [dp, i, ctypes.POINTER(ctypes.c_int64)]
        L.mss_ssd_time_split.argtypes = [ctypes.POINTER(SsdDims), ctypes.POINTER(ctypes.c_int64)]
        gd, gs = ctypes.POINTER(GatedDims), ctypes.POINTER(GatedStrides)
        nd, ns = ctypes.POINTER(NormDims), ctypes.POINTER(NormStrides)
        L.mss_gated_workspace_bytes.argtypes = [gd, i, ctypes.POINTER(sz)]
        L.mss_gated_scan.argtypes = [gd, gs] + [p] * 11 + [sz, p]
        L.mss_gated_scan_backward.argtypes = [gd, gs] + [p] * 16 + [sz, p]
        L.mss_gated_step.argtypes = [gd, gs] + [p] * 8
        L.mss_norm_workspace_bytes.argtypes = [nd, i, ctypes.POINTER(sz)]
        L.mss_add_norm.argtypes = [nd, ns] + [p] * 8
        L.mss_add_norm_backward.argtypes = [nd, ns] + [p] * 12 + [sz, p]
        L.mss_gated_norm.argtypes = [nd, ns] + [p] * 8
        L.mss_gated_norm_backward.argtypes = [nd, ns] + [p] * 12 + [sz, p]
        ed, es = ctypes.POINTER(EmbedDims), ctypes.POINTER(EmbedStrides)
        hd, hs = ctypes.POINTER(HeadDims), ctypes.POINTER(HeadStrides)
        f32, i64 = ctypes.c_float, ctypes.c_int64
        L.mss_embedding.argtypes = [ed, es] + [p] * 4
        L.mss_embedding_backward.argtypes = [ed, es] + [p] * 4 + [sz, p]
        L.mss_embed_workspace_bytes.argtypes = [ed, ctypes.POINTER(sz)]
        L.mss_head_workspace_bytes.argtypes = [hd, i, ctypes.POINTER(sz)]
        L.mss_head_loss.argtypes = [hd, hs] + [p] * 6 + [sz, p]
        L.mss_head_loss_backward.argtypes = [hd, hs] + [p] * 9 + [sz, p]
        L.mss_clip_workspace_bytes.argtypes = [i64, ctypes.POINTER(sz)]
        L.mss_grad_norm.argtypes = [p, i64, f32, p, p, sz, p]
        L.mss_clip_grads.argtypes = [p, i64, f32, f32, p, p, sz, p]
        for f in ("mss_embedding", "mss_embedding_backward", "mss_embed_workspace_bytes",
                  "mss_head_workspace_bytes", "mss_head_loss", "mss_head_loss_backward",
                  "mss_clip_workspace_bytes", "mss_grad_norm", "mss_clip_grads"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("mss_gated_workspace_bytes", "mss_gated_scan", "mss_gated_scan_backward",
                  "mss_gated_step", "mss_norm_workspace_bytes", "mss_add_norm",
                  "mss_add_norm_backward", "mss_gated_norm", "mss_gated_norm_backward"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("mss_conv1d_silu", "mss_selective_scan", "mss_mamba1_core",
                  "mss_selective_step", "mss_selective_scan_strided", "mss_mamba1_core_strided",
                  "mss_workspace_bytes", "mss_selective_scan_backward",
                  "mss_conv1d_silu_backward", "mss_ssd_scan", "mss_time_split",
                  "mss_ssd_time_split", "mss_selective_scan_backward_noalloc", "mss_version",
                  "mss_last_hip_error"):
            getattr(L, f).restype = ctypes.c_int
        L.mss_strerror.argtypes = [ctypes.c_int]
        L.mss_strerror.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(fn, status):
    if status != MSS_OK:
        L = lib()
        raise MssError(fn, status, L.mss_strerror(status).decode(), L.mss_last_hip_error())


def _disc(disc) -> int:
    key = disc.lower() if isinstance(disc, str) else disc
    if key not in _DISC:
        raise ValueError("disc must be 'zoh' or 'euler'")
    return _DISC[key]


def _torch():
    import torch
    return torch


def _ptr(t, name, shape, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    _same_device(t, name)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr() or None


def _rows(t, name, rows, cols, required=True):
    """(pointer, row stride) of a (rows, cols) fp32 GPU tensor whose rows may be
    strided (a column slice of a wider buffer); columns must be unit-stride."""
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None, cols
    torch = _torch()
    if not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or not t.is_cuda:
        raise TypeError(f"{name} must be a float32 GPU tensor")
    _same_device(t, name)
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name}: expected shape {(rows, cols)}, got {tuple(t.shape)}")
    if rows > 0 and cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: columns must be contiguous")
    ld = t.stride(0) if rows > 1 else cols
    return (t.data_ptr() or None), ld


def _same_device(t, name):
    # the kernels run on the current device: every tensor must live there
    dev = _torch().cuda.current_device()
    if t.device.index != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _dense(*ts):
    return all(t is None or t.is_contiguous() for t in ts)


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    if s.device.index != torch.cuda.current_device():
        raise ValueError(f"stream is on {s.device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")
    return ctypes.c_void_p(s.cuda_stream)


def _empty(shape, like, stream=None, dtype=None):
    if stream is not None:
        return _own_memory(stream, lambda: _empty(shape, like, dtype=dtype))
    return _torch().empty(shape, dtype=dtype or like.dtype, device=like.device)


def _own_memory(stream, make):
    """make(), a fresh tensor, in the memory of the stream that a call is given.

    Memory of the current stream may be handed out again, or still be in use,
    by that stream's own work, which is not ordered with the call's.  What the
    call returns may be used on the current stream afterwards: dropped, it is
    not handed out before that work is done either."""
    torch = _torch()
    _stream(stream)
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(torch.cuda.current_stream())
    return t


def conv1d_silu(x, w_conv, b_conv=None, *, batch, seq_len, out=None, stream=None):
    """u = SiLU(causal depthwise conv1d(x) + b_conv), (batch*seq_len, D)."""
    D, K = w_conv.shape
    M = batch * seq_len
    u = out if out is not None else _empty((M, D), x, stream)
    dims = make_dims(batch, seq_len, D, 1, K)
    _check("mss_conv1d_silu", lib().mss_conv1d_silu(
        ctypes.byref(dims), _ptr(x, "x", (M, D)), _ptr(w_conv, "w_conv", (D, K)),
        _ptr(b_conv, "b_conv", (D,), False), _ptr(u, "u", (M, D)), _stream(stream)))
    return u


def ckpt_steps(seq_len) -> int:
    """Rows of an 8-step checkpoint tensor: ceil(seq_len / 8)."""
    return (seq_len + 7) // 8


def _scan_outputs(x, batch, seq_len, D, N, out, h_cache, h_last, ckpt8, stream):
    M = batch * seq_len
    y = out if out is not None else _empty((M, D), x, stream)
    Lc = ckpt_steps(seq_len) if ckpt8 else seq_len
    hc = (h_cache if not isinstance(h_cache, bool) else
          (_empty((batch, Lc, D, N), x, stream) if h_cache else None))
    hl = (h_last if not isinstance(h_last, bool) else
          (_empty((batch, D, N), x, stream) if h_last else None))
    return y, hc, hl


def selective_scan(u, delta, A_log, B, C, D_vec=None, z=None, h0=None, *, batch, seq_len, disc,
                   h_cache=False, h_last=False, out=None, stream=None, exact=False, ckpt8=False):
    """Selective scan + gate on a given u.  Returns (y, h_cache, h_last).

    ``h_cache`` / ``h_last``: False (skip), True (allocate) or an output tensor.
    u, delta, z, B, C and ``out`` may be row-strided views (column slices).
    ``exact``: no time split (the plain sequential recurrence, less parallel).
    ``ckpt8``: h_cache is (batch, ceil(seq_len/8), D, N), the state entering
    steps 0, 8, 16, ... (the backward's checkpoints)."""
    D, N = A_log.shape
    M = batch * seq_len
    Lc = ckpt_steps(seq_len) if ckpt8 else seq_len
    y, hc, hl = _scan_outputs(u, batch, seq_len, D, N, out, h_cache, h_last, ckpt8,
                              stream)
    dims = make_dims(batch, seq_len, D, N, 1, exact, ckpt8)
    common = (_ptr(A_log, "A_log", (D, N)),)
    tail = (_ptr(D_vec, "D_vec", (D,), False),)
    if _dense(u, delta, B, C, z, y):
        _check("mss_selective_scan", lib().mss_selective_scan(
            ctypes.byref(dims), _disc(disc), _ptr(u, "u", (M, D)), _ptr(delta, "delta", (M, D)),
            *common, _ptr(B, "B", (M, N)), _ptr(C, "C", (M, N)), *tail,
            _ptr(z, "z", (M, D), False), _ptr(h0, "h0", (batch, D, N), False),
            _ptr(y, "y", (M, D)), _ptr(hc, "h_cache", (batch, Lc, D, N), False),
            _ptr(hl, "h_last", (batch, D, N), False), _stream(stream)))
        return y, hc, hl
    pu, lu = _rows(u, "u", M, D)
    pd, ldd = _rows(delta, "delta", M, D)
    pb, lb = _rows(B, "B", M, N)
    pc, lc = _rows(C, "C", M, N)
    pz, lz = _rows(z, "z", M, D, False)
    py, ly = _rows(y, "y", M, D)
    st = make_strides(lu, lz, ldd, lb, lc, ly)
    _check("mss_selective_scan_strided", lib().mss_selective_scan_strided(
        ctypes.byref(dims), ctypes.byref(st), _disc(disc), pu, pd, *common, pb, pc, *tail, pz,
        _ptr(h0, "h0", (batch, D, N), False), py,
        _ptr(hc, "h_cache", (batch, Lc, D, N), False),
        _ptr(hl, "h_last", (batch, D, N), False), _stream(stream)))
    return y, hc, hl


def mamba1_core(x, w_conv, b_conv, delta, A_log, B, C, D_vec=None, z=None, h0=None, *, batch,
                seq_len, disc, h_cache=False, h_last=False, out=None, stream=None, exact=False,
                ckpt8=False):
    """Fused conv1d + SiLU + selective scan + gate from x.  Returns (y, h_cache, h_last).

    x, delta, z, B, C and ``out`` may be row-strided views (column slices).
    ``exact``: no time split (the plain sequential recurrence, less parallel).
    ``ckpt8``: h_cache is the state entering every 8th step (see selective_scan)."""
    D, N = A_log.shape
    K = w_conv.shape[1]
    M = batch * seq_len
    Lc = ckpt_steps(seq_len) if ckpt8 else seq_len
    y, hc, hl = _scan_outputs(x, batch, seq_len, D, N, out, h_cache, h_last, ckpt8,
                              stream)
    dims = make_dims(batch, seq_len, D, N, K, exact, ckpt8)
    conv = (_ptr(w_conv, "w_conv", (D, K)), _ptr(b_conv, "b_conv", (D,), False))
    if _dense(x, delta, B, C, z, y):
        _check("mss_mamba1_core", lib().mss_mamba1_core(
            ctypes.byref(dims), _disc(disc), _ptr(x, "x", (M, D)), *conv,
            _ptr(delta, "delta", (M, D)), _ptr(A_log, "A_log", (D, N)), _ptr(B, "B", (M, N)),
            _ptr(C, "C", (M, N)), _ptr(D_vec, "D_vec", (D,), False), _ptr(z, "z", (M, D), False),
            _ptr(h0, "h0", (batch, D, N), False), _ptr(y, "y", (M, D)),
            _ptr(hc, "h_cache", (batch, Lc, D, N), False),
            _ptr(hl, "h_last", (batch, D, N), False), _stream(stream)))
        return y, hc, hl
    px, lx = _rows(x, "x", M, D)
    pd, ldd = _rows(delta, "delta", M, D)
    pb, lb = _rows(B, "B", M, N)
    pc, lc = _rows(C, "C", M, N)
    pz, lz = _rows(z, "z", M, D, False)
    py, ly = _rows(y, "y", M, D)
    st = make_strides(lx, lz, ldd, lb, lc, ly)
    _check("mss_mamba1_core_strided", lib().mss_mamba1_core_strided(
        ctypes.byref(dims), ctypes.byref(st), _disc(disc), px, *conv, pd,
        _ptr(A_log, "A_log", (D, N)), pb, pc, _ptr(D_vec, "D_vec", (D,), False), pz,
        _ptr(h0, "h0", (batch, D, N), False), py,
        _ptr(hc, "h_cache", (batch, Lc, D, N), False),
        _ptr(hl, "h_last", (batch, D, N), False), _stream(stream)))
    return y, hc, hl


def selective_step(x, z, delta, A_log, B, C, D_vec, w_conv, b_conv, conv_state, h, *, disc,
                   out=None, stream=None):
    """One decode step; updates ``conv_state`` and ``h`` in place.  Returns y (batch, D)."""
    batch, D = x.shape
    N = A_log.shape[1]
    K = w_conv.shape[1]
    y = out if out is not None else _empty((batch, D), x, stream)
    dims = make_dims(batch, 1, D, N, K)
    _check("mss_selective_step", lib().mss_selective_step(
        ctypes.byref(dims), _disc(disc), _ptr(x, "x", (batch, D)),
        _ptr(z, "z", (batch, D), False), _ptr(delta, "delta", (batch, D)),
        _ptr(A_log, "A_log", (D, N)), _ptr(B, "B", (batch, N)), _ptr(C, "C", (batch, N)),
        _ptr(D_vec, "D_vec", (D,), False), _ptr(w_conv, "w_conv", (D, K)),
        _ptr(b_conv, "b_conv", (D,), False),
        _ptr(conv_state, "conv_state", (batch, K - 1, D), K > 1),
        _ptr(h, "h", (batch, D, N)), _ptr(y, "y", (batch, D)), _stream(stream)))
    return y


def workspace_bytes(op, *, batch, seq_len, d_inner, d_state, d_conv=1, exact=False,
                    ckpt8=False) -> int:
    """Workspace bytes a backward entry point needs (``op``: OP_* constant;
    ``ckpt8``: the scan backward is given the forward's checkpoints)."""
    dims = make_dims(batch, seq_len, d_inner, d_state, d_conv, exact, ckpt8)
    n = ctypes.c_size_t(0)
    _check("mss_workspace_bytes", lib().mss_workspace_bytes(ctypes.byref(dims), op,
                                                             ctypes.byref(n)))
    return int(n.value)


def _workspace(op, like, workspace, stream, **dims):
    """The caller's workspace (a uint8 GPU tensor), or a fresh one of the size
    the library asks for; returns (pointer, bytes, tensor)."""
    need = workspace_bytes(op, **dims)
    if workspace is None:
        if need == 0:
            return None, 0, None
        # 256 bytes of slack so that the pointer can be aligned to 256.
        workspace = _empty(need + 256, like, stream, _torch().uint8)
    if workspace.dtype != _torch().uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 GPU tensor")
    _same_device(workspace, "workspace")
    base = workspace.data_ptr()
    pad = (-base) % 256
    return base + pad, max(0, workspace.numel() - pad), workspace


def time_split(op, *, batch, seq_len, d_inner, d_state, d_conv=1, exact=False) -> int:
    """Segment length in steps of the flattened (channel tile, t) space that
    ``op`` (OP_SELECTIVE_SCAN or OP_SELECTIVE_SCAN_BACKWARD) uses."""
    dims = make_dims(batch, seq_len, d_inner, d_state, d_conv, exact)
    n = ctypes.c_int64(0)
    _check("mss_time_split", lib().mss_time_split(ctypes.byref(dims), op, ctypes.byref(n)))
    return int(n.value)


def ssd_time_split(*, batch, seq_len, n_heads, head_dim, d_state, n_groups=1,
                   exact=False) -> int:
    """Segment length in steps of every (batch row, head) sequence of ssd_scan."""
    dims = make_ssd_dims(batch, seq_len, n_heads, head_dim, d_state, n_groups, exact)
    n = ctypes.c_int64(0)
    _check("mss_ssd_time_split", lib().mss_ssd_time_split(ctypes.byref(dims), ctypes.byref(n)))
    return int(n.value)


def selective_scan_backward(u, delta, A_log, B, C, D_vec, z, h0, dout, *, batch, seq_len, disc,
                            need_dh0=False, workspace=None, stream=None, exact=False,
                            h_ckpt=None):
    """Gradients of ``selective_scan``'s output against ``dout`` (batch*seq_len, D).

    Returns a dict: du, ddelta (M, D); dA_log (D, N); dB, dC (M, N);
    dD (D,) or None when D_vec is None; dz (M, D) or None when z is None;
    dh0 (batch, D, N) when ``need_dh0``.  ``workspace``: optional uint8 GPU
    tensor of at least ``workspace_bytes(OP_SELECTIVE_SCAN_BACKWARD, ...)``
    + 256 bytes (allocated here when omitted).  ``exact``: no time split.
    ``h_ckpt``: the forward's 8-step checkpoints (``h_cache`` of a forward
    call with ``ckpt8=True``), from which every 8-step block starts.
    """
    D, N = A_log.shape
    M = batch * seq_len
    g = {"du": _empty((M, D), u, stream), "ddelta": _empty((M, D), u, stream),
         "dA_log": _empty((D, N), u, stream), "dB": _empty((M, N), u, stream), "dC": _empty((M, N), u, stream),
         "dD": _empty((D,), u, stream) if D_vec is not None else None,
         "dz": _empty((M, D), u, stream) if z is not None else None,
         "dh0": _empty((batch, D, N), u, stream) if need_dh0 else None}
    ck = h_ckpt is not None
    wp, wn, _keep = _workspace(OP_SELECTIVE_SCAN_BACKWARD, u, workspace, stream, batch=batch,
                               seq_len=seq_len, d_inner=D, d_state=N, exact=exact, ckpt8=ck)
    dims = make_dims(batch, seq_len, D, N, 1, exact, ck)
    _check("mss_selective_scan_backward", lib().mss_selective_scan_backward(
        ctypes.byref(dims), _disc(disc), _ptr(u, "u", (M, D)), _ptr(delta, "delta", (M, D)),
        _ptr(A_log, "A_log", (D, N)), _ptr(B, "B", (M, N)), _ptr(C, "C", (M, N)),
        _ptr(D_vec, "D_vec", (D,), False), _ptr(z, "z", (M, D), False),
        _ptr(h0, "h0", (batch, D, N), False),
        _ptr(h_ckpt, "h_ckpt", (batch, ckpt_steps(seq_len), D, N), False),
        _ptr(dout, "dout", (M, D)),
        _ptr(g["du"], "du", (M, D)), _ptr(g["ddelta"], "ddelta", (M, D)),
        _ptr(g["dA_log"], "dA_log", (D, N)), _ptr(g["dB"], "dB", (M, N)),
        _ptr(g["dC"], "dC", (M, N)), _ptr(g["dD"], "dD", (D,), False),
        _ptr(g["dz"], "dz", (M, D), False), _ptr(g["dh0"], "dh0", (batch, D, N), False),
        wp, wn, _stream(stream)))
    return g


def selective_scan_backward_noalloc(u, delta, A_log, B, C, D_vec, z, h0, dout, *, batch,
                                    seq_len, disc, need_dh0=False, out=None, stream=None,
                                    exact=False, h_ckpt=None):
    """``selective_scan_backward`` through the entry point whose workspace is the
    library's static scratch array (for callers that cannot allocate; at most
    NOALLOC_SCRATCH_BYTES of workspace; calls overlapping on one GPU race).
    ``out``: optional dict of preallocated gradient tensors (the keys of the
    result), so that the call itself allocates nothing."""
    D, N = A_log.shape
    M = batch * seq_len
    shapes = {"du": (M, D), "ddelta": (M, D), "dA_log": (D, N), "dB": (M, N), "dC": (M, N),
              "dD": (D,), "dz": (M, D), "dh0": (batch, D, N)}
    want = {"du": True, "ddelta": True, "dA_log": True, "dB": True, "dC": True,
            "dD": D_vec is not None, "dz": z is not None, "dh0": need_dh0}
    out = dict(out or {})
    g = {k: (out[k] if k in out else _empty(shapes[k], u, stream)) if want[k] else None for k in shapes}
    dims = make_dims(batch, seq_len, D, N, 1, exact, h_ckpt is not None)
    _check("mss_selective_scan_backward_noalloc", lib().mss_selective_scan_backward_noalloc(
        ctypes.byref(dims), _disc(disc), _ptr(u, "u", (M, D)), _ptr(delta, "delta", (M, D)),
        _ptr(A_log, "A_log", (D, N)), _ptr(B, "B", (M, N)), _ptr(C, "C", (M, N)),
        _ptr(D_vec, "D_vec", (D,), False), _ptr(z, "z", (M, D), False),
        _ptr(h0, "h0", (batch, D, N), False),
        _ptr(h_ckpt, "h_ckpt", (batch, ckpt_steps(seq_len), D, N), False),
        _ptr(dout, "dout", (M, D)),
        _ptr(g["du"], "du", (M, D)), _ptr(g["ddelta"], "ddelta", (M, D)),
        _ptr(g["dA_log"], "dA_log", (D, N)), _ptr(g["dB"], "dB", (M, N)),
        _ptr(g["dC"], "dC", (M, N)), _ptr(g["dD"], "dD", (D,), False),
        _ptr(g["dz"], "dz", (M, D), False), _ptr(g["dh0"], "dh0", (batch, D, N), False),
        _stream(stream)))
    return g


def conv1d_silu_backward(x, w_conv, b_conv, du, *, batch, seq_len, workspace=None, stream=None):
    """Gradients of ``conv1d_silu`` against ``du``: (dx, dw_conv, db_conv)."""
    D, K = w_conv.shape
    M = batch * seq_len
    dx, dw, db = (_empty(shape, x, stream) for shape in ((M, D), (D, K), (D,)))
    wp, wn, _keep = _workspace(OP_CONV1D_SILU_BACKWARD, x, workspace, stream, batch=batch,
                               seq_len=seq_len, d_inner=D, d_state=1, d_conv=K)
    dims = make_dims(batch, seq_len, D, 1, K)
    _check("mss_conv1d_silu_backward", lib().mss_conv1d_silu_backward(
        ctypes.byref(dims), _ptr(x, "x", (M, D)), _ptr(w_conv, "w_conv", (D, K)),
        _ptr(b_conv, "b_conv", (D,), False), _ptr(du, "du", (M, D)), _ptr(dx, "dx", (M, D)),
        _ptr(dw, "dw_conv", (D, K)), _ptr(db, "db_conv", (D,)), wp, wn, _stream(stream)))
    return dx, dw, db


def ssd_scan(x, dt, A_log, B, C, D_vec=None, dt_bias=None, h0=None, *, batch, seq_len,
             head_dim, d_state, n_groups=1, disc, h_last=False, out=None, stream=None,
             exact=False):
    """Mamba-2 SSD scan: y (batch*seq_len, H*head_dim) and, when ``h_last`` is
    True (or a tensor), the final state (batch, H, head_dim, d_state).
    ``exact``: no time split."""
    H = A_log.shape[0]
    P, N, G = head_dim, d_state, n_groups
    M = batch * seq_len
    y = out if out is not None else _empty((M, H * P), x, stream)
    hl = (h_last if not isinstance(h_last, bool) else
          (_empty((batch, H, P, N), x, stream) if h_last else None))
    dims = make_ssd_dims(batch, seq_len, H, P, N, G, exact)
    _check("mss_ssd_scan", lib().mss_ssd_scan(
        ctypes.byref(dims), _disc(disc), _ptr(x, "x", (M, H * P)), _ptr(dt, "dt", (M, H)),
        _ptr(A_log, "A_log", (H,)), _ptr(B, "B", (M, G * N)), _ptr(C, "C", (M, G * N)),
        _ptr(D_vec, "D_vec", (H,), False), _ptr(dt_bias, "dt_bias", (H,), False),
        _ptr(h0, "h0", (batch, H, P, N), False), _ptr(y, "y", (M, H * P)),
        _ptr(hl, "h_last", (batch, H, P, N), False), _stream(stream)))
    return y, hl


# ---- gated linear recurrence and block norms ---------------------------------

GATES = {"sigmoid": 0, "decay": 1, "log": 2}      # MSS_GATE_*
NORM_KINDS = {"rms": 0, "layer": 1}               # MSS_NORM_*
GATE_ORDERS = {"before": 0, "after": 1}           # MSS_GATE_*_NORM


def _choice(table, value, name):
    try:
        return table[value]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {', '.join(map(repr, table))}") from None


@functools.lru_cache(maxsize=None)
def _dtype_codes():
    torch = _torch()
    return {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}     # MSS_F32, ...


def make_gated_dims(batch, seq_len, d_inner, dtype, gate, gate_scale=8.0) -> GatedDims:
    """Parameter block of the mss_gated_* calls (dtype, gate: MSS_* codes)."""
    return GatedDims(ctypes.sizeof(GatedDims), 0, dtype, gate, batch, seq_len, d_inner,
                     gate_scale, 0)


def make_gated_strides(*strides) -> GatedStrides:
    """Row strides x, r, i, z, y, dx, dr, di, dz (trailing ones may be left out)."""
    return GatedStrides(ctypes.sizeof(GatedStrides), 0, *strides)


def make_norm_dims(rows, width, dtype, res_dtype, kind, order=0, groups=1, eps=1e-6,
                   alpha=1.0) -> NormDims:
    """Parameter block of the norm calls (dtype, res_dtype, kind, order: MSS_* codes)."""
    return NormDims(ctypes.sizeof(NormDims), 0, dtype, res_dtype, kind, order, rows, width, groups,
                    eps, alpha)


def make_norm_strides(*strides) -> NormStrides:
    """Row strides x, z, residual, s, y, ds, dx, dz, dresidual (trailing ones may be left out)."""
    return NormStrides(ctypes.sizeof(NormStrides), 0, *strides)


# The blocks that the calls below pass, which nobody else holds.  They are kept by
# the values in them, so the calls make plain numbers of what they are given
# first (a tensor would be kept by its identity, and alpha = -0.0 taken for 0.0).
_gated_dims = functools.lru_cache(maxsize=1024)(make_gated_dims)
_gated_strides = functools.lru_cache(maxsize=1024)(make_gated_strides)
_norm_dims = functools.lru_cache(maxsize=1024)(make_norm_dims)
_norm_strides = functools.lru_cache(maxsize=1024)(make_norm_strides)


class _Call:
    """Argument checks of one call: the current device, the activation type and the stream."""

    __slots__ = ("torch", "Tensor", "f32", "dev", "like", "dtype", "code", "on")

    def __init__(self, like, name, stream):
        self.torch = torch = _torch()
        self.on = stream
        self.Tensor, self.f32 = torch.Tensor, torch.float32
        if not isinstance(like, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if not like.is_cuda:
            raise ValueError(f"{name} must be on the GPU")
        self.like, self.dtype = like, like.dtype
        self.code = _dtype_codes().get(self.dtype)
        if self.code is None:
            raise TypeError(f"{name} must be float32, bfloat16 or float16, got {like.dtype}")
        self.dev = torch.cuda.current_device()

    def _refuse(self, t, name, dtype, shape):
        if not isinstance(t, self.torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.get_device() != self.dev:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{self.dev}")
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")

    def rows(self, t, name, rows, cols, dtype=None, required=True):
        """(pointer, row stride) of a (rows, cols) activation whose rows may be strided."""
        if t is None:
            if required:
                raise ValueError(f"{name} is required")
            return None, cols
        dtype = dtype or self.dtype
        if (not isinstance(t, self.Tensor) or t.dtype is not dtype or t.get_device() != self.dev
                or t.shape != (rows, cols)):
            self._refuse(t, name, dtype, (rows, cols))
        row, col = t.stride()
        if col != 1 and cols > 1 and rows > 0:
            raise ValueError(f"{name}: columns must be contiguous")
        return t.data_ptr() or None, row if rows > 1 else cols

    def dense(self, t, name, shape, dtype=None, required=False):
        """Pointer of a contiguous tensor (float32 unless said otherwise)."""
        if t is None:
            if required:
                raise ValueError(f"{name} is required")
            return None
        dtype = dtype or self.f32
        if (not isinstance(t, self.Tensor) or t.dtype is not dtype or t.get_device() != self.dev
                or t.shape != shape):
            self._refuse(t, name, dtype, shape)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr() or None

    def empty(self, shape, dtype=None, like=None):
        """An uninitialised tensor; ``like``: one that may be of its shape and type (cheaper)."""
        if self.on is not None:
            return _empty(shape, self.like, self.on, dtype or self.dtype)
        dtype, like = dtype or self.dtype, self.like if like is None else like
        if like.shape == shape and like.dtype is dtype and like.is_contiguous():
            return self.torch.empty_like(like)
        return self.torch.empty(shape, dtype=dtype, device=like.device)

    def output(self, t, name, rows, cols, dtype=None, like=None):
        """(tensor, pointer, row stride) of an output: the caller's, or a fresh one."""
        if t is None:
            t = self.empty((rows, cols), dtype, like)
            return t, t.data_ptr() or None, cols
        return (t, *self.rows(t, name, rows, cols, dtype))

    def stream(self):
        """The handle of the call's stream (the current stream's where none is given)."""
        if self.on is None:
            return self.torch._C._cuda_getCurrentRawStream(self.dev)
        return _stream(self.on)

    def workspace(self, need, workspace):
        """(pointer, bytes, tensor) of the caller's workspace, or of a fresh one."""
        if workspace is None:
            if need == 0:
                return None, 0, None
            workspace = self.empty((need + 256,), self.torch.uint8)
        elif (not isinstance(workspace, self.torch.Tensor)
              or workspace.dtype != self.torch.uint8 or workspace.get_device() != self.dev
              or not workspace.is_contiguous()):
            raise TypeError("workspace must be a contiguous uint8 tensor on the current GPU")
        base = workspace.data_ptr()
        pad = (-base) % 256
        return base + pad, max(0, workspace.numel() - pad), workspace


def gated_workspace_bytes(op, *, batch, seq_len, d_inner, gate) -> int:
    """Workspace bytes of ``gated_scan`` (OP_GATED_SCAN) or ``gated_scan_backward``
    (OP_GATED_SCAN_BACKWARD)."""
    return _gated_need(op, _index(batch), _index(seq_len), _index(d_inner), _choice(GATES, gate, "gate"))


@functools.lru_cache(maxsize=1024)
def _gated_need(op, batch, seq_len, d_inner, gate):
    dims = make_gated_dims(batch, seq_len, d_inner, 0, gate)
    n = ctypes.c_size_t(0)
    _check("mss_gated_workspace_bytes",
           lib().mss_gated_workspace_bytes(ctypes.byref(dims), op, ctypes.byref(n)))
    return int(n.value)


def norm_workspace_bytes(op, *, rows, width, groups=1) -> int:
    """Workspace bytes of ``add_norm_backward`` (OP_ADD_NORM_BACKWARD) or
    ``gated_norm_backward`` (OP_GATED_NORM_BACKWARD)."""
    return _norm_need(op, _index(rows), _index(width), _index(groups))


@functools.lru_cache(maxsize=1024)
def _norm_need(op, rows, width, groups):
    dims = make_norm_dims(rows, width, 0, 0, 0, 0, groups)
    n = ctypes.c_size_t(0)
    _check("mss_norm_workspace_bytes",
           lib().mss_norm_workspace_bytes(ctypes.byref(dims), op, ctypes.byref(n)))
    return int(n.value)


def _ref(block):
    return ctypes.byref(block)


def _flag(t, shape, call, like=None):
    """An optional float32 output given as False / True (allocate) or a tensor."""
    if isinstance(t, bool):
        return call.empty(shape, call.f32, like) if t else None
    return t


def _gated_inputs(c, x, r, i, decay, z, rows, D, gate):
    if gate != "decay" and (i is not None or decay is not None):
        raise ValueError(f"i and decay belong to gate='decay', not {gate!r}")
    return (c.rows(x, "x", rows, D), c.rows(r, "r", rows, D),
            c.rows(i, "i", rows, D, required=gate == "decay"),
            c.dense(decay, "decay", (D,), required=gate == "decay"),
            c.rows(z, "z", rows, D, required=False))


def _reset(c, reset, rows):
    if isinstance(reset, c.Tensor) and reset.dtype is c.torch.bool:
        reset = reset.view(c.torch.uint8)
    return c.dense(reset, "reset", (rows,), c.torch.uint8)


def gated_ckpt_steps(seq_len) -> int:
    """Rows of gated_scan's checkpoints: ceil(seq_len / 64)."""
    return -(-seq_len // GATED_CKPT_STEPS)


def gated_scan(x, r, i=None, decay=None, z=None, h0=None, reset=None, *, batch, seq_len, gate,
               gate_scale=8.0, h_ckpt=False, h_last=False, out=None, workspace=None, stream=None):
    """Gated linear recurrence h_t = v_t + a_t h_{t-1}, y_t = h_t SiLU(z_t) (h_t without z).
    Returns (y, h_ckpt, h_last).

    ``gate``: "sigmoid" (a = sigma(r), v = (1 - a) x), "decay" (a = exp(-gate_scale
    softplus(decay) sigma(r)), v = sqrt(1 - a^2) sigma(i) x) or "log" (a = exp(r), v = x).
    x, r, i, z, out: (batch*seq_len, D) float32, bfloat16 or float16, all the same, rows may
    be strided; decay (D,), h0 (batch, D) float32; reset (batch*seq_len,) uint8 or bool: where
    set, the state carried into that step is dropped.
    ``h_ckpt`` / ``h_last``: False (skip), True (allocate) or an output tensor: the state
    entering every 64th step (batch, ceil(seq_len/64), D), which the backward pass takes, and
    the final state (batch, D), both float32.
    ``workspace``: uint8 GPU tensor of at least ``gated_workspace_bytes(OP_GATED_SCAN, ...)``
    + 256 bytes (allocated here when omitted)."""
    batch, seq_len, gate_scale = _index(batch), _index(seq_len), float(gate_scale)
    D, M = x.shape[-1], batch * seq_len
    c = _Call(x, "x", stream)
    code = _choice(GATES, gate, "gate")
    (px, lx), (pr, lr), (pi, li), pdec, (pz, lz) = _gated_inputs(c, x, r, i, decay, z, M, D, gate)
    y, py, ly = c.output(out, "out", M, D)
    ck = _flag(h_ckpt, (batch, gated_ckpt_steps(seq_len), D), c)
    hl = _flag(h_last, (batch, D), c, h0)
    need = _gated_need(OP_GATED_SCAN, batch, seq_len, D, code)
    wp, wn, _keep = c.workspace(need, workspace)
    _check("mss_gated_scan", lib().mss_gated_scan(
        _ref(_gated_dims(batch, seq_len, D, c.code, code, gate_scale)),
        _ref(_gated_strides(lx, lr, li, lz, ly)), px, pr, pi, pdec, pz,
        c.dense(h0, "h0", (batch, D)), _reset(c, reset, M), py,
        c.dense(ck, "h_ckpt", (batch, gated_ckpt_steps(seq_len), D)),
        c.dense(hl, "h_last", (batch, D)), wp, wn, c.stream()))
    return y, ck, hl


def gated_scan_backward(x, r, i, decay, z, reset, h_ckpt, dout, *, batch, seq_len, gate,
                        gate_scale=8.0, dh_last=None, need_dh0=False, out=None, workspace=None,
                        stream=None):
    """Gradients of ``gated_scan`` against ``dout`` (batch*seq_len, D), the gradient of y, and
    ``dh_last`` (batch, D), that of h_last (0 when None).

    ``h_ckpt``: the forward's checkpoints (a call with the same inputs and ``h_ckpt=True``).
    Returns a dict: dx, dr, di, dz (M, D) in x's type, ddecay (D,) and dh0 (batch, D) float32;
    di and ddecay are None unless gate is "decay", dz is None when z is, dh0 unless
    ``need_dh0``.  ``out``: optional dict of output tensors for some of them (dx, dr, di, dz
    may be row-strided).  ``workspace`` as in gated_scan, with OP_GATED_SCAN_BACKWARD."""
    batch, seq_len, gate_scale = _index(batch), _index(seq_len), float(gate_scale)
    D, M = x.shape[-1], batch * seq_len
    c = _Call(x, "x", stream)
    code = _choice(GATES, gate, "gate")
    (px, lx), (pr, lr), (pi, li), pdec, (pz, lz) = _gated_inputs(c, x, r, i, decay, z, M, D, gate)
    has_decay, MD, f32 = gate == "decay", (M, D), c.f32
    g, at = _outputs(c, out, {
        "dx": (True, MD, None, x, True), "dr": (True, MD, None, r, True),
        "di": (has_decay, MD, None, i, True), "ddecay": (has_decay, (D,), f32, decay, False),
        "dz": (z is not None, MD, None, z, True),
        "dh0": (need_dh0, (batch, D), f32, dh_last, False)})
    (pdx, ldx), (pdr, ldr), (pdi, ldi), (pdz, ldz) = at["dx"], at["dr"], at["di"], at["dz"]
    po, lo = c.rows(dout, "dout", M, D)
    need = _gated_need(OP_GATED_SCAN_BACKWARD, batch, seq_len, D, code)
    wp, wn, _keep = c.workspace(need, workspace)
    _check("mss_gated_scan_backward", lib().mss_gated_scan_backward(
        _ref(_gated_dims(batch, seq_len, D, c.code, code, gate_scale)),
        _ref(_gated_strides(lx, lr, li, lz, lo, ldx, ldr, ldi, ldz)), px, pr, pi, pdec, pz,
        _reset(c, reset, M),
        c.dense(h_ckpt, "h_ckpt", (batch, gated_ckpt_steps(seq_len), D), required=True), po,
        c.dense(dh_last, "dh_last", (batch, D)), pdx, pdr, pdi,
        at["ddecay"][0], pdz, at["dh0"][0], wp, wn, c.stream()))
    return g


def _outputs(c, out, results):
    """Results, each given as (wanted, shape, dtype, a tensor like it, rows may be strided):
    the caller's tensors, fresh ones, or None where not wanted; and their (pointer, row
    stride)."""
    if out:
        unknown = [k for k in out if k not in results]
        if unknown:
            raise ValueError(f"out has no place for {', '.join(unknown)}")
    g, at = {}, {}
    for k, (wanted, shape, dtype, like, strided) in results.items():
        given = out.get(k) if out and wanted else None
        if not wanted:
            g[k], at[k] = None, (None, shape[-1])
        elif given is None:
            g[k] = t = c.empty(shape, dtype, like)
            at[k] = t.data_ptr() or None, shape[-1]
        else:
            g[k] = given
            at[k] = (c.rows(given, k, *shape, dtype) if strided else
                     (c.dense(given, k, shape, dtype), shape[-1]))
    return g, at


def gated_step(x, r, i, decay, z, h, *, gate, gate_scale=8.0, out=None, stream=None):
    """One token per sequence of ``gated_scan``: x, r, i, z (batch, D); updates ``h``
    (batch, D) float32 in place.  Returns y (batch, D)."""
    batch, D = x.shape
    c, gate_scale = _Call(x, "x", stream), float(gate_scale)
    code = _choice(GATES, gate, "gate")
    (px, lx), (pr, lr), (pi, li), pdec, (pz, lz) = _gated_inputs(c, x, r, i, decay, z, batch, D,
                                                                 gate)
    y, py, ly = c.output(out, "out", batch, D)
    _check("mss_gated_step", lib().mss_gated_step(
        _ref(_gated_dims(batch, 1, D, c.code, code, gate_scale)),
        _ref(_gated_strides(lx, lr, li, lz, ly)), px, pr, pi, pdec, pz,
        c.dense(h, "h", (batch, D), required=True), py, c.stream()))
    return y


def _res_code(c, dtype, name):
    if dtype is not c.dtype and dtype is not c.f32:
        raise TypeError(f"{name} must be {c.dtype} or float32, got {dtype}")
    return _dtype_codes()[dtype]


def add_norm(x, residual, weight, bias=None, scale=None, *, kind="rms", eps=1e-6, alpha=1.0,
             res_dtype=None, out=None, residual_out=None, stream=None):
    """Before a block: s = residual + alpha scale x, y = norm(s) weight + bias.  Returns (y, s).

    x (M, D) float32, bfloat16 or float16; residual (M, D) of x's type or float32, or None (0);
    weight, bias, scale (D,) float32; ``kind``: "rms" or "layer".  s has the residual's type
    (``res_dtype``, x's by default, where residual is None) and the norm reads s as that type
    holds it.  ``residual_out`` may be ``residual`` itself: updated in place.  Rows of x,
    residual and the outputs may be strided."""
    M, D = x.shape
    c, eps, alpha = _Call(x, "x", stream), float(eps), float(alpha) + 0.0
    rt = (residual.dtype if residual is not None else
          residual_out.dtype if residual_out is not None else res_dtype or c.dtype)
    rc = _res_code(c, rt, "the residual stream")
    s, ps, ls = c.output(residual_out, "residual_out", M, D, rt, residual)
    px, lx = c.rows(x, "x", M, D)
    pr, lr = c.rows(residual, "residual", M, D, rt, False)
    y, py, ly = c.output(out, "out", M, D)
    _check("mss_add_norm", lib().mss_add_norm(
        _ref(_norm_dims(M, D, c.code, rc, _choice(NORM_KINDS, kind, "kind"), 0, 1, eps, alpha)),
        _ref(_norm_strides(lx, 0, lr, ls, ly)), px, pr,
        c.dense(weight, "weight", (D,), required=True), c.dense(bias, "bias", (D,)),
        c.dense(scale, "scale", (D,)), ps, py, c.stream()))
    return y, s


def add_norm_backward(s, weight, dy, ds=None, x=None, scale=None, *, bias=False, kind="rms",
                      eps=1e-6, alpha=1.0, need_dx=True, out=None, workspace=None, stream=None):
    """Gradients of ``add_norm`` against ``dy`` (M, D), the gradient of y, and ``ds`` (M, D),
    what else reaches s (0 when None).

    ``s``: the forward's residual stream; ``x``: the forward's x, needed with ``scale``.
    Returns a dict: dx in dy's type (None unless ``need_dx``), dresidual in s's, dweight,
    dbias (with ``bias``) and dscale (with ``scale``) float32.  ``out`` and ``workspace`` as in
    gated_scan_backward (``norm_workspace_bytes(OP_ADD_NORM_BACKWARD, ...)``)."""
    M, D = dy.shape
    c, eps, alpha = _Call(dy, "dy", stream), float(eps), float(alpha) + 0.0
    rc = _res_code(c, s.dtype, "s")
    g, at = _outputs(c, out, {
        "dx": (need_dx, (M, D), None, dy, True), "dresidual": (True, (M, D), s.dtype, s, True),
        "dweight": (True, (D,), c.f32, weight, False),
        "dbias": (bool(bias), (D,), c.f32, weight, False),
        "dscale": (scale is not None, (D,), c.f32, scale, False)})
    ps, ls = c.rows(s, "s", M, D, s.dtype)
    po, lo = c.rows(dy, "dy", M, D)
    pds, lds = c.rows(ds, "ds", M, D, s.dtype, False)
    px, lx = c.rows(x, "x", M, D, required=scale is not None)
    (pdx, ldx), (pdr, ldr) = at["dx"], at["dresidual"]
    wp, wn, _keep = c.workspace(_norm_need(OP_ADD_NORM_BACKWARD, M, D, 1), workspace)
    _check("mss_add_norm_backward", lib().mss_add_norm_backward(
        _ref(_norm_dims(M, D, c.code, rc, _choice(NORM_KINDS, kind, "kind"), 0, 1, eps, alpha)),
        _ref(_norm_strides(lx, 0, 0, ls, lo, lds, ldx, 0, ldr)), ps,
        c.dense(weight, "weight", (D,), required=True), po, pds, px,
        c.dense(scale, "scale", (D,)), pdx, pdr, at["dweight"][0], at["dbias"][0], at["dscale"][0],
        wp, wn, c.stream()))
    return g


def gated_norm(x, z, weight, bias=None, residual=None, scale=None, *, groups=1, order="before",
               kind="rms", eps=1e-6, alpha=1.0, out=None, stream=None):
    """After a block: n = norm(x SiLU(z)) weight + bias (``order="before"``) or
    n = (norm(x) weight + bias) SiLU(z) (``order="after"``); y = alpha scale n, plus residual
    when given.  Returns y.

    x, z, residual, y (M, D) float32, bfloat16 or float16, all the same, rows may be strided;
    z, residual may be None; weight, bias, scale (D,) float32; the norm runs over each of
    ``groups`` equal groups of channels."""
    M, D = x.shape
    c, groups, eps, alpha = _Call(x, "x", stream), _index(groups), float(eps), float(alpha) + 0.0
    px, lx = c.rows(x, "x", M, D)
    pz, lz = c.rows(z, "z", M, D, required=False)
    pr, lr = c.rows(residual, "residual", M, D, required=False)
    y, py, ly = c.output(out, "out", M, D)
    _check("mss_gated_norm", lib().mss_gated_norm(
        _ref(_norm_dims(M, D, c.code, c.code, _choice(NORM_KINDS, kind, "kind"),
                            _choice(GATE_ORDERS, order, "order"), groups, eps, alpha)),
        _ref(_norm_strides(lx, lz, lr, 0, ly)), px, pz,
        c.dense(weight, "weight", (D,), required=True), c.dense(bias, "bias", (D,)), pr,
        c.dense(scale, "scale", (D,)), py, c.stream()))
    return y


def gated_norm_backward(x, z, weight, bias, scale, dout, *, groups=1, order="before", kind="rms",
                        eps=1e-6, alpha=1.0, out=None, workspace=None, stream=None):
    """Gradients of ``gated_norm`` against ``dout`` (M, D) (the residual's is dout itself).

    Returns a dict: dx, dz in x's type (dz None when z is), dweight, dbias (with ``bias``) and
    dscale (with ``scale``) float32.  ``out`` and ``workspace`` as in gated_scan_backward
    (``norm_workspace_bytes(OP_GATED_NORM_BACKWARD, ...)``)."""
    M, D = x.shape
    c, groups, eps, alpha = _Call(x, "x", stream), _index(groups), float(eps), float(alpha) + 0.0
    g, at = _outputs(c, out, {
        "dx": (True, (M, D), None, x, True), "dz": (z is not None, (M, D), None, z, True),
        "dweight": (True, (D,), c.f32, weight, False),
        "dbias": (bias is not None, (D,), c.f32, bias, False),
        "dscale": (scale is not None, (D,), c.f32, scale, False)})
    px, lx = c.rows(x, "x", M, D)
    pz, lz = c.rows(z, "z", M, D, required=False)
    po, lo = c.rows(dout, "dout", M, D)
    (pdx, ldx), (pdz, ldz) = at["dx"], at["dz"]
    wp, wn, _keep = c.workspace(_norm_need(OP_GATED_NORM_BACKWARD, M, D, groups), workspace)
    _check("mss_gated_norm_backward", lib().mss_gated_norm_backward(
        _ref(_norm_dims(M, D, c.code, c.code, _choice(NORM_KINDS, kind, "kind"),
                            _choice(GATE_ORDERS, order, "order"), groups, eps, alpha)),
        _ref(_norm_strides(lx, lz, 0, 0, lo, 0, ldx, ldz)), px, pz,
        c.dense(weight, "weight", (D,), required=True), c.dense(bias, "bias", (D,)),
        c.dense(scale, "scale", (D,)), po, pdx, pdz, at["dweight"][0], at["dbias"][0], at["dscale"][0],
        wp, wn, c.stream()))
    return g


# ---- the ends of a model -------------------------------------------------------

def make_embed_dims(rows, vocab, width, dtype, out_dtype, id_bytes, scale=1.0, accumulate=False) -> EmbedDims:
    """Parameter block of the embedding calls (dtype: the table's, out_dtype: the rows', MSS_* codes)."""
    return EmbedDims(ctypes.sizeof(EmbedDims), EMBED_ACCUMULATE if accumulate else 0, dtype, out_dtype,
                     id_bytes, 0, rows, vocab, width, scale, 0)


def make_embed_strides(weight, y) -> EmbedStrides:
    return EmbedStrides(ctypes.sizeof(EmbedStrides), 0, weight, y)


def make_head_dims(rows, vocab, width, dtype, id_bytes, logit_scale=1.0) -> HeadDims:
    """Parameter block of the head calls (dtype: MSS_* code)."""
    return HeadDims(ctypes.sizeof(HeadDims), 0, dtype, id_bytes, rows, vocab, width, logit_scale, 0)


def make_head_strides(*strides) -> HeadStrides:
    """Row strides x, weight, dx, dweight (trailing ones may be left out)."""
    return HeadStrides(ctypes.sizeof(HeadStrides), 0, *strides)


_embed_dims = functools.lru_cache(maxsize=1024)(make_embed_dims)
_embed_strides = functools.lru_cache(maxsize=1024)(make_embed_strides)
_head_dims = functools.lru_cache(maxsize=1024)(make_head_dims)
_head_strides = functools.lru_cache(maxsize=1024)(make_head_strides)


def embed_workspace_bytes(*, rows, vocab, width) -> int:
    """Workspace bytes of ``embedding_backward``."""
    return _embed_need(_index(rows), _index(vocab), _index(width))


@functools.lru_cache(maxsize=1024)
def _embed_need(rows, vocab, width):
    dims = make_embed_dims(rows, vocab, width, 0, 0, 8)
    n = ctypes.c_size_t(0)
    _check("mss_embed_workspace_bytes", lib().mss_embed_workspace_bytes(ctypes.byref(dims), ctypes.byref(n)))
    return int(n.value)


def head_workspace_bytes(op, *, rows, vocab, width, dtype) -> int:
    """Workspace bytes of ``head_loss`` (OP_HEAD_LOSS) or ``head_loss_backward``
    (OP_HEAD_LOSS_BACKWARD); ``dtype``: the torch type of x."""
    return _head_need(op, _index(rows), _index(vocab), _index(width), _dtype_code(dtype, "dtype"))


@functools.lru_cache(maxsize=1024)
def _head_need(op, rows, vocab, width, code):
    dims = make_head_dims(rows, vocab, width, code, 8)
    n = ctypes.c_size_t(0)
    _check("mss_head_workspace_bytes", lib().mss_head_workspace_bytes(ctypes.byref(dims), op, ctypes.byref(n)))
    return int(n.value)


def clip_workspace_bytes(count) -> int:
    """Workspace bytes of ``grad_norm`` and ``clip_grads`` for ``count`` tensors."""
    return _clip_need(_index(count))


@functools.lru_cache(maxsize=1024)
def _clip_need(count):
    n = ctypes.c_size_t(0)
    _check("mss_clip_workspace_bytes", lib().mss_clip_workspace_bytes(count, ctypes.byref(n)))
    return int(n.value)


def _dtype_code(dtype, name):
    code = _dtype_codes().get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def _ids(c, t, name, rows):
    """(pointer, bytes of an id) of a tensor of token ids."""
    if not isinstance(t, c.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is c.torch.int64:
        return c.dense(t, name, (rows,), c.torch.int64, True), 8
    return c.dense(t, name, (rows,), c.torch.int32, True), 4


def _id_rows(ids, name):
    """The number of ids, before there is anything to check them against."""
    if not isinstance(ids, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if ids.dim() != 1:
        raise ValueError(f"{name} must have one dimension, got shape {tuple(ids.shape)}")
    return ids.shape[0]


def embedding(ids, weight, *, scale=1.0, out_dtype=None, out=None, stream=None):
    """Rows of a table by token: y_m = scale weight[ids_m].  Returns y (M, D).

    ids (M,) int64 or int32; one outside 0 .. V-1 marks a padded place (or a token that another
    shard of the table holds): its row is zeros.  weight (V, D) float32, bfloat16 or float16;
    y of ``out_dtype`` (weight's by default): weight's type or float32, or any of the three where
    weight is float32.  Rows of weight and out may be strided."""
    M = _id_rows(ids, "ids")
    c, scale = _Call(weight, "weight", stream), float(scale) + 0.0
    V, D = weight.shape
    yt = out.dtype if out is not None else out_dtype or c.dtype
    yc = _dtype_code(yt, "the output")
    if yc and c.code and yc != c.code:
        raise TypeError(f"the output must be {c.dtype} or float32, got {yt}")
    pid, nid = _ids(c, ids, "ids", M)
    pw, lw = c.rows(weight, "weight", V, D)
    y, py, ly = c.output(out, "out", M, D, yt)
    _check("mss_embedding", lib().mss_embedding(
        _ref(_embed_dims(M, V, D, c.code, yc, nid, scale)), _ref(_embed_strides(lw, ly)), pid, pw, py,
        c.stream()))
    return y


def embedding_backward(ids, dy, *, vocab, scale=1.0, dtype=None, accumulate=False, out=None,
                       workspace=None, stream=None):
    """Gradient of ``embedding`` against dy (M, D): dweight (vocab, D), in ``dtype`` (dy's by default).

    Row v is scale times the sum of the dy of the places where v stands, in their order, in fp32;
    zeros where it does not occur.  ``accumulate``: the sums are added to ``out``, which is then
    required, and its other rows are left as they are (a table tied to the head: ``out`` holds
    the dweight of ``head_loss_backward``).  dy and dweight of the same type, or one of them
    float32; rows of dy and out may be strided.  ``workspace``: uint8 GPU tensor of at least
    ``embed_workspace_bytes(...)`` + 256 bytes (allocated here when omitted)."""
    M, V = _id_rows(ids, "ids"), _index(vocab)
    c, scale = _Call(dy, "dy", stream), float(scale) + 0.0
    D = dy.shape[-1]
    wt = out.dtype if out is not None else dtype or c.dtype
    wc = _dtype_code(wt, "dweight")
    if wc and c.code and wc != c.code:
        raise TypeError(f"dweight must be {c.dtype} or float32, got {wt}")
    if accumulate and out is None:
        raise ValueError("accumulate needs out, the gradient to add to")
    if V < 0:
        raise ValueError(f"vocab must not be negative, got {V}")
    pid, nid = _ids(c, ids, "ids", M)
    pd, ld = c.rows(dy, "dy", M, D)
    dw, pw, lw = c.output(out, "out", V, D, wt)
    wp, wn, _keep = c.workspace(_embed_need(M, V, D), workspace)
    _check("mss_embedding_backward", lib().mss_embedding_backward(
        _ref(_embed_dims(M, V, D, wc, c.code, nid, scale, bool(accumulate))), _ref(_embed_strides(lw, ld)),
        pid, pd, pw, wp, wn, c.stream()))
    return dw


def head_loss(x, weight, targets, *, logit_scale=1.0, out=None, workspace=None, stream=None):
    """Softmax cross entropy of the logits logit_scale x weight^T, which are not kept.
    Returns (loss, lse), both (M,) float32.

    x (M, D), weight (V, D) float32, bfloat16 or float16, both the same, rows may be strided;
    targets (M,) int64 or int32.  lse_m is the log of the sum of the exponentials, loss_m = lse_m
    minus the target's logit; a target outside 0 .. V-1 marks a padded row, whose loss is 0 (its lse
    is that of its logits).
    ``out``: optional pair of output tensors.  ``workspace``: uint8 GPU tensor of at least
    ``head_workspace_bytes(OP_HEAD_LOSS, ...)`` + 256 bytes (allocated here when omitted)."""
    c, logit_scale = _Call(x, "x", stream), float(logit_scale) + 0.0
    M, D = x.shape
    V = weight.shape[0]
    px, lx = c.rows(x, "x", M, D)
    pw, lw = c.rows(weight, "weight", V, D)
    pt, nt = _ids(c, targets, "targets", M)
    loss, lse = out if out is not None else (c.empty((M,), c.f32), c.empty((M,), c.f32))
    wp, wn, _keep = c.workspace(_head_need(OP_HEAD_LOSS, M, V, D, c.code), workspace)
    _check("mss_head_loss", lib().mss_head_loss(
        _ref(_head_dims(M, V, D, c.code, nt, logit_scale)), _ref(_head_strides(lx, lw)), px, pw, pt,
        c.dense(loss, "loss", (M,), required=True), c.dense(lse, "lse", (M,), required=True), wp, wn,
        c.stream()))
    return loss, lse


def head_loss_backward(x, weight, targets, lse, dloss, dlse=None, *, logit_scale=1.0, need_dx=True,
                       need_dweight=True, out=None, workspace=None, stream=None):
    """Gradients of ``head_loss`` against dloss (M,) and dlse (M,) (0 when None), float32.

    ``lse``: the forward's.  Returns a dict: dx (M, D) and dweight (V, D) in x's type, None where
    not needed.  A padded row takes no part: its dx is 0, and its x, dloss and dlse are not used.
    A vocabulary in shards: ``lse`` is the log sum over all shards; a row whose target is in another
    shard is given any token of this one, dloss 0 and dlse its dloss + dlse (as a padded row it would
    lose this shard's part); dx is the sum over the shards.
    In 2-byte types the gradient of each logit is rounded once before the products that make
    dx and dweight.  ``out`` and ``workspace`` as in gated_scan_backward
    (``head_workspace_bytes(OP_HEAD_LOSS_BACKWARD, ...)``)."""
    c, logit_scale = _Call(x, "x", stream), float(logit_scale) + 0.0
    M, D = x.shape
    V = weight.shape[0]
    px, lx = c.rows(x, "x", M, D)
    pw, lw = c.rows(weight, "weight", V, D)
    pt, nt = _ids(c, targets, "targets", M)
    g, at = _outputs(c, out, {"dx": (need_dx, (M, D), None, x, True),
                              "dweight": (need_dweight, (V, D), None, weight, True)})
    (pdx, ldx), (pdw, ldw) = at["dx"], at["dweight"]
    need = _head_need(OP_HEAD_LOSS_BACKWARD, M, V, D, c.code)
    wp, wn, _keep = c.workspace(need, workspace)
    _check("mss_head_loss_backward", lib().mss_head_loss_backward(
        _ref(_head_dims(M, V, D, c.code, nt, logit_scale)), _ref(_head_strides(lx, lw, ldx, ldw)), px, pw, pt,
        c.dense(lse, "lse", (M,), required=True), c.dense(dloss, "dloss", (M,), required=True),
        c.dense(dlse, "dlse", (M,)), pdx, pdw, wp, wn, c.stream()))
    return g


def _refuse_tensor(c, t, name):
    if not isinstance(t, c.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _dtype_codes():
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.get_device() != c.dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{c.dev}")
    raise ValueError(f"{name} must be contiguous")


def _tensor_list(c, grads, out):
    """The mss_tensors of the tensors that are not None, with their outputs: (bytes, how many)."""
    if len(out) != len(grads):
        raise ValueError(f"out has {len(out)} tensors, grads {len(grads)}")
    codes, dev, Tensor = _dtype_codes(), c.dev, c.Tensor
    flat = []
    for k, g in enumerate(grads):
        o = out[k]
        if g is None:
            if o is not None:
                raise ValueError(f"grads[{k}] is None, out[{k}] is not")
            continue
        code = codes.get(g.dtype) if isinstance(g, Tensor) else None
        if code is None or g.get_device() != dev or not g.is_contiguous():
            _refuse_tensor(c, g, f"grads[{k}]")
        at = g.data_ptr()
        if o is g:
            flat += at, at, g.numel(), code, code
            continue
        to = codes.get(o.dtype) if isinstance(o, Tensor) else None
        if to is None or o.get_device() != dev or not o.is_contiguous():
            _refuse_tensor(c, o, f"out[{k}]")
        if o.shape != g.shape:
            raise ValueError(f"out[{k}]: expected shape {tuple(g.shape)}, got {tuple(o.shape)}")
        if to != code and to != 0:
            raise TypeError(f"out[{k}] must be {g.dtype} or float32, got {o.dtype}")
        flat += at, o.data_ptr(), g.numel(), code, to
    n = len(flat) // 5
    return struct.pack("PPqii" * n, *flat), n


def _list_call(grads, stream):
    like = next((g for g in grads if g is not None), None)
    if like is None:
        raise ValueError("grads holds no tensor")
    return _Call(like, "grads", stream)


def grad_norm(grads, *, scale=1.0, out=None, workspace=None, stream=None):
    """scale times the 2-norm of all elements of a list of tensors: a float32 tensor without dimensions.

    Tensors are float32, bfloat16 or float16, of any sizes, dense; None is passed over.  Squares
    and sums are fp64.  ``workspace``: uint8 GPU tensor of at least
    ``clip_workspace_bytes(len(grads))`` + 256 bytes (allocated here when omitted)."""
    grads = list(grads)
    c, scale = _list_call(grads, stream), float(scale)
    entries, n = _tensor_list(c, grads, grads)
    norm = out if out is not None else c.empty((), c.f32)
    wp, wn, _keep = c.workspace(_clip_need(n), workspace)
    _check("mss_grad_norm", lib().mss_grad_norm(entries, n, scale, c.dense(norm, "out", (), required=True),
                                                wp, wn, c.stream()))
    return norm


def clip_grads(grads, max_norm, *, scale=1.0, out=None, norm=None, workspace=None, stream=None):
    """The norm of ``grad_norm`` and the tensors times scale min(1, max_norm / norm).
    Returns (tensors, norm).

    ``scale``: what the gradients are to be multiplied with first (1 / the loss scale, or 1 / the
    number of micro-batches in them).  The tensors are updated in place, or written to ``out``, a
    list of tensors of their types or float32 (each may be its input).  Where a value is infinite or
    NaN they are left as they are (``out``: copied), so that the caller can look at the norm, which
    is not finite then, and pass over the step.  A tensor may stand in the list once.  ``norm``:
    optional output tensor without dimensions.  ``workspace`` as in ``grad_norm``."""
    grads = list(grads)
    c, scale, max_norm = _list_call(grads, stream), float(scale), float(max_norm)
    out = grads if out is None else list(out)
    entries, n = _tensor_list(c, grads, out)
    norm = norm if norm is not None else c.empty((), c.f32)
    wp, wn, _keep = c.workspace(_clip_need(n), workspace)
    _check("mss_clip_grads", lib().mss_clip_grads(entries, n, scale, max_norm,
                                                  c.dense(norm, "norm", (), required=True), wp, wn,
                                                  c.stream()))
    return out, norm
