"""Thin Python binding over libfa's C ABI (include/fa.h).

Argument marshalling only: every step of the attention path runs in libfa's
CUDA kernels.  torch supplies device memory and the current stream.  If the
library has not been built, every call raises: there is no other code path.

API
  fwd(q, k, v, o, lse, causal, scale)               -> None   (fa_fwd)
  bwd_preprocess(o, do, delta)                       -> None   (fa_bwd_preprocess)
  bwd(q, k, v, do, lse, delta, dq, dk, dv, causal, scale) -> None (fa_bwd)
  attention_fwd(q, k, v, causal, scale)             -> (o, lse)   allocates outputs
  attention_bwd(q, k, v, o, lse, do, causal, scale) -> (dq, dk, dv)
  attention(q, k, v, causal, scale)                 -> o with autograd; double
                                                       backward raises
Tensors are CUDA [B, H, N, D] with unit last stride (any other strides), all of
one dtype (float32, float16, bfloat16); lse and delta are contiguous float32
[B, H, N].

General problems (fa_fwd_ex / fa_bwd_ex): K and V may have fewer heads than Q
(Hq % Hkv == 0) and another length; sequences may be packed with cu_seqlens;
attention weights may be dropped (Philox4x32-10 mask, regenerated by the
backward from the same seed and offset, or stored by the forward into a
keep-mask buffer that the backward reads).
  fwd_ex(q, k, v, o, lse, causal, scale, *, cu_seqlens_q, cu_seqlens_k,
         max_seqlen_q, max_seqlen_k, dropout_p, seed, offset,
         dropout_mask)                                             (fa_fwd_ex)
  dropout_mask_bytes(q, k, causal, scale, ...)  size of the keep mask
  fill_dropout_mask(q, k, mask, causal, scale, ...)   draws it without a forward
                                                (fa_dropout_mask)
  make_dropout_mask(q, k, causal, scale, ...)   allocates and draws it
  bwd_ex(q, k, v, do, lse, delta, dq, dk, dv, causal, scale, ...)  (fa_bwd_ex)
  bwd_fused(q, k, v, do, lse, delta, dq, dk, dv, causal, scale, *, workspace, ...)
                                    single-pass backward, dQ summed in an fp32
                                    workspace (fa_bwd_fused; dQ not bitwise
                                    reproducible); workspace_bytes(...) sizes it
  attention_ex_fwd / attention_ex_bwd: the same with outputs allocated
                                    (attention_ex_bwd(..., deterministic=False)
                                    takes the single-pass backward)
  attention(q, k, v, causal, scale, dropout_p=..., seed=..., offset=...)
  attention_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                   max_seqlen_k, causal, scale, dropout_p, seed, offset)
Rotation of query and key heads by positions with one or several axes, and the
RMS norm of every head in the same pass (fa_rotary_fwd / fa_rotary_bwd):
  rotary(q, k, positions, inv_freq, sections, interleaved)      -> (q', k') with autograd
  qk_norm_rotary(q, k, q_weight, k_weight, positions, inv_freq, sections,
                 interleaved, eps)                              -> (q', k') with autograd
  rotary_fwd / rotary_bwd, qk_norm_rotary_fwd / qk_norm_rotary_bwd: the same with
                                    outputs allocated (or given as out=)
  Rotary(...)                       the same choices as one value, which
                                    attention_gqa(..., rotary=),
                                    attention_varlen(..., rotary=) and
                                    attention_varlen_prefix(..., rotary=) apply first

Packed sequences behind one shared prefix (fa_fwd_prefix / fa_bwd_prefix): every
query sees the whole prefix and its own sequence's keys:
  attention_varlen_prefix(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_k,
                          max_seqlen_q, max_seqlen_k, causal, scale, rotary)
                                    -> o with autograd, also for the prefix
  attention_prefix_fwd / attention_prefix_bwd: the same with outputs allocated
  fwd_prefix / bwd_prefix_delta / bwd_prefix    write the tensors given

Serving (fa_decode): the newest tokens of a batch whose keys are a prefix that
all requests share, followed by each request's own cache rows:
  attention_decode(q, k_prefix, v_prefix, k, v, seq_lens, causal, scale)
                                    -> (o, lse)   allocates outputs and workspace
  decode(q, k_prefix, v_prefix, k, v, seq_lens, o, lse, causal, scale, *, workspace)
  decode_workspace_bytes(q, k_prefix, k)

Fixed lengths: q, o, do [B, Hq, Nq, D]; k, v [B, Hkv, Nk, D]; lse [B, Hq, Nq].
Packed: q, o, do [total_q, Hq, D]; k, v [total_k, Hkv, D]; lse [Hq, total_q];
cu_seqlens_* int32 CUDA tensors of B+1 offsets, max_seqlen_* host ints.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import struct
import threading
from typing import NamedTuple, Optional, Sequence

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")

FA_F32, FA_F16, FA_BF16 = 0, 1, 2
_DTYPE_CODE = {torch.float32: FA_F32, torch.float16: FA_F16, torch.bfloat16: FA_BF16}
FA_PATH_AUTO, FA_PATH_FFMA = 0, 1

STATUS_NAMES = {
    0: "FA_OK", 1: "FA_ERR_NULL", 2: "FA_ERR_SHAPE", 3: "FA_ERR_HEADDIM",
    4: "FA_ERR_DTYPE", 5: "FA_ERR_STRIDE", 6: "FA_ERR_ALIGN", 7: "FA_ERR_LAUNCH",
    8: "FA_ERR_TIMEOUT", 9: "FA_ERR_ARCH", 10: "FA_ERR_SCALE", 11: "FA_ERR_ARG",
    12: "FA_ERR_SCRATCH", 13: "FA_ERR_SEQLENS",
}

EXPORTED = ("fa_fwd", "fa_bwd_preprocess", "fa_bwd", "fa_get_device_status",
            "fa_status_string", "fa_set_path", "fa_set_wait_timeout_ns",
            "fa_set_profile_events", "fa_version", "fa_bwd_noalloc",
            "fa_test_withhold_next_arrival", "fa_fwd_ex", "fa_bwd_ex",
            "fa_bwd_fused_workspace_bytes", "fa_bwd_fused", "fa_dropout_mask_bytes",
            "fa_dropout_mask", "fa_test_set_l2_bytes", "fa_rotary_fwd",
            "fa_rotary_bwd_workspace_bytes", "fa_rotary_bwd", "fa_decode_workspace_bytes",
            "fa_decode", "fa_fwd_prefix", "fa_bwd_prefix_delta", "fa_bwd_prefix")


class Problem(ctypes.Structure):
    """struct fa_problem of include/fa.h."""
    _fields_ = [("B", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hkv", ctypes.c_int64),
                ("Nq", ctypes.c_int64), ("Nk", ctypes.c_int64), ("D", ctypes.c_int64),
                ("cu_seqlens_q", ctypes.c_void_p), ("cu_seqlens_k", ctypes.c_void_p),
                ("total_q", ctypes.c_int64), ("total_k", ctypes.c_int64),
                ("causal", ctypes.c_int), ("scale", ctypes.c_float), ("dtype", ctypes.c_int),
                ("dropout_p", ctypes.c_float), ("seed", ctypes.c_uint64),
                ("offset", ctypes.c_uint32), ("dropout_mask", ctypes.c_void_p)]


class RotaryProblem(ctypes.Structure):
    """struct fa_rotary of include/fa.h."""
    _fields_ = [("B", ctypes.c_int64), ("N", ctypes.c_int64), ("Hq", ctypes.c_int64),
                ("Hkv", ctypes.c_int64), ("D", ctypes.c_int64), ("dtype", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("n_axes", ctypes.c_int64),
                ("sections", ctypes.c_int64 * 4), ("inv_freq", ctypes.c_void_p),
                ("positions", ctypes.c_void_p), ("pos_stride", ctypes.c_int64 * 3),
                ("positions_64", ctypes.c_int), ("weight_f32", ctypes.c_int),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class DecodeProblem(ctypes.Structure):
    """struct fa_decode_problem of include/fa.h."""
    _fields_ = [("B", ctypes.c_int64), ("Hq", ctypes.c_int64), ("Hkv", ctypes.c_int64),
                ("Nq", ctypes.c_int64), ("D", ctypes.c_int64), ("P", ctypes.c_int64),
                ("S", ctypes.c_int64), ("seq_lens", ctypes.c_void_p), ("causal", ctypes.c_int),
                ("scale", ctypes.c_float), ("dtype", ctypes.c_int)]


class FAError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)}")


_lock = threading.Lock()
_lib = None
_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_s4 = ctypes.c_void_p      # int64[4]: a ctypes array or packed bytes


def load_library(path: str = LIB_PATH):
    """Load libfa.so and declare its signatures.  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libfa.so is not built ({path}); run __graft_entry__.build()")
        lib = ctypes.CDLL(path)
        lib.fa_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64,
                               _s4, _s4, _s4, _s4, ctypes.c_int, ctypes.c_float,
                               ctypes.c_int, _vp]
        lib.fa_fwd.restype = ctypes.c_int
        lib.fa_bwd_preprocess.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64,
                                          _s4, _s4, ctypes.c_int, _vp]
        lib.fa_bwd_preprocess.restype = ctypes.c_int
        lib.fa_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _i64, _i64, _i64, _i64, _s4, _s4, _s4, _s4, _s4,
                               _s4, _s4, ctypes.c_int, ctypes.c_float, ctypes.c_int,
                               _vp]
        lib.fa_bwd.restype = ctypes.c_int
        lib.fa_bwd_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                       _i64, _i64, _i64, _i64, _s4, _s4, _s4, _s4, _s4,
                                       _s4, _s4, _s4, ctypes.c_int, ctypes.c_float,
                                       ctypes.c_int, _vp]
        lib.fa_bwd_noalloc.restype = ctypes.c_int
        _pp = ctypes.POINTER(Problem)
        lib.fa_fwd_ex.argtypes = [_pp, _vp, _s4, _vp, _s4, _vp, _s4, _vp, _s4, _vp, _vp]
        lib.fa_fwd_ex.restype = ctypes.c_int
        lib.fa_bwd_ex.argtypes = [_pp, _vp, _s4, _vp, _s4, _vp, _s4, _vp, _s4, _vp, _vp,
                                  _vp, _s4, _vp, _s4, _vp, _s4, _vp]
        lib.fa_bwd_ex.restype = ctypes.c_int
        lib.fa_bwd_fused_workspace_bytes.argtypes = [_pp]
        lib.fa_bwd_fused_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_bwd_fused.argtypes = [_pp, _vp, _s4, _vp, _s4, _vp, _s4, _vp, _s4, _vp, _vp,
                                     _vp, _s4, _vp, _s4, _vp, _s4, _vp, ctypes.c_size_t, _vp]
        lib.fa_bwd_fused.restype = ctypes.c_int
        lib.fa_dropout_mask_bytes.argtypes = [_pp]
        lib.fa_dropout_mask_bytes.restype = ctypes.c_size_t
        lib.fa_dropout_mask.argtypes = [_pp, _vp, ctypes.c_size_t, _vp]
        lib.fa_dropout_mask.restype = ctypes.c_int
        # structs and strides as plain addresses: ctypes objects and packed bytes pass
        lib.fa_rotary_fwd.argtypes = [_vp] * 10
        lib.fa_rotary_fwd.restype = ctypes.c_int
        lib.fa_rotary_bwd_workspace_bytes.argtypes = [_vp]
        lib.fa_rotary_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_rotary_bwd.argtypes = [_vp] * 16 + [ctypes.c_size_t, _vp]
        lib.fa_rotary_bwd.restype = ctypes.c_int
        lib.fa_fwd_prefix.argtypes = [_vp, _i64] + [_vp] * 14
        lib.fa_fwd_prefix.restype = ctypes.c_int
        lib.fa_bwd_prefix_delta.argtypes = [_vp, _i64] + [_vp] * 17
        lib.fa_bwd_prefix_delta.restype = ctypes.c_int
        lib.fa_bwd_prefix.argtypes = [_vp, _i64] + [_vp] * 25
        lib.fa_bwd_prefix.restype = ctypes.c_int
        lib.fa_decode_workspace_bytes.argtypes = [_vp]
        lib.fa_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.fa_decode.argtypes = [_vp] * 15 + [ctypes.c_size_t, _vp]
        lib.fa_decode.restype = ctypes.c_int
        lib.fa_get_device_status.argtypes = [_vp]
        lib.fa_get_device_status.restype = ctypes.c_int
        lib.fa_status_string.argtypes = [ctypes.c_int]
        lib.fa_status_string.restype = ctypes.c_char_p
        lib.fa_set_path.argtypes = [ctypes.c_int]
        lib.fa_set_path.restype = ctypes.c_int
        lib.fa_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
        lib.fa_set_wait_timeout_ns.restype = None
        lib.fa_set_profile_events.argtypes = [ctypes.c_void_p]
        lib.fa_set_profile_events.restype = None
        lib.fa_version.restype = ctypes.c_int
        lib.fa_test_withhold_next_arrival.argtypes = []
        lib.fa_test_withhold_next_arrival.restype = None
        lib.fa_test_set_l2_bytes.argtypes = [_i64]
        lib.fa_test_set_l2_bytes.restype = None
        if os.environ.get("FA_WAIT_TIMEOUT_NS"):
            lib.fa_set_wait_timeout_ns(int(os.environ["FA_WAIT_TIMEOUT_NS"]))
        _lib = lib
        return lib


def _strides(t: torch.Tensor):
    return (ctypes.c_int64 * 4)(*t.stride())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _check(code: int, where: str):
    if code != 0:
        raise FAError(code, where)


def _dims(q: torch.Tensor):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, D] tensors")
    if q.dtype not in _DTYPE_CODE:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if not q.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    return q.shape


def _same(ref: torch.Tensor, *ts):
    for t in ts:
        if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
            raise ValueError("q, k, v, o, do, dq, dk, dv must share shape, dtype and device")


def _scale(D: int, scale):
    return 1.0 / math.sqrt(D) if scale is None else float(scale)


def fwd(q, k, v, o, lse, causal: bool, scale=None):
    B, H, N, D = _dims(q)
    _same(q, k, v, o)
    lib = load_library()
    with torch.cuda.device(q.device):
        code = lib.fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                          lse.data_ptr(), B, H, N, D, _strides(q), _strides(k),
                          _strides(v), _strides(o), int(bool(causal)),
                          _scale(D, scale), _DTYPE_CODE[q.dtype], _stream(q))
    _check(code, "fa_fwd")


def bwd_preprocess(o, do, delta):
    B, H, N, D = _dims(o)
    _same(o, do)
    lib = load_library()
    with torch.cuda.device(o.device):
        code = lib.fa_bwd_preprocess(o.data_ptr(), do.data_ptr(), delta.data_ptr(),
                                     B, H, N, D, _strides(o), _strides(do),
                                     _DTYPE_CODE[o.dtype], _stream(o))
    _check(code, "fa_bwd_preprocess")


def bwd(q, k, v, do, lse, delta, dq, dk, dv, causal: bool, scale=None):
    B, H, N, D = _dims(q)
    _same(q, k, v, do, dq, dk, dv)
    lib = load_library()
    with torch.cuda.device(q.device):
        code = lib.fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), do.data_ptr(),
                          lse.data_ptr(), delta.data_ptr(), dq.data_ptr(),
                          dk.data_ptr(), dv.data_ptr(), B, H, N, D, _strides(q),
                          _strides(k), _strides(v), _strides(do), _strides(dq),
                          _strides(dk), _strides(dv), int(bool(causal)),
                          _scale(D, scale), _DTYPE_CODE[q.dtype], _stream(q))
    _check(code, "fa_bwd")


def bwd_noalloc(q, k, v, o, do, lse, dq, dk, dv, causal: bool, scale=None):
    """fa_bwd_noalloc: the backward for callers that cannot allocate device
    memory; Delta lives in a fixed buffer inside libfa (B*H*N must not exceed
    its FA_NOALLOC_MAX_ROWS rows).  Calls must not overlap on the GPU."""
    B, H, N, D = _dims(q)
    _same(q, k, v, o, do, dq, dk, dv)
    lib = load_library()
    with torch.cuda.device(q.device):
        code = lib.fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                  do.data_ptr(), lse.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                  dv.data_ptr(), B, H, N, D, _strides(q), _strides(k),
                                  _strides(v), _strides(o), _strides(do), _strides(dq),
                                  _strides(dk), _strides(dv), int(bool(causal)),
                                  _scale(D, scale), _DTYPE_CODE[q.dtype], _stream(q))
    _check(code, "fa_bwd_noalloc")


def device_status(device=None) -> int:
    """fa_get_device_status on the current stream of `device` (syncs it)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    lib = load_library()
    with torch.cuda.device(dev):
        return lib.fa_get_device_status(ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream))


def set_path(path: int) -> None:
    _check(load_library().fa_set_path(int(path)), "fa_set_path")


def set_wait_timeout_ns(ns: int) -> None:
    load_library().fa_set_wait_timeout_ns(int(ns))


def test_set_l2_bytes(nbytes: int) -> None:
    """fa_test_set_l2_bytes: the L2 size the block order assumes (0: the device's)."""
    load_library().fa_test_set_l2_bytes(int(nbytes))


def set_profile_events(events) -> None:
    """events: three torch.cuda.Event(enable_timing=True) recorded by later
    fa_bwd calls before dK/dV, between dK/dV and dQ, and after dQ; None turns
    the hook off."""
    lib = load_library()
    if events is None:
        lib.fa_set_profile_events(None)
        return
    handles = (ctypes.c_void_p * 3)(*[ev.cuda_event for ev in events])
    lib.fa_set_profile_events(ctypes.cast(handles, ctypes.c_void_p))


def attention_fwd(q, k, v, causal: bool = False, scale=None):
    B, H, N, D = _dims(q)
    o = torch.empty((B, H, N, D), dtype=q.dtype, device=q.device)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    fwd(q, k, v, o, lse, causal, scale)
    return o, lse


def attention_bwd(q, k, v, o, lse, do, causal: bool = False, scale=None):
    B, H, N, D = _dims(q)
    delta = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    bwd_preprocess(o, do, delta)
    dq = torch.empty((B, H, N, D), dtype=q.dtype, device=q.device)
    dk = torch.empty_like(dq)
    dv = torch.empty_like(dq)
    bwd(q, k, v, do, lse, delta, dq, dk, dv, causal, scale)
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale):
        o, lse = attention_fwd(q, k, v, causal, scale)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.scale = causal, scale
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        if do.stride(-1) != 1:
            do = do.contiguous()
        dq, dk, dv = attention_bwd(q, k, v, o, lse, do, ctx.causal, ctx.scale)
        return dq, dk, dv, None, None


def attention(q, k, v, causal: bool = False, scale=None):
    """Exact softmax attention with autograd.  Second-order gradients are
    refused (once_differentiable raises) rather than silently wrong."""
    return _Attention.apply(q, k, v, causal, scale)


# ----------------------------------------------------------------------------
# Rotation of query and key heads by their positions, and their norm


class Rotary(NamedTuple):
    """A rotation (and, with weights, a head norm) of queries and keys.

    positions: int32 or int64 CUDA tensor.  Beside [B, H, N, D] heads: [A, B, N]
    for A axes ([A, 1, N] shares them over the batch; with one axis also [B, N]
    or [N]); beside packed [T, H, D] heads: [A, T], or [T] with one axis.
    inv_freq: float32 CUDA vector, one frequency per rotated pair (a multiple of
    8 of them, at most D / 2).  sections: rotated pairs of each axis, in the
    order of inv_freq (None: one axis).  interleaved: pairs (2i, 2i + 1) instead
    of (i, n + i).  q_weight, k_weight: norm weights of D elements, float32 or
    the heads' type (None: no norm); eps: the norm's."""
    positions: torch.Tensor
    inv_freq: torch.Tensor
    sections: Optional[Sequence[int]] = None
    interleaved: bool = False
    q_weight: Optional[torch.Tensor] = None
    k_weight: Optional[torch.Tensor] = None
    eps: float = 1e-6


# The calls below run once per layer and token in serving, where their host
# time is what a step waits for: strides and structs are packed straight into
# bytes (the C layouts of int64[4], fa_rotary, fa_decode_problem and fa_problem) instead of
# through ctypes objects and views, and the device is only switched when it is
# not the current one.
_PACK4 = struct.Struct("@4q").pack
_PACK_ROTARY = struct.Struct("@5q2iq4qPP3q2iPPf0q").pack
_PACK_DECODE = struct.Struct("@7qPifi0q").pack
_PACK_PROBLEM = struct.Struct("@6qPP2qififQIP").pack


def _call(fn, where: str, dev: int, *args):
    """fn(*args, stream) with the current stream of device `dev`."""
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        code = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, stream)
    if code != 0:
        raise FAError(code, where)


def _strides4(t: torch.Tensor) -> bytes:
    """int64[4] strides (b, h, n, d) of [B, H, N, D] or packed [N, H, D]."""
    st = t.stride()
    return _PACK4(*st) if len(st) == 4 else _PACK4(0, st[1], st[0], st[2])


def _rotary_problem(q, k, rot: Rotary) -> bytes:
    """struct fa_rotary of a call."""
    dt = q.dtype
    if dt not in _DTYPE_CODE or not q.is_cuda:
        raise TypeError("tensors must be CUDA float32, float16 or bfloat16")
    dev = q.get_device()
    qs, ks = q.shape, k.shape
    if len(qs) == 4:
        B, Hq, N, D = qs
        packed = False
    elif len(qs) == 3:
        N, Hq, D = qs
        B, packed = 1, True
    else:
        raise ValueError("expected [B, H, N, D] or packed [T, H, D] tensors")
    if k.dtype != dt or k.get_device() != dev or len(ks) != len(qs) or ks[-1] != D:
        raise ValueError("q and k must share dtype, device, layout and head dimension")
    Hkv = ks[1]
    if (ks[0] != N) if packed else (ks[0] != B or ks[2] != N):
        raise ValueError("q and k must share batch and length")
    pos, freq, sections, interleaved, qw, kw, eps = rot
    pairs = freq.numel()
    if freq.dtype != torch.float32 or freq.get_device() != dev or freq.dim() != 1 \
            or not freq.is_contiguous():
        raise ValueError("inv_freq: a contiguous float32 vector on q's device")
    pos64 = pos.dtype == torch.int64
    if not (pos64 or pos.dtype == torch.int32) or pos.get_device() != dev:
        raise ValueError("positions: int32 or int64 on q's device")
    sec = [pairs] if sections is None else [int(n) for n in sections]
    A = len(sec)
    if A < 1 or A > 4 or sum(sec) != pairs:
        raise ValueError("sections: one to four counts that add up to inv_freq's length")
    sec += [0] * (4 - A)
    # extents and strides (axis, b, n); one axis may leave out the axis
    # dimension, and then also the batch's
    ps, pst = list(pos.shape), list(pos.stride())
    full = 2 if packed else 3
    while A == 1 and len(ps) < full:
        ps.insert(0, 1)
        pst.insert(0, 0)
    if packed and len(ps) == 2:
        ps.insert(1, 1)
        pst.insert(1, 0)
    if len(ps) != 3 or ps[0] != A or ps[2] != N or (ps[1] != B and ps[1] != 1):
        raise ValueError(f"positions: expected {[A, N] if packed else [A, B, N]}, got {list(pos.shape)}")
    if ps[1] != B:
        pst[1] = 0
    wq = wk = w32 = 0
    if qw is not None or kw is not None:
        if qw is None or kw is None:
            raise ValueError("q_weight and k_weight: both or none")
        for w in (qw, kw):
            if w.get_device() != dev or w.dim() != 1 or w.numel() != D or not w.is_contiguous() \
                    or (w.dtype != torch.float32 and w.dtype != dt) or w.dtype != qw.dtype:
                raise ValueError("q_weight, k_weight: contiguous [D] of one dtype, float32 or q's")
        wq, wk, w32 = qw.data_ptr(), kw.data_ptr(), qw.dtype == torch.float32
    return _PACK_ROTARY(B, N, Hq, Hkv, D, _DTYPE_CODE[dt], bool(interleaved), A, *sec,
                        freq.data_ptr(), pos.data_ptr(), *pst, pos64, w32, wq, wk, float(eps))


def _rotary_out(x, out):
    if out is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    if out.shape != x.shape or out.dtype != x.dtype or out.device != x.device:
        raise ValueError("out: the shape, dtype and device of its input")
    return out


def _apply_fwd(q, k, rot, out):
    pr = _rotary_problem(q, k, rot)
    qo, ko = out or (None, None)
    qo, ko = _rotary_out(q, qo), _rotary_out(k, ko)
    _call(load_library().fa_rotary_fwd, "fa_rotary_fwd", q.get_device(), pr, q.data_ptr(),
          _strides4(q), k.data_ptr(), _strides4(k), qo.data_ptr(), _strides4(qo), ko.data_ptr(),
          _strides4(ko))
    return qo, ko


def _apply_bwd(q, k, dqo, dko, rot, out):
    """q, k are not read when rot has no weights (and may be None)."""
    pr = _rotary_problem(dqo, dko, rot)
    norm = rot.q_weight is not None
    if norm:
        for x, g in ((q, dqo), (k, dko)):
            if x.shape != g.shape or x.dtype != g.dtype or x.device != g.device:
                raise ValueError("gradients: the shape, dtype and device of their inputs")
    dq, dk = out or (None, None)
    dq, dk = _rotary_out(dqo, dq), _rotary_out(dko, dk)
    lib = load_library()
    if norm:
        D = dqo.shape[-1]
        dev = q.device
        dqw = torch.empty(D, dtype=torch.float32, device=dev)
        dkw = torch.empty(D, dtype=torch.float32, device=dev)
        nbytes = lib.fa_rotary_bwd_workspace_bytes(pr)
        ws = torch.empty(nbytes // 4, dtype=torch.float32, device=dev)
        extra = (dqw.data_ptr(), dkw.data_ptr(), ws.data_ptr(), nbytes)
    else:
        q, k = dqo, dko
        extra = (0, 0, 0, 0)
    _call(lib.fa_rotary_bwd, "fa_rotary_bwd", dqo.get_device(), pr, q.data_ptr(), _strides4(q),
          k.data_ptr(), _strides4(k), dqo.data_ptr(), _strides4(dqo), dko.data_ptr(), _strides4(dko),
          dq.data_ptr(), _strides4(dq), dk.data_ptr(), _strides4(dk), *extra)
    return (dq, dk, dqw, dkw) if norm else (dq, dk)


def rotary_fwd(q, k, positions, inv_freq, sections=None, interleaved: bool = False, out=None):
    """fa_rotary_fwd without a norm: (q', k'), the heads rotated by their
    positions (see Rotary).  q [B, Hq, N, D], k [B, Hkv, N, D], or packed
    [T, H, D].  out: the two tensors to write, which may be q and k themselves."""
    return _apply_fwd(q, k, Rotary(positions, inv_freq, sections, interleaved), out)


def rotary_bwd(dq_out, dk_out, positions, inv_freq, sections=None, interleaved: bool = False,
               out=None):
    """fa_rotary_bwd without a norm: (dq, dk) from the gradients of rotary_fwd's
    outputs.  out: the two tensors to write, which may be the gradients themselves."""
    return _apply_bwd(None, None, dq_out, dk_out, Rotary(positions, inv_freq, sections, interleaved),
                      out)


def qk_norm_rotary_fwd(q, k, q_weight, k_weight, positions, inv_freq, sections=None,
                       interleaved: bool = False, eps: float = 1e-6, out=None):
    """fa_rotary_fwd with the RMS norm of every head before the rotation."""
    return _apply_fwd(q, k, Rotary(positions, inv_freq, sections, interleaved, q_weight, k_weight,
                                   eps), out)


def qk_norm_rotary_bwd(q, k, q_weight, k_weight, dq_out, dk_out, positions, inv_freq,
                       sections=None, interleaved: bool = False, eps: float = 1e-6, out=None):
    """fa_rotary_bwd with the norm: (dq, dk, dq_weight, dk_weight), the weight
    gradients in float32."""
    return _apply_bwd(q, k, dq_out, dk_out, Rotary(positions, inv_freq, sections, interleaved,
                                                   q_weight, k_weight, eps), out)


def _dense(t: torch.Tensor) -> torch.Tensor:
    """t, or a contiguous copy when its layout is not one the kernels take
    (e.g. the expanded gradient of a sum)."""
    es = t.element_size()
    ok = t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(
        n == 1 or (s > 0 and s * es % 16 == 0) for n, s in zip(t.shape[:-1], t.stride()[:-1]))
    return t if ok else t.contiguous()


class _ApplyRotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, rot):
        # Positions and frequencies are saved like inputs, so that a change in
        # place before the backward is an error; without a norm the gradient
        # needs neither q nor k.
        norm = (q, k, q_weight, k_weight) if q_weight is not None else ()
        ctx.save_for_backward(rot.positions, rot.inv_freq, *norm)
        ctx.rot = rot._replace(positions=None, inv_freq=None, q_weight=None, k_weight=None)
        return _apply_fwd(q, k, rot, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dqo, dko):
        dqo, dko = _dense(dqo), _dense(dko)
        positions, inv_freq, *norm = ctx.saved_tensors
        rot = ctx.rot._replace(positions=positions, inv_freq=inv_freq)
        if not norm:
            return (*_apply_bwd(None, None, dqo, dko, rot, None), None, None, None)
        q, k, qw, kw = norm
        dq, dk, dqw, dkw = _apply_bwd(q, k, dqo, dko, rot._replace(q_weight=qw, k_weight=kw), None)
        return dq, dk, dqw.to(qw.dtype), dkw.to(kw.dtype), None


def apply_rotary(q, k, rot: Rotary):
    """(q', k') of a Rotary, with autograd for q, k and the norm's weights.
    Second-order gradients are refused, and so are frequencies that want one."""
    if rot.inv_freq.requires_grad and torch.is_grad_enabled():
        raise ValueError("inv_freq takes no gradient")
    return _ApplyRotary.apply(_dense(q), _dense(k), rot.q_weight, rot.k_weight, rot)


def rotary(q, k, positions, inv_freq, sections=None, interleaved: bool = False):
    """rotary_fwd with autograd."""
    return apply_rotary(q, k, Rotary(positions, inv_freq, sections, interleaved))


def qk_norm_rotary(q, k, q_weight, k_weight, positions, inv_freq, sections=None,
                   interleaved: bool = False, eps: float = 1e-6):
    """qk_norm_rotary_fwd with autograd."""
    return apply_rotary(q, k, Rotary(positions, inv_freq, sections, interleaved, q_weight, k_weight,
                                     eps))


# ----------------------------------------------------------------------------
# Serving: new tokens over a shared prefix and each request's own rows


def _decode_sizes(q, k_prefix, k):
    """(B, Hq, Hkv, Nq, D, P, S) of a decode call."""
    qs, ps, ks = q.shape, k_prefix.shape, k.shape
    if len(qs) != 4 or len(ks) != 4 or len(ps) != 3:
        raise ValueError("expected q [B, Hq, Nq, D], k, v [B, Hkv, S, D], prefixes [Hkv, P, D]")
    B, Hq, Nq, D = qs
    Hkv, P, Dp = ps
    if ks[0] != B or ks[1] != Hkv or ks[3] != D or Dp != D:
        raise ValueError("q, k and the prefix must share batch, key/value heads and head dimension")
    return B, Hq, Hkv, Nq, D, P, ks[2]


@functools.lru_cache(maxsize=256)
def _decode_bytes(sizes) -> int:
    # the lengths, type and scale do not change the size
    pr = _PACK_DECODE(*sizes, 16, 1, 1.0, FA_F16)
    return int(load_library().fa_decode_workspace_bytes(pr))


def decode_workspace_bytes(q, k_prefix, k) -> int:
    """Bytes of the workspace decode needs for these shapes (0 if none, or if they
    are invalid)."""
    return _decode_bytes(_decode_sizes(q, k_prefix, k))


def decode(q, k_prefix, v_prefix, k, v, seq_lens, o, lse, causal: bool = True, scale=None, *,
           workspace: Optional[torch.Tensor] = None):
    """fa_decode.  workspace: a contiguous CUDA tensor of at least
    decode_workspace_bytes(q, k_prefix, k) bytes, 16-byte aligned (None when
    that is 0); calls that may overlap on the GPU need one each."""
    sizes = _decode_sizes(q, k_prefix, k)
    if o.shape != q.shape or o.dtype != q.dtype or o.device != q.device:
        raise ValueError("o: the shape, dtype and device of q")
    if lse.dtype != torch.float32 or lse.shape != q.shape[:3] or lse.device != q.device \
            or not lse.is_contiguous():
        raise ValueError("lse: contiguous float32 [B, Hq, Nq] on q's device")
    if workspace is not None and (workspace.device != q.device or not workspace.is_contiguous()):
        raise ValueError("workspace: a contiguous tensor on q's device")
    _decode(sizes, q, k_prefix, v_prefix, k, v, seq_lens, o, lse, causal, scale, workspace)


def _decode(sizes, q, k_prefix, v_prefix, k, v, seq_lens, o, lse, causal, scale, workspace):
    """decode with its outputs and workspace known to fit."""
    dt = q.dtype
    if (dt != torch.bfloat16 and dt != torch.float16) or not q.is_cuda:
        raise TypeError("decode takes CUDA float16 or bfloat16 tensors")
    dev = q.get_device()
    for t in (k_prefix, v_prefix, k, v):
        if t.dtype != dt or t.get_device() != dev:
            raise ValueError("all tensors must share dtype and device")
    if v.shape != k.shape or v_prefix.shape != k_prefix.shape:
        raise ValueError("v and v_prefix take the shapes of k and k_prefix")
    if seq_lens.dtype != torch.int32 or seq_lens.shape != (sizes[0],) or seq_lens.get_device() != dev \
            or not seq_lens.is_contiguous():
        raise ValueError("seq_lens: a contiguous int32 vector of B lengths on q's device")
    ws = nbytes = 0
    if workspace is not None:
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    pr = _PACK_DECODE(*sizes, seq_lens.data_ptr(), bool(causal), _scale(sizes[4], scale),
                      _DTYPE_CODE[dt])
    _call(load_library().fa_decode, "fa_decode", dev, pr, q.data_ptr(), _PACK4(*q.stride()),
          k_prefix.data_ptr(), _PACK4(0, *k_prefix.stride()), v_prefix.data_ptr(),
          _PACK4(0, *v_prefix.stride()), k.data_ptr(), _PACK4(*k.stride()), v.data_ptr(),
          _PACK4(*v.stride()), o.data_ptr(), _PACK4(*o.stride()), lse.data_ptr(), ws, nbytes)


def attention_decode(q, k_prefix, v_prefix, k, v, seq_lens, causal: bool = True, scale=None,
                     workspace: Optional[torch.Tensor] = None):
    """Attention of the newest Nq (1 to 16) tokens of B requests: returns
    (o [B, Hq, Nq, D], lse [B, Hq, Nq]).  q [B, Hq, Nq, D]; k_prefix, v_prefix
    [Hkv, P, D], keys that every request sees in full; k, v [B, Hkv, S, D], the
    requests' own cache rows, of which request b's first seq_lens[b] count (int32
    CUDA vector; the new tokens' rows among them, as the last Nq).  causal: token
    t sees own rows up to its own.  float16 and bfloat16; no gradient."""
    sizes = _decode_sizes(q, k_prefix, k)
    dev = q.device
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty((sizes[0], sizes[1], sizes[3]), dtype=torch.float32, device=dev)
    if workspace is None:
        nbytes = _decode_bytes(sizes)
        if nbytes:
            workspace = torch.empty(nbytes // 4, dtype=torch.float32, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor on q's device")
    _decode(sizes, q, k_prefix, v_prefix, k, v, seq_lens, o, lse, causal, scale, workspace)
    return o, lse


# ----------------------------------------------------------------------------
# General problems: Nq != Nk, grouped key/value heads, packed sequences, dropout


def _as4(t: torch.Tensor, packed: bool) -> torch.Tensor:
    """Packed [total, H, D] -> the [1, H, total, D] view the C ABI takes."""
    if packed:
        if t.dim() != 3:
            raise ValueError("packed tensors are [total, H, D]")
        return t.permute(1, 0, 2).unsqueeze(0)
    if t.dim() != 4:
        raise ValueError("expected [B, H, N, D] tensors")
    return t


def _problem(q4, k4, causal, scale, cu_q, cu_k, max_q, max_k, dropout_p, seed, offset,
             dropout_mask=None):
    if q4.dtype not in _DTYPE_CODE or not q4.is_cuda:
        raise TypeError("tensors must be CUDA float32, float16 or bfloat16")
    for t in (k4,):
        if t.dtype != q4.dtype or t.device != q4.device or t.shape[-1] != q4.shape[-1]:
            raise ValueError("q, k, v must share dtype, device and head dimension")
    pr = Problem()
    D = q4.shape[3]
    pr.Hq, pr.Hkv, pr.D = q4.shape[1], k4.shape[1], D
    if cu_q is not None:
        for cu in (cu_q, cu_k):
            if cu is None or cu.dtype != torch.int32 or not cu.is_cuda or cu.dim() != 1:
                raise ValueError("cu_seqlens_q and cu_seqlens_k: int32 CUDA vectors of B+1")
        if cu_q.numel() != cu_k.numel() or cu_q.numel() < 2:
            raise ValueError("cu_seqlens_q and cu_seqlens_k need the same B+1 >= 2 entries")
        pr.B = cu_q.numel() - 1
        pr.Nq, pr.Nk = int(max_q), int(max_k)
        pr.cu_seqlens_q, pr.cu_seqlens_k = cu_q.data_ptr(), cu_k.data_ptr()
        pr.total_q, pr.total_k = q4.shape[2], k4.shape[2]
    else:
        if q4.shape[0] != k4.shape[0]:
            raise ValueError("q and k need the same batch")
        pr.B, pr.Nq, pr.Nk = q4.shape[0], q4.shape[2], k4.shape[2]
    pr.causal = int(bool(causal))
    pr.scale = _scale(D, scale)
    pr.dtype = _DTYPE_CODE[q4.dtype]
    pr.dropout_p = float(dropout_p)
    pr.seed = int(seed) & ((1 << 64) - 1)
    pr.offset = int(offset) & 0xFFFFFFFF
    if dropout_mask is not None:
        if (dropout_mask.dtype != torch.uint8 or dropout_mask.device != q4.device
                or not dropout_mask.is_contiguous()):
            raise ValueError("dropout_mask: a contiguous uint8 tensor on q's device")
        pr.dropout_mask = dropout_mask.data_ptr()
    return pr


def fwd_ex(q, k, v, o, lse, causal: bool = False, scale=None, *, cu_seqlens_q=None,
           cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None, dropout_p: float = 0.0,
           seed: int = 0, offset: int = 0, dropout_mask=None):
    packed = cu_seqlens_q is not None
    q4, k4, v4, o4 = (_as4(t, packed) for t in (q, k, v, o))
    pr = _problem(q4, k4, causal, scale, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                  max_seqlen_k, dropout_p, seed, offset, dropout_mask)
    lib = load_library()
    with torch.cuda.device(q.device):
        code = lib.fa_fwd_ex(ctypes.byref(pr), q4.data_ptr(), _strides(q4), k4.data_ptr(),
                             _strides(k4), v4.data_ptr(), _strides(v4), o4.data_ptr(),
                             _strides(o4), lse.data_ptr(), _stream(q))
    _check(code, "fa_fwd_ex")


def bwd_ex(q, k, v, do, lse, delta, dq, dk, dv, causal: bool = False, scale=None, *,
           cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=None, max_seqlen_k=None,
           dropout_p: float = 0.0, seed: int = 0, offset: int = 0, dropout_mask=None):
    packed = cu_seqlens_q is not None
    q4, k4, v4, do4, dq4, dk4, dv4 = (_as4(t, packed) for t in (q, k, v, do, dq, dk, dv))
    pr = _problem(q4, k4, causal, scale, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                  max_seqlen_k, dropout_p, seed, offset, dropout_mask)
    lib = load_library()
    with torch.cuda.device(q.device):
        code = lib.fa_bwd_ex(ctypes.byref(pr), q4.data_ptr(), _strides(q4), k4.data_ptr(),
                             _strides(k4), v4.data_ptr(), _strides(v4), do4.data_ptr(),
                             _strides(do4), lse.data_ptr(), delta.data_ptr(), dq4.data_ptr(),
                             _strides(dq4), dk4.data_ptr(), _strides(dk4), dv4.data_ptr(),
                             _strides(dv4), _stream(q))
    _check(code, "fa_bwd_ex")


_EX_KEYS = ("cu_seqlens_q", "cu_seqlens_k", "max_seqlen_q", "max_seqlen_k", "dropout_p",
            "seed", "offset", "dropout_mask")


def _ex_call(tensors, causal, scale, kw):
    """The [1, H, total, D] views of packed tensors (tensors[0], tensors[1]:
    q and k) and the fa_problem of a general call."""
    unknown = set(kw) - set(_EX_KEYS)
    if unknown:
        raise TypeError(f"unexpected keyword arguments {sorted(unknown)}")
    packed = kw.get("cu_seqlens_q") is not None
    t4 = [_as4(t, packed) for t in tensors]
    pr = _problem(t4[0], t4[1], causal, scale, kw.get("cu_seqlens_q"), kw.get("cu_seqlens_k"),
                  kw.get("max_seqlen_q"), kw.get("max_seqlen_k"), kw.get("dropout_p", 0.0),
                  kw.get("seed", 0), kw.get("offset", 0), kw.get("dropout_mask"))
    return t4, pr


def dropout_mask_bytes(q, k, causal: bool = False, scale=None, **kw) -> int:
    """Bytes of the keep mask fa_dropout_mask draws for this problem (0 when
    dropout_p = 0 or the problem is invalid)."""
    _, pr = _ex_call((q, k), causal, scale, kw)
    return int(load_library().fa_dropout_mask_bytes(ctypes.byref(pr)))


def fill_dropout_mask(q, k, mask, causal: bool = False, scale=None, **kw):
    """fa_dropout_mask: draws the keep decisions of the problem into `mask`, a
    contiguous uint8 CUDA tensor of at least dropout_mask_bytes(...) bytes,
    without a forward (fwd_ex given dropout_mask= stores the same bytes)."""
    kw = {key: val for key, val in kw.items() if key != "dropout_mask"}
    (q4, _), pr = _ex_call((q, k), causal, scale, kw)
    if mask.dtype != torch.uint8 or mask.device != q.device or not mask.is_contiguous():
        raise ValueError("mask: a contiguous uint8 tensor on q's device")
    lib = load_library()
    with torch.cuda.device(q.device):
        code = lib.fa_dropout_mask(ctypes.byref(pr), mask.data_ptr(), mask.numel(), _stream(q))
    _check(code, "fa_dropout_mask")


def make_dropout_mask(q, k, causal: bool = False, scale=None, **kw) -> torch.Tensor:
    """Allocates and draws the keep mask of a dropout problem (see
    fill_dropout_mask), e.g. for bwd_ex after a forward that kept none."""
    kw = {key: val for key, val in kw.items() if key != "dropout_mask"}
    nbytes = dropout_mask_bytes(q, k, causal, scale, **kw)
    if nbytes == 0:
        raise ValueError("no keep mask for this problem (dropout_p = 0 or invalid)")
    mask = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    fill_dropout_mask(q, k, mask, causal, scale, **kw)
    return mask


def workspace_bytes(q, k, causal: bool = False, scale=None, **kw) -> int:
    """Bytes of the fp32 dQ workspace bwd_fused needs for this problem (0 if invalid)."""
    _, pr = _ex_call((q, k), causal, scale, kw)
    return int(load_library().fa_bwd_fused_workspace_bytes(ctypes.byref(pr)))


def bwd_fused(q, k, v, do, lse, delta, dq, dk, dv, causal: bool = False, scale=None, *,
              workspace: torch.Tensor, **kw):
    """fa_bwd_fused: like bwd_ex, with dQ summed in `workspace` (a CUDA tensor of
    at least workspace_bytes(...) bytes, 16-byte aligned; zeroed by the call)."""
    (q4, k4, v4, do4, dq4, dk4, dv4), pr = _ex_call((q, k, v, do, dq, dk, dv), causal, scale,
                                                   kw)
    if not workspace.is_cuda or workspace.device != q.device:
        raise ValueError("workspace must be a CUDA tensor on q's device")
    nbytes = workspace.numel() * workspace.element_size()
    lib = load_library()
    with torch.cuda.device(q.device):
        code = lib.fa_bwd_fused(ctypes.byref(pr), q4.data_ptr(), _strides(q4), k4.data_ptr(),
                                _strides(k4), v4.data_ptr(), _strides(v4), do4.data_ptr(),
                                _strides(do4), lse.data_ptr(), delta.data_ptr(),
                                dq4.data_ptr(), _strides(dq4), dk4.data_ptr(), _strides(dk4),
                                dv4.data_ptr(), _strides(dv4), workspace.data_ptr(), nbytes,
                                _stream(q))
    _check(code, "fa_bwd_fused")


def _lse_shape(q, packed):
    return (q.shape[1], q.shape[0]) if packed else (q.shape[0], q.shape[1], q.shape[2])


def attention_ex_fwd(q, k, v, causal: bool = False, scale=None, **kw):
    """Allocating forward of a general problem: returns (o, lse)."""
    packed = kw.get("cu_seqlens_q") is not None
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty(_lse_shape(q, packed), dtype=torch.float32, device=q.device)
    fwd_ex(q, k, v, o, lse, causal, scale, **kw)
    return o, lse


def attention_ex_bwd(q, k, v, o, lse, do, causal: bool = False, scale=None, *,
                     deterministic: bool = True, **kw):
    """Allocating backward of a general problem: returns (dq, dk, dv).  With
    deterministic=False the single-pass backward runs (fp16/bf16 only)."""
    packed = kw.get("cu_seqlens_q") is not None
    o4, do4 = _as4(o, packed), _as4(do, packed)
    delta = torch.empty(_lse_shape(q, packed), dtype=torch.float32, device=q.device)
    bwd_preprocess(o4, do4, delta)
    dq = torch.empty_like(q, memory_format=torch.contiguous_format)
    dk = torch.empty_like(k, memory_format=torch.contiguous_format)
    dv = torch.empty_like(v, memory_format=torch.contiguous_format)
    if deterministic:
        bwd_ex(q, k, v, do, lse, delta, dq, dk, dv, causal, scale, **kw)
    else:
        nbytes = workspace_bytes(q, k, causal, scale, **kw)
        ws = torch.empty(max(nbytes // 4, 4), dtype=torch.float32, device=q.device)
        bwd_fused(q, k, v, do, lse, delta, dq, dk, dv, causal, scale, workspace=ws, **kw)
    return dq, dk, dv


# The autograd functions give the forward a keep-mask buffer to store its
# dropout decisions in, which the backward then reads instead of evaluating
# the generator again, when the buffer takes at most this many bytes
# (keep_mask=None); larger problems draw the decisions again in the backward.
# Either way the decisions, and so the results, are bitwise the same.
DROPOUT_MASK_AUTO_BYTES = 4 << 30


def _with_mask(q, k, causal, scale, kw, keep_mask):
    """kw with a keep-mask buffer (filled by the forward) when the policy asks
    for one."""
    if keep_mask is False or kw.get("dropout_p", 0.0) <= 0.0 or kw.get("dropout_mask") is not None:
        return kw
    nbytes = dropout_mask_bytes(q, k, causal, scale, **kw)
    if nbytes == 0 or (keep_mask is None and nbytes > DROPOUT_MASK_AUTO_BYTES):
        return kw
    return dict(kw, dropout_mask=torch.empty(nbytes, dtype=torch.uint8, device=q.device))


class _AttentionEx(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale, kw, deterministic, keep_mask):
        kw = _with_mask(q, k, causal, scale, kw, keep_mask)
        o, lse = attention_ex_fwd(q, k, v, causal, scale, **kw)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.causal, ctx.scale, ctx.kw, ctx.deterministic = causal, scale, kw, deterministic
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        if do.stride(-1) != 1:
            do = do.contiguous()
        dq, dk, dv = attention_ex_bwd(q, k, v, o, lse, do, ctx.causal, ctx.scale,
                                      deterministic=ctx.deterministic, **ctx.kw)
        return dq, dk, dv, None, None, None, None, None


def attention_gqa(q, k, v, causal: bool = False, scale=None, dropout_p: float = 0.0,
                  seed: int = 0, offset: int = 0, deterministic: bool = True,
                  keep_mask: bool | None = None, rotary: Optional[Rotary] = None):
    """Autograd attention for q [B, Hq, Nq, D], k, v [B, Hkv, Nk, D] (Hq % Hkv == 0),
    with optional dropout of the attention weights.  deterministic=False takes
    the single-pass backward (dQ not bitwise reproducible).  keep_mask: let
    the forward store its dropout decisions in a buffer the backward reads
    (True), never (False), or when it fits DROPOUT_MASK_AUTO_BYTES (None).
    rotary: the rotation (and head norm) to apply to q and k first; they need
    one length then."""
    if rotary is not None:
        q, k = apply_rotary(q, k, rotary)
    kw = dict(dropout_p=dropout_p, seed=seed, offset=offset)
    return _AttentionEx.apply(q, k, v, causal, scale, kw, deterministic, keep_mask)


def attention_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q: int,
                     max_seqlen_k: int, causal: bool = False, scale=None,
                     dropout_p: float = 0.0, seed: int = 0, offset: int = 0,
                     deterministic: bool = True, keep_mask: bool | None = None,
                     rotary: Optional[Rotary] = None):
    """Autograd attention over packed sequences: q [total_q, Hq, D],
    k, v [total_k, Hkv, D], cu_seqlens_* int32 CUDA offsets (B+1); keep_mask
    and rotary as for attention_gqa."""
    if rotary is not None:
        q, k = apply_rotary(q, k, rotary)
    kw = dict(cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k,
              max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k,
              dropout_p=dropout_p, seed=seed, offset=offset)
    return _AttentionEx.apply(q, k, v, causal, scale, kw, deterministic, keep_mask)


# ----------------------------------------------------------------------------
# Packed sequences behind one shared prefix


def _prefix_problem(q, k, v, k_prefix, v_prefix, cu_q, cu_k, max_q, max_k, causal, scale) -> bytes:
    """struct fa_problem of a prefix call, its inputs checked."""
    dt = q.dtype
    if dt not in _DTYPE_CODE or not q.is_cuda:
        raise TypeError("tensors must be CUDA float32, float16 or bfloat16")
    qs, ks, ps = q.shape, k.shape, k_prefix.shape
    if len(qs) != 3 or len(ks) != 3 or len(ps) != 3:
        raise ValueError("expected q [total_q, Hq, D], k, v [total_k, Hkv, D], prefixes [P, Hkv, D]")
    dev = q.get_device()
    if v.shape != ks or v_prefix.shape != ps or ks[2] != qs[2] or ps[1:] != ks[1:]:
        raise ValueError("q, k, v and the prefixes must share head dimension and key/value heads")
    for t in (k, v, k_prefix, v_prefix):
        if t.dtype != dt or t.get_device() != dev:
            raise ValueError("all tensors must share dtype and device")
    n = cu_q.numel()
    for cu in (cu_q, cu_k):
        if cu.dtype != torch.int32 or cu.get_device() != dev or cu.dim() != 1 \
                or not cu.is_contiguous() or cu.numel() != n or n < 2:
            raise ValueError("cu_seqlens_q and cu_seqlens_k: contiguous int32 CUDA vectors of B+1")
    return _PACK_PROBLEM(n - 1, qs[1], ks[1], int(max_q), int(max_k), qs[2], cu_q.data_ptr(),
                         cu_k.data_ptr(), qs[0], ks[0], bool(causal), _scale(qs[2], scale),
                         _DTYPE_CODE[dt], 0.0, 0, 0, 0)


def _like(ref, *ts):
    for t in ts:
        if t.shape != ref.shape or t.dtype != ref.dtype or t.device != ref.device:
            raise ValueError("tensors of one kind must share shape, dtype and device")


def _lse_like(q, *ts):
    for t in ts:
        if t.dtype != torch.float32 or t.device != q.device or not t.is_contiguous() \
                or t.shape != (q.shape[1], q.shape[0]):
            raise ValueError("lse, delta: contiguous float32 [Hq, total_q] on q's device")


def _addr(*ts):
    """Address and strides of packed tensors, in turn."""
    return [x for t in ts for x in (t.data_ptr(), _strides4(t))]


def _fwd_prefix(pr, q, k, v, k_prefix, v_prefix, o, lse):
    _call(load_library().fa_fwd_prefix, "fa_fwd_prefix", q.get_device(), pr, k_prefix.shape[0],
          *_addr(q, k_prefix, v_prefix, k, v, o), lse.data_ptr())


def _bwd_prefix_delta(pr, q, k, v, k_prefix, v_prefix, o, do, lse, delta):
    _call(load_library().fa_bwd_prefix_delta, "fa_bwd_prefix_delta", q.get_device(), pr,
          k_prefix.shape[0], *_addr(q, k_prefix, v_prefix, k, v, o, do), lse.data_ptr(),
          delta.data_ptr())


def _bwd_prefix(pr, q, k, v, k_prefix, v_prefix, do, lse, delta, dq, dk, dv, dk_prefix, dv_prefix):
    _call(load_library().fa_bwd_prefix, "fa_bwd_prefix", q.get_device(), pr, k_prefix.shape[0],
          *_addr(q, k_prefix, v_prefix, k, v, do), lse.data_ptr(), delta.data_ptr(),
          *_addr(dq, dk_prefix, dv_prefix, dk, dv))


def fwd_prefix(q, k, v, k_prefix, v_prefix, o, lse, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
               max_seqlen_k, causal: bool = True, scale=None):
    """fa_fwd_prefix: q, o [total_q, Hq, D], k, v [total_k, Hkv, D], k_prefix,
    v_prefix [P, Hkv, D], lse [Hq, total_q]."""
    pr = _prefix_problem(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                         max_seqlen_k, causal, scale)
    _like(q, o)
    _lse_like(q, lse)
    _fwd_prefix(pr, q, k, v, k_prefix, v_prefix, o, lse)


def bwd_prefix_delta(q, k, v, k_prefix, v_prefix, o, do, lse, delta, cu_seqlens_q, cu_seqlens_k,
                     max_seqlen_q, max_seqlen_k, causal: bool = True, scale=None):
    """fa_bwd_prefix_delta: delta [Hq, total_q] for bwd_prefix, without the rounding
    of o in rows that see few keys."""
    pr = _prefix_problem(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                         max_seqlen_k, causal, scale)
    _like(q, o, do)
    _lse_like(q, lse, delta)
    _bwd_prefix_delta(pr, q, k, v, k_prefix, v_prefix, o, do, lse, delta)


def bwd_prefix(q, k, v, k_prefix, v_prefix, do, lse, delta, dq, dk, dv, dk_prefix, dv_prefix,
               cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal: bool = True,
               scale=None):
    """fa_bwd_prefix: the gradients of fwd_prefix from its lse and bwd_prefix_delta's
    delta = rowsum(do * o), [Hq, total_q]."""
    pr = _prefix_problem(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                         max_seqlen_k, causal, scale)
    _like(q, do, dq)
    _like(k, dk, dv)
    _like(k_prefix, dk_prefix, dv_prefix)
    _lse_like(q, lse, delta)
    _bwd_prefix(pr, q, k, v, k_prefix, v_prefix, do, lse, delta, dq, dk, dv, dk_prefix, dv_prefix)


def attention_prefix_fwd(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                         max_seqlen_k, causal: bool = True, scale=None):
    """Allocating fwd_prefix: (o, lse)."""
    pr = _prefix_problem(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                         max_seqlen_k, causal, scale)
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    _fwd_prefix(pr, q, k, v, k_prefix, v_prefix, o, lse)
    return o, lse


def attention_prefix_bwd(q, k, v, k_prefix, v_prefix, o, lse, do, cu_seqlens_q, cu_seqlens_k,
                         max_seqlen_q, max_seqlen_k, causal: bool = True, scale=None):
    """Allocating bwd_prefix: (dq, dk, dv, dk_prefix, dv_prefix)."""
    pr = _prefix_problem(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                         max_seqlen_k, causal, scale)
    _like(q, o, do)
    _lse_like(q, lse)
    delta = torch.empty_like(lse)
    _bwd_prefix_delta(pr, q, k, v, k_prefix, v_prefix, o, do, lse, delta)
    grads = [torch.empty_like(t, memory_format=torch.contiguous_format)
             for t in (q, k, v, k_prefix, v_prefix)]
    _bwd_prefix(pr, q, k, v, k_prefix, v_prefix, do, lse, delta, *grads)
    return tuple(grads)


class _AttentionPrefix(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, k_prefix, v_prefix, cu_q, cu_k, max_q, max_k, causal, scale):
        o, lse = attention_prefix_fwd(q, k, v, k_prefix, v_prefix, cu_q, cu_k, max_q, max_k, causal,
                                      scale)
        ctx.save_for_backward(q, k, v, k_prefix, v_prefix, o, lse, cu_q, cu_k)
        ctx.args = (max_q, max_k, causal, scale)
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, kp, vp, o, lse, cu_q, cu_k = ctx.saved_tensors
        grads = attention_prefix_bwd(q, k, v, kp, vp, o, lse, _dense(do), cu_q, cu_k, *ctx.args)
        return (*grads, None, None, None, None, None, None)


def attention_varlen_prefix(q, k, v, k_prefix, v_prefix, cu_seqlens_q, cu_seqlens_k,
                            max_seqlen_q: int, max_seqlen_k: int, causal: bool = True, scale=None,
                            rotary: Optional[Rotary] = None):
    """Autograd attention over packed sequences that share a prefix: q
    [total_q, Hq, D], k, v [total_k, Hkv, D], k_prefix, v_prefix [P, Hkv, D]
    (every query sees all of it; its gradients sum over the sequences),
    cu_seqlens_* int32 CUDA offsets (B+1).  causal: within each sequence, counted
    from its first row.  rotary: the rotation (and head norm) to apply to q and k
    first (not to the prefix, which is used as it is)."""
    if rotary is not None:
        q, k = apply_rotary(q, k, rotary)
    return _AttentionPrefix.apply(*(_dense(t) for t in (q, k, v, k_prefix, v_prefix)), cu_seqlens_q,
                                  cu_seqlens_k, max_seqlen_q, max_seqlen_k, causal, scale)
