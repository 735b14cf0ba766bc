"""ctypes binding of the C ABI in include/attn_bwd.h (argument marshalling only).

Every step of the computation runs in the CUDA kernels of ``libattn_bwd.so``;
this module only fills the parameter structs from torch tensors, allocates
outputs / workspace with torch (the library itself allocates nothing) and
passes the caller's current CUDA stream.  ``load()`` raises if the library has
not been built: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn_bwd.so")

ATTN_BF16, ATTN_FP16, ATTN_FP32 = 0, 1, 2
MASK_NONE, MASK_CAUSAL_TOP_LEFT, MASK_CAUSAL_BOTTOM_RIGHT, MASK_WINDOW = 0, 1, 2, 3
BIAS_NONE, BIAS_11SS, BIAS_1HSS, BIAS_BHSS, BIAS_B1SS = 0, 1, 2, 3, 4   # attn_bias_t
DET_ATOMIC, DET_ORDERED, DET_SPLIT = 0, 1, 2   # attn_det_t
STATUS = {0: "ATTN_OK", -1: "ATTN_ERR_INVALID_ARG", -2: "ATTN_ERR_UNSUPPORTED_HEADDIM",
          -3: "ATTN_ERR_WORKSPACE_TOO_SMALL", -4: "ATTN_ERR_CUDA", -5: "ATTN_ERR_DEVICE_FLAG",
          -6: "ATTN_ERR_TIMEOUT", -7: "ATTN_ERR_BAD_SEQLENS", -8: "ATTN_ERR_BAD_PAGE",
          -9: "ATTN_ERR_OUT_OF_PAGES"}
# attn_status_t codes by name (ATTN_OK, ATTN_ERR_INVALID_ARG, ...)
globals().update({name: code for code, name in STATUS.items()})

_DTYPES = {torch.bfloat16: ATTN_BF16, torch.float16: ATTN_FP16, torch.float32: ATTN_FP32}

_i32, _vp, _f32 = ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
_i64x3 = ctypes.c_int64 * 3


class AttnBwdParams(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("batch", _i32), ("nhead_q", _i32), ("nhead_kv", _i32),
                ("seqlen_q", _i32), ("seqlen_k", _i32), ("total_q", _i32), ("total_k", _i32),
                ("d_qk", _i32), ("d_v", _i32), ("cu_seqlens_q", _vp), ("cu_seqlens_k", _vp),
                ("cu_seqlens_q_padded", _vp), ("cu_seqlens_k_padded", _vp), ("mask", _i32), ("window_left", _i32), ("window_right", _i32),
                ("softmax_scale", _f32), ("deterministic", _i32),
                ("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("dout", _vp), ("lse", _vp),
                ("dq", _vp), ("dk", _vp), ("dv", _vp),
                ("stride_q", _i64x3), ("stride_k", _i64x3), ("stride_v", _i64x3), ("stride_o", _i64x3),
                ("stride_dout", _i64x3), ("stride_dq", _i64x3), ("stride_dk", _i64x3), ("stride_dv", _i64x3),
                ("bias_type", _i32), ("dropout_p", _f32), ("bias", _vp), ("dbias", _vp), ("philox_seed", _vp),
                ("philox_offset", _vp)]


class AttnFwdParams(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("batch", _i32), ("nhead_q", _i32), ("nhead_kv", _i32),
                ("seqlen_q", _i32), ("seqlen_k", _i32), ("total_q", _i32), ("total_k", _i32),
                ("d_qk", _i32), ("d_v", _i32), ("cu_seqlens_q", _vp), ("cu_seqlens_k", _vp),
                ("cu_seqlens_q_padded", _vp), ("cu_seqlens_k_padded", _vp), ("mask", _i32), ("window_left", _i32), ("window_right", _i32),
                ("softmax_scale", _f32), ("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("lse", _vp),
                ("stride_q", _i64x3), ("stride_k", _i64x3), ("stride_v", _i64x3), ("stride_o", _i64x3),
                ("bias_type", _i32), ("dropout_p", _f32), ("bias", _vp), ("philox_seed", _vp), ("philox_offset", _vp)]


class AttnHostTensors(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("o", _vp), ("dout", _vp), ("lse", _vp),
                ("dq", _vp), ("dk", _vp), ("dv", _vp)]


class AttnRopeParams(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("batch", _i32), ("seqlen", _i32), ("nhead_q", _i32), ("nhead_kv", _i32),
                ("head_dim", _i32), ("rot_dim", _i32), ("n_axes", _i32), ("interleaved", _i32), ("inverse", _i32),
                ("positions", _vp), ("stride_pos", _i64x3), ("inv_freq", _vp), ("pair_axis", _vp),
                ("q", _vp), ("k", _vp), ("q_out", _vp), ("k_out", _vp),
                ("stride_q", _i64x3), ("stride_k", _i64x3), ("stride_q_out", _i64x3), ("stride_k_out", _i64x3)]


class AttnKvCache(ctypes.Structure):
    _fields_ = [("num_pages", _i32), ("page_size", _i32), ("nhead_kv", _i32), ("d_qk", _i32), ("d_v", _i32),
                ("reserved", _i32), ("k", _vp), ("v", _vp), ("k_exp", _vp), ("v_exp", _vp),
                ("stride_k", _i64x3), ("stride_v", _i64x3)]


class AttnKvPlanParams(ctypes.Structure):
    _fields_ = [("batch", _i32), ("page_size", _i32), ("num_pages", _i32), ("max_blocks", _i32),
                ("max_tokens", _i32), ("reserved", _i32), ("new_lens", _vp), ("seqlens", _vp), ("seqlens_out", _vp),
                ("block_table", _vp), ("table_stride", ctypes.c_int64), ("free_pages", _vp), ("free_count", _vp),
                ("free_count_out", _vp), ("cu_seqlens", _vp), ("positions", _vp), ("slots", _vp), ("status", _vp)]


class AttnKvAppendParams(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("tokens", _i32), ("k", _vp), ("v", _vp), ("stride_k", _i64x3),
                ("stride_v", _i64x3), ("slots", _vp), ("cache", AttnKvCache)]


class AttnKvFwdParams(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("batch", _i32), ("nhead_q", _i32), ("total_q", _i32), ("max_seqlen_q", _i32),
                ("max_seqlen_k", _i32), ("max_blocks", _i32), ("mask", _i32), ("window_left", _i32),
                ("window_right", _i32), ("softmax_scale", _f32), ("reserved", _i32), ("cu_seqlens_q", _vp),
                ("cu_seqlens_q_padded", _vp), ("seqlens_k", _vp), ("block_table", _vp),
                ("table_stride", ctypes.c_int64), ("q", _vp), ("o", _vp), ("lse", _vp), ("stride_q", _i64x3),
                ("stride_o", _i64x3), ("cache", AttnKvCache)]


EXPORTS = ["attn_bwd_workspace_size", "attn_bwd", "attn_bwd_timed", "attn_bwd_read_status",
           "attn_fwd", "attn_status_string", "attn_bwd_static_ws", "attn_selftest_waits", "attn_bwd_host",
           "attn_rope", "attn_kv_plan", "attn_kv_append", "attn_kv_fwd_workspace_size", "attn_kv_fwd",
           "attn_kv_fwd_read_status"]

_lib = None


def load(path: str = LIB_PATH):
    """Load libattn_bwd.so and declare its signatures.  Raises if missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first (python -m head_attention_backward_gb300.build)")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.attn_bwd_workspace_size.argtypes = [P(AttnBwdParams), P(ctypes.c_size_t)]
    lib.attn_bwd_workspace_size.restype = ctypes.c_int
    lib.attn_bwd.argtypes = [P(AttnBwdParams), _vp, ctypes.c_size_t, _vp]
    lib.attn_bwd.restype = ctypes.c_int
    lib.attn_bwd_timed.argtypes = [P(AttnBwdParams), _vp, ctypes.c_size_t, _vp, P(ctypes.c_float)]
    lib.attn_bwd_timed.restype = ctypes.c_int
    lib.attn_bwd_read_status.argtypes = [_vp, _vp, P(ctypes.c_int)]
    lib.attn_bwd_read_status.restype = ctypes.c_int
    lib.attn_fwd.argtypes = [P(AttnFwdParams), _vp]
    lib.attn_fwd.restype = ctypes.c_int
    lib.attn_rope.argtypes = [P(AttnRopeParams), _vp]
    lib.attn_rope.restype = ctypes.c_int
    lib.attn_kv_plan.argtypes = [P(AttnKvPlanParams), _vp]
    lib.attn_kv_plan.restype = ctypes.c_int
    lib.attn_kv_append.argtypes = [P(AttnKvAppendParams), _vp]
    lib.attn_kv_append.restype = ctypes.c_int
    lib.attn_kv_fwd_workspace_size.argtypes = [P(AttnKvFwdParams), P(ctypes.c_size_t)]
    lib.attn_kv_fwd_workspace_size.restype = ctypes.c_int
    lib.attn_kv_fwd.argtypes = [P(AttnKvFwdParams), _vp, ctypes.c_size_t, _vp]
    lib.attn_kv_fwd.restype = ctypes.c_int
    lib.attn_kv_fwd_read_status.argtypes = [P(AttnKvFwdParams), _vp, ctypes.c_size_t, _vp, P(ctypes.c_int)]
    lib.attn_kv_fwd_read_status.restype = ctypes.c_int
    lib.attn_status_string.argtypes = [ctypes.c_int]
    lib.attn_status_string.restype = ctypes.c_char_p
    lib.attn_bwd_host.argtypes = [P(AttnBwdParams), P(AttnHostTensors), _vp, ctypes.c_size_t, _vp, _vp, _vp,
                                  ctypes.c_int]
    lib.attn_bwd_host.restype = ctypes.c_int
    _lib = lib
    return lib


class AttnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({attn_status_string(status)})")


# ------------------------------------------------------------ raw entry points

def attn_bwd_workspace_size(p: AttnBwdParams):
    n = ctypes.c_size_t(0)
    st = load().attn_bwd_workspace_size(ctypes.byref(p), ctypes.byref(n))
    return st, n.value


def attn_bwd(p: AttnBwdParams, workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    return load().attn_bwd(ctypes.byref(p), workspace, workspace_bytes, stream)


def attn_bwd_timed(p: AttnBwdParams, workspace: int, workspace_bytes: int, stream: int = 0):
    ms = (ctypes.c_float * 4)()
    st = load().attn_bwd_timed(ctypes.byref(p), workspace, workspace_bytes, stream, ms)
    return st, list(ms)


def attn_bwd_read_status(workspace: int, stream: int = 0):
    s = ctypes.c_int(0)
    st = load().attn_bwd_read_status(workspace, stream, ctypes.byref(s))
    return st, s.value


def attn_fwd(p: AttnFwdParams, stream: int = 0) -> int:
    return load().attn_fwd(ctypes.byref(p), stream)


def attn_rope(p: AttnRopeParams, stream: int = 0) -> int:
    return load().attn_rope(ctypes.byref(p), stream)


def attn_kv_plan(p: AttnKvPlanParams, stream: int = 0) -> int:
    return load().attn_kv_plan(ctypes.byref(p), stream)


def attn_kv_append(p: AttnKvAppendParams, stream: int = 0) -> int:
    return load().attn_kv_append(ctypes.byref(p), stream)


def attn_kv_fwd_workspace_size(p: AttnKvFwdParams):
    n = ctypes.c_size_t(0)
    st = load().attn_kv_fwd_workspace_size(ctypes.byref(p), ctypes.byref(n))
    return st, n.value


def attn_kv_fwd(p: AttnKvFwdParams, workspace: int, workspace_bytes: int, stream: int = 0) -> int:
    return load().attn_kv_fwd(ctypes.byref(p), workspace, workspace_bytes, stream)


def attn_kv_fwd_read_status(p: AttnKvFwdParams, workspace: int, workspace_bytes: int, stream: int = 0):
    s = ctypes.c_int(0)
    st = load().attn_kv_fwd_read_status(ctypes.byref(p), workspace, workspace_bytes, stream, ctypes.byref(s))
    return st, s.value


def attn_bwd_host(p: AttnBwdParams, host: AttnHostTensors, workspace: int, workspace_bytes: int, stream: int,
                  copy_in: int, copy_out: int, chunks: int) -> int:
    return load().attn_bwd_host(ctypes.byref(p), ctypes.byref(host), workspace, workspace_bytes, stream, copy_in,
                                copy_out, chunks)


def host_tensors(q, k, v, o, do, lse, dq, dk, dv) -> AttnHostTensors:
    """Pinned host tensors (contiguous) for attn_bwd_host."""
    h = AttnHostTensors()
    for name, t in zip(("q", "k", "v", "o", "dout", "lse", "dq", "dk", "dv"), (q, k, v, o, do, lse, dq, dk, dv)):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"host tensor {name} must be a contiguous CPU tensor (pinned for overlap)")
        setattr(h, name, t.data_ptr())
    return h


def attn_status_string(st: int) -> str:
    return load().attn_status_string(st).decode()


STATIC_WS_BYTES = 64 << 20


SELFTEST_SCRATCH_BYTES = 3 * 128 * 4 + 16


def attn_selftest_waits(scratch_ptr: int, scratch_bytes: int, stream: int = 0):
    """Runs the bounded-wait self-test; returns (rc, [status0, status1, status2])."""
    lib = load()
    fn = lib.attn_selftest_waits
    fn.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.POINTER(ctypes.c_int)]
    fn.restype = ctypes.c_int
    out = (ctypes.c_int * 3)()
    rc = fn(ctypes.c_void_p(scratch_ptr), ctypes.c_size_t(scratch_bytes), ctypes.c_void_p(stream), out)
    return rc, list(out)


def attn_bwd_static_ws(p: AttnBwdParams, stream: int = 0) -> int:
    """attn_bwd with the library's own fixed device workspace: for callers
    that cannot allocate device memory.  Problems needing more than
    STATIC_WS_BYTES of workspace are rejected (ATTN_ERR_WORKSPACE_TOO_SMALL);
    calls overlapping on the GPU share that workspace and race."""
    lib = load()
    fn = lib.attn_bwd_static_ws
    fn.argtypes = [ctypes.POINTER(AttnBwdParams), _vp]
    fn.restype = ctypes.c_int
    return fn(ctypes.byref(p), stream)


# ------------------------------------------------------- tensor marshalling

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _strides(t, group: bool):
    """{batch, row, head} element strides of a [B,S,H,D] or [T,H,D] tensor
    whose last dimension is contiguous."""
    if t.stride(-1) != 1:
        raise ValueError("the head dimension must be contiguous (stride 1)")
    if group:
        return (0, t.stride(0), t.stride(1))
    return (t.stride(0), t.stride(1), t.stride(2))


def _set_strides(p, group: bool, **tensors):
    for name, t in tensors.items():
        getattr(p, "stride_" + name)[:] = _strides(t, group)


def _shape_args(q, k, v, cu_seqlens_q, max_seqlen_q, max_seqlen_k):
    if cu_seqlens_q is None:
        b, sq, hq, dqk = q.shape
        sk, hkv, dv = k.shape[1], k.shape[2], v.shape[3]
        return dict(batch=b, nhead_q=hq, nhead_kv=hkv, seqlen_q=sq, seqlen_k=sk, total_q=0,
                    total_k=0, d_qk=dqk, d_v=dv)
    tq, hq, dqk = q.shape
    tk, hkv, dv = k.shape[0], k.shape[1], v.shape[2]
    return dict(batch=cu_seqlens_q.numel() - 1, nhead_q=hq, nhead_kv=hkv, seqlen_q=max_seqlen_q,
                seqlen_k=max_seqlen_k, total_q=tq, total_k=tk, d_qk=dqk, d_v=dv)


def bias_type_of(bias: Optional[torch.Tensor], batch: int, nhead_q: int) -> int:
    """attn_bias_t of a [bias_b, bias_h, Sq, Sk] bias (bias_b in {1, B}, bias_h
    in {1, Hq})."""
    if bias is None:
        return BIAS_NONE
    bb, bh = bias.shape[0], bias.shape[1]
    if bias.dim() != 4 or bb not in (1, batch) or bh not in (1, nhead_q):
        raise ValueError("bias must be [1 or B, 1 or Hq, Sq, Sk]")
    if bb == 1 and bh == 1:
        return BIAS_11SS
    if bb == 1:
        return BIAS_1HSS
    return BIAS_B1SS if bh == 1 else BIAS_BHSS


def _set_extras(p, q, bias, dropout_p, philox_seed, philox_offset, dbias=None):
    if bias is not None:
        if not bias.is_contiguous():
            raise ValueError("the bias must be contiguous")
        p.bias_type = bias_type_of(bias, q.shape[0], q.shape[2])
        p.bias = bias.data_ptr()
    if dbias is not None:
        p.dbias = dbias.data_ptr()
    p.dropout_p = float(dropout_p)
    p.philox_seed, p.philox_offset = _ptr(philox_seed), _ptr(philox_offset)


def bwd_params(q, k, v, o, do, lse, dq, dk, dv, *, scale, mask=MASK_NONE, left=-1, right=-1,
               deterministic=False, cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=0,
               max_seqlen_k=0, cu_seqlens_q_padded=None, cu_seqlens_k_padded=None, bias=None, dbias=None,
               dropout_p=0.0, philox_seed=None, philox_offset=None) -> AttnBwdParams:
    p = AttnBwdParams()
    p.dtype = _DTYPES[q.dtype]
    for name, val in _shape_args(q, k, v, cu_seqlens_q, max_seqlen_q, max_seqlen_k).items():
        setattr(p, name, val)
    p.cu_seqlens_q, p.cu_seqlens_k = _ptr(cu_seqlens_q), _ptr(cu_seqlens_k)
    p.cu_seqlens_q_padded, p.cu_seqlens_k_padded = _ptr(cu_seqlens_q_padded), _ptr(cu_seqlens_k_padded)
    p.mask, p.window_left, p.window_right = mask, left, right
    p.softmax_scale = scale
    p.deterministic = int(deterministic)   # False/True or an attn_det_t value (0, 1, 2)
    p.q, p.k, p.v, p.o, p.dout, p.lse = (_ptr(t) for t in (q, k, v, o, do, lse))
    p.dq, p.dk, p.dv = _ptr(dq), _ptr(dk), _ptr(dv)
    _set_strides(p, cu_seqlens_q is not None, q=q, k=k, v=v, o=o, dout=do, dq=dq, dk=dk, dv=dv)
    _set_extras(p, q, bias, dropout_p, philox_seed, philox_offset, dbias)
    return p


def fwd_params(q, k, v, o, lse, *, scale, mask=MASK_NONE, left=-1, right=-1, cu_seqlens_q=None,
               cu_seqlens_k=None, max_seqlen_q=0, max_seqlen_k=0, cu_seqlens_q_padded=None,
               cu_seqlens_k_padded=None, bias=None, dropout_p=0.0, philox_seed=None,
               philox_offset=None) -> AttnFwdParams:
    p = AttnFwdParams()
    p.dtype = _DTYPES[q.dtype]
    for name, val in _shape_args(q, k, v, cu_seqlens_q, max_seqlen_q, max_seqlen_k).items():
        setattr(p, name, val)
    p.cu_seqlens_q, p.cu_seqlens_k = _ptr(cu_seqlens_q), _ptr(cu_seqlens_k)
    p.cu_seqlens_q_padded, p.cu_seqlens_k_padded = _ptr(cu_seqlens_q_padded), _ptr(cu_seqlens_k_padded)
    p.mask, p.window_left, p.window_right = mask, left, right
    p.softmax_scale = scale
    p.q, p.k, p.v, p.o, p.lse = (_ptr(t) for t in (q, k, v, o, lse))
    _set_strides(p, cu_seqlens_q is not None, q=q, k=k, v=v, o=o)
    _set_extras(p, q, bias, dropout_p, philox_seed, philox_offset)
    return p


def workspace_bytes(p: AttnBwdParams) -> int:
    st, n = attn_bwd_workspace_size(p)
    if st != 0:
        raise AttnError(st, "attn_bwd_workspace_size")
    return n


def alloc_workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _empty_in_order_of(t, last: int):
    """An uninitialised tensor shaped like t but with last dimension `last`,
    its other dimensions laid out in t's memory order (so BHSD or SBHD inputs
    give a BHSD or SBHD output and the strides fold the same way)."""
    n = t.dim() - 1
    order = sorted(range(n), key=lambda i: -t.stride(i))
    buf = torch.empty([t.shape[i] for i in order] + [last], dtype=t.dtype, device=t.device)
    return buf.permute([order.index(i) for i in range(n)] + [n])


def attn_forward(q, k, v, *, scale, mask=MASK_NONE, left=-1, right=-1, cu_seqlens_q=None,
                 cu_seqlens_k=None, max_seqlen_q=0, max_seqlen_k=0, cu_seqlens_q_padded=None,
                 cu_seqlens_k_padded=None, stream=None, bias=None, dropout_p=0.0, philox_seed=None,
                 philox_offset=None):
    """O and LSE from the library's forward helper (outputs allocated here; the
    padding rows of a padded layout, which the helper leaves alone, hold O = 0
    and LSE = -inf)."""
    o = _empty_in_order_of(q, v.shape[-1])
    if cu_seqlens_q is None:
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device=q.device)
    else:
        o.zero_()
        lse = torch.full((q.shape[1], q.shape[0]), -math.inf, dtype=torch.float32, device=q.device)
    p = fwd_params(q, k, v, o, lse, scale=scale, mask=mask, left=left, right=right,
                   cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k,
                   max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k,
                   cu_seqlens_q_padded=cu_seqlens_q_padded, cu_seqlens_k_padded=cu_seqlens_k_padded,
                   bias=bias, dropout_p=dropout_p, philox_seed=philox_seed, philox_offset=philox_offset)
    st = attn_fwd(p, _stream(stream))
    if st != 0:
        raise AttnError(st, "attn_fwd")
    return o, lse


def attn_backward(q, k, v, o, do, lse, *, scale, mask=MASK_NONE, left=-1, right=-1,
                  deterministic=False, cu_seqlens_q=None, cu_seqlens_k=None, max_seqlen_q=0,
                  max_seqlen_k=0, cu_seqlens_q_padded=None, cu_seqlens_k_padded=None,
                  workspace=None, out=None, stream=None, check_status=True, bias=None, return_dbias=False,
                  dropout_p=0.0, philox_seed=None, philox_offset=None):
    """dQ, dK, dV (and dbias [B, Hq, Sq, Sk] when return_dbias) through attn_bwd
    (outputs and workspace allocated here unless given).  `bias` is a
    [1 or B, 1 or Hq, Sq, Sk] tensor in the dtype of q; dropout takes a
    probability and one-element int64 device tensors for the philox seed and
    offset."""
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(k), torch.empty_like(v))
    dq, dk, dv = out
    dbias = None
    if return_dbias:
        dbias = torch.empty((q.shape[0], q.shape[2], q.shape[1], k.shape[1]), dtype=q.dtype, device=q.device)
    p = bwd_params(q, k, v, o, do, lse, dq, dk, dv, scale=scale, mask=mask, left=left, right=right,
                   deterministic=deterministic, cu_seqlens_q=cu_seqlens_q, cu_seqlens_k=cu_seqlens_k,
                   max_seqlen_q=max_seqlen_q, max_seqlen_k=max_seqlen_k,
                   cu_seqlens_q_padded=cu_seqlens_q_padded, cu_seqlens_k_padded=cu_seqlens_k_padded,
                   bias=bias, dbias=dbias, dropout_p=dropout_p, philox_seed=philox_seed,
                   philox_offset=philox_offset)
    n = workspace_bytes(p)
    if workspace is None or workspace.numel() < n:
        workspace = alloc_workspace(n, q.device)
    s = _stream(stream)
    st = attn_bwd(p, workspace.data_ptr(), workspace.numel(), s)
    if st != 0:
        raise AttnError(st, "attn_bwd")
    if check_status:
        st, dev = attn_bwd_read_status(workspace.data_ptr(), s)
        if st != 0:
            raise AttnError(st, "attn_bwd_read_status")
        if dev != 0:
            raise AttnError(dev, "attn_bwd (device status)")
    if return_dbias:
        return dq, dk, dv, dbias
    return dq, dk, dv


# ------------------------------------------- rotary positions and the cache
#
# These run once per layer or step of a serving loop, often for a few
# microseconds of device time, so the marshalling is kept short: each tensor's
# attributes are read once, the whole argument struct is packed in one go (the
# layouts below are those of the ctypes mirrors above), and what is wrong is
# only worked out once something is.

_F16 = (torch.bfloat16, torch.float16)
_FLOATS = tuple(_DTYPES)
_BYTES = (torch.float8_e4m3fn, torch.uint8)
_I32, _I64 = torch.int32, torch.int64
_current_device = torch._C._cuda_getDevice
_current_raw_stream = torch._C._cuda_getCurrentRawStream

_ROPE = struct.Struct("<10i Q 3q 2Q 4Q 12q")
_CACHE = struct.Struct("<6i 4Q 6q")
_PLAN = struct.Struct("<6i 4Q q 7Q")
_APPEND = struct.Struct("<2i 2Q 6q Q")
_FWD = struct.Struct("<10i f i 4Q q 3Q 6q")
for _s, _c, _tail in ((_ROPE, AttnRopeParams, 0), (_CACHE, AttnKvCache, 0), (_PLAN, AttnKvPlanParams, 0),
                      (_APPEND, AttnKvAppendParams, 1), (_FWD, AttnKvFwdParams, 1)):
    assert _s.size + (_tail and _CACHE.size) == ctypes.sizeof(_c), _c


def _entry(name: str, nargs: int):
    """The library's function `name` for packed structs (bytes)."""
    global _entries
    f = load()[name]
    f.argtypes = [_vp] * nargs
    f.restype = ctypes.c_int
    _entries[name] = f
    return f


_entries = {}


def _check(t: torch.Tensor, what: str, dtypes, shape=None, device=None):
    """Raises ValueError if t is not of these types, shape and device."""
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype} is not one of {tuple(dtypes)}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_cuda or (device is not None and t.get_device() != device):
        raise ValueError(f"{what} must be on cuda:{device if device is not None else '?'}, not on {t.device}")


def _vector(t: torch.Tensor, what: str, n: int, index: int, dtype=_I32) -> int:
    """Address of a contiguous vector of n whole numbers on device `index`."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{what} must be a contiguous {dtype} vector of {n} on cuda:{index}; "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _rows3(t: torch.Tensor, what: str):
    """{0, row, head} strides of a [T, H, D] tensor; a dimension of one entry
    may carry any stride, so it is given the contiguous one."""
    row, head, one = t.stride()
    n, h, d = t.shape
    if one != 1 and d > 1:
        raise ValueError(f"{what}: the head dimension must be contiguous (stride 1)")
    if h == 1:
        head = d
    return 0, (row if n > 1 else h * head), head


def _on(index: int, stream):
    """(raw stream, context for allocations) of a call on device `index`.  With
    an explicit stream the outputs are allocated on it, so that the allocator
    does not hand their memory to other work while the kernels may still write
    it."""
    if index != _current_device():
        raise ValueError(f"tensors on device {index}, but the current device is {_current_device()}")
    raw = _current_raw_stream(index)
    if stream is None:
        return raw, None
    want = _stream(stream)
    if want == raw:
        return raw, None
    return want, torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(want))


def _empty(shape, dtype, device, ctx):
    if ctx is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with ctx:
        return torch.empty(shape, dtype=dtype, device=device)


def rope_frequencies(rot_dim: int, base: float = 10000.0) -> torch.Tensor:
    """The usual ladder base^(-2 i / rot_dim), i < rot_dim / 2, in 64 bits on
    the host: the inv_freq of rope()."""
    return base ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)


def rope(q, k, positions, inv_freq, *, pair_axis=None, interleaved=False, inverse=False, out=None, stream=None):
    """q and k (or None) with their rotary positions applied (attn_rope), as
    new tensors or into `out` = (q_out, k_out), which may be (q, k).

    q [T, H, D] or [B, S, H, D], k likewise with its own heads; positions int32
    [T] / [B, S], or with a leading axis dimension [n_axes, ...] for several
    axes; inv_freq and pair_axis are host tensors (float64 and uint8,
    rot_dim / 2 entries).  inverse=True is the gradient: rope(dq, dk, ...,
    inverse=True) after attn_backward."""
    dtype, index, qs = q.dtype, q.get_device(), q.shape
    code, packed = _DTYPES.get(dtype), len(qs) == 3
    if code is None or index < 0 or not (packed or len(qs) == 4):
        _check(q, "q", _FLOATS)
        raise ValueError("q must be [T, H, D] or [B, S, H, D]")
    if packed:
        batch, (seqlen, heads, dim) = 1, qs
    else:
        batch, seqlen, heads, dim = qs
    if (inv_freq.dtype is not torch.float64 or inv_freq.get_device() >= 0 or inv_freq.dim() != 1
            or not inv_freq.is_contiguous()):
        raise ValueError("inv_freq must be a contiguous float64 vector on the host")
    half = inv_freq.shape[0]
    axis_ptr = 0
    if pair_axis is not None:
        if (pair_axis.dtype is not torch.uint8 or pair_axis.get_device() >= 0 or pair_axis.shape != (half,)
                or not pair_axis.is_contiguous()):
            raise ValueError("pair_axis must be a contiguous uint8 vector on the host, as long as inv_freq")
        axis_ptr = pair_axis.data_ptr()
    # strides {axis, batch entry, row}
    ps, sp = positions.shape, positions.stride()
    n_axes = 1
    if ps == qs[:-2]:
        sp = (0, 0, *sp) if packed else (0, *sp)
    elif ps[1:] == qs[:-2]:
        n_axes = ps[0]
        if packed:
            sp = (sp[0], 0, sp[1])
    else:
        raise ValueError(f"positions {tuple(ps)} do not fit rows {tuple(qs[:-2])}")
    if positions.dtype is not _I32 or positions.get_device() != index:
        _check(positions, "positions", (_I32,), None, index)
    raw, ctx = _on(index, stream)
    if out is not None:
        qo, ko = out
        _check(qo, "out[0]", (dtype,), qs, index)
        if k is not None:
            _check(ko, "out[1]", (dtype,), k.shape, index)
    elif ctx is None:
        qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
    else:
        with ctx:
            qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
    sq, so = q.stride(), qo.stride()
    if sq[-1] != 1 or so[-1] != 1:
        raise ValueError("the head dimension must be contiguous (stride 1)")
    nk, kp, kop, sk, sko = 0, 0, 0, (0, 0, 0, 1), (0, 0, 0, 1)
    if k is not None:
        ks = k.shape
        nk = ks[-2]
        if k.dtype is not dtype or k.get_device() != index or ks[-1] != dim or ks[:-2] != qs[:-2]:
            _check(k, "k", (dtype,), (*qs[:-2], nk, dim), index)
        kp, kop, sk, sko = k.data_ptr(), ko.data_ptr(), k.stride(), ko.stride()
        if sk[-1] != 1 or sko[-1] != 1:
            raise ValueError("the head dimension must be contiguous (stride 1)")
        if packed:
            sk, sko = (0, *sk), (0, *sko)
    if packed:
        sq, so = (0, *sq), (0, *so)
    p = _ROPE.pack(code, batch, seqlen, heads, nk, dim, 2 * half, n_axes, 1 if interleaved else 0,
                   1 if inverse else 0, positions.data_ptr(), *sp, inv_freq.data_ptr(), axis_ptr, q.data_ptr(), kp,
                   qo.data_ptr(), kop, sq[0], sq[1], sq[2], sk[0], sk[1], sk[2], so[0], so[1], so[2], sko[0], sko[1],
                   sko[2])
    st = (_entries.get("attn_rope") or _entry("attn_rope", 2))(p, raw)
    if st != 0:
        raise AttnError(st, "attn_rope")
    return qo, (None if k is None else ko)


class KvCache:
    """Handle of a paged 8-bit cache (attn_kv_cache): k [pages, page_size,
    kv heads, d_qk] and v [..., d_v] as torch.float8_e4m3fn (or uint8), any
    strides with a contiguous head dimension, and the scale exponents k_exp,
    v_exp uint8 [pages, kv heads].  It keeps the tensors and their packed
    description; make it once per cache."""

    __slots__ = ("k", "v", "k_exp", "v_exp", "num_pages", "page_size", "nhead_kv", "d_qk", "d_v", "index", "packed")

    def __init__(self, k, v, k_exp, v_exp):
        index, ks, vs = k.get_device(), k.shape, v.shape
        pages, size, heads, dqk = ks
        dv = vs[3]
        sk, sv = k.stride(), v.stride()
        if (index < 0 or k.dtype not in _BYTES or v.dtype is not k.dtype or vs != (pages, size, heads, dv)
                or v.get_device() != index or sk[3] != 1 or sv[3] != 1):
            _check(k, "k", _BYTES)
            _check(v, "v", (k.dtype,), (pages, size, heads, dv), index)
            raise ValueError("the head dimension must be contiguous (stride 1)")
        es = (pages, heads)
        for name, e in (("k_exp", k_exp), ("v_exp", v_exp)):
            if e.dtype is not torch.uint8 or e.get_device() != index or e.shape != es or not e.is_contiguous():
                _check(e, name, (torch.uint8,), es, index)
                raise ValueError(f"{name} must be contiguous")
        self.k, self.v, self.k_exp, self.v_exp = k, v, k_exp, v_exp
        self.num_pages, self.page_size, self.nhead_kv, self.d_qk, self.d_v, self.index = pages, size, heads, dqk, dv, index
        self.packed = _CACHE.pack(pages, size, heads, dqk, dv, 0, k.data_ptr(), v.data_ptr(), k_exp.data_ptr(),
                                  v_exp.data_ptr(), sk[0], sk[1], sk[2], sv[0], sv[1], sv[2])

    @classmethod
    def empty(cls, num_pages, page_size, nhead_kv, d_qk, d_v, device="cuda"):
        """A new cache, zero everywhere."""
        k, v = (torch.zeros((num_pages, page_size, nhead_kv, d), dtype=torch.uint8, device=device)
                .view(torch.float8_e4m3fn) for d in (d_qk, d_v))
        e = [torch.full((num_pages, nhead_kv), 127, dtype=torch.uint8, device=device) for _ in range(2)]
        return cls(k, v, *e)


class KvPlan(NamedTuple):
    """What attn_kv_plan computes: packed segment offsets, the requests' new
    lengths, one position and slot per token, the free pages left, the status
    word (0 = ATTN_OK), all on the device."""
    cu_seqlens: torch.Tensor
    seqlens: torch.Tensor
    positions: torch.Tensor
    slots: torch.Tensor
    free_count: torch.Tensor
    status: torch.Tensor

    def check(self):
        """Synchronises; raises AttnError if the step was refused."""
        s = int(self.status)
        if s != 0:
            raise AttnError(s, "attn_kv_plan (device status)")


def _table(t: torch.Tensor, n: int, index: int):
    """(columns, row stride) of an int32 [n, columns] block table."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not _I32 or t.get_device() != index or len(shape) != 2 or shape[0] != n or stride[1] != 1:
        _check(t, "block_table", (_I32,), (n, shape[-1]), index)
        raise ValueError("block_table rows must be contiguous")
    return shape[1], (stride[0] if n > 1 else shape[1])


def kv_plan(new_lens, seqlens, block_table, free_pages, free_count, *, page_size, max_tokens, out=None, stream=None):
    """Pages, positions and slots for one step (attn_kv_plan).  new_lens and
    seqlens int32 [B] (KV_RELEASE ends a request), block_table int32
    [B, max_blocks] and free_pages int32 [num_pages] are updated in place,
    free_count int32 [1].  Returns a KvPlan, `out` itself when given: its
    seqlens and free_count may be the inputs', so that a captured call
    advances its state at every replay."""
    index, n = new_lens.get_device(), new_lens.shape[0]
    pages = free_pages.shape[0]
    cols, row = _table(block_table, n, index)
    new_p, len_p = _vector(new_lens, "new_lens", n, index), _vector(seqlens, "seqlens", n, index)
    free_p, count_p = _vector(free_pages, "free_pages", pages, index), _vector(free_count, "free_count", 1, index)
    raw, ctx = _on(index, stream)
    if out is None:
        # two blocks for six vectors: the words, the slots
        device = new_lens.device
        words, slots = _empty((2 * n + 3 + max_tokens,), _I32, device, ctx), _empty((max_tokens,), _I64, device, ctx)
        cu, lens, count, status, pos = words.split((n + 1, n, 1, 1, max_tokens))
        out = KvPlan(cu, lens, pos, slots, count, status)
        w = words.data_ptr()
        cu_p, out_p, left_p, status_p, pos_p = w, w + 4 * (n + 1), w + 4 * (2 * n + 1), w + 4 * (2 * n + 2), w + 4 * (2 * n + 3)
        slots_p = slots.data_ptr()
    else:
        cu_p, out_p = _vector(out.cu_seqlens, "out.cu_seqlens", n + 1, index), _vector(out.seqlens, "out.seqlens", n, index)
        left_p, status_p = _vector(out.free_count, "out.free_count", 1, index), _vector(out.status, "out.status", 1, index)
        pos_p = _vector(out.positions, "out.positions", max_tokens, index)
        slots_p = _vector(out.slots, "out.slots", max_tokens, index, _I64)
    p = _PLAN.pack(n, page_size, pages, cols, max_tokens, 0, new_p, len_p, out_p, block_table.data_ptr(), row, free_p,
                   count_p, left_p, cu_p, pos_p, slots_p, status_p)
    st = (_entries.get("attn_kv_plan") or _entry("attn_kv_plan", 2))(p, raw)
    if st != 0:
        raise AttnError(st, "attn_kv_plan")
    return out


def kv_append(k, v, slots, cache: KvCache, *, stream=None):
    """New keys and values into the cache (attn_kv_append): k [T, kv heads,
    d_qk] and v [T, kv heads, d_v] in bf16 or fp16, slots int64 [T] as from
    kv_plan (-1: skipped)."""
    index, ks, dtype = cache.index, k.shape, k.dtype
    n, heads = ks[0], cache.nhead_kv
    if (dtype not in _F16 or v.dtype is not dtype or ks != (n, heads, cache.d_qk) or v.shape != (n, heads, cache.d_v)
            or k.get_device() != index or v.get_device() != index):
        _check(k, "k", _F16, (n, heads, cache.d_qk), index)
        _check(v, "v", (dtype,), (n, heads, cache.d_v), index)
    raw, _ = _on(index, stream)
    p = _APPEND.pack(_DTYPES[dtype], n, k.data_ptr(), v.data_ptr(), *_rows3(k, "k"), *_rows3(v, "v"),
                     _vector(slots, "slots", n, index, _I64)) + cache.packed
    st = (_entries.get("attn_kv_append") or _entry("attn_kv_append", 2))(p, raw)
    if st != 0:
        raise AttnError(st, "attn_kv_append")


def attn_kv_forward(q, cache: KvCache, block_table, seqlens_k, cu_seqlens_q, *, scale, mask=MASK_CAUSAL_BOTTOM_RIGHT,
                    left=-1, right=-1, max_seqlen_q, max_seqlen_k, cu_seqlens_q_padded=None, out=None, workspace=None,
                    stream=None, check_status=False):
    """O [T, Hq, d_v] and LSE [Hq, T] of packed queries q [T, Hq, d_qk] over the
    cache (attn_kv_fwd).  block_table int32 [B, max_blocks], seqlens_k int32
    [B], cu_seqlens_q int32 [B + 1] as from kv_plan.  Rows of no segment are
    not written: pass `out` = (o, lse) to choose what they hold, in outputs
    allocated here they are undefined.  check_status=True synchronises and
    raises what the kernels found (lengths beyond their bounds, pages outside
    the cache)."""
    index, qs, dtype = cache.index, q.shape, q.dtype
    t, hq = qs[0], qs[1]
    if dtype not in _F16 or q.get_device() != index or len(qs) != 3 or qs[2] != cache.d_qk:
        _check(q, "q", _F16, (t, hq, cache.d_qk), index)
    n = seqlens_k.shape[0]
    cols, row = _table(block_table, n, index)
    cu_p, len_p = _vector(cu_seqlens_q, "cu_seqlens_q", n + 1, index), _vector(seqlens_k, "seqlens_k", n, index)
    pad_p = 0
    if cu_seqlens_q_padded is not None:
        pad_p = _vector(cu_seqlens_q_padded, "cu_seqlens_q_padded", n + 1, index)
    raw, ctx = _on(index, stream)
    dv = cache.d_v
    if out is None:
        device = q.device
        o, lse = _empty((t, hq, dv), dtype, device, ctx), _empty((hq, t), torch.float32, device, ctx)
        so = (0, hq * dv, dv)
    else:
        o, lse = out
        _check(o, "out[0]", (dtype,), (t, hq, dv), index)
        _check(lse, "out[1]", (torch.float32,), (hq, t), index)
        if not lse.is_contiguous():
            raise ValueError("out[1] must be contiguous")
        so = _rows3(o, "out[0]")
    p = _FWD.pack(_DTYPES[dtype], n, hq, t, max_seqlen_q, max_seqlen_k, cols, mask, left, right, scale, 0, cu_p, pad_p,
                  len_p, block_table.data_ptr(), row, q.data_ptr(), o.data_ptr(), lse.data_ptr(), *_rows3(q, "q"),
                  *so) + cache.packed
    need = ctypes.c_size_t(0)
    st = (_entries.get("attn_kv_fwd_workspace_size") or _entry("attn_kv_fwd_workspace_size", 2))(p, ctypes.addressof(need))
    if st != 0:
        raise AttnError(st, "attn_kv_fwd_workspace_size")
    if workspace is None:
        workspace = _empty((need.value,), torch.uint8, q.device, ctx)
    elif workspace.get_device() != index or workspace.dtype is not torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    ws, nbytes = workspace.data_ptr(), workspace.numel()
    st = (_entries.get("attn_kv_fwd") or _entry("attn_kv_fwd", 4))(p, ws, nbytes, raw)
    if st != 0:
        raise AttnError(st, "attn_kv_fwd")
    if check_status:
        found = ctypes.c_int(0)
        f = _entries.get("attn_kv_fwd_read_status") or _entry("attn_kv_fwd_read_status", 5)
        st = f(p, ws, nbytes, raw, ctypes.addressof(found))
        if st != 0:
            raise AttnError(st, "attn_kv_fwd_read_status")
        if found.value != 0:
            raise AttnError(found.value, "attn_kv_fwd (device status)")
    return o, lse


KV_RELEASE = -1   # ATTN_KV_RELEASE
