"""ctypes binding of libpa.so: argument marshalling only.

Every function here checks the tensors' dtype, device, contiguity and shape,
passes raw device pointers, sizes and the current CUDA stream to the C entry
point of the same name (``include/pa.h``), and raises ``PAError`` on a
non-zero status.  All computation happens in the library's kernels; if the
library is missing this module fails to import -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

library_path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpa.so")
if not os.path.exists(library_path):
    raise ImportError(f"{library_path} is missing: build it with `python -m paged_kv_cache_445_b200.csrc.build` "
                      "(needs nvcc); there is no CPU fallback")
_lib = ctypes.CDLL(library_path)

_vp, _ci, _i32p = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
_lib.pa_cache_append.argtypes = [_vp, _vp, _vp, _vp, _i32p, _ci, _ci, _ci, _ci, _ci, _vp, _vp]
_lib.pa_cache_append.restype = _ci
_lib.pa_workspace_bytes.argtypes = [_ci, _ci, _ci, _ci, _ci, _ci]
_lib.pa_workspace_bytes.restype = ctypes.c_size_t
_lib.pa_decode.argtypes = [_vp, _vp, _vp, _vp, _i32p, _ci, _i32p, _ci, _ci, _ci, _ci, _ci, _ci, ctypes.c_float,
                           _vp, ctypes.c_size_t, _vp, _vp]
_lib.pa_decode.restype = _ci
_lib.pa_prefill_chunk.argtypes = [_vp, _vp, _i32p, _vp, _vp, _i32p, _ci, _i32p, _ci, _ci, _ci, _ci, _ci, _ci, _ci,
                                  ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]
_lib.pa_prefill_chunk.restype = _ci
_lib.pa_decode_append.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32p, _ci, _i32p, _ci, _ci, _ci, _ci, _ci, _ci,
                                  ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]
_lib.pa_decode_append.restype = _ci
_lib.pa_cascade_workspace_bytes.argtypes = [_ci, _ci, _ci, _ci, _ci, _ci]
_lib.pa_cascade_workspace_bytes.restype = ctypes.c_size_t
_lib.pa_decode_cascade.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32p, _ci, _i32p, _ci, _ci, _ci, _ci, _ci, _ci,
                                   ctypes.c_float, _i32p, _i32p, _ci, _vp, ctypes.c_size_t, _vp, _vp]
_lib.pa_decode_cascade.restype = _ci
_lib.pa_cache_append_fp8.argtypes = [_vp, _vp, _vp, _vp, _i32p, _ci, _ci, _ci, _ci, _ci, ctypes.c_float,
                                     ctypes.c_float, _vp, _vp]
_lib.pa_cache_append_fp8.restype = _ci
_lib.pa_decode_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i32p, _ci, _i32p, _ci, _ci, _ci, _ci, _ci, _ci,
                               ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]
_lib.pa_decode_fp8.restype = _ci
_lib.pa_prefill_chunk_fp8.argtypes = [_vp, _vp, _i32p, _vp, _vp, _i32p, _ci, _i32p, _ci, _ci, _ci, _ci, _ci, _ci, _ci,
                                      ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp, ctypes.c_size_t, _vp, _vp]
_lib.pa_prefill_chunk_fp8.restype = _ci
_lib.pa_decode_static_scratch.argtypes = [_vp, _vp, _vp, _vp, _i32p, _ci, _i32p, _ci, _ci, _ci, _ci, _ci, _ci,
                                          ctypes.c_float, _vp, _vp]
_lib.pa_decode_static_scratch.restype = _ci
_lib.pa_status_string.argtypes = [_ci]
_lib.pa_status_string.restype = ctypes.c_char_p
PLAN_WORDS = 16  # PA_PLAN_WORDS of include/pa.h


class Plan(ctypes.Structure):
    """pa_plan: the host plan of a varlen batch (opaque words)."""
    _fields_ = [("words", ctypes.c_int32 * PLAN_WORDS)]


_lib.pa_plan_batch.argtypes = [_vp, _vp, _ci, _ci, _ci, _ci, _ci, _ci, ctypes.POINTER(Plan)]
_lib.pa_plan_batch.restype = _ci
_lib.pa_prefill_chunk_planned.argtypes = [_vp, _vp, _i32p, _vp, _vp, _i32p, _ci, _i32p, _ci, _ci, _ci, _ci, _ci, _ci,
                                          _ci, ctypes.c_float, _vp, ctypes.c_size_t, ctypes.POINTER(Plan), _vp, _vp]
_lib.pa_prefill_chunk_planned.restype = _ci
_lib.pa_calibrate_bytes.argtypes = []
_lib.pa_calibrate_bytes.restype = ctypes.c_size_t
_lib.pa_calibrate.argtypes = [_vp, ctypes.c_size_t, _vp, _vp]
_lib.pa_calibrate.restype = _ci
_lib.pa_calibration.argtypes = [ctypes.POINTER(_ci), _vp]
_lib.pa_calibration.restype = _ci
_lib.pa_calibration_clear.argtypes = []
_lib.pa_calibration_clear.restype = None
_lib.pa_last_cuda_error.argtypes = []
_lib.pa_last_cuda_error.restype = _ci
_lib.pa_last_cuda_error_string.argtypes = []
_lib.pa_last_cuda_error_string.restype = ctypes.c_char_p

_ll, _cf, _cd = ctypes.c_longlong, ctypes.c_float, ctypes.c_double


class RopeScaling(ctypes.Structure):
    """pa_rope_scaling: how rotary frequencies are scaled for long contexts."""
    _fields_ = [("type", ctypes.c_int32), ("original_positions", ctypes.c_int32), ("factor", _cd), ("low", _cd),
                ("high", _cd), ("attention_factor", _cd)]


_lib.pa_step_slots.argtypes = [_i32p] * 6 + [_ci] + [_i32p] * 3 + [_ci] * 3 + [_i32p] * 3 + [_ci, _vp, _vp]
_lib.pa_step_slots.restype = _ci
_lib.pa_rope_table.argtypes = [_vp, _ci, _ci, _cd, ctypes.POINTER(RopeScaling), _vp]
_lib.pa_rope_table.restype = _ci
_rope_args = [_vp, _vp, _ll, _vp, _ll, _vp, _ll, _vp, _vp, _vp, _ci, _ci, _ci, _i32p, _i32p] + [_ci] * 6
_lib.pa_rope_append.argtypes = _rope_args + [_vp, _vp]
_lib.pa_rope_append.restype = _ci
_lib.pa_rope_append_fp8.argtypes = _rope_args + [_cf, _cf, _vp, _vp]
_lib.pa_rope_append_fp8.restype = _ci
_lib.pa_rope_append_int4.argtypes = _rope_args + [_vp, _vp]
_lib.pa_rope_append_int4.restype = _ci
_lib.pa_cache_append_int4.argtypes = [_vp, _vp, _vp, _vp, _i32p, _ci, _ci, _ci, _ci, _ci, _vp, _vp]
_lib.pa_cache_append_int4.restype = _ci
_lib.pa_cache_read_int4.argtypes = [_vp, _vp, _vp, _vp, _i32p, _ci, _ci, _ci, _ci, _ci, _vp, _vp]
_lib.pa_cache_read_int4.restype = _ci
_lib.pa_int4_workspace_bytes.argtypes = [_ci, _ci, _ci]
_lib.pa_int4_workspace_bytes.restype = ctypes.c_size_t
_lib.pa_decode_int4.argtypes = _lib.pa_decode.argtypes
_lib.pa_decode_int4.restype = _ci
_lib.pa_prefill_chunk_int4.argtypes = _lib.pa_prefill_chunk.argtypes
_lib.pa_prefill_chunk_int4.restype = _ci
_lib.pa_accept_drafts.argtypes = [_i32p, _i32p, _vp, _ll, _vp, _ll, _ci, _i32p, _i32p, _vp, _ci, _ci, _ci, _i32p,
                                  _i32p, _vp, _vp]
_lib.pa_accept_drafts.restype = _ci

PA_OK = 0
PA_ERR_NULL, PA_ERR_SHAPE, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE = -1, -2, -3, -4
PA_ERR_RANGE, PA_ERR_CUDA, PA_ERR_TIMEOUT = -5, -6, -7
PA_ERR_NO_BLOCKS = -8
STATIC_SCRATCH_BYTES = 64 * 1024 * 1024  # PA_STATIC_SCRATCH_BYTES of include/pa.h


def status_bit(code: int) -> int:
    """Bit a kernel ORs into the device status word for device error ``code``."""
    return 1 << (-code)


class PAError(RuntimeError):
    def __init__(self, code: int, detail: str | None = None):
        self.code = code
        msg = pa_status_string(code)
        super().__init__(f"{msg} ({detail})" if detail else msg)


def pa_status_string(code: int) -> str:
    return _lib.pa_status_string(int(code)).decode()


def pa_last_cuda_error() -> int:
    """cudaError_t (or CUresult) behind the last PA_ERR_CUDA on this thread; 0 if none."""
    return int(_lib.pa_last_cuda_error())


def pa_last_cuda_error_string() -> str:
    return _lib.pa_last_cuda_error_string().decode()


def _check(rc: int) -> None:
    if rc != PA_OK:
        raise PAError(rc, pa_last_cuda_error_string() if rc == PA_ERR_CUDA else None)


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int | None = None) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a CUDA device")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {tuple(t.shape)}")
    return t.data_ptr()


def _status_ptr(dev_status) -> int | None:
    if dev_status is None:
        return None
    return _dev(dev_status, "dev_status", torch.int32)


def _stream_ptr(stream) -> int | None:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream if hasattr(s, "cuda_stream") else int(s)


def pa_cache_append(k_new, v_new, k_cache, v_cache, slot_mapping, dev_status=None, stream=None) -> None:
    """Scatter k_new/v_new [T, Hkv, d] (bf16) into k_cache/v_cache
    [num_blocks, Hkv, block_size, d] at slot_mapping [T] (int32; < 0 = skip)."""
    kp = _dev(k_new, "k_new", torch.bfloat16, 3)
    vp = _dev(v_new, "v_new", torch.bfloat16, 3)
    kc = _dev(k_cache, "k_cache", torch.bfloat16, 4)
    vc = _dev(v_cache, "v_cache", torch.bfloat16, 4)
    sm = _dev(slot_mapping, "slot_mapping", torch.int32, 1)
    nb, hkv, bs, d = k_cache.shape
    if v_cache.shape != k_cache.shape or k_new.shape != v_new.shape:
        raise ValueError("k and v tensors must have the same shapes")
    if k_new.shape[1:] != (hkv, d) or slot_mapping.shape[0] != k_new.shape[0]:
        raise ValueError("k_new must be [T, Hkv, d] and slot_mapping [T]")
    _check(_lib.pa_cache_append(kp, vp, kc, vc, sm, k_new.shape[0], nb, hkv, d, bs, _status_ptr(dev_status),
                                _stream_ptr(stream)))


def pa_workspace_bytes(num_query_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                       max_blocks_per_seq: int, block_size: int) -> int:
    n = int(_lib.pa_workspace_bytes(num_query_tokens, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                                    block_size))
    if n == 0:
        raise PAError(PA_ERR_UNSUPPORTED)
    return n


def make_workspace(num_query_tokens: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                   max_blocks_per_seq: int, block_size: int, device=None) -> torch.Tensor:
    """A zero-filled workspace of pa_workspace_bytes() bytes (the zero fill is required once)."""
    n = pa_workspace_bytes(num_query_tokens, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def _attention_args(out, q, k_cache, v_cache, block_tables, context_lens, workspace):
    op = _dev(out, "out", torch.bfloat16, 3)
    qp = _dev(q, "q", torch.bfloat16, 3)
    kc = _dev(k_cache, "k_cache", torch.bfloat16, 4)
    vc = _dev(v_cache, "v_cache", torch.bfloat16, 4)
    bt = _dev(block_tables, "block_tables", torch.int32, 2)
    cl = _dev(context_lens, "context_lens", torch.int32, 1)
    ws = _dev(workspace, "workspace", torch.uint8, 1)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if v_cache.shape != k_cache.shape or k_cache.shape[3] != q.shape[2]:
        raise ValueError("k_cache/v_cache must be [num_blocks, Hkv, block_size, d] with q's d")
    if block_tables.shape[0] != context_lens.shape[0]:
        raise ValueError("block_tables and context_lens must have one row per sequence")
    return op, qp, kc, vc, bt, cl, ws


def pa_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace, dev_status=None,
              stream=None) -> None:
    """One decode row per sequence: q/out [B, Hq, d]; see include/pa.h."""
    op, qp, kc, vc, bt, cl, ws = _attention_args(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    nb, hkv, bs, d = k_cache.shape
    if q.shape[0] != context_lens.shape[0]:
        raise ValueError("pa_decode takes exactly one query row per sequence")
    _check(_lib.pa_decode(op, qp, kc, vc, bt, block_tables.shape[1], cl, context_lens.shape[0], q.shape[1], hkv, d,
                          bs, nb, float(scale), ws, workspace.numel(), _status_ptr(dev_status), _stream_ptr(stream)))


def pa_decode_append(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                     dev_status=None, stream=None) -> None:
    """pa_cache_append of each sequence's newest row (k_new / v_new [B, Hkv, d],
    written at position context_lens[s] - 1 through the block table) and
    pa_decode, in one launch; see include/pa.h."""
    op, qp, kc, vc, bt, cl, ws = _attention_args(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    kn = _dev(k_new, "k_new", torch.bfloat16, 3)
    vn = _dev(v_new, "v_new", torch.bfloat16, 3)
    nb, hkv, bs, d = k_cache.shape
    if q.shape[0] != context_lens.shape[0]:
        raise ValueError("pa_decode_append takes exactly one query row per sequence")
    if k_new.shape != (context_lens.shape[0], hkv, d) or v_new.shape != k_new.shape:
        raise ValueError("k_new / v_new must be [num_seqs, Hkv, d]")
    _check(_lib.pa_decode_append(op, qp, kn, vn, kc, vc, bt, block_tables.shape[1], cl, context_lens.shape[0],
                                 q.shape[1], hkv, d, bs, nb, float(scale), ws, workspace.numel(),
                                 _status_ptr(dev_status), _stream_ptr(stream)))


def pa_cascade_workspace_bytes(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                               max_blocks_per_seq: int, block_size: int) -> int:
    n = int(_lib.pa_cascade_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq,
                                            block_size))
    if n == 0:
        raise PAError(PA_ERR_UNSUPPORTED)
    return n


def make_cascade_workspace(num_seqs: int, num_q_heads: int, num_kv_heads: int, head_dim: int,
                           max_blocks_per_seq: int, block_size: int, device=None) -> torch.Tensor:
    """A zero-filled workspace of pa_cascade_workspace_bytes() bytes."""
    n = pa_cascade_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, head_dim, max_blocks_per_seq, block_size)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def pa_decode_cascade(out, q, k_cache, v_cache, block_tables, context_lens, scale, group_start, group_prefix,
                      workspace, k_new=None, v_new=None, dev_status=None, stream=None) -> None:
    """Decode attention for a batch with shared-prefix groups (sequences
    group_start[g] .. group_start[g+1]-1 share their first group_prefix[g]
    tokens); with k_new / v_new the step's append is fused in.  See include/pa.h."""
    op, qp, kc, vc, bt, cl, ws = _attention_args(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    gs = _dev(group_start, "group_start", torch.int32, 1)
    gp = _dev(group_prefix, "group_prefix", torch.int32, 1)
    if group_start.shape[0] != group_prefix.shape[0] + 1:
        raise ValueError("group_start must have one more entry than group_prefix")
    nb, hkv, bs, d = k_cache.shape
    if q.shape[0] != context_lens.shape[0]:
        raise ValueError("pa_decode_cascade takes exactly one query row per sequence")
    kn = vn = None
    if k_new is not None or v_new is not None:
        kn = _dev(k_new, "k_new", torch.bfloat16, 3)
        vn = _dev(v_new, "v_new", torch.bfloat16, 3)
        if k_new.shape != (context_lens.shape[0], hkv, d) or v_new.shape != k_new.shape:
            raise ValueError("k_new / v_new must be [num_seqs, Hkv, d]")
    _check(_lib.pa_decode_cascade(op, qp, kn, vn, kc, vc, bt, block_tables.shape[1], cl, context_lens.shape[0],
                                  q.shape[1], hkv, d, bs, nb, float(scale), gs, gp, group_prefix.shape[0], ws,
                                  workspace.numel(), _status_ptr(dev_status), _stream_ptr(stream)))


def pa_cache_append_fp8(k_new, v_new, k_cache, v_cache, slot_mapping, k_scale, v_scale, dev_status=None,
                        stream=None) -> None:
    """Append into an FP8 (E4M3 codes, uint8) cache with per-tensor scales; see include/pa.h."""
    kp = _dev(k_new, "k_new", torch.bfloat16, 3)
    vp = _dev(v_new, "v_new", torch.bfloat16, 3)
    kc = _dev(k_cache, "k_cache", torch.uint8, 4)
    vc = _dev(v_cache, "v_cache", torch.uint8, 4)
    sm = _dev(slot_mapping, "slot_mapping", torch.int32, 1)
    nb, hkv, bs, d = k_cache.shape
    if v_cache.shape != k_cache.shape or k_new.shape[1:] != (hkv, d) or v_new.shape != k_new.shape:
        raise ValueError("k_new/v_new [T, Hkv, d] and caches [num_blocks, Hkv, block_size, d] must agree")
    _check(_lib.pa_cache_append_fp8(kp, vp, kc, vc, sm, k_new.shape[0], nb, hkv, d, bs, float(k_scale),
                                    float(v_scale), _status_ptr(dev_status), _stream_ptr(stream)))


def pa_decode_fp8(out, q, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale, workspace,
                  k_new=None, v_new=None, dev_status=None, stream=None) -> None:
    """Decode over an FP8 cache; with k_new / v_new the step's append is fused in.  See include/pa.h."""
    op = _dev(out, "out", torch.bfloat16, 3)
    qp = _dev(q, "q", torch.bfloat16, 3)
    kc = _dev(k_cache, "k_cache", torch.uint8, 4)
    vc = _dev(v_cache, "v_cache", torch.uint8, 4)
    bt = _dev(block_tables, "block_tables", torch.int32, 2)
    cl = _dev(context_lens, "context_lens", torch.int32, 1)
    ws = _dev(workspace, "workspace", torch.uint8, 1)
    nb, hkv, bs, d = k_cache.shape
    if out.shape != q.shape or v_cache.shape != k_cache.shape or q.shape[2] != d:
        raise ValueError("out/q [B, Hq, d] and caches [num_blocks, Hkv, block_size, d] must agree")
    if q.shape[0] != context_lens.shape[0] or block_tables.shape[0] != context_lens.shape[0]:
        raise ValueError("one query row, one block-table row and one length per sequence")
    kn = vn = None
    if k_new is not None or v_new is not None:
        kn = _dev(k_new, "k_new", torch.bfloat16, 3)
        vn = _dev(v_new, "v_new", torch.bfloat16, 3)
        if k_new.shape != (context_lens.shape[0], hkv, d) or v_new.shape != k_new.shape:
            raise ValueError("k_new / v_new must be [num_seqs, Hkv, d]")
    _check(_lib.pa_decode_fp8(op, qp, kn, vn, kc, vc, bt, block_tables.shape[1], cl, context_lens.shape[0],
                              q.shape[1], hkv, d, bs, nb, float(scale), float(k_scale), float(v_scale), ws,
                              workspace.numel(), _status_ptr(dev_status), _stream_ptr(stream)))


def pa_prefill_chunk(out, q, query_start, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                     dev_status=None, stream=None) -> None:
    """Varlen batch of prefill chunks, multi-token verification rows and
    decodes: q/out [Tq, Hq, d], query_start [B + 1]; see include/pa.h (which
    kernel takes which sequences)."""
    op, qp, kc, vc, bt, cl, ws = _attention_args(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    qs = _dev(query_start, "query_start", torch.int32, 1)
    if query_start.shape[0] != context_lens.shape[0] + 1:
        raise ValueError("query_start must have num_seqs + 1 entries")
    nb, hkv, bs, d = k_cache.shape
    _check(_lib.pa_prefill_chunk(op, qp, qs, kc, vc, bt, block_tables.shape[1], cl, context_lens.shape[0], q.shape[0],
                                 q.shape[1], hkv, d, bs, nb, float(scale), ws, workspace.numel(),
                                 _status_ptr(dev_status), _stream_ptr(stream)))


def _host_i32(a, name):
    import numpy as np
    if isinstance(a, torch.Tensor):
        if a.is_cuda:
            raise ValueError(f"{name} must be a host array (the plan is made on the host)")
        a = a.numpy()
    a = np.ascontiguousarray(a, dtype=np.int32)
    if a.ndim != 1:
        raise ValueError(f"{name} must be one-dimensional")
    return a


def pa_prefill_chunk_fp8(out, q, query_start, k_cache, v_cache, block_tables, context_lens, scale, k_scale, v_scale,
                         workspace, dev_status=None, stream=None) -> None:
    """pa_prefill_chunk over E4M3 caches (uint8 [num_blocks, Hkv, block_size, d])
    with per-tensor scales, as pa_decode_fp8."""
    op = _dev(out, "out", torch.bfloat16, 3)
    qp = _dev(q, "q", torch.bfloat16, 3)
    kc = _dev(k_cache, "k_cache", torch.uint8, 4)
    vc = _dev(v_cache, "v_cache", torch.uint8, 4)
    bt = _dev(block_tables, "block_tables", torch.int32, 2)
    cl = _dev(context_lens, "context_lens", torch.int32, 1)
    qs = _dev(query_start, "query_start", torch.int32, 1)
    ws = _dev(workspace, "workspace", torch.uint8, 1)
    if out.shape != q.shape or v_cache.shape != k_cache.shape or k_cache.shape[3] != q.shape[2]:
        raise ValueError("out/q [Tq, Hq, d] and caches [num_blocks, Hkv, block_size, d] must agree")
    if query_start.shape[0] != context_lens.shape[0] + 1 or block_tables.shape[0] != context_lens.shape[0]:
        raise ValueError("query_start must have num_seqs + 1 entries, one table row per sequence")
    nb, hkv, bs, d = k_cache.shape
    _check(_lib.pa_prefill_chunk_fp8(op, qp, qs, kc, vc, bt, block_tables.shape[1], cl, context_lens.shape[0],
                                     q.shape[0], q.shape[1], hkv, d, bs, nb, float(scale), float(k_scale),
                                     float(v_scale), ws, workspace.numel(), _status_ptr(dev_status),
                                     _stream_ptr(stream)))


def pa_plan_batch(query_start, context_lens, num_q_heads: int, num_kv_heads: int, head_dim: int, block_size: int,
                  max_blocks_per_seq: int) -> Plan:
    """Host plan of a varlen batch from HOST copies of query_start [B + 1] and
    context_lens [B]: which kernels have work, and how decode rows and
    prefill chunks share the SMs.  Make it with the device current that runs
    the call."""
    qs = _host_i32(query_start, "query_start")
    cl = _host_i32(context_lens, "context_lens")
    if qs.shape[0] != cl.shape[0] + 1:
        raise ValueError("query_start must have num_seqs + 1 entries")
    plan = Plan()
    _check(_lib.pa_plan_batch(qs.ctypes.data, cl.ctypes.data, cl.shape[0], num_q_heads, num_kv_heads, head_dim,
                              block_size, max_blocks_per_seq, ctypes.byref(plan)))
    return plan


def pa_prefill_chunk_planned(out, q, query_start, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                             plan: Plan, dev_status=None, stream=None) -> None:
    """pa_prefill_chunk with a plan from pa_plan_batch (made for this batch)."""
    op, qp, kc, vc, bt, cl, ws = _attention_args(out, q, k_cache, v_cache, block_tables, context_lens, workspace)
    qs = _dev(query_start, "query_start", torch.int32, 1)
    if query_start.shape[0] != context_lens.shape[0] + 1:
        raise ValueError("query_start must have num_seqs + 1 entries")
    if not isinstance(plan, Plan):
        raise TypeError("plan must come from pa_plan_batch")
    nb, hkv, bs, d = k_cache.shape
    _check(_lib.pa_prefill_chunk_planned(op, qp, qs, kc, vc, bt, block_tables.shape[1], cl, context_lens.shape[0],
                                         q.shape[0], q.shape[1], hkv, d, bs, nb, float(scale), ws, workspace.numel(),
                                         ctypes.byref(plan), _status_ptr(dev_status), _stream_ptr(stream)))


def pa_calibrate(buffer: torch.Tensor | None = None, dev_status=None, stream=None) -> list[int]:
    """Time the decode kernel on every SM of the current device and keep per-SM
    weights for its split of the work; returns the weights.  ``buffer``: a
    CUDA tensor of at least pa_calibrate_bytes() bytes (overwritten); one is
    allocated for the call if None.  Waits for its own work."""
    need = int(_lib.pa_calibrate_bytes())
    if need == 0:
        raise PAError(PA_ERR_CUDA, "no CUDA device")
    if buffer is None:
        buffer = torch.empty(need, dtype=torch.uint8, device="cuda")
    if not buffer.is_cuda or not buffer.is_contiguous():
        raise ValueError("buffer must be a contiguous CUDA tensor")
    _check(_lib.pa_calibrate(buffer.data_ptr(), buffer.numel() * buffer.element_size(), _status_ptr(dev_status),
                             _stream_ptr(stream)))
    return pa_calibration()


def pa_calibration() -> list[int]:
    """The per-SM rates recorded for the current device ([] if none)."""
    n = _ci(0)
    rates = (ctypes.c_uint16 * 256)()
    rc = _lib.pa_calibration(ctypes.byref(n), rates)
    if rc == PA_ERR_RANGE:
        return []
    _check(rc)
    return list(rates[:n.value])


def pa_calibration_clear() -> None:
    """Forget every device's rates: decode splits its work equally again."""
    _lib.pa_calibration_clear()


def pa_decode_static_scratch(out, q, k_cache, v_cache, block_tables, context_lens, scale, dev_status=None,
                             stream=None) -> None:
    """pa_decode without a workspace argument, for callers that cannot allocate
    device memory when they launch: the library's own per-device scratch array
    (STATIC_SCRATCH_BYTES) is used instead.  Overlapping calls on one device
    race on that array; make the first call on a device before any stream
    capture.  See include/pa.h."""
    op = _dev(out, "out", torch.bfloat16, 3)
    qp = _dev(q, "q", torch.bfloat16, 3)
    kc = _dev(k_cache, "k_cache", torch.bfloat16, 4)
    vc = _dev(v_cache, "v_cache", torch.bfloat16, 4)
    bt = _dev(block_tables, "block_tables", torch.int32, 2)
    cl = _dev(context_lens, "context_lens", torch.int32, 1)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if v_cache.shape != k_cache.shape or k_cache.shape[3] != q.shape[2]:
        raise ValueError("k_cache/v_cache must be [num_blocks, Hkv, block_size, d] with q's d")
    if block_tables.shape[0] != context_lens.shape[0] or q.shape[0] != context_lens.shape[0]:
        raise ValueError("one query row, one block-table row and one length per sequence")
    nb, hkv, bs, d = k_cache.shape
    rc = _lib.pa_decode_static_scratch(op, qp, kc, vc, bt, block_tables.shape[1], cl, context_lens.shape[0],
                                       q.shape[1], hkv, d, bs, nb, float(scale), _status_ptr(dev_status),
                                       _stream_ptr(stream))
    if rc == PA_ERR_WORKSPACE:
        raise PAError(rc, f"this batch needs more scratch than the {STATIC_SCRATCH_BYTES}-byte static array: "
                          "use pa_decode with a workspace")
    _check(rc)


# ---- the step around the attention -------------------------------------------------
# These calls run once or more per layer and step, and the small ones take less time on the GPU than a check of
# twenty tensors can take here: the checks below are few attribute reads, and say what is wrong only when something is.
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda d: torch.cuda.current_stream(d).cuda_stream)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_Tensor, _BF16, _F32, _I32, _U8 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32, torch.uint8


def _device_of(t, name: str) -> int:
    """Index of the CUDA device of a call's first tensor; all its tensors must be there."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    return dev


def _refuse(t, name, dtype, dev, shape, layout):
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the CUDA device of the call's other tensors")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be {layout}")


def _at(t, name, dtype, dev, shape) -> int:
    """Device pointer of a contiguous tensor of this type, device and shape."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev \
            and t.is_contiguous():
        return t.data_ptr()
    _refuse(t, name, dtype, dev, shape, "contiguous")


def _rows_at(t, name, dtype, dev, shape):
    """Device pointer and row stride (elements) of a tensor whose rows are contiguous."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev:
        width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
        if t.is_contiguous():
            return t.data_ptr(), width
        st = t.stride()
        if st[-1] == 1 and (len(st) == 2 or st[1] == shape[2] or shape[1] == 1):
            return t.data_ptr(), st[0] if shape[0] > 1 else width
    _refuse(t, name, dtype, dev, shape, "contiguous within each row")


def _status_at(dev_status, dev):
    return None if dev_status is None else _at(dev_status, "dev_status", _I32, dev, (1,))


def _shape(t, name, ndim):
    if not isinstance(t, _Tensor) or t.dim() != ndim:
        raise ValueError(f"{name} must be a tensor of {ndim} dimensions")
    return t.shape


def _call(fn, dev, stream, *args) -> None:
    """fn(*args, stream) with device `dev` current, on `stream` or that device's current one."""
    if _current_device() == dev:
        rc = fn(*args, _raw_stream(dev) if stream is None else _stream_ptr(stream))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if rc != PA_OK:
        _check(rc)


def pa_step_slots(new_tokens, context_lens, blocks_held, block_tables, free_blocks, free_state, block_size,
                  query_start, positions, slot_mapping, context_lens_out=None, blocks_held_out=None,
                  free_state_out=None, dev_status=None, stream=None) -> None:
    """Block tables, row offsets, positions and slots of a step from request
    lengths, all int32 on the GPU; see include/pa.h.  new_tokens, context_lens,
    blocks_held [B], block_tables [B, max_blocks], free_blocks [num_blocks],
    free_state [2] (head, count); query_start [B + 1], positions and
    slot_mapping [max_tokens] are written.  The lengths, held counts and queue
    state are updated in place unless other outputs are given."""
    if context_lens_out is None:
        context_lens_out = context_lens
    if blocks_held_out is None:
        blocks_held_out = blocks_held
    if free_state_out is None:
        free_state_out = free_state
    dev = _device_of(new_tokens, "new_tokens")
    (b,), (t,), (nb,) = _shape(new_tokens, "new_tokens", 1), _shape(positions, "positions", 1), _shape(
        free_blocks, "free_blocks", 1)
    width = _shape(block_tables, "block_tables", 2)[1]
    _call(_lib.pa_step_slots, dev, stream, _at(new_tokens, "new_tokens", _I32, dev, (b,)),
          _at(context_lens, "context_lens", _I32, dev, (b,)),
          _at(context_lens_out, "context_lens_out", _I32, dev, (b,)),
          _at(blocks_held, "blocks_held", _I32, dev, (b,)), _at(blocks_held_out, "blocks_held_out", _I32, dev, (b,)),
          _at(block_tables, "block_tables", _I32, dev, (b, width)), width,
          _at(free_blocks, "free_blocks", _I32, dev, (nb,)), _at(free_state, "free_state", _I32, dev, (2,)),
          _at(free_state_out, "free_state_out", _I32, dev, (2,)), b, nb, block_size,
          _at(query_start, "query_start", _I32, dev, (b + 1,)), _at(positions, "positions", _I32, dev, (t,)),
          _at(slot_mapping, "slot_mapping", _I32, dev, (t,)), t, _status_at(dev_status, dev))


ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}  # pa_rope_type of include/pa.h


def pa_rope_table(table, base=10000.0, scaling="none", factor=1.0, original_positions=0, low=None, high=None,
                  attention_factor=0.0, stream=None) -> None:
    """Fill table [positions, rot_dim] (float32) with the cosines, then the
    sines, of rotary positions; scaling: "none", "linear", "ntk", "yarn" or
    "bands" (low and high default to 1 and 32, for bands 1 and 4).  See
    include/pa.h."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
    dev = _device_of(table, "table")
    shape = _shape(table, "table", 2)
    sc = RopeScaling(ROPE_SCALINGS[scaling], int(original_positions), float(factor), 1.0 if low is None else float(low),
                     (4.0 if scaling == "bands" else 32.0) if high is None else float(high), float(attention_factor))
    _call(_lib.pa_rope_table, dev, stream, _at(table, "table", _F32, dev, shape), shape[0], shape[1], float(base),
          ctypes.byref(sc))


def _rope_call(fn, cache_dtype, int4, q_out, q, k_new, v_new, k_cache, v_cache, table, positions, slot_mapping,
               interleaved, scales, dev_status, stream):
    dev = _device_of(q, "q")
    t, hq, d = shape = _shape(q, "q", 3)
    hkv = _shape(k_new, "k_new", 3)[1]
    new = (t, hkv, d)
    nb, _, bs, _ = _shape(k_cache, "k_cache", 4)
    cache = (nb, hkv, bs, d * 9 // 16 if int4 else d)
    length, rot = _shape(table, "table", 2)
    qp, qs = _rows_at(q, "q", _BF16, dev, shape)
    kp, ks = _rows_at(k_new, "k_new", _BF16, dev, new)
    vp, vs = _rows_at(v_new, "v_new", _BF16, dev, new)
    _call(fn, dev, stream, _at(q_out, "q_out", _BF16, dev, shape), qp, qs, kp, ks, vp, vs,
          _at(k_cache, "k_cache", cache_dtype, dev, cache), _at(v_cache, "v_cache", cache_dtype, dev, cache),
          _at(table, "table", _F32, dev, (length, rot)), length, rot, 1 if interleaved else 0,
          _at(positions, "positions", _I32, dev, (t,)), _at(slot_mapping, "slot_mapping", _I32, dev, (t,)), t, nb, hq,
          hkv, d, bs, *scales, _status_at(dev_status, dev))


def pa_rope_append(q_out, q, k_new, v_new, k_cache, v_cache, table, positions, slot_mapping, interleaved=False,
                   dev_status=None, stream=None) -> None:
    """Rotate q [T, Hq, d] into q_out and k_new [T, Hkv, d] into the bf16 cache
    by table row positions[t]; v_new goes to the cache unrotated.  q, k_new and
    v_new may be views of one projection's output (contiguous within a token);
    q_out may be q.  See include/pa.h."""
    _rope_call(_lib.pa_rope_append, _BF16, False, q_out, q, k_new, v_new, k_cache, v_cache, table, positions,
               slot_mapping, interleaved, (), dev_status, stream)


def pa_rope_append_fp8(q_out, q, k_new, v_new, k_cache, v_cache, table, positions, slot_mapping, k_scale, v_scale,
                       interleaved=False, dev_status=None, stream=None) -> None:
    """pa_rope_append into an FP8 (E4M3 codes, uint8) cache with per-tensor scales."""
    _rope_call(_lib.pa_rope_append_fp8, _U8, False, q_out, q, k_new, v_new, k_cache, v_cache, table, positions,
               slot_mapping, interleaved, (float(k_scale), float(v_scale)), dev_status, stream)


def pa_rope_append_int4(q_out, q, k_new, v_new, k_cache, v_cache, table, positions, slot_mapping, interleaved=False,
                        dev_status=None, stream=None) -> None:
    """pa_rope_append into a 4-bit cache (uint8 [num_blocks, Hkv, block_size, d * 9 / 16])."""
    _rope_call(_lib.pa_rope_append_int4, _U8, True, q_out, q, k_new, v_new, k_cache, v_cache, table, positions,
               slot_mapping, interleaved, (), dev_status, stream)


def _int4_rows(fn, names, dtype, k, v, k_cache, v_cache, slot_mapping, dev_status, stream):
    dev = _device_of(k, names[0])
    t, hkv, d = shape = _shape(k, names[0], 3)
    nb, _, bs, _ = _shape(k_cache, "k_cache", 4)
    cache = (nb, hkv, bs, d * 9 // 16)
    _call(fn, dev, stream, _at(k, names[0], dtype, dev, shape), _at(v, names[1], dtype, dev, shape),
          _at(k_cache, "k_cache", _U8, dev, cache), _at(v_cache, "v_cache", _U8, dev, cache),
          _at(slot_mapping, "slot_mapping", _I32, dev, (t,)), t, nb, hkv, d, bs, _status_at(dev_status, dev))


def pa_cache_append_int4(k_new, v_new, k_cache, v_cache, slot_mapping, dev_status=None, stream=None) -> None:
    """Quantise k_new / v_new [T, Hkv, d] (bf16) into a 4-bit cache (uint8
    [num_blocks, Hkv, block_size, d * 9 / 16]) at slot_mapping [T]; see include/pa.h."""
    _int4_rows(_lib.pa_cache_append_int4, ("k_new", "v_new"), _BF16, k_new, v_new, k_cache, v_cache, slot_mapping,
               dev_status, stream)


def pa_cache_read_int4(k_out, v_out, k_cache, v_cache, slot_mapping, dev_status=None, stream=None) -> None:
    """The rows of a 4-bit cache in slot_mapping [T] as values: k_out / v_out
    [T, Hkv, d] (float32); rows of negative slots are left as they are."""
    _int4_rows(_lib.pa_cache_read_int4, ("k_out", "v_out"), _F32, k_out, v_out, k_cache, v_cache, slot_mapping,
               dev_status, stream)


def pa_int4_workspace_bytes(num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    n = int(_lib.pa_int4_workspace_bytes(num_q_heads, num_kv_heads, head_dim))
    if n == 0:
        raise PAError(PA_ERR_UNSUPPORTED)
    return n


def make_int4_workspace(num_q_heads: int, num_kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for pa_decode_int4 / pa_prefill_chunk_int4 (the zero fill is required once; one from
    make_workspace for the same heads does too, and serves calls on other caches in turn)."""
    with torch.cuda.device(device):  # None: the current device
        n = pa_int4_workspace_bytes(num_q_heads, num_kv_heads, head_dim)
        return torch.zeros(n, dtype=torch.uint8, device="cuda")


def _int4_attention(fn, out, q, query_start, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                    dev_status, stream):
    dev = _device_of(q, "q")
    t, hq, d = shape = _shape(q, "q", 3)
    (b,) = _shape(context_lens, "context_lens", 1)
    width = _shape(block_tables, "block_tables", 2)[1]
    nb, hkv, bs, _ = _shape(k_cache, "k_cache", 4)
    cache = (nb, hkv, bs, d * 9 // 16)
    op, qp = _at(out, "out", _BF16, dev, shape), _at(q, "q", _BF16, dev, shape)
    if query_start is not None:
        head, rows = (op, qp, _at(query_start, "query_start", _I32, dev, (b + 1,))), (t,)
    elif t == b:
        head, rows = (op, qp), ()
    else:
        raise ValueError("pa_decode_int4 takes exactly one query row per sequence")
    (size,) = _shape(workspace, "workspace", 1)
    _call(fn, dev, stream, *head, _at(k_cache, "k_cache", _U8, dev, cache), _at(v_cache, "v_cache", _U8, dev, cache),
          _at(block_tables, "block_tables", _I32, dev, (b, width)), width,
          _at(context_lens, "context_lens", _I32, dev, (b,)), b, *rows, hq, hkv, d, bs, nb, float(scale),
          _at(workspace, "workspace", _U8, dev, (size,)), size, _status_at(dev_status, dev))


def pa_decode_int4(out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace, dev_status=None,
                   stream=None) -> None:
    """pa_decode over a 4-bit cache (uint8 [num_blocks, Hkv, block_size, d * 9 / 16]); see include/pa.h."""
    _int4_attention(_lib.pa_decode_int4, out, q, None, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                    dev_status, stream)


def pa_prefill_chunk_int4(out, q, query_start, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                          dev_status=None, stream=None) -> None:
    """pa_prefill_chunk over a 4-bit cache, as pa_decode_int4."""
    if query_start is None:
        raise TypeError("query_start must be a torch.Tensor")
    _int4_attention(_lib.pa_prefill_chunk_int4, out, q, query_start, k_cache, v_cache, block_tables, context_lens,
                    scale, workspace, dev_status, stream)


def pa_accept_drafts(out_tokens, num_accepted, target_probs, draft_probs, tokens, query_start, uniforms,
                     context_lens=None, context_lens_out=None, dev_status=None, stream=None) -> None:
    """Which drafted tokens a verification step keeps and the token after them:
    target_probs [rows, vocab] and draft_probs (the same, or None: drafts that
    were looked up) in float32 or bfloat16, tokens [rows] the token fed at each
    row, query_start [B + 1], uniforms [rows] in [0, 1).  out_tokens [rows] and
    num_accepted [B] are written; context_lens [B], if given, lose the rows not
    kept (in place, or into context_lens_out).  See include/pa.h."""
    dev = _device_of(target_probs, "target_probs")
    dtype = target_probs.dtype
    if dtype is not _F32 and dtype is not _BF16:
        raise TypeError("target_probs must be float32 or bfloat16")
    r, v = shape = _shape(target_probs, "target_probs", 2)
    (b,) = _shape(num_accepted, "num_accepted", 1)
    cp = co = None
    if context_lens is not None:
        cp = _at(context_lens, "context_lens", _I32, dev, (b,))
        co = cp if context_lens_out is None else _at(context_lens_out, "context_lens_out", _I32, dev, (b,))
    elif context_lens_out is not None:
        raise ValueError("context_lens_out needs context_lens")
    tp, ts = _rows_at(target_probs, "target_probs", dtype, dev, shape)
    dp, ds = (None, 0) if draft_probs is None else _rows_at(draft_probs, "draft_probs", dtype, dev, shape)
    _call(_lib.pa_accept_drafts, dev, stream, _at(out_tokens, "out_tokens", _I32, dev, (r,)),
          _at(num_accepted, "num_accepted", _I32, dev, (b,)), tp, ts, dp, ds, 1 if dtype is _BF16 else 0,
          _at(tokens, "tokens", _I32, dev, (r,)), _at(query_start, "query_start", _I32, dev, (b + 1,)),
          _at(uniforms, "uniforms", _F32, dev, (r,)), b, r, v, cp, co, _status_at(dev_status, dev))


def exported_symbols() -> list[str]:
    return ["pa_cache_append", "pa_workspace_bytes", "pa_decode", "pa_decode_append", "pa_cache_append_fp8",
            "pa_decode_fp8", "pa_cascade_workspace_bytes", "pa_decode_cascade", "pa_prefill_chunk",
            "pa_decode_static_scratch", "pa_status_string", "pa_last_cuda_error", "pa_last_cuda_error_string",
            "pa_plan_batch", "pa_prefill_chunk_planned", "pa_prefill_chunk_fp8", "pa_calibrate_bytes", "pa_calibrate", "pa_calibration",
            "pa_calibration_clear", "pa_step_slots", "pa_rope_table", "pa_rope_append", "pa_rope_append_fp8",
            "pa_rope_append_int4", "pa_cache_append_int4", "pa_cache_read_int4", "pa_int4_workspace_bytes",
            "pa_decode_int4", "pa_prefill_chunk_int4", "pa_accept_drafts"]
