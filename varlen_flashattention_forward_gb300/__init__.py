"""GB300 (sm_103a) variable-length attention forward -- Python binding.

Thin ctypes marshalling over the C ABI of ``libfa_gb300.so`` (declared in
``include/fa_gb300.h``).  Every step of the computation runs in the library's
CUDA kernels; this module only checks tensor shapes/dtypes, passes raw device
pointers and sizes, and turns status codes into exceptions.  There is no CPU
or PyTorch fallback: if the library is missing, the entry points raise.

Entry points (same names as the C ABI):
  fa_varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                max_seqlen_k, softmax_scale, causal=False, window_left=-1,
                window_right=-1, out=None, lse=None, return_lse=False,
                stream=None)
  fa_varlen_fwd_plan(batch, total_q, total_k, num_heads, num_heads_k, d_qk, d_v,
                     max_seqlen_q=0, max_seqlen_k=0, causal=False, window_left=-1,
                     window_right=-1)
  fa_sparse_mla_decode(q, kv_cache, page_table, topk_idx, softmax_scale,
                       out=None, lse=None, return_lse=False, stream=None)
  fa_sparse_mla_decode_plan(num_tokens, num_heads, topk)
  fa_sparse_mla_decode_noalloc(q, kv_cache, page_table, topk_idx, softmax_scale,
                               out, lse=None, stream=None)
  fa_merge_attn_states(prefix_out, prefix_lse, suffix_out, suffix_lse,
                       out=None, out_lse=None, stream=None)
  fa_qk_norm_rope(q, k, positions, cos_sin, q_weight=None, k_weight=None, eps=1e-6,
                  interleaved=False, q_out=None, k_out=None, stream=None)
  fa_paged_kv_append(k, v, cu_seqlens, seq_lens, page_table, k_cache, v_cache, k_scale,
                     v_scale, cos_sin=None, k_weight=None, eps=1e-6, interleaved=False,
                     stream=None)
  fa_paged_attn(q, k_cache, v_cache, k_scale, v_scale, cu_seqlens_q, seq_lens, page_table,
                max_seqlen_q=0, max_seqlen_k=0, softmax_scale=None, causal=True,
                window_left=-1, out=None, lse=None, return_lse=False, workspace=None,
                stream=None)
  fa_paged_attn_plan(batch, total_q, num_heads, num_heads_k, head_dim, max_seqlen_q=0)
  fa_paged_kv_gather(k_cache, v_cache, k_scale, v_scale, cu_seqlens, page_table, total_k,
                     k_out=None, v_out=None, stream=None)
  fa_get_device_status()
  fa_set_wait_limit_ns(ns)
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

FA_OK = 0
FA_ERR_INVALID_ARG = 1
FA_ERR_UNSUPPORTED = 2
FA_ERR_ARCH = 3
FA_ERR_LAUNCH = 4
FA_ERR_DEVICE_TIMEOUT = 5
FA_ERR_SCRATCH = 6
NOALLOC_SCRATCH_BYTES = 48 << 20  # FA_NOALLOC_SCRATCH_BYTES

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa_gb300.so")

# Exported C symbols (kept in sync with include/fa_gb300.h; a CPU test checks).
EXPORTS = ("fa_varlen_fwd", "fa_varlen_fwd_plan", "fa_varlen_fwd_strided", "fa_sparse_mla_decode",
           "fa_sparse_mla_decode_plan", "fa_sparse_mla_decode_noalloc", "fa_merge_attn_states",
           "fa_qk_norm_rope", "fa_paged_kv_append", "fa_paged_attn", "fa_paged_attn_plan",
           "fa_paged_kv_gather", "fa_get_device_status", "fa_set_wait_limit_ns", "fa_status_string")

_lib = None


class FaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def load_library():
    """Loads libfa_gb300.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (needs nvcc)")
    lib = ctypes.CDLL(LIB_PATH)
    p, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_varlen_fwd.argtypes = [p, p, p, p, p, i32, i32, i32, i32, i32, i32,
                                  i32, i32, i32, f32, i32, i32, i32, p, p, p]
    lib.fa_varlen_fwd.restype = i32
    i64 = ctypes.c_longlong
    lib.fa_varlen_fwd_strided.argtypes = [p, i64, i64, p, i64, i64, p, i64, i64, p, p, i32,
                                          i32, i32, i32, i32, i32, i32, i32, i32, f32, i32,
                                          i32, i32, p, p, p]
    lib.fa_varlen_fwd_strided.restype = i32
    lib.fa_sparse_mla_decode.argtypes = [p, p, p, p, i32, i32, i32, i32, i32,
                                         f32, p, p, p]
    lib.fa_sparse_mla_decode.restype = i32
    pi = ctypes.POINTER(i32)
    lib.fa_varlen_fwd_plan.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32, i32, i32, i32,
                                       i32, pi, pi, pi]
    lib.fa_varlen_fwd_plan.restype = i32
    lib.fa_sparse_mla_decode_plan.argtypes = [i32, i32, i32, ctypes.POINTER(i32),
                                              ctypes.POINTER(ctypes.c_size_t)]
    lib.fa_sparse_mla_decode_plan.restype = i32
    lib.fa_sparse_mla_decode_noalloc.argtypes = [p, p, p, p, i32, i32, i32, i32, i32,
                                                 f32, p, p, p]
    lib.fa_sparse_mla_decode_noalloc.restype = i32
    lib.fa_merge_attn_states.argtypes = [p, p, p, p, p, p, i32, i32, i32, p]
    lib.fa_merge_attn_states.restype = i32
    lib.fa_qk_norm_rope.argtypes = [p, i64, i64, p, i64, i64, p, p, p, p, i32, i32, i32, i32,
                                    i32, i32, i32, f32, p, i64, i64, p, i64, i64, p]
    lib.fa_qk_norm_rope.restype = i32
    lib.fa_paged_kv_append.argtypes = [p, i64, i64, p, i64, i64, p, p, p, i32, i32, i32, i32, i32,
                                       i32, p, f32, p, i32, i32, i32, p, p, p, p, p]
    lib.fa_paged_kv_append.restype = i32
    size = ctypes.c_size_t
    lib.fa_paged_attn.argtypes = [p, i64, i64, p, p, p, p, p, p, p, i32, i32, i32, i32, i32, i32,
                                  i32, i32, i32, f32, i32, i32, p, p, p, size, p]
    lib.fa_paged_attn.restype = i32
    lib.fa_paged_attn_plan.argtypes = [i32, i32, i32, i32, i32, i32, pi, pi,
                                       ctypes.POINTER(size)]
    lib.fa_paged_attn_plan.restype = i32
    lib.fa_paged_kv_gather.argtypes = [p, p, p, p, p, p, i32, i32, i32, i32, i32, i32, p, p, p]
    lib.fa_paged_kv_gather.restype = i32
    lib.fa_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.fa_set_wait_limit_ns.restype = i32
    lib.fa_get_device_status.argtypes = []
    lib.fa_get_device_status.restype = i32
    lib.fa_status_string.argtypes = [i32]
    lib.fa_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(status: int) -> str:
    try:
        return load_library().fa_status_string(int(status)).decode()
    except Exception:  # library unavailable: still give a readable message
        return f"status {status}"


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_ptr(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _window(n):
    """A window's size as a 32-bit argument: sizes past every position mean the
    same, and what is below -1 stays so (the library refuses it)."""
    return max(-2, min(int(n), 2 ** 31 - 1))


def _check(t, name, dtype, ndim, view=False):
    if t.dtype is dtype and t.dim() == ndim:
        if t.is_contiguous() or (view and t.stride(-1) == 1):
            return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    if view:
        # A strided view is passed as (pointer, row stride, head stride); the
        # library checks the strides, the innermost dimension must be dense.
        if t.stride(-1) != 1:
            raise ValueError(f"{name} must have a contiguous last dimension")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def fa_varlen_fwd(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q=0,
                  max_seqlen_k=0, softmax_scale=None, causal=False,
                  window_left=-1, window_right=-1, out=None, lse=None,
                  return_lse=False, stream=None):
    """Varlen attention forward; see fa_varlen_fwd in include/fa_gb300.h.

    q [total_q, H, d_qk], k [total_k, H_k, d_qk], v [total_k, H_k, d_v] bf16
    CUDA tensors; cu_seqlens_* int32 [batch+1] CUDA tensors.  Returns out
    [total_q, H, d_v] bf16, or (out, lse [H, total_q] fp32) if an lse buffer
    is given or return_lse is set.  q, k and v may be strided views with a
    contiguous last dimension (for example V taken out of a combined
    [tokens, heads, nope + v] buffer); they then go through
    fa_varlen_fwd_strided.
    """
    import torch
    lib = load_library()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check(t, name, torch.bfloat16, 3, view=True)
    _check(cu_seqlens_q, "cu_seqlens_q", torch.int32, 1)
    _check(cu_seqlens_k, "cu_seqlens_k", torch.int32, 1)
    total_q, H, d_qk = q.shape
    total_k, H_k, d_v = v.shape
    if k.shape[0] != total_k or k.shape[1] != H_k or k.shape[2] != d_qk:
        raise ValueError(f"k shape {tuple(k.shape)} inconsistent with q/v")
    batch = cu_seqlens_q.shape[0] - 1
    if cu_seqlens_k.shape[0] != batch + 1:
        raise ValueError("cu_seqlens_q and cu_seqlens_k differ in length")
    if softmax_scale is None:
        softmax_scale = d_qk ** -0.5
    if out is None:
        out = torch.empty((total_q, H, d_v), dtype=torch.bfloat16, device=q.device)
    else:
        _check(out, "out", torch.bfloat16, 3)
    if lse is None and return_lse:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check(lse, "lse", torch.float32, 2)
    if q.is_contiguous() and k.is_contiguous() and v.is_contiguous():
        st = lib.fa_varlen_fwd(
            _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
            batch, total_q, total_k, H, H_k, d_qk, d_v, int(max_seqlen_q),
            int(max_seqlen_k), float(softmax_scale), int(bool(causal)),
            _window(window_left), _window(window_right), _ptr(out), _ptr(lse),
            _stream_ptr(stream))
    else:
        st = lib.fa_varlen_fwd_strided(
            _ptr(q), q.stride(0), q.stride(1), _ptr(k), k.stride(0), k.stride(1),
            _ptr(v), v.stride(0), v.stride(1), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
            batch, total_q, total_k, H, H_k, d_qk, d_v, int(max_seqlen_q),
            int(max_seqlen_k), float(softmax_scale), int(bool(causal)),
            _window(window_left), _window(window_right), _ptr(out), _ptr(lse),
            _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_varlen_fwd")
    return (out, lse) if lse is not None else out


def fa_sparse_mla_decode(q, kv_cache, page_table, topk_idx, softmax_scale=None,
                         out=None, lse=None, return_lse=False, stream=None):
    """Sparse-MLA decode; see fa_sparse_mla_decode in include/fa_gb300.h.

    q [T, H, 576] bf16, kv_cache [num_pages, 64, 576] bf16, page_table
    [T, max_pages] int32, topk_idx [T, topk] int32 (CUDA tensors).  Returns
    out [T, H, 512] bf16, or (out, lse [H, T] fp32).
    """
    import torch
    lib = load_library()
    _check(q, "q", torch.bfloat16, 3)
    _check(kv_cache, "kv_cache", torch.bfloat16, 3)
    _check(page_table, "page_table", torch.int32, 2)
    _check(topk_idx, "topk_idx", torch.int32, 2)
    T, H, dq = q.shape
    if dq != 576 or kv_cache.shape[1] != 64 or kv_cache.shape[2] != 576:
        raise ValueError("q must be [T, H, 576] and kv_cache [pages, 64, 576]")
    if page_table.shape[0] != T or topk_idx.shape[0] != T:
        raise ValueError("page_table / topk_idx must have one row per token")
    if softmax_scale is None:
        softmax_scale = 576 ** -0.5
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    else:
        _check(out, "out", torch.bfloat16, 3)
    if lse is None and return_lse:
        lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    if lse is not None:
        _check(lse, "lse", torch.float32, 2)
    st = lib.fa_sparse_mla_decode(
        _ptr(q), _ptr(kv_cache), _ptr(page_table), _ptr(topk_idx), T, H,
        topk_idx.shape[1], kv_cache.shape[0], page_table.shape[1],
        float(softmax_scale), _ptr(out), _ptr(lse), _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_sparse_mla_decode")
    return (out, lse) if lse is not None else out


def fa_varlen_fwd_plan(batch, total_q, total_k, num_heads, num_heads_k, d_qk, d_v,
                       max_seqlen_q=0, max_seqlen_k=0, causal=False, window_left=-1,
                       window_right=-1):
    """(grid, split, heads_per_tile) of an fa_varlen_fwd call of these sizes
    on the current device: split > 1 means split-KV in clusters of `split`
    CTAs, heads_per_tile > 1 GQA head-group packing; see fa_varlen_fwd_plan
    in include/fa_gb300.h."""
    lib = load_library()
    g, s, p = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    st = lib.fa_varlen_fwd_plan(int(batch), int(total_q), int(total_k), int(num_heads),
                                int(num_heads_k), int(d_qk), int(d_v), int(max_seqlen_q),
                                int(max_seqlen_k), int(bool(causal)), _window(window_left),
                                _window(window_right), ctypes.byref(g), ctypes.byref(s),
                                ctypes.byref(p))
    if st != FA_OK:
        raise FaError(st, "fa_varlen_fwd_plan")
    return g.value, s.value, p.value


def fa_sparse_mla_decode_plan(num_tokens, num_heads, topk):
    """(launches, workspace_bytes) of a decode call of this size on the
    current device; see fa_sparse_mla_decode_plan in include/fa_gb300.h."""
    lib = load_library()
    n = ctypes.c_int(0)
    b = ctypes.c_size_t(0)
    st = lib.fa_sparse_mla_decode_plan(int(num_tokens), int(num_heads), int(topk),
                                       ctypes.byref(n), ctypes.byref(b))
    if st != FA_OK:
        raise FaError(st, "fa_sparse_mla_decode_plan")
    return n.value, b.value


def fa_sparse_mla_decode_noalloc(q, kv_cache, page_table, topk_idx, softmax_scale, out,
                                 lse=None, stream=None):
    """fa_sparse_mla_decode_noalloc (include/fa_gb300.h): the same decode with
    no device allocation, by the library or here.  `out` [T, H, 512] bf16 and
    (optionally) `lse` [H, T] fp32 are caller-provided.  Overlapping calls on
    one device race on the library's fixed scratch; the caller orders them."""
    import torch
    lib = load_library()
    _check(q, "q", torch.bfloat16, 3)
    _check(kv_cache, "kv_cache", torch.bfloat16, 3)
    _check(page_table, "page_table", torch.int32, 2)
    _check(topk_idx, "topk_idx", torch.int32, 2)
    _check(out, "out", torch.bfloat16, 3)
    if lse is not None:
        _check(lse, "lse", torch.float32, 2)
    T, H, dq = q.shape
    if dq != 576 or kv_cache.shape[1] != 64 or kv_cache.shape[2] != 576:
        raise ValueError("q must be [T, H, 576] and kv_cache [pages, 64, 576]")
    if page_table.shape[0] != T or topk_idx.shape[0] != T or tuple(out.shape) != (T, H, 512):
        raise ValueError("page_table / topk_idx / out must have one row per token")
    st = lib.fa_sparse_mla_decode_noalloc(
        _ptr(q), _ptr(kv_cache), _ptr(page_table), _ptr(topk_idx), T, H,
        topk_idx.shape[1], kv_cache.shape[0], page_table.shape[1],
        float(softmax_scale), _ptr(out), _ptr(lse), _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_sparse_mla_decode_noalloc")
    return out


def fa_merge_attn_states(prefix_out, prefix_lse, suffix_out, suffix_lse, out=None,
                         out_lse=None, stream=None):
    """LSE-weighted merge; see fa_merge_attn_states in include/fa_gb300.h.

    *_out bf16 [T, H, d], *_lse fp32 [H, T] CUDA tensors.  Returns (out, out_lse).
    """
    import torch
    lib = load_library()
    for name, t in (("prefix_out", prefix_out), ("suffix_out", suffix_out)):
        _check(t, name, torch.bfloat16, 3)
    for name, t in (("prefix_lse", prefix_lse), ("suffix_lse", suffix_lse)):
        _check(t, name, torch.float32, 2)
    T, H, d = prefix_out.shape
    if tuple(suffix_out.shape) != (T, H, d) or tuple(prefix_lse.shape) != (H, T) \
            or tuple(suffix_lse.shape) != (H, T):
        raise ValueError("merge inputs must be [T, H, d] outputs and [H, T] LSEs")
    if out is None:
        out = torch.empty_like(prefix_out)
    if out_lse is None:
        out_lse = torch.empty_like(prefix_lse)
    st = lib.fa_merge_attn_states(_ptr(out), _ptr(out_lse), _ptr(prefix_out), _ptr(prefix_lse),
                                  _ptr(suffix_out), _ptr(suffix_lse), T, H, d,
                                  _stream_ptr(stream))
    if st != FA_OK:
        raise FaError(st, "fa_merge_attn_states")
    return out, out_lse


def _device(stream, first, *others):
    """Index of the CUDA device that the tensors (None: left out) are on, and a
    context that makes it and the call's stream current where they are not:
    what is allocated in it belongs to that stream."""
    import torch
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on {t.device} and {first.device}: one CUDA device is needed")
    if index < 0:
        raise ValueError(f"CUDA tensors are needed, got {first.device}")
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
        return index, torch.cuda.stream(stream)
    if index != torch._C._cuda_getDevice():
        return index, torch.cuda.device(index)
    return index, _NO_CONTEXT


_NO_CONTEXT = contextlib.nullcontext()


def _raw_stream(index):
    """Pointer of the current stream of a device."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index)


def _p(t):
    """A tensor's address for an argument declared c_void_p (None: NULL)."""
    return None if t is None else t.data_ptr()


def _shape(t, name, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_rope(cos_sin, weights, d):
    """rot_dim and max_pos of a rotation table (None: no rotation)."""
    import torch
    for name, w in weights:
        if w is not None:
            _check(w, name, torch.float32, 1)
            _shape(w, name, (d,))
    if cos_sin is None:
        return 0, 0
    _check(cos_sin, "cos_sin", torch.float32, 2)
    return cos_sin.shape[1], cos_sin.shape[0]


def _check_cache(k_cache, v_cache, k_scale, v_scale, cu_seqlens, page_table):
    """(batch, pages, kv heads, head dim, pages of a sequence) of a cache."""
    import torch
    f8, f32, i32 = torch.float8_e4m3fn, torch.float32, torch.int32
    # (In one expression: these calls are made at every decode step.)
    if not (k_cache.dtype is f8 and v_cache.dtype is f8 and k_scale.dtype is f32
            and v_scale.dtype is f32 and cu_seqlens.dtype is i32 and page_table.dtype is i32
            and k_cache.dim() == 4 and k_scale.dim() == 2 and cu_seqlens.dim() == 1
            and page_table.dim() == 2 and k_cache.is_contiguous() and v_cache.is_contiguous()
            and k_scale.is_contiguous() and v_scale.is_contiguous()
            and cu_seqlens.is_contiguous() and page_table.is_contiguous()):
        _check(k_cache, "k_cache", f8, 4)
        _check(v_cache, "v_cache", f8, 4)
        _check(k_scale, "k_scale", f32, 2)
        _check(v_scale, "v_scale", f32, 2)
        _check(cu_seqlens, "cu_seqlens", i32, 1)
        _check(page_table, "page_table", i32, 2)
    shape = k_cache.shape
    pages, hk, page, d = shape
    if page != 64:
        raise ValueError(f"a cache page has 64 tokens, got {page}")
    if v_cache.shape != shape:
        _shape(v_cache, "v_cache", shape)
    scales = (pages, hk)
    if k_scale.shape != scales or v_scale.shape != scales:
        _shape(k_scale, "k_scale", scales)
        _shape(v_scale, "v_scale", scales)
    rows, width = page_table.shape
    batch = cu_seqlens.shape[0] - 1
    if rows != batch:
        raise ValueError("page_table must have one row per sequence")
    return batch, pages, hk, d, width


def fa_qk_norm_rope(q, k, positions, cos_sin, q_weight=None, k_weight=None, eps=1e-6,
                    interleaved=False, q_out=None, k_out=None, stream=None):
    """Per-head RMS norm of q and k with the position rotation, in one pass;
    see fa_qk_norm_rope in include/fa_gb300.h.

    q [T, H, d], k [T, H_k, d] bf16 (strided views allowed; either may be
    None), positions [T] int32, cos_sin [max_pos, rot_dim] fp32 (cosines, then
    sines; None: no rotation, positions may be None too), weights [d] fp32 or
    None (no norm).  Returns (q_out, k_out), contiguous unless given; q_out=q
    works in place.
    """
    import torch
    lib = load_library()
    bf16 = torch.bfloat16
    if q is not None:
        _check(q, "q", bf16, 3, view=True)
        T, H, d = q.shape
        qr, qh, _ = q.stride()
    if k is not None:
        _check(k, "k", bf16, 3, view=True)
        Tk, Hk, dk = k.shape
        kr, kh, _ = k.stride()
        if q is None:
            T, H, d, qr, qh = Tk, 0, dk, 0, 0
        elif Tk != T or dk != d:
            raise ValueError(f"k shape {tuple(k.shape)} inconsistent with q")
    elif q is None:
        raise ValueError("one of q and k is needed")
    else:
        Hk, kr, kh = 0, 0, 0
    rot, max_pos = _check_rope(cos_sin, (("q_weight", q_weight), ("k_weight", k_weight)), d)
    if positions is not None:
        _check(positions, "positions", torch.int32, 1)
        _shape(positions, "positions", (T,))
    elif rot:
        raise ValueError("positions are needed for the rotation")
    index, here = _device(stream, k if q is None else q, k, positions, cos_sin, q_weight, k_weight,
                          q_out, k_out)
    with here:
        qor = qoh = kor = koh = 0
        if q is not None and q_out is None:
            q_out = torch.empty((T, H, d), dtype=bf16, device=q.device)
            qor, qoh = H * d, d
        elif q_out is not None:
            _check(q_out, "q_out", bf16, 3, view=True)
            _shape(q_out, "q_out", (T, H, d))
            qor, qoh, _ = q_out.stride()
        if k is not None and k_out is None:
            k_out = torch.empty((T, Hk, d), dtype=bf16, device=k.device)
            kor, koh = Hk * d, d
        elif k_out is not None:
            _check(k_out, "k_out", bf16, 3, view=True)
            _shape(k_out, "k_out", (T, Hk, d))
            kor, koh, _ = k_out.stride()
        st = lib.fa_qk_norm_rope(
            _p(q), qr, qh, _p(k), kr, kh, _p(positions), _p(cos_sin), _p(q_weight), _p(k_weight),
            T, H, Hk, d, rot, max_pos, bool(interleaved), eps, _p(q_out), qor, qoh, _p(k_out),
            kor, koh, _raw_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_qk_norm_rope")
    return q_out, k_out


def fa_paged_kv_append(k, v, cu_seqlens, seq_lens, page_table, k_cache, v_cache, k_scale,
                       v_scale, cos_sin=None, k_weight=None, eps=1e-6, interleaved=False,
                       stream=None):
    """Writes new keys (normed and rotated on the way) and values into the
    paged 8-bit cache; see fa_paged_kv_append in include/fa_gb300.h.

    k, v [total, H_k, d] bf16 (strided views allowed), cu_seqlens [batch+1] and
    seq_lens [batch] int32 (lengths with the new tokens), page_table [batch,
    pages of a sequence] int32, caches [pages, H_k, 64, d] float8_e4m3fn and
    scales [pages, H_k] fp32, updated in place.
    """
    import torch
    lib = load_library()
    for name, t in (("k", k), ("v", v)):
        _check(t, name, torch.bfloat16, 3, view=True)
    batch, pages, hk, d, width = _check_cache(k_cache, v_cache, k_scale, v_scale, cu_seqlens,
                                              page_table)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    _shape(seq_lens, "seq_lens", (batch,))
    _shape(k, "k", (k.shape[0], hk, d))
    _shape(v, "v", k.shape)
    rot, max_pos = _check_rope(cos_sin, (("k_weight", k_weight),), d)
    index, here = _device(stream, k, v, cu_seqlens, seq_lens, page_table, k_cache, v_cache,
                          k_scale, v_scale, cos_sin, k_weight)
    kr, kh, _ = k.stride()
    vr, vh, _ = v.stride()
    with here:
        st = lib.fa_paged_kv_append(
            k.data_ptr(), kr, kh, v.data_ptr(), vr, vh, cu_seqlens.data_ptr(),
            seq_lens.data_ptr(), page_table.data_ptr(), batch, k.shape[0], hk, d, pages, width,
            _p(k_weight), eps, _p(cos_sin), rot, max_pos, bool(interleaved), k_cache.data_ptr(),
            v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), _raw_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_paged_kv_append")


def fa_paged_attn_plan(batch, total_q, num_heads, num_heads_k, head_dim, max_seqlen_q=0):
    """(grid, rows_per_tile, workspace_bytes) of a fa_paged_attn call of these
    sizes on the current device; see fa_paged_attn_plan in
    include/fa_gb300.h."""
    lib = load_library()
    g, r, w = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_size_t(0)
    st = lib.fa_paged_attn_plan(int(batch), int(total_q), int(num_heads), int(num_heads_k),
                                int(head_dim), int(max_seqlen_q), ctypes.byref(g),
                                ctypes.byref(r), ctypes.byref(w))
    if st != FA_OK:
        raise FaError(st, "fa_paged_attn_plan")
    return g.value, r.value, w.value


def fa_paged_attn(q, k_cache, v_cache, k_scale, v_scale, cu_seqlens_q, seq_lens, page_table,
                  max_seqlen_q=0, max_seqlen_k=0, softmax_scale=None, causal=True,
                  window_left=-1, out=None, lse=None, return_lse=False, workspace=None,
                  stream=None):
    """Attention of a few query rows per sequence over the paged 8-bit cache;
    see fa_paged_attn in include/fa_gb300.h.  (From about 64 rows a sequence on,
    fa_paged_kv_gather and fa_varlen_fwd are faster.)

    q [total_q, H, d] bf16 (strided view allowed), caches and scales as
    fa_paged_kv_append, cu_seqlens_q [batch+1], seq_lens [batch] and
    page_table [batch, pages of a sequence] int32.  Returns out [total_q, H, d]
    bf16, or (out, lse [H, total_q] fp32) if an lse buffer is given or
    return_lse is set.  workspace: a uint8 CUDA tensor of the bytes
    fa_paged_attn_plan gives; None allocates one for the call.
    """
    import torch
    lib = load_library()
    _check(q, "q", torch.bfloat16, 3, view=True)
    batch, pages, hk, d, width = _check_cache(k_cache, v_cache, k_scale, v_scale, cu_seqlens_q,
                                              page_table)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    _shape(seq_lens, "seq_lens", (batch,))
    T, H, dq = q.shape
    if dq != d:
        raise ValueError(f"q has head dim {dq}, the cache {d}")
    # (Now: the workspace's size is looked up by the values of these sizes.)
    max_seqlen_q, max_seqlen_k = int(max_seqlen_q), int(max_seqlen_k)
    if softmax_scale is None:
        softmax_scale = d ** -0.5
    index, here = _device(stream, q, k_cache, v_cache, k_scale, v_scale, cu_seqlens_q, seq_lens,
                          page_table, out, lse, workspace)
    with here:
        if out is None:
            out = torch.empty((T, H, d), dtype=torch.bfloat16, device=q.device)
        else:
            _check(out, "out", torch.bfloat16, 3)
            _shape(out, "out", (T, H, d))
        if lse is not None:
            _check(lse, "lse", torch.float32, 2)
            _shape(lse, "lse", (H, T))
        elif return_lse:
            lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
        if workspace is None:
            need = _attn_workspace(index, batch, T, H, hk, d, max_seqlen_q)
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        else:
            _check(workspace, "workspace", torch.uint8, 1)
            need = workspace.shape[0]
        qr, qh, _ = q.stride()
        st = lib.fa_paged_attn(
            q.data_ptr(), qr, qh, k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
            v_scale.data_ptr(), cu_seqlens_q.data_ptr(), seq_lens.data_ptr(),
            page_table.data_ptr(), batch, T, H, hk, d, pages, width, max_seqlen_q, max_seqlen_k,
            softmax_scale, bool(causal), _window(window_left), out.data_ptr(), _p(lse),
            workspace.data_ptr(), need, _raw_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_paged_attn")
    return (out, lse) if lse is not None else out


@functools.lru_cache(maxsize=1024)
def _attn_workspace(index, batch, total_q, num_heads, num_heads_k, head_dim, max_seqlen_q):
    """Workspace bytes of a fa_paged_attn call on the current device `index`."""
    return fa_paged_attn_plan(batch, total_q, num_heads, num_heads_k, head_dim, max_seqlen_q)[2]


def fa_paged_kv_gather(k_cache, v_cache, k_scale, v_scale, cu_seqlens, page_table, total_k,
                       k_out=None, v_out=None, stream=None):
    """The first cu_seqlens[b+1] - cu_seqlens[b] cached tokens of each sequence
    as packed bf16 k and v [total_k, H_k, d], ready for fa_varlen_fwd; see
    fa_paged_kv_gather in include/fa_gb300.h.  total_k is cu_seqlens[-1], on
    the host."""
    import torch
    lib = load_library()
    batch, pages, hk, d, width = _check_cache(k_cache, v_cache, k_scale, v_scale, cu_seqlens,
                                              page_table)
    index, here = _device(stream, k_cache, v_cache, k_scale, v_scale, cu_seqlens, page_table,
                          k_out, v_out)
    with here:
        shape = (total_k, hk, d)
        if k_out is None:
            k_out = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
        else:
            _check(k_out, "k_out", torch.bfloat16, 3)
            _shape(k_out, "k_out", shape)
        if v_out is None:
            v_out = torch.empty(shape, dtype=torch.bfloat16, device=k_cache.device)
        else:
            _check(v_out, "v_out", torch.bfloat16, 3)
            _shape(v_out, "v_out", shape)
        st = lib.fa_paged_kv_gather(
            k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
            cu_seqlens.data_ptr(), page_table.data_ptr(), batch, total_k, hk, d, pages, width,
            k_out.data_ptr(), v_out.data_ptr(), _raw_stream(index))
    if st != FA_OK:
        raise FaError(st, "fa_paged_kv_gather")
    return k_out, v_out


def fa_set_wait_limit_ns(ns: int) -> None:
    """Time limit of the kernels' pipeline waits for later launches (0 = the
    default of 4 s); a test hook, see fa_set_wait_limit_ns in
    include/fa_gb300.h."""
    load_library().fa_set_wait_limit_ns(int(ns))


def fa_get_device_status() -> int:
    """Reads and clears the device status word (synchronises the device)."""
    return int(load_library().fa_get_device_status())
