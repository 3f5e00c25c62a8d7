"""Thin Python binding of libverify_attn.so (C ABI in include/verify_attn.h).

Argument marshalling only: every function here takes torch tensors that live
on the GPU, checks dtypes/shapes enough to build the C call, passes raw device
pointers and the current CUDA stream, and raises ``VerifyAttnError`` when the
library returns a non-OK status.  All computation happens in the CUDA kernels;
there is no fallback path, and importing the library fails loudly when it has
not been built.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

VA_OK, VA_ERR_INVALID_ARG, VA_ERR_UNSUPPORTED, VA_ERR_WORKSPACE, VA_ERR_CUDA, VA_ERR_TIMEOUT, \
    VA_ERR_DEVICE_BOUNDS, VA_ERR_DEVICE_INVALID = range(8)
VA_DTYPE_BF16, VA_DTYPE_FP32 = 0, 2
STATUS_NAMES = {0: "VA_OK", 1: "VA_ERR_INVALID_ARG", 2: "VA_ERR_UNSUPPORTED", 3: "VA_ERR_WORKSPACE",
                4: "VA_ERR_CUDA", 5: "VA_ERR_TIMEOUT", 6: "VA_ERR_DEVICE_BOUNDS", 7: "VA_ERR_DEVICE_INVALID"}


class VerifyAttnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class VaScoreMod(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("window", ctypes.c_int), ("slopes", ctypes.c_void_p),
                ("key_start", ctypes.c_void_p), ("token_pos", ctypes.c_void_p)]


class VaShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("Hq", ctypes.c_int), ("Hkv", ctypes.c_int),
                ("D", ctypes.c_int), ("dtype", ctypes.c_int), ("scale", ctypes.c_float),
                ("rope_base", ctypes.c_float)]


class VaRows(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64)]


_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_SIGS = {
    "verify_attn_workspace_size": (_SZ, [ctypes.POINTER(VaShape)]),
    "verify_attn_workspace_init": (_I, [_P, _SZ, _P]),
    "verify_attn_dense": (_I, [ctypes.POINTER(VaShape), _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "verify_attn_paged": (_I, [ctypes.POINTER(VaShape), _P, _P, _P, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P,
                               _SZ, _P]),
    "verify_attn_sparse": (_I, [ctypes.POINTER(VaShape), _P, _P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P,
                                _SZ, _P]),
    "verify_attn_combine": (_I, [_I, _I, _I, _P, _P, _I, _P, _P, _P]),
    "verify_tree_mask_from_parents": (_I, [_I, _I, _P, _P, _P, _P]),
    "verify_build_index": (_I, [_I, _I, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "verify_accept_greedy": (_I, [_I, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "verify_commit_kv_dense": (_I, [ctypes.POINTER(VaShape), _P, _P, _I, _P, _P, _P, _P, _P, _P]),
    "verify_commit_kv_paged": (_I, [ctypes.POINTER(VaShape), _P, _P, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P]),
    "verify_rope_draft_dense": (_I, [ctypes.POINTER(VaShape), _P, _P, _I, _P, _P, ctypes.c_float, _P, _P]),
    "verify_rope_draft_paged": (_I, [ctypes.POINTER(VaShape), _P, _P, _I, _I, _P, _I, _P, _P, ctypes.c_float, _P,
                                     _P]),
    "verify_head_importance_scratch_size": (_SZ, [_I, _I, _I, _I]),
    "verify_head_importance": (_I, [ctypes.POINTER(VaShape), _P, _P, _I, _P, _P, _I, _P, _I, _P, _SZ, _P, _P]),
    "verify_attn_dense_mod": (_I, [ctypes.POINTER(VaShape), ctypes.POINTER(VaScoreMod), _P, _P, _P, _I, _P, _P, _P, _P,
                                   _P, _P, _SZ, _P]),
    "verify_attn_paged_mod": (_I, [ctypes.POINTER(VaShape), ctypes.POINTER(VaScoreMod), _P, _P, _P, _I, _I, _P, _I, _P,
                                   _P, _P, _P, _P, _P, _SZ, _P]),
    "verify_accumulate_weight_dense": (_I, [ctypes.POINTER(VaShape), ctypes.POINTER(VaScoreMod), _P, _P, _I, _P, _P, _P,
                                            _P, ctypes.c_float, _P, _I, _P, _P]),
    "verify_accumulate_weight_paged": (_I, [ctypes.POINTER(VaShape), ctypes.POINTER(VaScoreMod), _P, _P, _I, _I, _P, _I,
                                            _P, _P, _P, _P, ctypes.c_float, _P, _I, _P, _P]),
    "verify_evict_kv_scratch_size": (_SZ, [_I, _I, _I]),
    "verify_evict_kv_dense": (_I, [ctypes.POINTER(VaShape), _P, _P, _I, _P, _P, _P, _I, _P, _I, _P, _P, _SZ, _P, _P]),
    "verify_evict_kv_paged": (_I, [ctypes.POINTER(VaShape), _P, _P, _I, _I, _P, _I, _P, _P, _P, _I, _P, _I, _P, _P,
                                   _SZ, _P, _P]),
    "verify_attn_dense_quant": (_I, [_P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "verify_attn_paged_quant": (_I, [_P, _I, _P, _P, _P, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "verify_norm_rope": (_I, [_P, _P, _P, _P, _P, ctypes.c_float, _P, _P, _P, _P]),
    "verify_kv_row_bytes": (_SZ, [_I, _I]),
    "verify_quantize_kv_dense": (_I, [_P, _I, _P, _P, _P, _P, _I, _P, _P, _P, _P]),
    "verify_quantize_kv_paged": (_I, [_P, _I, _P, _P, _P, _P, _I, _I, _P, _I, _P, _P, _P, _P]),
    "verify_dequantize_kv_dense": (_I, [_P, _I, _P, _P, _I, _P, _P, _P, _P, _P, _P]),
    "verify_dequantize_kv_paged": (_I, [_P, _I, _P, _P, _I, _I, _P, _I, _P, _P, _P, _P, _P, _P]),
    "verify_attn_check_status": (_I, [_P, _P]),
    "verify_attn_last_error": (ctypes.c_char_p, []),
    "verify_attn_version": (ctypes.c_char_p, []),
    "verify_attn_selftest_wait_timeout": (_I, [_P, ctypes.c_ulonglong, _P]),
    "verify_attn_test_inject": (_I, [ctypes.c_ulonglong, _I]),
    "verify_attn_test_stall": (_I, [ctypes.c_ulonglong, _I]),
    "verify_attn_test_index_path": (_I, [_I]),
    "verify_attn_dense_noalloc": (_I, [ctypes.POINTER(VaShape), _P, _P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
}


def library_path() -> str:
    return _build.LIB


def lib(build_if_missing: bool = True):
    """The loaded ctypes library (built on first use when nvcc is available)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if build_if_missing and not _build.up_to_date():
                _build.build()
            if not os.path.exists(path):
                raise RuntimeError(f"libverify_attn.so is not built ({path}); run __graft_entry__.build()")
            L = ctypes.CDLL(path)
            for name, (res, args) in _SIGS.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def _check(status: int):
    if status != VA_OK:
        msg = lib().verify_attn_last_error().decode()
        raise VerifyAttnError(status, msg)


def _ptr(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensor arguments must be contiguous")
    return t.data_ptr()


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return VA_DTYPE_BF16
    if t.dtype == torch.float32:
        return VA_DTYPE_FP32
    raise TypeError(f"unsupported element type {t.dtype}; use bfloat16 or float32")


def make_shape(B, T, Hq, Hkv, D, dtype_code, scale=None, rope_base=0.0) -> VaShape:
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    return VaShape(int(B), int(T), int(Hq), int(Hkv), int(D), int(dtype_code), float(scale), float(rope_base))


def workspace_size(shape: VaShape) -> int:
    return int(lib().verify_attn_workspace_size(ctypes.byref(shape)))


class Workspace:
    """Caller-owned device scratch for the attention calls, initialised once."""

    def __init__(self, nbytes: int, device=None, stream=None):
        nbytes = max(int(nbytes), 256)
        self.buffer = torch.empty(nbytes + 256, dtype=torch.uint8, device=device or "cuda")
        base = self.buffer.data_ptr()
        self.offset = (-base) % 256
        self.nbytes = nbytes
        _check(lib().verify_attn_workspace_init(self.ptr, self.nbytes, _stream(stream)))

    @property
    def ptr(self) -> int:
        return self.buffer.data_ptr() + self.offset

    @classmethod
    def for_shape(cls, shape: VaShape, device=None, stream=None) -> "Workspace":
        n = workspace_size(shape)
        if n == 0:
            _check(VA_ERR_INVALID_ARG)
        return cls(n, device=device, stream=stream)


# ----------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ----------------------------------------------------------------------------

def _shape_of(q, Hkv, scale, rope_base=0.0):
    B, T, Hq, D = q.shape
    return make_shape(B, T, Hq, Hkv, D, _dtype_code(q), scale, rope_base)


def _outputs(q, out, lse):
    B, T, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Hq, T, dtype=torch.float32, device=q.device)
    return out, lse


def verify_attn_dense(q, k_cache, v_cache, seqlens, tree_parent=None, tree_mask=None, positions=None,
                      out=None, lse=None, workspace: Workspace = None, scale=None, stream=None, rope_base=0.0):
    """Dense-cache verification attention; returns (out [B][T][Hq][D], lse [B][Hq][T]).
    With positions [B][T] int32 (and rope_base > 0) q and the draft keys are
    rotated inside the kernels."""
    shape = _shape_of(q, k_cache.shape[2], scale, rope_base)
    out, lse = _outputs(q, out, lse)
    ws = workspace or Workspace.for_shape(shape, q.device, stream)
    _check(lib().verify_attn_dense(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[1],
                                   _ptr(seqlens), _ptr(tree_parent), _ptr(tree_mask), _ptr(positions), _ptr(out),
                                   _ptr(lse), ws.ptr, ws.nbytes, _stream(stream)))
    return out, lse


def verify_attn_dense_noalloc(q, k_cache, v_cache, seqlens, tree_parent=None, tree_mask=None, positions=None,
                              out=None, lse=None, device_status=None, scale=None, stream=None, rope_base=0.0):
    """verify_attn_dense without a workspace (fixed 8 MiB static device scratch inside
    the library) for callers that cannot allocate; see include/verify_attn.h."""
    shape = _shape_of(q, k_cache.shape[2], scale, rope_base)
    out, lse = _outputs(q, out, lse)
    _check(lib().verify_attn_dense_noalloc(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                           k_cache.shape[1], _ptr(seqlens), _ptr(tree_parent), _ptr(tree_mask),
                                           _ptr(positions), _ptr(out), _ptr(lse), _ptr(device_status),
                                           _stream(stream)))
    return out, lse


def verify_attn_paged(q, k_pages, v_pages, page_table, seqlens, tree_parent=None, tree_mask=None, positions=None,
                      out=None, lse=None, workspace: Workspace = None, scale=None, stream=None, rope_base=0.0):
    """Paged-cache verification attention; pages [P][page][Hkv][D], page_table int32 [B][max_pages]."""
    shape = _shape_of(q, k_pages.shape[2], scale, rope_base)
    out, lse = _outputs(q, out, lse)
    ws = workspace or Workspace.for_shape(shape, q.device, stream)
    _check(lib().verify_attn_paged(ctypes.byref(shape), _ptr(q), _ptr(k_pages), _ptr(v_pages), k_pages.shape[0],
                                   k_pages.shape[1], _ptr(page_table), page_table.shape[1], _ptr(seqlens),
                                   _ptr(tree_parent), _ptr(tree_mask), _ptr(positions), _ptr(out), _ptr(lse),
                                   ws.ptr, ws.nbytes, _stream(stream)))
    return out, lse


def verify_attn_sparse(q, k_cache, v_cache, seqlens, indices, n_indices, tree_parent=None, tree_mask=None,
                       positions=None, out=None, lse=None, workspace: Workspace = None, scale=None, stream=None,
                       rope_base=0.0):
    """Sparse verification over per-(sequence, kv-head) verify index sets [B][Hkv][max_indices]."""
    shape = _shape_of(q, k_cache.shape[2], scale, rope_base)
    out, lse = _outputs(q, out, lse)
    ws = workspace or Workspace.for_shape(shape, q.device, stream)
    _check(lib().verify_attn_sparse(ctypes.byref(shape), _ptr(q), _ptr(k_cache), _ptr(v_cache), k_cache.shape[1],
                                    _ptr(seqlens), _ptr(indices), _ptr(n_indices), indices.shape[2],
                                    _ptr(tree_parent), _ptr(tree_mask), _ptr(positions), _ptr(out), _ptr(lse),
                                    ws.ptr, ws.nbytes, _stream(stream)))
    return out, lse


def verify_attn_combine(o_parts, lse_parts, out_dtype=torch.float32, out=None, lse=None, stream=None):
    """Log-sum-exp merge of partials: o_parts f32 [S][R][D], lse_parts f32 [S][R] -> (out [R][D], lse [R])."""
    S, R, D = o_parts.shape
    if out is None:
        out = torch.empty(R, D, dtype=out_dtype, device=o_parts.device)
    if lse is None:
        lse = torch.empty(R, dtype=torch.float32, device=o_parts.device)
    _check(lib().verify_attn_combine(R, S, D, _ptr(o_parts), _ptr(lse_parts), _dtype_code(out), _ptr(out), _ptr(lse),
                                     _stream(stream)))
    return out, lse


def verify_tree_mask_from_parents(parent, mask=None, workspace: Workspace = None, stream=None):
    """Ancestor-or-self bitmask uint32-as-int32 [B][T][ceil(T/32)] from parent int32 [B][T]."""
    B, T = parent.shape
    if mask is None:
        mask = torch.empty(B, T, (T + 31) // 32, dtype=torch.int32, device=parent.device)
    _check(lib().verify_tree_mask_from_parents(B, T, _ptr(parent), _ptr(mask),
                                               workspace.ptr if workspace is not None else None, _stream(stream)))
    return mask


def verify_build_index(seqlens, score_draft, score_target, n_sink, window, m_draft, budget, indices=None,
                       n_indices=None, workspace: Workspace = None, stream=None):
    """Verify index sets: returns (indices int32 [B][Hkv][budget], n_indices int32 [B][Hkv])."""
    B, Hkv, stride = score_draft.shape
    if indices is None:
        indices = torch.empty(B, Hkv, budget, dtype=torch.int32, device=score_draft.device)
    if n_indices is None:
        n_indices = torch.empty(B, Hkv, dtype=torch.int32, device=score_draft.device)
    _check(lib().verify_build_index(B, Hkv, _ptr(seqlens), _ptr(score_draft), _ptr(score_target), stride, n_sink,
                                    window, m_draft, budget, _ptr(indices), _ptr(n_indices),
                                    workspace.ptr if workspace is not None else None, _stream(stream)))
    return indices, n_indices


def verify_accept_greedy(parent, draft_tokens, target_next, path=None, n_accept=None, bonus=None,
                         workspace: Workspace = None, stream=None):
    """Greedy tree acceptance: returns (path int32 [B][T], n_accept int32 [B], bonus int32 [B])."""
    B, T = parent.shape
    dev = parent.device
    if path is None:
        path = torch.empty(B, T, dtype=torch.int32, device=dev)
    if n_accept is None:
        n_accept = torch.empty(B, dtype=torch.int32, device=dev)
    if bonus is None:
        bonus = torch.empty(B, dtype=torch.int32, device=dev)
    _check(lib().verify_accept_greedy(B, T, _ptr(parent), _ptr(draft_tokens), _ptr(target_next), _ptr(path),
                                      _ptr(n_accept), _ptr(bonus), workspace.ptr if workspace is not None else None,
                                      _stream(stream)))
    return path, n_accept, bonus


def _bf16_rows(cache):
    """A cache whose rows are moved as they are: quantised rows (uint8) as bf16 rows of half as many elements."""
    if isinstance(cache, torch.Tensor) and cache.dtype == torch.uint8 and cache.dim() == 4:
        if cache.shape[-1] % 16 != 0 or not cache.is_contiguous():
            raise ValueError("caches held in 8 or 4 bits must be contiguous, in rows of 16-byte multiples")
        return cache.view(torch.bfloat16)
    return cache


def _bf16_pair(k, v):
    """_bf16_rows of a K and a V cache, which are held alike."""
    if isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and torch.uint8 in (k.dtype, v.dtype) and \
            (k.dtype != v.dtype or k.shape != v.shape):
        raise ValueError(f"caches of {k.dtype} {list(k.shape)} and {v.dtype} {list(v.shape)} are not of the same rows")
    return _bf16_rows(k), _bf16_rows(v)


def verify_commit_kv_dense(k_cache, v_cache, seqlens, path, n_accept, seqlens_out=None,
                           workspace: Workspace = None, stream=None):
    """Move the accepted draft rows of k_cache / v_cache [B][len][Hkv][D] in
    place to the slots after each prefix; returns seqlens + n_accept.  (Here and
    in the eviction a cache may hold quantised rows, uint8 [..][kv_row_bytes].)"""
    k_cache, v_cache = _bf16_pair(k_cache, v_cache)
    B, cap, Hkv, D = k_cache.shape
    T = path.shape[1]
    if seqlens_out is None:
        seqlens_out = torch.empty(B, dtype=torch.int32, device=k_cache.device)
    shape = make_shape(B, T, Hkv, Hkv, D, _dtype_code(k_cache), 1.0)
    _check(lib().verify_commit_kv_dense(ctypes.byref(shape), _ptr(k_cache), _ptr(v_cache), cap, _ptr(seqlens),
                                        _ptr(path), _ptr(n_accept), _ptr(seqlens_out),
                                        workspace.ptr if workspace is not None else None, _stream(stream)))
    return seqlens_out


def verify_commit_kv_paged(k_pages, v_pages, page_table, seqlens, path, n_accept, seqlens_out=None,
                           workspace: Workspace = None, stream=None):
    """The same commit through a page table; pages [P][page][Hkv][D]."""
    k_pages, v_pages = _bf16_pair(k_pages, v_pages)
    P, ps, Hkv, D = k_pages.shape
    B, max_pages = page_table.shape
    T = path.shape[1]
    if seqlens_out is None:
        seqlens_out = torch.empty(B, dtype=torch.int32, device=k_pages.device)
    shape = make_shape(B, T, Hkv, Hkv, D, _dtype_code(k_pages), 1.0)
    _check(lib().verify_commit_kv_paged(ctypes.byref(shape), _ptr(k_pages), _ptr(v_pages), P, ps, _ptr(page_table),
                                        max_pages, _ptr(seqlens), _ptr(path), _ptr(n_accept), _ptr(seqlens_out),
                                        workspace.ptr if workspace is not None else None, _stream(stream)))
    return seqlens_out


def verify_rope_draft_dense(q, k_cache, seqlens, positions, rope_base=10000.0, workspace: Workspace = None,
                            stream=None):
    """Rotate, in place, every head of q [B][T][Hq][D] and the draft key rows
    (slots L_b .. L_b+T-1) of k_cache [B][len][Hkv][D] at positions [B][T]."""
    B, T, Hq, D = q.shape
    _, cap, Hkv, _ = k_cache.shape
    shape = make_shape(B, T, Hq, Hkv, D, _dtype_code(q), 1.0)
    _check(lib().verify_rope_draft_dense(ctypes.byref(shape), _ptr(q), _ptr(k_cache), cap, _ptr(seqlens),
                                         _ptr(positions), float(rope_base),
                                         workspace.ptr if workspace is not None else None, _stream(stream)))


def verify_rope_draft_paged(q, k_pages, page_table, seqlens, positions, rope_base=10000.0,
                            workspace: Workspace = None, stream=None):
    """The same rotation through a page table; pages [P][page][Hkv][D]."""
    B, T, Hq, D = q.shape
    P, ps, Hkv, _ = k_pages.shape
    shape = make_shape(B, T, Hq, Hkv, D, _dtype_code(q), 1.0)
    _check(lib().verify_rope_draft_paged(ctypes.byref(shape), _ptr(q), _ptr(k_pages), P, ps, _ptr(page_table),
                                         page_table.shape[1], _ptr(seqlens), _ptr(positions), float(rope_base),
                                         workspace.ptr if workspace is not None else None, _stream(stream)))


class ScoreScratch:
    """Caller-owned device scratch of the scoring pass (256-byte aligned)."""

    def __init__(self, B, T, n_heads, max_cache_len, device=None):
        n = int(lib().verify_head_importance_scratch_size(int(B), int(T), int(n_heads), int(max_cache_len)))
        if n == 0:
            _check(VA_ERR_INVALID_ARG)
        self.buffer = torch.empty(n + 256, dtype=torch.uint8, device=device or "cuda")
        self.offset = (-self.buffer.data_ptr()) % 256
        self.nbytes = n

    @property
    def ptr(self) -> int:
        return self.buffer.data_ptr() + self.offset


def verify_head_importance(q, k_cache, seqlens, heads, score=None, score_stride=None, scale=None,
                           scratch: ScoreScratch = None, workspace: Workspace = None, stream=None):
    """Importance map of the committed positions from the listed query heads:
    returns score fp32 [B][Hkv][score_stride] (entries past each L_b untouched;
    a new tensor is zero-filled there)."""
    B, T, Hq, D = q.shape
    _, cap, Hkv, _ = k_cache.shape
    heads = [int(h) for h in heads]
    if score is None:
        score = torch.zeros(B, Hkv, score_stride or cap, dtype=torch.float32, device=q.device)
    stride = score.shape[-1]
    if scratch is None:
        scratch = ScoreScratch(B, T, len(heads), cap, device=q.device)
    shape = make_shape(B, T, Hq, Hkv, D, _dtype_code(q), scale)
    harr = (ctypes.c_int32 * len(heads))(*heads)
    _check(lib().verify_head_importance(ctypes.byref(shape), _ptr(q), _ptr(k_cache), cap, _ptr(seqlens),
                                        ctypes.cast(harr, ctypes.c_void_p), len(heads), _ptr(score), stride,
                                        scratch.ptr, scratch.nbytes,
                                        workspace.ptr if workspace is not None else None, _stream(stream)))
    return score


# ----------------------------------------------------------------------------
# score shaping, accumulated attention weight, eviction
# ----------------------------------------------------------------------------

_I32, _F32 = torch.int32, torch.float32


def _arg(t, name, shape, dtype, dev):
    """Device pointer of a contiguous tensor of this shape and type on GPU `dev`; None stays None."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name}: expected a torch.Tensor or None") from None
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, q or the cache on cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")
    raise ValueError("tensor arguments must be contiguous")


def _req(t, name, shape, dtype, dev):
    """The same for an argument that has to be given."""
    if t is None:
        raise TypeError(f"{name}: expected a torch.Tensor")
    return _arg(t, name, shape, dtype, dev)


def _sizes(t, name, dim):
    """Sizes of a GPU tensor of `dim` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    if t.dim() != dim:
        raise ValueError(f"{name}: expected {dim} dimensions, got {list(t.shape)}")
    return t.shape


def _cache_args(layout, n0, n1, B, table, dev):
    """Geometry arguments of a cache: [cache length], or [pages, page size, table, table width]."""
    if layout == "dense":
        if n0 != B:
            raise ValueError(f"the key cache: expected {B} sequences, got {n0}")
        return (n1,)
    width = _sizes(table, "page_table", 2)[1]
    return n0, n1, _arg(table, "page_table", (B, width), _I32, dev), width


def _run_on(dev, stream, name, *args):
    """Call library function `name` with GPU `dev` current, on `stream` (that GPU's
    current stream by default); args end before the stream."""
    f = getattr(_lib or lib(), name)
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == dev:
        status = f(*args, s)
    else:
        with torch.cuda.device(dev):
            status = f(*args, s)
    if status != VA_OK:
        _check(status)


def _made(make, dev, stream):
    """What make() allocates for a call on `stream`, from that stream's memory pool: neither
    the memory's last user nor its next one overlaps with the call."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return make()
    with torch.cuda.device(dev):
        return make()


class ScoreMod:
    """Score shaping of a target model (see va_score_mod in include/verify_attn.h):
    tanh cap, sliding window, distance slopes fp32 [Hq], first visible prefix
    slots int32 [B], positions of the draft tokens int32 [B][T].  Keeps
    references to the tensors; they are read when a call runs."""

    def __init__(self, softcap=0.0, window=0, slopes=None, key_start=None, token_pos=None):
        self.softcap, self.window = float(softcap), int(window)
        self.slopes, self.key_start, self.token_pos = slopes, key_start, token_pos

    def struct(self, B, T, Hq, dev) -> VaScoreMod:
        return VaScoreMod(self.softcap, self.window, _arg(self.slopes, "slopes", (Hq,), _F32, dev),
                          _arg(self.key_start, "key_start", (B,), _I32, dev),
                          _arg(self.token_pos, "token_pos", (B, T), _I32, dev))


def _mod_call(layout, q, k, v, table, seqlens, mod, tree_parent, tree_mask, out, lse, workspace, scale, stream):
    B, T, Hq, D = rows = _sizes(q, "q", 4)
    n0, n1, Hkv, _ = _sizes(k, "the key cache", 4)
    dev, dtype, cache = q.get_device(), q.dtype, (n0, n1, Hkv, D)
    if not isinstance(mod, ScoreMod):
        raise TypeError("mod: expected a ScoreMod")
    shape = VaShape(B, T, Hq, Hkv, D, _dtype_code(q), D ** -0.5 if scale is None else scale, 0.0)
    if out is None or lse is None:
        out, lse = _made(lambda: _outputs(q, out, lse), dev, stream)
    ws = workspace
    if ws is None:
        ws = _made(lambda: Workspace.for_shape(shape, q.device, stream), dev, stream)
    elif ws.buffer.get_device() != dev:
        raise ValueError(f"workspace is on {ws.buffer.device}, q on cuda:{dev}")
    _run_on(dev, stream, "verify_attn_dense_mod" if layout == "dense" else "verify_attn_paged_mod",
            ctypes.byref(shape), ctypes.byref(mod.struct(B, T, Hq, dev)), _arg(q, "q", rows, dtype, dev),
            _arg(k, "the key cache", cache, dtype, dev), _req(v, "the value cache", cache, dtype, dev),
            *_cache_args(layout, n0, n1, B, table, dev), _req(seqlens, "seqlens", (B,), _I32, dev),
            _arg(tree_parent, "tree_parent", (B, T), _I32, dev),
            _arg(tree_mask, "tree_mask", (B, T, (T + 31) // 32), _I32, dev), _arg(out, "out", rows, dtype, dev),
            _arg(lse, "lse", (B, Hq, T), _F32, dev), ws.ptr, ws.nbytes)
    return out, lse


def verify_attn_dense_mod(q, k_cache, v_cache, seqlens, mod: ScoreMod, tree_parent=None, tree_mask=None, out=None,
                          lse=None, workspace: Workspace = None, scale=None, stream=None):
    """verify_attn_dense with score shaping; returns (out [B][T][Hq][D], lse [B][Hq][T])."""
    return _mod_call("dense", q, k_cache, v_cache, None, seqlens, mod, tree_parent, tree_mask, out, lse, workspace,
                     scale, stream)


def verify_attn_paged_mod(q, k_pages, v_pages, page_table, seqlens, mod: ScoreMod, tree_parent=None, tree_mask=None,
                          out=None, lse=None, workspace: Workspace = None, scale=None, stream=None):
    """verify_attn_paged with score shaping; pages [P][page][Hkv][D], page_table int32 [B][max_pages]."""
    return _mod_call("paged", q, k_pages, v_pages, page_table, seqlens, mod, tree_parent, tree_mask, out, lse,
                     workspace, scale, stream)


def _status_ptr(workspace, dev):
    if workspace is None:
        return None
    if workspace.buffer.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.buffer.device}, the cache on cuda:{dev}")
    return workspace.ptr


def _weight_call(layout, q, k, table, seqlens, lse, weight, mod, path, n_accept, decay, scale, workspace, stream):
    B, T, Hq, D = rows = _sizes(q, "q", 4)
    n0, n1, Hkv, _ = _sizes(k, "the key cache", 4)
    stride = _sizes(weight, "weight", 3)[2]
    dev, dtype = q.get_device(), q.dtype
    shape = VaShape(B, T, Hq, Hkv, D, _dtype_code(q), D ** -0.5 if scale is None else scale, 0.0)
    if mod is not None and not isinstance(mod, ScoreMod):
        raise TypeError("mod: expected a ScoreMod or None")
    _run_on(dev, stream, "verify_accumulate_weight_dense" if layout == "dense" else "verify_accumulate_weight_paged",
            ctypes.byref(shape), ctypes.byref(mod.struct(B, T, Hq, dev)) if mod is not None else None,
            _arg(q, "q", rows, dtype, dev), _arg(k, "the key cache", (n0, n1, Hkv, D), dtype, dev),
            *_cache_args(layout, n0, n1, B, table, dev), _req(seqlens, "seqlens", (B,), _I32, dev),
            _arg(path, "path", (B, T), _I32, dev), _arg(n_accept, "n_accept", (B,), _I32, dev),
            _req(lse, "lse", (B, Hq, T), _F32, dev), decay, _arg(weight, "weight", (B, Hkv, stride), _F32, dev), stride,
            _status_ptr(workspace, dev))
    return weight


def verify_accumulate_weight_dense(q, k_cache, seqlens, lse, weight, mod: ScoreMod = None, path=None, n_accept=None,
                                   decay=1.0, scale=None, workspace: Workspace = None, stream=None):
    """Add the attention the accepted tokens gave to every cached key to weight
    fp32 [B][Hkv][stride], in place (after the commit, with the seqlens from
    before it and the verification call's q and lse); returns weight."""
    return _weight_call("dense", q, k_cache, None, seqlens, lse, weight, mod, path, n_accept, decay, scale, workspace,
                        stream)


def verify_accumulate_weight_paged(q, k_pages, page_table, seqlens, lse, weight, mod: ScoreMod = None, path=None,
                                   n_accept=None, decay=1.0, scale=None, workspace: Workspace = None, stream=None):
    """The same totals over a paged cache."""
    return _weight_call("paged", q, k_pages, page_table, seqlens, lse, weight, mod, path, n_accept, decay, scale,
                        workspace, stream)


class EvictScratch(Workspace):
    """Caller-owned device scratch of the eviction, initialised once."""

    def __init__(self, B, Hkv, max_indices, device=None, stream=None):
        n = int(lib().verify_evict_kv_scratch_size(int(B), int(Hkv), int(max_indices)))
        if n == 0:
            _check(VA_ERR_INVALID_ARG)
        super().__init__(n, device=device, stream=stream)


def _evict_call(layout, k, v, table, seqlens, indices, n_indices, weight, seqlens_out, scratch, workspace, stream):
    k, v = _bf16_pair(k, v)
    n0, n1, Hkv, D = cache = _sizes(k, "the key cache", 4)
    B, _, m = _sizes(indices, "indices", 3)
    stride = _sizes(weight, "weight", 3)[2] if weight is not None else 0
    dev, dtype = k.get_device(), k.dtype
    if seqlens_out is None:
        seqlens_out = _made(lambda: torch.empty(B, dtype=_I32, device=k.device), dev, stream)
    shape = VaShape(B, 1, Hkv, Hkv, D, _dtype_code(k), 1.0, 0.0)
    sc = scratch
    if sc is None:
        sc = _made(lambda: EvictScratch(B, Hkv, max(m, 1), k.device, stream), dev, stream)
    elif sc.buffer.get_device() != dev:
        raise ValueError(f"scratch is on {sc.buffer.device}, the cache on cuda:{dev}")
    _run_on(dev, stream, "verify_evict_kv_dense" if layout == "dense" else "verify_evict_kv_paged", ctypes.byref(shape),
            _arg(k, "the key cache", cache, dtype, dev), _req(v, "the value cache", cache, dtype, dev),
            *_cache_args(layout, n0, n1, B, table, dev), _req(seqlens, "seqlens", (B,), _I32, dev),
            _arg(indices, "indices", (B, Hkv, m), _I32, dev), _req(n_indices, "n_indices", (B, Hkv), _I32, dev), m,
            _arg(weight, "weight", (B, Hkv, stride), _F32, dev), stride,
            _arg(seqlens_out, "seqlens_out", (B,), _I32, dev), sc.ptr, sc.nbytes, _status_ptr(workspace, dev))
    return seqlens_out


def verify_evict_kv_dense(k_cache, v_cache, seqlens, indices, n_indices, weight=None, seqlens_out=None,
                          scratch: EvictScratch = None, workspace: Workspace = None, stream=None):
    """Move the kept rows indices [B][Hkv][n] of k_cache / v_cache [B][len][Hkv][D]
    (and of weight fp32 [B][Hkv][stride]) to the front, in place; returns the
    new lengths."""
    return _evict_call("dense", k_cache, v_cache, None, seqlens, indices, n_indices, weight, seqlens_out, scratch,
                       workspace, stream)


def verify_evict_kv_paged(k_pages, v_pages, page_table, seqlens, indices, n_indices, weight=None, seqlens_out=None,
                          scratch: EvictScratch = None, workspace: Workspace = None, stream=None):
    """The same eviction through a page table; pages [P][page][Hkv][D]."""
    return _evict_call("paged", k_pages, v_pages, page_table, seqlens, indices, n_indices, weight, seqlens_out,
                       scratch, workspace, stream)


# ----------------------------------------------------------------------------
# norm with rotation, caches held in 8 or 4 bits
# ----------------------------------------------------------------------------

KV_FORMATS = {"e4m3": 0, "e2m1": 1}
_ROW_BYTES = {}


def kv_row_bytes(fmt, D) -> int:
    """Bytes of a quantised row (one token of one kv-head): caches of format `fmt`
    ("e4m3" or "e2m1") are uint8 [B][len][Hkv][kv_row_bytes], or pages of such rows."""
    n = _ROW_BYTES.get((fmt, D))
    if n is None:
        n = int(lib().verify_kv_row_bytes(_format(fmt), int(D)))
        if n == 0:
            raise ValueError(f"caches held in {fmt} take D = 64 or 128, not {D}")
        _ROW_BYTES[fmt, D] = n
    return n


def _format(fmt) -> int:
    try:
        return KV_FORMATS[fmt]
    except (KeyError, TypeError):
        raise ValueError(f"unknown cache format {fmt!r}; use 'e4m3' or 'e2m1'") from None


def _rows(t, name, shape, dtype, dev):
    """Rows of D elements of a [B][T][heads][D] tensor, by reference: heads side by
    side, any batch and token stride (a part of a projection's output)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            sb, st, sh, sd = t.stride()
            if (sd == 1 or shape[3] == 1) and (sh == shape[3] or shape[2] == 1):
                return ctypes.byref(VaRows(t.data_ptr(), sb, st))
            raise ValueError(f"{name}: the heads of a token must be contiguous")
    except AttributeError:
        raise TypeError(f"{name}: expected a torch.Tensor") from None
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the others on cuda:{dev}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    raise ValueError(f"{name}: expected shape {list(shape)}, got {list(t.shape)}")


def verify_norm_rope(q, k, q_weight=None, k_weight=None, positions=None, eps=1e-6, rope_base=10000.0, q_out=None,
                     k_out=None, stream=None):
    """RMS norm of every head of q [B][T][Hq][D] and k [B][T][Hkv][D] (weights [D];
    None: no norm) and the rotation at positions int32 [B][T] (None: no rotation),
    in one pass.  q and k may be parts of one projection's output; returns (q_out,
    k_out), contiguous unless given (an output may be its own input)."""
    B, T, Hq, D = _sizes(q, "q", 4)
    Hkv = _sizes(k, "k", 4)[2]
    dev, dtype = q.get_device(), q.dtype
    shape = VaShape(B, T, Hq, Hkv, D, _dtype_code(q), 1.0, rope_base)
    sq, sk = (B, T, Hq, D), (B, T, Hkv, D)
    if q_out is None or k_out is None:
        new = _made(lambda: [torch.empty(s, dtype=dtype, device=q.device) if o is None else o
                             for s, o in ((sq, q_out), (sk, k_out))], dev, stream)
        q_out, k_out = new
    _run_on(dev, stream, "verify_norm_rope", ctypes.byref(shape), _rows(q, "q", sq, dtype, dev),
            _rows(k, "k", sk, dtype, dev), _arg(q_weight, "q_weight", (D,), dtype, dev),
            _arg(k_weight, "k_weight", (D,), dtype, dev), eps, _arg(positions, "positions", (B, T), _I32, dev),
            _rows(q_out, "q_out", sq, dtype, dev), _rows(k_out, "k_out", sk, dtype, dev))
    return q_out, k_out


_QUANT_CALLS = {(w, y): f"verify_{w}_kv_{y}" for w in ("quantize", "dequantize") for y in ("dense", "paged")}


def _quant_call(what, layout, k, v, k_cache, v_cache, table, start, fmt, n_tokens, workspace, stream):
    B, T, Hkv, D = rows = _sizes(k, "k", 4)
    n0, n1, _, _ = _sizes(k_cache, "the key cache", 4)
    dev, dtype = k.get_device(), k.dtype
    shape = VaShape(B, T, Hkv, Hkv, D, _dtype_code(k), 1.0, 0.0)
    code, cache = _format(fmt), (n0, n1, Hkv, kv_row_bytes(fmt, D))
    plain = _rows(k, "k", rows, dtype, dev), _rows(v, "v", rows, dtype, dev)
    caches = (_arg(k_cache, "the key cache", cache, torch.uint8, dev),
              _req(v_cache, "the value cache", cache, torch.uint8, dev), *_cache_args(layout, n0, n1, B, table, dev))
    first = _req(start, "start" if what == "dequantize" else "seqlens", (B,), _I32, dev)
    count = _arg(n_tokens, "n_tokens", (B,), _I32, dev)
    args = (*plain, *caches, first, count) if what == "quantize" else (*caches, first, count, *plain)
    _run_on(dev, stream, _QUANT_CALLS[what, layout], ctypes.byref(shape), code, *args, _status_ptr(workspace, dev))


def verify_quantize_kv_dense(k, v, k_cache, v_cache, seqlens, fmt, n_tokens=None, workspace: Workspace = None,
                             stream=None):
    """Quantise rows k, v [B][T][Hkv][D] into caches held in `fmt`, uint8
    [B][len][Hkv][kv_row_bytes], at slots seqlens[b] + t for t < n_tokens[b] (None: T)."""
    _quant_call("quantize", "dense", k, v, k_cache, v_cache, None, seqlens, fmt, n_tokens, workspace, stream)


def verify_quantize_kv_paged(k, v, k_pages, v_pages, page_table, seqlens, fmt, n_tokens=None,
                             workspace: Workspace = None, stream=None):
    """The same through a page table; pages uint8 [P][page][Hkv][kv_row_bytes]."""
    _quant_call("quantize", "paged", k, v, k_pages, v_pages, page_table, seqlens, fmt, n_tokens, workspace, stream)


def _read_back(layout, k_cache, v_cache, table, start, fmt, n, dtype, n_tokens, k_out, v_out, workspace, stream):
    _, _, Hkv, nbytes = _sizes(k_cache, "the key cache", 4)
    B = _sizes(start, "start", 1)[0]
    if k_out is None or v_out is None:
        if n is None:
            raise TypeError("n: the number of slots is needed without k_out and v_out")
        D = {kv_row_bytes(fmt, d): d for d in (64, 128)}.get(nbytes)
        if D is None:
            raise ValueError(f"the key cache: rows of {nbytes} bytes are no {fmt} rows")
        # (rows past n_tokens stay as they are made: zero)
        k_out, v_out = _made(lambda: [torch.zeros(B, n, Hkv, D, dtype=dtype, device=k_cache.device) if o is None else o
                                      for o in (k_out, v_out)], k_cache.get_device(), stream)
    _quant_call("dequantize", layout, k_out, v_out, k_cache, v_cache, table, start, fmt, n_tokens, workspace, stream)
    return k_out, v_out


def verify_dequantize_kv_dense(k_cache, v_cache, start, fmt, n=None, dtype=torch.bfloat16, n_tokens=None, k_out=None,
                               v_out=None, workspace: Workspace = None, stream=None):
    """Read slots start[b] .. start[b] + n - 1 of caches held in `fmt` back (only the
    first n_tokens[b] of them, if given); returns (k, v) [B][n][Hkv][D]."""
    return _read_back("dense", k_cache, v_cache, None, start, fmt, n, dtype, n_tokens, k_out, v_out, workspace, stream)


def verify_dequantize_kv_paged(k_pages, v_pages, page_table, start, fmt, n=None, dtype=torch.bfloat16, n_tokens=None,
                               k_out=None, v_out=None, workspace: Workspace = None, stream=None):
    """The same through a page table."""
    return _read_back("paged", k_pages, v_pages, page_table, start, fmt, n, dtype, n_tokens, k_out, v_out, workspace,
                      stream)


def _attn_quant(layout, q, k, v, table, seqlens, fmt, tree_parent, tree_mask, out, lse, workspace, scale, stream):
    B, T, Hq, D = rows = _sizes(q, "q", 4)
    n0, n1, Hkv, _ = _sizes(k, "the key cache", 4)
    dev, dtype = q.get_device(), q.dtype
    shape = VaShape(B, T, Hq, Hkv, D, _dtype_code(q), D ** -0.5 if scale is None else scale, 0.0)
    code, cache = _format(fmt), (n0, n1, Hkv, kv_row_bytes(fmt, D))
    if out is None or lse is None:
        out, lse = _made(lambda: _outputs(q, out, lse), dev, stream)
    ws = workspace
    if ws is None:
        ws = _made(lambda: Workspace.for_shape(shape, q.device, stream), dev, stream)
    elif ws.buffer.get_device() != dev:
        raise ValueError(f"workspace is on {ws.buffer.device}, q on cuda:{dev}")
    _run_on(dev, stream, "verify_attn_dense_quant" if layout == "dense" else "verify_attn_paged_quant",
            ctypes.byref(shape), code, _arg(q, "q", rows, dtype, dev), _arg(k, "the key cache", cache, torch.uint8, dev),
            _req(v, "the value cache", cache, torch.uint8, dev), *_cache_args(layout, n0, n1, B, table, dev),
            _req(seqlens, "seqlens", (B,), _I32, dev), _arg(tree_parent, "tree_parent", (B, T), _I32, dev),
            _arg(tree_mask, "tree_mask", (B, T, (T + 31) // 32), _I32, dev), _arg(out, "out", rows, dtype, dev),
            _arg(lse, "lse", (B, Hq, T), _F32, dev), ws.ptr, ws.nbytes)
    return out, lse


def verify_attn_dense_quant(q, k_cache, v_cache, seqlens, fmt, tree_parent=None, tree_mask=None, out=None, lse=None,
                            workspace: Workspace = None, scale=None, stream=None):
    """verify_attn_dense over caches held in `fmt` ("e4m3" or "e2m1"), uint8
    [B][len][Hkv][kv_row_bytes]; returns (out [B][T][Hq][D], lse [B][Hq][T])."""
    return _attn_quant("dense", q, k_cache, v_cache, None, seqlens, fmt, tree_parent, tree_mask, out, lse, workspace,
                       scale, stream)


def verify_attn_paged_quant(q, k_pages, v_pages, page_table, seqlens, fmt, tree_parent=None, tree_mask=None, out=None,
                            lse=None, workspace: Workspace = None, scale=None, stream=None):
    """verify_attn_paged over pages of quantised rows, uint8 [P][page][Hkv][kv_row_bytes]."""
    return _attn_quant("paged", q, k_pages, v_pages, page_table, seqlens, fmt, tree_parent, tree_mask, out, lse,
                       workspace, scale, stream)


def verify_attn_check_status(workspace: Workspace, stream=None):
    """Synchronise the stream and raise if a kernel recorded a device-side error."""
    _check(lib().verify_attn_check_status(workspace.ptr, _stream(stream)))


def version() -> str:
    return lib().verify_attn_version().decode()
