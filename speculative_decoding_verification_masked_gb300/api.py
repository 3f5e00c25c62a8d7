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


def verify_commit_kv_dense(k_cache, v_cache, seqlens, path, n_accept, seqlens_out=None,
                           workspace: Workspace = None, stream=None):
    """Move the accepted draft rows of k_cache / v_cache [B][len][Hkv][D] in
    place to the slots after each prefix; returns seqlens + n_accept."""
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


def verify_attn_check_status(workspace: Workspace, stream=None):
    """Synchronise the stream and raise if a kernel recorded a device-side error."""
    _check(lib().verify_attn_check_status(workspace.ptr, _stream(stream)))


def version() -> str:
    return lib().verify_attn_version().decode()
