"""Norms of queries and keys, the paged key/value cache, and attention over it.

Signatures and documentation of the corresponding entry points of
``include/sparse_attn.h``; as in the package's other calls, every step runs in the
library's kernels, and arguments are checked before anything is launched: shapes,
types and devices of the tensors in ``csrc/sa_binding.cpp``, values in the library.

    # training: norm, then the attention that rotates by itself
    q, k = qk_norm_rope(x_q, x_k, w_q, w_k, rotate=False)
    dx_q, dx_k, dw_q, dw_k = qk_norm_rope_bwd(x_q, x_k, w_q, w_k, dq, dk, rotate=False)

    # serving: any mix of prefill chunks and single tokens, layer by layer or all at once
    cache = paged_cache(L, n_pages, heads, page_size, D, torch.float8_e4m3fn)
    q = cache_append(x_q, x_k, x_v, cache, page_table, cu_q, cached, q_weight=w_q, k_weight=w_k)
    O, lse = chunk_attn(q, cache, page_table, cu_q, cached, alpha, window=12)

All tensors of a call are on one CUDA device, which need not be the current
one; the work goes to that device's current stream, or to ``stream=`` (every
call takes it). Outputs, the pages of an append and workspaces share no memory with
the call's other tensors, but where a call says that an output may be an input;
others are refused.
"""
import ctypes
from typing import NamedTuple, Optional

import torch

from . import FIB15, SA_DTYPE_BF16, SA_DTYPE_F32, _check, lib

SA_CACHE_PLAIN, SA_CACHE_E4M3 = 0, 1

_DTYPES = {torch.float32: SA_DTYPE_F32, torch.bfloat16: SA_DTYPE_BF16}


# The C structures, for calls of lib()'s entry points themselves
class HeadStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("layer", "batch", "head", "row")]


class RowStrides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("layer", "row", "head")]


class QkNormParams(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("L", "B", "Hq", "Hkv", "T", "D", "pos0", "rotate")]
                + [("eps", ctypes.c_float), ("rope_base", ctypes.c_float),
                   ("dtype", ctypes.c_int32)])


class PagedParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("L", "N", "B", "Hq", "Hkv", "D", "n_pages",
                                               "page_size", "max_pages", "dtype", "format")]


class Pages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "page_table")]


class PagedCache(NamedTuple):
    """Pages of keys and values, [L, n_pages, Hkv, page_size, D], and for
    float8_e4m3fn pages the rows' fp32 scales, [L, n_pages, Hkv, page_size]."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None


def paged_cache(layers, n_pages, heads, page_size, head_dim, dtype=torch.bfloat16, device="cuda"):
    """An empty (zeroed) PagedCache; dtype float32, bfloat16 or float8_e4m3fn."""
    if dtype not in (torch.float32, torch.bfloat16, torch.float8_e4m3fn):
        raise TypeError(f"unsupported cache dtype {dtype}")
    shape = (int(layers), int(n_pages), int(heads), int(page_size), int(head_dim))
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype != torch.float8_e4m3fn:
        return PagedCache(k, v)
    return PagedCache(k, v, *(torch.zeros(shape[:4], dtype=torch.float32, device=device)
                              for _ in range(2)))


_native = None      # the extension module, once one of its calls was made


def _calls():
    """The extension module, given the library's entry points."""
    global _native
    if _native is None:
        L = lib()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError(f"{__package__}._binding cannot be loaded ({e}): build it with "
                               f"`python -m {__package__}.build`") from e
        _binding.bind(_check, *[ctypes.cast(getattr(L, "sparse_attn_" + n), ctypes.c_void_p).value
                                for n in ("qk_norm_workspace_size", "qk_norm_rope",
                                          "qk_norm_rope_bwd", "cache_append", "cache_read",
                                          "chunk")])
        _native = _binding
    return _native


# ---- norms of queries and keys ------------------------------------------------
def qk_norm_rope(q, k, q_weight, k_weight, *, eps=1e-6, rotate=True, rope_base=10000.0, pos0=0,
                 q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head, and the position rotation, in one
    pass (sparse_attn_qk_norm_rope): returns contiguous (q', k').

    q [L, B, Hq, T, D], k [L, B, Hkv, T, D]: bf16 or fp32 with contiguous rows,
    otherwise of any strides (views of a projection's output).  q_weight,
    k_weight: fp32 [L, D], or both None for the rotation alone.  Row t is at
    position pos0 + t.  rotate=False leaves the rotation to the attention: with
    fwd(), bwd() and decode(), which rotate by themselves, it has to be False, or
    rows are rotated twice; the default is for attention over rotated rows.  q_out
    may be a contiguous q, k_out a contiguous k."""
    return _calls().qk_norm_rope(stream, q, k, q_weight, k_weight, eps, rotate, rope_base, pos0,
                                 q_out, k_out)


def qk_norm_rope_bwd(q, k, q_weight, k_weight, dq_out, dk_out, *, eps=1e-6, rotate=True,
                     rope_base=10000.0, pos0=0, dq=None, dk=None, dq_weight=None, dk_weight=None,
                     workspace=None, stream=None):
    """Gradients of qk_norm_rope, called with the same rotate, for its outputs'
    gradients dq_out, dk_out (shaped like q and k, rows contiguous): returns contiguous (dq, dk) and the
    fp32 [L, D] gradients of the weights (None, None without weights), summed in a
    fixed order.  dq may be a contiguous dq_out, dk a contiguous dk_out.
    workspace: an optional CUDA uint8 buffer of qk_norm_workspace_size() bytes, for
    one call at a time (else one is allocated per call)."""
    return _calls().qk_norm_rope_bwd(stream, q, k, q_weight, k_weight, eps, rotate, rope_base, pos0,
                                     dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace)


def qk_norm_workspace_size(q_shape, k_shape, dtype=torch.bfloat16) -> int:
    """Bytes of qk_norm_rope_bwd's workspace for q and k of these shapes."""
    L_, B, Hq, T, D = q_shape
    p = QkNormParams(L_, B, Hq, k_shape[2], T, D, 0, 1, 0.0, 10000.0, _DTYPES[dtype])
    return int(lib().sparse_attn_qk_norm_workspace_size(p))


# ---- paged cache ----------------------------------------------------------------
def cache_append(q, k, v, cache, page_table, cu_q, cached, *, q_weight=None, k_weight=None,
                 eps=1e-6, rope_base=10000.0, q_out=None, stream=None):
    """Writes new tokens into the cache (sparse_attn_cache_append): their keys
    rotated (and normed, with weights), their values as they are, both quantised
    for float8_e4m3fn pages; returns their rotated queries [L, N, Hq, D].

    q [L, N, Hq, D], k and v [L, N, Hkv, D]: bf16 or fp32 with contiguous rows,
    otherwise of any strides.  Rows cu_q[b] .. cu_q[b + 1] - 1 are sequence b's new
    tokens, at positions cached[b], cached[b] + 1, ...; other rows are padding,
    whose values do not matter and whose q_out stays as it was.  Row r of a sequence
    lies in slot r % page_size of page page_table[b, r // page_size].  cu_q [B + 1],
    cached [B] and page_table [B, max_pages] are int32 and read on the device.  No
    two sequences with new tokens may share the pages that are written.  A table of
    cosines for all max_pages * page_size positions (4 D bytes each) is kept on the
    device."""
    return _calls().cache_append(stream, q, k, v, cache, page_table, cu_q, cached, q_weight,
                                 k_weight, eps, rope_base, q_out)


def cache_read(cache, page_table, lengths, *, rows=None, dtype=None, k_out=None, v_out=None,
               stream=None):
    """The first lengths[b] rows of every sequence (int32 [B]) as contiguous
    (k, v) [L, B, Hkv, rows, D] (sparse_attn_cache_read): the stored, rotated keys
    and the values; float8_e4m3fn pages are read as dtype (bf16 by default).
    rows defaults to all that the page table covers, or to k_out's (whose rows and
    dtype any given rows= and dtype= have to be); rows from lengths[b] on are left
    as they were (zeros where the output is made here, which is filled with them
    first: a large read takes twice as long as into given outputs)."""
    return _calls().cache_read(stream, cache, page_table, lengths, rows, dtype, k_out, v_out)


def chunk_attn(q, cache, page_table, cu_q, cached, alpha, *, window, offsets=FIB15, sinks=0,
               scale=0.0, beta=None, out=None, lse=None, want_lse=True, stream=None):
    """Sparse attention of new tokens over the paged cache, which holds their own
    rows already (sparse_attn_chunk): returns (O [L, N, Hq, D], LSE [L, N, Hq] or
    None).  One token per sequence is a decode step, many are a prefill chunk, and
    a call may mix them.

    q [L, N, Hq, D]: rotated queries (cache_append's), rows contiguous; Hq a
    multiple of the cache's heads.  page_table, cu_q, cached: as given to
    cache_append.  alpha: fp32 [L].  beta: optional fp32 [L, N, Hq] log-prior on the
    offset members.  window, offsets, sinks, scale: as in fwd().  Rows that belong
    to no sequence keep what out and lse held."""
    return _calls().chunk_attn(stream, q, cache, page_table, cu_q, cached, alpha, window, offsets,
                               sinks, scale, beta, out, lse, want_lse)


def _bind(L):
    """Argument types of the entry points (structures are passed by reference)."""
    vp, sz, i32, f32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.c_float
    NP, HS = ctypes.POINTER(QkNormParams), ctypes.POINTER(HeadStrides)
    PP, PG, RS = ctypes.POINTER(PagedParams), ctypes.POINTER(Pages), ctypes.POINTER(RowStrides)
    L.sparse_attn_qk_norm_workspace_size.restype = sz
    L.sparse_attn_qk_norm_workspace_size.argtypes = [NP]
    for name, args in (
            ("qk_norm_rope", [NP, vp, HS, vp, HS, vp, vp, vp, vp, vp]),
            ("qk_norm_rope_bwd", [NP, vp, HS, vp, HS, vp, vp, vp, HS, vp, HS, vp, vp, vp, vp, vp,
                                  sz, vp]),
            ("cache_append", [PP, PG, vp, vp, vp, RS, vp, RS, vp, RS, vp, vp, f32, f32, vp, vp]),
            ("cache_read", [PP, PG, vp, i32, vp, vp, vp]),
            ("chunk", [PP, PG, vp, vp, vp, RS, vp, vp, i32, i32, vp, i32, f32, vp, vp, vp])):
        f = getattr(L, "sparse_attn_" + name)
        f.restype, f.argtypes = ctypes.c_int, args
