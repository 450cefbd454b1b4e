"""Norms of queries and keys, the paged key/value cache, and attention over it.

Binding of the corresponding entry points of ``include/sparse_attn.h``; as in
the package's other calls, every step runs in the library's kernels, and
arguments are checked here or in the library before anything is launched.

    # training: norm, then the attention that rotates by itself
    q, k = qk_norm_rope(x_q, x_k, w_q, w_k, rotate=False)
    dx_q, dx_k, dw_q, dw_k = qk_norm_rope_bwd(x_q, x_k, w_q, w_k, dq, dk, rotate=False)

    # serving: any mix of prefill chunks and single tokens, layer by layer or all at once
    cache = paged_cache(L, n_pages, heads, page_size, D, torch.float8_e4m3fn)
    q = cache_append(x_q, x_k, x_v, cache, page_table, cu_q, cached, q_weight=w_q, k_weight=w_k)
    O, lse = chunk_attn(q, cache, page_table, cu_q, cached, alpha, window=12)

All tensors of a call are on one CUDA device, which need not be the current
one; the work goes to that device's current stream, or to ``stream=`` (every
call takes it).
"""
import contextlib
import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import (FIB15, SA_DTYPE_BF16, SA_DTYPE_F32, _check, lib)

SA_CACHE_PLAIN, SA_CACHE_E4M3 = 0, 1

_DTYPES = {torch.float32: SA_DTYPE_F32, torch.bfloat16: SA_DTYPE_BF16}


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


# Single calls of this module take a few microseconds of kernel time, so what a
# call does in Python counts: devices are compared by index and the stream is
# taken as the raw handle.
_raw_stream = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
               or (lambda index: torch.cuda.current_stream(index).cuda_stream))
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _int32(x):
    """x, or the C int nearest to it, which means the same (a window past every row)
    or is refused like it; ctypes would cut its upper bits off."""
    return max(-(1 << 31), min(int(x), (1 << 31) - 1))


def _empty_like(t):
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _addr(t):
    return t.data_ptr() if t is not None else None


@contextlib.contextmanager
def _entered(index, stream):
    if stream is not None and stream.device.index != index:
        raise ValueError(f"stream must be on cuda:{index}")
    with torch.cuda.device(index), (contextlib.nullcontext() if stream is None
                                    else torch.cuda.stream(stream)):
        yield


def _on_its_device(call):
    """Runs call(first, ..., stream=) with the device of its first tensor current
    and stream (of that device) its current stream: allocations and launches go there."""
    @functools.wraps(call)
    def wrapped(*args, stream=None, **kw):
        first = args[0] if args else kw.get("q", kw.get("cache"))
        t = first.k if isinstance(first, PagedCache) else first
        if t is None:
            return call(*args, **kw)      # which says what is missing
        index = t.get_device()
        if index < 0:
            raise ValueError("the tensors must be on a CUDA device")
        if stream is None and _current_device() == index:
            return call(*args, **kw)
        with _entered(index, stream):
            return call(*args, **kw)
    return wrapped


def _whole(name, t, shape, dtype, index):
    """t: a contiguous tensor of that shape, type and device."""
    if (t.dtype != dtype or t.shape != shape or t.get_device() != index
            or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"on cuda:{index}")


def _rows(name, t, shape, dtype, index, kind):
    """t: rows of that shape, their elements contiguous; its strides (0 where there
    is one)."""
    strides = t.stride()
    if (t.dtype != dtype or t.shape != shape or t.get_device() != index or strides[-1] != 1):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on "
                         f"cuda:{index} with contiguous rows")
    return kind(*[s if n > 1 else 0 for s, n in zip(strides[:-1], shape)])


def _span(t):
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _output(name, out, like, others):
    """out, checked, or a new contiguous tensor like `like`."""
    if out is None:
        return _empty_like(like)
    _whole(name, out, like.shape, like.dtype, like.get_device())
    _apart(name, out, like, others)
    return out


def _overlap(a, b):
    a0, a1 = _span(a)
    b0, b1 = _span(b)
    return a0 < b1 and b0 < a1


def _apart(name, out, own, others):
    """out is `own` (contiguous) or shares no memory with it, and none with others."""
    if not out.numel():
        return
    if own is not None and own.numel() and _overlap(out, own):
        if out.data_ptr() != own.data_ptr() or not own.is_contiguous():
            raise ValueError(f"{name} overlaps its input")
    for o in others:
        if o is not None and o.numel() and _overlap(out, o):
            raise ValueError(f"{name} overlaps another tensor of the call")


# ---- norms of queries and keys ------------------------------------------------
def _norm_args(q, k, q_weight, k_weight, eps, rotate, rope_base, pos0):
    dev = q.get_device()
    if q.dim() != 5 or k.dim() != 5:
        raise ValueError("q and k must be [L, B, H, T, D]")
    if q.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}")
    L_, B, Hq, T, D = q.shape
    Hkv = k.shape[2]
    qs = _rows("q", q, q.shape, q.dtype, dev, HeadStrides)
    ks = _rows("k", k, (L_, B, Hkv, T, D), q.dtype, dev, HeadStrides)
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight: both or neither")
    if q_weight is not None:
        _whole("q_weight", q_weight, (L_, D), torch.float32, dev)
        _whole("k_weight", k_weight, (L_, D), torch.float32, dev)
    elif not rotate:
        raise ValueError("without weights there is only the rotation")
    p = QkNormParams(L_, B, Hq, Hkv, _int32(T), D, _int32(pos0), int(bool(rotate)), float(eps),
                     float(rope_base), _DTYPES[q.dtype])
    return dev, p, qs, ks


@_on_its_device
def qk_norm_rope(q, k, q_weight, k_weight, *, eps=1e-6, rotate=True, rope_base=10000.0, pos0=0,
                 q_out=None, k_out=None):
    """RMS norm of every query and key head, and the position rotation, in one
    pass (sparse_attn_qk_norm_rope): returns contiguous (q', k').

    q [L, B, Hq, T, D], k [L, B, Hkv, T, D]: bf16 or fp32 with contiguous rows,
    otherwise of any strides (views of a projection's output).  q_weight,
    k_weight: fp32 [L, D], or both None for the rotation alone.  Row t is at
    position pos0 + t; rotate=False leaves the rotation to the attention (fwd()
    and decode() rotate by themselves).  q_out may be a contiguous q, k_out a
    contiguous k."""
    dev, p, qs, ks = _norm_args(q, k, q_weight, k_weight, eps, rotate, rope_base, pos0)
    q_out = _output("q_out", q_out, q, (k, k_out))
    k_out = _output("k_out", k_out, k, (q,))
    _check("sparse_attn_qk_norm_rope",
           lib().sparse_attn_qk_norm_rope(p, _addr(q), qs, _addr(k), ks, _addr(q_weight),
                                          _addr(k_weight), _addr(q_out), _addr(k_out),
                                          _raw_stream(dev)))
    return q_out, k_out


@_on_its_device
def qk_norm_rope_bwd(q, k, q_weight, k_weight, dq_out, dk_out, *, eps=1e-6, rotate=True,
                     rope_base=10000.0, pos0=0, dq=None, dk=None, dq_weight=None, dk_weight=None,
                     workspace=None):
    """Gradients of qk_norm_rope for its outputs' gradients dq_out, dk_out
    (shaped like q and k, rows contiguous): returns contiguous (dq, dk) and the
    fp32 [L, D] gradients of the weights (None, None without weights), summed in a
    fixed order.  dq may be a contiguous dq_out, dk a contiguous dk_out.
    workspace: an optional CUDA uint8 buffer of qk_norm_workspace_size() bytes, for
    one call at a time (else one is allocated per call)."""
    dev, p, qs, ks = _norm_args(q, k, q_weight, k_weight, eps, rotate, rope_base, pos0)
    dqs = _rows("dq_out", dq_out, q.shape, q.dtype, dev, HeadStrides)
    dks = _rows("dk_out", dk_out, k.shape, k.dtype, dev, HeadStrides)
    dq = _output("dq", dq, dq_out, (q, k, dk_out, dk))
    dk = _output("dk", dk, dk_out, (q, k, dq_out))
    if q_weight is not None:
        dq_weight = _output("dq_weight", dq_weight, q_weight, ())
        dk_weight = _output("dk_weight", dk_weight, k_weight, (dq_weight,))
        if workspace is None:
            need = int(lib().sparse_attn_qk_norm_workspace_size(p))
            workspace = q.new_empty(need, dtype=torch.uint8)
        elif workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be a contiguous buffer on cuda:{dev}")
    elif dq_weight is not None or dk_weight is not None:
        raise ValueError("no weights, no gradients of them")
    n = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("sparse_attn_qk_norm_rope_bwd",
           lib().sparse_attn_qk_norm_rope_bwd(
               p, _addr(q), qs, _addr(k), ks, _addr(q_weight), _addr(k_weight), _addr(dq_out),
               dqs, _addr(dk_out), dks, _addr(dq), _addr(dk), _addr(dq_weight),
               _addr(dk_weight), _addr(workspace), n, _raw_stream(dev)))
    return dq, dk, dq_weight, dk_weight


def qk_norm_workspace_size(q_shape, k_shape, dtype=torch.bfloat16) -> int:
    """Bytes of qk_norm_rope_bwd's workspace for q and k of these shapes."""
    L_, B, Hq, T, D = q_shape
    p = QkNormParams(L_, B, Hq, k_shape[2], T, D, 0, 1, 0.0, 10000.0, _DTYPES[dtype])
    return int(lib().sparse_attn_qk_norm_workspace_size(p))


# ---- paged cache ----------------------------------------------------------------
def _paged_args(cache, page_table, dtype, L_, N, Hq):
    k, v, k_scale, v_scale = cache
    dev = k.get_device()
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if k.dim() != 5:
        raise ValueError("cache.k must be [L, n_pages, Hkv, page_size, D]")
    _, n_pages, Hkv, page_size, D = k.shape
    L_ = k.shape[0] if L_ is None else L_
    quantised = k.dtype == torch.float8_e4m3fn
    if dtype not in _DTYPES or (not quantised and k.dtype != dtype):
        raise TypeError(f"rows of {dtype} and a cache of {k.dtype}")
    shape = (L_, n_pages, Hkv, page_size, D)
    _whole("cache.k", k, shape, k.dtype, dev)
    _whole("cache.v", v, shape, k.dtype, dev)
    if quantised:
        if k_scale is None or v_scale is None:
            raise ValueError("float8_e4m3fn pages need k_scale and v_scale")
        _whole("cache.k_scale", k_scale, shape[:4], torch.float32, dev)
        _whole("cache.v_scale", v_scale, shape[:4], torch.float32, dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales belong to float8_e4m3fn pages only")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, max_pages = page_table.shape
    _whole("page_table", page_table, (B, max_pages), torch.int32, dev)
    if max(N, B, n_pages, page_size, max_pages) >= 1 << 31:
        raise ValueError("every size must fit 32 bits")
    p = PagedParams(L_, N, B, Hkv if Hq is None else Hq, Hkv, D, n_pages, page_size, max_pages,
                    _DTYPES[dtype], SA_CACHE_E4M3 if quantised else SA_CACHE_PLAIN)
    c = Pages(k.data_ptr(), v.data_ptr(), _addr(k_scale), _addr(v_scale), page_table.data_ptr())
    return dev, p, c


def _sequences(cu_q, cached, B, dev):
    _whole("cu_q", cu_q, (B + 1,), torch.int32, dev)
    _whole("cached", cached, (B,), torch.int32, dev)


@_on_its_device
def cache_append(q, k, v, cache, page_table, cu_q, cached, *, q_weight=None, k_weight=None,
                 eps=1e-6, rope_base=10000.0, q_out=None):
    """Writes new tokens into the cache (sparse_attn_cache_append): their keys
    rotated (and normed, with weights), their values as they are, both quantised
    for float8_e4m3fn pages; returns their rotated queries [L, N, Hq, D].

    q [L, N, Hq, D], k and v [L, N, Hkv, D]: bf16 or fp32 with contiguous rows,
    otherwise of any strides.  Rows cu_q[b] .. cu_q[b + 1] - 1 are sequence b's new
    tokens, at positions cached[b], cached[b] + 1, ...; other rows are padding,
    whose values do not matter and whose q_out stays as it was.  Row r of a sequence lies in slot r % page_size of
    page page_table[b, r // page_size].  cu_q [B + 1], cached [B] and page_table
    [B, max_pages] are int32 and read on the device.  No two sequences with new
    tokens may share the pages that are written."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q, k and v must be [L, N, heads, D]")
    L_, N, Hq, D = q.shape
    dev, p, c = _paged_args(cache, page_table, q.dtype, L_, N, Hq)
    kv = (L_, N, p.Hkv, p.D)
    qs = _rows("q", q, (L_, N, Hq, p.D), q.dtype, dev, RowStrides)
    ks = _rows("k", k, kv, q.dtype, dev, RowStrides)
    vs = _rows("v", v, kv, q.dtype, dev, RowStrides)
    _sequences(cu_q, cached, p.B, dev)
    if (q_weight is None) != (k_weight is None):
        raise ValueError("q_weight and k_weight: both or neither")
    if q_weight is not None:
        _whole("q_weight", q_weight, (L_, D), torch.float32, dev)
        _whole("k_weight", k_weight, (L_, D), torch.float32, dev)
    if q_out is None:
        q_out = _empty_like(q)
    else:
        _whole("q_out", q_out, q.shape, q.dtype, dev)
        _apart("q_out", q_out, None, (q, k, v))
    _check("sparse_attn_cache_append",
           lib().sparse_attn_cache_append(
               p, c, cu_q.data_ptr(), cached.data_ptr(), q.data_ptr(), qs, k.data_ptr(), ks,
               v.data_ptr(), vs, _addr(q_weight), _addr(k_weight), float(eps),
               float(rope_base), q_out.data_ptr(), _raw_stream(dev)))
    return q_out


@_on_its_device
def cache_read(cache, page_table, lengths, *, rows=None, dtype=None, k_out=None, v_out=None):
    """The first lengths[b] rows of every sequence (int32 [B]) as contiguous
    (k, v) [L, B, Hkv, rows, D] (sparse_attn_cache_read): the stored, rotated keys
    and the values; float8_e4m3fn pages are read as dtype (bf16 by default).
    rows defaults to all that the page table covers, or to k_out's; rows from
    lengths[b] on are left as they were (zeros where the output is made here)."""
    if k_out is not None:
        dtype, rows = k_out.dtype, k_out.shape[3] if k_out.dim() == 5 else -1
    if dtype is None:
        dtype = torch.bfloat16 if cache.k.dtype == torch.float8_e4m3fn else cache.k.dtype
    dev, p, c = _paged_args(cache, page_table, dtype, None, 0, None)
    _whole("lengths", lengths, (p.B,), torch.int32, dev)
    rows = p.max_pages * p.page_size if rows is None else _int32(rows)
    if rows < 0:
        raise ValueError("k_out and v_out must be [L, B, Hkv, rows, D], rows at least 0")
    shape = (p.L, p.B, p.Hkv, rows, p.D)
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out: both or neither")
    if k_out is None:
        k_out, v_out = (cache.k.new_zeros(shape, dtype=dtype) for _ in range(2))
    else:
        _whole("k_out", k_out, shape, dtype, dev)
        _whole("v_out", v_out, shape, dtype, dev)
        _apart("v_out", v_out, None, (k_out,))
    _check("sparse_attn_cache_read",
           lib().sparse_attn_cache_read(p, c, lengths.data_ptr(), rows, k_out.data_ptr(),
                                        v_out.data_ptr(), _raw_stream(dev)))
    return k_out, v_out


@_on_its_device
def chunk_attn(q, cache, page_table, cu_q, cached, alpha, *, window, offsets=FIB15, sinks=0,
               scale=0.0, beta=None, out=None, lse=None, want_lse=True):
    """Sparse attention of new tokens over the paged cache, which holds their own
    rows already (sparse_attn_chunk): returns (O [L, N, Hq, D], LSE [L, N, Hq] or
    None).  One token per sequence is a decode step, many are a prefill chunk, and
    a call may mix them.

    q [L, N, Hq, D]: rotated queries (cache_append's), rows contiguous; Hq a
    multiple of the cache's heads.  page_table, cu_q, cached: as given to
    cache_append.  alpha: fp32 [L].  beta: optional fp32 [L, N, Hq] log-prior on the
    offset members.  window, offsets, sinks, scale: as in fwd().  Rows that belong
    to no sequence keep what out and lse held."""
    if q.dim() != 4:
        raise ValueError("q must be [L, N, Hq, D]")
    L_, N, Hq, D = q.shape
    dev, p, c = _paged_args(cache, page_table, q.dtype, L_, N, Hq)
    qs = _rows("q", q, (L_, N, Hq, p.D), q.dtype, dev, RowStrides)
    _sequences(cu_q, cached, p.B, dev)
    _whole("alpha", alpha, (L_,), torch.float32, dev)
    if beta is not None:
        _whole("beta", beta, (L_, N, Hq), torch.float32, dev)
    if out is None:
        out = _empty_like(q)
    else:
        _whole("out", out, q.shape, q.dtype, dev)
        _apart("out", out, None, (q,))
    if lse is not None:
        _whole("lse", lse, (L_, N, Hq), torch.float32, dev)
    elif want_lse:
        lse = alpha.new_empty((L_, N, Hq))
    offs = _offsets(tuple(offsets))
    _check("sparse_attn_chunk",
           lib().sparse_attn_chunk(p, c, cu_q.data_ptr(), cached.data_ptr(), q.data_ptr(), qs,
                                   alpha.data_ptr(), _addr(beta), _int32(window), len(offs),
                                   offs, _int32(sinks), float(scale), out.data_ptr(), _addr(lse),
                                   _raw_stream(dev)))
    return out, lse


@functools.lru_cache(maxsize=64)
def _offsets(offsets):
    """The offset table as a C array (copied by the library during the call)."""
    offsets = [int(x) for x in offsets]
    if any(x != _int32(x) for x in offsets):
        raise ValueError("offsets must fit 32 bits")
    return (ctypes.c_int32 * len(offsets))(*offsets)


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
