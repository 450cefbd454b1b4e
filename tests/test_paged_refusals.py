"""Refusals of the query/key norm, the paged cache and the chunk attention: the C
entry points reject bad arguments on the host before anything is launched (these
tests need no GPU; the pointers are never dereferenced), and the binding rejects
tensors that do not fit together."""
import ctypes

import pytest
import torch

import structured_sparse_attention_fibonacci_b200 as sa
from structured_sparse_attention_fibonacci_b200 import build as sa_build
from structured_sparse_attention_fibonacci_b200 import paged

OK = 1 << 20
ODD = OK + 8
INVALID, UNSUPPORTED = sa.SA_ERR_INVALID_ARG, sa.SA_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    sa_build.build()
    return sa.lib()


NORM = dict(L=1, B=1, Hq=2, Hkv=1, T=4, D=64, pos0=0, rotate=1, eps=1e-6, rope_base=1e4,
            dtype=sa.SA_DTYPE_BF16)
NORM_BAD = [
    (dict(L=0), INVALID), (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(D=48), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(pos0=-1), INVALID), (dict(pos0=(1 << 24) - 3), UNSUPPORTED), (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=INF), INVALID), (dict(rope_base=0.0), INVALID),
    (dict(rope_base=NAN), INVALID), (dict(dtype=7), INVALID), (dict(L=70000), UNSUPPORTED),
    (dict(B=1 << 20, T=1 << 12), UNSUPPORTED), (dict(Hq=65535), UNSUPPORTED),
]


def _norm(lib, kw=(), hs=(64, 64, 64, 64), q=OK, qw=OK, kwt=OK, out=OK):
    p = paged.QkNormParams(**{**NORM, **dict(kw)})
    s = paged.HeadStrides(*hs)
    return lib.sparse_attn_qk_norm_rope(p, q, s, OK, s, qw, kwt, out, OK, None)


def _norm_bwd(lib, kw=(), hs=(64, 64, 64, 64), dy=OK, qw=OK, kwt=OK, dqw=OK, dkw=OK, ws=OK,
              n=1 << 30):
    p = paged.QkNormParams(**{**NORM, **dict(kw)})
    s = paged.HeadStrides(*hs)
    return lib.sparse_attn_qk_norm_rope_bwd(p, OK, s, OK, s, qw, kwt, dy, s, OK, s, OK, OK, dqw,
                                            dkw, ws, n, None)


@pytest.mark.parametrize("bad,code", NORM_BAD)
def test_norm_params(lib, bad, code):
    assert _norm(lib, bad) == code
    assert _norm_bwd(lib, bad) == code
    assert lib.sparse_attn_qk_norm_workspace_size(paged.QkNormParams(**{**NORM, **bad})) == 0


def test_norm_pointers(lib):
    for kw in (dict(q=None), dict(q=ODD), dict(out=None), dict(out=ODD), dict(qw=None),
               dict(kwt=None), dict(qw=OK + 4), dict(hs=(64, 64, 4, 64)), dict(hs=(64, 64, 64, 7))):
        assert _norm(lib, **kw) == INVALID, kw
    assert _norm(lib, dict(rotate=0), qw=None, kwt=None) == INVALID      # nothing to do
    for kw in (dict(dy=None), dict(dy=ODD), dict(dqw=None), dict(dkw=OK + 2),
               dict(qw=None, kwt=None), dict(hs=(64, 1, 64, 64))):
        assert _norm_bwd(lib, **kw) == INVALID, kw
    assert _norm_bwd(lib, ws=None) == sa.SA_ERR_WORKSPACE
    assert _norm_bwd(lib, ws=ODD) == sa.SA_ERR_WORKSPACE
    assert _norm_bwd(lib, n=16) == sa.SA_ERR_WORKSPACE
    assert lib.sparse_attn_qk_norm_rope(None, OK, None, OK, None, OK, OK, OK, OK, None) == INVALID
    p = paged.QkNormParams(**NORM)
    assert lib.sparse_attn_qk_norm_rope(p, OK, None, OK, None, OK, OK, OK, OK, None) == INVALID


PAGED = dict(L=1, N=3, B=2, Hq=4, Hkv=2, D=64, n_pages=8, page_size=16, max_pages=4,
             dtype=sa.SA_DTYPE_BF16, format=0)
PAGED_BAD = [
    (dict(L=0), INVALID), (dict(N=-1), INVALID), (dict(B=-1), INVALID), (dict(Hq=3), INVALID),
    (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(D=80), UNSUPPORTED),
    (dict(n_pages=0), INVALID), (dict(page_size=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(dtype=2), INVALID), (dict(format=2), INVALID),
    (dict(page_size=1 << 20, max_pages=17), UNSUPPORTED),
    (dict(n_pages=1 << 30, page_size=16), UNSUPPORTED), (dict(L=65536), UNSUPPORTED),
    (dict(Hq=65536, Hkv=1), UNSUPPORTED), (dict(N=(1 << 30) + 1), UNSUPPORTED),
]


def _pages(fmt, **kw):
    sc = OK if fmt else None
    f = dict(k=OK, v=OK, k_scale=sc, v_scale=sc, page_table=OK)
    return paged.Pages(**{**f, **kw})


def _append(lib, kw=(), pages=None, rs=(64, 64, 64), q=OK, cu=OK, cached=OK, qw=None, kwt=None,
            eps=1e-6, base=1e4, out=OK):
    f = {**PAGED, **dict(kw)}
    s = paged.RowStrides(*rs)
    return lib.sparse_attn_cache_append(paged.PagedParams(**f), pages or _pages(f["format"]), cu,
                                        cached, q, s, OK, s, OK, s, qw, kwt, eps, base, out, None)


def _read(lib, kw=(), pages=None, lengths=OK, rows=5, k=OK):
    f = {**PAGED, **dict(kw)}
    return lib.sparse_attn_cache_read(paged.PagedParams(**f), pages or _pages(f["format"]), lengths,
                                      rows, k, OK, None)


def _chunk(lib, kw=(), pages=None, rs=(64, 64, 64), q=OK, alpha=OK, beta=None, W=12, offs=(1, 2),
           S=0, scale=0.0, o=OK, lse=None):
    f = {**PAGED, **dict(kw)}
    a = (ctypes.c_int32 * max(1, len(offs)))(*offs)
    return lib.sparse_attn_chunk(paged.PagedParams(**f), pages or _pages(f["format"]), OK, OK, q,
                                 paged.RowStrides(*rs), alpha, beta, W, len(offs), a, S, scale, o,
                                 lse, None)


@pytest.mark.parametrize("bad,code", PAGED_BAD)
def test_paged_params(lib, bad, code):
    assert _append(lib, bad) == code
    assert _chunk(lib, bad) == code
    if "N" not in bad or bad["N"] < 0:
        assert _read(lib, bad) == code


def test_paged_pointers(lib):
    for f in (_append, _read, _chunk):
        for kw in (dict(k=None), dict(k=ODD), dict(v=None), dict(page_table=None),
                   dict(page_table=OK + 2), dict(k_scale=OK)):
            assert f(lib, pages=_pages(0, **kw)) == INVALID, kw
        for kw in (dict(k_scale=None), dict(v_scale=None), dict(v_scale=OK + 1)):
            assert f(lib, dict(format=1), pages=_pages(1, **kw)) == INVALID, kw
    for kw in (dict(q=None), dict(q=ODD), dict(cu=None), dict(cached=OK + 1), dict(out=ODD),
               dict(qw=OK), dict(kwt=OK), dict(qw=ODD, kwt=OK), dict(eps=-1.0), dict(eps=NAN),
               dict(base=0.0), dict(base=INF), dict(rs=(64, 64, 3))):
        assert _append(lib, **kw) == INVALID, kw
    for kw in (dict(q=None), dict(alpha=None), dict(alpha=OK + 2), dict(beta=OK + 1),
               dict(lse=OK + 1), dict(o=None), dict(o=ODD), dict(W=0), dict(S=-1), dict(offs=(1, 0)),
               dict(scale=NAN), dict(scale=INF), dict(rs=(64, 9, 64))):
        assert _chunk(lib, **kw) == INVALID, kw
    assert _chunk(lib, S=17) == UNSUPPORTED
    assert _chunk(lib, offs=tuple(range(1, 34))) == UNSUPPORTED
    for kw in (dict(lengths=None), dict(k=None), dict(k=ODD), dict(rows=-1)):
        assert _read(lib, **kw) == INVALID, kw
    assert _read(lib, dict(B=65536)) == UNSUPPORTED
    assert _read(lib, rows=(1 << 24) + 1) == UNSUPPORTED


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((1, 1, 2, 4, 16))
    w = torch.ones((1, 16))
    with pytest.raises(ValueError):
        sa.qk_norm_rope(x, x, w, w)
    cache = sa.paged_cache(1, 2, 2, 4, 16, torch.float32, device="cpu")
    i32 = lambda t: torch.tensor(t, dtype=torch.int32)
    with pytest.raises(ValueError):
        sa.cache_append(x[0], x[0], x[0], cache, i32([[0, 1]]), i32([0, 2]), i32([0]))
    with pytest.raises(ValueError):
        sa.cache_read(cache, i32([[0, 1]]), i32([0]))
    with pytest.raises(ValueError):
        sa.chunk_attn(x[0], cache, i32([[0, 1]]), i32([0, 2]), i32([0]), torch.ones(1), window=2)
    with pytest.raises(TypeError):
        sa.paged_cache(1, 2, 2, 4, 16, torch.float16, device="cpu")


@pytest.mark.gpu
def test_binding_refuses_tensors_that_do_not_fit():
    dev = "cuda"
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype, device=dev)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=dev)
    q, k, w = z(1, 1, 4, 6, 64), z(1, 1, 2, 6, 64), z(1, 64, dtype=torch.float32)
    for args, kw in (((q, k[:, :, :, :5], w, w), {}), ((q, k.float(), w, w), {}),
                     ((q, k, w, None), {}), ((q, k, w.bfloat16(), w), {}),
                     ((q, k, None, None), dict(rotate=False)),
                     ((q[..., ::2], k[..., ::2], w[:, :32], w[:, :32]), {}),
                     ((q, k, w, w), dict(q_out=q[:, :, :2])),
                     ((q, k, w, w), dict(q_out=z(1, 1, 4, 6, 64, dtype=torch.float32))),
                     ((q[:, :, :2], k, w, w), dict(q_out=k))):
        with pytest.raises((ValueError, TypeError)):
            sa.qk_norm_rope(*args, **kw)
    with pytest.raises(TypeError):
        sa.qk_norm_rope(q.half(), k.half(), w, w)
    with pytest.raises(sa.SparseAttnError):
        sa.qk_norm_rope(q, k, w, w, eps=-1.0)
    big = z(2, 1, 4, 6, 64)
    with pytest.raises(ValueError):      # an output that overlaps its input, shifted
        sa.qk_norm_rope(big.view(-1)[64:64 + q.numel()].view(q.shape), k, w, w,
                        q_out=big.view(-1)[:q.numel()].view(q.shape))
    with pytest.raises(ValueError):      # one tensor for both outputs
        sa.qk_norm_rope(q, q, w, w, q_out=q, k_out=q)
    with pytest.raises(ValueError):
        sa.qk_norm_rope_bwd(q, k, w, w, q, k[:, :, :1])
    with pytest.raises(sa.SparseAttnError):
        sa.qk_norm_rope_bwd(q, k, w, w, q.clone(), k.clone(), workspace=z(4, dtype=torch.uint8))
    x, y = z(1, 3, 4, 64), z(1, 3, 2, 64)
    cache, table, cu, old = sa.paged_cache(1, 4, 2, 16, 64), i32([[0, 1], [2, 3]]), i32([0, 1, 3]), i32([0, 0])
    alpha = torch.ones(1, device=dev)
    good = (x, y, y, cache, table, cu, old)
    sa.cache_append(*good)
    q8 = sa.paged_cache(1, 4, 2, 16, 64, torch.float8_e4m3fn)
    for i, bad in ((0, x.float()), (0, x[..., :32]), (1, y[:, :2]), (2, x), (3, sa.paged_cache(2, 4, 2, 16, 64)),
                   (3, sa.PagedCache(q8.k, q8.v)), (3, sa.PagedCache(cache.k, cache.v, q8.k_scale, q8.v_scale)),
                   (3, sa.PagedCache(cache.k, cache.v[:, :3])), (4, table.long()), (4, table[0]),
                   (4, table.t()), (5, cu[:2]), (5, cu.float()), (6, old[:1]), (6, old.cpu())):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError)):
            sa.cache_append(*args)
    with pytest.raises(ValueError):
        sa.cache_append(*good, q_weight=w)
    with pytest.raises(ValueError):
        sa.cache_append(*good, q_out=x)
    with pytest.raises(sa.SparseAttnError):     # rows of 8-byte alignment
        odd = z(3 * 4 * 64 + 4)[4:].view(1, 3, 4, 64)
        sa.cache_append(odd, y, y, cache, table, cu, old)
    for kw in (dict(window=0), dict(window=3, offsets=(0,)), dict(window=3, sinks=-1),
               dict(window=3, sinks=17)):
        with pytest.raises(sa.SparseAttnError):
            sa.chunk_attn(x, cache, table, cu, old, alpha, **kw)
    for kw in (dict(beta=z(1, 3, 4)), dict(out=x), dict(out=z(1, 3, 4, 64, dtype=torch.float32)),
               dict(lse=z(1, 3, 2, dtype=torch.float32))):
        with pytest.raises(ValueError):
            sa.chunk_attn(x, cache, table, cu, old, alpha, window=3, **kw)
    with pytest.raises(sa.SparseAttnError):
        sa.chunk_attn(z(1, 3, 3, 64), cache, table, cu, old, alpha, window=3)
    for kw in (dict(rows=-1), dict(dtype=torch.float16), dict(k_out=z(1, 2, 2, 8, 64))):
        with pytest.raises((ValueError, TypeError)):
            sa.cache_read(cache, table, old, **kw)
