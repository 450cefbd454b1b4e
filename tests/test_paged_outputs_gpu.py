"""What the paged and norm calls write: outputs that lie in another tensor of the call are
refused before anything is launched, and outputs given are what the call is for."""
import pytest
import torch

import structured_sparse_attention_fibonacci_b200 as sa

DEV = "cuda"
BF, F32, Q8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
pytestmark = pytest.mark.gpu

# sizes that every tensor below can lie in: L, N, Hq, Hkv, D, pages, rows of a page, B, max_pages
L, N, HQ, HKV, D, P, PAGE, B, MP = 1, 3, 4, 2, 64, 4, 16, 2, 2


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _inside(host, shape, dtype):
    """A contiguous tensor in the first bytes of another one's memory."""
    n = torch.empty(shape, dtype=dtype).nbytes
    raw = torch.empty(0, dtype=torch.uint8, device=DEV).set_(
        host.untyped_storage(), host.storage_offset() * host.element_size(), (n,))
    return raw.view(dtype).view(shape)


def _tensors(dtype, fmt):
    """The tensors of a cache call, each with memory enough for any output to lie in it."""
    room = 1 << 15

    def make(shape, t, value=0):
        x = torch.zeros(room, dtype=torch.uint8, device=DEV)
        x = _inside(x, shape, t)
        return x.fill_(value) if t != Q8 else x
    pool = (L, P, HKV, PAGE, D)
    t = dict(q=make((L, N, HQ, D), dtype), k=make((L, N, HKV, D), dtype), v=make((L, N, HKV, D), dtype),
             kc=make(pool, Q8 if fmt == "e4m3" else dtype), vc=make(pool, Q8 if fmt == "e4m3" else dtype),
             ks=None, vs=None, table=make((B, MP), torch.int32), cu=make((B + 1,), torch.int32),
             cached=make((B,), torch.int32), qw=make((L, D), F32, 1), kw=make((L, D), F32, 1),
             alpha=make((L,), F32, 1), beta=make((L, N, HQ), F32))
    if fmt == "e4m3":
        t["ks"], t["vs"] = make(pool[:4], F32, 1), make(pool[:4], F32, 1)
    t["table"].copy_(i32([[0, 1], [2, 3]]))
    t["cu"].copy_(i32([0, 1, 3]))
    return t


def _append(t, **kw):
    return sa.cache_append(t["q"], t["k"], t["v"], sa.PagedCache(t["kc"], t["vc"], t["ks"], t["vs"]),
                           t["table"], t["cu"], t["cached"], q_weight=t["qw"], k_weight=t["kw"], **kw)


def _chunk(t, **kw):
    return sa.chunk_attn(t["q"], sa.PagedCache(t["kc"], t["vc"], t["ks"], t["vs"]), t["table"],
                         t["cu"], t["cached"], t["alpha"], window=4, beta=t["beta"], **kw)


def _read(t, **kw):
    return sa.cache_read(sa.PagedCache(t["kc"], t["vc"], t["ks"], t["vs"]), t["table"], t["cached"], **kw)


@pytest.mark.parametrize("dtype,fmt", [(BF, "plain"), (F32, "e4m3")])
def test_outputs_inside_other_tensors_of_a_cache_call_are_refused(dtype, fmt):
    t = _tensors(dtype, fmt)
    rows = (L, N, HQ, D)
    for host in ("q", "k", "v", "kc", "vc", "ks", "vs", "table", "cu", "cached", "qw", "kw"):
        if t[host] is not None:
            with pytest.raises(ValueError, match="overlaps"):
                _append(t, q_out=_inside(t[host], rows, dtype))
    for host in ("q", "kc", "vc", "ks", "vs", "table", "cu", "cached", "alpha", "beta"):
        if t[host] is not None:
            with pytest.raises(ValueError, match="overlaps"):
                _chunk(t, out=_inside(t[host], rows, dtype))
            with pytest.raises(ValueError, match="overlaps"):
                _chunk(t, lse=_inside(t[host], (L, N, HQ), F32))
    both = torch.zeros(1 << 12, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):
        _chunk(t, out=_inside(both, rows, dtype), lse=_inside(both, (L, N, HQ), F32))
    out = (L, B, HKV, 5, D)
    other = torch.zeros(out, dtype=dtype, device=DEV)
    for host in ("kc", "vc", "ks", "vs", "table", "cached"):
        if t[host] is not None:
            x = _inside(t[host], out, dtype)
            for kw in (dict(k_out=x, v_out=other), dict(k_out=other, v_out=x)):
                with pytest.raises(ValueError, match="overlaps"):
                    _read(t, **kw)
    with pytest.raises(ValueError, match="overlaps"):
        _read(t, k_out=other, v_out=other)
    # an append writes the pages: no input and no other part of the cache lies in them
    for host in ("kc", "vc", "ks", "vs"):
        if t[host] is None:
            continue
        for name, shape, ty in (("q", rows, dtype), ("k", (L, N, HKV, D), dtype), ("v", (L, N, HKV, D), dtype),
                                ("cu", (B + 1,), torch.int32), ("table", (B, MP), torch.int32),
                                ("qw", (L, D), F32)):
            with pytest.raises(ValueError, match="overlaps"):
                _append({**t, name: _inside(t[host], shape, ty)})
    with pytest.raises(ValueError, match="overlaps"):
        _append({**t, "vc": t["kc"]})
    if fmt == "e4m3":
        with pytest.raises(ValueError, match="overlaps"):
            _append({**t, "vs": t["ks"]})
    _append(t)
    _chunk(t)
    # reading is not writing: one tensor may hold keys and values
    o, _ = _chunk({**t, "vc": t["kc"], "vs": t["ks"]})
    assert torch.isfinite(o.float()).all()
    torch.cuda.synchronize()


def test_outputs_inside_other_tensors_of_a_norm_call_are_refused():
    room = 1 << 14
    make = lambda s, v=0.0: _inside(torch.zeros(room, dtype=torch.uint8, device=DEV), s, F32).fill_(v)
    sq, sk = (L, 1, 2, 4, D), (L, 1, 1, 4, D)
    q, k, qw, kw, dyq, dyk = make(sq, 1), make(sk, 1), make((L, D), 1), make((L, D), 1), make(sq), make(sk)
    for host in (k, qw, kw):
        with pytest.raises(ValueError, match="overlaps"):
            sa.qk_norm_rope(q, k, qw, kw, q_out=_inside(host, sq, F32))
    for host in (q, qw, kw):
        with pytest.raises(ValueError, match="overlaps"):
            sa.qk_norm_rope(q, k, qw, kw, k_out=_inside(host, sk, F32))
    bwd = lambda **o: sa.qk_norm_rope_bwd(q, k, qw, kw, dyq, dyk, **o)
    n = sa.qk_norm_workspace_size(sq, sk, F32)
    assert n <= room
    for host in (q, k, qw, kw, dyk):
        with pytest.raises(ValueError, match="overlaps"):
            bwd(dq=_inside(host, sq, F32))
    for host in (q, k, qw, kw, dyq):
        with pytest.raises(ValueError, match="overlaps"):
            bwd(dk=_inside(host, sk, F32))
    for host in (q, k, dyq, dyk):
        for name in ("dq_weight", "dk_weight"):
            with pytest.raises(ValueError, match="overlaps"):
                bwd(**{name: _inside(host, (L, D), F32)})
    out = make(sq)
    for name in ("dq_weight", "dk_weight"):
        with pytest.raises(ValueError, match="overlaps"):
            bwd(dq=out, **{name: _inside(out, (L, D), F32)})
    same = make((L, D))
    with pytest.raises(ValueError, match="overlaps"):
        bwd(dq_weight=same, dk_weight=same)
    for host in (q, k, qw, kw, dyq, dyk):
        with pytest.raises(ValueError, match="overlaps"):
            bwd(workspace=_inside(host, (n,), torch.uint8))
    for kw_ in (dict(dq=out), dict(dq_weight=_inside(out, (L, D), F32))):
        with pytest.raises(ValueError, match="overlaps"):
            bwd(workspace=_inside(out, (n,), torch.uint8), **kw_)
    # in place, as documented
    d1, d2 = dyq.clone(), dyk.clone()
    for a, b in zip(bwd(), sa.qk_norm_rope_bwd(q, k, qw, kw, d1, d2, dq=d1, dk=d2)):
        assert torch.equal(a, b)


def test_read_outputs_are_what_the_call_asks_for():
    """rows= and dtype= beside outputs that have others: refused, not passed over."""
    cache = sa.paged_cache(L, P, HKV, PAGE, D, Q8)
    table, lengths = i32([[0, 1], [2, 3]]), i32([9, 3])
    k, v = (torch.zeros((L, B, HKV, 8, D), dtype=BF, device=DEV) for _ in range(2))
    for kw in (dict(rows=5), dict(rows=9), dict(rows=0), dict(dtype=F32), dict(rows=8, dtype=F32)):
        with pytest.raises(ValueError):
            sa.cache_read(cache, table, lengths, k_out=k, v_out=v, **kw)
    for kw in (dict(), dict(rows=8), dict(dtype=BF), dict(rows=8, dtype=BF)):
        got = sa.cache_read(cache, table, lengths, k_out=k, v_out=v, **kw)
        assert got[0].data_ptr() == k.data_ptr() and got[1].data_ptr() == v.data_ptr()
    with pytest.raises(TypeError):
        sa.cache_read(cache, table, lengths, k_out=k, v_out=v, dtype="bf16")
