"""The paged cache (append, read back) and the chunk attention on the GPU against
their plain 64-bit forms, and the operators used together.

Tolerances, per element, from the arithmetic: a stored value is off by at most
half a step, u = torch.finfo(dtype).eps / 2 of its size (bf16 2^-8, fp32 2^-24;
e4m3 2^-4, or half its smallest step 2^-10 under the row's scale).  With A = sum
p |v| and Q = max over members of sum |q k| scale:
  LSE    2^-20 (Q + |LSE| + 1)                    fp32 sums of D products, exp2 and log2
  O fp32 (2^-18 (Q + 1) + 2^-24 members) A        the scores' errors through exp, sums
  O bf16 that, + 2^-8 A for the rounded probabilities, + 2^-8 |O| for the output
|v| of an interpolated member in A is (1 - w) |row a| + w |row b|: its two rows have
rounded probabilities p (1 - w) and p w of their own, each off by up to 2^-8 of
itself, whose errors do not cancel where the rows themselves do.
"""
import math

import pytest
import torch

import structured_sparse_attention_fibonacci_b200 as sa
import paged_plain as plain

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu

FIB = sa.FIB15
MANY = tuple(sorted(set(FIB + (7, 7, 11, 16, 30, 60, 64, 100, 200, 400))))[:24] + (2, 2)


def _run_chunk(t, q, alpha, **kw):
    cache, table, cu, cached = t.device(sa)
    beta = kw.pop("beta", None)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, dtype=F32, device=DEV)
    sa.chunk_attn(q.to(DEV), cache, table, cu, cached, torch.tensor(alpha, device=DEV), out=out,
                  lse=lse, beta=None if beta is None else beta.to(DEV), **kw)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def _check_chunk(t, q, out, lse, ref, dtype, n_members):
    o, l, mag, big = ref
    live = ~torch.isnan(l)
    inside = torch.zeros(t.N, dtype=torch.bool)
    inside[t.cu[0]:t.cu[-1]] = True
    assert (out[:, ~inside] == 7.0).all() and (lse[:, ~inside] == 7.0).all()
    assert live[:, inside].all()
    tol = 2.0 ** -20 * (big + l.abs() + 1)
    bad = ((lse.double() - l).abs() - tol)[:, inside]
    assert (bad <= 0).all(), f"LSE beyond its bound by {bad.max().item():.3g}"
    tol = (2.0 ** -18 * (big[..., None] + 1) + 2.0 ** -24 * n_members) * mag
    if dtype == BF:
        tol = tol + 2.0 ** -8 * mag + 2.0 ** -8 * o.abs()
    bad = ((out.double() - o).abs() - tol)[:, inside]
    assert (bad <= 0).all(), f"O beyond its bound by {bad.max().item():.3g}"


# (id, dtype, format, D, Hq, Hkv, page, W, S, offsets, alphas, old, new, lead, tail)
CHUNK = [
    ("bf16_d64_mha", BF, "plain", 64, 2, 2, 16, 12, 0, FIB, [1.0, 0.5], [0, 40, 1100, 3],
     [20, 1, 9, 0], 0, 0),
    ("bf16_d64_sinks_pad", BF, "plain", 64, 3, 3, 7, 64, 4, FIB, [1.37], [0, 5, 130],
     [70, 3, 33], 2, 5),
    ("bf16_d64_e4m3", BF, "e4m3", 64, 2, 1, 16, 12, 2, FIB, [0.83, 1.5], [0, 200, 17],
     [31, 1, 8], 0, 1),
    ("bf16_d128_gqa4_e4m3", BF, "e4m3", 128, 8, 2, 16, 12, 0, FIB, [1.1], [0, 300], [19, 6], 0, 0),
    ("bf16_d128_gqa8", BF, "plain", 128, 8, 1, 32, 5, 1, (16,), [1.0], [0, 33, 0], [4, 1, 40], 0, 0),
    ("bf16_d32_gqa3", BF, "plain", 32, 6, 2, 5, 9, 0, FIB, [0.7, 1.0], [0, 64], [33, 2], 0, 0),
    ("bf16_d16_gqa6_e4m3", BF, "e4m3", 16, 6, 1, 1, 3, 16, (1, 4, 9), [1.25], [0, 20], [25, 1],
     0, 0),
    ("bf16_d16_mha", BF, "plain", 16, 1, 1, 64, 1, 0, FIB, [1.0], [0], [130], 0, 0),
    ("bf16_d32_gqa12_e4m3", BF, "e4m3", 32, 12, 1, 16, 17, 3, FIB, [0.9], [50], [7], 0, 0),
    ("bf16_d64_gqa9_many", BF, "plain", 64, 9, 1, 16, 12, 0, MANY, [0.77], [0, 700], [11, 9], 0, 0),
    ("bf16_d64_none", BF, "plain", 64, 4, 2, 16, 33, 0, (), [1.0], [0, 70], [40, 1], 0, 0),
    ("bf16_d64_w1", BF, "plain", 64, 2, 2, 16, 1, 0, (), [1.0], [0], [1], 0, 0),
    ("bf16_d64_w300", BF, "e4m3", 64, 1, 1, 128, 300, 4, FIB, [1.0], [0, 900], [50, 1], 0, 0),
    ("bf16_d64_wide_window", BF, "plain", 64, 1, 1, 16, 1 << 30, 0, (3,), [1.5], [0, 90], [20, 1],
     0, 0),
    ("f32_d16", F32, "plain", 16, 2, 2, 16, 6, 0, FIB, [1.0, 0.66], [0, 40], [64, 1], 1, 2),
    ("f32_d32_gqa_e4m3", F32, "e4m3", 32, 6, 2, 7, 12, 2, FIB, [1.3], [0, 100], [20, 3], 0, 0),
    ("f32_d64", F32, "plain", 64, 2, 1, 16, 40, 4, MANY, [0.8], [0, 500], [30, 1], 0, 0),
    ("f32_d64_e4m3", F32, "e4m3", 64, 2, 2, 16, 12, 0, (), [1.0], [3], [10], 0, 0),
    ("f32_d128", F32, "plain", 128, 3, 1, 3, 12, 0, FIB, [1.45], [0, 200], [17, 1], 0, 0),
    ("f32_d16_e4m3", F32, "e4m3", 16, 4, 4, 16, 50, 0, FIB, [1.0], [0], [60], 0, 0),
    ("f32_d128_e4m3", F32, "e4m3", 128, 2, 2, 16, 4, 16, (5,), [0.9], [0, 60], [18, 1], 0, 0),
]


# Integer distances, in and out of the window, twice the same, at its edge, at 0, all of them in
# it, more than 8 outside; and rows enough for several key tiles
for n, (offs, alphas, W) in enumerate([
        ((1, 2, 3), [1.0, 2.0], 12), ((5, 5, 1, 12, 11, 13, 5), [1.0], 12), (FIB, [1.0, 2.0], 22),
        (FIB, [3.0, 0.0], 64), ((63, 64, 65, 1, 31, 32, 33, 90, 2, 3), [1.0], 80),
        (tuple(range(1, 17)), [1.0, 4.0], 8), (tuple(range(1, 17)), [1.0], 100)]):
    for dtype, fmt, D, Hq, Hkv in ((BF, "plain", 64, 2, 2), (BF, "e4m3", 32, 4, 1),
                                   (BF, "plain", 16, 6, 2), (F32, "plain", 16, 1, 1)):
        CHUNK.append((f"integer_{n}_{fmt}_{Hq}x{D}", dtype, fmt, D, Hq, Hkv, 16, W, n % 3, offs, alphas,
                      [0, 130, 9], [21, 1, 14], 0, 0))


# Interpolated distances, one query head per key head: tokens share each other's rows
for D in (16, 32, 64, 128):
    for fmt in ("plain", "e4m3"):
        for n, (offs, W) in enumerate(((FIB, 12), (MANY, 5), ((1,), 20), ((3, 900, 1, 2, 6), 1))):
            CHUNK.append((f"shared_{n}_{fmt}_{D}", BF, fmt, D, 2, 2, (16, 5, 64, 1)[n], W, 2 * (n % 2), offs,
                          [0.77, 1.37], [0, 300, 77, 12], [37, 9, 4, 3], n, n))


@pytest.mark.parametrize("prior", [False, True], ids=["", "prior"])
@pytest.mark.parametrize("case", CHUNK, ids=[c[0] for c in CHUNK])
def test_chunk_matches_the_plain_form(case, prior):
    name, dtype, fmt, D, Hq, Hkv, page, W, S, offs, alpha, old, new, lead, tail = case
    t = plain.Batch(len(alpha), Hkv, D, page, old, new, dtype, fmt, seed=len(name), lead=lead,
                    tail=tail)
    g = torch.Generator().manual_seed(7)
    # queries as views with a stride of their own, NaN where no sequence has a row
    q = torch.randn((len(alpha), t.N, Hq + 2, D), generator=g).to(dtype)[:, :, 1:Hq + 1]
    q[:, :lead] = math.nan
    q[:, t.cu[-1]:] = math.nan
    beta = torch.randn((len(alpha), t.N, Hq), generator=g) if prior else None
    out, lse = _run_chunk(t, q.to(DEV), alpha, window=W, sinks=S, offsets=offs, beta=beta)
    ref = plain.chunk(q.double(), t.keys, t.vals, t.cu, t.old, alpha, W, S, offs,
                      beta=None if beta is None else beta.double())
    _check_chunk(t, q, out, lse, ref, dtype, min(W, max(t.held)) + S + 2 * len(offs))


# (format, D, Hq, Hkv, W, S, offsets, old, new): few tokens with windows that the warps of one,
# two, four and eight CTAs share, short sequences beside long ones
LONG = [("plain", 64, 2, 2, 400, 4, FIB, [4200, 3], [1, 1]),
        ("plain", 64, 2, 2, 700, 0, (3,), [4200, 650], [1, 2]),
        ("e4m3", 64, 4, 2, 1500, 4, FIB, [4200, 0], [9, 3]),
        ("plain", 128, 8, 1, 4000, 0, FIB, [4200], [1]), ("e4m3", 128, 8, 1, 4000, 4, FIB, [4200, 40], [1, 1]),
        ("plain", 32, 1, 1, 4000, 16, (), [4200, 0], [5, 1]), ("e4m3", 16, 6, 2, 2500, 0, MANY, [4200], [2])]


@pytest.mark.parametrize("alpha", [1.0, 1.3])
@pytest.mark.parametrize("case", LONG, ids=[f"{c[0]}_{c[2]}x{c[1]}_w{c[4]}" for c in LONG])
def test_long_windows_of_few_tokens(case, alpha):
    """As the cases above; LSE has 2^-24 per member more, for the sum's additions."""
    fmt, D, Hq, Hkv, W, S, offs, old, new = case
    t = plain.Batch(1, Hkv, D, 64, old, new, BF, fmt, seed=D)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((1, t.N, Hq, D), generator=g).to(BF)
    beta = torch.randn((1, t.N, Hq), generator=g)
    out, lse = _run_chunk(t, q, [alpha], window=W, sinks=S, offsets=offs, beta=beta)
    o, l, mag, big = plain.chunk(q.double(), t.keys, t.vals, t.cu, t.old, [alpha], W, S, offs,
                                 beta=beta.double())
    n = min(W, max(t.held)) + S + 2 * len(offs)
    assert ((lse.double() - l).abs() <= 2.0 ** -20 * (big + l.abs() + 1) + 2.0 ** -24 * n).all()
    tol = (2.0 ** -18 * (big[..., None] + 1) + 2.0 ** -24 * n + 2.0 ** -8) * mag
    assert ((out.double() - o).abs() <= tol + 2.0 ** -8 * o.abs()).all()


@pytest.mark.device_error_expected
@pytest.mark.parametrize("fmt,D,W", [("plain", 64, 400), ("e4m3", 32, 1200), ("plain", 128, 4000)])
def test_a_bad_page_anywhere_in_a_shared_window(fmt, D, W):
    t = plain.Batch(1, 1, D, 64, [4200], [1], BF, fmt, seed=1)
    cache, table, cu, cached = t.device(sa)
    q = torch.randn((1, 1, 2, D), generator=torch.Generator().manual_seed(0)).to(BF).to(DEV)
    alpha = torch.ones(1, device=DEV)
    call = lambda: sa.chunk_attn(q, cache, table, cu, cached, alpha, window=W, offsets=(5,))
    want = call()
    assert sa.device_error(clear=True) == 0
    for page in range(table.shape[1]):
        good = table[0, page].clone()
        table[0, page] = 1 << 20
        o, lse = call()
        table[0, page] = good
        inside = (page + 1) * 64 > 4200 - W + 1 and page * 64 <= 4200
        assert sa.device_error(clear=True) == (sa.ERR_PAGE if inside else 0), page
        assert bool(torch.isnan(o).all()) == inside and bool(torch.isnan(lse).all()) == inside
        assert inside or (torch.equal(o, want[0]) and torch.equal(lse, want[1]))


@pytest.mark.parametrize("dtype,fmt,Hq,Hkv", [(BF, "plain", 1, 1), (BF, "e4m3", 4, 2),
                                              (F32, "plain", 2, 1), (F32, "e4m3", 1, 1)])
def test_masked_rows_with_infinities_and_nan_do_not_reach_a_query(dtype, fmt, Hq, Hkv):
    """Rows 30 (Inf in V), 37 (NaN in K) and 45 (NaN in V): queries that attend one are
    not finite exactly where the plain form is not; all others agree with it."""
    alpha, W, offs = [1.2], 5, (3, 8)
    t = plain.Batch(1, Hkv, 64, 16, [10], [60], dtype, fmt, seed=3)
    cache, table, cu, cached = t.device(sa)
    spoiled = {30: ("v", math.inf), 37: ("k", math.nan), 45: ("v", math.nan)}
    for r, (which, x) in spoiled.items():
        page, slot = int(t.table[0, r // 16]), r % 16
        pool = cache.k if which == "k" else cache.v
        held = t.keys[0] if which == "k" else t.vals[0]
        if fmt == "e4m3":       # as an append of such a row: a NaN scale
            (cache.k_scale if which == "k" else cache.v_scale)[:, page, :, slot] = math.nan
            held[:, :, r] = math.nan
        else:
            pool[:, page, :, slot, 5] = x
            held[:, :, r, 5] = x
    g = torch.Generator().manual_seed(1)
    q = torch.randn((1, t.N, Hq, 64), generator=g).to(dtype)
    o, lse = sa.chunk_attn(q.to(DEV), cache, table, cu, cached, torch.tensor(alpha, device=DEV),
                           window=W, offsets=offs)
    o, lse = o.cpu().double(), lse.cpu().double()
    ro, rl, mag, big = plain.chunk(q.double(), t.keys, t.vals, t.cu, t.old, alpha, W, 0, offs)
    assert torch.equal(torch.isfinite(o), torch.isfinite(ro))
    assert torch.equal(torch.isnan(o), torch.isnan(ro))
    assert torch.equal(torch.isnan(lse), torch.isnan(rl))
    ok = torch.isfinite(ro)
    assert 0.3 < ok.float().mean().item() < 0.9
    tol = (2.0 ** -18 * (big[..., None] + 1) + 2.0 ** -19) * mag
    tol = tol + (2.0 ** -8 * (mag + ro.abs()) if dtype == BF else 0.0)
    assert ((o - ro).abs() <= tol)[ok].all()


def test_scores_of_the_lowest_values_and_huge_scores():
    """Keys of +-1e4 along one axis: scores of +-1e4 spread over the members, so that all
    but the largest underflow; no NaN, and LSE is the largest."""
    t = plain.Batch(1, 1, 64, 16, [0], [40], BF, "plain", seed=5)
    cache, table, cu, cached = t.device(sa)
    big = torch.linspace(-1e4, 1e4, 40).to(BF)
    for r in range(40):
        cache.k[:, int(t.table[0, r // 16]), :, r % 16] = 0
        cache.k[:, int(t.table[0, r // 16]), :, r % 16, 3] = big[r].item()
        t.keys[0][:, :, r] = 0
        t.keys[0][:, :, r, 3] = big[r].double()
    q = torch.zeros((1, 40, 1, 64), dtype=BF)
    q[..., 3] = 8.0
    alpha = [1.0]
    o, lse = sa.chunk_attn(q.to(DEV), cache, table, cu, cached, torch.tensor(alpha, device=DEV),
                           window=9)
    ro, rl, mag, bigq = plain.chunk(q.double(), t.keys, t.vals, t.cu, t.old, alpha, 9, 0, FIB)
    assert ((lse.cpu().double() - rl).abs() <= 2.0 ** -20 * (bigq + rl.abs() + 1)).all()
    assert ((o.cpu().double() - ro).abs() <= (2.0 ** -18 * (bigq[..., None] + 1) + 2.0 ** -8) * mag
            + 2.0 ** -8 * ro.abs()).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_alpha_without_rows_makes_its_layer_nan(dtype):
    t = plain.Batch(3, 1, 32, 16, [5, 0], [9, 4], dtype, "plain", seed=2)
    q = torch.randn((3, t.N, 2, 32), generator=torch.Generator().manual_seed(0)).to(dtype)
    out, lse = _run_chunk(t, q, [1.0, math.nan, -0.5], window=4)
    assert torch.isfinite(out[0].float()).all() and torch.isfinite(lse[0]).all()
    assert torch.isnan(out[1:].float()).all() and torch.isnan(lse[1:]).all()


# ---- append and read ------------------------------------------------------------
# (id, dtype, format, L, Hq, Hkv, D, page, old, new, lead, tail, norm)
APPEND = [
    ("bf16_decode", BF, "plain", 3, 8, 8, 64, 16, [0, 5, 15, 16, 31], [1, 1, 1, 1, 1], 0, 0, False),
    ("bf16_norm_pad", BF, "plain", 2, 6, 2, 128, 16, [0, 100, 3], [37, 0, 5], 3, 4, True),
    ("bf16_e4m3_norm", BF, "e4m3", 2, 4, 1, 64, 7, [0, 9], [50, 1], 0, 2, True),
    ("bf16_e4m3_d16", BF, "e4m3", 1, 3, 3, 16, 1, [4, 0, 2], [3, 9, 1], 0, 0, False),
    ("bf16_e4m3_d128", BF, "e4m3", 1, 16, 2, 128, 64, [1000], [70], 0, 0, True),
    ("bf16_d32", BF, "plain", 1, 5, 5, 32, 5, [0], [23], 0, 0, True),
    ("f32_norm", F32, "plain", 2, 2, 2, 16, 16, [0, 30], [20, 1], 1, 0, True),
    ("f32_d64", F32, "plain", 1, 12, 3, 64, 16, [7], [40], 0, 0, False),
    ("f32_e4m3", F32, "e4m3", 1, 2, 1, 32, 16, [0, 0, 9], [1, 0, 20], 0, 0, True),
    ("f32_e4m3_d128", F32, "e4m3", 2, 2, 2, 128, 3, [11], [13], 0, 0, False),
]


@pytest.mark.parametrize("case", APPEND, ids=[c[0] for c in APPEND])
def test_append_and_read_match_the_plain_form(case):
    name, dtype, fmt, L, Hq, Hkv, D, page, old, new, lead, tail, normed = case
    t = plain.Batch(L, Hkv, D, page, old, new, dtype, fmt, seed=len(name))
    cu = [lead + c for c in t.cu]
    N, eps = cu[-1] + tail, 1e-5
    g = torch.Generator().manual_seed(11)
    x = torch.randn((L, N, Hq + 2 * Hkv, D), generator=g) * torch.logspace(-3, 3, N)[None, :, None, None]
    x = x.to(dtype)
    x[:, :lead] = math.nan
    x[:, cu[-1]:] = math.nan
    qw, kw = (1 + 0.3 * torch.randn((L, D), generator=g) for _ in range(2))
    cache, table, _, cached = t.device(sa)
    before = [None if y is None else y.clone() for y in cache]
    xd = x.to(DEV)
    q, k, v = xd[:, :, :Hq], xd[:, :, Hq:Hq + Hkv], xd[:, :, Hq + Hkv:]
    q_out = torch.full((L, N, Hq, D), 7.0, dtype=dtype, device=DEV)
    w = dict(q_weight=qw.to(DEV), k_weight=kw.to(DEV)) if normed else {}
    sa.cache_append(q, k, v, cache, table, torch.tensor(cu, dtype=torch.int32, device=DEV), cached,
                    eps=eps, q_out=q_out, **w)
    held = torch.tensor(t.held, dtype=torch.int32, device=DEV)
    kr, vr = sa.cache_read(cache, table, held, dtype=dtype)
    torch.cuda.synchronize()
    inside = torch.zeros(N, dtype=torch.bool)
    inside[cu[0]:cu[-1]] = True
    assert (q_out.cpu()[:, ~inside] == 7.0).all()
    u = torch.finfo(dtype).eps / 2
    xf = x.double()
    for b in range(len(old)):
        rows, pos = slice(cu[b], cu[b + 1]), old[b] + torch.arange(new[b])
        # (1) queries: norm and rotation in fp32, one rounding to the type
        def turned(y, weight):
            y = plain.norm(y, weight.double()[:, None, None, :], eps) if normed else y
            return plain.rope(y, pos[:, None]), y.abs().amax(-1, keepdim=True)
        rq, big = turned(xf[:, rows, :Hq], qw)
        assert ((q_out[:, rows].cpu().double() - rq).abs() <= u * rq.abs() + 2.0 ** -20 * big).all()
        # (2) keys and values as read back; rows held before are untouched
        rk, big = turned(xf[:, rows, Hq:Hq + Hkv], kw)
        rk, big = rk.transpose(1, 2), big.transpose(1, 2)
        got_k, got_v = kr[:, b].cpu().double(), vr[:, b].cpu().double()
        assert torch.equal(got_k[:, :, :old[b]], t.keys[b][:, :, :old[b]].to(dtype).double())
        assert torch.equal(got_v[:, :, :old[b]], t.vals[b][:, :, :old[b]].to(dtype).double())
        assert (got_k[:, :, t.held[b]:] == 0).all() and (got_v[:, :, t.held[b]:] == 0).all()
        now_k, now_v = got_k[:, :, old[b]:t.held[b]], got_v[:, :, old[b]:t.held[b]]
        rv = x[:, rows, Hq + Hkv:].transpose(1, 2)
        if fmt == "plain":
            assert ((now_k - rk).abs() <= u * rk.abs() + 2.0 ** -20 * big).all()
            assert torch.equal(now_v, rv.double())
        else:
            codes, scale = plain.quantise(rv.float())
            assert torch.equal(now_v, (codes.double() * scale.double()[..., None]).to(dtype).double())
            # half a step of the code (of the subnormals at least), the scale's power of
            # two up to one step apart where amax sits on its border
            step = 2.0 ** -9 * torch.exp2(torch.ceil(torch.log2(rk.abs().amax(-1, keepdim=True) / 448)))
            assert ((now_k - rk).abs() <= (2.0 ** -4 + u) * rk.abs() + step + 2.0 ** -20 * big).all()
    # (3) nothing else was written
    touched = torch.zeros(cache.k.shape[1], cache.k.shape[3], dtype=torch.bool)
    for b in range(len(old)):
        for r in range(old[b], t.held[b]):
            touched[int(t.table[b, r // page]), r % page] = True
    for y, z in zip(before, cache):
        if y is None:
            continue
        y, z = y.cpu().view(torch.uint8), z.cpu().view(torch.uint8)
        y = y.view(*cache.k.shape[:4], -1).transpose(2, 3)[:, ~touched]
        z = z.view(*cache.k.shape[:4], -1).transpose(2, 3)[:, ~touched]
        assert torch.equal(y, z)


def test_eight_bit_rows_at_their_borders():
    """Zero rows, rows of one tiny or huge value, amax on and next to 1.75 * 2^k, ties of the
    code, and rows with an infinity or a NaN, as values (which are not rotated)."""
    D, up = 16, lambda x: torch.nextafter(torch.tensor(x), torch.tensor(math.inf)).item()
    tops = [0.0, 1e-45, 1e-38, 2.0 ** -100, 448 * 2.0 ** -100, 1.75, up(1.75), 448.0, up(448.0),
            1.0, 3e38, 3.4e38, math.inf, math.nan]
    x = torch.zeros((1, len(tops), 3, D), dtype=F32)
    for i, a in enumerate(tops):
        x[0, i, 2] = torch.linspace(-1, 1, D) * (a if math.isfinite(a) else 1.0)
        x[0, i, 2, 3] = a
        x[0, i, 2, 4] = -a * 0.75           # a tie between two codes where the scale is 2^k
    n = len(tops)
    cache = sa.paged_cache(1, 2, 1, 16, D, torch.float8_e4m3fn)
    table = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device=DEV)
    xd = x.to(DEV)
    sa.cache_append(xd[:, :, :1], xd[:, :, 1:2], xd[:, :, 2:], cache, table, i32([0, n]), i32([0]))
    _, got = sa.cache_read(cache, table, i32([n]), dtype=F32)
    codes, scale = plain.quantise(x[0, :, 2])
    assert torch.equal(torch.nan_to_num(cache.v_scale[0, 1, 0, :n].cpu(), nan=-1.0),
                       torch.nan_to_num(scale, nan=-1.0))
    want = codes * scale[:, None]
    got = got[0, 0, 0, :n].cpu()
    assert torch.isnan(got[-2:]).all()
    assert torch.equal(got[:-2], want[:-2])
    assert (cache.k[0, 0].float() == 0).all()       # the other page


def test_read_of_given_rows_leaves_the_rest():
    t = plain.Batch(2, 2, 64, 16, [33, 0, 5], [0, 0, 0], BF, "e4m3", seed=4)
    cache, table, _, _ = t.device(sa)
    k = torch.full((2, 3, 2, 20, 64), 7.0, dtype=F32, device=DEV)
    v = k.clone()
    sa.cache_read(cache, table, torch.tensor(t.held, dtype=torch.int32, device=DEV), k_out=k, v_out=v)
    for b, n in enumerate((20, 0, 5)):
        assert torch.equal(k[:, b, :, :n].cpu().double(), t.keys[b][:, :, :n])
        assert torch.equal(v[:, b, :, :n].cpu().double(), t.vals[b][:, :, :n])
        assert (k[:, b, :, n:] == 7.0).all() and (v[:, b, :, n:] == 7.0).all()


# ---- bad pages, empty calls -------------------------------------------------------
@pytest.mark.device_error_expected
@pytest.mark.parametrize("dtype,fmt", [(BF, "plain"), (BF, "e4m3"), (F32, "plain")])
def test_bad_pages_and_positions_are_reported_and_touch_nothing(dtype, fmt):
    assert sa.device_error() == 0
    t = plain.Batch(1, 2, 64, 16, [20, 20, 20], [4, 4, 4], dtype, fmt, seed=6)
    x = torch.randn((1, 12, 8, 64), generator=torch.Generator().manual_seed(0)).to(dtype).to(DEV)
    alpha = torch.ones(1, device=DEV)

    def both(table, cached):
        cache, _, cu, _ = t.device(sa)
        before = [y.clone() for y in cache if y is not None]
        q = sa.cache_append(x[:, :, :4], x[:, :, 4:6], x[:, :, 6:], cache, table, cu, cached)
        word_a = sa.device_error()
        n_same = [torch.equal(y.view(torch.uint8), z.view(torch.uint8))
                  for y, z in zip(before, (c for c in cache if c is not None))]
        o, lse = sa.chunk_attn(q, cache, table, cu, cached, alpha, window=12)
        word_c = sa.device_error()
        return q, o, lse, word_a, word_c, n_same
    good = t.table.to(DEV)
    cached = torch.tensor(t.old, dtype=torch.int32, device=DEV)
    for bad_page in (-1, t.n_pages, 1 << 30, -(1 << 31)):
        table = good.clone()
        table[1, 1] = bad_page                 # rows 16 .. 31 of sequence 1
        q, o, lse, wa, wc, _ = both(table, cached)
        assert wa == sa.ERR_PAGE and wc == sa.ERR_PAGE
        assert torch.isnan(o[:, 4:8]).all() and torch.isnan(lse[:, 4:8]).all()
        assert torch.isfinite(o[:, :4].float()).all() and torch.isfinite(o[:, 8:].float()).all()
        assert torch.isfinite(q.float()).all()
    for start in (-1, -5, t.width * 16 - 3, 1 << 30, (1 << 31) - 2):
        c = cached.clone()
        c[1] = start
        table = good.clone()
        table[1] = table[1, 0]                 # every page of sequence 1 exists
        q, o, lse, wa, wc, _ = both(table, c)
        assert wa == sa.ERR_PAGE and wc == sa.ERR_PAGE
        assert torch.isnan(o[:, 4:8]).any() and torch.isnan(q[:, 4:8].float()).any()
        assert torch.isfinite(o[:, :4].float()).all() and torch.isfinite(o[:, 8:].float()).all()
    # all sequences bad: the cache stays as it was
    *_, same = both(torch.full_like(good, -1), cached)
    assert all(same)
    table = good.clone()
    table[2, 0] = t.n_pages
    cache, _, _, _ = t.device(sa)
    k, v = sa.cache_read(cache, table, torch.tensor(t.held, dtype=torch.int32, device=DEV))
    assert sa.device_error() == sa.ERR_PAGE
    assert torch.isnan(k[:, 2, :, :16].float()).all() and torch.isfinite(k[:, 2, :, 16:].float()).all()
    assert torch.isfinite(k[:, :2].float()).all() and torch.isfinite(v[:, :2].float()).all()


def test_calls_without_work():
    cache = sa.paged_cache(2, 3, 2, 16, 64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    x = torch.empty((2, 0, 2, 64), dtype=BF, device=DEV)
    alpha = torch.ones(2, device=DEV)
    table = i32([[0, 1], [2, 0]])
    assert sa.cache_append(x, x, x, cache, table, i32([0, 0, 0]), i32([4, 0])).shape == x.shape
    o, lse = sa.chunk_attn(x, cache, table, i32([0, 0, 0]), i32([4, 0]), alpha, window=3)
    assert o.shape == x.shape and lse.shape == (2, 0, 2)
    none = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    y = torch.ones((2, 5, 2, 64), dtype=BF, device=DEV)         # padding only
    out = torch.full_like(y, 7.0)
    sa.chunk_attn(y, cache, none, i32([0]), i32([]), alpha, window=3, out=out)
    assert (out == 7.0).all()
    sa.cache_append(y, y, y, cache, none, i32([0]), i32([]), q_out=out)
    assert (out == 7.0).all() and (cache.k == 0).all()
    k, v = sa.cache_read(cache, none, i32([]))
    assert k.shape == (2, 0, 2, 32, 64)
    k, v = sa.cache_read(cache, table, i32([0, 0]), rows=0)
    assert k.shape == (2, 2, 2, 0, 64)


# ---- together ----------------------------------------------------------------------
@pytest.mark.parametrize("dtype,fmt,D", [(F32, "plain", 32), (BF, "plain", 64), (BF, "e4m3", 64)])
def test_chunks_over_the_cache_equal_the_forward_over_the_sequence(dtype, fmt, D):
    """Two sequences are prefilled in ragged chunks and then decoded token by token; every
    output equals the training forward's row on the normed queries and keys."""
    L, H, page, eps = 2, 2, 16, 1e-6
    lens, g = [150, 77], torch.Generator().manual_seed(5)
    alpha = torch.tensor([0.8, 1.0], device=DEV)
    xs = [torch.randn((L, n, 3 * H, D), generator=g).to(dtype).to(DEV) for n in lens]
    qw, kw = (1 + 0.1 * torch.randn((L, D), generator=g).to(DEV) for _ in range(2))
    kw_ = dict(window=12, sinks=2)
    want = []
    for x in xs:
        heads = x.permute(0, 2, 1, 3)[:, None]                 # [L, 1, 3 H, n, D]
        q, k = sa.qk_norm_rope(heads[:, :, :H], heads[:, :, H:2 * H], qw, kw, eps=eps, rotate=False)
        o, lse = sa.fwd(q, k, heads[:, :, 2 * H:].contiguous(), alpha, **kw_)
        want.append((o[:, 0].transpose(1, 2), lse[:, 0].transpose(1, 2)))
    width = 10
    cache = sa.paged_cache(L, 2 * width, H, page, D, torch.float8_e4m3fn if fmt == "e4m3" else dtype)
    table = torch.randperm(2 * width, generator=g).view(2, width).to(torch.int32).to(DEV)
    done = [0, 0]
    steps = [(64, 0), (1, 40), (17, 20)] + [(1, 1)] * 17 + [(51, 0)]
    worst = 0.0
    for step in steps:
        new = [min(s, n - d) for s, n, d in zip(step, lens, done)]
        x = torch.cat([y[:, d:d + s] for y, d, s in zip(xs, done, new)], 1)
        cu = torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device=DEV)
        cached = torch.tensor(done, dtype=torch.int32, device=DEV)
        q = sa.cache_append(x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:], cache, table, cu, cached,
                            q_weight=qw, k_weight=kw, eps=eps)
        o, lse = sa.chunk_attn(q, cache, table, cu, cached, alpha, **kw_)
        at = 0
        for b in range(2):
            ro, rl = (y[:, done[b]:done[b] + new[b]] for y in want[b])
            go, gl = o[:, at:at + new[b]], lse[:, at:at + new[b]]
            at += new[b]
            if fmt == "e4m3":      # 3-bit mantissas: relative in the 2-norm, 2^-4 per element
                worst = max(worst, *[((a.double() - r.double()).norm() / r.double().norm()).item()
                                     for a, r in ((go, ro),) if r.numel()] or [0.0])
            else:
                tol = 1e-5 if dtype == F32 else 2e-2
                assert (go.float() - ro.float()).abs().max().item() <= tol if new[b] else True
                assert (gl - rl).abs().max().item() <= tol if new[b] else True
            done[b] += new[b]
    assert done == lens
    # keys and values are each off by at most 2^-4 (on average a third of that): the output's
    # 2-norm by less than 2 * 2^-4 for scores of order one
    assert worst <= 2.0 ** -3


def test_decode_agrees_with_the_contiguous_cache():
    """One token of three sequences with common lengths: chunk_attn over pages and decode()
    over a contiguous cache (which rotates its raw keys itself)."""
    L, B, H, T, D, pos = 2, 3, 4, 100, 64, 99
    g = torch.Generator().manual_seed(8)
    k, v = (torch.randn((L, B, H, T, D), generator=g).to(DEV) for _ in range(2))
    q = torch.randn((L, B, H, D), generator=g).to(DEV)
    beta = torch.randn((L, B, H), generator=g).to(DEV)
    alpha = torch.tensor([0.7, 1.3], device=DEV)
    cache = sa.paged_cache(L, B * 8, H, 16, D, F32)
    table = torch.randperm(B * 8, generator=g).view(B, 8).to(torch.int32).to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    flat = lambda x: x.transpose(2, 3).reshape(L, B * T, H, D)
    sa.cache_append(flat(k), flat(k), flat(v), cache, table, i32([0, T, 2 * T, 3 * T]), i32([0, 0, 0]))
    qr = sa.cache_append(q, k[:, :, :, pos], v[:, :, :, pos], cache, table, i32([0, 1, 2, 3]),
                         i32([pos] * 3))
    o, lse = sa.chunk_attn(qr, cache, table, i32([0, 1, 2, 3]), i32([pos] * 3), alpha, window=12,
                           sinks=3, beta=beta)
    ro, rl = sa.decode(q, k, v, alpha, pos, window=12, sinks=3, beta=beta)
    assert (o - ro).abs().max().item() <= 1e-5 and (lse - rl).abs().max().item() <= 1e-5


def test_strides_and_streams_and_graphs():
    """A step captured once and replayed after its lengths, pages and rows changed; and the
    same step on a side stream."""
    L, H, D = 2, 4, 64
    t = plain.Batch(L, H, D, 16, [30, 0, 12], [3, 5, 0], BF, "e4m3", seed=9, tail=2)
    cache, table, cu, cached = t.device(sa)
    g = torch.Generator().manual_seed(2)
    alpha = torch.tensor([0.9, 1.0], device=DEV)
    xs = [torch.randn((L, t.N, 3 * H, D), generator=g).to(BF).to(DEV) for _ in range(2)]
    x = xs[0].clone()
    q = torch.zeros((L, t.N, H, D), dtype=BF, device=DEV)
    o, lse = torch.zeros_like(q), torch.zeros((L, t.N, H), device=DEV)

    def step(stream=None):
        sa.cache_append(x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:], cache, table, cu, cached,
                        q_out=q, stream=stream)
        sa.chunk_attn(q, cache, table, cu, cached, alpha, window=12, out=o, lse=lse, stream=stream)

    plans = [(xs[0], t.cu, t.old, t.table),
             (xs[1], [0, 1, 2, 8], [32, 4, 6], t.table[[1, 0, 2]])]

    def load(plan):
        x.copy_(plan[0])
        cu.copy_(torch.tensor(plan[1]))
        cached.copy_(torch.tensor(plan[2]))
        table.copy_(plan[3])
    plans[1][3][0] = t.table[0]      # sequence 0 keeps its pages, 1 and 2 take others that exist
    plans[1][3][1:, 1:] = plans[1][3][1:, :1]
    saved = [y.clone() for y in cache]

    def fresh():
        for y, z in zip(cache, saved):
            y.copy_(z)
        for y in (q, o, lse):
            y.zero_()
    eager = []
    side = torch.cuda.Stream()
    for plan in plans:
        fresh()
        load(plan)
        side.wait_stream(torch.cuda.current_stream())
        step(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        eager.append([y.clone() for y in (q, o, lse, *cache)])
    fresh()
    load(plans[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for plan, want in zip(plans, eager):
        fresh()
        load(plan)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((q, o, lse, *cache), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_a_long_cache_past_32_bit_offsets():
    """A pool of more than 2^31 elements per tensor: rows at its far end."""
    L, P, H, page, D = 1, 70000, 8, 64, 64          # 2.3e9 elements of one byte
    assert P * H * page * D > 1 << 31
    cache = sa.PagedCache(*(torch.zeros((L, P, H, page, D), dtype=torch.float8_e4m3fn, device=DEV)
                            for _ in range(2)),
                          *(torch.ones((L, P, H, page), device=DEV) for _ in range(2)))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    table = i32([[P - 1, P - 2]])
    g = torch.Generator().manual_seed(3)
    x = torch.randn((L, 70, 3 * H, D), generator=g).to(BF).to(DEV)
    q = sa.cache_append(x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:], cache, table, i32([0, 70]),
                        i32([0]))
    o, lse = sa.chunk_attn(q, cache, table, i32([0, 70]), i32([0]), torch.ones(1, device=DEV),
                           window=12)
    k, v = sa.cache_read(cache, table, i32([70]))
    small = sa.paged_cache(L, 2, H, page, D, torch.float8_e4m3fn)
    t2 = i32([[1, 0]])
    q2 = sa.cache_append(x[:, :, :H], x[:, :, H:2 * H], x[:, :, 2 * H:], small, t2, i32([0, 70]),
                         i32([0]))
    o2, lse2 = sa.chunk_attn(q2, small, t2, i32([0, 70]), i32([0]), torch.ones(1, device=DEV),
                             window=12)
    k2, v2 = sa.cache_read(small, t2, i32([70]))
    for a, b in ((q, q2), (o, o2), (lse, lse2), (k, k2), (v, v2)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("W,S,offs", [(12, 0, FIB), (64, 4, FIB), (200, 16, (3, 77)), (500, 0, ()),
                                      (1, 0, (1,)), (20, 1, MANY)])
@pytest.mark.parametrize("dtype,fmt,D,Hq,Hkv,B", [
    (BF, "plain", 64, 2, 2, 3), (BF, "e4m3", 128, 8, 2, 2), (BF, "plain", 16, 1, 1, 1),
    (BF, "e4m3", 16, 20, 2, 2), (BF, "plain", 128, 3, 1, 40), (F32, "plain", 64, 2, 1, 2)])
def test_single_tokens(dtype, fmt, D, Hq, Hkv, B, W, S, offs):
    """Decode steps: the smallest calls, whose blocks are shared by several warps, and one of
    more blocks than that."""
    alpha = [1.0, 0.9]
    old = [(37 * b * b + 450 * (b % 2)) % 701 for b in range(B)]
    t = plain.Batch(2, Hkv, D, 16, old, [1] * B, dtype, fmt, seed=W + S)
    g = torch.Generator().manual_seed(1)
    q = torch.randn((2, t.N, Hq, D), generator=g).to(dtype)
    beta = torch.randn((2, t.N, Hq), generator=g)
    out, lse = _run_chunk(t, q.to(DEV), alpha, window=W, sinks=S, offsets=offs, beta=beta)
    ref = plain.chunk(q.double(), t.keys, t.vals, t.cu, t.old, alpha, W, S, offs, beta=beta.double())
    _check_chunk(t, q, out, lse, ref, dtype, min(W, max(t.held)) + S + 2 * len(offs))


def test_many_sequences_and_shared_pages():
    """1100 sequences with none to two new tokens; all of them read one sequence's first two pages
    as their own (a shared prompt), the rest lies in a page of their own."""
    B, page, D = 1100, 16, 32
    new = [(b * 7) % 3 for b in range(B)]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    g = torch.Generator().manual_seed(0)
    kp, vp = (torch.randn((1, B + 2, 1, page, D), generator=g).to(BF) for _ in range(2))
    table = torch.stack([torch.full((B,), B), torch.full((B,), B + 1), torch.randperm(B, generator=g)],
                        1).to(torch.int32)
    old = [32 + b % 13 for b in range(B)]
    q = torch.randn((1, cu[-1], 2, D), generator=g).to(BF)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    alpha = [0.75]
    o, lse = sa.chunk_attn(q.to(DEV), sa.PagedCache(kp.to(DEV), vp.to(DEV)), table.to(DEV), i32(cu),
                           i32(old), torch.tensor(alpha, device=DEV), window=10, sinks=2)
    seqs = [[x[:, t.long()].transpose(1, 2).flatten(2, 3).double() for t in table] for x in (kp, vp)]
    ro, rl, mag, big = plain.chunk(q.double(), *seqs, cu, old, alpha, 10, 2, FIB)
    assert ((lse.cpu().double() - rl).abs() <= 2.0 ** -20 * (big + rl.abs() + 1)).all()
    tol = (2.0 ** -18 * (big[..., None] + 1) + 2.0 ** -19 + 2.0 ** -8) * mag + 2.0 ** -8 * ro.abs()
    assert ((o.cpu().double() - ro).abs() <= tol).all()
    # and without the sums
    o2, none = sa.chunk_attn(q.to(DEV), sa.PagedCache(kp.to(DEV), vp.to(DEV)), table.to(DEV), i32(cu),
                             i32(old), torch.tensor(alpha, device=DEV), window=10, sinks=2,
                             want_lse=False)
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("qscale", [1.0, 1e-12, 1e9])
def test_scales_and_queries_of_any_size(dtype, qscale):
    """8-bit rows with scales that no append writes: not powers of two, zero, negative, from 1e-30
    to 1e10 side by side; queries of any size against keys that keep the scores moderate."""
    t = plain.Batch(1, 1, 64, 16, [40, 0], [30, 9], dtype, "e4m3", seed=12)
    g = torch.Generator().manual_seed(4)
    vs = torch.randn(t.vs.shape, generator=g) * 10.0 ** torch.randint(-30, 11, t.vs.shape, generator=g)
    vs = torch.where(torch.rand(t.vs.shape, generator=g) < 0.1, torch.zeros(()), vs)
    ks = torch.rand(t.ks.shape, generator=g) * 0.02 / qscale
    t.ks, t.vs = ks, vs
    for b in range(2):
        for r in range(t.held[b]):
            at = (slice(None), int(t.table[b, r // 16]), slice(None), r % 16)
            t.keys[b][:, :, r] = t.k[at].double() * ks[at].double()[..., None]
            t.vals[b][:, :, r] = t.v[at].double() * vs[at].double()[..., None]
    q = (torch.randn((1, t.N, 1, 64), generator=g) * qscale).to(dtype)
    alpha = [1.3]
    out, lse = _run_chunk(t, q.to(DEV), alpha, window=12)
    ref = plain.chunk(q.double(), t.keys, t.vals, t.cu, t.old, alpha, 12, 0, FIB)
    _check_chunk(t, q, out, lse, ref, dtype, 27)


@pytest.mark.parametrize("dtype,fmt", [(BF, "plain"), (BF, "e4m3"), (F32, "plain")])
def test_a_query_of_nan_or_infinities_stays_alone(dtype, fmt):
    t = plain.Batch(1, 1, 64, 16, [30], [16], dtype, fmt, seed=13)
    q = torch.randn((1, 16, 2, 64), generator=torch.Generator().manual_seed(6)).to(dtype)
    good, _ = _run_chunk(t, q.to(DEV), [1.0], window=20)
    q2 = q.clone()
    q2[0, 3, 1, 5] = math.nan
    q2[0, 9, 0, 7] = math.inf
    out, lse = _run_chunk(t, q2.to(DEV), [1.0], window=20)
    spoiled = torch.zeros((16, 2), dtype=torch.bool)
    spoiled[3, 1] = spoiled[9, 0] = True
    assert torch.isnan(out[0][spoiled].float()).all() and torch.isnan(lse[0][spoiled]).all()
    # (a block with such a query is computed query by query: both results are within 2^-8 (A + |O|)
    # of the exact one, for |O| <= A <= 3)
    assert ((out[0][~spoiled].float() - good[0][~spoiled].float()).abs() <= 0.05).all()
    assert torch.isfinite(lse[0][~spoiled]).all()


def test_calls_by_keyword_and_with_other_numbers():
    import numpy as np
    t = plain.Batch(1, 1, 32, 16, [5], [6], BF, "plain", seed=1)
    cache, table, cu, cached = t.device(sa)
    q = torch.randn((1, 6, 1, 32), generator=torch.Generator().manual_seed(0)).to(BF).to(DEV)
    alpha = torch.ones(1, device=DEV)
    a = sa.chunk_attn(q, cache, table, cu, cached, alpha, window=4, sinks=1)
    b = sa.chunk_attn(q=q, cache=cache, page_table=table, cu_q=cu, cached=cached, alpha=alpha,
                      window=np.int64(4), sinks=np.int32(1), offsets=np.array(FIB), scale=np.float32(0))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # windows past 32 bits are windows past every row; other numbers there are refused
    wide = sa.chunk_attn(q, cache, table, cu, cached, alpha, window=100)
    for window in (1 << 31, 1 << 32, (1 << 32) + 3):
        x = sa.chunk_attn(q, cache, table, cu, cached, alpha, window=window)
        assert torch.equal(x[0], wide[0]) and torch.equal(x[1], wide[1])
    for kw in (dict(window=-(1 << 32) + 4), dict(window=4, sinks=-(1 << 32)),
               dict(window=4, sinks=1 << 32)):
        with pytest.raises(sa.SparseAttnError):
            sa.chunk_attn(q, cache, table, cu, cached, alpha, **kw)
    for offset in ((1 << 32) + 3, -(1 << 32) + 3):
        with pytest.raises(ValueError):
            sa.chunk_attn(q, cache, table, cu, cached, alpha, window=4, offsets=(2, offset))
    k, v = sa.cache_read(cache=cache, page_table=table,
                         lengths=torch.tensor([11], dtype=torch.int32, device=DEV))
    assert torch.equal(k, sa.cache_read(cache, table, cached + 6)[0]) and bool(k[..., :11, :].any())
    with pytest.raises(TypeError):
        sa.chunk_attn(cache=cache)
    with pytest.raises(TypeError):
        sa.chunk_attn()


def test_tensors_without_storage_are_refused():
    from torch._subclasses.fake_tensor import FakeTensorMode
    real = sa.paged_cache(1, 2, 1, 16, 32)
    with FakeTensorMode(allow_non_fake_inputs=True):
        q = torch.empty((1, 2, 1, 5, 32), device=DEV)
        with pytest.raises(Exception):
            sa.qk_norm_rope(q, q, None, None)
        x = torch.empty((1, 5, 1, 32), dtype=BF, device=DEV)
        i32 = lambda *n: torch.empty(n, dtype=torch.int32, device=DEV)
        with pytest.raises(Exception):
            sa.cache_append(x, x, x, real, i32(1, 2), i32(2), i32(1))
        with pytest.raises(Exception):
            sa.chunk_attn(x, real, i32(1, 2), i32(2), i32(1), torch.ones(1, device=DEV), window=3)
    assert sa.device_error() == 0
