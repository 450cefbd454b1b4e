"""Norms and appends of many rows: the passes of a warp over a token's heads, and the walks of a
thread over the rows of its tiles, on batches that need several of each. Against 64-bit plain
forms on the GPU.

Tolerances per element: half a step of the type, u = torch.finfo(dtype).eps / 2, of the result,
plus 2^-20 of the row's largest term for fp32 arithmetic; weight gradients (rows + 24) 2^-24 of
the sum of their terms' sizes: fp32 sums of a thread's rows (at most 40 here), then over 5 lanes' and
8 warps' steps, with a few roundings in each term; the rest is summed in 64 bits."""
import pytest
import torch

import paged_device as dev
import structured_sparse_attention_fibonacci_b200 as sa

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu


def _ceil(a, b):
    return -(-a // b)


# (id, dtype, L, B, Hq, Hkv, T, D, packed, heads that a lane group walks at least, rows of a thread
# of the backward at least): the last tile is partial, the heads no multiple of the walk
NORM = [
    ("bf16_d64", BF, 6, 3, 8, 3, 6667, 64, True, 8, 16),
    ("bf16_d64_long", BF, 1, 1, 7, 4, 50001, 64, False, 8, 16),
    ("bf16_d128", BF, 2, 2, 9, 2, 5001, 128, False, 8, 16),
    ("bf16_d32", BF, 3, 2, 13, 4, 4999, 32, True, 4, 8),
    ("bf16_d16", BF, 4, 2, 21, 4, 4999, 16, False, 2, 6),
    ("f32_d64", F32, 3, 3, 8, 3, 7001, 64, True, 8, 16),
    ("f32_d128", F32, 1, 2, 9, 3, 10001, 128, False, 8, 16),
    ("f32_d16", F32, 4, 3, 9, 4, 6001, 16, True, 2, 8),
]


@pytest.mark.parametrize("mode", ["norm_rope", "norm", "rope"])
@pytest.mark.parametrize("case", NORM, ids=[c[0] for c in NORM])
def test_norm_of_many_rows_and_its_gradients(case, mode):
    name, dtype, L, B, Hq, Hkv, T, D, packed, heads, rows = case
    per, tokens, H = 256 // (D // 16), B * T, Hq + Hkv
    tiles = _ceil(tokens, per)
    assert tokens % per
    walk = 8                                   # fwd_t's choice
    while walk > 1 and tiles * L * _ceil(H, walk) < 148 * 8:
        walk //= 2
    waves = min(4, max(1, tiles * H * L // (296 * 16)))      # bwd_grid's
    want = max(2, _ceil(296 * waves, L))
    most = max(_ceil(tiles * Hq, max(1, want * Hq // H)), _ceil(tiles * Hkv, max(1, want - want * Hq // H)))
    assert walk >= heads and H % walk and rows <= most <= 40, (walk, most)
    g = torch.Generator(device=DEV).manual_seed(len(name))

    def pair(packed):
        if packed:
            x = torch.randn((L, B, T, H, D), generator=g, device=DEV).to(dtype).permute(0, 1, 3, 2, 4)
            return x[:, :, :Hq], x[:, :, Hq:]
        return tuple(torch.randn((L, B, h, T, D), generator=g, device=DEV).to(dtype) for h in (Hq, Hkv))
    (q, k), (dqo, dko) = pair(packed), pair(not packed)
    qw, kw = (1 + 0.3 * torch.randn((L, D), generator=g, device=DEV) for _ in range(2))
    if mode == "rope":
        qw = kw = None
    rotate, eps, u, pos0 = mode != "norm", 1e-5, torch.finfo(dtype).eps / 2, 11
    args = dict(eps=eps, rotate=rotate, pos0=pos0)
    ys = sa.qk_norm_rope(q, k, qw, kw, **args)
    grads = sa.qk_norm_rope_bwd(q, k, qw, kw, dqo, dko, **args)
    again = sa.qk_norm_rope_bwd(q, k, qw, kw, dqo, dko, **args)
    assert all(a is None or torch.equal(a, b) for a, b in zip(grads, again))
    pos = pos0 + torch.arange(T, device=DEV)
    for x_, w_, dy_, y_, dx_, dw_ in ((q, qw, dqo, ys[0], grads[0], grads[2]),
                                      (k, kw, dko, ys[1], grads[1], grads[3])):
        for l in range(L):      # a layer at a time: 64-bit copies are large
            x, dy, w = x_[l].double(), dy_[l].double(), None if w_ is None else w_[l].double()
            n = x if w is None else dev.norm(x, w, eps)
            ref = dev.rope(n, pos) if rotate else n
            tol = u * ref.abs() + 2.0 ** -20 * n.abs().amax(-1, keepdim=True)
            assert ((y_[l].double() - ref).abs() <= tol).all()
            gr = dev.rope(dy, pos, sign=-1.0) if rotate else dy
            big = dy.abs().amax(-1, keepdim=True)
            if w is None:
                rdx = gr
                assert dw_ is None
            else:
                r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
                m, gw = x * r, gr * w
                rdx = r * (gw - m * (gw * m).mean(-1, keepdim=True))
                big = big * r * w.abs().amax() * (1 + m.abs().amax(-1, keepdim=True) ** 2)
                terms = (gr * m).abs().sum((0, 1, 2))
                assert ((dw_[l].double() - (gr * m).sum((0, 1, 2))).abs() <= (most + 24) * 2.0 ** -24 * terms).all()
            assert ((dx_[l].double() - rdx).abs() <= u * rdx.abs() + 2.0 ** -20 * big).all()


# (id, dtype, format, L, Hq, Hkv, D, old, new, warps of a token, passes of a warp at least)
APPEND = [
    ("bf16_32x128", BF, "plain", 2, 32, 8, 128, [40, 0], [1000, 300], 1, 12),
    ("bf16_e4m3_32x128", BF, "e4m3", 2, 32, 8, 128, [0, 7], [1200, 100], 1, 12),
    ("f32_32x128", F32, "plain", 1, 32, 8, 128, [5], [2400], 1, 12),
    ("f32_e4m3_32x128", F32, "e4m3", 2, 32, 8, 128, [0], [1200], 1, 12),
    ("bf16_8x64", BF, "plain", 2, 8, 8, 64, [0, 3], [1250, 17], 1, 3),
    ("bf16_e4m3_8x64", BF, "e4m3", 2, 8, 8, 64, [0, 3], [1250, 17], 1, 3),
    ("bf16_odd", BF, "e4m3", 1, 5, 5, 128, [9], [2401], 1, 4),
    ("bf16_d16", BF, "plain", 1, 40, 8, 16, [9], [2401], 1, 2),
    ("f32_d32", F32, "e4m3", 1, 21, 7, 32, [0], [2500], 1, 3),
    ("bf16_four_warps", BF, "e4m3", 2, 32, 8, 128, [0, 5], [300, 100], 4, 3),
    ("bf16_d64_two_warps", BF, "plain", 1, 30, 10, 64, [0], [1500], 2, 4),
]


@pytest.mark.parametrize("normed", [False, True], ids=["", "norm"])
@pytest.mark.parametrize("case", APPEND, ids=[c[0] for c in APPEND])
def test_appends_of_several_passes(case, normed):
    name, dtype, fmt, L, Hq, Hkv, D, old, new, warps, passes = case
    t = dev.Batch(L, Hkv, D, 16, old, new, dtype, fmt, seed=len(name))
    need = _ceil(Hq + 2 * Hkv, 512 // D)          # launch_cache_append's choice
    parts = 1
    while parts < need and t.N * L * parts < 148 * 16:
        parts *= 2
    assert min(parts, need) == warps and _ceil(need, warps) >= passes
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn((L, t.N, Hq + 2 * Hkv, D), generator=g, device=DEV).to(dtype)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    qw, kw = (1 + 0.3 * torch.randn((L, D), generator=g, device=DEV) for _ in range(2))
    cache, table, cu, cached = t.call(sa)
    before = [None if y is None else y.clone() for y in cache]
    eps, u = 1e-5, torch.finfo(dtype).eps / 2
    qo = sa.cache_append(q, k, v, cache, table, cu, cached, eps=eps,
                         **(dict(q_weight=qw, k_weight=kw) if normed else {}))
    b = torch.cat([torch.full((n,), i) for i, n in enumerate(new)]).to(DEV)
    pos = torch.cat([o + torch.arange(n) for o, n in zip(old, new)]).to(DEV)
    page, slot = t.table.to(DEV)[b, pos // 16], pos % 16

    def turned(y, w):
        y = y.double()
        y = dev.norm(y, w.double()[:, None, None, :], eps) if normed else y
        return dev.rope(y, pos[:, None]), y.abs().amax(-1, keepdim=True)
    ref, big = turned(q, qw)
    assert ((qo.double() - ref).abs() <= u * ref.abs() + 2.0 ** -20 * big).all()
    # rows of the pages: [L, N, Hkv, D]
    def held(pool, scale):
        y = pool[:, page, :, slot].transpose(0, 1).double()
        return y if scale is None else y * scale[:, page, :, slot].transpose(0, 1).double()[..., None]
    ref, big = turned(k, kw)
    got = held(cache.k, cache.k_scale)
    if fmt == "plain":
        assert ((got - ref).abs() <= u * ref.abs() + 2.0 ** -20 * big).all()
        assert torch.equal(held(cache.v, None), v.double())
    else:
        step = 2.0 ** -9 * torch.exp2(torch.ceil(torch.log2(ref.abs().amax(-1, keepdim=True) / 448)))
        assert ((got - ref).abs() <= 2.0 ** -4 * ref.abs() + step + 2.0 ** -20 * big).all()
        codes, scale = dev.quantise(v.float())
        assert torch.equal(held(cache.v, cache.v_scale), codes.double() * scale.double()[..., None])
    touched = torch.zeros(cache.k.shape[1], 16, dtype=torch.bool, device=DEV)
    touched[page, slot] = True
    for y, z in zip(before, cache):
        if y is not None:
            y, z = (a.view(torch.uint8).view(*cache.k.shape[:4], -1).transpose(2, 3)[:, ~touched] for a in (y, z))
            assert torch.equal(y, z)


def test_weight_gradients_of_a_long_batch_keep_their_bits():
    """9 million rows that are all the same, so that every rounding of a running fp32 sum falls the
    same way: n equal terms are off by up to n / 2 2^-24 of their sum. A thread may add 66 rows before
    the sums go on in 64 bits: 33, and 16 for the warp's, the CTA's and each term's own roundings."""
    T, Hq, Hkv, D = 2_280_011, 4, 1, 128
    g = torch.Generator(device=DEV).manual_seed(1)
    x, dy = (torch.randn(D, generator=g, device=DEV).to(BF) for _ in range(2))
    all_ = lambda r, h: r.expand(1, 1, h, T, D)
    w = torch.ones((1, D), device=DEV)
    _, _, dqw, dkw = sa.qk_norm_rope_bwd(all_(x, Hq), all_(x, Hkv), w, w, all_(dy, Hq), all_(dy, Hkv),
                                         eps=0.0, rotate=False)
    term = dy.double() * x.double() / torch.sqrt(x.double().square().mean())
    for got, h in ((dqw, Hq), (dkw, Hkv)):
        want = term * (T * h)
        assert ((got[0].double() - want).abs() <= 49 * 2.0 ** -24 * want.abs()).all()
