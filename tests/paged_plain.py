"""Plain 64-bit forms of the query/key norm, the paged cache and the chunk
attention, from their definitions (include/sparse_attn.h), on the CPU: one row,
one query, one member at a time where that is the plainest.  Test infrastructure
only."""
import math

import torch


def rope(x, pos, base=10000.0, sign=1.0):
    """x [..., D] rotated at positions pos (broadcast against x's leading shape)."""
    D = x.shape[-1]
    theta = base ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)
    a = sign * torch.as_tensor(pos, dtype=torch.float64)[..., None] * theta
    x1, x2 = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()], -1)


def norm(x, w, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def norm_rope(x, w, eps, rotate, pos0=0, base=10000.0):
    """x [L, B, H, T, D] fp64; w [L, D] or None."""
    y = x if w is None else norm(x, w[:, None, None, None, :], eps)
    return rope(y, pos0 + torch.arange(x.shape[3]), base) if rotate else y


def norm_rope_bwd(x, w, eps, rotate, dy, pos0=0, base=10000.0):
    """(dx, dw, sum of |terms| of dw) by the formulas."""
    g = rope(dy, pos0 + torch.arange(x.shape[3]), base, -1.0) if rotate else dy
    if w is None:
        return g, None, None
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, gw = x * r, g * w[:, None, None, None, :]
    dx = r * (gw - n * (gw * n).mean(-1, keepdim=True))
    return dx, (g * n).sum((1, 2, 3)), (g * n).abs().sum((1, 2, 3))


def quantise(x):
    """fp32 rows [..., D] -> (e4m3 values as fp32 before the scale, scale), exact arithmetic."""
    x = x.double()
    top = x.abs().amax(-1)
    scale = torch.empty_like(top)
    flat, out = top.reshape(-1), scale.view(-1)
    for i, t in enumerate(flat.tolist()):
        if not math.isfinite(t):
            out[i] = math.nan
            continue
        e = -100
        if t > 0:
            m, ex = math.frexp(t / 448.0)           # t / 448 = m 2^ex, m in [0.5, 1)
            e = max(-100, ex - 1 if m == 0.5 else ex)
        out[i] = 2.0 ** e
    y = x / scale[..., None]
    a = y.abs().clamp(min=2.0 ** -30)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6.0) - 3)
    return (torch.round(y / step) * step).float(), scale.float()


def geometry(alpha, f):
    d = float(torch.tensor(alpha, dtype=torch.float32) * torch.tensor(float(f), dtype=torch.float32))
    lo = math.floor(d)
    return lo, math.ceil(d), d - lo


def members(pos, W, S, offsets, alpha):
    """[(row a, weight a, row b or None, weight b, is offset)] of the query at pos."""
    out = [(pos - t, 1.0, None, 0.0, False) for t in range(min(W, pos + 1))]
    out += [(j, 1.0, None, 0.0, False) for j in range(S) if j <= pos]
    for f in offsets:
        lo, up, w = geometry(alpha, f)
        if pos - up >= 0:
            out.append((pos - lo, 1.0 - w, pos - lo - 1 if w else None, w, True))
    return out


def chunk(q, keys, vals, cu, cached, alpha, W, S, offsets, scale=None, beta=None):
    """q [L, N, Hq, D] fp64; keys, vals: per sequence [L, Hkv, rows, D] fp64.
    Returns (o, lse, sum p |v|, max over members of sum |q k| scale), rows of no
    sequence NaN; |v| of an interpolated member is (1 - w) |row a| + w |row b|."""
    L, N, Hq, D = q.shape
    Hkv = keys[0].shape[1] if keys else 1
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(D) if not scale or scale <= 0 else scale
    o = torch.full((L, N, Hq, D), math.nan, dtype=torch.float64)
    mag = torch.full((L, N, Hq, D), math.nan, dtype=torch.float64)
    lse = torch.full((L, N, Hq), math.nan, dtype=torch.float64)
    big = torch.zeros((L, N, Hq), dtype=torch.float64)
    for b in range(len(cached)):
        for n in range(cu[b], cu[b + 1]):
            pos = cached[b] + n - cu[b]
            for l in range(L):
                ms = members(pos, W, S, offsets, alpha[l])
                ra = torch.tensor([m[0] for m in ms])
                wa = torch.tensor([m[1] for m in ms], dtype=torch.float64)[None, :, None]
                rb = torch.tensor([m[0] if m[2] is None else m[2] for m in ms])
                wb = torch.tensor([m[3] for m in ms], dtype=torch.float64)[None, :, None]
                off = torch.tensor([m[4] for m in ms])

                def rows(x):
                    two = torch.where(wb > 0, wa * x[l][:, ra] + wb * x[l][:, rb], x[l][:, ra])
                    return two.repeat_interleave(G, 0)          # [Hq, M, D]
                K, V = rows(keys[b]), rows(vals[b])
                size = rows(vals[b].abs())
                s = (q[l, n][:, None, :] * K).sum(-1) * scale
                big[l, n] = (q[l, n][:, None, :] * K).abs().sum(-1).amax(-1) * scale
                if beta is not None:
                    s = s + off[None, :] * beta[l, n][:, None]
                lse[l, n] = torch.logsumexp(s, -1)
                p = torch.exp(s - lse[l, n][:, None])
                o[l, n] = (p[..., None] * V).sum(1)
                mag[l, n] = (p[..., None] * size).sum(1)
    return o, lse, mag, big


class Batch:
    """Sequences with random lengths' worth of rows, spread over a shuffled pool of
    pages.  Slots that no sequence holds are NaN; table entries behind a sequence's
    last page name no page."""

    def __init__(self, L, Hkv, D, page, old, new, dtype, fmt, seed, lead=0, tail=0, magnitude=1.0):
        g = torch.Generator().manual_seed(seed)
        self.L, self.Hkv, self.D, self.page, self.g = L, Hkv, D, page, g
        self.old, self.new = list(old), list(new)
        B = len(old)
        self.held = [a + b for a, b in zip(old, new)]
        self.width = max(1, max([-(-h // page) for h in self.held] or [1])) + 1
        need = [-(-h // page) for h in self.held]
        self.n_pages = sum(need) + 2
        order = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = torch.full((B, self.width), -7, dtype=torch.int32)
        at = 0
        for b in range(B):
            for i in range(need[b]):
                self.table[b, i] = order[at]
                at += 1
        cu = [lead]
        for n in new:
            cu.append(cu[-1] + n)
        self.cu, self.N = cu, cu[-1] + tail
        self.dtype, self.fmt = dtype, fmt
        shape = (L, self.n_pages, Hkv, page, D)
        self.rows = [torch.randn((L, h, Hkv, D), generator=g) * magnitude for h in self.held], \
                    [torch.randn((L, h, Hkv, D), generator=g) for h in self.held]
        self.k, self.v = (torch.full(shape, math.nan) for _ in range(2))
        self.ks, self.vs = (torch.full(shape[:4], math.nan) for _ in range(2))
        self.keys, self.vals = [], []
        for xs, pool, sc, held in ((self.rows[0], self.k, self.ks, self.keys),
                                   (self.rows[1], self.v, self.vs, self.vals)):
            for b, x in enumerate(xs):
                x = x.to(dtype).float()
                s = torch.ones(x.shape[:3])
                if fmt == "e4m3":
                    x, s = quantise(x)
                for r in range(self.held[b]):
                    p = int(self.table[b, r // page])
                    pool[:, p, :, r % page] = x[:, r]
                    sc[:, p, :, r % page] = s[:, r]
                held.append((x.double() * s.double()[..., None]).transpose(1, 2).contiguous())

    def device(self, sa, dev="cuda"):
        """(cache, table, cu, cached) on the device."""
        if self.fmt == "e4m3":
            cache = sa.PagedCache(self.k.to(torch.float8_e4m3fn).to(dev),
                                  self.v.to(torch.float8_e4m3fn).to(dev),
                                  self.ks.to(dev), self.vs.to(dev))
        else:
            cache = sa.PagedCache(self.k.to(self.dtype).to(dev), self.v.to(self.dtype).to(dev))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
        return cache, self.table.to(dev), i32(self.cu), i32(self.old)
