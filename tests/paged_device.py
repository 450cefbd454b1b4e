"""The chunk attention's plain 64-bit form on the GPU, for batches that the form in
paged_plain.py, which goes query by query, would take too long for; and such batches.
Test infrastructure only."""
import math

import torch

DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def quantise(x):
    """fp32 rows -> (e4m3 codes, power-of-two scales: the smallest with |x| / scale <= 448)."""
    m, e = torch.frexp(x.abs().amax(-1))
    scale = torch.ldexp(torch.ones_like(m), torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-100))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


class Batch:
    """Random rows of sequences in a shuffled pool of pages: old[b] rows held before, new[b]
    new tokens. Slots that no sequence holds are NaN."""

    def __init__(self, L, Hkv, D, page, old, new, dtype, fmt, seed):
        self.old, self.new = list(old), list(new)
        self.held = [a + b for a, b in zip(old, new)]
        self.L, self.Hkv, self.D, self.page, self.dtype, self.fmt = L, Hkv, D, page, dtype, fmt
        B, self.width = len(old), max(1, -(-max(self.held) // page))
        g = torch.Generator().manual_seed(seed)
        n_pages = B * self.width + 1
        self.table = torch.randperm(n_pages, generator=g)[:B * self.width].view(B, -1)
        self.cu = [sum(new[:b]) for b in range(B + 1)]
        self.N = self.cu[-1]
        held = torch.zeros((n_pages, page), dtype=torch.bool)
        for b, n in enumerate(self.held):
            r = torch.arange(n)
            held[self.table[b, r // page], r % page] = True
        held = held.to(DEV)
        gd = torch.Generator(device=DEV).manual_seed(seed)
        shape = (L, n_pages, Hkv, page, D)
        pools, self.values = [], []
        for _ in range(2):
            x = torch.randn(shape, generator=gd, device=DEV).to(dtype).float()
            x = torch.where(held[None, :, None, :, None], x, math.nan)
            if fmt == "e4m3":
                codes, scale = quantise(x)
                scale = torch.where(held[None, :, None], scale, math.nan)
                pools.append((codes, scale))
                self.values.append(codes.double() * scale.double()[..., None])
            else:
                pools.append((x.to(dtype), None))
                self.values.append(x.to(dtype).double())
        self.pools = pools

    def call(self, sa):
        """(cache, page_table, cu_q, cached)"""
        (k, ks), (v, vs) = self.pools
        return sa.PagedCache(k, v, ks, vs), i32(self.table.tolist()), i32(self.cu), i32(self.old)

    def queries(self, Hq, seed=1):
        g = torch.Generator(device=DEV).manual_seed(seed)
        return torch.randn((self.L, self.N, Hq, self.D), generator=g, device=DEV).to(self.dtype)

    def is_shared(self, Hq, W, S):
        """How many CTAs' warps share a block of 16-bit queries in launch_chunk_attn (0: a warp has
        a block and its whole window for itself)."""
        G = Hq // self.Hkv
        groups = -(-G // 8)
        per = -(-G // groups)
        shift = {1: 3, 2: 2, 3: 1, 4: 1}.get(per, 0)
        blocks = (self.N >> shift) + len(self.old) if shift else self.N
        warps = blocks * self.Hkv * groups * self.L
        tiles = -(-(min(W, self.width * self.page) + (1 << shift) - 1) // 16) + (S > 0)
        room = 148 * (3 if self.D == 128 and self.fmt == "plain" else 4)
        team = 1 if tiles >= 3 and warps <= room else 0
        while 0 < team < 8 and -(-tiles // 2) > 4 * (4 * team - 1) and warps * team * 2 <= room:
            team *= 2
        return team


def members(pos, W, S, offsets, alpha):
    """Rows a and b [n, M], their weights, whether an offset, whether there, of queries at pos [n]."""
    f = torch.tensor(offsets, dtype=torch.float32)
    d = (torch.tensor(alpha, dtype=torch.float32) * f).double().to(DEV)
    lo, up, w = d.floor().long(), d.ceil().long(), d - d.floor()
    p = pos[:, None]
    near = p - torch.arange(W, device=DEV)
    lead = torch.arange(S, device=DEV).expand(len(pos), S)
    far = p - lo
    ra = torch.cat([near, lead, far], 1)
    rb = torch.cat([near, lead, far - (w > 0).long()], 1)
    there = torch.cat([near >= 0, lead <= p, p - up >= 0], 1)
    wb = torch.cat([torch.zeros(W + S, dtype=torch.float64, device=DEV), w])
    off = torch.arange(W + S + len(offsets), device=DEV) >= W + S
    return ra, rb, wb, off, there


def chunk(t, q, alpha, W, S, offsets, beta=None, pick=None):
    """(o, lse, A, Q, M, top) of the picked token rows (all by default): o [L, n, Hq, D]; with
    normalised weights p, A = sum p ((1 - w) |row a| + w |row b|), Q = max over members of sum
    |q k| scale, M = rows that are summed, top = max over members of p times the largest |value|
    of its rows."""
    pick = torch.arange(t.N, device=DEV) if pick is None else pick
    L, Hq, D, G = t.L, q.shape[2], t.D, q.shape[2] // t.Hkv
    cu, old, table = (torch.tensor(x, device=DEV) for x in (t.cu, t.old, t.table.tolist()))
    W = min(W, max(t.held))
    outs = []
    step = max(1, (1 << 25) // ((W + S + len(offsets)) * Hq * D))
    for part in pick.split(step):
        b = (part[:, None] >= cu[None, 1:]).sum(1)
        pos = old[b] + part - cu[b]
        layers = []
        for l in range(L):
            ra, rb, wb, off, there = members(pos, W, S, offsets, alpha[l])

            def rows(x, r):
                r = torch.where(there, r, pos[:, None])
                page = table[b[:, None], r // t.page]
                return x[l][page, :, r % t.page].permute(0, 2, 1, 3).repeat_interleave(G, 1)  # [n, Hq, M, D]
            w = wb[None, None, :, None]
            K, V = ((1 - w) * rows(x, ra) + w * rows(x, rb) for x in t.values)
            va, vb = rows(t.values[1].abs(), ra), rows(t.values[1].abs(), rb)
            terms = q[l, part].double()[:, :, None] * K / math.sqrt(D)
            s, size = terms.sum(-1), terms.abs().sum(-1)
            if beta is not None:
                s = s + off * beta[l, part].double()[:, :, None]
            s = s.masked_fill(~there[:, None], -math.inf)
            lse = torch.logsumexp(s, -1)
            p = torch.exp(s - lse[..., None])
            o = (p[..., None] * V).sum(2)
            mag = (p[..., None] * ((1 - w) * va + w * vb)).sum(2)
            top = (p * torch.maximum(va, vb).amax(-1)).amax(-1)
            layers.append((o, lse, mag, size.masked_fill(~there[:, None], 0).amax(-1), top))
        outs.append([torch.stack(x) for x in zip(*layers)])
    o, lse, mag, big, top = (torch.cat(x, 1) for x in zip(*outs))
    return o, lse, mag, big, W + S + 2 * len(offsets), top


def beyond(t, out, lse, ref):
    """How far O and LSE are beyond their bounds (0 or less: within). fp32 sums of D products,
    exponentials and logarithms: LSE 2^-20 (Q + |LSE| + 1) + 2^-24 M, O (2^-18 (Q + 1) + 2^-24 M) A,
    and half a step of the output, 2^-8 |O| for bf16. 16-bit queries' probabilities go into the
    products as sums of two 16-bit values: over bf16 rows two bf16, 2^-8 2^-8 A; over 8-bit rows two
    fp16, 2^-11 2^-11 A and half of their smallest step, 2^-25, of each of the M weights where
    the largest is 1, times codes of up to 448: with value = code * scale and 448 scale < 2 max |value|
    2^-24 M top."""
    o, l, mag, big, M, top = ref
    tol = (2.0 ** -18 * (big[..., None] + 1) + 2.0 ** -24 * M) * mag
    if t.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * o.abs()
        if t.fmt == "plain":
            tol = tol + 2.0 ** -16 * mag
        else:
            tol = tol + 2.0 ** -22 * mag + 2.0 ** -24 * M * top[..., None]
    else:
        tol = tol + 2.0 ** -24 * o.abs()
    bad = ((out.double() - o).abs() - tol).amax().item()
    return bad, ((lse.double() - l).abs() - 2.0 ** -20 * (big + l.abs() + 1) - 2.0 ** -24 * M).amax().item()


def rope(x, pos, base=10000.0, sign=1.0):
    """x [..., D] in 64 bits, rotated at positions pos (broadcast against x's leading shape)."""
    D = x.shape[-1]
    theta = base ** (-2.0 * torch.arange(D // 2, dtype=torch.float64, device=DEV) / D)
    a = sign * pos.double()[..., None] * theta
    x1, x2 = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([x1 * a.cos() - x2 * a.sin(), x2 * a.cos() + x1 * a.sin()], -1)


def norm(x, w, eps):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
