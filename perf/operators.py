"""Cases that measure the query/key norm, the paged cache and the chunk attention.

Six kinds of case, one per way a program calls the operators:
  norm      norms of queries and keys per head, with or without the position rotation
  norm_bwd  its gradients: dq, dk and the two weights'
  append    new tokens' rotated queries, and their keys and values into the pages of a cache
  handover  the same into an 8-bit cache, which is then read back (what a prefill worker sends)
  read      the rows of every sequence of a paged cache, as contiguous tensors
  chunk     attention of the new tokens (one or many per sequence) over a paged cache
``run`` computes them in elementary torch operations, or, where ``own`` is
true, by the package's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
FIB15 = (1, 2, 3, 5, 8, 13, 21, 34, 55, 89, 144, 233, 377, 610, 987)
OFFSETS = {"fib": FIB15, "pi": (16,), "pow2": tuple(1 << i for i in range(12))}
EPS = 1e-6
BASE = 10000.0


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # the 16-layer training batch (8 heads of 64), before a forward that rotates by itself
        dict(name="norm_train", kind="norm", L=16, B=8, hq=8, hkv=8, T=1024, D=64, dtype="bf16",
             rotate=False, packed=False),
        # the tiny fp32 configuration: latency
        dict(name="norm_tiny", kind="norm", L=1, B=1, hq=2, hkv=2, T=64, D=16, dtype="f32",
             rotate=True, packed=False),
        # the backward of the training batch
        dict(name="norm_bwd_train", kind="norm_bwd", L=16, B=8, hq=8, hkv=8, T=1024, D=64,
             dtype="bf16", rotate=False, packed=False),
        # grouped heads of 128 as views of one projection, an odd length, rotated
        dict(name="norm_bwd_grouped", kind="norm_bwd", L=2, B=3, hq=12, hkv=4, T=777, D=128,
             dtype="bf16", rotate=True, packed=True),
        # one token of each of 8 sequences, all 16 layers: a decode step's cache write
        dict(name="append_decode", kind="append", L=16, B=8, hq=8, hkv=8, D=64, dtype="bf16",
             cache="same", page=64, old=1023, new=1, ragged=False, norm=False),
        # prefill of six prompts into an 8-bit cache, read back for another worker
        dict(name="handover_prefill", kind="handover", L=4, B=6, hq=32, hkv=8, D=128, dtype="bf16",
             cache="e4m3", page=16, old=200, new=2048, ragged=True, norm=True),
        # four long sequences out of an 8-bit cache
        dict(name="read_long", kind="read", L=16, B=4, hq=8, hkv=8, D=64, dtype="bf16",
             cache="e4m3", page=64, old=8192, new=0, ragged=False, norm=False),
        # short ragged sequences, pages of an odd size
        dict(name="read_small", kind="read", L=1, B=3, hq=4, hkv=4, D=32, dtype="bf16",
             cache="same", page=7, old=100, new=0, ragged=True, norm=False),
        # one token of one sequence with a long window and sinks: latency
        dict(name="chunk_one", kind="chunk", L=1, B=1, hq=16, hkv=16, D=64, dtype="bf16",
             cache="e4m3", page=64, old=32767, new=1, ragged=False, W=64, S=4, offsets="fib",
             alpha="one", prior=False),
        # the 16-layer decode step at position 4095
        dict(name="chunk_decode", kind="chunk", L=16, B=8, hq=8, hkv=8, D=64, dtype="bf16",
             cache="same", page=64, old=4095, new=1, ragged=False, W=12, S=0, offsets="fib",
             alpha="stagger", prior=False),
        # the second half of a 32768-token prompt, long window and sinks
        dict(name="chunk_prefill", kind="chunk", L=1, B=1, hq=16, hkv=16, D=64, dtype="bf16",
             cache="same", page=64, old=16384, new=16384, ragged=False, W=64, S=4, offsets="fib",
             alpha="one", prior=False),
        # a mixed batch of grouped heads of 128 over an 8-bit cache, with the log-prior
        dict(name="chunk_mixed", kind="chunk", L=4, B=40, hq=32, hkv=8, D=128, dtype="bf16",
             cache="e4m3", page=16, old=3000, new=300, ragged=True, W=12, S=0, offsets="fib",
             alpha="stagger", prior=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {k: max(_cost(c) for c in listed() if c["kind"] == k)
            for k in ("norm", "norm_bwd", "append", "handover", "read", "chunk")}
    most["append"] = most["handover"]
    while True:
        kind = rng.choice(("norm", "norm_bwd", "append", "handover", "read", "chunk", "chunk"))
        dtype = rng.choice(("bf16", "bf16", "f32"))
        D = rng.choice((16, 32, 64, 64, 128))
        hkv = _log_int(rng, 1, 16)
        group = rng.choice((1, 1, 2, 3, 4, 6, 8, 12))
        c = dict(kind=kind, L=_log_int(rng, 1, 16), B=_log_int(rng, 1, 48), hq=hkv * group, hkv=hkv,
                 D=D, dtype=dtype)
        if kind in ("norm", "norm_bwd"):
            c.update(T=_log_int(rng, 1, 4096), rotate=rng.random() < 0.6,
                     packed=rng.random() < 0.5)
        else:
            c.update(cache=rng.choice(("same", "e4m3")), page=rng.choice((1, 7, 16, 32, 64, 128)),
                     old=_log_int(rng, 1, 8192) - 1,
                     new=rng.choice((1, _log_int(rng, 1, 4096))), ragged=rng.random() < 0.6)
            if kind == "append":
                c["cache"] = "same"
            if kind == "handover":      # an 8-bit key is returned as the 16-bit value it stands for
                c["cache"], c["dtype"] = "e4m3", "bf16"
            if kind == "read":
                c["new"] = 0
            if kind == "chunk":
                c.update(W=_log_int(rng, 1, 300), S=rng.choice((0, 0, 1, 4, 16)),
                         offsets=rng.choice(("fib", "fib", "pi", "pow2")),
                         alpha=rng.choice(("one", "stagger")), prior=rng.random() < 0.3)
            else:
                c["norm"] = rng.random() < 0.5
        if kind not in ("norm", "norm_bwd") and (c["L"] * c["B"] > 256 or sum(_new(c) + _old(c)) == 0):
            continue
        if kind not in ("norm", "norm_bwd", "read") and sum(_new(c)) == 0:
            continue
        pool = 0 if "page" not in c else c["L"] * c["B"] * _rows(c) * hkv * D
        if pool <= 1 << 28 and _cost(c) <= most[kind]:
            return c


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 50


def _share(i):
    """A fixed spread of shares of the longest length over the sequences; the third has none."""
    return (1.0, 0.37, 0.0, 0.71, 0.05, 0.53)[i % 6] * (1.0 if i < 6 else 0.5 + 0.5 / (1 + i % 7))


def _new(c):
    """New tokens of each sequence."""
    n = [int(c["new"] * _share(i)) if c["ragged"] else c["new"] for i in range(c["B"])]
    if c["ragged"] and c["new"] and c["B"] > 6:    # a mixed batch: most sequences decode
        n = [1 if i >= 6 and i % 5 else x for i, x in enumerate(n)]
    return n


def _old(c):
    """Rows that each sequence has in the cache before."""
    return [int(c["old"] * (1.0 - 0.9 * _share(i + 1))) if c["ragged"] else c["old"]
            for i in range(c["B"])]


def _rows(c):
    """Rows that a page table row covers."""
    longest = max(a + b for a, b in zip(_new(c), _old(c)))
    return max(1, -(-longest // c["page"])) * c["page"]


def _alpha(c):
    if c["alpha"] == "one":
        return [1.0] * c["L"]
    return [0.5 + l / (c["L"] - 1) for l in range(c["L"])] if c["L"] > 1 else [1.37]


def _geometry(c):
    """(lo, ceil, w) of every layer's offsets: the product is one fp32 rounding."""
    d = torch.tensor(_alpha(c), dtype=torch.float32)[:, None] * torch.tensor(
        OFFSETS[c["offsets"]], dtype=torch.float32)[None, :]
    return d.floor().long(), d.ceil().long(), d - d.floor()


def _attended_rows(c):
    """Rows that the chunk reads, each once: the union over each sequence's new tokens, all layers."""
    lo, hi, w = _geometry(c)
    total = 0
    for l in range(c["L"]):
        reach = [(0, c["W"] - 1)] + [(int(a), int(a) + (1 if x > 0 else 0))
                                     for a, x in zip(lo[l].tolist(), w[l].tolist())]
        for old, new in zip(_old(c), _new(c)):
            if not new:
                continue
            spans = sorted((max(0, old - far), old + new - 1 - near) for near, far in reach
                           if old + new - 1 - near >= 0)
            if c["S"]:
                spans = sorted(spans + [(0, min(c["S"], old + new) - 1)])
            end = -1
            for a, b in spans:
                total += max(0, b - max(a, end + 1) + 1)
                end = max(end, b)
    return total


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    heads, D, L = c["hq"] + c["hkv"], c["D"], c["L"]
    if c["kind"] in ("norm", "norm_bwd"):
        n = L * c["B"] * c["T"] * heads * D
        if c["kind"] == "norm":
            return {"bytes": 2 * n * e, "flops": 8 * n}
        return {"bytes": 3 * n * e, "flops": 16 * n}
    row = D * e if c["cache"] == "same" else D + 4     # bytes of a cache row
    N = sum(_new(c))
    held = sum(_new(c)) + sum(_old(c))
    put = L * N * ((2 * c["hq"] + 2 * c["hkv"]) * D * e + 2 * c["hkv"] * row)
    get = L * held * 2 * c["hkv"] * (row + D * e)
    if c["kind"] == "append":
        return {"bytes": put, "flops": 8 * L * N * heads * D}
    if c["kind"] == "handover":
        return {"bytes": put + get, "flops": 8 * L * N * heads * D}
    if c["kind"] == "read":
        return {"bytes": get, "flops": L * held * 2 * c["hkv"] * D}
    members = c["W"] + c["S"] + 2 * len(OFFSETS[c["offsets"]])
    if c["alpha"] == "one":
        members = c["W"] + c["S"] + len(OFFSETS[c["offsets"]])
    return {"bytes": L * N * c["hq"] * (2 * D * e + 4 + (4 if c["prior"] else 0))
            + _attended_rows(c) * 2 * c["hkv"] * row,
            "flops": L * N * c["hq"] * members * 4 * D}


# ---- inputs -----------------------------------------------------------------
def _normal(g, *shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _weights(g, L, D):
    return 1.0 + 0.2 * torch.randn((L, D), generator=g, device="cuda")


def prepare(case, seed):
    c, g = case, torch.Generator(device="cuda").manual_seed(seed)
    dt, L, B, D = DTYPES[c["dtype"]], c["L"], c["B"], c["D"]
    s = {"case": c}
    if c["kind"] in ("norm", "norm_bwd"):
        hq, hkv, T = c["hq"], c["hkv"], c["T"]

        def heads():
            if c["packed"]:     # views of one projection's output
                x = _normal(g, L, B, T, (hq + hkv) * D, dtype=dt).view(L, B, T, hq + hkv, D)
                x = x.permute(0, 1, 3, 2, 4)
                return x[:, :, :hq], x[:, :, hq:]
            return _normal(g, L, B, hq, T, D, dtype=dt), _normal(g, L, B, hkv, T, D, dtype=dt)
        s["q"], s["k"] = heads()
        s["qw"], s["kw"] = _weights(g, L, D), _weights(g, L, D)
        if c["kind"] == "norm_bwd":
            s["dq"], s["dk"] = heads()
        return s
    new, old = _new(c), _old(c)
    N, width = sum(new), _rows(c) // c["page"]
    s["cu"] = torch.tensor([sum(new[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    s["old"] = torch.tensor(old, dtype=torch.int32, device="cuda")
    s["held"] = torch.tensor([a + b for a, b in zip(new, old)], dtype=torch.int32, device="cuda")
    pages = B * width + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:B * width]
    s["table"] = table.view(B, width).to(torch.int32).contiguous()
    shape = (L, pages, c["hkv"], c["page"], D)
    rows = [_normal(g, *shape, dtype=dt) for _ in range(2)]
    if c["cache"] == "e4m3":
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = (_quantise(x.float()) for x in rows)
    else:
        s["kc"], s["vc"], s["ks"], s["vs"] = rows[0], rows[1], None, None
    del rows
    if c["kind"] in ("append", "handover"):
        hq, hkv = c["hq"], c["hkv"]
        x = _normal(g, L, N, (hq + 2 * hkv) * D, dtype=dt).view(L, N, hq + 2 * hkv, D)
        s["q"], s["k"], s["v"] = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:]
        s["qw"] = _weights(g, L, D) if c["norm"] else None
        s["kw"] = _weights(g, L, D) if c["norm"] else None
    if c["kind"] in ("handover", "read"):
        out = (L, B, c["hkv"], _rows(c), D)
        s["ko"] = torch.zeros(out, dtype=dt, device="cuda")
        s["vo"] = torch.zeros(out, dtype=dt, device="cuda")
    if c["kind"] == "chunk":
        s["q"] = _normal(g, L, N, c["hq"], D, dtype=dt)
        s["alpha"] = torch.tensor(_alpha(c), dtype=torch.float32, device="cuda")
        s["f"] = torch.tensor(OFFSETS[c["offsets"]], dtype=torch.float32, device="cuda")
        s["beta"] = (torch.randn((L, N, c["hq"]), generator=g, device="cuda") if c["prior"]
                     else None)
    return s


# ---- plain forms ------------------------------------------------------------
def _quantise(x):
    """e4m3 codes of rows and their power-of-two scales, the smallest with |x| / scale <= 448."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)
    k = torch.clamp(e - 9 + (m > 0.875).to(torch.int32), min=-100)
    scale = torch.ldexp(torch.ones_like(top), k)
    scale = torch.where(torch.isfinite(top), scale, torch.full_like(top, float("nan")))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _turns(pos, D):
    """cos and sin of pos * base^(-2j/D): the angles in 64 bits."""
    j = torch.arange(D // 2, device="cuda", dtype=torch.float64)
    a = pos.to(torch.float64)[..., None] * torch.pow(BASE, -2.0 * j / D)
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(x, cos, sin):
    a, b = x[..., :x.shape[-1] // 2], x[..., x.shape[-1] // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def _norm_plain(s, which):
    c, x = s["case"], s[which].float()
    y = _norm(x, s[which + "w"][:, None, None, None, :])
    if c["rotate"]:
        cos, sin = _turns(torch.arange(c["T"], device="cuda"), c["D"])
        y = _turn(y, cos, sin)
    return y.to(DTYPES[c["dtype"]])


def _norm_bwd_plain(s, which):
    c, x, g = s["case"], s[which].float(), s["d" + which].float()
    if c["rotate"]:
        cos, sin = _turns(torch.arange(c["T"], device="cuda"), c["D"])
        g = _turn(g, cos, -sin)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * r
    dw = (g * n).sum(dim=(1, 2, 3), dtype=torch.float64).float()
    g = g * s[which + "w"][:, None, None, None, :]
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    return dx.to(DTYPES[c["dtype"]]), dw


def _places(s):
    """Sequence and position of each new token."""
    N = sum(_new(s["case"]))
    n = torch.arange(N, device="cuda")
    b = (n[:, None] >= s["cu"][None, 1:]).sum(-1)
    return b, s["old"].long()[b] + n - s["cu"].long()[b]


def _put(codes, scales, at, x):
    if scales is None:
        codes[at] = x.to(codes.dtype)
    else:
        y, scales[at] = _quantise(x.float())
        codes.view(torch.uint8)[at] = y.view(torch.uint8)


def _append_plain(s):
    c = s["case"]
    b, pos = _places(s)
    cos, sin = _turns(pos, c["D"])
    q, k, v = s["q"].float(), s["k"].float(), s["v"]
    if c["norm"]:
        q, k = _norm(q, s["qw"][:, None, None, :]), _norm(k, s["kw"][:, None, None, :])
    q, k = _turn(q, cos[:, None], sin[:, None]), _turn(k, cos[:, None], sin[:, None])
    page, slot = s["table"].long()[b, pos // c["page"]], pos % c["page"]
    l = torch.arange(c["L"], device="cuda")[:, None, None]
    h = torch.arange(c["hkv"], device="cuda")[None, None, :]
    at = (l, page[None, :, None], h, slot[None, :, None])
    _put(s["kc"], s["ks"], at, k)
    _put(s["vc"], s["vs"], at, v)
    return q.to(DTYPES[c["dtype"]])


def _rows_of(codes, scales, at):
    """Cache rows as 32-bit values."""
    if scales is None:
        return codes[at].float()
    return codes.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scales[at][..., None]


def _read_plain(s):
    c = s["case"]
    r = torch.arange(_rows(c), device="cuda")
    page, slot = s["table"].long()[:, r // c["page"]], r % c["page"]
    l = torch.arange(c["L"], device="cuda")[:, None, None, None]
    h = torch.arange(c["hkv"], device="cuda")[None, None, :, None]
    at = (l, page[None, :, None, :], h, slot[None, None, None, :])
    live = (r[None, :] < s["held"][:, None])[None, :, None, :, None]
    k, v = _rows_of(s["kc"], s["ks"], at), _rows_of(s["vc"], s["vs"], at)
    s["ko"].copy_(torch.where(live, k.to(s["ko"].dtype), s["ko"]))
    s["vo"].copy_(torch.where(live, v.to(s["vo"].dtype), s["vo"]))
    return s["ko"], s["vo"]


def _chunk_plain(s):
    c = s["case"]
    L, hkv, D, W, S = c["L"], c["hkv"], c["D"], c["W"], c["S"]
    G = c["hq"] // hkv
    b, pos = _places(s)
    N = pos.numel()
    d = s["alpha"][:, None] * s["f"][None, :]
    lo, w = d.floor(), d - d.floor()
    near = pos[:, None] - torch.arange(W, device="cuda")[None, :]
    lead = torch.arange(S, device="cuda")[None, :].expand(N, S)
    rows = torch.cat([near, lead], 1)[None].expand(L, N, W + S)
    there = torch.cat([near >= 0, lead <= pos[:, None]], 1)[None].expand(L, N, W + S)
    first = pos[None, :, None] - lo.long()[:, None, :]
    second = first - 1
    offs = pos[None, :, None] - d.ceil().long()[:, None, :] >= 0
    n_off = first.shape[-1]
    M = W + S + n_off
    every = torch.cat([rows, first, second], -1).clamp(min=0)
    page = s["table"].long()[b[None, :, None], every // c["page"]]
    l = torch.arange(L, device="cuda")[:, None, None, None]
    h = torch.arange(hkv, device="cuda")[None, None, :, None]
    at = (l, page[:, :, None, :], h, (every % c["page"])[:, :, None, :])
    there = torch.cat([there, offs], -1)[:, :, None, None, :]

    def members(x):     # interpolated rows of the offsets in their places
        u = w[:, None, None, :, None]
        y = torch.where(u > 0, (1 - u) * x[..., W + S:M, :] + u * x[..., M:, :], x[..., W + S:M, :])
        return torch.cat([x[..., :W + S, :], y], -2)

    q = s["q"].float().view(L, N, hkv, G, D)
    score = torch.matmul(q, members(_rows_of(s["kc"], s["ks"], at)).transpose(-1, -2))
    score = score / math.sqrt(D)
    if s["beta"] is not None:
        score[..., W + S:] += s["beta"].view(L, N, hkv, G, 1)
    score = torch.where(there, score, torch.full_like(score, float("-inf")))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p / total, members(_rows_of(s["vc"], s["vs"], at)))
    lse = (top + torch.log(total)).view(L, N, c["hq"])
    return out.view(L, N, c["hq"], D).to(DTYPES[c["dtype"]]), lse


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["kind"] == "norm":
        return {"q": _norm_plain(s, "q"), "k": _norm_plain(s, "k")}
    if c["kind"] == "norm_bwd":
        (dq, dqw), (dk, dkw) = _norm_bwd_plain(s, "q"), _norm_bwd_plain(s, "k")
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    if c["kind"] == "append":
        q = _append_plain(s)
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    if c["kind"] == "handover":
        q = _append_plain(s)
        k, v = _read_plain(s)
        return {"q": q, "k": k, "v": v}
    if c["kind"] == "read":
        k, v = _read_plain(s)
        return {"k": k, "v": v}
    o, lse = _chunk_plain(s)
    return {"o": o, "lse": lse}


def _run_own(s, c):
    import structured_sparse_attention_fibonacci_b200 as sa
    if c["kind"] == "norm":
        q, k = sa.qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], eps=EPS, rotate=c["rotate"])
        return {"q": q, "k": k}
    if c["kind"] == "norm_bwd":
        dq, dk, dqw, dkw = sa.qk_norm_rope_bwd(s["q"], s["k"], s["qw"], s["kw"], s["dq"], s["dk"],
                                               eps=EPS, rotate=c["rotate"])
        return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}
    cache = sa.PagedCache(s["kc"], s["vc"], s["ks"], s["vs"])
    if c["kind"] in ("append", "handover"):
        q = sa.cache_append(s["q"], s["k"], s["v"], cache, s["table"], s["cu"], s["old"],
                            q_weight=s["qw"], k_weight=s["kw"], eps=EPS)
        if c["kind"] == "append":
            return {"q": q, "k": s["kc"], "v": s["vc"]}
        k, v = sa.cache_read(cache, s["table"], s["held"], k_out=s["ko"], v_out=s["vo"])
        return {"q": q, "k": k, "v": v}
    if c["kind"] == "read":
        k, v = sa.cache_read(cache, s["table"], s["held"], k_out=s["ko"], v_out=s["vo"])
        return {"k": k, "v": v}
    o, lse = sa.chunk_attn(s["q"], cache, s["table"], s["cu"], s["old"], s["alpha"],
                           window=c["W"], sinks=c["S"], offsets=OFFSETS[c["offsets"]],
                           beta=s["beta"])
    return {"o": o, "lse": lse}


# ---- from the definitions, in 64 bits -----------------------------------------
def _turned(x, pos, sign=1.0):
    """Every pair (x_j, x_{j + D/2}) as a complex number, times e^(i pos theta_j)."""
    D = x.shape[-1]
    theta = torch.exp(-math.log(BASE) * 2.0 / D
                      * torch.arange(D // 2, device="cuda", dtype=torch.float64))
    angle = sign * pos.to(torch.float64)[..., None] * theta
    z = torch.complex(x[..., :D // 2], x[..., D // 2:]) * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], -1)


def _normed(x, w):
    return w * x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def _decoded(codes, scales):
    """The values that cache rows stand for."""
    return codes.double() if scales is None else codes.double() * scales.double()[..., None]


def _coded(x):
    """Rows through 8 bits and back: rounded to the nearest multiple of their step, ties to even."""
    top = x.abs().amax(-1, keepdim=True)
    k = torch.ceil(torch.log2(torch.clamp(top, min=1e-300) / 448.0))
    k = torch.clamp(torch.where(top / torch.exp2(k - 1) <= 448.0, k - 1, k), min=-100.0)
    y = x / torch.exp2(k)
    e = torch.clamp(torch.floor(torch.log2(torch.clamp(y.abs(), min=1e-30))), min=-6.0)
    step = torch.exp2(e - 3)
    return torch.round(y / step) * step * torch.exp2(k)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["kind"] in ("norm", "norm_bwd"):
        t = torch.arange(c["T"], device="cuda")
        found = {}
        for which in ("q", "k"):
            x = s[which].double().requires_grad_(c["kind"] == "norm_bwd")
            w = s[which + "w"].double().requires_grad_(c["kind"] == "norm_bwd")
            y = _normed(x, w[:, None, None, None, :])
            y = _turned(y, t) if c["rotate"] else y
            if c["kind"] == "norm":
                found[which] = y
            else:
                dx, dw = torch.autograd.grad(y, (x, w), s["d" + which].double())
                found["d" + which], found["d" + which + "w"] = dx, dw
        return found
    old, new = _old(c), _new(c)
    if c["kind"] in ("append", "handover", "read"):
        found = {}
        k, v = _decoded(s["kc"], s["ks"]), _decoded(s["vc"], s["vs"])
        if c["kind"] != "read":
            pos = torch.cat([torch.arange(o, o + n, device="cuda") for o, n in zip(old, new)])
            qx, kx, vx = s["q"].double(), s["k"].double(), s["v"].double()
            if c["norm"]:
                qx = _normed(qx, s["qw"].double()[:, None, None, :])
                kx = _normed(kx, s["kw"].double()[:, None, None, :])
            found["q"] = _turned(qx, pos[:, None])
            kx = _turned(kx, pos[:, None])
            if c["cache"] == "e4m3":
                kx, vx = _coded(kx), _coded(vx)
            at = 0
            for b, (o, n) in enumerate(zip(old, new)):
                r = torch.arange(o, o + n, device="cuda")
                page = s["table"][b].long()[r // c["page"]]
                for x, y in ((k, kx), (v, vx)):
                    x[:, page, :, r % c["page"]] = y[:, at:at + n].transpose(0, 1)
                at += n
            if c["kind"] == "append":
                return {"q": found["q"], "k": k, "v": v}
        for name, x in (("k", k), ("v", v)):
            out = torch.zeros(s["ko"].shape, dtype=torch.float64, device="cuda")
            for b, (o, n) in enumerate(zip(old, new)):
                if o + n:
                    seq = x[:, s["table"][b].long()].transpose(1, 2).flatten(2, 3)
                    out[:, b, :, :o + n] = seq[:, :, :o + n]
            found[name] = out
        return found
    L, D, G = c["L"], c["D"], c["hq"] // c["hkv"]
    if L * c["B"] * (c["W"] + c["S"] + 15) > 30000:
        return None     # too many steps of the loops below
    lo, hi, w = _geometry(c)
    o_all = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse_all = torch.zeros(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    for l in range(L):
        far = list(zip(lo[l].tolist(), hi[l].tolist(), w[l].double().tolist()))
        at = 0
        for b, (o, n) in enumerate(zip(old, new)):
            if not n:
                continue
            used = s["table"][b].long()[:-(-(o + n) // c["page"])]
            k, v = (_decoded(x[l][used], None if y is None else y[l][used]).transpose(0, 1)
                    .flatten(1, 2).repeat_interleave(G, 0)
                    for x, y in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))    # [hq, rows, D]
            q = s["q"][l, at:at + n].double().transpose(0, 1)                # [hq, n, D]
            p = torch.arange(o, o + n, device="cuda")

            def keys():
                """(row of each query, second row, weight of the second, which queries, prior?)"""
                for t in range(min(c["W"], o + n)):
                    yield p - t, None, 0.0, p - t >= 0, False
                for j in range(c["S"]):
                    yield torch.full_like(p, j), None, 0.0, p >= j, False
                for a, up, x in far:
                    if up < o + n:
                        yield p - a, (p - a - 1 if x else None), x, p - up >= 0, True

            def value(x, first, second, share):
                y = x[:, first.clamp(0, x.shape[1] - 1)]
                if second is None:
                    return y
                return (1 - share) * y + share * x[:, second.clamp(min=0)]

            scores = []
            for first, second, share, live, prior in keys():
                sc = (q * value(k, first, second, share)).sum(-1) / math.sqrt(D)
                if prior and s["beta"] is not None:
                    sc = sc + s["beta"][l, at:at + n].double().T
                scores.append(sc.masked_fill(~live, float("-inf")))
            scores = torch.stack(scores)
            lse = torch.logsumexp(scores, 0)
            out = torch.zeros_like(q)
            for sc, (first, second, share, live, prior) in zip(scores, keys()):
                out += torch.exp(sc - lse)[..., None] * value(v, first, second, share)
            o_all[l, at:at + n] = out.transpose(0, 1)
            lse_all[l, at:at + n] = lse.T
            at += n
    return {"o": o_all, "lse": lse_all}
