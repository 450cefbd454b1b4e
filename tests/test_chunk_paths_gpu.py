"""The chunk attention on batches large enough for the kernels that a prefill runs, against
the 64-bit plain form on the GPU (paged_device.py, which has the bounds and their derivation)."""
import functools
import threading

import pytest
import torch

import paged_device as dev
import structured_sparse_attention_fibonacci_b200 as sa

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu

FIB = sa.FIB15


def _run(t, q, alpha, beta=None, **kw):
    return sa.chunk_attn(q, *t.call(sa), torch.tensor(alpha, device=DEV), beta=beta, **kw)


# (format, D, Hq, Hkv, window, alpha): one and several query heads per key head; interpolated and
# integer distances
@pytest.mark.parametrize("fmt", ["plain", "e4m3"])
@pytest.mark.parametrize("D,Hq,Hkv,W,alpha", [
    (64, 4, 4, 12, 1.3), (64, 4, 4, 12, 1.0), (128, 8, 2, 12, 1.3), (32, 12, 2, 20, 0.7),
    (16, 2, 1, 5, 2.0)])
def test_probabilities_of_16_bit_queries_keep_16_bits_or_more(fmt, D, Hq, Hkv, W, alpha):
    t = dev.Batch(1, Hkv, D, 16, [700, 0, 90], [60, 300, 1], BF, fmt, seed=D + W)
    q = t.queries(Hq)
    out, lse = _run(t, q, [alpha], window=W, sinks=2)
    ref = dev.chunk(t, q, [alpha], W, 2, FIB)
    o_bad, lse_bad = dev.beyond(t, out, lse, ref)
    assert o_bad <= 0 and lse_bad <= 0, (o_bad, lse_bad)


@pytest.mark.parametrize("new", [1, 9], ids=["team", "own"])
def test_calls_of_two_threads_leave_each_other_their_shared_memory(new):
    """One kernel instance, two sizes of shared memory (one query head per key head, and several),
    from two threads on streams of their own."""
    window = 64 if new == 1 else 12
    calls, want, errors = [], [], []
    for Hq, Hkv in ((1, 1), (2, 1)):
        t = dev.Batch(1, Hkv, 128, 16, [40], [new], BF, "plain", seed=Hq)
        assert (t.is_shared(Hq, window, 0) > 0) == (new == 1)
        q, args, alpha = t.queries(Hq), t.call(sa), torch.ones(1, device=DEV)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
        call = functools.partial(sa.chunk_attn, q, *args, alpha, window=window, out=out, lse=lse)
        call()
        calls.append((call, out))
        want.append(out.clone())
    torch.cuda.synchronize()

    def run(call):
        try:
            stream = torch.cuda.Stream()
            for i in range(20000):
                call(stream=stream)
                if i % 1000 == 999:
                    stream.synchronize()
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=run, args=(c[0],)) for c in calls]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for (_, out), w in zip(calls, want):
        assert torch.equal(out, w)


MANY = tuple(sorted(set(FIB + (7, 7, 11, 16, 30, 60, 64, 100, 200, 400))))[:24] + (2, 2)
EDGES = (1, 31, 32, 33, 62, 63, 64, 65, 90, 31)      # whose near distances fill two words' ends
PROMPT = ([900, 0, 37], [400, 290, 33])
STEP = ([(61 * b) % 500 for b in range(200)], [1] * 200)

# (format, D, Hq, Hkv, L, (old, new), window, sinks, offsets, alphas): blocks enough that every warp
# has one and its whole window for itself, windows of several pairs of tiles
OWN = [
    ("plain", 64, 8, 8, 1, PROMPT, 64, 4, FIB, [1.0]),
    ("plain", 64, 8, 8, 1, PROMPT, 64, 0, FIB, [1.3]),
    ("plain", 64, 8, 8, 1, PROMPT, 300, 4, FIB, [1.0]),
    ("plain", 64, 8, 8, 1, PROMPT, 300, 0, MANY, [1.3]),
    ("plain", 64, 4, 4, 2, PROMPT, 100, 16, EDGES, [1.0, 1.0]),
    ("plain", 64, 8, 8, 1, PROMPT, 64, 0, EDGES, [1.0]),
    ("plain", 64, 8, 8, 1, PROMPT, 40, 0, EDGES, [1.0]),
    ("plain", 64, 8, 8, 1, PROMPT, 100, 0, (), [1.0]),
    ("plain", 64, 16, 4, 2, PROMPT, 100, 4, FIB, [1.0, 0.7]),
    ("plain", 64, 4, 4, 1, STEP, 64, 4, FIB, [1.0]),
    ("plain", 64, 4, 4, 1, STEP, 300, 0, FIB, [1.3]),
    ("e4m3", 64, 8, 8, 1, PROMPT, 64, 4, FIB, [1.0]),
    ("e4m3", 64, 8, 8, 1, PROMPT, 300, 0, FIB, [1.3]),
    ("e4m3", 64, 6, 3, 2, PROMPT, 100, 2, EDGES, [1.0, 1.0]),
    ("e4m3", 64, 4, 4, 1, STEP, 100, 4, FIB, [0.6]),
    ("plain", 128, 4, 4, 2, PROMPT, 100, 4, FIB, [1.0, 1.3]),
    ("plain", 128, 8, 2, 1, PROMPT, 64, 0, FIB, [1.3]),
    ("plain", 128, 24, 2, 1, PROMPT, 64, 4, FIB, [1.0]),
    ("e4m3", 128, 8, 2, 2, PROMPT, 100, 4, FIB, [1.0, 1.3]),
    ("e4m3", 128, 8, 8, 1, PROMPT, 300, 0, FIB, [1.0]),
    ("e4m3", 128, 8, 1, 1, PROMPT, 64, 0, MANY, [1.0]),
    ("plain", 32, 12, 4, 1, PROMPT, 100, 4, EDGES, [1.0]),
    ("e4m3", 32, 8, 8, 1, PROMPT, 300, 4, FIB, [1.3]),
    ("plain", 16, 8, 8, 1, PROMPT, 300, 0, EDGES, [1.0]),
    ("e4m3", 16, 8, 8, 1, PROMPT, 64, 16, FIB, [0.9]),
    ("e4m3", 16, 20, 4, 1, PROMPT, 100, 0, FIB, [1.0]),
]


@pytest.mark.parametrize("prior", [False, True], ids=["", "prior"])
@pytest.mark.parametrize("case", OWN, ids=[f"{c[0]}_{c[2]}x{c[1]}_{c[3]}_w{c[6]}_s{c[7]}_n{len(c[8])}_{c[9][0]}_{len(c[5][1])}"
                                           for c in OWN])
def test_long_windows_of_many_blocks(case, prior):
    fmt, D, Hq, Hkv, L, (old, new), W, S, offs, alpha = case
    t = dev.Batch(L, Hkv, D, 16, old, new, BF, fmt, seed=D + W + S)
    assert t.is_shared(Hq, W, S) == 0 and min(W, max(t.held)) > 32
    q = t.queries(Hq)
    beta = torch.randn((L, t.N, Hq), generator=torch.Generator().manual_seed(2)).to(DEV) if prior else None
    out, lse = _run(t, q, alpha, beta, window=W, sinks=S, offsets=offs)
    o_bad, lse_bad = dev.beyond(t, out, lse, dev.chunk(t, q, alpha, W, S, offs, beta))
    assert o_bad <= 0 and lse_bad <= 0, (o_bad, lse_bad)


# (D, Hq, Hkv, heads that one warp takes)
@pytest.mark.parametrize("fmt", ["plain", "e4m3"])
@pytest.mark.parametrize("D,Hq,Hkv,heads", [(64, 8, 2, 4), (64, 12, 2, 4), (64, 6, 2, 2), (128, 6, 2, 2),
                                            (128, 8, 2, 2), (32, 14, 2, 4), (16, 10, 2, 4), (64, 3, 3, 1)])
def test_heads_of_32_bit_queries_that_share_rows(fmt, D, Hq, Hkv, heads):
    t = dev.Batch(1, Hkv, D, 16, [300, 0, 20], [900, 401, 1], F32, fmt, seed=D)
    most, G = (2 if D == 128 else 4), Hq // Hkv      # launch_f32's choice
    while most > 1 and (G < most or t.N * Hkv * -(-G // most) < 148 * 16):
        most //= 2
    assert most == heads
    q = t.queries(Hq)
    beta = torch.randn((1, t.N, Hq), generator=torch.Generator().manual_seed(2)).to(DEV)
    out, lse = _run(t, q, [0.8], beta, window=20, sinks=3)
    o_bad, lse_bad = dev.beyond(t, out, lse, dev.chunk(t, q, [0.8], 20, 3, FIB, beta))
    assert o_bad <= 0 and lse_bad <= 0, (o_bad, lse_bad)
