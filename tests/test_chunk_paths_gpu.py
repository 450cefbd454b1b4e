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
