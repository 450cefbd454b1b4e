"""The chunk attention on batches large enough for the kernels that a prefill runs, against
the 64-bit plain form on the GPU (paged_device.py, which has the bounds and their derivation)."""
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
