"""Norms of queries and keys with the rotation, forward and backward, against
their plain 64-bit form, and as a part of the training step.

Tolerances per element: half a step of the type, u = torch.finfo(dtype).eps / 2,
of the result, plus 2^-20 of the row's largest term for fp32 arithmetic; weight
gradients 2^-18 of the sum of their terms' sizes (fp32 sums of at most 48 rows per
thread in these cases, joined in shared memory and then in 64 bits)."""
import numpy as np
import pytest
import torch

import oracle
import structured_sparse_attention_fibonacci_b200 as sa
import paged_plain as plain
from parity import to_np

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
pytestmark = pytest.mark.gpu

# (id, dtype, L, B, Hq, Hkv, T, D, packed, pos0)
CASES = [
    ("f32_tiny", F32, 1, 1, 2, 2, 64, 16, False, 0),
    ("f32_gqa", F32, 2, 3, 6, 2, 37, 32, True, 5),
    ("f32_d64", F32, 1, 2, 3, 1, 1, 64, False, 1000),
    ("f32_d128", F32, 2, 1, 1, 1, 129, 128, True, 0),
    ("bf16_d64", BF, 3, 2, 4, 4, 333, 64, False, 0),
    ("bf16_packed", BF, 1, 2, 8, 2, 100, 64, True, 70000),
    ("bf16_d128", BF, 2, 1, 5, 3, 61, 128, True, 0),
    ("bf16_d16", BF, 1, 5, 1, 1, 7, 16, False, 3),
    ("bf16_d32_one", BF, 1, 1, 1, 1, 1, 32, False, 0),
    ("bf16_many_rows", BF, 1, 4, 9, 3, 600, 64, True, 0),
]


def _heads(g, L, B, Hq, Hkv, T, D, dtype, packed, scale=1.0):
    """(q, k) on the device; packed: views of one [L, B, T, heads, D] tensor."""
    x = torch.randn((L, B, T, Hq + Hkv, D), generator=g)
    x = x * scale * torch.logspace(-2, 2, T)[None, None, :, None, None]
    x = x.to(dtype).to(DEV).permute(0, 1, 3, 2, 4)
    q, k = x[:, :, :Hq], x[:, :, Hq:]
    return (q, k) if packed else (q.contiguous(), k.contiguous())


@pytest.mark.parametrize("mode", ["norm_rope", "norm", "rope"])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_norm_and_its_gradients(case, mode):
    name, dtype, L, B, Hq, Hkv, T, D, packed, pos0 = case
    g = torch.Generator().manual_seed(len(name))
    q, k = _heads(g, L, B, Hq, Hkv, T, D, dtype, packed)
    dqo, dko = _heads(g, L, B, Hq, Hkv, T, D, dtype, not packed)
    qw, kw = (1 + 0.3 * torch.randn((L, D), generator=g) for _ in range(2))
    if mode == "rope":
        qw = kw = None
    rotate, eps, u = mode != "norm", 1e-5, torch.finfo(dtype).eps / 2
    dev = lambda w: None if w is None else w.to(DEV)
    kwargs = dict(eps=eps, rotate=rotate, pos0=pos0)
    yq, yk = sa.qk_norm_rope(q, k, dev(qw), dev(kw), **kwargs)
    dq, dk, dqw, dkw = sa.qk_norm_rope_bwd(q, k, dev(qw), dev(kw), dqo, dko, **kwargs)
    torch.cuda.synchronize()
    for x, w, dy, y, dx, dw in ((q, qw, dqo, yq, dq, dqw), (k, kw, dko, yk, dk, dkw)):
        x, dy = x.double().cpu(), dy.double().cpu()
        w = None if w is None else w.double()
        ref = plain.norm_rope(x, w, eps, rotate, pos0)
        big = plain.norm_rope(x, w, eps, False).abs().amax(-1, keepdim=True)
        assert y.is_contiguous() and y.shape == x.shape
        assert ((y.double().cpu() - ref).abs() <= u * ref.abs() + 2.0 ** -20 * big).all()
        rdx, rdw, terms = plain.norm_rope_bwd(x, w, eps, rotate, dy, pos0)
        big = dy.abs().amax(-1, keepdim=True)
        if w is not None:
            r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
            big = big * r * w.abs().amax() * (1 + (x * r).abs().amax(-1, keepdim=True) ** 2)
        assert ((dx.double().cpu() - rdx).abs() <= u * rdx.abs() + 2.0 ** -20 * big).all()
        if w is None:
            assert dw is None
        else:
            assert ((dw.double().cpu() - rdw).abs() <= 2.0 ** -18 * terms + 1e-30).all()


def test_zero_rows_and_no_eps():
    """A zero row: with eps its output and gradient are finite (g w / sqrt(eps)); with eps = 0 it
    is 0 * inf, NaN, and no other row is touched."""
    q = torch.zeros((1, 1, 1, 3, 16), device=DEV)
    q[..., 1, :] = 2.0
    w = torch.ones((1, 16), device=DEV)
    dy = torch.ones_like(q)
    y, _ = sa.qk_norm_rope(q, q, w, w, eps=0.25, rotate=False)
    assert (y[0, 0, 0, 0] == 0).all() and torch.isfinite(y).all()
    dx, _, dw, _ = sa.qk_norm_rope_bwd(q, q, w, w, dy, dy, eps=0.25, rotate=False)
    assert (dx[0, 0, 0, 0] == 2.0).all() and torch.isfinite(dw).all()
    y, _ = sa.qk_norm_rope(q, q, w, w, eps=0.0, rotate=False)
    assert torch.isnan(y[0, 0, 0, 0]).all() and (y[0, 0, 0, 1] == 1).all()


def test_in_place_and_repeatable():
    g = torch.Generator().manual_seed(3)
    q, k = _heads(g, 2, 2, 4, 2, 200, 64, BF, False)
    dqo, dko = _heads(g, 2, 2, 4, 2, 200, 64, BF, False)
    w = torch.rand((2, 64), generator=g).to(DEV)
    a = sa.qk_norm_rope(q, k, w, w)
    q2, k2 = q.clone(), k.clone()
    b = sa.qk_norm_rope(q2, k2, w, w, q_out=q2, k_out=k2)
    assert b[0] is q2 and torch.equal(a[0], q2) and torch.equal(a[1], k2)
    ref = sa.qk_norm_rope_bwd(q, k, w, w, dqo, dko)
    ws = torch.empty(sa.qk_norm_workspace_size(q.shape, k.shape), dtype=torch.uint8, device=DEV)
    d1, d2 = dqo.clone(), dko.clone()
    got = sa.qk_norm_rope_bwd(q, k, w, w, d1, d2, dq=d1, dk=d2, workspace=ws)
    for x, y in zip(ref, got):
        assert torch.equal(x, y)


def test_no_rows():
    w = torch.ones((2, 32), device=DEV)
    q = torch.empty((2, 0, 3, 5, 32), device=DEV)
    y, z = sa.qk_norm_rope(q, q[:, :, :1], w, w)
    assert y.shape == q.shape and z.shape == (2, 0, 1, 5, 32)
    dq, dk, dqw, dkw = sa.qk_norm_rope_bwd(q, q[:, :, :1], w, w, q, q[:, :, :1])
    assert (dqw == 0).all() and (dkw == 0).all() and dqw.shape == (2, 32)


def test_training_step_gradients_against_the_oracle_and_differences():
    """norm -> sparse attention -> loss <dO, O>, fp32: gradients of the raw queries and keys and
    of the weights from the chained backward calls, against the oracle's backward chained with
    the plain form's, and against a central difference of the loss in 64 bits."""
    L, B, H, T, D = 2, 1, 2, 40, 16
    g = torch.Generator().manual_seed(17)
    xq, xk, v, do = (torch.randn((L, B, H, T, D), generator=g) for _ in range(4))
    qw, kw = (1 + 0.2 * torch.randn((L, D), generator=g) for _ in range(2))
    alpha, eps, kw_ = torch.tensor([0.8, 1.3]), 1e-5, dict(window=5, sinks=1)
    d = lambda t: t.to(DEV)
    q, k = sa.qk_norm_rope(d(xq), d(xk), d(qw), d(kw), eps=eps, rotate=False)
    o, lse = sa.fwd(q, k, d(v), d(alpha), **kw_)
    dq, dk, dv, dal = sa.bwd(q, k, d(v), o, lse, d(do), d(alpha), **kw_)
    got = sa.qk_norm_rope_bwd(d(xq), d(xk), d(qw), d(kw), dq, dk, eps=eps, rotate=False)
    got = [to_np(t) for t in got]

    def normed(x, w):
        return plain.norm_rope(x.double(), w.double(), eps, False)
    rq, rk = normed(xq, qw), normed(xk, kw)
    r = oracle.bwd(rq.numpy(), rk.numpy(), to_np(v), to_np(do), alpha.numpy(), **kw_)
    want = []
    for x, w, dy in ((xq, qw, r[0]), (xk, kw, r[1])):
        want.append(plain.norm_rope_bwd(x.double(), w.double(), eps, False, torch.tensor(dy)))
    want = [want[0][0], want[1][0], want[0][1], want[1][1]]
    for a, b in zip(got, want):
        b = b.numpy()
        assert np.abs(a - b).max() <= 1e-5 * max(1.0, np.abs(b).max())

    def loss(xq_, xk_, qw_, kw__):
        a, b = (plain.norm_rope(x, w, eps, False) for x, w in ((xq_, qw_), (xk_, kw__)))
        oo, _ = oracle.fwd(a.numpy(), b.numpy(), to_np(v), alpha.numpy(), **kw_)
        return float((oo * to_np(do)).sum())
    base = [t.double() for t in (xq, xk, qw, kw)]
    step = [torch.randn(t.shape, generator=g, dtype=torch.float64) for t in base]
    h = 1e-5
    diff = (loss(*[b + h * s for b, s in zip(base, step)])
            - loss(*[b - h * s for b, s in zip(base, step)])) / (2 * h)
    mine = sum(float((torch.tensor(a) * s).sum()) for a, s in zip(got, step))
    assert abs(diff - mine) <= 1e-4 * (abs(diff) + 1)


def test_backward_replays_from_graphs_with_their_own_workspaces():
    g = torch.Generator().manual_seed(4)
    sets = []
    for T in (300, 50):
        q, k = _heads(g, 1, 2, 4, 2, T, 64, BF, True)
        dy = _heads(g, 1, 2, 4, 2, T, 64, BF, False)
        w = torch.rand((1, 64), generator=g).to(DEV)
        ws = torch.empty(sa.qk_norm_workspace_size(q.shape, k.shape), dtype=torch.uint8, device=DEV)
        want = sa.qk_norm_rope_bwd(q, k, w, w, *dy)
        sets.append((q, k, w, dy, ws, want))
    torch.cuda.synchronize()
    graphs = []
    for q, k, w, dy, ws, _ in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = sa.qk_norm_rope_bwd(q, k, w, w, *dy, workspace=ws)
        graphs.append((graph, out))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        graphs[0][0].replay()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
    torch.cuda.synchronize()
    for (_, out), s in zip(graphs, sets):
        for a, b in zip(out, s[5]):
            assert torch.equal(a, b)


def test_a_capture_that_needs_a_new_table_is_refused_and_goes_on():
    q, k = (torch.randn(1, 1, 2, 9, 32, device=DEV) for _ in range(2))
    base = 4321.0      # used nowhere else
    out = torch.zeros_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        with pytest.raises(sa.SparseAttnError):
            sa.qk_norm_rope(q, k, None, None, rope_base=base)
        out.copy_(q)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, q)
    want = sa.qk_norm_rope(q, k, None, None, rope_base=base)[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        sa.qk_norm_rope(q, k, None, None, rope_base=base, q_out=out, k_out=torch.empty_like(k))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
