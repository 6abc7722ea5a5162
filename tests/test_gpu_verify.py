"""dsa_verify_drafts through the C ABI against the float64 oracle: accepted counts
and tokens equal.  The comparisons are of float64 values on both sides; a drawn
token could differ only where the random number meets a border of the cumulative
weights within float64 rounding (1e-13 of the weight)."""
import numpy as np
import pytest
import torch

from dsa_indexer_top_b200 import binding as B
from oracle import paged as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _run(p, q, x, n_draft, u, us, status=B.DSA_OK):
    n, d1, _ = p.shape
    tok = torch.full((n, d1), -9, dtype=torch.int32, device=DEV)
    acc = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    B.dsa_verify_drafts(p, x, u, us, tok, acc, ws, draft=q, n_draft=n_draft)
    got_status = B.dsa_check_status(ws)
    h = lambda t: None if t is None else t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()
    wt, wa = P.verify_drafts(h(p), h(q), h(x), h(n_draft), h(u), h(us))
    if (wt[np.arange(n), wa] < 0).any():     # a distribution without weight
        status = B.DSA_ERR_INVALID
    assert got_status == status
    np.testing.assert_array_equal(acc.cpu().numpy(), wa)
    np.testing.assert_array_equal(tok.cpu().numpy(), wt)
    return tok, acc


def _inputs(n, D, V, dt, greedy, seed, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    logits = 2 * torch.randn(n, D + 1, V, generator=g, device=DEV)
    near = logits[:, :D] + 0.7 * torch.randn(n, D, V, generator=g, device=DEV)
    pp = torch.zeros(n, D + 1, V + pad, dtype=dt, device=DEV)
    qq = torch.zeros(n, D, V + pad, dtype=dt, device=DEV)
    pp[..., :V] = torch.softmax(logits, -1).to(dt)
    qq[..., :V] = torch.softmax(near, -1).to(dt)
    p, q = pp[..., :V], qq[..., :V]
    x = near.argmax(-1) if greedy or V < 2 else torch.multinomial(q.reshape(-1, V).float(), 1, generator=g).view(n, D) \
        if D else torch.zeros(n, 0, device=DEV)
    u = torch.rand(n, D, generator=g, device=DEV)
    us = torch.rand(n, generator=g, device=DEV)
    k = torch.randint(0, D + 1, (n,), generator=g, device=DEV, dtype=torch.int32)
    return p, (None if greedy else q), x.to(torch.int32), k, u, us


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("n,D,V,pad", [(1, 1, 1, 0), (3, 2, 7, 0), (9, 1, 31, 1), (5, 4, 1000, 8), (2, 40, 513, 0),
                                       (33, 3, 4099, 0), (4, 0, 777, 0), (6, 2, 65537, 0), (200, 5, 2048, 0), (3, 2, 131071, 1)])
def test_verify(cuda_ok, dt, greedy, n, D, V, pad):
    p, q, x, k, u, us = _inputs(n, D, V, dt, greedy, seed=n * 100 + D, pad=pad)
    _run(p, q, x, k, u, us)
    _run(p, q, x, None, u, us)


@pytest.mark.parametrize("V", [5, 300, 20000])
def test_verify_borders(cuda_ok, V):
    """Random numbers at 0 and just under 1, one-hot and tied distributions, zero
    tails: exact sums, so the borders themselves are tested."""
    one = torch.zeros(6, 2, V, device=DEV)
    one[:, :, V // 2] = 1.0
    even = torch.full((6, 2, V), 1.0 / 1024, device=DEV)
    even[:, :, V // 3:] = 0
    even[:, 0, 0] = 0
    us = torch.tensor([0.0, 0.5, 1 - 2.0 ** -24, 0.25, 2.0 ** -30, 0.75], device=DEV)
    x = torch.full((6, 1), V // 2, dtype=torch.int32, device=DEV)
    for p in (one, even):
        for u in (0.0, 0.999):
            au = torch.full((6, 1), u, device=DEV)
            _run(p, None, x, None, au, us)
            _run(p, even[:, :1].contiguous(), x, None, au, us)
            _run(p, one[:, :1].contiguous(), x, None, au, us)
            _run(p, p[:, :1].contiguous(), x, None, au, us)      # p == q: nothing left, drawn from p


def test_verify_odd_values(cuda_ok):
    """Negative, NaN and infinite entries count as 0; random numbers out of range
    still give a token with weight; no weight at all gives -1 and an error."""
    p, q, x, k, u, us = _inputs(8, 2, 600, torch.float32, False, seed=3)
    p[:, :, 10], p[:, :, 11], p[:, :, 599] = float("nan"), float("inf"), -5.0
    q[:, :, 20], q[:, :, 21] = float("nan"), float("inf")
    x[0, 0], x[1, 1] = 10, 11
    _run(p, q, x, None, u, us)
    wild = torch.tensor([1.0, 7.0, -3.0, float("nan"), float("inf"), 0.5, 1.0, 0.0], device=DEV)
    tok = torch.empty(8, 3, dtype=torch.int32, device=DEV)
    acc = torch.empty(8, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    B.dsa_verify_drafts(p, x, u, wild, tok, acc, ws, draft=q)
    assert B.dsa_check_status(ws) == B.DSA_OK
    drawn = tok.gather(1, acc.long()[:, None])[:, 0]
    assert ((drawn >= 0) & (drawn < 600)).all()
    assert (p[torch.arange(8, device=DEV), acc.long(), drawn.long()] > 0).all()
    p[3] = 0
    _run(p, q, x, None, u, us, status=B.DSA_ERR_INVALID)


def test_verify_reports_bad_drafts(cuda_ok):
    p, q, x, k, u, us = _inputs(4, 3, 50, torch.float32, False, seed=4)
    u.zero_()
    x[1, 1], x[2, 0] = 50, -1
    _run(p, q, x, None, u, us, status=B.DSA_ERR_INVALID)
    _run(p, None, x, None, u, us, status=B.DSA_ERR_INVALID)
    x.clamp_(0, 49)
    _run(p, q, x, torch.tensor([4, -1, 2, 3], dtype=torch.int32, device=DEV), u, us, status=B.DSA_ERR_INVALID)


def test_verify_strides_and_graph(cuda_ok):
    """Rows of a wider tensor, one target row shared by every request, a captured call."""
    p, q, x, k, u, us = _inputs(5, 2, 1001, torch.bfloat16, False, seed=5, pad=7)
    shared = p[:1].expand(5, -1, -1)
    _run(shared, q, x, None, u, us)
    tok, acc = _run(p, q, x, k, u, us)
    out = torch.empty_like(tok), torch.empty_like(acc)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    B.dsa_verify_drafts(p, x, u, us, *out, ws, draft=q, n_draft=k)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        B.dsa_verify_drafts(p, x, u, us, *out, ws, draft=q, n_draft=k)
    for t in out:
        t.fill_(-9)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], tok) and torch.equal(out[1], acc)
