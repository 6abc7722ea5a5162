"""Draft verification with every size of cluster, from eight CTAs a request down to
one, over short vocabularies, where a CTA has next to nothing to do before it writes
to the others of its cluster."""
import pytest
import torch

from dsa_indexer_top_b200 import binding as B
from tests.test_gpu_verify import _inputs, _run

pytestmark = pytest.mark.gpu
DEV = "cuda"


# (148 SMs with four CTAs each: the requests share 592 places)
@pytest.mark.parametrize("n", [2, 80, 90, 110, 140, 190, 290, 600, 701])
@pytest.mark.parametrize("greedy,dt", [(False, torch.float32), (True, torch.bfloat16)])
@pytest.mark.parametrize("V", [3, 129, 1031])
def test_verify_cluster_sizes(cuda_ok, n, greedy, dt, V):
    p, q, x, k, u, us = _inputs(n, 2, V, dt, greedy, seed=n + V)
    _run(p, q, x, k, u, us)


def test_verify_short_rows_under_load(cuda_ok):
    """The same tokens each time while another stream keeps the SMs busy."""
    p, q, x, k, u, us = _inputs(70, 1, 33, torch.float32, False, seed=8)
    tok, acc = _run(p, q, x, k, u, us)
    side = torch.cuda.Stream()
    busy = torch.randn(1 << 25, device=DEV)
    out = torch.empty_like(tok), torch.empty_like(acc)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    for _ in range(50):
        for t in out:
            t.fill_(-9)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            busy.mul_(1.0)
        for _ in range(8):
            B.dsa_verify_drafts(p, x, u, us, *out, ws, draft=q, n_draft=k)
        torch.cuda.synchronize()
        assert B.dsa_check_status(ws) == B.DSA_OK
        assert torch.equal(out[0], tok) and torch.equal(out[1], acc)
