"""Attention over paged caches where its roles run at different speeds: many short
pieces (one or two tiles of 128 rows each) on every cluster, with other work on the
same SMs.  Sums, maxima and results pass between warps and between the two CTAs of a
cluster once per piece, so a missing wait would show as a result that changes from
one call to the next."""
import numpy as np
import pytest
import torch

from dsa_indexer_top_b200 import binding as B
from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _short_sequences(n, seed):
    rng = np.random.default_rng(seed)
    return [(int(rng.integers(0, 200)), int(rng.integers(1, 6))) for _ in range(n)]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("heads", [64, 48])
def test_many_short_pieces_under_load(cuda_ok, kind, heads):
    """Row tiles of more than 64 rows (two tokens): the oracle's result, the same bits each time."""
    c = Case(_short_sequences(230, seed=31), heads=heads, page=16, kind=kind, seed=31).run().check()
    out, lse = c.out.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    busy = torch.randn(1 << 25, device=DEV)
    wide = torch.randn(2048, 2048, device=DEV)
    for _ in range(25):
        c.out.fill_(77.0)
        c.lse.fill_(77.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(3):
                busy.mul_(1.0)
                torch.sin(wide)
        B.dsa_paged_mla(c.batch, c.mla, c.ws)
        torch.cuda.synchronize()
        assert B.dsa_check_status(c.ws) == B.DSA_OK
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_results_are_out_before_the_next_piece(cuda_ok, kind):
    """One-tile pieces: a result is staged where the next piece's weights arrive."""
    c = Case([(i % 120, 1) for i in range(600)], heads=64, page=32, kind=kind, seed=32).run().check()
    out, lse = c.out.clone(), c.lse.clone()
    for _ in range(25):
        c.out.fill_(77.0)
        c.lse.fill_(77.0)
        for _ in range(4):
            B.dsa_paged_mla(c.batch, c.mla, c.ws)
        torch.cuda.synchronize()
        assert B.dsa_check_status(c.ws) == B.DSA_OK
        assert torch.equal(c.out, out) and torch.equal(c.lse, lse)
