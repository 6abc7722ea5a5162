"""Attention over a paged bf16 cache where one row has all the weight."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("heads,page", [(64, 16), (128, 64), (3, 8)])
def test_one_visible_row_is_returned_as_it_is(cuda_ok, heads, page):
    """One row: its weight over the sum of weights is 1, whatever the weight is rounded
    to.  The quotient in float32 is off by at most 2^-22, and a bf16 value times that
    rounds to itself."""
    c = Case([(0, 1)] * 300, heads=heads, page=page, seed=41).run()
    row = torch.from_numpy(np.stack([c.rows[c.table[b, 0], 0, :512] for b in range(300)])).to(DEV)
    assert torch.equal(c.out.double(), row[:, None].expand(-1, heads, -1))
    x = c.scale * torch.einsum("nhd,nd->nh", c.q.double(), torch.from_numpy(np.stack(
        [c.rows[c.table[b, 0], 0] for b in range(300)])).to(DEV))
    assert (c.lse.double() - x).abs().max() <= 1e-3


@pytest.mark.parametrize("total,where", [(500, 3), (500, 499), (40000, 7), (40000, 39000)])
def test_one_row_with_all_the_weight(cuda_ok, total, where):
    """A row whose logit is 40 above the others': the others add less than 40000 e^-40 (1e-13)
    of their values, the row is returned as it is, also where parts are joined (each part's
    quotient and the join's are float32: under 2^-20 together)."""
    c = Case([(total - 1, 1)], heads=64, page=64, seed=42)
    c.q[..., 512] = 8.0                              # one RoPE dim carries the difference
    c.pool[..., 512] = 0.0
    c.rows[..., 512] = 0.0
    at = c.table[0, where // 64], where % 64
    for x in (c.pool, c.rows):
        x[at][512] = 128.0
    c.run()
    # logits of the others are N(0, 1.5): below 9 in 40000 x 64 of them; 64 - 9 - 9 = 46
    assert torch.equal(c.out[0].double(), torch.from_numpy(c.rows[at][:512]).to(DEV).expand(64, -1))
