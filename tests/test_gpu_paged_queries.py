"""Queries that are not finite, in attention over paged caches."""
import pytest
import torch

from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_query_that_is_not_finite(cuda_ok, kind, value):
    """A (token, head) whose query holds an infinity or NaN gives NaN, the others what they
    give without it."""
    shape = dict(d_lat=64, d_rope=16) if kind == "f32" else {}
    heads = 4 if kind == "f32" else 64
    c = Case([(200, 3), (1500, 1)], heads=heads, page=16, kind=kind, seed=46, **shape).run()
    out, lse = c.out.clone(), c.lse.clone()
    hit = [(0, 1, 10), (2, 3, 40), (3, 0, 63)]
    for i, h, d in hit:
        c.q[i, h, d] = value
    c.run()
    bad = torch.zeros(4, heads, dtype=torch.bool, device=DEV)
    for i, h, _ in hit:
        bad[i, h] = True
    assert torch.isnan(c.out[bad]).all() and not torch.isfinite(c.lse[bad]).any()
    assert torch.equal(c.out[~bad], out[~bad]) and torch.equal(c.lse[~bad], lse[~bad])


def test_fp8_infinite_query_over_small_codes(cuda_ok):
    """Every row's code in the query's infinite dim is small: the logits have to be infinite
    all the same, not the largest finite query's."""
    c = Case([(200, 3), (1500, 1)], heads=64, page=16, kind="fp8", seed=48)
    c.pool[..., 10] = 0x18
    c.run()
    out, lse = c.out.clone(), c.lse.clone()
    c.q[1, 7, 10] = float("inf")
    c.q[3, 2, 10] = float("-inf")
    c.run()
    bad = torch.zeros(4, 64, dtype=torch.bool, device=DEV)
    bad[1, 7] = bad[3, 2] = True
    assert torch.isnan(c.out[bad]).all() and not torch.isfinite(c.lse[bad]).any()
    assert torch.equal(c.out[~bad], out[~bad]) and torch.equal(c.lse[~bad], lse[~bad])
