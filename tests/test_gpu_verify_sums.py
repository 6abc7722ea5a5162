"""Draft verification where float64 sums of the weights round: the token drawn is one
whose interval of the cumulative weights holds the target, or a neighbour within the
sums' rounding, never one from elsewhere in the vocabulary."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from dsa_indexer_top_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _draw(rows, u):
    """Tokens drawn from rows [n, V] without drafts."""
    p = torch.from_numpy(np.asarray(rows, dtype=np.float32)).to(DEV)[:, None]
    n = p.shape[0]
    tok = torch.full((n, 1), -9, dtype=torch.int32, device=DEV)
    acc = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    B.dsa_verify_drafts(p, torch.empty(n, 0, dtype=torch.int32, device=DEV), torch.empty(n, 0, device=DEV),
                        torch.tensor(u, dtype=torch.float32, device=DEV), tok, acc, ws)
    assert B.dsa_check_status(ws) == B.DSA_OK and (acc == 0).all()
    return tok[:, 0].tolist()


def _holds(row, u, token):
    """Whether the exact cumulative weights hold u * total at `token`, within 2^-48 of the total."""
    w = {int(j): Fraction(float(row[j])) for j in np.nonzero(row)[0]}
    total = sum(w.values())
    target, before = Fraction(float(np.float32(u))) * total, sum(x for j, x in w.items() if j < token)
    slack = total / 2 ** 48
    return token in w and before <= target + slack and target < before + w[token] + slack


@pytest.mark.parametrize("V,gap", [(16384, 32), (16384, 64), (70000, 32)])
def test_target_between_two_orders_of_summation(cuda_ok, V, gap):
    """1 and twice 2^-53 sum to 1 + 2^-52 or to 1, by their order; the target is 1, and a
    last entry of next to no weight stands at the vocabulary's end."""
    row = np.zeros(V)
    row[0], row[1], row[1 + gap], row[V // 2], row[V - 1] = 1.0, 2.0 ** -53, 2.0 ** -53, 1.0, 2.0 ** -60
    tok, = _draw([row], [0.5])
    assert tok in (0, 1, 1 + gap, V // 2) and _holds(row, 0.5, tok)


@pytest.mark.parametrize("V", [40, 2000, 16384, 50000])
def test_borders_of_wide_ranges(cuda_ok, V):
    """Weights over 60 powers of two, random numbers at and next to the borders of the
    cumulative weights."""
    rng = np.random.default_rng(V)
    rows, us = [], []
    for _ in range(40):
        row = np.zeros(V, dtype=np.float32)
        at = rng.choice(V, min(V, 300), replace=False)
        row[at] = 2.0 ** rng.integers(-60, 1, len(at)) * (1 + rng.integers(0, 4, len(at)) / 4)
        cdf = np.cumsum(row.astype(np.float64))
        u = np.float32(cdf[rng.choice(at)] / cdf[-1])
        rows.append(row)
        us.append(min(np.nextafter(u, np.float32(rng.integers(0, 2))) if rng.random() < 0.5 else u, 1 - 2.0 ** -24))
    for row, u, tok in zip(rows, us, _draw(rows, us)):
        assert _holds(row, u, tok)
