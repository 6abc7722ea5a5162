"""Attention over packed FP8 rows whose scales lie far apart."""
import numpy as np
import pytest
import torch

from oracle import paged as P
from tests.test_gpu_paged import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _fp8_case(seqs, seed, **kw):
    """Query latent dims 0..7 are zero: a row with codes in those dims alone has a logit
    from its RoPE key only, whatever its scale."""
    c = Case(seqs, page=16, kind="fp8", seed=seed, **kw)
    c.q[..., :8] = 0
    c.q[..., 512] = 4.0
    return c


def _set_row(c, b, s, scale, key):
    """Row s of sequence b: code 1.0 in dims 0..7, the scale given, RoPE key (key, 0, ...)."""
    at = c.table[b, s // 16], s % 16
    raw = torch.zeros(656, dtype=torch.uint8)
    raw[:8] = 0x38
    raw[512:514] = torch.tensor([key], dtype=torch.bfloat16).view(torch.uint8)
    raw[640:644] = torch.tensor([scale], dtype=torch.float32).view(torch.uint8)
    c.pool[at][:656] = raw.to(DEV)
    c.rows[at] = 0
    c.rows[at][:8] = scale
    c.rows[at][512] = key


@pytest.mark.parametrize("k", [6, 12, 20, 30, 60])
@pytest.mark.parametrize("heads", [16, 64])
def test_fp8_large_scale_without_weight(cuda_ok, k, heads):
    """Rows whose scale is 2^k times the others' but whose logit is 75 under them (e^-75 2^60
    adds nothing), and rows with that scale that some tokens do not see."""
    c = _fp8_case([(300, 1), (128, 5), (1000, 2), (20, 40)], seed=43, heads=heads)
    for b, s in [(0, 5), (0, 299), (0, 140), (1, 131), (1, 0), (2, 700), (2, 1001), (3, 30)]:
        _set_row(c, b, s, 2.0 ** (k - 7), -300.0)
    c.run().check()


@pytest.mark.parametrize("k", [4, 9, 16, 24, 40])
@pytest.mark.parametrize("heads", [16, 64])
def test_fp8_small_scale_with_all_the_weight(cuda_ok, k, heads):
    """A row whose logit is 75 above the others' and whose scale is 2^-k of theirs: the
    result is that row, in proportion to itself.  Latent part: code times scale, a power of
    two; its weight over the sum: fp16 (2^-11) and float32 roundings; bf16 result 2^-8.  The
    others add 2^40 e^-60 1000 values of their own size, 1e-11 of the row's."""
    c = _fp8_case([(300, 1), (1000, 2), (20, 40)], seed=44, heads=heads)
    spots = [(0, 150), (1, 3), (2, 0)]
    for b, s in spots:
        _set_row(c, b, s, 2.0 ** (-7 - k), 300.0)
    c.run()
    for b, s in spots:
        got = c.out[c.begin[b]:c.begin[b + 1]].double().cpu().numpy()
        want = c.rows[c.table[b, s // 16], s % 16, :512]
        assert (np.abs(got[..., :8] - want[:8]) <= (2.0 ** -8 + 2.0 ** -10) * want[:8]).all()
        assert (np.abs(got[..., 8:]) <= 1e-10 * want[0]).all()


def test_fp8_rows_of_zeros_before_others(cuda_ok):
    """Tiles whose rows all have scale zero and logits 40 above the rows that follow: the
    result is e^-40 of those rows, in proportion to itself (the zeros' weight divides them)."""
    c = _fp8_case([(500, 1)], seed=45, heads=64)
    for s in range(256):
        _set_row(c, 0, s, 0.0, 160.0)
    c.run()
    want, lse, _ = P.paged_mla(c.q.double().cpu().numpy(), c.rows, c.table, c.begin, c.total, 16, 512, c.scale)
    mag = c._weighted_abs(c.q.double().cpu().numpy(), c.table)
    got = c.out.double().cpu().numpy()
    # weights: float32 logits (1e-3 each) and fp16; bf16 result
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.1e-3 + 2.0 ** -10) * mag).all()
    assert np.abs(c.lse.double().cpu().numpy() - lse).max() <= 1e-3


def test_fp8_scales_far_apart_in_long_pieces(cuda_ok):
    """The same with many sequences, so that a piece runs over several tiles: scales 2^-24 of
    the others' with all the weight, 2^24 without, zeros in front of everything."""
    c = _fp8_case([(600, 1), (700, 1), (500, 1), (400, 5)] * 30, seed=47, heads=64)
    for b in range(0, 120, 4):
        _set_row(c, b, (37 * b) % 601, 2.0 ** -31, 300.0)
        _set_row(c, b + 1, (41 * b) % 700, 2.0 ** 17, -300.0)
        for s in range(256):
            _set_row(c, b + 2, s, 0.0, 160.0)
        _set_row(c, b + 3, 403, 2.0 ** 20, -300.0)
    c.run()
    q = c.q.double().cpu().numpy()
    want, lse, _ = P.paged_mla(q, c.rows, c.table, c.begin, c.total, 16, 512, c.scale)
    mag = c._weighted_abs(q, c.table)
    # (in proportion to the result's own size: no absolute term but what fp16 weights leave,
    # 2^-20 of the largest weight times scale, here under 2^-20 of the row's largest |c|)
    big = np.abs(want).max(-1, keepdims=True)
    err = np.abs(c.out.double().cpu().numpy() - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + (2.1e-3 + 2.0 ** -10) * mag + 2.0 ** -19 * big).all()
    assert np.abs(c.lse.double().cpu().numpy() - lse).max() <= 1e-3
