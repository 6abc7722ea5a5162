"""Pins of the paged-cache oracle (CPU): hand-worked page tables, paged attention
against dense float64 attention, the packed FP8 decoder, and draft verification
against the identity it exists for (the emitted token follows the target)."""
import numpy as np
import torch

from oracle import paged as P


def test_page_tables_by_hand():
    # pages of 4 rows; sequence 0 grows into a second page, 1 stays inside its page,
    # 2 has no token, 3 starts from nothing and takes three pages
    table = [[7, -1, -1], [5, -1, -1], [-1, -1, -1], [-1, -1, -1]]
    r = P.page_tables([3, 1, 0, 0], [2, 1, 0, 9], [1, 1, 0, 0], [0, 2, 4, 6, 8], 1, table, 4, 14)
    assert r["table"].tolist() == [[7, 2, -1], [5, -1, -1], [-1, -1, -1], [4, 6, 8]]
    assert r["q_begin"].tolist() == [0, 2, 3, 3, 12] and r["seq_len"].tolist() == [5, 2, 0, 9]
    assert r["q_seq"].tolist() == [0, 0, 1] + [3] * 9 + [0, 0]
    assert r["q_pos"].tolist() == [3, 4, 1] + list(range(9)) + [0, 0]
    assert r["slot_map"].tolist() == [31, 8, 21, 16, 17, 18, 19, 24, 25, 26, 27, 32, -1, -1]
    assert r["held_out"].tolist() == [2, 1, 0, 3] and r["free_used"] == 4


def test_paged_attention_equals_dense():
    g = np.random.default_rng(3)
    H, dl, dr, page = 3, 8, 4, 4
    lens, new = [9, 1, 14], [3, 1, 14]
    rows = g.standard_normal((12, page, dl + dr))
    table = np.array([[3, 0, 11, -1], [5, -1, -1, -1], [1, 2, 9, 4]])
    begin = np.concatenate([[0], np.cumsum(new)])
    q = g.standard_normal((begin[-1], H, dl + dr))
    out, lse, touched = P.paged_mla(q, rows, table, begin, lens, page, dl, 0.3)
    assert touched.all()
    for b in range(3):
        k = -(-lens[b] // page)
        key = torch.from_numpy(rows[table[b, :k]].reshape(-1, dl + dr)[: lens[b]])
        qb = torch.from_numpy(q[begin[b]:begin[b + 1]]).transpose(0, 1)
        mask = torch.arange(lens[b])[None, :] <= torch.arange(lens[b] - new[b], lens[b])[:, None]
        ref = torch.nn.functional.scaled_dot_product_attention(qb, key.expand(H, -1, -1), key[:, :dl].expand(H, -1, -1),
                                                               attn_mask=mask, scale=0.3)
        np.testing.assert_allclose(out[begin[b]:begin[b + 1]], ref.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)
        logit = (0.3 * qb @ key.T).masked_fill(~mask, -np.inf)
        np.testing.assert_allclose(lse[begin[b]:begin[b + 1]], torch.logsumexp(logit, -1).T.numpy(), rtol=1e-12)


def test_unpack_fp8_matches_torch():
    g = torch.Generator().manual_seed(1)
    c = torch.randn(5, 512, generator=g)
    sigma = c.abs().amax(-1, keepdim=True) / 448
    codes = (c / sigma).to(torch.float8_e4m3fn)
    rope = torch.randn(5, 64, generator=g).bfloat16()
    raw = torch.zeros(5, 656, dtype=torch.uint8)
    raw[:, :512], raw[:, 512:640], raw[:, 640:644] = codes.view(torch.uint8), rope.view(torch.uint8), sigma.view(torch.uint8)
    decode = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    want = torch.cat([codes.double() * sigma.double(), rope.double()], -1).numpy()
    np.testing.assert_array_equal(P.unpack_fp8(raw.numpy(), decode), want)


def test_verified_tokens_follow_the_target():
    """Sum over the draft's choice and a grid of both random numbers: the first
    emitted token's distribution is p_0, within the grid's resolution."""
    p = np.array([0.5, 0.25, 0.0, 0.25])
    q = np.array([0.125, 0.25, 0.25, 0.375])
    K = 64
    grid = (np.arange(K) + 0.5) / K
    au, su = [a.ravel() for a in np.meshgrid(grid, grid)]
    target = np.broadcast_to(np.stack([p, p]), (K * K, 2, 4))
    draft = np.broadcast_to(q[None], (K * K, 1, 4))
    got = np.zeros(4)
    for x in range(4):
        tok, _ = P.verify_drafts(target, draft, np.full((K * K, 1), x), None, au[:, None], su)
        got += q[x] * np.bincount(tok[:, 0], minlength=4) / (K * K)
    np.testing.assert_allclose(got, p, atol=2.0 / K)


def test_verify_by_hand():
    # greedy draft of token 1: accepted at u < p(1) = 0.25, else drawn from the rest
    t = np.array([[[0.5, 0.25, 0.25], [0.0, 0.0, 1.0]]])
    x = np.array([[1]])
    run = lambda u, s: [a.tolist() for a in P.verify_drafts(t, None, x, None, [[u]], [s])]
    assert run(0.2, 0.9) == [[[1, 2]], [1]]
    assert run(0.25, 0.6) == [[[0, -1]], [0]]      # rest (0.5, 0, 0.25): 0.6 * 0.75 = 0.45 < 0.5
    assert run(0.25, 0.7) == [[[2, -1]], [0]]
    # no weight left where p <= q: drawn from p; no weight at all: -1
    same = np.array([[[0.5, 0.5, 0.0]]])
    tok, acc = P.verify_drafts(np.concatenate([same, same], 1), same, np.array([[2]]), None, [[0.5]], [0.75])
    assert tok.tolist() == [[1, -1]] and acc.tolist() == [0]
    tok, _ = P.verify_drafts(np.zeros((1, 1, 3)), None, np.zeros((1, 0), int), None, np.zeros((1, 0)), [0.5])
    assert tok.tolist() == [[-1]]
    # an inverse cumulative weight that meets the border takes the next token
    even = np.array([[[0.25, 0.25, 0.5]]])
    tok, _ = P.verify_drafts(even, None, np.zeros((1, 0), int), None, np.zeros((1, 0)), [0.5])
    assert tok.tolist() == [[2]]
