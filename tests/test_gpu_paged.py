"""Paged caches through the C ABI against the float64 oracle (oracle/paged.py):
page tables and slot maps, the cache-row writer through a slot map, attention of
new tokens over a paged latent cache, and a serving step made of all of them.

Attention tolerance, per output element: with p the softmax weights and
A = sum_s p_s |c_s|, rounding each weight to bf16 (half a step: 2^-8 relative)
moves the output by at most 2^-8 A; logits summed in float32 over 576 products
are off by at most 576 * 2^-24 * scale * sum |q c| < 1e-3 for these inputs
(sum |q c| < 460 at N(0, 1), scale 1/16), which moves every weight by at most 1e-3
relative and the output by 2e-3 A; the float32 sums add less than 1e-4 A.  The
output's own rounding is 2^-8 |o|.  Packed FP8 rows: the weight times the row
scale is rounded to fp16 (2^-11), less than the bf16 case.  lse: 1e-3 (logits)."""
import numpy as np
import pytest
import torch

from dsa_indexer_top_b200 import binding as B
from oracle import paged as P
from oracle import producers as PR

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a), dtype=np.int32)).to(DEV)


# ------------------------------------------------------------------ page tables
def _plan(ctx, new, held, table, free, free_begin, page, n_pages, n_tok, fill=-9):
    n = len(ctx)
    e = lambda k: torch.full((k,), fill, dtype=torch.int32, device=DEV)
    t = _i32(table)
    return B.PagePlan(_i32(ctx), _i32(new), _i32(held), _i32(free), None if free_begin is None else _i32([free_begin]),
                      t, e(n + 1), e(n), e(n_tok), e(n_tok), e(n_tok), e(n), e(1), n_pages=n_pages, page_rows=page)


def _layout(rng, ctx, new, page, reserve=0.2):
    ctx, new = np.asarray(ctx), np.asarray(new)
    held = -(-ctx // page) + (rng.random(len(ctx)) < reserve)
    need = np.maximum(held, -(-(ctx + new) // page))
    n_pages = int(need.sum()) + 4
    perm = rng.permutation(n_pages)
    table = np.full((len(ctx), int(need.max(initial=0)) + 1), -1)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        at += int(h)
    return held, table, perm[at:], n_pages


CHECKS = ("q_begin", "seq_len", "q_seq", "q_pos", "slot_map", "held_out")


@pytest.mark.parametrize("n_seq,new_hi,ctx_hi,page,pad", [
    (1, 1, 1, 1, 0), (1, 900, 0, 16, 5), (64, 1, 32767, 64, 0), (300, 40, 900, 8, 17), (1500, 3, 50, 16, 100),
    (5000, 2, 30, 128, 0), (7, 9000, 5, 24, 1), (33, 0, 70, 16, 3)])
def test_page_tables(cuda_ok, n_seq, new_hi, ctx_hi, page, pad):
    rng = np.random.default_rng(n_seq + page)
    ctx, new = rng.integers(0, ctx_hi + 1, n_seq), rng.integers(0, new_hi + 1, n_seq)
    held, table, free, n_pages = _layout(rng, ctx, new, page)
    begin = 2
    free = np.concatenate([[-1, -1], free])
    n_tok = int(new.sum()) + pad
    p = _plan(ctx, new, held, table, free, begin, page, n_pages, n_tok)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    want = P.page_tables(ctx, new, held, free, begin, table, page, n_tok)
    for _ in range(2):       # a repeated call gives the same
        B.dsa_page_tables(p, ws)
        assert B.dsa_check_status(ws) == B.DSA_OK
        np.testing.assert_array_equal(p.block_table.cpu().numpy(), want["table"])
        for k in CHECKS:
            np.testing.assert_array_equal(getattr(p, k).cpu().numpy(), want[k], err_msg=k)
        assert int(p.free_used) == want["free_used"]


def test_page_tables_strided_table_and_no_sequences(cuda_ok):
    rng = np.random.default_rng(5)
    ctx, new = [10, 3], [9, 0]
    held, table, free, n_pages = _layout(rng, ctx, new, 4)
    p = _plan(ctx, new, held, table, free, None, 4, n_pages, 9)
    wide = torch.full((2, 40), -7, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = p.block_table
    p.block_table = wide[:, :table.shape[1]]
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    B.dsa_page_tables(p, ws)
    want = P.page_tables(ctx, new, held, free, 0, table, 4, 9)
    np.testing.assert_array_equal(p.block_table.cpu().numpy(), want["table"])
    assert (wide[:, table.shape[1]:] == -7).all()
    empty = _plan([], [], [], np.zeros((0, 1)), [], None, 4, 10, 3)
    B.dsa_page_tables(empty, ws)
    assert B.dsa_check_status(ws) == B.DSA_OK
    assert empty.q_begin.tolist() == [0] and empty.slot_map.tolist() == [-1] * 3 and int(empty.free_used) == 0


def test_page_tables_report_bad_input(cuda_ok):
    """Every error keeps to the buffers: missing pages give -1, lengths are clamped."""
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)

    def run(ctx, new, held, table, free, begin=0, n_pages=20, n_tok=8):
        p = _plan(ctx, new, held, table, free, begin, 4, n_pages, n_tok)
        B.dsa_page_tables(p, ws)
        return p, B.dsa_check_status(ws)

    p, s = run([4], [6], [1], [[3, -1, -1]], [7])                       # one page short
    assert s == B.DSA_ERR_INVALID and p.block_table.tolist() == [[3, 7, -1]]
    assert p.slot_map.tolist() == [28, 29, 30, 31, -1, -1, -1, -1] and int(p.free_used) == 1
    p, s = run([0], [2], [0], [[-1]], [25])                             # a page outside the pool
    assert s == B.DSA_ERR_INVALID and p.slot_map.tolist()[:2] == [-1, -1]
    p, s = run([2], [2], [1], [[99]], [5])                              # a held page outside the pool
    assert s == B.DSA_ERR_INVALID and p.slot_map.tolist()[:2] == [-1, -1]
    p, s = run([0], [7], [0], [[-1]], [5, 6])                           # longer than the table
    assert s == B.DSA_ERR_INVALID and p.slot_map.tolist()[:7] == [20, 21, 22, 23, -1, -1, -1]
    assert p.held_out.tolist() == [1]
    p, s = run([-3, 1], [-1, 1], [-1, 1], [[-1], [2]], [5])             # negative lengths
    assert s == B.DSA_ERR_INVALID and p.q_begin.tolist() == [0, 0, 1] and p.slot_map.tolist()[0] == 9
    p, s = run([0, 0], [6, 6], [0, 0], [[-1, -1], [-1, -1]], [1, 2, 3, 4])  # more tokens than capacity
    assert s == B.DSA_ERR_INVALID and p.q_begin.tolist() == [0, 6, 8] and p.slot_map.tolist() == [4, 5, 6, 7, 8, 9, 12, 13]
    p, s = run([0], [1], [0], [[-1]], [1], begin=-5)                    # a bad list start hands out nothing
    assert s == B.DSA_ERR_INVALID and p.slot_map.tolist()[0] == -1 and int(p.free_used) == 0
    p, s = run([2**31 - 1], [5], [0], [[-1]], [1])                      # length past int32
    assert s == B.DSA_ERR_INVALID


# ------------------------------------------------------------------ writer
@pytest.mark.parametrize("n_tok,page", [(1, 16), (4, 16), (5, 8), (7, 8), (16, 64), (40, 24), (300, 64), (1030, 16)])
def test_write_paged_rows(cuda_ok, n_tok, page):
    """The oracle's rows at the slots; nothing else written."""
    rng = np.random.default_rng(n_tok)
    g = torch.Generator(device=DEV).manual_seed(n_tok)
    H = 640
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    h, w = rn(n_tok, H).bfloat16(), (rn(704, H) / H ** 0.5).bfloat16()
    norms = (1 + 0.1 * rn(512), 1 + 0.1 * rn(128), 0.1 * rn(128))
    pos = _i32(rng.choice(1 << 20, n_tok, replace=False))
    n_pages = -(-n_tok // page) + 2
    slots = rng.permutation(n_pages * page)[:n_tok]
    slots[n_tok // 2::5] = -1
    kv = torch.full((n_pages, page, 592), float("nan"), dtype=torch.bfloat16, device=DEV)
    kidx = torch.full((n_pages, page + 1, 128), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :page]
    ws = torch.zeros(B.dsa_cache_writer_workspace_bytes(n_tok, H), dtype=torch.uint8, device=DEV)
    B.dsa_write_paged_rows(B.CacheWriter(h, w, *norms, None, pos, kv, kidx), _i32(slots), ws)
    assert B.dsa_check_status(ws) == B.DSA_OK
    hf, wf = h.float().cpu().numpy(), w.float().cpu().numpy()
    p64 = pos.cpu().numpy()
    rows = PR.latent_rows(hf, wf[:576].T, norms[0].cpu().numpy(), p64)
    keys = PR.indexer_keys(hf, wf[576:].T, norms[1].cpu().numpy(), norms[2].cpu().numpy(), p64)
    # rows N(0, 1): bf16 half step 2^-8 relative plus float32 sums (1e-5 of them)
    for got_pool, ref64 in ((kv, rows), (kidx, keys)):
        got = got_pool.float().cpu().numpy()
        mask = np.zeros((n_pages, page), dtype=bool)
        for i, s in enumerate(slots):
            if s >= 0:
                mask[s // page, s % page] = True
                row = got[s // page, s % page, :ref64.shape[1]]
                assert (np.abs(row - ref64[i]) <= 2.0 ** -8 * np.abs(ref64[i]) + 5e-5).all()
        assert np.isnan(got[~mask]).all()
    assert torch.isnan(kv[..., 576:].float()).all()


def test_write_paged_rows_bad_slots(cuda_ok):
    H, n = 64, 4
    h, w = torch.ones(n, H, device=DEV).bfloat16(), torch.ones(704, H, device=DEV).bfloat16()
    norms = (torch.ones(512, device=DEV), torch.ones(128, device=DEV), torch.zeros(128, device=DEV))
    ws = torch.zeros(B.dsa_cache_writer_workspace_bytes(n, H), dtype=torch.uint8, device=DEV)
    for slots, pos, written in (([3, -2, 8, 5], [0, 1, 2, 3], [3, 5]), ([0, 1, 2, 3], [0, -1, 2, 3], [0, 2, 3])):
        kv = torch.full((2, 4, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
        B.dsa_write_paged_rows(B.CacheWriter(h, w, *norms, None, _i32(pos), kv, None), _i32(slots), ws)
        assert B.dsa_check_status(ws) == B.DSA_ERR_INVALID
        done = ~torch.isnan(kv.float()).any(-1).flatten()
        assert done.nonzero().flatten().tolist() == written


# ------------------------------------------------------------------ attention
DECODE = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()


class Case:
    """Inputs of one attention call; unused pool rows hold NaN."""

    def __init__(self, seqs, heads=64, page=16, kind="bf16", d_lat=512, d_rope=64, seed=0, row_pad=0, page_pad=0,
                 lead=0, tail=0, table_pad=0, scale=1 / 16, hot=0.0, lse=True):
        rng = np.random.default_rng([seed, len(seqs), heads, page])
        g = torch.Generator(device=DEV).manual_seed(seed + 17)
        self.ctx, self.new = [c for c, _ in seqs], [n for _, n in seqs]
        total = np.array(self.ctx) + np.array(self.new)
        need = -(-total // page)
        n_pages = int(need.sum()) + 2
        dk = d_lat + d_rope
        perm = rng.permutation(n_pages)
        self.table = np.full((len(seqs), int(need.max()) + table_pad), -1)
        live = np.zeros((n_pages, page), dtype=bool)
        at = 0
        for b, k in enumerate(need):
            self.table[b, :k] = perm[at:at + k]
            for s in range(int(total[b])):
                live[self.table[b, s // page], s % page] = True
            at += int(k)
        n_tok = lead + int(np.sum(self.new)) + tail
        self.begin = lead + np.concatenate([[0], np.cumsum(self.new)])
        dt = torch.float32 if kind == "f32" else torch.bfloat16
        rows = torch.randn(n_pages, page, dk, generator=g, device=DEV)
        if hot:  # logits that grow along the sequence: the running maximum moves
            rows *= (1 + hot * torch.rand(n_pages, page, 1, generator=g, device=DEV) ** 6)
        rows = rows.to(dt)
        q = torch.randn(n_tok, heads, dk, generator=g, device=DEV).to(dt)
        live_t = torch.from_numpy(live).to(DEV)
        if kind == "fp8":
            c = rows[..., :d_lat].float()
            sigma = c.abs().amax(-1, keepdim=True) / 448
            raw = torch.full((n_pages, page + page_pad, 656 + row_pad), 0xFF, dtype=torch.uint8, device=DEV)  # NaN codes
            raw[:, :page, :d_lat] = (c / sigma).to(torch.float8_e4m3fn).view(torch.uint8)
            raw[:, :page, d_lat:d_lat + 128] = rows[..., d_lat:].contiguous().view(torch.uint8)
            raw[:, :page, 640:644] = sigma.contiguous().view(torch.uint8)
            raw[:, :page][~live_t] = 0xFF
            self.pool = raw[:, :page]
            self.rows = P.unpack_fp8(np.where(live[..., None], raw[:, :page].cpu().numpy(), 0), DECODE)
        else:
            pool = torch.full((n_pages, page + page_pad, dk + row_pad), float("nan"), dtype=dt, device=DEV)
            pool[:, :page, :dk] = torch.where(live_t[..., None], rows, float("nan"))
            self.pool = pool[:, :page]
            self.rows = torch.where(live_t[..., None], rows, 0).double().cpu().numpy()
        self.q, self.page, self.n_pages, self.n_tok, self.d_lat, self.scale = q, page, n_pages, n_tok, d_lat, scale
        self.kind, self.heads, self.total = kind, heads, total
        self.out = torch.full((n_tok, heads, d_lat), 77.0, dtype=dt, device=DEV)
        self.lse = torch.full((n_tok, heads), 77.0, dtype=torch.float32, device=DEV) if lse else None
        self.batch = B.PagedBatch(_i32(self.table), _i32(self.begin), _i32(total), n_tok, n_pages, page)
        self.mla = B.Mla(q, self.pool, self.out, d_lat, scale, self.lse)
        self.ws = B.paged_workspace(self.batch, self.mla)

    def run(self, status=B.DSA_OK, stream=None):
        B.dsa_paged_mla(self.batch, self.mla, self.ws, stream)
        assert B.dsa_check_status(self.ws) == status
        return self

    def check(self, table=None, total=None, skip=(), nan=(), any_value=()):
        """skip: sequences left alone; nan: tokens whose row is NaN; any_value: tokens not compared."""
        table = self.table if table is None else table
        q = self.q.double().cpu().numpy()
        want, lse, touched = P.paged_mla(q, self.rows, table, self.begin, self.total, self.page, self.d_lat, self.scale)
        mag = self._weighted_abs(q, table)
        for b in skip:
            touched[self.begin[b]:self.begin[b + 1]] = False
        got = self.out.double().cpu().numpy()
        assert (got[~touched] == 77).all(), "rows outside the sequences were written"
        left = ~touched
        for i in nan:
            assert np.isnan(got[i]).all()
            assert self.lse is None or torch.isnan(self.lse[i]).all()
        touched[list(nan) + list(any_value)] = False
        half = 2.0 ** -24 if self.kind == "f32" else 2.0 ** -8
        tol = half * np.abs(want) + (2.1e-3 + (0 if self.kind == "f32" else 2.0 ** -8)) * mag + 1e-6
        err = np.abs(got - want)[touched] / tol[touched]
        assert np.isfinite(got[touched]).all() and err.max(initial=0) <= 1, f"{err.max():.3f} of the tolerance"
        if self.lse is not None:
            gl = self.lse.double().cpu().numpy()
            assert (gl[left] == 77).all()
            seen = np.isfinite(lse) & touched[:, None]
            assert (np.abs(gl[seen] - lse[seen]) <= 1e-3).all()
            assert (gl[touched[:, None] & ~np.isfinite(lse)] == -np.inf).all()
        return self

    def _weighted_abs(self, q, table):
        """sum_s p_s |c_s| per output element."""
        out = np.zeros((self.n_tok, self.heads, self.d_lat))
        for b in range(len(self.total)):
            for i in range(int(self.begin[b]), int(self.begin[b + 1])):
                seen = int(self.total[b]) - (int(self.begin[b + 1]) - i) + 1
                pg = np.asarray(table[b])[np.arange(seen) // self.page]
                ok = (pg >= 0) & (pg < self.n_pages)
                key = self.rows[pg[ok], np.arange(seen)[ok] % self.page]
                if len(key):
                    x = self.scale * (q[i] @ key.T)
                    e = np.exp(x - x.max(-1, keepdims=True))
                    out[i] = (e / e.sum(-1, keepdims=True)) @ np.abs(key[:, :self.d_lat])
        return out


EDGES = [(0, 1), (0, 2), (1, 1), (62, 1), (63, 1), (64, 1), (126, 1), (127, 1), (128, 1), (255, 2), (300, 3)]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,page", [(64, 64), (64, 16), (16, 32), (128, 64), (1, 8), (5, 128), (48, 256)])
def test_attention_edges(cuda_ok, kind, heads, page):
    """Sequences of one row up to a few hundred, at the borders of 64 and 128 rows, in one call."""
    Case(EDGES, heads=heads, page=page, kind=kind, seed=1).run().check()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("heads,seqs", [
    (64, [(0, 130)]), (64, [(77, 65), (0, 1), (500, 33)]), (16, [(129, 100), (3, 17)]), (128, [(40, 21)]),
    (7, [(10, 80), (200, 19)]), (33, [(64, 9)])])
def test_attention_chunks(cuda_ok, kind, heads, seqs):
    """Causal chunks: new tokens attend over one another too; tiles that end inside a token run."""
    Case(seqs, heads=heads, page=16, kind=kind, seed=2).run().check()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("seqs,page", [([(20000, 1)], 64), ([(5000, 2), (9, 1), (3333, 1)], 16), ([(1900, 1)] * 9, 128)])
def test_attention_long_rows_are_split_and_joined(cuda_ok, kind, seqs, page):
    Case(seqs, heads=64, page=page, kind=kind, seed=3, hot=1.5).run().check()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_attention_strides_and_outer_rows(cuda_ok, kind):
    """Padded rows, pages and table rows; query rows before the first and behind the last sequence."""
    Case([(100, 3), (0, 1), (31, 2)], heads=64, page=16, kind=kind, row_pad=16, page_pad=3, table_pad=5, lead=4, tail=7,
         seed=4).run().check()


def test_attention_without_lse_and_with_empty_sequences(cuda_ok):
    Case([(0, 0), (50, 1), (40, 0), (9, 4), (0, 0)], heads=64, page=16, seed=5, lse=False).run().check()


@pytest.mark.parametrize("heads,d_lat,d_rope,kind,page", [
    (4, 64, 16, "f32", 16), (3, 96, 0, "f32", 5), (200, 512, 64, "bf16", 16), (4, 64, 16, "bf16", 16),
    (64, 512, 64, "bf16", 5), (2, 512, 64, "fp8", 12)])
def test_attention_other_shapes(cuda_ok, heads, d_lat, d_rope, kind, page):
    """float32, other dims, more heads than a tile, pages that are no multiple of eight rows."""
    Case([(0, 1), (140, 6), (300, 1)], heads=heads, page=page, kind=kind, d_lat=d_lat, d_rope=d_rope, seed=6).run().check()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "f32"])
def test_attention_missing_pages(cuda_ok, kind):
    """Pages outside the pool are rows nobody sees; a token left with none gives 0 and -inf."""
    shape = dict(d_lat=64, d_rope=16) if kind == "f32" else {}
    c = Case([(200, 2), (20, 1), (150, 1)], heads=64 if kind != "f32" else 4, page=16, kind=kind, seed=7, **shape)
    c.table[0, 3] = -1
    c.table[0, 9] = c.n_pages + 1000000
    c.table[1, :] = -1
    c.batch.block_table = _i32(c.table)
    c.run(B.DSA_ERR_INVALID).check()


@pytest.mark.parametrize("kind,what", [("bf16", "nan"), ("bf16", "inf"), ("f32", "nan"), ("fp8", "nan"),
                                       ("fp8", "scale nan"), ("fp8", "scale inf")])
@pytest.mark.parametrize("heads", [16, 64])
def test_attention_later_rows_that_are_not_finite(cuda_ok, kind, what, heads):
    """A row with NaN or infinities is NaN in the tokens that see it and nothing in those before it."""
    seqs = [(100, 7), (0, 3), (126, 4), (1500, 20), (300, 1)]
    where = [103, 1, 128, 1500, None]                # the row of each sequence
    shape = dict(d_lat=64, d_rope=16) if kind == "f32" else {}
    c = Case(seqs, heads=heads, page=16, kind=kind, seed=13, **shape)
    nan = []
    for b, s in enumerate(where):
        if s is None:
            continue
        at = c.table[b, s // 16], s % 16
        c.rows[at] = 0
        if kind != "fp8":
            c.pool[at][5:8] = float("nan") if what == "nan" else float("inf")
        elif what == "nan":
            c.pool[at][5:8] = 0x7F
        else:
            c.pool[at][640:644] = torch.tensor([float(what.split()[1])], device=DEV).view(torch.uint8)
        nan += range(int(c.begin[b]) + s - c.ctx[b], int(c.begin[b + 1]))
    # (an infinite row's logit may also be -infinity)
    c.run().check(**{"nan" if "nan" in what else "any_value": nan})


@pytest.mark.parametrize("heads", [8, 64])
def test_attention_fp8_rows_without_latent_part(cuda_ok, heads):
    """A scale of zero: the latent part is zero, the RoPE part counts; scales far apart."""
    c = Case([(300, 1), (128, 2), (200, 5), (20, 1)], heads=heads, page=16, kind="fp8", seed=14)
    for b, rows in enumerate([[0, 5, 130, 299, 300], list(range(130)), [203, 7], list(range(21))]):
        for s in rows:
            at = c.table[b, s // 16], s % 16
            # scale 0; every other row 2^-60 of what it was
            f = 0.0 if s % 2 or b == 3 else 2.0 ** -60
            c.pool[at][640:644] = (c.pool[at][640:644].view(torch.float32) * f).view(torch.uint8)
            c.rows[at][:512] *= f
    c.run().check()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_attention_lengths_at_the_end_of_int32(cuda_ok, kind):
    """Positions past int32's end are refused; nothing of that sequence is read or written."""
    shape = dict(d_lat=64, d_rope=16) if kind == "f32" else {}
    c = Case([(30, 2), (40, 1)], heads=4, page=16, kind=kind, seed=15, **shape)
    wide = torch.zeros(2, (1 << 27) + 1, dtype=torch.int32, device=DEV)   # page 0 wherever it is read
    wide[:, :c.table.shape[1]] = _i32(c.table)
    c.batch.block_table = wide
    for length in (2 ** 31 - 1, 2 ** 31 - 1025):
        c.batch.seq_len = _i32([length, 41])
        c.run(B.DSA_ERR_INVALID).check(skip=[0])


def test_attention_bad_sequences_are_skipped(cuda_ok):
    c = Case([(30, 2), (40, 1), (50, 1)], heads=64, page=16, seed=8)
    for bad in (1, 5000):        # shorter than its new tokens; longer than its table
        lens = c.total.copy()
        lens[0] = bad
        c.out.fill_(77.0)
        c.lse.fill_(77.0)
        c.batch.seq_len = _i32(lens)
        c.run(B.DSA_ERR_INVALID).check(skip=[0])


def test_attention_many_sequences(cuda_ok):
    rng = np.random.default_rng(9)
    Case([(int(rng.integers(0, 90)), int(rng.integers(0, 3))) for _ in range(700)], heads=8, page=16, seed=9).run().check()


def test_attention_one_page_twice_and_shared_prefix(cuda_ok):
    """Two sequences over the same pages, and a table that names one page twice."""
    c = Case([(127, 1), (127, 1)], heads=64, page=32, seed=10)
    c.table[1] = c.table[0]
    c.table[1, 2] = c.table[1, 1]
    c.batch.block_table = _i32(c.table)
    c.run().check()


def test_attention_second_call_stream_and_graph(cuda_ok):
    """Repeated calls agree bit for bit; on another stream; captured and replayed on new lengths."""
    c = Case([(700, 1), (90, 2), (1500, 1)], heads=64, page=16, seed=11).run().check()
    first = c.out.clone()
    c.run()
    assert torch.equal(first, c.out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.out.fill_(77.0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        B.dsa_paged_mla(c.batch, c.mla, c.ws)
    s.synchronize()
    assert torch.equal(first, c.out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.dsa_paged_mla(c.batch, c.mla, c.ws)
    c.total = c.total - np.array([333, 0, 64])
    c.batch.seq_len.copy_(_i32(c.total))
    graph.replay()
    torch.cuda.synchronize()
    assert B.dsa_check_status(c.ws) == B.DSA_OK
    c.check()


def test_attention_calls_at_the_same_time(cuda_ok):
    """Calls on three streams, each with a workspace of its own, give what they give alone."""
    cases = [Case([(900, 1), (3000, 2), (70, 40)], heads=64, page=16, kind=k, seed=16 + i)
             for i, k in enumerate(["bf16", "fp8", "bf16"])]
    alone = [c.run().out.clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        for c in cases:
            c.out.fill_(77.0)
        torch.cuda.synchronize()
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                B.dsa_paged_mla(c.batch, c.mla, c.ws)
        torch.cuda.synchronize()
        for c, want in zip(cases, alone):
            assert B.dsa_check_status(c.ws) == B.DSA_OK and torch.equal(c.out, want)


def test_attention_two_graphs_share_a_workspace(cuda_ok):
    """Two captured calls over one workspace, replayed in turn on one stream."""
    a = Case([(2000, 1), (31, 2)], heads=64, page=16, kind="fp8", seed=19).run().check()
    b = Case([(5, 60), (1100, 1), (64, 1)], heads=16, page=32, seed=20).run().check()
    ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    want = [a.out.clone(), b.out.clone()]
    graphs = []
    for c in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            B.dsa_paged_mla(c.batch, c.mla, ws)
    for _ in range(3):
        a.out.fill_(77.0)
        b.out.fill_(77.0)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert B.dsa_check_status(ws) == B.DSA_OK
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_tables_and_rows_captured(cuda_ok):
    """Tables and rows in one graph, replayed on other lengths: rows at the new slots."""
    rng = np.random.default_rng(22)
    page, n_tok, H = 16, 40, 256
    ctx, new = np.array([30, 0, 7]), np.array([9, 20, 3])
    held, table, free, n_pages = _layout(rng, ctx, new, page)
    free = np.concatenate([free, free])                     # (room for either step's pages)
    table = np.concatenate([table, np.full((3, 2), -1)], 1)
    p = _plan(ctx, new, held, table, free, 0, page, n_pages, n_tok)
    g = torch.Generator(device=DEV).manual_seed(22)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    h, w = rn(n_tok, H).bfloat16(), (rn(704, H) / H ** 0.5).bfloat16()
    norms = (1 + 0.1 * rn(512), 1 + 0.1 * rn(128), 0.1 * rn(128))
    kv = torch.empty(n_pages, page, 576, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(max(256, B.dsa_cache_writer_workspace_bytes(n_tok, H)), dtype=torch.uint8, device=DEV)
    writer = B.CacheWriter(h, w, *norms, None, p.q_pos, kv, None)

    def step():
        B.dsa_page_tables(p, ws)
        B.dsa_write_paged_rows(writer, p.slot_map, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for c2, n2 in ((ctx, new), (ctx - [1, 0, 7], np.array([2, 1, 31]))):
        p.ctx_len.copy_(_i32(c2))
        p.new_len.copy_(_i32(n2))
        p.block_table.copy_(_i32(table))
        kv.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert B.dsa_check_status(ws) == B.DSA_OK
        want = P.page_tables(c2, n2, held, free, 0, table, page, n_tok)
        for k in CHECKS:
            np.testing.assert_array_equal(getattr(p, k).cpu().numpy(), want[k], err_msg=k)
        rows = PR.latent_rows(h.float().cpu().numpy(), w[:576].float().cpu().numpy().T, norms[0].cpu().numpy(), want["q_pos"])
        got = kv.flatten(0, 1).double().cpu().numpy()
        slots = want["slot_map"][:int(n2.sum())]
        assert (np.abs(got[slots] - rows[:len(slots)]) <= 2.0 ** -8 * np.abs(rows[:len(slots)]) + 5e-5).all()
        got[slots] = np.nan
        assert np.isnan(got).all()


def test_attention_far_offsets(cuda_ok):
    """Pages whose byte and element offsets pass 32 bits."""
    page, n_pages = 64, 62000                      # 62000 * 64 * 576 = 2.29e9 elements, 4.6 GB
    pool = torch.empty(n_pages, page, 576, dtype=torch.bfloat16, device=DEV)
    use = [n_pages - 1, n_pages - 2, 1, 31000]
    g = torch.Generator(device=DEV).manual_seed(12)
    rows = torch.randn(4, page, 576, generator=g, device=DEV).bfloat16()
    pool[use] = rows
    q = torch.randn(1, 64, 576, generator=g, device=DEV).bfloat16()
    out = torch.empty(1, 64, 512, dtype=torch.bfloat16, device=DEV)
    batch = B.PagedBatch(_i32([use]), _i32([0, 1]), _i32([250]), 1, n_pages, page)
    mla = B.Mla(q, pool, out, 512, 1 / 16)
    ws = B.paged_workspace(batch, mla)
    B.dsa_paged_mla(batch, mla, ws)
    assert B.dsa_check_status(ws) == B.DSA_OK
    want, _, _ = P.paged_mla(q.double().cpu().numpy(), rows.double().cpu().numpy(), [[0, 1, 2, 3]], [0, 1], [250], page,
                             512, 1 / 16)
    # weights of about 1/250 over N(0, 1) values: A < 1
    assert np.abs(out.double().cpu().numpy() - want).max() <= 2.0 ** -7 + 2.1e-3


# ------------------------------------------------------------------ a serving step
def test_serving_step(cuda_ok):
    """Two steps of a small server: tables, rows, absorbed queries, attention and
    verification, the second step on the lengths the verification left."""
    g = torch.Generator(device=DEV).manual_seed(21)
    rng = np.random.default_rng(21)
    hidden, heads, page, n_seq, V, D = 256, 64, 16, 3, 50, 2
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    w = (rn(704, hidden) / hidden ** 0.5).bfloat16()
    norms = (1 + 0.1 * rn(512), 1 + 0.1 * rn(128), 0.1 * rn(128))
    w_uk = (rn(heads, 512, 192) / 192 ** 0.5).bfloat16()
    n_pages, width = 40, 8
    pool = torch.full((n_pages, page, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    table = torch.full((n_seq, width), -1, dtype=torch.int32, device=DEV)
    free = _i32(rng.permutation(n_pages))
    ctx, held, head = _i32([0, 0, 0]), _i32([0, 0, 0]), _i32([0])
    history = [np.zeros((0, 576)) for _ in range(n_seq)]       # each sequence's cache rows, float64
    news = [[35, 1, 18], [D + 1] * 3]
    for new in news:
        n_tok = sum(new) + 2                                   # two padding rows
        e = lambda k: torch.empty(k, dtype=torch.int32, device=DEV)
        plan = B.PagePlan(ctx, _i32(new), held, free, head, table, e(n_seq + 1), e(n_seq), e(n_tok), e(n_tok), e(n_tok),
                          e(n_seq), e(1), n_pages=n_pages, page_rows=page)
        ws = torch.zeros(max(256, B.dsa_cache_writer_workspace_bytes(n_tok, hidden)), dtype=torch.uint8, device=DEV)
        h = rn(n_tok, hidden).bfloat16()
        q_nope, q_rope = rn(n_tok, heads, 192).bfloat16(), rn(n_tok, heads, 64).bfloat16()
        q = torch.empty(n_tok, heads, 576, dtype=torch.bfloat16, device=DEV)
        out = torch.full((n_tok, heads, 512), 77.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((n_tok, heads), 77.0, device=DEV)
        B.dsa_page_tables(plan, ws)
        B.dsa_write_paged_rows(B.CacheWriter(h, w, *norms, None, plan.q_pos, pool, None), plan.slot_map, ws)
        B.dsa_absorb_queries(q_nope, q_rope, w_uk, plan.q_pos, 8e6, q, ws)
        batch = B.PagedBatch(table, plan.q_begin, plan.seq_len, n_tok, n_pages, page)
        mla = B.Mla(q, pool, out, 512, 1 / 16, lse)
        aws = B.paged_workspace(batch, mla)
        B.dsa_paged_mla(batch, mla, aws)
        assert B.dsa_check_status(ws) == B.DSA_OK and B.dsa_check_status(aws) == B.DSA_OK
        assert (out[sum(new):] == 77).all() and (lse[sum(new):] == 77).all()
        # the rows, read back from the pool as bf16, against the oracle's; then dense attention over them
        begin, pos = plan.q_begin.cpu().numpy(), plan.q_pos.cpu().numpy()
        want_rows = PR.latent_rows(h.float().cpu().numpy(), w[:576].float().cpu().numpy().T, norms[0].cpu().numpy(), pos)
        tab = table.cpu().numpy()
        for b in range(n_seq):
            c0 = int(ctx[b])
            assert pos[begin[b]:begin[b + 1]].tolist() == list(range(c0, c0 + new[b]))
            got = pool[tab[b, :-(-(c0 + new[b]) // page)].tolist()].flatten(0, 1)[:c0 + new[b]].double().cpu().numpy()
            wr = want_rows[begin[b]:begin[b + 1]]
            assert (np.abs(got[c0:] - wr) <= 2.0 ** -8 * np.abs(wr) + 5e-5).all()
            np.testing.assert_array_equal(got[:c0], history[b][:c0])   # earlier rows stay
            history[b] = got
            for i in range(begin[b], begin[b + 1]):
                key = got[:pos[i] + 1]
                x = q[i].double().cpu().numpy() @ key.T / 16
                p = np.exp(x - x.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                o, mag = p @ key[:, :512], p @ np.abs(key[:, :512])
                err = np.abs(out[i].double().cpu().numpy() - o)
                assert (err <= 2.0 ** -8 * np.abs(o) + (2.1e-3 + 2.0 ** -8) * mag + 1e-6).all()
        if new is news[-1]:
            break
        # drafts verified: the next step's lengths
        tgt = torch.softmax(rn(n_seq, D + 1, V), -1)
        drf = torch.softmax(rn(n_seq, D, V), -1)
        x = _i32(rng.integers(0, V, (n_seq, D)))
        au, su = torch.rand(n_seq, D, generator=g, device=DEV), torch.rand(n_seq, generator=g, device=DEV)
        tok, acc = torch.empty(n_seq, D + 1, dtype=torch.int32, device=DEV), torch.empty(n_seq, dtype=torch.int32, device=DEV)
        B.dsa_verify_drafts(tgt, x, au, su, tok, acc, ws, draft=drf)
        assert B.dsa_check_status(ws) == B.DSA_OK
        wt, wa = P.verify_drafts(tgt.cpu().numpy(), drf.cpu().numpy(), x.cpu().numpy(), None, au.cpu().numpy(), su.cpu().numpy())
        np.testing.assert_array_equal(tok.cpu().numpy(), wt)
        np.testing.assert_array_equal(acc.cpu().numpy(), wa)
        # (of the chunk's tokens the drafts were the last D: those rejected are taken back)
        short = torch.minimum(plan.seq_len, torch.full_like(plan.seq_len, D)) - acc
        ctx, held, head = (plan.seq_len - short.clamp_min(0)).to(torch.int32), plan.held_out, head + plan.free_used
