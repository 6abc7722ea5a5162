"""Host-side refusals of the paged-cache entry points (no GPU needed): every bad
argument is rejected before any launch; and the binding's own checks."""
import ctypes

import pytest
import torch

from dsa_indexer_top_b200 import binding as B

WS, BIG = 0x10000, 1 << 40


def _plan(**kw):
    p = B._PagePlan(4, 8, 100, 16, 6, 5, 0x1000, 0x2000, 0x3000, 0x4000, 0x5000, 0x6000, 6, 0x7000, 0x8000, 0x9000,
                    0xa000, 0xb000, 0xc000, 0xd000)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw", [
    dict(n_seq=-1), dict(n_tok=-1), dict(n_free=-1), dict(max_pages=0), dict(n_pages=0), dict(page_rows=0),
    dict(n_pages=1 << 20, page_rows=1 << 11), dict(table_stride=5), dict(ctx_len=None), dict(new_len=None),
    dict(held=None), dict(free_pages=None), dict(block_table=None), dict(q_begin=None), dict(seq_len=None),
    dict(q_seq=None), dict(q_pos=None), dict(slot_map=None), dict(held_out=None), dict(free_used=None),
    dict(held_out=0x3000), dict(seq_len=0x1000), dict(free_used=0x5000), dict(q_pos=0x9000)])
def test_page_tables_rejects(kw):
    p = _plan(**kw)
    assert B.lib().dsa_page_tables(ctypes.byref(p), WS, BIG, None) == B.DSA_ERR_INVALID


def test_page_tables_rejects_null_and_workspace():
    lib, p = B.lib(), _plan()
    assert lib.dsa_page_tables(None, WS, BIG, None) == B.DSA_ERR_INVALID
    for ws, n in ((None, BIG), (WS + 16, BIG), (WS, 255)):
        assert lib.dsa_page_tables(ctypes.byref(p), ws, n, None) == B.DSA_ERR_WORKSPACE


def _batch(**kw):
    b = B._PagedBatch(4, 8, 100, 16, 6, 0x1000, 6, 0x2000, 0x3000)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def _mla(**kw):
    m = B._Mla(64, 512, 64, B.DSA_BF16, 0.0625, 0, 0x6000, 0x7000, 16 * 576, 576, 0x8000, None)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


@pytest.mark.parametrize("b,m", [
    (dict(n_seq=-1), {}), (dict(n_tok=-1), {}), (dict(n_pages=0), {}), (dict(page_rows=0), {}), (dict(max_pages=0), {}),
    (dict(n_pages=1 << 21, page_rows=1 << 10), {}), (dict(table_stride=5), {}), (dict(block_table=None), {}),
    (dict(q_begin=None), {}), (dict(seq_len=None), {}), ({}, dict(q=None)), ({}, dict(kv=None)), ({}, dict(out=None)),
    ({}, dict(heads=0)), ({}, dict(d_latent=0)), ({}, dict(d_rope=-1)), ({}, dict(dtype=7)), ({}, dict(kv_dtype=9)),
    ({}, dict(kv_row_stride=575)), ({}, dict(kv_seq_stride=-1)),
    ({}, dict(kv_dtype=B.DSA_FP8_E4M3, kv_row_stride=640, kv_seq_stride=640 * 16))])
def test_paged_mla_rejects(b, m):
    lib, bc, mc = B.lib(), _batch(**b), _mla(**m)
    assert lib.dsa_paged_mla(ctypes.byref(bc), ctypes.byref(mc), WS, BIG, None) == B.DSA_ERR_INVALID
    assert lib.dsa_paged_mla_workspace_bytes(ctypes.byref(bc), ctypes.byref(mc)) == 0


@pytest.mark.parametrize("m", [
    dict(kv_dtype=B.DSA_FP8_E4M3, kv_row_stride=664, kv_seq_stride=664 * 16),                # not 16-byte rows
    dict(kv_dtype=B.DSA_FP8_E4M3, kv_row_stride=656, kv_seq_stride=656 * 16, dtype=B.DSA_F32),
    dict(kv_dtype=B.DSA_FP8_E4M3, kv_row_stride=656, kv_seq_stride=656 * 16, d_latent=256),
    dict(kv_dtype=B.DSA_FP8_E4M3, kv_row_stride=656, kv_seq_stride=656 * 16, kv=0x7008),
    dict(heads=70000), dict(d_latent=9000, kv_row_stride=9064, kv_seq_stride=9064 * 16)])
def test_paged_mla_unsupported(m):
    bc, mc = _batch(), _mla(**m)
    assert B.lib().dsa_paged_mla(ctypes.byref(bc), ctypes.byref(mc), WS, BIG, None) == B.DSA_ERR_UNSUPPORTED


def test_paged_mla_workspace_and_empty():
    lib, bc, mc = B.lib(), _batch(), _mla()
    need = lib.dsa_paged_mla_workspace_bytes(ctypes.byref(bc), ctypes.byref(mc))
    assert need >= 256
    call = lambda b, ws, n: lib.dsa_paged_mla(ctypes.byref(b), ctypes.byref(mc), ws, n, None)
    for ws, n in ((None, need), (WS + 128, need), (WS, need - 1)):
        assert call(bc, ws, n) == B.DSA_ERR_WORKSPACE
    assert call(_batch(n_tok=0), WS, need) == B.DSA_OK
    assert call(_batch(n_seq=0, block_table=None, seq_len=None), WS, need) == B.DSA_OK


def _writer(**kw):
    w = B._CacheWriter(4, 64, 0x1000, 64, 0x2000, 0x3000, 0x4000, 0x5000, None, 0x6000, 10, 16, 0x7000, 16 * 576, 576,
                       None, 0, 0, 1e-5, 8e6)
    for k, v in kw.items():
        setattr(w, k, v)
    return w


def test_write_paged_rows_rejects():
    lib = B.lib()
    call = lambda w, s=0x8000, ws=WS, n=BIG: lib.dsa_write_paged_rows(w and ctypes.byref(w), s, ws, n, None)
    assert call(None) == B.DSA_ERR_INVALID
    assert call(_writer(), s=None) == B.DSA_ERR_INVALID
    assert call(_writer(n_seq=1 << 20, max_ctx=1 << 12)) == B.DSA_ERR_INVALID      # slots are int32
    for kw in (dict(n_tok=-1), dict(n_seq=0), dict(max_ctx=0), dict(tok_pos=None), dict(kv=None), dict(hidden=60),
               dict(kv_row_stride=500), dict(eps=0.0), dict(h_row_stride=60)):
        assert call(_writer(**kw)) == B.DSA_ERR_INVALID, kw
    assert call(_writer(), n=256) == B.DSA_ERR_WORKSPACE
    assert call(_writer(n_tok=0)) == B.DSA_OK
    # the contiguous writer still needs its token sequences
    w = _writer()
    assert lib.dsa_write_cache_rows(ctypes.byref(w), WS, BIG, None) == B.DSA_ERR_INVALID


def _verify(**kw):
    v = B._Verify(3, 2, 100, B.DSA_F32, 0x1000, 300, 100, 0x2000, 200, 100, 0x3000, None, 0x4000, 0x5000, 0x6000, 0x7000)
    for k, x in kw.items():
        setattr(v, k, x)
    return v


@pytest.mark.parametrize("kw", [
    dict(n_req=-1), dict(n_draft=-1), dict(vocab=0), dict(dtype=5), dict(target=None), dict(target=0x1002),
    dict(draft=0x2001), dict(draft_tokens=None), dict(accept_u=None), dict(sample_u=None), dict(tokens=None),
    dict(n_accept=None), dict(t_req_stride=-1), dict(t_row_stride=-1), dict(d_req_stride=-1), dict(d_row_stride=-1),
    dict(tokens=0x3000), dict(tokens=0x1000), dict(n_accept=0x4000), dict(n_accept=0x6000)])
def test_verify_rejects(kw):
    v = _verify(**kw)
    assert B.lib().dsa_verify_drafts(ctypes.byref(v), WS, BIG, None) == B.DSA_ERR_INVALID


def test_verify_other_statuses():
    lib = B.lib()
    call = lambda v, ws=WS, n=BIG: lib.dsa_verify_drafts(ctypes.byref(v), ws, n, None)
    assert lib.dsa_verify_drafts(None, WS, BIG, None) == B.DSA_ERR_INVALID
    assert call(_verify(dtype=B.DSA_FP8_E4M3)) == B.DSA_ERR_UNSUPPORTED
    assert call(_verify(vocab=(1 << 30) + 1)) == B.DSA_ERR_UNSUPPORTED
    for ws, n in ((None, BIG), (WS + 8, BIG), (WS, 128)):
        assert call(_verify(), ws, n) == B.DSA_ERR_WORKSPACE
    assert call(_verify(n_req=0)) == B.DSA_OK


def test_binding_checks_tensors():
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    plan = dict(ctx_len=i(2), new_len=i(2), held=i(2), free_pages=i(3), free_begin=None, block_table=i(2, 4),
                q_begin=i(3), seq_len=i(2), q_seq=i(5), q_pos=i(5), slot_map=i(5), held_out=i(2), free_used=i(1),
                n_pages=9, page_rows=4)
    c = B.PagePlan(**plan).c()
    assert (c.n_seq, c.n_tok, c.max_pages, c.n_free, c.table_stride) == (2, 5, 4, 3, 4)
    for bad in (dict(new_len=i(3)), dict(q_begin=i(2)), dict(slot_map=i(4)), dict(block_table=i(3, 4))):
        with pytest.raises(ValueError):
            B.PagePlan(**{**plan, **bad}).c()
    for bad in (dict(ctx_len=torch.zeros(2, dtype=torch.int64)), dict(block_table=i(4, 2).t()), dict(held=i(4)[::2])):
        with pytest.raises(TypeError):
            B.PagePlan(**{**plan, **bad}).c()
    with pytest.raises(ValueError):
        B.PagedBatch(i(2, 4), i(2), i(2), 5, 9, 4).c()
    ws = torch.zeros(256, dtype=torch.uint8)
    t, x, u = torch.zeros(2, 3, 7), i(2, 2), torch.zeros(2, 2)
    ok = dict(target=t, draft_tokens=x, accept_u=u, sample_u=torch.zeros(2), tokens=i(2, 3), n_accept=i(2), ws=ws)
    for bad in (dict(draft_tokens=i(2, 3)), dict(tokens=i(2, 2)), dict(draft=torch.zeros(2, 3, 7)),
                dict(n_draft=i(3))):
        with pytest.raises(ValueError):
            B.dsa_verify_drafts(**{**ok, **bad})
    for bad in (dict(target=torch.zeros(2, 7, 3).transpose(1, 2)), dict(draft=torch.zeros(2, 2, 7).bfloat16()),
                dict(accept_u=u.double()), dict(n_accept=torch.zeros(2))):
        with pytest.raises(TypeError):
            B.dsa_verify_drafts(**{**ok, **bad})


def test_cache_writers_take_an_empty_batch():
    lib, w = B.lib(), _writer(n_tok=0, tok_seq=0x9000)
    need = B.dsa_cache_writer_workspace_bytes(0, 64)
    assert need >= 256
    assert lib.dsa_write_cache_rows(ctypes.byref(w), WS, need, None) == B.DSA_OK
    assert lib.dsa_write_paged_rows(ctypes.byref(w), None, WS, need, None) == B.DSA_OK
