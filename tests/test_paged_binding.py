"""The paged calls' own checks of their tensors (no GPU needed): what would make a kernel
read or write outside a tensor is refused before the call."""
import pytest
import torch

from dsa_indexer_top_b200 import binding as B

i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
WS = torch.zeros(256, dtype=torch.uint8)


def _batch(**kw):
    return B.PagedBatch(**{**dict(block_table=i32(2, 4), q_begin=i32(3), seq_len=i32(2), n_tok=3, n_pages=9, page_rows=16),
                           **kw})


def _mla(**kw):
    return B.Mla(**{**dict(q=bf(3, 8, 576), kv=bf(9, 16, 576), out=bf(3, 8, 512), d_latent=512, scale=0.1,
                           lse=torch.zeros(3, 8)), **kw})


@pytest.mark.parametrize("kw,err", [
    (dict(kv=bf(8, 16, 576)), ValueError), (dict(kv=bf(9, 15, 576)), ValueError), (dict(kv=bf(9, 16, 570)), ValueError),
    (dict(kv=torch.zeros(9, 16, 640, dtype=torch.uint8)), ValueError), (dict(out=bf(3, 4, 512)), ValueError),
    (dict(out=bf(2, 8, 512)), ValueError), (dict(lse=torch.zeros(3, 7)), ValueError), (dict(d_latent=600), ValueError),
    (dict(lse=bf(3, 8)), TypeError), (dict(kv=torch.zeros(9, 16, 576)), TypeError),
    (dict(out=torch.zeros(3, 8, 512)), TypeError), (dict(q=bf(3, 8, 1152)[..., ::2]), TypeError),
    (dict(out=bf(3, 8, 1024)[..., ::2]), TypeError), (dict(kv=bf(9, 16, 1152)[..., ::2]), TypeError),
    (dict(lse=torch.zeros(8, 3).t()), TypeError)])
def test_attention_refuses_tensors_that_do_not_fit(kw, err):
    with pytest.raises(err):
        B.dsa_paged_mla(_batch(), _mla(**kw), WS)


def test_a_descriptor_is_checked_again_when_it_changes():
    batch, mla = _batch(), _mla(lse=bf(3, 8))
    for _ in range(2):
        with pytest.raises(TypeError):
            B.dsa_paged_mla(batch, mla, WS)
    mla.lse = None
    with pytest.raises(ValueError, match="GPU"):     # (host tensors: everything else fits)
        B.dsa_paged_mla(batch, mla, WS)


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [dict(n_tok=4), dict(n_pages=10), dict(page_rows=17)])
def test_a_batch_that_one_layer_has_no_room_for(cuda_ok, kw):
    """Layers share a batch; each one's tensors are held to it."""
    dev = lambda m: B.Mla(m.q.cuda(), m.kv.cuda(), m.out.cuda(), 512, 0.1, m.lse.cuda())
    batch = _batch(block_table=i32(2, 4).cuda(), q_begin=i32(3).cuda(), seq_len=i32(2).cuda())
    layers = [dev(_mla()), dev(_mla())]
    ws = B.paged_workspace(batch, layers[0])
    for layer in layers:
        B.dsa_paged_mla(batch, layer, ws)          # (no sequence has tokens: nothing is read)
    for k, v in kw.items():
        setattr(batch, k, v)
    for layer in layers:
        with pytest.raises(ValueError):
            B.dsa_paged_mla(batch, layer, ws)
    torch.cuda.synchronize()


def _writer(**kw):
    return B.CacheWriter(**{**dict(h=bf(5, 64), w=bf(704, 64), rms_weight=torch.ones(512), ln_weight=torch.ones(128),
                                   ln_bias=torch.ones(128), tok_seq=None, tok_pos=i32(5), kv=bf(4, 8, 576),
                                   k_idx=bf(4, 8, 128)), **kw})


@pytest.mark.parametrize("kw,err", [
    (dict(tok_pos=i32(4)), ValueError), (dict(tok_pos=torch.zeros(5, dtype=torch.int64)), TypeError),
    (dict(w=bf(700, 64)), TypeError), (dict(w=bf(704, 128)[:, ::2]), TypeError), (dict(w=torch.zeros(704, 64)), TypeError),
    (dict(h=torch.zeros(5, 64)), TypeError), (dict(rms_weight=torch.ones(511)), TypeError),
    (dict(ln_bias=bf(128)), TypeError), (dict(kv=torch.zeros(4, 8, 576)), TypeError), (dict(kv=bf(4, 8, 575)), ValueError),
    (dict(k_idx=bf(4, 8, 127)), ValueError), (dict(k_idx=bf(4, 9, 128)), ValueError), (dict(kv=bf(32, 576), k_idx=None), ValueError)])
def test_writer_refuses_tensors_that_do_not_fit(kw, err):
    with pytest.raises(err):
        B.dsa_write_paged_rows(_writer(**kw), i32(5), WS)


def test_tensors_that_are_not_on_the_gpu_are_refused():
    """Host tensors, which a kernel could not read."""
    plan = B.PagePlan(i32(2), i32(2), i32(2), i32(3), None, i32(2, 4), i32(3), i32(2), i32(5), i32(5), i32(5), i32(2), i32(1),
                      n_pages=9, page_rows=4)
    calls = [lambda: B.dsa_page_tables(plan, WS), lambda: B.dsa_write_paged_rows(_writer(), i32(5), WS),
             lambda: B.dsa_paged_mla(_batch(), _mla(), WS),
             lambda: B.dsa_verify_drafts(torch.zeros(2, 3, 7), i32(2, 2), torch.zeros(2, 2), torch.zeros(2), i32(2, 3),
                                         i32(2), WS)]
    for call in calls:
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.mark.gpu
def test_another_current_device_is_refused(cuda_ok, monkeypatch):
    """The kernels would run on the current device; a call with another device's tensors is not made."""
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")
    f = lambda *s: z(*s, dtype=torch.float32)
    ws = z(256, dtype=torch.uint8)
    plan = B.PagePlan(z(2), z(2), z(2), z(3), None, z(2, 4), z(3), z(2), z(5), z(5), z(5), z(2), z(1), n_pages=9, page_rows=4)
    verify = lambda: B.dsa_verify_drafts(f(2, 3, 7) + 1, z(2, 2), f(2, 2), f(2), z(2, 3), z(2), ws)
    for call in (lambda: B.dsa_page_tables(plan, ws), verify):
        call()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: B.dsa_page_tables(plan, ws), verify):
        with pytest.raises(ValueError, match="current device"):
            call()
