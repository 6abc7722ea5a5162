"""Workspaces of the two cache-row writers: each is held to its own plan."""
import ctypes

import numpy as np
import pytest
import torch

from dsa_indexer_top_b200 import binding as B

HIDDEN = 6144
# tokens and the contiguous writer's splits along K: at most 144 tiles of 128 x 128 over
# tiles of the result, at least 4 of the 96 blocks along K each
SPLITS = [(4, 24), (300, 8), (1024, 3), (2048, 1), (3000, 1)]


def _need(n_tok, splits):
    return 256 + (splits * n_tok * 704 * 4 + 255) // 256 * 256


@pytest.mark.parametrize("n_tok,splits", SPLITS)
def test_workspaces_that_are_too_small_are_refused(n_tok, splits):
    lib, P, ws = B.lib(), 0xD000, 0x10000
    w = B._CacheWriter(n_tok, HIDDEN, P, HIDDEN, P, P, P, P, P, P, 1, 4096, P, 4096 * 576, 576, P, 4096 * 128, 128, 1e-5, 8e6)
    need = _need(n_tok, splits)
    assert lib.dsa_cache_writer_workspace_bytes(n_tok, HIDDEN) >= need
    assert lib.dsa_write_cache_rows(ctypes.byref(w), ws, need - 1, None) == B.DSA_ERR_WORKSPACE
    assert lib.dsa_write_paged_rows(ctypes.byref(w), P, ws, need - 1, None) == B.DSA_ERR_WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("n_tok,splits", SPLITS)
def test_contiguous_writer_takes_its_own_size(cuda_ok, n_tok, splits):
    """The contiguous writer runs in the bytes of its own plan, writes none behind them and gives
    the rows it gives in a larger workspace."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(n_tok)
    rn = lambda *s: torch.randn(*s, generator=g, device=dev)
    h, w = rn(n_tok, HIDDEN).bfloat16(), (rn(704, HIDDEN) / HIDDEN ** 0.5).bfloat16()
    norms = (1 + 0.1 * rn(512), 1 + 0.1 * rn(128), 0.1 * rn(128))
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).to(dev)
    seq, pos = i32([0] * n_tok), i32(range(n_tok))
    need, got = _need(n_tok, splits), []
    for room in (need, B.dsa_cache_writer_workspace_bytes(n_tok, HIDDEN)):
        buf = torch.zeros(room + 4096, dtype=torch.uint8, device=dev)
        buf[room:] = 0x5A
        kv = torch.zeros(1, n_tok, 576, dtype=torch.bfloat16, device=dev)
        kidx = torch.zeros(1, n_tok, 128, dtype=torch.bfloat16, device=dev)
        B.dsa_write_cache_rows(B.CacheWriter(h, w, *norms, seq, pos, kv, kidx), buf[:room])
        assert B.dsa_check_status(buf[:room]) == B.DSA_OK
        assert (buf[room:] == 0x5A).all()
        got.append((kv, kidx))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
