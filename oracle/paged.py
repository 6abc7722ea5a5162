"""Plain oracle of the paged-cache operators (test infrastructure only): page
tables in Python integers, dense causal absorbed MLA over paged caches and draft
verification in float64."""
from __future__ import annotations

import numpy as np


def page_tables(ctx, new, held, free, free_begin, table, page_rows, n_tok):
    """Tables, token positions and slots of one step (valid inputs only); `table` is copied."""
    table = np.array(table, dtype=np.int64)
    begin, seq, pos, slot, held_out = [0], [], [], [], []
    at = int(free_begin)
    for b in range(len(ctx)):
        h = int(held[b])
        while h * page_rows < int(ctx[b]) + int(new[b]):
            table[b, h] = free[at]
            at += 1
            h += 1
        held_out.append(h)
        begin.append(begin[-1] + int(new[b]))
        for t in range(int(ctx[b]), int(ctx[b]) + int(new[b])):
            seq.append(b)
            pos.append(t)
            slot.append(int(table[b, t // page_rows]) * page_rows + t % page_rows)
    pad = n_tok - len(seq)
    return dict(table=table, q_begin=np.array(begin), seq_len=np.array(ctx) + np.array(new),
                q_seq=np.array(seq + [0] * pad), q_pos=np.array(pos + [0] * pad),
                slot_map=np.array(slot + [-1] * pad), held_out=np.array(held_out), free_used=at - int(free_begin))


def unpack_fp8(raw, decode, d_lat=512, d_rope=64):
    """Packed FP8 rows (uint8 [..., >= 656]) as float64 [..., d_lat + d_rope]; decode: 256 E4M3 values."""
    raw = np.ascontiguousarray(raw)
    codes = decode[raw[..., :d_lat]].astype(np.float64)
    rope = np.ascontiguousarray(raw[..., d_lat:d_lat + 2 * d_rope]).view(np.uint16).astype(np.uint32) << 16
    sigma = np.ascontiguousarray(raw[..., d_lat + 2 * d_rope:d_lat + 2 * d_rope + 4]).view(np.float32)
    return np.concatenate([codes * sigma.astype(np.float64), rope.view(np.float32).astype(np.float64)], -1)


def paged_mla(q, rows, table, q_begin, seq_len, page_rows, d_lat, scale):
    """q [n_tok, H, dk], rows [n_pages, page_rows, dk] (float64) -> out [n_tok, H, d_lat], lse, touched [n_tok]."""
    n_tok, heads, dk = q.shape
    out = np.zeros((n_tok, heads, d_lat))
    lse = np.full((n_tok, heads), -np.inf)
    touched = np.zeros(n_tok, dtype=bool)
    for b in range(len(seq_len)):
        first, last, total = int(q_begin[b]), int(q_begin[b + 1]), int(seq_len[b])
        for i in range(first, last):
            touched[i] = True
            seen = total - (last - i) + 1
            pages = np.asarray(table[b])[np.arange(seen) // page_rows]
            ok = (pages >= 0) & (pages < rows.shape[0])
            key = rows[pages[ok], np.arange(seen)[ok] % page_rows].astype(np.float64)
            if not len(key):
                continue
            logit = scale * (q[i].astype(np.float64) @ key.T)
            m = logit.max(-1, keepdims=True)
            e = np.exp(logit - m)
            z = e.sum(-1, keepdims=True)
            out[i] = (e / z) @ key[:, :d_lat]
            lse[i] = (m + np.log(z))[:, 0]
    return out, lse, touched


def _clean(p):
    p = np.asarray(p, dtype=np.float64)
    return np.where(np.isfinite(p) & (p > 0), p, 0.0)


def verify_drafts(target, draft, x, draft_len, accept_u, sample_u):
    """target [n, D + 1, V], draft [n, D, V] or None, x [n, D] -> tokens [n, D + 1], n_accept [n]."""
    n, d1, V = target.shape
    d = d1 - 1
    accept_u, x = np.asarray(accept_u), np.asarray(x)
    tokens, n_accept = np.full((n, d1), -1, dtype=np.int64), np.zeros(n, dtype=np.int64)
    for r in range(n):
        k = d if draft_len is None else min(max(int(draft_len[r]), 0), d)
        i = 0
        while i < k:
            t = int(x[r, i])
            if not 0 <= t < V:
                break
            p = _clean(target[r, i, t])
            q = 1.0 if draft is None else _clean(draft[r, i, t])
            if not float(accept_u[r, i]) * q < p:
                break
            tokens[r, i] = t
            i += 1
        p = _clean(target[r, i])
        w = p
        if i < k:
            if draft is not None:
                w = np.maximum(p - _clean(draft[r, i]), 0.0)
            elif 0 <= int(x[r, i]) < V:
                w = p.copy()
                w[int(x[r, i])] = 0.0
            if not w.any():
                w = p
        n_accept[r] = i
        if w.any():
            cdf = np.cumsum(w)
            u = max(float(sample_u[r]), 0.0)
            j = int(np.searchsorted(cdf, u * cdf[-1], side="right"))
            tokens[r, i] = min(j, int(np.nonzero(w)[0][-1]))
    return tokens, n_accept
