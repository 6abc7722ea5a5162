"""Measured cases of the paged-cache operators: page tables, the cache-row writer
through a slot map, attention of new tokens over a paged latent cache, and the
verification of drafted tokens.

`run` computes a case in its plain form (elementary torch operations in float32,
float64 where a sum decides an integer) or, with `own` set, through the library's
entry points.  Shapes are the package's own: latent 512 + RoPE key 64, indexer
key 128, hidden 6144, 64 heads (fewer where heads are divided over ranks).
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
LATENT, ROPE, IDX = 512, 64, 128
ROW = LATENT + ROPE
FP8_ROW = 656
HIDDEN = 6144
EPS = 1e-5
THETA = 8.0e6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step of 64 requests: where the call's latency is all of it
        dict(name="tables-decode-64", op="tables", n_seq=64, new_lo=1, new_hi=1, ctx_hi=32767, page=64, pad=0),
        # a step that mixes prompt chunks and single tokens, small pages, a padded token count
        dict(name="tables-mixed-700", op="tables", n_seq=700, new_lo=0, new_hi=160, ctx_hi=9000, page=16, pad=133),
        # cache rows of one decode step, some slots of the padded batch empty
        dict(name="write-decode-13", op="write", n_tok=13, page=64, skip=3),
        # cache rows of a prompt chunk
        dict(name="write-chunk-2048", op="write", n_tok=2048, page=64, skip=0),
        # one short request, one token: the smallest attention call
        dict(name="attend-one-777", op="attend", n_seq=1, new_lo=1, new_hi=1, ctx_lo=776, ctx_hi=776, heads=64,
             page=64, fp8=False, chunk=0),
        # decode of 8 requests at 32K rows each
        dict(name="attend-decode-8x32k", op="attend", n_seq=8, new_lo=1, new_hi=1, ctx_lo=32767, ctx_hi=32767,
             heads=64, page=64, fp8=False, chunk=0),
        # ragged decode over packed FP8 pages
        dict(name="attend-decode-fp8-32", op="attend", n_seq=32, new_lo=1, new_hi=1, ctx_lo=900, ctx_hi=24000,
             heads=64, page=64, fp8=True, chunk=0),
        # a base token and its drafts per request, small pages
        dict(name="attend-drafts-16", op="attend", n_seq=16, new_lo=2, new_hi=5, ctx_lo=1000, ctx_hi=12000,
             heads=64, page=16, fp8=False, chunk=0),
        # heads divided over four ranks, a prompt chunk among single tokens
        dict(name="attend-mixed-16h", op="attend", n_seq=25, new_lo=1, new_hi=1, ctx_lo=300, ctx_hi=7000, heads=16,
             page=32, fp8=False, chunk=601),
        # a prompt chunk of 2048 tokens behind 16K cached rows
        dict(name="attend-chunk-2048", op="attend", n_seq=1, new_lo=2048, new_hi=2048, ctx_lo=16384, ctx_hi=16384,
             heads=64, page=64, fp8=False, chunk=0),
        # verification of greedy drafts, bf16 probabilities, few requests
        dict(name="verify-greedy-5", op="verify", n_req=5, drafts=2, vocab=32000, bf16=True, greedy=True),
        # verification of sampled drafts of a full batch, odd vocabulary
        dict(name="verify-sampled-96", op="verify", n_req=96, drafts=4, vocab=131071, bf16=False, greedy=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "write", "attend", "attend", "attend", "verify"])
    if op == "tables":
        n_seq = _log_int(rng, 1, 1024)
        page = rng.choice([8, 16, 32, 64, 128])
        hi = rng.choice([1, 5, _log_int(rng, 1, max(2, 60000 // n_seq))])
        return dict(op=op, n_seq=n_seq, new_lo=rng.choice([0, 1]), new_hi=max(1, hi), ctx_hi=_log_int(rng, 1, 32767),
                    page=page, pad=rng.choice([0, rng.randrange(1, 300)]))
    if op == "write":
        n_tok = _log_int(rng, 1, 2048)
        return dict(op=op, n_tok=n_tok, page=rng.choice([8, 16, 64]), skip=rng.choice([0, n_tok // 5]))
    if op == "verify":
        return dict(op=op, n_req=_log_int(rng, 1, 96), drafts=rng.randrange(1, 6), vocab=_log_int(rng, 1000, 131071),
                    bf16=rng.random() < 0.5, greedy=rng.random() < 0.5)
    heads = rng.choice([8, 16, 32, 64, 64, 128])
    page = rng.choice([16, 32, 64, 64, 128])
    fp8 = rng.random() < 0.4
    kind = rng.choice(["decode", "drafts", "chunk", "mixed"])
    if kind == "chunk":
        n_seq = rng.randrange(1, 5)
        new = _log_int(rng, 40, 1000)
        ctx = rng.choice([0, _log_int(rng, 1, 7000)])
        while n_seq * new * (ctx + new) * heads > 2.0e9:
            new //= 2
        return dict(op=op, n_seq=n_seq, new_lo=max(1, new // 2), new_hi=new, ctx_lo=ctx // 2, ctx_hi=ctx, heads=heads,
                    page=page, fp8=fp8, chunk=0)
    n_seq = _log_int(rng, 1, 48)
    ctx = _log_int(rng, 1, 20000)
    hi = 1 if kind != "drafts" else rng.randrange(2, 7)
    return dict(op=op, n_seq=n_seq, new_lo=1, new_hi=hi, ctx_lo=ctx // 4, ctx_hi=ctx, heads=heads, page=page, fp8=fp8,
                chunk=_log_int(rng, 20, 700) if kind == "mixed" else 0)


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """(ctx_len, new_len) of a case's sequences: fixed by the case, not by the seed."""
    r = np.random.default_rng([case["n_seq"], case["new_hi"], case["ctx_hi"], case["page"]])
    n = case["n_seq"]
    ctx = r.integers(case.get("ctx_lo", 0), case["ctx_hi"] + 1, n)
    new = r.integers(case["new_lo"], case["new_hi"] + 1, n)
    if case.get("chunk"):
        new[n // 2] = case["chunk"]
    return ctx.astype(np.int64), new.astype(np.int64)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a), dtype=np.int32)).to(DEV)


def _page_layout(total_rows, page, rng, slack=3):
    """Block table with pages in random order; returns table, pages in the pool."""
    need = [-(-int(t) // page) for t in total_rows]
    n_pages = max(1, sum(need) + slack)
    perm = rng.permutation(n_pages)
    width = max(1, max(need, default=1))
    table = np.full((len(need), width), -1, dtype=np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = perm[at:at + k]
        at += k
    return table, n_pages


def _prepare_tables(case, rng):
    ctx, new = _lengths(case)
    page, n = case["page"], case["n_seq"]
    held = -(-ctx // page)
    more = rng.random(n) < 0.1            # pages kept after rejected drafts
    held = held + more
    total = -(-(ctx + new) // page)
    width = int(max(1, np.maximum(total, held).max())) + 2
    n_held, n_new = int(held.sum()), int(np.maximum(total - held, 0).sum())
    n_pages = n_held + n_new + 7
    perm = rng.permutation(n_pages)
    table = np.full((n, width), -1, dtype=np.int32)
    at = 0
    for b in range(n):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += int(held[b])
    free_begin = 3
    free = np.concatenate([np.full(free_begin, -1), perm[at:]])   # the list's first entries are used up
    n_tok = int(new.sum()) + case["pad"]
    e = lambda k: torch.empty(k, dtype=torch.int32, device=DEV)
    st = dict(ctx=_i32(ctx), new=_i32(new), held=_i32(held), free=_i32(free), free_begin=_i32([free_begin]),
              table=_i32(table), page=page, n_tok=n_tok, n_pages=n_pages,
              out=dict(q_begin=e(n + 1), seq_len=e(n), q_seq=e(n_tok), q_pos=e(n_tok), slot_map=e(n_tok),
                       held_out=e(n), free_used=e(1)))
    if own:
        from dsa_indexer_top_b200 import binding as B
        o = st["out"]
        st["plan"] = B.PagePlan(st["ctx"], st["new"], st["held"], st["free"], st["free_begin"], st["table"],
                                o["q_begin"], o["seq_len"], o["q_seq"], o["q_pos"], o["slot_map"], o["held_out"],
                                o["free_used"], n_pages=n_pages, page_rows=page)
        st["ws"] = _status_ws(B, 256)
    return st


def _status_ws(B, nbytes):
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=DEV)
    B.dsa_workspace_init(ws)
    return ws


def _prepare_write(case, rng, g):
    n, page = case["n_tok"], case["page"]
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    n_pages = -(-n // page) + 5
    slots = rng.permutation(n_pages * page)[:n].astype(np.int32)
    if case["skip"]:
        slots[n - case["skip"]:] = -1     # the padded end of the batch
    st = dict(h=rn(n, HIDDEN).bfloat16(), w=(rn(704, HIDDEN) / math.sqrt(HIDDEN)).bfloat16(),
              rms=1 + 0.1 * rn(LATENT), lnw=1 + 0.1 * rn(IDX), lnb=0.1 * rn(IDX),
              pos=_i32(rng.integers(0, 1 << 20, n)), slots=_i32(slots), page=page,
              kv=rn(n_pages, page, ROW).bfloat16(), k_idx=rn(n_pages, page, IDX).bfloat16())
    if own:
        from dsa_indexer_top_b200 import binding as B
        st["writer"] = B.CacheWriter(st["h"], st["w"], st["rms"], st["lnw"], st["lnb"], None, st["pos"], st["kv"],
                                     st["k_idx"], eps=EPS, rope_theta=THETA)
        st["ws"] = _status_ws(B, B.dsa_cache_writer_workspace_bytes(n, HIDDEN))
    return st


def _pack_fp8(rows):
    """bf16 rows [.., 576] as packed FP8 rows: codes, bf16 RoPE key, float32 scale."""
    c = rows[..., :LATENT].float()
    sigma = (c.abs().amax(-1, keepdim=True) / 448.0).clamp_min(1e-12)
    codes = (c / sigma).to(torch.float8_e4m3fn)
    out = torch.zeros((*rows.shape[:-1], FP8_ROW), dtype=torch.uint8, device=rows.device)
    out[..., :LATENT] = codes.view(torch.uint8)
    out[..., LATENT:LATENT + 2 * ROPE] = rows[..., LATENT:].contiguous().view(torch.uint8)
    out[..., LATENT + 2 * ROPE:LATENT + 2 * ROPE + 4] = sigma.contiguous().view(torch.uint8)
    return out


def _prepare_attend(case, rng, g):
    ctx, new = _lengths(case)
    page, heads = case["page"], case["heads"]
    total = ctx + new
    table, n_pages = _page_layout(total, page, rng)
    n_tok = int(new.sum())
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV)
    rows = rn(n_pages, page, ROW)
    # a few rows that attract attention, as first tokens and delimiters do
    hot = torch.rand(n_pages, page, 1, generator=g, device=DEV) < 0.004
    rows = torch.where(hot, 2.5 * rows, rows).bfloat16()
    kv = _pack_fp8(rows) if case["fp8"] else rows
    begin = np.concatenate([[0], np.cumsum(new)])
    st = dict(q=rn(n_tok, heads, ROW).bfloat16(), kv=kv, fp8=case["fp8"], table=_i32(table), q_begin=_i32(begin),
              seq_len=_i32(total), ctx=ctx, new=new, page=page, heads=heads, scale=1.0 / 16.0,
              out=torch.empty(n_tok, heads, LATENT, dtype=torch.bfloat16, device=DEV),
              lse=torch.empty(n_tok, heads, dtype=torch.float32, device=DEV))
    if own:
        from dsa_indexer_top_b200 import binding as B
        st["batch"] = B.PagedBatch(st["table"], st["q_begin"], st["seq_len"], n_tok=n_tok, n_pages=n_pages,
                                   page_rows=page)
        st["mla"] = B.Mla(st["q"], kv, st["out"], LATENT, st["scale"], st["lse"])
        st["ws"] = B.paged_workspace(st["batch"], st["mla"])
    return st


def _prepare_verify(case, rng, g):
    n, d, v = case["n_req"], case["drafts"], case["vocab"]
    dt = torch.bfloat16 if case["bf16"] else torch.float32
    logits = 2.5 * torch.randn(n, d + 1, v, generator=g, device=DEV)
    p = torch.softmax(logits, -1).to(dt)
    near = logits[:, :d] + 0.5 * torch.randn(n, d, v, generator=g, device=DEV)
    q = torch.softmax(near, -1).to(dt)
    if case["greedy"]:
        x = near.argmax(-1)
    else:
        cdf = q.double().cumsum(-1)
        u = torch.rand(n, d, 1, generator=g, device=DEV, dtype=torch.float64) * cdf[..., -1:]
        x = (cdf <= u).sum(-1).clamp_max(v - 1)
    st = dict(p=p, q=None if case["greedy"] else q, x=x.to(torch.int32), n_draft=_i32(rng.integers(0, d + 1, n)),
              u=torch.rand(n, d, generator=g, device=DEV), us=torch.rand(n, generator=g, device=DEV),
              tokens=torch.empty(n, d + 1, dtype=torch.int32, device=DEV),
              n_accept=torch.empty(n, dtype=torch.int32, device=DEV))
    if own:
        from dsa_indexer_top_b200 import binding as B
        st["ws"] = _status_ws(B, 256)
    return st


def prepare(case, seed):
    rng = np.random.default_rng([seed, 77])
    g = torch.Generator(device=DEV).manual_seed(1000003 * (seed % 100000) + 12345)
    if case["op"] == "tables":
        st = _prepare_tables(case, rng)
    elif case["op"] == "write":
        st = _prepare_write(case, rng, g)
    elif case["op"] == "attend":
        st = _prepare_attend(case, rng, g)
    else:
        st = _prepare_verify(case, rng, g)
    st["op"] = case["op"]
    return st


# ------------------------------------------------------------------ plain forms
def _plain_tables(s):
    page, n_tok = s["page"], s["n_tok"]
    ctx, new, held = s["ctx"].long(), s["new"].long(), s["held"].long()
    n = ctx.numel()
    total = ctx + new
    need = torch.maximum(held, (total + page - 1) // page)
    fresh = need - held
    first = fresh.cumsum(0) - fresh + s["free_begin"].long()
    cols = torch.arange(s["table"].shape[1], device=DEV)
    is_new = (cols[None] >= held[:, None]) & (cols[None] < need[:, None])
    src = (first[:, None] + cols[None] - held[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(is_new, s["free"][src], s["table"])
    begin = torch.zeros(n + 1, dtype=torch.int64, device=DEV)
    begin[1:] = new.cumsum(0)
    tok = torch.arange(n_tok, device=DEV)
    seq = torch.searchsorted(begin[1:].contiguous(), tok, right=True)
    live = seq < n
    seq = torch.where(live, seq, 0)
    pos = torch.where(live, ctx[seq] + tok - begin[seq], 0)
    slot = torch.where(live, table[seq, pos // page].long() * page + pos % page, -1)
    i = lambda t: t.to(torch.int32)
    return dict(table=table, q_begin=i(begin), seq_len=i(total), q_seq=i(seq), q_pos=i(pos), slot_map=i(slot),
                held_out=i(need), free_used=i(fresh.sum().reshape(1)))


def _rope(x, pos):
    """Adjacent pairs of the last axis (64) turned by pos * theta^(-2i/64), angles in float64."""
    half = x.shape[-1] // 2
    freq = THETA ** (-2.0 * torch.arange(half, device=x.device, dtype=torch.float64) / x.shape[-1])
    ang = pos.double()[:, None] * freq
    c, s = ang.cos().float(), ang.sin().float()
    a, b = x[:, 0::2], x[:, 1::2]
    return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(1)


def _plain_write(s):
    y = s["h"].float() @ s["w"].float().T
    c, r, k = y[:, :LATENT], y[:, LATENT:ROW], y[:, ROW:]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["rms"]
    kc = k - k.mean(-1, keepdim=True)
    k = kc * torch.rsqrt((kc * kc).mean(-1, keepdim=True) + EPS) * s["lnw"] + s["lnb"]
    rows = torch.cat([c, _rope(r, s["pos"])], -1).bfloat16()
    keys = torch.cat([k[:, :IDX - ROPE], _rope(k[:, IDX - ROPE:], s["pos"])], -1).bfloat16()
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    at = s["slots"].long()[keep]
    s["kv"].view(-1, ROW)[at] = rows[keep]
    s["k_idx"].view(-1, IDX)[at] = keys[keep]
    return dict(kv=s["kv"], k_idx=s["k_idx"])


def _rows32(s, b, total):
    """Sequence b's cache rows in order, float32 [total, 576]."""
    k = -(-total // s["page"])
    raw = s["kv"][s["table"][b, :k].long()].flatten(0, 1)[:total]
    if not s["fp8"]:
        return raw.float()
    codes = raw[:, :LATENT].contiguous().view(torch.float8_e4m3fn).float()
    rope = raw[:, LATENT:LATENT + 2 * ROPE].contiguous().view(torch.bfloat16).float()
    sigma = raw[:, LATENT + 2 * ROPE:LATENT + 2 * ROPE + 4].contiguous().view(torch.float32)
    return torch.cat([codes * sigma, rope], -1)


def _plain_attend(s):
    at = 0
    for b in range(len(s["ctx"])):
        n, ctx = int(s["new"][b]), int(s["ctx"][b])
        rows = _rows32(s, b, ctx + n)
        step = max(1, (1 << 28) // (s["heads"] * (ctx + n)))
        for j0 in range(0, n, step):
            j1 = min(n, j0 + step)
            seen = ctx + j1
            q = s["q"][at + j0:at + j1].float()
            logit = (q.flatten(0, 1) @ rows[:seen].T).view(j1 - j0, s["heads"], seen) * s["scale"]
            pos = torch.arange(ctx + j0, ctx + j1, device=DEV)
            hidden = torch.arange(seen, device=DEV)[None, :] > pos[:, None]
            logit = logit.masked_fill(hidden[:, None, :], float("-inf"))
            m = logit.amax(-1, keepdim=True)
            e = (logit - m).exp()
            z = e.sum(-1, keepdim=True)
            s["lse"][at + j0:at + j1] = (m + z.log()).squeeze(-1)
            o = (e.flatten(0, 1) @ rows[:seen, :LATENT]).view(j1 - j0, s["heads"], LATENT) / z
            s["out"][at + j0:at + j1] = o.bfloat16()
        at += n
    return dict(out=s["out"], lse=s["lse"])


def _plain_verify(s):
    n, d = s["x"].shape
    x = s["x"].long()[..., None]
    px = s["p"][:, :d].gather(-1, x).squeeze(-1).double()
    qx = torch.ones_like(px) if s["q"] is None else s["q"].gather(-1, x).squeeze(-1).double()
    idx = torch.arange(d, device=DEV)
    ok = (s["u"].double() * qx < px) & (idx[None] < s["n_draft"][:, None])
    acc = ok.long().cumprod(-1).sum(-1)
    rows = torch.arange(n, device=DEV)
    p = s["p"][rows, acc].double()
    rejected = acc < s["n_draft"]
    at = acc.clamp_max(d - 1)
    if s["q"] is None:
        q = torch.zeros_like(p)
        q[rows, s["x"].long()[rows, at]] = float("inf")
    else:
        q = s["q"][rows, at].double()
    res = torch.where(rejected[:, None], (p - q).clamp_min(0), p)
    res = torch.where((res.sum(-1) > 0)[:, None], res, p)
    cdf = res.cumsum(-1)
    t = (cdf <= s["us"].double()[:, None] * cdf[:, -1:]).sum(-1)
    tokens = torch.where(idx[None] < acc[:, None], s["x"], -1)
    tokens = torch.cat([tokens, torch.full_like(tokens[:, :1], -1)], -1)
    tokens[rows, acc] = t.to(torch.int32)
    return dict(tokens=tokens, n_accept=acc.to(torch.int32))


# ------------------------------------------------------------------ the library's calls
def _own_tables(s):
    from dsa_indexer_top_b200 import binding as B
    B.dsa_page_tables(s["plan"], s["ws"])
    return dict(table=s["table"], **s["out"])


def _own_write(s):
    from dsa_indexer_top_b200 import binding as B
    B.dsa_write_paged_rows(s["writer"], s["slots"], s["ws"])
    return dict(kv=s["kv"], k_idx=s["k_idx"])


def _own_attend(s):
    from dsa_indexer_top_b200 import binding as B
    B.dsa_paged_mla(s["batch"], s["mla"], s["ws"])
    return dict(out=s["out"], lse=s["lse"])


def _own_verify(s):
    from dsa_indexer_top_b200 import binding as B
    B.dsa_verify_drafts(s["p"], s["x"], s["u"], s["us"], s["tokens"], s["n_accept"], s["ws"], draft=s["q"],
                        n_draft=s["n_draft"])
    return dict(tokens=s["tokens"], n_accept=s["n_accept"])


def run(state):
    form = {"tables": (_plain_tables, _own_tables), "write": (_plain_write, _own_write),
            "attend": (_plain_attend, _own_attend), "verify": (_plain_verify, _own_verify)}[state["op"]]
    return form[1 if own else 0](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "tables":
        ctx, new = _lengths(case)
        page = case["page"]
        fresh = int(np.maximum(-(-(ctx + new) // page) - -(-ctx // page), 0).sum())
        n, n_tok = case["n_seq"], int(new.sum()) + case["pad"]
        return {"bytes": 4 * (3 * n + 2 * fresh + n + 1 + 2 * n + 1 + 3 * n_tok), "flops": 0}
    if case["op"] == "write":
        n = case["n_tok"]
        live = n - case["skip"]
        return {"bytes": 2 * n * HIDDEN + 2 * 704 * HIDDEN + 4 * (LATENT + 2 * IDX) + 8 * n + 2 * live * 704,
                "flops": 2 * live * HIDDEN * 704}
    if case["op"] == "attend":
        ctx, new = _lengths(case)
        h = case["heads"]
        pairs = int((new * ctx + new * (new + 1) // 2).sum())
        row = FP8_ROW - 12 if case["fp8"] else 2 * ROW
        n_tok = int(new.sum())
        table = int((-(-(ctx + new) // case["page"])).sum())
        return {"bytes": int((ctx + new).sum()) * row + n_tok * h * (2 * ROW + 2 * LATENT + 4) + 4 * table,
                "flops": 2 * pairs * h * (ROW + LATENT)}
    n, d, v = case["n_req"], case["drafts"], case["vocab"]
    e = 2 if case["bf16"] else 4
    rows = 1 if case["greedy"] else 2
    return {"bytes": n * (rows * v * e + d * (8 + rows * e) + 4 + 4 + 4 * (d + 1) + 4), "flops": 2 * n * v}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    host = lambda k: st[k].cpu().numpy()
    if case["op"] == "tables":
        page, n_tok = st["page"], st["n_tok"]
        ctx, new, held, free, table = host("ctx"), host("new"), host("held"), host("free"), host("table").copy()
        head = int(host("free_begin")[0])
        begin, seq, pos, slot, out_held = [0], [], [], [], []
        start = head
        for b in range(len(ctx)):
            have = int(held[b])
            while have * page < ctx[b] + new[b]:
                table[b, have] = free[head]
                head += 1
                have += 1
            out_held.append(have)
            begin.append(begin[-1] + int(new[b]))
            for t in range(int(ctx[b]), int(ctx[b] + new[b])):
                seq.append(b)
                pos.append(t)
                slot.append(int(table[b, t // page]) * page + t % page)
        pad = n_tok - len(seq)
        return dict(table=_i32(table), q_begin=_i32(begin), seq_len=_i32(ctx + new), q_seq=_i32(seq + [0] * pad),
                    q_pos=_i32(pos + [0] * pad), slot_map=_i32(slot + [-1] * pad), held_out=_i32(out_held),
                    free_used=_i32([head - start]))
    if case["op"] == "write":
        y = torch.einsum("nk,fk->nf", st["h"].double(), st["w"].double())
        lat, rope, key = y.split([LATENT, ROPE, IDX], dim=1)
        lat = lat / (lat.pow(2).mean(1, keepdim=True) + EPS).sqrt() * st["rms"].double()
        mu, var = key.mean(1, keepdim=True), key.var(1, unbiased=False, keepdim=True)
        key = (key - mu) / (var + EPS).sqrt() * st["lnw"].double() + st["lnb"].double()

        def turn(v):
            i = torch.arange(ROPE // 2, dtype=torch.float64, device=DEV)
            w = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV),
                            st["pos"].double()[:, None] * torch.exp(-2 * i / ROPE * math.log(THETA)))
            return torch.view_as_real(torch.view_as_complex(v.reshape(-1, ROPE // 2, 2).contiguous()) * w).flatten(1)

        kv, k_idx = st["kv"].double(), st["k_idx"].double()
        rows = torch.cat([lat, turn(rope)], 1)
        keys = torch.cat([key[:, :IDX - ROPE], turn(key[:, IDX - ROPE:])], 1)
        for i, slot in enumerate(st["slots"].tolist()):
            if slot >= 0:
                kv[slot // st["page"], slot % st["page"]] = rows[i]
                k_idx[slot // st["page"], slot % st["page"]] = keys[i]
        return dict(kv=kv, k_idx=k_idx)
    if case["op"] == "attend":
        out = torch.empty(st["out"].shape, dtype=torch.float64, device=DEV)
        lse = torch.empty(st["lse"].shape, dtype=torch.float64, device=DEV)
        table, begin = host("table"), host("q_begin")
        for b, total in enumerate(host("seq_len").tolist()):
            pages = [st["kv"][int(p)] for p in table[b, : -(-total // st["page"])]]
            raw = torch.cat(pages)[:total]
            if st["fp8"]:
                lat = raw[:, :LATENT].contiguous().view(torch.float8_e4m3fn).to(torch.float64)
                lat = lat * raw[:, 640:644].contiguous().view(torch.float32).to(torch.float64)
                key = torch.cat([lat, raw[:, 512:640].contiguous().view(torch.bfloat16).to(torch.float64)], 1)
            else:
                key = raw.to(torch.float64)
            first, last = int(begin[b]), int(begin[b + 1])
            block = max(1, (1 << 27) // (case["heads"] * total))
            for i0 in range(first, last, block):
                i1 = min(last, i0 + block)
                limit = total - (last - torch.arange(i0, i1, device=DEV))      # last visible row
                logit = torch.einsum("nhd,sd->nhs", st["q"][i0:i1].double(), key) * st["scale"]
                far = torch.arange(total, device=DEV)[None, None, :] > limit[:, None, None]
                logit[far.expand_as(logit)] = -math.inf
                lse[i0:i1] = torch.logsumexp(logit, -1)
                out[i0:i1] = torch.einsum("nhs,sd->nhd", (logit - lse[i0:i1, :, None]).exp(), key[:, :LATENT])
        return dict(out=out, lse=lse)
    x, u, us, n_draft = host("x"), host("u").astype(np.float64), host("us").astype(np.float64), host("n_draft")
    n, d = x.shape
    tokens, n_accept = np.full((n, d + 1), -1), np.zeros(n, dtype=np.int64)
    for r in range(n):
        i = 0
        while i < n_draft[r]:
            pi = float(st["p"][r, i, int(x[r, i])])
            qi = 1.0 if st["q"] is None else float(st["q"][r, i, int(x[r, i])])
            if not u[r, i] * qi < pi:
                break
            tokens[r, i] = x[r, i]
            i += 1
        left = st["p"][r, i].double().cpu().numpy()
        if i < n_draft[r]:
            if st["q"] is None:
                rest = left.copy()
                rest[x[r, i]] = 0.0
            else:
                rest = np.maximum(left - st["q"][r, i].double().cpu().numpy(), 0.0)
            left = rest if rest.sum() > 0 else left
        cdf = np.cumsum(left)
        tokens[r, i] = int(np.searchsorted(cdf, us[r] * cdf[-1], side="right"))
        n_accept[r] = i
    return dict(tokens=_i32(tokens), n_accept=_i32(n_accept))
