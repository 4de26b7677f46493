"""Cases of the dense attention over (paged) caches and of the page operations, with their plain forms.

``run`` computes an operator in elementary torch operations, or, with ``own``, through the package's entry points
(``dense_attn``, ``idx_page_copy``, ``idx_page_update``, ``idx_page_compact``) on the same state.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "i8": torch.int8}
TRASH = 1   # spare pages behind every cache of the page operations: where a plain form sends what it need not write

# cache rows of the page operations: (trailing shape, type) of each cache that shares the page numbers
CACHES = {
    "mla": (((128,), "f16"), ((576,), "bf16")),                     # indexer keys and the latent
    "gqa": (((128,), "bf16"), ((4, 128), "bf16"), ((4, 128), "bf16")),   # raw indexer keys, K and V
    "q8": (((132,), "i8"), ((576,), "bf16")),                       # coded keys with their scale inline, the latent
    "small": (((4, 33), "f32"),),                                   # rows that are no multiple of 16 bytes
}


def _attn(name, batch, new, cached, hq, hkv, d, dtype, page, cap=0.0, window=0, slopes=False, docs=0, prefix=False,
          ragged=False):
    c = dict(kind="attn", batch=batch, new=new, cached=cached, hq=hq, hkv=hkv, d=d, dtype=dtype, page=page, cap=cap,
             window=window, slopes=slopes, docs=docs, prefix=prefix, ragged=ragged)
    return dict(c, name=name) if name else c


def _pages(name, kind, seqs, per_seq, page, caches, used, part):
    """seqs rows of a page table with at most per_seq pages each, `used` of them in use; part: the share of the slots
    that are forked (update), of the pages that are copied (copy) or of the sequences that have ended (compact)."""
    c = dict(kind=kind, seqs=seqs, per_seq=per_seq, page=page, caches=caches, used=used, part=part)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of one short sequence, the tiny f32 configuration's heads: latency is all
        _attn("one_token_f32", 1, 1, 256, 4, 1, 32, "f32", 0),
        # one decode step of 16 long sequences over 64-row pages, the block-pooled configuration's heads
        _attn("decode_gqa_bf16", 16, 1, 32768, 32, 4, 128, "bf16", 64, ragged=True),
        # a long prompt's last chunk: 4096 new tokens on 12288 cached ones
        _attn("chunk_long_bf16", 1, 4096, 16384, 32, 4, 128, "bf16", 0),
        # a dense layer beside the sparse ones: one decode step over the paged latent cache of 8 sequences
        _attn("decode_latent_bf16", 8, 1, 8192, 128, 1, 576, "bf16", 64, ragged=True),
        # capped scores in a sliding window: chunks of two sequences over small pages
        _attn("capped_window_bf16", 2, 1024, 8192, 32, 4, 128, "bf16", 16, cap=30.0, window=2048),
        # packed documents with a bidirectional prefix and a distance bias, ragged chunks, three query heads a kv head
        _attn("documents_distance_f16", 8, 512, 4096, 24, 8, 64, "f16", 64, slopes=True, docs=700, prefix=True,
              ragged=True),
        # swapping eight pages in: the smallest copy
        _pages("copy_8_pages", "copy", 8, 16, 64, "mla", 0.9, 0.07),
        # moving a long context's pages between pools of the same cache
        _pages("copy_4096_pages", "copy", 32, 320, 64, "mla", 1.0, 0.4),
        # one step of 8 short decode rows: some rows grow, some fork, one ends
        _pages("update_8_seqs", "update", 8, 128, 64, "mla", 0.7, 0.4),
        # one step of a large batch with many forks of long sequences
        _pages("update_256_seqs", "update", 256, 256, 64, "gqa", 0.5, 0.6),
        # a few sequences have ended in a small pool
        _pages("compact_small", "compact", 8, 128, 16, "q8", 0.6, 0.25),
        # a large fragmented pool
        _pages("compact_large", "compact", 64, 512, 64, "mla", 0.9, 0.4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "copy", "update", "compact"])
    while kind == "attn":
        heads = rng.choice([(4, 1, 32), (32, 4, 128), (32, 8, 128), (24, 8, 64), (16, 16, 64), (14, 2, 64), (8, 8, 96),
                            (20, 4, 80), (128, 1, 576)])
        dtype = rng.choice(["bf16", "f16", "f32"]) if heads[2] in (32, 64, 128) else rng.choice(["bf16", "f16"])
        new, cached, batch = _log(rng, 1, 4096), _log(rng, 1, 32768), _log(rng, 1, 32)
        if heads[2] == 576:     # the latent cache: bf16, few new tokens
            dtype, new = "bf16", min(new, 64)
        if rng.random() < 0.3:
            new = 1
        new = min(new, cached)
        c = _attn("", batch, new, cached, *heads, dtype, rng.choice([0, 8, 16, 32, 64, 128]),
                  cap=rng.choice([0.0, 0.0, 20.0, 50.0]) if heads[2] <= 128 else 0.0,
                  window=rng.choice([0, 0, _log(rng, 1, cached)]),
                  slopes=rng.random() < 0.25 and heads[2] <= 128, docs=rng.choice([0, 0, _log(rng, 1, cached)]),
                  prefix=rng.random() < 0.25, ragged=rng.random() < 0.7)
        w = work(c)
        dense = 4.0 * batch * new * cached * heads[0] * heads[2]
        # f32 runs at a sixteenth of the 16-bit rate or less: its calls are smaller
        most = 1.1e12 if dtype != "f32" else 5e10
        if w["bytes"] <= 1.1e9 and dense <= most and batch * cached <= 16 * 32768 and batch * new * cached * heads[0] <= 2.2e9:
            return c
    seqs, per_seq = _log(rng, 1, 256), _log(rng, 1, 512)
    page = rng.choice([1, 8, 16, 24, 64, 128])
    caches = rng.choice(sorted(CACHES))
    per_seq = max(1, min(per_seq, 2 * 2**30 // (_page_bytes(page, caches) * seqs)))
    return _pages("", kind, seqs, per_seq, page, caches, rng.uniform(0.3, 1.0), rng.uniform(0.05, 0.9))


# --------------------------------------------------------------------------------------------- inputs

def _page_bytes(page, caches):
    return page * sum(math.prod(s) * torch.empty((), dtype=DTYPES[t]).element_size() for s, t in CACHES[caches])


def _lengths(case):
    """Host numbers of an attention case: cached tokens and new tokens of each sequence."""
    B, T, N = case["batch"], case["new"], case["cached"]
    if not case["ragged"]:
        return [N] * B, [min(T, N)] * B
    r = np.random.RandomState(B * 1000003 + T * 101 + N)
    n_kv = [int(x) for x in r.randint(max(1, N // 2), N + 1, B)]
    n_kv[0] = N
    n_new = [min(n, int(x)) for n, x in zip(n_kv, r.randint(max(1, T // 2), T + 1, B))]
    return n_kv, n_new


def _positions(case):
    """Host arrays of an attention case: q_pos, doc_start (or None), prefix_len (or None), as rows need them."""
    n_kv, n_new = _lengths(case)
    B, T = case["batch"], case["new"]
    pos = np.full((B, T), -1, np.int64)
    for b in range(B):
        pos[b, :n_new[b]] = np.arange(n_kv[b] - n_new[b], n_kv[b])
    r = np.random.RandomState(B * 7919 + T * 31 + case["cached"])
    docs = prefix = None
    if case["docs"]:
        docs = np.zeros((B, T), np.int64)
        for b in range(B):
            cuts = np.unique(np.concatenate([[0], r.randint(0, n_kv[b], max(1, n_kv[b] // case["docs"]))]))
            docs[b] = cuts[np.searchsorted(cuts, np.maximum(pos[b], 0), side="right") - 1]
    if case["prefix"]:
        prefix = np.array([r.randint(0, n + 1) for n in n_kv], np.int64)
    return np.array(n_kv), pos, docs, prefix


def _bounds(case):
    """[lo, hi) of the positions that each row sees (host, int64 [B, T])."""
    n_kv, pos, docs, prefix = _positions(case)
    hi = pos + 1
    if prefix is not None:
        hi = np.maximum(hi, prefix[:, None])
    hi = np.where(pos < 0, 0, np.minimum(hi, n_kv[:, None]))
    lo = np.zeros_like(pos)
    if docs is not None:
        lo = np.maximum(lo, docs)
    if case["window"]:
        lo = np.maximum(lo, pos - case["window"] + 1)
    return lo, hi


def _prepare_attn(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    B, T, N, Hq, Hkv, d, page = (case[k] for k in ("batch", "new", "cached", "hq", "hkv", "d", "page"))
    dt = DTYPES[case["dtype"]]
    latent = d == 576
    n_kv, pos, docs, prefix = _positions(case)
    i32 = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)  # noqa: E731
    P = -(-N // page) if page else 0
    rows = B * P * page if page else B * N

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)
    q = rand(B * T, Hq, d)
    k = rand(rows, Hkv, d) if not latent else rand(rows, d)
    v = None if latent else rand(rows, Hkv, d)
    table = None
    s = {"case": case, "q": q, "k": k, "v": v, "scale": 1 / math.sqrt(192 if latent else d), "n_kv": i32(n_kv),
         "pos": i32(pos.reshape(-1)), "docs": i32(None if docs is None else docs.reshape(-1)), "prefix": i32(prefix),
         "slopes": None}
    j = torch.arange(N, device="cuda")
    if page:
        table = torch.randperm(B * P, generator=g, device="cuda").to(torch.int32).view(B, P)
        s["rows"] = table.long()[:, j // page] * page + j % page
    else:
        s["rows"] = torch.arange(B, device="cuda")[:, None] * N + j
    s["table"] = table
    # rows that hold no token yet: whatever a page held before
    free = torch.ones(rows, dtype=torch.bool, device="cuda")
    free[s["rows"][j[None] < s["n_kv"][:, None]]] = False
    for c in (k, v):
        if c is not None:
            c[free] = float("nan")
    if case["slopes"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device="cuda", dtype=torch.float32) / Hq)
    return s


def _page_state(case, seed):
    """Host numbers of a page case: the table, the lengths and what the call asks for."""
    r = np.random.RandomState(seed % (1 << 31))
    B, S, page = case["seqs"], case["per_seq"], case["page"]
    n_pages = B * S + (B * S) // 4 + 8
    most = max(1, int(round(S * case["used"])))
    n_len = r.randint(max(0, most - 1 - most // 4) * page, most * page + 1, B)
    need = -(-n_len // page)
    table = np.full((B, S), -1, np.int32)
    order = r.permutation(n_pages)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    held = np.zeros(n_pages, np.uint8)
    held[order[at:at + min(4, (n_pages - at) // 4)]] = 1
    return r, n_pages, n_len, table, held


def _prepare_pages(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r, n_pages, n_len, table, held = _page_state(case, seed)
    B, S, page = case["seqs"], case["per_seq"], case["page"]
    caches = []
    for shape, t in CACHES[case["caches"]]:
        full = ((n_pages + TRASH) * page,) + shape
        if t == "i8":
            caches.append(torch.randint(-127, 128, full, generator=g, device="cuda", dtype=torch.int8))
        else:
            caches.append(torch.randn(full, generator=g, device="cuda", dtype=DTYPES[t]))
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", torch.int32)  # noqa: E731
    s = {"case": case, "n_pages": n_pages, "caches": caches, "live": [c[:n_pages * page] for c in caches],
         "table": i32(table), "held": torch.from_numpy(held).cuda()}
    if case["kind"] == "copy":
        n = max(1, min(n_pages // 2, int(round(B * S * case["part"]))))
        order = r.permutation(n_pages)
        s["src"], s["dst"] = i32(order[:n]), i32(order[n:2 * n])
    elif case["kind"] == "update":
        # most rows go on, growing by a token; some give way to forks of others at some length; some end
        parent = np.arange(B)
        keep = n_len.copy()
        fork = r.rand(B) < case["part"]
        parent[fork] = r.randint(0, B, int(fork.sum()))
        keep = n_len[parent]
        cut = fork & (r.rand(B) < 0.5)
        keep[cut] = (keep[cut] * r.rand(int(cut.sum()))).astype(np.int64)
        new = np.minimum(keep + r.choice([1, 1, 1, page], B), S * page)
        end = r.rand(B) < 0.1
        parent[end], keep[end], new[end] = -1, 0, 0
        s["parent"], s["keep"], s["new"] = i32(parent), i32(keep), i32(new)
    else:
        ended = r.rand(B) < case["part"]
        s["len"] = i32(np.where(ended, 0, n_len))
    return s


def prepare(case, seed):
    return _prepare_attn(case, seed) if case["kind"] == "attn" else _prepare_pages(case, seed)


# --------------------------------------------------------------------------------------------- plain forms

def _plain_attn(s):
    c = s["case"]
    B, T, N, Hq, Hkv, d = (c[k] for k in ("batch", "new", "cached", "hq", "hkv", "d"))
    G = Hq // Hkv
    j = torch.arange(N, device="cuda")
    n_kv = s["n_kv"].long()[:, None]
    p = s["pos"].long().view(B, T)
    hi = p + 1
    if s["prefix"] is not None:
        hi = torch.maximum(hi, s["prefix"].long()[:, None])
    hi = torch.where(p < 0, 0, torch.minimum(hi, n_kv))
    lo = torch.zeros_like(p)
    if s["docs"] is not None:
        lo = torch.maximum(lo, s["docs"].long().view(B, T))
    if c["window"]:
        lo = torch.maximum(lo, p - c["window"] + 1)
    seen = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None, None]                      # [B, 1, 1, T, N]
    held = (j < n_kv)[..., None, None]
    k = s["k"][s["rows"]].view(B, N, Hkv, d)
    v = k[..., :512] if s["v"] is None else s["v"][s["rows"]].view(B, N, Hkv, d)
    k = torch.where(held, k, 0).float().permute(0, 2, 3, 1)                                   # [B, Hkv, d, N]
    v = torch.where(held, v, 0).float().permute(0, 2, 1, 3)                                   # [B, Hkv, N, dv]
    q = s["q"].float().view(B, T, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, d)
    x = (q @ k).view(B, Hkv, G, T, N).mul_(s["scale"])
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, Hkv, G, 1, 1) * (p[..., None] - j).abs().float()[:, None, None]
    x = x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    none = m == -math.inf
    x = x.sub_(m.masked_fill(none, 0)).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x.view(B, Hkv, G * T, N) @ v).view(B, Hkv, G, T, -1) / total.masked_fill(none, 1)
    lse = (m + total.log()).squeeze(-1)
    return (out.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, -1).to(s["q"].dtype),
            lse.permute(0, 3, 1, 2).reshape(B * T, Hq))


def _by_page(s):
    return [c.view(s["n_pages"] + TRASH, s["case"]["page"], *c.shape[1:]) for c in s["caches"]]


def _plain_copy(s):
    for c in _by_page(s):
        c[s["dst"].long()] = c[s["src"].long()]
    return s["live"]


def _plain_update(s):
    n_pages, page = s["n_pages"], s["case"]["page"]
    B, S = s["table"].shape
    dev = "cuda"
    i = torch.arange(S, device=dev)
    b = torch.arange(B, device=dev)
    keep, new = s["keep"].long(), s["new"].long()
    whole, part, need = keep // page, keep % page, (new + page - 1) // page
    old = s["table"].long()[s["parent"].long().clamp(min=0)]
    shared = i < whole[:, None]
    used = torch.zeros(n_pages + 1, dtype=torch.bool, device=dev)
    used[:n_pages] = s["held"].bool()
    used[torch.where(shared, old, n_pages)] = True
    last = torch.where(part > 0, old.gather(1, whole.clamp(max=S - 1)[:, None]).squeeze(1), n_pages)
    first = torch.full((n_pages + 1,), B, device=dev).scatter_reduce_(0, last, b, "amin")
    stays = (part > 0) & ~used[last] & (first[last] == b)
    used[torch.where(stays, last, n_pages)] = True
    used = used[:n_pages]
    stays_at = stays[:, None] & (i == whole[:, None])
    fresh = (i >= whole[:, None]) & (i < need[:, None]) & ~stays_at
    free = torch.argsort(used.to(torch.uint8), stable=True)
    rank = (fresh.reshape(-1).cumsum(0) - 1).clamp(0, n_pages - 1).view(B, S)
    table = torch.where(fresh, free[rank], torch.where(shared | stays_at, old, -1))
    left = n_pages - used.sum() - fresh.sum()
    # the kept rows of the pages that are copied; every other row goes to the spare page and back
    copied = ((part > 0) & ~stays & (left >= 0))[:, None]
    row = torch.arange(page, device=dev)
    moves = copied & (row < part[:, None])
    dst = table.gather(1, whole.clamp(max=S - 1)[:, None])
    src = torch.where(moves, last[:, None] * page + row, n_pages * page + row)
    dst = torch.where(moves, dst * page + row, n_pages * page + row)
    for c in s["caches"]:
        c[dst] = c[src]
    return [table.to(torch.int32), left.to(torch.int32).view(1)] + s["live"]


def _plain_compact(s):
    n_pages, page = s["n_pages"], s["case"]["page"]
    B, S = s["table"].shape
    i = torch.arange(S, device="cuda")
    p = torch.arange(n_pages, device="cuda")
    old = s["table"].long()
    live = i < ((s["len"].long() + page - 1) // page)[:, None]
    used = torch.zeros(n_pages + 1, dtype=torch.bool, device="cuda")
    used[torch.where(live, old, n_pages)] = True
    held = s["held"].bool()
    used = used[:n_pages] | held
    n = used.sum()
    moves = used & ~held & (p >= n)
    holes = ~used & (p < n)
    most = max(1, n_pages // 2)     # each moving page has a free number below it
    src = torch.argsort((~moves).to(torch.uint8), stable=True)[:most]
    dst = torch.argsort((~holes).to(torch.uint8), stable=True)[:most]
    real = torch.arange(most, device="cuda") < moves.sum()
    rank = (moves.cumsum(0) - 1).clamp(0, most - 1)
    remap = torch.where(moves, dst[rank], p)
    table = torch.where(live, remap[old.clamp(min=0)], -1)
    src, dst = torch.where(real, src, n_pages), torch.where(real, dst, n_pages)
    for c in _by_page(s):
        c[dst] = c[src]
    return [table.to(torch.int32), n.to(torch.int32).view(1), remap.to(torch.int32)] + s["live"]


# --------------------------------------------------------------------------------------------- the framework's calls

def _own(s):
    import lightning_indexer_top_gb300 as L
    c = s["case"]
    if c["kind"] == "attn":
        lse = torch.empty(s["q"].shape[:2], device="cuda", dtype=torch.float32)
        batch = L.Batch(s["n_kv"], c["new"], c["cached"], kv_seq_stride=c["cached"], q_pos=s["pos"],
                        page_table=s["table"], page_size=c["page"])
        out = L.dense_attn(s["q"], s["k"], s["v"], batch, s["scale"], softcap=c["cap"], window=c["window"],
                           slopes=s["slopes"], doc_start=s["docs"], prefix_len=s["prefix"], lse=lse)
        return out, lse
    if c["kind"] == "copy":
        L.idx_page_copy(s["live"], c["page"], s["src"], s["dst"])
        return s["live"]
    if c["kind"] == "update":
        table, left = L.idx_page_update(s["table"], s["parent"], s["keep"], s["new"], c["page"], s["live"],
                                        held=s["held"])
        return [table, left] + s["live"]
    table, n, remap = L.idx_page_compact(s["table"], s["len"], c["page"], s["live"], held=s["held"])
    return [table, n, remap] + s["live"]


def run(state):
    if own:
        return _own(state)
    return {"attn": _plain_attn, "copy": _plain_copy, "update": _plain_update,
            "compact": _plain_compact}[state["case"]["kind"]](state)


# --------------------------------------------------------------------------------------------- floors

def work(case):
    if case["kind"] == "attn":
        B, Hq, Hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
        dv = 512 if d == 576 else d
        lo, hi = _bounds(case)
        n = np.maximum(hi - lo, 0)
        size = torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
        # cached rows that some row of the sequence sees
        seen = 0
        for b in range(B):
            edge = np.zeros(case["cached"] + 1, np.int64)
            ok = n[b] > 0
            np.add.at(edge, lo[b][ok], 1)
            np.add.at(edge, hi[b][ok], -1)
            seen += int((np.cumsum(edge) > 0).sum())
        kv = Hkv * (d if d == 576 else 2 * d) * size
        rows = int((n > 0).sum())
        return {"bytes": seen * kv + rows * Hq * (d * size) + n.size * Hq * (dv * size + 4),
                "flops": 2.0 * float(n.sum()) * Hq * (d + dv)}
    _, n_pages, n_len, table, held = _page_state(case, 1)
    B, S, page = case["seqs"], case["per_seq"], case["page"]
    pb = _page_bytes(page, case["caches"])
    if case["kind"] == "copy":
        n = max(1, min(n_pages // 2, int(round(B * S * case["part"]))))
        return {"bytes": 2 * n * pb + 8 * n, "flops": 0}
    if case["kind"] == "update":
        # about part * 0.9 of the rows copy half a page; the tables are read and written, the held marks read
        return {"bytes": 8 * B * S + 12 * B + n_pages + int(0.9 * case["part"] * B * pb), "flops": 0}
    alive = int((1 - case["part"]) * sum(-(-n_len // page)))
    used = alive + int(held.sum())
    moves = int(alive * max(0, n_pages - used) / n_pages)
    return {"bytes": 8 * B * S + 4 * B + 5 * n_pages + 2 * moves * pb, "flops": 0}


# --------------------------------------------------------------------------------------------- 64-bit values

def _exact_attn(case, seed):
    B, T, N, Hq, Hkv, d = (case[k] for k in ("batch", "new", "cached", "hq", "hkv", "d"))
    s = _prepare_attn(case, seed)
    lo, hi = (torch.from_numpy(a).cuda() for a in _bounds(case))
    _, pos, _, _ = _positions(case)
    G, dv = Hq // Hkv, 512 if s["v"] is None else d
    if 2.0 * B * T * N * Hq * (d + dv) > 8e12:
        return None
    out = torch.zeros(B * T, Hq, dv, dtype=torch.float64, device="cuda")
    lse = torch.full((B * T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(B, T, Hq, d)
    for b in range(B):
        n = int(s["n_kv"][b])
        at = s["rows"][b, :n]
        j = torch.arange(n, device="cuda")
        seen = (j[None] >= lo[b][:, None]) & (j[None] < hi[b][:, None])
        far = (torch.from_numpy(pos[b]).cuda()[:, None] - j[None]).abs().double()
        some = seen.any(1)
        for g in range(Hkv):
            kk = (s["k"][at] if s["v"] is None else s["k"][at, g]).double()
            vv = kk[:, :dv] if s["v"] is None else s["v"][at, g].double()
            for h in range(g * G, (g + 1) * G) if T > 1 else [slice(g * G, (g + 1) * G)]:
                qq = q[b, :, h] if T > 1 else q[b, 0, h]
                y = torch.matmul(qq, kk.T) * s["scale"]
                if case["cap"]:
                    y = torch.tanh(y / case["cap"]) * case["cap"]
                if s["slopes"] is not None:
                    sl = s["slopes"][h].double()
                    y = y - (sl * far if T > 1 else sl[:, None] * far)
                y = torch.where(seen, y, -math.inf)
                t = torch.logsumexp(y, -1)
                w = torch.exp(y - torch.where(some, t, 0.0)[:, None])
                o = torch.matmul(w, vv)
                if T > 1:
                    lse[b * T:(b + 1) * T, h] = t
                    out[b * T:(b + 1) * T, h] = o
                else:
                    lse[b, h] = t
                    out[b, h] = o
    return out, lse


def _exact_pages(case, seed):
    """The page operations step by step on the host; the pages follow on the device."""
    s = _prepare_pages(case, seed)
    n_pages, page, B, S = s["n_pages"], case["page"], case["seqs"], case["per_seq"]
    old = s["table"].tolist()
    held = set(np.nonzero(s["held"].cpu().numpy())[0].tolist())
    first, moves = [], []      # whole numbers that come first, and (source page, target page, rows)
    if case["kind"] == "copy":
        moves = [(a, b, page) for a, b in zip(s["src"].tolist(), s["dst"].tolist())]
    elif case["kind"] == "update":
        parent, keep, new = s["parent"].tolist(), s["keep"].tolist(), s["new"].tolist()
        rows = [old[parent[b]][:keep[b] // page] if keep[b] else [] for b in range(B)]
        taken = set(held)
        for r in rows:
            taken.update(r)
        kept = {}
        for b in range(B):
            if keep[b] % page:
                last = old[parent[b]][keep[b] // page]
                if last not in taken:
                    taken.add(last)
                    kept[b] = last
        free = iter([p for p in range(n_pages) if p not in taken])
        n_new = 0
        for b in range(B):
            want = -(-new[b] // page)
            if b in kept:
                rows[b] = rows[b] + [kept[b]]
            elif keep[b] % page:
                p = next(free)
                n_new += 1
                moves.append((old[parent[b]][keep[b] // page], p, keep[b] % page))
                rows[b] = rows[b] + [p]
            more = [next(free) for _ in range(want - len(rows[b]))]
            n_new += len(more)
            rows[b] = rows[b] + more + [-1] * (S - want)
        first = [torch.tensor(rows, dtype=torch.int32).view(B, S), torch.tensor([n_pages - len(taken) - n_new], dtype=torch.int32)]
    else:
        need = [-(-x // page) for x in s["len"].tolist()]
        used = held.union(*[set(old[b][:need[b]]) for b in range(B)])
        n = len(used)
        to = dict(zip(sorted(p for p in used - held if p >= n), [p for p in range(n) if p not in used]))
        moves = [(a, b, page) for a, b in to.items()]
        rows = [[to.get(p, p) for p in old[b][:need[b]]] + [-1] * (S - need[b]) for b in range(B)]
        first = [torch.tensor(rows, dtype=torch.int32).view(B, S), torch.tensor([n], dtype=torch.int32),
                 torch.tensor([to.get(p, p) for p in range(n_pages)], dtype=torch.int32)]
    m = np.array(moves, np.int64).reshape(-1, 3)
    n_rows = m[:, 2].sum()
    within = np.arange(n_rows) - np.repeat(np.cumsum(m[:, 2]) - m[:, 2], m[:, 2])
    src = torch.from_numpy(np.repeat(m[:, 0], m[:, 2]) * page + within).cuda()
    dst = torch.from_numpy(np.repeat(m[:, 1], m[:, 2]) * page + within).cuda()
    for c in s["live"]:
        c.index_copy_(0, dst, c.index_select(0, src))
    return first + s["live"]


def exact(case, seed):
    return _exact_attn(case, seed) if case["kind"] == "attn" else _exact_pages(case, seed)
