"""Cases of appending to caches (with the position rotation, also into 4 bits), of attention over a 4-bit cache and of a
beam search's step, with their plain forms.

``run`` computes an operator in elementary torch operations, or, with ``own``, through the package's entry points
(``idx_cache_append``, ``idx_cache_append_q4`` with ``idx_cache_read_q4``, ``dense_attn_q4``, ``idx_beam_step``) on the
same state.

A row of a 4-bit cache: for each kv head d/2 bytes of codes (column c in byte c/2, the even one in the low half), then
for each kv head scale and minimum in f32, then bytes that make the row a multiple of 16; code n stands for
scale * n + minimum.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _append(name, kind, batch, new, room, hq, hkv, dk, dv, dtype, page, rot, start=0, inter=False, ragged=False,
            base=10000.0):
    """batch sequences of at most `room` cached positions get at most `new` rows each; hq 0: no queries beside them; dv 0:
    no values (the latent); rot columns of each head are rotated, from `start` on, in neighbouring pairs (inter) or halves."""
    c = dict(kind=kind, batch=batch, new=new, room=room, hq=hq, hkv=hkv, dk=dk, dv=dv, dtype=dtype, page=page, rot=rot,
             start=start, inter=inter, ragged=ragged, base=base)
    return dict(c, name=name) if name else c


def _attn(name, batch, new, cached, hq, hkv, d, dtype, page, cap=0.0, window=0, ragged=False):
    c = dict(kind="attn", batch=batch, new=new, cached=cached, hq=hq, hkv=hkv, d=d, dtype=dtype, page=page, cap=cap,
             window=window, ragged=ragged)
    return dict(c, name=name) if name else c


def _beam(name, seqs, beams, out, vocab, dtype, length, ended):
    """beams rows of logits for each sequence, `out` of their continuations are kept; histories of at most `length`
    tokens; a share `ended` of the beams has ended."""
    c = dict(kind="beam", seqs=seqs, beams=beams, out=out, vocab=vocab, dtype=dtype, length=length, ended=ended)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one new token of one short sequence, the tiny f32 configuration's heads: latency is all
        _append("append_token_f32", "append", 1, 1, 256, 4, 1, 32, 32, "f32", 0, 32),
        # the rows of one decode step: 16 long sequences over 64-row pages, the block-pooled configuration's heads
        _append("append_decode_bf16", "append", 16, 1, 16384, 32, 4, 128, 128, "bf16", 64, 128, ragged=True, base=1e6),
        # a chunk of a long prompt with its queries
        _append("append_chunk_bf16", "append", 1, 4096, 16384, 32, 4, 128, 128, "bf16", 64, 128, base=1e6),
        # chunks of eight prompts into the paged latent cache, whose last 64 columns carry the position
        _append("append_latent_bf16", "append", 8, 1024, 2048, 0, 1, 576, 0, "bf16", 16, 64, 512, True, True),
        # one decode step into 4-bit pages, heads of 64, half of whose columns are rotated
        _append("append4_decode_f16", "append4", 64, 1, 512, 24, 8, 64, 64, "f16", 16, 32, ragged=True),
        # prompts into 4-bit pages
        _append("append4_chunk_bf16", "append4", 4, 2048, 4096, 32, 8, 128, 128, "bf16", 64, 128, ragged=True),
        # one new token on a short 4-bit cache
        _attn("attn4_token_f16", 1, 1, 256, 8, 2, 64, "f16", 0),
        # one decode step of 16 long sequences over 4-bit pages
        _attn("attn4_decode_bf16", 16, 1, 32768, 32, 4, 128, "bf16", 64, ragged=True),
        # four proposed tokens of each sequence are looked at in a sliding window, capped scores, three heads a kv head
        _attn("attn4_window_f16", 8, 4, 8192, 24, 8, 64, "f16", 16, cap=30.0, window=2048, ragged=True),
        # a long prompt's last chunk
        _attn("attn4_chunk_bf16", 1, 4096, 16384, 32, 4, 128, "bf16", 64),
        # a search of four beams for one request
        _beam("beam_4_f32", 1, 4, 4, 32000, "f32", 64, 0.0),
        # 64 requests of eight beams each that keep twice as many continuations, some beams have ended
        _beam("beam_64x8_bf16", 64, 8, 16, 131072, "bf16", 512, 0.1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "append4", "attn", "attn", "beam"])
    if kind in ("append", "append4"):
        four = kind == "append4"
        hq, hkv, dk, dv = rng.choice([(32, 4, 128, 128), (32, 8, 128, 128), (24, 8, 64, 64), (16, 16, 64, 64), (14, 2, 64, 64),
                                      (8, 8, 96, 96), (20, 4, 80, 80)] + ([] if four else [(4, 1, 32, 32), (0, 1, 576, 0),
                                                                                          (0, 1, 128, 0), (5, 5, 20, 12)]))
        dtype = rng.choice(["bf16", "f16", "f32"])
        batch, room = _log(rng, 1, 64), _log(rng, 1, 16384)
        room = min(room, max(1, 131072 // batch))
        new = min(room, max(1, 16384 // batch), rng.choice([1, _log(rng, 1, 4096)]))
        rot = rng.choice([dk, dk // 2 // 4 * 4, 0]) if dk != 576 else 64
        if rng.random() < 0.25:
            hq = 0
        return _append("", kind, batch, new, room, hq, hkv, dk, dv, dtype, rng.choice([0, 1, 8, 16, 24, 64, 128]), rot,
                       512 if dk == 576 else rng.choice([0, dk - rot]), rng.random() < 0.3, rng.random() < 0.7,
                       rng.choice([1e4, 1e6]))
    while kind == "attn":
        heads = rng.choice([(32, 4, 128), (32, 8, 128), (32, 2, 128), (24, 8, 64), (16, 16, 64), (14, 2, 64), (8, 8, 96),
                            (20, 4, 80), (4, 1, 32)])
        dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
        new, cached, batch = _log(rng, 1, 4096), _log(rng, 1, 32768), _log(rng, 1, 32)
        if rng.random() < 0.5:
            new = rng.choice([1, 1, 2, 5])
        new = min(new, cached)
        c = _attn("", batch, new, cached, *heads, dtype, rng.choice([0, 1, 8, 16, 24, 64, 128]),
                  cap=rng.choice([0.0, 0.0, 20.0, 50.0]), window=rng.choice([0, 0, _log(rng, 1, cached)]),
                  ragged=rng.random() < 0.7)
        dense = 4.0 * batch * new * cached * heads[0] * heads[2]
        # f32 runs at a sixteenth of the 16-bit rate or less: its calls are smaller
        if dense <= (1.1e12 if dtype != "f32" else 5e10) and batch * cached <= 16 * 32768 and batch * new * cached * heads[0] <= 2.2e9:
            return c
    while True:
        seqs, beams, vocab = _log(rng, 1, 64), _log(rng, 1, 16), _log(rng, 100, 200000)
        out = min(32, vocab, rng.choice([1, beams, 2 * beams, 2 * beams + 1]))
        if seqs * beams * vocab <= 64 * 8 * 131072:
            return _beam("", seqs, beams, out, vocab, rng.choice(["bf16", "f16", "f32"]), _log(rng, 1, 2048),
                         rng.choice([0.0, 0.0, 0.2]))


# --------------------------------------------------------------------------------------------- inputs

def _row_bytes(heads, d):
    return -(-heads * (d // 2 + 8) // 16) * 16


def _lengths(case):
    """Host numbers: cached tokens (the new ones among them) and new tokens of each sequence."""
    B, T, N = case["batch"], case["new"], case["cached"] if case["kind"] == "attn" else case["room"]
    if not case["ragged"]:
        return np.full(B, N), np.full(B, min(T, N))
    r = np.random.RandomState(B * 1000003 + T * 101 + N)
    n_kv = r.randint(max(1, N // 2), N + 1, B)
    n_kv[0] = N
    return n_kv, np.minimum(n_kv, r.randint(max(1, T // 2), T + 1, B))


def _positions(case):
    """Host arrays: cached tokens of each sequence, the position of each new row (-1: padding)."""
    n_kv, n_new = _lengths(case)
    t = np.arange(case["new"])
    return n_kv, np.where(t < n_new[:, None], (n_kv - n_new)[:, None] + t, -1)


def _where(case, g, N):
    """The page table (or None), the cache rows there are, and the cache row of each position [B, N]."""
    B, page = case["batch"], case["page"]
    j = torch.arange(N, device="cuda")
    if not page:
        return None, B * N, torch.arange(B, device="cuda")[:, None] * N + j
    P = -(-N // page)
    table = torch.randperm(B * P, generator=g, device="cuda").to(torch.int32).view(B, P)
    return table, B * P * page, table.long()[:, j // page] * page + j % page


def _prepare_append(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    B, T, N, hq, hkv, dk, dv = (case[k] for k in ("batch", "new", "room", "hq", "hkv", "dk", "dv"))
    dt = DTYPES[case["dtype"]]
    n_kv, pos = _positions(case)
    table, rows, at = _where(case, g, N)
    # queries, keys and values are columns of one projection's output
    proj = torch.randn((B * T, hq * dk + hkv * (dk + dv)), generator=g, device="cuda", dtype=torch.float32).to(dt)
    q, k, v = proj.split([hq * dk, hkv * dk, hkv * dv], dim=1)
    s = {"case": case, "table": table, "q": q.unflatten(1, (hq, dk)) if hq else None, "k": k.unflatten(1, (hkv, dk)),
         "v": v.unflatten(1, (hkv, dv)) if dv else None, "n_kv": torch.from_numpy(n_kv).to("cuda", torch.int32),
         "pos": torch.from_numpy(pos.reshape(-1)).to("cuda", torch.int32), "inv_freq": None}
    if case["rot"]:
        i = torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64)
        s["inv_freq"] = (case["base"] ** (-i / case["rot"])).float()
    p = s["pos"].long().view(B, T)
    s["rows"] = at.gather(1, p.clamp(min=0)).view(-1)      # cache row of each new row (of padding: any)
    if case["kind"] == "append":
        s["k_cache"] = torch.randn((rows, hkv, dk), generator=g, device="cuda", dtype=dt)
        s["v_cache"] = torch.randn((rows, hkv, dv), generator=g, device="cuda", dtype=dt) if dv else None
    else:
        s["k_cache"] = torch.randint(0, 256, (rows, _row_bytes(hkv, dk)), generator=g, device="cuda", dtype=torch.uint8)
        s["v_cache"] = torch.randint(0, 256, (rows, _row_bytes(hkv, dv)), generator=g, device="cuda", dtype=torch.uint8)
        s["k_out"] = torch.zeros((B * T, hkv, dk), device="cuda", dtype=dt)
        s["v_out"] = torch.zeros((B * T, hkv, dv), device="cuda", dtype=dt)
    return s


def _pack(codes, scale, low, heads, d):
    """Rows of a 4-bit cache from codes [n, heads, d], scale and minimum [n, heads]."""
    c = codes.to(torch.uint8)
    c = (c[..., 0::2] | (c[..., 1::2] << 4)).flatten(1)
    pairs = torch.stack([scale.float(), low.float()], -1).flatten(1).contiguous().view(torch.uint8)
    rest = torch.zeros((c.shape[0], _row_bytes(heads, d) - c.shape[1] - pairs.shape[1]), device=c.device, dtype=torch.uint8)
    return torch.cat([c, pairs, rest], 1)


def _prepare_attn(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    B, T, N, Hq, Hkv, d = (case[k] for k in ("batch", "new", "cached", "hq", "hkv", "d"))
    n_kv, pos = _positions(case)
    table, rows, at = _where(case, g, N)
    q = torch.randn((B * T, Hq, d), generator=g, device="cuda", dtype=torch.float32).to(DTYPES[case["dtype"]])
    s = {"case": case, "q": q, "scale": 1 / math.sqrt(d), "table": table, "rows": at,
         "n_kv": torch.from_numpy(n_kv).to("cuda", torch.int32),
         "pos": torch.from_numpy(pos.reshape(-1)).to("cuda", torch.int32)}
    # rows that hold no token: bytes that are no numbers
    held = torch.zeros(rows, dtype=torch.bool, device="cuda")
    held[at[torch.arange(N, device="cuda") < s["n_kv"].long()[:, None]]] = True
    for name in ("k_cache", "v_cache"):
        cache = torch.empty((rows, _row_bytes(Hkv, d)), device="cuda", dtype=torch.uint8)
        for r0 in range(0, rows, 65536):
            x = torch.randn((min(65536, rows - r0), Hkv, d), generator=g, device="cuda")
            low, high = x.aminmax(dim=-1)
            scale = (high - low) / 15
            codes = ((x - low[..., None]) / scale[..., None]).round_().clamp_(0, 15)
            cache[r0:r0 + x.shape[0]] = _pack(codes, scale, low, Hkv, d)
        cache[~held] = 255
        s[name] = cache
    return s


def _prepare_beam(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    B, W, V, S = case["seqs"], case["beams"], case["vocab"], case["length"]
    rows = B * W
    logits = torch.randn((rows, V), generator=g, device="cuda").mul_(2.5).to(DTYPES[case["dtype"]])
    scores = torch.rand(rows, generator=g, device="cuda") * -6
    lengths = torch.full((rows,), S - 1, device="cuda", dtype=torch.int32)
    done = torch.rand(rows, generator=g, device="cuda") < case["ended"]
    short = (torch.rand(rows, generator=g, device="cuda") * S).to(torch.int32)
    lengths = torch.where(done, short, lengths)
    history = torch.randint(0, V, (rows, S), generator=g, device="cuda", dtype=torch.int32)
    return {"case": case, "logits": logits, "scores": scores, "done": done.to(torch.uint8), "lengths": lengths,
            "history": history, "history_out": torch.zeros((B * case["out"], S), device="cuda", dtype=torch.int32),
            "end": V // 2}


def prepare(case, seed):
    return {"append": _prepare_append, "append4": _prepare_append, "attn": _prepare_attn, "beam": _prepare_beam}[case["kind"]](case, seed)


# --------------------------------------------------------------------------------------------- plain forms

def _rotated(s, x):
    """x [rows, heads, dk] in 64 bits, turned by its rows' positions."""
    c = s["case"]
    x = x.double()
    n, a = c["rot"], c["start"]
    if not n:
        return x
    angle = s["pos"].clamp(min=0).double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    r = x[..., a:a + n]
    if c["inter"]:
        u, w = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
    else:
        u, w = r[..., :n // 2], r[..., n // 2:]
        r = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    r = torch.where((s["pos"] >= 0)[:, None, None], r, x[..., a:a + n])
    return torch.cat([x[..., :a], r, x[..., a + n:]], -1)


def _put(s, cache, x):
    """Rows of x into the cache; padding rows put back what their place holds (that of their own position 0's row)."""
    real = (s["pos"] >= 0).view([-1] + [1] * (x.dim() - 1))
    B, T = s["case"]["batch"], s["case"]["new"]
    # a padding row writes what the sequence's first row, which is none, writes
    first = torch.arange(B, device="cuda").repeat_interleave(T) * T
    src = torch.where(real.view(-1), torch.arange(B * T, device="cuda"), first)
    cache[s["rows"][src]] = x.to(cache.dtype)[src]


def _plain_append(s):
    q = None if s["q"] is None else _rotated(s, s["q"]).to(s["q"].dtype)
    _put(s, s["k_cache"], _rotated(s, s["k"]))
    if s["v"] is not None:
        _put(s, s["v_cache"], s["v"])
    return [x for x in (q, s["k_cache"], s["v_cache"]) if x is not None]


def _quantized(x):
    """Codes, scale and minimum of rows in 64 bits."""
    low, high = x.aminmax(dim=-1)
    span = (high - low)[..., None]
    codes = torch.where(span > 0, (x - low[..., None]) * 15 / span, 0).round()
    return codes, (high - low) / 15, low


def _values(cache, heads, d):
    """The f32 values [n, heads, d] that rows of a 4-bit cache stand for."""
    n = cache.shape[0]
    c = cache[:, :heads * d // 2].view(n, heads, d // 2)
    codes = torch.stack([c & 15, c >> 4], -1).flatten(-2).float()
    pairs = cache[:, heads * d // 2:heads * (d // 2 + 8)].contiguous().view(torch.float32).view(n, heads, 2)
    return codes * pairs[..., :1] + pairs[..., 1:]


def _plain_append4(s):
    c = s["case"]
    q = None if s["q"] is None else _rotated(s, s["q"]).to(s["q"].dtype)
    _put(s, s["k_cache"], _pack(*_quantized(_rotated(s, s["k"])), c["hkv"], c["dk"]))
    _put(s, s["v_cache"], _pack(*_quantized(s["v"].double()), c["hkv"], c["dv"]))
    real = (s["pos"] >= 0)[:, None, None]
    k = torch.where(real, _values(s["k_cache"][s["rows"]], c["hkv"], c["dk"]).to(s["k"].dtype), s["k_out"])
    v = torch.where(real, _values(s["v_cache"][s["rows"]], c["hkv"], c["dv"]).to(s["v"].dtype), s["v_out"])
    return [k, v] if q is None else [q, k, v]


def _plain_attn(s):
    c = s["case"]
    B, T, N, Hq, Hkv, d = (c[k] for k in ("batch", "new", "cached", "hq", "hkv", "d"))
    G = Hq // Hkv
    j = torch.arange(N, device="cuda")
    n_kv = s["n_kv"].long()[:, None]
    p = s["pos"].long().view(B, T)
    hi = torch.where(p < 0, 0, torch.minimum(p + 1, n_kv))
    lo = (p - c["window"] + 1).clamp(min=0) if c["window"] else torch.zeros_like(p)
    seen = ((j >= lo[..., None]) & (j < hi[..., None]))[:, None, None]                      # [B, 1, 1, T, N]
    held = (j < n_kv)[..., None, None]
    k = _values(s["k_cache"][s["rows"].view(-1)], Hkv, d).view(B, N, Hkv, d)
    v = _values(s["v_cache"][s["rows"].view(-1)], Hkv, d).view(B, N, Hkv, d)
    k = torch.where(held, k, 0).permute(0, 2, 3, 1)                                           # [B, Hkv, d, N]
    v = torch.where(held, v, 0).permute(0, 2, 1, 3)                                           # [B, Hkv, N, d]
    q = s["q"].float().view(B, T, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, d)
    x = (q @ k).view(B, Hkv, G, T, N).mul_(s["scale"])
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    x = x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    none = m == -math.inf
    x = x.sub_(m.masked_fill(none, 0)).exp_()
    total = x.sum(-1, keepdim=True)
    out = (x.view(B, Hkv, G * T, N) @ v).view(B, Hkv, G, T, -1) / total.masked_fill(none, 1)
    lse = (m + total.log()).squeeze(-1)
    return (out.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, -1).to(s["q"].dtype),
            lse.permute(0, 3, 1, 2).reshape(B * T, Hq))


def _plain_beam(s):
    c = s["case"]
    B, W, K, V, S = (c[k] for k in ("seqs", "beams", "out", "vocab", "length"))
    done = s["done"].bool()
    # scores that lie close together are told apart in 64 bits
    x = s["logits"].double()
    x = x - torch.logsumexp(x, -1, keepdim=True)
    alone = torch.where(torch.arange(V, device="cuda") == s["end"], 0.0, -math.inf).double()    # an ended beam's
    x = torch.where(done[:, None], alone, x) + s["scores"].double()[:, None]
    value, at = torch.sort(x.view(B, W * V), dim=-1, descending=True, stable=True)
    value, at = value[:, :K], at[:, :K]
    if W * V < K:
        value = torch.nn.functional.pad(value, (0, K - W * V), value=-math.inf)
        at = torch.nn.functional.pad(at, (0, K - W * V))
    none = (value == -math.inf).view(-1)
    parent = (at // V + torch.arange(B, device="cuda")[:, None] * W).view(-1)
    token = torch.where(none, -1, (at % V).view(-1))
    was = done[parent]
    length = s["lengths"].long()[parent]
    grown = torch.where(none, 0, length + (~was).long())
    ends = none | was | (token == s["end"])
    i = torch.arange(S, device="cuda")
    history = torch.where(i < length[:, None], s["history"][parent], s["history_out"])
    history = torch.where((i == length[:, None]) & ~was[:, None], token[:, None].to(torch.int32), history)
    history = torch.where(none[:, None], s["history_out"], history)
    i32 = lambda t: t.to(torch.int32)  # noqa: E731
    return [value.float().view(-1), i32(torch.where(none, -1, parent)), i32(token), ends.to(torch.uint8), i32(grown), history]


# --------------------------------------------------------------------------------------------- the framework's calls

def _own(s):
    import lightning_indexer_top_gb300 as L
    c = s["case"]
    if c["kind"] == "beam":
        r = L.idx_beam_step(s["logits"], s["scores"], c["beams"], n_out=c["out"], done=s["done"], end_token=s["end"],
                            lengths=s["lengths"], history=s["history"], history_out=s["history_out"])
        return [r.scores, r.parent, r.token, r.done, r.lengths, r.history]
    N = c["cached"] if c["kind"] == "attn" else c["room"]
    batch = L.Batch(s["n_kv"], c["new"], N, kv_seq_stride=N, q_pos=s["pos"], page_table=s["table"], page_size=c["page"])
    if c["kind"] == "attn":
        lse = torch.empty(s["q"].shape[:2], device="cuda", dtype=torch.float32)
        out = L.dense_attn_q4(s["q"], s["k_cache"], s["v_cache"], batch, s["scale"], c["hkv"], softcap=c["cap"],
                              window=c["window"], lse=lse)
        return out, lse
    call = L.idx_cache_append if c["kind"] == "append" else L.idx_cache_append_q4
    q = call(s["k"], s["v"], s["k_cache"], s["v_cache"], batch, q=s["q"], inv_freq=s["inv_freq"], rot_start=c["start"],
             interleaved=c["inter"])
    if c["kind"] == "append":
        return [x for x in (q, s["k_cache"], s["v_cache"]) if x is not None]
    k, v = L.idx_cache_read_q4(s["k_cache"], s["v_cache"], batch, c["hkv"], c["dk"], c["dv"], k_out=s["k_out"], v_out=s["v_out"])
    return [k, v] if q is None else [q, k, v]


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "append4": _plain_append4, "attn": _plain_attn,
            "beam": _plain_beam}[state["case"]["kind"]](state)


# --------------------------------------------------------------------------------------------- floors

def work(case):
    if case["kind"] == "beam":
        rows = case["seqs"] * case["beams"]
        size = torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
        kept = case["seqs"] * case["out"]
        return {"bytes": int(rows * (1 - case["ended"])) * case["vocab"] * size + 9 * rows + kept * (17 + 8 * case["length"]),
                "flops": 2.0 * rows * (1 - case["ended"]) * case["vocab"]}
    size = torch.empty((), dtype=DTYPES[case["dtype"]]).element_size()
    n_kv, pos = _positions(case)
    if case["kind"] == "attn":
        Hq, Hkv, d = case["hq"], case["hkv"], case["d"]
        hi = np.minimum(pos + 1, n_kv[:, None])
        lo = np.maximum(pos - case["window"] + 1, 0) if case["window"] else np.zeros_like(pos)
        n = np.where(pos < 0, 0, hi - lo)
        # rows of a sequence lie one behind the other: what they see is one piece
        seen = int((hi.max(1) - np.where(pos < 0, 1 << 40, lo).min(1)).sum())
        return {"bytes": seen * Hkv * (d + 16) + int((n > 0).sum()) * Hq * d * size + n.size * Hq * (d * size + 4),
                "flops": 4.0 * float(n.sum()) * Hq * d}
    rows = int((pos >= 0).sum())
    hq, hkv, dk, dv = (case[k] for k in ("hq", "hkv", "dk", "dv"))
    new = hkv * (dk + dv) * size
    q = 2 * pos.size * hq * dk * size
    flops = 3.0 * rows * (hq + hkv) * case["rot"]
    if case["kind"] == "append":
        return {"bytes": 2 * rows * new + q + 4 * pos.size, "flops": flops}
    # the new rows, their 4-bit form written and read, their values written
    return {"bytes": 2 * rows * new + 2 * rows * hkv * ((dk + dv) // 2 + 16) + q + 8 * pos.size, "flops": flops}


# --------------------------------------------------------------------------------------------- 64-bit values

def _turn(case, x, pos, inv_freq):
    """Rows [heads, dk] in 64 bits as complex numbers, multiplied by those of their angles."""
    n, a = case["rot"], case["start"]
    y = x.double().clone()
    if n:
        part = y[:, :, a:a + n]
        z = torch.complex(part[..., 0::2], part[..., 1::2]) if case["inter"] else torch.complex(part[..., :n // 2], part[..., n // 2:])
        t = pos.double()[:, None, None] * inv_freq.double()
        z = z * torch.polar(torch.ones_like(t), t)
        if case["inter"]:
            y[:, :, a:a + n:2], y[:, :, a + 1:a + n:2] = z.real, z.imag
        else:
            y[:, :, a:a + n // 2], y[:, :, a + n // 2:a + n] = z.real, z.imag
    return y


def _exact_append(case, seed):
    s = _prepare_append(case, seed)
    real = torch.nonzero(s["pos"] >= 0).view(-1)
    pos, to = s["pos"][real], s["rows"][real]
    outs = []
    if s["q"] is not None:
        q = s["q"].double().clone()
        q[real] = _turn(case, s["q"][real], pos, s["inv_freq"])
        outs.append(q)
    new = [_turn(case, s["k"][real], pos, s["inv_freq"])] + ([] if s["v"] is None else [s["v"][real].double()])
    for x, cache, out in zip(new, (s["k_cache"], s["v_cache"]), (s.get("k_out"), s.get("v_out"))):
        if case["kind"] == "append":
            y = cache.double()
            y[to] = x
        else:
            low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
            span = high - low
            y = out.double()
            y[real] = torch.round(15 * (x - low) / torch.where(span > 0, span, 1.0)) * (span / 15) + low
        outs.append(y)
    return outs


def _exact_attn(case, seed):
    B, T, N, Hq, Hkv, d = (case[k] for k in ("batch", "new", "cached", "hq", "hkv", "d"))
    if 4.0 * B * T * N * Hq * d > 8e12:
        return None
    s = _prepare_attn(case, seed)
    n_kv, pos = _positions(case)
    G = Hq // Hkv
    out = torch.zeros(B * T, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B * T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    q = s["q"].double().view(B, T, Hq, d)
    for b in range(B):
        n = int(n_kv[b])
        p = torch.from_numpy(pos[b]).cuda()[:, None]
        j = torch.arange(n, device="cuda")
        seen = (j <= p) & (p >= 0)
        if case["window"]:
            seen &= j > p - case["window"]
        some = seen.any(1)
        raw = [s[x][s["rows"][b, :n]] for x in ("k_cache", "v_cache")]
        for g in range(Hkv):
            kk, vv = [], []
            for x, to in zip(raw, (kk, vv)):
                byte = x[:, g * d // 2:(g + 1) * d // 2].to(torch.int64)
                code = torch.empty((n, d), dtype=torch.float64, device="cuda")
                code[:, 0::2], code[:, 1::2] = (byte % 16).double(), (byte // 16).double()
                f = x[:, Hkv * d // 2 + 8 * g:Hkv * d // 2 + 8 * g + 8].contiguous().view(torch.float32).double()
                to.append(code * f[:, :1] + f[:, 1:])
            for h in range(g * G, (g + 1) * G):
                y = torch.matmul(q[b, :, h], kk[0].T) * s["scale"]
                if case["cap"]:
                    y = torch.tanh(y / case["cap"]) * case["cap"]
                y = torch.where(seen, y, -math.inf)
                t = torch.logsumexp(y, -1)
                lse[b * T:(b + 1) * T, h] = t
                out[b * T:(b + 1) * T, h] = torch.matmul(torch.exp(y - torch.where(some, t, 0.0)[:, None]), vv[0])
    return out, lse


def _exact_beam(case, seed):
    """Candidate by candidate on the host, from each row's best ones."""
    s = _prepare_beam(case, seed)
    B, W, K, V = (case[k] for k in ("seqs", "beams", "out", "vocab"))
    x = s["logits"].cpu().numpy() if case["dtype"] == "f32" else s["logits"].float().cpu().numpy()
    base, done, lens, old = (s[k].cpu().numpy() for k in ("scores", "done", "lengths", "history"))
    history = s["history_out"].cpu().numpy().copy()
    res = [[], [], [], [], []]
    for b in range(B):
        cands = []
        for row in range(b * W, (b + 1) * W):
            if done[row]:
                cands.append((-float(base[row]), row, s["end"]))
                continue
            y = x[row].astype(np.float64)
            top = float(y.max())
            z = top + math.log(float(np.exp(y - top).sum()))
            edge = np.partition(x[row], V - min(K, V))[V - min(K, V)]
            cands += [(-(float(base[row]) + float(y[i]) - z), row, int(i)) for i in np.nonzero(x[row] >= edge)[0]]
        cands.sort()
        for i in range(K):
            if i >= len(cands):
                res = [r + [e] for r, e in zip(res, (-math.inf, -1, -1, 1, 0))]
                continue
            v, row, token = cands[i]
            n = int(lens[row])
            history[b * K + i, :n] = old[row, :n]
            if not done[row]:
                history[b * K + i, n] = token
            grown = n + (0 if done[row] else 1)
            res = [r + [e] for r, e in zip(res, (-v, row, token, int(bool(done[row]) or token == s["end"]), grown))]
    kinds = (torch.float64, torch.int32, torch.int32, torch.uint8, torch.int32)
    return [torch.tensor(r, dtype=t) for r, t in zip(res, kinds)] + [torch.from_numpy(history)]


def exact(case, seed):
    return {"append": _exact_append, "append4": _exact_append, "attn": _exact_attn, "beam": _exact_beam}[case["kind"]](case, seed)
