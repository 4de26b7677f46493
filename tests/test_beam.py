"""idx_beam_step against 64-bit code, its refusals, and whole searches: with idx_page_update, the cache writes and the
attention over 16-bit and 4-bit pages, against the same search on contiguous tensors.

Worths: an f32 sum of n exponentials, each off by 2^-22 and by 2^-24 of its exponent, is off by less than (2^-20 + n 2^-24 /
threads) relative; log and the rest run in 64 bits, the result is rounded to f32: |error| <= 2^-19 + 2^-24 |worth|.  Inputs are
drawn until no two worths at the border or within the kept ones lie closer than twice that, so that the choice is exact."""

import ctypes
import math

import numpy as np
import pytest
import torch

import lightning_indexer_top_gb300 as L

DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def reference(logits, scores, W, K, done=None, end=-1):
    """Kept continuations as lists per sequence: (worth, row, token), best first; and how near the closest two of the first
    K + 1 worths of different beams are."""
    rows, V = logits.shape
    x = logits.double().cpu()
    out, near = [], math.inf
    for s in range(rows // W):
        cand = []
        for r in range(s * W, (s + 1) * W):
            base = float(scores[r])
            if base == -math.inf or base != base or base == math.inf:
                continue
            if done is not None and bool(done[r]):
                cand.append((-base, r, end))
                continue
            y = x[r]
            if torch.isnan(y).any() or (y == math.inf).any() or (y == -math.inf).all():
                continue
            z = torch.logsumexp(y, 0)
            w = (y - z + base).numpy()
            best = np.lexsort((np.arange(V), -w))[:K + 1]
            cand += [(-float(w[i]), r, int(i)) for i in best if w[i] > -math.inf]
        cand.sort()
        first = cand[:K + 1]
        for a, b in zip(first, first[1:]):
            if a[1] != b[1] and a[0] != b[0]:
                near = min(near, b[0] - a[0])
        out.append([(-v, r, t) for v, r, t in cand[:K]])
    return out, near


def check(res, want, K, end, lengths=None, history=None, done=None, old=None):
    n = len(want) * K
    rows = [c for s in want for c in s + [None] * (K - len(s))]
    assert res.parent.tolist() == [-1 if c is None else c[1] for c in rows]
    assert res.token.tolist() == [-1 if c is None else c[2] for c in rows]
    was = [c is not None and done is not None and bool(done[c[1]]) for c in rows]
    assert res.done.tolist() == [int(c is None or w or c[2] == end) for c, w in zip(rows, was)]
    got = res.scores.cpu().double()
    ref = torch.tensor([-math.inf if c is None else c[0] for c in rows], dtype=torch.float64)
    assert torch.equal(torch.isneginf(got), torch.isneginf(ref))
    fin = ~torch.isneginf(ref)
    assert ((got - ref)[fin].abs() <= 2.0 ** -19 + 2.0 ** -24 * ref[fin].abs()).all()
    assert all(float(got[i]) == float(np.float32(c[0])) for i, c in enumerate(rows) if was[i])
    if lengths is not None:
        new = old.clone()
        lens = []
        for i, c in enumerate(rows):
            if c is None:
                lens.append(0)
                continue
            m = int(lengths[c[1]])
            new[i, :m] = history[c[1], :m]
            if not was[i]:
                new[i, m] = c[2]
                m += 1
            lens.append(m)
        assert res.lengths.tolist() == lens and torch.equal(res.history.cpu(), new)
    assert len(rows) == n


def inputs(rows, V, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, V, generator=g) * spread).to(dtype), (torch.rand(rows, generator=g) * -5).float(), g


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs,W,K,V", [(1, 1, 1, 1), (1, 1, 5, 3), (1, 4, 4, 1000), (3, 2, 5, 257), (2, 5, 11, 2048), (2, 3, 32, 2049), (5, 1, 32, 8193),
                                        (1, 16, 32, 40000), (40, 8, 16, 9001), (1, 2, 3, 131072), (2, 130, 7, 300)])
def test_steps(dtype, seqs, W, K, V):
    for seed in range(20):
        x, scores, g = inputs(seqs * W, V, dtype, seed)
        want, near = reference(x, scores, W, K)
        if near > 2.0 ** -18:
            break
    lengths = torch.randint(0, 9, (seqs * W,), generator=g).to(torch.int32)
    history = torch.randint(0, V, (seqs * W, 9), generator=g, dtype=torch.int32)
    old = torch.randint(0, V, (seqs * K, 9), generator=g, dtype=torch.int32)
    res = L.idx_beam_step(x.cuda(), scores.cuda(), W, n_out=K, lengths=lengths.cuda(), history=history.cuda(), history_out=old.cuda())
    check(res, want, K, -1, lengths, history, None, old)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("apart", [0, 3, 8])
def test_beams_that_are_done_dead_or_short_of_tokens(dtype, apart):
    seqs, W, K, V, end = 6, 4, 9, 500, 17
    for seed in range(20):
        x, scores, g = inputs(seqs * W, V, dtype, seed)
        done = torch.zeros(seqs * W, dtype=torch.uint8)
        done[[0, 5, 6, 8, 9, 10, 11]] = 1                       # sequence 2: all done
        scores[[3, 12, 13, 14, 15]] = -math.inf                 # sequence 3: all dead
        scores[17:20] = -math.inf                               # a first step: one beam lives
        x[20:24] = -math.inf                                    # sequence 5: seven tokens in all, one beam without any
        for r, t in ((20, 3), (20, 499), (21, 0), (21, 1), (21, 2), (22, 17), (22, 18)):
            x[r, t] = float(torch.randn((), generator=g))
        want, near = reference(x, scores, W, K, done, end)
        if near > 2.0 ** -18:
            break
    lengths = torch.randint(0, 12, (seqs * W,), generator=g).to(torch.int32)
    history = torch.randint(0, V, (seqs * W, 12), generator=g, dtype=torch.int32)
    old = torch.zeros(seqs * K, 12, dtype=torch.int32)
    wide = torch.zeros(seqs * W, V + apart, dtype=dtype, device="cuda")
    wide[:, :V] = x.cuda()
    wide[:, V:] = math.nan
    for d in (done.cuda(), done.bool().cuda()):
        res = L.idx_beam_step(wide[:, :V], scores.cuda(), W, n_out=K, done=d, end_token=end, lengths=lengths.cuda(), history=history.cuda())
        check(res, want, K, end, lengths, history, done, old)
    assert [len(w) for w in want][2:4] == [4, 0] and len(want[5]) == 7
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [7, 2000, 40000, 131072])
@pytest.mark.parametrize("K", [1, 6, 32])
def test_ties_go_to_the_lower_beam_then_token(dtype, V, K):
    # equal rows with equal scores, and rows of equal logits (every key is at the bound)
    x, _, g = inputs(1, V, dtype, 3)
    for rows in (x, torch.zeros(1, V, dtype=dtype), torch.full((1, V), -0.0, dtype=dtype), (x > 1).to(dtype)):
        x4 = rows.expand(4, V).contiguous()
        scores = torch.tensor([-1.0, -1.0, -1.0, -1.0])
        want, _ = reference(x4, scores, 4, K)
        check(L.idx_beam_step(x4.cuda(), scores.cuda(), 4, n_out=K), want, K, -1)
        if V % 8:
            continue
        # (rows of another alignment than the first)
        wide = torch.zeros(4, V + 3, dtype=dtype, device="cuda")
        wide[:, :V] = x4.cuda()
        check(L.idx_beam_step(wide[:, :V], scores.cuda(), 4, n_out=K), want, K, -1)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("seqs,W,K,V", [(2, 4, 9, 5), (1, 4, 32, 40000), (3, 130, 32, 300), (1, 2, 1, 9001), (2, 3, 7, 131072)])
@pytest.mark.parametrize("live", [0, 1])
def test_worths_that_64_bits_do_not_tell_apart(dtype, seqs, W, K, V, live):
    # beams kept out of the race by the lowest finite score: every token of theirs is worth the same
    x, scores, _ = inputs(seqs * W, V, dtype, 9)
    scores[:] = torch.finfo(torch.float32).min
    if live:      # one beam lives, with fewer tokens than are kept
        scores[::W] = -1.0
        x[::W, max(K - 3, 1):] = -math.inf
        x[::W, 0] = 30.0 if dtype != torch.float16 else 8.0
    for done in (None, (torch.arange(seqs * W) % W == 1).to(torch.uint8)):      # (one that is done is worth as much)
        end = -1 if done is None else 2
        want, _ = reference(x, scores, W, K, done, end)
        res = L.idx_beam_step(x.cuda(), scores.cuda(), W, n_out=K, done=None if done is None else done.cuda(), end_token=end)
        check(res, want, K, end, done=done)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("W,K,V", [(1, 4, 5000), (2, 32, 20000), (3, 1, 700)])
@pytest.mark.parametrize("up", [1, -1])
def test_logits_that_64_bits_do_not_tell_apart(W, K, V, up):
    # tiny logits, all different, that the sum's logarithm swallows; the lower token, whatever its logit
    x = torch.full((W, V), -20.0)
    at = torch.arange(3, V, 61)
    n = torch.arange(1.0, len(at) + 1)
    x[:, at] = (n if up > 0 else n.flip(0)) * 1e-30
    scores = torch.full((W,), -2.0)
    want, _ = reference(x, scores, W, K)
    assert [c[2] for c in want[0]][:3] == at[:min(K, 3)].tolist()
    check(L.idx_beam_step(x.cuda(), scores.cuda(), W, n_out=K), want, K, -1)


@pytest.mark.gpu
def test_histories_that_are_columns_of_one_tensor():
    # a step reads one half of each row and writes the other: nothing written is read
    x, scores, g = inputs(8, 500, torch.float32, 10)
    both = torch.randint(0, 500, (8, 24), generator=g, dtype=torch.int32).cuda()
    lengths = torch.full((8,), 5, dtype=torch.int32, device="cuda")
    call = lambda new: L.idx_beam_step(x.cuda(), scores.cuda(), 4, lengths=lengths, history=both[:, :12], history_out=new)  # noqa: E731
    want = call(both[:, 12:].clone())
    before = both[:, :12].clone()
    got = call(both[:, 12:])
    assert torch.equal(both[:, 12:], want.history) and torch.equal(both[:, :12], before) and torch.equal(got.lengths, want.lengths)
    with pytest.raises(L.LidxError):      # one column is in both
        call(both[:, 11:23])


@pytest.mark.gpu
def test_no_numbers_are_flagged():
    x, scores, _ = inputs(8, 3000, torch.float32, 4)
    x[1, 2999], x[2, 0] = math.nan, math.inf
    scores[4], scores[5] = math.nan, math.inf
    want, _ = reference(x, scores, 4, 6)
    check(L.idx_beam_step(x.cuda(), scores.cuda(), 4, n_out=6), want, 6, -1)
    assert L.idx_device_status(reset=True) == L.IDX_ERR_INEXACT
    # done beams' logits are not looked at
    done = torch.tensor([0, 1, 1, 0, 1, 1, 0, 0], dtype=torch.uint8)
    scores[4:6] = -3
    want, _ = reference(x, scores, 4, 6, done, 5)
    check(L.idx_beam_step(x.cuda(), scores.cuda(), 4, n_out=6, done=done.cuda(), end_token=5), want, 6, 5, done=done)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_far_apart_logits():
    # one token holds all the weight; logits as far down as f32 goes
    x = torch.full((2, 5000), -3e38)
    x[0, 7], x[0, 4999], x[1, 0] = 3e38, 2.9e38, 0.0
    res = L.idx_beam_step(x.cuda(), torch.zeros(2, device="cuda"), 2, n_out=3)
    assert res.parent.tolist() == [0, 1, 0] and res.token.tolist() == [7, 0, 4999]
    assert res.scores[:2].tolist() == [0.0, 0.0] and abs(float(res.scores[2]) + 1e37) < 1e31 * 10


@pytest.mark.gpu
def test_lengths_out_of_range_are_flagged():
    x, scores, g = inputs(4, 50, torch.float16, 5)
    history = torch.randint(0, 50, (4, 3), generator=g, dtype=torch.int32).cuda()
    scores[:] = torch.tensor([0.0, -50.0, -100.0, -150.0])
    for lens, flagged in (([0, 1, 2, 2], False), ([3, 0, 0, 0], True), ([-1, 0, 0, 0], True), ([9, 1, 1, 1], True)):
        old = torch.full((4, 3), 99, dtype=torch.int32, device="cuda")
        res = L.idx_beam_step(x.cuda(), scores.cuda(), 4, n_out=1, lengths=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                              history=history, history_out=old[:1])
        assert (L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS) == flagged
        n = min(max(lens[0], 0), 3)
        assert res.lengths.tolist() == [n + (not flagged)]
        assert torch.equal(old[0, :n], history[0, :n]) and (old[1:] == 99).all() and (old[0, n + (not flagged):] == 99).all()


@pytest.mark.gpu
def test_captured_and_written_to_given_tensors():
    x, scores, g = inputs(12, 9000, torch.bfloat16, 6)
    xs, sc = x.cuda(), scores.cuda()
    lens, hist = torch.full((12,), 4, dtype=torch.int32, device="cuda"), torch.randint(0, 9, (12, 8), device="cuda", dtype=torch.int32)
    first = L.idx_beam_step(xs, sc, 4, n_out=4, lengths=lens, history=hist, end_token=0)
    ws = torch.empty(L.idx_beam_workspace_size(3, 4, 4, 9000), dtype=torch.uint8, device="cuda")
    out = L.BeamStep(*[torch.zeros_like(t) for t in first])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.idx_beam_step(xs, sc, 4, n_out=4, lengths=lens, history=hist, end_token=0, out=out, workspace=ws)
    ws.fill_(255)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, out))
    # a step that continues from the last one's results, on another stream
    y, _, _ = inputs(12, 9000, torch.bfloat16, 7)
    xs.copy_(y.cuda())
    second = L.idx_beam_step(xs, first.scores, 4, done=first.done, lengths=first.lengths, history=first.history, end_token=0)
    sc.copy_(first.scores)
    lens.copy_(first.lengths)
    hist.copy_(first.history)
    if not first.done.any():
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            graph.replay()
        torch.cuda.current_stream().wait_stream(s)
        assert all(torch.equal(a, b) for a, b in zip(second[:5], out[:5]))
        assert all(torch.equal(second.history[i, :n], out.history[i, :n]) for i, n in enumerate(second.lengths.tolist()))


# --------------------------------------------------------------------------------------------- a search

class Model:
    """A layer of attention with random weights: tokens to logits, through the caches."""

    def __init__(self, V, Hq, Hkv, d, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: (torch.randn(*s, generator=g) / math.sqrt(s[0])).cuda()  # noqa: E731
        self.V, self.Hq, self.Hkv, self.d = V, Hq, Hkv, d
        # (every token's projection once: a product's bits go with its number of rows)
        self.qkv, self.out = (torch.randn(V, 64, generator=g).cuda() @ r(64, (Hq + 2 * Hkv) * d) * 2).half(), r(Hq * d, V) * 6
        self.freq = (100.0 ** (-torch.arange(0, d, 2).double() / d)).float().cuda()

    def project(self, tokens):
        q, k, v = self.qkv[tokens].split([self.Hq * self.d, self.Hkv * self.d, self.Hkv * self.d], 1)
        return [t.unflatten(1, (-1, self.d)) for t in (q, k, v)]

    def logits(self, attended):
        return attended.flatten(1).float() @ self.out


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_a_search_over_paged_caches(four):
    """Three requests of four beams over pages of eight rows: prompts are written as one chunk of ragged rows, then every
    step selects, forks pages, appends and attends.  Each kept beam's attention is held against its own token sequence
    attended anew from empty contiguous caches: the same rows in other places, so the results agree bit for bit in 4 bits and
    in 16."""
    m, W, steps, ps, end = Model(97, 8, 2, 64), 4, 12, 8, 5
    prompts = [[3, 14, 15, 92, 65, 35, 89, 79, 32, 38], [46], [26, 43, 38, 32]]
    B, T, cols = len(prompts), max(len(p) for p in prompts), 4
    n_pages, w = 60, L.idx_q4_row_bytes(2, 64)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def caches(rows):
        return [torch.zeros(rows, w, dtype=torch.uint8, device="cuda") if four else
                torch.zeros(rows, 2, 64, dtype=torch.float16, device="cuda") for _ in range(2)]

    def attend(tokens, kc, vc, batch):
        q, k, v = m.project(tokens)
        if four:
            q = L.idx_cache_append_q4(k, v, kc, vc, batch, q=q, inv_freq=m.freq)
            return L.dense_attn_q4(q, kc, vc, batch, 0.125, 2)
        q = L.idx_cache_append(k, v, kc, vc, batch, q=q, inv_freq=m.freq)
        return L.dense_attn(q, kc, vc, batch, 0.125)

    pool = caches(n_pages * ps)
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    lens = [len(p) for p in prompts]
    table, left = L.idx_page_update(table, i32([-1] * B), i32([0] * B), i32(lens), ps, pool)
    tokens = torch.zeros(B, T, dtype=torch.int64)
    pos = torch.full((B, T), -1)
    for b, p in enumerate(prompts):
        tokens[b, :len(p)], pos[b, :len(p)] = torch.tensor(p), torch.arange(len(p))
    out = attend(tokens.view(-1).cuda(), *pool, L.Batch(i32(lens), T, cols * ps, q_pos=i32(pos.view(-1).tolist()), page_table=table, page_size=ps))
    last = out.view(B, T, 8, 64)[torch.arange(B), torch.tensor(lens) - 1]
    # the first step: one beam lives in each sequence
    logits = m.logits(last).repeat_interleave(W, 0)
    scores = torch.full((B, W), -math.inf, device="cuda")
    scores[:, 0] = 0
    S = T + steps + 1
    history = torch.zeros(B * W, S, dtype=torch.int32, device="cuda")
    for b, p in enumerate(prompts):
        history[b * W:(b + 1) * W, :len(p)] = i32(p)
    res = L.BeamStep(scores.view(-1), None, None, torch.zeros(B * W, dtype=torch.uint8, device="cuda"), i32([n for n in lens for _ in range(W)]), history)
    table = table.repeat_interleave(W, 0).contiguous()
    for step in range(steps):
        lengths = res.lengths
        res = L.idx_beam_step(logits, res.scores, W, done=res.done, end_token=end, lengths=res.lengths, history=res.history)
        assert (res.parent >= 0).all()
        keep = lengths[res.parent.long()] if step == 0 else held[res.parent.long()]
        held = keep + (1 - res.done.int())            # a beam that is done gets no row for its last token
        table, left = L.idx_page_update(table, res.parent, keep, held, ps, pool)
        assert int(left) >= 0
        q_pos = torch.where(res.done.bool(), -1, keep)
        batch = L.Batch(held, 1, cols * ps, q_pos=q_pos, page_table=table, page_size=ps)
        out = attend(res.token.long(), *pool, batch)
        logits = m.logits(out)
        # every live beam anew
        for r in torch.nonzero(res.done == 0).view(-1).tolist()[::3 if step < steps - 1 else 1]:
            n = int(res.lengths[r])
            assert n == int(held[r])
            seq = res.history[r, :n].long()
            fresh = caches(n)
            one = None
            for i in range(n):      # token by token: what the steps did (the prompt's chunk gives the same rows)
                b1 = L.Batch(i32([i + 1]), 1, cols * ps, kv_seq_stride=0, q_pos=i32([i]))
                one = attend(seq[i:i + 1], *fresh, b1)
            got = [c.view(n_pages, ps, -1)[table[r, :-(-n // ps)].long()].view(-1, c[0].numel())[:n] for c in pool]
            assert all(torch.equal(a, b.view(n, -1)) for a, b in zip(got, fresh))
            assert torch.equal(one[0], out[r])
    assert L.idx_device_status(reset=True) == 0


# --------------------------------------------------------------------------------------------- refusals

def _call(**kw):
    p = ctypes.c_void_p
    beam = dict(logits=1 << 20, logit_stride=100, scores=1 << 12, done=None, lengths=None, history=None, history_stride=0, out_scores=2 << 12,
                parent=3 << 12, token=4 << 12, out_done=5 << 12, out_lengths=None, out_history=None, out_history_stride=0, history_cols=0)
    a = dict(dtype=L.IDX_F32, n=2, W=4, K=4, V=100, end=-1, ws=p(1 << 24), size=1 << 20)
    for k, v in kw.items():
        (beam if k in beam else a)[k] = v
    return L.load().idx_beam_step(ctypes.byref(L._Beam(**beam)), a["dtype"], a["n"], a["W"], a["K"], a["V"], a["end"], a["ws"], a["size"], None)


HIST = dict(lengths=6 << 12, history=7 << 12, out_lengths=8 << 12, out_history=9 << 12, history_stride=8, out_history_stride=8, history_cols=8)


@pytest.mark.parametrize("bad,word", [
    (dict(dtype=7), b"dtype"), (dict(n=-1), b"n_seq"), (dict(W=0), b"n_beams"), (dict(V=0), b"n_vocab"), (dict(K=0), b"n_out"), (dict(K=33), b"n_out"),
    (dict(W=1 << 16, V=1 << 15, logit_stride=1 << 15), b"continuations"), (dict(n=1 << 20, W=1 << 12), b"rows"), (dict(end=-2), b"end_token"),
    (dict(end=100), b"end_token"), (dict(done=1 << 13), b"done"), (dict(logit_stride=99), b"logit_stride"), (dict(history_cols=-1), b"history_cols"),
    (dict(HIST, history_cols=9), b"history_cols"), (dict(W=1025), b"n_beams"), (dict(W=1, V=2 ** 31 - 1, logit_stride=2 ** 31), b"n_vocab"), (dict(logits=None), b"NULL"), (dict(scores=None), b"NULL"),
    (dict(out_scores=None), b"NULL"), (dict(parent=None), b"NULL"), (dict(token=None), b"NULL"), (dict(out_done=None), b"NULL"),
    (dict(HIST, history=None), b"together"), (dict(HIST, out_lengths=None), b"together"), (dict(HIST, out_history=None), b"together"),
    (dict(out_scores=(1 << 12) + 4), b"overlaps"), (dict(HIST, out_history=(7 << 12) + 64), b"overlaps"), (dict(token=(1 << 20) + 16), b"overlaps"),
    (dict(ws=None), b"workspace"), (dict(ws=ctypes.c_void_p(24)), b"workspace"), (dict(size=8), b"workspace")])
def test_refusals(bad, word):
    assert _call(**bad) in (L.IDX_ERR_INVALID_ARG, L.IDX_ERR_UNSUPPORTED)
    assert word in L.load().idx_last_error()


def test_workspace_of_nonsense_sizes_is_0():
    for a in ((0, 1, 1, 10), (1, 0, 1, 10), (1, 1, 0, 10), (1, 1, 33, 10), (1, 1, 1, 0)):
        assert L.idx_beam_workspace_size(*a) == 0
    assert _call(n=0) == L.IDX_OK


@pytest.mark.gpu
def test_binding_refuses():
    x, s = torch.zeros(8, 50, device="cuda"), torch.zeros(8, device="cuda")
    i = lambda *a: torch.zeros(*a, dtype=torch.int32, device="cuda")  # noqa: E731
    L.idx_beam_step(x, s, 4)
    for bad in (dict(x=x[:7]), dict(x=x.T), dict(x=x[:1].expand(8, 50)), dict(x=x.int()), dict(s=s[:7]), dict(s=s.double()), dict(s=s.cpu()),
                dict(W=0), dict(W=3), dict(end_token=2 ** 32 + 3), dict(done=s, end_token=3), dict(done=torch.zeros(7, dtype=torch.uint8, device="cuda"), end_token=3),
                dict(lengths=i(8)), dict(history=i(8, 4)), dict(lengths=i(7), history=i(8, 4)), dict(lengths=i(8), history=i(7, 4)),
                dict(lengths=i(8), history=i(8, 4), history_out=i(8, 5)), dict(lengths=i(8), history=i(8, 4), history_out=i(7, 4)),
                dict(out=L.BeamStep(s, i(7), i(8), torch.zeros(8, dtype=torch.uint8, device="cuda"), None, None)),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda").expand(1000, 16))):
        a = {**dict(x=x, s=s, W=4), **bad}
        with pytest.raises((ValueError, TypeError)):
            L.idx_beam_step(a["x"], a["s"], a["W"], **{k: v for k, v in a.items() if k not in ("x", "s", "W")})
    with pytest.raises(L.LidxError):
        L.idx_beam_step(x, s, 4, end_token=50)
