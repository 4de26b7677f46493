"""dense_attn against softmax attention in 64 bits, and its refusals.

Tolerance of an output element, from the arithmetic: with u = 2^-24 and A_j = sum_i |q_i k_ji|,
  scores   an f32 dot product of dk terms is off by at most (dk + 2) u A; scaling, cap, bias and the
           maximum's subtraction add 8 u (|x| + cap + slope * distance + 1) each rounded: dx;
  weights  off by a factor within e^(2 dx) (1 + 2^-20) (exponentials to a few units of 2^-22), and, where
           16-bit inputs use the tensor cores, by half a step of the inputs' type (the weights are rounded
           to it; the sum of the weights is not);
  sums     n f32 additions: n u relative to the sum of magnitudes.
With S = sum_j p_j |v_j|: |error| <= 2 (2 dx + n u + 2^-20 + half(T)) S + half(T) |out|, where half(T) =
finfo(T).eps / 2 (f32: no weight rounding).  lse: dx + n u + 2^-20 + u |lse|."""

import ctypes
import math

import numpy as np
import pytest
import torch

import lightning_indexer_top_gb300 as L

U = 2.0 ** -24


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def intervals(n_kv, pos, window=0, prefix=None, docs=None):
    """lo, hi, int64 [B, T]; pos None: every cached key."""
    B = len(n_kv)
    n = torch.tensor(n_kv)[:, None]
    if pos is None:
        T = 1 if docs is None else docs.shape[1]
        lo, hi = torch.zeros(B, T, dtype=torch.int64), n.expand(B, T).clone()
    else:
        hi = pos + 1
        if prefix is not None:
            hi = torch.maximum(hi, torch.tensor(prefix)[:, None])
        hi = torch.where(pos < 0, 0, torch.minimum(hi, n))
        lo = torch.clamp(pos - window + 1, min=0) if window else torch.zeros_like(pos)
    if docs is not None:
        lo = torch.maximum(lo, docs)
    return lo, hi


def reference(q, k, v, rows, lo, hi, pos, scale, cap=0.0, slopes=None):
    """q [B, T, Hq, dk]; k [cache rows, Hkv, dk], v likewise (CPU tensors); rows: per sequence the cache row of each
    position.  Returns out, lse, and the tolerances of both, f64."""
    B, T, Hq, dk = q.shape
    Hkv, dv = k.shape[1], v.shape[2]
    G = Hq // Hkv
    half = _half(q.dtype)
    weights = half if q.dtype != torch.float32 else 0.0
    out = torch.zeros(B, T, Hq, dv, dtype=torch.float64)
    lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b in range(B):
        for t in range(T):
            l, h = int(lo[b, t]), int(hi[b, t])
            if l >= h:
                continue
            at = rows[b][l:h]
            kk = k[at].double().repeat_interleave(G, 1)
            vv = v[at].double().repeat_interleave(G, 1)
            qq = q[b, t].double()
            x = torch.einsum("hd,nhd->hn", qq, kk) * scale
            A = torch.einsum("hd,nhd->hn", qq.abs(), kk.abs()) * abs(scale)
            size = x.abs() + 1
            if cap:
                x = cap * torch.tanh(x / cap)
                size = size + cap
            if slopes is not None:
                dist = (int(pos[b, t]) - torch.arange(l, h)).abs().double()
                x = x - slopes.double()[:, None] * dist
                size = size + slopes.double()[:, None] * dist
            dx = ((dk + 2) * U * A + 8 * U * size).amax(1, keepdim=True)
            lse[b, t] = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1)
            p = torch.where(torch.isnan(p) & torch.isneginf(lse[b, t])[:, None], 0.0, p)   # every score -inf
            out[b, t] = torch.einsum("hn,nhd->hd", p, vv)
            S = torch.einsum("hn,nhd->hd", p, vv.abs())
            n = h - l
            tol[b, t] = 2 * (2 * dx + n * U + 2.0 ** -20 + weights) * S + half * out[b, t].abs() + 1e-30
            tol_lse[b, t] = dx[:, 0] + n * U + 2.0 ** -20 + U * lse[b, t].abs()
    return out, lse, tol, tol_lse


class Case:
    """A batch of chunks over a cache; rows of the cache that hold no visible key are NaN."""

    def __init__(self, n_kv, T, Hq, Hkv, dk, dv=None, dtype=torch.bfloat16, page=0, n_new=None, causal=True, latent=False,
                 window=0, prefix=None, docs=None, cap=0.0, slopes=False, seed=0, spread=1.0, extra=0):
        g = torch.Generator().manual_seed(seed)
        dv = dk if dv is None else dv
        B, N = len(n_kv), max(max(n_kv), 1)
        self.B, self.T, self.N, self.dv, self.latent = B, T, N, dv, latent
        self.scale = 1 / math.sqrt(dk)
        self.cap, self.window, self.prefix = cap, window, prefix
        n_new = [min(T, n) for n in n_kv] if n_new is None else n_new
        self.pos = None
        if causal:
            self.pos = torch.full((B, T), -1, dtype=torch.int64)
            for b in range(B):
                self.pos[b, :n_new[b]] = torch.arange(n_kv[b] - n_new[b], n_kv[b])
        self.docs = None
        if docs:
            at = self.pos.clamp(min=0) if causal else torch.zeros(B, T, dtype=torch.int64)
            self.docs = at // docs * docs
        P = -(-N // page) if page else 0
        n_rows = B * P * page if page else B * N + extra
        if page:
            self.table = torch.randperm(B * P, generator=g).view(B, P).to(torch.int32)
            j = torch.arange(N)
            self.rows = [(self.table[b].long()[j // page] * page + j % page)[:n_kv[b]] for b in range(B)]
        else:
            self.table = None
            self.rows = [b * N + torch.arange(n_kv[b]) for b in range(B)]
        self.q = (torch.randn(B, T, Hq, dk, generator=g) * spread).to(dtype)
        self.k = torch.randn(n_rows, Hkv, dk, generator=g).to(dtype)
        self.v = self.k[..., :dv] if latent else torch.randn(n_rows, Hkv, dv, generator=g).to(dtype)
        used = torch.zeros(n_rows, dtype=torch.bool)
        for r in self.rows:
            used[r] = True
        self.k[~used] = float("nan")
        if not latent:
            self.v[~used] = float("nan")
        self.n_kv, self.page = list(n_kv), page
        self.slopes = torch.exp2(-8.0 * torch.arange(1, Hq + 1) / Hq).float() if slopes else None
        self.lo, self.hi = intervals(self.n_kv, self.pos, window, prefix, self.docs)
        if self.pos is None and self.lo.shape[1] != T:
            self.lo, self.hi = self.lo.expand(B, T), self.hi.expand(B, T)

    def batch(self):
        i32 = lambda x: None if x is None else x.reshape(-1).to("cuda", torch.int32)  # noqa: E731
        return L.Batch(torch.tensor(self.n_kv, dtype=torch.int32, device="cuda"), self.T, self.N, kv_seq_stride=self.N,
                       q_pos=i32(self.pos), page_table=None if self.table is None else self.table.cuda(),
                       page_size=self.page)

    def mods(self):
        m = dict(softcap=self.cap, window=self.window)
        if self.slopes is not None:
            m["slopes"] = self.slopes.cuda()
        if self.prefix is not None:
            m["prefix_len"] = torch.tensor(self.prefix, dtype=torch.int32, device="cuda")
        if self.docs is not None:
            m["doc_start"] = self.docs.reshape(-1).to("cuda", torch.int32)
        return m

    def run(self, **kw):
        q = self.q.reshape(self.B * self.T, *self.q.shape[2:]).cuda()
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        k = self.k.cuda()
        out = L.dense_attn(q, k, None if self.latent else self.v.cuda(), self.batch(), self.scale, lse=lse,
                           dv=self.dv, **self.mods(), **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, what=""):
        ref, ref_lse, tol, tol_lse = reference(self.q, self.k, self.v, self.rows, self.lo, self.hi, self.pos, self.scale,
                                               self.cap, self.slopes)
        out = out.cpu().double().view(ref.shape)
        lse = lse.cpu().double().view(ref_lse.shape)
        assert torch.isfinite(out).all(), what
        bad = (out - ref).abs() > tol
        assert not bad.any(), (what, int(bad.sum()), float(((out - ref).abs() / tol.clamp(min=1e-30)).max()))
        none = self.lo >= self.hi
        assert (out[none] == 0).all() and torch.isneginf(lse[none]).all(), what
        some = ~none
        assert ((lse - ref_lse)[some].abs() <= tol_lse[some]).all(), (what, float((lse - ref_lse)[some].abs().max()))


DTYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [(4, 1, 32), (8, 2, 64), (16, 2, 128), (6, 2, 80), (3, 3, 96), (14, 2, 64), (2, 1, 5)])
@pytest.mark.parametrize("page", [0, 16, 64, 7])
def test_decode(dtype, heads, page):
    c = Case([1, 700, 33, 0, 128, 256], 1, *heads, dtype=dtype, page=page, seed=1)
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [32, 64, 80, 128])
@pytest.mark.parametrize("T", [1, 16, 17, 40])
@pytest.mark.parametrize("cap", [0.0, 1000.0])
def test_every_column_counts_once(dtype, d, T, cap):
    # query rows that are basis vectors against one key: row m's score is the key's column m % d, and lse is the score
    c = Case([1], T, 8, 1, d, dtype=dtype, causal=False, cap=cap, seed=21)
    c.scale = 1.0
    c.k[0, 0] = (torch.arange(1, d + 1) / 8).to(dtype)
    at = torch.arange(T * 8) % d
    c.q = torch.nn.functional.one_hot(at, d).to(dtype).view(1, T, 8, d)
    out, lse = c.run()
    want = c.k[0, 0].double()[at]
    want = cap * torch.tanh(want / cap) if cap else want
    assert ((lse.view(-1).cpu().double() - want).abs() <= 2.0 ** -20 * want).all()
    assert torch.equal(out.view(T * 8, d).cpu(), c.v[0, 0].expand(T * 8, d))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [2, 17, 100])
@pytest.mark.parametrize("heads", [(4, 1, 32), (8, 2, 64), (16, 2, 128), (5, 1, 72)])
@pytest.mark.parametrize("page", [0, 32])
def test_chunks(dtype, T, heads, page):
    n_kv = [300, T, 129, 257 if T < 257 else T]
    c = Case(n_kv, T, *heads, dtype=dtype, page=page, n_new=[T, T, max(1, T // 3), T - 1], seed=2)
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mods", [
    dict(cap=5.0), dict(window=1), dict(window=40), dict(slopes=True), dict(docs=37), dict(prefix=[0, 300, 50]),
    dict(cap=2.0, slopes=True, window=100, prefix=[90, 10, 0]), dict(docs=64, prefix=[200, 200, 200], slopes=True),
    dict(docs=1)])
@pytest.mark.parametrize("T,heads", [(1, (8, 1, 128)), (45, (8, 1, 128)), (45, (3, 3, 64)), (130, (4, 2, 128))])
def test_modified_scores(dtype, mods, T, heads):
    c = Case([300, 131, 70 if T <= 70 else T], T, *heads, dtype=dtype, page=16, n_new=[T, T - T // 4, T], seed=3,
             spread=4.0, **mods)
    c.check(*c.run(), what=str(mods))
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,Hq,page", [(1, 128, 64), (1, 128, 0), (5, 128, 16), (1, 16, 64), (3, 7, 0)])
def test_latent(dtype, T, Hq, page):
    c = Case([300, 65, T, 5 + T], T, Hq, 1, 576, dv=512, dtype=dtype, page=page, latent=True, seed=4)
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("mods", [dict(cap=4.0), dict(window=70), dict(slopes=True), dict(docs=50), dict(prefix=[300, 0, 20]),
                                  dict(cap=30.0, slopes=True, prefix=[200, 60, 0], docs=20)])
@pytest.mark.parametrize("T", [1, 4])
def test_latent_modified_scores(mods, T):
    for Hq in (128, 8):
        c = Case([300, 65, 130], T, Hq, 1, 576, dv=512, dtype=torch.bfloat16, page=16, n_new=[T, 1, T], latent=True, seed=19,
                 spread=2.0, **mods)
        c.check(*c.run(), what=(mods, Hq))


@pytest.mark.gpu
def test_long_latent_without_a_workspace_and_with_one():
    # more keys than one unit of the tensor-core kernel takes: split with a workspace, on the CUDA cores without
    c = Case([5000, 2100], 1, 128, 1, 576, dv=512, dtype=torch.bfloat16, page=64, latent=True, seed=20)
    c.check(*c.run())
    c.check(*c.run(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")))
    n = L.dense_attn_workspace_size(torch.bfloat16, 2, 1, c.N, 128, 1, 576, 512)
    c.check(*c.run(workspace=torch.empty(n // 2 // 16 * 16, dtype=torch.uint8, device="cuda")))


@pytest.mark.gpu
def test_latent_beyond_one_split():
    # 8192 keys are the most that a unit takes: splits they are with a workspace, the CUDA cores without
    c = Case([9000, 2100], 1, 128, 1, 576, dv=512, dtype=torch.bfloat16, page=64, latent=True, seed=31)
    c.check(*c.run())
    c.check(*c.run(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq", [128, 5])
def test_latent_infinite_scores(Hq):
    # column 550 is no part of the values: scores of -inf in the first tiles, or everywhere
    for keys in (128, 300):
        c = Case([300], 1, Hq, 1, 576, dv=512, dtype=torch.bfloat16, page=64, latent=True, seed=35)
        c.q[..., 550] = 0.5
        c.k[c.rows[0][:keys], 0, 550] = -math.inf
        out, lse = c.run()
        if keys == 300:
            assert (out == 0).all() and torch.isneginf(lse).all()
            continue
        ref, ref_lse, tol, tol_lse = reference(c.q, c.k, c.v, [c.rows[0][keys:]], c.lo, c.hi.clamp(max=300 - keys), c.pos,
                                               c.scale)
        assert ((out.cpu().double() - ref[0]).abs() <= tol[0]).all()
        assert ((lse.cpu().double() - ref_lse[0]).abs() <= tol_lse[0]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 8, 64])
def test_latent_more_rows_than_clusters(page):
    # a cluster takes several units in turn; some rows see nothing, one tile, an odd number of tiles
    c = Case([700, 130], 100, 128, 1, 576, dv=512, dtype=torch.bfloat16, page=page, n_new=[100, 37], latent=True, seed=32)
    c.check(*c.run())
    c = Case([700, 130], 100, 128, 1, 576, dv=512, dtype=torch.bfloat16, page=page, n_new=[100, 37], latent=True, seed=33,
             window=60)
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [24, 192, 256, 8])
@pytest.mark.parametrize("heads", [(4, 2, 128), (3, 1, 8)])
def test_other_pages_and_narrow_heads(dtype, page, heads):
    for T in (1, 70):
        c = Case([500, 131, T], T, *heads, dtype=dtype, page=page, seed=22)
        c.check(*c.run(), what=(page, T))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [0.0, -0.1])
@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_scales_that_are_not_positive(dtype, scale, cap):
    for T in (1, 30):
        c = Case([200, 77], T, 4, 2, 64, dtype=dtype, cap=cap, seed=23)
        c.scale = scale
        c.check(*c.run(), what=T)


@pytest.mark.gpu
def test_results_feed_the_next_call():
    # the output is the next call's q, with nothing between them; a later call sees it whole
    for T in (1, 96):
        c = Case([4000, 3000], T, 32, 4, 128, page=64, seed=24)
        q = c.q.reshape(-1, 32, 128).cuda()
        k, v, b = c.k.cuda(), c.v.cuda(), c.batch()
        idx = torch.arange(512, dtype=torch.int32, device="cuda").repeat(2 * T, 1)
        n_sel = torch.full((2 * T,), 512, dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)
        L.dense_attn(q, k, v, b, c.scale, out=out)
        torch.cuda.synchronize()
        want = L.sparse_attn_decode(out, k, v, b, idx, n_sel, c.scale)
        want2 = L.dense_attn(out, k, v, b, c.scale)
        torch.cuda.synchronize()
        for _ in range(20):
            out.fill_(float("nan"))
            L.dense_attn(q, k, v, b, c.scale, out=out)
            got = L.sparse_attn_decode(out, k, v, b, idx, n_sel, c.scale)
            out.fill_(float("nan"))
            L.dense_attn(q, k, v, b, c.scale, out=out)
            got2 = L.dense_attn(out, k, v, b, c.scale)
            assert torch.equal(got, want) and torch.equal(got2, want2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_latent_other_widths(dtype):
    c = Case([200, 1, 64], 3, 8, 1, 96, dv=40, dtype=dtype, page=8, latent=True, n_new=[3, 1, 2], seed=5)
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 128), (192, 128), (40, 24), (128, 512)])
def test_values_of_another_width(dtype, dk, dv):
    for T in (1, 40):
        c = Case([150, 41], T, 4, 2, dk, dv=dv, dtype=dtype, page=16, seed=6)
        c.check(*c.run(), what=(dk, dv, T))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_all_cached_keys_without_positions(dtype):
    for T in (1, 30):
        c = Case([100, 1, 0, 200], T, 8, 2, 64, dtype=dtype, causal=False, seed=7)
        c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 300])
def test_long_rows(dtype, T):
    # many tiles and key splits; rising and falling maxima
    c = Case([9000, 8200], T, 2, 1, 128, dtype=dtype, page=64, seed=8, spread=3.0)
    ramp = torch.linspace(0.2, 2.0, 9000)
    for b, r in enumerate(c.rows):
        c.k[r] = (c.k[r].float() * (ramp if b == 0 else ramp.flip(0))[:len(r), None, None]).to(dtype)
    keep = torch.linspace(0, T - 1, min(T, 6)).long()     # rows that the reference computes
    out, lse = c.run()
    full = c.q, c.lo, c.hi, c.pos
    c.q, c.lo, c.hi, c.pos = (x[:, keep] for x in full)
    pick = lambda x: x.view(c.B, T, *x.shape[1:])[:, keep].reshape(-1, *x.shape[1:])  # noqa: E731
    c.check(pick(out), pick(lse))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads", [(4, 1, 128), (4, 4, 64), (2, 1, 40)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_masked_keys_do_not_reach_a_row(dtype, heads, bad):
    # one position's K and V are NaN (or infinite): rows that see it may be anything, all others are exact
    T, n = 200, 333
    for at in (0, 150, 260, 332):
        c = Case([n], T, *heads, dtype=dtype, page=16, seed=9, window=120)
        c.k[c.rows[0][at]] = bad
        c.v[c.rows[0][at]] = bad
        out, lse = c.run()
        sees = (c.lo[0] <= at) & (at < c.hi[0])
        assert torch.isfinite(out.view(T, -1)[~sees.cuda()]).all()
        if math.isnan(bad) and sees.any():
            assert torch.isnan(out.view(T, -1)[sees.cuda()]).all()
        keep = torch.nonzero(~sees).flatten()[::17]
        c.k[c.rows[0][at]] = 0
        c.v[c.rows[0][at]] = 0
        c.q, c.lo, c.hi, c.pos = (x[:, keep] for x in (c.q, c.lo, c.hi, c.pos))
        c.check(out[keep.cuda()], lse[keep.cuda()], what=at)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 40])
def test_infinite_scores(dtype, d):
    # scores of -inf weigh nothing; a row that has no other gets zeros and lse -inf; +inf gives NaN
    n = 200
    c = Case([n], 1, 2, 2, d, dtype=dtype, seed=10)
    c.q[..., 0] = 1.0
    c.k[:, :, 0] = torch.where(torch.arange(n)[:, None] % 3 == 0, 0.0, -math.inf).to(dtype)
    c.k[:, 1, 0] = -math.inf
    out, lse = c.run()
    ref, ref_lse, tol, _ = reference(c.q, c.k[::3, :1], c.v[::3, :1], [torch.arange(67)], c.lo, c.hi.clamp(max=67), c.pos,
                                     c.scale)
    assert ((out[:, 0].cpu().double() - ref[0, :, 0]).abs() <= tol[0, :, 0]).all()
    assert (out[:, 1] == 0).all() and torch.isneginf(lse[0, 1])
    c.k[5, 0, 0] = math.inf
    out, _ = c.run()
    assert torch.isnan(out[:, 0]).all()


@pytest.mark.gpu
def test_pages_out_of_range_are_skipped_and_flagged():
    for dtype, heads in ((torch.bfloat16, (8, 2, 128)), (torch.float32, (4, 1, 32)), (torch.bfloat16, (4, 2, 40))):
        for T in (1, 50):
            c = Case([200, 150], T, *heads, dtype=dtype, page=16, seed=11)
            lo, hi, rows = c.lo.clone(), c.hi.clone(), list(c.rows)
            c.table[0, 3] = 1 << 20
            c.table[1, 0] = -5
            assert L.idx_device_status(reset=True) == 0
            out, lse = c.run()
            assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS
            # the same attention without those positions
            keep = [torch.cat([torch.arange(48), torch.arange(64, 200)]), torch.arange(16, 150)]
            for b in range(2):
                for t in (0, T - 1):
                    kept = keep[b][(keep[b] >= lo[b, t]) & (keep[b] < hi[b, t])]
                    n = torch.tensor([[len(kept)]])
                    ref, _, tol, _ = reference(c.q[b:b + 1, t:t + 1], c.k, c.v, [rows[b][kept]], n * 0, n,
                                               c.pos[b:b + 1, t:t + 1], c.scale)
                    got = out.view(2, T, *out.shape[1:])[b, t].cpu().double()
                    assert ((got - ref[0, 0]).abs() <= tol[0, 0]).all(), (dtype, heads, T, b, t)


@pytest.mark.gpu
def test_strides_views_and_unaligned_caches():
    for dtype in DTYPES:
        for d in (64, 128):
            for T in (1, 20):
                c = Case([100, 77], T, 4, 2, d, dtype=dtype, seed=12)
                ref = c.run()
                q = c.q.reshape(2 * T, 4, d).cuda()
                kv = torch.full((c.k.shape[0], 4 * d + 8), float("nan"), dtype=dtype, device="cuda")
                k, v = kv[:, :2 * d].view(-1, 2, d), kv[:, 2 * d + 8:].view(-1, 2, d)
                k.copy_(c.k), v.copy_(c.v)
                assert torch.equal(L.dense_attn(q, k, v, c.batch(), c.scale), ref[0])
                # caches that start one element past an aligned address
                odd = torch.empty(c.k.numel() + 1, dtype=dtype, device="cuda")[1:].view(c.k.shape)
                odd.copy_(c.k)
                lse = torch.empty_like(ref[1])
                c.check(L.dense_attn(q, odd, c.v.cuda(), c.batch(), c.scale, lse=lse), lse)
                oddq = torch.empty(q.numel() + 1, dtype=dtype, device="cuda")[1:].view(q.shape)
                oddq.copy_(q)
                oddo = torch.empty(q.numel() + 1, dtype=dtype, device="cuda")[1:].view(q.shape)
                c.check(L.dense_attn(oddq, c.k.cuda(), c.v.cuda(), c.batch(), c.scale, lse=lse, out=oddo), lse)


@pytest.mark.gpu
def test_ragged_starts_and_neighbours_untouched():
    # kv_start addresses the sequences; rows before, between and after them are NaN and out is written exactly
    for dtype, heads in ((torch.bfloat16, (8, 2, 128)), (torch.float32, (8, 2, 128)), (torch.float16, (2, 2, 64))):
        Hq, Hkv, d = heads
        for T in (1, 33):
            c = Case([130, 64, 40], T, *heads, dtype=dtype, seed=13)
            starts = [5, 140, 207]
            k = torch.full((250, Hkv, d), float("nan"), dtype=dtype)
            v = k.clone()
            for b, s in enumerate(starts):
                k[s:s + c.n_kv[b]], v[s:s + c.n_kv[b]] = c.k[c.rows[b]], c.v[c.rows[b]]
            b = c.batch()
            b.kv_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
            buf = torch.full((3 * T + 2, Hq, d), 3.0, dtype=dtype, device="cuda")
            lse = torch.full((3 * T + 2, Hq), 3.0, device="cuda")
            L.dense_attn(c.q.reshape(-1, Hq, d).cuda(), k.cuda(), v.cuda(), b, c.scale, out=buf[1:-1], lse=lse[1:-1])
            c.check(buf[1:-1], lse[1:-1])
            assert (buf[0] == 3).all() and (buf[-1] == 3).all() and (lse[0] == 3).all() and (lse[-1] == 3).all()


@pytest.mark.gpu
def test_workspace_sizes_change_splits_not_results():
    for dtype, heads in ((torch.bfloat16, (8, 2, 128)), (torch.float32, (8, 2, 64)), (torch.bfloat16, (4, 1, 40))):
        c = Case([9000, 1700], 1, *heads, dtype=dtype, page=64, seed=14)      # more splits than a cluster merges
        need = L.dense_attn_workspace_size(dtype, 2, 1, c.N, heads[0], heads[1], heads[2], heads[2])
        assert need > 0
        for n in (16, need // 3 // 16 * 16, need // 2 // 16 * 16, need):
            ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            c.check(*c.run(workspace=ws), what=(dtype, n))


@pytest.mark.gpu
def test_repeats_bit_for_bit():
    for dtype, T in ((torch.bfloat16, 1), (torch.float16, 300), (torch.float32, 40)):
        c = Case([2500, 1900], T, 8, 2, 128, dtype=dtype, page=64, seed=15)
        a = c.run()
        for _ in range(3):
            b = c.run()
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    cases = [Case([900, 700], T, 8, 2, 128, dtype=dt, page=64, seed=16 + i)
             for i, (dt, T) in enumerate(((torch.bfloat16, 1), (torch.bfloat16, 64), (torch.float32, 1)))]
    for c in cases:
        ref = c.run()
        q = c.q.reshape(-1, *c.q.shape[2:]).cuda()
        k, v, b, m = c.k.cuda(), c.v.cuda(), c.batch(), c.mods()
        lse = torch.empty_like(ref[1])
        out = torch.empty_like(ref[0])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            L.dense_attn(q, k, v, b, c.scale, out=out, lse=lse, **m)
        side.synchronize()
        assert torch.equal(out, ref[0]) and torch.equal(lse, ref[1])
        g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        o1, o2 = torch.zeros_like(out), torch.zeros_like(out)
        with torch.cuda.graph(g1):
            L.dense_attn(q, k, v, b, c.scale, out=o1, lse=lse, **m)
        with torch.cuda.graph(g2):
            L.dense_attn(q, k, v, b, c.scale, out=o2, **m)
        for _ in range(3):
            g1.replay()
            g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(o1, ref[0]) and torch.equal(o2, ref[0])
        # a replay follows its inputs
        q.neg_()
        g1.replay()
        torch.cuda.synchronize()
        c.q = -c.q
        c.check(o1, lse)


@pytest.mark.gpu
def test_empty_batches():
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(8, 2, 64, dtype=torch.bfloat16, device="cuda")
    b = L.Batch(torch.empty(0, dtype=torch.int32, device="cuda"), 1, 8)
    assert L.dense_attn(q, k, k, b, 1.0).shape == (0, 4, 64)
    # no cached key at all
    b = L.Batch(torch.zeros(2, dtype=torch.int32, device="cuda"), 1, 0)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.ones(2, 4, device="cuda")
    assert (L.dense_attn(q, k[:0], k[:0], b, 1.0, lse=lse) == 0).all() and torch.isneginf(lse).all()


# ------------------------------------------------------------------------------------------ refusals (CPU)

def _call(**kw):
    L.build()
    lib = L.load()
    b = L._Batch(1, 1, ctypes.c_void_p(16), None, 16, ctypes.c_void_p(16), 16)
    a = dict(q=16, dtype=L.IDX_BF16, Hq=8, Hkv=2, dk=128, dv=128, k=16, v=16, ks=256, vs=256, rows=16, b=b, mods=None,
             scale=1.0, out=16, lse=None, ws=None, wb=0)
    a.update(kw)
    m = None if a["mods"] is None else ctypes.byref(L._Mods(**a["mods"]))
    st = lib.dense_attn(a["q"], a["dtype"], a["Hq"], a["Hkv"], a["dk"], a["dv"], a["k"], a["v"], a["ks"], a["vs"],
                        a["rows"], a["b"], m, a["scale"], a["out"], a["lse"], a["ws"], a["wb"], None)
    return st, lib.idx_last_error().decode()


@pytest.mark.parametrize("kw,word", [
    (dict(dtype=7), "dtype"), (dict(Hq=6, Hkv=4), "Hq"), (dict(Hq=0), "Hq"), (dict(Hkv=0), "Hq"), (dict(dk=577), "dk"),
    (dict(dv=513), "dv"), (dict(dk=0), "dk"), (dict(ks=255), "kv_row_stride"), (dict(vs=255), "v_row_stride"),
    (dict(v=None), "latent"), (dict(v=None, Hkv=1, Hq=4, dk=64, dv=128), "latent"), (dict(rows=-1), "kv_rows"),
    (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"), (dict(q=None), "NULL"),
    (dict(k=None), "NULL"), (dict(out=None), "NULL"), (dict(ws=ctypes.c_void_p(24), wb=64), "aligned"),
    (dict(mods=dict(softcap=-1.0)), "softcap"), (dict(mods=dict(softcap=float("inf"))), "softcap"),
    (dict(mods=dict(softcap=float("nan"))), "softcap"), (dict(mods=dict(softcap=1e-40)), "softcap"), (dict(mods=dict(window=-1)), "window"),
    (dict(b=L._Batch(1, 0, ctypes.c_void_p(16), None, 16, None, 16)), "n_q_per_seq"),
    (dict(b=L._Batch(-1, 1, ctypes.c_void_p(16), None, 16, None, 16)), "n_seq"),
    (dict(b=L._Batch(1, 1, None, None, 16, None, 16)), "n_kv"),
    (dict(b=L._Batch(1, 1, ctypes.c_void_p(16), None, 16, None, 256, ctypes.c_void_p(16), 3, 64)), "page_table_stride"),
    (dict(b=L._Batch(1, 1, ctypes.c_void_p(16), None, 16, None, 16), mods=dict(window=4)), "q_pos"),
    (dict(b=L._Batch(1, 1, ctypes.c_void_p(16), None, 16, None, 16), mods=dict(slopes=16)), "q_pos"),
    (dict(b=L._Batch(1, 1, ctypes.c_void_p(16), None, 16, None, 16), mods=dict(prefix_len=16)), "q_pos"),
])
def test_bad_arguments_are_refused_on_the_host(kw, word):
    st, msg = _call(**kw)
    assert st == L.IDX_ERR_INVALID_ARG and word in msg and msg.startswith("dense_attn"), msg


def test_empty_batch_needs_no_pointers():
    st, _ = _call(q=None, k=None, out=None, b=L._Batch(0, 1, None, None, 0, None, 0))
    assert st == L.IDX_OK


def test_workspace_size_is_host_arithmetic():
    L.build()
    assert L.dense_attn_workspace_size(torch.bfloat16, 0, 1, 16, 8, 2, 128, 128) == 0
    assert L.dense_attn_workspace_size(torch.bfloat16, 1, 1, 16, 8, 3, 128, 128) == 0
    assert L.dense_attn_workspace_size(torch.bfloat16, 1, 1, 16, 8, 2, 1000, 128) == 0
    n = L.dense_attn_workspace_size(torch.float32, 1, 1, 4096, 8, 2, 128, 128)
    assert n > 0 and n % (8 * 130 * 4) == 0


def test_binding_refuses_bad_tensors():
    cpu = torch.zeros(1, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        L.dense_attn(cpu, cpu, cpu, L.Batch(torch.zeros(1, dtype=torch.int32), 1, 16), 1.0)


@pytest.mark.gpu
def test_binding_refuses_mismatched_tensors():
    dev = dict(device="cuda", dtype=torch.bfloat16)
    q, k = torch.zeros(1, 4, 64, **dev), torch.zeros(16, 2, 64, **dev)
    b = L.Batch(torch.tensor([16], dtype=torch.int32, device="cuda"), 1, 16,
                q_pos=torch.tensor([15], dtype=torch.int32, device="cuda"))
    ok = lambda **kw: L.dense_attn(kw.pop("q", q), kw.pop("k", k), kw.pop("v", k), b, 1.0, **kw)  # noqa: E731
    ok()
    for kw in (dict(q=q[:, :, ::2]), dict(k=k.half()), dict(v=k.float()), dict(k=k[:, :, :32]), dict(k=k[:8]),
               dict(slopes=torch.zeros(3, device="cuda")), dict(slopes=torch.zeros(4, device="cuda").half()),
               dict(prefix_len=torch.zeros(1, device="cuda", dtype=torch.int64)),
               dict(doc_start=torch.zeros(0, device="cuda", dtype=torch.int32)), dict(out=torch.zeros(1, 4, 64, device="cuda")),
               dict(lse=torch.zeros(1, 4, **dev)), dict(v=None), dict(dv=32),
               dict(k=torch.zeros(16, 4, 64, **dev)[:, ::2], v=torch.zeros(16, 4, 64, **dev)[:, ::2])):
        with pytest.raises(ValueError):
            ok(**kw)
    with pytest.raises(L.LidxError):
        ok(softcap=-1.0)


@pytest.mark.gpu
def test_binding_refuses_a_window_beyond_int32():
    q, k = torch.zeros(1, 4, 64, device="cuda"), torch.zeros(16, 2, 64, device="cuda")
    b = L.Batch(torch.tensor([16], dtype=torch.int32, device="cuda"), 1, 16,
                q_pos=torch.tensor([15], dtype=torch.int32, device="cuda"))
    L.dense_attn(q, k, k, b, 1.0, window=2**31 - 1)
    for window in (2**31, 2**32 + 4):
        with pytest.raises(ValueError, match="window"):
            L.dense_attn(q, k, k, b, 1.0, window=window)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 130, 1000, 2600])
@pytest.mark.parametrize("dtype,heads", [(torch.bfloat16, (8, 2, 128)), (torch.float32, (8, 2, 64))])
def test_key_splits_share_what_a_window_leaves(dtype, heads, window):
    # a row's splits divide the tiles that it sees, wherever they lie in a long cache; latent: the same
    for T in (1, 3):
        c = Case([5000, 900, 2049], T, *heads, dtype=dtype, page=16, window=window, seed=36)
        c.check(*c.run(), what=T)
    if dtype is torch.bfloat16:
        c = Case([5000, 900], 1, 128, 1, 576, dv=512, dtype=dtype, page=64, window=window, latent=True, seed=37)
        c.check(*c.run())
    assert L.idx_device_status(reset=True) == 0
