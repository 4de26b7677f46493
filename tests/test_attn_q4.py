"""dense_attn_q4 against softmax attention in 64 bits over the values that the codes stand for, and its refusals.

Tolerance of an output element, with u = 2^-24, half(T) = finfo(T).eps / 2, code n, scale s, minimum m, and m' = m + 8 s, so
that a value is s (n - 8) + m':
  scores   sums of dk terms in f32, either of q (s n + m) or as s sum q (n - 8) + m' sum q: off by at most (dk + 6) u A, where
           A = sum |q| (s |n - 8| + |m'|) (in which q's rounding to f16 at its row's scale, 2^-25 of its largest element, is
           counted too; an odd column's code is taken as 72 too much, which is taken off again: (dk + 6) u 72 sum |q| s more);
           many rows, or other heads: K is a sum of two numbers of the inputs' type, half(T)^2 sum |q k| more;
           scaling, cap, bias and maximum 8 u (|x| + cap + slope * distance + 1): dx;
  weights  off by a factor within e^(2 dx) (1 + 2^-20), and on the tensor cores by half a step of f16, to which they (few rows
           of 64 or 128 columns: their product with the value's scale) are rounded for the second product;
  values   many rows, or other heads: half a step of f16 each;
  sums     n f32 additions: n u of the sum of magnitudes, S = sum p (s |n - 8| + |m'|).
|error| <= 2 (2 dx + n u + 2^-20 + rounded weights and values) S + half(T) |out|.  lse: dx + n u + 2^-20 + u |lse|."""

import ctypes
import dataclasses
import math

import pytest
import torch

import lightning_indexer_top_gb300 as L
from test_dense_attn import Case

U = 2.0 ** -24
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def half(t):
    return torch.finfo(t).eps / 2


def pack(codes, scale, low, pad=0):
    """Rows of a 4-bit cache (uint8, CPU) from codes [rows, heads, d] and f32 scale and minimum [rows, heads]."""
    n, h, d = codes.shape
    c = codes.to(torch.uint8)
    c = (c[..., 0::2] | (c[..., 1::2] << 4)).reshape(n, -1)
    f = torch.stack([scale, low], -1).reshape(n, -1).contiguous().view(torch.uint8)
    w = L.idx_q4_row_bytes(h, d) + pad
    return torch.cat([c, f, torch.full((n, w - c.shape[1] - f.shape[1]), 255, dtype=torch.uint8)], 1)


class Case4(Case):
    """A dense attention case whose K and V are 4-bit rows; rows that hold no cached key are bytes that are no numbers."""

    def __init__(self, n_kv, T, Hq, Hkv, dk, dv=None, dtype=torch.bfloat16, seed=0, pad=0, offset=0.0, **kw):
        super().__init__(n_kv, T, Hq, Hkv, dk, dv=dv, dtype=dtype, seed=seed, **kw)
        g = torch.Generator().manual_seed(seed + 1000)
        self.Hkv, self.dtype = Hkv, dtype
        used = torch.zeros(self.k.shape[0], dtype=torch.bool)
        for r in self.rows:
            used[r] = True
        self.coded, self.caches = [], []
        for d in (dk, self.dv):
            x = torch.randn(self.k.shape[0], Hkv, d, generator=g) + offset
            low, high = x.aminmax(dim=-1)
            scale = (high - low) / 15
            codes = ((x - low[..., None]) / scale[..., None]).round().clamp(0, 15)
            c = pack(codes, scale, low, pad)
            c[~used] = 255
            self.coded.append((codes.double(), scale.double(), low.double()))
            self.caches.append(c)
        self.sync()

    def sync(self):
        self.k, self.v = (c * s[..., None] + m[..., None] for c, s, m in self.coded)

    def recode(self, which, row, head, codes=None, scale=None, low=None):
        """Changes one head row of a cache (0: K, 1: V)."""
        c, s, m = (t[row:row + 1].clone() for t in self.coded[which])
        if codes is not None:
            c[0, head] = codes
        if scale is not None:
            s[0, head] = scale
        if low is not None:
            m[0, head] = low
        for t, x in zip(self.coded[which], (c, s, m)):
            t[row] = x[0]
        w = self.caches[which].shape[1]
        self.caches[which][row] = pack(c, s.float(), m.float(), w - L.idx_q4_row_bytes(c.shape[1], c.shape[2]))[0]
        self.sync()

    def run(self, caches=None, **kw):
        q = self.q.reshape(self.B * self.T, *self.q.shape[2:]).cuda()
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        kc, vc = caches or [c.cuda() for c in self.caches]
        out = L.dense_attn_q4(q, kc, vc, self.batch(), self.scale, self.Hkv, dv=self.dv, lse=lse, **self.mods(), **kw)
        torch.cuda.synchronize()
        return out, lse

    def reference(self):
        B, T, Hq, dk = self.q.shape
        G = Hq // self.Hkv
        small = self.dtype == torch.float32
        codes = not small and T * G <= 256 and dk == self.dv and dk in (64, 128)      # (the codes themselves may be multiplied)
        rounded = 0.0 if small else (1 if codes else 2) * half(torch.float16)
        out = torch.zeros(B, T, Hq, self.dv, dtype=torch.float64)
        lse = torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
        tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
        expand = lambda t: t.repeat_interleave(G, 1)     # noqa: E731
        for b in range(B):
            for t in range(T):
                l, h = int(self.lo[b, t]), int(self.hi[b, t])
                if l >= h:
                    continue
                at = self.rows[b][l:h]
                at = at[at >= 0]
                if not len(at):
                    continue
                qq = self.q[b, t].double()
                (kc, ks, km), (vc, vs, vm) = ([expand(x[at]) for x in c] for c in self.coded)
                k, v = kc * ks[..., None] + km[..., None], vc * vs[..., None] + vm[..., None]
                x = torch.einsum("hd,nhd->hn", qq, k) * self.scale
                A = torch.einsum("hd,nhd->hn", qq.abs(), (kc - 8).abs() * ks[..., None] + (km + 8 * ks).abs()[..., None]) * abs(self.scale)
                if codes:
                    A = A + 72 * torch.einsum("hd,nh->hn", qq.abs(), ks) * abs(self.scale)
                size = x.abs() + 1
                if self.cap:
                    x = self.cap * torch.tanh(x / self.cap)
                    size = size + self.cap
                if self.slopes is not None:
                    dist = (int(self.pos[b, t]) - torch.nonzero(self.rows[b][l:h] >= 0)[:, 0] - l).abs().double()
                    x = x - self.slopes.double()[:, None] * dist
                    size = size + self.slopes.double()[:, None] * dist
                if not small:
                    A = A + half(self.dtype) ** 2 / U / (dk + 6) * torch.einsum("hd,nhd->hn", qq.abs(), k.abs()) * abs(self.scale)
                dx = ((dk + 6) * U * A + 8 * U * size).amax(1, keepdim=True)
                lse[b, t] = torch.logsumexp(x, 1)
                p = torch.softmax(x, 1)
                out[b, t] = torch.einsum("hn,nhd->hd", p, v)
                S = torch.einsum("hn,nhd->hd", p, (vc - 8).abs() * vs[..., None] + (vm + 8 * vs).abs()[..., None])
                n = h - l
                tol[b, t] = 2 * (2 * dx + n * U + 2.0 ** -20 + rounded) * S + half(self.dtype) * out[b, t].abs() + 1e-30
                tol_lse[b, t] = dx[:, 0] + n * U + 2.0 ** -20 + U * lse[b, t].abs()
        return out, lse, tol, tol_lse

    def check(self, out, lse, what="", skip=None):
        ref, ref_lse, tol, tol_lse = self.reference()
        out, lse = out.cpu().double().view(ref.shape), lse.cpu().double().view(ref_lse.shape)
        if skip is not None:
            out, ref, tol, lse, ref_lse, tol_lse = (t[~skip] for t in (out, ref, tol, lse, ref_lse, tol_lse))
        assert torch.isfinite(out).all(), what
        bad = (out - ref).abs() > tol
        assert not bad.any(), (what, int(bad.sum()), float(((out - ref).abs() / tol.clamp(min=1e-30)).max()))
        none = torch.isneginf(ref_lse)
        assert (out[none] == 0).all() and torch.isneginf(lse[none]).all(), what
        assert ((lse - ref_lse)[~none].abs() <= tol_lse[~none]).all(), (what, float((lse - ref_lse)[~none].abs().max()))


HEADS = [(4, 1, 32), (8, 2, 64), (16, 2, 128), (32, 2, 128), (6, 2, 80), (3, 3, 96), (14, 2, 64), (2, 1, 8), (5, 5, 128), (17, 1, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("page,pad", [(0, 0), (16, 4), (64, 16), (7, 0), (1, 0)])
def test_decode(dtype, heads, page, pad):
    c = Case4([1, 700, 33, 0, 128, 256, 2100], 1, *heads, dtype=dtype, page=page, pad=pad, seed=1)
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [32, 64, 80, 128])
@pytest.mark.parametrize("T", [1, 2, 16, 40])
def test_every_column_counts_once(dtype, d, T):
    # query rows that are basis vectors against one key: row m's score is the key's column m % d
    c = Case4([1], T, 8, 1, d, dtype=dtype, causal=False, seed=21)
    c.scale = 1.0
    codes = torch.arange(d) % 16
    c.recode(0, 0, 0, (codes * 7 + torch.arange(d) // 16) % 16, 0.5, -2.0)
    c.recode(1, 0, 0, codes, 2.0, -16.0)
    at = torch.arange(T * 8) % d
    c.q = torch.nn.functional.one_hot(at, d).to(dtype).view(1, T, 8, d)
    out, lse = c.run()
    assert ((lse.view(-1).cpu().double() - c.k[0, 0][at]).abs() <= 2.0 ** -20 * c.k[0, 0][at].abs() + 2.0 ** -21).all()
    assert torch.equal(out.view(T * 8, d).cpu().double(), c.v[0, 0].expand(T * 8, d))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [2, 5, 17, 100, 140])
@pytest.mark.parametrize("heads", [(4, 1, 32), (8, 2, 64), (16, 2, 128), (6, 1, 72), (4, 4, 128)])
@pytest.mark.parametrize("page", [0, 32, 3])
def test_chunks(dtype, T, heads, page):
    n_kv = [300, T, 129, 257 if T < 257 else T]
    c = Case4(n_kv, T, *heads, dtype=dtype, page=page, n_new=[T, T, max(1, T // 3), T - 1], seed=2)
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("mods", [
    dict(cap=5.0), dict(window=1), dict(window=40), dict(slopes=True), dict(docs=37), dict(prefix=[0, 300, 50]),
    dict(cap=2.0, slopes=True, window=100, prefix=[90, 10, 0]), dict(docs=64, prefix=[200, 200, 200], slopes=True),
    dict(docs=1)])
@pytest.mark.parametrize("T,heads", [(1, (8, 1, 128)), (3, (6, 2, 64)), (45, (8, 1, 128)), (45, (3, 3, 64)), (130, (4, 2, 128))])
def test_modified_scores(dtype, mods, T, heads):
    c = Case4([300, 131, 70 if T <= 70 else T], T, *heads, dtype=dtype, page=16, n_new=[T, T - T // 4, T], seed=3,
              spread=4.0, **mods)
    c.check(*c.run(), what=str(mods))
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 4, 60])
def test_keys_and_values_of_different_widths(dtype, T):
    for dk, dv in ((64, 128), (128, 64), (192, 128), (64, 256)):
        c = Case4([200, 90], T, 4, 2, dk, dv=dv, dtype=dtype, page=16, seed=4)
        c.check(*c.run(), what=(dk, dv))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 6, 70])
@pytest.mark.parametrize("share", [0.0, 0.3, 1.0])
def test_workspaces_of_any_size(dtype, T, share):
    c = Case4([5000, 2100], T, 8, 2, 128, dtype=dtype, page=16, seed=5)
    n = L.dense_attn_q4_workspace_size(dtype, 2, T, c.N, 8, 2, 128, 128)
    c.check(*c.run(workspace=torch.empty(max(16, int(n * share) // 16 * 16), dtype=torch.uint8, device="cuda")))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 2, 40])
@pytest.mark.parametrize("spread", [1e-3, 1.0, 2.0 ** 7])
def test_queries_of_any_size(dtype, T, spread):
    # (f16: up to 128 times five; bf16 and f32 far beyond f16's range, the scale undoes it)
    big = spread * (2.0 ** 60 if dtype != torch.float16 else 1.0)
    c = Case4([150, 40], T, 8, 1, 64, dtype=dtype, seed=6, spread=big)
    c.scale = 1 / (8 * big)
    c.check(*c.run())
    c.q[:, :, 3] = 0          # a query of zeros weighs all keys alike
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 40])
def test_negative_and_zero_scales(dtype, T):
    c = Case4([150, 40], T, 8, 2, 128, dtype=dtype, seed=7)
    for s in (0.0, -0.1):
        c.scale = s
        c.check(*c.run(), what=s)
    # head rows without a span, and one with a negative scale
    c.scale = 0.1
    c.recode(0, 3, 1, torch.zeros(128), 0.0, 1.5)
    c.recode(1, 5, 0, torch.zeros(128), 0.0, -0.25)
    c.recode(1, 6, 0, None, -0.3, 2.0)
    c.recode(0, 7, 0, None, -0.3, 2.0)
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 5, 40])
@pytest.mark.parametrize("d", [64, 128, 80])
def test_a_nan_reaches_the_rows_that_see_it_and_no_other(dtype, T, d):
    c = Case4([300, 200], T, 8, 2, d, dtype=dtype, page=16, window=30, seed=8)
    j = 300 - 1 - T // 2
    at = int(c.rows[0][j])
    for which, value in ((0, math.nan), (1, math.nan), (1, math.inf)):
        c = Case4([300, 200], T, 8, 2, d, dtype=dtype, page=16, window=30, seed=8)
        seen = (c.lo[0] <= j) & (j < c.hi[0])
        assert seen.any() and (T == 1 or not seen.all())
        c.recode(which, at, 1, None, value if which == 0 or math.isnan(value) else None, value)
        out, lse = c.run()
        o = out.view(2, T, 2, 4, d)
        assert not torch.isfinite(o[0, seen.cuda(), 1]).any(), (which, value)
        assert torch.isfinite(o[1]).all() and torch.isfinite(o[0, :, 0]).all() and torch.isfinite(o[0, ~seen.cuda()]).all()
        skip = torch.zeros(2, T, 8, dtype=torch.bool)
        skip[0, :, 4:] = seen[:, None]
        c.recode(which, at, 1, None, 0.1, -1.0)      # (what the others are to be)
        c.check(out, lse, skip=skip)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 6, 60])
@pytest.mark.parametrize("page", [16, 5])
def test_pages_out_of_range_are_skipped_and_flagged_where_seen(dtype, T, page):
    c = Case4([200, 180], T, 8, 2, 128, dtype=dtype, page=page, window=75, seed=9)
    lost = 130 // page
    c.table[0, lost], c.table[0, 0], c.table[1, lost] = -1, c.k.shape[0] // page, 10 ** 6      # page 0 is seen by nobody
    for b in (0, 1):
        c.rows[b] = c.rows[b].clone()
        c.rows[b][lost * page:(lost + 1) * page] = -1
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS
    c = Case4([200, 180], T, 8, 2, 128, dtype=dtype, page=page, window=20, seed=9)
    c.table[:, 0] = -1
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [16, 5])
def test_many_rows_and_pages_out_of_range(dtype, page):
    c = Case4([200, 180], 70, 8, 2, 128, dtype=dtype, page=page, window=75, seed=9)
    lost = 130 // page
    c.table[0, lost], c.table[0, 0], c.table[1, lost] = -1, c.k.shape[0] // page, 10 ** 6      # page 0 is seen by nobody
    for b in (0, 1):
        c.rows[b] = c.rows[b].clone()
        c.rows[b][lost * page:(lost + 1) * page] = -1
    c.check(*c.run())
    assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", [(1, 128), (5, 64), (70, 128), (70, 64), (3, 80)])
@pytest.mark.parametrize("page", [0, 16])
def test_values_of_any_size(dtype, T, d, page):
    # (f16: its results have to hold them)
    c = Case4([300, 41], T, 8, 2, d, dtype=dtype, seed=13, page=page)
    big = 2.0 ** (6 if dtype == torch.float16 else 60)
    for h, f in ((0, 1 / big), (1, big)):
        for x in c.coded[1][1:]:
            x[:, h] *= f
    codes, scale, low = c.coded[1]
    c.caches[1] = pack(codes, scale.float(), low.float())
    c.sync()
    c.check(*c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,d", [(1, 128), (40, 64), (70, 128), (70, 64), (3, 80)])
def test_values_beyond_half_precision(dtype, T, d):
    c = Case4([200, 180], T, 8, 2, d, dtype=dtype, seed=11)
    c.q = (c.q * 1e-4).to(c.q.dtype)
    c.recode(0, int(c.rows[0][5]), 1, None, 1e4, -2e4)
    c.recode(1, int(c.rows[1][6]), 0, None, 1e4, -2e4)
    c.check(*c.run())


def check_without_floor(c, out, lse):
    """c.check, for results that 1e-30 is not small beside: their types' least numbers instead."""
    ref, ref_lse, tol, tol_lse = c.reference()
    out, lse = out.cpu().double().view(ref.shape), lse.cpu().double().view(ref_lse.shape)
    none = torch.isneginf(ref_lse)
    tol[none] = 1e-30
    tol = tol - 1e-30 + {torch.float16: 2.0 ** -25}.get(c.dtype, 2.0 ** -134)
    assert torch.isfinite(out).all()
    bad = (out - ref).abs() > tol
    assert not bad.any(), (int(bad.sum()), float(((out - ref).abs() / tol).max()))
    assert (out[none] == 0).all() and torch.isneginf(lse[none]).all()
    assert ((lse - ref_lse)[~none].abs() <= tol_lse[~none]).all(), float((lse - ref_lse)[~none].abs().max())


def rescale(c, which, head, factors):
    """Multiplies head `head` of K (0) or V (1) by factors [cache rows] (powers of two)."""
    codes, scale, low = c.coded[which]
    scale[:, head] = (scale[:, head].float() * factors.float()).double()
    low[:, head] = (low[:, head].float() * factors.float()).double()
    pad = c.caches[which].shape[1] - L.idx_q4_row_bytes(codes.shape[1], codes.shape[2])
    c.caches[which] = pack(codes, scale.float(), low.float(), pad)
    c.sync()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(70, 128), (70, 64), (130, 96), (3, 80)])
def test_values_that_a_row_does_not_see_cost_it_nothing(dtype, T, d):
    # the last key but one is far larger than the others, and far smaller ones lie between: seen by the last rows alone
    for power in (20, 45, -45, 100):
        c = Case4([200, 180], T, 8, 2, d, dtype=dtype, page=16, seed=14)
        f = torch.ones(c.k.shape[0])
        f[c.rows[0][198]] = 2.0 ** power
        f[c.rows[1][10 if power < 0 else 178]] = 2.0 ** power
        rescale(c, 1, 1, f)
        check_without_floor(c, *c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 128), (5, 64), (30, 128), (70, 128), (3, 80)])
@pytest.mark.parametrize("page", [0, 16, 5])
def test_values_of_every_size(dtype, T, d, page):
    # head 0: all of one size; head 1: sizes that differ from key to key
    for power in (-115, -90, -78, -63, -57, 60, 64, 90, 115):
        c = Case4([300, 41], T, 8, 2, d, dtype=dtype, seed=15, page=page)
        g = torch.Generator().manual_seed(abs(power))
        n = c.k.shape[0]
        rescale(c, 1, 0, torch.full((n,), 2.0 ** power))
        rescale(c, 1, 1, torch.exp2(torch.randint(min(power, -power), abs(power) + 1, (n,), generator=g).float()))
        check_without_floor(c, *c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 128), (5, 64), (70, 128), (3, 80)])
def test_constant_values_of_every_size(dtype, T, d):
    # rows without a span, beside rows with one
    for power in (-115, -60, 30, 60, 115):
        for share in (1.0, 0.5):
            c = Case4([300, 41], T, 8, 2, d, dtype=dtype, seed=16)
            g = torch.Generator().manual_seed(power + 200)
            codes, scale, low = c.coded[1]
            flat = torch.rand(scale.shape, generator=g) < share
            codes[flat] = 0.0
            scale[flat] = 0.0
            low[flat] = (torch.where(torch.rand(scale.shape, generator=g) < 0.5, -1.0, 1.0) * 2.0 ** power).double()[flat]
            c.caches[1] = pack(codes, scale.float(), low.float())
            c.sync()
            check_without_floor(c, *c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 128), (5, 64), (70, 128), (3, 80)])
@pytest.mark.parametrize("mods", [{}, dict(cap=4.0)])
def test_keys_and_queries_of_every_size(dtype, T, d, mods):
    # (keys, queries, scale): together as they were
    for k, q, s in ((100, -100, 0), (-100, 100, 0), (100, 0, -100), (-100, 0, 100), (0, 100, -100), (0, -100, 100), (55, 55, -110), (-55, -55, 110)):
        c = Case4([300, 41], T, 8, 2, d, dtype=dtype, seed=17, **mods)
        for h in (0, 1):
            rescale(c, 0, h, torch.full((c.k.shape[0],), 2.0 ** k))
        c.q = c.q * 2.0 ** q
        c.scale *= 2.0 ** s
        check_without_floor(c, *c.run())


@pytest.mark.gpu
@pytest.mark.parametrize("T,heads", [(1, (8, 2, 128)), (5, (8, 2, 64)), (70, (8, 2, 128)), (150, (4, 2, 64)), (3, (6, 2, 80)), (90, (6, 2, 96))])
@pytest.mark.parametrize("mods", [{}, dict(cap=4.0), dict(slopes=True, window=60)])
def test_f16_keys_of_every_size(T, heads, mods):
    # head 0: all of one size, which the scale undoes; head 1: a key of another size, which the last rows alone see
    for power in (-45, -20, -12, 12, 40):
        c = Case4([300, 170], T, *heads, dtype=torch.float16, seed=20, page=16, **mods)
        n = c.k.shape[0]
        f = torch.full((n,), 2.0 ** power)
        rescale(c, 0, 0, f)
        f[c.rows[0][298]] *= 2.0 ** (power // 2)
        rescale(c, 0, 1, f)
        c.scale *= 2.0 ** -power
        check_without_floor(c, *c.run())
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,heads", [(1, (8, 2, 64)), (1, (16, 2, 128)), (4, (24, 8, 64)), (20, (8, 1, 128)), (1, (20, 4, 80)), (1, (8, 8, 96)),
                                     (5, (4, 1, 32)), (70, (8, 2, 128)), (150, (4, 2, 64)), (90, (6, 2, 96)), (300, (2, 1, 128))])
@pytest.mark.parametrize("n_kv", [(400, 130), (1, 2), (17, 33)])
@pytest.mark.parametrize("mods", [{}, dict(cap=3.0, slopes=True)])
def test_f16_results_are_as_near_as_their_own_rounding(T, heads, n_kv, mods):
    # What is not the result's rounding (2^-12 of an element at most, in the mean half of that) is f32's: sums of 128 terms, off by
    # some 2^-24 sqrt(128) of scores of size 4, 2^-17.  Errors that know nothing of each other add in squares: 1 + 2^-8.
    c = Case4([max(n, T) for n in n_kv], T, *heads, dtype=torch.float16, page=16, seed=19, **mods)
    out, _ = c.run()
    ref, ref_lse, _, _ = c.reference()
    seen = ~torch.isneginf(ref_lse)
    err = (out.cpu().double().view(ref.shape) - ref)[seen].square().mean().sqrt()
    own = (ref.half().double() - ref)[seen].square().mean().sqrt()
    assert err <= 1.05 * own, float(err / own)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("page", [0, 16, 5])
def test_caches_beyond_32_bit_offsets(dtype, page):
    # rows that lie more than 2^32 bytes behind the caches' first
    w = L.idx_q4_row_bytes(8, 128)
    big = [torch.empty(2 ** 32 // w + 4096, w, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for T in (1, 5, 70):
        c = Case4([300, 170], T, 8, 8, 128, dtype=dtype, page=page, seed=21)
        n = c.k.shape[0]
        at = (big[0].shape[0] - n) // max(page, 1) * max(page, 1)
        for x, y in zip(big, c.caches):
            x[at:at + n] = y.cuda()
        real = c.batch
        if page:
            c.table = c.table + at // page
        else:
            c.batch = lambda: dataclasses.replace(real(), kv_start=torch.tensor([at, at + c.N], dtype=torch.int32, device="cuda"))
        c.check(*c.run(caches=big))
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,d", [(3, 80), (70, 128)])
def test_a_workspace_that_does_not_fit_is_done_without(T, d):
    c = Case4([300, 41], T, 8, 2, d, dtype=torch.bfloat16, seed=18)
    real = c.batch
    c.batch = lambda: dataclasses.replace(real(), max_n_kv=2 ** 22)      # (gigabytes; the sequences are as short as they were)
    n = L.dense_attn_q4_workspace_size(torch.bfloat16, 2, T, 2 ** 22, 8, 2, d, d)
    assert n > 2 ** 32
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + 2 ** 30) / torch.cuda.get_device_properties(0).total_memory)
    try:
        out, lse = c.run()
        with pytest.raises(torch.cuda.OutOfMemoryError):
            torch.empty(n, dtype=torch.uint8, device="cuda")
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    c.check(out, lse)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_rows_captured_with_a_page_that_comes_back(dtype):
    c = Case4([200, 180], 70, 8, 2, 128, dtype=dtype, page=16, seed=12)
    q = c.q.reshape(c.B * c.T, 8, 128).cuda()
    caches, batch, lse = [x.cuda() for x in c.caches], c.batch(), torch.zeros(c.B * c.T, 8, device="cuda")
    ws = torch.empty(L.dense_attn_q4_workspace_size(dtype, 2, 70, batch.max_n_kv, 8, 2, 128, 128), dtype=torch.uint8, device="cuda")
    call = lambda: L.dense_attn_q4(q, *caches, batch, c.scale, 2, lse=lse, workspace=ws)  # noqa: E731
    first, first_lse = call().clone(), lse.clone()
    c.check(first, first_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    entry = batch.page_table[1, 3].clone()
    batch.page_table[1, 3] = -1
    graph.replay()
    torch.cuda.synchronize()
    assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS
    kept = c.rows[1]
    c.rows[1] = kept.clone()
    c.rows[1][48:64] = -1
    c.check(out, lse)
    c.rows[1] = kept
    batch.page_table[1, 3] = entry
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(lse, first_lse) and L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40])
def test_rows_past_a_contiguous_cache_are_skipped(T):
    c = Case4([120, 120], T, 8, 2, 64, dtype=torch.bfloat16, seed=10)
    c.rows[1] = c.rows[1].clone()
    c.rows[1][100:] = -1
    short = [x[:220].cuda() for x in c.caches]
    c.check(*c.run(caches=short))
    assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 30])
def test_empty_batches_and_rows(dtype, T):
    c = Case4([60, 9, 0], T, 4, 1, 128, dtype=dtype, n_new=[min(T, 1), 0, 0], seed=11)
    c.check(*c.run())
    b = L.Batch(torch.zeros(0, dtype=torch.int32, device="cuda"), T, 60)
    assert L.dense_attn_q4(torch.zeros(0, 4, 128, dtype=dtype, device="cuda"), *[x.cuda() for x in c.caches], b, 1.0, 1).shape == (0, 4, 128)
    none = [x[:0].cuda() for x in c.caches]
    b = L.Batch(torch.zeros(2, dtype=torch.int32, device="cuda"), T, 0)
    out = L.dense_attn_q4(torch.ones(2 * T, 4, 128, dtype=dtype, device="cuda"), *none, b, 1.0, 1)
    assert (out == 0).all() and L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T,heads", [(1, (32, 4, 128)), (4, (24, 8, 64)), (64, (8, 2, 128))])
def test_same_bits_again_captured_and_on_two_streams(T, heads):
    c = Case4([3000, 900, 2000], T, *heads, dtype=torch.bfloat16, page=16, seed=12)
    caches = [x.cuda() for x in c.caches]
    a, la = c.run(caches=caches)
    q = c.q.reshape(c.B * T, *c.q.shape[2:]).cuda()
    b = c.batch()
    outs = [torch.empty_like(a) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, o in zip(streams, outs):
            with torch.cuda.stream(s):
                L.dense_attn_q4(q, *caches, b, c.scale, heads[1], out=o)
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    n = L.dense_attn_q4_workspace_size(torch.bfloat16, c.B, T, c.N, *heads[:2], heads[2], heads[2])
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.dense_attn_q4(q, *caches, b, c.scale, heads[1], out=outs[2], workspace=ws)
    ws.fill_(255)
    graph.replay()
    assert all(torch.equal(o, a) for o in outs)
    # other lengths and rows, read by the replay
    b.n_kv.copy_(torch.tensor([2990, 10, 64]))
    b.q_pos.copy_(torch.where(b.q_pos < 0, b.q_pos, b.q_pos.clamp(max=9)))
    graph.replay()
    assert torch.equal(outs[2], L.dense_attn_q4(q, *caches, b, c.scale, heads[1]))
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_agrees_with_dense_attn_over_the_values():
    # the values read back in f32, attended by dense_attn: the same up to f32's rounding
    c = Case4([500, 77], 3, 8, 2, 80, dtype=torch.float32, page=8, seed=13)
    out, lse = c.run()
    caches = [x.cuda() for x in c.caches]
    n = c.caches[0].shape[0]
    every = L.Batch(torch.tensor([n], dtype=torch.int32, device="cuda"), n, n)
    k, v = L.idx_cache_read_q4(*caches, every, 2, 80, 80, dtype=torch.float32)
    ref = L.dense_attn(c.q.reshape(6, 8, 80).cuda(), k, v, c.batch(), c.scale)
    assert (out - ref).abs().max() <= 2.0 ** -18 * ref.abs().max()


# --------------------------------------------------------------------------------------------- refusals

def _call(**kw):
    p = ctypes.c_void_p
    a = dict(q=p(16), dtype=L.IDX_BF16, hq=8, hkv=2, dk=64, dv=64, kc=p(16), ks=80, vc=p(16), vs=80, n=16, pos=p(16), T=1, N=16, mods=None,
             scale=1.0, out=p(16), ws=None)
    a.update(kw)
    mods = None if a["mods"] is None else ctypes.byref(L._Mods(**a["mods"]))
    b = L._Batch(1, a["T"], p(16), None, 16, a["pos"], a["N"])
    return L.load().dense_attn_q4(a["q"], a["dtype"], a["hq"], a["hkv"], a["dk"], a["dv"], a["kc"], a["ks"], a["vc"], a["vs"], a["n"], b, mods,
                                  a["scale"], a["out"], None, a["ws"], 0, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(hq=7), dict(hkv=0), dict(dk=0), dict(dk=60), dict(dk=584), dict(dv=0), dict(dv=12), dict(dv=520), dict(ks=79), dict(ks=78),
    dict(vs=60), dict(vs=82), dict(kc=ctypes.c_void_p(18)), dict(n=-1), dict(T=0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=2e38),
    dict(mods=dict(softcap=-1.0)), dict(mods=dict(softcap=math.inf)), dict(mods=dict(softcap=1e-30), scale=1e20), dict(mods=dict(window=-1)),
    dict(mods=dict(window=4), pos=None), dict(mods=dict(slopes=ctypes.c_void_p(16)), pos=None), dict(ws=ctypes.c_void_p(24)), dict(q=None),
    dict(out=None), dict(kc=None), dict(vc=None), dict(N=2 ** 31 - 1)])
def test_refusals(bad):
    a = dict(bad)
    assert _call(**a) in (L.IDX_ERR_INVALID_ARG, L.IDX_ERR_UNSUPPORTED)
    assert b"dense_attn_q4" in L.load().idx_last_error()


def test_workspace_of_nonsense_sizes_is_0():
    good = (torch.bfloat16, 1, 1, 32768, 8, 2, 128, 128)
    for i, x in ((1, 0), (2, 0), (3, 0), (4, 7), (5, 0), (6, 12), (6, 584), (7, 0), (7, 520)):
        a = list(good)
        a[i] = x
        assert L.dense_attn_q4_workspace_size(*a) == 0


def test_the_workspace_is_bounded():
    for n, h in ((1, 1), (64, 8), (2 ** 20, 128), (2 ** 31 - 1, 2 ** 20)):
        assert 0 <= L.dense_attn_q4_workspace_size(torch.bfloat16, n, 4096, 2 ** 31 - 1025, 8 * h, h, 128, 128) <= 2 ** 36 + 16 * n + 16


@pytest.mark.gpu
def test_binding_refuses():
    q, kc = torch.zeros(2, 8, 64, device="cuda", dtype=torch.float16), torch.zeros(16, 80, device="cuda", dtype=torch.uint8)
    b = L.Batch(torch.tensor([8, 8], dtype=torch.int32, device="cuda"), 1, 8, kv_seq_stride=8)
    L.dense_attn_q4(q, kc, kc, b, 1.0, 2)
    for bad in (dict(q=q[:1]), dict(q=q.transpose(0, 1)), dict(k=kc[:8]), dict(k=kc[:, :64]), dict(k=kc.float()), dict(k=kc.cpu()), dict(h=0),
                dict(out=q.float()), dict(lse=torch.zeros(2, 4, device="cuda")), dict(window=2 ** 31), dict(dv=60), dict(dv=0),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda").expand(100, 16)),
                dict(slopes=torch.zeros(7, device="cuda")), dict(b=L.Batch(b.n_kv, 1, 8, q_pos=torch.zeros(1, dtype=torch.int32, device="cuda")))):
        a = {**dict(q=q, k=kc, b=b, h=2), **bad}
        rest = {i: a[i] for i in a if i not in ("q", "k", "b", "h")}
        with pytest.raises(ValueError):
            L.dense_attn_q4(a["q"], a["k"], kc, a["b"], 1.0, a["h"], **rest)
