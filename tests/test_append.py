"""idx_cache_append, idx_cache_append_q4 and idx_cache_read_q4 against 64-bit code, and their refusals.

Tolerances.  u = 2^-24.  An angle is off by pi * 2^-25 (its f32 in half turns) and 2^-51 of p * f (its 64-bit fraction), cosine
and sine by an ulp more, and a column's two products and their sum are rounded: at most 1.25 * 2^-22 + 2^-51 |p f| of the
pair's |a| + |b| in all.  The result is then rounded to the type: half a step (and half of the smallest subnormal).
Codes are exact; scale and minimum are f32 of such columns."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import lightning_indexer_top_gb300 as L

PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
DTYPES = [torch.float32, torch.float16, torch.bfloat16]


def turn(x, pos, freq, start, inter):
    """x f64 [rows, heads, d] turned by pos [rows]; and the pairs' |a| + |b| where a column was turned, 0 elsewhere; angles
    reduced as fractions."""
    y, size = x.clone(), torch.zeros_like(x)
    n = len(freq)
    at = torch.arange(n)
    c0, c1 = (start + 2 * at, start + 2 * at + 1) if inter else (start + at, start + n + at)
    for r, p in enumerate(pos):
        if p < 0:
            continue
        t = torch.tensor([2 * math.pi * float((Fraction(int(p)) * Fraction(float(f)) / (2 * PI)) % 1) for f in freq], dtype=torch.float64)
        a, b = x[r][:, c0], x[r][:, c1]
        y[r][:, c0] = a * t.cos() - b * t.sin()
        y[r][:, c1] = b * t.cos() + a * t.sin()
        size[r][:, c0] = size[r][:, c1] = a.abs() + b.abs()
    return y, size


class Rows:
    """New rows of a batch over contiguous or paged caches."""

    def __init__(self, n_kv, T, hq, hkv, dk, dv, dtype, page=0, n_new=None, n_rot=0, start=0, inter=False, seed=0, apart=True,
                 base=10000.0):
        g = torch.Generator().manual_seed(seed)
        B, N = len(n_kv), max(max(n_kv), 1)
        n_new = [min(T, n) for n in n_kv] if n_new is None else n_new
        self.B, self.T, self.N, self.page, self.inter, self.start, self.n_kv = B, T, N, page, inter, start, n_kv
        self.pos = torch.full((B, T), -1, dtype=torch.int64)
        for b in range(B):
            self.pos[b, :n_new[b]] = torch.arange(n_kv[b] - n_new[b], n_kv[b])
        self.pos = self.pos.view(-1)
        P = -(-N // page) if page else 0
        self.n_rows = B * P * page if page else B * N
        self.table = torch.randperm(B * P, generator=g).view(B, P).to(torch.int32) if page else None
        seq = torch.arange(B).repeat_interleave(T)
        p = self.pos.clamp(min=0)
        self.to = seq * N + p if not page else self.table.long()[seq, p // page] * page + p % page
        # (eight columns more where rows lie apart)
        x = torch.randn(B * T, hq * dk + hkv * (dk + dv) + (8 if apart else 0), generator=g).to(dtype)
        self.proj, self.heads, self.apart = x, ((hq, dk), (hkv, dk), (hkv, dv)), apart
        self.q, self.k, self.v = self.split(x)
        self.freq = (base ** (-torch.arange(0, n_rot, 2).double() / max(n_rot, 1))).float() if n_rot else None
        self.g = g

    def split(self, x):
        """q, k, v (None where there is none) as columns of the projection's output x."""
        parts = x[:, :sum(h * d for h, d in self.heads)].split([h * d for h, d in self.heads], 1)
        return [(t if self.apart else t.contiguous()).unflatten(1, hd) if hd[0] * hd[1] else None for t, hd in zip(parts, self.heads)]

    def gpu(self):
        return self.split(self.proj.cuda())

    def batch(self, **kw):
        i32 = lambda x: x.to("cuda", torch.int32)  # noqa: E731
        a = dict(kv_seq_stride=self.N, q_pos=i32(self.pos), page_table=None if self.table is None else i32(self.table),
                 page_size=self.page)
        return L.Batch(i32(torch.tensor(self.n_kv)), self.T, self.N, **{**a, **kw})

    def rope(self):
        return dict(inv_freq=None if self.freq is None else self.freq.cuda(), rot_start=self.start, interleaved=self.inter)

    def turned(self, x):
        if self.freq is None:
            return x.double(), torch.zeros_like(x, dtype=torch.float64)
        return turn(x.double(), self.pos.tolist(), self.freq.tolist(), self.start, self.inter)

    def error(self, size):
        far = 0.0 if self.freq is None else float(self.pos.max()) * float(self.freq.abs().max()) * 2.0 ** -51
        return size * (1.25 * 2.0 ** -22 + far)

    def close(self, got, want, size, what=""):
        dt = got.dtype
        tol = torch.finfo(dt).eps / 2 * want.abs() * (size > 0) + self.error(size) * 1.01 + TINY[dt] * (size > 0)
        bad = (got.cpu().double() - want).abs() > tol
        assert not bad.any(), (what, int(bad.sum()), float((got.cpu().double() - want).abs().max()))


SHAPES = [  # hq, hkv, dk, dv, n_rot, start, interleaved
    (4, 1, 32, 32, 32, 0, False), (32, 4, 128, 128, 128, 0, False), (32, 8, 128, 128, 64, 64, True), (0, 1, 576, 0, 64, 512, True),
    (14, 2, 64, 64, 32, 0, False), (5, 5, 20, 12, 8, 3, False), (3, 1, 7, 9, 4, 1, True), (2, 2, 96, 40, 0, 0, False),
    (8, 1, 128, 0, 48, 16, False), (1, 1, 2, 1, 2, 0, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("page", [0, 1, 16, 24])
@pytest.mark.parametrize("apart", [True, False])
def test_append(dtype, shape, page, apart):
    hq, hkv, dk, dv, n_rot, start, inter = shape
    c = Rows([300, 7, 41, 64], 9, hq, hkv, dk, dv, dtype, page, [9, 7, 4, 1], n_rot, start, inter, seed=1, apart=apart)
    q, k, v = c.gpu()
    kc = torch.randn(c.n_rows, hkv, dk, generator=c.g).to(dtype).cuda()
    vc = torch.randn(c.n_rows, hkv, dv, generator=c.g).to(dtype).cuda() if dv else None
    before = [None if t is None else t.clone() for t in (q, k, v, kc, vc)]
    out = L.idx_cache_append(k, v, kc, vc, c.batch(), q=q, **c.rope())
    real = c.pos >= 0
    if hq:
        want, size = c.turned(c.q)
        c.close(out, want, size, "q")
        assert torch.equal(out.cpu()[~real], c.q[~real])
    else:
        assert out is None
    want, size = c.turned(c.k)
    c.close(kc[c.to[real]], want[real], size[real], "k")
    if dv:
        assert torch.equal(vc.cpu()[c.to[real]], c.v[real])
    others = torch.ones(c.n_rows, dtype=torch.bool)
    others[c.to[real]] = False
    for t, b in ((kc, before[3]), (vc, before[4])):
        assert t is None or torch.equal(t.cpu()[others], b.cpu()[others])
    for t, b in zip((q, k, v), before):
        assert t is None or torch.equal(t, b)
    if hq:      # in place
        L.idx_cache_append(k, v, kc, vc, c.batch(), q=q, q_out=q, **c.rope())
        assert torch.equal(q, out)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("p", [0, 1, 65535, 1048577, 16777217, 2 ** 31 - 1025])
def test_far_positions(p):
    # the cache row of position p is row 1: the sequence starts at a negative row
    c = Rows([3], 1, 2, 1, 64, 64, torch.float32, 0, [1], 64)
    c.pos = torch.tensor([p])
    kc, vc = torch.zeros(3, 1, 64, device="cuda"), torch.zeros(3, 1, 64, device="cuda")
    b = L.Batch(torch.tensor([p + 1], dtype=torch.int32, device="cuda"), 1, p + 1,
                kv_start=torch.tensor([1 - p], dtype=torch.int32, device="cuda"), q_pos=c.pos.to("cuda", torch.int32))
    q, k, v = c.gpu()
    out = L.idx_cache_append(k, v, kc, vc, b, q=q, **c.rope())
    for got, x in ((out, c.q), (kc[1:2], c.k)):
        want, size = c.turned(x)
        c.close(got, want, size, p)
    assert (kc[[0, 2]] == 0).all() and L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("base", [1e6, 5e8, 1e20])
@pytest.mark.parametrize("p", [1, 65535, 16777217, 2 ** 31 - 1025])
def test_low_frequencies_at_far_positions(base, p):
    # each pair by itself: f32's part, and the phase's 2^-63 of a turn times the position, whatever the pair's frequency
    c = Rows([3], 1, 2, 1, 128, 64, torch.float32, 0, [1], 128, base=base)
    c.pos = torch.tensor([p])
    kc, vc = torch.zeros(3, 1, 128, device="cuda"), torch.zeros(3, 1, 64, device="cuda")
    b = L.Batch(torch.tensor([p + 1], dtype=torch.int32, device="cuda"), 1, p + 1,
                kv_start=torch.tensor([1 - p], dtype=torch.int32, device="cuda"), q_pos=c.pos.to("cuda", torch.int32))
    q, k, v = c.gpu()
    out = L.idx_cache_append(k, v, kc, vc, b, q=q, **c.rope())
    for got, x in ((out, c.q), (kc[1:2], c.k)):
        want, size = c.turned(x)
        tol = size * (1.25 * 2.0 ** -22 + 2 * math.pi * p * 2.0 ** -63) + 2.0 ** -24 * want.abs()
        assert ((got.cpu().double() - want).abs() <= tol).all()


@pytest.mark.gpu
def test_frequencies_of_any_sign_and_size():
    c = Rows([40], 7, 1, 1, 16, 16, torch.float32, 0, None, 16)
    c.freq = torch.tensor([-1.0, 3.5, -100.25, 1e-20, 0.0, 6.2831855, 1e4, -1e-3])
    kc, vc = torch.zeros(40, 1, 16, device="cuda"), torch.zeros(40, 1, 16, device="cuda")
    q, k, v = c.gpu()
    out = L.idx_cache_append(k, v, kc, vc, c.batch(), q=q, **c.rope())
    want, size = c.turned(c.q)
    c.close(out, want, size)


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_rows_without_positions_are_the_last_ones(four):
    c = Rows([50, 2, 9], 3, 4, 2, 64, 64, torch.bfloat16, 16, [3, 2, 3], 64, seed=2)
    c.pos = torch.tensor([47, 48, 49, -1, 0, 1, 6, 7, 8])      # n_kv - T + t, negative ones are padding
    p = c.pos.clamp(min=0)
    c.to = c.table.long()[torch.arange(3).repeat_interleave(3), p // 16] * 16 + p % 16
    q, k, v = c.gpu()
    w = L.idx_q4_row_bytes(2, 64)
    caches = [torch.zeros(c.n_rows, w, dtype=torch.uint8, device="cuda") if four else
              torch.zeros(c.n_rows, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    call = L.idx_cache_append_q4 if four else L.idx_cache_append
    a = call(k, v, *caches[:2], c.batch(), q=q, **c.rope())
    b = call(k, v, *caches[2:], c.batch(q_pos=None), q=q, **c.rope())
    assert torch.equal(a, b) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    if four:
        x, y = (L.idx_cache_read_q4(*caches[:2], bb, 2, 64, 64) for bb in (c.batch(), c.batch(q_pos=None)))
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_rows_out_of_range_are_flagged_and_not_written(four):
    c = Rows([20, 20], 2, 0, 1, 16, 16, torch.float16, 4, None)
    c.table[0, 4] = -1                       # positions 16 .. 19
    c.table[1, 4] = c.n_rows // 4            # one page past the cache
    _, k, v = c.gpu()
    shape = (c.n_rows, L.idx_q4_row_bytes(1, 16)) if four else (c.n_rows, 1, 16)
    kc, vc = (torch.zeros(shape, dtype=torch.uint8 if four else torch.float16, device="cuda") for _ in range(2))
    call = L.idx_cache_append_q4 if four else L.idx_cache_append
    call(k, v, kc, vc, c.batch())
    assert (kc == 0).all() and (vc == 0).all() and L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS
    c.table[0, 4], c.table[1, 4] = 0, 1
    c.pos = torch.tensor([20, 18, 19, 21])   # at and past n_kv
    call(k, v, kc, vc, c.batch())
    assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS
    written = torch.zeros(c.n_rows, dtype=torch.bool)
    written[[2, 4 + 3]] = True
    assert ((kc != 0).flatten(1).any(1).cpu() == written).all()
    if four:
        out = torch.full((4, 1, 16), 5.0, dtype=torch.float16, device="cuda")
        L.idx_cache_read_q4(kc, vc, c.batch(), 1, 16, 16, k_out=out)
        assert (out[[0, 3]] == 5).all() and (out[[1, 2]] != 5).any() and L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS


def parts(cache, heads, d):
    """codes, scale, minimum of a 4-bit cache on the host."""
    c = cache.cpu()
    b = c[:, :heads * d // 2].reshape(-1, heads, d // 2)
    codes = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    f = torch.from_numpy(np.ascontiguousarray(c[:, heads * d // 2:heads * (d // 2 + 8)].numpy()).view(np.float32).copy()).view(-1, heads, 2)
    return codes, f[..., 0], f[..., 1]


def codes_of(y):
    lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
    return torch.where(hi > lo, (y - lo) * 15 / torch.where(hi > lo, hi - lo, 1.0), 0.0).round(), ((hi - lo) / 15)[..., 0], lo[..., 0]


SHAPES4 = [(4, 1, 32, 32, 32, 0, False), (32, 4, 128, 128, 128, 0, False), (8, 8, 128, 128, 64, 64, True), (0, 1, 576, 0, 64, 512, True),
           (14, 2, 64, 64, 32, 0, False), (5, 5, 24, 8, 10, 3, False), (2, 2, 96, 40, 0, 0, False), (4, 2, 80, 256, 80, 0, True)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES4)
@pytest.mark.parametrize("page,pad", [(0, 0), (16, 4), (24, 16)])
def test_append_q4(dtype, shape, page, pad):
    hq, hkv, dk, dv, n_rot, start, inter = shape
    c = Rows([700, 100, 41, 640], 90, hq, hkv, dk, dv, dtype, page, [90, 77, 40, 1], n_rot, start, inter, seed=3)
    q, k, v = c.gpu()
    kc = torch.randint(0, 256, (c.n_rows, L.idx_q4_row_bytes(hkv, dk) + pad), generator=c.g, dtype=torch.uint8).cuda()
    vc = torch.randint(0, 256, (c.n_rows, L.idx_q4_row_bytes(hkv, dv) + pad), generator=c.g, dtype=torch.uint8).cuda() if dv else None
    before = [kc.clone(), None if vc is None else vc.clone()]
    out = L.idx_cache_append_q4(k, v, kc, vc, c.batch(), q=q, **c.rope())
    real = c.pos >= 0
    if hq:
        want, size = c.turned(c.q)
        c.close(out, want, size, "q")
    read = L.idx_cache_read_q4(kc, vc, c.batch(), hkv, dk, dv, dtype=torch.float32)
    for cache, was, x, d, got in ((kc, before[0], c.k, dk, read[0]), (vc, before[1], c.v, dv, read[1])):
        if cache is None:
            assert got is None
            continue
        y, size = c.turned(x) if cache is kc else (x.double(), torch.zeros(x.shape, dtype=torch.float64))
        want, scale, low = codes_of(y[real])
        codes, s, m = (t[c.to[real]] for t in parts(cache, hkv, d))
        assert torch.equal(codes.double(), want)
        off = c.error(size[real].amax(-1)) * 1.01
        assert ((s.double() - scale).abs() <= 2 * off / 15 + 2.0 ** -23 * scale).all()
        assert ((m.double() - low).abs() <= off + 2.0 ** -24 * low.abs()).all()
        # nothing else is written: other rows, and the bytes past a row's payload
        others = torch.ones(c.n_rows, dtype=torch.bool)
        others[c.to[real]] = False
        assert torch.equal(cache.cpu()[others], was.cpu()[others])
        assert torch.equal(cache[:, hkv * (d // 2 + 8):], was[:, hkv * (d // 2 + 8):])
        # and back: one f32 rounding
        value = codes.double() * s.double()[..., None] + m.double()[..., None]
        got = got.cpu()
        assert ((got[real].double() - value).abs() <= 2.0 ** -24 * value.abs()).all() and (got[~real] == 0).all()
        if dtype != torch.float32:
            rounded = L.idx_cache_read_q4(kc, vc, c.batch(), hkv, dk, dv, dtype=dtype)[0 if cache is kc else 1]
            assert torch.equal(rounded.cpu(), got.to(dtype))
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_q4_of_rows_that_f32_cannot_tell_apart():
    # half-way values (ties go to the even code), equal columns, tiny and huge spans, a large offset, and no numbers
    base = torch.tensor([0.0, 15.0, 0.5, 1.5, 2.5, 6.5, 7.5, 13.5], dtype=torch.float64)
    rows = [base, base * 2 ** -20 + 1, base * 2.0 ** -140, base * 2.0 ** 123, torch.full((8,), 3.0), torch.zeros(8),
            -base, torch.tensor([1e30, 1e30, 1e30, -1e30, 1, 2, 3, 4.0]), torch.tensor([3e38, -3e38, 0, 1, 2, 1e38, -1e38, 2e38]),
            torch.tensor([0.0, -0.0, 0.0, 0.0, 0.0, 0.0, 0.0, -0.0])]
    x = torch.stack([r.double() for r in rows]).float()
    nan = [x[0].clone() for _ in range(3)]
    nan[0][3], nan[1][0], nan[2][7] = math.nan, math.inf, -math.inf
    x = torch.cat([x, torch.stack(nan)])[:, None]
    n = x.shape[0]
    w = L.idx_q4_row_bytes(1, 8)
    for freq in (None, torch.zeros(4, device="cuda")):       # a rotation by nothing
        kc, vc = (torch.zeros(n, w, dtype=torch.uint8, device="cuda") for _ in range(2))
        b = L.Batch(torch.tensor([n], dtype=torch.int32, device="cuda"), n, n)
        L.idx_cache_append_q4(x.cuda(), x.cuda(), kc, vc, b, inv_freq=freq)
        for cache in (kc, vc):
            codes, s, m = parts(cache, 1, 8)
            want, scale, low = codes_of(x[:-3].double())
            assert torch.equal(codes[:-3].double(), want)
            assert torch.equal(codes[-3:], torch.zeros_like(codes[-3:])) and torch.isnan(s[-3:]).all() and torch.isnan(m[-3:]).all()
            assert ((s[:-3].double() - scale).abs() <= 2.0 ** -22 * scale + 2.0 ** -150).all() and torch.equal(m[:-3].double(), low)
        k, v = L.idx_cache_read_q4(kc, vc, b, 1, 8, 8, dtype=torch.float32)
        assert torch.isnan(k[-3:]).all() and torch.isfinite(k[:-3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,n_rot,start,inter", [
    (16, 0, 0, False), (16, 16, 0, False), (64, 32, 0, False), (64, 64, 0, True), (80, 80, 0, False), (80, 16, 8, True), (96, 0, 0, False),
    (128, 128, 0, False), (128, 64, 64, True), (512, 64, 448, False), (576, 64, 512, False), (24, 10, 3, False)])
def test_q4_rows_without_a_number_stand_for_nan_and_leave_the_others(dtype, d, n_rot, start, inter):
    # a NaN or an infinity first, in the middle and last, and rows of nothing else, between rows of numbers (which share their warp)
    values, n, h, dv = [math.nan, math.inf, -math.inf], 24, 3, min(d, 512)
    c = Rows([n], n, 0, h, d, dv, dtype, 0, None, n_rot, start, inter, seed=8, apart=False)
    bad = torch.zeros(n, h, dtype=torch.bool)
    rows = [(v, at) for v in values for at in ([0], [-1], [d // 2], slice(None))]
    c.k, c.v = c.k.clone(), c.v.clone()
    good = [t.clone() for t in (c.k, c.v)]
    for i, (value, at) in enumerate(rows):
        bad[2 * i, i % h] = True
        c.k[2 * i, i % h, at] = value
        c.v[2 * i, i % h, at if at != [d // 2] else dv // 2] = value
    new = lambda w: torch.zeros(n, L.idx_q4_row_bytes(h, w), dtype=torch.uint8, device="cuda")  # noqa: E731
    got, want = (new(d), new(dv)), (new(d), new(dv))
    L.idx_cache_append_q4(c.k.cuda(), c.v.cuda(), *got, c.batch(), **c.rope())
    L.idx_cache_append_q4(*[t.cuda() for t in good], *want, c.batch(), **c.rope())
    for a, b, w in zip(got, want, (d, dv)):
        codes, s, m = parts(a, h, w)
        assert torch.isnan(s[bad]).all() and torch.isnan(m[bad]).all() and (codes[bad] == 0).all()
        for x, y in zip((codes, s, m), parts(b, h, w)):
            assert torch.equal(x[~bad], y[~bad]) and torch.isfinite(x[~bad].float()).all()
    k, v = L.idx_cache_read_q4(*got, c.batch(), h, d, dv, dtype=torch.float32)
    for t in (k, v):
        assert torch.isnan(t[bad.cuda()]).all() and torch.isfinite(t[~bad.cuda()]).all()
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("four", [False, True])
def test_caches_beyond_32_bit_offsets(four):
    # rows that lie more than 2^32 bytes behind the caches' first
    c = Rows([300, 41], 60, 4, 8, 128, 128, torch.bfloat16, 16, [60, 41], 128, seed=9)
    w = L.idx_q4_row_bytes(8, 128)
    shape, size, dt = ((w,), w, torch.uint8) if four else ((8, 128), 2048, torch.bfloat16)
    n = (2 ** 32 // size + 4096) // 16 * 16
    big, small = ([torch.zeros(k, *shape, dtype=dt, device="cuda") for _ in range(2)] for k in (n, c.n_rows))
    call = L.idx_cache_append_q4 if four else L.idx_cache_append
    q, k, v = c.gpu()
    a = call(k, v, *small, c.batch(), q=q, **c.rope())
    far = c.batch(page_table=(c.table + (n - c.n_rows) // 16).cuda())
    b = call(k, v, *big, far, q=q, **c.rope())
    assert torch.equal(a, b)
    for x, y in zip(big, small):
        assert torch.equal(x[n - c.n_rows:], y) and not x[:4096].any()
    if four:
        x, y = (L.idx_cache_read_q4(*t, bb, 8, 128, 128) for t, bb in ((big, far), (small, c.batch())))
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_many_rows_have_exact_codes():
    # half a million columns, some of which lie within f32's error of a border
    c = Rows([2048], 2048, 0, 2, 128, 128, torch.bfloat16, 0, None, 128, seed=5, base=1e6)
    _, k, v = c.gpu()
    w = L.idx_q4_row_bytes(2, 128)
    kc, vc = (torch.zeros(2048, w, dtype=torch.uint8, device="cuda") for _ in range(2))
    L.idx_cache_append_q4(k, v, kc, vc, c.batch(), **c.rope())
    y, _ = c.turned(c.k)
    assert torch.equal(parts(kc, 2, 128)[0].double(), codes_of(y)[0])
    assert torch.equal(parts(vc, 2, 128)[0].double(), codes_of(c.v.double())[0])


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    c = Rows([64, 30], 1, 8, 2, 64, 64, torch.float16, 16, None, 64, seed=6)
    q, k, v = c.gpu()
    w = L.idx_q4_row_bytes(2, 64)
    fresh = lambda: [torch.zeros(c.n_rows, 2, 64, dtype=torch.float16, device="cuda"), torch.zeros(c.n_rows, 2, 64, dtype=torch.float16, device="cuda"),  # noqa: E731
                     torch.zeros(c.n_rows, w, dtype=torch.uint8, device="cuda"), torch.zeros(c.n_rows, w, dtype=torch.uint8, device="cuda")]
    b, rope = c.batch(), c.rope()

    def step(t, out):
        L.idx_cache_append(k, v, t[0], t[1], b, q=q, q_out=out, **rope)
        L.idx_cache_append_q4(k, v, t[2], t[3], b, q=q, q_out=out, **rope)
    want, o0 = fresh(), torch.empty(2, 8, 64, dtype=torch.float16, device="cuda")
    step(want, o0)
    got, o1 = fresh(), torch.empty_like(o0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(got, o1)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(x, y) for x, y in zip(want + [o0], got + [o1]))
    for t in got:
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got, o1)
    # the next step's positions and rows, read by the replay
    b.q_pos.sub_(1)
    k.neg_()
    graph.replay()
    want = fresh()
    step(want, o0)
    assert all(torch.equal(x, y) for x, y in zip(want + [o0], got + [o1]))


# --------------------------------------------------------------------------------------------- refusals

def _c_args(**kw):
    p = lambda x: ctypes.c_void_p(x)  # noqa: E731
    a = dict(rows=dict(k=p(4096), k_stride=64, v=p(4096), v_stride=64, q=None, q_stride=0, q_out=None, q_out_stride=0), dtype=L.IDX_F16,
             hq=0, hkv=1, dk=64, dv=64, T=1, rope=None, kc=p(4096), ks=64, vc=p(4096), vs=64, n=16)
    rows = {**a["rows"], **kw.pop("rows", {})}
    a.update(kw)
    return [ctypes.byref(L._NewRows(**rows)), a["dtype"], a["hq"], a["hkv"], a["dk"], a["dv"],
            L._Batch(1, a["T"], p(16), None, 16, None, 16), None if a["rope"] is None else ctypes.byref(L._Rope(*a["rope"])), a["kc"],
            a["ks"], a["vc"], a["vs"], a["n"], None]


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("bad,word", [
    (dict(dtype=5), b"dtype"), (dict(hkv=0), b"heads"), (dict(hq=-1), b"heads"), (dict(dk=0), b"dk"), (dict(dk=584), b"dk"), (dict(dv=-1), b"dv"),
    (dict(dv=0), b"need dv"), (dict(dv=520), b"dv"), (dict(T=0), b"n_q_per_seq"), (dict(n=-1), b"kv_rows"), (dict(rope=(16, 3, 0, 0)), b"n_rot"),
    (dict(rope=(16, -2, 0, 0)), b"n_rot"), (dict(rope=(16, 64, 2, 0)), b"n_rot"), (dict(rope=(16, 32, -1, 0)), b"n_rot"),
    (dict(rope=(None, 32, 0, 0)), b"inv_freq"), (dict(rope=(16, 66, 0, 0)), b"n_rot"),
    (dict(rows=dict(k_stride=63)), b"stride"), (dict(rows=dict(v_stride=63)), b"stride"), (dict(rows=dict(k=None)), b"NULL"),
    (dict(rows=dict(v=None)), b"NULL"), (dict(hq=2), b"stride"), (dict(hq=2, rows=dict(q_stride=128, q_out_stride=128)), b"NULL"),
    (dict(hq=2, rows=dict(q=16, q_out=16, q_stride=128, q_out_stride=130)), b"in place"),
    (dict(kc=None), b"NULL"), (dict(vc=None), b"NULL"), (dict(ks=10), b"stride"), (dict(vs=10), b"stride"), (dict(hkv=2 ** 30), b"wide")])
def test_refusals(four, bad, word):
    lib = L.load()
    fn = lib.idx_cache_append_q4 if four else lib.idx_cache_append
    wide = {"hkv": 2 ** 30}
    good = {} if bad != wide else dict(rows=dict(k_stride=2 ** 40, v_stride=2 ** 40), ks=2 ** 40, vs=2 ** 40)
    assert fn(*_c_args(**{**good, **bad})) in (L.IDX_ERR_INVALID_ARG, L.IDX_ERR_UNSUPPORTED)
    assert word in lib.idx_last_error()


def test_refusals_of_4_bit_rows():
    lib = L.load()
    for bad in (dict(dk=60), dict(dv=60), dict(ks=39), dict(ks=42), dict(vs=41), dict(kc=ctypes.c_void_p(4098))):
        a = {**dict(ks=40, vs=40), **bad}
        assert lib.idx_cache_append_q4(*_c_args(**a)) == L.IDX_ERR_INVALID_ARG, bad
    p = ctypes.c_void_p
    read = lambda **k: lib.idx_cache_read_q4(*[{**dict(kc=p(16), ks=40, vc=p(16), vs=40, n=4, h=1, dk=64, dv=64, b=L._Batch(  # noqa: E731
        1, 1, p(16), None, 16, None, 16), dt=L.IDX_F16, ko=p(16), vo=p(16), st=None), **k}[x] for x in
        ("kc", "ks", "vc", "vs", "n", "h", "dk", "dv", "b", "dt", "ko", "vo", "st")])
    for bad in (dict(dt=9), dict(h=0), dict(dk=0), dict(dk=65), dict(dv=0), dict(n=-1), dict(ks=38), dict(vs=36), dict(ko=None), dict(vo=None),
                dict(ko=p(24)), dict(kc=None), dict(vc=None), dict(kc=p(18))):
        assert read(**bad) == L.IDX_ERR_INVALID_ARG, bad
    assert L.idx_q4_row_bytes(4, 128) == 288 and L.idx_q4_row_bytes(1, 8) == 16 and L.idx_q4_row_bytes(3, 64) == 128
    for n, d in ((0, 8), (1, 0), (1, 12), (-1, 8)):
        with pytest.raises(ValueError):
            L.idx_q4_row_bytes(n, d)


def test_nothing_to_do_launches_nothing():
    lib = L.load()
    a = _c_args()
    a[6] = L._Batch(0, 1, None, None, 16, None, 16)
    assert lib.idx_cache_append(*a) == L.IDX_OK


@pytest.mark.gpu
def test_binding_refuses():
    x = lambda *s, **k: torch.zeros(*s, device="cuda", dtype=k.get("dtype", torch.float16))  # noqa: E731
    n_kv = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    b = L.Batch(n_kv, 2, 4, kv_seq_stride=4)
    k, v, kc, vc = x(4, 2, 64), x(4, 2, 64), x(8, 2, 64), x(8, 2, 64)
    f = torch.zeros(32, device="cuda")
    ok = lambda **a: L.idx_cache_append(*[{**dict(k=k, v=v, kc=kc, vc=vc, b=b), **a}[i] for i in ("k", "v", "kc", "vc", "b")],  # noqa: E731
                                        **{i: a[i] for i in a if i in ("q", "q_out", "inv_freq", "rot_start")})
    ok(inv_freq=f)
    for bad in (dict(k=x(3, 2, 64)), dict(k=x(4, 128)), dict(v=None), dict(vc=None), dict(v=x(4, 1, 64)), dict(v=x(4, 2, 64, dtype=torch.float32)),
                dict(kc=x(8, 2, 32)), dict(kc=x(8, 2, 64, dtype=torch.bfloat16)), dict(kc=x(6, 2, 64)), dict(kc=x(8, 64, 2).transpose(1, 2)),
                dict(k=x(4, 2, 128)[..., ::2]), dict(k=x(1, 2, 64).expand(4, 2, 64)), dict(q=x(4, 3, 32)), dict(q_out=x(4, 3, 64)),
                dict(q=x(4, 3, 64), q_out=x(4, 2, 64)), dict(inv_freq=f.double()), dict(inv_freq=f[::2]), dict(k=k.cpu()), dict(v=v.cpu()),
                dict(inv_freq=f, rot_start=2 ** 32), dict(inv_freq=f, rot_start=-1),
                dict(b=L.Batch(n_kv, 2, 4, kv_start=torch.zeros(1, dtype=torch.int32, device="cuda"))),
                dict(b=L.Batch(n_kv, 2, 4, q_pos=torch.zeros(3, dtype=torch.int32, device="cuda")))):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(L.LidxError):
        ok(inv_freq=f, rot_start=1)
    w = L.idx_q4_row_bytes(2, 64)
    for bad in (x(8, w - 16, dtype=torch.uint8), x(8, w), x(8, w, 1, dtype=torch.uint8), x(w, 8, dtype=torch.uint8).T,
                x(1, w, dtype=torch.uint8).expand(8, w), x(7, w, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            L.idx_cache_append_q4(k, v, bad, x(8, w, dtype=torch.uint8), b)
        with pytest.raises(ValueError):
            L.idx_cache_read_q4(bad, x(8, w, dtype=torch.uint8), b, 2, 64, 64)
