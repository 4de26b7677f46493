"""dense_attn at widths, caps and masks where its kernels' limits lie; tolerances as in test_dense_attn.py."""

import ctypes
import math

import pytest
import torch

import lightning_indexer_top_gb300 as L
from test_dense_attn import DTYPES, Case, intervals

# dk, dv of K and V apart / of a latent; every one with two to eight key splits that a cluster merges.  Narrow keys
# beside wide values, and latents just past a step of the value width: the merged rows are longer than Q, K, V and the
# scores, or nearly so.
NARROW = [(1, 128), (4, 128), (8, 128), (12, 126), (13, 128), (4, 65)]
NARROW_LATENT = [(1, 1), (8, 8), (16, 16), (20, 20), (12, 5), (129, 129), (136, 136), (140, 140), (144, 130), (144, 144)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", NARROW)
def test_merged_rows_of_narrow_keys(dtype, dk, dv):
    for T, n_kv in ((5, [256, 90]), (1, [200]), (9, [64, 40, 60])):
        c = Case(n_kv, T, 8, 1, dk, dv=dv, dtype=dtype, page=16, seed=41)
        c.check(*c.run(), what=(T, n_kv))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv", NARROW_LATENT)
def test_merged_rows_of_narrow_latents(dtype, dk, dv):
    for T, Hq, n_kv in ((1, 16, [256, 90]), (5, 8, [200, 33]), (3, 5, [64])):
        c = Case(n_kv, T, Hq, 1, dk, dv=dv, dtype=dtype, latent=True, seed=42)
        c.check(*c.run(), what=(T, Hq, n_kv))
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dk,dv,latent", [(576, 128, False), (576, 64, False), (529, 128, False), (528, 128, False),
                                          (549, 64, False), (576, 128, True), (573, 40, True), (576, 512, False)])
def test_wide_keys_of_many_rows(dtype, dk, dv, latent):
    # 64 rows of keys this wide are more than a CTA's shared memory holds
    for T, Hq in ((5, 8), (17, 1)):
        c = Case([150, 33], T, Hq, 1, dk, dv=dv, dtype=dtype, page=16, latent=latent, seed=43)
        c.check(*c.run(), what=(T, Hq))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("cap", [1e-40, 1e-30, 1e-7, 1e-5, 1e-4, 1e-2])
def test_small_caps(dtype, d, cap):
    # every score is within the cap of 0, to which a product of exactly 0 belongs beside large ones
    c = Case([150, 40], 3, 128 if d == 576 else 4, 1, d, dv=min(d, 512), dtype=dtype, latent=d == 576, cap=cap, seed=44)
    c.scale = 1.0 if cap > 1e-38 else 1e-3      # (scale / softcap has to be finite)
    c.q[0, 1] = 0
    for r in c.rows:
        c.k[r[3:20]] = 0
    c.v = c.k[..., :c.dv] if c.latent else c.v
    c.check(*c.run(), what=cap)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("d", [64, 128, 576])
@pytest.mark.parametrize("top", [0.14, 0.29, 0.9, 1e-3])
def test_large_caps(dtype, T, d, top):
    # one key, query rows that are multiples of basis vectors: lse is the score, up to `top` of a cap of millions.
    # tanh by its series is off by 2^-24 of the score and the roundings of its dozen operations, by the exponential
    # within a few of them of the cap, which is below 1 / top of the score
    Hq = 128 if d == 576 else 8
    c = Case([1], T, Hq, 1, d, dv=min(d, 512), dtype=dtype, latent=d == 576, causal=False, seed=45)
    c.scale = 1.0
    c.k[0, 0] = (torch.arange(1, d + 1) * (2.0 ** 15 / d)).to(dtype)
    at = (torch.arange(T * Hq) * 7 + d - 1) % d
    c.q = (torch.nn.functional.one_hot(at, d) * 256).to(dtype).view(1, T, Hq, d)
    c.v = c.k[..., :c.dv] if c.latent else c.v
    c.cap = float((c.k[0, 0].double().max() * 256 / top).float())
    out, lse = c.run()
    x = c.k[0, 0].double()[at] * 256
    want = c.cap * torch.tanh(x / c.cap)
    tol = 2.0 ** -20 * want + (2.0 ** -20 * c.cap if top > 0.3 else 0.0)
    assert ((lse.view(-1).cpu().double() - want).abs() <= tol).all()
    assert torch.equal(out.view(T * Hq, -1).cpu(), c.v[0, 0].expand(T * Hq, c.dv))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,heads", [(200, (4, 2, 128)), (70, (3, 3, 64)), (1, (8, 1, 128)), (9, (128, 1, 576))])
@pytest.mark.parametrize("window", [0, 50])
def test_packed_documents_with_prefixes(dtype, T, heads, window):
    # rows i, keys j of one sequence: j is seen if it is of i's document, and no later than i or in the document's prefix
    n_kv = [200, 133, 64 if T <= 64 else T]
    c = Case(n_kv, T, *heads, dv=min(heads[2], 512), dtype=dtype, page=16, n_new=[T, min(T, 100), T], latent=heads[2] == 576,
             seed=46)
    g = torch.Generator().manual_seed(7)
    seen = torch.zeros(c.B, T, c.N, dtype=torch.bool)
    start, end = torch.zeros(c.B, T, dtype=torch.int32), torch.zeros(c.B, T, dtype=torch.int32)
    for b, n in enumerate(n_kv):
        doc = (torch.rand(n, generator=g) < 0.03).cumsum(0)
        first = torch.searchsorted(doc, doc)
        length = torch.bincount(doc)[doc]
        prefix = (torch.rand(int(doc[-1]) + 1, generator=g)[doc] * (length + 1)).long()     # none of it to all of it
        j = torch.arange(n)
        for t in range(T):
            i = int(c.pos[b, t])
            if i < 0:
                continue
            seen[b, t, :n] = (doc == doc[i]) & ((j <= i) | (j - first[i] < prefix[i]))
            if window:
                seen[b, t, :n] &= j > i - window
            start[b, t], end[b, t] = first[i], first[i] + prefix[i]
    some = seen.any(-1)
    c.lo = torch.where(some, seen.long().argmax(-1), 0)
    c.hi = torch.where(some, c.N - seen.flip(-1).long().argmax(-1), 0)
    assert torch.equal(seen.sum(-1), c.hi - c.lo) and (T == 1 or (c.hi > c.pos + 1).any())
    q = c.q.reshape(c.B * T, *c.q.shape[2:]).cuda()
    lse = torch.empty(q.shape[:2], device="cuda")
    out = L.dense_attn(q, c.k.cuda(), None if c.latent else c.v.cuda(), c.batch(), c.scale, dv=c.dv, lse=lse, window=window,
                       doc_start=start.cuda().view(-1), prefix_end=end.cuda().view(-1))
    c.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("heads", [(4, 2, 128), (8, 1, 40), (128, 1, 576)])
def test_pages_that_no_row_sees_may_be_gone(dtype, heads):
    # rows at far apart positions under a window: the pages between are not in the cache, and nothing says so
    c = Case([400], 3, *heads, dv=min(heads[2], 512), dtype=dtype, page=16, n_new=[3], window=20, latent=heads[2] == 576,
             seed=48)
    c.pos = torch.tensor([[30, 200, 399]])
    c.lo, c.hi = intervals(c.n_kv, c.pos, window=20)
    for gone in (-1, 1 << 20):
        used = {j // 16 for t in range(3) for j in range(int(c.lo[0, t]), int(c.hi[0, t]))}
        for p in range(c.table.shape[1]):
            if p not in used:
                c.table[0, p] = gone
        c.check(*c.run(), what=gone)
        assert L.idx_device_status(reset=True) == 0
    c.table[0, 199 // 16] = -1
    c.run()
    assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS


@pytest.mark.gpu
def test_the_further_of_two_prefixes():
    c = Case([150, 90], 20, 4, 2, 64, dtype=torch.bfloat16, prefix=[140, 20], seed=47)
    ends = torch.arange(40, dtype=torch.int32).view(2, 20) * 9 - 30
    c.hi = torch.minimum(torch.maximum(c.hi, ends.long()), torch.tensor(c.n_kv)[:, None])
    c.check(*c.run(prefix_end=ends.cuda().view(-1)))


def _call(scale, softcap):
    m = L._Mods(softcap, None, 0, None, None)
    one = ctypes.c_void_p(16)
    b = L._Batch(1, 1, one, None, 8, None, 8, None, 0, 0)
    return L.load().dense_attn(one, 1, 1, 1, 64, 64, one, one, 64, 64, 8, b, m, scale, one, None, None, 0, None)


@pytest.mark.parametrize("scale,softcap,word", [(3e38, 0.0, "scale"), (-3e38, 0.0, "scale"), (math.inf, 0.0, "scale"),
                                                (1.0, 3e38, "softcap"), (1.0, math.nan, "softcap")])
def test_scales_and_caps_beyond_the_kernels_range_are_refused(scale, softcap, word):
    assert _call(scale, softcap) == L.IDX_ERR_INVALID_ARG
    assert word in L.load().idx_last_error().decode()


def test_a_prefix_by_row_needs_positions():
    one = ctypes.c_void_p(16)
    m = L._Mods(prefix_end=16)
    b = L._Batch(1, 1, one, None, 8, None, 8, None, 0, 0)
    st = L.load().dense_attn(one, 1, 1, 1, 64, 64, one, one, 64, 64, 8, b, m, 1.0, one, None, None, 0, None)
    assert st == L.IDX_ERR_INVALID_ARG and "q_pos" in L.load().idx_last_error().decode()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,heads,T,page", [(torch.bfloat16, (4, 2, 128), 1, 64), (torch.float16, (8, 2, 64), 70, 32),
                                                (torch.bfloat16, (128, 1, 576), 2, 64), (torch.float32, (4, 2, 128), 3, 16),
                                                (torch.bfloat16, (4, 2, 40), 3, 0)])
def test_rows_beyond_32_bit_offsets(dtype, heads, T, page):
    # a cache of more than 2^31 elements, the sequences' rows at its two ends
    Hq, Hkv, d = heads
    rows = ((1 << 31) // (Hkv * d) + 4096) // 64 * 64
    c = Case([200, 150], T, Hq, Hkv, d, dv=min(d, 512), dtype=dtype, page=page, latent=d == 576, seed=49)
    b = c.batch()
    if page:
        far = c.table.long() + torch.where(c.table >= c.table.numel() // 2, rows // page - c.table.numel(), 0)
        b.page_table = far.to(torch.int32).cuda()
        at = (far[:, torch.arange(c.N) // page] * page + torch.arange(c.N) % page)
    else:
        b.kv_start = torch.tensor([0, rows - 150], dtype=torch.int32, device="cuda")
        at = torch.arange(c.N) + b.kv_start.cpu().long()[:, None]

    def spread(x):
        big = torch.empty((rows, *x.shape[1:]), dtype=dtype, device="cuda")
        for i, n in enumerate(c.n_kv):
            big[at[i, :n].cuda()] = x[c.rows[i]].cuda()
        return big
    k = spread(c.k)
    assert k.numel() > 1 << 31 and max(int(at[i, :n].max()) for i, n in enumerate(c.n_kv)) > rows - 4096
    v = None if c.latent else spread(c.v)
    q = c.q.reshape(c.B * T, Hq, d).cuda()
    lse = torch.empty(q.shape[:2], device="cuda")
    out = L.dense_attn(q, k, v, b, c.scale, dv=c.dv, lse=lse)
    c.check(out, lse)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_long_latent_in_a_workspace_of_too_few_splits():
    # a unit of the tensor-core kernel takes 8192 keys: 20000 of them need three splits, and with room for fewer the call
    # runs on the CUDA cores, in as many splits as the room holds
    c = Case([20000, 900], 1, 128, 1, 576, dv=512, dtype=torch.bfloat16, page=64, latent=True, seed=50)
    split = 2 * 128 * (512 + 2) * 4
    for n in (3, 2, 1):
        c.check(*c.run(workspace=torch.empty(n * split, dtype=torch.uint8, device="cuda")), what=n)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_calls_on_several_streams_at_once():
    # every kernel and way of merging, each on a stream of its own with its own workspace, against the calls one by one
    cases = [Case([900, 300], 1, 32, 4, 128, page=64, seed=51), Case([700, 500], 200, 8, 2, 128, seed=52),
             Case([300] * 8, 60, 6, 2, 64, dtype=torch.float16, slopes=True, seed=53), Case([30000], 1, 8, 2, 64, page=16, seed=54),
             Case([4000, 900], 2, 128, 1, 576, dv=512, page=64, latent=True, seed=55),
             Case([2000, 100], 1, 8, 2, 128, dtype=torch.float32, seed=56),
             Case([400], 50, 4, 1, 64, dtype=torch.float32, seed=57)]
    jobs = []
    for c in cases:
        q = c.q.reshape(c.B * c.T, *c.q.shape[2:]).cuda()
        need = L.dense_attn_workspace_size(q.dtype, c.B, c.T, c.N, q.shape[1], c.k.shape[1], q.shape[2], c.dv)
        kw = dict(dv=c.dv, workspace=torch.empty(max(need, 16), dtype=torch.uint8, device="cuda"), **c.mods())
        jobs.append((q, c.k.cuda(), None if c.latent else c.v.cuda(), c.batch(), c.scale, kw))
    want = [L.dense_attn(*j[:5], **j[5]) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[] for _ in jobs]
    for _ in range(25):
        for i, j in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(L.dense_attn(*j[:5], **j[5]))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for x in g:
            assert torch.equal(x, w)
    assert L.idx_device_status(reset=True) == 0
