"""idx_page_copy, idx_page_update and idx_page_compact against step-by-step host code, their refusals, and a run of
them together with the attention that reads the pages."""

import ctypes
import math

import numpy as np
import pytest
import torch

import lightning_indexer_top_gb300 as L

INT_MIN = -2 ** 31


def host_update(table, parent, keep, new, ps, n_pages, held, cols):
    """(rows, left, copies) with copies = [(source page, target page, rows)]; rows None if there are too few pages."""
    B = len(parent)
    rows = [list(table[parent[b]][:keep[b] // ps]) if keep[b] else [] for b in range(B)]
    taken = set(held)
    for r in rows:
        taken.update(r)
    kept, copies = {}, []
    for b in range(B):
        if keep[b] % ps:
            last = table[parent[b]][keep[b] // ps]
            if last not in taken:
                taken.add(last)
                kept[b] = last
    free = [p for p in range(n_pages) if p not in taken]
    at = 0
    need = sum(-(-new[b] // ps) - len(rows[b]) - (b in kept) for b in range(B))
    if need > len(free):
        return None, len(free) - need, []
    for b in range(B):
        want = -(-new[b] // ps)
        if b in kept:
            rows[b].append(kept[b])
        elif keep[b] % ps:
            copies.append((table[parent[b]][keep[b] // ps], free[at], keep[b] % ps))
            rows[b].append(free[at])
            at += 1
        n = want - len(rows[b])
        rows[b] += free[at:at + n] + [-1] * (cols - want)
        at += n
    return rows, len(free) - at, copies


def host_compact(table, lens, ps, n_pages, held):
    need = [-(-n // ps) for n in lens]
    used = set(held).union(*[set(table[b][:need[b]]) for b in range(len(lens))]) if lens else set(held)
    n = len(used)
    to = dict(zip(sorted(p for p in used - set(held) if p >= n), [p for p in range(n) if p not in used]))
    rows = [[to.get(p, p) for p in table[b][:need[b]]] + [-1] * (len(table[b]) - need[b]) for b in range(len(lens))]
    return rows, n, [to.get(p, p) for p in range(n_pages)], [(a, b, ps) for a, b in to.items()]


def make_caches(n_pages, ps, kinds, seed=0):
    """Caches with NaN-free random bytes; "wide" ones are slices of wider rows."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for kind in kinds:
        shape, dtype, wide = kind
        n = math.prod(shape)
        full = torch.randint(-120, 120, (n_pages * ps, n + wide), generator=g).to(dtype).cuda()
        out.append(full[:, :n] if wide else full.view(n_pages * ps, *shape))
    return out


def expect_caches(caches, ps, copies):
    want = [c.clone() for c in caches]
    for c, w in zip(caches, want):
        for a, b, n in copies:
            w[b * ps:b * ps + n] = c[a * ps:a * ps + n]
    return want


KINDS = [
    [((128,), torch.float16, 0), ((576,), torch.bfloat16, 0)],
    [((4, 128), torch.bfloat16, 0), ((4, 128), torch.bfloat16, 0), ((132,), torch.int8, 0)],
    [((33,), torch.float32, 0)],
    [((5,), torch.int8, 0), ((7,), torch.int16, 2), ((64,), torch.float16, 24), ((1,), torch.int8, 0)],
    [((8,), torch.float16, 0)] * 8,
]


@pytest.mark.gpu
@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("ps", [1, 3, 16, 64, 300])
def test_copy(kinds, ps):
    n_pages = 40
    caches = make_caches(n_pages, ps, kinds, seed=ps)
    order = np.random.RandomState(ps).permutation(n_pages)
    for n in (1, 5, 20):
        src, dst = order[:n].tolist(), order[20:20 + n].tolist()
        want = expect_caches(caches, ps, [(a, b, ps) for a, b in zip(src, dst)])
        L.idx_page_copy(caches, ps, torch.tensor(src, dtype=torch.int32, device="cuda"),
                        torch.tensor(dst, dtype=torch.int32, device="cuda"))
        for c, w in zip(caches, want):
            assert torch.equal(c, w)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_copy_skips_what_it_is_told_to_and_what_is_out_of_range():
    ps, n_pages = 4, 10
    caches = make_caches(n_pages, ps, [((16,), torch.float32, 0)])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    want = expect_caches(caches, ps, [(0, 5, ps)])
    L.idx_page_copy(caches, ps, i32([-1, 0, 3, 2]), i32([1, 5, -1, 2]))
    assert torch.equal(caches[0], want[0]) and L.idx_device_status(reset=True) == 0
    L.idx_page_copy(caches, ps, i32([10, 1, 0]), i32([1, 10, 2 ** 31 - 1]))
    assert torch.equal(caches[0], want[0]) and L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS
    L.idx_page_copy(caches, ps, i32([]), i32([]))
    # rows past the last whole page stay
    odd = [torch.arange(43, device="cuda")]
    L.idx_page_copy(odd, ps, i32([0]), i32([9]))
    assert odd[0].tolist() == list(range(36)) + [0, 1, 2, 3] + [40, 41, 42]


def random_state(r, B, cols, ps, n_pages, shared=True):
    """A table as updates leave it: rows share whole pages."""
    table = np.full((B, cols), -1, np.int64)
    lens = r.randint(0, cols * ps + 1, B)
    order = list(r.permutation(n_pages))
    for b in range(B):
        need = -(-lens[b] // ps)
        n_shared = 0
        if shared and b and r.rand() < 0.5:
            a = r.randint(b)
            n_shared = min(lens[a] // ps, need, r.randint(0, cols + 1))
            table[b, :n_shared] = table[a, :n_shared]
        need = min(need, n_shared + len(order))
        lens[b] = min(lens[b], need * ps)
        for i in range(n_shared, need):
            table[b, i] = order.pop()
    held = [int(p) for p in order[:r.randint(0, 3)]]
    return table, lens, held


def call_update(table, parent, keep, new, ps, caches, held, n_pages, cols=None):
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")  # noqa: E731
    h = None
    if held is not None:
        h = torch.zeros(n_pages, dtype=torch.uint8, device="cuda")
        h[held] = 1
    t = i32(table).view(len(table), -1)
    out = torch.full((len(parent), t.shape[1] if cols is None else cols), -77, dtype=torch.int32, device="cuda")
    return L.idx_page_update(t, i32(parent), i32(keep), i32(new), ps, caches, held=h, new_table=out)


@pytest.mark.gpu
@pytest.mark.parametrize("ps", [1, 5, 64])
@pytest.mark.parametrize("B,cols,n_pages", [(1, 1, 1), (3, 4, 20), (8, 16, 130), (40, 33, 1500), (70, 3, 5000), (1100, 2, 3000)])
def test_update(ps, B, cols, n_pages):
    r = np.random.RandomState(B * ps + cols)
    for step in range(4):
        table, lens, held = random_state(r, B, cols, ps, n_pages)
        caches = make_caches(n_pages, ps, KINDS[step], seed=step)
        Bn = B if step % 2 == 0 else max(1, B - 1)
        new_cols = cols + (step == 3)
        parent = r.randint(-1, B, Bn) if step else np.arange(Bn)
        keep = np.where(parent < 0, 0, (lens[parent] * r.choice([0.0, 0.5, 1.0, 1.0], Bn)).astype(np.int64))
        new = np.minimum(keep + r.choice([0, 1, ps, 3 * ps], Bn), new_cols * ps)
        rows, left, copies = host_update(table.tolist(), parent, keep, new, ps, n_pages, held, new_cols)
        want = expect_caches(caches, ps, copies)
        out, n_free = call_update(table, parent, keep, new, ps, caches, held, n_pages, new_cols)
        assert int(n_free) == left
        if rows is None:
            assert (out == -77).all()
        else:
            assert out.tolist() == rows
        for c, w in zip(caches, want):
            assert torch.equal(c, w)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_update_cases_by_hand():
    ps, n_pages = 4, 12
    caches = make_caches(n_pages, ps, [((3,), torch.float32, 0)])
    table = [[5, 9, -1, -1], [2, -1, -1, -1]]
    # row 0 (6 positions) is forked three times: the first keeps page 9, the others copy its 2 rows; row 1 ends
    want = expect_caches(caches, ps, [(9, 0, 2), (9, 1, 1)])
    out, n_free = call_update(table, [0, 0, 0], [6, 6, 5], [7, 6, 9], ps, caches, None, n_pages)
    assert out.tolist() == [[5, 9, -1, -1], [5, 0, -1, -1], [5, 1, 2, -1]] and int(n_free) == 7
    assert torch.equal(caches[0], want[0])
    # a row that keeps the page whole: the row that wants part of it copies
    want = expect_caches(caches, ps, [(9, 0, 1)])
    out, n_free = call_update(table, [0, 0], [5, 8], [5, 8], ps, caches, None, n_pages)
    assert out.tolist() == [[5, 0, -1, -1], [5, 9, -1, -1]]
    assert torch.equal(caches[0], want[0])
    # a held page is copied too, and never handed out
    want = expect_caches(caches, ps, [(9, 1, 2)])
    out, n_free = call_update(table, [0], [6], [6], ps, caches, [9, 0], n_pages)
    assert out.tolist() == [[5, 1, -1, -1]] and int(n_free) == 8
    assert torch.equal(caches[0], want[0])
    # too few pages: the number missing, nothing written
    before = caches[0].clone()
    out, n_free = call_update(table, [0, 1, -1], [6, 3, 0], [16, 16, 31], ps, caches, None, n_pages, cols=8)
    assert int(n_free) == 12 - (2 + 1) - (2 + 3 + 8) and int(n_free) == -4
    assert (out == -77).all() and torch.equal(caches[0], before)
    # exactly enough
    out, n_free = call_update(table, [0, 1, -1], [6, 3, 0], [16, 16, 13], ps, caches, None, n_pages)
    assert int(n_free) == 0 and sorted(p for row in out.tolist() for p in row) == list(range(12))
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("parent,keep,new,cols", [
    ([2], [0], [0], 4), ([-2], [0], [0], 4), ([0], [-1], [0], 4), ([0], [4], [3], 4), ([0], [17], [17], 8),
    ([0], [4], [17], 4), ([-1], [1], [1], 4), ([1], [3], [3], 4), ([1], [8], [8], 4), ([0], [0], [-1], 4)])
def test_impossible_updates_change_nothing(parent, keep, new, cols):
    ps, n_pages = 4, 12
    caches = make_caches(n_pages, ps, [((3,), torch.float32, 0)])
    before = caches[0].clone()
    table = [[5, 9, 1, 2], [99, -1, -1, -1]]
    for more in (([], [], []), ([0], [6], [6])):
        out, n_free = call_update(table, parent + more[0], keep + more[1], new + more[2], ps, caches, None, n_pages, cols)
        assert int(n_free) == INT_MIN and (out == -77).all() and torch.equal(caches[0], before)
        assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS


@pytest.mark.gpu
@pytest.mark.parametrize("ps", [1, 5, 64])
@pytest.mark.parametrize("B,cols,n_pages", [(1, 1, 1), (3, 4, 20), (8, 16, 200), (40, 33, 1500), (70, 3, 5000)])
def test_compact(ps, B, cols, n_pages):
    r = np.random.RandomState(B * ps + cols)
    for step in range(4):
        table, lens, held = random_state(r, B, cols, ps, n_pages)
        lens = np.where(r.rand(B) < 0.3, 0, lens)
        held = [] if step == 0 else held
        caches = make_caches(n_pages, ps, KINDS[step], seed=step)
        rows, n, remap, moves = host_compact(table.tolist(), lens.tolist(), ps, n_pages, held)
        want = expect_caches(caches, ps, moves)
        i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")  # noqa: E731
        h = torch.zeros(n_pages, dtype=torch.bool, device="cuda")
        h[held] = True
        t = i32(table).view(B, cols)
        in_place = t if step % 2 else None
        out, n_used, m = L.idx_page_compact(t, i32(lens), ps, caches, held=h if held else None, new_table=in_place)
        assert out.tolist() == rows and int(n_used) == n and m.tolist() == remap
        for c, w in zip(caches, want):
            # pages that nobody uses any more keep what they held
            assert torch.equal(c, w)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
def test_compact_flags_bad_entries_and_lengths():
    ps, n_pages = 4, 8
    caches = make_caches(n_pages, ps, [((3,), torch.float32, 0)])
    t = torch.tensor([[7, 8], [3, 5]], dtype=torch.int32, device="cuda")
    out, n, _ = L.idx_page_compact(t, torch.tensor([8, 9], dtype=torch.int32, device="cuda"), ps, caches)
    assert out.tolist() == [[2, -1], [0, 1]] and int(n) == 3
    assert L.idx_device_status(reset=True) == L.IDX_ERR_DEVICE_BOUNDS
    out, n, _ = L.idx_page_compact(t[:0], torch.zeros(0, dtype=torch.int32, device="cuda"), ps, caches)
    assert out.shape == (0, 2) and int(n) == 0


@pytest.mark.gpu
def test_strided_tables():
    ps, n_pages = 4, 30
    caches = make_caches(n_pages, ps, [((3,), torch.float32, 0)])
    wide = torch.full((3, 9), 1000, dtype=torch.int32, device="cuda")
    t = wide[:, 2:6]
    t.copy_(torch.tensor([[5, 9, 1, -1], [20, 21, 22, 23], [8, -1, -1, -1]]))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    room = torch.full((3, 7), 55, dtype=torch.int32, device="cuda")
    L.idx_page_update(t, i32([0, 1, 2]), i32([10, 16, 2]), i32([13, 16, 2]), ps, caches, new_table=room[:, 1:5])
    assert room[:, 1:5].tolist() == [[5, 9, 1, 0], [20, 21, 22, 23], [8, -1, -1, -1]]
    assert (room[:, 0] == 55).all() and (room[:, 5:] == 55).all() and (wide[:, :2] == 1000).all()
    out, n, _ = L.idx_page_compact(t, i32([12, 16, 4]), ps, caches, new_table=room[:, 1:5])
    assert int(n) == 8 and out.tolist() == [[5, 2, 1, -1], [3, 4, 6, 7], [0, -1, -1, -1]]
    assert (room[:, 0] == 55).all() and (room[:, 5:] == 55).all()


@pytest.mark.gpu
def test_captured_twice_and_replayed():
    # two captured updates and a captured compaction, replayed in turn, each with its own workspace
    ps, n_pages, B, cols = 8, 400, 20, 12
    r = np.random.RandomState(3)
    table, lens, _ = random_state(r, B, cols, ps, n_pages)
    caches = make_caches(n_pages, ps, KINDS[0], seed=5)
    start = [c.clone() for c in caches]
    i32 = lambda x: torch.tensor(np.asarray(x, np.int32), device="cuda")  # noqa: E731
    t, parent = i32(table), r.randint(0, B, B)
    keep = lens[parent] // 2
    new = np.minimum(keep + 3, cols * ps)
    args = (i32(parent), i32(keep), i32(new))
    zero, hold = i32(lens), torch.empty(B, cols, dtype=torch.int32, device="cuda")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    got = []
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0]):
        got.append(L.idx_page_update(t, *args, ps, caches, new_table=hold))
    with torch.cuda.graph(graphs[1]):
        got.append(L.idx_page_compact(t, zero, ps, caches))
    rows, left, copies = host_update(table.tolist(), parent, keep, new, ps, n_pages, [], cols)
    for _ in range(3):
        for c, s in zip(caches, start):
            c.copy_(s)
        graphs[0].replay()
        want = expect_caches(start, ps, copies)
        assert hold.tolist() == rows and int(got[0][1]) == left
        for c, w in zip(caches, want):
            assert torch.equal(c, w)
        for c, s in zip(caches, start):
            c.copy_(s)
        graphs[1].replay()
        rows2, n, remap, moves = host_compact(table.tolist(), lens.tolist(), ps, n_pages, [])
        want = expect_caches(start, ps, moves)
        assert got[1][0].tolist() == rows2 and int(got[1][1]) == n and got[1][2].tolist() == remap
        for c, w in zip(caches, want):
            assert torch.equal(c, w)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,heads", [(torch.bfloat16, (8, 2, 128)), (torch.float32, (4, 2, 64)),
                                         (torch.bfloat16, (128, 1, 576))])
def test_a_served_batch(dtype, heads):
    """Prompts arrive in chunks, are decoded, forked and dropped, the pool is compacted; every step's attention equals
    the attention over each sequence's own contiguous copy of its tokens."""
    Hq, Hkv, d = heads
    latent = d == 576
    dv = 512 if latent else d
    ps, n_pages, cols, slots = 16, 64, 12, 4
    g = torch.Generator().manual_seed(7)
    shape = (n_pages * ps, d) if latent else (n_pages * ps, Hkv, d)
    caches = [torch.full(shape, float("nan"), dtype=dtype, device="cuda") for _ in range(1 if latent else 2)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((slots, cols), -1, dtype=torch.int32, device="cuda")
    own = [[torch.empty(0, *shape[1:], dtype=dtype, device="cuda") for _ in caches] for _ in range(slots)]
    lens = [0] * slots
    # (parents, kept, new tokens, compact) of each step
    script = [([-1, -1, -1, -1], None, [37, 20, 1, 0], False), ([0, 1, 2, 2], None, [1, 1, 1, 1], False),
              ([0, 0, 0, 1], None, [1, 1, 1, 1], False), ([0, 1, 3, 2], [30, None, None, 20], [9, 1, 1, 3], True),
              ([3, 3, -1, 0], None, [1, 1, 40, 1], False), ([0, 1, 2, 3], None, [1, 1, 1, 1], True)]
    for parent, kept, fresh, compact in script:
        keep = [0 if p < 0 else lens[p] if kept is None or kept[b] is None else kept[b] for b, p in enumerate(parent)]
        new = [k + f for k, f in zip(keep, fresh)]
        table, n_free = L.idx_page_update(table, i32(parent), i32(keep), i32(new), ps, caches)
        assert int(n_free) >= 0
        own = [[o[:keep[b]] for o in (own[p] if p >= 0 else own[b])] for b, p in enumerate(parent)]
        T = max(fresh)
        pos = torch.full((slots, T), -1, dtype=torch.int32)
        for b in range(slots):
            rows = torch.arange(keep[b], new[b], device="cuda")
            at = table[b].long()[rows // ps] * ps + rows % ps
            for c, cache in enumerate(caches):
                x = torch.randn(fresh[b], *shape[1:], generator=g).to(dtype).cuda()
                cache[at] = x
                own[b][c] = torch.cat([own[b][c], x])
            pos[b, :fresh[b]] = torch.arange(keep[b], new[b], dtype=torch.int32)
        lens = new
        q = torch.randn(slots * T, Hq, d, generator=g).to(dtype).cuda()
        n_max = max(lens)
        paged = L.Batch(i32(lens), T, n_max, q_pos=pos.flatten().cuda(), page_table=table, page_size=ps)
        flat = L.Batch(i32(lens), T, n_max, kv_seq_stride=n_max, q_pos=pos.flatten().cuda())
        rows = [torch.full((slots * n_max, *shape[1:]), float("nan"), dtype=dtype, device="cuda") for _ in caches]
        for b in range(slots):
            for r, o in zip(rows, own[b]):
                r[b * n_max:b * n_max + lens[b]] = o
        kw = dict(dv=dv)
        v = lambda x: None if latent else x[1]  # noqa: E731
        want = L.dense_attn(q, rows[0], v(rows), flat, 0.1, **kw)
        got = L.dense_attn(q, caches[0], v(caches), paged, 0.1, **kw)
        assert torch.isfinite(got).all()
        assert torch.equal(got, want)
        if compact:
            table, n_used, _ = L.idx_page_compact(table, i32(lens), ps, caches)
            assert int(table.max()) < int(n_used)
            paged.page_table = table
            assert torch.equal(L.dense_attn(q, caches[0], v(caches), paged, 0.1, **kw), want)
    assert L.idx_device_status(reset=True) == 0


# ------------------------------------------------------------------------------------------ refusals (CPU)

def _lib():
    L.build()
    return L.load()


def _caches(n=1, data=16, stride=256, row=256):
    arr = (L._PageCache * max(n, 1))()
    for i in range(n):
        arr[i] = L._PageCache(data, stride, row)
    return arr


@pytest.mark.parametrize("kw,word", [
    (dict(n_caches=0), "n_caches"), (dict(n_caches=9), "n_caches"), (dict(caches=None), "caches"), (dict(ps=0), "page_size"),
    (dict(n_pages=-1), "n_pages"), (dict(caches=_caches(row=0)), "row_bytes"), (dict(caches=_caches(stride=8, row=16)), "row_bytes"),
    (dict(caches=_caches(data=None)), "data"), (dict(n=-1), "n < 0"), (dict(src=None), "NULL"), (dict(dst=None), "NULL"),
    (dict(caches=_caches(stride=2 ** 61, row=16)), "address space")])
def test_copy_refusals(kw, word):
    lib = _lib()
    a = dict(caches=_caches(), n_caches=1, ps=16, n_pages=8, src=16, dst=16, n=2)
    a.update(kw)
    st = lib.idx_page_copy(a["caches"], a["n_caches"], a["ps"], a["n_pages"], a["src"], a["dst"], a["n"], None)
    assert st == L.IDX_ERR_INVALID_ARG and word in lib.idx_last_error().decode()


def test_nothing_to_copy_is_fine():
    lib = _lib()
    assert lib.idx_page_copy(_caches(), 1, 16, 8, None, None, 0, None) == L.IDX_OK


@pytest.mark.parametrize("kw,word", [
    (dict(n_caches=9), "n_caches"), (dict(n_caches=-1), "n_caches"), (dict(ps=0), "page_size"), (dict(n_old=-1), "n_seq"), (dict(n=-1), "n_seq"),
    (dict(stride=3), "columns"), (dict(cols=-1), "columns"), (dict(new_stride=3), "columns"), (dict(parent=None), "NULL"),
    (dict(keep=None), "NULL"), (dict(new=None), "NULL"), (dict(table=None), "NULL"), (dict(out=None), "NULL"),
    (dict(n_free=None), "NULL"), (dict(ws=None), "workspace"), (dict(wb=8), "workspace"), (dict(ws=24), "workspace"),
    (dict(out=4096 + 16), "overlaps"), (dict(n=2 ** 30, new_cols=4), "entries")])
def test_update_refusals(kw, word):
    lib = _lib()
    a = dict(table=4096, stride=4, cols=4, n_old=2, parent=16, keep=16, new=16, n=2, ps=16, n_pages=8, held=None, out=8192,
             new_stride=4, new_cols=4, n_free=16, caches=_caches(), n_caches=1, ws=65536, wb=1 << 20)
    a.update(kw)
    st = lib.idx_page_update(a["table"], a["stride"], a["cols"], a["n_old"], a["parent"], a["keep"], a["new"], a["n"],
                             a["ps"], a["n_pages"], a["held"], a["out"], a["new_stride"], a["new_cols"], a["n_free"],
                             a["caches"], a["n_caches"], a["ws"], a["wb"], None)
    assert st == L.IDX_ERR_INVALID_ARG and word in lib.idx_last_error().decode(), lib.idx_last_error()


@pytest.mark.parametrize("kw,word", [
    (dict(n_caches=9), "n_caches"), (dict(ps=0), "page_size"), (dict(n=-1), "n_seq"), (dict(stride=3), "table_cols"),
    (dict(new_stride=3), "table_cols"), (dict(lens=None), "NULL"), (dict(table=None), "NULL"), (dict(out=None), "NULL"),
    (dict(n_used=None), "NULL"), (dict(ws=None), "workspace"), (dict(wb=8), "workspace"), (dict(ws=24), "workspace"),
    (dict(out=4096 + 16), "overlaps"), (dict(out=4096, new_stride=5), "overlaps"), (dict(n=2 ** 30), "entries")])
def test_compact_refusals(kw, word):
    lib = _lib()
    a = dict(table=4096, stride=4, cols=4, n=2, lens=16, ps=16, n_pages=8, held=None, out=8192, new_stride=4, n_used=16,
             remap=None, caches=_caches(), n_caches=1, ws=65536, wb=1 << 20)
    a.update(kw)
    st = lib.idx_page_compact(a["table"], a["stride"], a["cols"], a["n"], a["lens"], a["ps"], a["n_pages"], a["held"],
                              a["out"], a["new_stride"], a["n_used"], a["remap"], a["caches"], a["n_caches"], a["ws"],
                              a["wb"], None)
    assert st == L.IDX_ERR_INVALID_ARG and word in lib.idx_last_error().decode(), lib.idx_last_error()


def test_workspace_grows_with_the_pages():
    _lib()
    assert L.idx_page_workspace_size(-1, 8) == 0 and L.idx_page_workspace_size(1, -1) == 0
    assert 0 < L.idx_page_workspace_size(1, 8) < L.idx_page_workspace_size(1, 8000) < L.idx_page_workspace_size(8000, 8000)


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(8, 4)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        L.idx_page_copy([x], 4, i, i)


@pytest.mark.gpu
def test_binding_refuses_mismatched_tensors():
    x = torch.zeros(32, 4, device="cuda")
    i = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    for f in (lambda: L.idx_page_copy([], 4, i, i), lambda: L.idx_page_copy([x], 0, i, i),
              lambda: L.idx_page_copy([x, x[:16]], 4, i, i), lambda: L.idx_page_copy([x[:, ::2]], 4, i, i),
              lambda: L.idx_page_copy([x], 4, i.long(), i), lambda: L.idx_page_copy([x], 4, i, t.view(-1)),
              lambda: L.idx_page_copy([x] * 9, 4, i, i), lambda: L.idx_page_update(t.view(-1), i, i, i, 4, [x]),
              lambda: L.idx_page_update(t, i, t.view(-1), i, 4, [x]), lambda: L.idx_page_update(t.long(), i, i, i, 4, [x]),
              lambda: L.idx_page_update(t, i, i, i, 4, [x], held=torch.zeros(7, dtype=torch.uint8, device="cuda")),
              lambda: L.idx_page_update(t, i, i, i, 4, [x], new_table=torch.zeros(2, 4, dtype=torch.int32, device="cuda")),
              lambda: L.idx_page_compact(t, t.view(-1), 4, [x]), lambda: L.idx_page_compact(t.t(), i, 4, [x]),
              lambda: L.idx_page_compact(t, i, 4, [x], new_table=t[:, :2])):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(L.LidxError, match="overlaps"):
        L.idx_page_update(t, i, i, i, 4, [x], new_table=t)
