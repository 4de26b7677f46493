"""The page operations beside other work and at the ends of their ranges."""

import numpy as np
import pytest
import torch

import lightning_indexer_top_gb300 as L
from test_pages import host_update, random_state


def _i32(x):
    return torch.tensor(np.asarray(x, np.int32), device="cuda")


@pytest.mark.gpu
def test_updates_beside_other_work():
    # plans on two streams, while a third keeps the SMs busy: a plan's CTAs start at different times
    ps, n_pages, B, cols = 4, 3000, 90, 16
    r = np.random.RandomState(17)
    load = torch.randn(1 << 24, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(3)]
    jobs = []
    for _ in range(2):
        table, lens, held = random_state(r, B, cols, ps, n_pages)
        parent = r.randint(0, B, B)
        keep = (lens[parent] * r.choice([0.5, 1.0], B)).astype(np.int64)
        new = np.minimum(keep + 3, cols * ps)
        want, left, _ = host_update(table.tolist(), parent, keep, new, ps, n_pages, held, cols)
        h = torch.zeros(n_pages, dtype=torch.uint8, device="cuda")
        h[held] = 1
        cache = torch.zeros(n_pages * ps, 16, device="cuda")
        ws = torch.empty(L.idx_page_workspace_size(B, n_pages), dtype=torch.uint8, device="cuda")
        jobs.append(((_i32(table).view(B, cols), _i32(parent), _i32(keep), _i32(new), ps, [cache]),
                     dict(held=h, workspace=ws), want, left))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(40):
        with torch.cuda.stream(streams[2]):
            load.mul_(1.0)
        for i, (args, kw, _, _) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(L.idx_page_update(*args, **kw))
    torch.cuda.synchronize()
    for g, (_, _, want, left) in zip(got, jobs):
        for table, n_free in g:
            assert int(n_free) == left and table.tolist() == (want if want is not None else table.tolist())
    assert all(w is not None for _, _, w, _ in jobs)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("n_pages", [6291456, 6500001])
def test_pools_around_the_largest_bitmap_in_shared_memory(n_pages):
    # a slice of the plans' bitmap is kept in shared memory up to 24576 words: 6291456 pages; beyond, in the workspace
    ps, B, cols = 2, 30, 40
    r = np.random.RandomState(5)
    cache = torch.randint(0, 256, (n_pages * ps, 1), dtype=torch.uint8, device="cuda",
                          generator=torch.Generator("cuda").manual_seed(6))
    lens = r.randint(1, cols * ps + 1, B)
    need = -(-lens // ps)
    order = np.unique(np.concatenate([r.randint(0, n_pages, 3000), [0, 31, 32, n_pages - 1]]))
    r.shuffle(order)
    table = np.full((B, cols), -1, np.int64)
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    held = [int(p) for p in order[at:at + 3]]
    h = torch.zeros(n_pages, dtype=torch.uint8, device="cuda")
    h[held] = 1
    parent = r.randint(0, B, B)
    keep = (lens[parent] * r.choice([0.5, 1.0], B)).astype(np.int64)
    new = np.minimum(keep + 5, cols * ps)
    want, left, copies = host_update(table.tolist(), parent, keep, new, ps, n_pages, held, cols)
    rows = cache.clone()
    out, n_free = L.idx_page_update(_i32(table), _i32(parent), _i32(keep), _i32(new), ps, [rows], held=h)
    assert int(n_free) == left and out.tolist() == want
    expect = cache.clone()
    for a, b, n in copies:
        expect[b * ps:b * ps + n] = cache[a * ps:a * ps + n]
    assert copies and torch.equal(rows, expect)
    rows.copy_(cache)
    out, n_used, remap = L.idx_page_compact(_i32(table), _i32(lens), ps, [rows], held=h)
    used = np.unique(np.concatenate([table[b, :need[b]] for b in range(B)] + [held]))
    n = len(used)
    moves = np.setdiff1d(used[used >= n], held)
    holes = np.setdiff1d(np.arange(n), used)[:len(moves)]
    to = np.arange(n_pages)
    to[moves] = holes
    assert int(n_used) == n and np.array_equal(remap.cpu().numpy(), to)
    assert np.array_equal(out.cpu().numpy(), np.where(table >= 0, to[table], -1))
    expect = cache.clone()
    for a, b in zip(moves, holes):
        expect[b * ps:(b + 1) * ps] = cache[a * ps:(a + 1) * ps]
    assert torch.equal(rows, expect)
    assert L.idx_device_status(reset=True) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("wide", [0, 8])
def test_pages_beyond_32_bit_offsets(wide):
    # pages at both ends of a cache of more than 2^32 bytes; wide: rows with bytes between them that stay as they are
    ps, row = 64, 1152
    n_pages = (1 << 32) // (ps * row) + 200
    cache = torch.empty(n_pages * ps, row + wide, dtype=torch.uint8, device="cuda")
    for p in range(8):
        cache[p * ps:(p + 1) * ps] = p
        cache[(n_pages - 1 - p) * ps:(n_pages - p) * ps] = 100 + p
    view = cache[:, :row]
    L.idx_page_copy([view], ps, _i32([0, n_pages - 1]), _i32([n_pages - 3, 2]))
    for p, want in ((n_pages - 3, 0), (2, 100), (n_pages - 2, 101), (n_pages - 4, 103), (1, 1), (3, 3)):
        assert (view[p * ps:(p + 1) * ps] == want).all()
    if wide:
        assert (cache[2 * ps:3 * ps, row:] == 2).all() and (cache[(n_pages - 3) * ps:(n_pages - 2) * ps, row:] == 102).all()
    # the used pages at the far end come down
    table = _i32([[n_pages - 1, n_pages - 2], [n_pages - 1, -1]])
    new, n_used, _ = L.idx_page_compact(table, _i32([2 * ps, ps]), ps, [view])
    assert new.tolist() == [[1, 0], [1, -1]] and int(n_used) == 2
    assert (view[:ps] == 101).all() and (view[ps:2 * ps] == 100).all()
