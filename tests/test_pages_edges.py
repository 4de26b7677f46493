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
