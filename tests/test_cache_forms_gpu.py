"""The paged cache's form for single tokens where some users ask with many rows: users of
17 to 400 (row, head) pairs in batches whose mean stays within the form; and the
accumulated weights where scores outgrow a sum's base and where pages are gone."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from cache_harness import DT, Case, check_attend, close, mass_bound

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("bf16", 40), ("fp32", 32), ("fp32", 256)]


@pytest.mark.parametrize("dtype,rank", KINDS)
@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("window,sink", [(0, 0), (70, 5)])
def test_users_of_many_pairs_among_users_of_few(dtype, rank, heads, window, sink):
    many = [17, 33, 64, 100, 200]            # pairs, to be divided by the heads
    new = [-(-n // heads) for n in many]
    rows = sum(new)
    # users without rows bring the mean to 8 pairs a user or less
    idle = -(-rows * heads // 8)
    lengths = [300, 129, 64, 1000, 450] + [20] * idle
    c = Case(dtype, heads, rank, 32, lengths, seed=80)
    check_attend(c, new + [0] * idle, window=window, n_sink=sink, accumulate=True)


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("fp32", 32)])
def test_one_long_chunk_among_idle_users(dtype, rank):
    c = Case(dtype, 4, rank, 64, [1500] + [30] * 215, seed=81)
    check_attend(c, [400] + [0] * 215, n_cand=0, accumulate=True)


@pytest.mark.parametrize("dtype,rank", KINDS)
@pytest.mark.parametrize("rows", [2, 70])
def test_weights_where_maxima_outgrow_the_base(dtype, rank, rows):
    # scores rise by 18 (26 in log2 units) every 64 events, for the last head not at all
    n, heads = 640, 2
    c = Case(dtype, heads, rank, 32, [n], seed=53)
    at = tuple(torch.from_numpy(a).cuda() for a in oc.slots(c.table[0], n, 32))
    t = (torch.arange(n) // 64).float()[:, None]
    c.pool[at] = (t * torch.ones(rank)).to(DT[dtype]).cuda()
    q, off = c.queries([rows], 0)
    q[:, 0] = 1.0
    q[:, 1] = 0.0
    scale = 18.0 / rank
    sp = {}
    mass = c.host_mass()
    oc.attend(c.host_pool(), mass, q.double().cpu().numpy(), off, c.table, c.lengths, 0, scale, 0, 0,
              sp)
    c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"), scale=scale,
                   accumulate=True)
    assert c.cache.status() == 0
    close(c.mass, mass, mass_bound(rank, n, sp, mass), "mass")


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("bf16", 40), ("fp32", 32)])
@pytest.mark.parametrize("new", [1, 30])
def test_weights_where_pages_outside_every_window_are_gone(dtype, rank, new):
    c = Case(dtype, 4, rank, 16, [500, 64], seed=57)
    q, off = c.queries([new, new], 0)
    kw = dict(scale=0.1, window=50, n_sink=20)
    gone = c.table.copy()
    # user 0: the first 20 events lie in pages 0 and 1, its windows begin at event
    # 500 - new - 49 or later
    gone[0, 2:(500 - new - 49) // 16] = -7
    for table in (c.table, gone):
        before, mass, sp = c.mass.clone(), c.host_mass(), {}
        oc.attend(c.host_pool(), mass, q.double().cpu().numpy(), off, c.table, c.lengths, 0,
                  kw["scale"], kw["window"], kw["n_sink"], sp)
        c.cache.attend(q, torch.from_numpy(off).cuda(), torch.from_numpy(table).cuda(),
                       c.dev("lengths"), accumulate=True, **kw)
        assert c.cache.status() == 0
        close(c.mass, mass, mass_bound(rank, 500, sp, mass), "mass")
        unseen = torch.from_numpy(sp["hits"] == 0).cuda()
        assert unseen.any() and torch.equal(c.mass[unseen], before[unseen])
