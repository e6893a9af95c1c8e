"""What callers of the paged cache get back for users that a call leaves out, from
repeated calls and from several threads, and numbers that it cannot take."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import oracle.cache as oc
from cache_harness import DT, Case, attend_bounds, close, mass_bound
from latent_attention_jagged_b200 import LatentCache
from latent_attention_jagged_b200.binding import DEV_BAD_OFFSETS, DEV_TOO_LONG, LLATTE_ERR_ARG

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("budget", [8, 100])
@pytest.mark.parametrize("apart", [False, True])
def test_lengths_that_eviction_returns_for_users_left_out(budget, apart):
    c = Case("bf16", 2, 64, 16, [40, 40, 40, 5], seed=13, spare=16, stale=0.25)
    lengths = c.lengths.copy()
    lengths[0], lengths[1] = -5, 10 ** 6
    dst = torch.tensor(c.free[:12], dtype=torch.int32).reshape(4, 3).cuda() if apart else None
    for _ in range(3):                       # blocks of freed memory hold other numbers
        junk = torch.full((4,), 23, dtype=torch.int32, device="cuda")
        del junk
        got = c.cache.evict(c.dev("table"), torch.from_numpy(lengths).cuda(), budget,
                            dst_table=dst)
        assert c.cache.status() == DEV_TOO_LONG
        assert got.cpu().tolist() == [-5, 10 ** 6, min(40, budget), 5]


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("bf16", 40), ("fp32", 32), ("fp32", 256)])
@pytest.mark.parametrize("new", [1, 40])
def test_rows_of_users_left_out_are_zeros(dtype, rank, new):
    c = Case(dtype, 4, rank, 32, [70, 130, 64, 90], seed=7)
    q, off = c.queries([new] * 4, 1)
    ref, ref_lse = oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table,
                             c.lengths, 1, 0.1)
    lengths = c.lengths.copy()
    lengths[1], lengths[2] = 1 << 20, -1
    if new == 1:
        lengths[3] = 0                       # fewer events than new rows
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 3.0, device="cuda")
    before = c.mass.clone()
    c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"),
                   torch.from_numpy(lengths).cuda(), n_cand=1, scale=0.1, out=out, lse=lse,
                   accumulate=True)
    assert c.cache.status() == DEV_TOO_LONG | (DEV_BAD_OFFSETS if new == 1 else 0)
    left = [1, 2] + ([3] if new == 1 else [])
    for u in range(4):
        a, b = off[u], off[u + 1]
        pages = torch.from_numpy(c.table[u][:-(-int(c.lengths[u]) // 32)]).long().cuda()
        if u in left:
            assert (out[a:b] == 0).all() and (lse[a:b] == -float("inf")).all()
            assert torch.equal(c.mass[pages], before[pages])
        else:
            sp = {}
            oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table, c.lengths, 1,
                      0.1, 0, 0, sp)
            b_out, b_lse = attend_bounds(dtype, rank, 130, sp, ref, ref_lse)
            close(out[a:b], ref[a:b], b_out[a:b], "out")
            close(lse[a:b], ref_lse[a:b], b_lse[a:b], "lse")


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("fp32", 32)])
def test_appending_again_clears_what_the_events_collected(dtype, rank):
    # the latents stay, the masses of the appended rows start over, those of the events
    # before them do not
    c = Case(dtype, 2, rank, 32, [100, 40], seed=9, stale=0.0)
    new = [10, 3]
    x = torch.from_numpy(c.rng.standard_normal((13, rank)).astype(np.float32)).to(DT[dtype]).cuda()
    off = torch.tensor([0, 10, 13]).cuda()
    args = (x, off, c.dev("table"), c.dev("lengths"))
    c.mass.zero_()
    c.cache.append(*args)
    q, qoff = c.queries(new, 1)
    sp = {}
    mass = c.host_mass()
    oc.attend(c.host_pool(), mass, q.double().cpu().numpy(), qoff, c.table, c.lengths, 1, 0.1, 0, 0,
              sp)
    c.cache.attend(q, torch.from_numpy(qoff).cuda(), c.dev("table"), c.dev("lengths"), n_cand=1,
                   scale=0.1, accumulate=True)
    bound = mass_bound(rank, 100, sp, mass)
    close(c.mass, mass, bound, "mass")
    pool = c.pool.clone()
    c.cache.append(*args)
    assert torch.equal(c.pool, pool) and c.cache.status() == 0
    for u, m in enumerate(new):
        pg, rw = oc.slots(c.table[u], int(c.lengths[u]), 32)
        mass[pg[-m:], rw[-m:]] = 0.0
        bound[pg[-m:], rw[-m:]] = 0.0
    close(c.mass, mass, bound, "mass after the second append")


def test_caches_of_other_ranks_in_several_threads():
    # the same kernel with more and with less shared memory, from threads of their own
    ranks = [100, 128, 100, 128, 68, 128]
    cases = [Case("fp32", 2, r, 32, [60, 40], seed=70) for r in ranks]
    calls, failed = [], []
    for x in cases:
        q, off = x.queries([1, 1], 0)
        args = (q, torch.from_numpy(off).cuda(), x.dev("table"), x.dev("lengths"))
        want = x.cache.attend(*args, scale=0.1).clone()
        out = torch.empty_like(q)
        stream = torch.cuda.Stream()
        calls.append((x.cache, args, out, stream, want))
    torch.cuda.synchronize()

    def work(cache, args, out, stream, want):
        try:
            for _ in range(2000):
                cache.attend(*args, scale=0.1, out=out, stream=stream)
        except Exception as e:               # noqa: BLE001 - reported by the test
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    assert all(torch.equal(out, want) for _, _, out, _, want in calls)


def test_numbers_that_do_not_fit_are_refused():
    c = Case("bf16", 4, 128, 64, [70, 30], seed=6)
    q, off = c.queries([1, 1], 1)
    o, t, n = torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths")
    pool, mass = c.pool.clone(), c.mass.clone()
    for k in (dict(n_cand=1 << 32), dict(window=(1 << 32) + 5), dict(n_sink=1 << 31),
              dict(window=-(1 << 31) - 1)):
        with pytest.raises(ValueError):
            c.cache.attend(q, o, t, n, **k)
    for k in (dict(budget=(1 << 32) + 4), dict(budget=8, n_sink=1 << 32),
              dict(budget=8, n_recent=(1 << 32) + 1)):
        with pytest.raises(ValueError):
            c.cache.evict(t, n, **k)
    for k in (dict(heads=(1 << 32) + 4), dict(max_batch=(1 << 32) + 2), dict(max_pages=1 << 32),
              dict(max_rows=1 << 64)):
        with pytest.raises(ValueError):
            LatentCache(c.pool, **dict(dict(heads=4), **k))
    torch.cuda.synchronize()
    assert c.cache.status() == 0
    assert torch.equal(torch.nan_to_num(c.pool), torch.nan_to_num(pool))
    assert torch.equal(c.mass, mass)


def test_append_refuses_more_rows_than_it_can_count():
    c = Case("bf16", 4, 64, 16, [20], seed=6)
    x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 2]).cuda()
    v, _ = c.cache._view(c.dev("table"), c.dev("lengths"))
    for rows in (-1, 1 << 29, 1 << 31, 1 << 61, 1 << 62, (1 << 63) - 1):
        assert c.cache.lib.llatte_cache_append(
            c.cache.h, ctypes.byref(v), x.data_ptr(), rows, off.data_ptr(), None, 1e-6,
            None) == LLATTE_ERR_ARG
