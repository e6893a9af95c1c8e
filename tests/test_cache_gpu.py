"""GPU parity of the paged latent cache (append, attention with window and
sinks, accumulated weights, eviction) against the fp64 oracle, with bounds
derived from the roundings (see cache_harness)."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from cache_harness import DT, Case, attend_bounds, check_attend, close
from latent_attention_jagged_b200 import LatentCache, LlatteError
from latent_attention_jagged_b200.binding import (DEV_BAD_ID, DEV_BAD_OFFSETS, DEV_TOO_LONG,
                                                  LLATTE_ERR_ARG)

pytestmark = pytest.mark.gpu

SHAPES = [("bf16", 4, 128, 64), ("bf16", 8, 256, 128), ("bf16", 3, 64, 16), ("bf16", 5, 40, 32),
          ("bf16", 1, 128, 128), ("bf16", 130, 64, 32), ("fp32", 2, 32, 16), ("fp32", 4, 128, 64),
          ("fp32", 3, 100, 32), ("fp32", 8, 256, 128)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("window,sink", [(0, 0), (1, 0), (50, 0), (130, 3), (37, 200)])
def test_attend(shape, window, sink):
    dtype, heads, rank, page = shape
    # empty, one event, page and tile edges, odd lengths
    lengths = [0, 1, page, 129, 300, 256, 2, 515]
    new = [0, 1, 3, 129, 40, 0, 2, 7]
    if heads > 100:
        lengths, new = lengths[:5], [0, 1, 3, 5, 2]
    c = Case(dtype, heads, rank, page, lengths, seed=window + sink, spare=2)
    check_attend(c, new, n_cand=3, window=window, n_sink=sink)


@pytest.mark.parametrize("shape", SHAPES[:5] + SHAPES[6:8], ids=str)
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 4)])
def test_single_tokens(shape, window, sink):
    dtype, heads, rank, page = shape
    lengths = [1, 17, 128, 129, 4000, 1000, 333]
    c = Case(dtype, heads, rank, page, lengths, seed=5)
    check_attend(c, [1] * 7, window=window, n_sink=sink, accumulate=True)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_accumulate(shape):
    dtype, heads, rank, page = shape
    lengths, new = [300, 0, 1, 140, 2 * page], [60, 0, 1, 140, 0]
    if heads > 100:
        new = [5, 0, 1, 3, 0]
    c = Case(dtype, heads, rank, page, lengths, seed=8)
    check_attend(c, new, n_cand=2, accumulate=True)
    before = c.mass.clone()
    check_attend(c, new, n_cand=1, window=33, n_sink=2, accumulate=True, sharp=6.0)
    assert not torch.equal(before, c.mass)


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("bf16", 256), ("fp32", 64)])
def test_same_bits_on_every_run(dtype, rank):
    c = Case(dtype, 4, rank, 64, [700, 90, 2500, 31], seed=1)
    q, off = c.queries([90, 33, 1, 4], 5)
    off_d, tab, ln = torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths")
    first = None
    mass0 = c.mass.clone()
    for _ in range(5):
        c.mass.copy_(mass0)
        out = c.cache.attend(q, off_d, tab, ln, n_cand=5, scale=0.1, accumulate=True)
        got = out.clone(), c.mass.clone()
        if first is None:
            first = got
        assert torch.equal(first[0], got[0]) and torch.equal(
            torch.nan_to_num(first[1]), torch.nan_to_num(got[1]))


def test_rescaling_over_growing_scores():
    # every tile of events scores far above the ones before
    for dtype, rank in (("bf16", 128), ("bf16", 256), ("fp32", 128)):
        c = Case(dtype, 2, rank, 32, [900], seed=2)
        at = tuple(torch.from_numpy(a) for a in oc.slots(c.table[0], 900, 32))
        d = torch.ones(rank)
        t = torch.arange(900, dtype=torch.float32)[:, None] / 16
        c.pool[at[0].cuda(), at[1].cuda()] = (t * d).to(DT[dtype]).cuda()
        q, off = c.queries([4], 2)
        q.fill_(1.0)
        sp = {}
        ref, ref_lse = oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table,
                                 c.lengths, 2, 1 / 32, 0, 0, sp)
        lse = torch.empty(q.shape[:2], device="cuda")
        out = c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"),
                             n_cand=2, scale=1 / 32, lse=lse)
        b_out, b_lse = attend_bounds(dtype, rank, 900, sp, ref, ref_lse)
        close(out, ref, b_out, "out")
        close(lse, ref_lse, b_lse, "lse")


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("bf16", 64), ("bf16", 40), ("fp32", 32)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_hidden_values_have_no_effect(dtype, rank, value):
    # rows of no event are NaN already (Case); here the newest event and one
    # outside every window are not finite either
    c = Case(dtype, 4, rank, 32, [200, 90], seed=4)
    q, off = c.queries([10, 10], 0)
    args = (q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"))
    kw = dict(scale=0.1, window=60, n_sink=3)
    clean = c.cache.attend(*args, **kw).clone()
    for u, t in ((0, 199), (0, 100), (1, 89), (1, 5)):
        pg, rw = c.table[u][t // 32], t % 32
        c.pool[int(pg), rw] = value
    lse = torch.empty(q.shape[:2], device="cuda")
    got = c.cache.attend(*args, lse=lse, accumulate=True, **kw)
    sees = torch.zeros(20, dtype=torch.bool)
    sees[[9, 19]] = True                      # only the newest rows see a bad event
    assert torch.equal(got[~sees.cuda()], clean[~sees.cuda()])
    assert torch.isfinite(lse[~sees.cuda()]).all()
    assert not torch.isfinite(got[sees.cuda()]).any()


def test_rows_of_no_user_stay_and_offsets_may_start_late():
    c = Case("bf16", 4, 128, 64, [70, 130], seed=6)
    q, off = c.queries([1, 2], 1, first=3, behind=5)
    out = torch.full_like(q, 3.0)
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"), n_cand=1,
                   scale=0.1, out=out, lse=lse)
    ref, _ = oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table, c.lengths, 1,
                       0.1)
    for t in (out, lse):
        assert (t[:3] == 3).all() and (t[8:] == 3).all()
    assert np.abs(out[3:8].double().cpu().numpy() - ref[3:8]).max() < 0.05


def test_users_with_fewer_rows_than_query_tokens():
    c = Case("bf16", 4, 128, 64, [70, 0, 10], seed=6)
    q, _ = c.queries([0, 0, 0], 2)
    off = np.array([0, 1, 2, 2])              # one row, one row without events, none
    q = q[:2].contiguous()
    out = c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"),
                         n_cand=5, scale=0.1)
    ref, _ = oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table, c.lengths, 5,
                       0.1)
    assert np.abs(out.double().cpu().numpy() - ref).max() < 0.05 and (out[1] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_faulty_users_are_left_out(dtype):
    c = Case(dtype, 4, 128, 64, [70, 130, 64, 5, 9], seed=7, spare=1)
    q, off = c.queries([1, 2, 1, 1, 1], 1)
    ref, _ = oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table, c.lengths, 1,
                       0.1)
    lengths, table = c.lengths.copy(), c.table.copy()
    lengths[1], lengths[2] = 1 << 20, -1              # longer than its pages, negative
    lengths[3] = 0                                    # fewer events than new rows
    args = [q, torch.from_numpy(off).cuda(), torch.from_numpy(table).cuda(),
            torch.from_numpy(lengths).cuda()]
    out = c.cache.attend(*args, n_cand=1, scale=0.1, accumulate=True)
    assert c.cache.status() == DEV_TOO_LONG | DEV_BAD_OFFSETS and c.cache.status() == 0
    good = list(range(0, 2)) + list(range(9, 11))
    assert np.abs(out.double().cpu().numpy()[good] - ref[good]).max() < 0.05
    # offsets past the rows, and decreasing ones
    bad = off.copy()
    bad[5] = 1000
    bad[2] = 1
    args[1], args[3] = torch.from_numpy(bad).cuda(), c.dev("lengths")
    out = c.cache.attend(*args, n_cand=1, scale=0.1)
    assert c.cache.status() & DEV_BAD_OFFSETS
    assert np.abs(out.double().cpu().numpy()[7:9] - ref[7:9]).max() < 0.05
    # pages outside the pool read as zero rows
    bad = table.copy()
    bad[0, 0], bad[0, 1] = -3, 1 << 29
    args[1], args[2] = torch.from_numpy(off).cuda(), torch.from_numpy(bad).cuda()
    out = c.cache.attend(*args, n_cand=1, scale=0.1, accumulate=True)
    assert c.cache.status() == DEV_BAD_ID
    assert (out[:2] == 0).all()
    assert np.abs(out.double().cpu().numpy()[2:] - ref[2:]).max() < 0.05


@pytest.mark.parametrize("dtype,rank,page", [("bf16", 128, 64), ("bf16", 8, 16), ("bf16", 256, 32),
                                             ("fp32", 256, 16), ("fp32", 36, 128)])
@pytest.mark.parametrize("norm", [False, True])
def test_append(dtype, rank, page, norm):
    lengths, new = [100, 0, 7, 128, 65, 3000], [100, 0, 3, 1, 0, 2999]
    c = Case(dtype, 2, rank, page, lengths, seed=9, stale=1.5)
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    x = torch.from_numpy(c.rng.standard_normal((int(off[-1]) + 2, rank)).astype(np.float32) * 3)
    x = x.to(DT[dtype]).cuda()
    gain = torch.from_numpy(1 + 0.1 * c.rng.standard_normal(rank).astype(np.float32))
    gain = gain.to(DT[dtype]).cuda() if norm else None
    pool, mass = c.host_pool(), c.host_mass()
    oc.append(pool, mass, x.double().cpu().numpy(), off, c.table, c.lengths,
              gain.double().cpu().numpy() if norm else None, 1e-5)
    for _ in range(2):                                # the same rows again change nothing
        c.cache.append(x, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"),
                       gain=gain, eps=1e-5)
        assert c.cache.status() == 0
        # the sum of squares: rank adds; its root, the quotient and two products: 4 more
        half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
        tol = (half + (rank + 8) * 2.0 ** -24) * np.abs(pool) if norm else 0.0 * pool
        close(c.pool, pool, tol, "pool")
        assert np.array_equal(c.host_mass(), mass)


def test_append_faults():
    c = Case("bf16", 2, 64, 16, [20, 20, 20], seed=9, stale=0.0)
    pool = c.pool.clone()
    x = torch.ones(9, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 3, 6, 9]).cuda()
    table = c.table.copy()
    table[0, 1] = c.n_pages                            # slots 17..19 lie in its second page
    lengths = c.lengths.copy()
    lengths[1] = 2                                     # fewer events than new rows
    c.cache.append(x, off, torch.from_numpy(table).cuda(), torch.from_numpy(lengths).cuda())
    assert c.cache.status() == DEV_BAD_ID | DEV_BAD_OFFSETS
    at = tuple(torch.from_numpy(a[17:]).cuda() for a in oc.slots(c.table[2], 20, 16))
    pool[at] = 1
    assert torch.equal(c.pool, pool)


def _evict_case(dtype, rank, page, lengths, seed, spare, ties):
    c = Case(dtype, 2, rank, page, lengths, seed=seed, spare=spare, stale=0.25)
    m = np.exp(2 * c.rng.standard_normal((c.n_pages, page))).astype(np.float32)
    if ties:
        m = np.floor(m)                                # many equal masses
        m[c.rng.random(m.shape) < 0.05] = np.nan
        m[c.rng.random(m.shape) < 0.05] = -0.0
        m[c.rng.random(m.shape) < 0.02] = np.inf
        m[c.rng.random(m.shape) < 0.05] *= -1
    c.mass.copy_(torch.from_numpy(m))
    return c


@pytest.mark.parametrize("dtype,rank,page", [("bf16", 128, 64), ("bf16", 256, 16),
                                             ("fp32", 32, 32), ("bf16", 40, 128)])
@pytest.mark.parametrize("budget,sink,recent", [(1, 0, 0), (1, 1, 0), (100, 4, 32), (128, 0, 0),
                                                (64, 30, 34), (300, 1, 299), (5000, 4, 4)])
@pytest.mark.parametrize("apart,ties", [(False, True), (True, False), (True, True)])
def test_evict(dtype, rank, page, budget, sink, recent, apart, ties):
    lengths = [0, 1, 5, 100, 101, 129, 513, 2100]
    need = sum(-(-min(n, budget) // page) for n in lengths)
    c = _evict_case(dtype, rank, page, lengths, 11, need, ties)
    dst = None
    if apart:
        free = list(c.free)
        dst = np.zeros((len(lengths), max(1, -(-min(max(lengths), budget) // page))), np.int32)
        if dst.shape[1] * page < min(budget, c.width * page):
            dst = np.zeros((len(lengths), -(-min(budget, c.width * page) // page)), np.int32)
        for u, n in enumerate(lengths):
            for i in range(-(-min(n, budget) // page)):
                dst[u, i] = free.pop()
    pool, mass = c.host_pool(), c.host_mass()
    new, kept = oc.evict(pool, mass, c.table, c.lengths, budget, sink, recent, dst)
    lens = c.dev("lengths")
    got_kept = torch.full((len(lengths), budget), -7, dtype=torch.int32, device="cuda")
    got = c.cache.evict(c.dev("table"), lens, budget, n_sink=sink, n_recent=recent,
                        dst_table=torch.from_numpy(dst).cuda() if apart else None, kept=got_kept,
                        new_lengths=lens if not apart else None)
    assert c.cache.status() == 0
    assert got.cpu().numpy().tolist() == new.tolist()
    for u, k in enumerate(kept):
        row = got_kept[u].cpu().numpy()
        assert row[:len(k)].tolist() == k and (row[len(k):] == -7).all()
    assert np.array_equal(c.host_pool(), pool)
    assert np.array_equal(c.host_mass(), mass, equal_nan=True)


def test_evict_long_history():
    # more events than one block's threads hold at once
    c = _evict_case("bf16", 64, 128, [70000, 33], 12, 0, True)
    pool, mass = c.host_pool(), c.host_mass()
    new, kept = oc.evict(pool, mass, c.table, c.lengths, 20000, 4, 128)
    got_kept = torch.zeros((2, 20000), dtype=torch.int32, device="cuda")
    got = c.cache.evict(c.dev("table"), c.dev("lengths"), 20000, n_sink=4, n_recent=128,
                        kept=got_kept)
    assert got.cpu().tolist() == new.tolist()
    assert got_kept[0].cpu().tolist() == kept[0]
    assert np.array_equal(c.host_pool(), pool)
    assert np.array_equal(c.host_mass(), mass, equal_nan=True)


def test_evict_faults():
    c = _evict_case("bf16", 64, 16, [40, 40, 40], 13, 0, False)
    pool, mass = c.host_pool(), c.host_mass()
    table, lengths = c.table.copy(), c.lengths.copy()
    lengths[0] = -5
    lengths[1] = 10 ** 6
    new = torch.full((3,), 77, dtype=torch.int32, device="cuda")
    oc.evict(pool, mass, c.table[2:], c.lengths[2:], 8)
    c.cache.evict(torch.from_numpy(table).cuda(), torch.from_numpy(lengths).cuda(), 8,
                  new_lengths=new)
    assert c.cache.status() == DEV_TOO_LONG
    assert new.cpu().tolist() == [77, 77, 8]
    assert np.array_equal(c.host_pool(), pool) and np.array_equal(c.host_mass(), mass)
    # a page outside the pool: nothing of it is read or written
    table[2, 0] = -1
    c.cache.evict(torch.from_numpy(table).cuda(), c.dev("lengths"), 8, new_lengths=new)
    assert c.cache.status() == DEV_BAD_ID


def test_refusals():
    c = Case("bf16", 4, 128, 64, [70, 130], seed=6, max_rows=8)
    q, off = c.queries([1, 1], 1)
    o, t, n = torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths")

    def arg(f, *a, **k):
        with pytest.raises(LlatteError) as e:
            f(*a, **k)
        assert e.value.code == LLATTE_ERR_ARG

    for k in (dict(n_cand=-1), dict(window=-1), dict(n_sink=-1), dict(scale=float("nan"))):
        arg(c.cache.attend, q, o, t, n, **k)
    big = torch.zeros(9, 4, 128, dtype=torch.bfloat16, device="cuda")
    arg(c.cache.attend, big, o, t, n)                       # more rows than max_rows
    for k in (dict(budget=0), dict(budget=4, n_sink=3, n_recent=2), dict(budget=4, n_sink=-1),
              dict(budget=4, n_recent=-1)):
        arg(c.cache.evict, t, n, **k)
    arg(c.cache.evict, t, n, 100, dst_table=t[:, :1].contiguous())      # 64 slots for 100 events
    arg(c.cache.append, torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda"),
        torch.tensor([0, 1, 2]).cuda(), t, n, gain=torch.ones(128, dtype=torch.bfloat16,
                                                            device="cuda"), eps=0.0)
    plain = LatentCache(c.pool, 4, max_batch=1, max_rows=8, max_pages=c.width)
    arg(plain.attend, q, o, t, n, accumulate=True)          # no masses, and more users than 1
    arg(plain.attend, q[:2].contiguous(), o[:2].contiguous(), t[:1].contiguous(),
        n[:1].contiguous(), accumulate=True)
    arg(plain.evict, t[:1].contiguous(), n[:1].contiguous(), 4)
    for bad in (q.float(), q[:, :3], q[:, :, :64], q.transpose(0, 1), q.cpu()):
        with pytest.raises(ValueError):
            c.cache.attend(bad, o, t, n)
    for o2, t2, n2 in ((o[:2], t, n), (o.int(), t, n), (o, t.long(), n), (o, t, n.long()),
                       (o, t[:, :1].expand(2, 4), n), (o, t.cpu(), n)):
        with pytest.raises(ValueError):
            c.cache.attend(q, o2, t2, n2)
    with pytest.raises(ValueError):
        c.cache.attend(q, o, t, n, out=torch.empty_like(q).float())
    with pytest.raises(ValueError):
        c.cache.evict(t, n, 8, kept=torch.zeros(2, 7, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        LatentCache(c.pool, 4, mass=c.mass[:, :3])
    assert c.cache.status() == 0


def test_empty_calls():
    c = Case("bf16", 4, 128, 64, [70], seed=6)
    t, n = c.dev("table"), c.dev("lengths")
    e = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    z = torch.zeros(2, dtype=torch.int64, device="cuda")
    assert c.cache.attend(e, z, t, n).shape == (0, 4, 128)
    c.cache.append(e[:, 0], z, t, n)
    none = torch.zeros(1, dtype=torch.int64, device="cuda")
    c.cache.attend(e, none, t[:0], n[:0])
    assert c.cache.evict(t[:0], n[:0], 4).shape == (0,)
    assert c.cache.status() == 0


def _session(cache, c, x, gain, q, off_x, off_q, table, n1, n2, kept):
    """Append, attend with weights, evict in place, append again, attend."""
    cache.append(x, off_x, table, n1, gain=gain)
    a = cache.attend(q, off_q, table, n1, n_cand=3, scale=0.1, accumulate=True)
    short = cache.evict(table, n1, 96, n_sink=2, n_recent=20, kept=kept)
    n2.copy_(short + 4)
    cache.append(x, off_x, table, n2, gain=gain)
    b = cache.attend(q, off_q, table, n2, n_cand=3, scale=0.1, window=50, n_sink=2,
                     accumulate=True)
    return a, b, short


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("fp32", 32)])
def test_a_session_eager_captured_and_on_another_stream(dtype, rank):
    B, h = 5, 4
    lengths = [300, 4, 97, 130, 260]
    c = Case(dtype, h, rank, 32, lengths, seed=20, stale=0.0, width=12)
    pool0, mass0 = c.pool.clone(), c.mass.clone()
    x = torch.from_numpy(c.rng.standard_normal((4 * B, rank)).astype(np.float32)).to(DT[dtype]).cuda()
    gain = torch.ones(rank, dtype=DT[dtype], device="cuda")
    q, off = c.queries([4] * B, 3)
    off_x = torch.arange(0, 4 * B + 1, 4).cuda()
    off_q = torch.from_numpy(off).cuda()
    table, n1 = c.dev("table"), c.dev("lengths")

    # the oracle's session, on the kernel's own stored rows where a rounding decides
    pool, mass = c.host_pool(), c.host_mass()
    oc.append(pool, mass, x.double().cpu().numpy(), off_x.cpu().numpy(), c.table, c.lengths,
              np.ones(rank))
    pool = torch.from_numpy(pool).to(DT[dtype]).double().numpy()
    ra, _ = oc.attend(pool, mass, q.double().cpu().numpy(), off, c.table, c.lengths, 3, 0.1)

    def state():
        c.pool.copy_(pool0)
        c.mass.copy_(mass0)
        return torch.zeros_like(n1), torch.full((B, 96), -1, dtype=torch.int32, device="cuda")

    n2, kept = state()
    a, b, short = _session(c.cache, c, x, gain, q, off_x, off_q, table, n1, n2, kept)
    torch.cuda.synchronize()
    assert c.cache.status() == 0
    # each step's result from the state the kernels left before it
    assert np.abs(a.double().cpu().numpy() - ra).max() < 0.05
    new, ref_kept = oc.evict(pool.copy(), mass.copy(), c.table, c.lengths, 96, 2, 20)
    assert short.cpu().tolist() == new.tolist() == [96, 4, 96, 96, 96]
    same = [len(set(k) & set(kept[u, :len(k)].cpu().tolist())) / len(k)
            for u, k in enumerate(ref_kept)]
    assert min(same) > 0.95                      # near ties may fall either way
    rb, _ = oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table,
                      n2.cpu().numpy(), 3, 0.1, 50, 2)
    assert np.abs(b.double().cpu().numpy() - rb).max() < 0.05
    want = a.clone(), b.clone(), c.pool.clone(), c.mass.clone(), kept.clone()

    # captured and replayed, twice
    n2, kept = state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ga, gb, _ = _session(c.cache, c, x, gain, q, off_x, off_q, table, n1, n2, kept)
    for _ in range(2):
        c.pool.copy_(pool0)
        c.mass.copy_(mass0)
        g.replay()
        torch.cuda.synchronize()
        for u, v in zip((ga, gb, c.pool, c.mass, kept), want):
            assert torch.equal(u, v)
    del g

    # on a stream given by hand
    n2, kept = state()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c.cache.append(x, off_x, table, n1, gain=gain, stream=s)
    oa = c.cache.attend(q, off_q, table, n1, n_cand=3, scale=0.1, accumulate=True, stream=s)
    s.synchronize()
    assert torch.equal(oa, want[0])


def test_two_caches_share_a_pool():
    # a pool whose pages belong to two layers, each with its own tables
    c = Case("bf16", 4, 128, 64, [300, 70], seed=30)
    other = LatentCache(c.pool, 4, max_batch=1, max_rows=64, max_pages=c.width)
    q, off = c.queries([2, 2], 0)
    tab, ln = c.dev("table"), c.dev("lengths")
    both = c.cache.attend(q, torch.from_numpy(off).cuda(), tab, ln, scale=0.1)
    s1 = torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    one = other.attend(q[:2].contiguous(), torch.tensor([0, 2]).cuda(), tab[:1].contiguous(),
                       ln[:1].contiguous(), scale=0.1)
    torch.cuda.synchronize()
    assert torch.equal(one, both[:2])
    other.close()


def test_many_users_and_long_rows():
    lengths = [int(n) for n in np.random.default_rng(1).integers(0, 60, 2000)]
    c = Case("bf16", 2, 64, 16, lengths, seed=40)
    check_attend(c, [1 if n else 0 for n in lengths], n_cand=1, accumulate=True)
