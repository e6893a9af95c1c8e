"""GPU parity of the paged cache's kernels where they switch, cut and join: blocks of
pairs that fill, end inside and pass the tensor-core blocks, blocks cut between
SMs, maxima that outgrow a sum's base, every sign of the scale, hidden values next
to single tokens, pages that are gone, pages that users share, and the largest
batch.  Bounds as in cache_harness."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from cache_harness import DT, Case, attend_bounds, check_attend, close, mass_bound
from latent_attention_jagged_b200 import LatentCache, LlatteError
from latent_attention_jagged_b200.binding import DEV_BAD_ID, LLATTE_ERR_ARG

pytestmark = pytest.mark.gpu

KINDS = [("bf16", 64), ("bf16", 128), ("bf16", 256), ("bf16", 40), ("fp32", 32), ("fp32", 256)]


@pytest.mark.parametrize("dtype,rank", KINDS)
@pytest.mark.parametrize("heads,page", [(1, 16), (3, 32), (4, 128)])
def test_blocks_of_pairs(dtype, rank, heads, page):
    # pairs: 1 .. 16 (one block of the token kernel), 31 .. 33 (a quadrant), 127 .. 129
    # (a block), several blocks; together they take the kernel of long blocks
    new = [1, 5, 11, 32, 33, 43, 128, 150]
    lengths = [64, 65, 127, 128, 129, 300, 256, 190]
    c = Case(dtype, heads, rank, page, lengths, seed=50)
    check_attend(c, new, n_cand=1, accumulate=True)


@pytest.mark.parametrize("dtype,rank", KINDS)
@pytest.mark.parametrize("pairs", [1, 7, 8, 9, 16])
def test_few_pairs(dtype, rank, pairs):
    lengths = [1, 15, 16, 17, 128, 129, 700, 0]
    c = Case(dtype, pairs, rank, 64, lengths, seed=51)
    check_attend(c, [1] * 7 + [0], accumulate=True, window=0)
    check_attend(c, [1] * 7 + [0], window=20, n_sink=2, accumulate=True)


@pytest.mark.parametrize("dtype,rank", KINDS)
@pytest.mark.parametrize("new", [1, 40])
def test_one_long_history_is_cut_between_sms(dtype, rank, new):
    c = Case(dtype, 4, rank, 64, [9000], seed=52)
    check_attend(c, [new], accumulate=True)
    check_attend(c, [new], window=5000, n_sink=300, accumulate=True)


@pytest.mark.parametrize("dtype,rank", KINDS)
@pytest.mark.parametrize("rows", [2, 70])
def test_maxima_outgrow_the_base(dtype, rank, rows):
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
    ref, ref_lse = oc.attend(c.host_pool(), mass, q.double().cpu().numpy(), off, c.table,
                             c.lengths, 0, scale, 0, 0, sp)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"),
                         scale=scale, lse=lse, accumulate=True)
    b_out, b_lse = attend_bounds(dtype, rank, n, sp, ref, ref_lse)
    close(out, ref, b_out, "out")
    close(lse, ref_lse, b_lse, "lse")


@pytest.mark.parametrize("dtype,rank", KINDS)
@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30])
@pytest.mark.parametrize("new", [1, 50])
def test_any_scale(dtype, rank, scale, new):
    c = Case(dtype, 3, rank, 32, [200, 129], seed=54)
    check_attend(c, [new, new], n_cand=1, scale=scale, accumulate=True)
    check_attend(c, [new, new], n_cand=1, scale=scale, window=70, n_sink=5)


@pytest.mark.parametrize("dtype,rank", KINDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_hidden_values_next_to_a_single_token(dtype, rank, value):
    c = Case(dtype, 4, rank, 32, [200, 90, 130], seed=55)
    q, off = c.queries([1, 1, 1], 0)
    args = (q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"))
    kw = dict(scale=0.1, window=60, n_sink=3)
    clean = c.cache.attend(*args, **kw).clone()
    for u, t in ((0, 100), (0, 3), (1, 20), (2, 129)):
        c.pool[int(c.table[u][t // 32]), t % 32] = value
    lse = torch.empty(q.shape[:2], device="cuda")
    before = c.mass.clone()
    got = c.cache.attend(*args, lse=lse, accumulate=True, **kw)
    assert torch.equal(got[:2], clean[:2]) and torch.isfinite(lse[:2]).all()
    assert not torch.isfinite(got[2]).any()
    # the weights of the users that see nothing bad are those of a clean cache
    for u in (0, 1):
        pages = torch.from_numpy(c.table[u][:-(-int(c.lengths[u]) // 32)]).long().cuda()
        added = (c.mass[pages] - before[pages]).double().sum().item()
        assert abs(added - 4.0) < 1e-3


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("bf16", 256), ("bf16", 64), ("fp32", 64)])
def test_rows_behind_the_last_user_stay(dtype, rank):
    # full and partial quadrants of a block, rows before the first and after the last
    c = Case(dtype, 4, rank, 64, [300, 150], seed=56)
    q, off = c.queries([40, 9], 1, first=2, behind=3)
    out, lse = torch.full_like(q, 3.0), torch.full(q.shape[:2], 3.0, device="cuda")
    c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"), n_cand=1,
                   scale=0.1, out=out, lse=lse)
    sp = {}
    ref, ref_lse = oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table,
                             c.lengths, 1, 0.1, 0, 0, sp)
    b_out, b_lse = attend_bounds(dtype, rank, 300, sp, ref, ref_lse)
    for t in (out, lse):
        assert (t[:2] == 3).all() and (t[53:] == 3).all()
    close(out[2:53], ref[2:53], b_out[2:53], "out")
    close(lse[2:53], ref_lse[2:53], b_lse[2:53], "lse")


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("bf16", 40), ("fp32", 32)])
@pytest.mark.parametrize("new", [1, 30])
def test_pages_outside_every_window_may_be_gone(dtype, rank, new):
    c = Case(dtype, 4, rank, 16, [500, 64], seed=57)
    q, off = c.queries([new, new], 0)
    kw = dict(scale=0.1, window=50, n_sink=20, accumulate=True)
    off = torch.from_numpy(off).cuda()
    want = c.cache.attend(q, off, c.dev("table"), c.dev("lengths"), **kw)
    mass = c.mass.clone()
    gone = c.table.copy()
    # user 0: the first 20 events lie in pages 0 and 1, its windows begin at event
    # 500 - new - 49 or later
    gone[0, 2:(500 - new - 49) // 16] = -7
    got = c.cache.attend(q, off, torch.from_numpy(gone).cuda(), c.dev("lengths"), **kw)
    assert c.cache.status() == 0
    assert torch.equal(got, want)
    added, again = mass, c.mass
    assert torch.isfinite(again).all() and (again >= added - 1e-6).all()
    gone[0, 1] = -7                                # a page of the first events
    c.cache.attend(q, off, torch.from_numpy(gone).cuda(), c.dev("lengths"), **kw)
    assert c.cache.status() == DEV_BAD_ID


@pytest.mark.parametrize("dtype,rank", [("bf16", 128), ("fp32", 64)])
def test_users_may_share_pages(dtype, rank):
    # two users with the same first pages, each with its own last one
    c = Case(dtype, 4, rank, 32, [100, 100], seed=58)
    table = c.table.copy()
    table[1, :3] = table[0, :3]
    for new in (1, 40):
        q, off = c.queries([new, new], 2)
        mass = c.host_mass()
        sp = {}
        ref, ref_lse = oc.attend(c.host_pool(), mass, q.double().cpu().numpy(), off, table,
                                 c.lengths, 2, 0.1, 0, 0, sp)
        out = c.cache.attend(q, torch.from_numpy(off).cuda(), torch.from_numpy(table).cuda(),
                             c.dev("lengths"), n_cand=2, scale=0.1, accumulate=True)
        b_out, _ = attend_bounds(dtype, rank, 100, sp, ref, ref_lse)
        close(out, ref, b_out, "out")
        # what a user adds rounds once more when it meets the other's
        close(c.mass, mass, mass_bound(rank, 100, sp, mass) + 2.0 ** -24 * np.abs(mass), "mass")


def test_the_largest_batch():
    B = 4096
    lengths = [int(n) for n in np.random.default_rng(2).integers(0, 40, B)]
    lengths[4095] = 700
    c = Case("bf16", 1, 64, 16, lengths, seed=59, max_rows=2 * B)
    check_attend(c, [1 if n else 0 for n in lengths], accumulate=True)
    x = torch.ones(B, 64, dtype=torch.bfloat16, device="cuda")
    off = torch.from_numpy(np.concatenate([[0], np.cumsum([1 if n else 0 for n in lengths])])).cuda()
    c.cache.append(x, off, c.dev("table"), c.dev("lengths"))
    for u in (0, 1000, 4094, 4095):
        if lengths[u]:
            t = lengths[u] - 1
            assert (c.pool[int(c.table[u][t // 16]), t % 16] == 1).all()
    assert c.cache.status() == 0


def test_two_caches_at_once_on_two_streams():
    # caches do not share workspaces: calls on two of them may overlap
    c = [Case("bf16", 4, 128, 64, [3000, 200], seed=60 + i) for i in range(2)]
    qs = [x.queries([1, 1], 0) for x in c]
    want = [x.cache.attend(q, torch.from_numpy(o).cuda(), x.dev("table"), x.dev("lengths"),
                           scale=0.1).clone() for x, (q, o) in zip(c, qs)]
    args = [(q, torch.from_numpy(o).cuda(), x.dev("table"), x.dev("lengths"))
            for x, (q, o) in zip(c, qs)]
    outs = [torch.zeros_like(q) for q, _ in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in c]
    for _ in range(20):
        for x, a, o, s in zip(c, args, outs, streams):
            x.cache.attend(*a, scale=0.1, out=o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_a_closed_cache_refuses():
    c = Case("bf16", 4, 128, 64, [70], seed=62)
    q, off = c.queries([1], 0)
    extra = LatentCache(c.pool, 4, max_batch=1, max_rows=4, max_pages=2)
    extra.close()
    with pytest.raises(LlatteError):
        extra.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"))


def test_the_result_may_not_replace_the_queries():
    c = Case("bf16", 4, 128, 64, [70], seed=63)
    q, off = c.queries([1], 0)
    with pytest.raises(LlatteError) as e:
        c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"), out=q)
    assert e.value.code == LLATTE_ERR_ARG
