"""The forward pass over cached histories where it has to refuse or to leave a user
out: models whose layers drop rows, histories longer than the layers keep, and users
whose length or pages are wrong."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
import oracle.cache as oc
from latent_attention_jagged_b200 import LatentCache, Llatte, LlatteError
from latent_attention_jagged_b200.binding import (DEV_BAD_OFFSETS, DEV_TOO_LONG, LLATTE_ERR_ARG,
                                                  LLATTE_ERR_UNSUPPORTED)
from oracle.model import rmsnorm, silu

from gpu_harness import assert_close
from test_forward_cached_gpu import Served, _inputs

pytestmark = pytest.mark.gpu


def _first_events(inp, lengths):
    """The same users and weights, with the first `lengths` events only."""
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    values = np.concatenate([inp.values[int(a):int(a) + n] for a, n in zip(inp.offsets, lengths)])
    return dataclasses.replace(inp, lengths=np.asarray(lengths, np.int64), offsets=off,
                               values=values)


def _events(s, first, last):
    rows = [s.inp.values[int(s.inp.offsets[u]) + a:int(s.inp.offsets[u]) + b]
            for u, (a, b) in enumerate(zip(first, last))]
    values = torch.from_numpy(np.concatenate(rows)).cuda().to(s.dt).contiguous()
    return values, torch.tensor([0] + list(np.cumsum([len(r) for r in rows]))).cuda()


def _call(s, first, last, lengths=None, table=None, **kw):
    """A request without the checks of the status words."""
    values, off = _events(s, first, last)
    ln = torch.tensor(last if lengths is None else lengths, dtype=torch.int32).cuda()
    return s.h.forward_cached(values, off, s.caches, s.table_d if table is None else table, ln,
                              context=s.ctx, cand=s.cand, **kw)


@pytest.mark.parametrize("dtype,kw", [("bf16", dict(rank=64)), ("fp32", dict(rank=32))])
def test_a_model_whose_layers_drop_rows_is_refused(dtype, kw):
    # the handle takes 16 new events at most, every layer keeps more than that, but the
    # caches hold histories that the whole-history pass would cut
    inp = _inputs(dtype, lengths=[120, 40], keep=(100, 60), **kw)
    s = Served(inp, max_new=16)
    with pytest.raises(LlatteError) as e:
        _call(s, [110, 30], [120, 40])
    assert e.value.code == LLATTE_ERR_UNSUPPORTED
    # the same model over caches of no more events than its layers keep
    short = [LatentCache(c.pool, inp.dims.heads, mass=c.mass, max_batch=2,
                         max_rows=s.h.query_rows(), max_pages=2) for c in s.caches]
    s.caches = short
    for a in range(0, 60, 15):
        at = [a, min(a, 33)], [a + 15, min(a + 15, 33)]
        out = _call(s, *at)
    torch.cuda.synchronize()
    assert s.h.status() == 0 and all(c.status() == 0 for c in s.caches)
    assert_close(out.double().cpu().numpy(), oracle.forward(_first_events(inp, [60, 33])), dtype,
                 "no more events than the layers keep")


def test_a_history_longer_than_the_layers_keep_is_left_out():
    # 10 pages of 32 events hold 320, the layers keep 300
    inp = _inputs(lengths=[320, 50])
    s = Served(inp, max_new=40)
    n = [0, 0]
    while n != [300, 50]:
        last = [min(n[0] + 40, 300), min(n[1] + 40, 50)]
        out = _call(s, n, last)
        n = last
    torch.cuda.synchronize()
    assert s.h.status() == 0 and all(c.status() == 0 for c in s.caches)
    ref = oracle.forward(_first_events(inp, [300, 50]))
    assert_close(out.double().cpu().numpy(), ref, "bf16", "as many events as the layers keep")
    pools = [c.pool.clone() for c in s.caches]
    out = _call(s, [300, 50], [301, 50]).double().cpu().numpy()
    assert s.h.status() == 0 and all(c.status() == DEV_TOO_LONG for c in s.caches)
    assert all(torch.equal(c.pool, p) for c, p in zip(s.caches, pools))     # nothing appended
    assert np.abs(out[0] - _without_attention(inp, 0)).max() < 0.03
    assert_close(out[1:], ref[1:], "bf16", "the user beside it")


def _without_attention(inp, u):
    """fp64 layers of a user's query tokens when the attention gives zeros."""
    D, Y = inp.dims, inp.cand[u].astype(np.float64)
    for w in inp.layers:
        f = {k: np.asarray(v, np.float64) for k, v in w.items() if v is not None}
        Z = rmsnorm(Y, f["g1"], D.eps)
        Y = rmsnorm(Z + silu(Z @ f["W1"].T) @ f["W2"].T, f["g2"], D.eps)
    return Y


@pytest.mark.parametrize("dtype,kw", [
    ("bf16", {}), ("bf16", dict(rank=40)), ("fp32", dict(rank=32))])
@pytest.mark.parametrize("max_new", [2, 60])
def test_rows_of_a_user_left_out_hold_nothing_of_earlier_calls(dtype, kw, max_new):
    # a handle for a few new rows (the form for single tokens) and one for many
    if max_new == 2:
        kw = dict(kw, n_q=2, heads=2, d_head=64)
    inp = _inputs(dtype, lengths=[60, 80, 50, 33], **kw)
    n = [int(x) for x in inp.lengths]
    old = [x - 2 for x in n]
    s = Served(inp, max_new=max_new)
    a = [0] * 4
    while a != old:
        b = [min(x + max_new, y) for x, y in zip(a, old)]
        _call(s, a, b)
        a = b
    wrong = list(n)
    wrong[1], wrong[2] = 1 << 20, 1             # beyond its pages; fewer than its new rows
    outs = []
    for before in (old, [x - 1 for x in old]):  # two calls that leave other rows behind
        s.cand.mul_(-1)
        _call(s, before, [x + 1 for x in before])
        s.cand.copy_(torch.from_numpy(inp.cand).cuda().to(s.dt))
        torch.cuda.synchronize()
        assert s.h.status() == 0 and all(c.status() == 0 for c in s.caches)
        outs.append(_call(s, old, n, lengths=wrong))
        torch.cuda.synchronize()
        assert all(c.status() == DEV_TOO_LONG | DEV_BAD_OFFSETS for c in s.caches)
        assert s.h.status() == 0
    assert torch.equal(outs[0], outs[1])
    got = outs[0].double().cpu().numpy()
    tol = 0.03 if dtype == "bf16" else 1e-4
    for u in (1, 2):
        assert np.abs(got[u] - _without_attention(inp, u)).max() < tol
    ref = oracle.forward(inp)
    assert_close(got[[0, 3]], ref[[0, 3]], dtype, "users beside those left out")


@pytest.mark.parametrize("dtype,kw", [
    ("bf16", {}), ("bf16", dict(rank=128, heads=2, d_head=64)), ("fp32", dict(rank=32, n_q=1)),
    ("bf16", dict(d=512, heads=8, d_head=64, rank=256, n_q=1))])
def test_single_events_on_a_handle_for_single_events(dtype, kw):
    # one new event and few query tokens a user: the attention's form for single tokens
    inp = _inputs(dtype, **dict(dict(n_q=2), **kw))
    big = Served(inp)
    n = np.asarray(inp.lengths)
    old = [int(x) for x in np.maximum(n - 1, 0)]
    big.request([0] * len(n), old, accumulate=True)
    h = Llatte(inp.dims, inp.layers, None, max_batch=len(n), max_len=1)
    caches = [LatentCache(c.pool, inp.dims.heads, mass=c.mass, max_batch=len(n),
                          max_rows=h.query_rows(), max_pages=big.table.shape[1])
              for c in big.caches]
    big.h, big.caches = h, caches
    before = [c.mass.double().sum().item() for c in caches]
    out = big.request(old, [int(x) for x in n], accumulate=True)
    assert_close(out, oracle.forward(inp), dtype, f"single events {kw}")
    rows = sum(inp.dims.n_q + 1 for x in n if x)
    for c, b in zip(caches, before):             # every row that sees an event spends 1 a head
        spent = c.mass.double().sum().item() - b
        assert abs(spent - inp.dims.heads * rows) < 1e-3 * inp.dims.heads * rows


def test_two_layers_may_not_write_the_same_pages():
    inp = _inputs(lengths=[40, 7])
    s = Served(inp, max_new=40)
    one = s.caches
    s.caches = [one[0], one[0]]
    with pytest.raises(LlatteError) as e:
        _call(s, [0, 0], [40, 7])
    assert e.value.code == LLATTE_ERR_ARG
    twin = LatentCache(one[0].pool, inp.dims.heads, max_batch=2, max_rows=s.h.query_rows(),
                       max_pages=s.table.shape[1])
    s.caches = [one[0], twin]                    # another cache over the same pool and table
    with pytest.raises(LlatteError) as e:
        _call(s, [0, 0], [40, 7])
    assert e.value.code == LLATTE_ERR_ARG
    # one cache for both layers, whose tables name other pages
    both = torch.zeros(2 * one[0].n_pages, 32, 64, dtype=torch.bfloat16, device="cuda")
    c = LatentCache(both, inp.dims.heads, max_batch=2, max_rows=s.h.query_rows(),
                    max_pages=s.table.shape[1])
    s.caches = [c, c]
    out = _call(s, [0, 0], [40, 7], table=[s.table_d, s.table_d + one[0].n_pages])
    torch.cuda.synchronize()
    assert s.h.status() == 0 and c.status() == 0
    assert_close(out.double().cpu().numpy(), oracle.forward(inp), "bf16", "one pool, two layers")


def test_the_same_request_again():
    # the same result; older events are counted a second time, the new ones start over
    inp = _inputs(lengths=[130, 40])
    s = Served(inp)
    s.request([0, 0], [100, 39])
    first = s.request([100, 39], [130, 40], accumulate=True)
    once = [c.mass.double() for c in s.caches]
    again = s.request([100, 39], [130, 40], accumulate=True)
    assert np.array_equal(first, again)
    for c, m in zip(s.caches, once):
        for u, (old, n) in enumerate(((100, 130), (39, 40))):
            at = tuple(torch.from_numpy(x).cuda() for x in oc.slots(s.table[u], n, s.page))
            was, now = m[at], c.mass.double()[at]
            assert torch.allclose(now[:old], 2 * was[:old], rtol=1e-5, atol=0)
            assert torch.allclose(now[old:], was[old:], rtol=1e-5, atol=0)
            assert (was > 0).all()
