"""The forward pass over cached histories where it has to refuse or to leave a user
out: models whose layers drop rows, and histories longer than the layers keep."""
import dataclasses

import numpy as np
import pytest
import torch

import oracle
from latent_attention_jagged_b200 import LatentCache, LlatteError
from latent_attention_jagged_b200.binding import DEV_TOO_LONG, LLATTE_ERR_UNSUPPORTED

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
    assert_close(out[1:], ref[1:], "bf16", "the user beside it")
