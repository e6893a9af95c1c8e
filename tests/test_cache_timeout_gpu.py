"""Failure detection in the paged cache's tensor-core kernels, without a fault: a wait is
made to run out (20 us limit) in every CTA that has work.  The call must return and
report the timeout, and the next call, on the same cache and in its workspace, must
give the same bits as one before it, also where blocks are summed from parts."""
import ctypes

import pytest
import torch

from cache_harness import Case
from latent_attention_jagged_b200 import LlatteError, binding

pytestmark = pytest.mark.gpu

# lengths, new events, query tokens, heads
FORMS = {
    "many rows, blocks cut": ([3000, 40, 900], [70, 20, 33], 3, 4),
    "many rows, short blocks": ([100, 64, 33, 90], [40, 20, 33, 9], 2, 4),
    "single tokens, blocks cut": ([20000, 700, 0, 5], [1, 1, 0, 1], 0, 8),
    "single tokens, short blocks": ([100, 64, 33, 90], [1, 1, 1, 1], 0, 4),
}


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rank", [64, 128, 256])
@pytest.mark.parametrize("form", list(FORMS))
def test_a_wait_that_runs_out_is_reported_and_the_cache_recovers(form, rank, accumulate):
    lengths, new, cand, heads = FORMS[form]
    c = Case("bf16", heads, rank, 64, lengths, seed=77)
    q, off = c.queries(new, cand)
    args = (q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"))
    mass0 = c.mass.clone()

    def call():
        c.mass.copy_(mass0)
        lse = torch.empty(q.shape[:2], device="cuda")
        out = c.cache.attend(*args, n_cand=cand, scale=0.1, lse=lse, accumulate=accumulate)
        torch.cuda.synchronize()
        return out, lse, c.mass.clone()

    good = call()
    assert c.cache.status() == 0
    for _ in range(3):
        c.cache.inject_timeout(True)
        call()
        assert c.cache.status() == binding.DEV_TIMEOUT
        c.cache.inject_timeout(False)
        again = call()
        assert c.cache.status() == 0
        assert all(torch.equal(a, b) for a, b in zip(good, again))


def test_append_and_eviction_go_on_beside_an_injection():
    c = Case("bf16", 4, 128, 64, [300, 90], seed=78, stale=0.0)
    c.cache.inject_timeout(True)
    new = c.cache.evict(c.dev("table"), c.dev("lengths"), 64)
    assert new.cpu().tolist() == [64, 64] and c.cache.status() == 0
    c.cache.inject_timeout(False)


def test_injection_needs_the_tensor_cores():
    c = Case("fp32", 4, 32, 64, [70], seed=79)
    with pytest.raises(LlatteError) as e:
        c.cache.inject_timeout(True)
    assert e.value.code == binding.LLATTE_ERR_UNSUPPORTED
    lib = c.cache.lib
    t = Case("bf16", 4, 64, 64, [70], seed=79)
    for n in (-1, 2, 1 << 30):
        assert lib.llatte_cache_inject_timeout(t.cache.h, n) == binding.LLATTE_ERR_ARG
    assert lib.llatte_cache_inject_timeout(ctypes.c_void_p(), 1) == binding.LLATTE_ERR_ARG
