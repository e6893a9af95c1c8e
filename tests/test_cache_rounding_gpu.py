"""What the rounding of softmax weights costs the tensor-core form of single tokens (bf16).

Up to 8 (row, head) pairs a block carries every weight as a bf16 number and a bf16 rest:
rounding the first leaves at most 2^-8 of it, rounding that at most 2^-8 of the rest,
2^-16 together.  A block of 9 to 16 pairs carries one bf16 number w' = w (1 + d),
|d| <= 2^-8, and divides by the sum of the rounded numbers:
    sum w' c / sum w' - sum w c / sum w = sum w d (c - o) / sum w',
at most 2^-8 (1 + 2^-7) sum_t P_t |c_t - o|, which vanishes as one event takes all
weight.  A block summed from parts divides part by part, each around its own mean: that
sum is at most twice the one around o."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from cache_harness import Case, attend_bounds, close, dot_error

pytestmark = pytest.mark.gpu

ROUNDED = 2 * 2.0 ** -8 * (1 + 2.0 ** -7)


def _run(c, q, off, n_cand, scale, window=0, n_sink=0):
    sp = {}
    ref, ref_lse = oc.attend(c.host_pool(), None, q.double().cpu().numpy(), off, c.table, c.lengths,
                             n_cand, scale, window, n_sink, sp)
    lse = torch.empty(q.shape[:2], device="cuda")
    out = c.cache.attend(q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"),
                         n_cand=n_cand, scale=scale, window=window, n_sink=n_sink, lse=lse)
    assert c.cache.status() == 0
    return out, lse, ref, ref_lse, sp


def _bound(c, sp, ref, spread, weight):
    """|out - exact|: the scores and sums (see attend_bounds), `weight` of what the
    rounded weights are spread over, and the result's own rounding."""
    T = int(c.lengths.max())
    rel = 2 * dot_error(c.rank, sp["dot"]) + 2.0 ** -22 + (2 * T + 16) * 2.0 ** -24
    return (sp["abs"] * 2 * rel[..., None] + weight * spread + 2.0 ** -8 * np.abs(ref)) \
        * (1 + 2.0 ** -6)


def _spread(c, q, off, n_cand, scale, ref, window=0, n_sink=0):
    """sum_t P_t |c_t - o| of every row and head."""
    pool, res = c.host_pool(), np.zeros(ref.shape)
    qd = q.double().cpu().numpy()
    for u in range(len(c.lengths)):
        a, b = int(off[u]), int(off[u + 1])
        cand = min(n_cand, b - a)
        see = oc.visible(b - a - cand, cand, int(c.lengths[u]), window, n_sink)
        ct = pool[oc.slots(c.table[u], int(c.lengths[u]), c.page)]
        for i in range(a, b):
            k = np.flatnonzero(see[i - a])
            if len(k):
                s = scale * (qd[i] @ ct[k].T)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                res[i] = np.einsum("ht,htr->hr", p, np.abs(ct[k][None] - ref[i][:, None]))
    return res


def _check(c, q, off, n_cand, scale, window=0, n_sink=0):
    out, lse, ref, ref_lse, sp = _run(c, q, off, n_cand, scale, window, n_sink)
    if c.heads <= 8:
        bound = _bound(c, sp, ref, sp["abs"], 2.0 ** -16)
    else:
        bound = _bound(c, sp, ref, _spread(c, q, off, n_cand, scale, ref, window, n_sink), ROUNDED)
    close(out, ref, bound, "out")
    T = int(c.lengths.max())
    close(lse, ref_lse, attend_bounds("bf16", c.rank, T, sp, ref, ref_lse)[1], "lse")
    return ref


@pytest.mark.parametrize("rank", [64, 128, 256])
@pytest.mark.parametrize("heads", [1, 4, 8, 9, 11, 16])
@pytest.mark.parametrize("window,sink", [(0, 0), (100, 4)])
def test_single_tokens(rank, heads, window, sink):
    c = Case("bf16", heads, rank, 64, [1, 17, 128, 129, 4000, 1000, 333], seed=90)
    q, off = c.queries([1] * 7, 0)
    _check(c, q, off, 0, rank ** -0.5, window, sink)


@pytest.mark.parametrize("rank", [64, 128, 256])
@pytest.mark.parametrize("heads", [2, 11])
def test_maxima_that_grow_within_and_beyond_a_base(rank, heads):
    # scores rise by 6 (8.7 in log2 units) every 64 events: some steps keep the base
    n = 900
    c = Case("bf16", heads, rank, 32, [n], seed=93)
    at = tuple(torch.from_numpy(x).cuda() for x in oc.slots(c.table[0], n, 32))
    c.pool[at[0], at[1], 0] = (torch.arange(n) // 64).to(torch.bfloat16).cuda()
    q, off = c.queries([1], 0)
    q[..., 0] = 6.0 * 16
    q[..., 1:] *= 0.05
    _check(c, q, off, 0, 1 / 16)


@pytest.mark.parametrize("rank", [64, 128, 256])
@pytest.mark.parametrize("heads", [2, 11])
def test_one_event_takes_all_weight(rank, heads):
    # the last event of every history scores 10.1 to 10.4 above the others (14.6 to 15 in
    # log2 units, within the growth that keeps a sum's base): the result is its latent
    for gain in (10.1, 10.2, 10.3, 10.4):
        c = Case("bf16", heads, rank, 32, [200, 500], seed=92)
        for u, n in enumerate((200, 500)):
            at = tuple(torch.from_numpy(x).cuda() for x in oc.slots(c.table[u], n, 32))
            c.pool[at[0], at[1], 0] = 0.0
            c.pool[at[0][-1], at[1][-1], 0] = 1.0
        q, off = c.queries([0, 0], 1)
        q.zero_()
        q[..., 0] = 1.0
        ref = _check(c, q, off, 1, gain)
        assert _spread(c, q, off, 1, gain, ref)[..., 1:].max() < 0.5   # latents of up to 3
