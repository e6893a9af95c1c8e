"""Shared helpers of the paged-cache tests: seeded caches on the device, their
fp64 copies, and error bounds derived from the roundings a kernel makes."""
from __future__ import annotations

import numpy as np
import torch

import oracle.cache as oc
from latent_attention_jagged_b200 import LatentCache

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


class Case:
    """A pool with shuffled pages, a page table for users of the given lengths
    (and `spare` more pages), random latents everywhere a user has an event.
    Rows no event lies in hold `stale` (NaN unless told otherwise)."""

    def __init__(self, dtype, heads, rank, page, lengths, seed=0, spare=0, width=None,
                 stale=float("nan"), max_rows=4096, max_pages=None):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.heads, self.rank, self.page = rng, dtype, heads, rank, page
        self.lengths = np.asarray(lengths, np.int32)
        counts = [-(-int(n) // page) for n in lengths]
        self.width = width or max(1, max(counts, default=1))
        self.n_pages = max(1, sum(counts) + spare)
        ids = list(rng.permutation(self.n_pages))
        self.table = np.zeros((len(lengths), self.width), np.int32)
        for u, n in enumerate(counts):
            self.table[u, :n] = [ids.pop() for _ in range(n)]
        self.free = [int(i) for i in ids]
        pool = torch.full((self.n_pages, page, rank), stale, dtype=DT[dtype])
        for u in range(len(lengths)):
            at = oc.slots(self.table[u], int(lengths[u]), page)
            pool[at] = torch.from_numpy(
                rng.standard_normal((int(lengths[u]), rank)).astype(np.float32)).to(DT[dtype])
        self.pool = pool.cuda()
        self.mass = torch.from_numpy(rng.random((self.n_pages, page)).astype(np.float32)).cuda()
        self.cache = LatentCache(self.pool, heads, mass=self.mass, max_batch=max(1, len(lengths)),
                                 max_rows=max_rows, max_pages=max_pages or self.width)

    def dev(self, name):
        return torch.from_numpy(np.ascontiguousarray(getattr(self, name))).cuda()

    def host_pool(self):
        return self.pool.double().cpu().numpy()

    def host_mass(self):
        return self.mass.double().cpu().numpy()

    def queries(self, new, n_cand, sharp=2.0, first=0, behind=0):
        """(q on the device, offsets): `new` events per user, then n_cand tokens."""
        n = np.asarray(new) + n_cand
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int64) + first
        q = self.rng.standard_normal((int(off[-1]) + behind, self.heads, self.rank)) * sharp
        return torch.from_numpy(q.astype(np.float32)).to(DT[self.dtype]).cuda(), off


def dot_error(rank, dot):
    """A score's error: `rank` products accumulated in fp32, each add off by at
    most one fp32 step (2^-23, accumulators that truncate included) of a partial
    sum no larger than `dot`, plus four for the scaling and the exponent's
    argument."""
    return (rank + 4) * 2.0 ** -23 * dot


def attend_bounds(dtype, rank, lengths_max, sp, out, lse):
    """Elementwise bounds of |out - exact| and |lse - exact|.

    A weight exp(s - m) is off by the score's error twice (s and the maximum it
    is taken from cancel only in exact arithmetic), the exponential (2^-22) and,
    on the tensor cores, one bf16 rounding before the product with c (half a
    step: 2^-8).  Sums over at most T events and the rescaling of running sums add
    (2 T + 16) half steps of fp32.  The result is rounded once."""
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    ds = dot_error(rank, sp["dot"])
    rel = 2 * ds + 2.0 ** -22 + (2 * lengths_max + 16) * 2.0 ** -24
    p_round = 2.0 ** -8 if dtype == "bf16" else 0.0
    b_out = (sp["abs"] * (2 * rel[..., None] + p_round) + half * np.abs(out)) * (1 + 2.0 ** -6)
    fin = np.where(np.isfinite(lse), lse, 0.0)
    b_lse = rel + 2.0 ** -22 * (np.abs(fin) + 1) + 1e-30
    return b_out, b_lse


def mass_bound(rank, lengths_max, sp, mass):
    """Bound of |mass - exact|: every added weight is off by the relative error of
    a weight over its row's sum, and the sum over the rows that see the event
    rounds at most once per row and head."""
    rel = 4 * dot_error(rank, sp["maxdot"]) + 2.0 ** -21 + (2 * lengths_max + 16) * 2.0 ** -24
    return sp["got"] * rel + (sp["hits"] + 4) * 2.0 ** -24 * np.abs(mass) + 1e-30


def check_attend(case, new, n_cand=0, scale=None, window=0, n_sink=0, accumulate=False,
                 sharp=2.0, **kw):
    """One attend call against the oracle; returns (out, lse, the queries, offsets)."""
    scale = case.rank ** -0.5 if scale is None else scale
    q, off = case.queries(new, n_cand, sharp)
    pool, mass = case.host_pool(), case.host_mass()
    sp = {}
    ref, ref_lse = oc.attend(pool, mass if accumulate else None, q.double().cpu().numpy(), off,
                             case.table, case.lengths, n_cand, scale, window, n_sink, sp)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = case.cache.attend(q, torch.from_numpy(off).cuda(), case.dev("table"),
                            case.dev("lengths"), n_cand=n_cand, scale=scale, window=window,
                            n_sink=n_sink, lse=lse, accumulate=accumulate, **kw)
    torch.cuda.synchronize()
    assert case.cache.status() == 0
    T = int(case.lengths.max(initial=1))
    b_out, b_lse = attend_bounds(case.dtype, case.rank, T, sp, ref, ref_lse)
    close(out, ref, b_out, "out")
    close(lse, ref_lse, b_lse, "lse")
    if accumulate:
        close(case.mass, mass, mass_bound(case.rank, T, sp, mass), "mass")
    return out, lse, q, off


def close(got, ref, bound, what):
    got = got.double().cpu().numpy()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what
    same = np.where(inf, 0.0, ref)
    err = np.abs(np.where(inf, 0.0, got) - same)
    bad = ~(err <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, first at "
                           f"{np.argwhere(bad)[0]}: {got[bad][0]} for {ref[bad][0]}, bound "
                           f"{np.broadcast_to(bound, ref.shape)[bad][0]:.3e}")
