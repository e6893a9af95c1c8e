"""GPU parity of the forward pass over cached histories: new events in several
requests against the oracle's one pass over the whole histories (a model whose
layers keep every row), windowed and evicted caches against per-layer attention
over what is left, and the call's refusals."""
import numpy as np
import pytest
import torch

import oracle
import oracle.cache as oc
from latent_attention_jagged_b200 import LatentCache, Llatte, LlatteError
from latent_attention_jagged_b200.binding import LLATTE_ERR_ARG, LLATTE_ERR_UNSUPPORTED
from oracle.model import absorb, rmsnorm, silu
from workloads import Dims, Workload, make_inputs

from gpu_harness import assert_close

pytestmark = pytest.mark.gpu

LENGTHS = [0, 1, 40, 128, 131, 300, 7, 64]


def _inputs(dtype="bf16", lengths=LENGTHS, **kw):
    base = dict(d=128, heads=4, d_head=32, rank=64, d_ctx=16, n_q=5, keep=(300, 300), dtype=dtype,
                attn_form=1)
    base.update(kw)
    wl = Workload(name="cached", dims=Dims(**base), batch=1, lengths=("fixed", 1), seed=31)
    return make_inputs(wl, lengths=lengths, random_gains=True)


class Served:
    """A model and one cache per layer, all layers sharing one page table."""

    def __init__(self, inp, page=32, max_new=300, events=None):
        D, self.inp = inp.dims, inp
        self.B, self.page = inp.batch, page
        events = [int(n) for n in inp.lengths] if events is None else events
        counts = [-(-n // page) for n in events]
        ids = np.random.default_rng(3).permutation(max(1, sum(counts)))
        self.table = np.zeros((self.B, max(1, max(counts))), np.int32)
        for u, n in enumerate(counts):
            self.table[u, :n], ids = ids[:n], ids[n:]
        self.h = Llatte(D, inp.layers, None, max_batch=self.B, max_len=max_new,
                        summaries=inp.summaries)
        dt = torch.bfloat16 if D.dtype == "bf16" else torch.float32
        self.dt = dt
        shape = (max(1, sum(counts)), page, D.rank)
        self.caches = [LatentCache(torch.zeros(shape, dtype=dt, device="cuda"), D.heads,
                                   mass=torch.zeros(shape[:2], device="cuda"), max_batch=self.B,
                                   max_rows=self.h.query_rows(), max_pages=self.table.shape[1])
                       for _ in D.keep]
        self.table_d = torch.from_numpy(self.table).cuda()
        self.ctx = torch.from_numpy(inp.ctx).cuda().to(dt) if D.d_ctx else None
        self.cand = torch.from_numpy(inp.cand).cuda().to(dt) if D.n_q else None

    def request(self, first, last, lengths=None, **kw):
        """Events first[u] .. last[u] - 1 of every user as new ones."""
        rows = [self.inp.values[int(self.inp.offsets[u]) + a:int(self.inp.offsets[u]) + b]
                for u, (a, b) in enumerate(zip(first, last))]
        values = torch.from_numpy(np.concatenate(rows)).cuda().to(self.dt).contiguous()
        off = torch.tensor([0] + list(np.cumsum([len(r) for r in rows]))).cuda()
        ln = torch.tensor(last if lengths is None else lengths, dtype=torch.int32).cuda()
        out = self.h.forward_cached(values, off, self.caches, self.table_d, ln, context=self.ctx,
                                    cand=self.cand, **kw)
        torch.cuda.synchronize()
        assert self.h.status() == 0 and all(c.status() == 0 for c in self.caches)
        return out.double().cpu().numpy()


@pytest.mark.parametrize("dtype,kw", [
    ("bf16", {}),                                                   # tensor cores
    ("bf16", dict(rank=128, heads=2, d_head=64, d_ctx=0)),
    ("bf16", dict(rank=40)),                                        # CUDA cores
    ("bf16", dict(q_rank=64)),                                      # low-rank query
    ("bf16", dict(d=512, heads=8, d_head=64, rank=256)),
    ("bf16", dict(n_sum=2, sum_rank=16, d_seq=8)),                  # summaries of the tokens
    ("fp32", dict(rank=32)),
])
def test_requests_in_turn_equal_one_pass(dtype, kw):
    inp = _inputs(dtype, **kw)
    s = Served(inp)
    n = np.asarray(inp.lengths)
    cuts = [np.zeros_like(n), n // 2, np.maximum(n - 1, n // 2), n]
    for a, b in zip(cuts, cuts[1:]):
        out = s.request([int(x) for x in a], [int(x) for x in b])
    assert_close(out, oracle.forward(inp), dtype, f"forward over a cache {kw}")


def _over_cache(inp, u, old, first, window=0, n_sink=0):
    """fp64 layers of user u: `old` holds the layers' cached latents, the events
    from `first` on are new; returns the final token rows."""
    D = inp.dims
    a, b = int(inp.offsets[u]), int(inp.offsets[u + 1])
    c = inp.ctx[u].astype(np.float64)
    H, Y = inp.values[a + first:b].astype(np.float64), inp.cand[u].astype(np.float64)
    for l, w in enumerate(inp.layers):
        f = {k: np.asarray(v, np.float64) for k, v in w.items() if v is not None}
        ab = absorb(w, D)
        C = np.concatenate([old[l], rmsnorm(H @ f["W_dkv"].T, f["g_kv"], D.eps)])
        R = np.concatenate([H, Y])
        RC = np.concatenate([R, np.broadcast_to(c, (len(R), len(c)))], axis=1)
        see = oc.visible(len(H), len(Y), len(C), window, n_sink)
        A = np.zeros_like(R)
        for j in range(D.heads):
            S = np.where(see, RC @ ab["W_QK"][j].T @ C.T, -np.inf)
            m = S.max(1, keepdims=True, initial=-np.inf)
            P = np.where(see, np.exp(S - np.where(np.isfinite(m), m, 0.0)), 0.0)
            P = P / np.maximum(P.sum(1, keepdims=True), 1e-300)
            A += P @ C @ ab["W_OV"][j].T
        Z = rmsnorm(R + A, f["g1"], D.eps)
        X = rmsnorm(Z + silu(Z @ f["W1"].T) @ f["W2"].T, f["g2"], D.eps)
        H, Y = X[:len(H)], X[len(H):]
    return Y


def _cached(s, u, n):
    """The latents of user u's first n events, layer by layer, as they are stored."""
    at = oc.slots(s.table[u], n, s.page)
    return [c.pool.double().cpu().numpy()[at] for c in s.caches]


def test_window_with_first_events_kept():
    inp = _inputs()
    s = Served(inp)
    n = [int(x) for x in inp.lengths]
    s.request([0] * len(n), n, window=50, n_sink=3)
    whole = np.stack([_over_cache(inp, u, [np.zeros((0, 64))] * 2, 0, 50, 3)
                      for u in range(len(n))])
    half = [x // 2 for x in n]
    t = Served(inp)
    t.request([0] * len(n), half, window=50, n_sink=3)
    out = t.request(half, n, window=50, n_sink=3)
    assert_close(out, whole, "bf16", "forward over a windowed cache")


def test_a_session_with_eviction():
    """Requests, eviction by the weights they left, a request over what is left in
    every layer's cache (each layer keeps its own events)."""
    inp = _inputs(lengths=[300, 200, 90, 257])
    s = Served(inp)
    n = [int(x) for x in inp.lengths]
    old = [x - 20 for x in n]
    s.request([0] * 4, old, accumulate=True)
    rows = np.array(old) + inp.dims.n_q
    for c in s.caches:                          # every row and head spends a weight of 1
        spent = sum(float(c.mass[torch.from_numpy(s.table[u, :-(-old[u] // 32)]).long().cuda()]
                          .double().sum()) for u in range(4))
        assert abs(spent - inp.dims.heads * rows.sum()) < 1e-3 * spent
    lengths = torch.tensor(old, dtype=torch.int32, device="cuda")
    short = [c.evict(s.table_d, lengths, 64, n_sink=2, n_recent=16) for c in s.caches]
    assert all(x.cpu().tolist() == [64, 64, 64, 64] for x in short)
    ref = np.stack([_over_cache(inp, u, _cached(s, u, 64), old[u]) for u in range(4)])
    assert_close(s.request(old, n, lengths=[84] * 4), ref, "bf16", "forward over an evicted cache")


def test_captured_and_replayed():
    inp = _inputs(lengths=[130, 40])
    s = Served(inp)
    first, n = [100, 39], [130, 40]
    s.request([0, 0], first)
    rows = [inp.values[int(inp.offsets[u]) + a:int(inp.offsets[u]) + b]
            for u, (a, b) in enumerate(zip(first, n))]
    values = torch.from_numpy(np.concatenate(rows)).cuda().to(s.dt).contiguous()
    off = torch.tensor([0, 30, 31]).cuda()
    ln = torch.tensor(n, dtype=torch.int32).cuda()
    args = (values, off, s.caches, s.table_d, ln)
    want = s.h.forward_cached(*args, context=s.ctx, cand=s.cand).clone()
    out = torch.zeros_like(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.h.forward_cached(*args, context=s.ctx, cand=s.cand, out=out, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.h.forward_cached(*args, context=s.ctx, cand=s.cand, out=out, stream=side)
    for _ in range(2):                          # the same events again change nothing
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert_close(out.double().cpu().numpy(), oracle.forward(inp), "bf16", "captured cached forward")
    del g


def test_refusals():
    inp = _inputs(lengths=[40, 7])
    s = Served(inp, max_new=40)
    vals = torch.zeros(3, 128, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 2, 3]).cuda()
    ln = torch.tensor([2, 1], dtype=torch.int32, device="cuda")

    def call(h=s.h, caches=None, **kw):
        return h.forward_cached(vals, off, caches or s.caches, s.table_d, ln, context=s.ctx,
                                cand=s.cand, **kw)

    for kw in (dict(window=-1), dict(n_sink=-1)):
        with pytest.raises(LlatteError) as e:
            call(**kw)
        assert e.value.code == LLATTE_ERR_ARG
    with pytest.raises(ValueError):
        call(caches=s.caches[:1])
    c = s.caches[0]
    small = LatentCache(c.pool, 4, mass=c.mass, max_batch=2, max_rows=3, max_pages=2)
    other = LatentCache(c.pool, 2, mass=c.mass, max_batch=2, max_rows=500, max_pages=2)
    plain = LatentCache(c.pool, 4, max_batch=2, max_rows=s.h.query_rows(), max_pages=2)
    for bad, kw in ((small, {}), (other, {}), (plain, dict(accumulate=True))):
        with pytest.raises(LlatteError) as e:
            call(caches=[c, bad], **kw)
        assert e.value.code == LLATTE_ERR_ARG
    for kw in (dict(keep=(300, 100)), dict(d_time=8), dict(n_q=0, d_ctx=16, d_out=8),
               dict(d_head=64, heads=2, attn_form=2)):
        t = _inputs(lengths=[40, 7], **kw)
        h = Llatte(t.dims, t.layers, t.W_e, max_batch=2, max_len=300)
        cs = [LatentCache(c.pool, t.dims.heads, max_batch=2, max_rows=h.query_rows(), max_pages=2)
              for _ in t.dims.keep]
        with pytest.raises(LlatteError) as e:
            h.forward_cached(vals, off, cs, s.table_d, ln, context=s.ctx,
                             cand=s.cand if t.dims.n_q else None)
        assert e.value.code == LLATTE_ERR_UNSUPPORTED
        h.close()
    call()                                       # and the call as it should be
    torch.cuda.synchronize()
    assert s.h.status() == 0
