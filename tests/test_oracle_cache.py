"""The paged-cache oracle against the forward oracle's masking and against
closed forms, and the host-side refusals of the cache's entry points (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.cache as oc
from latent_attention_jagged_b200 import LatentCache, binding
from latent_attention_jagged_b200.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


def test_visible_is_causal_and_query_tokens_see_all():
    see = oc.visible(3, 2, 5, 0, 0)
    assert see.tolist() == [[True, True, True, False, False], [True, True, True, True, False],
                            [True] * 5, [True] * 5, [True] * 5]


@pytest.mark.parametrize("window,sink", [(1, 0), (2, 1), (3, 5), (100, 2)])
def test_visible_window_counts(window, sink):
    n, m = 9, 9
    see = oc.visible(m, 1, n, window, sink)
    for p in range(n):
        want = {t for t in range(p + 1) if t > p - window or t < sink}
        assert set(np.flatnonzero(see[p])) == want
    assert np.array_equal(see[-1], see[-2])          # a query token sees what the last event sees


def test_attend_matches_a_dense_softmax_and_masses_sum_to_rows():
    rng = np.random.default_rng(3)
    P, table, lengths = 4, np.array([[2, 0, 5], [1, 3, 4]]), np.array([9, 4])
    pool, mass = rng.standard_normal((6, P, 3)), np.zeros((6, P))
    q, off = rng.standard_normal((7, 2, 3)), np.array([0, 4, 7])
    out, lse = oc.attend(pool, mass, q, off, table, lengths, n_cand=1, scale=0.7)
    assert np.isclose(mass.sum(), 7 * 2)
    c = pool[table[0]].reshape(-1, 3)[:9]
    s = 0.7 * q[3, 1] @ c.T                          # the first user's query token
    w = np.exp(s) / np.exp(s).sum()
    assert np.allclose(out[3, 1], w @ c) and np.isclose(lse[3, 1], np.log(np.exp(s).sum()))


def test_evict_keeps_ends_heaviest_and_earlier_ties():
    P, table = 2, np.array([[0, 1, 2, 3]])
    pool = np.arange(8.0).reshape(4, 2, 1)
    mass = np.array([[9, 1], [5, 5], [5, 0], [0, np.nan]], np.float64)
    new, kept = oc.evict(pool, mass, table, [7], budget=4, n_sink=1, n_recent=1)
    assert list(new) == [4] and kept[0] == [0, 2, 3, 6]
    assert pool.reshape(-1)[:4].tolist() == [0, 2, 3, 6]


def _dims(**kw):
    f = dict(heads=4, rank=128, dtype=binding.LLATTE_BF16, page_size=64, n_pages=10, max_batch=4,
             max_pages=3, max_rows=64)
    f.update(kw)
    return binding.llatte_cache_dims(**f)


def test_struct_layouts():
    assert ctypes.sizeof(binding.llatte_cache_dims) == 7 * 4 + 4 + 8
    assert ctypes.sizeof(binding.llatte_cache_view) == 8 + 8 + 8 + 8
    assert ctypes.sizeof(binding.llatte_cache_attn) == 8 * 3 + 16 + 8 + 8 + 8
    assert ctypes.sizeof(binding.llatte_cache_evict_args) == 16 + 8 + 8 + 8 + 8


@pytest.mark.parametrize("kw,code", [
    (dict(heads=0), "ARG"), (dict(rank=0), "ARG"), (dict(rank=512), "UNSUPPORTED"),
    (dict(rank=12), "UNSUPPORTED"), (dict(rank=6, dtype=1), "UNSUPPORTED"), (dict(dtype=2), "ARG"),
    (dict(page_size=8), "UNSUPPORTED"), (dict(page_size=48), "UNSUPPORTED"),
    (dict(n_pages=0), "ARG"), (dict(n_pages=1 << 25, page_size=64), "UNSUPPORTED"),
    (dict(max_batch=0), "ARG"), (dict(max_batch=4097), "UNSUPPORTED"), (dict(max_pages=0), "ARG"),
    (dict(max_pages=1 << 25), "UNSUPPORTED"), (dict(max_rows=0), "ARG"),
    (dict(max_rows=1 << 30), "UNSUPPORTED"), (dict(), "ARG")])
def test_create_refuses(lib, kw, code):
    d, h = _dims(**kw), ctypes.c_void_p()
    want = getattr(binding, "LLATTE_ERR_" + code)
    assert lib.llatte_cache_create(ctypes.byref(h), ctypes.byref(d), None, None) == want
    if kw:
        assert lib.llatte_cache_workspace_bytes(ctypes.byref(d)) == 0
    else:                                           # good dims, no pool
        assert lib.llatte_cache_workspace_bytes(ctypes.byref(d)) > 4 * 64 * 4


def test_calls_refuse_a_null_cache(lib):
    v, a, e = (binding.llatte_cache_view(), binding.llatte_cache_attn(),
               binding.llatte_cache_evict_args())
    st = ctypes.c_int32()
    A = binding.LLATTE_ERR_ARG
    assert lib.llatte_cache_create(None, ctypes.byref(_dims()), None, None) == A
    assert lib.llatte_cache_append(None, ctypes.byref(v), None, 1, None, None, 1e-6, None) == A
    assert lib.llatte_cache_attend(None, ctypes.byref(v), ctypes.byref(a), None) == A
    assert lib.llatte_cache_evict(None, ctypes.byref(v), ctypes.byref(e), None) == A
    assert lib.llatte_cache_get_status(None, ctypes.byref(st)) == A
    assert lib.llatte_cache_uses_tensor_cores(None) == A
    lib.llatte_cache_destroy(None)


def test_binding_refuses_host_tensors(lib):
    with pytest.raises(ValueError):
        LatentCache(torch.zeros(4, 16, 64, dtype=torch.bfloat16), heads=2)
