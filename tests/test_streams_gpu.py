"""Results that a call makes for a stream given by hand: their memory is not shared with
work of the current stream that the call does not wait for."""
import pytest
import torch

from cache_harness import Case
from test_forward_cached_gpu import Served, _inputs

from gpu_harness import make_handle, to_device

pytestmark = pytest.mark.gpu


def _behind_a_write(call):
    """`call(stream)` on another stream while the current one still has to write into
    memory that it has already given back."""
    side = torch.cuda.Stream()
    shape, dt = call(None).shape, call(None).dtype
    torch.cuda.synchronize()
    want = call(None).clone()
    torch.cuda.synchronize()
    keep = [torch.empty(shape, dtype=dt, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)            # about 10 ms
    for k in keep:
        k.fill_(7)
    del keep, k                              # free for the current stream's next tensors
    got = call(side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def _cache_call():
    c = Case("bf16", 4, 128, 64, [700, 90], seed=3)
    q, off = c.queries([40, 40], 0)
    return c, (q, torch.from_numpy(off).cuda(), c.dev("table"), c.dev("lengths"))


def test_attention():
    c, args = _cache_call()
    _behind_a_write(lambda s: c.cache.attend(*args, scale=0.1, stream=s))


def test_a_stream_given_by_its_address():
    c, args = _cache_call()
    _behind_a_write(lambda s: c.cache.attend(*args, scale=0.1,
                                             stream=None if s is None else s.cuda_stream))


def test_the_default_stream_given_by_its_address():
    # 0 is a stream like any other: the memory is the default stream's, not a third one's
    c, args = _cache_call()
    want = c.cache.attend(*args, scale=0.1).clone()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        _behind_a_write(lambda s: c.cache.attend(*args, scale=0.1, stream=None if s is None else 0))
        out = c.cache.attend(*args, scale=0.1, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    held = out.data_ptr()
    del out
    torch.cuda.synchronize()
    blocks = [torch.empty_like(want) for _ in range(64)]         # of the default stream
    assert held in [b.data_ptr() for b in blocks]


def test_eviction():
    c, args = _cache_call()
    _behind_a_write(lambda s: c.cache.evict(args[2], args[3], 5000, stream=s))


def test_forward():
    inp = _inputs()
    h, args = make_handle(inp), to_device(inp)
    _behind_a_write(lambda s: h.forward(*args, stream=s))
    _behind_a_write(lambda s: h.forward_export(*args, layer=1, stream=s)[1])


def test_forward_over_a_cache():
    inp = _inputs()
    s, (values, off, ctx, cand) = Served(inp), to_device(inp)
    ln = torch.from_numpy(inp.lengths).int().cuda()
    _behind_a_write(lambda st: s.h.forward_cached(values, off, s.caches, s.table_d, ln, context=ctx,
                                                  cand=cand, stream=st))


def test_memory_that_the_current_stream_still_reads_is_not_used_again():
    c, args = _cache_call()
    side = torch.cuda.Stream()
    want = c.cache.attend(*args, scale=0.1).clone()
    turned = (-args[0],) + args[1:]
    other = c.cache.attend(*turned, scale=0.1).clone()
    torch.cuda.synchronize()
    out = c.cache.attend(*args, scale=0.1, stream=side)
    side.synchronize()
    torch.cuda._sleep(20_000_000)            # about 10 ms
    copy = out.clone()
    del out
    again = c.cache.attend(*turned, scale=0.1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and torch.equal(again, other)
