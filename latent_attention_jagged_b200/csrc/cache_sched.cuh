// Work split of the paged-cache attention kernels.
//
// A user's (query row, head) pairs, heads innermost, are cut into blocks of MT;
// a block reads the tiles of KT events that any of its rows sees: the tiles that
// hold the first n_sink events, then those from the earliest row's window to the
// latest row's position.  All blocks' tiles in one line, user by user, are cut
// into gridDim.x equal runs, one per CTA.  So every CTA gets the same number of
// tiles whatever the batch looks like (one long history, or many short ones),
// and only a block that a cut goes through is summed from parts: at most two
// parts per CTA.  Every CTA works the split out for itself (one pass over the
// users and a scan in shared memory), which saves a planning launch.
#pragma once

#include "cache_call.cuh"

namespace llatte {

// The events that one block of one user's pairs reads.
struct CacheBlock {
  int32_t pmin, pmax;        // positions of its first and last row (-1: no events)
  int32_t sink_tiles;        // leading tiles read for the first n_sink events
  int32_t first_tile;        // first tile of the rest
  int32_t tiles;             // both together (0: the user has no events)
};

template <int MT, int KT>
__device__ __forceinline__ CacheBlock cache_block(const CacheCall& c, const CacheUser& x, int b) {
  CacheBlock k;
  // pairs of a call fit 31 bits, so 32-bit unsigned arithmetic is exact
  const uint32_t pairs = (uint32_t)x.n * (uint32_t)c.heads;
  const uint32_t q0 = (uint32_t)b * MT, q1 = min(q0 + MT, pairs) - 1;
  k.pmin = cache_pos(x, (int)(q0 / (uint32_t)c.heads));
  k.pmax = cache_pos(x, (int)(q1 / (uint32_t)c.heads));
  const int32_t all = k.pmax < 0 ? 0 : k.pmax / KT + 1;
  k.first_tile = cache_low(c, k.pmin) / KT;
  const int32_t sink = min(c.n_sink, k.pmax + 1);
  k.sink_tiles = sink <= 0 ? 0 : min((sink - 1) / KT + 1, k.first_tile);
  k.tiles = k.sink_tiles + (all - min(k.first_tile, all));
  return k;
}

__device__ __forceinline__ int32_t cache_tile(const CacheBlock& k, int i) {
  return i < k.sink_tiles ? i : k.first_tile + (i - k.sink_tiles);
}

// Does a row of the block see any of the events [t0, t1)?  Events of a page that
// no row sees are not looked at, nor is the page's entry in the table.
__device__ __forceinline__ bool cache_seen(const CacheCall& c, const CacheBlock& k, int32_t t0,
                                           int32_t t1) {
  return t0 <= k.pmax && (t1 > cache_low(c, k.pmin) || t0 < c.n_sink);
}

// The line of the attention kernels: blocks of MT pairs; a block takes a place for
// each of its tiles, or one when it has none (its rows still get their zeros).
template <int MT, int KT>
struct ByRows {
  __device__ __forceinline__ static int blocks(const CacheCall& c, const CacheUser& x) {
    return (int)(((uint32_t)x.n * (uint32_t)c.heads + (MT - 1)) / MT);
  }
  __device__ __forceinline__ static int32_t places(const CacheCall& c, const CacheUser& x, int b) {
    return max(1, cache_block<MT, KT>(c, x, b).tiles);
  }
};

// The events that any row of a user reads, as one block.
template <int KT>
__device__ __forceinline__ CacheBlock cache_all(const CacheCall& c, const CacheUser& x) {
  CacheBlock k;
  k.pmin = cache_pos(x, 0);
  k.pmax = x.len - 1;
  const int32_t all = k.pmax < 0 ? 0 : k.pmax / KT + 1;
  k.first_tile = cache_low(c, k.pmin) / KT;
  const int32_t sink = min(c.n_sink, k.pmax + 1);
  k.sink_tiles = sink <= 0 ? 0 : min((sink - 1) / KT + 1, k.first_tile);
  k.tiles = x.n == 0 ? 0 : k.sink_tiles + (all - min(k.first_tile, all));
  return k;
}

// The line of the accumulation kernel: blocks are a user's tiles of KT events; a
// block takes a place for each block of NP pairs with a row that sees the tile.
template <int NP, int KT>
struct ByTiles {
  __device__ __forceinline__ static int blocks(const CacheCall& c, const CacheUser& x) {
    return cache_all<KT>(c, x).tiles;
  }
  // First and last block of pairs that sees tile `tile`.  The rows that see it lie
  // between the first one at or after its start and the last one whose window
  // reaches back to its end.
  __device__ __forceinline__ static int2 range(const CacheCall& c, const CacheUser& x,
                                               int32_t tile) {
    const int64_t t0 = (int64_t)tile * KT, start = x.len - x.m;
    int64_t lo = max((int64_t)0, t0 - start), hi = x.n - 1;
    const int64_t last = t0 + KT - 2 + c.window;       // last position that sees its end
    if (c.window > 0 && t0 >= c.n_sink && x.len - 1 > last) hi = last - start;
    return make_int2((int)((uint32_t)lo * (uint32_t)c.heads / NP),
                     (int)(((uint32_t)hi * (uint32_t)c.heads + c.heads - 1) / NP));
  }
  __device__ __forceinline__ static int32_t places(const CacheCall& c, const CacheUser& x, int b) {
    const int2 r = range(c, x, cache_tile(cache_all<KT>(c, x), b));
    return r.y - r.x + 1;
  }
};

// Where a CTA's run of places lies.
struct CacheSplit {
  int32_t begin, end, quota;   // this CTA's run of places
  int32_t u, b, t;             // where it starts: user, block, place in the block
};

// The cut at place `at` of `base` (a whole warp calls this): user, block and place
// in the block.  A cut inside a block that is short against a CTA's run moves to
// the nearer end of the block: the imbalance is at most an eighth of a run, and
// the block need not be summed from parts.
template <class W>
__device__ __forceinline__ void cache_cut(const CacheCall& c, const int32_t* prefix, int64_t at,
                                          int64_t base, int32_t quota, CacheSplit* s) {
  const int lane = threadIdx.x & 31;
  s->begin = s->end = (int32_t)at;
  s->u = c.B; s->b = s->t = 0;
  if (at >= base) return;
  // the last user whose places start at or before the cut (skips empty users)
  int lo = 0, hi = c.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= at) lo = mid; else hi = mid - 1;
  }
  s->u = lo;
  const CacheUser x = cache_user(c, lo);
  const int nb = W::blocks(c, x);
  int32_t left = (int32_t)at - prefix[lo];
  for (int b0 = 0; b0 < nb; b0 += 32) {
    const int b = b0 + lane;
    const int32_t own = b < nb ? W::places(c, x, b) : 0;
    int32_t v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t w = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += w;
    }
    const uint32_t in = __ballot_sync(0xffffffffu, b < nb && v > left);
    if (in) {
      const int l = __ffs(in) - 1;
      const int32_t places = __shfl_sync(0xffffffffu, own, l);
      s->b = b0 + l;
      s->t = left - __shfl_sync(0xffffffffu, v - own, l);
      if (s->t > 0 && places <= quota / 4) {
        if (2 * s->t < places) {
          s->begin -= s->t;
        } else {
          s->begin += places - s->t;
          ++s->b;                       // the walk goes on to the next user if need be
        }
        s->t = 0;
      }
      break;
    }
    left -= __shfl_sync(0xffffffffu, v, 31);
  }
}

// Every thread of the CTA calls this (it synchronises); prefix has B + 1 entries
// of shared memory, prefix[u] = places before user u.  A call of 2^31 places or
// more gets no work and LLATTE_DEV_TOO_LONG.
template <class W>
__device__ __forceinline__ void cache_split(const CacheCall& c, int min_quota, int32_t* prefix,
                                            CacheSplit* out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  constexpr int64_t kTop = (int64_t)1 << 31;
  int64_t mine = 0;                       // places this warp has found (all lanes)
  for (int u0 = warp * 32; u0 < c.B; u0 += warps * 32) {
    const int u = u0 + lane;
    CacheUser x = {0, 0, 0, 0};
    if (u < c.B) x = cache_user(c, u);
    const int nb = W::blocks(c, x);
    int64_t places = 0;
    if (nb <= 4)
      for (int b = 0; b < nb; ++b) places += W::places(c, x, b);
    // users of many blocks: the whole warp, one block per lane
    for (uint32_t big = __ballot_sync(0xffffffffu, nb > 4); big; big &= big - 1) {
      const int l = __ffs(big) - 1;
      CacheUser y;
      y.row0 = 0;
      y.n = __shfl_sync(0xffffffffu, x.n, l);
      y.m = __shfl_sync(0xffffffffu, x.m, l);
      y.len = __shfl_sync(0xffffffffu, x.len, l);
      const int nby = __shfl_sync(0xffffffffu, nb, l);
      int64_t sum = 0;
      for (int b = lane; b < nby; b += 32) sum += W::places(c, y, b);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == l) places = sum;
    }
    mine += places;
    if (u < c.B) prefix[u + 1] = (int32_t)min(places, kTop - 1);
  }
  const int too_many = __syncthreads_or(mine >= kTop);
  if (warp == 0) {
    int64_t base = 0;
    for (int u0 = 0; u0 < c.B; u0 += 32) {
      const int u = u0 + lane;
      int64_t v = u < c.B ? prefix[u + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t w = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += w;
      }
      if (u < c.B) prefix[u + 1] = (int32_t)min(base + v, kTop - 1);
      base += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) prefix[0] = 0;
    __syncwarp();
    if (too_many || base >= kTop) {
      if (lane == 0) atomicOr(c.status, LLATTE_DEV_TOO_LONG);
      base = 0;
    }
    CacheSplit s, e;
    s.quota = (int32_t)max((int64_t)min_quota, (base + gridDim.x - 1) / gridDim.x);
    const int64_t first = (int64_t)blockIdx.x * s.quota;
    cache_cut<W>(c, prefix, min(first, base), base, s.quota, &s);
    e.quota = s.quota;
    cache_cut<W>(c, prefix, min(first + s.quota, base), base, s.quota, &e);
    s.end = e.begin;
    if (lane == 0) *out = s;
  }
  __syncthreads();
}

// One piece of work: places [t0, t1) of block b of user u.
struct CacheItem {
  int32_t u, b;
  CacheUser x;
  int32_t t0, t1;
  bool whole;                  // the block is not cut
  bool starts;                 // it starts in this CTA
  int32_t parts;               // CTAs that share it
};

// Walks the pieces of this CTA's run.  The next user's offsets and length are
// loaded one user ahead, so that no role waits for them.
template <class W>
struct CacheItems {
  int32_t pos, end, quota, u, b, t;
  CacheUser x;
  int32_t nb;
  int64_t next_a, next_b;      // offsets and length of user u + 1, as they were read
  int32_t next_len;

  __device__ __forceinline__ void fetch(const CacheCall& c, int v) {
    next_a = next_b = 0;
    next_len = 0;
    if (v < c.B) {
      next_a = c.qoff[v];
      next_b = c.qoff[v + 1];
      next_len = c.lengths[v];
    }
  }
  __device__ __forceinline__ void start(const CacheCall& c, const CacheSplit& s) {
    pos = s.begin; end = s.end; quota = s.quota; u = s.u; b = s.b; t = s.t;
    nb = 0;
    if (pos < end) {
      fetch(c, u);
      x = cache_user_of(c, next_a, next_b, next_len);
      nb = W::blocks(c, x);
      fetch(c, u + 1);
    }
  }
  __device__ __forceinline__ bool next(const CacheCall& c, CacheItem& it) {
    if (pos >= end) return false;
    while (b >= nb) {                       // on to the next user with rows
      ++u;
      if (u >= c.B) return false;
      b = 0;
      x = cache_user_of(c, next_a, next_b, next_len);
      nb = W::blocks(c, x);
      fetch(c, u + 1);
    }
    it.u = u; it.b = b; it.x = x;
    const int32_t places = W::places(c, x, b);
    it.t0 = t;
    it.t1 = min(places, t + (end - pos));
    const int32_t g0 = pos - t;             // the block's first place in the line
    it.whole = it.t0 == 0 && it.t1 == places;
    it.parts = (g0 + places - 1) / quota - g0 / quota + 1;
    it.starts = it.t0 == 0;
    pos += it.t1 - it.t0;
    t = 0;
    ++b;
    return true;
  }
};

}  // namespace llatte
