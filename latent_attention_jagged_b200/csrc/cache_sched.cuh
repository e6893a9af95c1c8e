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

// Growth of a row's maximum (log2 units) up to which its sums keep their base.  Any base
// leaves a weight the same relative rounding (2^-8 in bf16; only at the running maximum
// would the largest weight, 1, have none), so that the base only has to keep sums in
// range: weights up to 2^20 leave latents up to 2^70 and 2^31 events room.  With 2^8 some row of a block outgrew its first 64 events in many items, and
// a rescale waits for every product before it (64 candidates for 256 users: 44.3 us).
constexpr float kGrow = 20.f;

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
  k.pmin = cache_pos(x, cache_div(c, q0));
  k.pmax = cache_pos(x, cache_div(c, q1));
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
  using Block = CacheBlock;
  __device__ __forceinline__ static int blocks(const CacheCall& c, const CacheUser& x) {
    return (int)(((uint32_t)x.n * (uint32_t)c.heads + (MT - 1)) / MT);
  }
  __device__ __forceinline__ static Block block(const CacheCall& c, const CacheUser& x, int b) {
    return cache_block<MT, KT>(c, x, b);
  }
  __device__ __forceinline__ static int32_t places(const Block& k) { return max(1, k.tiles); }
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
struct CacheTile {
  CacheBlock all;              // what the user's rows read
  int32_t tile;
  int32_t first, last;         // blocks of pairs that see the tile
};

template <int NP, int KT>
struct ByTiles {
  using Block = CacheTile;
  __device__ __forceinline__ static int blocks(const CacheCall& c, const CacheUser& x) {
    return cache_all<KT>(c, x).tiles;
  }
  // The rows that see a tile lie between the first one at or after its start and
  // the last one whose window reaches back to its end.
  __device__ __forceinline__ static Block block(const CacheCall& c, const CacheUser& x, int b) {
    Block k;
    k.all = cache_all<KT>(c, x);
    k.tile = cache_tile(k.all, b);
    const int64_t t0 = (int64_t)k.tile * KT, start = x.len - x.m;
    int64_t lo = max((int64_t)0, t0 - start), hi = x.n - 1;
    const int64_t last = t0 + KT - 2 + c.window;       // last position that sees its end
    if (c.window > 0 && t0 >= c.n_sink && x.len - 1 > last) hi = last - start;
    k.first = (int)((uint32_t)lo * (uint32_t)c.heads / NP);
    k.last = (int)(((uint32_t)hi * (uint32_t)c.heads + c.heads - 1) / NP);
    return k;
  }
  __device__ __forceinline__ static int32_t places(const Block& k) { return k.last - k.first + 1; }
};

// Where a CTA's run of places lies.
struct CacheSplit {
  int32_t begin, end, quota;   // this CTA's run of places
  int32_t u, b, t;             // where it starts: user, block, place in the block
  CacheUser x;                 // that user
};

// Shared memory that a split works in: places before every user, and the users.
struct CacheSplitSpace {
  int32_t prefix[LLATTE_CACHE_MAX_BATCH + 4];
  int2 user[LLATTE_CACHE_MAX_BATCH];        // rows, cached events
  int64_t row0[LLATTE_CACHE_MAX_BATCH];     // first row
};

// The cut at place `at` of `base` (a whole warp calls this): where it lies and the
// user there.  A cut inside a block that is short against a CTA's run moves to the
// nearer end of the block: the imbalance is at most an eighth of a run, and the
// block need not be summed from parts.  With `never` every cut moves.
template <class W>
__device__ __forceinline__ void cache_cut(const CacheCall& c, const CacheSplitSpace& w, int64_t at,
                                          int64_t base, int32_t quota, bool never,
                                          CacheSplit* s) {
  const int lane = threadIdx.x & 31;
  s->begin = (int32_t)at;
  s->u = c.B; s->b = s->t = 0;
  s->x = {0, 0, 0, 0};
  if (at >= base) return;
  // the last user whose places start at or before the cut (skips empty users): a
  // 32-way search
  int lo = 0, n = c.B;                      // it is one of n users from lo
#pragma unroll 1
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const uint32_t le = __ballot_sync(0xffffffffu, lane * step < n && w.prefix[min(i, c.B)] <= at);
    const int k = 31 - __clz(le);           // lane 0 always answers yes
    n = min(step, n - k * step);
    lo += k * step;
  }
  s->u = lo;
  const int2 d = w.user[lo];
  const CacheUser x = {w.row0[lo], d.x, max(0, d.x - c.n_cand), d.y};
  s->x = x;
  const int nb = W::blocks(c, x);
  int32_t left = (int32_t)at - w.prefix[lo];
#pragma unroll 1
  for (int b0 = 0; b0 < nb; b0 += 32) {
    const int b = b0 + lane;
    const int32_t own = b < nb ? W::places(W::block(c, x, b)) : 0;
    int32_t v = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    const uint32_t in = __ballot_sync(0xffffffffu, b < nb && v > left);
    if (in) {
      const int l = __ffs(in) - 1;
      const int32_t places = __shfl_sync(0xffffffffu, own, l);
      s->b = b0 + l;
      s->t = left - __shfl_sync(0xffffffffu, v - own, l);
      if (s->t > 0 && (never || places <= quota / 4)) {
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

constexpr int kFewBlocks = 16;

// Every thread of the CTA calls this (it synchronises).  A run has min_quota places
// or more.  A call of 2^31 places or more gets no work and LLATTE_DEV_TOO_LONG.
template <class W>
__device__ __forceinline__ void cache_split(const CacheCall& c, int min_quota, bool never,
                                            CacheSplitSpace& w, CacheSplit* out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  constexpr int64_t kTop = (int64_t)1 << 31;
  bool many = false, too_many = false;
#pragma unroll 1
  for (int u = threadIdx.x; u < c.B; u += blockDim.x) {
    const CacheUser x = cache_user(c, u);
    const int nb = W::blocks(c, x);
    int64_t places = 0;
    if (nb <= kFewBlocks) {
#pragma unroll 1
      for (int b = 0; b < nb; ++b) places += W::places(W::block(c, x, b));
    } else {
      many = true;
      places = -1;
    }
    w.user[u] = make_int2(x.n, x.len);
    w.row0[u] = x.row0;
    w.prefix[u + 1] = (int32_t)min(places, kTop - 1);
  }
  // users of many blocks: a warp each, a block per lane (a thread takes about 40 cycles
  // a block, a warp 400 a user)
  if (__syncthreads_or(many)) {
    for (int u = warp; u < c.B; u += warps) {
      if (w.prefix[u + 1] >= 0) continue;
      const int2 d = w.user[u];
      const CacheUser x = {0, d.x, max(0, d.x - c.n_cand), d.y};
      const int nb = W::blocks(c, x);
      int64_t sum = 0;
#pragma unroll 1
      for (int b = lane; b < nb; b += 32) sum += W::places(W::block(c, x, b));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      too_many |= sum >= kTop;
      __syncwarp();
      if (lane == 0) w.prefix[u + 1] = (int32_t)min(sum, kTop - 1);
    }
    too_many = __syncthreads_or(too_many);
  }
  // warps 0 and 1 sum up the users, 32 runs of them, and find the CTA's two cuts
  if (warp < 2) {
    const int per = (c.B + 31) / 32, u0 = min(lane * per, c.B), u1 = min(u0 + per, c.B);
    int64_t v = 0;
#pragma unroll 1
    for (int u = u0; u < u1; ++u) v += w.prefix[u + 1];
    int64_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    int64_t base = __shfl_sync(0xffffffffu, incl, 31);
    if (too_many || base >= kTop) {
      if (lane == 0 && warp == 0) atomicOr(c.status, LLATTE_DEV_TOO_LONG);
      base = 0;
    }
    asm volatile("bar.sync 1, 64;" ::: "memory");       // both have read the places
    if (warp == 0) {
      int64_t sum = incl - v;
#pragma unroll 1
      for (int u = u0; u < u1; ++u) {
        sum += w.prefix[u + 1];
        w.prefix[u + 1] = (int32_t)min(sum, kTop - 1);
      }
      if (lane == 0) w.prefix[0] = 0;
    }
    asm volatile("bar.sync 1, 64;" ::: "memory");
    const int32_t quota = (int32_t)max((int64_t)min_quota, (base + gridDim.x - 1) / gridDim.x);
    const int64_t at = (int64_t)(blockIdx.x + warp) * quota;
    CacheSplit s;
    cache_cut<W>(c, w, min(at, base), base, quota, never, &s);
    if (lane == 0) {
      if (warp == 0) {
        out->begin = s.begin; out->quota = quota;
        out->u = s.u; out->b = s.b; out->t = s.t; out->x = s.x;
      } else {
        out->end = s.begin;
      }
    }
  }
  __syncthreads();
}

// One piece of work: places [t0, t1) of block b of user u.
template <class W>
struct CacheItem {
  int32_t u, b;
  CacheUser x;
  typename W::Block k;
  int32_t t0, t1;
  bool whole;                  // the block is not cut
  bool starts;                 // it starts in this CTA
  int32_t parts;               // CTAs that share it, from CTA `lead` on
  int32_t lead;
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
      x = s.x;
      nb = W::blocks(c, x);
      fetch(c, u + 1);
    }
  }
  __device__ __forceinline__ bool next(const CacheCall& c, CacheItem<W>& it) {
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
    it.k = W::block(c, x, b);
    const int32_t places = W::places(it.k);
    it.t0 = t;
    it.t1 = min(places, t + (end - pos));
    const int32_t g0 = pos - t;             // the block's first place in the line
    it.whole = it.t0 == 0 && it.t1 == places;
    it.lead = g0 / quota;
    it.parts = (g0 + places - 1) / quota - it.lead + 1;
    it.starts = it.t0 == 0;
    pos += it.t1 - it.t0;
    t = 0;
    ++b;
    return true;
  }
};

}  // namespace llatte
