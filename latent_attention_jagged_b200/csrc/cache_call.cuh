// Device helpers of the paged latent cache: a call's users, their rows'
// positions and the place of an event in the pool.
#pragma once

#include "cache.h"
#include "common.cuh"

namespace llatte {

struct CacheUser {
  int64_t row0;      // first row of the user
  int32_t n;         // rows
  int32_t m;         // of them new events (the rest are query tokens)
  int32_t len;       // cached events
};

// n / heads for 0 <= n < 2^31.  With 2^(s-1) < heads <= 2^s and m = floor(2^(31+s) /
// heads) + 1 < 2^32, m heads = 2^(31+s) + e with 0 < e <= 2^s, so that n m / 2^(31+s)
// exceeds n / heads by n e / (heads 2^(31+s)) < 1 / heads: the quotient is exact.
__device__ __forceinline__ int32_t cache_div(const CacheCall& c, uint32_t n) {
  return (int32_t)(c.head_mul ? __umulhi(n, c.head_mul) >> c.head_shift : n);
}

// A user of the call from its offsets and length; a user the header leaves out
// (bad offsets or length) gets no rows and no events, and its fault goes to the
// status word.  With zero_left_out it keeps the rows that good offsets name, as rows
// that see nothing.
__device__ __forceinline__ CacheUser cache_user_of(const CacheCall& c, int64_t a, int64_t b,
                                                   int32_t len) {
  CacheUser x = {0, 0, 0, 0};
  int bad = (len < 0 || len > c.cap) ? LLATTE_DEV_TOO_LONG : 0;
  const bool named = !(a < 0 || b < a || b > c.rows);
  if (!named) bad |= LLATTE_DEV_BAD_OFFSETS;
  if (!bad) {
    x.row0 = a;
    x.n = (int32_t)(b - a);
    x.m = max(0, x.n - c.n_cand);
    x.len = len;
    if (x.m > len) bad = LLATTE_DEV_BAD_OFFSETS;
  }
  if (bad) {
    atomicOr(c.status, bad);
    x = {0, 0, 0, 0};
    if (named && c.zero_left_out) {
      x.row0 = a;
      x.n = (int32_t)(b - a);
    }
  }
  return x;
}

__device__ __forceinline__ CacheUser cache_user(const CacheCall& c, int u) {
  int64_t a = 0, b = 0;
  if (c.qoff) {
    a = c.qoff[u];
    b = c.qoff[u + 1];
  }
  return cache_user_of(c, a, b, c.lengths[u]);
}

// Last event that row j of the user may see (-1: none).
__device__ __forceinline__ int32_t cache_pos(const CacheUser& x, int j) {
  return j < x.m ? x.len - x.m + j : x.len - 1;
}

// First event inside the window of position p (0 without a window).
__device__ __forceinline__ int32_t cache_low(const CacheCall& c, int32_t p) {
  return c.window > 0 ? max(0, p - c.window + 1) : 0;
}

// Pool row of event t of user u, or -1 (and the fault in the status word) for a
// page outside the pool.
__device__ __forceinline__ int64_t cache_row(const CacheCall& c, const int32_t* table,
                                             int32_t stride, int u, int32_t t) {
  const int32_t page = __ldg(table + (int64_t)u * stride + (t >> c.page_shift));
  if ((uint32_t)page >= (uint32_t)c.n_pages) {
    atomicOr(c.status, LLATTE_DEV_BAD_ID);
    return -1;
  }
  return ((int64_t)page << c.page_shift) + (t & ((1 << c.page_shift) - 1));
}

}  // namespace llatte
