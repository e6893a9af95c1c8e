// Attention over the paged latent cache on CUDA cores: fp32 storage, and bf16 at ranks
// that the tensor-core kernels do not take.
//
//   s_it = scale q_i . c_t over the events row i sees,  P = softmax(s),
//   o_i = sum_t P_it c_t,  lse_i = log sum_t exp(s_it),  mass_t += sum_i P_it
//
// Scores are kept in log2 units (scale * log2 e folded into one factor).  Three
// kernels share the work split of cache_sched.cuh:
//   rows    blocks of 64 pairs x tiles of 64 events, 4 x 4 scores and 4 x r/16 results
//           of a thread in registers, two fp32 lanes an instruction; bound by the
//           shared-memory reads that feed the FMA pipe (32 users, 100 to 300 new of
//           500 to 1000 events, 4 heads: 28 TFLOP/s at r = 128, 24 at r = 64; 21 and
//           19 with one CTA an SM and two buffers for its tiles)
//   tokens  blocks of 8 pairs; a warp takes every 32 events by itself (a lane owns an
//           event for the scores and columns for the result), and the warps meet at
//           the end; bound by latency at small sizes (64 users behind a window of 256,
//           2 heads, r = 32: 14 us, of which the cache's 2 MB are 0.3)
//   mass    tiles of 64 events against all blocks of 64 pairs; a thread sums its events
#include <algorithm>
#include <atomic>

#include "cache.h"
#include "cache_call.cuh"
#include "cache_sched.cuh"
#include "tc_common.cuh"

namespace llatte {

using tc::add_f2;
using tc::ex2_approx;
using tc::fma_f2;

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int MT = 64, KT = 64;           // pairs and events of a tile
constexpr int TP = 8, TK = 32;            // the same of the token kernel
constexpr int kSmemMax = 232448;          // shared memory of a CTA

__device__ __forceinline__ float4 ld4(const float* p) { return *(const float4*)p; }
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p) {
  const uint2 u = *(const uint2*)p;
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void st4(float* p, float4 v) { *(float4*)p = v; }
__device__ __forceinline__ void st4(__nv_bfloat16* p, float4 v) {
  *(uint2*)p = make_uint2(tc::pack_bf16(v.x, v.y), tc::pack_bf16(v.z, v.w));
}

// 16 bytes to shared memory; zeros where `src` is null.
__device__ __forceinline__ void copy16(void* dst, const void* any, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tc::smem_u32(dst)),
               "l"(src ? src : any), "r"(src ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Elements between rows in shared memory: 16 bytes more than a row, so that the same
// column of 8 rows falls on different banks.
template <typename T> __device__ __forceinline__ int row_pitch(int r) { return r + 16 / (int)sizeof(T); }

// Pool row of event t as block k of user u sees it: -1 when no row of the block sees
// it or its page is outside the pool.
__device__ __forceinline__ int64_t seen_row(const CacheCall& c, const CacheBlock& k, int u,
                                            int32_t t) {
  return cache_seen(c, k, t, t + 1) ? cache_row(c, c.table, c.stride, u, t) : -1;
}

// Copies `n` rows of `r` elements: row i from src(i) (null: zeros).
template <typename T, typename F>
__device__ __forceinline__ void copy_rows(T* dst, const T* any, int n, int r, int tid, int threads,
                                          F src) {
  constexpr int EV = 16 / sizeof(T);
  const int nvec = r / EV, pitch = row_pitch<T>(r);
  const int drow = threads / nvec, dcol = threads % nvec;
  int row = tid / nvec, col = tid % nvec;
  while (row < n) {
    const T* s = src(row);
    copy16(dst + row * pitch + col * EV, any, s ? s + col * EV : nullptr);
    row += drow;
    col += dcol;
    if (col >= nvec) { col -= nvec; ++row; }
  }
}

// s[i][j] = q row (4 ty + i) . k row (tx + 16 j)
template <typename T>
__device__ __forceinline__ void score_tile(const T* q, const T* k, int r, int ty, int tx,
                                           float (&s)[4][4]) {
  const int pitch = row_pitch<T>(r);
  float2 a[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) a[i][j] = make_float2(0.f, 0.f);
#pragma unroll 2
  for (int c = 0; c < r; c += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = ld4(q + (4 * ty + i) * pitch + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = ld4(k + (tx + 16 * j) * pitch + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        a[i][j] = fma_f2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), a[i][j]);
        a[i][j] = fma_f2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), a[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = a[i][j].x + a[i][j].y;
}

// Clears the rows of a tile that hold an infinity or NaN, so that a weight of 0 hides
// them.
template <typename T>
__device__ __forceinline__ void clear_rows(T* k, int n, int r, int tid, int threads) {
  const int pitch = row_pitch<T>(r);
  for (int row = tid; row < n; row += threads) {
    bool bad = false;
    for (int c = 0; c < r; c += 4) {
      const float4 x = ld4(k + row * pitch + c);
      bad |= !(fabsf(x.x) < INFINITY && fabsf(x.y) < INFINITY && fabsf(x.z) < INFINITY &&
               fabsf(x.w) < INFINITY);
    }
    if (bad)
      for (int c = 0; c < r; c += 4) st4(k + row * pitch + c, make_float4(0.f, 0.f, 0.f, 0.f));
  }
}

// ---------------------------------------------------------------- rows
// Two CTAs an SM hide each other's loads and barriers where shared memory has the room
// (r <= 128); at r = 256 one CTA has two buffers for its tiles.
template <typename T, int RC>
__global__ void __launch_bounds__(256, RC <= 2 ? 2 : 1) cache_rows_kernel(CacheAttn p) {
  constexpr int BUFS = RC <= 2 ? 1 : 2;
  using Line = ByRows<MT, KT>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ CacheSplit split;
  const CacheCall& c = p.c;
  const int r = c.r, pitch = row_pitch<T>(r), tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  T* sQ = (T*)smem;
  T* sK = sQ + MT * pitch;                 // [BUFS][KT][pitch]
  float* sP = (float*)(sK + BUFS * KT * pitch);   // [MT][KT + 4]
  constexpr int PP = KT + 4;
  tc::pdl_trigger();
  tc::pdl_wait();
  cache_split<Line>(c, p.min_quota, p.never_cut, *(CacheSplitSpace*)smem, &split);
  const CacheSplit run = split;
  CacheJoin* join = p.join + blockIdx.x;
  if (tid == 0) join->rows = 0;
  CacheItems<Line> items;
  items.start(c, run);
  CacheItem<Line> it;
  while (items.next(c, it)) {
    const uint32_t pair0 = (uint32_t)it.b * MT;
    const int rows = (int)min((uint32_t)MT, (uint32_t)it.x.n * (uint32_t)c.heads - pair0);
    const int64_t at0 = it.x.row0 * c.heads + pair0;
    T* out = (T*)p.out + at0 * r;
    if (it.x.len == 0) {
      for (int i = tid; i < rows * (r / 4); i += 256) st4(out + 4 * i, make_float4(0, 0, 0, 0));
      for (int i = tid; i < rows; i += 256) {
        if (p.lse) p.lse[at0 + i] = -INFINITY;
        if (p.lse2) p.lse2[at0 + i] = -INFINITY;
      }
      continue;
    }
    const T* q = (const T*)p.q + at0 * r;
    const T* pool = (const T*)p.pool;
    auto fetch = [&](int i, int buf) {
      const int32_t t0 = cache_tile(it.k, i) * KT;
      copy_rows(sK + buf * KT * pitch, pool, KT, r, tid, 256, [&](int row) -> const T* {
        const int64_t at = seen_row(c, it.k, it.u, t0 + row);
        return at < 0 ? nullptr : pool + at * r;
      });
      copy_commit();
    };
    __syncthreads();                       // the last item's reads are done
    copy_rows(sQ, q, MT, r, tid, 256, [&](int row) { return row < rows ? q + row * r : nullptr; });
    if (BUFS == 2) fetch(it.t0, 0);
    int32_t pos[4], low[4];
    float m[4], l[4];
    bool poison[4];
    float2 o[4][RC * 2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = min(4 * ty + i, rows - 1);
      pos[i] = cache_pos(it.x, cache_div(c, pair0 + row));
      low[i] = cache_low(c, pos[i]);
      m[i] = -INFINITY;
      l[i] = 0.f;
      poison[i] = false;
#pragma unroll
      for (int k = 0; k < RC * 2; ++k) o[i][k] = make_float2(0.f, 0.f);
    }
    for (int i = it.t0; i < it.t1; ++i) {
      const int buf = (i - it.t0) % BUFS;
      T* k = sK + buf * KT * pitch;
      if (BUFS == 1) fetch(i, 0);
      if (BUFS == 2 && i + 1 < it.t1) {
        fetch(i + 1, buf ^ 1);
        copy_wait<1>();
      } else {
        copy_wait<0>();
      }
      __syncthreads();
      const int32_t t0 = cache_tile(it.k, i) * KT;
      float s[4][4];
      score_tile(sQ, k, r, ty, tx, s);
      const bool masked = it.k.pmin < t0 + KT - 1 || cache_low(c, it.k.pmax) > t0;
      bool odd = false;
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[a][j] *= p.scale2;
          if (masked) {
            const int32_t t = t0 + tx + 16 * j;
            const bool fin = fabsf(s[a][j]) < INFINITY;
            const bool see = t <= pos[a] && (t >= low[a] || t < c.n_sink);
            if (!fin && 4 * ty + a < rows) {
              odd = true;
              poison[a] |= see;
            }
            s[a][j] = see && fin ? s[a][j] : -INFINITY;
          }
        }
      if (masked && __syncthreads_or(odd)) clear_rows(k, KT, r, tid, 256);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        float mt = fmaxf(fmaxf(s[a][0], s[a][1]), fmaxf(s[a][2], s[a][3]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
        const float mn = fmaxf(m[a], mt), mu = mn > -INFINITY ? mn : 0.f;
        if (mn != m[a]) {
          const float f = m[a] > -INFINITY ? ex2_approx(m[a] - mn) : 0.f;
          m[a] = mn;
          l[a] *= f;
#pragma unroll
          for (int b = 0; b < RC * 2; ++b) {
            o[a][b].x *= f;
            o[a][b].y *= f;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = ex2_approx(s[a][j] - mu);
          l[a] += e;
          sP[(4 * ty + a) * PP + tx + 16 * j] = e;
        }
      }
      __syncthreads();
      // O += P C: this thread's rows, columns 64 b + 4 tx
#pragma unroll 2
      for (int t = 0; t < KT; t += 4) {
        float4 w[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) w[a] = ld4(sP + (4 * ty + a) * PP + t);
#pragma unroll
        for (int b = 0; b < RC; ++b) {
          if (64 * b + 4 * tx >= r) continue;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const float4 v = ld4(k + (t + d) * pitch + 64 * b + 4 * tx);
#pragma unroll
            for (int a = 0; a < 4; ++a) {
              const float e = d == 0 ? w[a].x : d == 1 ? w[a].y : d == 2 ? w[a].z : w[a].w;
              o[a][2 * b] = fma_f2(make_float2(e, e), make_float2(v.x, v.y), o[a][2 * b]);
              o[a][2 * b + 1] = fma_f2(make_float2(e, e), make_float2(v.z, v.w), o[a][2 * b + 1]);
            }
          }
        }
      }
      __syncthreads();
    }
    const int64_t slot0 = ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * MT;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) {
        l[a] += __shfl_xor_sync(0xffffffffu, l[a], d);
        poison[a] |= __shfl_xor_sync(0xffffffffu, (int)poison[a], d) != 0;
      }
      if (poison[a] || m[a] == INFINITY) l[a] = NAN;
      const int row = 4 * ty + a;
      if (row >= rows) continue;
      const float inv = it.whole ? (l[a] != 0.f ? 1.f / l[a] : 0.f) : 1.f;
#pragma unroll
      for (int b = 0; b < RC; ++b) {
        const int col = 64 * b + 4 * tx;
        if (col >= r) continue;
        const float4 v = make_float4(o[a][2 * b].x * inv, o[a][2 * b].y * inv,
                                     o[a][2 * b + 1].x * inv, o[a][2 * b + 1].y * inv);
        if (it.whole) st4(out + row * r + col, v);
        else st4(p.part_o + (slot0 + row) * r + col, v);
      }
      if (tx == 0) {
        if (it.whole) {
          const float l2 = l[a] != 0.f ? m[a] + log2f(l[a]) : -INFINITY;
          if (p.lse) p.lse[at0 + row] = l2 * kLn2;
          if (p.lse2) p.lse2[at0 + row] = l2;
        } else {
          p.part_ml[slot0 + row] = make_float2(m[a], l[a]);
        }
      }
    }
    if (tid == 0 && !it.whole && it.starts) {
      join->pair0 = at0;
      join->parts = it.parts;
      join->rows = rows;
    }
  }
}

// ---------------------------------------------------------------- tokens
// Shared memory: queries [TP][r] (fp32), then for each warp two tiles [TK][pitch] and
// weights [TP][TK]; at the end the warps' results [warps][TP][r] in place of the tiles.
template <typename T, int RV>
__global__ void __launch_bounds__(256) cache_tokens_kernel(CacheAttn p) {
  using Line = ByRows<TP, TK>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ CacheSplit split;
  __shared__ float s_m[8][TP], s_l[8][TP];
  const CacheCall& c = p.c;
  const int r = c.r, pitch = row_pitch<T>(r), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int warps = blockDim.x >> 5;
  float* sQ = (float*)smem;
  float* sW = sQ + TP * r + warp * TP * TK;
  T* sK = (T*)(sQ + TP * r + warps * TP * TK) + warp * 2 * TK * pitch;
  float* sO = sQ + TP * r + warps * TP * TK;
  tc::pdl_trigger();
  tc::pdl_wait();
  cache_split<Line>(c, p.min_quota, p.never_cut, *(CacheSplitSpace*)smem, &split);
  const CacheSplit run = split;
  CacheJoin* join = p.join + blockIdx.x;
  if (tid == 0) join->rows = 0;
  CacheItems<Line> items;
  items.start(c, run);
  CacheItem<Line> it;
  while (items.next(c, it)) {
    const uint32_t pair0 = (uint32_t)it.b * TP;
    const int rows = (int)min((uint32_t)TP, (uint32_t)it.x.n * (uint32_t)c.heads - pair0);
    const int64_t at0 = it.x.row0 * c.heads + pair0;
    T* out = (T*)p.out + at0 * r;
    if (it.x.len == 0) {
      for (int i = tid; i < rows * (r / 4); i += blockDim.x)
        st4(out + 4 * i, make_float4(0, 0, 0, 0));
      if (tid < rows) {
        if (p.lse) p.lse[at0 + tid] = -INFINITY;
        if (p.lse2) p.lse2[at0 + tid] = -INFINITY;
      }
      continue;
    }
    const T* pool = (const T*)p.pool;
    auto fetch = [&](int i, int buf) {
      const int32_t t0 = cache_tile(it.k, i) * TK;
      const int64_t mine = seen_row(c, it.k, it.u, t0 + lane);
      // every lane takes part in every shuffle: whole steps of 32 chunks
      constexpr int EV = 16 / sizeof(T);
      const int nvec = r / EV;
      for (int id = lane; id < TK * nvec; id += 32) {
        const int row = id / nvec, col = id - row * nvec;
        const int64_t at = __shfl_sync(0xffffffffu, mine, row);
        copy16(sK + (buf * TK + row) * pitch + col * EV, pool,
               at < 0 ? nullptr : pool + at * r + col * EV);
      }
      copy_commit();
    };
    __syncthreads();                       // the last item's reads are done
    if (it.t0 + warp < it.t1) fetch(it.t0 + warp, 0);
    for (int i = tid; i < TP * r / 4; i += blockDim.x)
      st4(sQ + 4 * i, 4 * i < rows * r ? ld4((const T*)p.q + at0 * r + 4 * i)
                                       : make_float4(0, 0, 0, 0));
    __syncthreads();
    const int32_t low_max = cache_low(c, it.k.pmax);
    float m[TP], l[TP], o[TP][RV];
    uint32_t poison = 0;
#pragma unroll
    for (int a = 0; a < TP; ++a) {
      m[a] = -INFINITY;
      l[a] = 0.f;
#pragma unroll
      for (int b = 0; b < RV; ++b) o[a][b] = 0.f;
    }
    int buf = 0;
    for (int i = it.t0 + warp; i < it.t1; i += warps, buf ^= 1) {
      T* k = sK + buf * TK * pitch;
      if (i + warps < it.t1) {
        fetch(i + warps, buf ^ 1);
        copy_wait<1>();
      } else {
        copy_wait<0>();
      }
      __syncwarp();
      const int32_t t = cache_tile(it.k, i) * TK + lane;     // this lane's event
      float2 s2[TP];
#pragma unroll
      for (int a = 0; a < TP; ++a) s2[a] = make_float2(0.f, 0.f);
      for (int col = 0; col < r; col += 4) {
        const float4 y = ld4(k + lane * pitch + col);
#pragma unroll
        for (int a = 0; a < TP; ++a) {
          if (a >= rows) break;
          const float4 x = ld4(sQ + a * r + col);
          s2[a] = fma_f2(make_float2(x.x, x.y), make_float2(y.x, y.y), s2[a]);
          s2[a] = fma_f2(make_float2(x.z, x.w), make_float2(y.z, y.w), s2[a]);
        }
      }
      const bool masked = it.k.pmin < t - lane + TK - 1 || low_max > t - lane;
      float s[TP];
      bool odd = false;
#pragma unroll
      for (int a = 0; a < TP; ++a) {
        if (a >= rows) break;
        s[a] = (s2[a].x + s2[a].y) * p.scale2;
        if (masked) {
          const int32_t pos = cache_pos(it.x, cache_div(c, pair0 + a));
          const bool fin = fabsf(s[a]) < INFINITY;
          const bool see = t <= pos && (t >= cache_low(c, pos) || t < c.n_sink);
          odd |= !fin;
          if (!fin && see) poison |= 1u << a;
          s[a] = see && fin ? s[a] : -INFINITY;
        }
      }
      if (__any_sync(0xffffffffu, odd)) {
        clear_rows(k, TK, r, lane, 32);
        __syncwarp();
      }
#pragma unroll
      for (int a = 0; a < TP; ++a) {
        if (a >= rows) break;
        const float mn = fmaxf(m[a], warp_max(s[a])), mu = mn > -INFINITY ? mn : 0.f;
        if (mn != m[a]) {
          const float f = m[a] > -INFINITY ? ex2_approx(m[a] - mn) : 0.f;
          m[a] = mn;
          l[a] *= f;
#pragma unroll
          for (int b = 0; b < RV; ++b) o[a][b] *= f;
        }
        const float e = ex2_approx(s[a] - mu);
        l[a] += e;                         // this lane's share
        sW[a * TK + lane] = e;
      }
      __syncwarp();
      for (int d = 0; d < TK; d += 4) {
        float v[4][RV];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int b = 0; b < RV; ++b) {
            const int col = lane + 32 * b;
            v[e][b] = col < r ? to_f(k[(d + e) * pitch + col]) : 0.f;
          }
#pragma unroll
        for (int a = 0; a < TP; ++a) {
          if (a >= rows) break;
          const float4 w = ld4(sW + a * TK + d);
#pragma unroll
          for (int b = 0; b < RV; ++b)
            o[a][b] = fmaf(w.w, v[3][b], fmaf(w.z, v[2][b], fmaf(w.y, v[1][b],
                      fmaf(w.x, v[0][b], o[a][b]))));
        }
      }
      __syncwarp();
    }
    // ---- the warps' results meet
    poison = __reduce_or_sync(0xffffffffu, poison);
#pragma unroll
    for (int a = 0; a < TP; ++a) {
      if (a >= rows) break;
      l[a] = warp_sum(l[a]);
      if ((poison >> a) & 1 || m[a] == INFINITY) l[a] = NAN;
      if (lane == 0) {
        s_m[warp][a] = m[a];
        s_l[warp][a] = l[a];
      }
    }
    __syncthreads();                       // every warp is done with its tiles
#pragma unroll
    for (int a = 0; a < TP; ++a) {
      if (a >= rows) break;
      float mall = -INFINITY;
      for (int w = 0; w < warps; ++w) mall = fmaxf(mall, s_m[w][a]);
      const float f = m[a] > -INFINITY ? ex2_approx(m[a] - mall) : 0.f;
#pragma unroll
      for (int b = 0; b < RV; ++b)
        if (lane + 32 * b < r) sO[(warp * TP + a) * r + lane + 32 * b] = o[a][b] * f;
    }
    __syncthreads();
    const int64_t slot0 = ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * TP;
    for (int a = warp; a < rows; a += warps) {
      float mall = -INFINITY, lall = 0.f;
      for (int w = 0; w < warps; ++w) mall = fmaxf(mall, s_m[w][a]);
      const float mu = mall > -INFINITY ? mall : 0.f;
      for (int w = 0; w < warps; ++w) lall = fmaf(s_l[w][a], ex2_approx(s_m[w][a] - mu), lall);
      const float inv = it.whole ? (lall != 0.f ? 1.f / lall : 0.f) : 1.f;
      for (int col = lane; col < r; col += 32) {
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += sO[(w * TP + a) * r + col];
        if (it.whole) out[a * r + col] = from_f<T>(v * inv);
        else p.part_o[(slot0 + a) * r + col] = v;
      }
      if (lane == 0) {
        if (it.whole) {
          const float l2 = lall != 0.f ? mall + log2f(lall) : -INFINITY;
          if (p.lse) p.lse[at0 + a] = l2 * kLn2;
          if (p.lse2) p.lse2[at0 + a] = l2;
        } else {
          p.part_ml[slot0 + a] = make_float2(mall, lall);
        }
      }
    }
    if (tid == 0 && !it.whole && it.starts) {
      join->pair0 = at0;
      join->parts = it.parts;
      join->rows = rows;
    }
  }
}

// The block that CTA blockIdx.x began and did not finish, part by part in the order of
// the events.  One warp per row.
template <typename T>
__global__ void __launch_bounds__(256) cache_simt_join_kernel(CacheAttn p, int mt) {
  tc::pdl_trigger();
  tc::pdl_wait();
  const CacheJoin j = p.join[blockIdx.x];
  const int lane = threadIdx.x & 31, r = p.c.r;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (row >= j.rows) return;
  auto slot = [&](int i) -> int64_t {
    return ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * mt + row;
  };
  float m = -INFINITY, l = 0.f;
  for (int i = 0; i < j.parts; ++i) m = fmaxf(m, p.part_ml[slot(i)].x);
  const float mu = m > -INFINITY ? m : 0.f;
  for (int i = 0; i < j.parts; ++i) {
    const float2 ml = p.part_ml[slot(i)];
    l = fmaf(ex2_approx(ml.x - mu), ml.y, l);
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int64_t at = j.pair0 + row;
  for (int col = lane; col < r; col += 32) {
    float v = 0.f;
    for (int i = 0; i < j.parts; ++i)
      v = fmaf(ex2_approx(p.part_ml[slot(i)].x - mu), p.part_o[slot(i) * r + col], v);
    ((T*)p.out)[at * r + col] = from_f<T>(v * inv);
  }
  if (lane == 0) {
    const float l2 = l != 0.f ? m + log2f(l) : -INFINITY;
    if (p.lse) p.lse[at] = l2 * kLn2;
    if (p.lse2) p.lse2[at] = l2;
  }
}

// ---------------------------------------------------------------- mass
template <typename T>
__global__ void __launch_bounds__(256, 2) cache_mass_rows_kernel(CacheAttn p) {
  using Line = ByTiles<MT, KT>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ CacheSplit split;
  __shared__ float s_lse[MT];
  __shared__ int32_t s_pos[MT];
  __shared__ float s_sum[16][KT];
  const CacheCall& c = p.c;
  const int r = c.r, pitch = row_pitch<T>(r), tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  T* sK = (T*)smem;
  T* sQ = sK + KT * pitch;
  tc::pdl_trigger();
  tc::pdl_wait();
  cache_split<Line>(c, 1, false, *(CacheSplitSpace*)smem, &split);
  const CacheSplit run = split;
  CacheJoin* join = p.join + blockIdx.x;
  if (tid == 0) join->rows = 0;
  CacheItems<Line> items;
  items.start(c, run);
  CacheItem<Line> it;
  while (items.next(c, it)) {
    const CacheBlock& all = it.k.all;
    const int32_t t0 = it.k.tile * KT;
    const uint32_t pairs = (uint32_t)it.x.n * (uint32_t)c.heads;
    const T* pool = (const T*)p.pool;
    __syncthreads();
    copy_rows(sK, pool, KT, r, tid, 256, [&](int row) -> const T* {
      const int64_t at = seen_row(c, all, it.u, t0 + row);
      return at < 0 ? nullptr : pool + at * r;
    });
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = it.t0; i < it.t1; ++i) {
      const uint32_t pair0 = (uint32_t)(it.k.first + i) * MT;
      const int64_t at0 = it.x.row0 * c.heads + pair0;
      const int rows = (int)min((uint32_t)MT, pairs - pair0);
      if (i > it.t0) __syncthreads();
      copy_rows(sQ, (const T*)p.q, MT, r, tid, 256, [&](int row) -> const T* {
        return row < rows ? (const T*)p.q + (at0 + row) * r : nullptr;
      });
      copy_commit();
      if (tid < MT) {
        s_lse[tid] = tid < rows ? p.lse2[at0 + tid] : 0.f;
        s_pos[tid] = tid < rows ? cache_pos(it.x, cache_div(c, pair0 + tid)) : -1;
      }
      copy_wait<0>();
      __syncthreads();
      float s[4][4];
      score_tile(sQ, sK, r, ty, tx, s);
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int32_t pos = s_pos[4 * ty + a], low = cache_low(c, pos);
        const float lse = s_lse[4 * ty + a];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int32_t t = t0 + tx + 16 * j;
          const float e = ex2_approx(fmaf(s[a][j], p.scale2, -lse));
          if (t <= pos && (t >= low || t < c.n_sink)) sum[j] += e;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) s_sum[ty][tx + 16 * j] = sum[j];
    __syncthreads();
    if (tid < KT) {
      const int32_t t = t0 + tid;
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) v += s_sum[k][tid];
      if (!it.whole) {
        p.part_ml[((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * KT + tid].x = v;
      } else if (cache_seen(c, all, t, t + 1)) {
        const int64_t at = cache_row(c, c.table, c.stride, it.u, t);
        if (at >= 0) atomicAdd(&p.mass[at], v);
      }
    }
    if (tid == 0 && !it.whole && it.starts) {
      join->pair0 = ((int64_t)it.u << 32) | (uint32_t)t0;
      join->parts = it.parts;
      join->rows = min(KT, all.pmax + 1 - t0);
    }
  }
}

__global__ void __launch_bounds__(KT) cache_mass_rows_join_kernel(CacheAttn p) {
  tc::pdl_trigger();
  tc::pdl_wait();
  const CacheJoin j = p.join[blockIdx.x];
  if ((int)threadIdx.x >= j.rows) return;
  const CacheCall& c = p.c;
  const int u = (int)(j.pair0 >> 32);
  const int32_t t = (int32_t)(uint32_t)j.pair0 + threadIdx.x;
  if (!cache_seen(c, cache_all<KT>(c, cache_user(c, u)), t, t + 1)) return;
  float sum = 0.f;
  for (int i = 0; i < j.parts; ++i)
    sum += p.part_ml[((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * KT + threadIdx.x].x;
  const int64_t at = cache_row(c, c.table, c.stride, u, t);
  if (at >= 0) atomicAdd(&p.mass[at], sum);
}

// ---------------------------------------------------------------- launches
// A kernel's limit of dynamic shared memory is set once for a device, to all there is beside
// its static part: set to each launch's own need, a call of a cache of another rank could
// lower it between another thread's setting and its launch.
template <void (*Kernel)(CacheAttn)>
cudaError_t launch_with(int grid, int threads, size_t smem, const CacheAttn& a, cudaStream_t s) {
  static std::atomic<uint64_t> attr_devices{0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(attr_devices.load() >> (dev & 63) & 1)) {
    cudaFuncAttributes f;
    cudaError_t e = cudaFuncGetAttributes(&f, Kernel);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemMax - (int)f.sharedSizeBytes);
    if (e != cudaSuccess) return e;
    attr_devices |= 1ull << (dev & 63);
  }
  smem = std::max(smem, sizeof(CacheSplitSpace));
  return tc::launch_dependent(Kernel, dim3(grid), dim3(threads), smem, s, 1, a);
}

template <typename T>
cudaError_t attn_t(CacheAttn a, int num_sms, cudaStream_t s) {
  const int r = a.c.r, pitch = r + 16 / (int)sizeof(T);
  a.min_quota = 1;
  int mt, grid = num_sms;
  cudaError_t e;
  if (a.pairs <= TP * (int64_t)a.c.B) {
    mt = TP;
    // as many warps as two tiles of each leave room for
    const size_t warp = 2 * TK * pitch * sizeof(T) + TP * TK * 4;
    const int warps = (int)std::min<size_t>(8, (208 * 1024 - TP * r * 4) / warp);
    const size_t tiles = std::max<size_t>(warps * 2 * TK * pitch * sizeof(T),
                                          (size_t)warps * TP * r * 4);
    const size_t smem = TP * r * 4 + warps * TP * TK * 4 + tiles;
    a.never_cut = cache_most_tiles(a.c, TP, TK) <= 16;
    if (r <= 32) e = launch_with<cache_tokens_kernel<T, 1>>(num_sms, 32 * warps, smem, a, s);
    else if (r <= 64) e = launch_with<cache_tokens_kernel<T, 2>>(num_sms, 32 * warps, smem, a, s);
    else if (r <= 128) e = launch_with<cache_tokens_kernel<T, 4>>(num_sms, 32 * warps, smem, a, s);
    else e = launch_with<cache_tokens_kernel<T, 8>>(num_sms, 32 * warps, smem, a, s);
  } else {
    mt = MT;
    const size_t smem = (MT + (r <= 128 ? 1 : 2) * KT) * pitch * sizeof(T) + MT * (KT + 4) * 4;
    a.never_cut = cache_most_tiles(a.c, MT, KT) <= 4;
    if (r <= 128) grid = 2 * num_sms;
    if (r <= 64) e = launch_with<cache_rows_kernel<T, 1>>(grid, 256, smem, a, s);
    else if (r <= 128) e = launch_with<cache_rows_kernel<T, 2>>(grid, 256, smem, a, s);
    else e = launch_with<cache_rows_kernel<T, 4>>(grid, 256, smem, a, s);
  }
  cache_launched(a, a.never_cut ? 1 : 2);
  if (e != cudaSuccess || a.never_cut) return e;
  return tc::launch_dependent(cache_simt_join_kernel<T>, dim3(grid, mt / 8), dim3(256), 0, s, 1, a,
                              mt);
}

template <typename T>
cudaError_t mass_t(const CacheAttn& a, int num_sms, cudaStream_t s) {
  const size_t smem = (MT + KT) * (a.c.r + 16 / sizeof(T)) * sizeof(T);
  const int grid = a.c.r <= 128 ? 2 * num_sms : num_sms;
  cudaError_t e = launch_with<cache_mass_rows_kernel<T>>(grid, 256, smem, a, s);
  if (e != cudaSuccess) return e;
  cache_launched(a, 2);
  return tc::launch_dependent(cache_mass_rows_join_kernel, dim3(grid), dim3(KT), 0, s, 1, a);
}

}  // namespace

cudaError_t launch_cache_attn_simt(int elem, const CacheAttn& a, int num_sms, cudaStream_t s) {
  return elem == 4 ? attn_t<float>(a, num_sms, s) : attn_t<__nv_bfloat16>(a, num_sms, s);
}
cudaError_t launch_cache_mass_simt(int elem, const CacheAttn& a, int num_sms, cudaStream_t s) {
  return elem == 4 ? mass_t<float>(a, num_sms, s) : mass_t<__nv_bfloat16>(a, num_sms, s);
}

}  // namespace llatte
