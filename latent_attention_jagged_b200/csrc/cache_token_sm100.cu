// Attention of few new rows over the paged latent cache (bf16, rank 64, 128 or 256):
// the form for single tokens.
//
// With 16 (query row, head) pairs or fewer the floor is reading the cache: 4 r flops per
// pair and event against 2 r bytes.  The 128-row tensor-memory products of
// cache_attn_sm100.cu would run on padding, and every tile would wait for the chain
// S -> softmax -> P C; here the warps do not wait for one another at all.  A block of
// 16 pairs is one m16 operand; of a tile of 128 events each of 8 warps takes 16, with
// its own running maximum, sum and 16 x r result in registers (mma.sync, scores and
// weights never leave them), and the 8 results meet once per item.  A ninth warp keeps
// 192 KB of tiles on their way.
//
// Measured (64 users, 2000 to 8000 events, 8 heads, rank 256: 159 MB): 45 us, half the
// rate of HBM.  Its loads do not bound it (DRAM 41 % busy, tensor pipe 25 %, issue slots
// 17 %): each of two warps a scheduler waits for its own chain of
// ldmatrix, products and softmax, 64 products a tile of which half are padding at 8
// pairs.
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "cache.h"
#include "cache_call.cuh"
#include "cache_issue.cuh"
#include "cache_sched.cuh"
#include "tc_common.cuh"
#include "tc_drain.cuh"

namespace llatte {

using namespace tc;

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int MT = 16;                    // pairs of a block
constexpr int KT = 128;                   // events of a tile
constexpr int NW = 8;                     // consumer warps, 16 events of a tile each
// Three warpgroups, the third for the producer: the launch's 168 registers a thread
// are dealt out again, 128 threads x (232 + 232 + 40) = 384 x 168.  At r = 256 queries
// and results alone take 192, and what does not fit is read back from local memory in
// every tile (with all of shared memory in use little of it stays in L1), so that the
// consumers take 240 and leave the producer 24 (64 users of 2000 to 8000 events, 8 heads:
// 48 -> 45 us; at r = 128 the producer's own spills cost more, 29 -> 30 us).
constexpr int kThreads = 384;
template <int R> constexpr int kRegsConsume = R == 256 ? 240 : 232;
template <int R> constexpr int kRegsProduce = R == 256 ? 24 : 40;
static_assert(2 * kRegsConsume<128> + kRegsProduce<128> <= 504 &&
              2 * kRegsConsume<256> + kRegsProduce<256> <= 504, "registers of the launch");

template <int R>
struct Cfg {
  static constexpr int RSUB = R / 64;
  static constexpr int KS = 768 / R;                   // 192 KB of tiles
  static constexpr uint32_t KV_SUB = KT * 128;
  static constexpr uint32_t KV_BYTES = RSUB * KV_SUB;
  static constexpr uint32_t MEET = NW * MT * 64 * 4;   // 64 columns of every warp's result
  static constexpr uint32_t BAR_BYTES = 512;
  static constexpr size_t SMEM = 1024 + KS * KV_BYTES + MEET + BAR_BYTES + 3 * NW * MT * 4;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(KS * KV_BYTES >= sizeof(CacheSplitSpace), "split");
};

// The consumer warps meet.
__device__ __forceinline__ void meet_sync() {
  asm volatile("bar.sync 2, %0;" ::"n"(32 * NW) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The two bf16 numbers of a register in fp32.
__device__ __forceinline__ float2 unpack_bf16(uint32_t p) {
  return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}

// The warp clears the latents of its 16 events that are not finite.
template <int R>
__device__ __forceinline__ void clear_rows(uint8_t* kv, int first) {
  const int lane = threadIdx.x & 31, k = first + (lane & 15);
  bool bad = false;
  for (int s = lane >> 4; s < R / 64; s += 2) {
    const uint4* e = (const uint4*)(kv + s * (KT * 128) + k * 128);
    for (int j = 0; j < 8; ++j) {
      const uint4 x = e[j];
      for (uint32_t y : {x.x, x.y, x.z, x.w})
        bad |= (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
    }
  }
  bad |= __shfl_xor_sync(0xffffffffu, (int)bad, 16) != 0;
  if (bad) {
    for (int s = lane >> 4; s < R / 64; s += 2)
      for (int j = 0; j < 8; ++j)
        ((uint4*)(kv + s * (KT * 128) + k * 128))[j] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();               // the slot's next writes come from TMA
  __syncwarp();
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1)
cache_token_kernel(const __grid_constant__ CUtensorMap tmC, const CacheAttn p) {
  using C = Cfg<R>;
  using Line = ByRows<MT, KT>;
  constexpr int RSUB = C::RSUB, KS = C::KS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sKV = smem;
  float* meet = (float*)(sKV + KS * C::KV_BYTES);          // [NW][MT][64]
  uint64_t* bars = (uint64_t*)((uint8_t*)meet + C::MEET);
  uint64_t* kv_full = bars;                // [KS]
  uint64_t* kv_empty = kv_full + KS;       // [KS]
  volatile int* abort_flag = (volatile int*)(kv_empty + KS);
  volatile int* last_flag = abort_flag + 1;
  uint64_t* never = kv_empty + KS + 1;     // nothing arrives (injected timeout)
  CacheSplit* split = (CacheSplit*)(never + 1);
  static_assert((2 * KS + 2) * 8 + sizeof(CacheSplit) <= C::BAR_BYTES, "barriers");
  float* sm_m = (float*)((uint8_t*)bars + C::BAR_BYTES);   // [NW][MT]
  float* sm_l = sm_m + NW * MT;
  float* sm_r = sm_l + NW * MT;

  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheCall& c = p.c;
  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], NW); }
    mbar_init(never, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmC);
  }
  pdl_wait();
  cache_split<Line>(c, p.min_quota, p.never_cut, *(CacheSplitSpace*)sKV, split);
  fence_proxy_async_smem();               // the ring's next writes come from TMA
  __syncthreads();
  const CacheSplit run = *split;

  if (warp >= NW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsProduce<R>));
    if (warp == NW) {
    CacheItems<Line> items;
    items.start(c, run);
    CacheItem<Line> it;
    // ------------------------------------------------------------ producer
    // Lane l < boxes of a tile gathers box l (as in cache_attn_sm100.cu).
    uint32_t g = 0;
    const uint64_t policy = policy_stream(!p.lse2);   // the accumulation reads them again
    const int32_t P = min(1 << c.page_shift, kCacheBox);
    const int np = KT / P;
    const int32_t outside = c.n_pages << c.page_shift;
    bool ok = true;
    while (ok && items.next(c, it)) {
      if (it.x.len == 0) continue;
      const int32_t* row = c.table + (int64_t)it.u * c.stride;
      auto place = [&](int i) -> int32_t {
        const int32_t t = cache_tile(it.k, i) * KT + lane * P;
        if (lane >= np || !cache_seen(c, it.k, t, t + P)) return outside;
        const int32_t page = __ldg(row + (t >> c.page_shift));
        if ((uint32_t)page < (uint32_t)c.n_pages)
          return (page << c.page_shift) + (t & ((1 << c.page_shift) - 1));
        atomicOr(c.status, LLATTE_DEV_BAD_ID);
        return outside;
      };
      int32_t y = place(it.t0);
      for (int i = it.t0; i < it.t1; ++i, ++g) {
        const int32_t y_next = i + 1 < it.t1 ? place(i + 1) : 0;
        const int st = g % KS;
        if (lane == 0) {
          ok = mbar_wait(&kv_empty[st], ((g / KS) & 1) ^ 1, abort_flag, c.status);
          if (ok) mbar_arrive_expect_tx(&kv_full[st], C::KV_BYTES);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < np) {
          uint8_t* dst = sKV + st * C::KV_BYTES + lane * P * 128;
#pragma unroll
          for (int s = 0; s < RSUB; ++s)
            tma_load_2d_hint(&tmC, &kv_full[st], dst + s * C::KV_SUB, s * 64, y, policy);
        }
        y = y_next;
      }
    }
    __syncwarp();
    if (lane == 0) drain_ring(kv_full, KS, g, c.status);   // (see cache_attn_sm100.cu)
    __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsConsume<R>));
    CacheItems<Line> items;
    items.start(c, run);
    CacheItem<Line> it;
    // ------------------------------------------------------------ consumers
    const int grp = lane >> 2, t4 = lane & 3;          // row (and row + 8), column pair
    uint32_t g = 0;
    // an injected timeout: this warp has given up before its first tile
    bool ok = !(p.inject && warp == 0) ||
              warp_wait(never, 0, abort_flag, c.status, kInjectTimeoutNs);
    // ldmatrix rows of this lane: events 8 * (lane / 16) + lane % 8 for S, and
    // 8 * (lane / 8 % 2) + lane % 8 for P C; 16-byte chunks are XORed with event % 8
    const uint32_t k_row = (warp * 16 + ((lane >> 4) << 3) + (lane & 7)) * 128;
    const uint32_t v_row = (warp * 16 + (((lane >> 3) & 1) << 3) + (lane & 7)) * 128;
    const uint32_t k_chunk = (lane >> 3) & 1, v_chunk = lane >> 4, xr = lane & 7;
    while (items.next(c, it)) {
      const int64_t pair0 = (int64_t)it.b * MT;
      const int32_t rows = (int32_t)min((int64_t)MT, (int64_t)it.x.n * c.heads - pair0);
      const int64_t at0 = it.x.row0 * c.heads + pair0;
      const bool few = rows <= 8;
      if (it.x.len == 0) {                 // no event: zeros
        for (int i = threadIdx.x; i < rows * (R / 8); i += 32 * NW)
          ((uint4*)((__nv_bfloat16*)p.out + at0 * R))[i] = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; i < rows; i += 32 * NW) {
          if (p.lse) p.lse[at0 + i] = -INFINITY;
          if (p.lse2) p.lse2[at0 + i] = -INFINITY;
        }
        continue;
      }
      // the block's queries as A operands: rows grp and grp + 8 (zeros past the last)
      uint32_t qa[R / 16][4];
#pragma unroll
      for (int k = 0; k < R / 16; ++k) {
        const uint32_t* q0 = (const uint32_t*)((const __nv_bfloat16*)p.q + (at0 + grp) * R) + k * 8 + t4;
        const uint32_t* q1 = q0 + 8 * (R / 2);
        qa[k][0] = grp < rows ? __ldg(q0) : 0u;
        qa[k][1] = grp + 8 < rows ? __ldg(q1) : 0u;
        qa[k][2] = grp < rows ? __ldg(q0 + 4) : 0u;
        qa[k][3] = grp + 8 < rows ? __ldg(q1 + 4) : 0u;
      }
      int32_t pos[2], low[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t r = min(grp + 8 * h, rows - 1);
        pos[h] = cache_pos(it.x, cache_div(c, (uint32_t)(pair0 + r)));
        low[h] = cache_low(c, pos[h]);
      }
      const int32_t low_max = cache_low(c, it.k.pmax);
      float o[R / 8][4];
#pragma unroll
      for (int k = 0; k < R / 8; ++k) o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.f;
      // maximum, sum of the weights and of the rounded ones
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lr[2] = {0.f, 0.f};
      for (int i = it.t0; ok && i < it.t1; ++i, ++g) {
        const int st = g % KS;
        bool w = mbar_wait(&kv_full[st], (g / KS) & 1, abort_flag, c.status);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        const int32_t t0 = cache_tile(it.k, i) * KT + warp * 16;
        if (t0 > it.k.pmax) {              // nothing of this warp's events is there
          __syncwarp();
          if (lane == 0) mbar_arrive(&kv_empty[st]);
          continue;
        }
        uint8_t* kv = sKV + st * C::KV_BYTES;
        const uint32_t kv_addr = smem_u32(kv);
        // S = Q C^T: 16 pairs x 8 events twice (even and odd steps in accumulators of their
        // own cost 8 registers more than they gain)
        float v[2][4];                     // [event group j][row half * 2 + event]
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] = 0.f;
#pragma unroll
        for (int k = 0; k < R / 16; ++k) {
          uint32_t b[4];
          ldsm4(kv_addr + (k >> 2) * C::KV_SUB + k_row + (((2 * (k & 3) + k_chunk) ^ xr) << 4), b);
          mma16816(v[0], qa[k], b[0], b[1]);
          mma16816(v[1], qa[k], b[2], b[3]);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] *= p.scale2;
        bool poison[2] = {false, false};
        if (it.k.pmin < t0 + 15 || low_max > t0) {
          // some row hides some of the 16 events
          bool odd = false;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool fin = fabsf(v[j][e]) < INFINITY;
              const int h = e >> 1;
              const int32_t t = t0 + 8 * j + 2 * t4 + (e & 1);
              const bool see = t <= pos[h] && (t >= low[h] || t < c.n_sink);
              if (!fin && grp + 8 * h < rows) {
                odd = true;
                poison[h] |= see;
              }
              v[j][e] = see && fin ? v[j][e] : -INFINITY;
            }
          if (__any_sync(0xffffffffu, odd)) clear_rows<R>(kv, warp * 16);
        }
        // running maxima; O and the sums keep their base until one grows by more than
        // kGrow (a row that has seen nothing yet takes the first maximum it meets)
        float mt[2];
        bool grow = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mt[h] = fmaxf(fmaxf(v[0][2 * h], v[0][2 * h + 1]), fmaxf(v[1][2 * h], v[1][2 * h + 1]));
          mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 1));
          mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 2));
          grow |= mt[h] > m[h] + kGrow;
        }
        if (__any_sync(0xffffffffu, grow)) {
          float f[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float mn = fmaxf(m[h], mt[h]);
            f[h] = m[h] > -INFINITY ? ex2_approx(m[h] - mn) : 0.f;
            m[h] = mn;
            l[h] *= f[h];
            lr[h] *= f[h];
          }
          if (few) f[1] = f[0];
#pragma unroll
          for (int k = 0; k < R / 8; ++k) {
            o[k][0] *= f[0];
            o[k][1] *= f[0];
            o[k][2] *= f[1];
            o[k][3] *= f[1];
          }
        }
        // Weights.  For the product they are rounded to bf16.  Where rows 8 to 15 of the
        // operand are free what the rounding took goes there, rounded too, and the halves
        // of the result are added at the end: weights are then off by 2^-16 at most, for no
        // product more.  With more rows the result is divided by the sum of the rounded
        // weights, so that only their spread is left of the error (a second product for
        // the rests: 64 users of 2000 to 8000 events, 16 heads, r = 256, 59 -> 69 us).
        // The log sum is always that of the unrounded ones.
        uint32_t pa[4];
#pragma unroll
        for (int h = 1; h >= 0; --h) {
          const float mu = m[h] > -INFINITY ? m[h] : 0.f;
          const float a = ex2_approx(v[0][2 * h] - mu), b = ex2_approx(v[0][2 * h + 1] - mu);
          const float d = ex2_approx(v[1][2 * h] - mu), e = ex2_approx(v[1][2 * h + 1] - mu);
          l[h] += (a + b) + (d + e);
          if (poison[h]) l[h] = NAN;
          pa[h] = pack_bf16(a, b);
          pa[2 + h] = pack_bf16(d, e);
          const float2 x = unpack_bf16(pa[h]), y = unpack_bf16(pa[2 + h]);
          if (few && h == 0) {
            pa[1] = pack_bf16(a - x.x, b - x.y);
            pa[3] = pack_bf16(d - y.x, e - y.y);
          }
          if (!few) lr[h] += (x.x + x.y) + (y.x + y.y);
        }
        // O += P C: 16 columns a step
#pragma unroll
        for (int k = 0; k < R / 16; ++k) {
          uint32_t b[4];
          ldsm4t(kv_addr + (k >> 2) * C::KV_SUB + v_row + (((2 * (k & 3) + v_chunk) ^ xr) << 4), b);
          mma16816(o[2 * k], pa, b[0], b[1]);
          mma16816(o[2 * k + 1], pa, b[2], b[3]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&kv_empty[st]);
      }
      if (few) {
#pragma unroll
        for (int k = 0; k < R / 8; ++k) {
          o[k][0] += o[k][2];
          o[k][1] += o[k][3];
        }
      }
      // ---- the warps' results meet (after an abort too: every warp makes the same
      // number of meets, so none waits alone)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (few) lr[h] = l[h];
#pragma unroll
        for (int d = 1; d <= 2; d *= 2) {
          l[h] += __shfl_xor_sync(0xffffffffu, l[h], d);
          lr[h] += __shfl_xor_sync(0xffffffffu, lr[h], d);
        }
        if (t4 == 0) {
          sm_m[warp * MT + grp + 8 * h] = m[h];
          sm_l[warp * MT + grp + 8 * h] = l[h];
          sm_r[warp * MT + grp + 8 * h] = lr[h];
        }
      }
      meet_sync();
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mall = -INFINITY;
#pragma unroll
        for (int k = 0; k < NW; ++k) mall = fmaxf(mall, sm_m[k * MT + grp + 8 * h]);
        f[h] = m[h] > -INFINITY ? ex2_approx(m[h] - mall) : 0.f;
      }
      // A round sums 128 results of 16 (row, 64 columns): of 16 rows, or, where there
      // are no more than 8, of 8 rows and twice the columns.  A thread sums 4 columns
      // of a row.  Column pairs are XORed with the row, so that the 8 rows of a store
      // fall on different banks.
      const int line = threadIdx.x >> 4, c4 = threadIdx.x & 15, row = few ? line & 7 : line;
      float mall = -INFINITY, lall = 0.f, rall = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) mall = fmaxf(mall, sm_m[k * MT + row]);
      const float mu = mall > -INFINITY ? mall : 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) {
        const float w = ex2_approx(sm_m[k * MT + row] - mu);
        lall = fmaf(sm_l[k * MT + row], w, lall);
        rall = fmaf(sm_r[k * MT + row], w, rall);
      }
      if (mall == INFINITY) lall = NAN;
      const int64_t slot = ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * MT + row;
      // a whole block is divided by the sum of the rounded weights; a part becomes its mean
      // times the sum of the unrounded ones, which is what parts are joined by
      const float mul = lall != 0.f ? (it.whole ? 1.f : lall) / (lall == lall ? rall : NAN) : 0.f;
      auto put = [&](int unit, int q, int h) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          ((float2*)meet)[(warp * MT + 8 * unit + grp) * 32 + ((4 * k + t4) ^ (grp << 2))] =
              make_float2(o[8 * q + k][2 * h] * f[h], o[8 * q + k][2 * h + 1] * f[h]);
      };
      auto gather = [&](int q) {             // columns 64 q ..
        meet_sync();
        if (row < rows && q < R / 64) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < NW; ++k) {
            const float4 y = *(const float4*)(
                meet + ((k * MT + line) * 32 + ((2 * c4) ^ ((line & 7) << 2))) * 2);
            x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
          }
          if (it.whole)
            *(uint2*)((__nv_bfloat16*)p.out + (at0 + row) * R + q * 64 + c4 * 4) =
                make_uint2(pack_bf16(x.x * mul, x.y * mul), pack_bf16(x.z * mul, x.w * mul));
          else
            *(float4*)(p.part_o + slot * R + q * 64 + c4 * 4) =
                make_float4(x.x * mul, x.y * mul, x.z * mul, x.w * mul);
        }
        meet_sync();
      };
      if (few) {
#pragma unroll
        for (int q = 0; q < R / 64; q += 2) {
          put(0, q, 0);
          if (q + 1 < R / 64) put(1, q + 1, 0);
          gather(q + (line >> 3));
        }
      } else {
#pragma unroll
        for (int q = 0; q < R / 64; ++q) {
          put(0, q, 0);
          put(1, q, 1);
          gather(q);
        }
      }
      if (c4 == 0 && row < rows && !(few && line >= 8)) {
        if (it.whole) {
          const float l2 = lall != 0.f ? mall + log2f(lall) : -INFINITY;
          if (p.lse) p.lse[at0 + row] = l2 * kLn2;
          if (p.lse2) p.lse2[at0 + row] = l2;
        } else {
          p.part_ml[slot] = make_float2(mall, lall);
        }
      }
      if (it.whole) continue;
      // ---- a cut block: the CTA that comes last joins the parts, in the order of the
      // events (all CTAs come: none leaves its run early)
      __threadfence();
      meet_sync();
      if (threadIdx.x == 0) *last_flag = atomicAdd(&p.count[it.lead], 1) == it.parts - 1;
      meet_sync();
      if (!*last_flag) continue;
      __threadfence();
      if (threadIdx.x == 0) p.count[it.lead] = 0;        // for the next call
      for (int r = warp; r < rows; r += NW) {
        auto at_part = [&](int i) -> int64_t {
          return ((int64_t)(it.lead + i) * 2 + (i == 0 ? 1 : 0)) * MT + r;
        };
        float mj = -INFINITY, lj = 0.f;
        for (int i = lane; i < it.parts; i += 32) mj = fmaxf(mj, __ldcg(&p.part_ml[at_part(i)].x));
        mj = warp_max(mj);
        const float mju = mj > -INFINITY ? mj : 0.f;
        for (int i = lane; i < it.parts; i += 32) {
          const float2 ml = __ldcg(&p.part_ml[at_part(i)]);
          lj = fmaf(ex2_approx(ml.x - mju), ml.y, lj);
        }
        lj = warp_sum(lj);
        constexpr int CV = R / 64;           // column pairs of a lane
        float2 x[CV];
#pragma unroll
        for (int k = 0; k < CV; ++k) x[k] = make_float2(0.f, 0.f);
#pragma unroll 2
        for (int i = 0; i < it.parts; ++i) {
          const float w = ex2_approx(__ldcg(&p.part_ml[at_part(i)].x) - mju);
          const float2* src = (const float2*)(p.part_o + at_part(i) * R);
#pragma unroll
          for (int k = 0; k < CV; ++k) {
            const float2 y = __ldcg(src + lane + 32 * k);
            x[k].x = fmaf(w, y.x, x[k].x);
            x[k].y = fmaf(w, y.y, x[k].y);
          }
        }
        const float invj = lj != 0.f ? 1.f / lj : 0.f;
        uint32_t* dst = (uint32_t*)((__nv_bfloat16*)p.out + (at0 + r) * R);
#pragma unroll
        for (int k = 0; k < CV; ++k) dst[lane + 32 * k] = pack_bf16(x[k].x * invj, x[k].y * invj);
        if (lane == 0) {
          const float l2 = lj != 0.f ? mj + log2f(lj) : -INFINITY;
          if (p.lse) p.lse[at0 + r] = l2 * kLn2;
          if (p.lse2) p.lse2[at0 + r] = l2;
        }
      }
    }
  }
}

// Accumulated weights of few new rows: as in cache_mass_sm100.cu the scores are computed
// again transposed, here with mma.sync: a warp's 16 events are the m16 operand, the
// pairs come in groups of 8 columns, and the weights of an event are the sum over the
// columns of its row.  Nothing but the tiles' arrival is waited for.  A user's pairs
// beyond 16 take another pass over the tile in shared memory.
template <int R>
__global__ void __launch_bounds__(kThreads, 1)
cache_mass_token_kernel(const __grid_constant__ CUtensorMap tmC, const CacheAttn p) {
  using C = Cfg<R>;
  using Line = ByTiles<MT, KT>;
  constexpr int RSUB = C::RSUB, KS = C::KS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sKV = smem;
  uint64_t* bars = (uint64_t*)(sKV + KS * C::KV_BYTES + C::MEET);
  uint64_t* kv_full = bars;                // [KS]
  uint64_t* kv_empty = kv_full + KS;       // [KS]
  volatile int* abort_flag = (volatile int*)(kv_empty + KS);
  uint64_t* never = kv_empty + KS + 1;     // nothing arrives (injected timeout)
  CacheSplit* split = (CacheSplit*)(never + 1);

  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheCall& c = p.c;
  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], NW); }
    mbar_init(never, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmC);
  }
  pdl_wait();
  // no tile is cut: two CTAs that add to one event would do so in any order
  cache_split<Line>(c, 1, true, *(CacheSplitSpace*)sKV, split);
  fence_proxy_async_smem();
  __syncthreads();
  const CacheSplit run = *split;
  CacheItems<Line> items;
  items.start(c, run);
  CacheItem<Line> it;
  if (warp == NW) {
    uint32_t g = 0;
    const uint64_t policy = policy_stream(true);
    const int32_t P = min(1 << c.page_shift, kCacheBox);
    const int np = KT / P;
    const int32_t outside = c.n_pages << c.page_shift;
    bool ok = true;
    while (ok && items.next(c, it)) {
      int32_t y = outside;
      const int32_t t = it.k.tile * KT + lane * P;
      if (lane < np && cache_seen(c, it.k.all, t, t + P)) {
        const int32_t page = __ldg(c.table + (int64_t)it.u * c.stride + (t >> c.page_shift));
        if ((uint32_t)page < (uint32_t)c.n_pages)
          y = (page << c.page_shift) + (t & ((1 << c.page_shift) - 1));
        else
          atomicOr(c.status, LLATTE_DEV_BAD_ID);
      }
      const int st = g % KS;
      if (lane == 0) {
        ok = mbar_wait(&kv_empty[st], ((g / KS) & 1) ^ 1, abort_flag, c.status);
        if (ok) mbar_arrive_expect_tx(&kv_full[st], C::KV_BYTES);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (lane < np) {
        uint8_t* dst = sKV + st * C::KV_BYTES + lane * P * 128;
#pragma unroll
        for (int s = 0; s < RSUB; ++s)
          tma_load_2d_hint(&tmC, &kv_full[st], dst + s * C::KV_SUB, s * 64, y, policy);
      }
      ++g;
    }
    __syncwarp();
    if (lane == 0) drain_ring(kv_full, KS, g, c.status);   // (see cache_attn_sm100.cu)
    __syncwarp();
  } else if (warp < NW) {
    const int grp = lane >> 2, t4 = lane & 3;          // event (and event + 8), pair column
    // ldmatrix rows of this lane: events 8 * (lane / 8 % 2) + lane % 8, chunk lane / 16
    const uint32_t k_row = (warp * 16 + (((lane >> 3) & 1) << 3) + (lane & 7)) * 128;
    const uint32_t k_chunk = lane >> 4, xr = lane & 7;
    uint32_t g = 0;
    int held_u = -1, held_b = -1;                      // whose queries qb holds
    uint32_t qb[R / 16][4];
    float lse[2][2];
    int32_t pos[2][2];
    const bool ok = !(p.inject && warp == 0) ||        // an injected timeout (see above)
                    warp_wait(never, 0, abort_flag, c.status, kInjectTimeoutNs);
    while (ok && items.next(c, it)) {
      const int st = g % KS;
      bool w = mbar_wait(&kv_full[st], (g / KS) & 1, abort_flag, c.status);
      if (!__all_sync(0xffffffffu, w)) break;
      const int32_t t0 = it.k.tile * KT + warp * 16;
      const uint32_t kv_addr = smem_u32(sKV + st * C::KV_BYTES);
      const int32_t pairs = it.x.n * c.heads;
      float sum[2] = {0.f, 0.f};                       // of events grp and grp + 8
      for (int b = it.k.first; b <= it.k.last && t0 <= it.k.all.pmax; ++b) {
        if (it.u != held_u || b != held_b) {
          // 16 pairs as two B operands of 8 columns; pairs past the last are zeros
          held_u = it.u;
          held_b = b;
          const int64_t at0 = it.x.row0 * c.heads + (int64_t)b * MT;
          const int rows = min(MT, pairs - b * MT);
#pragma unroll
          for (int k = 0; k < R / 16; ++k) {
            const uint32_t* q0 =
                (const uint32_t*)((const __nv_bfloat16*)p.q + (at0 + grp) * R) + k * 8 + t4;
            const uint32_t* q1 = q0 + 8 * (R / 2);
            qb[k][0] = grp < rows ? __ldg(q0) : 0u;
            qb[k][1] = grp < rows ? __ldg(q0 + 4) : 0u;
            qb[k][2] = grp + 8 < rows ? __ldg(q1) : 0u;
            qb[k][3] = grp + 8 < rows ? __ldg(q1 + 4) : 0u;
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int a = 8 * n + 2 * t4 + e;        // this lane's column
              lse[n][e] = a < rows ? p.lse2[at0 + a] : 0.f;
              pos[n][e] = a < rows ? cache_pos(it.x, cache_div(c, b * MT + a)) : -1;
            }
        }
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < R / 16; ++k) {
          uint32_t a[4];
          ldsm4(kv_addr + (k >> 2) * C::KV_SUB + k_row + (((2 * (k & 3) + k_chunk) ^ xr) << 4), a);
          mma16816(s[0], a, qb[k][0], qb[k][1]);
          mma16816(s[1], a, qb[k][2], qb[k][3]);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t t = t0 + grp + 8 * (e >> 1), ps = pos[n][e & 1];
            const bool see = t <= ps && (t >= cache_low(c, ps) || t < c.n_sink);
            const float x = ex2_approx(fmaf(s[n][e], p.scale2, -lse[n][e & 1]));
            sum[e >> 1] += see ? x : 0.f;
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&kv_empty[st]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
        sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
        const int32_t t = t0 + grp + 8 * h;
        if (t4 == 0 && cache_seen(c, it.k.all, t, t + 1)) {
          const int64_t at = cache_row(c, c.table, c.stride, it.u, t);
          if (at >= 0) atomicAdd(&p.mass[at], sum[h]);
        }
      }
      ++g;
    }
  }
}

template <int R>
cudaError_t launch_mass_r(const CacheAttn& a, const CUtensorMap& tmC, int num_sms, cudaStream_t s) {
  using C = Cfg<R>;
  static std::atomic<uint64_t> attr_devices{0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(attr_devices.load() >> (dev & 63) & 1)) {
    cudaError_t e = cudaFuncSetAttribute(cache_mass_token_kernel<R>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    attr_devices |= 1ull << (dev & 63);
  }
  cache_launched(a, 1);
  return launch_dependent(cache_mass_token_kernel<R>, dim3(num_sms), dim3(kThreads), C::SMEM, s, 1,
                          tmC, a);
}

template <int R>
cudaError_t launch_r(CacheAttn a, const CUtensorMap& tmC, int num_sms, cudaStream_t s) {
  using C = Cfg<R>;
  static std::atomic<uint64_t> attr_devices{0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(attr_devices.load() >> (dev & 63) & 1)) {
    cudaError_t e = cudaFuncSetAttribute(cache_token_kernel<R>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    // the register split waits for what the launch does not have
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, cache_token_kernel<R>);
    if (e != cudaSuccess) return e;
    if (f.numRegs * 3 < 2 * kRegsConsume<R> + kRegsProduce<R>) return cudaErrorInvalidConfiguration;
    attr_devices |= 1ull << (dev & 63);
  }
  cache_launched(a, 1);
  return launch_dependent(cache_token_kernel<R>, dim3(num_sms), dim3(kThreads), C::SMEM, s, 1, tmC,
                          a);
}

}  // namespace

cudaError_t launch_cache_token(const CacheAttn& a, const CUtensorMap& tmC, int num_sms,
                               cudaStream_t s) {
  switch (a.c.r) {
    case 64: return launch_r<64>(a, tmC, num_sms, s);
    case 128: return launch_r<128>(a, tmC, num_sms, s);
    case 256: return launch_r<256>(a, tmC, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_cache_mass_token(const CacheAttn& a, const CUtensorMap& tmC, int num_sms,
                                    cudaStream_t s) {
  switch (a.c.r) {
    case 64: return launch_mass_r<64>(a, tmC, num_sms, s);
    case 128: return launch_mass_r<128>(a, tmC, num_sms, s);
    case 256: return launch_mass_r<256>(a, tmC, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace llatte
