// Attention over the paged latent cache for sm_100a (bf16, rank 64, 128 or 256).
//
//   s_it = scale q_i . c_t over the events row i sees,  P = softmax(s),
//   o_i = sum_t P_it c_t,  lse_i = log sum_t exp(s_it)
//
// One item = a block of MT (query row, head) pairs of one user and a run of its
// tiles of 128 events (cache_sched.cuh); K and V are one shared-memory copy of a
// tile, K-major for S = Q C^T and MN-major for O += P C, as in attn_sm100.cu.
// What differs from the batch kernel: a tile is gathered page by page (one TMA
// box per page and 64 columns, so pages of 16 to 128 rows cost the same bytes),
// rows hide events behind a window, a block may be cut between CTAs, and what a
// row does not see may hold any bits.
//
// MT = 128: blocks of many rows (chunks of new events, candidates), bound by the
// tensor pipe and the exponentials.  MT = 32: few pairs a user (single tokens),
// bound by reading the cache; the M = 128 products then use a quarter of their
// lanes, which costs nothing (about 1000 tensor cycles per 64 KB tile, of the 2750
// that HBM needs for it), the query block is 32 rows, and the ring gets the space.
//
// Hidden values.  P = 0 does not hide an infinity or NaN from the product P C, so
// in tiles where some row hides some event (the tile of the length's end, window
// edges, the diagonal) the softmax warps look for scores that are not finite; if
// there are any they clear the latents that are not finite in shared memory
// before the product, and rows that see one of them get NaN through their sum.
#include <cuda.h>

#include <algorithm>

#include "cache.h"
#include "cache_call.cuh"
#include "cache_sched.cuh"
#include "tc_common.cuh"
#include "tc_drain.cuh"
#include "tc_epilogue.cuh"
#include "tc_gemm.h"

namespace llatte {

using namespace tc;

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int KT = 128;                   // events of a tile

template <int R, int MT>
struct Cfg {
  static constexpr bool SMALL = MT == 32;
  static constexpr int KP = KT / 2;                    // events of a softmax warp
  static constexpr int RSUB = R / 64;
  static constexpr int OBUF = (2 * R + 2 * KT <= 512) ? 2 : 1;
  static constexpr int QBUF = SMALL || R <= 128 ? 2 : 1;
  static constexpr int KS = SMALL ? (R == 256 ? 3 : R == 128 ? 6 : 8) : (R == 256 ? 2 : 4);
  static constexpr uint32_t QSUB = MT * 128;           // one 64-wide sub-tile of a query block
  static constexpr uint32_t Q_BYTES = RSUB * QSUB;
  static constexpr uint32_t KV_SUB = KT * 128;
  static constexpr uint32_t KV_BYTES = RSUB * KV_SUB;
  static constexpr uint32_t S_COL = OBUF * R;
  // warps: MT = 128: producer 0, MMA 1, softmax 2..9, epilogue 10..13.  MT = 32:
  // softmax 0 and 4 (TMEM lanes 0..31 belong to warps 0 mod 4), producer 1,
  // MMA 2, epilogue 8.
  static constexpr int WARPS = SMALL ? 9 : 14;
  static constexpr int PROD = SMALL ? 1 : 0, MMA = SMALL ? 2 : 1;
  static constexpr int NSOFT = SMALL ? 2 : 8, EPI0 = SMALL ? 8 : 10, NEPI = SMALL ? 1 : 4;
  static constexpr uint32_t BAR_BYTES = 512;
  static constexpr uint32_t F_BYTES = 4 * MT * 8;      // sums, maxima, partial maxima
  static constexpr uint32_t STAGE = SMALL ? 0 : kStageBytes;
  static constexpr size_t SMEM = 1024 + QBUF * Q_BYTES + (size_t)KS * KV_BYTES + BAR_BYTES +
                                 F_BYTES + NEPI * STAGE;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(OBUF * R + 2 * KT <= 512, "TMEM budget");
  // an M = 128 product reads 16 KB from the start of a 32-row sub-tile
  static_assert(!SMALL || KS * KV_BYTES >= 16384, "operand reads stay in the buffers");
  // the split's prefix sums lie in the ring before its first load
  static_assert(KS * KV_BYTES >= 4 * (LLATTE_CACHE_MAX_BATCH + 1), "prefix sums");
};

// TMEM column (relative to the S buffer) of the packed bf16 P for events
// [16 kk, 16 kk + 16): each softmax warp packs its half into the first columns of
// its half of the buffer.
template <int KP>
__device__ __forceinline__ uint32_t p_col(int kk) {
  const int key = 16 * kk;
  return (uint32_t)((key / KP) * KP + (key % KP) / 2);
}

// Bits [lo, hi) of 64, both clamped.
__device__ __forceinline__ uint64_t bits_below(int64_t n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
}

// The 64 bytes x of this lane's row to dst (nullptr: none).
template <bool STAGED>
__device__ __forceinline__ void put64(uint32_t stg, const uint4 (&x)[4], void* dst) {
  if constexpr (STAGED) {
    stage_store(stg, x, dst);
  } else if (dst) {
#pragma unroll
    for (int j = 0; j < 4; ++j) ((uint4*)dst)[j] = x[j];
  }
}

template <int R, int MT>
__global__ void __launch_bounds__(32 * Cfg<R, MT>::WARPS, 1)
cache_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmC,
                  const CacheAttn p, const int min_quota) {
  using C = Cfg<R, MT>;
  using Line = ByRows<MT, KT>;
  constexpr int KP = C::KP, RSUB = C::RSUB, KS = C::KS, OBUF = C::OBUF, QBUF = C::QBUF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + QBUF * C::Q_BYTES;
  uint64_t* bars = (uint64_t*)(sKV + KS * C::KV_BYTES);
  uint64_t* q_full = bars;                 // [2]
  uint64_t* q_empty = bars + 2;            // [2]
  uint64_t* s_full = bars + 4;             // [2]
  uint64_t* p_full = bars + 6;             // [2] every softmax warp has written P
  uint64_t* p_empty = bars + 8;            // [2] P C done
  uint64_t* o_full = bars + 10;            // [2] last P C done, sums and maxima written
  uint64_t* o_free = bars + 12;            // [2] the epilogue has read O
  uint64_t* pair_bar = bars + 14;          // [4] the two softmax warps of a lane quadrant
  uint64_t* kv_full = bars + 18;           // [KS]
  uint64_t* kv_empty = kv_full + KS;       // [KS]
  uint64_t* drain = kv_empty + KS;
  uint32_t* tmem_slot = (uint32_t*)(drain + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  CacheSplit* split = (CacheSplit*)(tmem_slot + 2);
  static_assert((18 + 2 * KS + 1) * 8 + 8 + sizeof(CacheSplit) <= C::BAR_BYTES, "barriers");
  float* lbuf = (float*)((uint8_t*)bars + C::BAR_BYTES);     // [2][MT] row sums
  float* mbuf = lbuf + 2 * MT;                               // [2][MT] row maxima
  float* mx = mbuf + 2 * MT;                                 // [2][2][MT] partial maxima
  uint8_t* sStage = (uint8_t*)(mx + 4 * MT);

  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheCall& c = p.c;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], C::NSOFT);
      mbar_init(&p_empty[s], 1);
      mbar_init(&o_full[s], 1 + C::NSOFT);
      mbar_init(&o_free[s], C::NEPI);
    }
    for (int s = 0; s < KS; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 1); }
    for (int q = 0; q < 4; ++q) mbar_init(&pair_bar[q], 2);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmC);
  }
  for (int i = threadIdx.x; i < 2 * MT; i += blockDim.x) lbuf[i] = 0.f;
  if (warp == C::MMA) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // everything below reads what earlier kernels wrote
  pdl_wait();
  cache_split<Line>(c, min_quota, (int32_t*)sKV, split);
  fence_proxy_async_smem();               // the ring's next writes come from TMA
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const CacheSplit run = *split;

  if (warp == C::PROD) {
    // ------------------------------------------------------------ producer
    // Lane l < pages of a tile gathers page l; a page that no row of the block
    // sees, or that is outside the pool, reads as zeros (a box past the pool's
    // last row).
    uint32_t itm = 0, g = 0, qi = 0;
    const int32_t P = 1 << c.page_shift;
    const int np = KT >> c.page_shift;
    const int32_t outside = c.n_pages << c.page_shift;
    CacheItems<Line> items;
    items.start(c, run);
    CacheItem it;
    bool ok = true;
    while (ok && items.next(c, it)) {
      const CacheBlock blk = cache_block<MT, KT>(c, it.x, it.b);
      if (it.x.len == 0) continue;
      const int32_t* row = c.table + (int64_t)it.u * c.stride;
      // pool row of this lane's page in tile i of the piece
      auto place = [&](int i) -> int32_t {
        const int32_t t = cache_tile(blk, i) * KT + lane * P;
        if (lane >= np || !cache_seen(c, blk, t, t + P)) return outside;
        const int32_t page = __ldg(row + (t >> c.page_shift));
        if ((uint32_t)page < (uint32_t)c.n_pages) return page << c.page_shift;
        atomicOr(c.status, LLATTE_DEV_BAD_ID);
        return outside;
      };
      int32_t y = place(it.t0);
      const int qb = itm % QBUF;
      if (lane == 0) {
        ok = mbar_wait(&q_empty[qb], ((itm / QBUF) & 1) ^ 1, abort_flag, c.status);
        if (ok) {
          mbar_arrive_expect_tx(&q_full[qb], C::Q_BYTES);
          const int32_t qrow = (int32_t)(it.x.row0 * c.heads + (int64_t)it.b * MT);
#pragma unroll
          for (int s = 0; s < RSUB; ++s)
            tma_load_2d(&tmQ, &q_full[qb], sQ + qb * C::Q_BYTES + s * C::QSUB, s * 64, qrow);
          ++qi;
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
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
            tma_load_2d(&tmC, &kv_full[st], dst + s * C::KV_SUB, s * 64, y);
        }
        y = y_next;
      }
      ++itm;
    }
    __syncwarp();
    // after an abort the MMA thread may have left tiles unread
    if (lane == 0 && *abort_flag) {
      drain_ring(kv_full, KS, g, c.status);
      drain_ring(q_full, QBUF, qi, c.status);
    }
    __syncwarp();
  } else if (warp == C::MMA) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t IDESC_S = idesc_bf16(128, KT, false, false);
      constexpr uint32_t IDESC_O = idesc_bf16(128, R, false, true);
      uint32_t itm = 0, g = 0;
      bool ok = true;
      // S(gg) into S buffer gg & 1, which last held P(gg - 2): its product was
      // issued before this call and the tensor pipe works in order.
      auto issue_s = [&](uint32_t gg, uint32_t q_addr) -> bool {
        const int st = gg % KS;
        if (!mbar_wait(&kv_full[st], (gg / KS) & 1, abort_flag, c.status)) return false;
        tc_fence_after();
        const uint32_t kv_addr = smem_u32(sKV + st * C::KV_BYTES);
        const uint32_t d = tmem + C::S_COL + (gg & 1) * KT;
#pragma unroll
        for (int k = 0; k < R / 16; ++k) {
          const uint64_t ad = sdesc_sw128(q_addr + (k >> 2) * C::QSUB + (k & 3) * 32, 16, 1024);
          const uint64_t bd = sdesc_sw128(kv_addr + (k >> 2) * C::KV_SUB + (k & 3) * 32, 16, 1024);
          umma_bf16(d, ad, bd, IDESC_S, k > 0 ? 1u : 0u);
        }
        umma_commit(&s_full[gg & 1]);
        return true;
      };
      // O (+)= P(gg) C: P from TMEM, the tile read MN-major; `first` starts O anew.
      auto issue_pv = [&](uint32_t gg, bool first, int ob, uint32_t item) -> bool {
        if (!mbar_wait(&p_full[gg & 1], (gg >> 1) & 1, abort_flag, c.status)) return false;
        if (first && !mbar_wait(&o_free[ob], ((item / OBUF) & 1) ^ 1, abort_flag, c.status))
          return false;
        tc_fence_after();
        const int st = gg % KS;
        const uint32_t kv_addr = smem_u32(sKV + st * C::KV_BYTES);
        const uint32_t p_tmem = tmem + C::S_COL + (gg & 1) * KT;
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
          const uint64_t bd = sdesc_sw128(kv_addr + k * 2048, C::KV_SUB, 1024);
          umma_bf16_ts(tmem + ob * R, p_tmem + p_col<KP>(k), bd, IDESC_O,
                       (!first || k > 0) ? 1u : 0u);
        }
        umma_commit(&kv_empty[st]);
        umma_commit(&p_empty[gg & 1]);
        return true;
      };
      // The product of a tile is issued after the S of the next one, also across
      // items, so that a tile's softmax overlaps the next S.
      struct Pending { uint32_t g, item; int ob; bool first, last, valid; };
      Pending pend = {0, 0, 0, false, false, false};
      auto flush = [&]() -> bool {
        if (!pend.valid) return true;
        if (!issue_pv(pend.g, pend.first, pend.ob, pend.item)) return false;
        if (pend.last) umma_commit(&o_full[pend.ob]);
        pend.valid = false;
        return true;
      };
      CacheItems<Line> items;
      items.start(c, run);
      CacheItem it;
      while (ok && items.next(c, it)) {
        if (it.x.len == 0) continue;
        const int ob = itm % OBUF, qb = itm % QBUF;
        if (QBUF == 1 && !flush()) break;
        if (!mbar_wait(&q_full[qb], (itm / QBUF) & 1, abort_flag, c.status)) break;
        const uint32_t q_addr = smem_u32(sQ + qb * C::Q_BYTES);
        for (int i = it.t0; i < it.t1; ++i, ++g) {
          if (!issue_s(g, q_addr)) { ok = false; break; }
          if (i == it.t1 - 1) umma_commit(&q_empty[qb]);
          if (!flush()) { ok = false; break; }
          pend = {g, itm, ob, i == it.t0, i == it.t1 - 1, true};
        }
        ++itm;
      }
      if (ok) flush();
      umma_commit(drain);
      int dummy = 0;
      mbar_wait(drain, 0, &dummy, c.status);
    }
    __syncwarp();
  } else if (C::SMALL ? (warp == 0 || warp == 4) : (warp >= 2 && warp < 10)) {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3;
    const int part = C::SMALL ? warp >> 2 : (warp - 2) >> 2;    // half of the tile's events
    const int row = quad * 32 + lane;                  // pair in the block = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const float mul = p.scale2 == 0.f ? 1.f : fabsf(p.scale2);
    const float2 mul2 = make_float2(mul, mul);
    uint32_t g = 0, itm = 0, pphase = 0;
    bool ok = true;
    CacheItems<Line> items;
    items.start(c, run);
    CacheItem it;
    while (ok && items.next(c, it)) {
      const CacheBlock blk = cache_block<MT, KT>(c, it.x, it.b);
      if (it.x.len == 0) continue;
      const int ob = itm % OBUF;
      const uint32_t o_col = ob * R + part * (R / 2);          // this warp's half of O
      const uint32_t pairs = (uint32_t)it.x.n * (uint32_t)c.heads;
      const uint32_t pair = (uint32_t)it.b * MT + row;
      const bool valid = pair < pairs;
      const int32_t pos = valid ? cache_pos(it.x, (int)(pair / (uint32_t)c.heads)) : blk.pmax;
      const int32_t low = cache_low(c, pos);
      const bool idle = (uint32_t)it.b * MT + quad * 32 >= pairs;   // no row in this quadrant
      float m_run = -INFINITY, l_run = 0.f;     // running maximum (log2 units), partial sum
      bool poison = false;
      for (int i = it.t0; i < it.t1; ++i, ++g) {
        bool w = mbar_wait(&s_full[g & 1], (g >> 1) & 1, abort_flag, c.status);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        if (idle) {
          if (lane == 0) mbar_arrive(&p_full[g & 1]);
          continue;
        }
        tc_fence_after();
        const uint32_t s_addr = lane_base + C::S_COL + (g & 1) * KT + part * KP;
        const int32_t tile0 = cache_tile(blk, i) * KT;
        float v[KP];
        tmem_ld64(s_addr, v);
        if (p.scale2 <= 0.f) {
          const float f = p.scale2 == 0.f ? 0.f : -1.f;
#pragma unroll
          for (int k = 0; k < KP; ++k) v[k] *= f;
        }
        // some row hides some event of the tile (the same answer in every warp)
        if (blk.pmin < tile0 + KT - 1 || cache_low(c, blk.pmax) > tile0) {
          const int64_t t0 = tile0 + part * KP;
          uint64_t vis = bits_below((int64_t)pos + 1 - t0);
          if (c.window > 0) vis &= ~bits_below(low - t0) | bits_below(c.n_sink - t0);
          if (!valid) vis = ~0ull;
          float2 z2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < KP; k += 2)
            z2 = fma_f2(make_float2(v[k], v[k + 1]), make_float2(0.f, 0.f), z2);
          if (__any_sync(0xffffffffu, valid && !(z2.x + z2.y == 0.f))) {
            // a score is not finite: clear this warp's latents that are not
            uint8_t* kv = sKV + (g % KS) * C::KV_BYTES;
#pragma unroll 1
            for (int k = part * KP + lane; k < (part + 1) * KP; k += 32) {
              bool bad = false;
              for (int s = 0; s < RSUB; ++s) {
                const uint4* e = (const uint4*)(kv + s * C::KV_SUB + k * 128);
                for (int j = 0; j < 8; ++j) {
                  const uint4 x = e[j];
                  for (uint32_t y : {x.x, x.y, x.z, x.w})
                    bad |= (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
                }
              }
              if (!bad) continue;
              for (int s = 0; s < RSUB; ++s)
                for (int j = 0; j < 8; ++j)
                  ((uint4*)(kv + s * C::KV_SUB + k * 128))[j] = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
#pragma unroll
            for (int k = 0; k < KP; ++k) {
              const bool fin = fabsf(v[k]) < INFINITY;
              poison |= valid && !fin && ((vis >> k) & 1);
              v[k] = fin ? v[k] : -INFINITY;
            }
          }
#pragma unroll
          for (int k = 0; k < KP; ++k) v[k] = ((vis >> k) & 1) ? v[k] : -INFINITY;
        }
        float m8[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) m8[k] = -INFINITY;
#pragma unroll
        for (int k = 0; k < KP; k += 16) {
#pragma unroll
          for (int j = 0; j < 8; ++j) m8[j] = fmax3(m8[j], v[k + j], v[k + 8 + j]);
        }
        float mt = mul * fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])),
                               fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
        // the two halves of the row meet: both warps end with the same maximum
        float* mxs = mx + (g & 1) * 2 * MT;
        mxs[part * MT + row] = mt;
        if (!group_sync(&pair_bar[quad], pphase, abort_flag, c.status)) { ok = false; break; }
        mt = fmaxf(mt, mxs[(part ^ 1) * MT + row]);
        // O and l are rescaled only when the maximum grows by more than 2^8
        float scale = 1.f;
        bool resc = false;
        if (i == it.t0) {
          m_run = mt;
        } else if (mt > m_run + 8.f) {
          scale = ex2_approx(m_run - mt);
          m_run = mt;
          resc = true;
        }
        if (__any_sync(0xffffffffu, resc)) {
          // the previous product must be in O: the next phase of its p_empty
          bool w2 = mbar_wait(&p_empty[(g - 1) & 1], ((g - 1) >> 1) & 1, abort_flag, c.status);
          if (!__all_sync(0xffffffffu, w2)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int k = 0; k < R / 2; k += 32) {
            float o[32];
            tmem_ld32(lane_base + o_col + k, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= scale;
            tmem_st32(lane_base + o_col + k, o);
          }
          l_run *= scale;
        }
        // weights 2^(s - m), the sum in fp32 of the unrounded ones; a row that has
        // seen nothing yet subtracts 0 from its -inf
        const float m_use = m_run > -INFINITY ? m_run : 0.f;
        const float2 nm2 = make_float2(-m_use, -m_use);
        float2 l4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) l4[k] = make_float2(0.f, 0.f);
        float pk[KP / 2];                      // bf16 pairs
#pragma unroll
        for (int k = 0; k < KP / 2; ++k) {
          float2 x = fma_f2(make_float2(v[2 * k], v[2 * k + 1]), mul2, nm2);
          x.x = ex2_approx(x.x);
          x.y = ex2_approx(x.y);
          l4[k & 3] = add_f2(l4[k & 3], x);
          pk[k] = __uint_as_float(pack_bf16(x.x, x.y));
        }
        l_run += ((l4[0].x + l4[0].y) + (l4[1].x + l4[1].y)) +
                 ((l4[2].x + l4[2].y) + (l4[3].x + l4[3].y));
        tmem_st32(s_addr, pk);                 // waits for the store
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[g & 1]);
      }
      if (!ok) break;
      bool w4 = mbar_wait(&o_free[ob], ((itm / OBUF) & 1) ^ 1, abort_flag, c.status);
      if (!__all_sync(0xffffffffu, w4)) break;
      if (!idle) {
        if (poison || m_run == INFINITY) l_run = NAN;
        atomicAdd(&lbuf[ob * MT + row], l_run);     // zero before the two halves' sums
        if (part == 0) mbuf[ob * MT + row] = m_run;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_full[ob]);
      ++itm;
    }
  } else if (warp >= C::EPI0) {
    // ------------------------------------------------------------ epilogue
    const int quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t stg = smem_u32(sStage + (warp - C::EPI0) * C::STAGE);
    CacheJoin* join = p.join + blockIdx.x;
    const bool writer = warp == C::EPI0 && lane == 0;
    if (writer) join->rows = 0;
    uint32_t itm = 0;
    CacheItems<Line> items;
    items.start(c, run);
    CacheItem it;
    while (items.next(c, it)) {
      const uint32_t pairs = (uint32_t)it.x.n * (uint32_t)c.heads;
      const uint32_t pair = (uint32_t)it.b * MT + row;
      const bool valid = pair < pairs;
      const bool idle = (uint32_t)it.b * MT + quad * 32 >= pairs;
      const int64_t at = it.x.row0 * c.heads + pair;
      __nv_bfloat16* orow = valid ? (__nv_bfloat16*)p.out + at * R : nullptr;
      if (it.x.len == 0) {                 // no event: zeros
        if (idle) continue;
        const uint4 z[4] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0),
                            make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        for (int k = 0; k < R; k += 32) put64<!C::SMALL>(stg, z, orow ? orow + k : nullptr);
        if (valid && p.lse) p.lse[at] = -INFINITY;
        if (valid && p.lse2) p.lse2[at] = -INFINITY;
        continue;
      }
      const int ob = itm % OBUF;
      bool w = mbar_wait(&o_full[ob], (itm / OBUF) & 1, abort_flag, c.status);
      if (!__all_sync(0xffffffffu, w)) break;
      tc_fence_after();
      if (!idle) {
        const float l = lbuf[ob * MT + row], m = mbuf[ob * MT + row];
        lbuf[ob * MT + row] = 0.f;         // ready for the item that reuses this buffer
        if (it.whole) {
          const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll 1
          for (int k = 0; k < R; k += 64) {
            float v[64];
            tmem_ld64(lane_base + ob * R + k, v);
#pragma unroll
            for (int j = 0; j < 64; ++j) v[j] *= inv;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint4 x[4];
              pack_bf16x32(&v[32 * h], x);
              put64<!C::SMALL>(stg, x, orow ? orow + k + 32 * h : nullptr);
            }
          }
          if (valid) {
            const float l2 = l != 0.f ? m + log2f(l) : -INFINITY;
            if (p.lse) p.lse[at] = l2 * kLn2;
            if (p.lse2) p.lse2[at] = l2;
          }
        } else {
          // a part: O unnormalised, with its maximum and sum
          const int64_t slot = ((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * MT + row;
          float* prow = valid ? p.part_o + slot * R : nullptr;
#pragma unroll 1
          for (int k = 0; k < R; k += 64) {
            float v[64];
            tmem_ld64(lane_base + ob * R + k, v);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint4 x[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                x[j] = make_uint4(__float_as_uint(v[16 * h + 4 * j]),
                                  __float_as_uint(v[16 * h + 4 * j + 1]),
                                  __float_as_uint(v[16 * h + 4 * j + 2]),
                                  __float_as_uint(v[16 * h + 4 * j + 3]));
              put64<!C::SMALL>(stg, x, prow ? prow + k + 16 * h : nullptr);
            }
          }
          if (valid) p.part_ml[slot] = make_float2(m, l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[ob]);
      if (writer && !it.whole && it.starts) {
        join->pair0 = it.x.row0 * c.heads + (int64_t)it.b * MT;
        join->parts = it.parts;
        join->rows = (int32_t)min((uint32_t)MT, pairs - (uint32_t)it.b * MT);
      }
      ++itm;
    }
  }
  __syncthreads();
  if (warp == C::MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the block that CTA blockIdx.x of the attention kernel began
// and did not finish: out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p, part by
// part in the order of the events.  One warp per row.
template <int R>
__global__ void __launch_bounds__(256) cache_join_kernel(const CacheAttn p, const int mt) {
  pdl_trigger();
  pdl_wait();
  const CacheJoin j = p.join[blockIdx.x];
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (row >= j.rows) return;
  // part 0 is the beginning CTA's second slot, the others the first slots
  auto slot = [&](int i) -> int64_t {
    return ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * mt + row;
  };
  float m = -INFINITY;
  for (int i = lane; i < j.parts; i += 32) m = fmaxf(m, p.part_ml[slot(i)].x);
  m = warp_max(m);
  const float m_use = m > -INFINITY ? m : 0.f;
  float l = 0.f;
  for (int i = lane; i < j.parts; i += 32) {
    const float2 ml = p.part_ml[slot(i)];
    l = fmaf(ex2_approx(ml.x - m_use), ml.y, l);
  }
  l = warp_sum(l);
  constexpr int CV = R / 32;               // columns of a lane
  float o[CV];
#pragma unroll
  for (int k = 0; k < CV; ++k) o[k] = 0.f;
#pragma unroll 4
  for (int i = 0; i < j.parts; ++i) {
    const float w = ex2_approx(p.part_ml[slot(i)].x - m_use);
    const float2* src = (const float2*)(p.part_o + slot(i) * R);
#pragma unroll
    for (int k = 0; k < CV / 2; ++k) {
      const float2 v = src[lane + 32 * k];
      o[2 * k] = fmaf(w, v.x, o[2 * k]);
      o[2 * k + 1] = fmaf(w, v.y, o[2 * k + 1]);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const int64_t at = j.pair0 + row;
  uint32_t* dst = (uint32_t*)((__nv_bfloat16*)p.out + at * R);
#pragma unroll
  for (int k = 0; k < CV / 2; ++k)
    dst[lane + 32 * k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
  if (lane == 0) {
    const float l2 = l != 0.f ? m + log2f(l) : -INFINITY;
    if (p.lse) p.lse[at] = l2 * kLn2;
    if (p.lse2) p.lse2[at] = l2;
  }
}

template <int R, int MT>
cudaError_t launch_rm(const CacheAttn& a, const CUtensorMap& tmC, int num_sms, cudaStream_t s) {
  using C = Cfg<R, MT>;
  static uint64_t attr_devices = 0;
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(attr_devices >> (dev & 63) & 1)) {
    cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<R, MT>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    attr_devices |= 1ull << (dev & 63);
  }
  CUtensorMap tmQ;
  if (!make_tmap_bf16(&tmQ, a.q, (uint64_t)a.c.rows * a.c.heads, R, MT))
    return cudaErrorInvalidValue;
  cudaError_t e = launch_dependent(cache_attn_kernel<R, MT>, dim3(num_sms), dim3(32 * C::WARPS),
                                   C::SMEM, s, 1, tmQ, tmC, a, 1);
  if (e != cudaSuccess) return e;
  return launch_dependent(cache_join_kernel<R>, dim3(num_sms, MT / 8), dim3(256), 0, s, 1, a, MT);
}

template <int R>
cudaError_t launch_r(const CacheAttn& a, const CUtensorMap& tmC, int num_sms, cudaStream_t s) {
  // blocks of 32 pairs when a user has no more than that on average
  if (a.c.rows * a.c.heads <= 32 * (int64_t)a.c.B) return launch_rm<R, 32>(a, tmC, num_sms, s);
  return launch_rm<R, 128>(a, tmC, num_sms, s);
}

}  // namespace

bool cache_attn_tc_supported(int r) { return r == 64 || r == 128 || r == 256; }

cudaError_t launch_cache_attn_tc(const CacheAttn& a, const CUtensorMap& tmC, int num_sms,
                                 cudaStream_t s) {
  switch (a.c.r) {
    case 64: return launch_r<64>(a, tmC, num_sms, s);
    case 128: return launch_r<128>(a, tmC, num_sms, s);
    case 256: return launch_r<256>(a, tmC, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace llatte
