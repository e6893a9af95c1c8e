// Accumulated attention weights over the paged latent cache for sm_100a (bf16,
// rank 64, 128 or 256): after the attention kernel has left every row's log sum,
//
//   mass_t += sum over rows i and heads that see t of exp(scale q_i . c_t - lse_i).
//
// The weights of a row are known only after its last tile, so the scores are
// computed again, transposed: S^T = C Q^T with the tile's 128 events on the M = 128
// lanes of tensor memory and NP (row, head) pairs on its columns.  One thread then
// owns an event and sums its columns in registers: no exchange between threads, no
// atomics inside a call, and a fixed order (pairs ascending).  An event's row of
// S^T depends on its own latent alone, so what is stored beside it cannot reach it.
//
// One item = a tile of one user and a run of the blocks of pairs that see it; a
// tile cut between CTAs is summed from parts by a second kernel.
//
// What bounds it: a block is 1024 cycles of the exponentials (128 x 128, 16 a cycle) and
// about as many issue slots; it takes about 1600, and every item begins with the walk
// of the run and ends with a meeting of the warps (64 candidates for 256 users, r =
// 128: 34 us, of which 5 are the beginning).
#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "cache.h"
#include "cache_call.cuh"
#include "cache_issue.cuh"
#include "cache_sched.cuh"
#include "tc_common.cuh"
#include "tc_drain.cuh"
#include "tc_gemm.h"

namespace llatte {

using namespace tc;

namespace {

constexpr int KT = 128;                   // events of a tile
constexpr int NP = 128;                   // pairs of a block

// Four softmax warps share 32 events, a quarter of a block's pairs each; a warp goes on
// to the next block by itself.
constexpr int kSoft0 = 2, kSoft = 16;
constexpr int kThreads = 32 * (kSoft0 + kSoft);

template <int R>
struct Cfg {
  static constexpr int RSUB = R / 64;
  static constexpr int CP = NP / 4;                    // pairs of a softmax warp
  static constexpr int SB = 4;                         // S^T buffers in tensor memory
  static constexpr int KS = R == 256 ? 1 : 2;          // ring slots: a tile stays for many blocks
  static constexpr int QS = R == 256 ? 2 : 4;
  static constexpr uint32_t KSUB = KT * 128, K_BYTES = RSUB * KSUB;
  static constexpr uint32_t QSUB = NP * 128, Q_BYTES = RSUB * QSUB;
  static constexpr uint32_t BAR_BYTES = R == 256 ? 256 : 384;
  static constexpr uint32_t F_BYTES = kSoft * CP * 12 + 6 * 128 * 4;   // of the pairs; sums
  static constexpr size_t SMEM = 1024 + KS * K_BYTES + QS * Q_BYTES + BAR_BYTES + F_BYTES;
  static constexpr uint32_t TMEM_COLS = SB * NP;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(TMEM_COLS <= 512, "TMEM budget");
  static_assert(KS * K_BYTES + QS * Q_BYTES >= sizeof(CacheSplitSpace), "split");
  static_assert(KS * K_BYTES + QS * Q_BYTES <= 229376, "rings");
};


template <int R>
__global__ void __launch_bounds__(kThreads, 1)
cache_mass_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmC,
                  const CacheAttn p) {
  using C = Cfg<R>;
  using Line = ByTiles<NP, KT>;
  constexpr int CP = C::CP, RSUB = C::RSUB, KS = C::KS, QS = C::QS, SB = C::SB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sK = smem;
  uint8_t* sQ = sK + KS * C::K_BYTES;
  uint64_t* bars = (uint64_t*)(sQ + QS * C::Q_BYTES);
  uint64_t* k_full = bars;                 // [KS]
  uint64_t* k_empty = k_full + KS;         // [KS]
  uint64_t* q_full = k_empty + KS;         // [QS]
  uint64_t* q_empty = q_full + QS;         // [QS]
  uint64_t* s_full = q_empty + QS;         // [SB]
  uint64_t* s_empty = s_full + SB;         // [SB] every softmax warp has read S^T
  uint64_t* pair_bar = s_empty + SB;       // [4] the four softmax warps of a lane quadrant
  uint64_t* drain = pair_bar + 4;
  uint32_t* tmem_slot = (uint32_t*)(drain + 1);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  CacheSplit* split = (CacheSplit*)(tmem_slot + 2);
  static_assert((2 * KS + 2 * QS + 2 * SB + 5) * 8 + 8 + sizeof(CacheSplit) <= C::BAR_BYTES,
                "barriers");
  float* sums = (float*)((uint8_t*)bars + C::BAR_BYTES);   // [2][3][128]
  float* pbuf = sums + 6 * 128;                              // [kSoft][3][CP] of the pairs

  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheCall& c = p.c;

  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) { mbar_init(&k_full[s], 1); mbar_init(&k_empty[s], 1); }
    for (int s = 0; s < QS; ++s) { mbar_init(&q_full[s], 1); mbar_init(&q_empty[s], 1); }
    for (int s = 0; s < SB; ++s) { mbar_init(&s_full[s], 1); mbar_init(&s_empty[s], kSoft); }
    for (int q = 0; q < 4; ++q) mbar_init(&pair_bar[q], 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  cache_split<Line>(c, 1, false, *(CacheSplitSpace*)sK, split);
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const CacheSplit run = *split;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    uint32_t kn = 0, qn = 0;               // tiles and blocks of pairs asked for
    const int32_t P = min(1 << c.page_shift, kCacheBox);     // events of a box
    const int np = KT / P;
    const int32_t outside = c.n_pages << c.page_shift;
    CacheItems<Line> items;
    items.start(c, run);
    CacheItem<Line> it;
    bool ok = true;
    while (ok && items.next(c, it)) {
      const CacheBlock& all = it.k.all;
      const int32_t tile = it.k.tile;
      int32_t y = outside;
      const int32_t t = tile * KT + lane * P;
      if (lane < np && cache_seen(c, all, t, t + P)) {
        const int32_t page = __ldg(c.table + (int64_t)it.u * c.stride + (t >> c.page_shift));
        if ((uint32_t)page < (uint32_t)c.n_pages)
          y = (page << c.page_shift) + (t & ((1 << c.page_shift) - 1));
        else
          atomicOr(c.status, LLATTE_DEV_BAD_ID);
      }
      const int ks = kn % KS;
      if (lane == 0) {
        ok = mbar_wait(&k_empty[ks], ((kn / KS) & 1) ^ 1, abort_flag, c.status);
        if (ok) mbar_arrive_expect_tx(&k_full[ks], C::K_BYTES);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      if (lane < np) {
#pragma unroll
        for (int s = 0; s < RSUB; ++s)
          tma_load_2d(&tmC, &k_full[ks], sK + ks * C::K_BYTES + s * C::KSUB + lane * P * 128,
                      s * 64, y);
      }
      ++kn;
      if (lane == 0) {
        for (int i = it.t0; i < it.t1; ++i, ++qn) {
          const int qs = qn % QS;
          if (!mbar_wait(&q_empty[qs], ((qn / QS) & 1) ^ 1, abort_flag, c.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&q_full[qs], C::Q_BYTES);
          const int32_t qrow = (int32_t)(it.x.row0 * c.heads + (int64_t)(it.k.first + i) * NP);
#pragma unroll
          for (int s = 0; s < RSUB; ++s)
            tma_load_2d(&tmQ, &q_full[qs], sQ + qs * C::Q_BYTES + s * C::QSUB, s * 64, qrow);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    __syncwarp();
    if (lane == 0) {                       // (see cache_attn_sm100.cu)
      drain_ring(k_full, KS, kn, c.status);
      drain_ring(q_full, QS, qn, c.status);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // the warp stays converged and one lane issues (see cache_attn_sm100.cu)
    constexpr uint32_t IDESC = idesc_bf16(128, NP, false, false);
    const bool elect = elect_one();
    uint32_t kn = 0, qn = 0;
    bool ok = true;
    CacheItems<Line> items;
    items.start(c, run);
    CacheItem<Line> it;
    while (ok && items.next(c, it)) {
      const int ks = kn % KS;
      if (!warp_wait(&k_full[ks], (kn / KS) & 1, abort_flag, c.status)) break;
      const uint64_t ad = sdesc_sw128(smem_u32(sK + ks * C::K_BYTES), 16, 1024);
      for (int i = it.t0; i < it.t1; ++i, ++qn) {
        const int qs = qn % QS, sb = qn % SB;
        ok = warp_wait(&q_full[qs], (qn / QS) & 1, abort_flag, c.status) &&
             warp_wait(&s_empty[sb], ((qn / SB) & 1) ^ 1, abort_flag, c.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t bd = sdesc_sw128(smem_u32(sQ + qs * C::Q_BYTES), 16, 1024);
        const bool last = i == it.t1 - 1;
        if (elect) {
#pragma unroll
          for (int k = 0; k < R / 16; ++k)
            umma_bf16(tmem + sb * NP, ad + (((k >> 2) * C::KSUB + (k & 3) * 32) >> 4),
                      bd + (((k >> 2) * C::QSUB + (k & 3) * 32) >> 4), IDESC, k > 0 ? 1u : 0u);
          umma_commit(&s_full[sb]);
          umma_commit(&q_empty[qs]);
          if (last) umma_commit(&k_empty[ks]);
        }
        __syncwarp();
        // an injected timeout: with a product and loads in flight, a wait for what this
        // warp itself commits at its end
        if (p.inject && !warp_wait(drain, 0, abort_flag, c.status, kInjectTimeoutNs)) {
          ok = false;
          break;
        }
      }
      ++kn;
    }
    if (elect) umma_commit(drain);
    __syncwarp();
    int dummy = 0;
    mbar_wait(drain, 0, &dummy, c.status);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3, part = (warp - kSoft0) >> 2;   // events, quarter of the pairs
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    // of this warp's pairs: log sum, last and first event inside the window
    float* lw = pbuf + (warp - kSoft0) * 3 * CP;
    int32_t* pw = (int32_t*)(lw + CP);
    int32_t* ww = pw + CP;
    CacheJoin* join = p.join + blockIdx.x;
    const bool writer = warp == kSoft0 && lane == 0;
    if (writer) join->rows = 0;
    uint32_t qn = 0, pphase = 0;
    bool ok = true;
    CacheItems<Line> items;
    items.start(c, run);
    CacheItem<Line> it;
    while (ok && items.next(c, it)) {
      const CacheBlock& all = it.k.all;
      const int32_t tile0 = it.k.tile * KT;
      const int32_t t = tile0 + quad * 32 + lane;          // this lane's event
      const uint32_t pairs = (uint32_t)it.x.n * (uint32_t)c.heads;
      // the first events are inside every window
      const int32_t tw = t < c.n_sink ? INT32_MAX : t;
      // this lane's pair of block i, and its log sum
      const float* lse = p.lse2 + it.x.row0 * c.heads;
      auto pair_of = [&](int i) { return (uint32_t)(it.k.first + i) * NP + part * CP + lane; };
      auto ask = [&](int i) { return i < it.t1 && pair_of(i) < pairs ? lse[pair_of(i)] : 0.f; };
      // where the first quarter puts the sums
      int64_t at = -1;
      if (part == 0 && it.whole && t <= all.pmax &&
          (t >= cache_low(c, all.pmin) || t < c.n_sink))
        at = cache_row(c, c.table, c.stride, it.u, t);
      float sum = 0.f, next = ask(it.t0);
      for (int i = it.t0; i < it.t1; ++i, ++qn) {
        const int sb = qn % SB;
        __syncwarp();
        const int32_t pos = pair_of(i) < pairs ? cache_pos(it.x, cache_div(c, pair_of(i))) : -1;
        lw[lane] = next;
        pw[lane] = pos;
        ww[lane] = cache_low(c, pos);
        next = ask(i + 1);                 // on its way while this block is summed
        __syncwarp();
        bool w = mbar_wait(&s_full[sb], (qn / SB) & 1, abort_flag, c.status);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        tc_fence_after();
        float s4[4] = {0.f, 0.f, 0.f, 0.f};
        float v[CP];
        static_assert(CP == 32, "columns of a load");
        tmem_ld32(lane_base + sb * NP + part * CP, v);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[sb]);
#pragma unroll
        for (int k = 0; k < CP; k += 4) {
          const float4 l4 = *(const float4*)(lw + k);
          const int4 p4 = *(const int4*)(pw + k), w4 = *(const int4*)(ww + k);
          const float e0 = ex2_approx(fmaf(v[k], p.scale2, -l4.x));
          const float e1 = ex2_approx(fmaf(v[k + 1], p.scale2, -l4.y));
          const float e2 = ex2_approx(fmaf(v[k + 2], p.scale2, -l4.z));
          const float e3 = ex2_approx(fmaf(v[k + 3], p.scale2, -l4.w));
          if (t <= p4.x && tw >= w4.x) s4[0] += e0;
          if (t <= p4.y && tw >= w4.y) s4[1] += e1;
          if (t <= p4.z && tw >= w4.z) s4[2] += e2;
          if (t <= p4.w && tw >= w4.w) s4[3] += e3;
        }
        sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
      }
      if (!ok) break;
      // the quarters of the pairs meet, in this order (two sets of sums: the next
      // piece's are written while these are read)
      float* meet = sums + (pphase & 1) * 3 * 128;
      if (part) meet[(part - 1) * 128 + quad * 32 + lane] = sum;
      if (!group_sync(&pair_bar[quad], pphase, abort_flag, c.status)) break;
      if (part == 0) {
#pragma unroll
        for (int k = 0; k < 3; ++k) sum += meet[k * 128 + quad * 32 + lane];
        if (!it.whole)
          p.part_ml[((int64_t)blockIdx.x * 2 + (it.starts ? 1 : 0)) * KT + quad * 32 + lane].x = sum;
        else if (at >= 0)
          atomicAdd(&p.mass[at], sum);
      }
      if (writer && !it.whole && it.starts) {
        join->pair0 = ((int64_t)it.u << 32) | (uint32_t)tile0;
        join->parts = it.parts;
        join->rows = min(KT, all.pmax + 1 - tile0);
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// The tile that CTA blockIdx.x of the accumulation kernel began and did not finish:
// its parts in order of the pairs, one thread per event.
__global__ void __launch_bounds__(KT) cache_mass_join_kernel(const CacheAttn p) {
  pdl_trigger();
  pdl_wait();
  const CacheJoin j = p.join[blockIdx.x];
  if ((int)threadIdx.x >= j.rows) return;
  const CacheCall& c = p.c;
  const int u = (int)(j.pair0 >> 32);
  const int32_t t = (int32_t)(uint32_t)j.pair0 + threadIdx.x;
  const CacheBlock all = cache_all<KT>(c, cache_user(c, u));
  if (!(t >= cache_low(c, all.pmin) || t < c.n_sink)) return;
  float sum = 0.f;
  for (int i = 0; i < j.parts; ++i)
    sum += p.part_ml[((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * KT + threadIdx.x].x;
  const int64_t at = cache_row(c, c.table, c.stride, u, t);
  if (at >= 0) atomicAdd(&p.mass[at], sum);
}

template <int R>
cudaError_t launch_rn(const CacheAttn& a, const CUtensorMap& tmC, int num_sms, cudaStream_t s) {
  using C = Cfg<R>;
  static std::atomic<uint64_t> attr_devices{0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(attr_devices.load() >> (dev & 63) & 1)) {
    cudaError_t e = cudaFuncSetAttribute(cache_mass_kernel<R>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    attr_devices |= 1ull << (dev & 63);
  }
  CUtensorMap tmQ;
  if (!make_tmap_bf16(&tmQ, a.q, (uint64_t)a.c.rows * a.c.heads, R, NP))
    return cudaErrorInvalidValue;
  cache_launched(a, 2);
  cudaError_t e = launch_dependent(cache_mass_kernel<R>, dim3(num_sms), dim3(kThreads),
                                   C::SMEM, s, 1, tmQ, tmC, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(cache_mass_join_kernel, dim3(num_sms), dim3(KT), 0, s, 1, a);
}

template <int R>
cudaError_t launch_r(const CacheAttn& a, const CUtensorMap& tmC, int num_sms, cudaStream_t s) {
  // few pairs a user: 27 us there, 34 us here (128 users, 8 pairs, 800 to 1600 events)
  if (a.pairs <= 16 * (int64_t)a.c.B)
    return launch_cache_mass_token(a, tmC, num_sms, s);
  return launch_rn<R>(a, tmC, num_sms, s);
}

}  // namespace

cudaError_t launch_cache_mass_tc(const CacheAttn& a, const CUtensorMap& tmC, int num_sms,
                                 cudaStream_t s) {
  switch (a.c.r) {
    case 64: return launch_r<64>(a, tmC, num_sms, s);
    case 128: return launch_r<128>(a, tmC, num_sms, s);
    case 256: return launch_r<256>(a, tmC, num_sms, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace llatte
