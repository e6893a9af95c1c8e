// Attention over the paged latent cache for sm_100a (bf16, rank 64, 128 or 256).
//
//   s_it = scale q_i . c_t over the events row i sees,  P = softmax(s),
//   o_i = sum_t P_it c_t,  lse_i = log sum_t exp(s_it)
//
// A piece of work = a block of 128 (query row, head) pairs of one user and a run of its
// tiles of 128 events (cache_sched.cuh); K and V are one shared-memory copy of a tile,
// K-major for S = Q C^T and MN-major for O += P C, as in attn_sm100.cu.  What differs
// from the batch kernel: a tile is gathered page by page (one TMA box per page and 64
// columns, so pages of 16 to 128 rows cost the same bytes), rows hide events behind a
// window, a block may be cut between CTAs, and what a row does not see may hold any
// bits.  Few pairs a user (single tokens) run in cache_token_sm100.cu.
//
// What bounds it: a tile is 1024 (r = 128) or 2048 (r = 256) cycles of the tensor pipe
// and 1024 of the exponentials, but the chain S -> softmax -> P C of a tile is about
// 5500 cycles long, and tensor memory (r = 128) or shared memory (r = 256: two tiles
// beside the queries) holds two tiles at a time.  So a tile is handled in two halves by
// two of four softmax groups, only the running maximum goes from half to half, and the
// two issuing warps never wait for each other's operands.  A tile takes about 3800
// cycles in short blocks (64 candidates for 256 users) and 4000 in long ones (chunks
// of 500 to 800 events, r = 256).  Measured and dropped: one softmax group per tile
// (4800 a tile), one thread issuing all products (a divergent lane took 68 cycles per
// MMA), tiles of 64 events (an N = 64 product runs at 54 cycles for half the work),
// scores kept in registers instead of read twice (spills at 88 registers; with three
// groups at 112 the same time).
//
// Hidden values.  P = 0 does not hide an infinity or NaN from the product P C, so
// in tiles where some row hides some event (the tile of the length's end, window
// edges, the diagonal) the softmax warps look for scores that are not finite; if
// there are any they clear the latents that are not finite in shared memory
// before the product, and rows that see one of them get NaN through their sum.
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

constexpr float kLn2 = 0.6931471805599453f;
constexpr int MT = 128;                   // (row, head) pairs of a block
constexpr int KT = 128;                   // events of a tile
constexpr int HT = KT / 2;                // events of a half
constexpr int NG = 4;                     // softmax groups

// Six warpgroups: producer (warp 0), issuers of S (warp 1) and of P C (warp 2), the
// planner (warp 3); four of softmax; the epilogue.  The launch's 80 registers a thread
// are dealt out again: 128 threads x (56 + 4 x 80 + 104) = 768 x 80 (softmax keeps what
// it has).
constexpr int kThreads = 768;
constexpr int kRegsIssue = 56, kRegsSoft = 80, kRegsEpi = 104;
static_assert(kRegsIssue + NG * kRegsSoft + kRegsEpi <= 480, "registers of the launch");
template <int N> __device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// What the roles have to know about a piece of work.  One warp walks the CTA's run and
// hands the pieces round in a ring: with the walk in every role the kernel's code did
// not fit the instruction cache, and short pieces spent their time fetching it (64
// candidates for 256 users: 44 us).
struct __align__(16) Piece {
  int64_t at0;               // first (row, head) pair, in the call's rows
  int32_t u;                 // user (-1: the run is over)
  int32_t pair0, rows;       // the block's first pair in the user's, and its pairs
  int32_t m, len;            // the user's new events and cached events
  int32_t t0, t1;            // tiles of the piece
  CacheBlock k;
  int32_t parts;             // CTAs that share the block
  int32_t whole, starts;
};
constexpr int NPIECE = 4;

template <int R>
struct Cfg {
  static constexpr int RSUB = R / 64;
  static constexpr int NS = NG;                        // half S buffers
  static constexpr int OBUF = R <= 128 ? 2 : 1;        // O, over the pieces
  static constexpr int QBUF = R <= 128 ? 2 : 1;
  static constexpr int KS = R == 256 ? 4 : R == 128 ? 6 : 12;   // halves in the ring
  // 32 rows x 64 columns of output on their way to global memory, for each quadrant
  static constexpr int NSTG = R == 128 ? 2 : 1;
  static constexpr uint32_t STG_BYTES = 32 * 128;
  static constexpr uint32_t QSUB = MT * 128;           // one 64-wide sub-tile of a query block
  static constexpr uint32_t Q_BYTES = RSUB * QSUB;
  // The ring: for each 64 columns KS halves of 64 rows, so that the halves of a tile
  // (slots 2 j and 2 j + 1) are 128 rows of one operand.
  static constexpr uint32_t H_SUB = HT * 128;
  static constexpr uint32_t H_BYTES = RSUB * H_SUB;
  static constexpr uint32_t KV_SUB = KS * H_SUB;
  static_assert(KS % 2 == 0 && KS >= NG, "halves of a tile are neighbours");
  static constexpr uint32_t S_COL = OBUF * R;
  static constexpr uint32_t BAR_BYTES = 576 + NPIECE * (sizeof(Piece) + 16);
  static constexpr uint32_t F_BYTES = (OBUF * 2 + 1) * NG * MT * 4;   // sums, maxima
  static constexpr size_t SMEM = 1024 + QBUF * Q_BYTES + (size_t)KS * H_BYTES +
                                 4 * NSTG * STG_BYTES + BAR_BYTES + F_BYTES;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(OBUF * R + NS * HT <= 512, "TMEM budget");
  // the split works in the ring before its first load
  static_assert(KS * H_BYTES >= sizeof(CacheSplitSpace), "split");
};

// One column of this lane's row.
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  asm volatile("" : "+r"(r));
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr),
               "r"(__float_as_uint(v))
               : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// One warp clears the latents of half a tile that are not finite, so that a weight of
// 0 hides them (several warps may do so at once: they write the same zeros).
template <int R>
__device__ __forceinline__ void clear_rows(uint8_t* kv, uint32_t sub) {
  for (int k = threadIdx.x & 31; k < HT; k += 32) {
    bool bad = false;
    for (int s = 0; s < R / 64; ++s) {
      const uint4* e = (const uint4*)(kv + s * sub + k * 128);
      for (int j = 0; j < 8; ++j) {
        const uint4 x = e[j];
        for (uint32_t y : {x.x, x.y, x.z, x.w})
          bad |= (y & 0x7f80u) == 0x7f80u || (y & 0x7f800000u) == 0x7f800000u;
      }
    }
    if (!bad) continue;
    for (int s = 0; s < R / 64; ++s)
      for (int j = 0; j < 8; ++j) ((uint4*)(kv + s * sub + k * 128))[j] = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
}

template <int R>
__global__ void __launch_bounds__(kThreads, 1)
cache_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmC,
                  const __grid_constant__ CUtensorMap tmO, const CacheAttn p) {
  using C = Cfg<R>;
  using Line = ByRows<MT, KT>;
  constexpr int RSUB = C::RSUB, KS = C::KS, OBUF = C::OBUF, QBUF = C::QBUF, NS = C::NS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + QBUF * C::Q_BYTES;
  uint8_t* sStage = sKV + KS * C::H_BYTES;                   // [4][NSTG] of STG_BYTES
  uint64_t* bars = (uint64_t*)(sStage + 4 * C::NSTG * C::STG_BYTES);
  uint64_t* q_full = bars;                 // [2]
  uint64_t* q_empty = bars + 2;            // [2]
  uint64_t* o_full = bars + 4;             // [2] last P C done, sums and maxima written
  uint64_t* o_free = bars + 6;             // [2] the epilogue has read O
  uint64_t* s_full = bars + 8;             // [NS / 2] by tile
  uint64_t* p_full = bars + 11;            // [NS] every softmax warp of the group has written P
  uint64_t* p_empty = bars + 17;           // [NS] P C done
  uint64_t* m_full = bars + 23;            // [NG][4] a quadrant's maximum after a half
  uint64_t* kv_full = bars + 39;           // [KS]
  uint64_t* kv_empty = kv_full + KS;       // [KS]
  uint64_t* drain = kv_empty + KS;
  uint32_t* tmem_slot = (uint32_t*)(drain + 2);
  volatile int* abort_flag = (volatile int*)(tmem_slot + 1);
  CacheSplit* split = (CacheSplit*)(tmem_slot + 2);
  uint64_t* piece_full = (uint64_t*)((uint8_t*)bars + 576);  // [NPIECE]
  uint64_t* piece_empty = piece_full + NPIECE;               // [NPIECE]
  Piece* pieces = (Piece*)(piece_empty + NPIECE);
  static_assert((39 + 2 * KS + 2) * 8 + 8 + sizeof(CacheSplit) <= 576, "barriers");
  // of every row: by O buffer and group a sum and its base, by group the maximum so far
  float* lbuf = (float*)((uint8_t*)bars + C::BAR_BYTES);     // [OBUF][NG][MT]
  float* mbuf = lbuf + OBUF * NG * MT;                       // [OBUF][NG][MT]
  float* mrow = mbuf + OBUF * NG * MT;                       // [NG][MT]

  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3;
  const CacheCall& c = p.c;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
      mbar_init(&o_full[s], 1 + NG * 4);
      mbar_init(&o_free[s], 4);
    }
    for (int s = 0; s < NS / 2; ++s) mbar_init(&s_full[s], 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&p_full[s], 4);
      mbar_init(&p_empty[s], 1);
    }
    for (int s = 0; s < NG; ++s) {
      for (int q = 0; q < 4; ++q) mbar_init(&m_full[s * 4 + q], 1);
    }
    for (int s = 0; s < KS; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 1); }
    for (int s = 0; s < NPIECE; ++s) {
      mbar_init(&piece_full[s], 1);
      mbar_init(&piece_empty[s], 3 + 4 * (NG + 1));   // the warps that take it
    }
    mbar_init(drain, 1);
    mbar_init(drain + 1, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmC);
    tma_prefetch_desc(&tmO);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // everything below reads what earlier kernels wrote
  pdl_wait();
  cache_split<Line>(c, p.min_quota, p.never_cut, *(CacheSplitSpace*)sKV, split);
  fence_proxy_async_smem();               // the ring's next writes come from TMA
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const CacheSplit run = *split;

  // The next piece (a warp calls this): false after the last one, or an abort.
  uint32_t taken = 0;
  auto take = [&](Piece& it) -> bool {
    const int st = taken % NPIECE;
    if (!warp_wait(&piece_full[st], (taken / NPIECE) & 1, abort_flag, c.status)) return false;
    it = pieces[st];
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[st]);
    ++taken;
    return it.u >= 0;
  };

  if (warp < 4) {
    regs_down<kRegsIssue>();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      // Lane l < boxes of half a tile gathers box l, a page or, of a larger page, a
      // part; events that no row of the block sees, and pages outside the pool, read as
      // zeros (a box past the pool's last row).
      uint32_t itm = 0, g = 0, qi = 0;
      const int32_t P = min(1 << c.page_shift, kCacheBox);     // events of a box
      const int np = HT / P;
      const int32_t outside = c.n_pages << c.page_shift;
      Piece it;
      bool ok = true;
      while (ok && take(it)) {
        const CacheBlock& blk = it.k;
        if (it.len == 0) continue;
        const int32_t* row = c.table + (int64_t)it.u * c.stride;
        // pool row of this lane's box in half h of the piece's tiles
        auto place = [&](int h) -> int32_t {
          const int32_t t = cache_tile(blk, h >> 1) * KT + (h & 1) * HT + lane * P;
          if (lane >= np || !cache_seen(c, blk, t, t + P)) return outside;
          const int32_t page = __ldg(row + (t >> c.page_shift));
          if ((uint32_t)page < (uint32_t)c.n_pages)
            return (page << c.page_shift) + (t & ((1 << c.page_shift) - 1));
          atomicOr(c.status, LLATTE_DEV_BAD_ID);
          return outside;
        };
        int32_t y = place(2 * it.t0);
        const int qb = itm % QBUF;
        if (lane == 0) {
          ok = mbar_wait(&q_empty[qb], ((itm / QBUF) & 1) ^ 1, abort_flag, c.status);
          if (ok) {
            mbar_arrive_expect_tx(&q_full[qb], C::Q_BYTES);
            const int32_t qrow = (int32_t)it.at0;
#pragma unroll
            for (int s = 0; s < RSUB; ++s)
              tma_load_2d(&tmQ, &q_full[qb], sQ + qb * C::Q_BYTES + s * C::QSUB, s * 64, qrow);
            ++qi;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        for (int i = 2 * it.t0; i < 2 * it.t1; ++i, ++g) {
          const int32_t y_next = i + 1 < 2 * it.t1 ? place(i + 1) : 0;
          const int st = g % KS;
          if (lane == 0) {
            ok = mbar_wait(&kv_empty[st], ((g / KS) & 1) ^ 1, abort_flag, c.status);
            if (ok) mbar_arrive_expect_tx(&kv_full[st], C::H_BYTES);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          if (lane < np) {
            uint8_t* dst = sKV + st * C::H_SUB + lane * P * 128;
#pragma unroll
            for (int s = 0; s < RSUB; ++s)
              tma_load_2d(&tmC, &kv_full[st], dst + s * C::KV_SUB, s * 64, y);
          }
          y = y_next;
        }
        ++itm;
      }
      __syncwarp();
      // Its last loads land before the producer goes, whoever reads them: a role that gives
      // up later leaves them unread, and the CTA must not end before them.
      if (lane == 0) {
        drain_ring(kv_full, KS, g, c.status);
        drain_ring(q_full, QBUF, qi, c.status);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ S = Q C^T
      // Two warps issue, so that neither a tile on its way from memory nor a softmax
      // holds up the other's products.  Both stay converged and one lane issues:
      // descriptors then live in uniform registers (from one divergent lane an MMA took
      // 68 cycles to issue, more than it takes to run).
      constexpr uint32_t IDESC_S = idesc_bf16(128, KT, false, false);
      const bool elect = elect_one();
      uint32_t itm = 0, g = 0;               // items, tiles
      bool ok = true;
      Piece it;
      while (ok && take(it)) {
        if (it.len == 0) continue;
        const int qb = itm % QBUF;
        if (!warp_wait(&q_full[qb], (itm / QBUF) & 1, abort_flag, c.status)) break;
        const uint64_t ad = sdesc_sw128(smem_u32(sQ + qb * C::Q_BYTES), 16, 1024);
        for (int i = it.t0; i < it.t1; ++i, ++g) {
          const int st = (2 * g) % KS, sb = g % (NS / 2);
          // both halves are here; the products that read P in this S buffer are done
          ok = warp_wait(&kv_full[st], (2 * g / KS) & 1, abort_flag, c.status) &&
               warp_wait(&kv_full[st + 1], (2 * g / KS) & 1, abort_flag, c.status) &&
               warp_wait(&p_empty[2 * sb + 1], ((g / (NS / 2)) & 1) ^ 1, abort_flag, c.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bd = sdesc_sw128(smem_u32(sKV + st * C::H_SUB), 16, 1024);
          const uint32_t d = tmem + C::S_COL + sb * KT;
          const bool last = i == it.t1 - 1;
          if (elect) {
#pragma unroll
            for (int k = 0; k < R / 16; ++k)
              umma_bf16(d, ad + (((k >> 2) * C::QSUB + (k & 3) * 32) >> 4),
                        bd + (((k >> 2) * C::KV_SUB + (k & 3) * 32) >> 4), IDESC_S, k > 0 ? 1u : 0u);
            umma_commit(&s_full[sb]);
            if (last) umma_commit(&q_empty[qb]);
          }
          __syncwarp();
        }
        ++itm;
      }
      if (elect) umma_commit(drain);
      __syncwarp();
      int dummy = 0;
      mbar_wait(drain, 0, &dummy, c.status);
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------------------ O += P C
      // P from TMEM, half a tile read MN-major; the first half of an item starts O anew.
      constexpr uint32_t IDESC_O = idesc_bf16(128, R, false, true);
      const bool elect = elect_one();
      uint32_t itm = 0, g = 0;               // items, halves
      bool ok = true;
      Piece it;
      while (ok && take(it)) {
        if (it.len == 0) continue;
        const int ob = itm % OBUF;
        if (!warp_wait(&o_free[ob], ((itm / OBUF) & 1) ^ 1, abort_flag, c.status)) break;
        for (int i = 2 * it.t0; i < 2 * it.t1; ++i, ++g) {
          const int st = g % KS, sb = g % NS;
          ok = warp_wait(&p_full[sb], (g / NS) & 1, abort_flag, c.status);
          if (!ok) break;
          tc_fence_after();
          const uint64_t bd = sdesc_sw128(smem_u32(sKV + st * C::H_SUB), C::KV_SUB, 1024);
          const uint32_t p_tmem = tmem + C::S_COL + sb * HT;
          const bool first = i == 2 * it.t0, last = i == 2 * it.t1 - 1;
          if (elect) {
#pragma unroll
            for (int k = 0; k < HT / 16; ++k)
              umma_bf16_ts(tmem + ob * R, p_tmem + k * 8, bd + (k * 2048 >> 4), IDESC_O,
                           (!first || k > 0) ? 1u : 0u);
            umma_commit(&kv_empty[st]);
            umma_commit(&p_empty[sb]);
            if (last) umma_commit(&o_full[ob]);
          }
          __syncwarp();
        }
        ++itm;
      }
      if (elect) umma_commit(drain + 1);
      __syncwarp();
      int dummy = 0;
      mbar_wait(drain + 1, 0, &dummy, c.status);
      __syncwarp();
    } else {
      // ------------------------------------------------------------ planner
      CacheItems<Line> items;
      items.start(c, run);
      CacheItem<Line> it;
      uint32_t n = 0;
      for (bool more = true; more; ++n) {
        more = items.next(c, it);
        const int st = n % NPIECE;
        if (!warp_wait(&piece_empty[st], ((n / NPIECE) & 1) ^ 1, abort_flag, c.status)) break;
        if (lane == 0) {
          Piece q = {};
          q.u = -1;
          if (more) {
            q.u = it.u;
            q.pair0 = it.b * MT;
            q.at0 = it.x.row0 * c.heads + q.pair0;
            q.rows = (int32_t)min((uint32_t)MT, (uint32_t)it.x.n * (uint32_t)c.heads - q.pair0);
            q.m = it.x.m; q.len = it.x.len;
            q.t0 = it.t0; q.t1 = it.t1; q.k = it.k;
            q.parts = it.parts; q.whole = it.whole; q.starts = it.starts;
          }
          pieces[st] = q;
          mbar_arrive(&piece_full[st]);
        }
        __syncwarp();
        // An injected timeout: with the first piece handed round, a wait for the end of the
        // last product, which the pieces held back here keep from coming.
        if (p.inject && !warp_wait(drain + 1, 0, abort_flag, c.status, kInjectTimeoutNs)) break;
      }
    }
  } else if (warp < 20) {
    // ------------------------------------------------------------ softmax
    // The groups take the halves in turn, group g % NG half g; a thread owns a
    // row.  Only the running maximum goes from one group to the next,
    // as soon as it is known, so that the latencies of NG halves overlap.
    const int group = (warp >> 2) - 1, before = (group + NG - 1) % NG;
    const int row = quad * 32 + lane;                  // pair in the block = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const float mul = p.scale2 == 0.f ? 1.f : fabsf(p.scale2);
    const float2 mul2 = make_float2(mul, mul);
    uint32_t g = 0, itm = 0;
    bool ok = true;
    Piece it;
    while (ok && take(it)) {
      if (it.len == 0) continue;
      const CacheBlock& blk = it.k;
      const int ob = itm % OBUF;
      const bool valid = row < it.rows;
      const int j = cache_div(c, it.pair0 + row);
      const int32_t pos = !valid ? blk.pmax : j < it.m ? it.len - it.m + j : it.len - 1;
      const int32_t low = cache_low(c, pos), low_max = cache_low(c, blk.pmax);
      const bool idle = quad * 32 >= it.rows;          // no row in this quadrant
      float m_run = -INFINITY, l_run = 0.f;     // maximum (log2 units) that the sum is over
      bool poison = false;
      for (int i = 2 * it.t0; i < 2 * it.t1; ++i, ++g) {
        if ((int)(g % NG) != group) continue;
        const int sb = g % NS;
        const uint32_t s_addr = lane_base + C::S_COL + sb * HT;
        bool w = mbar_wait(&s_full[sb >> 1], (g / NS) & 1, abort_flag, c.status);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        tc_fence_after();
        float mt = -INFINITY;
        if (!idle) {
          // some row hides some event of the half (the same answer in every warp)
          const int32_t tile0 = cache_tile(blk, i >> 1) * KT + (i & 1) * HT;
          const bool masked = blk.pmin < tile0 + HT - 1 || low_max > tile0;
          bool clear = false;
#pragma unroll 1
          for (int h = 0; h < HT; h += 32) {
            float v[32];
            tmem_ld32(s_addr + h, v);
            if (p.scale2 <= 0.f) {
              const float f = p.scale2 == 0.f ? 0.f : -1.f;
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] *= f;
            }
            if (masked) {
              // events that the row sees: [0, hi) without [sk, lo)
              const int32_t t0 = tile0 + h;
              const int hi = max(min(pos + 1 - t0, 32), 0);
              const int lo = min(max(low - t0, 0), 32);
              const int sk = max(min(c.n_sink - t0, lo), 0);
              uint32_t vis = hi == 0 ? 0u : 0xffffffffu >> (32 - hi);
              if (sk < lo) vis &= ~((0xffffffffu >> (32 - lo)) & (0xffffffffu << sk));
              float2 z2 = make_float2(0.f, 0.f);
#pragma unroll
              for (int k = 0; k < 32; k += 2)
                z2 = fma_f2(make_float2(v[k], v[k + 1]), make_float2(0.f, 0.f), z2);
              if (__any_sync(0xffffffffu, valid && !(z2.x + z2.y == 0.f))) {
                // a score is not finite: column by column
                clear = true;
#pragma unroll 1
                for (int k = 0; k < 32; ++k) {
                  const float x = tmem_ld1(s_addr + h + k);
                  const bool fin = fabsf(x) < INFINITY;
                  poison |= valid && !fin && ((vis >> k) & 1);
                  tmem_st1(s_addr + h + k, fin ? x : -INFINITY);
                }
                tmem_ld32(s_addr + h, v);
                if (p.scale2 <= 0.f) {         // those that were not finite stay -inf
                  const float f = p.scale2 == 0.f ? 0.f : -1.f;
#pragma unroll 1
                  for (int k = 0; k < 32; ++k) {
                    const float x = tmem_ld1(s_addr + h + k);
                    tmem_st1(s_addr + h + k, x > -INFINITY ? f * x : x);
                  }
                  tmem_ld32(s_addr + h, v);
                }
              }
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = vis & (1u << k) ? v[k] : -INFINITY;
            }
            if (masked || p.scale2 <= 0.f) tmem_st32(s_addr + h, v);
            float m8[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) m8[k] = fmaxf(fmax3(v[k], v[k + 8], v[k + 16]), v[k + 24]);
            mt = fmaxf(mt, fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                                 fmaxf(m8[6], m8[7])));
          }
          if (clear) clear_rows<R>(sKV + (g % KS) * C::H_SUB, C::KV_SUB);
          mt *= mul;
        }
        // the maximum so far comes from the group before (a new block starts anew);
        // waiting for it in every tile also says that mrow[group] has been read
        if (g > 0) {
          w = mbar_wait(&m_full[before * 4 + quad], ((g - 1) / NG) & 1, abort_flag, c.status);
          if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        }
        const float m_prev = i == 2 * it.t0 ? -INFINITY : mrow[before * MT + row];
        // O and the sums keep their base until the maximum grows by more than kGrow
        const bool resc = i > 2 * it.t0 && mt > m_prev + kGrow;
        const float m_now = i == 2 * it.t0 || resc ? mt : m_prev;
        mrow[group * MT + row] = m_now;
        __syncwarp();
        if (lane == 0) mbar_arrive(&m_full[group * 4 + quad]);
        if (idle) {
          if (lane == 0) mbar_arrive(&p_full[sb]);
          continue;
        }
        if (__any_sync(0xffffffffu, resc)) {
          // the previous product must be in O: the next phase of its p_empty
          w = mbar_wait(&p_empty[(g - 1) % NS], ((g - 1) / NS) & 1, abort_flag, c.status);
          if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
          tc_fence_after();
          const float scale = resc ? ex2_approx(m_prev - m_now) : 1.f;
#pragma unroll 1
          for (int k = 0; k < R; k += 32) {
            float o[32];
            tmem_ld32(lane_base + ob * R + k, o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] *= scale;
            tmem_st32(lane_base + ob * R + k, o);
          }
        }
        // Weights 2^(s - m), rounded to bf16 for the product (off by up to 2^-8 each), the sum
        // in fp32 of the unrounded ones.  What the rounding takes could go into a second
        // product (its operand fits beside the first): error of the result against fp64
        // 0.0017 instead of 0.0021 (0.0017 is the result's own rounding), for 10 to 19 %
        // (64 candidates for 256 users 38.7 -> 42.6 us, chunks at r = 256 193 -> 230).  A row
        // that has seen nothing yet subtracts 0 from its -inf.  All of them take the special-
        // function unit (512 cycles a half and scheduler): a polynomial on the FMA pipe
        // for one pair in four cost more issue slots than it saved.
        const float m_use = m_now > -INFINITY ? m_now : 0.f;
        const float2 nm2 = make_float2(-m_use, -m_use);
        float2 l4[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) l4[k] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int h = 0; h < HT; h += 32) {
          float v[32];
          tmem_ld32(s_addr + h, v);
          uint32_t pk[16];                     // bf16 pairs
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 x = fma_f2(make_float2(v[2 * k], v[2 * k + 1]), mul2, nm2);
            x.x = ex2_approx(x.x);
            x.y = ex2_approx(x.y);
            l4[k & 1] = add_f2(l4[k & 1], x);
            pk[k] = pack_bf16(x.x, x.y);
          }
          tmem_st16u(s_addr + h / 2, pk);      // over scores already read
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[sb]);
        // the sum's base follows the maximum (also past changes of the other groups);
        // -inf: no sum yet
        if (m_now != m_run) {
          l_run = m_run > -INFINITY ? l_run * ex2_approx(m_run - m_now) : 0.f;
          m_run = m_now;
        }
        l_run += (l4[0].x + l4[0].y) + (l4[1].x + l4[1].y);
      }
      if (!ok) break;
      const bool w_free = mbar_wait(&o_free[ob], ((itm / OBUF) & 1) ^ 1, abort_flag, c.status);
      if (!__all_sync(0xffffffffu, w_free)) break;
      if (!idle) {
        if (poison || m_run == INFINITY) l_run = NAN;
        lbuf[(ob * NG + group) * MT + row] = l_run;
        mbuf[(ob * NG + group) * MT + row] = m_run;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_full[ob]);
      ++itm;
    }
  } else {
    regs_up<kRegsEpi>();
    // ------------------------------------------------------------ epilogue
    const int row = quad * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    CacheJoin* join = p.join + blockIdx.x;
    const bool writer = warp == 20 && lane == 0;
    if (writer) join->rows = 0;
    uint32_t itm = 0, stg = 0;             // items, staged boxes
    Piece it;
    while (take(it)) {
      const bool valid = row < it.rows;
      const bool box = quad * 32 + 32 <= it.rows;
      const bool idle = quad * 32 >= it.rows;
      const int64_t at = it.at0 + row;
      __nv_bfloat16* orow = (__nv_bfloat16*)p.out + at * R;
      if (it.len == 0) {                 // no event: zeros
        if (!valid) continue;
        for (int k = 0; k < R; k += 8) *(uint4*)(orow + k) = make_uint4(0, 0, 0, 0);
        if (p.lse) p.lse[at] = -INFINITY;
        if (p.lse2) p.lse2[at] = -INFINITY;
        continue;
      }
      const int ob = itm % OBUF;
      bool w = mbar_wait(&o_full[ob], (itm / OBUF) & 1, abort_flag, c.status);
      if (!__all_sync(0xffffffffu, w)) break;
      tc_fence_after();
      if (!idle) {
        // the groups' sums, each over its own last maximum; the largest is O's
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j) m = fmaxf(m, mbuf[(ob * NG + j) * MT + row]);
        const float m_use = m > -INFINITY ? m : 0.f;
#pragma unroll
        for (int j = 0; j < NG; ++j)
          l = fmaf(lbuf[(ob * NG + j) * MT + row],
                   ex2_approx(mbuf[(ob * NG + j) * MT + row] - m_use), l);
        const uint32_t o_addr = lane_base + ob * R;
        if (it.whole) {
          const float inv = l != 0.f ? 1.f / l : 0.f;
          if (box) {
            // all 32 rows are the user's: they leave as boxes, so that O is free as soon
            // as it has been read (64 stores of a lane's own row cost 3500 cycles)
#pragma unroll 1
            for (int k = 0; k < R; k += 64, ++stg) {
              uint8_t* buf = sStage + (quad * C::NSTG + stg % C::NSTG) * C::STG_BYTES;
              if (lane == 0)
                asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(C::NSTG - 1)
                             : "memory");
              __syncwarp();
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float v[32];
                tmem_ld32(o_addr + k + 32 * h, v);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float* e = v + 8 * j;
                  st_shared_v4(smem_u32(buf) + lane * 128 + (((4 * h + j) ^ (lane & 7)) << 4),
                               make_uint4(pack_bf16(e[0] * inv, e[1] * inv),
                                          pack_bf16(e[2] * inv, e[3] * inv),
                                          pack_bf16(e[4] * inv, e[5] * inv),
                                          pack_bf16(e[6] * inv, e[7] * inv)));
                }
              }
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_2d(&tmO, smem_u32(buf), k, (int32_t)(at - lane));
                tma_store_commit();
              }
            }
          }
#pragma unroll 1
          for (int k = box ? R : 0; k < R; k += 32) {
            float v[32];
            tmem_ld32(o_addr + k, v);
            if (valid) {
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                *(uint4*)(orow + k + j) =
                    make_uint4(pack_bf16(v[j] * inv, v[j + 1] * inv),
                               pack_bf16(v[j + 2] * inv, v[j + 3] * inv),
                               pack_bf16(v[j + 4] * inv, v[j + 5] * inv),
                               pack_bf16(v[j + 6] * inv, v[j + 7] * inv));
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
          float* prow = p.part_o + slot * R;
#pragma unroll 1
          for (int k = 0; k < R; k += 32) {
            float v[32];
            tmem_ld32(o_addr + k, v);
            if (valid) {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *(float4*)(prow + k + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            }
          }
          if (valid) p.part_ml[slot] = make_float2(m, l);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[ob]);
      if (writer && !it.whole && it.starts) {
        join->pair0 = it.at0;
        join->parts = it.parts;
        join->rows = it.rows;
      }
      ++itm;
    }
    if (lane == 0) tma_store_wait_all();
    __syncwarp();
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the block that CTA blockIdx.x of the attention kernel began
// and did not finish: out = sum_p 2^(m_p - M) O_p / sum_p 2^(m_p - M) l_p, part by
// part in the order of the events.  One warp per row.
template <int R>
__global__ void __launch_bounds__(256) cache_join_kernel(const CacheAttn p) {
  pdl_trigger();
  pdl_wait();
  const CacheJoin j = p.join[blockIdx.x];
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  if (row >= j.rows) return;
  // part 0 is the beginning CTA's second slot, the others the first slots
  auto slot = [&](int i) -> int64_t {
    return ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * MT + row;
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

template <int R>
cudaError_t launch_r(CacheAttn a, const CUtensorMap& tmC, int num_sms, cudaStream_t s) {
  using C = Cfg<R>;
  // Blocks of up to 4 tiles are not cut: the tiles that a CTA may have too many of
  // take less time than the launch that would join the parts.
  a.min_quota = 1;
  a.never_cut = cache_most_tiles(a.c, MT, KT) <= 4;
  // Few pairs a user on average: cache_token_sm100.cu.  Measured at 4 to 16 pairs, r = 128
  // (400 and 2000 events): 17 to 23 us there, 23 to 25 here; at 32 pairs 29 to 32 there.
  // At r = 256 its blocks cost more to begin and end, so that many short histories (8
  // pairs, 200 events, 256 users) take 35 us there and 27 here; 1000 events: 37 and 39.
  const bool many_short = R == 256 && a.never_cut && a.c.B > num_sms;
  if (a.pairs <= 16 * (int64_t)a.c.B && !many_short)
    return launch_cache_token(a, tmC, num_sms, s);
  static std::atomic<uint64_t> attr_devices{0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (!(attr_devices.load() >> (dev & 63) & 1)) {
    cudaError_t e = cudaFuncSetAttribute(cache_attn_kernel<R>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
    // the register split waits for what the launch does not have
    cudaFuncAttributes f;
    e = cudaFuncGetAttributes(&f, cache_attn_kernel<R>);
    if (e != cudaSuccess) return e;
    if (f.numRegs * (kThreads / 128) < kRegsIssue + NG * kRegsSoft + kRegsEpi)
      return cudaErrorInvalidConfiguration;
    attr_devices |= 1ull << (dev & 63);
  }
  CUtensorMap tmQ, tmO;
  const uint64_t pairs = (uint64_t)a.c.rows * a.c.heads;
  if (!make_tmap_bf16(&tmQ, a.q, pairs, R, MT) || !make_tmap_bf16(&tmO, a.out, pairs, R, 32))
    return cudaErrorInvalidValue;
  const cudaError_t e = launch_dependent(cache_attn_kernel<R>, dim3(num_sms), dim3(kThreads), C::SMEM,
                                         s, 1, tmQ, tmC, tmO, a);
  cache_launched(a, a.never_cut ? 1 : 2);
  if (e != cudaSuccess || a.never_cut) return e;
  return launch_dependent(cache_join_kernel<R>, dim3(num_sms, MT / 8), dim3(256), 0, s, 1, a);
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
