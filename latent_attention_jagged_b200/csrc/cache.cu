// Paged latent cache: host side of its entry points, and the two operators that
// move rows: append (RMSNorm of the new latents, written into their pages) and
// eviction (the heaviest events of every user, packed into fewer pages).
#include <algorithm>
#include <cmath>
#include <new>

#include "cache.h"
#include "cache_call.cuh"
#include "tc_common.cuh"
#include "tc_gemm.h"

using namespace llatte;

struct llatte_cache {
  llatte_cache_dims dims;
  int device;
  int elem;
  int num_sms;
  int page_shift;
  void* pool;            // caller-owned
  float* mass;           // caller-owned, or NULL
  char* ws;
  int32_t* status;
  int32_t* count;        // [max_batch]
  int32_t* list;         // [max_batch, max_pages * page_size] kept slots
  float* lse2;           // [max_rows, heads]
  bool tc;               // attention on the tensor cores
  bool inject;           // the next calls' kernels make a wait run out
  CUtensorMap tmC;       // the pool, a page a box (tc)
  float* part_o;         // [2 num_sms, block rows, rank]
  float2* part_ml;       // [2 num_sms, block rows]
  CacheJoin* join;       // [2 num_sms]
  int32_t* parts;        // [2 num_sms]
};

namespace llatte {
namespace {

// ---------------------------------------------------------------- append
// c = x / sqrt(mean(x^2) + eps) * g.  Bound by reading and writing the rows; what a row
// waits for is its place (offsets -> user -> length, page).  So a warp takes STEPS steps
// of 32 / G rows (G lanes a row, NV 16-byte vectors a lane), asks for all of them
// before it looks for their users, and one lane per row finds the place: a 32-way
// search by the warp for its first and last row, the rest between the two.
template <typename T, int G, int NV, int STEPS>
__global__ void __launch_bounds__(256) cache_append_kernel(CacheAppend a) {
  constexpr int EV = 16 / sizeof(T), STEP = 32 / G, ROWS = STEPS * STEP;
  static_assert(ROWS <= 32, "one lane finds the place of a row");
  tc::pdl_trigger();
  tc::pdl_wait();
  const CacheCall& c = a.c;
  const int lane = threadIdx.x & 31;
  const int64_t row0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * ROWS;
  // the search below may pass by a faulty user: the last block looks at them all
  if (blockIdx.x == gridDim.x - 1)
    for (int u = threadIdx.x; u < c.B; u += 256) cache_user(c, u);
  if (row0 >= min(c.rows, __ldg(c.qoff + c.B))) return;
  const int nvec = c.r / EV, sub = lane / G, k0 = lane % G;
  uint4 v[STEPS][NV];
#pragma unroll
  for (int i = 0; i < STEPS; ++i)
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int64_t row = row0 + i * STEP + sub;
      const int k = k0 + G * j;
      v[i][j] = make_uint4(0, 0, 0, 0);
      if (row < c.rows && k < nvec) v[i][j] = __ldg((const uint4*)a.x + row * nvec + k);
    }
  // the last user whose rows start at or before `row` (0 when there is none)
  auto find = [&](int64_t row) {
    int lo = 0, n = c.B;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const bool le = lane * step < n && __ldg(c.qoff + lo + lane * step) <= row;
      const uint32_t m = __ballot_sync(0xffffffffu, le);
      const int k = m ? 31 - __clz(m) : 0;
      n = min(step, n - k * step);
      lo += k * step;
    }
    return lo;
  };
  const int64_t last = min(row0 + ROWS, c.rows) - 1;
  const int u0 = find(row0), u1 = __ldg(c.qoff + min(u0 + 1, c.B)) > last ? u0 : find(last);
  int64_t dst = -1;
  if (lane < ROWS && row0 + lane <= last) {
    const int64_t row = row0 + lane;
    int lo = u0, hi = max(u0, u1);
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (__ldg(c.qoff + mid) <= row) lo = mid; else hi = mid - 1;
    }
    const CacheUser x = cache_user(c, lo);
    if (row >= x.row0 && row - x.row0 < x.n)
      dst = cache_row(c, c.table, c.stride, lo, x.len - x.n + (int32_t)(row - x.row0));
    if (dst >= 0 && a.mass) a.mass[dst] = 0.f;
  }
  float g[NV][EV];
  if (a.gain) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = k0 + G * j;
      const uint4 gv = k < nvec ? __ldg((const uint4*)a.gain + k) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < EV; ++e) g[j][e] = to_f(((const T*)&gv)[e]);
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int64_t to = __shfl_sync(0xffffffffu, dst, i * STEP + sub);
    if (a.gain) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < EV; ++e) {
          const float f = to_f(((const T*)&v[i][j])[e]);
          ss = fmaf(f, f, ss);
        }
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float inv = 1.f / sqrtf(ss / (float)c.r + a.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        T* e = (T*)&v[i][j];
#pragma unroll
        for (int b = 0; b < EV; ++b) e[b] = from_f<T>(to_f(e[b]) * inv * g[j][b]);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int k = k0 + G * j;
      if (to >= 0 && k < nvec) ((uint4*)a.pool)[to * nvec + k] = v[i][j];
    }
  }
}

// ---------------------------------------------------------------- evict
// Masses as unsigned keys in the same order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t mass_key(float f) {
  if (f != f) return 0u;
  const uint32_t b = __float_as_uint(f + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

constexpr int kSelThreads = 512;

// Kept slots of one user per block; left out, short and absent users.  Returns false
// when the block is done.
__device__ __forceinline__ bool select_start(const CacheEvict& a, int u, CacheUser* x) {
  const int tid = threadIdx.x;
  *x = cache_user(a.c, u);
  const bool left_out = a.c.lengths[u] != x->len;
  const int T = x->len, K = a.budget;
  __syncthreads();                      // new_lengths may be the lengths just read
  if (tid == 0) a.count[u] = left_out ? 0 : min(T, K);
  if (left_out) return false;
  if (tid == 0) a.new_lengths[u] = min(T, K);
  if (T > K) return true;
  for (int t = tid; t < T; t += kSelThreads) {
    a.list[(int64_t)u * a.list_stride + t] = t;
    if (a.kept) a.kept[(int64_t)u * K + t] = t;
  }
  return false;
}

// Exclusive sum of v over the block's threads, and the total in *all.
__device__ __forceinline__ int block_scan(int v, int* warps, int* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  const int w = lane < kSelThreads / 32 ? warps[lane] : 0;
  *all = __reduce_add_sync(0xffffffffu, w);
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
  __syncthreads();                      // warps[] may be written again
  return before + incl - v;
}

// Moves n kept rows of user u to other pages: a warp copies whole rows, 4 at a time, in
// turns of kCopyRows.  Bound by HBM where there are many users: 134 MB in 26 us (256
// users, 512 rows of 512 bytes).
constexpr int kCopyRows = 16;
__device__ __forceinline__ void copy_kept(const CacheEvict& a, int u, int n, int warp, int warps,
                                          int nvec) {
  const CacheCall& c = a.c;
  const int lane = threadIdx.x & 31;
  const int32_t* list = a.list + (int64_t)u * a.list_stride;
#pragma unroll 1
  for (int i0 = warp * kCopyRows; i0 < n; i0 += warps * kCopyRows) {
    // lane l: place of row i0 + l
    int64_t src = -1, dst = -1;
    if (lane < kCopyRows && i0 + lane < n) {
      src = cache_row(c, c.table, c.stride, u, list[i0 + lane]);
      dst = cache_row(c, a.dst_table, a.dst_stride, u, i0 + lane);
      if (dst >= 0) a.mass[dst] = src < 0 ? 0.f : a.mass[src];
    }
    const int rows = min(kCopyRows, n - i0);
    for (int r = 0; r < rows; r += 4) {
      int64_t s[4], d[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        s[k] = __shfl_sync(0xffffffffu, src, r + k);
        d[k] = __shfl_sync(0xffffffffu, dst, r + k);
      }
      for (int col = lane; col < nvec; col += 32) {
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = make_uint4(0, 0, 0, 0);
          if (s[k] >= 0) v[k] = __ldcs((const uint4*)a.pool + s[k] * nvec + col);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (d[k] >= 0) ((uint4*)a.pool)[d[k] * nvec + col] = v[k];
      }
    }
  }
}

// Users of up to NK * kSelThreads events: the keys are read once and stay in
// registers, NK neighbours a thread.  The threshold, the need-th largest key of the
// events that do not stay anyway, is found bit by bit from the highest bit in which
// the keys differ: the largest value that `need` keys reach.  Then two sums over the
// block place the kept slots in order, events at the threshold going to the earliest
// slots.  (Digits with histograms in shared memory took 31 us for 256 users of 700 to
// 1600 events: heavy-tailed masses fall into a few bins.)
// With copy_nvec > 0 the block then moves the rows as well.
template <int NK>
__global__ void __launch_bounds__(kSelThreads) cache_select_kernel(CacheEvict a, int copy_nvec) {
  __shared__ int s_warp[2][kSelThreads / 32];
  const CacheCall& c = a.c;
  const int u = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  CacheUser x;
  tc::pdl_trigger();
  tc::pdl_wait();
  const bool chosen = !select_start(a, u, &x);
  if (chosen && copy_nvec == 0) return;
  if (chosen) {                         // a user that keeps all its events, or none
    __syncthreads();
    copy_kept(a, u, a.count[u], warp, kSelThreads / 32, copy_nvec);
    return;
  }
  const int T = x.len, K = a.budget, lo = c.n_sink, hi = T - a.n_recent;   // [lo, hi): may go
  const int need = K - c.n_sink - a.n_recent;
  const int t0 = threadIdx.x * NK;
  uint32_t key[NK];
  uint32_t top = 0, low = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int t = t0 + i;
    key[i] = 0;
    if (t >= lo && t < hi && need > 0) {
      const int64_t row = cache_row(c, c.table, c.stride, u, t);
      key[i] = row < 0 ? 0u : mass_key(a.mass[row]);
      top = max(top, key[i]);
      low = min(low, key[i]);
    }
  }
  uint32_t thr = 0;
  int n_eq = 0;                         // events at the threshold that stay
  if (need > 0) {
    top = __reduce_max_sync(0xffffffffu, top);
    low = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) {
      s_warp[0][warp] = (int)top;
      s_warp[1][warp] = (int)low;
    }
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, (uint32_t)s_warp[0][lane & (kSelThreads / 32 - 1)]);
    low = __reduce_min_sync(0xffffffffu, (uint32_t)s_warp[1][lane & (kSelThreads / 32 - 1)]);
    __syncthreads();
    // events of the range that reach v
    int turn = 0;
    auto reach = [&](uint32_t v) -> int {
      int n = 0;
#pragma unroll
      for (int i = 0; i < NK; ++i) n += t0 + i >= lo && t0 + i < hi && key[i] >= v;
      n = __reduce_add_sync(0xffffffffu, n);
      int* w = s_warp[turn];
      turn ^= 1;                        // the last round's sums may still be read
      if (lane == 0) w[warp] = n;
      __syncthreads();
      return __reduce_add_sync(0xffffffffu, lane < kSelThreads / 32 ? w[lane] : 0);
    };
    const int bits = 32 - __clz(top ^ low);          // the keys share what is above
    thr = bits == 32 ? 0u : low >> bits << bits;
    for (int b = bits - 1; b >= 0; --b) {
      const uint32_t v = thr | 1u << b;
      if (reach(v) >= need) thr = v;
    }
    n_eq = need - (thr == 0xffffffffu ? 0 : reach(thr + 1));
    __syncthreads();
  }
  int eq = 0;
#pragma unroll
  for (int i = 0; i < NK; ++i) eq += need > 0 && t0 + i >= lo && t0 + i < hi && key[i] == thr;
  int all;
  int before = block_scan(eq, s_warp[0], &all);
  uint32_t keep = 0;
#pragma unroll
  for (int i = 0; i < NK; ++i) {
    const int t = t0 + i;
    if (t >= T) continue;
    if (t < lo || t >= hi) {
      keep |= 1u << i;
    } else if (need > 0) {
      if (key[i] > thr || (key[i] == thr && before < n_eq)) keep |= 1u << i;
      before += key[i] == thr;
    }
  }
  int at = block_scan(__popc(keep), s_warp[1], &all);
  int32_t* list = a.list + (int64_t)u * a.list_stride;
  int32_t* kept = a.kept ? a.kept + (int64_t)u * K : nullptr;
#pragma unroll
  for (int i = 0; i < NK; ++i)
    if ((keep >> i) & 1) {
      list[at] = t0 + i;
      if (kept) kept[at] = t0 + i;
      ++at;
    }
  if (copy_nvec == 0) return;
  __syncthreads();                      // the list is read by other threads
  copy_kept(a, u, min(T, K), warp, kSelThreads / 32, copy_nvec);
}

// Longer users: the threshold is found digit by digit (8 bits, from the top) with a
// histogram of the keys that share the digits found so far, reading the masses again
// for every digit; then one pass in slot order writes the kept slots.
__global__ void __launch_bounds__(kSelThreads) cache_select_long_kernel(CacheEvict a) {
  tc::pdl_trigger();
  tc::pdl_wait();
  __shared__ int hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int s_warp[2][kSelThreads / 32];
  const CacheCall& c = a.c;
  const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  CacheUser x;
  if (!select_start(a, u, &x)) return;
  const int T = x.len, K = a.budget;
  int32_t* list = a.list + (int64_t)u * a.list_stride;
  int32_t* kept = a.kept ? a.kept + (int64_t)u * K : nullptr;
  const int lo = c.n_sink, hi = T - a.n_recent;       // [lo, hi): may go
  auto key_of = [&](int t) -> uint32_t {
    const int64_t row = cache_row(c, c.table, c.stride, u, t);
    return row < 0 ? 0u : mass_key(a.mass[row]);
  };
  if (tid == 0) { s_prefix = 0; s_need = K - c.n_sink - a.n_recent; }
  __syncthreads();
  const bool any = s_need > 0;
  for (int shift = 24; any && shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int t = lo + tid; t < hi; t += kSelThreads) {
      const uint32_t k = key_of(t);
      if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int need = s_need, d = 255;
      while (hist[d] < need) need -= hist[d--];
      s_need = need;
      s_prefix = prefix | ((uint32_t)d << shift);
    }
    __syncthreads();
  }
  const uint32_t thr = s_prefix;
  const int n_eq = s_need;              // events at the threshold that stay
  int base_eq = 0, base = 0;
  for (int t0 = 0; t0 < T; t0 += kSelThreads) {
    const int t = t0 + tid;
    bool eq = false, keep = false;
    if (t < T) {
      if (t < lo || t >= hi) {
        keep = true;
      } else if (any) {
        const uint32_t k = key_of(t);
        keep = k > thr;
        eq = k == thr;
      }
    }
    uint32_t b = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) s_warp[0][warp] = __popc(b);
    __syncthreads();
    int before = base_eq + __popc(b & ((1u << lane) - 1));
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) before += s_warp[0][w];
      base_eq += s_warp[0][w];
    }
    if (eq && before < n_eq) keep = true;
    b = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) s_warp[1][warp] = __popc(b);
    __syncthreads();
    int at = base + __popc(b & ((1u << lane) - 1));
    for (int w = 0; w < kSelThreads / 32; ++w) {
      if (w < warp) at += s_warp[1][w];
      base += s_warp[1][w];
    }
    if (keep) {
      list[at] = t;
      if (kept) kept[at] = t;
    }
    __syncthreads();
  }
}

// Moves the kept rows in place.  A block owns one 64-byte column slice of one user's
// rows (the last slice index: the masses) and walks them in order, so that
// packing in place is safe without any other block: row i comes from a slot
// >= i, and a step's rows are all read before any of them is written.
constexpr int kMoveThreads = 256;
constexpr int kSliceBytes = 64;

__global__ void __launch_bounds__(kMoveThreads)
cache_move_kernel(CacheEvict a, int row_bytes, int slices) {
  tc::pdl_wait();
  const CacheCall& c = a.c;
  const int u = blockIdx.y, slice = blockIdx.x;
  const int n = a.count[u];
  const int32_t* list = a.list + (int64_t)u * a.list_stride;
  if (slice == slices) {
    for (int i0 = 0; i0 < n; i0 += kMoveThreads) {
      const int i = i0 + threadIdx.x;
      float v = 0.f;
      int64_t dst = -1;
      if (i < n) {
        const int t = list[i];
        const int64_t src = cache_row(c, c.table, c.stride, u, t);
        dst = t == i ? -1 : cache_row(c, a.dst_table, a.dst_stride, u, i);
        v = src < 0 ? 0.f : a.mass[src];
      }
      __syncthreads();
      if (dst >= 0) a.mass[dst] = v;
    }
    return;
  }
  const int vec = threadIdx.x % (kSliceBytes / 16);
  const int byte = slice * kSliceBytes + vec * 16;
  constexpr int ROWS = kMoveThreads / (kSliceBytes / 16);
  for (int i0 = 0; i0 < n; i0 += ROWS) {
    const int i = i0 + threadIdx.x / (kSliceBytes / 16);
    uint4 v = make_uint4(0, 0, 0, 0);
    int64_t dst = -1;
    if (i < n && byte < row_bytes) {
      const int t = list[i];
      const int64_t src = cache_row(c, c.table, c.stride, u, t);
      dst = t == i ? -1 : cache_row(c, a.dst_table, a.dst_stride, u, i);
      if (src >= 0) v = *(const uint4*)((const char*)a.pool + src * row_bytes + byte);
    }
    __syncthreads();
    if (dst >= 0) *(uint4*)((char*)a.pool + dst * row_bytes + byte) = v;
  }
}

__global__ void __launch_bounds__(kMoveThreads)
cache_copy_kernel(CacheEvict a, int nvec) {
  tc::pdl_wait();
  copy_kept(a, blockIdx.y, a.count[blockIdx.y], blockIdx.x * 8 + (threadIdx.x >> 5), gridDim.x * 8,
            nvec);
}

template <typename T, int G, int NV, int STEPS>
cudaError_t append_s(const CacheAppend& a, cudaStream_t s) {
  constexpr int rows = 8 * STEPS * 32 / G;
  return tc::launch_dependent(cache_append_kernel<T, G, NV, STEPS>,
                              dim3((unsigned)((a.c.rows + rows - 1) / rows)), dim3(256), 0, s, 1, a);
}

// A block lives as long as its chain of loads, whatever it moves: with more rows than one
// round of blocks of 4 steps takes (4 blocks an SM), 8 steps (256 users of 100 to
// 400 events, r = 128: 10.2 us with 4, 9.6 with 8).
template <typename T, int G, int NV>
cudaError_t append_g(const CacheAppend& a, cudaStream_t s) {
  constexpr bool more = NV == 1 && G >= 8;
  if constexpr (more) {
    if (a.c.rows > (int64_t)592 * 8 * 4 * 32 / G) return append_s<T, G, NV, 8>(a, s);
  }
  return append_s<T, G, NV, 4>(a, s);
}

template <typename T>
cudaError_t append_t(const CacheAppend& a, cudaStream_t s) {
  const int nvec = a.c.r * (int)sizeof(T) / 16;
  if (nvec <= 8) return append_g<T, 8, 1>(a, s);
  if (nvec <= 16) return append_g<T, 16, 1>(a, s);
  if (nvec <= 32) return append_g<T, 32, 1>(a, s);
  return append_g<T, 32, 2>(a, s);
}

}  // namespace

cudaError_t launch_cache_append(int elem, const CacheAppend& a, cudaStream_t s) {
  return elem == 4 ? append_t<float>(a, s) : append_t<__nv_bfloat16>(a, s);
}

cudaError_t launch_cache_evict(int elem, const CacheEvict& a, cudaStream_t s) {
  const int64_t most = std::min<int64_t>(a.c.cap, a.budget);    // kept events of a user
  const int row_bytes = a.c.r * elem;
  const bool apart = a.dst_table != a.c.table;
  // To other pages the selecting block moves its user's rows itself where they are few,
  // or where the users fill the GPU (256 users, 512 rows of 512 bytes: 35 us, 40 with a
  // second launch; 4 users, 128 rows of 128 bytes: 12.3 and 13.6); a launch that spreads
  // a user's rows over the GPU does it otherwise.
  const bool fused = apart && a.c.cap <= 16 * kSelThreads &&
                     (most * row_bytes <= 64 * 1024 || a.c.B >= 128);
  const int nvec = fused ? row_bytes / 16 : 0;
  const dim3 users(a.c.B), threads(kSelThreads);
  const cudaError_t e =
      a.c.cap <= 4 * kSelThreads
          ? tc::launch_dependent(cache_select_kernel<4>, users, threads, 0, s, 1, a, nvec)
      : a.c.cap <= 16 * kSelThreads
          ? tc::launch_dependent(cache_select_kernel<16>, users, threads, 0, s, 1, a, nvec)
          : tc::launch_dependent(cache_select_long_kernel, users, threads, 0, s, 1, a);
  if (e != cudaSuccess || fused) return e;
  if (apart) {
    const int blocks = (int)std::min<int64_t>((most + 8 * kCopyRows - 1) / (8 * kCopyRows), 64);
    return tc::launch_dependent(cache_copy_kernel, dim3(blocks, a.c.B), dim3(kMoveThreads), 0, s, 1,
                                a, row_bytes / 16);
  }
  const int slices = (row_bytes + kSliceBytes - 1) / kSliceBytes;
  return tc::launch_dependent(cache_move_kernel, dim3(slices + 1, a.c.B), dim3(kMoveThreads), 0, s,
                              1, a, row_bytes, slices);
}

}  // namespace llatte

// ---------------------------------------------------------------- host side
namespace {

constexpr float kLog2e = 1.4426950408889634f;

size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

int check_cache_dims(const llatte_cache_dims* d) {
  if (!d) return LLATTE_ERR_ARG;
  if (d->dtype != LLATTE_BF16 && d->dtype != LLATTE_FP32) return LLATTE_ERR_ARG;
  if (d->heads <= 0 || d->rank <= 0 || d->n_pages <= 0 || d->max_batch <= 0 ||
      d->max_pages <= 0 || d->max_rows <= 0)
    return LLATTE_ERR_ARG;
  const int e = d->dtype == LLATTE_BF16 ? 2 : 4;
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128)
    return LLATTE_ERR_UNSUPPORTED;
  if (d->rank * e % 16 != 0 || d->rank > 256) return LLATTE_ERR_UNSUPPORTED;
  if (d->max_batch > LLATTE_CACHE_MAX_BATCH) return LLATTE_ERR_UNSUPPORTED;
  const int64_t top = (int64_t)1 << 31;
  if ((int64_t)d->n_pages * d->page_size >= top || (int64_t)d->max_pages * d->page_size >= top)
    return LLATTE_ERR_UNSUPPORTED;
  if (d->max_rows >= top || d->max_rows * d->heads >= top) return LLATTE_ERR_UNSUPPORTED;
  return LLATTE_OK;
}

bool cache_uses_tc(const llatte_cache_dims& d) {
  return d.dtype == LLATTE_BF16 && cache_attn_tc_supported(d.rank);
}

struct CacheLayout { size_t status, count, list, lse2, part_o, part_ml, join, parts, zeros, total; };

// The parts' slots are counted for the largest part there is (148 SMs); a device
// with more SMs runs as many CTAs as there are slots.
constexpr int kCacheCtas = 148;

CacheLayout cache_layout(const llatte_cache_dims& d) {
  CacheLayout L = {};
  size_t o = 0;
  auto take = [&](size_t bytes) { size_t r = o; o += align_up(bytes); return r; };
  // first what starts as zeros
  L.status = take(sizeof(int32_t));
  L.join = take(sizeof(CacheJoin) * 2 * kCacheCtas);
  L.parts = take(sizeof(int32_t) * 2 * kCacheCtas);
  L.zeros = o;
  L.count = take(sizeof(int32_t) * d.max_batch);
  L.list = take(sizeof(int32_t) * (size_t)d.max_batch * d.max_pages * d.page_size);
  L.lse2 = take(sizeof(float) * (size_t)d.max_rows * d.heads);
  // two slots a CTA: blocks of kCacheBlockRows, or of 64 for up to two CTAs an SM
  const size_t slots = (size_t)2 * kCacheCtas * 128;
  static_assert(kCacheBlockRows == 128, "slots");
  L.part_o = take(sizeof(float) * slots * d.rank);
  L.part_ml = take(sizeof(float2) * slots);
  L.total = o;
  return L;
}

// Makes the cache's device current for one call.
struct DeviceGuard {
  int prev = -1;
  bool ok;
  explicit DeviceGuard(int device) {
    ok = cudaGetDevice(&prev) == cudaSuccess;
    if (ok && prev != device) ok = cudaSetDevice(device) == cudaSuccess;
    else prev = -1;
  }
  ~DeviceGuard() { if (prev >= 0) cudaSetDevice(prev); }
};

int check_view(const llatte_cache* h, const llatte_cache_view* v) {
  if (!h || !v) return LLATTE_ERR_ARG;
  if (v->B < 0 || v->B > h->dims.max_batch) return LLATTE_ERR_ARG;
  if (v->B > 0 && (!v->table || !v->lengths || v->table_stride <= 0)) return LLATTE_ERR_ARG;
  return LLATTE_OK;
}

CacheCall make_call(const llatte_cache* h, const llatte_cache_view* v, const int64_t* qoff,
                    int64_t rows) {
  CacheCall c = {};
  c.table = v->table; c.stride = v->table_stride; c.lengths = v->lengths; c.B = v->B;
  c.qoff = qoff; c.rows = rows;
  c.cap = (int64_t)std::min(v->table_stride, h->dims.max_pages) * h->dims.page_size;
  c.n_pages = h->dims.n_pages; c.page_shift = h->page_shift;
  c.heads = h->dims.heads; c.r = h->dims.rank; c.status = h->status;
  if (c.heads > 1) {         // see cache_div
    int sh = 0;
    while (((int64_t)1 << sh) < c.heads) ++sh;
    c.head_mul = (uint32_t)((((uint64_t)1 << (31 + sh)) / (uint64_t)c.heads) + 1);
    c.head_shift = sh - 1;
  }
  return c;
}

CacheAttn make_attn(const llatte_cache* h, const llatte_cache_view* v, const void* q,
                    const int64_t* qoff, int64_t rows, void* out) {
  CacheAttn a = {};
  a.c = make_call(h, v, qoff, rows);
  a.c.zero_left_out = 1;     // no row that a user's offsets name keeps an earlier call's bits
  a.pool = h->pool; a.mass = h->mass; a.q = q; a.out = out;
  a.part_o = h->part_o; a.part_ml = h->part_ml; a.join = h->join;
  a.count = h->parts;
  a.inject = h->inject;
  return a;
}

// The attention, and the accumulation when a.lse2 is set.
cudaError_t run_attn(llatte_cache* h, const CacheAttn& a, cudaStream_t s) {
  const cudaError_t e = h->tc ? launch_cache_attn_tc(a, h->tmC, h->num_sms, s)
                              : launch_cache_attn_simt(h->elem, a, h->num_sms, s);
  if (e != cudaSuccess || !a.lse2) return e;
  return h->tc ? launch_cache_mass_tc(a, h->tmC, h->num_sms, s)
               : launch_cache_mass_simt(h->elem, a, h->num_sms, s);
}

}  // namespace

namespace llatte {

int cache_layer_check(const llatte_cache* h, const llatte_cache_view* v, int heads, int rank,
                      int dtype, int64_t rows_q, int accumulate, int keep) {
  const int rc = check_view(h, v);
  if (rc != LLATTE_OK) return rc;
  if (h->dims.heads != heads || h->dims.rank != rank || h->dims.dtype != dtype ||
      h->dims.max_rows < rows_q || (accumulate && !h->mass))
    return LLATTE_ERR_ARG;
  // a history that some layer of one whole pass would cut must not fit into the pages
  // (but for the end of the last one: the kernels look at every user's length)
  const int64_t page = h->dims.page_size, pages = std::min(v->table_stride, h->dims.max_pages);
  if (v->B > 0 && pages > (keep + page - 1) / page) return LLATTE_ERR_UNSUPPORTED;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return LLATTE_ERR_CUDA;
  return dev == h->device ? LLATTE_OK : LLATTE_ERR_ARG;
}

const void* cache_layer_pool(const llatte_cache* h) { return h->pool; }

int cache_layer_run(llatte_cache* h, const llatte_cache_view* v, const CacheLayer& l,
                    int* launched, cudaStream_t s) {
  if (l.rows_h > 0) {
    ++*launched;
    CacheAppend ap = {};
    ap.c = make_call(h, v, l.hoff, l.rows_h);
    ap.c.cap = std::min<int64_t>(ap.c.cap, l.keep);
    ap.pool = h->pool; ap.mass = h->mass; ap.x = l.C;
    if (launch_cache_append(h->elem, ap, s) != cudaSuccess) return LLATTE_ERR_CUDA;
  }
  CacheAttn a = make_attn(h, v, l.q, l.qoff, l.rows_q, l.out);
  a.c.cap = std::min<int64_t>(a.c.cap, l.keep);
  a.c.n_cand = l.n_cand; a.c.window = l.window; a.c.n_sink = l.n_sink;
  a.lse2 = l.accumulate ? h->lse2 : nullptr;
  a.scale2 = l.scale2;
  a.pairs = l.pairs;
  a.launched = launched;
  return run_attn(h, a, s) == cudaSuccess ? LLATTE_OK : LLATTE_ERR_CUDA;
}

}  // namespace llatte

extern "C" {

size_t llatte_cache_workspace_bytes(const llatte_cache_dims* dims) {
  if (check_cache_dims(dims) != LLATTE_OK) return 0;
  return cache_layout(*dims).total;
}

int llatte_cache_create(llatte_cache** out, const llatte_cache_dims* dims, void* pool,
                        float* mass) {
  if (!out) return LLATTE_ERR_ARG;
  *out = nullptr;
  const int rc = check_cache_dims(dims);
  if (rc != LLATTE_OK) return rc;
  if (!pool || ((uintptr_t)pool & 15) || ((uintptr_t)mass & 3)) return LLATTE_ERR_ARG;
  for (const void* p : {(const void*)pool, (const void*)mass}) {
    if (!p) continue;
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess ||
        (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)) {
      cudaGetLastError();
      return LLATTE_ERR_ARG;    // the pools must be device memory
    }
  }
  llatte_cache* h = new (std::nothrow) llatte_cache();
  if (!h) return LLATTE_ERR_OOM;
  h->dims = *dims;
  h->elem = dims->dtype == LLATTE_BF16 ? 2 : 4;
  h->pool = pool;
  h->mass = mass;
  h->page_shift = 0;
  while ((1 << h->page_shift) < dims->page_size) ++h->page_shift;
  if (cudaGetDevice(&h->device) != cudaSuccess ||
      cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device) !=
          cudaSuccess) {
    llatte_cache_destroy(h);
    return LLATTE_ERR_CUDA;
  }
  const CacheLayout L = cache_layout(*dims);
  if (cudaMalloc((void**)&h->ws, L.total) != cudaSuccess) {
    cudaGetLastError();
    h->ws = nullptr;
    llatte_cache_destroy(h);
    return LLATTE_ERR_OOM;
  }
  h->status = (int32_t*)(h->ws + L.status);
  h->count = (int32_t*)(h->ws + L.count);
  h->list = (int32_t*)(h->ws + L.list);
  h->lse2 = (float*)(h->ws + L.lse2);
  h->num_sms = std::min(h->num_sms, kCacheCtas);
  h->tc = cache_uses_tc(*dims);
  h->part_o = (float*)(h->ws + L.part_o);
  h->part_ml = (float2*)(h->ws + L.part_ml);
  h->join = (CacheJoin*)(h->ws + L.join);
  h->parts = (int32_t*)(h->ws + L.parts);
  if (h->tc) {
    const uint64_t rows = (uint64_t)dims->n_pages * dims->page_size;
    if (!make_tmap_bf16(&h->tmC, pool, rows, dims->rank, std::min(dims->page_size, kCacheBox))) {
      llatte_cache_destroy(h);
      return LLATTE_ERR_CUDA;
    }
  }
  if (cudaMemset(h->ws, 0, L.zeros) != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) {
    llatte_cache_destroy(h);
    return LLATTE_ERR_CUDA;
  }
  *out = h;
  return LLATTE_OK;
}

int llatte_cache_append(llatte_cache* h, const llatte_cache_view* v, const void* x, int64_t rows,
                        const int64_t* offsets, const void* gain, float eps, void* stream) {
  const int rc = check_view(h, v);
  if (rc != LLATTE_OK) return rc;
  constexpr int64_t top = (int64_t)1 << 31;
  if (rows < 0 || rows >= top || rows * h->dims.heads >= top) return LLATTE_ERR_ARG;
  if (v->B == 0 || rows == 0) return LLATTE_OK;
  if (!x || !offsets || (((uintptr_t)x | (uintptr_t)gain) & 15)) return LLATTE_ERR_ARG;
  if (gain && !(eps > 0.f)) return LLATTE_ERR_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return LLATTE_ERR_CUDA;
  CacheAppend a = {};
  a.c = make_call(h, v, offsets, rows);
  a.pool = h->pool; a.mass = h->mass; a.x = x; a.gain = gain; a.eps = eps;
  return launch_cache_append(h->elem, a, (cudaStream_t)stream) == cudaSuccess ? LLATTE_OK
                                                                             : LLATTE_ERR_CUDA;
}

int llatte_cache_attend(llatte_cache* h, const llatte_cache_view* v, const llatte_cache_attn* p,
                        void* stream) {
  const int rc = check_view(h, v);
  if (rc != LLATTE_OK) return rc;
  if (!p || p->rows < 0 || p->rows > h->dims.max_rows || p->n_cand < 0 || p->window < 0 ||
      p->n_sink < 0 || (p->accumulate != 0 && p->accumulate != 1) || !std::isfinite(p->scale * kLog2e))
    return LLATTE_ERR_ARG;
  if (p->accumulate && !h->mass) return LLATTE_ERR_ARG;
  if (v->B == 0 || p->rows == 0) return LLATTE_OK;
  if (!p->q || !p->out || p->q == p->out || !p->q_offsets || (((uintptr_t)p->q | (uintptr_t)p->out) & 15))
    return LLATTE_ERR_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return LLATTE_ERR_CUDA;
  CacheAttn a = make_attn(h, v, p->q, p->q_offsets, p->rows, p->out);
  a.c.n_cand = p->n_cand; a.c.window = p->window; a.c.n_sink = p->n_sink;
  a.lse = p->lse; a.lse2 = p->accumulate ? h->lse2 : nullptr;
  a.scale2 = p->scale * kLog2e;
  a.pairs = p->rows * h->dims.heads;
  return run_attn(h, a, (cudaStream_t)stream) == cudaSuccess ? LLATTE_OK : LLATTE_ERR_CUDA;
}

int llatte_cache_evict(llatte_cache* h, const llatte_cache_view* v,
                       const llatte_cache_evict_args* p, void* stream) {
  const int rc = check_view(h, v);
  if (rc != LLATTE_OK) return rc;
  if (!p || p->budget < 1 || p->n_sink < 0 || p->n_recent < 0 ||
      (int64_t)p->n_sink + p->n_recent > p->budget || !h->mass)
    return LLATTE_ERR_ARG;
  if (v->B == 0) return LLATTE_OK;
  if (!p->new_lengths || (p->dst_table && p->dst_stride <= 0)) return LLATTE_ERR_ARG;
  // a destination row must be able to name the pages of every kept event
  const int64_t cap = (int64_t)std::min(v->table_stride, h->dims.max_pages) * h->dims.page_size;
  const int64_t most = std::min<int64_t>(p->budget, cap);
  if (p->dst_table && (int64_t)p->dst_stride * h->dims.page_size < most) return LLATTE_ERR_ARG;
  DeviceGuard g(h->device);
  if (!g.ok) return LLATTE_ERR_CUDA;
  CacheEvict a = {};
  a.c = make_call(h, v, nullptr, 0);
  a.c.n_sink = p->n_sink;
  a.pool = h->pool; a.mass = h->mass; a.budget = p->budget; a.n_recent = p->n_recent;
  a.dst_table = p->dst_table ? p->dst_table : v->table;
  a.dst_stride = p->dst_table ? p->dst_stride : v->table_stride;
  a.new_lengths = p->new_lengths; a.kept = p->kept;
  a.list = h->list; a.list_stride = (int64_t)h->dims.max_pages * h->dims.page_size;
  a.count = h->count;
  return launch_cache_evict(h->elem, a, (cudaStream_t)stream) == cudaSuccess ? LLATTE_OK
                                                                            : LLATTE_ERR_CUDA;
}

int llatte_cache_get_status(llatte_cache* h, int32_t* device_status) {
  if (!h || !device_status) return LLATTE_ERR_ARG;
  DeviceGuard g(h->device);
  int32_t v = 0;
  if (!g.ok || cudaDeviceSynchronize() != cudaSuccess ||
      cudaMemcpy(&v, h->status, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess ||
      cudaMemset(h->status, 0, sizeof(int32_t)) != cudaSuccess)
    return LLATTE_ERR_CUDA;
  *device_status = v;
  return v ? LLATTE_ERR_DEVICE : LLATTE_OK;
}

int llatte_cache_uses_tensor_cores(const llatte_cache* h) { return h ? h->tc : LLATTE_ERR_ARG; }

int llatte_cache_inject_timeout(llatte_cache* h, int enable) {
  if (!h || (enable != 0 && enable != 1)) return LLATTE_ERR_ARG;
  if (!h->tc) return LLATTE_ERR_UNSUPPORTED;
  h->inject = enable != 0;
  return LLATTE_OK;
}

void llatte_cache_destroy(llatte_cache* h) {
  if (!h) return;
  DeviceGuard g(h->device);
  cudaDeviceSynchronize();
  cudaFree(h->ws);
  delete h;
}

}  // extern "C"
