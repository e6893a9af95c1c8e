// Attention over the paged latent cache on CUDA cores: every rank and both
// storage types.
//
//   s_it = scale q_i . c_t   over the events row i sees,
//   out_i = sum_t softmax_t(s_i) c_t,   lse_i = log sum_t exp(s_it),
//   mass_t += sum_i exp(s_it - lse_i).
//
// Scores are kept in log2 units (scale * log2 e folded into one factor).
#include "cache.h"
#include "cache_call.cuh"

namespace llatte {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// One warp per (row, head): lanes split the rank, one pass over the events with
// the running maximum and sum.
template <typename T, int RV>
__global__ void __launch_bounds__(256) cache_attn_row_kernel(CacheAttn a) {
  const CacheCall& c = a.c;
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t row = w / c.heads;
  if (row < c.qoff[0] || row >= min(c.rows, c.qoff[c.B])) return;
  const int u = segment_of(c.qoff, c.B, row);
  const CacheUser x = cache_user(c, u);
  const int64_t j = row - x.row0;
  if (j < 0 || j >= x.n) return;
  const int32_t p = cache_pos(x, (int)j), low = cache_low(c, p);
  const int r = c.r;
  const T* q = (const T*)a.q + w * r;
  const T* pool = (const T*)a.pool;
  float qv[RV], o[RV];
#pragma unroll
  for (int i = 0; i < RV; ++i) {
    const int k = lane + 32 * i;
    qv[i] = k < r ? to_f(q[k]) : 0.f;
    o[i] = 0.f;
  }
  float mx = -INFINITY, l = 0.f;
  for (int32_t t = 0; t <= p; ++t) {
    if (t == c.n_sink && t < low) t = low;
    if (t >= c.n_sink && t < low) continue;
    const int64_t at = cache_row(c, c.table, c.stride, u, t);
    float kv[RV], part = 0.f;
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      const int k = lane + 32 * i;
      kv[i] = k < r && at >= 0 ? to_f(pool[at * r + k]) : 0.f;
      part = fmaf(qv[i], kv[i], part);
    }
    const float s = warp_sum(part) * a.scale2;
    const float mn = fmaxf(mx, s);
    const float corr = mx == mn ? 1.f : exp2f(mx - mn);
    const float pr = exp2f(s - mn);
    l = l * corr + pr;
#pragma unroll
    for (int i = 0; i < RV; ++i) o[i] = fmaf(pr, kv[i], o[i] * corr);
    mx = mn;
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  T* out = (T*)a.out + w * r;
#pragma unroll
  for (int i = 0; i < RV; ++i) {
    const int k = lane + 32 * i;
    if (k < r) out[k] = from_f<T>(o[i] * inv);
  }
  if (lane == 0) {
    const float l2 = l != 0.f ? mx + log2f(l) : -INFINITY;
    if (a.lse) a.lse[w] = l2 * kLn2;
    if (a.lse2) a.lse2[w] = l2;
  }
}

// One warp per (user, event): the weights of all rows and heads that see it,
// in row order.
template <typename T, int RV>
__global__ void __launch_bounds__(256) cache_mass_row_kernel(CacheAttn a) {
  const CacheCall& c = a.c;
  const int lane = threadIdx.x & 31, u = blockIdx.y;
  const CacheUser x = cache_user(c, u);
  const int r = c.r;
  for (int32_t t = blockIdx.x * 8 + (threadIdx.x >> 5); t < x.len; t += gridDim.x * 8) {
    const int64_t at = cache_row(c, c.table, c.stride, u, t);
    if (at < 0) continue;
    float kv[RV], sum = 0.f;
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      const int k = lane + 32 * i;
      kv[i] = k < r ? to_f(((const T*)a.pool)[at * r + k]) : 0.f;
    }
    for (int j = 0; j < x.n; ++j) {
      const int32_t p = cache_pos(x, j);
      if (t > p || (t < cache_low(c, p) && t >= c.n_sink)) continue;
      for (int h = 0; h < c.heads; ++h) {
        const int64_t w = (x.row0 + j) * c.heads + h;
        const T* q = (const T*)a.q + w * r;
        float part = 0.f;
#pragma unroll
        for (int i = 0; i < RV; ++i) {
          const int k = lane + 32 * i;
          if (k < r) part = fmaf(to_f(q[k]), kv[i], part);
        }
        sum += exp2f(warp_sum(part) * a.scale2 - a.lse2[w]);
      }
    }
    if (lane == 0) a.mass[at] += sum;
  }
}

template <typename T>
cudaError_t attn_t(const CacheAttn& a, cudaStream_t s) {
  const unsigned blocks = (unsigned)((a.c.rows * a.c.heads + 7) / 8);
  if (a.c.r <= 32) cache_attn_row_kernel<T, 1><<<blocks, 256, 0, s>>>(a);
  else if (a.c.r <= 64) cache_attn_row_kernel<T, 2><<<blocks, 256, 0, s>>>(a);
  else if (a.c.r <= 128) cache_attn_row_kernel<T, 4><<<blocks, 256, 0, s>>>(a);
  else cache_attn_row_kernel<T, 8><<<blocks, 256, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t mass_t(const CacheAttn& a, cudaStream_t s) {
  const dim3 grid(64, a.c.B);
  if (a.c.r <= 32) cache_mass_row_kernel<T, 1><<<grid, 256, 0, s>>>(a);
  else if (a.c.r <= 64) cache_mass_row_kernel<T, 2><<<grid, 256, 0, s>>>(a);
  else if (a.c.r <= 128) cache_mass_row_kernel<T, 4><<<grid, 256, 0, s>>>(a);
  else cache_mass_row_kernel<T, 8><<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_attn_simt(int elem, const CacheAttn& a, cudaStream_t s) {
  return elem == 4 ? attn_t<float>(a, s) : attn_t<__nv_bfloat16>(a, s);
}
cudaError_t launch_cache_mass_simt(int elem, const CacheAttn& a, cudaStream_t s) {
  return elem == 4 ? mass_t<float>(a, s) : mass_t<__nv_bfloat16>(a, s);
}

}  // namespace llatte
