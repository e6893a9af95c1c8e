// Internal interface of the paged latent cache (not part of the C ABI).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/llatte.h"

namespace llatte {

// One call's users and rows, as the kernels see them.
struct CacheCall {
  const int32_t* table;      // [B, stride] page ids
  const int32_t* lengths;    // [B] cached events, new ones included
  const int64_t* qoff;       // [B + 1] rows of every user (NULL: no rows, evict)
  int64_t rows;              // rows of the arrays behind qoff
  int64_t cap;               // most events of a user: pages a table row can name * page size
  int32_t stride, B;
  int32_t n_pages, page_shift;   // page size = 1 << page_shift
  int32_t heads, r;
  uint32_t head_mul;         // division by heads (cache_div); 0 for one head
  int32_t head_shift;
  int32_t n_cand, window, n_sink;
  int32_t zero_left_out;     // rows of a user left out for its length become zeros
  int32_t* status;
};

// A block of (row, head) pairs that one CTA began and others went on with: its
// first pair, rows and parts (rows = 0: none).
struct CacheJoin {
  int64_t pair0;
  int32_t rows, parts;
};

struct CacheAttn {
  CacheCall c;
  const void* pool;          // [n_pages, page, r]
  float* mass;               // [n_pages, page] or NULL
  const void* q;             // [rows, h, r]
  void* out;                 // [rows, h, r]
  float* lse;                // [rows, h] natural log, or NULL
  float* lse2;               // [rows, h] log2 units, workspace (needed when accumulating)
  // workspaces for blocks that are summed from parts: two slots per CTA
  float* part_o;             // [2 CTAs, block rows, r] unnormalised sums
  float2* part_ml;           // [2 CTAs, block rows] maximum (log2 units) and sum
  CacheJoin* join;           // [CTAs]
  int32_t* count;            // [CTAs] parts done of the block that begins there; 0 between calls
  int* launched;             // host: kernels launched are added here (or NULL)
  int64_t pairs;             // (row, head) pairs of the call, as far as the host can tell
  int32_t min_quota;         // fewest tiles of a CTA's run
  bool never_cut;            // no block is cut between CTAs (then there is nothing to join)
  bool inject;               // failure-detection test: every CTA makes one wait run out
  float scale2;              // scale * log2(e): scores in log2 units
};

// One layer of a forward pass over a cache (llatte_forward_cached): appends the latents
// C of the new events, then attends with the queries q of its rows.
struct CacheLayer {
  const void* C; const int64_t* hoff; int64_t rows_h;    // [rows_h, r], user offsets
  const void* q; const int64_t* qoff; int64_t rows_q;    // [rows_q, h, r]
  void* out;
  int64_t pairs;             // estimate of the pairs in use
  int32_t keep;              // most events of a user that every layer keeps
  int32_t n_cand, window, n_sink, accumulate;
  float scale2;              // scores in log2 units = scale2 * q . c
};
int cache_layer_check(const llatte_cache* h, const llatte_cache_view* v, int heads, int rank,
                      int dtype, int64_t rows_q, int accumulate, int keep);
const void* cache_layer_pool(const llatte_cache* h);
int cache_layer_run(llatte_cache* h, const llatte_cache_view* v, const CacheLayer& a,
                    int* launched, cudaStream_t s);

struct CacheAppend {
  CacheCall c;
  void* pool;
  float* mass;               // or NULL
  const void* x;             // [rows, r]
  const void* gain;          // [r] or NULL
  float eps;
};

struct CacheEvict {
  CacheCall c;
  void* pool;
  float* mass;
  int budget, n_recent;      // c.n_sink first events
  const int32_t* dst_table; int32_t dst_stride;   // == table when in place
  int32_t* new_lengths;
  int32_t* kept;             // [B, budget] or NULL
  int32_t* list;             // workspace: [B, list_stride] kept slots
  int64_t list_stride;
  int32_t* count;            // workspace: [B] kept events, -1 = nothing to move
};

// Most tiles of kt events that a block of mt pairs reads, as far as the host can tell.
inline int64_t cache_most_tiles(const CacheCall& c, int mt, int kt) {
  const int64_t t = (c.cap + kt - 1) / kt;
  if (c.window == 0) return t;
  const int64_t span = (int64_t)c.window + mt / c.heads;       // of the windows of its rows
  const int64_t w = (span + kt - 1) / kt + 1 + ((int64_t)c.n_sink + kt - 1) / kt;
  return t < w ? t : w;
}

inline void cache_launched(const CacheAttn& a, int n) {
  if (a.launched) *a.launched += n;
}

cudaError_t launch_cache_append(int elem, const CacheAppend& a, cudaStream_t s);
cudaError_t launch_cache_evict(int elem, const CacheEvict& a, cudaStream_t s);
// Tensor-core attention (bf16, rank 64, 128 or 256); tmC: the pool as a tensor
// [n_pages * page, r] in boxes of a page or kCacheBox rows.
bool cache_attn_tc_supported(int r);
cudaError_t launch_cache_attn_tc(const CacheAttn& a, const CUtensorMap& tmC, int num_sms,
                                 cudaStream_t s);
cudaError_t launch_cache_mass_tc(const CacheAttn& a, const CUtensorMap& tmC, int num_sms,
                                 cudaStream_t s);
// Their forms for blocks of 16 pairs.
cudaError_t launch_cache_token(const CacheAttn& a, const CUtensorMap& tmC, int num_sms,
                               cudaStream_t s);
cudaError_t launch_cache_mass_token(const CacheAttn& a, const CUtensorMap& tmC, int num_sms,
                                    cudaStream_t s);
constexpr int kCacheBox = 64;              // rows of a box of tmC, or a page if that is smaller
constexpr int kCacheBlockRows = 128;       // largest block of pairs
// CUDA-core attention (any rank up to 256, both types) and its accumulation.
cudaError_t launch_cache_attn_simt(int elem, const CacheAttn& a, int num_sms, cudaStream_t s);
cudaError_t launch_cache_mass_simt(int elem, const CacheAttn& a, int num_sms, cudaStream_t s);

}  // namespace llatte
