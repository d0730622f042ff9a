// Host-side checks and helpers shared by the files that define the C entry points.
#pragma once

#include <cuda_runtime.h>

#include "tsd.h"
#include "tsd_common.cuh"
#include "tsd_kvtile.cuh"
#include "tsd_plan.h"

namespace tsd {

bool is_pow2(int x);

// Host validation of the descriptors; fills the kernel views and shape summary.
tsd_status check_inputs(const tsd_kv_cache* c, const tsd_queries* q, KvView* kv, QView* qv, Shapes* sh);

// The queries with max_tokens_per_seq held to num_tokens: a loop may keep one bound for steps that
// draft fewer tokens in all.
inline tsd_queries bound_tokens(const tsd_queries& queries) {
  tsd_queries q = queries;
  if (q.q_indptr != nullptr && q.max_tokens_per_seq > q.num_tokens) q.max_tokens_per_seq = q.num_tokens;
  return q;
}

// check_inputs on shapes alone: device pointers may be NULL.
tsd_status sizes_for(const tsd_kv_cache* cache, const tsd_queries* queries, Shapes* sh);

// The cache descriptor alone.
tsd_status check_cache_only(const tsd_kv_cache* cache, KvView* kv, Shapes* sh);

// Tensor maps of K and V seen as [rows][128] bf16 with a {64, box} box and 128-byte swizzling,
// box = min(max_box, page_size) rows (max_box for the contiguous layout).  With `gather`, boxes are one
// row high for pages of less than 4 tokens (tile::gather4 loads); without it, maps are zeroed for pages
// of less than 8 (their tiles are copied with cp.async).
tsd_status make_kv_maps(const tsd_kv_cache* c, KvMaps* maps, int max_box = 16, bool gather = false);

// SM count of the current device (148 when none can be queried).
int current_sm_count();

// Whether two arrays share memory.
inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const char *x = static_cast<const char*>(a), *y = static_cast<const char*>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

inline tsd_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TSD_OK : TSD_ERR_CUDA; }

}  // namespace tsd
