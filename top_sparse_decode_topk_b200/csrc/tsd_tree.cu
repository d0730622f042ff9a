// Trees of drafted tokens: ancestor masks, and decode attention in which a draft sees the tokens
// before the drafts and the drafts named by its mask.
#include <math.h>
#include <string.h>

#include "tsd_host.h"

namespace tsd {

constexpr int kMaxTree = 512;   // drafts of a sequence

// ---------------------------------------------------------------------------
// Ancestor masks
// ---------------------------------------------------------------------------
// One block per sequence.  mask(j) = {j} u mask(parent(j)) by doubling: after round r row j holds
// j and its first 2^r - 1 ancestors and up[j] names the next one, so a chain of n drafts takes
// ceil(log2 n) rounds over shared memory instead of n dependent steps.
constexpr int kTmThreads = 256;

struct TreeMaskArgs {
  const int32_t* q_indptr;
  const int32_t* parents;
  uint32_t* mask;
  int32_t* depth;
  uint32_t* status;
  int32_t num_tokens, max_tokens, words;
};

__global__ void __launch_bounds__(kTmThreads) tree_mask_kernel(TreeMaskArgs a) {
  extern __shared__ int32_t tm_smem[];
  const int b = blockIdx.x, tid = threadIdx.x, W = a.words;
  const int t0 = a.q_indptr != nullptr ? __ldg(a.q_indptr + b) : b;
  const int t1 = a.q_indptr != nullptr ? __ldg(a.q_indptr + b + 1) : b + 1;
  const int n = t1 - t0;
  if (t0 < 0 || n < 0 || t1 > a.num_tokens || n > a.max_tokens) {
    if (tid == 0) flag_optional(a.status, TSD_DEV_BAD_SEQ);
    return;
  }
  int32_t* up = tm_smem;                                   // [2][max_tokens]
  uint32_t* rows = reinterpret_cast<uint32_t*>(tm_smem + 2 * a.max_tokens);   // [2][max_tokens][W]
  for (int j = tid; j < n; j += kTmThreads) {
    int p = __ldg(a.parents + t0 + j);
    if (p < -1 || p >= j) {
      flag_optional(a.status, TSD_DEV_BAD_TREE);
      p = -1;
    }
    up[j] = p;
  }
  for (int i = tid; i < n * W; i += kTmThreads) {
    const int j = i / W, w = i - j * W;
    rows[i] = (j >> 5) == w ? 1u << (j & 31) : 0u;
  }
  __syncthreads();
  int cur = 0;
  for (int reach = 1; reach < n; reach *= 2) {
    const int32_t* u = up + cur * a.max_tokens;
    const uint32_t* r = rows + (size_t)cur * a.max_tokens * W;
    int32_t* u2 = up + (cur ^ 1) * a.max_tokens;
    uint32_t* r2 = rows + (size_t)(cur ^ 1) * a.max_tokens * W;
    int any = 0;
    for (int i = tid; i < n * W; i += kTmThreads) {
      const int j = i / W, w = i - j * W;
      const int p = u[j];
      r2[i] = r[i] | (p >= 0 ? r[p * W + w] : 0u);
      if (w == 0) {
        const int next = p >= 0 ? u[p] : -1;
        u2[j] = next;
        any |= next >= 0;
      }
    }
    cur ^= 1;
    if (!__syncthreads_or(any)) break;
  }
  const uint32_t* r = rows + (size_t)cur * a.max_tokens * W;
  for (int i = tid; i < n * W; i += kTmThreads) a.mask[(int64_t)t0 * W + i] = r[i];
  if (a.depth != nullptr) {
    for (int j = tid; j < n; j += kTmThreads) {
      int d = -1;
      for (int w = 0; w < W; ++w) d += __popc(r[j * W + w]);
      a.depth[t0 + j] = d;
    }
  }
}

// ---------------------------------------------------------------------------
// Tree attention
// ---------------------------------------------------------------------------
struct TreeArgs {
  KvView kv;
  QView qv;
  const uint32_t* mask;
  int32_t words;
  void* out;
  int32_t out_f32;
  float* lse;
  uint32_t* status;
};

// One block per (token, q head); its warps take the visible tokens in turn, a lane holding four
// dims, and their states are merged at the end.
constexpr int kTaThreads = 256;

__global__ void __launch_bounds__(kTaThreads) tree_decode_kernel(TreeArgs a) {
  __shared__ float s_m[kTaThreads / 32], s_l[kTaThreads / 32], s_acc[kTaThreads / 32][kHeadDim];
  const int b = blockIdx.x / a.qv.max_tokens, j = blockIdx.x % a.qv.max_tokens, h = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqRaw raw = seq_load(a.kv, a.qv, b);
  const int n = raw.t1 - raw.t0, base = raw.len - n;
  if (raw.len < 0 || raw.len > a.kv.max_seq_len || raw.t0 < 0 || n < 0 || raw.t1 > a.qv.num_tokens ||
      n > a.qv.max_tokens || base < 0) {
    if (j == 0 && h == 0 && threadIdx.x == 0) flag_optional(a.status, TSD_DEV_BAD_SEQ);
    return;
  }
  if (j >= n) return;
  const int64_t list = (int64_t)(raw.t0 + j) * a.qv.hq + h;
  const int g = h / (a.qv.hq / a.kv.hkv);
  float q[4];
  if (a.qv.q_f32) {
    const float4 x = __ldg(static_cast<const float4*>(a.qv.q) + list * 32 + lane);
    q[0] = x.x; q[1] = x.y; q[2] = x.z; q[3] = x.w;
  } else {
    const uint2 x = __ldg(static_cast<const uint2*>(a.qv.q) + list * 32 + lane);
    q[0] = bf16lo(x.x); q[1] = bf16hi(x.x); q[2] = bf16lo(x.y); q[3] = bf16hi(x.y);
  }
  const float scale = a.qv.sm_scale * 1.44269504088896340736f;   // base-2 units
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = warp; i < raw.len; i += kTaThreads / 32) {
    if (i >= base) {
      const int d = i - base;
      const bool seen = a.mask != nullptr ? (__ldg(a.mask + (int64_t)(raw.t0 + j) * a.words + (d >> 5)) >> (d & 31)) & 1
                                          : d <= j;
      if (!seen) continue;
    }
    const uint32_t row = kv_row(a.kv, b, g, i);
    if (row == kInvalidRow) {
      if (lane == 0) flag_optional(a.status, TSD_DEV_BAD_PAGE);
      continue;
    }
    const uint2 kx = __ldg(reinterpret_cast<const uint2*>(a.kv.k) + (int64_t)row * 32 + lane);
    const uint2 vx = __ldg(reinterpret_cast<const uint2*>(a.kv.v) + (int64_t)row * 32 + lane);
    float z = q[0] * bf16lo(kx.x) + q[1] * bf16hi(kx.x) + q[2] * bf16lo(kx.y) + q[3] * bf16hi(kx.y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xFFFFFFFFu, z, o);
    z *= scale;
    if (z > m) {
      const float c = exp2f(m - z);
      l *= c;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] *= c;
      m = z;
    }
    const float p = m == -INFINITY ? 0.f : exp2f(z - m);
    l += p;
    acc[0] += p * bf16lo(vx.x);
    acc[1] += p * bf16hi(vx.x);
    acc[2] += p * bf16lo(vx.y);
    acc[3] += p * bf16hi(vx.y);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) s_acc[warp][4 * lane + e] = acc[e];
  __syncthreads();
  if (threadIdx.x >= kHeadDim) return;
  float mm = -INFINITY;
  for (int w = 0; w < kTaThreads / 32; ++w) mm = fmaxf(mm, s_m[w]);
  float ll = 0.f, o = 0.f;
  if (mm > -INFINITY) {
    for (int w = 0; w < kTaThreads / 32; ++w) {
      const float c = exp2f(s_m[w] - mm);
      if (s_m[w] == -INFINITY) continue;
      ll += c * s_l[w];
      o += c * s_acc[w][threadIdx.x];
    }
    o /= ll;
  }
  if (a.out_f32) static_cast<float*>(a.out)[list * kHeadDim + threadIdx.x] = o;
  else static_cast<uint16_t*>(a.out)[list * kHeadDim + threadIdx.x] = (uint16_t)cvt_bf16x2(o, 0.f);
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[list] = ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994530942f : (mm == -INFINITY ? -INFINITY : ll);
}

}  // namespace tsd

using namespace tsd;

extern "C" {

tsd_status tsd_tree_mask(int32_t batch, const int32_t* q_indptr, int32_t num_tokens, int32_t max_tokens,
                         const int32_t* parents, uint32_t* mask, int32_t* depth, uint32_t* status,
                         tsd_stream_t stream) {
  if (batch < 1 || num_tokens < 1 || parents == nullptr || mask == nullptr) return TSD_ERR_INVALID_ARGUMENT;
  if (q_indptr == nullptr) {
    if (num_tokens != batch) return TSD_ERR_INVALID_ARGUMENT;
    max_tokens = 1;
  }
  if (max_tokens < 1) return TSD_ERR_INVALID_ARGUMENT;
  if (max_tokens > kMaxTree) return TSD_ERR_UNSUPPORTED;
  TreeMaskArgs a;
  a.q_indptr = q_indptr;
  a.parents = parents;
  a.mask = mask;
  a.depth = depth;
  a.status = status;
  a.num_tokens = num_tokens;
  a.max_tokens = max_tokens;
  a.words = (max_tokens + 31) / 32;
  const size_t smem = (size_t)2 * max_tokens * (1 + a.words) * sizeof(int32_t);
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(tree_mask_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return TSD_ERR_CUDA;
  }
  tree_mask_kernel<<<batch, kTmThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

size_t tsd_tree_decode_workspace_size(const tsd_kv_cache* cache, const tsd_queries* queries) {
  Shapes sh;
  if (sizes_for(cache, queries, &sh) != TSD_OK || sh.max_tokens > kMaxTree) return 0;
  return 256;
}

tsd_status tsd_tree_decode(const tsd_kv_cache* cache, const tsd_queries* queries, const uint32_t* mask, void* out,
                           int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, uint32_t* status,
                           tsd_stream_t stream) {
  TreeArgs a;
  Shapes sh;
  memset(&a, 0, sizeof(a));
  const tsd_status st = check_inputs(cache, queries, &a.kv, &a.qv, &sh);
  if (st != TSD_OK) return st;
  if (out == nullptr || ws == nullptr || !queries->causal) return TSD_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)out & 15) || ((uintptr_t)ws & 255)) return TSD_ERR_INVALID_ARGUMENT;
  if (out_dtype != TSD_BF16 && out_dtype != TSD_F32) return TSD_ERR_UNSUPPORTED;
  if (sh.max_tokens > kMaxTree) return TSD_ERR_UNSUPPORTED;
  if (ws_bytes < tsd_tree_decode_workspace_size(cache, queries)) return TSD_ERR_WORKSPACE_TOO_SMALL;
  a.mask = mask;
  a.words = (int)(sh.max_tokens + 31) / 32;
  a.out = out;
  a.out_f32 = out_dtype == TSD_F32;
  a.lse = lse;
  a.status = status;
  if (sh.batch * sh.max_tokens > 0x7fffffffLL || sh.hq > 65535) return TSD_ERR_UNSUPPORTED;
  tree_decode_kernel<<<dim3((unsigned)(sh.batch * sh.max_tokens), (unsigned)sh.hq), kTaThreads, 0,
                       reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
