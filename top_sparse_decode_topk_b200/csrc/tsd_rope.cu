// Rotary positions fused with the append of a step's K and V rows to the cache.
//
// Pair i of a row is turned by p f_i radians, p the token's position.  In fp32 the product
// alone would be off by 2^-24 p f_i -- 0.01 radians at p = 128K -- so positions multiply the
// frequency in units of 2^-64 turns instead: p * turn[i] in 64-bit integers wraps at whole turns
// by itself, and its top 32 bits are the reduced angle to 2^-33 turns (7e-10 radians).  sincospi takes that
// angle as an fp32 fraction of half a turn, rounded to 2^-25 at most (9e-8 radians, near half a turn): the whole error
// at any position, with no 64-bit floating point and no range reduction.
//
// Bound by HBM: a token moves (Hq + Hkv) x 256 B in and out and Hkv x 512 B of V (bf16).  One
// block takes one or a few tokens of a sequence: its first threads compute the tokens' sines and cosines
// once (64 per token, shared by all heads), the rest of the work is 16-byte loads and stores.
// A thread takes two 16-byte chunks of a row that hold both elements of its pairs, so q can be
// rotated in place.  Measured, 32 + 8 + 8 heads: 32768 tokens 133 us = 6.1 TB/s (93% of a plain
// copy's rate), 8192 39 us, 64 6.3 us with the launch.
#include <math.h>
#include <string.h>

#include "tsd_host.h"

namespace tsd {

struct RopeArgs {
  KvView kv;
  QView qv;
  tsd_rope rope;
  const void* k_new;
  const void* v_new;
  int64_t q_stride, k_stride, v_stride;
  const int32_t* positions;
  const int32_t* depth;
  void* out_q;
  uint32_t* status;
  int32_t chunks;   // blocks per sequence
  int32_t toks;     // tokens per block
};

constexpr int kRopeThreads = 128;
constexpr int kRopeMaxToks = 4;

// Eight consecutive elements as fp32.
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int chunk, float* x) {
  if (F32) {
    const float4 a = *(reinterpret_cast<const float4*>(row) + 2 * chunk);
    const float4 b = *(reinterpret_cast<const float4*>(row) + 2 * chunk + 1);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  } else {
    unpack8(*(reinterpret_cast<const uint4*>(row) + chunk), x);
  }
}
template <bool F32>
__device__ __forceinline__ void store8(void* row, int chunk, const float* x) {
  if (F32) {
    *(reinterpret_cast<float4*>(row) + 2 * chunk) = make_float4(x[0], x[1], x[2], x[3]);
    *(reinterpret_cast<float4*>(row) + 2 * chunk + 1) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *(reinterpret_cast<uint4*>(row) + chunk) =
        make_uint4(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]), cvt_bf16x2(x[4], x[5]), cvt_bf16x2(x[6], x[7]));
  }
}

__device__ __forceinline__ void turn_pair(float& a, float& b, const float2 cs) {
  const float x = a, y = b;
  a = x * cs.x - y * cs.y;
  b = y * cs.x + x * cs.y;
}

// VEC: the rotated dims split into whole 16-byte chunks on both sides of every pair (half layout:
// rotary_dim a multiple of 16; interleaved: of 8); otherwise element by element (32768 tokens: 344 us;
// in the half layout a pair's elements then lie at different places of their chunks, and it goes by 2-byte accesses).
template <bool F32, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 cs[kRopeMaxToks][64];
  __shared__ int64_t s_row[kRopeMaxToks];   // cache row of (token, kv head 0), -1 when it has none
  const int b = blockIdx.x / a.chunks, j0 = (blockIdx.x % a.chunks) * a.toks;
  const int tid = threadIdx.x;
  const SeqRaw raw = seq_load(a.kv, a.qv, b);
  const int n = raw.t1 - raw.t0, base = raw.len - n;
  if (raw.len < 0 || raw.len > a.kv.max_seq_len || raw.t0 < 0 || n < 0 || raw.t1 > a.qv.num_tokens ||
      n > a.qv.max_tokens || base < 0) {
    if (j0 == 0 && tid == 0) flag_optional(a.status, TSD_DEV_BAD_SEQ);
    return;
  }
  const int nt = min(a.toks, n - j0);
  if (nt <= 0) return;
  const int half = a.rope.rotary_dim >> 1;
  for (int i = tid; i < nt * 64; i += kRopeThreads) {
    const int t = i >> 6, f = i & 63;
    if (f < half) {
      int pos = base + j0 + t;
      if (a.positions != nullptr) pos = __ldg(a.positions + raw.t0 + j0 + t);
      else if (a.depth != nullptr) pos = base + __ldg(a.depth + raw.t0 + j0 + t);
      const uint64_t phase = (uint64_t)(int64_t)pos * a.rope.turn[f] + 0x80000000ull;
      float s, c;
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &s, &c);
      cs[t][f] = make_float2(c * a.rope.mscale, s * a.rope.mscale);
    }
  }
  if (tid < nt) {
    const int r = base + j0 + tid;
    int64_t row;
    if (a.kv.page_table == nullptr) {
      row = (int64_t)b * a.kv.hkv * a.kv.max_seq_len + r;
    } else {
      const int32_t page = __ldg(a.kv.page_table + (int64_t)b * a.kv.max_pages + (r >> a.kv.page_shift));
      if (page < 0 || (int64_t)page >= a.kv.num_pages) {
        flag_optional(a.status, TSD_DEV_BAD_PAGE);
        row = -1;
      } else {
        row = (((int64_t)page * a.kv.hkv) << a.kv.page_shift) | (r & ((1 << a.kv.page_shift) - 1));
      }
    }
    s_row[tid] = row;
  }
  __syncthreads();
  const int64_t head_rows = a.kv.page_table == nullptr ? a.kv.max_seq_len : (int64_t)1 << a.kv.page_shift;
  const int hq = a.qv.hq, hkv = a.kv.hkv, rows = hq + 2 * hkv;
  constexpr int kUnits = VEC ? 8 : 64;        // pieces of a row, one per thread
  constexpr int kEsz = F32 ? 4 : 2;
  for (int i = tid; i < nt * rows * kUnits; i += kRopeThreads) {
    const int u = i % kUnits, tr = i / kUnits;
    const int t = tr / rows, h = tr - t * rows;
    const int64_t tok = raw.t0 + j0 + t;
    const char* src;
    char* dst;
    bool to_cache = true, rot = true;
    if (h < hq) {
      src = static_cast<const char*>(a.qv.q) + (tok * a.q_stride + (int64_t)h * kHeadDim) * kEsz;
      dst = static_cast<char*>(a.out_q) + (tok * hq + h) * kHeadDim * kEsz;
      to_cache = false;
    } else {
      const bool is_v = h >= hq + hkv;
      const int g = h - hq - (is_v ? hkv : 0);
      src = static_cast<const char*>(is_v ? a.v_new : a.k_new) +
            (tok * (is_v ? a.v_stride : a.k_stride) + (int64_t)g * kHeadDim) * kEsz;
      if (s_row[t] < 0) continue;
      dst = reinterpret_cast<char*>(const_cast<uint16_t*>(is_v ? a.kv.v : a.kv.k)) +
            (s_row[t] + g * head_rows) * kHeadDim * 2;
      rot = !is_v;
    }
    if (VEC) {
      // chunks c0 and c1 of eight elements
      int c0, c1;
      const bool turned = a.rope.interleaved ? true : u < (half >> 3);
      if (a.rope.interleaved) {
        c0 = 2 * u; c1 = 2 * u + 1;
      } else if (turned) {
        c0 = u; c1 = u + (half >> 3);
      } else {
        c0 = (half >> 2) + 2 * (u - (half >> 3)); c1 = c0 + 1;
      }
      float x[8], y[8];
      load8<F32>(src, c0, x);
      load8<F32>(src, c1, y);
      if (rot && turned) {
        if (a.rope.interleaved) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (8 * c0 < 2 * half) turn_pair(x[2 * e], x[2 * e + 1], cs[t][4 * c0 + e]);
            if (8 * c1 < 2 * half) turn_pair(y[2 * e], y[2 * e + 1], cs[t][4 * c1 + e]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) turn_pair(x[e], y[e], cs[t][8 * u + e]);
        }
      }
      if (to_cache || !F32) {
        store8<false>(dst, c0, x);
        store8<false>(dst, c1, y);
      } else {
        store8<true>(dst, c0, x);
        store8<true>(dst, c1, y);
      }
    } else {
      const bool turned = u < half;
      const int e0 = turned ? (a.rope.interleaved ? 2 * u : u) : 2 * u;
      const int e1 = turned && !a.rope.interleaved ? u + half : e0 + 1;
      float x, y;
      if (F32) {
        x = reinterpret_cast<const float*>(src)[e0];
        y = reinterpret_cast<const float*>(src)[e1];
      } else {
        x = bf16lo(reinterpret_cast<const uint16_t*>(src)[e0]);
        y = bf16lo(reinterpret_cast<const uint16_t*>(src)[e1]);
      }
      if (rot && turned) turn_pair(x, y, cs[t][u]);
      if (to_cache || !F32) {
        const uint32_t p = cvt_bf16x2(x, y);
        reinterpret_cast<uint16_t*>(dst)[e0] = (uint16_t)p;
        reinterpret_cast<uint16_t*>(dst)[e1] = (uint16_t)(p >> 16);
      } else {
        reinterpret_cast<float*>(dst)[e0] = x;
        reinterpret_cast<float*>(dst)[e1] = y;
      }
    }
  }
}

}  // namespace tsd

using namespace tsd;

extern "C" {

tsd_status tsd_rope_init(tsd_rope* rope, int32_t rotary_dim, double theta, int32_t interleaved,
                         const tsd_rope_scaling* scaling) {
  if (rope == nullptr || !(theta > 1.0) || !isfinite(theta)) return TSD_ERR_INVALID_ARGUMENT;
  if (rotary_dim < 2 || rotary_dim > 128 || (rotary_dim & 1)) return TSD_ERR_UNSUPPORTED;
  tsd_rope_scaling s;
  memset(&s, 0, sizeof(s));
  if (scaling != nullptr) s = *scaling;
  const int kind = s.kind;
  if (kind < TSD_ROPE_PLAIN || kind > TSD_ROPE_YARN) return TSD_ERR_INVALID_ARGUMENT;
  if (kind != TSD_ROPE_PLAIN && (!(s.factor >= 1.0) || !isfinite(s.factor))) return TSD_ERR_INVALID_ARGUMENT;
  if (kind == TSD_ROPE_BANDED || kind == TSD_ROPE_YARN) {
    if (!(s.original_max_len > 0.0) || !isfinite(s.original_max_len)) return TSD_ERR_INVALID_ARGUMENT;
  }
  if (kind == TSD_ROPE_BANDED &&
      (!(s.low_freq_factor > 0.0) || !(s.high_freq_factor > s.low_freq_factor) || !isfinite(s.high_freq_factor)))
    return TSD_ERR_INVALID_ARGUMENT;
  if (kind == TSD_ROPE_YARN && (!(s.beta_slow > 0.0) || !(s.beta_fast > s.beta_slow) || !isfinite(s.beta_fast) ||
                                !(s.attention_factor >= 0.0) || !isfinite(s.attention_factor)))
    return TSD_ERR_INVALID_ARGUMENT;
  const long double two_pi = 6.283185307179586476925286766559L;
  const int R = rotary_dim;
  long double th = theta;
  if (kind == TSD_ROPE_NTK && R > 2) th *= powl((long double)s.factor, (long double)R / (R - 2));
  memset(rope, 0, sizeof(*rope));
  rope->rotary_dim = R;
  rope->interleaved = interleaved != 0;
  rope->mscale = 1.f;
  long double lo = 0, hi = 0;
  if (kind == TSD_ROPE_YARN) {
    const long double L = s.original_max_len;
    lo = floorl(R * logl(L / (s.beta_fast * two_pi)) / (2 * logl(th)));
    hi = ceill(R * logl(L / (s.beta_slow * two_pi)) / (2 * logl(th)));
    if (lo < 0) lo = 0;
    if (hi > R - 1) hi = R - 1;
    rope->mscale = (float)(s.attention_factor > 0.0 ? s.attention_factor : 0.1 * log(s.factor) + 1.0);
  }
  for (int i = 0; i < R / 2; ++i) {
    long double f = powl(th, -2.0L * i / R);
    if (kind == TSD_ROPE_LINEAR) {
      f /= s.factor;
    } else if (kind == TSD_ROPE_BANDED) {
      const long double r = s.original_max_len * f / two_pi;
      long double t = (r - s.low_freq_factor) / ((long double)s.high_freq_factor - s.low_freq_factor);
      t = t < 0 ? 0 : (t > 1 ? 1 : t);
      f = (1 - t) * f / s.factor + t * f;
    } else if (kind == TSD_ROPE_YARN) {
      const long double width = hi - lo > 0.001L ? hi - lo : 0.001L;
      long double t = (i - lo) / width;
      t = t < 0 ? 0 : (t > 1 ? 1 : t);
      f = f / s.factor * t + f * (1 - t);
    }
    rope->turn[i] = (uint64_t)rintl(f / two_pi * 18446744073709551616.0L);   // f <= 1 rad: below 2^62
  }
  return TSD_OK;
}

tsd_status tsd_rope_append(const tsd_kv_cache* cache, const tsd_queries* queries, const tsd_rope* rope,
                           int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                           int64_t v_stride, const int32_t* positions, const int32_t* depth, void* out_q,
                           uint32_t* status, tsd_stream_t stream) {
  RopeArgs a;
  memset(&a, 0, sizeof(a));
  Shapes sh;
  if (queries == nullptr) return TSD_ERR_INVALID_ARGUMENT;
  const tsd_queries q = bound_tokens(*queries);
  const tsd_status st = check_inputs(cache, &q, &a.kv, &a.qv, &sh);
  if (st != TSD_OK) return st;
  if (rope == nullptr || k_new == nullptr || v_new == nullptr || out_q == nullptr) return TSD_ERR_INVALID_ARGUMENT;
  if (rope->rotary_dim < 2 || rope->rotary_dim > 128 || (rope->rotary_dim & 1)) return TSD_ERR_UNSUPPORTED;
  if (positions != nullptr && depth != nullptr) return TSD_ERR_INVALID_ARGUMENT;
  const int per16 = a.qv.q_f32 ? 4 : 8;
  if (q_stride < sh.hq * kHeadDim || k_stride < sh.hkv * kHeadDim || v_stride < sh.hkv * kHeadDim ||
      q_stride % per16 || k_stride % per16 || v_stride % per16)
    return TSD_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)k_new | (uintptr_t)v_new | (uintptr_t)out_q) & 15) return TSD_ERR_INVALID_ARGUMENT;
  // blocks write out_q while others read: only a row onto itself is safe
  const int64_t T = sh.tokens, esz = a.qv.q_f32 ? 4 : 2, out_bytes = T * sh.hq * kHeadDim * esz;
  auto span = [&](int64_t stride, int64_t heads) { return ((T - 1) * stride + heads * kHeadDim) * esz; };
  const bool in_place = out_q == a.qv.q && (T == 1 || q_stride == sh.hq * kHeadDim);
  if ((!in_place && overlap(out_q, out_bytes, a.qv.q, span(q_stride, sh.hq))) ||
      overlap(out_q, out_bytes, k_new, span(k_stride, sh.hkv)) || overlap(out_q, out_bytes, v_new, span(v_stride, sh.hkv)))
    return TSD_ERR_INVALID_ARGUMENT;
  a.rope = *rope;
  a.rope.interleaved = rope->interleaved != 0;
  a.k_new = k_new;
  a.v_new = v_new;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.positions = positions;
  a.depth = depth;
  a.out_q = out_q;
  a.status = status;
  // A token a block (four were no faster: 136 us against 133 at 32768 tokens, 47 against 39 at 8192),
  // unless the bound lies far above most sequences, where most blocks find no token.
  a.toks = (int64_t)sh.batch * sh.max_tokens > 4LL * sh.tokens ? kRopeMaxToks : 1;
  const int64_t per_seq = (sh.max_tokens + a.toks - 1) / a.toks;
  if (per_seq * sh.batch > 0x7fffffffLL) return TSD_ERR_UNSUPPORTED;
  a.chunks = (int)per_seq;
  const unsigned grid = (unsigned)(per_seq * sh.batch);
  const bool vec = rope->rotary_dim % (a.rope.interleaved ? 8 : 16) == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (a.qv.q_f32) {
    if (vec) rope_append_kernel<true, true><<<grid, kRopeThreads, 0, s>>>(a);
    else rope_append_kernel<true, false><<<grid, kRopeThreads, 0, s>>>(a);
  } else {
    if (vec) rope_append_kernel<false, true><<<grid, kRopeThreads, 0, s>>>(a);
    else rope_append_kernel<false, false><<<grid, kRopeThreads, 0, s>>>(a);
  }
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
