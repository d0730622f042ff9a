// Trees of drafted tokens: ancestor masks, and decode attention in which a draft sees the tokens
// before the drafts and the drafts named by its mask.
#include <math.h>
#include <stdlib.h>
#include <string.h>

#include "tsd_host.h"
#include "tsd_umma.cuh"

namespace tsd {

constexpr int kMaxTree = 512;   // drafts of a sequence

// ---------------------------------------------------------------------------
// Ancestor masks
// ---------------------------------------------------------------------------
// One block per sequence.  mask(j) = {j} u mask(parent(j)) by doubling: after round r row j holds
// j and its first 2^r - 1 ancestors and up[j] names the next one, so a chain of n drafts takes
// ceil(log2 n) rounds over shared memory instead of n dependent steps.  4 to 5 us for 1 to 37 trees with
// the launch, which is what bounds it.
constexpr int kTmThreads = 256;
constexpr size_t tree_mask_smem(int drafts, int words) { return (size_t)2 * drafts * (1 + words) * sizeof(int32_t); }

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
// Tree attention on the tensor cores
// ---------------------------------------------------------------------------
// The rows of a tile are lists: (draft, q head) pairs of one (sequence, kv head), list L = draft * G +
// head.  With R lists a tile, K and V are read once for all of them and every 512-byte K/V row costs
// 512 R flop, against a ridge of about 250 flop per byte: up to some 250 lists the cache's bytes bound
// the kernel, beyond them the tensor cores and the exponentials do.  Measured (bf16): 8 contexts of up
// to 32768 tokens, 16 drafts x 4 heads, 173 us = 6.2 TB/s, 95% of a plain copy's rate; one draft, 170 us;
// 4 contexts of up to 131072, 32 drafts x 8 heads, 543 us = 1.01 PFLOP/s, 62% of a large library product.
// There the chain maximum -> exponentials -> P -> products of each stream is what bounds it.
//
// Work: unit = (sequence, kv head, tile of kRows lists), cut along the context into tiles of TT tokens.
// All units' tiles form one line, of which every CTA (one per SM) takes an equal share, so a ragged
// batch keeps all SMs busy to the end and one long sequence spreads over all of them.  A share is a run
// of segments (stretches of one unit).  A unit inside one share is written directly; one that is cut
// leaves a partial state (m, l, O) per share, at most two a CTA, merged by tree_merge_kernel in the
// order of the shares.
//
// A CTA: warps 0-3 and 4-7 are two streams of 128 lists, one list a thread (= a tensor-memory lane);
// warps 8 and 9 issue a stream's MMAs; warps 10 and 12 load the K tiles by TMA, 11 and 13 the V tiles,
// every other tile each (one warp issues a box in some 80 cycles, too slow for pages of 16).
//   S_s = Q_s K^T   (M 128, N TT, K 128; operands in shared memory, fp32 in tensor memory)
//   softmax in registers: running maximum and sum per thread, P rounded to bf16 into tensor memory
//   O_s += P_s V    (M 128, N 128, K TT; P from tensor memory, V MN-major from shared memory)
// While one stream is in its softmax the tensor cores work for the other.  More than 128 lists: the
// streams hold different lists and share each K and V tile.  Up to 128 (DUAL false): both hold the
// same lists and take alternate tiles; their states are merged at the segment's end.
// O is rescaled lazily: only when a maximum grows by more than 2^8, so weights stay below 2^8.
// With different lists, a warp of each stream shares an SM quarter's exponential unit: they take it in
// turn, so that one's exponentials run under the other's waits (128K case: 576 us without).
//
// Precision: fp32 queries enter as three bf16 parts (QP = 3, exact to 2^-24); with fp32 outputs the
// weights do too (PP = 3).  With bf16 outputs the weights are rounded to bf16 once (2^-8 at most,
// averaged over the row), as the outputs are; the sum l is always of the unrounded fp32 weights.
// The 64-list case above: fp32 queries 221 us (three times the score products), fp32 outputs 283 us,
// both 354 us.  No unit is busy there (captured at 4 x 8K: tensor pipe 35%, tensor memory 39%, DRAM 24%, issue
// slots 21%): a stream's chain of dependent steps is longer, and sets the pace.
//
// Tiles that reach past the committed tokens ("special": drafts, or the end of the sequence) take a
// longer path: scores are masked by each list's bits; rows of V behind the sequence are zeroed in
// shared memory (0 x NaN is NaN), and so are drafts' rows that hold infinities or NaNs, whose
// products are then added for those lists alone that see them.
//
// Every wait is bounded; a wait that gives up raises `abort`, after which all waits return at once.  A
// producer or an issuer whose wait gave up stops, and no issuer begins another segment, so that a slot of the
// ring is called empty only when its products are done, and filled only when it is empty; the softmax warps
// run out over whatever their buffers hold.  The CTA ends with TSD_DEV_TIMEOUT set once its copies and MMAs in
// flight are through (waited for apart from `abort`).
struct TreeArgs {
  KvView kv;
  QView qv;
  const uint32_t* mask;
  int32_t words;       // 32-bit words of a mask row
  int32_t part_rows;   // rows of a partial state
  void* out;
  int32_t out_f32;
  float* lse;
  uint32_t* status;
  int32_t* line;       // [0] tiles in all, [1 + b] first tile of sequence b
  float2* part_ml;     // [2 * CTAs][part_rows] (maximum, sum), base-2 units
  float4* part_acc;    // [2 * CTAs][32][part_rows] four dims of an unnormalised row
  float4* sums;        // [CTAs][2][32][128] sums of a stream's products (fp32 outputs)
  int32_t ctas;
  uint32_t tries;      // of up to a microsecond each, after which a wait gives up
};

constexpr int kTaThreads = 512;
// 8 warps x 32 x (192 + 64) = the 65536 registers of 512 threads at 128.  A softmax thread holds a row
// of 64 scores; the other roles need no more than 64.
constexpr int kTaSoftmaxRegs = 192, kTaOtherRegs = 64;
constexpr int kTaRowsPerStream = 128;
constexpr int kTaTiles = 229376;               // Q tiles and the ring
constexpr size_t kTaSmem = 227 * 1024;         // then barriers and scratch: all of an SM's shared memory

template <int QP, int PP>
struct TreeShape {
  // Weights in three parts (PP = 3) take 1.5 tensor-memory columns a token, and a stream has 128 columns
  // for S and P.  fp32 queries: tiles of 64 tokens, P in two halves of 32 behind S (kSplit), which keeps
  // the scores' three parts at N 64.  bf16 queries: tiles of 32 tokens, whose S and P are double-buffered.
  // Measured (8 x 32K context, 64 lists), split and not (moving O every
  // 512 tokens): fp32 queries 344 and 387 us, bf16 310 and 287.
  static constexpr bool kSplit = QP == 3 && PP == 3;
  static constexpr int TT = PP == 1 || kSplit ? 64 : 32;     // tokens of a tile
  static constexpr int PT = kSplit ? 32 : TT;                // tokens whose weights P holds at a time
  static constexpr int kRows = QP == 1 ? 256 : 128;          // lists of a unit: two Q tiles, or one in three parts
  static constexpr int kQBytes = (QP == 1 ? 2 : 3) * 32768;
  static constexpr int kSlotBytes = TT * 256;                // one K or V tile
  // Ring slots of K and of V.  A K tile is done with once its scores are made, a V tile waits for the
  // softmax in between.
  static constexpr int kSlots = (kTaTiles - kQBytes) / kSlotBytes;
  // Both even: where the streams take alternate tiles, a slot then serves one stream throughout a
  // segment, and its waits see every phase of the slot's barriers (a parity says no more than that).
  static constexpr int kKSlots = (kSlots * 2 / 5 + 1) & ~1, kVSlots = kSlots - kKSlots;
  static_assert(kKSlots % 2 == 0 && kVSlots % 2 == 0 && kKSlots >= 4 && kVSlots >= 4, "ring slots");
  // Steps whose products add up in tensor memory before they are moved to fp32 sums in global
  // memory (fp32 outputs only; 0: never).  The tensor cores truncate each sum: measured, V = 1 came out
  // 6.6e-9 low per accumulation, 2e-5 over 80000 tokens.  Every 512, 256, 128 tokens: errors up to 1.5,
  // 1.25, 0.85 of a plain fp32 form's; 64 bf16 lists over 8 x 32K in 264, 283, 325 us.
  static constexpr int kFlush = PP == 1 ? 0 : 256 / TT;
};

// What one sequence contributes: its descriptor and its units.
struct TreeSeq {
  int t0, n, len, base, mtiles, tiles;
};
template <class SH>
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, int G, bool report) {
  TreeSeq s;
  const SeqRaw r = seq_load(a.kv, a.qv, b);
  const int n = r.t1 - r.t0;
  if (r.len < 0 || r.len > a.kv.max_seq_len || r.t0 < 0 || n < 0 || r.t1 > a.qv.num_tokens || n > a.qv.max_tokens ||
      n > r.len) {
    if (report) flag_optional(a.status, TSD_DEV_BAD_SEQ);
    s.t0 = s.n = s.len = s.base = s.mtiles = s.tiles = 0;
    return s;
  }
  s.t0 = r.t0;
  s.n = n;
  s.len = r.len;
  s.base = r.len - n;
  s.mtiles = (n * G + SH::kRows - 1) / SH::kRows;
  s.tiles = n > 0 ? (r.len + SH::TT - 1) / SH::TT : 0;
  return s;
}

// The line of `total` tiles cut into shares for C CTAs (C <= total): the first total % C shares have
// one tile more than the others.
struct TreeShares {
  int q, r;
  __device__ __forceinline__ TreeShares(int total, int C) : q(total / C), r(total % C) {}
  __device__ __forceinline__ int begin(int c) const { return c * q + min(c, r); }
  __device__ __forceinline__ int owner(int x) const {   // the CTA whose share holds tile x
    const int big = r * (q + 1);
    return x < big ? x / (q + 1) : r + (x - big) / q;
  }
};

// CTAs that share `total` tiles: two tiles each at least, one a stream.
__host__ __device__ __forceinline__ int tree_ctas(int ctas, int total) { return min(ctas, (total + 1) / 2); }

// The segments of a CTA's share, in order; every warp role walks them by itself.
template <class SH>
struct TreeWalk {
  TreeSeq s;
  int b, g, mt, k0, k1;   // segment: tiles [k0, k1) of unit (b, g, mt)
  int left;               // tiles of the share from k0 on

  __device__ __forceinline__ void start(const TreeArgs& a, int G, int b0, int off, int share) {
    b = b0;
    left = share;
    if (left <= 0) return;
    s = tree_seq<SH>(a, b, G, false);
    if (s.tiles == 0 || s.mtiles == 0) {   // only when lengths change under the call
      left = 0;
      return;
    }
    const int unit = off / s.tiles;
    g = unit / s.mtiles;
    mt = unit % s.mtiles;
    k0 = off - unit * s.tiles;
    cut();
  }
  __device__ __forceinline__ void cut() { k1 = min(s.tiles, k0 + left); }
  __device__ __forceinline__ bool live() const { return left > 0; }
  __device__ __forceinline__ void next(const TreeArgs& a, int G) {
    left -= k1 - k0;
    if (left <= 0) return;
    k0 = 0;
    if (++mt == s.mtiles) {
      mt = 0;
      if (++g == a.kv.hkv) {
        g = 0;
#pragma unroll 1
        do {
          if (++b >= a.kv.batch) {
            left = 0;
            return;
          }
          s = tree_seq<SH>(a, b, G, false);
        } while (s.tiles == 0 || s.mtiles == 0);
      }
    }
    cut();
  }
  __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == s.tiles; }
  // whether the streams hold different lists of the unit
  __device__ __forceinline__ bool dual(int G) const {
    return SH::kRows > kTaRowsPerStream && s.n * G - mt * SH::kRows > kTaRowsPerStream;
  }
};

// Shared-memory control block behind the Q tiles and the ring.
struct TreeCtl {
  uint64_t k_full[8], k_empty[8], v_full[12], v_empty[12];
  // A stream's 128 columns for S and P are two buffers: step k keeps both in buffer k % 2, with these
  // barriers' phase k / 2; s_full of step k implies that the products of step k - 2 are done, so no wait
  // is two phases behind.  Split: S has columns 0 to 63, free again (s_free) as soon as the softmax has
  // read it, P those behind it; p_ready[s][0] and o_done[s][0] count halves of steps.
  // q_ready[s] has a phase for each segment in which stream s has steps, since an issuer waits in those
  // alone: in a segment of one tile nothing holds the others until stream 1's issuer has come by, which over
  // a run of such segments could be more than one phase late.  fixed[s][buf] (not split): a special step is through
  // with the P of its buffer.  The scores of the step after it are made already, so its fixed can come before the
  // issuer has waited for this one's: hence one for each buffer.
  uint64_t q_ready[2], s_full[2][2], s_free[2], p_ready[2][2], o_done[2][2], fixed[2][2], drain[2];
  uint32_t abort, tries, tmem, nf[2][2];
  // Rows with a bad page of tile m (counted over the CTA's share), at m % 32: K is loaded at most
  // 4 (two steps of two streams) + kKSlots <= 12 tiles ahead of the softmax.
  uint32_t bad[32][2];
  int scan[kTaThreads / 32], off, b0;
  float2 ml[2][kTaRowsPerStream];
};
static_assert(sizeof(TreeCtl) <= kTaSmem - kTaTiles, "control block");

// Bounded wait that gives way to `abort`: up to c->tries tries of up to a microsecond each.  Counted, not
// timed, to keep the code small: the kernel's waits are many, and an instruction cache miss costs
// a warp some hundred cycles.
// Whether the phase was complete.
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, TreeCtl* c, uint32_t* status) {
#pragma unroll 1
  for (uint32_t tries = 0; !mbar_try_wait_suspend(bar, parity, 1000u);) {
    if (*reinterpret_cast<volatile uint32_t*>(&c->abort)) return false;
    if (++tries >= c->tries) {
      atomicOr(&c->abort, 1u);
      flag_optional(status, TSD_DEV_TIMEOUT);
      return false;
    }
  }
  return true;
}
// Whether the phase of the given parity is complete.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok)
               : "r"(smem_u32(bar)), "r"(parity)
               : "memory");
  return ok != 0;
}

// tree_wait by all lanes of a warp, converged again behind it (as .aligned instructions need).  Most
// phases are complete by the time they are waited for, and a test says so sooner than a try.
// Whether the phase was complete, the same answer for all lanes.
__device__ __forceinline__ bool tree_wait_warp(uint64_t* bar, uint32_t parity, TreeCtl* c, uint32_t* status) {
  if (__all_sync(0xFFFFFFFFu, mbar_test(bar, parity))) return true;
  const bool complete = tree_wait(bar, parity, c, status);
  return __all_sync(0xFFFFFFFFu, complete);
}

// Whether a wait of this CTA has given up, the same answer for all lanes.
__device__ __forceinline__ bool tree_gave_up(TreeCtl* c) {
  return __any_sync(0xFFFFFFFFu, *reinterpret_cast<volatile uint32_t*>(&c->abort) != 0);
}

template <int N>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xFFFFFFFF;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
// Of a whole warp, converged (bar.sync and bar.arrive are aligned instructions).
__device__ __forceinline__ void pair_wait(int id) { asm volatile("bar.sync %0, 64;\n" ::"r"(id) : "memory"); }
__device__ __forceinline__ void pair_arrive(int id) { asm volatile("bar.arrive %0, 64;\n" ::"r"(id) : "memory"); }
__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); }

// The tokens [tw, tw + 32) that draft j of the sequence sees, as bits.
__device__ __forceinline__ uint32_t tree_visible32(const TreeArgs& a, const TreeSeq& s, int j, int tw) {
  const int d0 = tw - s.base;   // draft index of the first token
  uint32_t bits = 0;
  if (d0 + 31 >= 0 && d0 < s.n) {
    if (a.mask == nullptr) {
      bits = low_bits(j + 1 - d0);
    } else {
      const uint32_t* row = a.mask + (int64_t)(s.t0 + j) * a.words;
      if (d0 < 0) {
        bits = __ldg(row) << -d0;
      } else {
        const int w = d0 >> 5;
        const uint32_t lo = w < a.words ? __ldg(row + w) : 0u, hi = w + 1 < a.words ? __ldg(row + w + 1) : 0u;
        bits = __funnelshift_r(lo, hi, d0 & 31);
      }
    }
  }
  return (low_bits(-d0) | bits) & low_bits(s.len - tw);
}
// The same for a tile of TT tokens.
template <int TT>
__device__ __noinline__ uint64_t tree_visible(const TreeArgs& a, TreeSeq s, int j, int tw) {
  uint64_t v = tree_visible32(a, s, j, tw);
  if (TT > 32) v |= (uint64_t)tree_visible32(a, s, j, tw + 32) << 32;
  return v;
}

// The paths that few tiles take stand outside the softmax loop, so that they cost it no registers
// (kTaSoftmaxRegs a thread; what spills goes to L2, since shared memory takes nearly all of the L1).
// Tensor memory is read and written by whole warps: the instructions need all 32 lanes, converged.  Every
// condition around one of these calls or such an instruction is therefore the same for a warp -- the role,
// warp_live, the step's number, `special`, the tile's marks, a ballot -- and what a lane decides for itself
// (valid, seen, m) is data: a factor, a mask or a store that is left out.

// O of this warp's lists times f.
__device__ __noinline__ void tree_scale(uint32_t to, float f) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float o[32];
    tmem_ld32(to + c * 32, o);
    tmem_wait_ld();
    tmem_loaded32(o);
#pragma unroll
    for (int d = 0; d < 32; ++d) o[d] *= f;
    tmem_st32(to + c * 32, o);
  }
  tmem_wait_st();
}

// Four floats are added to *p in L2 (by this thread alone, so in a fixed order; subnormal sums count as 0).
__device__ __forceinline__ void red_add4(float4* p, const float* x) {
  asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"l"(p), "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]) : "memory");
}

// sums = sums * f + O (sums are taken as 0 when !have): this list's column of [32][128] float4.  Added
// in L2, without a wait, when f is 1.
__device__ __noinline__ void tree_flush(uint32_t to, float4* sums, float f, bool have, bool valid) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float o[32];
    __syncwarp();
    tmem_ld32(to + c * 32, o);
    tmem_wait_ld();
    tmem_loaded32(o);
    if (!valid) continue;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      float4* p = sums + (8 * c + d) * kTaRowsPerStream;
      if (have && f == 1.f) {
        red_add4(p, o + 4 * d);
      } else {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (have) x = __ldcg(p);
        __stcg(p, make_float4(x.x * f + o[4 * d], x.y * f + o[4 * d + 1], x.z * f + o[4 * d + 2], x.w * f + o[4 * d + 3]));
      }
    }
  }
}

// O += sums * f.
__device__ __noinline__ void tree_unflush(uint32_t to, const float4* sums, float f, bool valid) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float o[32];
    __syncwarp();
    tmem_ld32(to + c * 32, o);
    tmem_wait_ld();
    tmem_loaded32(o);
    if (valid) {
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        const float4 x = __ldcg(sums + (8 * c + d) * kTaRowsPerStream);
        o[4 * d] += f * x.x;
        o[4 * d + 1] += f * x.y;
        o[4 * d + 2] += f * x.z;
        o[4 * d + 3] += f * x.w;
      }
    }
    __syncwarp();
    tmem_st32(to + c * 32, o);
  }
  tmem_wait_st();
}

// A special tile's V in shared memory (`threads` threads, index id, share the work; bar is theirs): rows
// behind the sequence and drafts' rows that are not finite become zeros.  Returns the latter as bits.
template <int TT>
__device__ __noinline__ uint64_t tree_clean_v(unsigned char* vt, uint32_t* found, int t0, int base, int len, int id,
                                              int threads, int bar) {
  named_sync(bar, threads);
  if (id < 2) found[id] = 0;
  named_sync(bar, threads);
#pragma unroll 1
  for (int e = id; e < TT * 16; e += threads) {
    const int r = e >> 4, ch = e & 15, t = t0 + r;
    if (t < base) continue;
    uint4* p = reinterpret_cast<uint4*>(vt + (ch >> 3) * (TT * 128) + sw128(r, ch & 7));
    if (t >= len) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 v = *p;
    uint32_t odd = 0;   // an exponent of all ones
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t u = w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
      odd |= ((u & 0x7F80u) == 0x7F80u) | ((u & 0x7F800000u) == 0x7F800000u);
    }
    if (odd) atomicOr(&found[r >> 5], 1u << (r & 31));
  }
  named_sync(bar, threads);
  const uint64_t any = (uint64_t)found[1] << 32 | found[0];
  if (any) {
#pragma unroll 1
    for (int e = id; e < TT * 16; e += threads) {
      const int r = e >> 4, ch = e & 15;
      if (any >> r & 1)
        *reinterpret_cast<uint4*>(vt + (ch >> 3) * (TT * 128) + sw128(r, ch & 7)) = make_uint4(0, 0, 0, 0);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
  if (threads == 256) named_sync(bar, threads);   // the other stream's products read these rows too
  __syncwarp();   // tensor-memory instructions follow
  return any;
}

// Adds to O the products of the rows of V that were zeroed for their infinities or NaNs (`rows`), for
// the lists that see them (`seen`).  P, of PT tokens, is still in tensor memory, at tp.
template <int PT, int PP>
__device__ __noinline__ void tree_add_nonfinite(const KvView& kv, int b, int g, int t0, uint64_t rows, uint64_t seen,
                                                uint32_t tp, uint32_t to) {
  for (; rows != 0; rows &= rows - 1) {
    const int r = __ffsll((long long)rows) - 1;
    float p = 0.f;
#pragma unroll 1
    for (int part = 0; part < PP; ++part) {
      uint32_t w = tmem_ld1(tp + part * (PT / 2) + ((r % PT) >> 1));
      tmem_wait_ld();
      asm volatile("" : "+r"(w));
      p += (r & 1) ? bf16hi(w) : bf16lo(w);
    }
    const uint32_t vr = kv_row(kv, b, g, t0 + r);
    if (vr == kInvalidRow) continue;
    const uint16_t* v = kv.v + (int64_t)vr * kHeadDim;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float o[32];
      __syncwarp();
      tmem_ld32(to + c * 32, o);
      tmem_wait_ld();
      tmem_loaded32(o);
      if (seen >> r & 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(v + c * 32) + e), x);
#pragma unroll
          for (int d = 0; d < 8; ++d) o[8 * e + d] += p * x[d];
        }
      }
      __syncwarp();
      tmem_st32(to + c * 32, o);
    }
    tmem_wait_st();
  }
}

template <int QP, int PP>
__global__ void __launch_bounds__(kTaThreads, 1)
    tree_decode_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ KvMaps maps) {
  using SH = TreeShape<QP, PP>;
  constexpr int TT = SH::TT, KS = SH::kKSlots, VS = SH::kVSlots;
  extern __shared__ __align__(1024) unsigned char ta_smem[];
  unsigned char* qtile = ta_smem;
  unsigned char* kring = ta_smem + SH::kQBytes;
  unsigned char* vring = kring + KS * SH::kSlotBytes;
  TreeCtl* ctl = reinterpret_cast<TreeCtl*>(ta_smem + kTaTiles);
  // the broadcast tells the compiler that the role, and what follows from it, is the same for a warp
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0), lane = tid & 31;
  const int G = a.qv.hq / a.kv.hkv;
  pdl_launch_dependents();
  if (smem_u32(ta_smem) & 1023u) {   // the swizzled tiles need 1024-byte alignment
    if (tid == 0) flag_optional(a.status, TSD_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < SH::kKSlots; ++i) {
      mbar_init(&ctl->k_full[i], 1);
      mbar_init(&ctl->k_empty[i], 2);
    }
    for (int i = 0; i < SH::kVSlots; ++i) {
      mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->v_empty[i], 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->q_ready[s], 256);
      for (int d = 0; d < 2; ++d) {
        mbar_init(&ctl->s_full[s][d], 1);
        mbar_init(&ctl->p_ready[s][d], 128);
        mbar_init(&ctl->o_done[s][d], 1);
        mbar_init(&ctl->fixed[s][d], 128);
      }
      mbar_init(&ctl->s_free[s], 128);
      mbar_init(&ctl->drain[s], 1);
    }
    ctl->abort = 0;
    ctl->tries = a.tries;
    ctl->b0 = ctl->off = 0;
    mbar_fence_init();
  }
  if (warp == 10) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  // The line of all units' tiles: running sums over the sequences, then the sequence this CTA's
  // share starts in.
  int total = 0, begin = -1, share = 0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    int run = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.kv.batch; b0 += kTaThreads) {
      const int b = b0 + tid;
      int cost = 0;
      if (b < a.kv.batch) {
        const TreeSeq s = tree_seq<SH>(a, b, G, pass == 0 && blockIdx.x == 0);
        cost = s.mtiles * s.tiles * a.kv.hkv;
      }
      int x = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) ctl->scan[warp] = x;
      __syncthreads();
      int before = run + x - cost;
#pragma unroll 1
      for (int w = 0; w < kTaThreads / 32; ++w) {
        if (w < warp) before += ctl->scan[w];
        run += ctl->scan[w];
      }
      if (pass == 0) {
        if (blockIdx.x == 0 && b < a.kv.batch) a.line[1 + b] = before;
      } else if (begin >= before && begin < before + cost) {
        ctl->b0 = b;
        ctl->off = begin - before;
      }
    }
    if (pass == 0) {
      total = run;
      const int C = tree_ctas(a.ctas, total);
      if ((int)blockIdx.x < C) {
        const TreeShares shares(total, C);
        begin = shares.begin(blockIdx.x);
        share = shares.begin(blockIdx.x + 1) - begin;
      }
    }
  }
  if (blockIdx.x == 0 && tid == 0) a.line[0] = total;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem;
  if (warp < 8) {
    take_registers<kTaSoftmaxRegs>();
    TreeWalk<SH> wk;
    wk.start(a, G, ctl->b0, ctl->off, share);
    // ---- softmax: a list a thread
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;   // this warp's tensor-memory lanes
    const uint32_t tm = tmem + lanes + s * 256, to = tm + 128;  // S and P (two buffers), O
    float scale = a.qv.sm_scale * 1.44269504088896340736f;   // base-2 units
    // The tensor cores truncate the sums of a score's products: measured, scores come out 2^-23 low on
    // average, which the scale makes up for (errors of fp32 outputs fall by a fifth, of lse by a third).  A score
    // whose products add up without a rounding comes out 2^-23 of itself high by it: a unit in its last place or two.
    if (PP == 3) scale = fmaf(scale, 0x1p-23f, scale);
    float4* sums = a.sums + ((int64_t)blockIdx.x * 2 + s) * 32 * kTaRowsPerStream + row;   // kFlush: this list's sums
    uint32_t done = 0, tiles_done = 0;
#pragma unroll 1
    for (; wk.live(); wk.next(a, G)) {
      const TreeSeq& sq = wk.s;
      const bool dual = wk.dual(G);
      const int ntile = wk.k1 - wk.k0;
      const int steps = dual ? ntile : (s ? ntile / 2 : (ntile + 1) / 2);
      const int lists = sq.n * G;
      const int first = wk.mt * SH::kRows + (dual ? s * kTaRowsPerStream : 0);
      const int list = first + row;
      const bool valid = list < lists, warp_live = first + 32 * (warp & 3) < lists;
      // the warp of the other stream on the same quarter of the SM has work too
      const bool pair = PP == 1 && dual && wk.mt * SH::kRows + kTaRowsPerStream + 32 * (warp & 3) < lists;
      __syncwarp();   // lanes without a list left the last segment's stores early
      if (pair && s == 1) pair_arrive(4 + 2 * (warp & 3));   // stream 0 goes first
      const int j = list / G, h = wk.g * G + (list - j * G);
      named_sync(1, 256);   // the previous segment's Q tiles and states are done with
      {
        unsigned char* q0 = qtile + (dual && s ? 32768 : 0);
        const int threads = dual ? 128 : 256, id = dual ? row : tid;
#pragma unroll 1
        for (int i = id; i < 128 * 16; i += threads) {
          const int r = i >> 4, ch = i & 15, ls = first + r;
          uint4 part[3];
          part[0] = part[1] = part[2] = make_uint4(0, 0, 0, 0);
          if (ls < lists) {
            const int jj = ls / G;
            const int64_t at = ((int64_t)(sq.t0 + jj) * a.qv.hq + wk.g * G + (ls - jj * G)) * kHeadDim + ch * 8;
            if (QP == 1) {
              part[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.qv.q) + at));
            } else {
              float x[8];
              const float4 u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.qv.q) + at));
              const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.qv.q) + at + 4));
              x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
              x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
#pragma unroll
              for (int p = 0; p < 3; ++p) {   // each part takes the next 8 bits
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  w[e] = cvt_bf16x2(x[2 * e], x[2 * e + 1]);
                  x[2 * e] -= bf16lo(w[e]);
                  x[2 * e + 1] -= bf16hi(w[e]);
                }
                part[p] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
          }
          const uint32_t off = (ch >> 3) * 16384 + sw128(r, ch & 7);
#pragma unroll
          for (int p = 0; p < QP; ++p) *reinterpret_cast<uint4*>(q0 + p * 32768 + off) = part[p];
        }
      }
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      mbar_arrive(&ctl->q_ready[0]);
      if (dual || ntile > 1) mbar_arrive(&ctl->q_ready[1]);   // stream 1 has steps

      float m = -INFINITY, l = 0.f;
      float m_sum = -INFINITY;   // reference of the sums moved to global memory; -inf: none yet
      uint64_t seen = 0;         // the special tile's tokens that this list sees
      auto products_done = [&](uint32_t step) {   // O holds all products up to this step's
        if (!SH::kSplit) tree_wait_warp(&ctl->o_done[s][step & 1], (step >> 1) & 1, ctl, a.status);
        else tree_wait_warp(&ctl->o_done[s][0], 1, ctl, a.status);   // its second half
        tc_fence_after_sync();
      };
#pragma unroll 1
      for (int i = 0; i < steps; ++i) {
        const int at = dual ? i : 2 * i + s, tile = wk.k0 + at;
        const uint32_t step = done + i, num = tiles_done + at;
        const bool special = (tile + 1) * TT > sq.base;
        const uint32_t buf = SH::kSplit ? 0 : step & 1, tb = tm + buf * 64;   // S
        if (SH::kFlush && i > 0 && i % (SH::kFlush ? SH::kFlush : 1) == 0 && warp_live) {
          products_done(step - 1);
          tree_flush(to, sums, m_sum == -INFINITY ? 0.f : fast_exp2(m_sum - m), m_sum != -INFINITY, valid);
          m_sum = m;
        }
        const uint32_t s_phase = (SH::kSplit ? step : step >> 1) & 1;
        tree_wait_warp(&ctl->s_full[s][buf], s_phase, ctl, a.status);
        tc_fence_after_sync();
        float x[TT];
        uint32_t bad0 = 0, bad1 = 0;
        if (warp_live) {
#pragma unroll
          for (int c = 0; c < TT / 32; ++c) tmem_ld32(tb + 32 * c, x + 32 * c);
          const volatile uint32_t* marks = ctl->bad[num & 31];
          bad0 = marks[0];
          if (TT > 32) bad1 = marks[1];
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < TT / 32; ++c) tmem_loaded32(x + 32 * c);
        }
        if (SH::kSplit) {
          tc_fence_before_sync();
          mbar_arrive(&ctl->s_free[s]);
        }
        if (warp_live) {
          if (special || (bad0 | bad1)) {   // the marks are the tile's: every lane comes here or none
            const uint64_t bad = (uint64_t)bad1 << 32 | bad0;
            seen = tree_visible<TT>(a, sq, valid ? j : 0, tile * TT) & ~bad;   // called by every lane
            if (!valid) seen = 0;
            __syncwarp();
#pragma unroll
            for (int c = 0; c < TT; ++c) x[c] = seen >> c & 1 ? x[c] : -INFINITY;
          }
          float mx8[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) mx8[c] = x[c];
#pragma unroll
          for (int c = 8; c < TT; c += 2) mx8[(c >> 1) & 7] = max3(mx8[(c >> 1) & 7], x[c], x[c + 1]);
          const float mx = max3(max3(mx8[0], mx8[1], mx8[2]), max3(mx8[3], mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])) * scale;
          if (i == 0) {
            m = mx;
          } else {
            const bool grow = mx > m + 8.f;
            if (__any_sync(0xFFFFFFFFu, grow)) {
              const float f = grow ? fast_exp2(m - mx) : 1.f;
              if (grow) m = mx;
              l *= f;
              products_done(step - 1);
              tree_scale(to, f);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;   // nothing seen yet: weights 0
        const float2 scale2 = make_float2(scale, scale), ref2 = make_float2(-ref, -ref);
        uint64_t odd = 0;
        auto clean_v = [&]() {
          const uint32_t slot = num % VS;
          tree_wait_warp(&ctl->v_full[slot], (num / VS) & 1, ctl, a.status);
          odd = tree_clean_v<TT>(vring + (size_t)slot * SH::kSlotBytes, ctl->nf[dual ? 0 : s], tile * TT, sq.base, sq.len,
                                 dual ? tid : row, dual ? 256 : 128, dual ? 1 : 2 + s);
        };
        // Weights of 32 tokens: exponentials and their sum, then P in PP parts.
        float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weigh = [&](float* p) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 z = __ffma2_rn(make_float2(p[e], p[e + 1]), scale2, ref2);
            p[e] = fast_exp2(z.x);
            p[e + 1] = fast_exp2(z.y);
            l2[(e >> 1) & 1] = __fadd2_rn(l2[(e >> 1) & 1], make_float2(p[e], p[e + 1]));
          }
        };
        auto store_p = [&](float* p, uint32_t at) {
#pragma unroll
          for (int part = 0; part < PP; ++part) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              w[e] = cvt_bf16x2(p[2 * e], p[2 * e + 1]);
              if (part + 1 < PP) {
                p[2 * e] -= bf16lo(w[e]);
                p[2 * e + 1] -= bf16hi(w[e]);
              }
            }
            tmem_st16(at + part * (SH::PT / 2), w);
          }
        };
        if constexpr (!SH::kSplit) {
          if (warp_live) {
            if (pair) pair_wait(4 + 2 * (warp & 3) + s);
#pragma unroll
            for (int c = 0; c < TT / 32; ++c) {
              weigh(x + 32 * c);
              store_p(x + 32 * c, tb + 16 * c);
            }
            if (pair) pair_arrive(4 + 2 * (warp & 3) + (s ^ 1));
            l2[0] = __fadd2_rn(l2[0], l2[1]);
            l += l2[0].x + l2[0].y;
            tmem_wait_st();
          }
          if (special) clean_v();
          tc_fence_before_sync();
          mbar_arrive(&ctl->p_ready[s][buf]);
          if (special) {
            if (odd != 0 && warp_live) {
              products_done(step);
              tree_add_nonfinite<SH::PT, PP>(a.kv, wk.b, wk.g, tile * TT, odd, seen, tb, to);
              tc_fence_before_sync();
            }
            if (i + 2 < steps) mbar_arrive(&ctl->fixed[s][buf]);
          }
        } else {
          if (special) clean_v();
          const uint32_t tp = tm + 64;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            if (warp_live) weigh(x + 32 * c);
            // the products of the half before this one
            if (c > 0 || step > 0) tree_wait_warp(&ctl->o_done[s][0], c ^ 1, ctl, a.status);
            if (warp_live) {
              store_p(x + 32 * c, tp);
              tmem_wait_st();
            }
            tc_fence_before_sync();
            mbar_arrive(&ctl->p_ready[s][0]);
            if (special) {
              const uint64_t here = odd & (c ? ~0ull << 32 : 0xFFFFFFFFull);
              if (here != 0) {
                tree_wait_warp(&ctl->o_done[s][0], c, ctl, a.status);
                tc_fence_after_sync();
                if (warp_live) tree_add_nonfinite<SH::PT, PP>(a.kv, wk.b, wk.g, tile * TT, here, seen, tp, to);
                tc_fence_before_sync();
              }
            }
          }
          l2[0] = __fadd2_rn(l2[0], l2[1]);
          if (warp_live) l += l2[0].x + l2[0].y;
        }
      }
      __syncwarp();
      if (pair && s == 0) pair_wait(4 + 2 * (warp & 3));   // the other stream's last turn
      if (steps > 0) products_done(done + steps - 1);
      tc_fence_after_sync();
      done += steps;
      tiles_done += ntile;

      // ---- the segment's state: O / l where the unit is whole, else a partial state
      float w0 = 1.f, w1 = 0.f;
      bool two = false;
      // The sums in global memory come on top.  Whether there are any is the same for a whole warp; a list that
      // had seen nothing when they were moved last (m_sum -inf) has zeros there, which count for nothing.
      if (SH::kFlush && steps > SH::kFlush && warp_live)
        tree_unflush(to, sums, m_sum == -INFINITY ? 0.f : fast_exp2(m_sum - m), valid);
      if (!dual) {
        ctl->ml[s][row] = make_float2(m, l);
        tc_fence_before_sync();
        named_sync(1, 256);
        const float2 x = ctl->ml[0][row], y = ctl->ml[1][row];
        two = ntile > 1;
        m = two ? fmaxf(x.x, y.x) : x.x;
        w0 = x.x == -INFINITY ? 0.f : fast_exp2(x.x - m);
        w1 = !two || y.x == -INFINITY ? 0.f : fast_exp2(y.x - m);
        if (x.x == INFINITY) w0 = 1.f;   // its sum is not a number already
        if (two && y.x == INFINITY) w1 = 1.f;
        l = w0 * x.y + (two ? w1 * y.y : 0.f);
      }
      tc_fence_after_sync();
      if (warp_live) {
        const bool whole = wk.whole();
        const float norm = !whole ? 1.f : (l == 0.f ? 0.f : 1.f / l);
        const int64_t lst = (int64_t)(sq.t0 + j) * a.qv.hq + h;
        const int64_t slot = 2 * (int64_t)blockIdx.x + (wk.k0 == 0);
        const int prow = (dual ? s * kTaRowsPerStream : 0) + row;
        const uint32_t o0 = tmem + lanes + 128 + (dual ? s * 256 : 0), o1 = tmem + lanes + 256 + 128;
        const int c0 = dual ? 0 : 2 * s, c1 = dual ? 4 : c0 + 2;   // 32-dim pieces of the row
        if (valid && (dual || s == 0)) {
          if (whole) {
            if (a.lse != nullptr)
              a.lse[lst] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
          } else {
            a.part_ml[slot * a.part_rows + prow] = make_float2(m, l);
          }
        }
#pragma unroll 1
        for (int c = c0; c < c1; ++c) {
          float o[32], o2[32];
          __syncwarp();
          tmem_ld32(o0 + 32 * c, o);
          if (two) tmem_ld32(o1 + 32 * c, o2);
          tmem_wait_ld();
          tmem_loaded32(o);
          if (two) {
            tmem_loaded32(o2);
#pragma unroll
            for (int d = 0; d < 32; ++d) o[d] = w0 * o[d] + w1 * o2[d];
          }
          if (!valid) continue;
          if (!whole) {
            float4* part = a.part_acc + (slot * 32 + 8 * c) * a.part_rows + prow;
#pragma unroll
            for (int d = 0; d < 8; ++d)
              part[(int64_t)d * a.part_rows] = make_float4(o[4 * d], o[4 * d + 1], o[4 * d + 2], o[4 * d + 3]);
          } else if (a.out_f32) {
            float4* out = static_cast<float4*>(a.out) + lst * 32 + 8 * c;
#pragma unroll
            for (int d = 0; d < 8; ++d)
              out[d] = make_float4(o[4 * d] * norm, o[4 * d + 1] * norm, o[4 * d + 2] * norm, o[4 * d + 3] * norm);
          } else {
            uint4* out = static_cast<uint4*>(a.out) + lst * 16 + 4 * c;
#pragma unroll
            for (int d = 0; d < 4; ++d)
              out[d] = make_uint4(cvt_bf16x2(o[8 * d] * norm, o[8 * d + 1] * norm),
                                  cvt_bf16x2(o[8 * d + 2] * norm, o[8 * d + 3] * norm),
                                  cvt_bf16x2(o[8 * d + 4] * norm, o[8 * d + 5] * norm),
                                  cvt_bf16x2(o[8 * d + 6] * norm, o[8 * d + 7] * norm));
          }
        }
      }
      tc_fence_before_sync();
    }
  } else {
    give_registers<kTaOtherRegs>();
    TreeWalk<SH> wk;
    wk.start(a, G, ctl->b0, ctl->off, share);
  if (warp >= 10 && warp < 14) {
    // ---- producers: warp 10 loads K, warp 11 V, tile n of the share into slot n % slots of its ring.
    // The TMA unit takes about 80 cycles for a box of 16 rows x 128 bytes, 25 bytes a cycle against
    // the 23 that are an SM's part of the HBM rate, so little may stand between the boxes: the page
    // numbers of 32 boxes are fetched and resolved at once, the next 32 while those are used.
    const bool is_v = warp & 1;
    const uint32_t odd = (warp - 10) >> 1;
    const CUtensorMap* map = is_v ? &maps.v : &maps.k;
    unsigned char* ring = is_v ? vring : kring;
    uint64_t *full = is_v ? ctl->v_full : ctl->k_full, *empty = is_v ? ctl->v_empty : ctl->k_empty;
    const uint32_t slots = is_v ? VS : KS;
    // Pages of 4 or more tokens: boxes of `per` rows, one a lane; smaller pages: four rows a lane.
    // Measured, 8 x 16 drafts over 32K: pages of 8 183 us in boxes, 280 gathered; of 4 256 and 280; of 1
    // 288 (a copy instruction for every four rows and half row).
    const bool paged = a.kv.page_table != nullptr, gather = paged && a.kv.page_shift < 2;
    const int shift = paged ? a.kv.page_shift : 0, in_page = (1 << shift) - 1;
    const int per = !paged ? TT : (gather ? 4 : min(TT, 1 << shift));
    const int per_tile = TT / per, window = 32 / per_tile;   // boxes of a tile, tiles of 32 boxes
    const int page_rows = a.kv.hkv << shift, no_row = (int)(a.kv.num_pages * page_rows);   // no_row: zeros arrive
    const uint32_t num_pages = (uint32_t)a.kv.num_pages;
    uint32_t n = 0;
    bool stop = false;
#pragma unroll 1
    for (; wk.live() && !stop; wk.next(a, G)) {
      const int len = wk.s.len;
      // rows that no other unit reads are the first to leave L2
      const uint64_t pol = wk.s.mtiles == 1 ? l2_evict_first() : l2_evict_normal();
      const int32_t* table = a.kv.page_table + (int64_t)wk.b * a.kv.max_pages;
      const int head_row = paged ? wk.g << shift : (wk.b * a.kv.hkv + wk.g) * a.kv.max_seq_len;
      int page[4], y[4];
      uint32_t bad = 0, any_bad = 0;
      auto fetch = [&](int tile) {   // asks for the page numbers of this lane's rows of 32 boxes
        const int t = tile * TT + lane * per;
        page[0] = paged && t < len ? __ldg(table + (t >> shift)) : 0;
        if (gather) {
#pragma unroll
          for (int e = 1; e < 4; ++e) page[e] = t + e < len ? __ldg(table + ((t + e) >> shift)) : 0;
        }
      };
      auto resolve = [&](int tile) {
        const int t = tile * TT + lane * per;
        if (!paged) {
          y[0] = head_row + t;
        } else {
          bad = (uint32_t)page[0] >= num_pages;
          y[0] = bad ? no_row : page[0] * page_rows + head_row + (t & in_page);
          if (gather) {
#pragma unroll
            for (int e = 1; e < 4; ++e) {
              const bool none = (uint32_t)page[e] >= num_pages;
              bad |= (uint32_t)none << e;
              y[e] = none ? no_row : page[e] * page_rows + head_row + ((t + e) & in_page);
            }
          }
          any_bad = __ballot_sync(0xFFFFFFFFu, bad != 0);
          if (bad && !is_v) flag_optional(a.status, TSD_DEV_BAD_PAGE);
        }
      };
      fetch(wk.k0);
#pragma unroll 1
      for (int tile = wk.k0, w = 0; tile < wk.k1; ++tile, ++n) {
        if (w == 0) {
          resolve(tile);
          if (tile + window < wk.k1) fetch(tile + window);
        }
        const uint32_t slot = n % slots, round = n / slots;
        const int box0 = w * per_tile, boxes = min(per_tile, (len - tile * TT + per - 1) / per);
        if (++w == window) w = 0;
        if ((n & 1) != odd) continue;
        if (round > 0 && !tree_wait_warp(&empty[slot], (round - 1) & 1, ctl, a.status)) {
          stop = true;
          break;
        }
        if (!is_v) {
          uint32_t* marks = ctl->bad[n & 31];
          if (lane < 2) marks[lane] = 0;
          if (any_bad >> box0 & low_bits(per_tile)) {   // rows of bad pages, as bits of the tile
            __syncwarp();
            const int r0 = (lane - box0) * per;
            if (lane >= box0 && r0 < TT)
#pragma unroll 1
              for (int e = 0; e < per; ++e)
                if (bad & (gather ? 1u << e : 1u)) atomicOr(&marks[(r0 + e) >> 5], 1u << ((r0 + e) & 31));
          }
          __syncwarp();
        }
        unsigned char* dst = ring + slot * SH::kSlotBytes;
        const bool one = elect_one();
        if (one) mbar_arrive_expect_tx(&full[slot], (uint32_t)(boxes * per * 256));
        // one thread issues: a TMA instruction with other operands in every lane is split up
        if (gather) {
#pragma unroll 1
          for (int i = 0; i < boxes; ++i) {
            int yi[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) yi[e] = __shfl_sync(0xFFFFFFFFu, y[e], box0 + i);
            if (one) {
              tma_gather4_hint(dst + i * 512, map, 0, yi, &full[slot], pol);
              tma_gather4_hint(dst + TT * 128 + i * 512, map, 64, yi, &full[slot], pol);
            }
          }
        } else {
#pragma unroll 1
          for (int i = 0; i < boxes; ++i) {
            const int yi = __shfl_sync(0xFFFFFFFFu, y[0], box0 + i);
            if (one) {
              tma_load_2d_hint(dst + i * per * 128, map, 0, yi, &full[slot], pol);
              tma_load_2d_hint(dst + TT * 128 + i * per * 128, map, 64, yi, &full[slot], pol);
            }
          }
        }
      }
    }
    // No copy may be in flight when the CTA ends: the last tiles that this warp asked for (those below n), whether
    // or not a wait has given up.
    bool landed = true;
#pragma unroll 1
    for (uint32_t i = n > slots ? n - slots : 0; i < n; ++i)
      if ((i & 1) == odd) landed &= mbar_wait(&full[i % slots], (i / slots) & 1);
    if (!landed) flag_optional(a.status, TSD_DEV_TIMEOUT);
    __syncwarp();
  }
  else if (warp == 8 || warp == 9) {
    // ---- MMA issuers: one thread for each stream.  A step's products are followed by the scores of the
    // step after next, into the buffer that the products have just read (MMAs run in order).
    {
      const int s = warp - 8;
      constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, TT), idesc_o = umma_idesc_bf16_f32_bmn(128, 128);
      const uint64_t q_desc = sw128_desc(smem_u32(qtile), 1024), ring_k = sw128_desc(smem_u32(kring), 1024),
                     ring_v = sw128_mn_desc(smem_u32(vring), TT * 128, 1024);
      const uint32_t tm = tmem + s * 256;
      uint32_t tiles_done = 0, done = 0, segs = 0;   // segs: those in which this stream has steps
      uint32_t fixes = 0;                            // bit b: parity of the next phase of fixed[s][b]
      bool stop = false;
#pragma unroll 1
      for (; wk.live() && !stop; wk.next(a, G)) {
        const bool dual = wk.dual(G);
        const int ntile = wk.k1 - wk.k0, stride = dual ? 1 : 2, first = dual ? 0 : s;
        const int steps = (ntile - first + stride - 1) / stride;
        const uint64_t qd = q_desc + (dual && s ? 32768 >> 4 : 0);
        if (steps > 0) {
          // The softmax warps announce queries even when a wait has given up: then the other stream's tiles may not
          // have come, and a slot's barrier may be a phase behind what a wait here takes it for.
          if (!tree_wait_warp(&ctl->q_ready[s], segs++ & 1, ctl, a.status) || tree_gave_up(ctl)) break;
          tc_fence_after_sync();
        }
        auto scores = [&](int i) -> bool {
          const uint32_t n = tiles_done + first + stride * i, slot = n % KS, buf = SH::kSplit ? 0 : (done + i) & 1;
          if (!tree_wait_warp(&ctl->k_full[slot], (n / KS) & 1, ctl, a.status)) return false;
          tc_fence_after_sync();
          if (elect_one()) {
            const uint64_t kd = ring_k + (uint64_t)(slot * (SH::kSlotBytes >> 4));
#pragma unroll 1
            for (int p = QP - 1; p >= 0; --p)   // the small parts first: every step rounds the sum so far
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                umma_bf16(tm + buf * 64, qd + ((p * 32768 + (ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                          kd + (((ks >> 2) * (TT * 128) + (ks & 3) * 32) >> 4), idesc_s, p < QP - 1 || ks > 0);
            umma_commit(&ctl->s_full[s][buf]);
            umma_commit(&ctl->k_empty[slot]);   // expects both streams; a tile of one stream counts twice
            if (!dual) umma_commit(&ctl->k_empty[slot]);
          }
          __syncwarp();
          return true;
        };
        // O += P V over the P's tokens, from k step k0 of the tile on; the small parts first
        auto products = [&](uint32_t pt, uint64_t vd, int k0, bool fresh) {
#pragma unroll
          for (int p = PP - 1; p >= 0; --p)
#pragma unroll
            for (int ks = 0; ks < SH::PT / 16; ++ks)
              umma_bf16_ts(tm + 128, pt + p * (SH::PT / 2) + ks * 8, vd + ((k0 + ks) * 2048 >> 4), idesc_o,
                           !fresh || p < PP - 1 || ks > 0);
        };
        if constexpr (!SH::kSplit) {
#pragma unroll 1
          for (int i = -2; i < steps; ++i) {
            const int at = first + stride * i;
            if (i >= 0) {
              const uint32_t n = tiles_done + at, slot = n % VS, buf = (done + i) & 1;
              stop = !tree_wait_warp(&ctl->v_full[slot], (n / VS) & 1, ctl, a.status) ||
                     !tree_wait_warp(&ctl->p_ready[s][buf], ((done + i) >> 1) & 1, ctl, a.status);
              if (stop) break;
              tc_fence_after_sync();
              if (elect_one()) {
                products(tm + buf * 64, ring_v + (uint64_t)(slot * (SH::kSlotBytes >> 4)), 0,
                         SH::kFlush ? i % (SH::kFlush ? SH::kFlush : 1) == 0 : i == 0);
                umma_commit(&ctl->o_done[s][buf]);
                umma_commit(&ctl->v_empty[slot]);
                if (!dual) umma_commit(&ctl->v_empty[slot]);
              }
              __syncwarp();
            }
            if (i + 2 < steps) {
              if (i >= 0 && (wk.k0 + at + 1) * TT > wk.s.base) {   // a special tile: P is read once more
                const uint32_t buf = (done + i) & 1;
                stop = !tree_wait_warp(&ctl->fixed[s][buf], fixes >> buf & 1, ctl, a.status);
                if (stop) break;
                fixes ^= 1u << buf;
                tc_fence_after_sync();
              }
              stop = !scores(i + 2);
              if (stop) break;
            }
          }
        } else {
#pragma unroll 1
          for (int i = -1; i < steps; ++i) {
            if (i + 1 < steps) {   // S(i + 1) is made while the weights of S(i) are
              stop = done + i + 1 > 0 && !tree_wait_warp(&ctl->s_free[s], (done + i) & 1, ctl, a.status);
              if (stop) break;
              tc_fence_after_sync();
              stop = !scores(i + 1);
              if (stop) break;
            }
            if (i < 0) continue;
            const uint32_t n = tiles_done + first + stride * i, slot = n % VS;
            const uint64_t vd = ring_v + (uint64_t)(slot * (SH::kSlotBytes >> 4));
            stop = !tree_wait_warp(&ctl->v_full[slot], (n / VS) & 1, ctl, a.status);
#pragma unroll 1
            for (int c = 0; c < 2 && !stop; ++c) {
              stop = !tree_wait_warp(&ctl->p_ready[s][0], c, ctl, a.status);
              if (stop) break;
              tc_fence_after_sync();
              if (elect_one()) {
                products(tm + 64, vd, 2 * c, c == 0 && i % (SH::kFlush ? SH::kFlush : 1) == 0);
                umma_commit(&ctl->o_done[s][0]);
                if (c == 1) {
                  umma_commit(&ctl->v_empty[slot]);
                  if (!dual) umma_commit(&ctl->v_empty[slot]);
                }
              }
              __syncwarp();
            }
            if (stop) break;
          }
        }
        tiles_done += ntile;
        done += steps;
      }
      // no MMA may be in flight when tensor memory is freed
      if (elect_one()) {
        umma_commit(&ctl->drain[s]);
        if (!mbar_wait(&ctl->drain[s], 0)) flag_optional(a.status, TSD_DEV_TIMEOUT);
      }
    }
    __syncwarp();
  }
  }
  __syncthreads();
  if (warp == 10) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Merge of the partial states of units cut over several CTAs, in the order of the shares.  One block
// per 32 lists of a (sequence, kv head) and 16 ND of their dims; a lane per list, so that the states'
// rows are read whole.  The warps find the weights of kTgShares shares at a time, which they keep in
// shared memory, then take 4 ND dims each, in two halves of the shares, with eight rows under way: a
// short step of one user has 33 shares to merge and few lists to do it with (ND = 1), a batch has more
// blocks than the SMs hold, each with its chain of dependent loads (ND = 4).
constexpr int kTgThreads = 256;
constexpr int kTgWarps = kTgThreads / 32;
constexpr int kTgShares = 32;

template <int QP, int PP, int ND>
__global__ void __launch_bounds__(kTgThreads) tree_merge_kernel(const __grid_constant__ TreeArgs a, int groups) {
  using SH = TreeShape<QP, PP>;
  __shared__ float weight[kTgShares][32];
  __shared__ float red[kTgWarps][32];
  __shared__ float4 half[4 * ND][32];
  constexpr int kSlices = 8 / ND, kAhead = 8 / ND;
  const int slice = blockIdx.x % kSlices, unit = blockIdx.x / kSlices;
  const int rg = unit % groups, g = (unit / groups) % a.kv.hkv, b = unit / groups / a.kv.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.qv.hq / a.kv.hkv;
  const TreeSeq sq = tree_seq<SH>(a, b, G, false);
  const int lists = sq.n * G;
  pdl_wait();
  if (rg * 32 >= lists) return;
  const int total = a.line[0];
  const TreeShares shares(total, tree_ctas(a.ctas, total));
  const int mt = rg * 32 / SH::kRows, u0 = a.line[1 + b] + (g * sq.mtiles + mt) * sq.tiles;
  const int c0 = shares.owner(u0), parts = shares.owner(u0 + sq.tiles - 1) - c0 + 1;
  if (parts == 1) return;   // written directly
  const int list = rg * 32 + lane, prow = list - mt * SH::kRows;
  const bool valid = list < lists;
  const int row = min(prow, a.part_rows - 1);
  // the first share of the unit starts at its first tile: its state is in the odd slot
  auto slot = [&](int p) { return 2 * (int64_t)(c0 + p) + (p == 0 ? 1 : 0); };
  // the first rows are on their way while the weights are found
  const int d4 = slice * 4 * ND + (warp & 3), p0 = warp >> 2;   // and every fourth after it
  float4 x[kAhead][ND];
  auto ask = [&](int q) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (q + 2 * i < parts) x[i][d] = __ldcg(a.part_acc + (slot(q + 2 * i) * 32 + d4 + 4 * d) * a.part_rows + row);
  };
  ask(p0);
  float m = -INFINITY;
#pragma unroll 2
  for (int p = warp; p < parts; p += kTgWarps) m = fmaxf(m, __ldcg(&a.part_ml[slot(p) * a.part_rows + row].x));
  red[warp][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTgWarps; ++w) m = fmaxf(m, red[w][lane]);
  float l = 0.f;
  float4 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < parts; s0 += kTgShares) {
    const int s1 = min(parts, s0 + kTgShares);
    if (s0 > 0) __syncthreads();
#pragma unroll 2
    for (int p = s0 + warp; p < s1; p += kTgWarps) {
      const float2 ml = __ldcg(a.part_ml + slot(p) * a.part_rows + row);
      // a share in which the list saw nothing (l = 0) counts for nothing; one whose scores were all -inf or NaN
      // has the maximum -inf and a sum that is not a number, which stays
      const float w = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : (ml.x == m ? 1.f : fast_exp2(ml.x - m));
      weight[p - s0][lane] = w;
      if (ml.x != -INFINITY || w != 0.f) l += w * ml.y;
    }
    __syncthreads();
    for (int q = s0 + p0; q < s1; q += 2 * kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float w = q + 2 * i < s1 ? weight[q + 2 * i - s0][lane] : 0.f;
        if (w != 0.f) {   // else the share adds nothing, whatever its state holds
#pragma unroll
          for (int d = 0; d < ND; ++d) {
            o[d].x += w * x[i][d].x;
            o[d].y += w * x[i][d].y;
            o[d].z += w * x[i][d].z;
            o[d].w += w * x[i][d].w;
          }
        }
      }
      ask(q + 2 * kAhead);
    }
  }
  __syncthreads();
  red[warp][lane] = l;
  if (warp >= 4) {
#pragma unroll
    for (int d = 0; d < ND; ++d) half[(warp - 4) * ND + d][lane] = o[d];
  }
  __syncthreads();
  if (warp >= 4 || !valid) return;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kTgWarps; ++w) l += red[w][lane];
  const float norm = l == 0.f ? 0.f : 1.f / l;
  const int j = list / G;
  const int64_t lst = (int64_t)(sq.t0 + j) * a.qv.hq + g * G + (list - j * G);
#pragma unroll
  for (int d = 0; d < ND; ++d) {
    const float4 y = half[warp * ND + d][lane];
    const float4 z = make_float4((o[d].x + y.x) * norm, (o[d].y + y.y) * norm, (o[d].z + y.z) * norm, (o[d].w + y.w) * norm);
    const int64_t at = lst * 32 + d4 + 4 * d;
    if (a.out_f32) static_cast<float4*>(a.out)[at] = z;
    else static_cast<uint2*>(a.out)[at] = make_uint2(cvt_bf16x2(z.x, z.y), cvt_bf16x2(z.z, z.w));
  }
  if (warp == 0 && slice == 0 && a.lse != nullptr)
    a.lse[lst] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}
static_assert(kTgShares % 16 == 0, "rows asked for ahead run on into the next shares");

struct TreeLayout {
  size_t line, ml, acc, sums, total;
  int part_rows;
};
static TreeLayout tree_layout(const Shapes& sh, int ctas, bool q_f32, bool out_f32) {
  TreeLayout l;
  const int64_t lists = (sh.group * sh.max_tokens + 31) / 32 * 32, rows = q_f32 ? 128 : 256;
  l.part_rows = (int)(lists < rows ? lists : rows);
  l.line = 0;
  l.ml = align256((size_t)(1 + sh.batch) * sizeof(int32_t));
  l.acc = l.ml + align256((size_t)2 * ctas * l.part_rows * sizeof(float2));
  l.sums = l.acc + align256((size_t)2 * ctas * 32 * l.part_rows * sizeof(float4));
  l.total = l.sums + (out_f32 ? (size_t)2 * ctas * 32 * kTaRowsPerStream * sizeof(float4) : 0);
  return l;
}

template <int QP, int PP>
static cudaError_t launch_tree(const TreeArgs& a, const KvMaps& maps, int64_t batch, int groups, cudaStream_t stream) {
  const cudaError_t e = cudaFuncSetAttribute(tree_decode_kernel<QP, PP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)kTaSmem);
  if (e != cudaSuccess) return e;
  tree_decode_kernel<QP, PP><<<a.ctas, kTaThreads, kTaSmem, stream>>>(a, maps);
  const cudaError_t e2 = cudaGetLastError();
  if (e2 != cudaSuccess) return e2;
  const int64_t units = batch * a.kv.hkv * groups;
  if (units * 8 > a.ctas)   // 2 units: 18.4 us of a step with ND = 1, 20.8 with 4; 128 units: 178.6 and 174.4
    return launch_dependent(tree_merge_kernel<QP, PP, 4>, dim3((unsigned)(units * 2)), dim3(kTgThreads), 0, stream, a, groups);
  return launch_dependent(tree_merge_kernel<QP, PP, 1>, dim3((unsigned)(units * 8)), dim3(kTgThreads), 0, stream, a, groups);
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
  const size_t smem = tree_mask_smem(max_tokens, a.words);
  if (smem > 48 * 1024) {   // the largest trees' size, whatever this call's: another thread may be about to launch
    const cudaError_t e = cudaFuncSetAttribute(tree_mask_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)tree_mask_smem(kMaxTree, kMaxTree / 32));
    if (e != cudaSuccess) return TSD_ERR_CUDA;
  }
  tree_mask_kernel<<<batch, kTmThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cuda_status(cudaGetLastError());
}

size_t tsd_tree_decode_workspace_size(const tsd_kv_cache* cache, const tsd_queries* queries, int32_t out_dtype) {
  Shapes sh;
  if (queries == nullptr || (queries->q_indptr != nullptr && queries->max_tokens_per_seq > kMaxTree)) return 0;
  const tsd_queries q = bound_tokens(*queries);
  if (sizes_for(cache, &q, &sh) != TSD_OK) return 0;
  if (out_dtype != TSD_BF16 && out_dtype != TSD_F32) return 0;
  return tree_layout(sh, current_sm_count(), queries->q_dtype == TSD_F32, out_dtype == TSD_F32).total;
}

tsd_status tsd_tree_decode(const tsd_kv_cache* cache, const tsd_queries* queries, const uint32_t* mask, void* out,
                           int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, uint32_t* status,
                           tsd_stream_t stream) {
  TreeArgs a;
  Shapes sh;
  memset(&a, 0, sizeof(a));
  if (queries == nullptr) return TSD_ERR_INVALID_ARGUMENT;
  const tsd_queries q = bound_tokens(*queries);
  tsd_status st = check_inputs(cache, &q, &a.kv, &a.qv, &sh);
  if (st != TSD_OK) return st;
  if (out == nullptr || ws == nullptr || !queries->causal) return TSD_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)out & 15) || ((uintptr_t)ws & 255)) return TSD_ERR_INVALID_ARGUMENT;
  if (out_dtype != TSD_BF16 && out_dtype != TSD_F32) return TSD_ERR_UNSUPPORTED;
  const int max_tokens = queries->q_indptr == nullptr ? 1 : queries->max_tokens_per_seq;
  if (max_tokens > kMaxTree) return TSD_ERR_UNSUPPORTED;
  a.ctas = current_sm_count();
  const TreeLayout l = tree_layout(sh, a.ctas, a.qv.q_f32, out_dtype == TSD_F32);
  if (ws_bytes < l.total) return TSD_ERR_WORKSPACE_TOO_SMALL;
  // outputs are written while other blocks read queries
  const int64_t elems = sh.tokens * sh.hq * kHeadDim;
  if (overlap(out, elems * (out_dtype == TSD_F32 ? 4 : 2), a.qv.q, elems * (a.qv.q_f32 ? 4 : 2)))
    return TSD_ERR_INVALID_ARGUMENT;
  const int64_t groups = (sh.group * sh.max_tokens + 31) / 32;
  // positions up to a tile (and a producer's 32 boxes) behind a sequence are 32-bit numbers
  if (sh.max_seq_len > 0x7fffffffLL - 4096) return TSD_ERR_UNSUPPORTED;
  // the line of tiles and the merge's grid are counted in 32 bits
  if ((double)sh.batch * sh.hkv * groups * ((double)sh.max_seq_len / 32 + 8) >= 2147483647.0) return TSD_ERR_UNSUPPORTED;
  a.mask = mask;
  a.words = (max_tokens + 31) / 32;
  a.part_rows = l.part_rows;
  a.out = out;
  a.out_f32 = out_dtype == TSD_F32;
  a.lse = lse;
  a.status = status;
  char* w = static_cast<char*>(ws);
  a.line = reinterpret_cast<int32_t*>(w + l.line);
  a.part_ml = reinterpret_cast<float2*>(w + l.ml);
  a.part_acc = reinterpret_cast<float4*>(w + l.acc);
  a.sums = reinterpret_cast<float4*>(w + l.sums);
  const char* tries = getenv("TSD_TREE_WAIT_TRIES");   // for the tests of waits that run out
  a.tries = tries != nullptr ? (uint32_t)strtoul(tries, nullptr, 10) : 1u << 20;
  KvMaps maps;
  st = make_kv_maps(cache, &maps, a.out_f32 && !a.qv.q_f32 ? TreeShape<1, 3>::TT : TreeShape<3, 3>::TT, true);
  static_assert(TreeShape<3, 3>::TT == TreeShape<1, 1>::TT && TreeShape<3, 3>::TT == TreeShape<3, 1>::TT, "boxes of a tile");
  if (st != TSD_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.qv.q_f32) e = a.out_f32 ? launch_tree<3, 3>(a, maps, sh.batch, (int)groups, s) : launch_tree<3, 1>(a, maps, sh.batch, (int)groups, s);
  else e = a.out_f32 ? launch_tree<1, 3>(a, maps, sh.batch, (int)groups, s) : launch_tree<1, 1>(a, maps, sh.batch, (int)groups, s);
  return cuda_status(e);
}

}  // extern "C"
