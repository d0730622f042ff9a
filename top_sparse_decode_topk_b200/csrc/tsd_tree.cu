// Trees of drafted tokens: ancestor masks, and decode attention in which a draft sees the tokens
// before the drafts and the drafts named by its mask.
#include <math.h>
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
// Tree attention on the tensor cores
// ---------------------------------------------------------------------------
// The rows of a tile are lists: (draft, q head) pairs of one (sequence, kv head), list L = draft * G +
// head.  With R lists a tile, K and V are read once for all of them and every 512-byte K/V row costs
// 512 R flop, against a ridge of about 250 flop per byte: up to some 250 lists the cache's bytes bound
// the kernel, beyond them the tensor cores and the exponentials do.
//
// Work: unit = (sequence, kv head, tile of kRows lists), cut along the context into tiles of TT tokens.
// All units' tiles form one line, of which every CTA (one per SM) takes an equal share, so a ragged
// batch keeps all SMs busy to the end and one long sequence spreads over all of them.  A share is a run
// of segments (stretches of one unit).  A unit inside one share is written directly; one that is cut
// leaves a partial state (m, l, O) per share, at most two a CTA, merged by tree_merge_kernel in the
// order of the shares.
//
// A CTA: warps 0-3 and 4-7 are two streams of 128 lists, one list a thread (= a tensor-memory lane);
// warp 8 issues the MMAs; warp 9 loads K and V tiles by TMA.
//   S_s = Q_s K^T   (M 128, N TT, K 128; operands in shared memory, fp32 in tensor memory)
//   softmax in registers: running maximum and sum per thread, P rounded to bf16 into tensor memory
//   O_s += P_s V    (M 128, N 128, K TT; P from tensor memory, V MN-major from shared memory)
// While one stream is in its softmax the tensor cores work for the other.  More than 128 lists: the
// streams hold different lists and share each K and V tile.  Up to 128 (DUAL false): both hold the
// same lists and take alternate tiles; their states are merged at the segment's end.
// O is rescaled lazily: only when a maximum grows by more than 2^8, so weights stay below 2^8.
//
// Precision: fp32 queries enter as three bf16 parts (QP = 3, exact to 2^-24); with fp32 outputs the
// weights do too (PP = 3), over tiles of 64 tokens so that the parts fit the tensor memory that S
// leaves free.  With bf16 outputs the weights are rounded to bf16 once (2^-8 at most, averaged over
// the row), as the outputs are; the sum l is always of the unrounded fp32 weights.
//
// Tiles that reach past the committed tokens ("special": drafts, or the end of the sequence) take a
// longer path: scores are masked by each list's bits; rows of V behind the sequence are zeroed in
// shared memory (0 x NaN is NaN), and so are drafts' rows that hold infinities or NaNs, whose
// products are then added for those lists alone that see them.
//
// Every wait is bounded; a wait that gives up raises `abort`, after which all waits return at once,
// the loops run out, and the CTA ends with TSD_DEV_TIMEOUT set.
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
  int64_t* line;       // [0] tiles in all, [1 + b] first tile of sequence b
  float2* part_ml;     // [2 * CTAs][part_rows] (maximum, sum), base-2 units
  float4* part_acc;    // [2 * CTAs][32][part_rows] four dims of an unnormalised row
  int32_t ctas;
};

constexpr int kTaThreads = 320;
constexpr int kTaRowsPerStream = 128;
constexpr int kTaTiles = 229376;               // Q tiles and the ring
constexpr size_t kTaSmem = kTaTiles + 3072;    // then barriers and scratch: all of an SM's shared memory

template <int QP, int PP>
struct TreeShape {
  static constexpr int TT = QP == 1 && PP == 1 ? 128 : 64;   // tokens of a tile
  static constexpr int kRows = QP == 1 ? 256 : 128;          // lists of a unit: two Q tiles, or one in three parts
  static constexpr int kQBytes = (QP == 1 ? 2 : 3) * 32768;
  static constexpr int kSlotBytes = TT * 256;                // one K or V tile
  static constexpr int kSlots = (kTaTiles - kQBytes) / kSlotBytes;
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

// CTA whose share holds tile x of `total` (CTA c starts at floor(total c / C)).
__device__ __forceinline__ int tree_owner(int64_t x, int64_t total, int64_t C) { return (int)(((x + 1) * C - 1) / total); }

// The segments of a CTA's share, in order; every warp role walks them by itself.
template <class SH>
struct TreeWalk {
  TreeSeq s;
  int b, g, mt, k0, k1;   // segment: tiles [k0, k1) of unit (b, g, mt)
  int64_t left;           // tiles of the share from k0 on

  __device__ __forceinline__ void start(const TreeArgs& a, int G, int b0, int64_t off, int64_t share) {
    b = b0;
    left = share;
    if (left <= 0) return;
    s = tree_seq<SH>(a, b, G, false);
    const int64_t unit = off / s.tiles;
    g = (int)(unit / s.mtiles);
    mt = (int)(unit % s.mtiles);
    k0 = (int)(off - unit * s.tiles);
    cut();
  }
  __device__ __forceinline__ void cut() { k1 = (int)min((int64_t)s.tiles, k0 + left); }
  __device__ __forceinline__ bool live() const { return left > 0; }
  __device__ __forceinline__ void next(const TreeArgs& a, int G) {
    left -= k1 - k0;
    if (left <= 0) return;
    k0 = 0;
    if (++mt == s.mtiles) {
      mt = 0;
      if (++g == a.kv.hkv) {
        g = 0;
        do s = tree_seq<SH>(a, ++b, G, false); while (s.tiles == 0 || s.mtiles == 0);
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
  uint64_t full[16], empty[16];
  uint64_t q_ready, s_full[2], p_ready[2], o_done[2], fixed[2], drain;
  uint32_t abort, tmem, nf[2][4];
  // Rows with a bad page of tile m (counted over the CTA's share), at m % 16: the producer is at
  // most (kSlots + 1) / 2 tiles ahead of the softmax, whose tile's V it waits for.
  uint32_t bad[16][4];
  int64_t scan[10];
  int64_t total, off;
  int b0;
  float2 ml[2][kTaRowsPerStream];
};
static_assert(sizeof(TreeCtl) <= kTaSmem - kTaTiles, "control block");

// Bounded wait that gives way to `abort`.
__device__ __forceinline__ void tree_wait(uint64_t* bar, uint32_t parity, TreeCtl* c, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  while (!mbar_try_wait_suspend(bar, parity, 20000u)) {
    if (*reinterpret_cast<volatile uint32_t*>(&c->abort)) return;
    if (clock64() - t0 > kWaitCycles) {
      atomicOr(&c->abort, 1u);
      flag_optional(status, TSD_DEV_TIMEOUT);
      return;
    }
  }
}

// The same by all lanes of a warp, converged again behind it (as .aligned instructions need).
__device__ __forceinline__ void tree_wait_warp(uint64_t* bar, uint32_t parity, TreeCtl* c, uint32_t* status) {
  tree_wait(bar, parity, c, status);
  __syncwarp();
}

__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u); }

// The tokens [tw, tw + 32) that draft j of the sequence sees, as bits.
__device__ __forceinline__ uint32_t tree_visible(const TreeArgs& a, const TreeSeq& s, int j, int tw) {
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

// K or V tile `tile` of a segment into shared memory by TMA, all 32 lanes of the producer issuing.
// y: this lane's box coordinates, one box a lane (pages of 8 or more tokens: box rows `bp`), or four
// rows a lane (smaller pages).
template <int TT>
__device__ __forceinline__ void tree_issue(const CUtensorMap* map, unsigned char* dst, uint64_t* bar, const int (&y)[4],
                                           int bp, int rows, int lane, uint64_t pol) {
  if (bp >= 8) {
    const int boxes = (rows + bp - 1) / bp;
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(boxes * bp * 256));
    __syncwarp();
    if (lane < boxes) {
      tma_load_2d_hint(dst + lane * bp * 128, map, 0, y[0], bar, pol);
      tma_load_2d_hint(dst + TT * 128 + lane * bp * 128, map, 64, y[0], bar, pol);
    }
  } else {
    const int groups = (rows + 3) >> 2;
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(groups * 4 * 256));
    __syncwarp();
    if (lane < groups) {
      tma_gather4_hint(dst + lane * 512, map, 0, y, bar, pol);
      tma_gather4_hint(dst + TT * 128 + lane * 512, map, 64, y, bar, pol);
    }
  }
}

template <int QP, int PP>
__global__ void __launch_bounds__(kTaThreads, 1)
    tree_decode_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ KvMaps maps) {
  using SH = TreeShape<QP, PP>;
  constexpr int TT = SH::TT, NS = SH::kSlots;
  extern __shared__ __align__(1024) unsigned char ta_smem[];
  unsigned char* qtile = ta_smem;
  unsigned char* ring = ta_smem + SH::kQBytes;
  TreeCtl* ctl = reinterpret_cast<TreeCtl*>(ta_smem + kTaTiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.qv.hq / a.kv.hkv;
  pdl_launch_dependents();
  if (smem_u32(ta_smem) & 1023u) {   // the swizzled tiles need 1024-byte alignment
    if (tid == 0) flag_optional(a.status, TSD_DEV_TIMEOUT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&ctl->full[i], 1);
      mbar_init(&ctl->empty[i], 1);
    }
    mbar_init(&ctl->q_ready, 256);
    mbar_init(&ctl->drain, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctl->s_full[s], 1);
      mbar_init(&ctl->p_ready[s], 128);
      mbar_init(&ctl->o_done[s], 1);
      mbar_init(&ctl->fixed[s], 128);
    }
    ctl->abort = 0;
    mbar_fence_init();
  }
  if (warp == 9) {
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  // The line of all units' tiles: running sums over the sequences, then the sequence this CTA's
  // share starts in.
  int64_t total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t run = 0;
    const int64_t C = total > 0 ? min((int64_t)a.ctas, total) : 1;
    const int64_t begin = total * min((int64_t)blockIdx.x, C) / C;
    for (int b0 = 0; b0 < a.kv.batch; b0 += kTaThreads) {
      const int b = b0 + tid;
      int64_t cost = 0;
      if (b < a.kv.batch) {
        const TreeSeq s = tree_seq<SH>(a, b, G, pass == 0 && blockIdx.x == 0);
        cost = (int64_t)s.mtiles * s.tiles * a.kv.hkv;
      }
      int64_t x = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) ctl->scan[warp] = x;
      __syncthreads();
      int64_t before = run;
      for (int w = 0; w < kTaThreads / 32; ++w) {
        if (w < warp) before += ctl->scan[w];
        run += ctl->scan[w];
      }
      before += x - cost;
      if (pass == 0) {
        if (blockIdx.x == 0 && b < a.kv.batch) a.line[1 + b] = before;
      } else if (begin >= before && begin < before + cost) {
        ctl->b0 = b;
        ctl->off = begin - before;
      }
    }
    if (pass == 0) total = run;
  }
  if (blockIdx.x == 0 && tid == 0) a.line[0] = total;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = ctl->tmem;
  int64_t share = 0;
  if (total > 0) {
    const int64_t C = min((int64_t)a.ctas, total);
    if (blockIdx.x < C) share = total * (blockIdx.x + 1) / C - total * blockIdx.x / C;
  }
  TreeWalk<SH> wk;
  wk.start(a, G, ctl->b0, ctl->off, share);

  if (warp == 9) {
    // ---- producer: K and V of every tile of every segment, in order, load n into slot n % NS
    const int bp = a.kv.page_table == nullptr ? TT : min(TT, 1 << a.kv.page_shift);
    uint32_t n = 0;
    for (; wk.live(); wk.next(a, G)) {
      // rows that no other unit reads are the first to leave L2
      const uint64_t pol = wk.s.mtiles == 1 ? l2_evict_first() : l2_evict_normal();
      // this lane's rows of a tile: one box, or (small pages) four rows
      auto coords = [&](int tile, int (&y)[4], uint32_t& bad) {
        bad = 0;
        const int per = bp >= 8 ? bp : 4;
        const int t = tile * TT + lane * per;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = 0;
          if (e > 0 && bp >= 8) continue;
          const int te = t + e;
          if (lane * per >= TT || t >= wk.s.len) continue;
          if (a.kv.page_table == nullptr) {
            y[e] = (wk.b * a.kv.hkv + wk.g) * a.kv.max_seq_len + te;
            continue;
          }
          const int32_t page = te < wk.s.len
                                   ? __ldg(a.kv.page_table + (int64_t)wk.b * a.kv.max_pages + (te >> a.kv.page_shift)) : 0;
          if (page < 0 || (int64_t)page >= a.kv.num_pages) {
            bad |= 1u << e;
            y[e] = (int)(a.kv.num_pages * a.kv.hkv << a.kv.page_shift);   // past the last row: zeros arrive
          } else {
            y[e] = (int)((((int64_t)page * a.kv.hkv + wk.g) << a.kv.page_shift) | (te & ((1 << a.kv.page_shift) - 1)));
          }
        }
      };
      int y[4], y2[4];
      uint32_t bad, bad2;
      coords(wk.k0, y, bad);
      for (int tile = wk.k0; tile < wk.k1; ++tile) {
        if (tile + 1 < wk.k1) coords(tile + 1, y2, bad2);   // the page numbers of the next tile are under way
        const int rows = min(TT, wk.s.len - tile * TT);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const uint32_t slot = n % NS;
          if (n >= NS) tree_wait_warp(&ctl->empty[slot], (n / NS - 1) & 1, ctl, a.status);
          if (kv == 0) {
            // rows of bad pages, as bits of the tile
            const bool any = __any_sync(0xFFFFFFFFu, bad != 0);
            uint32_t* marks = ctl->bad[(n >> 1) & 15];
            if (lane < 4) marks[lane] = 0;
            __syncwarp();
            if (any) {
              const int per = bp >= 8 ? bp : 4;
              if (bad) flag_optional(a.status, TSD_DEV_BAD_PAGE);
              for (int e = 0; e < per && lane * per < TT; ++e)
                if (bad & (bp >= 8 ? 1u : 1u << e)) 
                  atomicOr(&marks[(lane * per + e) >> 5], 1u << ((lane * per + e) & 31));
              __syncwarp();
            }
          }
          tree_issue<TT>(kv ? &maps.v : &maps.k, ring + (size_t)slot * SH::kSlotBytes, &ctl->full[slot], y, bp, rows, lane,
                         pol);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = y2[e];
        bad = bad2;
      }
    }
    // no copy may be in flight when the CTA ends
    for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i) tree_wait_warp(&ctl->full[i % NS], (i / NS) & 1, ctl, a.status);
  }
  else if (warp == 8) {
    // ---- MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc_s = umma_idesc_bf16_f32(128, TT), idesc_o = umma_idesc_bf16_f32_bmn(128, 128);
      uint32_t loads = 0, done[2] = {0, 0}, fixes[2] = {0, 0}, segs = 0;
      for (; wk.live(); wk.next(a, G), ++segs) {
        const bool dual = wk.dual(G);
        const int ntile = wk.k1 - wk.k0;
        const int steps[2] = {dual ? ntile : (ntile + 1) / 2, dual ? ntile : ntile / 2};
        tree_wait(&ctl->q_ready, segs & 1, ctl, a.status);
        tc_fence_after_sync();
        auto scores = [&](int s, int i) {
          const uint32_t n = loads + 2 * (dual ? i : 2 * i + s), slot = n % NS;
          tree_wait(&ctl->full[slot], (n / NS) & 1, ctl, a.status);
          tc_fence_after_sync();
          const uint32_t kb = smem_u32(ring + (size_t)slot * SH::kSlotBytes);
          const uint32_t qb = smem_u32(qtile) + (dual && s ? 32768u : 0u);
#pragma unroll
          for (int p = 0; p < QP; ++p)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              umma_bf16(tmem + s * 256, sw128_desc(qb + p * 32768 + (ks >> 2) * 16384 + (ks & 3) * 32, 1024),
                        sw128_desc(kb + (ks >> 2) * (TT * 128) + (ks & 3) * 32, 1024), idesc_s, p + ks > 0);
          umma_commit(&ctl->s_full[s]);
          if (!dual || s == 1) umma_commit(&ctl->empty[slot]);
        };
        for (int s = 0; s < 2; ++s)
          if (steps[s] > 0) scores(s, 0);
        for (int i = 0; i < steps[0]; ++i) {
          for (int s = 0; s < 2; ++s) {
            if (i >= steps[s]) continue;
            const int at = dual ? i : 2 * i + s;
            const uint32_t n = loads + 2 * at + 1, slot = n % NS;
            tree_wait(&ctl->p_ready[s], (done[s] + i) & 1, ctl, a.status);
            tree_wait(&ctl->full[slot], (n / NS) & 1, ctl, a.status);
            tc_fence_after_sync();
            const uint32_t vb = smem_u32(ring + (size_t)slot * SH::kSlotBytes);
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
              for (int ks = 0; ks < TT / 16; ++ks)
                umma_bf16_ts(tmem + s * 256 + 128, tmem + s * 256 + p * (TT / 2) + ks * 8,
                             sw128_mn_desc(vb + ks * 2048, TT * 128, 1024), idesc_o, i + p + ks > 0);
            umma_commit(&ctl->o_done[s]);
            if (!dual || s == 1) umma_commit(&ctl->empty[slot]);
            if (i + 1 < steps[s]) {
              if ((wk.k0 + at + 1) * TT > wk.s.base) {   // a special tile: P is read once more
                tree_wait(&ctl->fixed[s], fixes[s]++ & 1, ctl, a.status);
                tc_fence_after_sync();
              }
              scores(s, i + 1);
            }
          }
        }
        loads += 2 * ntile;
        done[0] += steps[0];
        done[1] += steps[1];
      }
      // no MMA may be in flight when tensor memory is freed
      umma_commit(&ctl->drain);
      if (!mbar_wait(&ctl->drain, 0)) flag_optional(a.status, TSD_DEV_TIMEOUT);
    }
    __syncwarp();
  } else {
    // ---- softmax: a list a thread
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;   // this warp's tensor-memory lanes
    const uint32_t tp = tmem + lanes + s * 256, to = tp + 128;  // S and P, O
    const float scale = a.qv.sm_scale * 1.44269504088896340736f;   // base-2 units
    uint32_t done = 0, tiles_done = 0;
    for (; wk.live(); wk.next(a, G)) {
      const TreeSeq& sq = wk.s;
      const bool dual = wk.dual(G);
      const int ntile = wk.k1 - wk.k0;
      const int steps = dual ? ntile : (s ? ntile / 2 : (ntile + 1) / 2);
      const int lists = sq.n * G;
      const int first = wk.mt * SH::kRows + (dual ? s * kTaRowsPerStream : 0);
      const int list = first + row;
      const bool valid = list < lists, warp_live = first + 32 * (warp & 3) < lists;
      const int j = list / G, h = wk.g * G + (list - j * G);
      named_sync(1, 256);   // the previous segment's Q tiles and states are done with
      {
        unsigned char* q0 = qtile + (dual && s ? 32768 : 0);
        const int threads = dual ? 128 : 256, id = dual ? row : tid;
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
      mbar_arrive(&ctl->q_ready);

      float m = -INFINITY, l = 0.f;
      uint32_t vis[TT / 32], nf[4] = {0, 0, 0, 0};
      // Adds to O the products of the rows of V that were zeroed for their infinities or NaNs, for
      // the lists that see them.  The tile's P is still in tensor memory.
      auto add_nonfinite = [&](int tile, uint32_t phase) {
        if ((nf[0] | nf[1] | nf[2] | nf[3]) == 0 || !warp_live) return;
        tree_wait_warp(&ctl->o_done[s], phase, ctl, a.status);
        tc_fence_after_sync();
        for (int r = 0; r < TT; ++r) {
          if (!(nf[r >> 5] >> (r & 31) & 1)) continue;
          float p = 0.f;
          for (int part = 0; part < PP; ++part) {
            uint32_t w = tmem_ld1(tp + part * (TT / 2) + (r >> 1));
            tmem_wait_ld();
            asm volatile("" : "+r"(w));
            p += (r & 1) ? bf16hi(w) : bf16lo(w);
          }
          bool seen = false;
#pragma unroll
          for (int w = 0; w < TT / 32; ++w)
            if ((r >> 5) == w) seen = vis[w] >> (r & 31) & 1;
          const uint32_t vr = kv_row(a.kv, wk.b, wk.g, tile * TT + r);
          if (vr == kInvalidRow) continue;
          const uint16_t* v = a.kv.v + (int64_t)vr * kHeadDim;
          for (int c = 0; c < 4; ++c) {
            float o[32];
            tmem_ld32(to + c * 32, o);
            tmem_wait_ld();
            tmem_loaded32(o);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x[8];
              unpack8(__ldg(reinterpret_cast<const uint4*>(v + c * 32) + e), x);
#pragma unroll
              for (int d = 0; d < 8; ++d)
                if (seen) o[8 * e + d] += p * x[d];
            }
            __syncwarp();
            tmem_st32(to + c * 32, o);
          }
          tmem_wait_st();
        }
        tc_fence_before_sync();
      };
      for (int i = 0; i < steps; ++i) {
        const int at = dual ? i : 2 * i + s, tile = wk.k0 + at;
        const uint32_t phase = (done + i) & 1, num = tiles_done + at;
        const bool special = (tile + 1) * TT > sq.base;
        tree_wait_warp(&ctl->s_full[s], phase, ctl, a.status);
        tc_fence_after_sync();
        if (warp_live) {
          float x[TT];
#pragma unroll
          for (int c = 0; c < TT / 32; ++c) tmem_ld32(tp + c * 32, x + 32 * c);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < TT / 32; ++c) tmem_loaded32(x + 32 * c);
          const volatile uint32_t* bad = ctl->bad[num & 15];
          uint32_t bw[TT / 32], any_bad = 0;
#pragma unroll
          for (int w = 0; w < TT / 32; ++w) any_bad |= bw[w] = bad[w];
          if (special || any_bad) {
#pragma unroll
            for (int w = 0; w < TT / 32; ++w) {
              vis[w] = valid ? tree_visible(a, sq, j, tile * TT + 32 * w) & ~bw[w] : 0u;
#pragma unroll
              for (int c = 0; c < 32; ++c) x[32 * w + c] = vis[w] >> c & 1 ? x[32 * w + c] : -INFINITY;
            }
          }
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < TT; ++c) mx4[c & 3] = fmaxf(mx4[c & 3], x[c]);
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * scale;
          if (i == 0) {
            m = mx;
          } else {
            const bool grow = mx > m + 8.f;
            if (__any_sync(0xFFFFFFFFu, grow)) {
              const float f = grow ? fast_exp2(m - mx) : 1.f;
              if (grow) m = mx;
              l *= f;
              tree_wait_warp(&ctl->o_done[s], phase ^ 1, ctl, a.status);
              tc_fence_after_sync();
              for (int c = 0; c < 4; ++c) {
                float o[32];
                tmem_ld32(to + c * 32, o);
                tmem_wait_ld();
                tmem_loaded32(o);
#pragma unroll
                for (int d = 0; d < 32; ++d) o[d] *= f;
                tmem_st32(to + c * 32, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;   // nothing seen yet: weights 0
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < TT / 32; ++c) {
            float* p = x + 32 * c;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              p[e] = fast_exp2(fmaf(p[e], scale, -ref));
              l4[e & 3] += p[e];
            }
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
              tmem_st16(tp + part * (TT / 2) + 16 * c, w);
            }
          }
          l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tmem_wait_st();
        }
        if (special) {
          // this tile's V in shared memory: rows behind the sequence and drafts' rows that are not
          // finite become zeros
          const uint32_t n = 2 * num + 1, slot = n % NS;
          unsigned char* vt = ring + (size_t)slot * SH::kSlotBytes;
          const int threads = dual ? 256 : 128, id = dual ? tid : row, bar = dual ? 1 : 2 + s;
          uint32_t* found = ctl->nf[dual ? 0 : s];
          tree_wait_warp(&ctl->full[slot], (n / NS) & 1, ctl, a.status);
          named_sync(bar, threads);
          if (id < 4) found[id] = 0;
          named_sync(bar, threads);
          for (int e = id; e < TT * 16; e += threads) {
            const int r = e >> 4, ch = e & 15, t = tile * TT + r;
            if (t < sq.base) continue;
            uint4* p = reinterpret_cast<uint4*>(vt + (ch >> 3) * (TT * 128) + sw128(r, ch & 7));
            if (t >= sq.len) {
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
          uint32_t any = 0;
#pragma unroll
          for (int w = 0; w < 4; ++w) any |= nf[w] = found[w];
          if (any) {
            for (int e = id; e < TT * 16; e += threads) {
              const int r = e >> 4, ch = e & 15;
              if (found[r >> 5] >> (r & 31) & 1)
                *reinterpret_cast<uint4*>(vt + (ch >> 3) * (TT * 128) + sw128(r, ch & 7)) = make_uint4(0, 0, 0, 0);
            }
          }
          asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
          if (dual) named_sync(bar, threads);   // the other stream's products read these rows too
        }
        tc_fence_before_sync();
        mbar_arrive(&ctl->p_ready[s]);
        if (special) {
          add_nonfinite(tile, phase);
          if (i + 1 < steps) mbar_arrive(&ctl->fixed[s]);
        }
      }
      if (steps > 0) tree_wait_warp(&ctl->o_done[s], (done + steps - 1) & 1, ctl, a.status);
      done += steps;
      tiles_done += ntile;

      // ---- the segment's state: O / l where the unit is whole, else a partial state
      float w0 = 1.f, w1 = 0.f;
      bool two = false;
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
  }
  __syncthreads();
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Merge of the partial states of units cut over several CTAs, in the order of the shares.  One block
// per 32 lists of a (sequence, kv head); a lane per list, so that the states' rows are read whole,
// and four dims of it at a time.
constexpr int kTgThreads = 256;

template <int QP, int PP>
__global__ void __launch_bounds__(kTgThreads) tree_merge_kernel(const __grid_constant__ TreeArgs a, int groups) {
  using SH = TreeShape<QP, PP>;
  const int rg = blockIdx.x % groups, g = (blockIdx.x / groups) % a.kv.hkv, b = blockIdx.x / groups / a.kv.hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.qv.hq / a.kv.hkv;
  const TreeSeq sq = tree_seq<SH>(a, b, G, false);
  const int lists = sq.n * G;
  pdl_wait();
  if (rg * 32 >= lists) return;
  const int64_t total = a.line[0], C = min((int64_t)a.ctas, total);
  const int mt = rg * 32 / SH::kRows;
  const int64_t u0 = a.line[1 + b] + ((int64_t)g * sq.mtiles + mt) * sq.tiles;
  const int c0 = tree_owner(u0, total, C), c1 = tree_owner(u0 + sq.tiles - 1, total, C);
  if (c0 == c1) return;   // written directly
  const int list = rg * 32 + lane, prow = list - mt * SH::kRows;
  if (list >= lists) return;
  auto slot = [&](int c) { return 2 * (int64_t)c + (c == c0 ? 1 : 0); };
  // the first share of the unit starts at its first tile: its state is in the odd slot
  float m = -INFINITY;
  for (int c = c0; c <= c1; ++c) m = fmaxf(m, __ldcg(&a.part_ml[slot(c) * a.part_rows + prow].x));
  float l = 0.f, o[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
#pragma unroll 4
  for (int c = c0; c <= c1; ++c) {
    const int64_t sl = slot(c);
    const float2 ml = __ldcg(a.part_ml + sl * a.part_rows + prow);
    const float w = ml.x == m ? 1.f : fast_exp2(ml.x - m);
    if (ml.x == -INFINITY) continue;   // nothing seen in this share
    l += w * ml.y;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = __ldcg(a.part_acc + (sl * 32 + warp + 8 * i) * a.part_rows + prow);
      o[i][0] += w * x.x;
      o[i][1] += w * x.y;
      o[i][2] += w * x.z;
      o[i][3] += w * x.w;
    }
  }
  const int j = list / G;
  const int64_t lst = (int64_t)(sq.t0 + j) * a.qv.hq + g * G + (list - j * G);
  const float norm = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = lst * 32 + warp + 8 * i;
    if (a.out_f32)
      static_cast<float4*>(a.out)[at] = make_float4(o[i][0] * norm, o[i][1] * norm, o[i][2] * norm, o[i][3] * norm);
    else
      static_cast<uint2*>(a.out)[at] =
          make_uint2(cvt_bf16x2(o[i][0] * norm, o[i][1] * norm), cvt_bf16x2(o[i][2] * norm, o[i][3] * norm));
  }
  if (warp == 0 && a.lse != nullptr) a.lse[lst] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
}

struct TreeLayout {
  size_t line, ml, acc, total;
  int part_rows;
};
static TreeLayout tree_layout(const Shapes& sh, int ctas, bool q_f32) {
  TreeLayout l;
  const int64_t lists = (sh.group * sh.max_tokens + 31) / 32 * 32, rows = q_f32 ? 128 : 256;
  l.part_rows = (int)(lists < rows ? lists : rows);
  l.line = 0;
  l.ml = align256((size_t)(1 + sh.batch) * sizeof(int64_t));
  l.acc = l.ml + align256((size_t)2 * ctas * l.part_rows * sizeof(float2));
  l.total = l.acc + align256((size_t)2 * ctas * 32 * l.part_rows * sizeof(float4));
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
  return launch_dependent(tree_merge_kernel<QP, PP>, dim3((unsigned)(batch * a.kv.hkv * groups)), dim3(kTgThreads), 0,
                          stream, a, groups);
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
  return tree_layout(sh, current_sm_count(), queries->q_dtype == TSD_F32).total;
}

tsd_status tsd_tree_decode(const tsd_kv_cache* cache, const tsd_queries* queries, const uint32_t* mask, void* out,
                           int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, uint32_t* status,
                           tsd_stream_t stream) {
  TreeArgs a;
  Shapes sh;
  memset(&a, 0, sizeof(a));
  tsd_status st = check_inputs(cache, queries, &a.kv, &a.qv, &sh);
  if (st != TSD_OK) return st;
  if (out == nullptr || ws == nullptr || !queries->causal) return TSD_ERR_INVALID_ARGUMENT;
  if (((uintptr_t)out & 15) || ((uintptr_t)ws & 255)) return TSD_ERR_INVALID_ARGUMENT;
  if (out_dtype != TSD_BF16 && out_dtype != TSD_F32) return TSD_ERR_UNSUPPORTED;
  if (sh.max_tokens > kMaxTree) return TSD_ERR_UNSUPPORTED;
  a.ctas = current_sm_count();
  const TreeLayout l = tree_layout(sh, a.ctas, a.qv.q_f32);
  if (ws_bytes < l.total) return TSD_ERR_WORKSPACE_TOO_SMALL;
  const int64_t groups = (sh.group * sh.max_tokens + 31) / 32;
  if (sh.batch * sh.hkv * groups > 0x7fffffffLL) return TSD_ERR_UNSUPPORTED;
  a.mask = mask;
  a.words = (int)(sh.max_tokens + 31) / 32;
  a.part_rows = l.part_rows;
  a.out = out;
  a.out_f32 = out_dtype == TSD_F32;
  a.lse = lse;
  a.status = status;
  char* w = static_cast<char*>(ws);
  a.line = reinterpret_cast<int64_t*>(w + l.line);
  a.part_ml = reinterpret_cast<float2*>(w + l.ml);
  a.part_acc = reinterpret_cast<float4*>(w + l.acc);
  KvMaps maps;
  const int tt = a.qv.q_f32 || a.out_f32 ? 64 : 128;
  st = make_kv_maps(cache, &maps, tt, true);
  if (st != TSD_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (a.qv.q_f32) e = a.out_f32 ? launch_tree<3, 3>(a, maps, sh.batch, (int)groups, s) : launch_tree<3, 1>(a, maps, sh.batch, (int)groups, s);
  else e = a.out_f32 ? launch_tree<1, 3>(a, maps, sh.batch, (int)groups, s) : launch_tree<1, 1>(a, maps, sh.batch, (int)groups, s);
  return cuda_status(e);
}

}  // extern "C"
