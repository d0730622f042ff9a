// Page management of the paged cache: sequences that share pages, pages taken (with copy on
// write) and released, accepted drafts moved to the front.
//
// State: the page table [batch][max_pages], the lengths and refs[page] = table entries that hold the
// page; a page is free when refs is 0.  There is no free list to keep consistent: the free pages
// are counted from refs on every call (4 B a page: 4 MB for a million pages), which also makes
// the outcome -- lowest free numbers first -- independent of the order in which anything ran.
#include <string.h>

#include "tsd_host.h"

namespace tsd {

constexpr int kMaxLayers = 128;

struct Layers {   // passed by value to the kernels
  void* k[kMaxLayers];
  void* v[kMaxLayers];
};

struct Pool {
  int32_t* table;
  int32_t* lens;
  int32_t* refs;
  int64_t num_pages;
  int32_t batch, max_pages, page_shift, max_seq_len;
};

__device__ __forceinline__ int pages_of(int len, int shift) { return (int)(((int64_t)len + (1 << shift) - 1) >> shift); }

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------
// One block per pair.  A pair reads only its src's row and length, and no src is any pair's dst,
// so nothing read is written in the same call.  4 us for 192 pairs with the launch, which is what bounds it.
__global__ void __launch_bounds__(256) cache_fork_kernel(Pool p, int num_pairs, const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst, uint32_t* status) {
  const int i = blockIdx.x;
  const int s = __ldg(src + i), d = __ldg(dst + i);
  bool bad = s < 0 || s >= p.batch || d < 0 || d >= p.batch || s == d;
  for (int j = threadIdx.x; j < num_pairs; j += 256) {
    const int dj = __ldg(dst + j);
    if (dj == s || (j < i && dj == d)) bad = true;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) flag_optional(status, TSD_DEV_BAD_SEQ);
    return;
  }
  const int len = p.lens[s];
  bad = len < 0 || len > p.max_seq_len || p.lens[d] != 0;
  if (__syncthreads_or(bad)) {   // also: every thread has read lens[d] before it is written
    if (threadIdx.x == 0) flag_optional(status, TSD_DEV_BAD_SEQ);
    return;
  }
  const int n = pages_of(len, p.page_shift);
  const int32_t* from = p.table + (int64_t)s * p.max_pages;
  int32_t* to = p.table + (int64_t)d * p.max_pages;
  for (int c = threadIdx.x; c < p.max_pages; c += 256) {
    int32_t page = -1;
    if (c < n) {
      page = from[c];
      if (page < 0 || (int64_t)page >= p.num_pages) flag_optional(status, TSD_DEV_BAD_PAGE);
      else atomicAdd(p.refs + page, 1);
    }
    to[c] = page;
  }
  if (threadIdx.x == 0) p.lens[d] = len;
}

// ---------------------------------------------------------------------------
// Resize
// ---------------------------------------------------------------------------
// One cluster of kRzCtas CTAs does the bookkeeping in three steps with cluster barriers between, so
// that a call is one launch (and one more for the copies) with no grid-wide wait:
//   1  CTA 0 finds what every sequence wants and the running sums of that; every warp of the others
//      counts the free pages of its slice of refs, keeping the first kRzKept groups' as bits;
//   2  the warps whose first free page has a rank below the total wanted list their free pages;
//   3  a warp per sequence hands out the listed pages, updates its row and the counts.
// Sequences are served from the list in order, so the outcome does not depend on timing.  Where a table names
// a page that refs has as free, that page may be handed out in the same call; so where a call both
// releases and takes, all releases (which leave such a page alone) come first, behind one more cluster barrier.  A call
// is a chain of dependent loads (length, page, count; listed page, row) more than it is bytes: for 256
// sequences over a pool with 70000 free pages, whose bytes take 0.1 us, 8 us where all grow or all shrink by a page or
// two and 16 where some end with hundreds of pages and others grow (2 of it the barrier between).
constexpr int kRzCtas = 8;
constexpr int kRzThreads = 1024;
constexpr int kRzWarps = kRzCtas * kRzThreads / 32;
constexpr int kRzCounters = (kRzCtas - 1) * kRzThreads / 32;   // warps that count
constexpr int kRzRelease = 8;
constexpr int kRzKept = 8;                                     // groups of 128 pages: 4 bits a lane each

struct ResizeArgs {
  Pool p;
  const int32_t* new_lens;
  int32_t* counts;   // [kRzCounters] free pages of each warp's slice
  int32_t* total;    // [2] pages wanted in all, whether any are released
  int2* want;        // [batch] (first rank, pages wanted | copy flag << 31); -1 first: leave alone
  int2* pairs;       // [batch] (from, to) page to copy, (-1, -1) for none
  int32_t* list;     // [num_pages] the free pages of ranks below the total
  uint32_t* status;
  int32_t aligned;   // refs is 16-byte aligned
};

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();   // lanes may come from different ends of a loop, and the barrier takes whole warps
  asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}

__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xFFFFFFFFu, v); }

__device__ __forceinline__ int warp_exclusive(int v, int lane) {
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  return x - v;
}

// Which of pages at .. at + 3 are free, as bits.
__device__ __forceinline__ uint32_t free_bits(const Pool& p, int64_t at, bool aligned) {
  uint32_t bits = 0;
  if (aligned && at + 4 <= p.num_pages) {
    const int4 r = *reinterpret_cast<const int4*>(p.refs + at);
    return (uint32_t)(r.x == 0) | (uint32_t)(r.y == 0) << 1 | (uint32_t)(r.z == 0) << 2 | (uint32_t)(r.w == 0) << 3;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (at + e < p.num_pages && p.refs[at + e] == 0) bits |= 1u << e;
  return bits;
}

__global__ void __cluster_dims__(kRzCtas, 1, 1) __launch_bounds__(kRzThreads) cache_resize_kernel(ResizeArgs a) {
  __shared__ int tmp[kRzThreads / 32 + 1];
  const Pool& p = a.p;
  const int tid = threadIdx.x, lane = tid & 31;
  const int gw = blockIdx.x * (kRzThreads / 32) + (tid >> 5);
  const int cw = gw - kRzThreads / 32;   // this warp among those that count
  pdl_launch_dependents();
  // ---- 1: slices of whole 128-page groups, lane l taking pages 4l .. 4l + 3 of a group
  int64_t g0 = 0, g1 = 0;
  uint32_t kept = 0;
  if (blockIdx.x == 0) {
    int running = 0, shrinks = 0;
    for (int b0 = 0; b0 < p.batch; b0 += kRzThreads) {
      const int b = b0 + tid;
      int need = 0, cow = 0;
      bool ok = false;
      if (b < p.batch) {
        const int old = p.lens[b], now = a.new_lens[b];
        ok = old >= 0 && old <= p.max_seq_len && now >= 0 && now <= p.max_seq_len;
        if (!ok) {
          flag_optional(a.status, TSD_DEV_BAD_SEQ);
        } else if (now > old) {
          const int have = pages_of(old, p.page_shift);
          need = pages_of(now, p.page_shift) - have;
          if (old & ((1 << p.page_shift) - 1)) {
            const int32_t page = p.table[(int64_t)b * p.max_pages + have - 1];
            if (page < 0 || (int64_t)page >= p.num_pages) flag_optional(a.status, TSD_DEV_BAD_PAGE);
            else cow = p.refs[page] > 1;
          }
        } else {
          shrinks |= now < old;
        }
      }
      int sum;
      const int first = running + block_exclusive_scan<kRzThreads>(need + cow, tmp, &sum);
      running += sum;
      if (b < p.batch) a.want[b] = make_int2(ok ? first : -1, (need + cow) | (cow << 31));
    }
    shrinks = __syncthreads_or(shrinks);
    if (tid == 0) {
      a.total[0] = running;
      a.total[1] = shrinks;
    }
  } else {
    const int64_t groups = (p.num_pages + 127) / 128;
    g0 = groups * cw / kRzCounters;
    g1 = groups * (cw + 1) / kRzCounters;
    int free_cnt = 0;
#pragma unroll
    for (int k = 0; k < kRzKept; ++k)
      if (g0 + k < g1) kept |= free_bits(p, (g0 + k) * 128 + 4 * lane, a.aligned) << (4 * k);
    free_cnt = __popc(kept);
#pragma unroll 4
    for (int64_t g = g0 + kRzKept; g < g1; ++g) free_cnt += __popc(free_bits(p, g * 128 + 4 * lane, a.aligned));
    free_cnt = warp_sum(free_cnt);
    if (lane == 0) a.counts[cw] = free_cnt;
  }
  cluster_sync();
  // ---- 2
  const int total = a.total[0];
  const bool apart = total > 0 && a.total[1];   // releases first
  int2 w = gw < p.batch ? a.want[gw] : make_int2(-1, 0);   // step 3's first sequence
  int old = gw < p.batch ? p.lens[gw] : 0, now = gw < p.batch ? a.new_lens[gw] : 0;
  int before = 0, free_all = 0;
#pragma unroll
  for (int i = lane; i < kRzCounters; i += 32) {
    const int c = a.counts[i];
    free_all += c;
    if (i < cw) before += c;
  }
  before = warp_sum(before);
  free_all = warp_sum(free_all);
  for (int64_t g = g0; g < g1 && before < total; ++g) {
    const int64_t at = g * 128 + 4 * lane;
    const uint32_t is_free = g - g0 < kRzKept ? kept >> (4 * (int)(g - g0)) & 15u : free_bits(p, at, a.aligned);
    const int mine = __popc(is_free);
    int rank = before + warp_exclusive(mine, lane);
    before += warp_sum(mine);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (is_free >> e & 1) {
        if (rank < total) a.list[rank] = (int32_t)(at + e);
        ++rank;
      }
  }
  cluster_sync();
  // ---- 3
#pragma unroll 1
  for (int pass = apart ? 0 : 1; pass < 2; ++pass) {
    if (pass == 1 && apart) cluster_sync();
    for (int b = gw; b < p.batch; b += kRzWarps) {
      if (b != gw || (apart && pass == 1 && p.batch > kRzWarps)) {   // else they are at hand
        w = a.want[b];
        old = p.lens[b];
        now = a.new_lens[b];
      }
      if (apart && (now < old) != (pass == 0)) continue;   // done sequences come by again with their new length
      int2 pair = make_int2(-1, -1);
      if (w.x >= 0) {
        const int need = w.y & 0x7fffffff, cow = (int)((uint32_t)w.y >> 31);
        const int have = pages_of(old, p.page_shift), end = pages_of(now, p.page_shift);
        int32_t* row = p.table + (int64_t)b * p.max_pages;
        if (need > 0 && (int64_t)w.x + need > free_all) {
          if (lane == 0) flag_optional(a.status, TSD_DEV_NO_PAGES);
        } else {
          if (cow) {
            pair = make_int2(row[have - 1], a.list[w.x]);
            __syncwarp();
            if (lane == 0) {
              row[have - 1] = pair.y;
              p.refs[pair.y] = 1;
              if (atomicSub(p.refs + pair.x, 1) < 1) {   // more tables name it than refs counts
                atomicAdd(p.refs + pair.x, 1);
                flag_optional(a.status, TSD_DEV_BAD_PAGE);
              }
            }
          }
          for (int i = have + lane; i < end; i += 32) {
            const int32_t page = a.list[w.x + cow + i - have];
            row[i] = page;
            p.refs[page] = 1;
          }
          // eight rounds' loads, then their counts, at once: an ended sequence gives back hundreds of pages
          for (int i0 = end + lane; i0 < have; i0 += 32 * kRzRelease) {
            int32_t page[kRzRelease], held[kRzRelease];
#pragma unroll
            for (int e = 0; e < kRzRelease; ++e) {
              page[e] = i0 + 32 * e < have ? row[i0 + 32 * e] : 0;
              held[e] = 1;
            }
#pragma unroll
            for (int e = 0; e < kRzRelease; ++e) {
              if (i0 + 32 * e >= have) continue;
              row[i0 + 32 * e] = -1;
              if (page[e] < 0 || (int64_t)page[e] >= p.num_pages) flag_optional(a.status, TSD_DEV_BAD_PAGE);
              else held[e] = atomicSub(p.refs + page[e], 1);
            }
#pragma unroll
            for (int e = 0; e < kRzRelease; ++e) {
              if (held[e] < 1) {   // it was free already
                atomicAdd(p.refs + page[e], 1);
                flag_optional(a.status, TSD_DEV_BAD_PAGE);
              }
            }
          }
          __syncwarp();
          if (lane == 0) p.lens[b] = now;
        }
      }
      if (lane == 0) a.pairs[b] = pair;
    }
  }
}

// Copies pairs[b].x to pairs[b].y in every layer's K and V, page_chunks 16-byte chunks a page.
// Grid (pieces of a page's copies over all layers, batch); a block copies kCpChunks chunks per
// thread, loads first.  Bound by HBM: 256 pages x 16 layers, 537 MB, in 72 us (sources that several
// sequences share stay in L2).
constexpr int kCpThreads = 256;
constexpr int kCpChunks = 4;

__global__ void __launch_bounds__(kCpThreads) page_copy_kernel(const __grid_constant__ Layers layers, int num_layers,
                                                               const int2* pairs, int64_t page_chunks) {
  pdl_wait();
  const int2 pr = pairs[blockIdx.y];
  if (pr.x < 0) return;
  const int64_t all = page_chunks * 2 * num_layers;
  const int64_t at0 = (int64_t)blockIdx.x * (kCpThreads * kCpChunks) + threadIdx.x;
  uint4 x[kCpChunks];
#pragma unroll
  for (int i = 0; i < kCpChunks; ++i) {
    const int64_t at = at0 + i * kCpThreads;
    if (at < all) {
      const int64_t which = at / page_chunks, off = at - which * page_chunks;
      const void* base = (which & 1) ? layers.v[which >> 1] : layers.k[which >> 1];
      x[i] = __ldcs(static_cast<const uint4*>(base) + (int64_t)pr.x * page_chunks + off);
    }
  }
#pragma unroll
  for (int i = 0; i < kCpChunks; ++i) {
    const int64_t at = at0 + i * kCpThreads;
    if (at < all) {
      const int64_t which = at / page_chunks, off = at - which * page_chunks;
      void* base = (which & 1) ? layers.v[which >> 1] : layers.k[which >> 1];
      static_cast<uint4*>(base)[(int64_t)pr.y * page_chunks + off] = x[i];
    }
  }
}

// ---------------------------------------------------------------------------
// Compact
// ---------------------------------------------------------------------------
// Rows move towards the front of the drafts, in place.  A group of 16 threads owns one stream --
// one (layer, kv head, K or V) of a sequence -- and each of its threads one 16-byte column of every
// row, which it moves in the order of the list, kCmBatch loads before their stores.  A row's new
// place i is at most its old place keep[i], which is below every later keep: no store reaches a
// row that is still to be read.  Nothing has to be staged and streams need not wait for one another.
// Bound by the dependent loads of a stream (list, page, row): 4.2 us for 8 sequences of one layer, 9.1
// for 64 sequences x 16 layers, whose bytes take 3.9.
constexpr int kCmThreads = 256;
constexpr int kCmStreams = kCmThreads / 16;
constexpr int kCmBatch = 4;
constexpr int kCmPart = 256;   // list entries resolved to rows at a time

struct CompactArgs {
  KvView kv;
  const int32_t* q_indptr;
  int32_t num_tokens, max_tokens, num_layers, k_max;
  const int32_t* keep;
  const int32_t* refs;
  int32_t* out_lens;
  uint32_t* status;
};

// Cache row of position r of sequence b (kv head 0), or -1; *page its page (paged).
__device__ __forceinline__ int64_t position_row(const KvView& kv, int b, int r, int32_t* page) {
  if (kv.page_table == nullptr) {
    *page = -1;
    return (int64_t)b * kv.hkv * kv.max_seq_len + r;
  }
  *page = __ldg(kv.page_table + (int64_t)b * kv.max_pages + (r >> kv.page_shift));
  if (*page < 0 || (int64_t)*page >= kv.num_pages) return -1;
  return (((int64_t)*page * kv.hkv) << kv.page_shift) | (r & ((1 << kv.page_shift) - 1));
}

__global__ void __launch_bounds__(kCmThreads, 7) cache_compact_kernel(const __grid_constant__ CompactArgs a,
                                                                   const __grid_constant__ Layers layers) {
  __shared__ int64_t s_src[kCmPart], s_dst[kCmPart];
  __shared__ int s_cnt;
  __shared__ uint32_t s_bad;
  const int b = blockIdx.y, tid = threadIdx.x;
  const bool lead = blockIdx.x == 0 && tid == 0;
  if (tid == 0) {
    s_cnt = 0;
    s_bad = 0;
  }
  __syncthreads();
  const int32_t* keep = a.keep + (int64_t)b * a.k_max;
  // the first part of the list does not wait for the descriptor
  int r = tid < a.k_max ? __ldg(keep + tid) : -1, prev = tid > 0 && tid < a.k_max ? __ldg(keep + tid - 1) : -1;
  const int len = __ldg(a.kv.seq_lens + b);
  const int t0 = a.q_indptr != nullptr ? __ldg(a.q_indptr + b) : b;
  const int t1 = a.q_indptr != nullptr ? __ldg(a.q_indptr + b + 1) : b + 1;
  const int n = t1 - t0, base = len - n;
  if (len < 0 || len > a.kv.max_seq_len || t0 < 0 || n < 0 || t1 > a.num_tokens || n > a.max_tokens || base < 0) {
    if (lead) {
      flag_optional(a.status, TSD_DEV_BAD_SEQ);
      a.out_lens[b] = len;
    }
    return;
  }
  // every block checks the whole list, so that all streams of a sequence move or none
  uint32_t bad = 0;
  int cnt = 0;
  for (int i = tid; i < a.k_max; i += kCmThreads) {
    if (i != tid) {
      r = __ldg(keep + i);
      prev = __ldg(keep + i - 1);
    }
    int64_t from = -1, to = -1;
    if (r < 0) {
      if (r != -1) bad |= TSD_DEV_BAD_INDEX;
    } else {
      ++cnt;
      if (r >= n || r <= prev || (i > 0 && prev < 0)) {
        bad |= TSD_DEV_BAD_INDEX;
      } else if (r != i) {   // else it stays where it is
        int32_t ps, pd;
        from = position_row(a.kv, b, base + r, &ps);
        to = position_row(a.kv, b, base + i, &pd);
        if (from < 0 || to < 0) bad |= TSD_DEV_BAD_PAGE;
        else if (a.refs != nullptr && pd >= 0 && __ldg(a.refs + pd) > 1) bad |= TSD_DEV_SHARED_PAGE;
      }
    }
    if (i < kCmPart) {   // kCmPart = kCmThreads: the first part of the list, resolved
      s_src[i] = from;
      s_dst[i] = to;
    }
  }
  if (cnt) atomicAdd(&s_cnt, cnt);
  if (bad) atomicOr(&s_bad, bad);
  __syncthreads();
  if (s_bad) {
    if (lead) {
      flag_optional(a.status, s_bad);
      a.out_lens[b] = len;
    }
    return;
  }
  if (lead) a.out_lens[b] = base + s_cnt;
  const int total = s_cnt;
  const int stream = blockIdx.x * kCmStreams + (tid >> 4), col = tid & 15;
  const int per_layer = 2 * a.kv.hkv;
  const bool live = stream < a.num_layers * per_layer;
  const int layer = live ? stream / per_layer : 0;
  const int which = (live ? stream % per_layer : 0) / a.kv.hkv, g = (live ? stream : 0) % a.kv.hkv;
  const int64_t head_rows = a.kv.page_table == nullptr ? a.kv.max_seq_len : (int64_t)1 << a.kv.page_shift;
  uint4* rows = static_cast<uint4*>(which ? layers.v[layer] : layers.k[layer]) + g * head_rows * 16 + col;
  for (int i0 = 0; i0 < total; i0 += kCmPart) {
    const int m = min(kCmPart, total - i0);
    if (i0 > 0) {
      __syncthreads();
      for (int i = tid; i < m; i += kCmThreads) {
        const int kr = __ldg(keep + i0 + i);
        int32_t page;
        s_src[i] = kr == i0 + i ? -1 : position_row(a.kv, b, base + kr, &page);
        s_dst[i] = position_row(a.kv, b, base + i0 + i, &page);
      }
      __syncthreads();
    }
    if (!live) continue;
    for (int i = 0; i < m; i += kCmBatch) {
      uint4 x[kCmBatch];
#pragma unroll
      for (int e = 0; e < kCmBatch; ++e)
        if (i + e < m && s_src[i + e] >= 0) x[e] = rows[s_src[i + e] * 16];
#pragma unroll
      for (int e = 0; e < kCmBatch; ++e)
        if (i + e < m && s_src[i + e] >= 0) rows[s_dst[i + e] * 16] = x[e];
    }
  }
}

static tsd_status fill_layers(int32_t num_layers, const tsd_layer* layers, Layers* out) {
  if (num_layers < 1 || layers == nullptr) return TSD_ERR_INVALID_ARGUMENT;
  if (num_layers > kMaxLayers) return TSD_ERR_UNSUPPORTED;
  memset(out, 0, sizeof(*out));
  for (int i = 0; i < num_layers; ++i) {
    if (layers[i].k == nullptr || layers[i].v == nullptr) return TSD_ERR_INVALID_ARGUMENT;
    if (((uintptr_t)layers[i].k | (uintptr_t)layers[i].v) & 15) return TSD_ERR_INVALID_ARGUMENT;
    out->k[i] = layers[i].k;
    out->v[i] = layers[i].v;
  }
  return TSD_OK;
}

static tsd_status fill_pool(const tsd_kv_cache* cache, int32_t* refs, Pool* p, Shapes* sh) {
  KvView kv;
  const tsd_status st = check_cache_only(cache, &kv, sh);
  if (st != TSD_OK) return st;
  if (cache->layout != TSD_LAYOUT_PAGED) return TSD_ERR_UNSUPPORTED;
  if (refs == nullptr) return TSD_ERR_INVALID_ARGUMENT;
  p->table = const_cast<int32_t*>(cache->page_table);
  p->lens = const_cast<int32_t*>(cache->seq_lens);
  p->refs = refs;
  p->num_pages = kv.num_pages;
  p->batch = kv.batch;
  p->max_pages = kv.max_pages;
  p->page_shift = kv.page_shift;
  p->max_seq_len = kv.max_seq_len;
  return TSD_OK;
}

struct ResizeLayout {
  size_t counts, total_off, want, pairs, list, total;
};
static ResizeLayout resize_layout(int64_t batch, int64_t num_pages) {
  ResizeLayout l;
  l.counts = 0;
  l.total_off = kRzCounters * sizeof(int32_t);
  l.want = align256(l.total_off + 2 * sizeof(int32_t));
  l.pairs = l.want + align256((size_t)batch * sizeof(int2));
  l.list = l.pairs + align256((size_t)batch * sizeof(int2));
  l.total = l.list + align256((size_t)num_pages * sizeof(int32_t));
  return l;
}

}  // namespace tsd

using namespace tsd;

extern "C" {

tsd_status tsd_cache_fork(const tsd_kv_cache* cache, int32_t* refs, int32_t num_pairs, const int32_t* src,
                          const int32_t* dst, uint32_t* status, tsd_stream_t stream) {
  Pool p;
  Shapes sh;
  const tsd_status st = fill_pool(cache, refs, &p, &sh);
  if (st != TSD_OK) return st;
  if (num_pairs < 0 || (num_pairs > 0 && (src == nullptr || dst == nullptr))) return TSD_ERR_INVALID_ARGUMENT;
  if (num_pairs == 0) return TSD_OK;
  cache_fork_kernel<<<num_pairs, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p, num_pairs, src, dst, status);
  return cuda_status(cudaGetLastError());
}

size_t tsd_cache_resize_workspace_size(const tsd_kv_cache* cache) {
  if (cache == nullptr || cache->layout != TSD_LAYOUT_PAGED || cache->batch < 1 || cache->num_pages < 1 ||
      cache->num_pages > 0x7fffffffLL)
    return 0;
  return resize_layout(cache->batch, cache->num_pages).total;
}

tsd_status tsd_cache_resize(const tsd_kv_cache* cache, int32_t num_layers, const tsd_layer* layers, int32_t* refs,
                            const int32_t* new_lens, void* ws, size_t ws_bytes, uint32_t* status,
                            tsd_stream_t stream) {
  ResizeArgs a;
  Layers ls;
  Shapes sh;
  memset(&a, 0, sizeof(a));
  tsd_status st = fill_pool(cache, refs, &a.p, &sh);
  if (st == TSD_OK) st = fill_layers(num_layers, layers, &ls);
  if (st != TSD_OK) return st;
  if (new_lens == nullptr || ws == nullptr || ((uintptr_t)ws & 255) != 0) return TSD_ERR_INVALID_ARGUMENT;
  if (a.p.num_pages > 0x7fffffffLL || a.p.batch > 65535) return TSD_ERR_UNSUPPORTED;
  // the pages that all sequences want, a copy each among them, are summed in 32 bits
  if ((int64_t)a.p.batch * ((int64_t)a.p.max_pages + 1) > 0x7fffffffLL) return TSD_ERR_UNSUPPORTED;
  const ResizeLayout l = resize_layout(a.p.batch, a.p.num_pages);
  if (ws_bytes < l.total) return TSD_ERR_WORKSPACE_TOO_SMALL;
  char* w = static_cast<char*>(ws);
  a.new_lens = new_lens;
  a.counts = reinterpret_cast<int32_t*>(w + l.counts);
  a.total = reinterpret_cast<int32_t*>(w + l.total_off);
  a.want = reinterpret_cast<int2*>(w + l.want);
  a.pairs = reinterpret_cast<int2*>(w + l.pairs);
  a.list = reinterpret_cast<int32_t*>(w + l.list);
  a.status = status;
  a.aligned = ((uintptr_t)refs & 15) == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cache_resize_kernel<<<kRzCtas, kRzThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return TSD_ERR_CUDA;
  const int64_t page_chunks = (int64_t)cache->num_kv_heads * cache->page_size * 16;
  const int64_t pieces = (page_chunks * 2 * num_layers + kCpThreads * kCpChunks - 1) / (kCpThreads * kCpChunks);
  if (pieces > 0x7fffffffLL) return TSD_ERR_UNSUPPORTED;
  return cuda_status(launch_dependent(page_copy_kernel, dim3((unsigned)pieces, (unsigned)a.p.batch), dim3(kCpThreads), 0,
                                      s, ls, (int)num_layers, (const int2*)a.pairs, page_chunks));
}

tsd_status tsd_cache_compact(const tsd_kv_cache* cache, int32_t num_layers, const tsd_layer* layers,
                             const int32_t* q_indptr, int32_t num_tokens, int32_t max_tokens, const int32_t* keep,
                             int32_t k_max, const int32_t* refs, int32_t* out_lens, uint32_t* status,
                             tsd_stream_t stream) {
  CompactArgs a;
  Layers ls;
  Shapes sh;
  memset(&a, 0, sizeof(a));
  tsd_status st = check_cache_only(cache, &a.kv, &sh);
  if (st == TSD_OK) st = fill_layers(num_layers, layers, &ls);
  if (st != TSD_OK) return st;
  if (keep == nullptr || out_lens == nullptr || k_max < 1 || num_tokens < 0) return TSD_ERR_INVALID_ARGUMENT;
  if (q_indptr == nullptr) {
    if (num_tokens != cache->batch) return TSD_ERR_INVALID_ARGUMENT;
    max_tokens = 1;
  } else if (max_tokens < 0) {
    return TSD_ERR_INVALID_ARGUMENT;
  }
  if (cache->batch > 65535) return TSD_ERR_UNSUPPORTED;
  // blocks read seq_lens while others write out_lens
  if (out_lens < cache->seq_lens + cache->batch && cache->seq_lens < out_lens + cache->batch)
    return TSD_ERR_INVALID_ARGUMENT;
  a.q_indptr = q_indptr;
  a.num_tokens = num_tokens;
  a.max_tokens = max_tokens;
  a.num_layers = num_layers;
  a.k_max = k_max;
  a.keep = keep;
  a.refs = refs;
  a.out_lens = out_lens;
  a.status = status;
  const int64_t blocks = ((int64_t)num_layers * 2 * cache->num_kv_heads + kCmStreams - 1) / kCmStreams;
  cache_compact_kernel<<<dim3((unsigned)blocks, (unsigned)cache->batch), kCmThreads, 0,
                         reinterpret_cast<cudaStream_t>(stream)>>>(a, ls);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
