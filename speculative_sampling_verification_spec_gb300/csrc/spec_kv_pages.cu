// spec_kv_pages.cu -- the pages of the paged cache: argument checks, kernels and the
// C ABI entry points of include/spec_kv_pages.h.
//
// Holding and forking are one kernel, which walks the page table and the counts:
//
//   1. every entry of the table is brought up to date but for the pages that are
//      missing: releases count down, shared pages count up, and what is missing
//      becomes a bit;
//   2. once all counts are final, every page that is free becomes a bit;
//   3. the k-th missing entry (sequence by sequence, page by page) takes the k-th free
//      page: a count of the bits before it, and a search for the page.
//
// Between the steps everything has to be known everywhere, so the kernel is one
// thread-block cluster, whose barrier costs well under a microsecond where another
// launch costs one or two.  Its CTAs each have a stretch of the table and of the pool;
// the bits and how many come before each word of them stay in their shared memory,
// where the others search them: nothing is kept in a workspace, and the order of the
// atomic counts (whole numbers) changes nothing.
//
// Forking ends with a second kernel that copies what the last pages hold (384 pages, 50 MB
// read and written, in 12 us of the 22 that the call takes).
#include "kernel_table.h"
#include "spec_kv_common.cuh"
#include "spec_kv_pages.h"

#include <algorithm>
#include <atomic>

namespace {

using namespace spec_kv_detail;

constexpr int kMostCtas = 16, kPortableCtas = 8;  // of a cluster
// Words of bits up to which one CTA takes a call on alone: it has no other to wait for, but 15 fewer to share the work
// with (8 sequences, 3000 pages, 128 words: 4.0 us a call either way; 32 and 2800, 216 words: 6.6, by a cluster 4.2).
constexpr int kWordsAlone = 128;
// Words up to which CTAs have 256 threads, past it 1024: fewer make for quicker barriers (128 rows of 128 entries, 100 000
// pages, 3637 words: 5.1 us a call, 6.3 with 1024; a fork 10.1 and 11.3), more have more of a large table under way (300
// rows, 120 000 pages, 4950 words: 6.9 us with 256, 6.6 with 1024, a fork 12.3 and 11.8; 256 x 8194 entries: 33 and 23).
constexpr int kWordsFew = 4096;
constexpr int kAhead = 4;      // loads of counts of a lane under way at once

struct PagesArgs {
  int32_t* refs;
  int32_t* table;
  int64_t table_stride;
  int32_t* free_pages;
  int32_t* status;
  int32_t num_pages, log_page, B, max_pages;
  const int32_t* new_lens;
  int32_t T, window, sinks;
  int32_t* seq_lens;  // written by forks
  const int32_t* parents;
  int32_t vec, refs_vec;            // the table, the counts can be read four at a time
  int32_t row_words;                // words of bits of a row of the table (a whole number of stretches)
  int32_t need_words, free_words;   // of all rows; of the pool
  int32_t need_share, free_share;   // of a CTA
  uint64_t row_recip;               // 2^64 over the stretches of a row
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// all threads of the cluster; what they wrote is seen by all
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a word of another CTA's shared memory
__device__ __forceinline__ uint32_t load_of(uint32_t rank, const uint32_t* here) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(here)), v;
  asm volatile(
      "{\n\t.reg .b32 there;\n\tmapa.shared::cluster.u32 there, %1, %2;\n\tld.shared::cluster.u32 %0, [there];\n\t}"
      : "=r"(v)
      : "r"(at), "r"(rank));
  return v;
}

// Four neighbouring entries of a row, or counts of pages.
struct Four {
  int32_t x[4];
  __device__ __forceinline__ void load(const int32_t* row, int c, int columns, bool vec) {
    if (vec && c + 4 <= columns) {
      *reinterpret_cast<int4*>(x) = *reinterpret_cast<const int4*>(row + c);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = c + e < columns ? row[c + e] : -1;
    }
  }
  __device__ __forceinline__ void store(int32_t* row, const Four& old, int c, int columns) const {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (x[e] != old.x[e] && c + e < columns) row[c + e] = x[e];
  }
  // (atomics have been at the counts: not from the first-level cache)
  __device__ __forceinline__ void load_counts(const PagesArgs& a, int page) {
    if (a.refs_vec && page + 4 <= a.num_pages) {
      *reinterpret_cast<int4*>(x) = __ldcg(reinterpret_cast<const int4*>(a.refs + page));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = page + e < a.num_pages ? __ldcg(a.refs + page + e) : 1;
    }
  }
};

// The bits of eight neighbouring lanes, four each, side by side.
__device__ __forceinline__ uint32_t word_of(uint32_t bits) {
  uint32_t w = bits << (4 * (threadIdx.x & 7));
  w |= __shfl_xor_sync(kFull, w, 1);
  w |= __shfl_xor_sync(kFull, w, 2);
  w |= __shfl_xor_sync(kFull, w, 4);
  return w;
}

// What a row of the table becomes.
struct Row {
  int last;        // hold: columns from this on are empty; fork: the parent's tokens.  -1: nothing happens to it
  int keep, from;  // hold: columns below `keep` and from `from` on are needed
};

__device__ __forceinline__ Row hold_row(const PagesArgs& a, int b) {
  Row r;
  const int L = a.seq_lens[b], n = a.new_lens ? a.new_lens[b] : a.T;
  const int64_t end = static_cast<int64_t>(L) + n;
  const bool out = L < 0 || n < 0 || end > (static_cast<int64_t>(a.max_pages) << a.log_page);
  r.last = out ? -1 : static_cast<int>((end + (1 << a.log_page) - 1) >> a.log_page);
  r.keep = a.sinks > 0 ? ((a.sinks - 1) >> a.log_page) + 1 : 0;
  r.from = a.window > 0 && L >= a.window ? (L + 1 - a.window) >> a.log_page : 0;
  return r;
}

// A copy's parent; -1: the row stays, -2: it should not, but its parent cannot be one.
__device__ __forceinline__ int parent_of(const PagesArgs& a, int b, int* L) {
  const int p = a.parents[b];
  if (p == -1 || p == b) return -1;
  if (p < 0 || p >= a.B) return -2;
  const int pp = a.parents[p];
  *L = a.seq_lens[p];
  if ((pp != -1 && pp != p) || *L < 0 || *L > (static_cast<int64_t>(a.max_pages) << a.log_page)) return -2;
  return p;
}

// n of four bits, from the lowest on
__device__ __forceinline__ uint32_t first_of(int n) { return (1u << min(max(n, 0), 4)) - 1; }

// A warp's columns of a row: four a lane, N times.  Tables of up to 128 columns take N = 1, others 4, because a
// stretch costs about as many instructions however long it is.
template <bool FORK, int N>
struct Stretch {
  static constexpr int kWords = 4 * N;  // of bits
  int b, c;  // row; the lane's first column
  Row row;
  Four entry[N], source[FORK ? N : 1];  // source: of the parent's row
  __device__ __forceinline__ int column(int k) const { return c + k * 128; }
  __device__ __forceinline__ void load(const PagesArgs& a, int i) {
    const int of_row = a.row_words / kWords;
    b = of_row == 1 ? i : static_cast<int>(__umul64hi(i, a.row_recip));
    c = (i - b * of_row) * N * 128 + (threadIdx.x & 31) * 4;
    const int32_t* const at = a.table + b * a.table_stride;
    if constexpr (FORK) {
      int L = 0;
      const int p = parent_of(a, b, &L);
      row.last = p < 0 ? -1 : L;
      if (p == -2 && c == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
      if (p < 0) return;
#pragma unroll
      for (int k = 0; k < N; ++k) source[k].load(a.table + p * a.table_stride, column(k), a.max_pages, a.vec);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) entry[k].load(at, column(k), a.max_pages, a.vec);
    if constexpr (!FORK) {
      row = hold_row(a, b);
      if (row.last < 0 && c == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
    }
  }
  // hold: whether this lane has something to do among the 128 columns of the k-th time.  Most are all needed and there,
  // or neither.
  __device__ __forceinline__ bool some(const PagesArgs& a, int k) const {
    const int c0 = column(k) - (threadIdx.x & 31) * 4, c1 = c0 + 128;
    const int32_t* const x = entry[k].x;
    if (c0 >= row.last || (c0 >= row.keep && c1 <= row.from)) return (x[0] & x[1] & x[2] & x[3]) != -1;
    if (c1 <= row.last && (c0 >= row.from || c1 <= row.keep)) {
      const auto u = [&](int e) { return static_cast<uint32_t>(x[e]); };
      return max(max(u(0), u(1)), max(u(2), u(3))) >= static_cast<uint32_t>(a.num_pages);
    }
    return true;
  }
};

// Exclusive counts of the bits of `words` words, and their total: by all threads.
template <int kThreads>
__device__ uint32_t count_before(const uint32_t* bits, uint32_t* before, int words, uint32_t* scratch) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per = (words + kThreads - 1) / kThreads;
  const int i0 = min(words, static_cast<int>(threadIdx.x) * per), i1 = min(words, i0 + per);
  uint32_t mine = 0;
  for (int i = i0; i < i1; ++i) mine += __popc(bits[i]);
  uint32_t inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  uint32_t at = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at += scratch[w];
    total += scratch[w];
  }
  for (int i = i0; i < i1; ++i) {
    before[i] = at;
    at += __popc(bits[i]);
  }
  __syncthreads();
  return total;
}

// The last of n ascending numbers, load(0) = 0 .. load(n - 1), that is at most k: seven looks at a time, since a look
// into another CTA's memory takes long.
template <typename Load>
__device__ __forceinline__ int last_at_most(uint32_t k, int n, const Load& load) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 7) / 8;
    int below = 0;
#pragma unroll
    for (int q = 1; q < 8; ++q) {
      const int at = lo + q * step;
      below += at < hi && load(min(at, n - 1)) <= k;
    }
    lo += below * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

// The place of the k-th bit (from 0) of a word.
__device__ __forceinline__ int bit_of(uint32_t word, uint32_t k) {
  for (; k; --k) word &= word - 1;
  return __ffs(word) - 1;
}

// Bound by latency (barriers, loads that depend on one another: 32 sequences and 2831 pages 5.4 us) and, where tables
// are large, by what the cluster's SMs can read and look through (256 rows of 8194 entries and 145 166 pages: 9 MB in
// 24 us; four CTAs took 64).
template <bool FORK, int N, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) spec_kv_pages_kernel(const __grid_constant__ PagesArgs a) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint32_t dyn[];
  __shared__ uint32_t scratch[kWarps], total[2];            // this CTA's missing entries and free pages
  __shared__ uint32_t need_at[kMostCtas + 1], free_at[kMostCtas + 1];
  uint32_t* const need = dyn;
  uint32_t* const need_before = need + a.need_share;
  uint32_t* const avail = need_before + a.need_share;
  uint32_t* const avail_before = avail + a.free_share;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank()), ctas = static_cast<int>(cluster_size());
  const int w0 = min(a.need_words, rank * a.need_share), nw = min(a.need_words - w0, a.need_share);
  const int f0 = min(a.free_words, rank * a.free_share), nf = min(a.free_words - f0, a.free_share);
  start_dependents();
  wait_for_grid();

  // ---- 1. the table: a stretch a warp, the next one under way
  // (of forks, whose stretches have two rows, one at a time)
  Stretch<FORK, N> now, next;
  constexpr int kStretchWords = Stretch<FORK, N>::kWords;
  if (!FORK && warp < nw / kStretchWords) now.load(a, w0 / kStretchWords + warp);
  for (int i = warp; i < nw / kStretchWords; i += kWarps) {
    if (FORK)
      now.load(a, w0 / kStretchWords + i);
    else if (i + kWarps < nw / kStretchWords)
      next.load(a, w0 / kStretchWords + i + kWarps);
    bool some = FORK;
    if constexpr (!FORK) {
#pragma unroll
      for (int k = 0; k < N; ++k) some |= now.some(a, k);
    }
    if (now.row.last < 0 || !__any_sync(kFull, some)) {
      if (lane < kStretchWords) need[i * kStretchWords + lane] = 0;
    } else {
      bool bad = false;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int c0 = now.column(k);
        const Four& old = now.entry[k];
        Four to = old;
        uint32_t missing = 0;
        if constexpr (FORK) {
          const int whole = now.row.last >> a.log_page;
          const bool rest = (now.row.last & ((1 << a.log_page) - 1)) != 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t src = now.source[k].x[e];
            const bool partly = rest && c0 + e == whole, page = src >= 0 && src < a.num_pages;
            if (old.x[e] >= 0 && old.x[e] < a.num_pages) atomicSub(&a.refs[old.x[e]], 1);
            if (c0 + e < whole && page) atomicAdd(&a.refs[src], 1);
            if (partly && page) missing |= 1u << e;
            to.x[e] = c0 + e < whole && page ? src : -1;
            bad |= (c0 + e < whole && src >= a.num_pages) || (partly && !page);
          }
        } else if (__any_sync(kFull, now.some(a, k))) {
          const uint32_t needed = first_of(now.row.last - c0) & (first_of(now.row.keep - c0) | ~first_of(now.row.from - c0));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((needed >> e) & 1) {
              if (old.x[e] < 0) missing |= 1u << e;
              bad |= old.x[e] >= a.num_pages;
            } else if (old.x[e] != -1) {
              if (old.x[e] >= 0 && old.x[e] < a.num_pages) atomicSub(&a.refs[old.x[e]], 1);
              to.x[e] = -1;
            }
          }
        }
        to.store(a.table + now.b * a.table_stride, old, c0, a.max_pages);
        const uint32_t word = word_of(missing);
        if ((lane & 7) == 0) need[i * kStretchWords + k * 4 + lane / 8] = word;
      }
      if (bad) report(a.status, SPEC_ERR_CACHE_RANGE);
      if (FORK && now.column(0) == 0) a.seq_lens[now.b] = now.row.last;
    }
    if (!FORK) now = next;
  }
  __syncthreads();
  {
    const uint32_t n = count_before<kThreads>(need, need_before, nw, scratch);
    if (tid == 0) total[0] = n;
  }
  cluster_sync();  // the counts are final
  if (warp == 0) {
    const uint32_t n = lane < ctas ? load_of(lane, &total[0]) : 0;
    uint32_t inc = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(kFull, inc, d);
      if (lane >= d) inc += o;
    }
    if (lane <= kMostCtas) need_at[lane] = inc - n;
  }
  __syncthreads();
  const uint32_t needs = need_at[ctas];
  if (needs > 0 || a.free_pages) {
    // ---- 2. the pool: 128 pages a warp
    for (int i0 = warp; i0 < nf / 4; i0 += kWarps * kAhead) {
      Four count[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i0 + k * kWarps < nf / 4) count[k].load_counts(a, (f0 / 4 + i0 + k * kWarps) * 128 + lane * 4);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * kWarps;
        if (i >= nf / 4) continue;
        uint32_t bits = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) bits |= count[k].x[e] <= 0 ? 1u << e : 0u;
        const uint32_t word = word_of(bits);
        if ((lane & 7) == 0) avail[i * 4 + lane / 8] = word;
      }
    }
    __syncthreads();
    {
      const uint32_t n = count_before<kThreads>(avail, avail_before, nf, scratch);
      if (tid == 0) total[1] = n;
    }
    cluster_sync();
    if (warp == 0) {
      const uint32_t n = lane < ctas ? load_of(lane, &total[1]) : 0;
      uint32_t inc = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(kFull, inc, d);
        if (lane >= d) inc += o;
      }
      if (lane <= kMostCtas) free_at[lane] = inc - n;
    }
    __syncthreads();
    const uint32_t frees = free_at[ctas];
    if (rank == 0 && tid == 0 && a.free_pages) *a.free_pages = static_cast<int32_t>(frees - min(frees, needs));

    // ---- 3. pages for the missing entries, one a thread
    const uint32_t mine = total[0];
    for (uint32_t n = tid; n < mine; n += kThreads) {
      uint32_t k = need_at[rank] + n;
      if (k >= frees) {
        report(a.status, SPEC_ERR_CACHE_FULL);
        break;
      }
      const int i = last_at_most(n, nw, [&](int w) { return need_before[w]; });
      const int b = (w0 + i) / a.row_words;
      const int c = (w0 + i - b * a.row_words) * 32 + bit_of(need[i], n - need_before[i]);
      int r = 0;
#pragma unroll
      for (int q = 1; q < kMostCtas; ++q) r += q < ctas && k >= free_at[q];
      k -= free_at[r];
      const int lo = last_at_most(k, min(a.free_words - r * a.free_share, a.free_share),
                                  [&](int w) { return load_of(r, avail_before + w); });
      const uint32_t word = load_of(r, avail + lo), before = load_of(r, avail_before + lo);
      const int page = (r * a.free_share + lo) * 32 + bit_of(word, k - before);
      a.table[b * a.table_stride + c] = page;
      a.refs[page] = 1;
    }
  }
  cluster_sync();  // others may still be reading here
}

// The filled slots and the scales of the last pages of copies.  A warp has the keys or
// the values of one head of a page: rows of D bytes, 16 a lane.
struct CopyArgs {
  PagesArgs a;
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
  int64_t page_stride, head_stride, token_stride, scale_page_stride, scale_head_stride;
  int32_t Hkv, vecs, blocks;  // heads; 16-byte pieces of a row, at most 16; blocks of a sequence
  int32_t vecs_recip;         // 2^16 / vecs, rounded up: i / vecs is (i * this) >> 16 for the 2048 pieces of a page
};

constexpr int kCopyThreads = 128, kCopyAhead = 8;

__global__ void __launch_bounds__(kCopyThreads) spec_kv_copy_kernel(const __grid_constant__ CopyArgs g) {
  const PagesArgs& a = g.a;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x / g.blocks;
  const int unit = (blockIdx.x - b * g.blocks) * (kCopyThreads / 32) + (threadIdx.x >> 5);
  start_dependents();
  wait_for_grid();
  int L = 0;
  const int p = parent_of(a, b, &L);
  const int filled = L & ((1 << a.log_page) - 1);
  if (p < 0 || filled == 0 || unit >= 2 * g.Hkv) return;
  const int c = L >> a.log_page;
  const int from = a.table[p * a.table_stride + c], to = a.table[b * a.table_stride + c];
  if (from < 0 || from >= a.num_pages || to < 0 || to >= a.num_pages) return;
  const bool values = unit & 1;
  const int h = unit >> 1;
  uint8_t* const codes = (values ? g.v_codes : g.k_codes) + h * g.head_stride;
  float* const scale = (values ? g.v_scale : g.k_scale) + h * g.scale_head_stride;
  if (lane == 0) scale[to * g.scale_page_stride] = scale[from * g.scale_page_stride];
  const uint8_t* const src = codes + from * g.page_stride;
  uint8_t* const dst = codes + to * g.page_stride;
  const int pieces = filled * g.vecs;
  for (int i0 = lane; i0 < pieces; i0 += 32 * kCopyAhead) {
    uint4 x[kCopyAhead];
    int64_t at[kCopyAhead];
#pragma unroll
    for (int k = 0; k < kCopyAhead; ++k) {
      const int i = i0 + 32 * k, tok = (i * g.vecs_recip) >> 16;
      at[k] = tok * g.token_stride + (i - tok * g.vecs) * 16;
      if (i < pieces) x[k] = *reinterpret_cast<const uint4*>(src + at[k]);
    }
#pragma unroll
    for (int k = 0; k < kCopyAhead; ++k)
      if (i0 + 32 * k < pieces) *reinterpret_cast<uint4*>(dst + at[k]) = x[k];
  }
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Launch {
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = {};
  Launch(int64_t grid, int threads, int cluster, int smem, void* stream) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

spec_status launch(const void* fn, int64_t grid, int threads, int cluster, int smem, void* stream, void** args) {
  const Launch l(grid, threads, cluster, smem, stream);
  if (cudaLaunchKernelExC(&l.cfg, fn, args) != cudaSuccess) return SPEC_ERR_CUDA;
  specv_units::count_launches(1);
  return SPEC_OK;
}

// how many clusters of this size the device has room for at once
int clusters(const void* fn, int ctas, int threads, int smem) {
  const Launch l(ctas, threads, ctas, smem, nullptr);
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fn, &l.cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

spec_status check(const spec_kv_pages* p) {
  if (!p || p->num_pages < 1 || p->B < 0 || p->max_pages < 1) return SPEC_ERR_INVALID_ARG;
  if (p->page_size != 16 && p->page_size != 32 && p->page_size != 64 && p->page_size != 128) return SPEC_ERR_INVALID_ARG;
  if (!p->refs || !aligned(p->refs, 4)) return SPEC_ERR_INVALID_ARG;
  if (p->B == 0) return SPEC_OK;
  if (!p->page_table || !aligned(p->page_table, 4)) return SPEC_ERR_INVALID_ARG;
  if (p->B > 1 && p->table_stride < p->max_pages) return SPEC_ERR_INVALID_ARG;
  // positions are counted in 32 bits
  if (static_cast<int64_t>(p->max_pages) * p->page_size > INT_MAX - 128) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// CTAs of the cluster, of at most `most`, and the shared memory of each; 0: too large.
constexpr int kMostSmem = 224 * 1024;
int plan(PagesArgs& a, int batch, int most, int* smem) {
  const int stretches = (a.max_pages + 128 * batch - 1) / (128 * batch), words = 4 * batch;
  a.row_words = stretches * words;
  a.row_recip = ~uint64_t(0) / static_cast<uint64_t>(stretches) + 1;
  const int64_t need = static_cast<int64_t>(a.B) * a.row_words, avail = (static_cast<int64_t>(a.num_pages) + 127) / 128 * 4;
  if (need + avail > static_cast<int64_t>(most) * kMostSmem / 8) return 0;
  a.need_words = static_cast<int32_t>(need);
  a.free_words = static_cast<int32_t>(avail);
  // a small call is quickest with one CTA, another with all that a cluster may have
  const int ctas = need + avail <= kWordsAlone ? 1 : most;
  a.need_share = (a.need_words / words + ctas - 1) / ctas * words;
  a.free_share = (a.free_words / 4 + ctas - 1) / ctas * 4;
  *smem = 8 * (a.need_share + a.free_share);
  return *smem <= kMostSmem ? ctas : 0;
}

template <bool FORK, int N, int kThreads>
spec_status launch_pages(PagesArgs& a, void* stream) {
  int smem = 0;
  if (plan(a, N, kMostCtas, &smem) == 0) return SPEC_ERR_UNSUPPORTED;
  const void* fn = reinterpret_cast<const void*>(&spec_kv_pages_kernel<FORK, N, kThreads>);
  // once for a kernel and device: allow what it takes, and ask whether the device has room for the largest cluster
  static std::atomic<int> most[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPEC_ERR_CUDA;
  int ctas = most[dev].load(std::memory_order_acquire);
  if (ctas == 0) {
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) != cudaSuccess ||
        cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
      return SPEC_ERR_CUDA;
    ctas = clusters(fn, kMostCtas, kThreads, kMostSmem) > 0 ? kMostCtas : kPortableCtas;
    most[dev].store(ctas, std::memory_order_release);
  }
  ctas = plan(a, N, ctas, &smem);
  if (ctas == 0) return SPEC_ERR_UNSUPPORTED;
  void* args[] = {&a};
  return launch(fn, ctas, kThreads, ctas, smem, stream, args);
}

template <bool FORK>
spec_status launch_pages(PagesArgs& a, void* stream) {
  const int64_t words = (static_cast<int64_t>(a.B) * a.max_pages + a.num_pages) / 32;
  if (words <= kWordsFew)
    return a.max_pages <= 128 ? launch_pages<FORK, 1, 256>(a, stream) : launch_pages<FORK, 4, 256>(a, stream);
  return a.max_pages <= 128 ? launch_pages<FORK, 1, 1024>(a, stream) : launch_pages<FORK, 4, 1024>(a, stream);
}

void fill(const spec_kv_pages* p, PagesArgs& a) {
  a.refs = p->refs;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.free_pages = p->free_pages;
  a.status = p->status;
  a.num_pages = p->num_pages;
  a.log_page = 0;
  while ((1 << a.log_page) < p->page_size) ++a.log_page;
  a.B = p->B;
  a.max_pages = p->max_pages;
  a.vec = aligned(p->page_table, 16) && (p->B == 1 || p->table_stride % 4 == 0);
  a.refs_vec = aligned(p->refs, 16);
}

}  // namespace

extern "C" {

spec_status spec_kv_hold(const spec_kv_pages* pages, const int32_t* seq_lens, const int32_t* new_lens, int32_t T,
                         int32_t window, int32_t sinks) {
  const spec_status s = check(pages);
  if (s != SPEC_OK) return s;
  if (T < 0 || window < 0 || sinks < 0) return SPEC_ERR_INVALID_ARG;
  if (pages->B > 0 && !seq_lens) return SPEC_ERR_INVALID_ARG;
  PagesArgs a = {};
  fill(pages, a);
  a.seq_lens = const_cast<int32_t*>(seq_lens);  // (not written by this)
  a.new_lens = new_lens;
  a.T = T;
  a.window = window;
  a.sinks = sinks;
  return launch_pages<false>(a, pages->stream);
}

spec_status spec_kv_fork(const spec_kv_pages* pages, const spec_kv_cache* cache, int32_t* seq_lens,
                         const int32_t* parents) {
  spec_status s = check(pages);
  if (s != SPEC_OK) return s;
  if (!cache || cache->num_pages != pages->num_pages || cache->page_size != pages->page_size) return SPEC_ERR_INVALID_ARG;
  if (cache->Hkv < 1 || cache->D < 16 || cache->D > 256 || cache->D % 16) return SPEC_ERR_INVALID_ARG;
  if (!cache->k_codes || !cache->v_codes || !cache->k_scale || !cache->v_scale) return SPEC_ERR_INVALID_ARG;
  if (!aligned(cache->k_codes, 16) || !aligned(cache->v_codes, 16)) return SPEC_ERR_INVALID_ARG;
  if (cache->page_stride < 0 || cache->head_stride < 0 || cache->token_stride < 0 || cache->page_stride % 16 ||
      cache->head_stride % 16 || cache->token_stride % 16 || cache->scale_page_stride < 0 || cache->scale_head_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  if (cache->token_stride == 0 || (cache->Hkv > 1 && (cache->head_stride == 0 || cache->scale_head_stride == 0)) ||
      (cache->num_pages > 1 && (cache->page_stride == 0 || cache->scale_page_stride == 0)))
    return SPEC_ERR_INVALID_ARG;
  if (pages->B > 0 && (!seq_lens || !parents)) return SPEC_ERR_INVALID_ARG;
  CopyArgs g = {};
  PagesArgs& a = g.a;
  fill(pages, a);
  a.seq_lens = seq_lens;
  a.parents = parents;
  constexpr int warps = kCopyThreads / 32;
  g.blocks = (2 * cache->Hkv + warps - 1) / warps;
  if (static_cast<int64_t>(a.B) * g.blocks > INT_MAX) return SPEC_ERR_UNSUPPORTED;
  s = launch_pages<true>(a, pages->stream);
  if (s != SPEC_OK || a.B == 0) return s;
  g.k_codes = cache->k_codes;
  g.v_codes = cache->v_codes;
  g.k_scale = cache->k_scale;
  g.v_scale = cache->v_scale;
  g.page_stride = cache->page_stride;
  g.head_stride = cache->head_stride;
  g.token_stride = cache->token_stride;
  g.scale_page_stride = cache->scale_page_stride;
  g.scale_head_stride = cache->scale_head_stride;
  g.Hkv = cache->Hkv;
  g.vecs = cache->D / 16;
  g.vecs_recip = (65536 + g.vecs - 1) / g.vecs;
  void* args[] = {&g};
  return launch(reinterpret_cast<const void*>(&spec_kv_copy_kernel), static_cast<int64_t>(a.B) * g.blocks, kCopyThreads, 1,
                0, pages->stream, args);
}

}  // extern "C"
