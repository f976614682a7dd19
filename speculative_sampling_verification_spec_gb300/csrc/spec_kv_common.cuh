#pragma once
// spec_kv_common.cuh -- what the paged-cache kernels share: their arguments, how
// the attention's work is cut into ranges of tiles, and small device helpers.
//
// The attention's work is a list of tiles of 2^log_tile tokens: sequence after
// sequence, within a sequence head after head, within a head in order of
// position.  Before each head's tiles come `overhead` places without one, for what
// it costs to take up a head.  The list is cut into `nranges` equal ranges (from
// the lengths on the device, so a batch of unequal sequences is spread evenly and
// no length crosses to the host); a range is walked by one CTA for one row tile.
// An item (sequence, head, row tile) that lies in one range is finished there; one
// that several ranges share leaves a partial result (unnormalised output,
// reference, sum) per range in the workspace.  They are added up in the order of
// the ranges, by the CTA that arrives last or by the join kernel.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "spec_kv.h"

namespace spec_kv_detail {

constexpr int kTile = 128;          // tokens of a tensor-core tile
constexpr int kMinScaleExp = -100;  // scales are at least 2^kMinScaleExp
constexpr float kNoRef = -3.4028234663852886e38f;  // softmax reference before any token: the lowest float
constexpr unsigned kFull = 0xffffffffu;

struct KvArgs {
  // cache
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scale;
  float* v_scale;
  int64_t page_stride, head_stride, token_stride, scale_page_stride, scale_head_stride;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* status;
  int32_t B, T, Hq, Hkv, G, D;
  int32_t log_page, num_pages, max_pages, window;
  // attention
  const void* q;
  void* out;
  float* lse;
  int64_t q_seq, q_tok, q_head, o_seq, o_tok, o_head;
  float scale2;       // scale * log2(e): scores are kept in log2 units
  int32_t rows;       // rows of a row tile (row = t * G + head in group)
  int32_t nrt;        // row tiles of a sequence
  int32_t log_tile;   // log2 of a tile's tokens
  int32_t nranges;    // ranges of the tile list
  int32_t overhead;   // places of the list before a head's tiles
  int32_t join_here;  // the last CTA of an item joins it, else the join kernel
  int32_t q_vec;      // queries may be loaded 16 bytes at a time
  int32_t o_vec;      // outputs may be stored four channels at a time
  int32_t slot_rows;  // rows a partial slot has room for
  int32_t* arrived;   // workspace: [B][Hkv][nrt] ranges that have left their part; zero between calls
  int32_t* prefix;    // workspace: [B + 1] places of the list before each sequence
  float* part_o;      // workspace: [slots][slot_rows][D]
  float2* part_ml;    // workspace: [slots][slot_rows] (reference, sum)
};

__device__ __forceinline__ void report(int32_t* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// Programmatic dependent launches.  A kernel of the cache may be scheduled while
// the one before it in the stream runs out; nothing of global memory is read or
// written before wait_for_grid (which every CTA passes), and the next such kernel
// may be scheduled once every CTA has called start_dependents.
__device__ __forceinline__ void start_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_grid() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_float(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }

// two e4m3 codes -> two floats (exact)
__device__ __forceinline__ float2 codes2_to_float2(uint16_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
  return __half22float2(__half2(h));
}

// The tokens of sequence b and the tiles its rows read: positions from tile
// t0 to L + n.  No tiles when it has no new token or its lengths are out of range.
struct SeqSpan {
  int L, n, t0, nt;
  int places;  // a head's in the list
  bool bad;
};
__device__ __forceinline__ SeqSpan seq_span(const KvArgs& a, int b) {
  SeqSpan s;
  s.L = a.seq_lens[b];
  s.n = a.new_lens ? a.new_lens[b] : a.T;
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.log_page;
  s.bad = s.L < 0 || s.n < 0 || s.n > a.T || static_cast<int64_t>(s.L) + s.n > cap;
  s.t0 = 0;
  s.nt = 0;
  s.places = 0;
  if (!s.bad && s.n > 0) {
    const int first = (a.window > 0 && s.L + 1 > a.window) ? s.L + 1 - a.window : 0;
    s.t0 = first >> a.log_tile;
    s.nt = ((s.L + s.n - 1) >> a.log_tile) + 1 - s.t0;
    s.places = s.nt + a.overhead;
  }
  return s;
}

// A CTA's view of the list: the range [w0, w1), and where w0 lies.
struct RangePlan {
  int per, w0, w1;
  int b, off;  // sequence that holds w0, and w0's offset in its places (all heads)
};

// All threads of the CTA (NT of them) take part, once; `plan` and `scratch` are in
// shared memory.  When prefix is given, it gets the places before each sequence.
template <int NT>
__device__ void make_plan_range(const KvArgs& a, int range, RangePlan* plan, int* scratch, int32_t* prefix) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = (a.B + NT - 1) / NT;
  const int b0 = min(a.B, tid * c), b1 = min(a.B, b0 + c);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += seq_span(a, b).places * a.Hkv;
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += o;
  }
  if (lane == 31) scratch[warp] = inc;
  __syncthreads();
  int before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
  }
  const int per = max(1, (total + a.nranges - 1) / a.nranges);
  const int64_t start = static_cast<int64_t>(range) * per;
  const int w0 = start < total ? static_cast<int>(start) : total;
  const int w1 = min(total, w0 + per);
  if (tid == 0) {
    plan->per = per;
    plan->w0 = w0;
    plan->w1 = w1;
    if (prefix) prefix[a.B] = total;
  }
  if (w0 < w1 && before <= w0 && w0 < before + mine) {
    int at = before;
    for (int b = b0; b < b1; ++b) {
      const int k = seq_span(a, b).places * a.Hkv;
      if (w0 < at + k) {
        plan->b = b;
        plan->off = w0 - at;
        break;
      }
      at += k;
    }
  }
  if (prefix) {
    int at = before;
    for (int b = b0; b < b1; ++b) {
      prefix[b] = at;
      at += seq_span(a, b).places * a.Hkv;
    }
  }
  __syncthreads();
}

// One piece of work: a (sequence, head, row tile) and the tiles of it that this
// range holds.  Every role of a CTA walks the same pieces.
struct Piece {
  int b, h;
  int L, n;          // tokens before the new ones; new tokens
  int row0, nrows;   // rows of this row tile
  int tile0, tile1;  // absolute tiles [tile0, tile1); may be empty
  int first;         // first position that a row sees
  int c0, c1;        // first and last range that hold tiles of the item
  int slot;          // where a partial result goes, when these differ
  __device__ bool whole() const { return c0 == c1; }
};

struct Walk {
  int w, w1, b, off;  // next place of the list; sequence and offset in it
  int per, range, rt;
};

__device__ __forceinline__ Walk walk_begin(const RangePlan& p, int range, int rt) {
  Walk k;
  k.w = p.w0;
  k.w1 = p.w1;
  k.b = p.b;
  k.off = p.off;
  k.per = p.per;
  k.range = range;
  k.rt = rt;
  return k;
}

// The slot of range c's part of an item that begins in range c0: a range holds at
// most one item that began before it and one that goes on after it.
__device__ __forceinline__ int part_slot(const KvArgs& a, int c, int c0, int rt) {
  return 2 * (c * a.nrt + rt) + (c == c0 ? 1 : 0);
}

// The next piece that has rows; false at the range's end.
__device__ __forceinline__ bool walk_next(const KvArgs& a, Walk& k, Piece& p) {
  while (k.w < k.w1) {
    const SeqSpan s = seq_span(a, k.b);
    if (k.off >= s.places * a.Hkv) {  // on to the next sequence
      ++k.b;
      k.off = 0;
      continue;
    }
    const int h = k.off / s.places, at = k.off - h * s.places;
    const int take = min(s.places - at, k.w1 - k.w);
    const int first = k.w - at + a.overhead;  // place of the item's first tile
    const int t0 = max(at - a.overhead, 0), t1 = at + take - a.overhead;
    p.c0 = first / k.per;
    p.c1 = (first + s.nt - 1) / k.per;
    p.slot = part_slot(a, k.range, p.c0, k.rt);
    k.w += take;
    k.off += take;
    p.b = k.b;
    p.h = h;
    p.L = s.L;
    p.n = s.n;
    p.row0 = k.rt * a.rows;
    p.nrows = min(a.rows, s.n * a.G - p.row0);
    if (p.nrows <= 0 || t1 <= 0) continue;
    // tiles that some row of this row tile sees
    const int t_first = p.row0 / a.G, t_last = (p.row0 + p.nrows - 1) / a.G;
    const int hi = ((s.L + t_last) >> a.log_tile) + 1;
    const int lo = (a.window > 0 && s.L + t_first + 1 > a.window) ? s.L + t_first + 1 - a.window : 0;
    p.first = lo;
    p.tile0 = max(s.t0 + t0, lo >> a.log_tile);
    p.tile1 = min(s.t0 + t1, hi);
    if (p.tile1 < p.tile0) p.tile1 = p.tile0;
    return true;
  }
  return false;
}

// page number of a token's page, -1 where it is not one of the pool's (an error
// only if some row sees a token of it: a tile may begin before the window)
__device__ __forceinline__ int page_of(const KvArgs& a, int b, int page_index) {
  const int pid = a.table[b * a.table_stride + page_index];
  return (pid >= 0 && pid < a.num_pages) ? pid : -1;
}

}  // namespace spec_kv_detail
