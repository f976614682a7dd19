#pragma once
// spec_kv_attn.cuh -- attention over the paged 8-bit cache: the kernel on the
// ordinary float units, which takes every type, head size and alignment, and the
// kernel that joins the ranges' partial results.
//
// One pass over the tokens with the running maximum m and sum l of each row's
// softmax, in log2 units:  m' = max(m, x);  o = o 2^(m - m') + 2^(x - m') v;
// l likewise.  All of it is held in float.
//
// float32 queries come here because 8-bit pieces cannot reach their precision (and
// the matrix unit's truncated sums would not keep it).  Bound by shared-memory
// reads: 16 sequences of 8000 tokens, 32 float32 query heads on 8 key/value heads:
// 263 MB in 299 us.
#include "spec_kv_common.cuh"

namespace spec_kv_detail {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// reference and sum -> natural logarithm of the sum of the weights
__device__ __forceinline__ float lse_of(float m, float l) { return (m + log2f(l)) * 0.69314718055994531f; }

template <typename E>
__device__ __forceinline__ void store4(const KvArgs& a, E* o, float4 x) {
  if constexpr (sizeof(E) == 4) {
    if (a.o_vec) {
      *reinterpret_cast<float4*>(o) = x;
      return;
    }
  } else {
    if (a.o_vec) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
      *reinterpret_cast<uint2*>(o) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      return;
    }
  }
  from_float(x.x, o);
  from_float(x.y, o + 1);
  from_float(x.z, o + 2);
  from_float(x.w, o + 3);
}

// The largest reference of a row's parts, in every lane.
__device__ __forceinline__ float top_of_parts(const KvArgs& a, int rt, int r, int c0, int c1) {
  float top = kNoRef;
  for (int c = c0 + (threadIdx.x & 31); c <= c1; c += 32)
    top = fmaxf(top, __ldcg(&a.part_ml[static_cast<int64_t>(part_slot(a, c, c0, rt)) * a.slot_rows + r]).x);
#pragma unroll
  for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
  return top;
}

// Adds up the parts of one row from `from` on, `step` apart, in order: lane by lane
// four channels (and four more from 128 on).  `top` gets the largest reference of
// all parts c0 .. c1.  The first outputs are asked for before the references are
// there: a join is a few trips to the L2 cache, one after the other.
__device__ __forceinline__ void add_parts(const KvArgs& a, int rt, int r, int c0, int c1, int from, int step, float& top,
                                          float4* acc, float& l) {
  constexpr int kAhead = 4;
  const int lane = threadIdx.x & 31;
  const auto slot_row = [&](int c) { return static_cast<int64_t>(part_slot(a, c, c0, rt)) * a.slot_rows + r; };
  const auto part_ml = [&](int cb) {  // of up to 32 parts, one a lane
    return cb + lane * step <= c1 ? __ldcg(&a.part_ml[slot_row(cb + lane * step)]) : make_float2(kNoRef, 0.0f);
  };
  float2 ml = part_ml(from);
  bool have_top = false;
  for (int cb = from; cb <= c1; cb += 32 * step) {
    if (cb != from) ml = part_ml(cb);
    float wl = 0.0f;
    const int m = min(32, (c1 - cb) / step + 1);
    for (int i0 = 0; i0 < m; i0 += kAhead) {
      float4 x[kAhead][2];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int d = lane * 4 + k * 128;
          x[i][k] = make_float4(0, 0, 0, 0);
          if (i0 + i < m && d < a.D)
            x[i][k] = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot_row(cb + (i0 + i) * step) * a.D + d));
        }
      }
      if (i0 == 0) {
        if (!have_top) {
          top = step == 1 && c1 - c0 < 32 ? ml.x : kNoRef;
          if (step == 1 && c1 - c0 < 32) {
#pragma unroll
            for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
          } else {
            top = top_of_parts(a, rt, r, c0, c1);
          }
          have_top = true;
        }
        wl = exp2f(ml.x - top);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float w = __shfl_sync(kFull, wl, i0 + i), li = __shfl_sync(kFull, ml.y, i0 + i);
        // a part without tokens for this row left no output
        if (i0 + i >= m || li == 0.0f) continue;
        l = fmaf(w, li, l);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          acc[k].x = fmaf(w, x[i][k].x, acc[k].x);
          acc[k].y = fmaf(w, x[i][k].y, acc[k].y);
          acc[k].z = fmaf(w, x[i][k].z, acc[k].z);
          acc[k].w = fmaf(w, x[i][k].w, acc[k].w);
        }
      }
    }
  }
  if (!have_top) top = top_of_parts(a, rt, r, c0, c1);
}

// A joined row's output and lse, by one warp.
template <typename E>
__device__ __forceinline__ void store_row(const KvArgs& a, int b, int t, int hq, const float4* acc, float top, float l) {
  const int lane = threadIdx.x & 31;
  E* o = static_cast<E*>(a.out) + b * a.o_seq + t * a.o_tok + hq * a.o_head;
  const float inv = 1.0f / l;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = lane * 4 + k * 128;
    if (d < a.D) store4(a, o + d, make_float4(acc[k].x * inv, acc[k].y * inv, acc[k].z * inv, acc[k].w * inv));
  }
  if (lane == 0 && a.lse) a.lse[(static_cast<int64_t>(b) * a.T + t) * a.Hq + hq] = lse_of(top, l);
}

// Whether this CTA is the last of its item to leave its part (all parts can then
// be read).  Called by one thread after the CTA's stores and a barrier.
__device__ __forceinline__ bool last_of_item(const KvArgs& a, const Piece& p, int rt) {
  int32_t* count = a.arrived + (static_cast<int64_t>(p.b) * a.Hkv + p.h) * a.nrt + rt;
  __threadfence();
  const bool last = atomicAdd(count, 1) == p.c1 - p.c0;
  if (last) {
    *count = 0;  // for the next call
    __threadfence();
  }
  return last;
}

// Joins an item's rows, by `warps` warps: a row is a warp's.
template <typename E>
__device__ __forceinline__ void join_item(const KvArgs& a, const Piece& p, int rt, int warp, int warps) {
  for (int r = warp; r < p.nrows; r += warps) {
    const int gr = p.row0 + r, t = gr / a.G, g = gr - t * a.G;
    float top;
    float4 acc[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
    float l = 0.0f;
    add_parts(a, rt, r, p.c0, p.c1, p.c0, 1, top, acc, l);
    store_row<E>(a, p.b, t, p.h * a.G + g, acc, top, l);
  }
}

// Slots without a new token are zero, those of a sequence with bad lengths NaN;
// (sequence, slot) pairs are spread over the grid's CTAs.
template <typename E>
__device__ __forceinline__ void fill_empty(const KvArgs& a, int tid, int threads) {
  const int64_t pairs = static_cast<int64_t>(a.B) * a.T;
  for (int64_t i = blockIdx.x; i < pairs; i += gridDim.x) {
    const int b = static_cast<int>(i / a.T), t = static_cast<int>(i - static_cast<int64_t>(b) * a.T);
    const SeqSpan s = seq_span(a, b);
    if (!s.bad && t < s.n) continue;
    const float x = s.bad ? __uint_as_float(0x7fc00000u) : 0.0f;
    if (s.bad && tid == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
    const int quads = a.D / 4;
    for (int e = tid; e < a.Hq * quads; e += threads) {
      const int h = e / quads, d = (e - h * quads) * 4;
      store4(a, static_cast<E*>(a.out) + b * a.o_seq + t * a.o_tok + h * a.o_head + d, make_float4(x, x, x, x));
      if (d == 0 && a.lse) a.lse[i * a.Hq + h] = s.bad ? x : -INFINITY;
    }
  }
}

constexpr int kGenThreads = 128;
constexpr int kGenRows = 8;    // rows of a row tile at most
constexpr int kGenLogTile = 6; // tokens of a tile: short, for latency
constexpr int kGenSub = 32;    // tokens staged at a time: a lane's token in the scores
constexpr int kGenMaxD = 256;
constexpr int gen_smem_bytes(int D, int rows) { return 4 * (rows * D + kGenSub * (D + 4)) + kGenSub * D; }

// A CTA walks its pieces 32 tokens at a time.  The next 32 tokens' codes are in
// registers (16-byte loads) while the present ones are worked on.  Scores: lane =
// token, a row's maximum and sum stay in its warp.  Output: thread = channel, all
// rows in registers.
// MAXD: 128 or 256, the head sizes that the registers are laid out for; ROWS: rows
// of a row tile, 4 or 8, a fourth of them a warp's.
template <typename E, int MAXD, int ROWS>
__global__ void __launch_bounds__(kGenThreads, MAXD == 128 ? 5 : 3)
    spec_kv_attention_kernel(const __grid_constant__ KvArgs a) {
  constexpr int kVecs = 2 * kGenSub * (MAXD / 16) / kGenThreads;  // 16-byte vectors a thread, keys and values
  constexpr int kCh = MAXD / kGenThreads;                         // channels a thread
  __shared__ RangePlan plan;
  __shared__ int scratch[kGenThreads / 32];
  extern __shared__ __align__(16) uint8_t dyn[];  // gen_smem_bytes(D, ROWS)
  __shared__ __align__(16) float sp[ROWS][kGenSub];
  __shared__ float sfac[ROWS], sl[ROWS], sm[ROWS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int range = blockIdx.x / a.nrt, rt = blockIdx.x - range * a.nrt;
  start_dependents();
  wait_for_grid();
  make_plan_range<kGenThreads>(a, range, &plan, scratch, blockIdx.x == 0 ? a.prefix : nullptr);
  fill_empty<E>(a, tid, kGenThreads);
  if (plan.w0 >= plan.w1) return;
  const int D = a.D, kst = D + 4, dv = D / 16;
  float* sq = reinterpret_cast<float*>(dyn);  // [ROWS][D]
  float* sk = sq + ROWS * D;              // [kGenSub][kst]: four floats of padding keep the lanes' banks apart
  uint8_t* sv = reinterpret_cast<uint8_t*>(sk + kGenSub * kst);  // [kGenSub][D]
  const int half_vecs = kGenSub * dv;  // vectors of the staged keys
  Walk walk = walk_begin(plan, range, rt);
  Piece p;
  while (walk_next(a, walk, p)) {
    const int j0 = p.tile0 << a.log_tile, j1 = min(p.tile1 << a.log_tile, p.L + p.n);
    // queries in log2 units, zero rows past the last
    for (int i = tid; i < ROWS * D; i += kGenThreads) {
      const int r = i / D, d = i - r * D;
      float x = 0.0f;
      if (r < p.nrows) {
        const int gr = p.row0 + r, t = gr / a.G, g = gr - t * a.G;
        x = to_float(static_cast<const E*>(a.q)[p.b * a.q_seq + t * a.q_tok + (p.h * a.G + g) * a.q_head + d]) * a.scale2;
      }
      sq[i] = x;
    }
    constexpr int RW = ROWS / 4;  // rows of a warp
    float m[RW], l[RW];
    int pos[RW], low[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int r = warp * RW + i;
      m[i] = kNoRef;
      l[i] = 0.0f;
      pos[i] = r < p.nrows ? p.L + (p.row0 + r) / a.G : -1;
      low[i] = a.window > 0 ? pos[i] - a.window : -1;  // sees positions in (low, pos]
    }
    float acc[kCh][ROWS];
#pragma unroll
    for (int i = 0; i < kCh; ++i)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) acc[i][r] = 0.0f;
    // positions that every row sees
    const int all_from = a.window > 0 ? p.L + (p.row0 + p.nrows - 1) / a.G - a.window + 1 : 0;
    const int all_to = p.L + p.row0 / a.G;

    uint4 reg[kVecs];
    auto fetch = [&](int base) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        int v = tid + i * kGenThreads;
        const bool val = v >= half_vecs;
        if (val) v -= half_vecs;
        reg[i] = make_uint4(0, 0, 0, 0);
        if (v < half_vecs) {
          const int tok = v / dv, c = v - tok * dv, j = base + tok;
          if (j < j1) {
            const int page = page_of(a, p.b, j >> a.log_page);
            if (page >= 0)
              reg[i] = *reinterpret_cast<const uint4*>((val ? a.v_codes : a.k_codes) + page * a.page_stride +
                                                       p.h * a.head_stride +
                                                       (j & ((1 << a.log_page) - 1)) * a.token_stride + c * 16);
          }
        }
      }
    };
    if (j0 < j1) fetch(j0);
    for (int base = j0; base < j1; base += kGenSub) {
      // scales of the lane's token; a page that is not the pool's gives NaN
      const int j = base + lane;
      float ks = 0.0f, vs = 0.0f;
      if (j < j1) {
        const int page = page_of(a, p.b, j >> a.log_page);
        if (page < 0) {
          ks = vs = __uint_as_float(0x7fc00000u);
          if (warp == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
        } else {
          const int64_t at = page * a.scale_page_stride + p.h * a.scale_head_stride;
          ks = a.k_scale[at];
          vs = a.v_scale[at];
        }
      }
      __syncthreads();  // the staged tokens before have been read
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        int v = tid + i * kGenThreads;
        const bool val = v >= half_vecs;
        if (val) v -= half_vecs;
        if (v < half_vecs) {
          const int tok = v / dv, c = v - tok * dv;
          if (val) {
            *reinterpret_cast<uint4*>(&sv[tok * D + c * 16]) = reg[i];
          } else {
            const uint32_t w[4] = {reg[i].x, reg[i].y, reg[i].z, reg[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 lo = codes2_to_float2(static_cast<uint16_t>(w[e] & 0xffffu));
              const float2 hi = codes2_to_float2(static_cast<uint16_t>(w[e] >> 16));
              *reinterpret_cast<float4*>(&sk[tok * kst + c * 16 + e * 4]) = make_float4(lo.x, lo.y, hi.x, hi.y);
            }
          }
        }
      }
      __syncthreads();
      if (base + kGenSub < j1) fetch(base + kGenSub);
      // scores of the warp's rows
      float sc[RW];
#pragma unroll
      for (int i = 0; i < RW; ++i) sc[i] = 0.0f;
      {
        const float4* kp = reinterpret_cast<const float4*>(&sk[lane * kst]);
        const float4* qp = reinterpret_cast<const float4*>(&sq[warp * RW * D]);
#pragma unroll 4
        for (int d = 0; d < D / 4; ++d) {
          const float4 k4 = kp[d];
#pragma unroll
          for (int i = 0; i < RW; ++i) {
            const float4 q4 = qp[i * (D / 4) + d];
            sc[i] = fmaf(k4.x, q4.x, fmaf(k4.y, q4.y, fmaf(k4.z, q4.z, fmaf(k4.w, q4.w, sc[i]))));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RW; ++i) {
        const int r = warp * RW + i;
        const bool see = j < j1 && j <= pos[i] && j > low[i];
        const float x = see ? sc[i] * ks : -INFINITY;
        float top = x;
#pragma unroll
        for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
        const float mn = fmaxf(m[i], top), f = ex2(m[i] - mn);
        const float w = ex2(x - mn);
        m[i] = mn;
        l[i] = fmaf(l[i], f, w);  // a lane's share of the sum
        sp[r][lane] = see ? w * vs : -0.0f;  // -0: not seen
        if (lane == 0) sfac[r] = f;
      }
      __syncthreads();
      const bool all = base >= all_from && base + kGenSub - 1 <= all_to;
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        const int d = tid + i * kGenThreads;
        if (d < D) {
#pragma unroll
          for (int r = 0; r < ROWS; ++r) acc[i][r] *= sfac[r];
#pragma unroll 2
          for (int t = 0; t < kGenSub; t += 4) {
            const uint8_t* v0 = &sv[t * D + d];
            const float2 va = codes2_to_float2(static_cast<uint16_t>(v0[0] | (v0[D] << 8)));
            const float2 vb = codes2_to_float2(static_cast<uint16_t>(v0[2 * D] | (v0[3 * D] << 8)));
            if (all) {
#pragma unroll
              for (int r = 0; r < ROWS; ++r) {
                const float4 w = *reinterpret_cast<const float4*>(&sp[r][t]);
                acc[i][r] = fmaf(w.w, vb.y, fmaf(w.z, vb.x, fmaf(w.y, va.y, fmaf(w.x, va.x, acc[i][r]))));
              }
            } else {
              // a token that the row does not see adds nothing, whatever its slot holds
              const float v[4] = {va.x, va.y, vb.x, vb.y};
#pragma unroll
              for (int r = 0; r < ROWS; ++r) {
                const float4 w4 = *reinterpret_cast<const float4*>(&sp[r][t]);
                const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (__float_as_uint(w[e]) != 0x80000000u) acc[i][r] = fmaf(w[e], v[e], acc[i][r]);
              }
            }
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
#pragma unroll
      for (int d = 16; d; d >>= 1) l[i] += __shfl_xor_sync(kFull, l[i], d);
      if (lane == 0) {
        sl[warp * RW + i] = l[i];
        sm[warp * RW + i] = m[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int d = tid + i * kGenThreads;
      if (d < D) {
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          if (r >= p.nrows) continue;
          if (p.whole()) {
            const int gr = p.row0 + r, t = gr / a.G, g = gr - t * a.G;
            from_float(acc[i][r] / sl[r], static_cast<E*>(a.out) + p.b * a.o_seq + t * a.o_tok + (p.h * a.G + g) * a.o_head + d);
          } else {
            a.part_o[(static_cast<int64_t>(p.slot) * a.slot_rows + r) * D + d] = acc[i][r];
          }
        }
      }
    }
    if (tid < p.nrows) {
      const int gr = p.row0 + tid, t = gr / a.G, g = gr - t * a.G;
      if (p.whole()) {
        if (a.lse) a.lse[(static_cast<int64_t>(p.b) * a.T + t) * a.Hq + p.h * a.G + g] = lse_of(sm[tid], sl[tid]);
      } else {
        a.part_ml[static_cast<int64_t>(p.slot) * a.slot_rows + tid] = make_float2(sm[tid], sl[tid]);
      }
    }
    __syncthreads();  // queries and statistics are rewritten by the next piece
    if (a.join_here && !p.whole()) {
      if (tid == 0) scratch[0] = last_of_item(a, p, rt);
      __syncthreads();
      if (scratch[0]) join_item<E>(a, p, rt, warp, kGenThreads / 32);
    }
  }
}

// The join kernel, for items of many rows and parts: a row (sequence, token, query
// head) is a CTA's, whose warps take every fourth part (the order of the sum is
// fixed too).
constexpr int kJoinWarps = 4;

template <typename E>
__global__ void __launch_bounds__(32 * kJoinWarps) spec_kv_join_kernel(const __grid_constant__ KvArgs a) {
  __shared__ __align__(16) float4 part_o[kJoinWarps][64];
  __shared__ float part_l[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = blockIdx.x;
  const int hq = static_cast<int>(row % a.Hq);
  const int64_t bt = row / a.Hq;
  const int b = static_cast<int>(bt / a.T), t = static_cast<int>(bt - static_cast<int64_t>(b) * a.T);
  start_dependents();
  wait_for_grid();  // the ranges' results are complete
  const SeqSpan s = seq_span(a, b);
  if (s.bad || t >= s.n) return;
  const int per = max(1, (a.prefix[a.B] + a.nranges - 1) / a.nranges);
  const int h = hq / a.G, g = hq - h * a.G;
  const int first = a.prefix[b] + h * s.places + a.overhead;
  const int c0 = first / per, c1 = (first + s.nt - 1) / per;
  if (c0 == c1) return;
  const int gr = t * a.G + g, rt = gr / a.rows, r = gr - rt * a.rows;
  float top;
  float4 acc[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
  float l = 0.0f;
  add_parts(a, rt, r, c0, c1, c0 + warp, kJoinWarps, top, acc, l);
#pragma unroll
  for (int k = 0; k < 2; ++k) part_o[warp][lane + 32 * k] = acc[k];
  if (lane == 0) part_l[warp] = l;
  __syncthreads();
  if (warp > 0) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) {
    l += part_l[w];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 x = part_o[w][lane + 32 * k];
      acc[k] = make_float4(acc[k].x + x.x, acc[k].y + x.y, acc[k].z + x.z, acc[k].w + x.w);
    }
  }
  store_row<E>(a, b, t, hq, acc, top, l);
}

}  // namespace spec_kv_detail
