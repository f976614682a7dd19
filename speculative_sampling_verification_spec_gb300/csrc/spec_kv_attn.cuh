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
// the matrix unit's truncated sums would not keep it).
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
        wl = exp2f(0.5f * (ml.x - top));
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float w = __shfl_sync(kFull, wl, i0 + i), li = __shfl_sync(kFull, ml.y, i0 + i);
        // a part without tokens for this row left no output
        if (i0 + i >= m || li == 0.0f) continue;
        // (references take in the values' scales, so a part far below the top may still have a large sum)
        l = fmaf(w, w * li, l);
        const float ww = w * w;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          acc[k].x = fmaf(ww, x[i][k].x, acc[k].x);
          acc[k].y = fmaf(ww, x[i][k].y, acc[k].y);
          acc[k].z = fmaf(ww, x[i][k].z, acc[k].z);
          acc[k].w = fmaf(ww, x[i][k].w, acc[k].w);
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

// sums over the 32 lanes of N = 8, 16 or 32 values each; lane r (mod N) gets value r's
template <int N>
__device__ __forceinline__ float lane_sums(float* v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 16; w >= N; w >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(kFull, v[i], w);
#pragma unroll
  for (int w = N / 2; w; w >>= 1) {
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const bool up = lane & w;
      const float keep = up ? v[i + w] : v[i], send = up ? v[i] : v[i + w];
      v[i] = keep + __shfl_xor_sync(kFull, send, w);
    }
  }
  return v[0];
}

constexpr int kGenThreads = 128, kGenWarps = kGenThreads / 32;
constexpr int kGenLogTile = 6;  // tokens of a tile: short, for latency
constexpr int kGenStep = 8;     // tokens of a warp's step; they share a page
constexpr int kGenMaxD = 256;

// Each warp walks the piece's tokens on its own, every fourth step of eight, with a
// softmax of its own; the four are added up at the end of the piece.  A lane holds
// CH consecutive channels of the queries, of the output, and of each token, whose
// codes it loads straight from the cache (a token's head is one coalesced load).
// Scores: a lane's share of four tokens times ROWS rows, summed over the lanes by
// halving, which leaves lane (row, token) with its score; weights go back to all
// lanes through shared memory.  The next step's codes are on their way meanwhile.
//
// Bound by the float units: a token and row cost 4 D / 32 multiply-adds a lane and
// about half as many instructions for the sums over lanes and the conversions (16
// sequences of 8000 tokens, 4 float32 rows a key/value head of 128 channels: 263 MB
// in 131 us; 8 of 4000 with 20 rows: 140 us).  An earlier form with keys and weights
// in shared memory took 299 and 293 us, bound by its reads.
//
// CH: 4 or 8, for head sizes up to 128 or 256; ROWS: rows of a row tile, 4 or 8.
// SINKS: first tokens may be seen beside the window, which costs the calls without
// them 2 to 6 % (16 sequences of 8000 as above 76.9 us for 72.7, 64 of up to 8192
// 328 for 310, 256 channels 60.4 for 58.8).
constexpr int gen_ctas_an_sm(int ch, int rows) { return ch == 8 ? 2 : rows == 4 ? 4 : 3; }

template <typename E, int CH, int ROWS, bool SINKS>
__global__ void __launch_bounds__(kGenThreads, gen_ctas_an_sm(CH, ROWS))
    spec_kv_attention_kernel(const __grid_constant__ KvArgs a) {
  constexpr int kWords = CH / 4;  // 32-bit words of codes a token and lane
  __shared__ RangePlan plan;
  __shared__ int scratch[kGenWarps];
  __shared__ __align__(16) float sp[kGenWarps][ROWS][4];  // weights of four tokens
  __shared__ __align__(16) float sf[kGenWarps][ROWS];     // what a step multiplies the sums by
  __shared__ float sm[kGenWarps][ROWS], sl[kGenWarps][ROWS];
  __shared__ __align__(16) float so[kGenWarps][ROWS][32 * CH];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int range = blockIdx.x / a.nrt, rt = blockIdx.x - range * a.nrt;
  start_dependents();
  wait_for_grid();
  make_plan_range<kGenThreads, SINKS>(a, range, &plan, scratch, blockIdx.x == 0 ? a.prefix : nullptr);
  fill_empty<E>(a, tid, kGenThreads);
  if (plan.w0 >= plan.w1) return;
  const int D = a.D, d0 = lane * CH;
  const bool mine = d0 < D;  // the lane has channels
  const int my_row = (lane >> 2) % ROWS, my_tok = lane & 3;
  Walk walk = walk_begin(plan, range, rt);
  Piece p;
  while (walk_next<SINKS>(a, walk, p)) {
    // The piece's tokens i without what is left out, `begin` to `end`; position_of: where they are.  They are counted
    // from 0, but from the first position on where 8 channels a lane leave no registers for that (256 channels without
    // sinks: 58.8 us for 59.5; 128 channels and 20 rows: 83.9 for 78.0).
    constexpr bool kFromZero = SINKS || CH == 4;
    const int skip = SINKS ? p.skip : 0, tile_at = p.tile0 << a.log_tile, j0 = kFromZero ? tile_at : 0;
    const int begin = tile_at - j0, near = p.near - j0, end = min(p.tile1 << a.log_tile, p.L + p.n - skip) - j0;
    const auto position_of = [&](int i) { return j0 + i + (SINKS && i >= near ? skip : 0); };
    float q[ROWS][CH], acc[ROWS][CH];  // queries in log2 units; zero past the last row and channel
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const int gr = p.row0 + r, t = gr / a.G, g = gr - t * a.G;
      const E* src = static_cast<const E*>(a.q) + p.b * a.q_seq + t * a.q_tok + (p.h * a.G + g) * a.q_head + d0;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        q[r][c] = mine && r < p.nrows ? to_float(src[c]) * a.scale2 : 0.0f;
        acc[r][c] = 0.0f;
      }
    }
    // positions that every row sees, and the lane's row's
    const int all_from = a.window > 0 ? p.L + (p.row0 + p.nrows - 1) / a.G - a.window + 1 : 0;
    const int all_to = p.L + p.row0 / a.G;
    const int pos = my_row < p.nrows ? p.L + (p.row0 + my_row) / a.G : -1;
    const int low = a.window > 0 ? pos - a.window : -1;  // sees positions in (low, pos]
    float m = kNoRef, l = 0.0f;

    uint32_t kc[kGenStep][kWords], vc[kGenStep][kWords];
    float ks, vs;
    const auto number = [&](int i) { return i < end ? page_of(a, p.b, position_of(i) >> a.log_page) : 0; };
    const auto fetch = [&](int i, int page) {
      ks = vs = __uint_as_float(0x7fc00000u);  // a page that is not the pool's, or, with sinks, tokens that no row sees
      const int base = position_of(i);
      const bool want = i < end && (!SINKS || piece_sees(a, p, base, base + kGenStep)), ok = want && page >= 0;
      if (want && page < 0 && lane == 0 && piece_sees<SINKS>(a, p, base, ((base >> a.log_page) + 1) << a.log_page))
        report(a.status, SPEC_ERR_CACHE_RANGE);
      if (ok) {
        const int64_t at = page * a.scale_page_stride + p.h * a.scale_head_stride;
        ks = a.k_scale[at];
        vs = a.v_scale[at];
      }
      const int64_t row = page * a.page_stride + p.h * a.head_stride +
                          (base & ((1 << a.log_page) - 1)) * a.token_stride + d0;
#pragma unroll
      for (int t = 0; t < kGenStep; ++t) {
        const bool get = ok && mine && i + t < end;
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          kc[t][w] = get ? *reinterpret_cast<const uint32_t*>(a.k_codes + row + t * a.token_stride + 4 * w) : 0u;
          vc[t][w] = get ? *reinterpret_cast<const uint32_t*>(a.v_codes + row + t * a.token_stride + 4 * w) : 0u;
        }
      }
    };
    constexpr int kStride = kGenStep * kGenWarps;
    int i = begin + warp * kGenStep;
    int page = number(i), next_page = number(i + kStride);
    if (i < end) fetch(i, page);
    for (; i < end; i += kStride) {
      const int base = position_of(i);
      float kf[kGenStep][CH];
      uint32_t vnow[kGenStep][kWords];
      const float ks_now = ks, vs_now = vs;
#pragma unroll
      for (int t = 0; t < kGenStep; ++t) {
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          const float2 lo = codes2_to_float2(static_cast<uint16_t>(kc[t][w] & 0xffffu));
          const float2 hi = codes2_to_float2(static_cast<uint16_t>(kc[t][w] >> 16));
          kf[t][4 * w] = lo.x;
          kf[t][4 * w + 1] = lo.y;
          kf[t][4 * w + 2] = hi.x;
          kf[t][4 * w + 3] = hi.y;
          vnow[t][w] = vc[t][w];
        }
      }
      page = next_page;
      next_page = number(i + 2 * kStride);
      if (i + kStride < end) fetch(i + kStride, page);
      const bool all = (base >= all_from || (SINKS && base + kGenStep <= a.sinks)) && base + kGenStep - 1 <= all_to;
#pragma unroll
      for (int t0 = 0; t0 < kGenStep; t0 += 4) {
        float s[ROWS * 4];
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            float x = q[r][0] * kf[t0 + t][0];
#pragma unroll
            for (int c = 1; c < CH; ++c) x = fmaf(q[r][c], kf[t0 + t][c], x);
            s[r * 4 + t] = x;
          }
        }
        const float score = lane_sums<ROWS * 4>(s) * ks_now;
        const int j = base + t0 + my_tok;
        const bool see = j <= pos && (j > low || (SINKS && j < a.sinks));  // (positions past the last are past every row's own)
        const float x = see ? score : -INFINITY;
        float top = fmaxf(x, __shfl_xor_sync(kFull, x, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        const float mn = fmaxf(m, top), f = ex2(m - mn), w = ex2(x - mn);
        m = mn;
        l = fmaf(l, f, w);  // this lane's tokens' share of the sum
        const bool raised = __any_sync(kFull, f != 1.0f);
        __syncwarp();  // the weights before have been read
        if (lane < ROWS * 4) {
          sp[warp][my_row][my_tok] = see ? w * vs_now : -0.0f;  // -0: not seen
          if (my_tok == 0) sf[warp][my_row] = f;
        }
        __syncwarp();
        float v[4][CH];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
          for (int e = 0; e < kWords; ++e) {
            const float2 lo = codes2_to_float2(static_cast<uint16_t>(vnow[t0 + t][e] & 0xffffu));
            const float2 hi = codes2_to_float2(static_cast<uint16_t>(vnow[t0 + t][e] >> 16));
            v[t][4 * e] = lo.x;
            v[t][4 * e + 1] = lo.y;
            v[t][4 * e + 2] = hi.x;
            v[t][4 * e + 3] = hi.y;
          }
        }
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          if (raised) {
            const float fr = sf[warp][r];
#pragma unroll
            for (int c = 0; c < CH; ++c) acc[r][c] *= fr;
          }
          const float4 w4 = *reinterpret_cast<const float4*>(sp[warp][r]);
          const float wr[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            // a token that the row does not see adds nothing, whatever its slot holds
            if (!all && __float_as_uint(wr[t]) == 0x80000000u) continue;
#pragma unroll
            for (int c = 0; c < CH; ++c) acc[r][c] = fmaf(wr[t], v[t][c], acc[r][c]);
          }
        }
      }
    }
    // the four warps' results: references and sums, then outputs
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    if (my_tok == 0 && lane < ROWS * 4) {
      sm[warp][my_row] = m;
      sl[warp][my_row] = l;
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int c = 0; c < CH; c += 4)
        *reinterpret_cast<float4*>(&so[warp][r][d0 + c]) =
            make_float4(acc[r][c], acc[r][c + 1], acc[r][c + 2], acc[r][c + 3]);
    __syncthreads();
    for (int r = warp; r < p.nrows; r += kGenWarps) {
      float top = sm[0][r];
#pragma unroll
      for (int w = 1; w < kGenWarps; ++w) top = fmaxf(top, sm[w][r]);
      float sum = 0.0f, o[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) o[c] = 0.0f;
#pragma unroll
      for (int w = 0; w < kGenWarps; ++w) {
        const float f = ex2(sm[w][r] - top), lw = sl[w][r];
        if (lw == 0.0f) continue;  // no tokens for this row
        sum = fmaf(f, lw, sum);
#pragma unroll
        for (int c = 0; c < CH; ++c) o[c] = fmaf(f, so[w][r][d0 + c], o[c]);
      }
      const int gr = p.row0 + r, t = gr / a.G, g = gr - t * a.G;
      if (p.whole()) {
        const float inv = 1.0f / sum;
        E* out = static_cast<E*>(a.out) + p.b * a.o_seq + t * a.o_tok + (p.h * a.G + g) * a.o_head + d0;
#pragma unroll
        for (int c = 0; c < CH; c += 4)
          if (mine) store4(a, out + c, make_float4(o[c] * inv, o[c + 1] * inv, o[c + 2] * inv, o[c + 3] * inv));
        if (lane == 0 && a.lse) a.lse[(static_cast<int64_t>(p.b) * a.T + t) * a.Hq + p.h * a.G + g] = lse_of(top, sum);
      } else {
        const int64_t at = static_cast<int64_t>(p.slot) * a.slot_rows + r;
#pragma unroll
        for (int c = 0; c < CH; c += 4)
          if (mine) *reinterpret_cast<float4*>(a.part_o + at * D + d0 + c) = make_float4(o[c], o[c + 1], o[c + 2], o[c + 3]);
        if (lane == 0) a.part_ml[at] = make_float2(top, sum);
      }
    }
    __syncthreads();  // the results' places are used again
    if (a.join_here && !p.whole()) {
      if (tid == 0) scratch[0] = last_of_item(a, p, rt);
      __syncthreads();
      if (scratch[0]) join_item<E>(a, p, rt, warp, kGenWarps);
      __syncthreads();
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
