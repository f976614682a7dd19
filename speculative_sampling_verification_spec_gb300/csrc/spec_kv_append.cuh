#pragma once
// spec_kv_append.cuh -- rotate the new tokens' queries and keys, store keys and
// values in the paged 8-bit cache.
//
// A unit is what one call writes to one (page, key/value head) of the keys or of
// the values: at most page_size tokens.  Its scale depends on all of them (the
// largest magnitude), so a unit is read, rotated and kept in registers, reduced,
// and only then written as codes: one pass over the inputs.  A unit with few
// elements is a warp's, a larger one a CTA's.  The queries need no reduction and
// go to CTAs of their own at the end of the grid.
//
// A thread handles chunks of PC rotation pairs, 2 * PC channels: PC = 8 moves 16
// bytes at a time and more where everything is aligned, PC = 1 single channels.
#include "spec_kv_common.cuh"

namespace spec_kv_detail {

struct AppendArgs {
  KvArgs a;
  const void* k;
  const void* v;
  const float* cos_sin;
  int64_t k_seq, k_tok, k_head, v_seq, v_tok, v_head;
  int32_t rot, rot_len, interleaved;
  int32_t units_page;    // pages a sequence can touch in this call
  int32_t unit_blocks;   // blocks that take units; the rest take queries
  int32_t units;         // B * units_page * Hkv * 2
  int32_t q_rows_block;  // (sequence, token) rows a query block takes
};

template <typename E, int N>
__device__ __forceinline__ void load_n(const E* p, float* x) {
  if constexpr (N == 1) {
    x[0] = to_float(*p);
  } else if constexpr (sizeof(E) == 2) {
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 r = reinterpret_cast<const float4*>(p)[i];
      x[4 * i] = r.x;
      x[4 * i + 1] = r.y;
      x[4 * i + 2] = r.z;
      x[4 * i + 3] = r.w;
    }
  }
}

template <typename E, int N>
__device__ __forceinline__ void store_n(E* p, const float* x) {
  if constexpr (N == 1) {
    from_float(x[0], p);
  } else if constexpr (sizeof(E) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}

// Channels of chunk c: the first PC from `lo` and the second PC from `hi`, as
// pairs (lo + i, hi + i) or, adjacent, (lo + 2i, lo + 2i + 1) over both.
struct ChunkAt {
  int lo, hi, angle;  // angle: the first pair's index
  bool turn;          // the chunk is rotated
};
template <int PC>
__device__ __forceinline__ ChunkAt chunk_at(const AppendArgs& g, int c) {
  ChunkAt k;
  const int half = g.rot >> 1, p = c * PC;
  k.turn = p < half;
  k.angle = p;
  if (k.turn && !g.interleaved) {
    k.lo = p;
    k.hi = p + half;
  } else {
    k.lo = 2 * p;
    k.hi = 2 * p + PC;
  }
  return k;
}

// The values of a chunk in the order lo.., hi.., rotated where `turn`.  Products
// and sums are rounded one by one, so the result does not depend on contraction.
template <typename E, int PC>
__device__ __forceinline__ void load_chunk(const AppendArgs& g, const E* row, const float* cs, const ChunkAt& k,
                                           float* y) {
  load_n<E, PC>(row + k.lo, y);
  load_n<E, PC>(row + k.hi, y + PC);
  if (!cs || !k.turn) return;
  float co[PC], si[PC];
  load_n<float, PC>(cs + k.angle, co);
  load_n<float, PC>(cs + (g.rot >> 1) + k.angle, si);
#pragma unroll
  for (int i = 0; i < PC; ++i) {
    // both forms are spelled out, so that the indices are constants
    const float x1 = g.interleaved ? y[2 * i] : y[i], x2 = g.interleaved ? y[2 * i + 1] : y[PC + i];
    const float a = __fsub_rn(__fmul_rn(x1, co[i]), __fmul_rn(x2, si[i]));
    const float b = __fadd_rn(__fmul_rn(x2, co[i]), __fmul_rn(x1, si[i]));
    if (g.interleaved) {
      y[2 * i] = a;
      y[2 * i + 1] = b;
    } else {
      y[i] = a;
      y[PC + i] = b;
    }
  }
}

__device__ __forceinline__ bool is_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// 2^e, e the least integer >= kMinScaleExp with amax <= 448 * 2^e (448 = 1.75 * 2^8,
// the largest e4m3 value): from the exponent and mantissa fields, with no rounding
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, kMinScaleExp);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// x / scale, through the reciprocal where that is exact (powers of two)
struct Divider {
  float scale, inv;
  bool exact;
  __device__ __forceinline__ explicit Divider(float s) : scale(s) {
    exact = (__float_as_uint(s) & 0x7fffffu) == 0 && s > 1e-37f && s < 1e37f;
    inv = exact ? 1.0f / s : 0.0f;
  }
  __device__ __forceinline__ float operator()(float x) const { return exact ? x * inv : __fdiv_rn(x, scale); }
};

// two floats -> two e4m3 codes (low byte first); infinities become NaN codes
__device__ __forceinline__ uint32_t to_codes2(float x, float y) {
  if (!is_finite(x)) x = __uint_as_float(0x7fc00000u);
  if (!is_finite(y)) y = __uint_as_float(0x7fc00000u);
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* x, const Divider& d) {
  if constexpr (N == 1) {
    *p = static_cast<uint8_t>(to_codes2(d(x[0]), 0.0f) & 0xffu);
  } else {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = to_codes2(d(x[4 * i]), d(x[4 * i + 1])) | (to_codes2(d(x[4 * i + 2]), d(x[4 * i + 3])) << 16);
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// lengths of sequence b against this call's limits
__device__ __forceinline__ bool append_span(const AppendArgs& g, int b, int* L, int* n) {
  const KvArgs& a = g.a;
  *L = a.seq_lens[b];
  *n = a.new_lens ? a.new_lens[b] : a.T;
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.log_page;
  const int64_t end = static_cast<int64_t>(*L) + *n;
  return !(*L < 0 || *n < 0 || *n > a.T || end > cap || (g.rot > 0 && *n > 0 && end > g.rot_len));
}

// ITER chunks a thread are kept in registers; a unit with more is read twice.
constexpr int kAppendIter = 4;

template <typename E, int PC, bool WARP>
__device__ __forceinline__ void append_unit(const AppendArgs& g, int unit, int t, int nt, float* red) {
  const KvArgs& a = g.a;
  const int kv = unit & 1;
  int u = unit >> 1;
  const int h = u % a.Hkv;
  u /= a.Hkv;
  const int pg = u % g.units_page, b = u / g.units_page;
  int L, n;
  if (!append_span(g, b, &L, &n)) {
    if (t == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
    return;
  }
  const int S = 1 << a.log_page;
  const int pi = (L >> a.log_page) + pg;  // page of the sequence
  const int p0 = max(L, pi << a.log_page), p1 = min(L + n, (pi + 1) << a.log_page);
  if (p0 >= p1) return;
  const int page = page_of(a, b, pi);
  if (page < 0) {
    if (t == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
    return;
  }
  const E* x = static_cast<const E*>(kv ? g.v : g.k) + b * (kv ? g.v_seq : g.k_seq) + h * (kv ? g.v_head : g.k_head);
  const int64_t x_tok = kv ? g.v_tok : g.k_tok;
  uint8_t* codes = (kv ? a.v_codes : a.k_codes) + page * a.page_stride + h * a.head_stride;
  float* sp = (kv ? a.v_scale : a.k_scale) + page * a.scale_page_stride + h * a.scale_head_stride;
  const int kept = p0 & (S - 1);  // earlier tokens of the sequence in this page
  const float before = kept ? *sp : 0.0f;
  const int per_tok = a.D / (2 * PC), total = (p1 - p0) * per_tok;
  const bool turn = !kv && g.rot > 0;
  const bool hold = total <= kAppendIter * nt;
  float y[kAppendIter][2 * PC];
  float amax = 0.0f;
  for (int base = 0; base < total; base += kAppendIter * nt) {
#pragma unroll
    for (int it = 0; it < kAppendIter; ++it) {
      const int i = base + it * nt + t;
      if (i < total) {
        const int tok = i / per_tok, c = i - tok * per_tok;
        const ChunkAt at = chunk_at<PC>(g, c);
        load_chunk<E, PC>(g, x + (p0 - L + tok) * x_tok, turn ? g.cos_sin + static_cast<int64_t>(p0 + tok) * g.rot : nullptr,
                          at, y[it]);
#pragma unroll
        for (int j = 0; j < 2 * PC; ++j) {
          const float m = fabsf(y[it][j]);
          amax = (is_finite(m) && m > amax) ? m : amax;
        }
      }
    }
  }
  // magnitudes are not negative: their bit patterns order them
  uint32_t bits = __reduce_max_sync(kFull, __float_as_uint(amax));
  if constexpr (!WARP) {
    if ((t & 31) == 0) red[t >> 5] = __uint_as_float(bits);
    __syncthreads();
    for (int w = 0; w < nt / 32; ++w) bits = max(bits, __float_as_uint(red[w]));
  }
  const float need = scale_for(__uint_as_float(bits));
  const float scale = before >= need ? before : need;
  if (kept && scale != before) {
    // the page's earlier codes at the grown scale
    const float f = before / scale;
    const int vec = a.D / 16;
    for (int i = t; i < kept * vec; i += nt) {
      const int tok = i / vec, c = i - tok * vec;
      uint4* p = reinterpret_cast<uint4*>(codes + tok * a.token_stride + c * 16);
      uint4 r = *p;
      uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 lo = codes2_to_float2(static_cast<uint16_t>(w[j] & 0xffffu));
        const float2 hi = codes2_to_float2(static_cast<uint16_t>(w[j] >> 16));
        w[j] = to_codes2(lo.x * f, lo.y * f) | (to_codes2(hi.x * f, hi.y * f) << 16);
      }
      *p = r;
    }
  }
  if (t == 0 && !(scale == before)) *sp = scale;
  const Divider div(scale);
  for (int base = 0; base < total; base += kAppendIter * nt) {
#pragma unroll
    for (int it = 0; it < kAppendIter; ++it) {
      const int i = base + it * nt + t;
      if (i < total) {
        const int tok = i / per_tok, c = i - tok * per_tok;
        const ChunkAt at = chunk_at<PC>(g, c);
        if (!hold)
          load_chunk<E, PC>(g, x + (p0 - L + tok) * x_tok,
                            turn ? g.cos_sin + static_cast<int64_t>(p0 + tok) * g.rot : nullptr, at, y[it]);
        uint8_t* dst = codes + ((p0 + tok) & (S - 1)) * a.token_stride;
        store_codes<PC>(dst + at.lo, y[it], div);
        store_codes<PC>(dst + at.hi, y[it] + PC, div);
      }
    }
  }
}

constexpr int kAppendWarpThreads = 128;  // units of a warp: four a CTA
constexpr int kAppendCtaThreads = 256;   // units of a CTA

template <typename E, int PC, bool WARP>
__global__ void __launch_bounds__(WARP ? kAppendWarpThreads : kAppendCtaThreads)
    spec_kv_append_kernel(const __grid_constant__ AppendArgs g) {
  const KvArgs& a = g.a;
  const int tid = threadIdx.x;
  if (blockIdx.x < static_cast<unsigned>(g.unit_blocks)) {
    __shared__ float red[WARP ? 1 : kAppendCtaThreads / 32];
    if constexpr (WARP) {
      const int unit = blockIdx.x * (kAppendWarpThreads / 32) + (tid >> 5);
      if (unit < g.units) append_unit<E, PC, true>(g, unit, tid & 31, 32, red);
    } else {
      append_unit<E, PC, false>(g, blockIdx.x, tid, kAppendCtaThreads, red);
    }
    return;
  }
  // queries
  const int per_tok = a.D / (2 * PC), per_row = a.Hq * per_tok;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x - g.unit_blocks) * g.q_rows_block;
  const int64_t nrows = static_cast<int64_t>(a.B) * a.T;
  for (int i = tid; i < g.q_rows_block * per_row; i += blockDim.x) {
    const int r = i / per_row, j = i - r * per_row;
    const int64_t row = row0 + r;
    if (row >= nrows) break;
    const int b = static_cast<int>(row / a.T), tok = static_cast<int>(row - static_cast<int64_t>(b) * a.T);
    const int h = j / per_tok, c = j - h * per_tok;
    int L, n;
    const bool ok = append_span(g, b, &L, &n);
    float y[2 * PC];
    const ChunkAt at = chunk_at<PC>(g, c);
    if (!ok || tok >= n) {
      const float fill = ok ? 0.0f : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int e = 0; e < 2 * PC; ++e) y[e] = fill;
      if (!ok && i == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
    } else {
      load_chunk<E, PC>(g, static_cast<const E*>(a.q) + b * a.q_seq + tok * a.q_tok + h * a.q_head,
                        g.rot > 0 ? g.cos_sin + static_cast<int64_t>(L + tok) * g.rot : nullptr, at, y);
    }
    E* o = static_cast<E*>(a.out) + b * a.o_seq + tok * a.o_tok + h * a.o_head;
    store_n<E, PC>(o + at.lo, y);
    store_n<E, PC>(o + at.hi, y + PC);
  }
}

}  // namespace spec_kv_detail
