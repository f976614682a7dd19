#pragma once
// spec_kv_append.cuh -- normalise each head of the new tokens' queries and keys where
// that is asked for, rotate them, store keys and values in the paged 8-bit cache.
//
// A unit is what one call writes to one (page, key/value head) of the keys or of
// the values: at most page_size tokens.  Its scale depends on all of them (the
// largest magnitude), so a unit is read, kept in registers, reduced,
// and only then written as codes: one pass over the inputs.  What is kept is the
// input as it came (half the registers in bfloat16, so twice as much is under
// way); keys are rotated once for the largest magnitude and again for the codes.  A unit with few
// elements is a warp's, a larger one a CTA's; where there are many, a warp or CTA
// takes several of one page.  The queries need no reduction and go to CTAs of
// their own at the end of the grid.
//
// Prompts are bound by memory and by the instructions of the conversions about
// alike: 8 sequences of up to 4096 new tokens (32 query and 8 key/value heads of
// 128 channels, 20 480 tokens; 472 MB, and 101 MB of zeros in empty query slots)
// take 105 us, 5.5 TB/s; with norms of queries and keys 137.  Few tokens are bound by the chain lengths - page - scale:
// 3 us, with norms 5.
//
// A thread handles chunks of PC rotation pairs, 2 * PC channels: PC = 8 moves 16
// bytes at a time and more where everything is aligned, PC = 1 single channels.
//
// Norms.  r = 1 / sqrt(mean x^2 + eps) of a head goes to the keys' scales and codes
// through comparisons and roundings, so it is made a function of the inputs alone: the
// sum of the squares and its root are carried in two floats (some 40 bits), and r is the
// nearest float but for one head in a hundred thousand.  (In 64 bits the sums of a prompt alone
// would take longer than the rest: the chip's rate of such multiply-adds is a hundredth
// of that in 32.)  The threads of a head are a power of two of neighbouring lanes, the
// last of them idle where its chunks are not, and add up by exchanging; with PC = 1 a
// warp first takes the norms of a unit's tokens, and a whole head of a query.  Prompts
// with norms are bound by latency: the heads of a thread need 128 registers, which leaves
// 16 warps an SM (with sums in chains of two-float additions, head after head, 172 us; all
// heads' sums side by side 150, weights kept 145, angles asked for before the sums and the
// next rows ahead 137).
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
  int32_t group_units;   // units of a group: a warp's or a CTA's
  int32_t groups_page;   // groups of a page's 2 * Hkv units
  int32_t groups;        // B * units_page * groups_page
  int32_t unit_blocks;   // blocks that take groups; the rest take queries
  int32_t q_rows_block;  // (sequence, token) rows a query block takes
  int32_t q_heads;       // heads a query thread takes: 1 or kAppendHeads
  float one;             // 1
  int32_t tok_threads;   // threads of a token's head: its chunks, or the power of two above
  // norms: weights (NULL: not normalised), and D * eps and sqrt(D) as sums of two floats
  const float* q_weight;
  const float* k_weight;
  int64_t q_weight_head, k_weight_head;
  float eps_hi, eps_lo, root_hi, root_lo;
  float bias;         // see squares
  int32_t least_exp;  // of what sums of squares are scaled by: below, the squares are nothing beside eps
};

// N consecutive elements as they are in memory: 8 of them in 16-byte words, or one
template <typename E, int N>
struct Raw {
  uint4 w[sizeof(E) * N / 16 > 0 ? sizeof(E) * N / 16 : 1];
  __device__ __forceinline__ void load(const E* p) {
    if constexpr (N == 1) {
      w[0].x = __float_as_uint(to_float(*p));
    } else {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(E) * N / 16); ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    }
  }
  // the largest magnitude, NaN aside
  __device__ __forceinline__ float top() const {
    if constexpr (N > 1 && sizeof(E) == 2) {
      const auto two = [](uint32_t u) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&u)); };
      const __nv_bfloat162 m = __hmax2(__hmax2(two(w[0].x), two(w[0].y)), __hmax2(two(w[0].z), two(w[0].w)));
      return fmaxf(__low2float(m), __high2float(m));
    } else {
      float x[N], m = 0.0f;
      values(x);
#pragma unroll
      for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(x[i]));
      return m;
    }
  }
  __device__ __forceinline__ void values(float* x) const {
    if constexpr (N == 1) {
      x[0] = __uint_as_float(w[0].x);
    } else if constexpr (sizeof(E) == 2) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 4; ++i) {
        x[4 * i] = __uint_as_float(w[i].x);
        x[4 * i + 1] = __uint_as_float(w[i].y);
        x[4 * i + 2] = __uint_as_float(w[i].z);
        x[4 * i + 3] = __uint_as_float(w[i].w);
      }
    }
  }
};
template <typename E, int N>
__device__ __forceinline__ void load_n(const E* p, float* x) {
  Raw<E, N> r;
  r.load(p);
  r.values(x);
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

// (x1, x2) rotated by an angle; products and sums are rounded one by one, so the
// result does not depend on contraction.
__device__ __forceinline__ void turn(float& x1, float& x2, float co, float si) {
  const float a = __fsub_rn(__fmul_rn(x1, co), __fmul_rn(x2, si));
  const float b = __fadd_rn(__fmul_rn(x2, co), __fmul_rn(x1, si));
  x1 = a;
  x2 = b;
}

// A chunk as it is in memory, and its values in the order lo.., hi..
template <typename E, int PC>
struct RawChunk {
  Raw<E, PC> lo, hi;
  __device__ __forceinline__ void load(const E* row, const ChunkAt& k) {
    lo.load(row + k.lo);
    hi.load(row + k.hi);
  }
  __device__ __forceinline__ float top() const {
    return fmaxf(lo.top(), hi.top());
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (uint4& u : lo.w) u = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (uint4& u : hi.w) u = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float* y) const {
    lo.values(y);
    hi.values(y + PC);
  }
};
// The cosines and sines of a chunk's pairs, from the position's row of them, and
// the rotation of a chunk.
template <int PC>
struct Angles {
  float co[PC], si[PC];
  __device__ __forceinline__ Angles(const AppendArgs& g, const float* cs, const ChunkAt& k) {
    if (!k.turn) return;
    load_n<float, PC>(cs + k.angle, co);
    load_n<float, PC>(cs + (g.rot >> 1) + k.angle, si);
  }
  __device__ __forceinline__ void turn_all(const AppendArgs& g, const ChunkAt& k, float* y) const {
    if (!k.turn) return;
    if (g.interleaved) {
#pragma unroll
      for (int i = 0; i < PC; ++i) turn(y[2 * i], y[2 * i + 1], co[i], si[i]);
    } else {
      if constexpr (PC == 1) {
        turn(y[0], y[1], co[0], si[0]);
      } else {
        // Two pairs at a time, rounded alike.  The sums are written as multiplications by a 1 that the assembler
        // does not know: a plain packed addition of a packed product it makes one operation, with one rounding.
        const u64 plus = pack2(g.one, g.one), minus = pack2(-g.one, -g.one);
#pragma unroll
        for (int i = 0; i < PC; i += 2) {
          const u64 a = pack2(y[i], y[i + 1]), b = pack2(y[PC + i], y[PC + i + 1]);
          const u64 c = pack2(co[i], co[i + 1]), d = pack2(si[i], si[i + 1]);
          unpack2(fma2(mul2(b, d), minus, mul2(a, c)), y[i], y[i + 1]);
          unpack2(fma2(mul2(a, d), plus, mul2(b, c)), y[PC + i], y[PC + i + 1]);
        }
      }
    }
  }
};
template <int PC>
__device__ __forceinline__ void turn_chunk(const AppendArgs& g, const float* cs, const ChunkAt& k, float* y) {
  const Angles<PC> at(g, cs, k);
  at.turn_all(g, k, y);
}

__device__ __forceinline__ bool is_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

// The sum of the squares of a head's channels, times the square of a power of two f that brings the largest to [1, 2):
// hi + lo.  A lane runs two sums side by side, of every second square, each on top of a bias, 2 D or the power of two above
// (32 at least), which neither reaches (8 squares below 4 at most): every addition leaves a multiple of the bias's last
// place in the sum, exactly, and the rest of the square, all but exactly, for a second sum of small numbers.  The multiples
// of all lanes add up exactly, too.
struct Squares {
  float hi, lo, f;
};

// Of R heads whose channels lie with `threads` neighbouring lanes (a power of two), N each: values(r, y) gives the
// lane's, top(r) the largest magnitude among them (NaN aside, which comes up in the sum).  Step by step for all heads,
// whose chains run side by side.
template <int N, int R, typename Values, typename Top>
__device__ __forceinline__ void squares(const AppendArgs& g, const Values& values, const Top& top, unsigned mask,
                                        int threads, Squares* a) {
  float m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) m[r] = top(r);
  for (int d = threads >> 1; d; d >>= 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) m[r] = fmaxf(m[r], __shfl_xor_sync(mask, m[r], d));
  }
  const u64 minus = pack2(-1.0f, -1.0f), bias = pack2(g.bias, g.bias);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int e = min(max(static_cast<int>(__float_as_uint(m[r]) >> 23), g.least_exp), 253);
    a[r].f = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    const u64 f = pack2(a[r].f, a[r].f);
    u64 sum = bias, rest = pack2(0.0f, 0.0f);
    float x[N];
    values(r, x);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const u64 y = mul2(pack2(x[i], x[i + 1]), f), next = fma2(y, y, sum);
      const u64 taken = fma2(next, minus, sum);  // less what the sum has grown by
      rest = add2(rest, fma2(y, y, taken));
      sum = next;
    }
    sum = fma2(bias, minus, sum);
    float b1, c1;
    unpack2(sum, a[r].hi, b1);
    unpack2(rest, a[r].lo, c1);
    a[r].hi += b1;
    a[r].lo += c1;
  }
  for (int d = threads >> 1; d; d >>= 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      a[r].hi += __shfl_xor_sync(mask, a[r].hi, d);
      a[r].lo += __shfl_xor_sync(mask, a[r].lo, d);
    }
  }
}

// sqrt(D) / sqrt(sum + D eps), to the nearest float: an approximate root and one step of Newton's in two floats.
__device__ __forceinline__ float norm_of(const AppendArgs& g, const Squares& a) {
  const float eps = g.eps_hi * a.f * a.f, u = __fadd_rn(a.hi, eps);
  const float b = __fsub_rn(u, a.hi);  // u's own rounding: (hi - (u - b)) + (eps - b)
  const float lost = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(u, b)), __fsub_rn(eps, b));
  const float ul = __fadd_rn(__fadd_rn(lost, a.lo), g.eps_lo * a.f * a.f);
  const float r = rsqrtf(__fadd_rn(u, ul));
  const float q = __fmul_rn(r, r), ql = fmaf(r, r, -q);
  const float p = __fmul_rn(u, q), pl = fmaf(ul, q, fmaf(u, ql, fmaf(u, q, -p)));
  const float step = __fmul_rn(__fmul_rn(0.5f, r), __fsub_rn(__fsub_rn(1.0f, p), pl));
  const float m = __fmul_rn(r, g.root_hi);
  const float n = __fadd_rn(m, fmaf(step, g.root_hi, fmaf(r, g.root_lo, fmaf(r, g.root_hi, -m))));
  // infinities: 0; NaN
  return a.hi < INFINITY ? n * a.f : a.hi > 0.0f ? 0.0f : a.hi;
}

// The lanes that share a head.
__device__ __forceinline__ unsigned lanes_of(int threads) {
  const unsigned lane = threadIdx.x & 31;
  return threads == 32 ? kFull : ((1u << threads) - 1) << (lane & ~(threads - 1u));
}

// The norm factors of R heads at once, whose chunks are raw[0] .. raw[R - 1]: with as many lanes to a head, each takes
// one of the roots.
template <int R, typename E, int PC>
__device__ __forceinline__ void norms_of(const AppendArgs& g, const RawChunk<E, PC>* raw, float* r, int threads) {
  const unsigned mask = lanes_of(threads);
  Squares a[R];
  squares<2 * PC, R>(
      g, [&](int k, float* y) { raw[k].values(y); }, [&](int k) { return raw[k].top(); }, mask, threads, a);
  if (R == 4 && threads >= 4) {
    const int mine = threadIdx.x & 3;
    Squares b = a[0];
#pragma unroll
    for (int k = 1; k < R; ++k) {
      b.hi = mine == k ? a[k].hi : b.hi;
      b.lo = mine == k ? a[k].lo : b.lo;
      b.f = mine == k ? a[k].f : b.f;
    }
    const float n = norm_of(g, b);
#pragma unroll
    for (int k = 0; k < R; ++k) r[k] = __shfl_sync(mask, n, ((threadIdx.x & 31) & ~3u) + k);
  } else {
#pragma unroll
    for (int k = 0; k < R; ++k) r[k] = norm_of(g, a[k]);
  }
}

// The weights of a chunk, and its normalised values: (x r) w, each product rounded.
template <int PC>
struct Weights {
  float w[2 * PC];
  __device__ __forceinline__ void load(const float* weight, const ChunkAt& k) {
    load_n<float, PC>(weight + k.lo, w);
    load_n<float, PC>(weight + k.hi, w + PC);
  }
  __device__ __forceinline__ void scale(float* y, float r) const {
    const u64 r2 = pack2(r, r);
#pragma unroll
    for (int i = 0; i < 2 * PC; i += 2)
      unpack2(mul2(mul2(pack2(y[i], y[i + 1]), r2), pack2(w[i], w[i + 1])), y[i], y[i + 1]);
  }
};

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

// two floats -> two e4m3 codes (low byte first)
__device__ __forceinline__ uint32_t to_codes2(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// infinities have no code (the conversion would take the largest one): NaN
__device__ __forceinline__ float no_infinity(float x) { return is_finite(x) ? x : __uint_as_float(0x7fc00000u); }

// N values of a chunk's half as codes: `plain`, all are finite and the scale is a power of two
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* x, const Divider& d, bool plain) {
  if constexpr (N == 1) {
    *p = static_cast<uint8_t>(to_codes2(no_infinity(d(x[0])), 0.0f) & 0xffu);
  } else {
    uint32_t w[2];
    if (plain) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = to_codes2(x[4 * i] * d.inv, x[4 * i + 1] * d.inv) |
               (to_codes2(x[4 * i + 2] * d.inv, x[4 * i + 3] * d.inv) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[i] = to_codes2(no_infinity(d(x[4 * i])), no_infinity(d(x[4 * i + 1]))) |
               (to_codes2(no_infinity(d(x[4 * i + 2])), no_infinity(d(x[4 * i + 3]))) << 16);
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// The norm factor of a head by a whole warp, straight from memory.
template <typename E>
__device__ __forceinline__ float row_norm(const AppendArgs& g, const E* x) {
  float y[8];  // channels lane, lane + 32, ... of at most 256
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = (threadIdx.x & 31) + 32 * i;
    y[i] = d < g.a.D ? to_float(x[d]) : 0.0f;
  }
  Squares a;
  squares<8, 1>(
      g, [&](int, float* z) { for (int i = 0; i < 8; ++i) z[i] = y[i]; },
      [&](int) {
        float m = 0.0f;
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));
        return m;
      },
      kFull, 32, &a);
  return norm_of(g, a);
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

// Threads of a CTA, and chunks a thread keeps in registers (a unit with more is
// read twice): units of a warp, four a CTA; units of a CTA.
constexpr int kAppendWarpThreads = 128, kAppendWarpIter = 4;
constexpr int kAppendCtaThreads = 256, kAppendCtas = 3;  // CTAs an SM
template <typename E>
constexpr int kAppendCtaIter = sizeof(E) == 2 ? 4 : 2;
// Heads a query thread turns by one load of a position's angles, where the call is
// large; chunks it has under way at once, and rows it takes in all.
constexpr int kAppendHeads = 4, kAppendQueryRows = 16;
constexpr int kMostSlots = 128;  // of a page

// A group of units: `units` consecutive (head, keys or values) of one page of a
// sequence, by a warp or a CTA.  What they share is worked out once.
template <typename E, int PC, bool WARP, bool NORM>
__device__ __forceinline__ void append_group(const AppendArgs& g, int group, int t, uint32_t* red, float* norms) {
  constexpr int nt = WARP ? 32 : kAppendCtaThreads;
  constexpr int ITER = WARP ? kAppendWarpIter : kAppendCtaIter<E>;
  const KvArgs& a = g.a;
  const int of_page = group / g.groups_page;  // (sequence, page)
  const int first = (group - of_page * g.groups_page) * g.group_units;
  const int b = of_page / g.units_page, pg = of_page - b * g.units_page;
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
  // a thread has one chunk of a token and every `step`th token, so that its chunk's
  // place is worked out once (threads past the last whole token have nothing)
  const int per_tok = NORM ? g.tok_threads : a.D / (2 * PC), tokens = p1 - p0;
  const int step = nt / per_tok, tok0 = t / per_tok;
  const bool has = !NORM || t - tok0 * per_tok < a.D / (2 * PC);  // the thread's chunk is one
  const ChunkAt at = chunk_at<PC>(g, has ? t - tok0 * per_tok : 0);
  const int mine = tok0 < step ? (tokens - tok0 + step - 1) / step : 0;  // this thread's tokens
  const bool hold = tokens <= ITER * step;
  const int kept = p0 & (S - 1);  // earlier tokens of the sequence in this page
  const int cs_step = step * g.rot;
  const float* const cs = g.cos_sin + (g.rot > 0 ? static_cast<int64_t>(p0 + tok0) * g.rot : 0);
  const int64_t token = p0 - L + tok0;
  const int last = min(first + g.group_units, 2 * a.Hkv);
  for (int unit = first; unit < last; ++unit) {
    const int kv = unit & 1, h = unit >> 1;
    const int64_t x_tok = kv ? g.v_tok : g.k_tok, x_step = step * x_tok;
    const E* const x = static_cast<const E*>(kv ? g.v : g.k) + b * (kv ? g.v_seq : g.k_seq) +
                       h * (kv ? g.v_head : g.k_head) + token * x_tok;
    const bool turned = !kv && g.rot > 0;
    const float* const weight = NORM && !kv && g.k_weight ? g.k_weight + h * g.k_weight_head : nullptr;
    if constexpr (NORM && PC == 1) {
      // the unit's tokens, a warp each
      if constexpr (!WARP) __syncthreads();  // the norms before have been used
      if (weight) {
        const E* const x0 = x - tok0 * x_tok;
        for (int i = WARP ? 0 : t >> 5; i < tokens; i += WARP ? 1 : nt / 32) {
          const float r = row_norm(g, x0 + i * x_tok);
          if ((t & 31) == 0) norms[i] = r;
        }
      }
      if constexpr (WARP)
        __syncwarp();
      else
        __syncthreads();
    }
    Weights<PC> weights;
    if (weight) weights.load(weight, at);
    RawChunk<E, PC> raw[ITER];
    float norm[ITER];
    const auto read = [&](int i0) {
#pragma unroll
      for (int it = 0; it < ITER; ++it)
        if (i0 + it < mine && has)
          raw[it].load(x + (i0 + it) * x_step, at);
        else if (NORM)
          raw[it].clear();
      if constexpr (NORM) {
        if (weight) {
          if constexpr (PC == 1) {
#pragma unroll
            for (int it = 0; it < ITER; ++it)
              if (i0 + it < mine) norm[it] = norms[tok0 + (i0 + it) * step];
          } else {
            norms_of<ITER>(g, raw, norm, per_tok);  // (of tokens that are not there, too: they are zero)
          }
        }
      }
    };
    const auto values = [&](int i0, int it, float* y) {
      raw[it].values(y);
      if constexpr (NORM)
        if (weight) weights.scale(y, norm[it]);
      if (turned) turn_chunk<PC>(g, cs + static_cast<int64_t>(i0 + it) * cs_step, at, y);
    };
    const auto largest = [&](uint32_t v) {
      v = __reduce_max_sync(kFull, v);
      if constexpr (!WARP) {
        __syncthreads();  // `red` has been read
        if ((t & 31) == 0) red[t >> 5] = v;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < nt / 32; w += 4) {
          const uint4 r = *reinterpret_cast<const uint4*>(&red[w]);
          v = max(max(v, max(r.x, r.y)), max(r.z, r.w));
        }
      }
      return v;
    };
    // bits of the largest magnitude: they order magnitudes, the infinities and NaN last
    uint32_t top = 0;
    int i0 = 0;
    do {
      read(i0);
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        if (i0 + it < mine) {
          float y[2 * PC];
          values(i0, it, y);
          if (!has) continue;  // (a neighbour's weights times zero may be NaN)
#pragma unroll
          for (int j = 0; j < 2 * PC; ++j) top = max(top, __float_as_uint(y[j]) & 0x7fffffffu);
        }
      }
      i0 += ITER;
    } while (!hold && i0 < mine);
    if (page < 0) {
      if (t == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
      return;
    }
    uint8_t* const page_codes = (kv ? a.v_codes : a.k_codes) + page * a.page_stride + h * a.head_stride;
    float* sp = (kv ? a.v_scale : a.k_scale) + page * a.scale_page_stride + h * a.scale_head_stride;
    const float before = kept ? *sp : 0.0f;
    top = largest(top);  // (all have read `before`)
    bool plain = top < 0x7f800000u;
    if (!plain) {  // NaN or infinities: the scale is that of the finite values
      top = 0;
      i0 = 0;
      do {
        if (!hold) read(i0);
#pragma unroll
        for (int it = 0; it < ITER; ++it) {
          if (i0 + it < mine) {
            float y[2 * PC];
            values(i0, it, y);
#pragma unroll
            for (int j = 0; j < 2 * PC; ++j) {
              const uint32_t m = __float_as_uint(y[j]) & 0x7fffffffu;
              top = max(top, has && m < 0x7f800000u ? m : 0u);
            }
          }
        }
        i0 += ITER;
      } while (!hold && i0 < mine);
      top = largest(top);
    }
    const float need = scale_for(__uint_as_float(top));
    const float scale = before >= need ? before : need;
    if constexpr (WARP) __syncwarp();
    if (kept && scale != before) {
      // the page's earlier codes at the grown scale
      const float f = before / scale;
      const int vec = a.D / 16;
#pragma unroll 1
      for (int i = t; i < kept * vec; i += nt) {
        const int tok = i / vec, c = i - tok * vec;
        uint4* p = reinterpret_cast<uint4*>(page_codes + tok * a.token_stride + c * 16);
        uint4 r = *p;
        uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 lo = codes2_to_float2(static_cast<uint16_t>(w[j] & 0xffffu));
          const float2 hi = codes2_to_float2(static_cast<uint16_t>(w[j] >> 16));
          w[j] = to_codes2(no_infinity(lo.x * f), no_infinity(lo.y * f)) |
                 (to_codes2(no_infinity(hi.x * f), no_infinity(hi.y * f)) << 16);
        }
        *p = r;
      }
    }
    if (t == 0 && !(scale == before)) *sp = scale;
    const Divider div(scale);
    plain = plain && div.exact;
    const int64_t code_step = step * a.token_stride;
    uint8_t* const codes = page_codes + (kept + tok0) * a.token_stride;
    i0 = 0;
    do {
      if (!hold) read(i0);
#pragma unroll
      for (int it = 0; it < ITER; ++it) {
        if (i0 + it < mine) {
          uint8_t* dst = codes + (i0 + it) * code_step;
          float y[2 * PC];
          values(i0, it, y);
          if (has) {
            store_codes<PC>(dst + at.lo, y, div, plain);
            store_codes<PC>(dst + at.hi, y + PC, div, plain);
          }
        }
      }
      i0 += ITER;
    } while (i0 < mine);
  }
}

// Queries of single channels with norms: a head of a row is a warp's, whose lanes read and write the same pairs.
template <typename E>
__device__ __forceinline__ void norm_queries(const AppendArgs& g, int row0, int row1, int warp, int warps) {
  const KvArgs& a = g.a;
  const int lane = threadIdx.x & 31;
  for (int i = warp; i < (row1 - row0) * a.Hq; i += warps) {
    const int row = row0 + i / a.Hq, h = i - (row - row0) * a.Hq, b = row / a.T, tok = row - b * a.T;
    int L, n;
    const bool ok = append_span(g, b, &L, &n);
    if (!ok && lane == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
    const E* q = static_cast<const E*>(a.q) + b * a.q_seq + h * a.q_head + tok * a.q_tok;
    E* o = static_cast<E*>(a.out) + b * a.o_seq + h * a.o_head + tok * a.o_tok;
    if (!ok || tok >= n) {
      const float fill = ok ? 0.0f : __uint_as_float(0x7fc00000u);
      for (int d = lane; d < a.D; d += 32) from_float(fill, o + d);
      continue;
    }
    const float r = row_norm(g, q);  // (every lane's channels are read before any is written)
    const float* cs = g.cos_sin + (g.rot > 0 ? static_cast<int64_t>(L + tok) * g.rot : 0);
    for (int p = lane; p < a.D / 2; p += 32) {
      const ChunkAt k = chunk_at<1>(g, p);
      float y[2] = {to_float(q[k.lo]), to_float(q[k.hi])};
      Weights<1> w;
      w.load(g.q_weight + h * g.q_weight_head, k);
      w.scale(y, r);
      turn_chunk<1>(g, cs, k, y);
      from_float(y[0], o + k.lo);
      from_float(y[1], o + k.hi);
    }
  }
}

template <typename E, int PC, bool WARP, bool NORM>
__global__ void __launch_bounds__(WARP ? kAppendWarpThreads : kAppendCtaThreads, WARP ? 1 : NORM ? 2 : kAppendCtas)
    spec_kv_append_kernel(const __grid_constant__ AppendArgs g) {
  constexpr int nt = WARP ? kAppendWarpThreads : kAppendCtaThreads;
  const KvArgs& a = g.a;
  const int tid = threadIdx.x;
  start_dependents();
  wait_for_grid();
  if (blockIdx.x < static_cast<unsigned>(g.unit_blocks)) {
    __shared__ __align__(16) uint32_t red[WARP ? 4 : kAppendCtaThreads / 32];
    __shared__ float norms[NORM && PC == 1 ? (WARP ? nt / 32 : 1) : 1][NORM && PC == 1 ? kMostSlots : 1];
    if constexpr (WARP) {
      const int group = blockIdx.x * (kAppendWarpThreads / 32) + (tid >> 5);
      if (group < g.groups)
        append_group<E, PC, true, NORM>(g, group, tid & 31, red, norms[NORM && PC == 1 ? tid >> 5 : 0]);
    } else {
      append_group<E, PC, false, NORM>(g, blockIdx.x, tid, red, norms[0]);
    }
    return;
  }
  if constexpr (NORM && PC == 1) {
    if (g.q_weight) {
      const int row0 = static_cast<int>(blockIdx.x - g.unit_blocks) * g.q_rows_block;
      norm_queries<E>(g, row0, min(a.B * a.T, row0 + g.q_rows_block), tid >> 5, nt / 32);
      return;
    }
  }
  // queries: rows (sequence, token); as many side by side as the CTA has threads for
  const int per_tok = NORM ? g.tok_threads : a.D / (2 * PC), heads = a.Hq / g.q_heads, per_row = heads * per_tok;
  const int beside = max(1, nt / per_row);
  const int r0 = tid / per_row;  // this thread's row among those side by side
  if (beside > 1 && r0 >= beside) return;
  const int nrows = a.B * a.T;
  const int row0 = static_cast<int>(blockIdx.x - g.unit_blocks) * g.q_rows_block;
  const int first = row0 + (beside > 1 ? r0 : 0), last = min(nrows, row0 + g.q_rows_block);
  for (int j = beside > 1 ? tid - r0 * per_row : tid; j < per_row; j += nt) {
    const int h = j / per_tok;
    const bool has = !NORM || j - h * per_tok < a.D / (2 * PC);  // the thread's chunk is one
    const ChunkAt k = chunk_at<PC>(g, has ? j - h * per_tok : 0);
    // (heads a thread takes lie `heads` apart)
    const float* const weight = NORM && g.q_weight ? g.q_weight + h * g.q_weight_head : nullptr;
    const int64_t w_heads = heads * g.q_weight_head;
    int b = first / a.T, tok = first - b * a.T;
    for (int row = first; row < last;) {
      // this sequence's rows among the CTA's: the new tokens, then the empty slots
      int L, n;
      const bool ok = append_span(g, b, &L, &n);
      if (!ok && j == 0) report(a.status, SPEC_ERR_CACHE_RANGE);
      const int rows = (min(last - row, a.T - tok) + beside - 1) / beside;
      const int full = ok && tok < n ? min(rows, (n - tok + beside - 1) / beside) : 0;
      const E* q = static_cast<const E*>(a.q) + b * a.q_seq + h * a.q_head + tok * a.q_tok;
      E* o = static_cast<E*>(a.out) + b * a.o_seq + h * a.o_head + tok * a.o_tok;
      const float* cs = g.cos_sin + (k.turn ? static_cast<int64_t>(L + tok) * g.rot : 0);
      const int64_t q_step = beside * a.q_tok, o_step = beside * a.o_tok;
      const int64_t q_heads = heads * a.q_head, o_heads = heads * a.o_head;
      if (g.q_heads == 1) {
        for (int i = 0; i < full; ++i, q += q_step, o += o_step, cs += beside * g.rot) {
          float y[2 * PC];
          RawChunk<E, PC> raw;
          if (has)
            raw.load(q, k);
          else
            raw.clear();
          raw.values(y);
          if constexpr (NORM && PC > 1) {
            if (weight) {
              float norm;
              norms_of<1>(g, &raw, &norm, per_tok);
              Weights<PC> w;
              w.load(weight, k);
              w.scale(y, norm);
            }
          }
          turn_chunk<PC>(g, cs, k, y);
          if (!has) continue;
          store_n<E, PC>(o + k.lo, y);
          store_n<E, PC>(o + k.hi, y + PC);
        }
      } else {
        for (int i = 0; i < full; ++i, q += q_step, o += o_step, cs += beside * g.rot) {
          RawChunk<E, PC> raw[kAppendHeads];
#pragma unroll
          for (int e = 0; e < kAppendHeads; ++e) {
            if (has)
              raw[e].load(q + e * q_heads, k);
            else
              raw[e].clear();
          }
          if (NORM && i + 1 < full) {
#pragma unroll
            for (int e = 0; e < kAppendHeads; ++e) {
              asm volatile("prefetch.global.L2 [%0];" ::"l"(q + q_step + e * q_heads + k.lo));
              asm volatile("prefetch.global.L2 [%0];" ::"l"(q + q_step + e * q_heads + k.hi));
            }
          }
          const Angles<PC> at(g, cs, k);
          float norm[kAppendHeads];
          if constexpr (NORM && PC > 1) {
            if (weight) norms_of<kAppendHeads>(g, raw, norm, per_tok);
          }
          Weights<PC> w;
          if (weight) w.load(weight, k);
#pragma unroll
          for (int e = 0; e < kAppendHeads; ++e) {
            float y[2 * PC];
            raw[e].values(y);
            if constexpr (NORM && PC > 1) {
              if (weight) {
                if (e > 0 && w_heads) w.load(weight + e * w_heads, k);
                w.scale(y, norm[e]);
              }
            }
            at.turn_all(g, k, y);
            if (!has) continue;
            store_n<E, PC>(o + e * o_heads + k.lo, y);
            store_n<E, PC>(o + e * o_heads + k.hi, y + PC);
          }
        }
      }
      float fill[PC];
#pragma unroll
      for (int e = 0; e < PC; ++e) fill[e] = ok ? 0.0f : __uint_as_float(0x7fc00000u);
      for (int i = full; has && i < rows; ++i, o += o_step) {
        for (int e = 0; e < g.q_heads; ++e) {
          store_n<E, PC>(o + e * o_heads + k.lo, fill);
          store_n<E, PC>(o + e * o_heads + k.hi, fill);
        }
      }
      row += rows * beside;
      tok += rows * beside;
      while (tok >= a.T) {
        tok -= a.T;
        ++b;
      }
    }
  }
}

}  // namespace spec_kv_detail
