#pragma once
// spec_kv_mma.cuh -- attention over the paged 8-bit cache on the tensor cores, for
// bfloat16 queries.
//
// The cache's bytes go from memory to the matrix instruction as they are: tensor
// maps bring a tile of 128 tokens into swizzled shared memory, and both products
// are 8-bit ones with float accumulators in tensor memory,
//
//   S^T [128 tokens x rows]   = K [128 x D]   Q^T [D x rows]
//   O^T [D x rows]           += V^T [D x 128] P^T [128 x rows].
//
// Tokens and channels are the instruction's 128 rows and the query rows its
// columns, so its cost goes with the rows there are (from 16) and not with 128.
// A row is a (new token, query head) of one key/value head; the two softmax groups
// take half of the rows each, four at a time, the first half in columns 0.. and
// the second in columns NR / 2...
//
// What is not 8 bits is carried in 8-bit pieces:
//   q / 2^e = hi + lo in e4m3, two products into one accumulator (a bfloat16 has 8
//     significant bits: exact but for 2^-17 of the row's largest channel; rows
//     within 2^kNear of each other share one e, for 2^-17 of the largest's, and
//     one factor of the scores with it);
//   p = p0 + p1 / 8 + p2 / 64 in e5m2, the pieces side by side as columns of one
//     product and added at the end (sums are of the float p).
// Long contexts are full of small weights that only count together, so each weight
// keeps its own precision: an error of 2^-9 of it at most down to 2^-23 of the
// largest weight of its row in the range, and of 2^-32 of the largest below.  (Two
// e4m3 pieces lost what lay under 2^-17 of it: 58 % of the output where a quarter of
// the weight is spread evenly over 32768 tokens.)
//
// A thread of the softmax warps holds one token: the token's two scales are
// scalars of the thread, applied to the scores in float (the value scale as
// exponent of 2, so that p is the weight of the 8-bit values).  The running
// maximum of a row is over the threads; it is not needed exactly, only as a
// reference that keeps p within the pieces' range, so it is raised (and the
// accumulators rescaled) only when a weight would pass 2^kSlack times the one at
// which it was set, and in the first tile of an item.
//
// The matrix unit adds to its float accumulators with truncation: about 2^-24 of
// the sum for each 32 tokens, always downwards in magnitude.  At a million tokens
// in one range that is 1e-3 of an output, of the order of its bfloat16 rounding.
//
// Roles: warps 0-3 and 4-7 softmax and epilogue, each four warps for half of the
// rows; warp 8 loads; one thread of warp 9 issues the products.  Scores are
// double-buffered, so the products of the next tile run under the softmax of this
// one.  Two CTAs share an SM.
//
// What bounds it.  Long caches: memory while few rows read them (64 sequences of
// up to 8192 tokens, 8 rows a key/value head: 653 MB in 106 us, 6.2 TB/s), the
// softmax warps' instructions beside it as rows grow (32 sequences of up to 32768
// tokens, 36 rows: 1.24 GB in 219 us, 5.7 TB/s; a tile costs a softmax warp about
// 3000 cycles beside three others on its scheduler, the tensor unit is busy a fifth
// of the time).  Part of a prompt (512 queries on 8192 tokens): the same instructions,
// 142 GFLOP in 299 us.  Short calls: the chain of dependent steps (lengths, page
// numbers, keys, scores, weights, output, join: 1000 tokens take 10.5 us).
#include <cuda_fp16.h>

#include "spec_kv_attn.cuh"
#include "spec_kv_append.cuh"
#include "spec_kv_ptx.cuh"

namespace spec_kv_detail {

// Rows of a row tile at most.  More would share one reading of the cache between
// more rows, but 64 do not fit the registers of the softmax threads (with two-piece
// weights, 512 queries on 8192 tokens took 472 us in row tiles of 64, 367 in tiles of
// 48, 414 in tiles of 32).
constexpr int kMmaRows = 48;
constexpr int kMmaThreads = 320;
constexpr int kSoftThreads = 256;  // two groups of 128, a token a thread
// Rings without a way back, because the loader cannot go round them: it is at most
// KS + 2 <= 5 tiles ahead of the softmax (stages of keys, and two buffers of scores),
// so at most five pieces with tiles, one more announced, then an empty one and the end.
constexpr int kPieceRing = 8;
constexpr uint32_t kUnset = 0x80000000u;  // bits of -0: scores are taken as they are
constexpr int kNear = 4;            // log2 of how far apart rows with one exponent may be
constexpr int kTop = 15;            // log2 of the largest weight (e5m2 and half hold more than 2^15)
// log2 of how far weights may pass the reference: a bit more costs the smallest weights one, a bit less makes
// references move more often (36 rows on 32768 tokens 236 us with 3, 222 with 5, 219 with 6, 219 with 7; 512 queries
// on 8192 351, 308, 299, 293)
constexpr int kSlack = 6;
constexpr float kShift = kTop - kSlack;  // a raised reference is kShift below the largest score
// The sums are of weights times this: with value scales down to 2^-100 those of 2^24 tokens stay finite.
constexpr int kSumExp = 12;
constexpr float kSumUnit = 1.0f / (1 << kSumExp);
constexpr int kPieces = 3;          // of a weight
// Value scales count as this times the largest that came before them in the piece, at least:
// below, a token's weight would leave the float range on its way to the sum.
constexpr float kLeastOfTop = 1.0f / (1ull << 40) / (1ull << 40);

// Stages of keys and of values, buffers of weights: what two CTAs an SM leave room
// for.  Keys are used up two tiles ahead of the weights (the scores are
// double-buffered), so values get the larger share (36 rows on 32768 tokens: 223 us,
// 236 with two stages of values; 20 rows on 131072: 52.8 us, 54.7 with a second buffer
// of weights in place of the third stage).
template <int D, int NR>
struct MmaCfg {
  static constexpr int kTileBytes = kTile * D;
  static constexpr int KS = D == 64 ? 3 : 2;
  static constexpr int VS = D == 64 ? 5 : 3;
  static constexpr int kScaleRing = KS == 2 ? 4 : 8;    // at least KS + 2: see kPieceRing
  static constexpr int PB = D == 64 || NR == 16 ? 2 : 1;
  static constexpr int kQBytes = NR * D;                // one piece
  static constexpr int kPBytes = kTile * kPieces * NR;  // all pieces
  static constexpr int kOffV = 0;                    // values first: a 64-channel operand reads on into what follows
  static constexpr int kOffK = kOffV + VS * kTileBytes;
  static constexpr int kOffQ = kOffK + KS * kTileBytes;
  static constexpr int kOffP = kOffQ + 2 * kQBytes;
  static constexpr int kOffSmall = kOffP + PB * kPBytes;
  static constexpr uint32_t kCols = NR == 16 ? 128 : 256;  // 2 x scores, 3 pieces of output
};

template <int D, int NR>
struct MmaSmall {
  using C = MmaCfg<D, NR>;
  uint64_t k_full[C::KS], k_empty[C::KS], v_full[C::VS], v_empty[C::VS];
  uint64_t s_full[2], p_full[C::PB], pv_done[C::PB], piece_full[kPieceRing], q_full, drain;
  alignas(16) float refs[NR];     // negated references of the rows; kUnset: none yet
  alignas(16) float factor[NR];   // of the scores, where rows have exponents of their own
  uint32_t q_top, q_least;        // largest and least of the rows' largest magnitudes
  float4 scales[C::kScaleRing][kTile / 16];  // of a page: key scale; value scale's log2, and kSumUnit over it
  int64_t out_at[NR];             // element of the output where a row begins
  alignas(16) float red[4][NR];   // a row's maxima or sums by warp; then, by the thread that has read them,
  __device__ float* up() { return red[0]; }   // what a rescaling raises the reference by,
  __device__ float* fac() { return red[1]; }  // what it multiplies by,
  __device__ float* root() { return red[2]; }  // and the root of that
  int pos[NR];
  RangePlan plan;
  int scratch[kMmaThreads / 32];
  uint32_t tmem;
  int gave_up, last;
  Piece pieces[kPieceRing];  // from the loader to the other roles; b < 0: no more
};

// two CTAs share an SM's 228 KB, of which each takes 1 KB beside its own
constexpr int kMostSmem = (228 / 2 - 1) * 1024;
template <int D, int NR>
constexpr int mma_smem_bytes() {
  constexpr int bytes = MmaCfg<D, NR>::kOffSmall + static_cast<int>(sizeof(MmaSmall<D, NR>));
  static_assert(bytes <= kMostSmem, "two CTAs an SM");
  return bytes;
}

// tensor maps of the pool: the channel, then token, head and page in the order of
// their strides
struct MmaMaps {
  CUtensorMap k, v;
  int32_t at_head, at_page;  // places among the three, 0 to 2
};

typedef unsigned long long u64;
__device__ __forceinline__ u64 pack2(float a, float b) {
  u64 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(u64 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
__device__ __forceinline__ u64 fma2(u64 a, u64 b, u64 c) {
  u64 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ u64 mul2(u64 a, u64 b) {
  u64 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ u64 add2(u64 a, u64 b) {
  u64 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// barriers 1 and 2: a group of four softmax warps; barrier 3: both groups
// (constant numbers: with a computed one the CTA would claim all sixteen)
__device__ __forceinline__ void group_sync(int group) {
  if (group == 0)
    asm volatile("bar.sync 1, 128;" ::: "memory");
  else
    asm volatile("bar.sync 2, 128;" ::: "memory");
}
__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 3, 256;" ::: "memory"); }
__device__ __forceinline__ bool group_any(int group, bool x) {
  uint32_t r;
  if (group == 0)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(x ? 1u : 0u)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.or.pred q, 2, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(x ? 1u : 0u)
        : "memory");
  return r != 0;
}
__device__ __forceinline__ bool soft_any(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 3, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(x ? 1u : 0u)
      : "memory");
  return r != 0;
}

// order-preserving integer image of a float (NaN aside), and back
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float of_order(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// Two weights as halves, in three pieces whose bytes are those of e5m2: a half's upper byte is an e5m2 (of the half
// rounded towards zero, 3 significant bits), so the first piece is the half without its lower byte; the second is that of
// eight times what it leaves, exactly; the third the nearest to eight times what that leaves.  a and b get the first two
// pieces in their upper bytes, c the third in two bytes.
__device__ __forceinline__ void three_pieces(float w0, float w1, uint32_t& a, uint32_t& b, uint32_t& c) {
  const auto bits = [](__half2 x) { return *reinterpret_cast<const uint32_t*>(&x); };
  const auto upper = [&](__half2 x, uint32_t& u) {
    u = bits(x) & 0xff00ff00u;
    return *reinterpret_cast<const __half2*>(&u);
  };
  const __half2 eight = __half2half2(__ushort_as_half(0x4800));
  const __half2 h = __floats2half2_rn(w0, w1);
  const __half2 d = __hmul2(__hsub2(h, upper(h, a)), eight);
  const __half2 e = __hmul2(__hsub2(d, upper(d, b)), eight);
  c = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(e), __NV_SATFINITE, __NV_E5M2);
}
// the upper bytes of the halves of x and y, in order
__device__ __forceinline__ uint32_t upper_bytes(uint32_t x, uint32_t y) { return __byte_perm(x, y, 0x7531); }

// 8 channels of a row that is not aligned, as if loaded 16 bytes at a time
static __device__ __noinline__ Raw<__nv_bfloat16, 8> gather8(const __nv_bfloat16* src) {
  Raw<__nv_bfloat16, 8> r;
  const unsigned short* s = reinterpret_cast<const unsigned short*>(src);
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) u[i] = s[2 * i] | (static_cast<uint32_t>(s[2 * i + 1]) << 16);
  r.w[0] = make_uint4(u[0], u[1], u[2], u[3]);
  return r;
}

// A wait of the CTA ran out: the range's pieces from the `done`th on become NaN.
static __device__ __noinline__ void abandon(const KvArgs& a, const RangePlan& plan, int range, int rt, int done,
                                            int* last) {
  const int tid = threadIdx.x;  // of the softmax warps
  const float nan = __uint_as_float(0x7fc00000u);
  if (tid == 0) report(a.status, SPEC_ERR_TIMEOUT);
  Walk walk = walk_begin(plan, range, rt);
  Piece p;
  for (int i = 0; walk_next(a, walk, p); ++i) {
    if (i < done) continue;
    for (int r = tid >> 5; r < p.nrows; r += kSoftThreads / 32) {
      const int gr = p.row0 + r, t = gr / a.G, hq = p.h * a.G + gr - t * a.G;
      if (!p.whole()) {
        if ((tid & 31) == 0) a.part_ml[static_cast<int64_t>(p.slot) * a.slot_rows + r] = make_float2(kNoRef, nan);
        continue;
      }
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + p.b * a.o_seq + t * a.o_tok + hq * a.o_head;
      for (int d = tid & 31; d < a.D; d += 32) from_float(nan, o + d);
      if (a.lse && (tid & 31) == 0) a.lse[(static_cast<int64_t>(p.b) * a.T + t) * a.Hq + hq] = nan;
    }
    if (a.join_here && !p.whole()) {
      soft_sync();
      if (tid == 0) *last = last_of_item(a, p, rt);
      soft_sync();
      if (*last) join_item<__nv_bfloat16>(a, p, rt, tid >> 5, kSoftThreads / 32);
    }
  }
}

// RU: rows that a softmax group keeps in registers, at most NR / 2
template <int D, int NR, int RU>
__global__ void __launch_bounds__(kMmaThreads, 2)
    spec_kv_attention_mma_kernel(const __grid_constant__ KvArgs a, const __grid_constant__ MmaMaps maps) {
  using C = MmaCfg<D, NR>;
  extern __shared__ __align__(1024) uint8_t dyn[];  // the swizzles repeat every 1024 bytes
  MmaSmall<D, NR>& sm = *reinterpret_cast<MmaSmall<D, NR>*>(dyn + C::kOffSmall);
  uint8_t* const sv = dyn + C::kOffV;
  uint8_t* const sk = dyn + C::kOffK;
  uint8_t* const sq = dyn + C::kOffQ;
  uint8_t* const sp = dyn + C::kOffP;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kSwizzle = D == 128 ? kSwizzle128 : kSwizzle64;

  if (tid == 0) {
    for (int i = 0; i < C::KS; ++i) {
      bar_init(&sm.k_full[i], 1);
      bar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < C::VS; ++i) {
      bar_init(&sm.v_full[i], 1);
      bar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) bar_init(&sm.s_full[i], 2);
    for (int i = 0; i < C::PB; ++i) {
      bar_init(&sm.p_full[i], kSoftThreads / 32);
      bar_init(&sm.pv_done[i], 1);
    }
    for (int i = 0; i < kPieceRing; ++i) bar_init(&sm.piece_full[i], 1);
    bar_init(&sm.q_full, 1);
    bar_init(&sm.drain, 1);
    sm.gave_up = 0;
    fence_bar_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_map(&maps.k);
    tma_prefetch_map(&maps.v);
  }
  if (warp == 9) tmem_alloc(&sm.tmem, C::kCols);
  const int range = blockIdx.x / a.nrt, rt = blockIdx.x - range * a.nrt;
  start_dependents();
  wait_for_grid();
  tc_fence_before();
  make_plan_range<kMmaThreads>(a, range, &sm.plan, sm.scratch, blockIdx.x == 0 ? a.prefix : nullptr);
  tc_fence_after();
  const uint32_t tm = sm.tmem;
  volatile int* const gave_up = &sm.gave_up;

  if (sm.plan.w0 < sm.plan.w1) {
    int n = 0;       // tiles so far, over all pieces
    int pieces = 0;  // pieces so far

    if (warp == 8) {
      // ---------------------------------------------------------------- loads
      const int np = kTile >> a.log_page;  // pages a tile
      const uint32_t page_bytes = static_cast<uint32_t>(D) << a.log_page;
      // a long cache goes through the L2 cache once a call: as lines to be evicted first it
      // took 106 us against 114 (653 MB), 217 against 232 (1.24 GB)
      const uint64_t policy = read_once_policy();
      bool ok = true;
      int nk = -1;
      Piece p;
      Walk walk = walk_begin(sm.plan, range, rt);
      while (ok) {
        if (!walk_next(a, walk, p)) p.b = -1;
        if (lane == 0) {
          sm.pieces[pieces % kPieceRing] = p;
          bar_arrive(&sm.piece_full[pieces % kPieceRing]);
        }
        ++pieces;
        if (p.b < 0) break;
        const int end = p.L + p.n;
        const int first = p.tile0 * np, last = min(p.tile1 * np, (end + (1 << a.log_page) - 1) >> a.log_page);
        // 32 pages at a time, one a lane: numbers, then scales; the next 32 are under way
        const auto number = [&](int base) {
          int pid = 0;
          if (base + lane < last) {
            pid = page_of(a, p.b, base + lane);
            if (pid < 0 && ((base + lane + 1) << a.log_page) > p.first) report(a.status, SPEC_ERR_CACHE_RANGE);
          }
          return pid;
        };
        const auto scales = [&](int base, int pid) {
          float2 s = make_float2(0.0f, 1.0f);
          if (base + lane < last) {
            if (pid < 0) {
              s.x = s.y = __uint_as_float(0x7fc00000u);
            } else {
              const int64_t at = pid * a.scale_page_stride + p.h * a.scale_head_stride;
              s.x = a.k_scale[at];
              s.y = a.v_scale[at];
            }
          }
          return s;
        };
        uint32_t v_top = 0;  // bits of the largest value scale so far
        int base = first;
        int pid = number(base), pid_next = 0;
        float2 sc = scales(base, pid), sc_next = make_float2(0.0f, 0.0f);
        for (int t = p.tile0; t < p.tile1; ++t, ++n) {
          int in = t * np - base;  // the tile's first page among the 32
          if (in == 32) {
            base += 32;
            in = 0;
            pid = pid_next;
            sc = sc_next;
          }
          const int mine = lane - in;  // this lane's page of the tile
          const bool has = mine >= 0 && mine < np && base + lane < last;
          const int cnt = min(np, last - (base + in));
          // coordinates after the channel: token 0, the head and the page, in the maps' order
          const int page = max(pid, 0);
          const int y = maps.at_head == 0 ? p.h : maps.at_page == 0 ? page : 0;
          const int z = maps.at_head == 1 ? p.h : maps.at_page == 1 ? page : 0;
          const int w = maps.at_head == 2 ? p.h : maps.at_page == 2 ? page : 0;
          const int ks = n % C::KS, vs = n % C::VS;
          if (n >= C::KS) ok = bar_wait(&sm.k_empty[ks], (n / C::KS - 1) & 1, gave_up);
          ok = __all_sync(kFull, ok);
          if (!ok) break;
          if (has)
            tma_load_4d(sk + ks * C::kTileBytes + mine * page_bytes, &maps.k, 0, y, z, w, &sm.k_full[ks], policy);
          // the tile's scales come with its keys: the arrival that the copies' bytes wait for is after them
          if (in == 0) {
            const bool counts = base + lane < last && sc.y > 0.0f && is_finite(sc.y);
            v_top = max(v_top, __reduce_max_sync(kFull, counts ? __float_as_uint(sc.y) : 0u));
          }
          if (mine >= 0 && mine < np) {
            const float least = fmaxf(7.8886090522101181e-31f, __uint_as_float(v_top) * kLeastOfTop);  // 2^-100
            const float v = sc.y < least ? least : sc.y;
            sm.scales[n % C::kScaleRing][mine] = make_float4(sc.x, log2f(v), kSumUnit / v, 0.0f);
          }
          __syncwarp();
          if (lane == 0) bar_arrive_expect(&sm.k_full[ks], cnt * page_bytes);
          if (n >= C::VS) ok = bar_wait(&sm.v_empty[vs], (n / C::VS - 1) & 1, gave_up);
          ok = __all_sync(kFull, ok);
          if (!ok) {
            nk = n + 1;  // this tile's keys are on their way
            break;
          }
          if (lane == 0) bar_arrive_expect(&sm.v_full[vs], cnt * page_bytes);
          __syncwarp();
          if (has)
            tma_load_4d(sv + vs * C::kTileBytes + mine * page_bytes, &maps.v, 0, y, z, w, &sm.v_full[vs], policy);
          if (in == 0) pid_next = number(base + 32);
          if (in == np) sc_next = scales(base + 32, pid_next);
        }
      }
      if (!ok) {
        // copies still under way have to land before the CTA ends
        int quiet = 0;
        if (nk < 0) nk = n;
        for (int i = max(0, nk - C::KS); i < nk; ++i) bar_wait(&sm.k_full[i % C::KS], (i / C::KS) & 1, &quiet);
        quiet = 0;
        for (int i = max(0, n - C::VS); i < n; ++i) bar_wait(&sm.v_full[i % C::VS], (i / C::VS) & 1, &quiet);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------- products
      if (lane == 0) {
        const uint32_t q0 = smem_u32(sq), k0 = smem_u32(sk), v0 = smem_u32(sv), p0 = smem_u32(sp);
        constexpr uint32_t kDescS = instr_desc(128, NR, false, false, kE4m3);
        constexpr uint32_t kDescO = instr_desc(128, kPieces * NR, true, true, kE5m2);
        bool ok = true;
        int queries = 0;
        const auto scores = [&](int i) {
          const int st = i % C::KS;
          ok = ok && bar_wait(&sm.k_full[st], (i / C::KS) & 1, gave_up);
          if (!ok) return;
          tc_fence_after();
          const uint32_t d = tm + (i & 1) * NR;
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int k = 0; k < D / 32; ++k)
              mma_f8(d, operand_desc(k0 + st * C::kTileBytes + k * 32, 16, 8 * D, kSwizzle),
                     operand_desc(q0 + half * C::kQBytes + k * 2 * NR * 16, NR * 16, 128, kSwizzleNone), kDescS,
                     half + k > 0);
          mma_commit(&sm.k_empty[st]);
          mma_commit(&sm.s_full[i & 1]);
          bar_arrive(&sm.s_full[i & 1]);  // passes the loader's scales on, as a commit alone need not
        };
        for (;; ++pieces) {
          ok = ok && bar_wait(&sm.piece_full[pieces % kPieceRing], (pieces / kPieceRing) & 1, gave_up);
          if (!ok) break;
          const Piece& p = sm.pieces[pieces % kPieceRing];
          if (p.b < 0) break;
          const int m = p.tile1 - p.tile0;
          if (m == 0) continue;
          ok = bar_wait(&sm.q_full, queries & 1, gave_up);
          if (!ok) break;
          ++queries;
          scores(n);
          if (m > 1) scores(n + 1);
          for (int i = 0; ok && i < m; ++i, ++n) {
            ok = bar_wait(&sm.p_full[n % C::PB], (n / C::PB) & 1, gave_up) &&
                 bar_wait(&sm.v_full[n % C::VS], (n / C::VS) & 1, gave_up);
            if (!ok) break;
            tc_fence_after();
            const uint32_t va = v0 + (n % C::VS) * C::kTileBytes, pa = p0 + (n % C::PB) * C::kPBytes;
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k)
              mma_f8(tm + 2 * NR, operand_desc(va + k * 32 * D, kTile * 64, 8 * D, kSwizzle),
                     operand_desc(pa + k * 32 * 16, 128, kTile * 16, kSwizzleNone), kDescO, i + k > 0);
            mma_commit(&sm.v_empty[n % C::VS]);
            mma_commit(&sm.pv_done[n % C::PB]);
            if (i + 2 < m) scores(n + 2);
          }
        }
        if (!ok) {  // products still running have to end before tensor memory is released
          int quiet = 0;
          mma_commit(&sm.drain);
          bar_wait(&sm.drain, 0, &quiet);
        }
      }
      __syncwarp();
    } else {
      // -------------------------------------------------------------- softmax
      constexpr int RT = NR / 2;         // columns of a group
      constexpr int CH = 4;              // rows at a time
      const int group = warp >> 2, token = tid & 127, r_base = group * RT;
      const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;  // tensor memory lanes of this warp
      const uint32_t tO = tm + lanes + 2 * NR + r_base;                     // first pieces; the others NR and 2 NR further
      bool fail = false;
      for (;; ++pieces) {
        // the piece stays in shared memory, out of the registers that the loop over the tiles needs
        const Piece& p = sm.pieces[pieces % kPieceRing];
        const auto half_of = [&]() { return min(RU, (p.nrows + 7) / 8 * 4); };  // rows of the first group
        const auto rows_mine = [&]() { return group == 0 ? min(half_of(), p.nrows) : p.nrows - half_of(); };
        const auto row_of = [&](int col) {  // of a column: nrows and more for none
          const int half = half_of();
          return col < RT ? (col < half ? col : p.nrows) : col - RT + half;
        };
        if (!fail) fail = !bar_wait(&sm.piece_full[pieces % kPieceRing], (pieces / kPieceRing) & 1, gave_up);
        if (tid == 0) {
          sm.q_top = 0;
          sm.q_least = 0x7f7fffffu;
        }
        fail = soft_any(fail);  // the piece before has been written out
        if (fail || p.b < 0) break;
        const int m = p.tile1 - p.tile0;
        const int fours = max(0, (rows_mine() + 3) / 4 * 4);  // this group's rows, in fours
        float l[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r) l[r] = 0.0f;
        if (tid < NR) {
          const int r = row_of(tid);
          const bool row = r < p.nrows;
          const int gr = p.row0 + r, t = gr / a.G, g = gr - t * a.G;
          sm.pos[tid] = row ? p.L + t : -1;
          sm.out_at[tid] = p.b * a.o_seq + t * a.o_tok + (p.h * a.G + g) * a.o_head;
        }
        bool one_factor = true;
        float factor = 0.0f;
        if (m > 0) {
          // queries: 8 channels a thread
          constexpr int kPer = D / 8;                  // threads a row
          constexpr int kStep = kSoftThreads / kPer;   // rows at a time
          constexpr int kTimes = (NR + kStep - 1) / kStep;
          Raw<__nv_bfloat16, 8> raw[kTimes];
          uint32_t tops[kTimes];  // bits of a row's largest magnitude (NaN above infinity)
#pragma unroll
          for (int i = 0; i < kTimes; ++i) {
            const int col = i * kStep + tid / kPer, c = tid % kPer, r = row_of(col);
            raw[i].w[0] = make_uint4(0, 0, 0, 0);
            if (col < NR && r < p.nrows) {
              const int gr = p.row0 + r, t = gr / a.G, g = gr - t * a.G;
              const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + p.b * a.q_seq + t * a.q_tok +
                                         (p.h * a.G + g) * a.q_head + c * 8;
              if (a.q_vec)
                raw[i].load(src);
              else
                raw[i] = gather8(src);
            }
          }
          uint32_t most = 0, least = 0x7f7fffffu;
#pragma unroll
          for (int i = 0; i < kTimes; ++i) {
            float x[8];
            raw[i].values(x);
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
            for (int d = kPer / 2; d; d >>= 1) top = max(top, __shfl_xor_sync(kFull, top, d));
            tops[i] = top;
            if (top > 0 && top < 0x7f800000u) {
              most = max(most, top);
              least = min(least, top);
            }
          }
          most = __reduce_max_sync(kFull, most);
          least = __reduce_min_sync(kFull, least);
          if (lane == 0) {
            atomicMax(&sm.q_top, most);
            atomicMin(&sm.q_least, least);
          }
          soft_sync();
          const uint32_t q_top = sm.q_top;
          const float common = scale_for(__uint_as_float(q_top));
          one_factor = q_top < sm.q_least + (static_cast<uint32_t>(kNear) << 23);
          factor = one_factor ? common * a.scale2 : a.scale2;
#pragma unroll
          for (int i = 0; i < kTimes; ++i) {
            const int col = i * kStep + tid / kPer, c = tid % kPer;
            if (col >= NR) continue;
            float x[8];
            raw[i].values(x);
            const bool fin = tops[i] < 0x7f800000u;  // a row that is not is NaN by its reference
            const float s = one_factor ? common : fin ? scale_for(__uint_as_float(tops[i])) : 1.0f;
            const float inv = 1.0f / s;
            uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 y = make_float2(fin ? x[e] * inv : 0.0f, fin ? x[e + 1] * inv : 0.0f);
              const uint16_t ch = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
              const float2 b = codes2_to_float2(ch);
              const uint16_t cl =
                  __nv_cvt_float2_to_fp8x2(make_float2(y.x - b.x, y.y - b.y), __NV_SATFINITE, __NV_E4M3);
              hi[e / 4] |= static_cast<uint32_t>(ch) << (8 * (e & 2));
              lo[e / 4] |= static_cast<uint32_t>(cl) << (8 * (e & 2));
            }
            uint8_t* dst = sq + (c >> 1) * (NR * 16) + col * 16 + (c & 1) * 8;
            *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(dst + C::kQBytes) = make_uint2(lo[0], lo[1]);
            if (c == 0) {
              // a row that is not there has a reference no score passes
              sm.refs[col] = row_of(col) >= p.nrows ? kNoRef : __uint_as_float(fin ? kUnset : 0x7fc00000u);
              sm.factor[col] = s;
            }
          }
          fence_async();
          soft_sync();
          if (tid == 0) bar_arrive(&sm.q_full);
        }
        const int tile0 = p.tile0, tile1 = p.tile1;
        const int pos_hi = p.L + (p.row0 + p.nrows - 1) / a.G;
        // tiles that some row sees only in part: from t_edge on, and up to t_win; and the tile from
        // which on every row has seen a token
        const int t_edge = (p.L + p.row0 / a.G + 1) / kTile;
        const int t_win = a.window > 0 && pos_hi >= a.window ? (pos_hi - a.window) / kTile : -1;
        const int t_unset = max(tile0, a.window > 0 ? (pos_hi + 1 - a.window) / kTile : 0);
        for (int t = tile0; t < tile1; ++t, ++n) {
          const int j = t * kTile + token;
          // scores of this tile; they come with its scales, and with the end of the products two
          // tiles back (issued before them): with two buffers of weights this one's is free
          if (!fail) fail = !bar_wait(&sm.s_full[n & 1], (n >> 1) & 1, gave_up);
          tc_fence_after();
          float4 sc = sm.scales[n % C::kScaleRing][token >> a.log_page];
          const bool edge = t >= t_edge || t <= t_win;
          bool poison = false;
          if (edge) {
            // no row may be touched by what it does not see: values that are not to be read are
            // zero, NaN codes and scales of a token that some rows see go to those rows' sums
            const int first = p.L + p.row0 / a.G, last = p.L + (p.row0 + p.nrows - 1) / a.G;
            const bool all_see = j <= first && (a.window <= 0 || j > last - a.window);
            const bool gone = j >= p.L + p.n;
            const bool bad_scale = !(sc.x == sc.x && sc.z == sc.z);
            uint8_t* row = sv + (n % C::VS) * C::kTileBytes + token * D;  // whole rows: the swizzle stays inside
            if (!fail) fail = !bar_wait(&sm.v_full[n % C::VS], (n / C::VS) & 1, gave_up);
            // (lanes begin at different places of their rows, which all start at one bank)
            if (!all_see && !gone) {
              uint32_t nan = 0;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint4 u = reinterpret_cast<const uint4*>(row)[(i + lane) % (D / 16)];
                nan |= __vcmpeq4(u.x & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(u.y & 0x7f7f7f7fu, 0x7f7f7f7fu) |
                       __vcmpeq4(u.z & 0x7f7f7f7fu, 0x7f7f7f7fu) | __vcmpeq4(u.w & 0x7f7f7f7fu, 0x7f7f7f7fu);
              }
              poison = nan != 0 || bad_scale;
            }
            soft_sync();  // both groups have looked
            if (gone || poison) {
#pragma unroll 4
              for (int i = 0; i < D / 16; ++i)
                reinterpret_cast<uint4*>(row)[(i + lane) % (D / 16)] = make_uint4(0, 0, 0, 0);
              if (gone || bad_scale) sc = make_float4(0.0f, 0.0f, 1.0f, 0.0f);
            }
          }
          const float ks = sc.x * factor;
          const u64 ks2 = pack2(ks, ks), lv2 = pack2(sc.y, sc.y), ivs2 = pack2(sc.z, sc.z);
          const uint32_t tS = tm + lanes + (n & 1) * NR + r_base;
          const auto sees = [&](int r) {
            const int q = sm.pos[r_base + r];
            return j <= q && (a.window <= 0 || j > q - a.window);
          };
          float x[RT];
#pragma unroll
          for (int c = 0; c < RT; c += 8) tmem_ld<8>(tS + c, &x[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < RT; c += 8) tmem_tie<8>(&x[c]);
          if (!one_factor) {
#pragma unroll
            for (int r = 0; r < RU; ++r) x[r] *= sm.factor[r_base + r];
          }
          // scores in log2 units against the rows' references
#pragma unroll
          for (int c = 0; c < RU; c += CH) {
            if (c < fours) {
              const float4 ref = *reinterpret_cast<const float4*>(&sm.refs[r_base + c]);
              unpack2(fma2(pack2(x[c], x[c + 1]), ks2, add2(lv2, pack2(ref.x, ref.y))), x[c], x[c + 1]);
              unpack2(fma2(pack2(x[c + 2], x[c + 3]), ks2, add2(lv2, pack2(ref.z, ref.w))), x[c + 2], x[c + 3]);
            }
          }
          if (edge) {
#pragma unroll
            for (int r = 0; r < RU; ++r) x[r] = sees(r) ? x[r] : -INFINITY;
          }
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < RU; c += CH)
            if (c < fours) top = fmaxf(fmaxf(top, fmaxf(x[c], x[c + 1])), fmaxf(x[c + 2], x[c + 3]));
          // would some weight leave the pieces' range, or has some row no reference yet?
          if (group_any(group, top > static_cast<float>(kTop) || t <= t_unset)) {
            float most = -INFINITY;  // of row `lane`, over the warp's tokens
#pragma unroll
            for (int c = 0; c < RU; c += CH) {
              if (c < fours) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                  const float w = of_order(__reduce_max_sync(kFull, order_of(x[c + i])));
                  if (lane == c + i) most = w;
                }
              }
            }
            if (lane < RT) sm.red[warp & 3][r_base + lane] = most;
            group_sync(group);
            if (token < fours) {
              const int r = r_base + token;
              const float now = fmaxf(fmaxf(sm.red[0][r], sm.red[1][r]), fmaxf(sm.red[2][r], sm.red[3][r])) - kShift;
              const float ref = sm.refs[r];
              const bool unset = __float_as_uint(ref) == kUnset;
              // raised by: nothing for a row that no token of this tile belongs to
              const float up = unset ? (now == -INFINITY ? 0.0f : now) : fmaxf(now, 0.0f);
              sm.up()[r] = up;
              sm.fac()[r] = unset ? 1.0f : ex2(-up);
              sm.root()[r] = unset ? 1.0f : ex2(-0.5f * up);
              // 0 - x is never the mark of an unset reference
              sm.refs[r] = unset && now == -INFINITY ? ref : (unset ? 0.0f : ref) - up;
            }
            group_sync(group);
#pragma unroll
            for (int c = 0; c < RU; c += CH) {
              if (c < fours) {
                const float4 u = *reinterpret_cast<const float4*>(&sm.up()[r_base + c]);
                x[c] -= u.x;
                x[c + 1] -= u.y;
                x[c + 2] -= u.z;
                x[c + 3] -= u.w;
              }
            }
            if (t > tile0) {
#pragma unroll
              for (int c = 0; c < RU; c += CH) {
                if (c < fours) {
                  const float4 f = *reinterpret_cast<const float4*>(&sm.root()[r_base + c]);
                  l[c] = l[c] * f.x * f.x;  // (a large value scale may raise a reference beyond the float range)
                  l[c + 1] = l[c + 1] * f.y * f.y;
                  l[c + 2] = l[c + 2] * f.z * f.z;
                  l[c + 3] = l[c + 3] * f.w * f.w;
                }
              }
              if (!fail) fail = !bar_wait(&sm.pv_done[(n - 1) % C::PB], ((n - 1) / C::PB) & 1, gave_up);
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < fours; c += 4) {
                float o[kPieces][4];
#pragma unroll
                for (int k = 0; k < kPieces; ++k) tmem_ld<4>(tO + c + k * NR, o[k]);
                tmem_wait_ld();
                const float4 f = *reinterpret_cast<const float4*>(&sm.fac()[r_base + c]);
#pragma unroll
                for (int k = 0; k < kPieces; ++k) {
                  tmem_tie<4>(o[k]);
                  o[k][0] *= f.x;
                  o[k][1] *= f.y;
                  o[k][2] *= f.z;
                  o[k][3] *= f.w;
                  tmem_st<4>(tO + c + k * NR, o[k]);
                }
              }
              tmem_wait_st();
            }
          }
          // weights: three 8-bit pieces each, 16 rows of a token side by side
          if (C::PB == 1 && n > 0 && !fail) fail = !bar_wait(&sm.pv_done[0], (n - 1) & 1, gave_up);
          uint8_t* dst = sp + (n % C::PB) * C::kPBytes + token * 16;
          constexpr int kNext = (NR / 16) * (kTile * 16);  // from a piece to the next
#pragma unroll
          for (int c = 0; c < RT; c += 16) {
            constexpr int kLast = RT % 16 ? 8 : 16;
            const int n16 = c + 16 <= RT ? 16 : kLast;
            uint32_t w[kPieces][4] = {};
#pragma unroll
            for (int i = 0; i < 16; i += CH) {
              if (i < n16 && c + i < RU && c + i < fours) {
                uint32_t u[kPieces][2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const int r = c + i + 2 * e;
                  const float w0 = ex2(x[r]), w1 = ex2(x[r + 1]);
                  unpack2(fma2(pack2(w0, w1), ivs2, pack2(l[r], l[r + 1])), l[r], l[r + 1]);
                  three_pieces(w0, w1, u[0][e], u[1][e], u[2][e]);
                }
                w[0][i / 4] = upper_bytes(u[0][0], u[0][1]);
                w[1][i / 4] = upper_bytes(u[1][0], u[1][1]);
                w[2][i / 4] = u[2][0] | (u[2][1] << 16);
              }
            }
            const int col = r_base + c;
            uint8_t* at = dst + (col / 16) * (kTile * 16) + (col % 16);
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
              if (RT % 16 == 0) {
                *reinterpret_cast<uint4*>(at + k * kNext) = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
              } else {  // eight columns at a time: a block of 16 may be shared with the other group
                *reinterpret_cast<uint2*>(at + k * kNext) = make_uint2(w[k][0], w[k][1]);
                if (n16 == 16) {
                  uint8_t* next = dst + ((col + 8) / 16) * (kTile * 16) + ((col + 8) % 16);
                  *reinterpret_cast<uint2*>(next + k * kNext) = make_uint2(w[k][2], w[k][3]);
                }
              }
            }
          }
          if (poison) {
#pragma unroll
            for (int r = 0; r < RU; ++r)
              if (sees(r)) l[r] = __uint_as_float(0x7fc00000u);
          }
          fence_async();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&sm.p_full[n % C::PB]);
        }
        // ---- results of the piece
        if (m > 0 && !fail) fail = !bar_wait(&sm.pv_done[(n - 1) % C::PB], ((n - 1) / C::PB) & 1, gave_up);
        fail = soft_any(fail);
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < RT; c += 8) {
          if (c < fours) {
            const float s = lane_sums<8>(l + c);
            if (lane < 8) sm.red[warp & 3][r_base + c + lane] = s;
          }
        }
        soft_sync();
        if (tid < NR && row_of(tid) < p.nrows) {
          const float ref = (m > 0 && __float_as_uint(sm.refs[tid]) != kUnset ? -sm.refs[tid] : kNoRef) + kSumExp;
          float s = sm.red[0][tid] + sm.red[1][tid] + sm.red[2][tid] + sm.red[3][tid];
          if (fail) s = __uint_as_float(0x7fc00000u);
          if (p.whole()) {
            const int gr = p.row0 + row_of(tid), t = gr / a.G, g = gr - t * a.G;
            if (a.lse) a.lse[(static_cast<int64_t>(p.b) * a.T + t) * a.Hq + p.h * a.G + g] = lse_of(ref, s);
            sm.fac()[tid] = kSumUnit / s;
          } else {
            a.part_ml[static_cast<int64_t>(p.slot) * a.slot_rows + row_of(tid)] = make_float2(ref, s);
          }
        }
        const bool whole = p.whole();
        if (whole) soft_sync();
        if (m > 0 && (warp & 3) * 32 < D) {
          const int row0 = group == 0 ? 0 : half_of(), mine = rows_mine();
          float* part = a.part_o + (static_cast<int64_t>(p.slot) * a.slot_rows + row0) * D + token;
          __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + token;
#pragma unroll 1
          for (int c = 0; c < fours; c += 8) {
            float o[8], o1[8], o2[8];  // the pieces of eight rows
            tmem_ld<8>(tO + c, o);
            tmem_ld<8>(tO + NR + c, o1);
            tmem_ld<8>(tO + 2 * NR + c, o2);
            tmem_wait_ld();
            tmem_tie<8>(o);
            tmem_tie<8>(o1);
            tmem_tie<8>(o2);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(fmaf(o2[i], 0.125f, o1[i]), 0.125f, o[i]);
            if (whole) {
              int64_t at[8];  // (read before the stores, which for all the compiler knows write there)
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                at[i] = sm.out_at[r_base + c + i];
                f[i] = sm.fac()[r_base + c + i];
              }
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (c + i < mine) from_float(o[i] * f[i], out + at[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (c + i < mine) part[(c + i) * D] = o[i] * kSumUnit;
            }
          }
        }
        tc_fence_before();
        if (a.join_here && !p.whole()) {
          soft_sync();  // the part is written
          if (tid == 0) sm.last = last_of_item(a, p, rt);
          soft_sync();
          if (sm.last) join_item<__nv_bfloat16>(a, p, rt, warp, kSoftThreads / 32);
        }
      }
      if (fail) abandon(a, sm.plan, range, rt, pieces, &sm.last);
    }
  }
  fill_empty<__nv_bfloat16>(a, tid, kMmaThreads);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free(tm, C::kCols);
}

}  // namespace spec_kv_detail
