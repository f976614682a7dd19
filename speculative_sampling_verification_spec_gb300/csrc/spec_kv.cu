// spec_kv.cu -- the paged 8-bit cache: argument checks, launch planning and the C
// ABI entry points of include/spec_kv.h, with the append, general attention and
// join kernels.
#include "kernel_table.h"
#include "spec_kv_append.cuh"
#include "spec_kv_attn.cuh"
#include "spec_kv_mma.cuh"
#include "spec_kv_units.h"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <utility>

namespace {

using namespace spec_kv_detail;

// CTAs the attention's tile list is cut for: the 152 SMs times the CTAs that stay
// resident on one (constants, so that the workspace size needs no device).
constexpr int kSMs = 152;
constexpr int kMmaCtas = kSMs * 2;
// What an item costs beside its tiles, in tiles.
constexpr int kGenOverhead = 1;
constexpr int kMmaOverhead = 4;
// limits of the norms' eps, which is added to squares of values scaled by powers of two
constexpr float kLeastEps = 0x1p-80f, kMostEps = 0x1p40f;

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool pow2_page(int s) { return s == 16 || s == 32 || s == 64 || s == 128; }

spec_status check_shapes(const spec_kv_cache* c, const spec_kv_params* p) {
  if (!c || !p) return SPEC_ERR_INVALID_ARG;
  if (c->num_pages < 1 || !pow2_page(c->page_size) || c->Hkv < 1) return SPEC_ERR_INVALID_ARG;
  if (c->D < 16 || c->D > kGenMaxD || c->D % 16) return SPEC_ERR_INVALID_ARG;
  if (p->B < 0 || p->T < 1 || p->Hq < 1 || p->Hq % c->Hkv) return SPEC_ERR_INVALID_ARG;
  if (p->dtype != SPEC_F32 && p->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  // rows and tiles are counted in 32 bits
  if (static_cast<int64_t>(p->B) * p->T * p->Hq > (int64_t(1) << 30)) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

spec_status check_cache(const spec_kv_cache* c, const spec_kv_params* p) {
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale) return SPEC_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16)) return SPEC_ERR_INVALID_ARG;
  if (c->page_stride < 0 || c->head_stride < 0 || c->token_stride < 0 || c->page_stride % 16 || c->head_stride % 16 ||
      c->token_stride % 16 || c->scale_page_stride < 0 || c->scale_head_stride < 0)
    return SPEC_ERR_INVALID_ARG;
  if (c->token_stride == 0 || (c->Hkv > 1 && (c->head_stride == 0 || c->scale_head_stride == 0)) ||
      (c->num_pages > 1 && (c->page_stride == 0 || c->scale_page_stride == 0)))
    return SPEC_ERR_INVALID_ARG;
  if (!p->page_table || !p->seq_lens || p->max_pages < 1 || p->table_stride < 0) return SPEC_ERR_INVALID_ARG;
  const int64_t tiles = ((static_cast<int64_t>(p->max_pages) * c->page_size) >> kGenLogTile) + 1;
  // positions, and tiles of the whole call, are counted in 32 bits
  if (static_cast<int64_t>(p->max_pages) * c->page_size > INT_MAX - kTile) return SPEC_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(std::max(1, p->B)) * c->Hkv > (int64_t(1) << 30) / (tiles + kMmaOverhead)) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

bool bad_strides(int64_t seq, int64_t tok, int64_t head) { return seq < 0 || tok < 0 || head < 0; }
// what is written may not overlap itself
bool bad_output(const spec_kv_params* p) {
  return bad_strides(p->o_seq_stride, p->o_tok_stride, p->o_head_stride) || (p->B > 1 && p->o_seq_stride == 0) ||
         (p->T > 1 && p->o_tok_stride == 0) || (p->Hq > 1 && p->o_head_stride == 0);
}

void fill_cache(const spec_kv_cache* c, const spec_kv_params* p, KvArgs& a) {
  a.k_codes = c->k_codes;
  a.v_codes = c->v_codes;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.page_stride = c->page_stride;
  a.head_stride = c->head_stride;
  a.token_stride = c->token_stride;
  a.scale_page_stride = c->scale_page_stride;
  a.scale_head_stride = c->scale_head_stride;
  a.table = p->page_table;
  a.table_stride = p->table_stride;
  a.seq_lens = p->seq_lens;
  a.new_lens = p->new_lens;
  a.status = p->status;
  a.B = p->B;
  a.T = p->T;
  a.Hq = p->Hq;
  a.Hkv = c->Hkv;
  a.G = p->Hq / c->Hkv;
  a.D = c->D;
  a.log_page = 0;
  while ((1 << a.log_page) < c->page_size) ++a.log_page;
  a.num_pages = c->num_pages;
  a.max_pages = p->max_pages;
  a.q_seq = p->q_seq_stride;
  a.q_tok = p->q_tok_stride;
  a.q_head = p->q_head_stride;
  a.o_seq = p->o_seq_stride;
  a.o_tok = p->o_tok_stride;
  a.o_head = p->o_head_stride;
}

// All kernels of the cache are programmatic dependent launches: see start_dependents.
spec_status launch(const void* fn, int64_t grid, int threads, int smem, void* stream, void** args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelExC(&cfg, fn, args) != cudaSuccess) return SPEC_ERR_CUDA;
  specv_units::count_launches(1);
  return SPEC_OK;
}

template <typename E, int PC, bool WARP>
const void* append_ptr(bool norm) {
  return norm ? reinterpret_cast<const void*>(&spec_kv_append_kernel<E, PC, WARP, true>)
              : reinterpret_cast<const void*>(&spec_kv_append_kernel<E, PC, WARP, false>);
}
template <typename E>
const void* append_fn(bool vec, bool warp, bool norm) {
  return vec ? (warp ? append_ptr<E, 8, true>(norm) : append_ptr<E, 8, false>(norm))
             : (warp ? append_ptr<E, 1, true>(norm) : append_ptr<E, 1, false>(norm));
}

// x as the sum of two floats
void split(double x, float* hi, float* lo) {
  *hi = static_cast<float>(x);
  *lo = static_cast<float>(x - *hi);
}

// How the attention's work is cut; a function of B, T, Hq, Hkv, D and the kernel.
struct AttnPlan {
  int rows = 0, nrt = 0, nranges = 0, slot_rows = 0;
  bool join_here = false, clear = false;
  size_t off_prefix = 0, off_ml = 0, off_o = 0, ws_bytes = 0;
};

// Bytes of an item's parts that a warp of its last CTA joins, at most.
constexpr int64_t kJoinBytes = 10 << 10;
// Workspace bytes kept zero between calls: counters of the items' parts.
constexpr size_t kPartCounters = 64 * 1024;

AttnPlan plan_attention(const spec_kv_cache* c, const spec_kv_params* p, bool mma) {
  AttnPlan pl;
  const int64_t rows = static_cast<int64_t>(p->T) * (p->Hq / c->Hkv);
  const int most = mma ? kMmaRows : c->D > 128 ? 4 : 8;
  pl.nrt = static_cast<int>((rows + most - 1) / most);
  // row tiles of equal size; the general kernel's have 4 or 8 rows (4 past 128 channels)
  pl.rows = static_cast<int>((rows + pl.nrt - 1) / pl.nrt);
  if (!mma) pl.rows = pl.rows <= 4 ? 4 : 8;
  pl.slot_rows = pl.rows;
  const int ctas = mma ? kMmaCtas : kSMs * gen_ctas_an_sm(c->D > 128 ? 8 : 4, pl.rows);
  pl.nranges = std::max(1, ctas / pl.nrt);
  // with one range nothing is shared, so no partial results
  const size_t slots = pl.nranges > 1 ? static_cast<size_t>(2) * pl.nranges * pl.nrt : 0;
  // The last CTA of an item adds up its parts where that is little to read (the
  // parts of one item, if all sequences are alike); else a kernel over all rows.
  const int64_t items = static_cast<int64_t>(std::max(1, p->B)) * c->Hkv;
  const int64_t parts = (pl.nranges + items - 1) / items;
  pl.join_here = parts * pl.rows * c->D * 4 <= kJoinBytes * (mma ? kSoftThreads : kGenThreads) / 32;
  const size_t counters = round_up(static_cast<size_t>(p->B) * c->Hkv * pl.nrt * sizeof(int32_t), 256);
  pl.clear = pl.join_here && pl.nranges > 1 && counters > kPartCounters;
  pl.off_prefix = std::max(kPartCounters, counters);
  pl.off_ml = pl.off_prefix + round_up((static_cast<size_t>(p->B) + 1) * sizeof(int32_t), 256);
  pl.off_o = pl.off_ml + round_up(slots * pl.slot_rows * sizeof(float2), 256);
  pl.ws_bytes = pl.off_o + round_up(slots * pl.slot_rows * c->D * sizeof(float), 256);
  return pl;
}

// The tensor-core kernel serves bfloat16 queries of 64 or 128 channels.
bool mma_shape(const spec_kv_cache* c, const spec_kv_params* p) {
  return p->dtype == SPEC_BF16 && (c->D == 64 || c->D == 128);
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    fn.store(f, std::memory_order_release);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// Order of the pool's token, head and page dimensions in a tensor map: by stride,
// each a multiple of the one before (a dimension of one entry fits anywhere).
// False: these strides are not a tensor map's, and the general kernel serves them.
struct MapOrder {
  int64_t extent[3], stride[3];
  int box[3], at_head, at_page;
};
bool map_order(const spec_kv_cache* c, MapOrder* o) {
  struct Dim {
    int64_t extent, stride;
    int which;
  } d[3] = {{c->page_size, c->token_stride, 0}, {c->Hkv, c->head_stride, 1}, {c->num_pages, c->page_stride, 2}};
  for (Dim& x : d)
    if (x.extent == 1) x.stride = c->D;
  for (int i = 1; i < 3; ++i)
    for (int k = i; k > 0 && d[k].stride < d[k - 1].stride; --k) std::swap(d[k], d[k - 1]);
  int64_t before = c->D;
  for (int i = 0; i < 3; ++i) {
    if (d[i].stride < before || d[i].stride % before || d[i].stride >= (int64_t(1) << 40)) return false;
    before = d[i].stride;
    o->extent[i] = d[i].extent;
    o->stride[i] = d[i].stride;
    o->box[i] = d[i].which == 0 ? c->page_size : 1;
    if (d[i].which == 1) o->at_head = i;
    if (d[i].which == 2) o->at_page = i;
  }
  return true;
}

bool make_map(EncodeTiled enc, const spec_kv_cache* c, const MapOrder& o, uint8_t* base, CUtensorMap* map) {
  const cuuint64_t extent[4] = {static_cast<cuuint64_t>(c->D), static_cast<cuuint64_t>(o.extent[0]),
                                static_cast<cuuint64_t>(o.extent[1]), static_cast<cuuint64_t>(o.extent[2])};
  const cuuint64_t stride[3] = {static_cast<cuuint64_t>(o.stride[0]), static_cast<cuuint64_t>(o.stride[1]),
                                static_cast<cuuint64_t>(o.stride[2])};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(c->D), static_cast<cuuint32_t>(o.box[0]),
                             static_cast<cuuint32_t>(o.box[1]), static_cast<cuuint32_t>(o.box[2])};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, extent, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             c->D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// dynamic shared memory above 48 KB has to be allowed once for a kernel and device
bool allow_smem(const void* fn, int slot, int bytes) {
  static std::atomic<int> allowed[64][16];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  if (allowed[dev][slot].load(std::memory_order_acquire) >= bytes) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  allowed[dev][slot].store(bytes, std::memory_order_release);
  return true;
}

template <typename E, int CH, int ROWS>
const void* general_ptr(bool sinks) {
  return sinks ? reinterpret_cast<const void*>(&spec_kv_attention_kernel<E, CH, ROWS, true>)
               : reinterpret_cast<const void*>(&spec_kv_attention_kernel<E, CH, ROWS, false>);
}
template <typename E>
const void* general_fn(int D, int rows, bool sinks) {
  if (D > 128) return general_ptr<E, 8, 4>(sinks);
  return rows == 4 ? general_ptr<E, 4, 4>(sinks) : general_ptr<E, 4, 8>(sinks);
}

spec_status launch_general(const KvArgs& args, bool f32, int grid, cudaStream_t st) {
  KvArgs a = args;
  void* params[] = {&a};
  const bool sinks = a.sinks > 0;
  const void* fn = f32 ? general_fn<float>(a.D, a.rows, sinks) : general_fn<__nv_bfloat16>(a.D, a.rows, sinks);
  return launch(fn, grid, kGenThreads, 0, st, params);
}

spec_status launch_mma(const KvArgs& args, const spec_kv_cache* c, const MapOrder& order, int grid, cudaStream_t st) {
  KvArgs a = args;
  MmaMaps maps;
  EncodeTiled enc = encode_tiled();
  if (!enc || !make_map(enc, c, order, c->k_codes, &maps.k) || !make_map(enc, c, order, c->v_codes, &maps.v))
    return SPEC_ERR_CUDA;
  maps.at_head = order.at_head;
  maps.at_page = order.at_page;
  int smem = 0;
  const void* fn = specv_units::kv_mma(a.D, a.rows, a.sinks > 0, &smem);
  const int kind = a.rows <= 16 ? 0 : a.rows <= 32 ? 1 : a.rows <= 40 ? 2 : 3;
  if (!fn || !allow_smem(fn, (a.sinks > 0 ? 8 : 0) + (a.D == 128 ? 4 : 0) + kind, smem)) return SPEC_ERR_CUDA;
  void* params[] = {&a, &maps};
  return launch(fn, grid, kMmaThreads, smem, st, params);
}

}  // namespace

extern "C" {

spec_status spec_kv_append(const void* q, const void* k, const void* v, const float* cos_sin,
                           const spec_kv_cache* cache, const spec_kv_params* params, void* q_out) {
  return spec_kv_append_norm(q, k, v, cos_sin, nullptr, cache, params, q_out);
}

spec_status spec_kv_append_norm(const void* q, const void* k, const void* v, const float* cos_sin,
                                const spec_kv_norms* norms, const spec_kv_cache* cache, const spec_kv_params* params,
                                void* q_out) {
  spec_status s = check_shapes(cache, params);
  if (s != SPEC_OK) return s;
  const spec_kv_params* p = params;
  if (p->rot_dim < 0 || p->rot_dim % 2 || p->rot_dim > cache->D) return SPEC_ERR_INVALID_ARG;
  if (p->rot_dim > 0 && (!cos_sin || p->rot_len < 1 || !aligned(cos_sin, 16))) return SPEC_ERR_INVALID_ARG;
  if (norms) {
    if (!(norms->eps >= kLeastEps && norms->eps <= kMostEps)) return SPEC_ERR_INVALID_ARG;
    if (norms->q_head_stride < 0 || norms->k_head_stride < 0) return SPEC_ERR_INVALID_ARG;
    if (!aligned(norms->q_weight, 4) || !aligned(norms->k_weight, 4)) return SPEC_ERR_INVALID_ARG;
    if (norms->q_weight && !q) return SPEC_ERR_INVALID_ARG;
  }
  if (p->B == 0) return SPEC_OK;
  s = check_cache(cache, p);
  if (s != SPEC_OK) return s;
  if (!k || !v || (q == nullptr) != (q_out == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (bad_strides(p->k_seq_stride, p->k_tok_stride, p->k_head_stride) ||
      bad_strides(p->v_seq_stride, p->v_tok_stride, p->v_head_stride))
    return SPEC_ERR_INVALID_ARG;
  if (q && (bad_strides(p->q_seq_stride, p->q_tok_stride, p->q_head_stride) ||
            bad_output(p)))
    return SPEC_ERR_INVALID_ARG;
  AppendArgs g = {};
  KvArgs& a = g.a;
  fill_cache(cache, p, a);
  a.q = q;
  a.out = q_out;
  g.k = k;
  g.v = v;
  g.cos_sin = cos_sin;
  g.k_seq = p->k_seq_stride;
  g.k_tok = p->k_tok_stride;
  g.k_head = p->k_head_stride;
  g.v_seq = p->v_seq_stride;
  g.v_tok = p->v_tok_stride;
  g.v_head = p->v_head_stride;
  g.rot = p->rot_dim;
  g.rot_len = p->rot_len;
  g.interleaved = p->interleaved ? 1 : 0;
  const int S = cache->page_size;
  const int64_t es = p->dtype == SPEC_F32 ? 4 : 2;
  const auto vec_ok = [&](const void* ptr, int64_t a1, int64_t a2, int64_t a3) {
    return aligned(ptr, 16) && (a1 * es) % 16 == 0 && (a2 * es) % 16 == 0 && (a3 * es) % 16 == 0;
  };
  const bool norm = norms && (norms->q_weight || norms->k_weight);
  if (norm) {
    g.q_weight = norms->q_weight;
    g.k_weight = norms->k_weight;
    g.q_weight_head = norms->q_head_stride;
    g.k_weight_head = norms->k_head_stride;
    split(static_cast<double>(norms->eps) * cache->D, &g.eps_hi, &g.eps_lo);
    split(std::sqrt(static_cast<double>(cache->D)), &g.root_hi, &g.root_lo);
    for (g.bias = 2; g.bias < 2 * cache->D;) g.bias *= 2;
    // D eps, scaled like the squares, stays below 2^60
    g.least_exp = 127 - (60 - (std::ilogb(static_cast<double>(norms->eps) * cache->D) + 1)) / 2;
  }
  // eight pairs a thread where every chunk starts on a 16-byte boundary
  const bool vec = p->rot_dim % 16 == 0 && aligned(g.q_weight, 16) && aligned(g.k_weight, 16) &&
                   g.q_weight_head % 4 == 0 && g.k_weight_head % 4 == 0 && vec_ok(k, g.k_seq, g.k_tok, g.k_head) &&
                   vec_ok(v, g.v_seq, g.v_tok, g.v_head) &&
                   (!q || (vec_ok(q, a.q_seq, a.q_tok, a.q_head) && vec_ok(q_out, a.o_seq, a.o_tok, a.o_head)));
  int per_tok = cache->D / (vec ? 16 : 2);
  if (norm && vec) per_tok = per_tok > 8 ? 16 : per_tok > 4 ? 8 : per_tok > 2 ? 4 : per_tok;
  g.tok_threads = per_tok;
  g.one = 1.0f;
  g.units_page = (p->T - 1 + S - 1) / S + 1;
  // a unit fits a warp's registers or takes a CTA
  const bool warp = per_tok <= 32 && std::min(p->T, S) <= 32 / per_tok * kAppendWarpIter;
  const int threads = warp ? kAppendWarpThreads : kAppendCtaThreads;
  // groups of units, as large as leaves several for every warp or CTA that can be resident
  const int64_t pages = static_cast<int64_t>(p->B) * g.units_page;
  const int64_t slots = warp ? kSMs * 4 * (2048 / 32) : kSMs * kAppendCtas * 4;
  g.group_units = 1;
  while (g.group_units < 2 * cache->Hkv && pages * 2 * cache->Hkv / (2 * g.group_units) >= slots) g.group_units *= 2;
  g.group_units = std::min(g.group_units, 2 * cache->Hkv);
  g.groups_page = (2 * cache->Hkv + g.group_units - 1) / g.group_units;
  if (pages * g.groups_page > INT_MAX) return SPEC_ERR_UNSUPPORTED;
  g.groups = static_cast<int>(pages * g.groups_page);
  constexpr int kWarps = kAppendWarpThreads / 32;
  g.unit_blocks = warp ? (g.groups + kWarps - 1) / kWarps : g.groups;
  // a query thread takes several heads and rows where that leaves enough threads for all SMs
  const int64_t rows = static_cast<int64_t>(p->B) * p->T;
  g.q_heads = p->Hq % kAppendHeads == 0 && rows * p->Hq * per_tok >= int64_t(4) * kAppendHeads * kSMs * 2048 ? kAppendHeads : 1;
  const int64_t beside = std::max(1, threads / (p->Hq / g.q_heads * per_tok));
  g.q_rows_block = static_cast<int>(
      beside * std::max<int64_t>(1, std::min<int64_t>(kAppendQueryRows, rows / (beside * kSMs * 2048 / threads))));
  const int64_t q_blocks = q ? (rows + g.q_rows_block - 1) / g.q_rows_block : 0;
  if (g.unit_blocks + q_blocks > INT_MAX) return SPEC_ERR_UNSUPPORTED;
  const void* fn = p->dtype == SPEC_F32 ? append_fn<float>(vec, warp, norm) : append_fn<__nv_bfloat16>(vec, warp, norm);
  void* args[] = {&g};
  return launch(fn, g.unit_blocks + q_blocks, threads, 0, p->stream, args);
}

size_t spec_kv_attention_workspace_size(const spec_kv_cache* cache, const spec_kv_params* params) {
  if (check_shapes(cache, params) != SPEC_OK) return 0;
  // which kernel serves a call also depends on the cache's strides: room for either
  const size_t general = plan_attention(cache, params, false).ws_bytes;
  return mma_shape(cache, params) ? std::max(general, plan_attention(cache, params, true).ws_bytes) : general;
}

uint64_t spec_kv_capture_id(void* stream) {
  cudaStreamCaptureStatus state = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(static_cast<cudaStream_t>(stream), &state, &id) != cudaSuccess) {
    cudaGetLastError();  // (the default stream, beside a capture: calls on it are not part of one)
    return 0;
  }
  return state == cudaStreamCaptureStatusActive ? id : 0;
}

spec_status spec_kv_attention(const void* q, const spec_kv_cache* cache, const spec_kv_params* params, void* out,
                              float* lse) {
  return spec_kv_attention_sinks(q, cache, params, 0, out, lse);
}

spec_status spec_kv_attention_sinks(const void* q, const spec_kv_cache* cache, const spec_kv_params* params,
                                    int32_t sinks, void* out, float* lse) {
  spec_status s = check_shapes(cache, params);
  if (s != SPEC_OK) return s;
  const spec_kv_params* p = params;
  if (p->window < 0 || sinks < 0 || !std::isfinite(p->scale)) return SPEC_ERR_INVALID_ARG;
  if (p->B == 0) return SPEC_OK;
  s = check_cache(cache, p);
  if (s != SPEC_OK) return s;
  if (!q || !out || bad_strides(p->q_seq_stride, p->q_tok_stride, p->q_head_stride) || bad_output(p))
    return SPEC_ERR_INVALID_ARG;
  if (!p->workspace || !aligned(p->workspace, 256) ||
      p->workspace_bytes < spec_kv_attention_workspace_size(cache, params))
    return SPEC_ERR_INVALID_ARG;
  MapOrder order = {};
  const bool mma = mma_shape(cache, p) && map_order(cache, &order);
  const AttnPlan pl = plan_attention(cache, p, mma);
  KvArgs a = {};
  fill_cache(cache, p, a);
  a.q = q;
  a.out = out;
  a.lse = lse;
  a.window = p->window;
  a.sinks = p->window > 0 ? sinks : 0;
  a.scale2 = static_cast<float>(static_cast<double>(p->scale) * 1.4426950408889634);
  a.rows = pl.rows;
  a.nrt = pl.nrt;
  a.log_tile = mma ? 7 : kGenLogTile;
  a.nranges = pl.nranges;
  a.overhead = mma ? kMmaOverhead : kGenOverhead;
  a.join_here = pl.join_here;
  a.slot_rows = pl.slot_rows;
  a.q_vec = aligned(q, 16) && a.q_seq % 8 == 0 && a.q_tok % 8 == 0 && a.q_head % 8 == 0;
  const int64_t ob = 4 * (p->dtype == SPEC_F32 ? 4 : 2);  // bytes of four channels
  a.o_vec = aligned(out, static_cast<uintptr_t>(ob)) && a.o_seq % 4 == 0 && a.o_tok % 4 == 0 && a.o_head % 4 == 0;
  char* ws = static_cast<char*>(p->workspace);
  a.arrived = reinterpret_cast<int32_t*>(ws);
  a.prefix = reinterpret_cast<int32_t*>(ws + pl.off_prefix);
  a.part_ml = reinterpret_cast<float2*>(ws + pl.off_ml);
  a.part_o = reinterpret_cast<float*>(ws + pl.off_o);
  const bool f32 = p->dtype == SPEC_F32;
  cudaStream_t st = static_cast<cudaStream_t>(p->stream);
  if (pl.clear && cudaMemsetAsync(ws, 0, pl.off_prefix, st) != cudaSuccess) return SPEC_ERR_CUDA;
  const int grid = pl.nranges * pl.nrt;
  s = mma ? launch_mma(a, cache, order, grid, st) : launch_general(a, f32, grid, st);
  if (s != SPEC_OK) return s;
  if (pl.join_here || pl.nranges == 1) return SPEC_OK;
  void* args[] = {&a};
  const void* jn = f32 ? reinterpret_cast<const void*>(&spec_kv_join_kernel<float>)
                       : reinterpret_cast<const void*>(&spec_kv_join_kernel<__nv_bfloat16>);
  return launch(jn, static_cast<int64_t>(a.B) * a.T * a.Hq, 32 * kJoinWarps, 0, st, args);
}

}  // extern "C"
