// spec_kv_mma.cu -- the instantiations of the tensor-core attention kernel.
#include "spec_kv_mma.cuh"
#include "spec_kv_units.h"

namespace specv_units {
namespace {
template <int D, int NR, int RU>
const void* entry(bool sinks, int* smem_bytes) {
  *smem_bytes = spec_kv_detail::mma_smem_bytes<D, NR>();
  return sinks ? reinterpret_cast<const void*>(&spec_kv_detail::spec_kv_attention_mma_kernel<D, NR, RU, true>)
               : reinterpret_cast<const void*>(&spec_kv_detail::spec_kv_attention_mma_kernel<D, NR, RU, false>);
}
// 33 to 40 rows have a kernel of their own: 20 rows of each half fit the registers
// where 24 do not quite (36 rows of 32768 tokens: 223 us against 228)
template <int D>
const void* of_rows(int rows, bool sinks, int* smem_bytes) {
  if (rows <= 16) return entry<D, 16, 8>(sinks, smem_bytes);
  if (rows <= 32) return entry<D, 32, 16>(sinks, smem_bytes);
  if (rows <= 40) return entry<D, 48, 20>(sinks, smem_bytes);
  return entry<D, 48, 24>(sinks, smem_bytes);
}
}  // namespace

const void* kv_mma(int D, int rows, bool sinks, int* smem_bytes) {
  return D == 64 ? of_rows<64>(rows, sinks, smem_bytes) : of_rows<128>(rows, sinks, smem_bytes);
}

}  // namespace specv_units
