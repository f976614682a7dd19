// spec_kv_mma.cu -- the instantiations of the tensor-core attention kernel.
#include "kernel_table.h"
#include "spec_kv_mma.cuh"

namespace specv_units {
namespace {
template <int D, int NR, int RU>
const void* entry(int* smem_bytes) {
  *smem_bytes = spec_kv_detail::mma_smem_bytes<D, NR>();
  return reinterpret_cast<const void*>(&spec_kv_detail::spec_kv_attention_mma_kernel<D, NR, RU>);
}
// 33 to 40 rows have a kernel of their own: 20 rows of each half fit the registers
// where 24 do not quite (36 rows of 32768 tokens: 223 us against 228)
template <int D>
const void* of_rows(int rows, int* smem_bytes) {
  if (rows <= 16) return entry<D, 16, 8>(smem_bytes);
  if (rows <= 32) return entry<D, 32, 16>(smem_bytes);
  if (rows <= 40) return entry<D, 48, 20>(smem_bytes);
  return entry<D, 48, 24>(smem_bytes);
}
}  // namespace

const void* kv_mma(int D, int rows, int* smem_bytes) {
  return D == 64 ? of_rows<64>(rows, smem_bytes) : of_rows<128>(rows, smem_bytes);
}

}  // namespace specv_units
