// spec_kv_mma.cu -- the instantiations of the tensor-core attention kernel.
#include "kernel_table.h"
#include "spec_kv_mma.cuh"

namespace specv_units {
namespace {
template <int D, int NR>
const void* entry(int* smem_bytes) {
  *smem_bytes = spec_kv_detail::mma_smem_bytes<D, NR>();
  return reinterpret_cast<const void*>(&spec_kv_detail::spec_kv_attention_mma_kernel<D, NR>);
}
template <int D>
const void* of_rows(int NR, int* smem_bytes) {
  switch (NR) {
    case 16: return entry<D, 16>(smem_bytes);
    case 32: return entry<D, 32>(smem_bytes);
    case 48: return entry<D, 48>(smem_bytes);
  }
  return nullptr;
}
}  // namespace

const void* kv_mma(int D, int NR, int* smem_bytes) {
  if (D == 64) return of_rows<64>(NR, smem_bytes);
  if (D == 128) return of_rows<128>(NR, smem_bytes);
  return nullptr;
}

}  // namespace specv_units
