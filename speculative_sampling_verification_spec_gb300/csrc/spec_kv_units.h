// spec_kv_units.h -- the paged cache's kernels that are compiled apart from their
// launches, so that units compile in parallel (kernel_table.h has verification's).
#pragma once

namespace specv_units {

// the tensor-core attention over the paged cache for head size D (64, 128) and up
// to `rows` rows (at most 48) a row tile, for calls with or without sinks, and its
// shared memory
const void* kv_mma(int D, int rows, bool sinks, int* smem_bytes);

}  // namespace specv_units
