// The prefill kernel of block-scaled pools: its launcher.
#pragma once

#include "block_common.cuh"

namespace int8kv {

// Attention of a prefill chunk, and the joining of a.n_splits splits (a.pool is not used).
// expire_us: 0, or the diagnostic that lets a wait of every block run out after so long.
cudaError_t launch_block_prefill(const BlockView& pool, const PrefillArgs& a, int head_dim, bool f8,
                                 uint32_t expire_us, cudaStream_t stream);

}  // namespace int8kv
