// The prefill kernel of block-scaled pools: its launcher.
#pragma once

#include "block_scored.cuh"

namespace int8kv {

struct PrefillShape {
  Shaping scores;
  int window, prefix;         // 0: none; positions 0 .. prefix - 1 are seen by every query
};

// Attention of a prefill chunk, and the joining of a.n_splits splits (a.pool is not used).
// expire_us: 0, or the diagnostic that lets a wait of every block run out after so long.
// shape: null for plain scores.
cudaError_t launch_block_prefill(const BlockView& pool, const PrefillArgs& a, int head_dim, bool f8,
                                 uint32_t expire_us, const PrefillShape* shape, cudaStream_t stream);

}  // namespace int8kv
