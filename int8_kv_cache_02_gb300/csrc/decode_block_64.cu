// Block-scaled decode at head_dim 64.
#include "decode_block.cuh"

namespace int8kv {
INT8KV_DECODE_BLOCK_INSTANCE(64)
}  // namespace int8kv
