// Block-scaled decode at head_dim 128.
#include "decode_block.cuh"

namespace int8kv {
INT8KV_DECODE_BLOCK_INSTANCE(128)
}  // namespace int8kv
