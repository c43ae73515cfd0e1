// Block-scaled decode at head_dim 256.
#include "decode_block.cuh"

namespace int8kv {
INT8KV_DECODE_SCORED_INSTANCE(256)
}  // namespace int8kv
