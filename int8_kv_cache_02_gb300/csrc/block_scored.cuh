// What the attention kernels over block-scaled pools share where scores are shaped: capped by a
// tanh, biased by distance, and masked to a prefix and a sliding window.
#pragma once

#include "block_common.cuh"

namespace int8kv {

// Scores z are in base-2 exponents (times log2 e), and so are the cap and the slopes here.
struct Shaping {
  float cap;                    // 0: none
  float over_cap;               // 1 / cap
  const float* slopes;          // [H], in natural units; or null
};

// c tanh(z / c).  Up to |z| = c the odd polynomial x + x x^2 P(x^2), P fitted to
// (tanh(x) / x - 1) / x^2 on [0, 1] for the least relative error of tanh (4.6e-9; with its
// roundings 1.3 * 2^-24): scores far below the cap, where all the weights can lie, keep
// fp32's relative precision, which 1 - 2 / (e^2x + 1) loses there, and nothing but
// multiply-adds is issued.  Larger ones are rare: a branch.
__device__ __forceinline__ float capped(float z, float cap, float over_cap) {
  const float x = z * over_cap, s = x * x;
  float p = -3.5845194e-4f;
  p = fmaf(p, s, 2.3013644e-3f);
  p = fmaf(p, s, -7.9461057e-3f);
  p = fmaf(p, s, 2.1486657e-2f);
  p = fmaf(p, s, -5.3879801e-2f);
  p = fmaf(p, s, 1.3332345e-1f);
  p = fmaf(p, s, -3.3333296e-1f);
  float y = fmaf(z, s * p, z);
  if (s > 1.f) {
    const float e = ptx::ex2(fabsf(x) * 2.8853900817779268f);      // e^2|x|; beyond fp32: tanh is 1
    y = copysignf(cap - cap * __fdividef(2.f, fminf(e, 1e30f) + 1.f), z);
  }
  return y;
}

// attn_decode_scored_int8's arguments beside those of a plain decode call.
struct BlockScoredArgs : BlockDecodeArgs {
  Shaping shape;
  const int32_t* prefix_lens;   // [B], or null: `prefix` for every sequence
  int prefix;
};

cudaError_t launch_block_decode_scored(const BlockScoredArgs& a, int head_dim, bool f8,
                                       cudaStream_t stream);

}  // namespace int8kv
