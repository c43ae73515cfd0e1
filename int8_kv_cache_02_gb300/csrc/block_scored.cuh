// What the attention kernels over block-scaled pools share where scores are shaped: capped by a
// tanh, biased by distance, and masked to a prefix and a sliding window.
#pragma once

#include "block_common.cuh"
#include "packed.cuh"

namespace int8kv {

// Scores z are in base-2 exponents (times log2 e), and so are the cap and the slopes here.
struct Shaping {
  float cap;                    // 0: none
  float over_cap;               // 1 / cap
  const float* slopes;          // [H], in natural units; or null
};

// The position that a row's bias is counted from, of those that a query at `last` sees (itself, the
// `window` positions up to it, 0: all, and the prefix).  A softmax is the same whatever is added to a
// whole row, so it is the one with the largest bias: the heaviest positions then have biases near 0,
// and nothing of their scores is rounded away.  (Counted from the query itself, as the formula has it,
// queries up to 3500 positions ahead of their prefix's end were 1.6e-4 off at slopes near 1.)
__device__ __forceinline__ int bias_origin(float slope, int last, int pre, int window) {
  if (slope < 0.f) return pre > 0 || window == 0 ? 0 : max(0, last - window + 1);
  return max(last, pre - 1);
}

// c tanh(z / c).  Up to |z| = c the odd polynomial x + x x^2 P(x^2), P fitted to
// (tanh(x) / x - 1) / x^2 on [0, 1] for the least relative error of tanh (4.6e-9; with its
// roundings 1.3 * 2^-24): scores far below the cap, where all the weights can lie, keep
// fp32's relative precision, which c - 2 c / (e^2x + 1) loses there (2^-22 of the cap), and nothing
// but multiply-adds is issued.  Larger ones are rare: both forms, of which each score takes its own.
// A score's bits are its own matter so, whatever stands around it, hidden or seen.
__device__ constexpr float cap_poly(int c) {
  return c == 0   ? -3.3333296e-1f
         : c == 1 ? 1.3332345e-1f
         : c == 2 ? -5.3879801e-2f
         : c == 3 ? 2.1486657e-2f
         : c == 4 ? -7.9461057e-3f
         : c == 5 ? 2.3013644e-3f
                  : -3.5845194e-4f;
}
constexpr float kTwoLog2E = 2.8853900817779268f;

// Two scores, neither beyond the cap; over: the pair of 1 / cap.
__device__ __forceinline__ uint64_t capped2(uint64_t z, uint64_t over) {
  const uint64_t x = mul2(z, over), s = mul2(x, x);
  uint64_t p = pack2(cap_poly(6), cap_poly(6));
#pragma unroll
  for (int c = 5; c >= 0; --c) p = fma2(p, s, pack2(cap_poly(c), cap_poly(c)));
  return fma2(z, mul2(s, p), z);
}

// One beyond it; per: 2 log2(e) / cap.  (e^2|x| + 1 is 1 and more, or infinite: tanh is 1 then.)
__device__ __forceinline__ float beyond_cap(float z, float cap, float per) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ptx::ex2(fabsf(z) * per) + 1.f));
  return copysignf(fmaf(-2.f * cap, r, cap), z);
}

// Two of any size.
__device__ __forceinline__ void capped_any(uint64_t z, float cap, float over_cap, float& y0, float& y1) {
  float z0, z1;
  unpack2(z, z0, z1);
  unpack2(capped2(z, pack2(over_cap, over_cap)), y0, y1);
  const float per = over_cap * kTwoLog2E;
  const float far0 = beyond_cap(z0, cap, per), far1 = beyond_cap(z1, cap, per);
  y0 = fabsf(z0) > cap ? far0 : y0;
  y1 = fabsf(z1) > cap ? far1 : y1;
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
