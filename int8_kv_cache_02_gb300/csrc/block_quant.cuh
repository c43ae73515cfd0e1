// Quantization into block-scaled pools, shared by the kernels that append to them.
#pragma once

#include "block_common.cuh"
#include "packed.cuh"

namespace int8kv {

__device__ __forceinline__ void scale8(const float (&v)[8], float f, float (&y)[8]) {
  const uint64_t f2 = pack2(f, f);
#pragma unroll
  for (int e = 0; e < 8; e += 2) unpack2(mul2(pack2(v[e], v[e + 1]), f2), y[e], y[e + 1]);
}

// Codes of eight values.  A code is decided by the IEEE quotient v / s; v * inv (inv = 1 / s) is
// within 2^-22 of it (two roundings, and the quotient's own).  Only where a rounding
// boundary of the codes lies that near to one of the eight, or the caller says so (`near`),
// are the divisions made:
//   e4m3: where v inv (1 - 2^-21) and v inv (1 + 2^-21), which enclose the quotient, have
//         different codes;
//   int8: where v inv is within 1e-4 of a half-integer (|v / s| < 128), which 127.5, the one
//         value that needs saturation, is too.
template <bool F8>
__device__ __forceinline__ uint2 quantize8(const float (&v)[8], float s, float inv, bool near) {
  float y[8];
  uint2 w;
  if constexpr (F8) {
    scale8(v, inv * (1.f - 0x1p-21f), y);
    w = round_codes8<F8>(y);
    scale8(v, inv * (1.f + 0x1p-21f), y);
    const uint2 u = round_codes8<F8>(y);
    near |= w.x != u.x || w.y != u.y;
  } else {
    scale8(v, inv, y);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      near |= fabsf(y[e] - ((y[e] + kRoundToInt) - kRoundToInt)) > 0.5f - 1.0e-4f;
    w = round_codes8<F8>(y);
  }
  if (near) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = __fdiv_rn(v[e], s);
      if constexpr (!F8) y[e] = fminf(fmaxf(y[e], -127.f), 127.f);
    }
    w = round_codes8<F8>(y);
  }
  return w;
}

// The scale of a block that holds earlier rows under scale s_old > 0, after doublings that let
// magnitude a fit; `shrink`: what its earlier codes are multiplied by.
template <bool F8>
__device__ __forceinline__ float grown_scale(float s_old, float a, float& shrink) {
  float s = s_old, lim = Codes<F8>::kFits * s_old;
  shrink = 1.f;
  for (int k = 0; k < 256 && a > lim; ++k) {   // (a finite a: fewer doublings of any scale)
    lim *= 2.f;
    s *= 2.f;
    shrink *= 0.5f;
  }
  return s;
}

// `bytes` code bytes at `codes` (16-byte aligned, a multiple of 16) become round(c * shrink), by
// threads tid of nt.
template <bool F8>
__device__ __forceinline__ void shrink_codes(uint8_t* codes, int bytes, float shrink, int tid,
                                             int nt) {
  for (int i = tid; i < bytes / 16; i += nt) {
    uint4 w = *reinterpret_cast<const uint4*>(codes + i * 16);
    uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float y[4];
      code_values<F8>(u[e], y);
#pragma unroll
      for (int f = 0; f < 4; ++f) y[f] *= shrink;
      u[e] = round_codes<F8>(y);      // (|y| <= 64, or e4m3)
    }
    *reinterpret_cast<uint4*>(codes + i * 16) = w;
  }
}

}  // namespace int8kv
