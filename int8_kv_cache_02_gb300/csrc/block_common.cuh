// Pieces shared by the kernels over block-scaled pools (INT8KV_K8V8_BLOCK,
// INT8KV_F8_BLOCK): the pool as they see it, and the conversions between codes
// and values.
//
// A block is T = group_size consecutive positions of one kv head, T dividing the
// page size; its codes share one fp32 scale s, value = code * s.
#pragma once

#include <cstdint>

#include <cuda_fp16.h>

#include "common.cuh"
#include "ptx.cuh"

namespace int8kv {

// ---- host side: what a pool's variant says, and limits ----------------------
inline bool block_variant(int variant) {
  return variant == INT8KV_K8V8_BLOCK || variant == INT8KV_F8_BLOCK;
}
inline bool is_block(const int8kv_pool* p) { return block_variant(p->variant); }
inline bool is_f8(const int8kv_pool* p) { return p->variant == INT8KV_F8_BLOCK; }

constexpr int kBlockKernel = 2;       // index of its decode kernel in int8kv_pool::resident,
constexpr int kBlockClusters = 0;     // and of how many clusters of its blocks run at once
constexpr int kBlockCluster = 8;      // blocks of a cluster that share a unit
constexpr int kBlockSingle = 65536;   // values (positions x head_dim) of a context decoded in one
                                      // block per unit: at most these, or half of them where
constexpr int kBlockJoined = 1 << 19; // clusters may take the unit, up to these
constexpr int kBlockMostPositions = 1 << 30;   // of a page-table row (positions count in 32 bits)

// Whether the pool's device is the current one, on which the launches go.
inline bool on_current_device(const int8kv_pool* p) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == p->device;
}

// The layer of a block-scaled pool that a kernel works on.
struct BlockView {
  uint8_t* k;        // codes [n_pages][Hkv][ps][D], one byte each
  uint8_t* v;
  float* ks;         // scales [n_pages][Hkv][ps / T]
  float* vs;
  int32_t* err;      // device error word, or null
  int n_pages, Hkv;
  int ps_log2, t_log2;   // page size and T
};

inline int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

inline BlockView block_view(const int8kv_pool* p, int layer) {
  const size_t rows = (size_t)p->n_pages * p->n_kv_heads * p->page_size;
  BlockView b;
  b.k = (uint8_t*)p->k_store + (size_t)layer * rows * p->head_dim;
  b.v = (uint8_t*)p->v_store + (size_t)layer * rows * p->head_dim;
  b.ks = (float*)p->k_scales + (size_t)layer * (rows / p->group_size);
  b.vs = (float*)p->v_scales + (size_t)layer * (rows / p->group_size);
  b.err = p->dev_error;
  b.n_pages = p->n_pages;
  b.Hkv = p->n_kv_heads;
  b.ps_log2 = log2_of(p->page_size);
  b.t_log2 = log2_of(p->group_size);
  return b;
}

// A page-table entry, or -1 (flagged) when it names no page of the pool.
__device__ __forceinline__ int block_page(const int32_t* row, int lp, const BlockView& p) {
  const int pg = __ldg(row + lp);
  if (pg < 0 || pg >= p.n_pages) {
    flag_error(p.err, INT8KV_DEVERR_PAGE_ID);
    return -1;
  }
  return pg;
}

// A length clamped to [0, what a page-table row holds]; a longer one is flagged.
__device__ __forceinline__ int block_length(int len, int max_pages, const BlockView& p) {
  const long long cap = (long long)max_pages << p.ps_log2;
  if (len > cap) {
    flag_error(p.err, INT8KV_DEVERR_LENGTH);
    return (int)cap;
  }
  return len < 0 ? 0 : len;
}

// Codes of one kind: largest code, and the largest |x| / s that still rounds to
// it without losing more than half a step (127 + 1/2; 448 + half the step 32).
template <bool F8>
struct Codes {
  static constexpr float kMax = F8 ? 448.f : 127.f;
  static constexpr float kFits = F8 ? 464.f : 127.5f;
};

// Two codes as an fp16 pair, exactly.  int8: bytes 0 and 2 of x (c ^ 0x80 = c + 128
// under the fp16 exponent of 1024, less 1152; Kim et al., "Who Says Elephants
// Can't Run", 2022).  e4m3: the two low bytes.
template <bool F8>
__device__ __forceinline__ uint32_t codes_to_h2(uint32_t x) {
  if constexpr (F8) {
    uint32_t h;
    asm("{ .reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(h)
        : "r"(x));
    return h;
  } else {
    const uint32_t b = (x & 0x00FF00FFu) ^ 0x64806480u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&b),
                              __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// The pair behind the one that codes_to_h2 takes from the same word: int8 bytes 1 and 3, e4m3 the
// two high bytes.
template <bool F8>
__device__ __forceinline__ uint32_t codes_behind_to_h2(uint32_t x) {
  if constexpr (F8) {
    uint32_t h;
    asm("{ .reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}"
        : "=r"(h)
        : "r"(x));
    return h;
  } else {
    return codes_to_h2<F8>(x >> 8);
  }
}

// Two words as words of pairs: the first and second byte of a beside those of b
// (first), and the third and fourth (second), in the order codes_to_h2 wants.
template <bool F8>
__device__ __forceinline__ void pair_words(uint32_t a, uint32_t b, uint32_t& first,
                                           uint32_t& second) {
  first = ptx::prmt(a, b, F8 ? 0x5140 : 0x5410);
  second = ptx::prmt(a, b, F8 ? 0x7362 : 0x7632);
}

constexpr float kRoundToInt = 12582912.f;   // 1.5 * 2^23

// Four values in units of the scale, rounded to nearest even, as four code bytes (y[0]
// in the lowest).  e4m3 saturates; int8 takes |y| < 127.5.
template <bool F8>
__device__ __forceinline__ uint32_t round_codes(const float (&y)[4]) {
  if constexpr (F8) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y[1]), "f"(y[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(y[3]), "f"(y[2]));
    return (uint32_t)lo | ((uint32_t)hi << 16);
  } else {
    // y + 1.5 * 2^23 is the nearest integer (ties to even) plus that, exactly: its low byte
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = __float_as_uint(y[i] + kRoundToInt);
    return ptx::prmt(ptx::prmt(c[0], c[1], 0x0040), ptx::prmt(c[2], c[3], 0x0040), 0x5410);
  }
}

template <bool F8>
__device__ __forceinline__ uint2 round_codes8(const float (&y)[8]) {
  const float a[4] = {y[0], y[1], y[2], y[3]}, b[4] = {y[4], y[5], y[6], y[7]};
  return make_uint2(round_codes<F8>(a), round_codes<F8>(b));
}

// Four code bytes as fp32 values in units of the scale.
template <bool F8>
__device__ __forceinline__ void code_values(uint32_t w, float (&y)[4]) {
  const uint32_t a = codes_to_h2<F8>(w), b = codes_behind_to_h2<F8>(w);
  const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
  y[0] = fa.x;
  y[1] = F8 ? fa.y : fb.x;
  y[2] = F8 ? fb.x : fa.y;
  y[3] = fb.y;
}

struct BlockDecodeArgs {
  BlockView pool;
  const uint16_t* q;          // [B][Q][H][D] fp16
  const int32_t* seq_lens;    // [B], or null: `length` for the one sequence (a prefill chunk)
  int length;
  const int32_t* page_table;  // [B][max_pages]
  float* out;                 // [B][Q][H][D]
  float* part_o;              // [slots][width][D] normalised partial outputs
  float2* part_ml;            // [slots][width] their softmax reference m and sum l, apart: in one
                              // float m + log2 l, a large m would round l away
  int2* part_units;           // [units] first partial and number of them (1: none, it is in out)
  int B, H, G, Q, max_pages, window;
  int n_cg, width;            // column groups per (sequence, kv head), columns of each
  int shares;                 // blocks of the balanced schedule, or 0: `cluster` blocks per unit
  int cluster;                // 1 or kBlockCluster
  float scale_log2;           // softmax_scale * log2(e)
  // Whether the kernel launched just before appends position seq_lens[b] - 1 of every
  // sequence: then only the blocks of those positions are waited for.
  bool appended;
};

cudaError_t launch_block_append(const BlockView& p, int head_dim, bool f8, const uint16_t* k_new,
                                const uint16_t* v_new, int n_seqs, int n_new,
                                const int32_t* seq_pos, int pos_offset, const int32_t* page_table,
                                int max_pages, cudaStream_t stream);
cudaError_t launch_block_decode(const BlockDecodeArgs& a, int head_dim, bool f8,
                                cudaStream_t stream);
// Blocks of the decode kernel resident at once on the current device (and the
// kernel's shared-memory attribute set there); <= 0 on a CUDA error.
int block_decode_resident(int head_dim, bool f8);
// Clusters of kBlockCluster of its blocks that run at once; 0 where none does.
int block_decode_clusters(int head_dim, bool f8);

}  // namespace int8kv
