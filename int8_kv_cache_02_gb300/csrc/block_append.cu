// kv_quant_append into block-scaled pools: fp16 K/V rows of new tokens -> 8-bit
// codes (int8 or e4m3) with one fp32 scale per (T positions, kv head).
//
// With qmax = 127 (int8) or 448 (e4m3), a = max |x| over the call's new rows of a
// block, and fits = 127.5 or 464 (the largest |x| / s that rounds to qmax within
// half a step):
//   a block without earlier rows (or whose scale is 0):  s = fl32(a / qmax)
//   else  s = s_old 2^k with the smallest k >= 0 such that a <= fl32(fits s_old) 2^k,
//         and the earlier rows' codes become round(c 2^-k)
//   new codes: round(fl32(x / s)), half to even, saturated; 0 where s = 0.
// Doubling keeps a growing block's error bounded: a code is off by half a step of
// its last scale, plus at most as much again from all halvings together (each is
// off by half a step of a scale, and the scales are a geometric series).  For e4m3
// halving a code is exact down to its subnormals.
//
// One group of threads (a warp, or a block of 256 threads) owns a (sequence,
// block, kv head, store): it loads the new rows once into registers, reduces a,
// and writes codes and scale; no two groups share a byte.  Traffic: 2 D bytes in
// and D out per row and store.
#include <cmath>

#include "block_quant.cuh"

namespace int8kv {
namespace {

// Codes of eight fp16 values.
template <bool F8>
__device__ __forceinline__ uint2 quantize_halves8(const uint4& x, float s, float inv) {
  const __half2* h = reinterpret_cast<const __half2*>(&x);
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(h[e]);
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
  }
  return quantize8<F8>(v, s, inv, false);
}

// NT threads per group; GROUPS groups per thread block; CH 16-byte pieces of new
// rows per thread (NT * CH >= rows * D / 8 for the most rows a block can get).
template <int D, bool F8, int NT, int GROUPS, int CH>
__global__ void __launch_bounds__(NT* GROUPS) block_append_kernel(
    const BlockView p, const uint16_t* __restrict__ k_new, const uint16_t* __restrict__ v_new,
    int n_seqs, int n_new, int nb, const int32_t* __restrict__ seq_pos, int pos_offset,
    const int32_t* __restrict__ page_table, int max_pages) {
  constexpr int PPR = D / 8;     // pieces per row
  static_assert(GROUPS == 1 || NT == 32, "groups of a block are single warps");
  __shared__ float red[NT / 32];
  // Dependents may start once everything before this kernel is complete (not earlier: a
  // decode of the same call reads what those kernels wrote without waiting again, which rests
  // on these two lines' order).
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  const int tid = threadIdx.x % NT;
  const unsigned unit = blockIdx.x * GROUPS + threadIdx.x / NT;     // (fewer than 2^31)
  // unit = ((sequence * nb + block) * Hkv + kv head) * 2 + store
  const bool is_v = unit & 1;
  const int kvh = (unit >> 1) % (unsigned)p.Hkv;
  const unsigned sb = (unit >> 1) / (unsigned)p.Hkv;
  const int j = sb % (unsigned)nb;
  const size_t b = sb / (unsigned)nb;
  if (b >= (size_t)n_seqs) return;
  const int T = 1 << p.t_log2;
  long long pos = (long long)__ldg(seq_pos + b) + pos_offset, skip = 0;
  if (pos < 0) {     // tokens at negative positions have no place
    skip = -pos;
    pos = 0;
    if (tid == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
  }
  const long long first = ((pos >> p.t_log2) + j) << p.t_log2;   // the block's first position
  const int r0 = j == 0 ? (int)(pos & (T - 1)) : 0;              // rows it held before
  const long long i0 = first + r0 - pos + skip;                  // its first new token
  const long long left = (long long)n_new - i0;                  // (below INT_MIN, it may be)
  if (left <= 0) return;
  const int rows = (int)min((long long)(T - r0), left);
  const long long lp = first >> p.ps_log2;
  if (lp >= max_pages) {
    if (tid == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
    return;
  }

  // the new rows, once (their loads and the table's are under way together)
  const uint16_t* src = (is_v ? v_new : k_new) + (((size_t)b * n_new + i0) * p.Hkv + kvh) * D;
  uint4 x[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = tid + c * NT, r = i / PPR;
    x[c] = r < rows ? ptx::ldg128(src + (size_t)r * p.Hkv * D + (i % PPR) * 8)
                    : make_uint4(0, 0, 0, 0);
  }
  const int page = block_page(page_table + b * max_pages, (int)lp, p);
  if (page < 0) return;
  const int slot = (int)(first & ((1 << p.ps_log2) - 1));
  const size_t ph = (size_t)page * p.Hkv + kvh;
  uint8_t* codes = (is_v ? p.v : p.k) + ((ph << p.ps_log2) + slot) * D;
  float* scale = (is_v ? p.vs : p.ks) + (ph << (p.ps_log2 - p.t_log2)) + (slot >> p.t_log2);
  const float s_old = r0 ? *scale : 0.f;

  float a = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const __half2* h = reinterpret_cast<const __half2*>(&x[c]);
    __half2 m = __habs2(h[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) m = __hmax2(m, __habs2(h[e]));
    const float2 f = __half22float2(m);
    a = fmaxf(a, fmaxf(f.x, f.y));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
  if constexpr (NT > 32) {
    if ((tid & 31) == 0) red[tid >> 5] = a;
    __syncthreads();
    a = red[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) a = fmaxf(a, red[w]);
  }

  float s;
  if (s_old > 0.f) {
    float shrink;
    s = grown_scale<F8>(s_old, a, shrink);
    if (shrink != 1.f) shrink_codes<F8>(codes, r0 * D, shrink, tid, NT);
  } else {
    s = __fdiv_rn(a, Codes<F8>::kMax);
  }
  if (tid == 0) *scale = s;
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int i = tid + c * NT, r = i / PPR;
    if (r < rows)
      *reinterpret_cast<uint2*>(codes + (size_t)(r0 + r) * D + (i % PPR) * 8) =
          s > 0.f ? quantize_halves8<F8>(x[c], s, inv) : make_uint2(0, 0);
  }
}

struct AppendCall {
  const BlockView& p;
  const uint16_t *k_new, *v_new;
  int n_seqs, n_new;
  const int32_t* seq_pos;
  int pos_offset;
  const int32_t* page_table;
  int max_pages;
  cudaStream_t stream;
};

template <int D, bool F8, int NT, int GROUPS, int CH>
cudaError_t launch(const AppendCall& c) {
  const int T = 1 << c.p.t_log2;
  const int nb = (c.n_new + T - 2) / T + 1;   // blocks that n_new tokens may touch
  const long long units = (long long)c.n_seqs * nb * c.p.Hkv * 2;
  const long long grid = (units + GROUPS - 1) / GROUPS;
  if (units > 0x7fffff00LL) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(NT * GROUPS);
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_append_kernel<D, F8, NT, GROUPS, CH>, c.p, c.k_new,
                            c.v_new, c.n_seqs, c.n_new, nb, c.seq_pos, c.pos_offset, c.page_table,
                            c.max_pages);
}

template <int D, bool F8>
cudaError_t dispatch(const AppendCall& c) {
  const int T = 1 << c.p.t_log2;
  const int pieces = (c.n_new < T ? c.n_new : T) * (D / 8);   // most new 16-byte pieces of a block
  if (pieces <= 32) return launch<D, F8, 32, 4, 1>(c);
  if (pieces <= 64) return launch<D, F8, 32, 4, 2>(c);
  if (pieces <= 128) return launch<D, F8, 32, 4, 4>(c);
  if (pieces <= 256) return launch<D, F8, 32, 4, 8>(c);
  if (pieces <= 512) return launch<D, F8, 64, 1, 8>(c);
  if (pieces <= 1024) return launch<D, F8, 128, 1, 8>(c);
  if constexpr (D >= 128)
    if (pieces > 1024 && pieces <= 2048) return launch<D, F8, 256, 1, 8>(c);
  if constexpr (D >= 256)
    if (pieces > 2048) return launch<D, F8, 512, 1, 8>(c);
  return cudaErrorNotSupported;
}

}  // namespace

cudaError_t launch_block_append(const BlockView& p, int head_dim, bool f8, const uint16_t* k_new,
                                const uint16_t* v_new, int n_seqs, int n_new,
                                const int32_t* seq_pos, int pos_offset, const int32_t* page_table,
                                int max_pages, cudaStream_t stream) {
  const AppendCall c{p, k_new, v_new, n_seqs, n_new, seq_pos, pos_offset, page_table, max_pages,
                     stream};
  switch (head_dim) {
    case 64: return f8 ? dispatch<64, true>(c) : dispatch<64, false>(c);
    case 128: return f8 ? dispatch<128, true>(c) : dispatch<128, false>(c);
    case 256: return f8 ? dispatch<256, true>(c) : dispatch<256, false>(c);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace int8kv
