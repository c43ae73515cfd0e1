// kv_rope_append: queries and keys of new tokens rotated by their positions, and keys and
// values appended as kv_quant_append does, in one kernel.
//
// Pair i of the first R values of a row, (a, b) = values (i, i + R/2) or (2i, 2i + 1), with c and s
// from the table's row of the position that pair i goes by:
//   a' = fl(fl(a c) - fl(b s)),   b' = fl(fl(b c) + fl(a s))
// in fp32, every operation rounded by itself, so that the result does not depend on how a
// compiler joins them.  Queries are rounded once, to fp16.  Keys are not rounded before
// they are quantized: scale and codes come from the fp32 values.
//
// What rotates together is kept together: a "twin" is two 16-byte pieces of a row (8 values each)
// that one thread takes, pieces t and t + R/16 for t < R/16, and neighbours behind the
// rotated part.  In either pairing a twin's eight pairs use eight cosines and eight sines
// in pieces of four, and a piece of four pairs that go by one position is two 16-byte loads.
#include <cmath>

#include "block_quant.cuh"
#include "quant_row.cuh"
#include "q4_row.cuh"

namespace int8kv {
namespace {

struct RopeArgs {
  const uint16_t *q, *k, *v;      // tokens q_stride, k_stride, v_stride values apart
  uint16_t* q_out;                // [n_seqs][n_new][H][D]
  long long q_stride, k_stride, v_stride;
  int n_seqs, n_new, H, Hkv;
  const int32_t* seq_pos;         // [n_seqs]
  const int32_t* new_lens;        // [n_seqs], or null: n_new each
  const float* table;             // [n_table][R]: R/2 cosines, R/2 sines
  int n_table, R;
  bool pairs;                     // values (2i, 2i + 1), else (i, i + R/2)
  const int32_t* positions;       // [axes][n_seqs][n_new], or null: seq_pos[b] + i
  uint8_t axes[32];               // which axis pair i goes by, two bits each
  const int32_t* page_table;
  int max_pages;
  int32_t* err;
  unsigned append_blocks;         // the blocks behind them rotate queries
  int heads;                      // query heads that one of their threads takes
};

// Tokens that sequence b brings.
__device__ __forceinline__ int tokens_of(const RopeArgs& a, size_t b) {
  if (!a.new_lens) return a.n_new;
  const int n = __ldg(a.new_lens + b);
  if (n > a.n_new) flag_error(a.err, INT8KV_DEVERR_LENGTH);
  return max(0, min(n, a.n_new));
}

// The table's row of the position that token i of sequence b has on an axis; null (flagged)
// outside the table.
__device__ __forceinline__ const float* table_row(const RopeArgs& a, size_t b, int i, int axis) {
  const long long at = a.positions
                           ? __ldg(a.positions + ((size_t)axis * a.n_seqs + b) * a.n_new + i)
                           : (long long)__ldg(a.seq_pos + b) + i;
  if (at < 0 || at >= a.n_table) {
    flag_error(a.err, INT8KV_DEVERR_LENGTH);
    return nullptr;
  }
  return a.table + (size_t)at * a.R;
}

// Cosines and sines of N consecutive pairs from pair i on (N a multiple of 4, i too).
template <int N>
__device__ __forceinline__ void load_turns(const RopeArgs& a, size_t b, int tok, int i, float* c,
                                           float* s) {
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    const unsigned by = a.axes[(i + k) >> 2], first = by & 3;
    if (by == first * 0x55u) {
      const float* row = table_row(a, b, tok, first);
      float4 x = make_float4(1.f, 1.f, 1.f, 1.f), y = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row) {
        x = __ldg(reinterpret_cast<const float4*>(row + i + k));
        y = __ldg(reinterpret_cast<const float4*>(row + a.R / 2 + i + k));
      }
      c[k] = x.x, c[k + 1] = x.y, c[k + 2] = x.z, c[k + 3] = x.w;
      s[k] = y.x, s[k + 1] = y.y, s[k + 2] = y.z, s[k + 3] = y.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* row = table_row(a, b, tok, by >> (2 * e) & 3);
        c[k + e] = row ? __ldg(row + i + k + e) : 1.f;
        s[k + e] = row ? __ldg(row + a.R / 2 + i + k + e) : 0.f;
      }
    }
  }
}

__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
  const float x = a;
  a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(x, s));
}

__device__ __forceinline__ void halves_to_floats(const uint4& x, float (&f)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(&x);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 y = __half22float2(h[e]);
    f[2 * e] = y.x;
    f[2 * e + 1] = y.y;
  }
}

// A twin's two pieces within a row.
__device__ __forceinline__ void twin_pieces(int t, int R, int& x, int& y) {
  if (t < R / 16) {
    x = t;
    y = t + R / 16;
  } else {
    x = 2 * t;
    y = x + 1;
  }
}

// The turns of twin t, and the twin turned.
struct Turns {
  float c[8], s[8];
};
__device__ __forceinline__ void twin_turns(const RopeArgs& a, size_t b, int tok, int t, Turns& w) {
  if (a.pairs) {
    load_turns<4>(a, b, tok, 4 * t, w.c, w.s);
    load_turns<4>(a, b, tok, a.R / 4 + 4 * t, w.c + 4, w.s + 4);
  } else {
    load_turns<8>(a, b, tok, 8 * t, w.c, w.s);
  }
}
__device__ __forceinline__ void turn_twin(bool pairs, const Turns& w, float (&x)[8], float (&y)[8]) {
  if (pairs) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      turn(x[2 * e], x[2 * e + 1], w.c[e], w.s[e]);
      turn(y[2 * e], y[2 * e + 1], w.c[4 + e], w.s[4 + e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) turn(x[e], y[e], w.c[e], w.s[e]);
  }
}

// Queries: a thread takes one twin of a token for `a.heads` heads, whose turns it loads once.
// (q_out may be q: a value is read and written by one thread, in this order, so not through
// the read-only path.)
template <int D>
__device__ __forceinline__ void rotate_queries(const RopeArgs& a, unsigned thread) {
  constexpr int TW = D / 16, TOGETHER = 4;
  const unsigned groups = (a.H + a.heads - 1) / a.heads;
  const int t = thread % TW;
  const unsigned job = thread / TW, tok = job / groups;
  const int h0 = job % groups * a.heads;
  if (tok >= (unsigned)a.n_seqs * a.n_new) return;
  const unsigned b = tok / a.n_new;
  const int i = tok % a.n_new;
  if (i >= tokens_of(a, b)) return;
  int px, py;
  twin_pieces(t, a.R, px, py);
  const bool turned = t < a.R / 16;
  Turns w;
  const int end = min(a.H, h0 + a.heads);
  const uint16_t* from = a.q + (size_t)tok * a.q_stride;
  uint16_t* to = a.q_out + (size_t)tok * a.H * D;
  for (int h = h0; h < end; h += TOGETHER) {
    uint4 x[TOGETHER], y[TOGETHER];
#pragma unroll
    for (int k = 0; k < TOGETHER; ++k)
      if (h + k < end) {
        x[k] = *reinterpret_cast<const uint4*>(from + (h + k) * D + 8 * px);
        y[k] = *reinterpret_cast<const uint4*>(from + (h + k) * D + 8 * py);
      }
    if (h == h0 && turned) twin_turns(a, b, i, t, w);
#pragma unroll
    for (int k = 0; k < TOGETHER; ++k)
      if (h + k < end) {
        if (turned) {
          float fx[8], fy[8];
          halves_to_floats(x[k], fx);
          halves_to_floats(y[k], fy);
          turn_twin(a.pairs, w, fx, fy);
          x[k] = make_uint4(ptx::pack_f16x2(fx[0], fx[1]), ptx::pack_f16x2(fx[2], fx[3]),
                            ptx::pack_f16x2(fx[4], fx[5]), ptx::pack_f16x2(fx[6], fx[7]));
          y[k] = make_uint4(ptx::pack_f16x2(fy[0], fy[1]), ptx::pack_f16x2(fy[2], fy[3]),
                            ptx::pack_f16x2(fy[4], fy[5]), ptx::pack_f16x2(fy[6], fy[7]));
        }
        *reinterpret_cast<uint4*>(to + (h + k) * D + 8 * px) = x[k];
        *reinterpret_cast<uint4*>(to + (h + k) * D + 8 * py) = y[k];
      }
  }
}

// ---- block-scaled pools ------------------------------------------------------
// As in the append kernel, one group of threads (a warp, or a block of NT threads) owns a
// (sequence, block, kv head, store): it loads the new rows once, turns K's, reduces the
// largest magnitude, and writes codes and scale.  CH twins per thread, as fp32.
template <int D, bool F8, int NT, int GROUPS, int CH>
__global__ void __launch_bounds__(NT* GROUPS)
    rope_block_kernel(const __grid_constant__ RopeArgs a, const BlockView p, int nb) {
  constexpr int TW = D / 16;     // twins per row
  static_assert(GROUPS == 1 || NT == 32, "groups of a block are single warps");
  __shared__ float red[NT / 32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  if (blockIdx.x >= a.append_blocks) {
    rotate_queries<D>(a, (blockIdx.x - a.append_blocks) * (NT * GROUPS) + threadIdx.x);
    return;
  }
  const int tid = threadIdx.x % NT;
  const unsigned unit = blockIdx.x * GROUPS + threadIdx.x / NT;     // (fewer than 2^31)
  // unit = ((sequence * nb + block) * Hkv + kv head) * 2 + store
  const bool is_v = unit & 1;
  const int kvh = (unit >> 1) % (unsigned)p.Hkv;
  const unsigned sb = (unit >> 1) / (unsigned)p.Hkv;
  const int j = sb % (unsigned)nb;
  const size_t b = sb / (unsigned)nb;
  if (b >= (size_t)a.n_seqs) return;
  const int T = 1 << p.t_log2;
  long long pos = __ldg(a.seq_pos + b), skip = 0;
  const int count = tokens_of(a, b);
  if (pos < 0) {     // tokens at negative positions have no place
    skip = -pos;
    pos = 0;
    if (tid == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
  }
  const long long first = ((pos >> p.t_log2) + j) << p.t_log2;   // the block's first position
  const int r0 = j == 0 ? (int)(pos & (T - 1)) : 0;              // rows it held before
  const long long i0 = first + r0 - pos + skip;                  // its first new token
  const int rows = (int)min((long long)(T - r0), (long long)count - i0);
  if (rows <= 0) return;
  const long long lp = first >> p.ps_log2;
  if (lp >= a.max_pages) {
    if (tid == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
    return;
  }
  const long long stride = is_v ? a.v_stride : a.k_stride;
  const uint16_t* src = (is_v ? a.v : a.k) + (size_t)(b * a.n_new + i0) * stride + kvh * D;
  uint4 raw[CH][2];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int n = tid + c * NT, r = n / TW;
    int px, py;
    twin_pieces(n % TW, a.R, px, py);
    raw[c][0] = raw[c][1] = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      raw[c][0] = ptx::ldg128(src + r * stride + 8 * px);
      raw[c][1] = ptx::ldg128(src + r * stride + 8 * py);
    }
  }
  const int page = block_page(a.page_table + b * a.max_pages, (int)lp, p);
  if (page < 0) return;
  const int slot = (int)(first & ((1 << p.ps_log2) - 1));
  const size_t ph = (size_t)page * p.Hkv + kvh;
  uint8_t* codes = (is_v ? p.v : p.k) + ((ph << p.ps_log2) + slot) * D;
  float* scale = (is_v ? p.vs : p.ks) + (ph << (p.ps_log2 - p.t_log2)) + (slot >> p.t_log2);
  const float s_old = r0 ? *scale : 0.f;

  float x[CH][2][8], top = 0.f;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int n = tid + c * NT, r = n / TW, t = n % TW;
    halves_to_floats(raw[c][0], x[c][0]);
    halves_to_floats(raw[c][1], x[c][1]);
    if (!is_v && t < a.R / 16 && r < rows) {
      Turns w;
      twin_turns(a, b, (int)i0 + r, t, w);
      turn_twin(a.pairs, w, x[c][0], x[c][1]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x[c][0][e]), fabsf(x[c][1][e])));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if constexpr (NT > 32) {
    if ((tid & 31) == 0) red[tid >> 5] = top;
    __syncthreads();
    top = red[0];
#pragma unroll
    for (int w = 1; w < NT / 32; ++w) top = fmaxf(top, red[w]);
  }
  float s;
  if (s_old > 0.f) {
    float shrink;
    s = grown_scale<F8>(s_old, top, shrink);
    if (shrink != 1.f) shrink_codes<F8>(codes, r0 * D, shrink, tid, NT);
  } else {
    s = __fdiv_rn(top, Codes<F8>::kMax);
  }
  if (tid == 0) *scale = s;
  // (products with a small sine may be far below what fp16 holds, where 1 / s has no fp32 value)
  const bool tiny = s < 0x1p-100f;
  const float inv = tiny ? 0.f : __frcp_rn(s);
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int n = tid + c * NT, r = n / TW;
    int px, py;
    twin_pieces(n % TW, a.R, px, py);
    if (r < rows) {
      uint8_t* row = codes + (size_t)(r0 + r) * D;
      *reinterpret_cast<uint2*>(row + 8 * px) =
          s > 0.f ? quantize8<F8>(x[c][0], s, inv, tiny) : make_uint2(0, 0);
      *reinterpret_cast<uint2*>(row + 8 * py) =
          s > 0.f ? quantize8<F8>(x[c][1], s, inv, tiny) : make_uint2(0, 0);
    }
  }
}

// ---- pools with a scale for each row --------------------------------------
// A warp takes a (sequence, token, kv head), lane l values [l VPL, (l + 1) VPL) of K and V, as
// the append kernel of these pools; a value's partner is in the lane R/2 values further.
template <int VPL>
__device__ __forceinline__ void turn_row(const RopeArgs& a, size_t b, int tok, int lane,
                                         float (&x)[VPL]) {
  const int at = lane * VPL, half = a.R / 2;
  if (a.pairs) {
    if (at < a.R) {
#pragma unroll
      for (int e = 0; e < VPL; e += 2) {
        const int i = (at + e) / 2;
        const float* row = table_row(a, b, tok, a.axes[i >> 2] >> (2 * (i & 3)) & 3);
        if (row) turn(x[e], x[e + 1], __ldg(row + i), __ldg(row + half + i));
      }
    }
    return;
  }
  const int away = half / VPL;
  const bool second = at >= half && at < a.R;
  const int partner = at < half ? lane + away : second ? lane - away : lane;
#pragma unroll
  for (int e = 0; e < VPL; ++e) {
    float mine = x[e], other = __shfl_sync(0xffffffffu, x[e], partner);
    if (at < a.R) {
      const int i = (second ? at - half : at) + e;
      const float* row = table_row(a, b, tok, a.axes[i >> 2] >> (2 * (i & 3)) & 3);
      if (row) {
        float& first = second ? other : mine;
        float& last = second ? mine : other;
        turn(first, last, __ldg(row + i), __ldg(row + half + i));
        x[e] = mine;
      }
    }
  }
}

template <int VPL>
__device__ __forceinline__ void store_row(const PoolView& p, bool is_v, bool i8, bool q4,
                                          size_t row, float (&x)[VPL], int lane, float norm) {
  constexpr int D = 32 * VPL;
  char* store = (char*)(is_v ? p.v : p.k);
  uint16_t* scales = (uint16_t*)(is_v ? p.vs : p.ks);
  if (q4) {
    fwht_row<VPL>(x, lane, norm);
    uint16_t scale;
    const uint32_t packed = q4_0_regs<VPL>(x, lane, scale);
#pragma unroll
    for (int n = 0; n < VPL / 2; ++n)
      store[row * (D / 2) + q4_byte_of(lane * VPL + 2 * n, D)] = (char)(packed >> (8 * n));
    if (lane % (32 / VPL) == 0) scales[row * (D / 32) + lane * VPL / 32] = scale;
  } else if (i8) {
    typename Vec<VPL>::B codes;
    uint16_t scale;
    const int lpg = p.gs / VPL;
    quantize_regs<VPL>(x, lpg, codes, scale);
    *reinterpret_cast<typename Vec<VPL>::B*>(store + row * D + lane * VPL) = codes;
    if (lane % lpg == 0) scales[row * p.ng + lane / lpg] = scale;
  } else {
    union { typename Vec<VPL>::H v; uint32_t w[VPL / 2]; } h;
#pragma unroll
    for (int e = 0; e < VPL; e += 2) h.w[e / 2] = ptx::pack_f16x2(x[e], x[e + 1]);
    *reinterpret_cast<typename Vec<VPL>::H*>(store + (row * D + lane * VPL) * 2) = h.v;
  }
}

constexpr int kRowWarps = 8;
template <int VPL>
__global__ void __launch_bounds__(kRowWarps * 32)
    rope_rows_kernel(const __grid_constant__ RopeArgs a, const PoolView p, bool k8, bool v8,
                     float norm) {
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  if (blockIdx.x >= a.append_blocks) {
    rotate_queries<32 * VPL>(a, (blockIdx.x - a.append_blocks) * (kRowWarps * 32) + threadIdx.x);
    return;
  }
  const int lane = threadIdx.x & 31;
  const unsigned n = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const unsigned tok = n / (unsigned)p.Hkv;
  const int kvh = n % (unsigned)p.Hkv;
  const size_t b = tok / (unsigned)a.n_new;
  const int i = tok % (unsigned)a.n_new;
  if (b >= (size_t)a.n_seqs || i >= tokens_of(a, b)) return;
  const long long pos = (long long)__ldg(a.seq_pos + b) + i;
  if (pos < 0 || pos / p.ps >= a.max_pages) {
    if (lane == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
    return;
  }
  float k[VPL], v[VPL];
  load_halves<VPL>(a.k + (size_t)tok * a.k_stride + kvh * p.D + lane * VPL, k);
  load_halves<VPL>(a.v + (size_t)tok * a.v_stride + kvh * p.D + lane * VPL, v);
  const int page = check_page(__ldg(a.page_table + b * a.max_pages + (int)(pos / p.ps)), p);
  if (page < 0) return;
  turn_row<VPL>(a, b, i, lane, k);
  const size_t row = row_index(p, page, kvh, (int)(pos % p.ps));
  store_row<VPL>(p, false, k8, p.k4, row, k, lane, norm);
  store_row<VPL>(p, true, v8, p.v4, row, v, lane, norm);
}

// ---- launches ------------------------------------------------------------
// Query heads per thread: a thread's turns cost twice its twin's bytes of one head, so a thread takes
// up to eight heads, but not fewer than two blocks of threads an SM are made of them.
unsigned query_blocks(RopeArgs& a, int D, int threads, int sms) {
  a.heads = 1;
  if (!a.q) return 0;
  const long long twins = (long long)a.n_seqs * a.n_new * (D / 16);
  while (a.heads < 8 && twins * ((a.H + 2 * a.heads - 1) / (2 * a.heads)) >= 512LL * sms) a.heads *= 2;
  return (unsigned)((twins * ((a.H + a.heads - 1) / a.heads) + threads - 1) / threads);
}

struct RopeLaunch {
  RopeArgs& a;
  const int8kv_pool* pool;
  int layer;
  cudaStream_t stream;
};

template <class... A>
cudaError_t launch_early(void (*kernel)(A...), unsigned grid, int threads, cudaStream_t stream,
                         A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int D, bool F8, int NT, int GROUPS, int CH>
cudaError_t launch_blocks(const RopeLaunch& c) {
  const BlockView p = block_view(c.pool, c.layer);
  const int T = 1 << p.t_log2;
  const int nb = (int)(((long long)c.a.n_new + T - 2) / T + 1);   // blocks that n_new tokens may touch
  const long long units = (long long)c.a.n_seqs * nb * p.Hkv * 2;
  if (units > 0x3fffff00LL) return cudaErrorNotSupported;
  c.a.append_blocks = (unsigned)((units + GROUPS - 1) / GROUPS);
  const unsigned q = query_blocks(c.a, D, NT * GROUPS, c.pool->num_sms);
  return launch_early(rope_block_kernel<D, F8, NT, GROUPS, CH>, c.a.append_blocks + q, NT * GROUPS,
                      c.stream, (const RopeArgs)c.a, p, nb);
}

template <int D, bool F8>
cudaError_t dispatch_blocks(const RopeLaunch& c) {
  const int T = c.pool->group_size;
  const int twins = (c.a.n_new < T ? c.a.n_new : T) * (D / 16);   // most new twins of a block
  if (twins <= 32) return launch_blocks<D, F8, 32, 4, 1>(c);
  if (twins <= 64) return launch_blocks<D, F8, 32, 4, 2>(c);
  if (twins <= 128) return launch_blocks<D, F8, 32, 4, 4>(c);
  if (twins <= 256) return launch_blocks<D, F8, 64, 1, 4>(c);
  if (twins <= 512) return launch_blocks<D, F8, 128, 1, 4>(c);
  if constexpr (D >= 128)
    if (twins <= 1024) return launch_blocks<D, F8, 256, 1, 4>(c);
  if constexpr (D >= 256)
    if (twins <= 2048) return launch_blocks<D, F8, 512, 1, 4>(c);
  return cudaErrorNotSupported;
}

template <int VPL>
cudaError_t launch_rows(const RopeLaunch& c) {
  const PoolView p = layer_view(c.pool, c.layer);
  const long long rows = (long long)c.a.n_seqs * c.a.n_new * p.Hkv;
  if (rows > 0x3fffff00LL) return cudaErrorNotSupported;
  c.a.append_blocks = (unsigned)((rows + kRowWarps - 1) / kRowWarps);
  const unsigned q = query_blocks(c.a, 32 * VPL, kRowWarps * 32, c.pool->num_sms);
  return launch_early(rope_rows_kernel<VPL>, c.a.append_blocks + q, kRowWarps * 32, c.stream,
                      (const RopeArgs)c.a, p, c.pool->k_int8, c.pool->v_int8,
                      (float)(1.0 / std::sqrt((double)p.D)));
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace
}  // namespace int8kv

using namespace int8kv;

extern "C" int kv_rope_append(const int8kv_pool* pool, int layer, const uint16_t* q,
                              const uint16_t* k_new, const uint16_t* v_new, long long q_stride,
                              long long k_stride, long long v_stride, int n_seqs, int n_new,
                              int n_heads, const int32_t* seq_pos, const int32_t* new_lens,
                              const float* rope_table, int n_table, int rope_dim, int rope_style,
                              const int32_t* positions, int n_axes, const uint8_t* pair_axis,
                              uint16_t* q_out, const int32_t* page_table, int max_pages_per_seq,
                              void* stream) {
  if (!pool) return INT8KV_ERR_NULL_PTR;
  const int D = pool->head_dim, Hkv = pool->n_kv_heads;
  if (layer < 0 || layer >= pool->n_layers || n_seqs < 0 || n_new < 0 || max_pages_per_seq <= 0 ||
      n_table <= 0 || rope_dim < 16 || rope_dim > D || rope_dim % 16 != 0 || n_axes < 1 || n_axes > 4 ||
      (rope_style != INT8KV_ROPE_HALVES && rope_style != INT8KV_ROPE_PAIRS))
    return INT8KV_ERR_INVALID_ARG;
  if (q && (n_heads <= 0 || q_stride < (long long)n_heads * D)) return INT8KV_ERR_INVALID_ARG;
  if (k_stride < (long long)Hkv * D || v_stride < (long long)Hkv * D) return INT8KV_ERR_INVALID_ARG;
  if (n_axes > 1 && !pair_axis) return INT8KV_ERR_NULL_PTR;
  RopeArgs a = {};
  if (pair_axis)
    for (int i = 0; i < rope_dim / 2; ++i) {
      if (pair_axis[i] >= n_axes) return INT8KV_ERR_INVALID_ARG;
      a.axes[i >> 2] |= pair_axis[i] << (2 * (i & 3));
    }
  if ((long long)n_seqs * n_new == 0) return INT8KV_OK;
  if (!k_new || !v_new || !seq_pos || !rope_table || !page_table || (q && !q_out) ||
      (n_axes > 1 && !positions))
    return INT8KV_ERR_NULL_PTR;
  if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(q_out) ||
      !aligned16(rope_table) || (q && q_stride % 8 != 0) || k_stride % 8 != 0 || v_stride % 8 != 0)
    return INT8KV_ERR_ALIGNMENT;
  if (!on_current_device(pool)) return INT8KV_ERR_INVALID_ARG;
  // the kernels count tokens, their rows and their queries' pieces in 32 bits
  if ((long long)n_seqs * n_new * (q ? n_heads : 1) > 0x7fffffffLL / (D / 16))
    return INT8KV_ERR_UNSUPPORTED;
  a.q = q;
  a.k = k_new;
  a.v = v_new;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.n_seqs = n_seqs;
  a.n_new = n_new;
  a.H = n_heads;
  a.Hkv = Hkv;
  a.seq_pos = seq_pos;
  a.new_lens = new_lens;
  a.table = rope_table;
  a.n_table = n_table;
  a.R = rope_dim;
  a.pairs = rope_style == INT8KV_ROPE_PAIRS;
  a.positions = positions;
  a.page_table = page_table;
  a.max_pages = max_pages_per_seq;
  a.err = pool->dev_error;
  const RopeLaunch c{a, pool, layer, (cudaStream_t)stream};
  cudaError_t e;
  if (is_block(pool)) {
    const bool f8 = is_f8(pool);
    e = D == 64    ? f8 ? dispatch_blocks<64, true>(c) : dispatch_blocks<64, false>(c)
        : D == 128 ? f8 ? dispatch_blocks<128, true>(c) : dispatch_blocks<128, false>(c)
                   : f8 ? dispatch_blocks<256, true>(c) : dispatch_blocks<256, false>(c);
  } else {
    e = D == 64 ? launch_rows<2>(c) : D == 128 ? launch_rows<4>(c) : launch_rows<8>(c);
  }
  if (e == cudaErrorNotSupported) return INT8KV_ERR_UNSUPPORTED;
  return e == cudaSuccess ? INT8KV_OK : INT8KV_ERR_CUDA;
}
