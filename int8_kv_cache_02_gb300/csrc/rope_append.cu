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
//
// Bound by HBM for prompts (rows in, queries and codes out; half of the issue slots are taken), by
// the launch and three dependent loads for single tokens (64 sequences: 3.3 us).
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
  int heads, kv_heads;            // query heads that one of their threads takes, kv heads of a group
};

// Tokens that sequence b brings.
__device__ __forceinline__ int tokens_of(const RopeArgs& a, size_t b) {
  if (!a.new_lens) return a.n_new;
  const int n = __ldg(a.new_lens + b);
  if (n > a.n_new) flag_error(a.err, INT8KV_DEVERR_LENGTH);
  return max(0, min(n, a.n_new));
}

// The table's row of the position that token i of sequence b has on an axis; outside the table `ok`
// is false and the row some other (loads go ahead without a branch, and in batches).
struct TableRow {
  const float* row;
  bool ok;
  __device__ __forceinline__ TableRow(const RopeArgs& a, size_t b, int i, int axis) {
    const long long at = a.positions
                             ? __ldg(a.positions + ((size_t)axis * a.n_seqs + b) * a.n_new + i)
                             : (long long)__ldg(a.seq_pos + b) + i;
    ok = at >= 0 && at < a.n_table;
    row = a.table + (size_t)(ok ? at : 0) * a.R;
  }
};

// Cosines and sines of N consecutive pairs from pair i on: 4 or 8 from a multiple of 4 on, else 1 or 2.
// What lies outside the table is flagged by the caller (`bad`) and does not turn.
template <int N>
__device__ __forceinline__ void load_turns(const RopeArgs& a, size_t b, int tok, int i, float* c,
                                           float* s, bool& bad) {
  if constexpr (N >= 4) {      // (mostly by one position)
    const unsigned by = a.axes[i >> 2], first = by & 3;
    if (by == first * 0x55u && (N == 4 || a.axes[(i >> 2) + 1] == by)) {
      const TableRow r(a, b, tok, first);
      bad |= !r.ok;
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(r.row + i + k));
        const float4 y = __ldg(reinterpret_cast<const float4*>(r.row + a.R / 2 + i + k));
        c[k] = r.ok ? x.x : 1.f, c[k + 1] = r.ok ? x.y : 1.f;
        c[k + 2] = r.ok ? x.z : 1.f, c[k + 3] = r.ok ? x.w : 1.f;
        s[k] = r.ok ? y.x : 0.f, s[k + 1] = r.ok ? y.y : 0.f;
        s[k + 2] = r.ok ? y.z : 0.f, s[k + 3] = r.ok ? y.w : 0.f;
      }
      return;
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const TableRow r(a, b, tok, a.axes[(i + k) >> 2] >> (2 * ((i + k) & 3)) & 3);
    const float x = __ldg(r.row + i + k), y = __ldg(r.row + a.R / 2 + i + k);
    bad |= !r.ok;
    c[k] = r.ok ? x : 1.f;
    s[k] = r.ok ? y : 0.f;
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
__device__ __forceinline__ void twin_turns(const RopeArgs& a, size_t b, int tok, int t, Turns& w,
                                           bool& bad) {
  if (a.pairs) {
    load_turns<4>(a, b, tok, 4 * t, w.c, w.s, bad);
    load_turns<4>(a, b, tok, a.R / 4 + 4 * t, w.c + 4, w.s + 4, bad);
  } else {
    load_turns<8>(a, b, tok, 8 * t, w.c, w.s, bad);
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

// Queries: a thread takes one twin of a token for `a.heads` heads, whose turns it loads once; the next
// heads' values are under way while it turns the last ones'.
// (q_out may be q: a value is read and written by one thread, in this order, so not through
// the read-only path.)
template <int D>
__device__ __forceinline__ void rotate_queries(const RopeArgs& a, unsigned thread) {
  constexpr int TW = D / 16, N = 2;
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
  const int end = min(a.H, h0 + a.heads);
  const uint16_t* from = a.q + (size_t)tok * a.q_stride;
  uint16_t* to = a.q_out + (size_t)tok * a.H * D;
  uint4 next[N][2];
  const auto load = [&](int h) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (h + k < end) {
        next[k][0] = *reinterpret_cast<const uint4*>(from + (h + k) * D + 8 * px);
        next[k][1] = *reinterpret_cast<const uint4*>(from + (h + k) * D + 8 * py);
      }
  };
  load(h0);
  Turns w;
  bool bad = false;
  if (turned) twin_turns(a, b, i, t, w, bad);
  if (bad) flag_error(a.err, INT8KV_DEVERR_LENGTH);
  for (int h = h0; h < end; h += N) {
    uint4 x[N][2];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[k][0] = next[k][0];
      x[k][1] = next[k][1];
    }
    load(h + N);
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (h + k < end) {
        if (turned) {
          float fx[8], fy[8];
          halves_to_floats(x[k][0], fx);
          halves_to_floats(x[k][1], fy);
          turn_twin(a.pairs, w, fx, fy);
          x[k][0] = make_uint4(ptx::pack_f16x2(fx[0], fx[1]), ptx::pack_f16x2(fx[2], fx[3]),
                               ptx::pack_f16x2(fx[4], fx[5]), ptx::pack_f16x2(fx[6], fx[7]));
          x[k][1] = make_uint4(ptx::pack_f16x2(fy[0], fy[1]), ptx::pack_f16x2(fy[2], fy[3]),
                               ptx::pack_f16x2(fy[4], fy[5]), ptx::pack_f16x2(fy[6], fy[7]));
        }
        *reinterpret_cast<uint4*>(to + (h + k) * D + 8 * px) = x[k][0];
        *reinterpret_cast<uint4*>(to + (h + k) * D + 8 * py) = x[k][1];
      }
  }
}

// ---- block-scaled pools ------------------------------------------------------
// As in the append kernel, one group of threads (a warp, or a block of NT threads) owns blocks of
// positions: it loads a block's new rows once, turns K's, reduces the largest magnitude, and writes
// codes and scale.  Here it takes the same positions of a.kv_heads heads, one after the other: their
// turns are the same, and loaded once (a row's are four times its own bytes), and the next head's
// rows are under way meanwhile.  CH twins per thread, as fp32; beyond two of them the turns
// are loaded again for each head, the registers holding no more.
// Compiled for 768 threads an SM: a prompt of 2 x 16381 tokens (32 / 8 heads of D 128, one axis) takes
// 123 us (90 % of the copy rate); when the three were measured it took 126, 138 with 512
// threads (128 registers), and 144 with 1024, whose spills the keys pay for.
constexpr int kResident = 768;
template <int D, bool F8, int NT, int GROUPS, int CH>
__global__ void __launch_bounds__(NT* GROUPS, kResident / (NT * GROUPS) ? kResident / (NT * GROUPS) : 1)
    rope_block_kernel(const __grid_constant__ RopeArgs a, const BlockView p, int nb) {
  constexpr int TW = D / 16;     // twins per row
  constexpr bool KEEP = CH <= 2;
  static_assert(GROUPS == 1 || NT == 32, "groups of a block are single warps");
  __shared__ float red[2][NT / 32];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  if (blockIdx.x >= a.append_blocks) {
    rotate_queries<D>(a, (blockIdx.x - a.append_blocks) * (NT * GROUPS) + threadIdx.x);
    return;
  }
  const int tid = threadIdx.x % NT;
  const unsigned unit = blockIdx.x * GROUPS + threadIdx.x / NT;     // (fewer than 2^31)
  // unit = ((sequence * nb + block) * head groups + group) * 2 + store
  const bool is_v = unit & 1;
  const unsigned groups = (p.Hkv + a.kv_heads - 1) / a.kv_heads;
  const int h0 = (unit >> 1) % groups * a.kv_heads, end = min(p.Hkv, h0 + a.kv_heads);
  const unsigned sb = (unit >> 1) / groups;
  const int j = sb % (unsigned)nb;
  const size_t b = sb / (unsigned)nb;
  if (b >= (size_t)a.n_seqs) return;
  const int T = 1 << p.t_log2;
  long long pos = __ldg(a.seq_pos + b), skip = 0;
  const int count = tokens_of(a, b);
  if (count == 0) return;      // (of a sequence that brings none the position does not matter)
  if (pos < 0) {     // tokens at negative positions have no place
    skip = -pos;
    pos = 0;
    if (tid == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
  }
  const long long first = ((pos >> p.t_log2) + j) << p.t_log2;   // the block's first position
  const int r0 = j == 0 ? (int)(pos & (T - 1)) : 0;              // rows it held before
  const long long i0 = first + r0 - pos + skip;                  // its first new token
  const long long left = (long long)count - i0;                  // (below INT_MIN, it may be)
  if (left <= 0) return;
  const int rows = (int)min((long long)(T - r0), left);
  const long long lp = first >> p.ps_log2;
  if (lp >= a.max_pages) {
    if (tid == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
    return;
  }
  const long long stride = is_v ? a.v_stride : a.k_stride;
  const uint16_t* src = (is_v ? a.v : a.k) + (size_t)(b * a.n_new + i0) * stride + h0 * D;
  // What a thread's twins are: where they come from (in the next head: D values on) and go to, how far
  // apart their pieces are, which are there, and which turn.
  const uint16_t* from[CH];
  int to[CH], apart[CH];
  unsigned there = 0, turned = 0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int n = tid + c * NT, r = n / TW, t = n % TW;
    int px, py;
    twin_pieces(t, a.R, px, py);
    apart[c] = 8 * (py - px);
    from[c] = src + r * stride + 8 * px;
    to[c] = (r0 + r) * D + 8 * px;
    there |= (r < rows) << c;
    turned |= (r < rows && !is_v && t < a.R / 16) << c;
  }
  uint4 raw[CH][2];
  const auto load = [&](bool more) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      raw[c][0] = raw[c][1] = make_uint4(0, 0, 0, 0);
      if (more && (there >> c & 1)) {
        raw[c][0] = ptx::ldg128(from[c]);
        raw[c][1] = ptx::ldg128(from[c] + apart[c]);
      }
      from[c] += D;
    }
  };
  load(true);
  const int page = block_page(a.page_table + b * a.max_pages, (int)lp, p);
  Turns turns[KEEP ? CH : 1];
  bool bad = false;
  const auto turns_of = [&](int c, Turns& w) {
    const int n = tid + c * NT;
    if (turned >> c & 1) twin_turns(a, b, (int)i0 + n / TW, n % TW, w, bad);
  };
  if constexpr (KEEP)
#pragma unroll
    for (int c = 0; c < CH; ++c) turns_of(c, turns[c]);
  if (page < 0) return;
  const int slot = (int)(first & ((1 << p.ps_log2) - 1));
  const size_t ph = (size_t)page * p.Hkv + h0;
  uint8_t* codes = (is_v ? p.v : p.k) + ((ph << p.ps_log2) + slot) * D;
  float* scale = (is_v ? p.vs : p.ks) + (ph << (p.ps_log2 - p.t_log2)) + (slot >> p.t_log2);
  for (int h = h0; h < end; ++h) {
    const float s_old = r0 ? *scale : 0.f;
    float x[CH][2][8], top = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      halves_to_floats(raw[c][0], x[c][0]);
      halves_to_floats(raw[c][1], x[c][1]);
    }
    load(h + 1 < end);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if constexpr (!KEEP) turns_of(c, turns[0]);
      if (turned >> c & 1) turn_twin(a.pairs, turns[KEEP ? c : 0], x[c][0], x[c][1]);
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x[c][0][e]), fabsf(x[c][1][e])));
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if constexpr (NT > 32) {      // (two places in turn: one barrier a head)
      float* at = red[h & 1];
      if ((tid & 31) == 0) at[tid >> 5] = top;
      __syncthreads();
      top = at[0];
#pragma unroll
      for (int w = 1; w < NT / 32; ++w) top = fmaxf(top, at[w]);
    }
    float s;
    if (s_old > 0.f) {
      float shrink;
      s = grown_scale<F8>(s_old, top, shrink);
      if (shrink != 1.f) shrink_codes<F8>(codes, r0 * D, shrink, tid, NT);
    } else {
      s = __fdiv_rn(top, Codes<F8>::kMax);
    }
    // (every thread has read the old scale: by the barrier, or by the warp's reduction)
    if (tid == 0) *scale = s;
    // (products with a small sine may be far below what fp16 holds, where 1 / s has no fp32 value)
    const bool tiny = s < 0x1p-100f;
    const float inv = tiny ? 0.f : __frcp_rn(s);
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (there >> c & 1) {
        *reinterpret_cast<uint2*>(codes + to[c]) =
            s > 0.f ? quantize8<F8>(x[c][0], s, inv, tiny) : make_uint2(0, 0);
        *reinterpret_cast<uint2*>(codes + to[c] + apart[c]) =
            s > 0.f ? quantize8<F8>(x[c][1], s, inv, tiny) : make_uint2(0, 0);
      }
    codes += (size_t)D << p.ps_log2;
    scale += 1 << (p.ps_log2 - p.t_log2);
  }
  if (bad) flag_error(p.err, INT8KV_DEVERR_LENGTH);
}

// ---- pools with a scale for each row --------------------------------------
// int8 and fp16 stores: D / 16 lanes take a row, a twin each, for a.kv_heads heads in turn; a scale's
// values are those of several pieces, whose largest magnitudes meet in shared memory.  The prompt of
// 2 x 16381 tokens (32 / 8 heads of D 128): 144 us with two int8 stores (109 at the copy rate), 132 with
// one of them fp16 (113); 16 / 2 heads of D 256, all values turned: 124 and 118 (94, 96).
constexpr int kRowThreads = 256;

// Eight codes under scale s (fp16's, as fp32); 1 / s and the products as in quantize8, but a scale
// rounded to a subnormal leaves quotients beyond 127: saturated first.
__device__ __forceinline__ uint2 quantize8_row(const float (&v)[8], float s, float inv) {
  float y[8];
  bool near = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    y[e] = fminf(fmaxf(v[e] * inv, -127.f), 127.f);
    near |= fabsf(y[e] - ((y[e] + kRoundToInt) - kRoundToInt)) > 0.5f - 1.0e-4f;
  }
  if (near)
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fminf(fmaxf(__fdiv_rn(v[e], s), -127.f), 127.f);
  return round_codes8<false>(y);
}

__device__ __forceinline__ float largest(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) m = fmaxf(m, fabsf(x[e]));
  return m;
}

// A row's twin (px: x, py: y) into a store.  tops: the warp's places, D / 8 for this row; all lanes
// of the warp take part.
template <int D>
__device__ __forceinline__ void store_twin(const PoolView& p, bool is_v, bool i8, size_t row, int px,
                                           int py, const float (&x)[8], const float (&y)[8],
                                           float* tops, bool there) {
  char* store = (char*)(is_v ? p.v : p.k);
  if (!i8) {
    if (there) {
      *reinterpret_cast<uint4*>(store + (row * D + 8 * px) * 2) =
          make_uint4(ptx::pack_f16x2(x[0], x[1]), ptx::pack_f16x2(x[2], x[3]),
                     ptx::pack_f16x2(x[4], x[5]), ptx::pack_f16x2(x[6], x[7]));
      *reinterpret_cast<uint4*>(store + (row * D + 8 * py) * 2) =
          make_uint4(ptx::pack_f16x2(y[0], y[1]), ptx::pack_f16x2(y[2], y[3]),
                     ptx::pack_f16x2(y[4], y[5]), ptx::pack_f16x2(y[6], y[7]));
    }
    return;
  }
  uint16_t* scales = (uint16_t*)(is_v ? p.vs : p.ks) + row * p.ng;
  float top[2] = {largest(x), largest(y)};
  const int per = p.gs / 8;      // pieces of a scale: 2 or more
  if (p.ng == 1) {
    top[0] = fmaxf(top[0], top[1]);
#pragma unroll
    for (int off = D / 32; off > 0; off >>= 1)
      top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], off));
    top[1] = top[0];
  } else {
    __syncwarp();      // (the last row's have been read)
    tops[px] = top[0];
    tops[py] = top[1];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float* from = tops + (k ? py : px) / per * per;
      float m = 0.f;
      for (int e = 0; e < per; e += 2) {
        const float2 f = *reinterpret_cast<const float2*>(from + e);
        m = fmaxf(m, fmaxf(f.x, f.y));
      }
      top[k] = m;
    }
  }
  if (!there) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int piece = k ? py : px;
    const __half s16 = __float2half_rn(__fdiv_rn(top[k], 127.f));
    const float s = __half2float(s16);
    *reinterpret_cast<uint2*>(store + row * D + 8 * piece) =
        s > 0.f ? quantize8_row(k ? y : x, s, __frcp_rn(s)) : make_uint2(0, 0);
    if (piece % per == 0) scales[piece / per] = __half_as_ushort(s16);
  }
}

template <int D>
__global__ void __launch_bounds__(kRowThreads, 3)
    rope_rows_kernel(const __grid_constant__ RopeArgs a, const PoolView p, bool k8, bool v8) {
  constexpr int TW = D / 16;
  __shared__ float tops[kRowThreads / TW][D / 8];
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  if (blockIdx.x >= a.append_blocks) {
    rotate_queries<D>(a, (blockIdx.x - a.append_blocks) * kRowThreads + threadIdx.x);
    return;
  }
  const int t = threadIdx.x % TW;
  const unsigned n = blockIdx.x * (kRowThreads / TW) + threadIdx.x / TW;
  const unsigned groups = (p.Hkv + a.kv_heads - 1) / a.kv_heads;
  const unsigned tokens = (unsigned)a.n_seqs * a.n_new;
  unsigned tok = n / groups;
  const int h0 = n % groups * a.kv_heads;
  bool there = tok < tokens;      // (a warp's lanes stay together)
  if (!there) tok = 0;
  const size_t b = tok / (unsigned)a.n_new;
  const int i = tok % (unsigned)a.n_new;
  there = there && i < tokens_of(a, b);
  const int end = there ? min(p.Hkv, h0 + a.kv_heads) : 0;
  const long long pos = (long long)__ldg(a.seq_pos + b) + i;
  if (there && (pos < 0 || pos / p.ps >= a.max_pages)) {
    if (t == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
    there = false;
  }
  int px, py;
  twin_pieces(t, a.R, px, py);
  const uint16_t* from_k = a.k + (size_t)tok * a.k_stride;
  const uint16_t* from_v = a.v + (size_t)tok * a.v_stride;
  uint4 raw[4] = {};
  const auto load = [&](int h) {
    if (there && h < end) {
      raw[0] = ptx::ldg128(from_k + h * D + 8 * px);
      raw[1] = ptx::ldg128(from_k + h * D + 8 * py);
      raw[2] = ptx::ldg128(from_v + h * D + 8 * px);
      raw[3] = ptx::ldg128(from_v + h * D + 8 * py);
    }
  };
  load(h0);
  const int page = there ? check_page(__ldg(a.page_table + b * a.max_pages + (int)(pos / p.ps)), p) : -1;
  const bool turned = t < a.R / 16 && there;
  Turns w;
  bool bad = false;
  if (turned) twin_turns(a, b, i, t, w, bad);
  if (bad) flag_error(p.err, INT8KV_DEVERR_LENGTH);
  there = there && page >= 0;
  for (int k = 0; k < a.kv_heads; ++k) {
    const int h = h0 + k;
    float kx[8], ky[8], vx[8], vy[8];
    halves_to_floats(raw[0], kx);
    halves_to_floats(raw[1], ky);
    halves_to_floats(raw[2], vx);
    halves_to_floats(raw[3], vy);
    load(h + 1);
    if (turned) turn_twin(a.pairs, w, kx, ky);
    const bool now = there && h < end;
    const size_t row = now ? row_index(p, page, h, (int)(pos % p.ps)) : 0;
    float* mine = tops[threadIdx.x / TW];
    store_twin<D>(p, false, k8, row, px, py, kx, ky, mine, now);
    store_twin<D>(p, true, v8, row, px, py, vx, vy, mine, now);
  }
}

// Pools with a 4-bit store: a warp takes a (sequence, token), lane l values [l VPL, (l + 1) VPL) of K
// and V, as their append kernel (whose transform runs over a whole row); a value's partner is in the
// lane R/2 values further.  Bound by issue: the transform's butterflies, the search for a block's first
// largest value and single-byte stores make 182 M warp-instructions of the prompt of 2 x 16381 tokens
// (32 / 8 heads of D 128; 82 M in block-scaled pools), at 2.6 a cycle and SM: 224 us with k8v4, 208
// with q4_0 (106 and 104 at the copy rate); keys and values alone 154 and 137, kv_quant_append's 158
// and 153.  64 single tokens: 3.9 and 3.7 us.
template <int VPL>
__device__ __forceinline__ void row_turns(const RopeArgs& a, size_t b, int tok, int lane,
                                          float (&c)[VPL], float (&s)[VPL], bool& bad) {
  const int at = lane * VPL, half = a.R / 2;
  if (at >= a.R) return;
  if (a.pairs)
    load_turns<VPL / 2>(a, b, tok, at / 2, c, s, bad);
  else
    load_turns<VPL>(a, b, tok, at >= half ? at - half : at, c, s, bad);
}

template <int VPL>
__device__ __forceinline__ void turn_row(const RopeArgs& a, int lane, float (&x)[VPL],
                                         const float (&c)[VPL], const float (&s)[VPL]) {
  const int at = lane * VPL, half = a.R / 2;
  if (a.pairs) {
    if (at < a.R) {
#pragma unroll
      for (int e = 0; e < VPL; e += 2) turn(x[e], x[e + 1], c[e / 2], s[e / 2]);
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
      if (second) turn(other, mine, c[e], s[e]);
      else turn(mine, other, c[e], s[e]);
      x[e] = mine;
    }
  }
}

template <int VPL>
__device__ __forceinline__ void halves_of(const typename Vec<VPL>::H& raw, float (&x)[VPL]) {
  const __half2* h = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
  for (int e = 0; e < VPL / 2; ++e) {
    const float2 f = __half22float2(h[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
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
    rope_q4_kernel(const __grid_constant__ RopeArgs a, const PoolView p, bool k8, bool v8,
                   float norm) {
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();
  if (blockIdx.x >= a.append_blocks) {
    rotate_queries<32 * VPL>(a, (blockIdx.x - a.append_blocks) * (kRowWarps * 32) + threadIdx.x);
    return;
  }
  // a warp: one token, a.kv_heads heads, whose turns are the same
  const int lane = threadIdx.x & 31;
  const unsigned n = blockIdx.x * kRowWarps + (threadIdx.x >> 5);
  const unsigned groups = (p.Hkv + a.kv_heads - 1) / a.kv_heads, tok = n / groups;
  const int h0 = n % groups * a.kv_heads, end = min(p.Hkv, h0 + a.kv_heads);
  const size_t b = tok / (unsigned)a.n_new;
  const int i = tok % (unsigned)a.n_new;
  if (b >= (size_t)a.n_seqs || i >= tokens_of(a, b)) return;
  const long long pos = (long long)__ldg(a.seq_pos + b) + i;
  if (pos < 0 || pos / p.ps >= a.max_pages) {
    if (lane == 0) flag_error(p.err, INT8KV_DEVERR_LENGTH);
    return;
  }
  const uint16_t* from_k = a.k + (size_t)tok * a.k_stride + lane * VPL;
  const uint16_t* from_v = a.v + (size_t)tok * a.v_stride + lane * VPL;
  using H = typename Vec<VPL>::H;
  constexpr int N = 2;      // heads under way
  H next_k[N], next_v[N];
  const auto load = [&](int h) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (h + e < end) {
        next_k[e] = __ldg(reinterpret_cast<const H*>(from_k + (h + e) * p.D));
        next_v[e] = __ldg(reinterpret_cast<const H*>(from_v + (h + e) * p.D));
      }
  };
  load(h0);
  const int page = check_page(__ldg(a.page_table + b * a.max_pages + (int)(pos / p.ps)), p);
  float c[VPL], s[VPL];
  bool bad = false;
  row_turns<VPL>(a, b, i, lane, c, s, bad);
  if (bad) flag_error(p.err, INT8KV_DEVERR_LENGTH);
  if (page < 0) return;
  for (int h = h0; h < end; h += N) {
    float k[N][VPL], v[N][VPL];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      halves_of<VPL>(next_k[e], k[e]);
      halves_of<VPL>(next_v[e], v[e]);
    }
    load(h + N);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (h + e < end) {
        turn_row<VPL>(a, lane, k[e], c, s);
        const size_t row = row_index(p, page, h + e, (int)(pos % p.ps));
        store_row<VPL>(p, false, k8, p.k4, row, k[e], lane, norm);
        store_row<VPL>(p, true, v8, p.v4, row, v[e], lane, norm);
      }
  }
}

// ---- launches ------------------------------------------------------------
// Query heads per thread: a thread's turns are twice its twin's bytes of one head, so it takes up to
// eight heads, but two blocks of threads an SM are made of them at least.  A prompt of 2 x 16381 tokens
// (32 / 8 heads of D 128, one axis) with 1, 2, 4, 8, 16 heads a thread: 197, 140, 128, 124, 126 us,
// with three axes 302, 205, 149, 133, 129; 16 heads of D 256, 64 values turned: 92, 64, 58, 56, 59;
// 2 x 1000 tokens, where the rule stops at four: 14.1 with one, 9.9.
unsigned query_blocks(RopeArgs& a, int D, int threads, int sms) {
  a.heads = 1;
  if (!a.q) return 0;
  const long long twins = (long long)a.n_seqs * a.n_new * (D / 16);
  while (a.heads < 8 && twins * ((a.H + 2 * a.heads - 1) / (2 * a.heads)) >= 512LL * sms) a.heads *= 2;
  return (unsigned)((twins * ((a.H + a.heads - 1) / a.heads) + threads - 1) / threads);
}

// Heads that a group of threads takes in turn, of `threads` that one head wants: up to eight, while
// two blocks' threads are left for every SM.  Keys and values of the prompt above with 1 and 8 heads a
// group: 76 and 57 us, with three axes 102 and 60.
int heads_of_a_group(long long threads, int heads, int sms) {
  int n = 1;
  while (n < 8 && n < heads && threads * ((heads + 2 * n - 1) / (2 * n)) >= 1024LL * sms) n *= 2;
  return n;
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
  const long long blocks = (long long)c.a.n_seqs * nb * 2;
  c.a.kv_heads = heads_of_a_group(blocks * NT, p.Hkv, c.pool->num_sms);
  const long long units = blocks * ((p.Hkv + c.a.kv_heads - 1) / c.a.kv_heads);
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
  if (twins <= 128) return launch_blocks<D, F8, 64, 1, 2>(c);
  if (twins <= 256) return launch_blocks<D, F8, 128, 1, 2>(c);
  if (twins <= 512) return launch_blocks<D, F8, 256, 1, 2>(c);
  if constexpr (D >= 128)
    if (twins <= 1024) return launch_blocks<D, F8, 512, 1, 2>(c);
  if constexpr (D >= 256)
    if (twins <= 2048) return launch_blocks<D, F8, 512, 1, 4>(c);
  return cudaErrorNotSupported;
}

template <int D>
cudaError_t launch_rows(const RopeLaunch& c) {
  const PoolView p = layer_view(c.pool, c.layer);
  const bool q4 = p.k4 || p.v4;
  const int threads = q4 ? kRowWarps * 32 : kRowThreads, lanes = q4 ? 32 : D / 16;
  const long long tokens = (long long)c.a.n_seqs * c.a.n_new;
  c.a.kv_heads = heads_of_a_group(tokens * lanes, p.Hkv, c.pool->num_sms);
  const long long rows = tokens * ((p.Hkv + c.a.kv_heads - 1) / c.a.kv_heads);
  if (rows > 0x3fffff00LL) return cudaErrorNotSupported;
  const int per = threads / lanes;
  c.a.append_blocks = (unsigned)((rows + per - 1) / per);
  const unsigned q = query_blocks(c.a, D, threads, c.pool->num_sms);
  if (q4)
    return launch_early(rope_q4_kernel<D / 32>, c.a.append_blocks + q, threads, c.stream,
                        (const RopeArgs)c.a, p, c.pool->k_int8, c.pool->v_int8,
                        (float)(1.0 / std::sqrt((double)D)));
  return launch_early(rope_rows_kernel<D>, c.a.append_blocks + q, threads, c.stream,
                      (const RopeArgs)c.a, p, c.pool->k_int8, c.pool->v_int8);
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
    e = D == 64 ? launch_rows<64>(c) : D == 128 ? launch_rows<128>(c) : launch_rows<256>(c);
  }
  if (e == cudaErrorNotSupported) return INT8KV_ERR_UNSUPPORTED;
  return e == cudaSuccess ? INT8KV_OK : INT8KV_ERR_CUDA;
}
