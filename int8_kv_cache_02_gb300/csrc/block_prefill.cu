// Causal attention of a chunk of new queries over a block-scaled pool (one fp32
// scale per T positions and kv head; int8 or e4m3 codes) on the 5th-generation
// tensor cores.  The chunk's own rows are appended before this runs; its query i
// sits at position start + i and sees positions 0 .. start + i.
//
//   z_j = (q . ck_j) sk(block of j) scale,  o = sum_j 2^(z_j) sv(block of j) cv_j / sum_j 2^(z_j)
//
// A block takes 128 (query, head) rows of one kv head, row R in lane R of tensor
// memory, and a range of tiles of 64 positions.  Its warps have three tasks, in step
// through mbarriers:
//   - warps 8 - 15 load codes, a tile ahead and in whole lines, and write them as fp16
//     (exact) into two shared-memory tiles each of K and V, 128-byte-swizzled boxes
//     [D / 64][64 positions][128 B].  A scale serves 16 positions and more, so no value is
//     multiplied by it: K scales multiply scores, V scales weights.
//   - warp 16 issues S = Q K^T (M 128, N 64) and O += W V (N = D; W as an fp16 hi + lo pair
//     from tensor memory), the next tile's scores ahead of this tile's weights: three S
//     buffers, so that scores never wait for the product that reads the last weights.
//   - warps 0 - 7 turn scores into weights, two threads a row with 32 positions each.  As in
//     the decode kernel a row has two references, m for the sum and m + e for weights
//     times their V scales, moved only when exceeded by 2^8, and then O in tensor memory is
//     rescaled.  w = 2^(z - m + c), c = log2 sv - e + 6, and the sum takes 2^-c times the
//     sum of a piece's 16 weights: one exponential and one multiply-add a score, which has
//     c - m as one summand.  That rounds the exponents to the last place of m, so where |m| > 64
//     (2^-18) the score meets m alone first (a chunk of such scores takes 4 to 16 % longer).
//
// Bound by the warps that convert and weigh, then by the tensor pipe (a tile costs 3 * 128 *
// 64 * D multiply-adds, W being in two parts): a tile takes 1.5 us at D 256 and 1.3 at 128,
// 0.8 and 0.4 at the tensor rate.  256 queries over 33,024 positions: 16 / 2 heads of D 256
// 200 us (int8, 690 TFLOP/s of the formula's operations) and 186 (e4m3), 32 / 8 of D 128 326
// and 301; the decode kernel's windows took 912, 784, 908 and 758.  What brought it there
// (D 256, int8): the products' first form 469 us; O in one product of N = D and one warp a
// row to join the splits 371; codes' addresses from one page entry a tile 253; packed fp32
// pairs in the weights, the queries loaded under the first codes, and splits that
// count a block's start and end 201 (200 as it is now).
// Slower: 16 converting warps with registers moved to the others (setmaxnreg; -2 % to +5 %), four
// threads a row for the scores (+20 %), K converted a tile ahead of V (+8 %), whichever
// product has its operands issued first (+5 %).
//
// The sums in tensor memory drop the bits below their last place instead of rounding: over
// n positions O loses up to n / 8 * 2^-23 of itself (measured: 2e-5 at 8192 positions).  So
// every kChain tiles the scoring threads add O to their rows' sums in global memory (where the
// output, or the split's partial, will be) and the next product starts from zero: at most
// 5120 / 8 * 2^-23 = 8e-5 is lost whatever the context.  131,072 positions in one block:
// 1.3e-5 off, 3.5e-4 as one chain; 1.5 us a chain of 109 us (D 128) or 129 (D 256).  The decode
// kernel, whose sums are in registers, has no such loss.
#include <cuda_fp16.h>

#include "block_prefill.h"
#include "decode_common.cuh"
#include "tc_common.cuh"

namespace int8kv {
namespace {

constexpr int kRows = 128;                 // (query, head) rows of a block
constexpr int kKeys = 64;                  // positions of a tile
constexpr int kBox = kKeys * 128;          // bytes of 64 dims of a tile
constexpr int kQBox = kRows * 128;
constexpr int kSoftmax = 256;              // threads that take scores
constexpr int kConvert = 256;              // and that convert codes
constexpr int kProducts = (kSoftmax + kConvert) / 32;      // the warp that issues products
constexpr int kThreads = kSoftmax + kConvert + 32;
constexpr uint64_t kPatience = 2000000000;      // ns after which a wait has run out
constexpr float kUnset = -1e30f;
constexpr float kLazy = 8.f;
constexpr float kWeightShift = 6.f;        // w <= 2^14 in fp16
constexpr int kChain = 80;                 // tiles that one sum in tensor memory takes
constexpr float kNear = 64.f;              // |m| up to here: c - m is one summand

template <int D>
struct Layout {
  static constexpr int Q = 0;                              // fp16 [D / 64][128 rows][128 B]
  static constexpr int TILE = kKeys * D * 2;
  static constexpr int K = Q + kRows * D * 2;              // two tiles
  static constexpr int V = K + 2 * TILE;
  static constexpr int SMEM = V + 2 * TILE + 1024;         // (tiles start on 1024 bytes)
  static constexpr int O = 3 * kKeys;                      // tensor-memory columns: S x 3, then O
  static constexpr int COLS = O + D <= 256 ? 256 : 512;
  static constexpr int CH = kKeys * D / 16 / kConvert;     // 16-byte pieces a thread converts a side
};

struct PrefillBlockArgs {
  BlockView pool;
  const uint16_t* q;          // [n_new][H][D] fp16
  const int32_t* page_table;  // [max_pages]
  float* out;                 // [n_new][H][D]
  float* part_o;              // [n_new][H][splits][D], relative to 2^m
  float2* part_ml;            // [n_new][H][splits] m, l
  int n_new, H, G, start, splits, n_cg;
  float scale_log2;
  uint64_t patience;          // ns after which a wait has run out
  int expire;                 // 1: diagnostic, V's barriers wait for a warp that never comes
};

struct Shared {
  uint64_t k_full[2], v_full[2], s_done[2], w_full[2], o_done[2], t_full[4], q_full, drain, stopped;
  uint32_t tmem;
  int failed;
  float k_scale[4][4], v_log2[4][4];       // of a tile's 16-position pieces; four tiles
  int none[4][4];                          // piece without a page
  float2 top[2][2][kRows];                 // largest z of a thread's two pieces, by tile and half
};

__device__ __forceinline__ int swizzled(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

__device__ __forceinline__ uint64_t now_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

// Bounded wait: true once the barrier's phase is complete, false where it has run out or
// another wait of the block has (failed: null for the last one, which the products in flight
// end).  A complete phase says nothing about the block's other waits.  But every wait is one
// that the products need, and they complete `drain` only when none was left out.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* failed,
                                     uint64_t patience) {
  uint64_t from = 0;
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (ptx::mbar_try_wait(bar, parity)) return true;
    if (failed && *(volatile int*)failed) return false;
    const uint64_t now = now_ns();
    if (from == 0) from = now;
    if (now - from > patience) break;
  }
  if (failed) *(volatile int*)failed = 1;
  return false;
}

// Two fp32 values in one operation.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void tmem_scale(uint32_t ta, int n, float f) {
  for (int c = 0; c < n; c += 16) {
    uint32_t v[16];
    tc::ld16(ta + c, v);
    tc::wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
    tc::st16(ta + c, v);
  }
  tc::wait_st();
}

// The sums of a scoring warp's rows over their earlier chains, D / 2 values of each, which lie
// where the rows' output will be (own: the lane's).  A whole warp keeps them in pieces of 512
// bytes, four values of every lane, D / 8 lanes to a row: a lane's own row would be 32
// lines at a time.  In a warp whose rows are not all there each lane that has one uses it.
template <int D>
struct Sums {
  float* own;
  bool whole, there;
  __device__ __forceinline__ float* at(int q) const {      // the lane's values 4q ..
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x & 31;
    const uint64_t other = __shfl_sync(0xffffffffu, (uint64_t)own, q * (32 / LANES) + lane / LANES);
    return whole ? (float*)other + lane % LANES * 4 : own + 4 * q;
  }
  // O (in tensor memory at `from`) times `by` is put there, or added: by reductions in L2, which
  // nothing waits for.  (Loads, adds and stores took 6.9 us a chain at D 256 instead of 1.5.)
  // Nobody else adds to them, so the order is the program's.
  __device__ __forceinline__ void take(uint32_t from, float by, bool first) const {
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 16) {
      uint32_t o[16];
      tc::ld16(from + c, o);
      tc::wait_ld();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float* to = at(c / 4 + k);
        const float4 x = make_float4(
            __uint_as_float(o[4 * k]) * by, __uint_as_float(o[4 * k + 1]) * by,
            __uint_as_float(o[4 * k + 2]) * by, __uint_as_float(o[4 * k + 3]) * by);
        if (there) {
          if (first)
            *reinterpret_cast<float4*>(to) = x;
          else
            asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to),
                         "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
                         : "memory");
        }
      }
    }
  }
  // the sums times `by`
  __device__ __forceinline__ void scale(float by) const {
#pragma unroll 1
    for (int q = 0; q < D / 8; ++q) {
      float4* to = reinterpret_cast<float4*>(at(q));
      if (there) {
        const float4 x = __ldcg(to);
        *to = make_float4(x.x * by, x.y * by, x.z * by, x.w * by);
      }
    }
  }
  // O gets them added, times `by`
  __device__ __forceinline__ void give(uint32_t to, float by) const {
#pragma unroll 1
    for (int c = 0; c < D / 2; c += 16) {
      float4 x[4];
      uint32_t o[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4* from = reinterpret_cast<const float4*>(at(c / 4 + k));
        x[k] = there ? __ldcg(from) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      tc::ld16(to + c, o);
      tc::wait_ld();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[4 * k] = __float_as_uint(fmaf(x[k].x, by, __uint_as_float(o[4 * k])));
        o[4 * k + 1] = __float_as_uint(fmaf(x[k].y, by, __uint_as_float(o[4 * k + 1])));
        o[4 * k + 2] = __float_as_uint(fmaf(x[k].z, by, __uint_as_float(o[4 * k + 2])));
        o[4 * k + 3] = __float_as_uint(fmaf(x[k].w, by, __uint_as_float(o[4 * k + 3])));
      }
      tc::st16(to + c, o);
    }
    tc::wait_st();
  }
};

// Sixteen codes as fp16 in the order codes_to_h2 gives (int8: dims 0 2 1 3 of every four).
template <bool F8>
__device__ __forceinline__ void halves_of(const uint4 w, uint4& lo, uint4& hi) {
  lo = make_uint4(codes_to_h2<F8>(w.x), codes_behind_to_h2<F8>(w.x), codes_to_h2<F8>(w.y),
                  codes_behind_to_h2<F8>(w.y));
  hi = make_uint4(codes_to_h2<F8>(w.z), codes_behind_to_h2<F8>(w.z), codes_to_h2<F8>(w.w),
                  codes_behind_to_h2<F8>(w.w));
}

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1) block_prefill_kernel(const PrefillBlockArgs a) {
  using L = Layout<D>;
  constexpr int CH = L::CH, CPR = D / 16;
  extern __shared__ unsigned char raw[];
  __shared__ Shared s;
  unsigned char* smem = raw + ((1024u - (ptx::smem_u32(raw) & 1023u)) & 1023u);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const BlockView& p = a.pool;

  // the units with the longest contexts first
  const int split = blockIdx.x % a.splits, unit = blockIdx.x / a.splits;
  const int kvh = unit % p.Hkv, cg = a.n_cg - 1 - unit / p.Hkv;
  const int rows = a.n_new * a.G, row0 = cg * kRows;      // columns (query, head of the group)
  const int hi = a.start + (min(row0 + kRows, rows) - 1) / a.G + 1;      // positions [0, hi)
  const int tiles = (hi + kKeys - 1) / kKeys;
  const int t0 = (int)((long long)tiles * split / a.splits);
  const int n = (int)((long long)tiles * (split + 1) / a.splits) - t0;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s.k_full[i], kConvert / 32);
      ptx::mbar_init(&s.v_full[i], kConvert / 32 + a.expire);
      ptx::mbar_init(&s.s_done[i], 1);
      ptx::mbar_init(&s.w_full[i], kSoftmax / 32);
      ptx::mbar_init(&s.o_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&s.t_full[i], 1);
    ptx::mbar_init(&s.q_full, kSoftmax / 32);
    ptx::mbar_init(&s.drain, 1);
    ptx::mbar_init(&s.stopped, 1);
    ptx::fence_mbar_init();
    s.failed = 0;
  }
  if (warp == kProducts) tc::alloc(&s.tmem, L::COLS);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = s.tmem;

  if (warp < kSoftmax / 32) {
    // ---- scores to weights
    const int half = warp >> 2, R = tid & (kRows - 1), gc = row0 + R;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int last = gc < rows ? a.start + gc / a.G : -1;      // the row's last position
    const int least = a.start + row0 / a.G;                    // of the block's first row
    // the queries, while the first codes come
    constexpr int PIECES = kRows * (D / 8) / kSoftmax, BATCH = PIECES < 8 ? PIECES : 8;
    for (int x0 = 0; x0 < PIECES; x0 += BATCH) {
      uint4 v[BATCH];
#pragma unroll
      for (int x = 0; x < BATCH; ++x) {
        const int c = tid + (x0 + x) * kSoftmax, col = row0 + c / (D / 8);
        v[x] = make_uint4(0, 0, 0, 0);
        if (col < rows)
          v[x] = ptx::ldg128(a.q + ((size_t)(col / a.G) * a.H + kvh * a.G + col % a.G) * D +
                             c % (D / 8) * 8);
      }
#pragma unroll
      for (int x = 0; x < BATCH; ++x) {
        const int c = tid + (x0 + x) * kSoftmax, r = c / (D / 8), ch = c % (D / 8);
        uint4 y = v[x];
        if (a.scale_log2 < 0.f)      // (the scores' factors are not negative)
          y = make_uint4(y.x ^ 0x80008000u, y.y ^ 0x80008000u, y.z ^ 0x80008000u, y.w ^ 0x80008000u);
        if constexpr (!F8)      // the order of the converted codes
          y = make_uint4(ptx::prmt(y.x, y.y, 0x5410), ptx::prmt(y.x, y.y, 0x7632),
                         ptx::prmt(y.z, y.w, 0x5410), ptx::prmt(y.z, y.w, 0x7632));
        *reinterpret_cast<uint4*>(smem + L::Q + (ch >> 3) * kQBox + swizzled(r, ch & 7)) = y;
      }
    }
    ptx::fence_proxy_async();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&s.q_full);
    // where the row's output goes, or its split's partial: until then the sum of earlier chains
    const auto row_h = [&](int g) { return (size_t)(g / a.G) * a.H + kvh * a.G + g % a.G; };
    const auto row_out = [&](int g) {
      return a.splits > 1 ? a.part_o + (row_h(g) * a.splits + split) * D : a.out + row_h(g) * D;
    };
    const auto sums = [&]() {
      int g = gc;
      asm volatile("" : "+r"(g));      // (computed where it is used, not kept over the loops)
      return Sums<D>{row_out(g) + half * (D / 2), (g | 31) < rows, g < rows};
    };
    const uint32_t my_o = lanes + L::O + half * (D / 2);
    float m = kUnset, e = kUnset, l = 0.f, e_sum = kUnset;      // (e_sum: e of that sum)
    bool far = false;    // whether a row of the warp has |m| > kNear
    bool ok = true;      // (once it is false the warp only keeps the barrier's count)
    for (int from = 0; from < n; from += kChain) {
      if (from > 0) {      // the sum in tensor memory starts anew with the next product
        ok = ok && wait(&s.o_done[(from - 1) & 1], ((from - 1) >> 1) & 1, &s.failed, a.patience);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc::fence_after();
          const Sums<D> sum = sums();
          if (from == kChain) {
            e_sum = e;
          } else if (__any_sync(0xffffffffu, e - e_sum > 64.f)) {      // (else O grows to it)
            sum.scale(ptx::ex2(e_sum - e));
            e_sum = e;
          }
          sum.take(my_o, ptx::ex2(e - e_sum), from == kChain);
        }
      }
      const int behind = min(n, from + kChain);
      for (int i = from; i < behind; ++i) {
        const int pos = (t0 + i) * kKeys + half * 32, tab = i & 3;
        ok = ok && wait(&s.t_full[tab], (i >> 2) & 1, &s.failed, a.patience);
        ok = ok && wait(&s.s_done[i & 1], (i >> 1) & 1, &s.failed, a.patience);
        ok = __all_sync(0xffffffffu, ok);
        const uint32_t sc = lanes + (i % 3) * kKeys + half * 32;
        uint32_t v[2][16];
        float f[2], lv[2], lo[2], most[2] = {-INFINITY, -INFINITY};
        if (ok) {
          tc::fence_after();
          tc::ld16(sc, v[0]);
          tc::ld16(sc + 16, v[1]);
          bool none[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            f[j] = s.k_scale[tab][2 * half + j];
            lv[j] = s.v_log2[tab][2 * half + j];
            lo[j] = s.v_log2[tab][2 * (half ^ 1) + j];      // (the other thread's)
            none[j] = s.none[tab][2 * half + j];
          }
          tc::wait_ld();
          const bool masked = pos + 31 > least || none[0] || none[1];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (masked) {
              const int to = none[j] ? -1 : last - pos - 16 * j;
#pragma unroll
              for (int k = 0; k < 16; ++k)
                v[j][k] = __float_as_uint(k > to ? -INFINITY : __uint_as_float(v[j][k]) * f[j]);
              f[j] = 1.f;
            }
            float x[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              x[k] = fmaxf(fmaxf(__uint_as_float(v[j][k]), __uint_as_float(v[j][k + 4])),
                           fmaxf(__uint_as_float(v[j][k + 8]), __uint_as_float(v[j][k + 12])));
            most[j] = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * f[j];
          }
        }
        s.top[i & 1][half][R] = make_float2(most[0], most[1]);
        ptx::named_barrier_sync(1, kSoftmax);      // (also once a wait has failed)
        if (!ok) continue;
        const float2 other = s.top[i & 1][half ^ 1][R];
        const float top = fmaxf(fmaxf(most[0], most[1]), fmaxf(other.x, other.y));
        const auto above_m = [&]() {      // the tile's largest z - m + log2 sv
          return fmaxf(fmaxf(most[0] - m + lv[0], most[1] - m + lv[1]),
                       fmaxf(other.x - m + lo[0], other.y - m + lo[1]));
        };
        if (__any_sync(0xffffffffu, top > m + kLazy || above_m() > e + kLazy)) {
          if (top > m + kLazy) {
            l *= ptx::ex2(m - top);
            e += m - top;      // (the same references, from the new m)
            e_sum += m - top;
            m = top;
          }
          const float topE = above_m();
          float r = 1.f;
          if (topE > e + kLazy) {
            r = ptx::ex2(e - topE);
            e = topE;
          }
          far = __any_sync(0xffffffffu, fabsf(m) > kNear && m != kUnset);
          if (i > 0 && __any_sync(0xffffffffu, r != 1.f)) {
            ok = wait(&s.o_done[(i - 1) & 1], ((i - 1) >> 1) & 1, &s.failed, a.patience);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            tc::fence_after();
            tmem_scale(lanes + L::O + half * (D / 2), D / 2, r);
          }
        }
        float to = m;
        if (far) {      // scores, rounded like m, less m, which is exact
#pragma unroll
          for (int j = 0; j < 2; ++j) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              v[j][k] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(v[j][k]), f[j]), m));
            f[j] = 1.f;
          }
          to = 0.f;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // w = 2^(z - m + c) and its share of the sum, w 2^-c.  A scale below 2^-60 of the
          // row's reference, or zero, counts as that: its weights only carry the sum.
          const float c = fmaxf(lv[j] - e + kWeightShift, -60.f), cm = c - to;
          const uint64_t f2 = pack2(f[j], f[j]), c2 = pack2(cm, cm), minus = pack2(-1.f, -1.f);
          uint64_t sum = pack2(0.f, 0.f);
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            float w0, w1, s0, s1;
            unpack2(fma2(pack2(__uint_as_float(v[j][2 * k]), __uint_as_float(v[j][2 * k + 1])), f2,
                         c2),
                    w0, w1);
            const uint64_t w2 = pack2(ptx::ex2(w0), ptx::ex2(w1));
            sum = add2(sum, w2);
            unpack2(w2, w0, w1);
            w[k] = ptx::pack_f16x2(w0, w1);
            const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
            unpack2(fma2(pack2(x.x, x.y), minus, w2), s0, s1);
            w[8 + k] = ptx::pack_f16x2(s0, s1);
          }
          tc::st16(sc + 16 * j, w);
          float s0, s1;
          unpack2(sum, s0, s1);
          l = fmaf(s0 + s1, ptx::ex2(-to - cm), l);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&s.w_full[i & 1]);
      }
    }
    s.top[n & 1][half][R] = make_float2(l, 0.f);      // (the last tile's may still be read)
    ptx::named_barrier_sync(1, kSoftmax);
    l += s.top[n & 1][half ^ 1][R].x;
    ok = __all_sync(0xffffffffu, wait(&s.drain, 0, &s.failed, a.patience));
    tc::fence_after();
    if (!ok && tid == 0) flag_error(p.err, INT8KV_DEVERR_TIMEOUT);
    {
      const bool live = ok && n > 0 && l > 0.f;      // (a block that failed counts for nothing)
      float f = live ? ptx::ex2(e - kWeightShift) : 0.f;
      float* const out = row_out(gc);
      if (n > kChain) {
        sums().give(my_o, ptx::ex2(e_sum - e));
        __syncwarp();      // (other lanes' sums lay where this lane's row goes)
      }
      if (a.splits > 1) {
        if (gc < rows && half == 0)
          a.part_ml[row_h(gc) * a.splits + split] = make_float2(live ? m : -INFINITY, live ? l : 0.f);
      } else if (live) {
        f /= l;
      }
#pragma unroll 1
      for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
        uint32_t v[16];
        tc::ld16(lanes + L::O + c, v);
        tc::wait_ld();
        constexpr int X = F8 ? 1 : 2, Y = F8 ? 2 : 1;
        if (gc < rows)
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            *reinterpret_cast<float4*>(out + c + k) =
                live ? make_float4(__uint_as_float(v[k]) * f, __uint_as_float(v[k + X]) * f,
                                   __uint_as_float(v[k + Y]) * f, __uint_as_float(v[k + 3]) * f)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
  } else if (warp < kProducts) {
    // ---- codes to fp16.  Piece x of a thread: 16 codes, row `row` + STEP x, 16-byte column ch.
    // A warp takes whole rows; eight lanes four pieces of two neighbouring rows, whose swizzled
    // places are all eight of a 128-byte line: no bank conflicts.
    constexpr int STEP = kConvert / CPR;      // rows between a thread's pieces
    const int ch = (lane >> 3) % (D / 64) * 4 + (lane & 3);
    const int row = (warp - kSoftmax / 32) * (32 / CPR) + (lane >> 3) / (D / 64) * 2 + (lane >> 2 & 1);
    const int box = (ch >> 2) * kBox, at = (ch & 3) * 2;
    const bool tables = warp == kSoftmax / 32 && lane < 8;
    const bool one_page = p.ps_log2 >= 6;      // for a tile
    const int in_page = (1 << p.ps_log2) - 1;
    const size_t page_bytes = ((size_t)p.Hkv << p.ps_log2) * D;
    const size_t base = ((size_t)kvh << p.ps_log2) * D + 16 * ch;
    uint4 k[CH], v[CH];
    size_t from[CH];                // the next pieces' codes in the pool
    int page[CH], have = 0;         // and which there are
    constexpr int kAll = 1 << CH;   // (all, STEP rows apart)
    int table_page = 0, none = 0;
    float scale = 0.f;
    bool bad = false;
    auto entry = [&](int pos) { return pos < hi ? __ldg(a.page_table + (pos >> p.ps_log2)) : -1; };
    auto find = [&](int tile) {
      const int pos = (t0 + tile) * kKeys + row;
      page[0] = entry(one_page ? pos - row : pos);
      if (!one_page)
#pragma unroll
        for (int x = 1; x < CH; ++x) page[x] = entry(pos + STEP * x);
      if (tables) table_page = entry((t0 + tile) * kKeys + (lane & 3) * 16);
    };
    auto locate = [&](int tile) {      // (the page ids have come by then)
      const int pos = (t0 + tile) * kKeys + row;
      have = 0;
      if (one_page) {
        const bool there = (unsigned)page[0] < (unsigned)p.n_pages;
        bad |= !there;
        from[0] = base + (size_t)page[0] * page_bytes + (size_t)(pos & in_page) * D;
        if (there && pos + STEP * (CH - 1) < hi) {
          have = kAll;
        } else {
#pragma unroll
          for (int x = 0; x < CH; ++x) {
            from[x] = from[0] + STEP * D * x;
            have |= (there && pos + STEP * x < hi) << x;
          }
        }
      } else {
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          const int at_pos = pos + STEP * x;
          const bool there = (unsigned)page[x] < (unsigned)p.n_pages;
          bad |= !there && at_pos < hi;
          from[x] = base + (size_t)page[x] * page_bytes + (size_t)(at_pos & in_page) * D;
          have |= there << x;
        }
      }
    };
    auto load = [&](const uint8_t* codes, uint4 (&w)[CH]) {
      if (have == kAll) {
#pragma unroll
        for (int x = 0; x < CH; ++x) w[x] = ptx::ldg128(codes + from[0] + STEP * D * x);
      } else {
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          w[x] = make_uint4(0, 0, 0, 0);
          if (have >> x & 1) w[x] = ptx::ldg128(codes + from[x]);
        }
      }
    };
    auto load_scale = [&](int tile) {
      if (!tables) return;
      const int pos = (t0 + tile) * kKeys + (lane & 3) * 16;
      none = (unsigned)table_page >= (unsigned)p.n_pages;
      scale = 0.f;
      if (!none)
        scale = __ldg((lane < 4 ? p.ks : p.vs) +
                      (((size_t)table_page * p.Hkv + kvh) << (p.ps_log2 - p.t_log2)) +
                      ((pos & in_page) >> p.t_log2));
    };
    auto store = [&](unsigned char* tile, const uint4 (&w)[CH]) {
#pragma unroll
      for (int x = 0; x < CH; ++x) {
        uint4 lo, hi2;
        halves_of<F8>(w[x], lo, hi2);
        const int r = row + STEP * x;
        *reinterpret_cast<uint4*>(tile + box + swizzled(r, at)) = lo;
        *reinterpret_cast<uint4*>(tile + box + swizzled(r, at + 1)) = hi2;
      }
    };
    if (n > 0) {
      find(0);
      locate(0);
      load(p.k, k);
      load(p.v, v);
      load_scale(0);
      find(1);
    }
    for (int i = 0; i < n; ++i) {
      const int b = i & 1, before = ((i - 2) >> 1) & 1;
      // K's place is free once the scores of tile i - 2 are done, V's once its output is
      bool ok = i < 2 || wait(&s.s_done[b], before, &s.failed, a.patience);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (tables) {      // (scores i - 2 were issued behind the output of tile i - 4: its entry is free)
        if (lane < 4) {
          s.k_scale[i & 3][lane] = scale * fabsf(a.scale_log2);
          s.none[i & 3][lane] = none;
        } else {
          s.v_log2[i & 3][lane - 4] = log2f(scale);
        }
      }
      store(smem + L::K + b * L::TILE, k);
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) {
        if (warp == kSoftmax / 32) ptx::mbar_arrive(&s.t_full[i & 3]);
        ptx::mbar_arrive(&s.k_full[b]);
      }
      if (i + 1 < n) {
        locate(i + 1);
        load(p.k, k);
        load_scale(i + 1);
        find(i + 2);
      }
      ok = i < 2 || wait(&s.o_done[b], before, &s.failed, a.patience);
      if (!__all_sync(0xffffffffu, ok)) break;
      store(smem + L::V + b * L::TILE, v);
      ptx::fence_proxy_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&s.v_full[b]);
      if (i + 1 < n) load(p.v, v);
    }
    if (bad) flag_error(p.err, INT8KV_DEVERR_PAGE_ID);
  } else {
    // ---- the products
    constexpr uint32_t id_s = tc::idesc_f16(kRows, kKeys, 0, 0), id_o = tc::idesc_f16(kRows, D, 0, 1);
    const uint64_t dq = tc::sdesc(ptx::smem_u32(smem + L::Q), 16, 1024);
    const uint64_t dk = tc::sdesc(ptx::smem_u32(smem + L::K), 16, 1024);
    const uint64_t dv = tc::sdesc(ptx::smem_u32(smem + L::V), kBox, 1024);
    auto scores = [&](int i) {
      bool ok = i < 3 || wait(&s.o_done[(i - 3) & 1], ((i - 3) >> 1) & 1, &s.failed, a.patience);
      ok = ok && wait(&s.k_full[i & 1], (i >> 1) & 1, &s.failed, a.patience);
      if (!__all_sync(0xffffffffu, ok)) return false;
      tc::fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc::mma_ss(tmem + i % 3 * kKeys, dq + (((ks >> 2) * kQBox + (ks & 3) * 32) >> 4),
                     dk + (((i & 1) * L::TILE + (ks >> 2) * kBox + (ks & 3) * 32) >> 4), id_s, ks > 0);
        tc::mma_commit(&s.s_done[i & 1]);
      }
      __syncwarp();
      return true;
    };
    bool ok = __all_sync(0xffffffffu, wait(&s.q_full, 0, &s.failed, a.patience)) && (n == 0 || scores(0));
    int i = 0;
    for (; ok && i < n; ++i) {
      if (i + 1 < n && !scores(i + 1)) break;
      ok = wait(&s.w_full[i & 1], (i >> 1) & 1, &s.failed, a.patience) &&
           wait(&s.v_full[i & 1], (i >> 1) & 1, &s.failed, a.patience);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc::fence_after();
      if (ptx::elect_one()) {
#pragma unroll
        for (int j = 0; j < kKeys / 16; ++j) {
          const uint64_t d = dv + (((i & 1) * L::TILE + j * 2048) >> 4);
          const uint32_t w = tmem + i % 3 * kKeys + j * 16;
          tc::mma_ts(tmem + L::O, w, d, id_o, i % kChain > 0 || j > 0);
          tc::mma_ts(tmem + L::O, w + 8, d, id_o, true);
        }
        tc::mma_commit(&s.o_done[i & 1]);
      }
      __syncwarp();
    }
    // all products: complete, or the ones issued before a wait ran out
    uint64_t* end = ok && i == n ? &s.drain : &s.stopped;
    if (ptx::elect_one()) tc::mma_commit(end);
    __syncwarp();
    wait(end, 0, nullptr, kPatience);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kProducts) {
    tc::fence_after();
    tc::dealloc(tmem, L::COLS);
  }
}

// The splits of a row: one warp each, with up to four splits' values under way.
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) block_prefill_join_kernel(
    const float* part_o, const float2* part_ml, float* out, long long rows, int splits) {
  constexpr int W = D / 32;      // values of a lane: 2, 4, or two times 4
  const int lane = threadIdx.x & 31;
  const long long h = (long long)blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  if (h >= rows) return;
  const float2* ml = part_ml + h * splits;
  float m = -INFINITY, l = 0.f;
  for (int k = lane; k < splits; k += 32) m = fmaxf(m, ml[k].x);
  m = warp_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float o[W] = {};
  const float* from = part_o + (size_t)h * splits * D;
  for (int k0 = 0; k0 < splits; k0 += 32) {
    const float2 x = k0 + lane < splits ? ml[k0 + lane] : make_float2(-INFINITY, 0.f);
    const float mine = ptx::ex2(x.x - ref);
    l += x.y * mine;
    const int end = min(32, splits - k0);
#pragma unroll 4
    for (int k = 0; k < end; ++k) {
      const float f = __shfl_sync(0xffffffffu, mine, k);
      const float* row = from + (size_t)(k0 + k) * D;
      if constexpr (W == 2) {
        const float2 y = *reinterpret_cast<const float2*>(row + 2 * lane);
        o[0] = fmaf(f, y.x, o[0]);
        o[1] = fmaf(f, y.y, o[1]);
      } else {
#pragma unroll
        for (int c = 0; c < W / 4; ++c) {
          const float4 y = *reinterpret_cast<const float4*>(row + 128 * c + 4 * lane);
          o[4 * c] = fmaf(f, y.x, o[4 * c]);
          o[4 * c + 1] = fmaf(f, y.y, o[4 * c + 1]);
          o[4 * c + 2] = fmaf(f, y.z, o[4 * c + 2]);
          o[4 * c + 3] = fmaf(f, y.w, o[4 * c + 3]);
        }
      }
    }
  }
  l = warp_sum(l);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  float* to = out + (size_t)h * D;
  if constexpr (W == 2) {
    *reinterpret_cast<float2*>(to + 2 * lane) = make_float2(o[0] * inv, o[1] * inv);
  } else {
#pragma unroll
    for (int c = 0; c < W / 4; ++c)
      *reinterpret_cast<float4*>(to + 128 * c + 4 * lane) = make_float4(
          o[4 * c] * inv, o[4 * c + 1] * inv, o[4 * c + 2] * inv, o[4 * c + 3] * inv);
  }
}

template <int D>
cudaError_t launch_join(const PrefillBlockArgs& a, cudaStream_t stream) {
  const long long rows = (long long)a.n_new * a.H, grid = (rows + kJoinWarps - 1) / kJoinWarps;
  if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_prefill_join_kernel<D>, (const float*)a.part_o,
                            (const float2*)a.part_ml, a.out, rows, a.splits);
}

template <int D, bool F8>
cudaError_t launch_typed(const PrefillBlockArgs& a, cudaStream_t stream) {
  auto kernel = block_prefill_kernel<D, F8>;
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = true;
  }
  const long long grid = (long long)a.n_cg * a.pool.Hkv * a.splits;
  if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
  kernel<<<(unsigned)grid, kThreads, Layout<D>::SMEM, stream>>>(a);
  e = cudaGetLastError();
  return e != cudaSuccess || a.splits == 1 ? e : launch_join<D>(a, stream);
}

template <int D>
cudaError_t launch_codes(const PrefillBlockArgs& a, bool f8, cudaStream_t stream) {
  return f8 ? launch_typed<D, true>(a, stream) : launch_typed<D, false>(a, stream);
}

}  // namespace

cudaError_t launch_block_prefill(const BlockView& pool, const PrefillArgs& a, int head_dim, bool f8,
                                 uint32_t expire_us, cudaStream_t stream) {
  PrefillBlockArgs b;
  b.pool = pool;
  b.q = a.q;
  b.page_table = a.page_table;
  b.out = a.out;
  b.part_o = a.ws.part_o;
  b.part_ml = a.ws.part_ml;
  b.n_new = a.n_new;
  b.H = a.H;
  b.G = a.G;
  b.start = a.start;
  b.splits = a.n_splits;
  b.n_cg = (int)(((long long)a.n_new * a.G + kRows - 1) / kRows);
  b.scale_log2 = a.scale_log2;
  b.patience = expire_us ? expire_us * 1000ull : kPatience;
  b.expire = expire_us != 0;
  switch (head_dim) {
    case 64: return launch_codes<64>(b, f8, stream);
    case 128: return launch_codes<128>(b, f8, stream);
    default: return launch_codes<256>(b, f8, stream);
  }
}

}  // namespace int8kv
