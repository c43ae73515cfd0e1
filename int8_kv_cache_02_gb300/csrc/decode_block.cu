// Split-K GQA decode attention over block-scaled pools (one fp32 scale per T
// positions and kv head; int8 or e4m3 codes), and the combine of its partials.
//
//   z_i = (q . ck_i) sk(block of i) scale,  o = sum_i 2^(z_i) sv(block of i) cv_i / sum_i 2^(z_i)
// in base-2 exponents, ck and cv the codes: a scale multiplies 16 scores at once
// instead of every row's, so dequantizing is a bare conversion of codes to fp16,
// which is exact.
//
// Tiles of 16 positions (T and the page size are multiples of 16, so a tile has
// one page and one scale of each store).  A warp owns its tiles alone:
//   S^T[16 x 8] = K[16 x D] q^T[D x 8]            mma.sync m16n8k16, heads on N
//   O^T[D x 8] += V^T[D x 16] W^T[16 x 8]         W = 2^(z - M) sv, as fp16 hi + lo
// The D index of the first product and the row order of the second are permuted so
// that a lane's operands are the 16 bytes it copied itself: each lane brings its
// own pieces with cp.async into a ring that only it reads.  No barrier, no bank
// conflict, zero fill in place of rows outside the context.
//
// Two references per head: m for the softmax sum and M for the weights times their
// V scales, both the running maximum of what they scale (moved only when exceeded by
// 2^8), so the fp16 pair of W keeps ~22 bits of the largest weight whatever
// the scales' range.
//
// Schedule: all tiles of all (sequence, kv head, column group) units in one line,
// cut into equal shares, one per resident block ("a.shares"); a unit that a share
// boundary cuts leaves partials, numbered unit + share, which the combine kernel
// joins.  With a.shares = 0 every block takes one whole unit and writes it out.
//
// Bound by HBM: 2 D bytes per position and kv head.
#include "block_common.cuh"
#include "decode_common.cuh"

namespace int8kv {
namespace {

constexpr int kTile = 16;
constexpr float kUnset = -1e30f;      // reference of a head that has seen nothing
constexpr float kLazy = 8.f;          // a reference moves when exceeded by 2^8
constexpr float kWeightShift = 6.f;   // W is scaled by 2^6: at most 2^14 in fp16

template <int D>
struct Shape {
  static constexpr int NW = 4;                        // warps per block
  static constexpr int NS = D == 64 ? 4 : 3;          // ring stages per warp
  static constexpr int KP = D / 32;                   // 16-byte K pieces per lane and tile
  static constexpr int STAGE = kTile * D * 2;         // bytes of one warp's stage
  static constexpr int RING = NW * NS * STAGE;
  static constexpr int MERGE = NW * 8 * (D + 4) * 4;  // the warps' outputs, over the ring
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  static constexpr int BLOCKS = D == 256 ? 2 : (D == 128 ? 4 : 6);   // per SM
};

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? BYTES : 0;    // 0: BYTES zeros
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The positions of sequence b that some query of it attends: [lo, hi).
__device__ __forceinline__ void unit_range(const BlockDecodeArgs& a, int b, int& lo, int& hi) {
  hi = block_length(__ldg(a.seq_lens + b), a.max_pages, a.pool);
  lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
}
__device__ __forceinline__ int unit_tiles(int lo, int hi) {
  return hi > lo ? (hi - 1) / kTile - lo / kTile + 1 : 0;
}

// Where sequence boundaries lie in the line of tiles.  Every thread sums a run of
// sequences; the run that holds tile `at` is walked by its thread.
struct Place {
  long long total;   // tiles of the whole batch
  long long start;   // first tile of sequence b
  int b;
};
template <int NT>
__device__ __forceinline__ long long batch_tiles(const BlockDecodeArgs& a, int per_seq,
                                                 long long* warp_sums, long long& mine) {
  const int run = (a.B + NT - 1) / NT;
  long long sum = 0;
  for (int i = 0; i < run; ++i) {
    const int b = threadIdx.x * run + i;
    if (b >= a.B) break;
    int lo, hi;
    unit_range(a, b, lo, hi);
    sum += (long long)unit_tiles(lo, hi) * per_seq;
  }
  long long inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, off);
    if ((threadIdx.x & 31) >= off) inc += o;
  }
  if ((threadIdx.x & 31) == 31) warp_sums[threadIdx.x >> 5] = inc;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < (int)(threadIdx.x >> 5)) before += warp_sums[w];
    total += warp_sums[w];
  }
  mine = before + inc - sum;     // tiles before this thread's run
  return total;
}

__device__ __forceinline__ long long share_tiles(long long total, int shares, int least) {
  const long long per = (total + shares - 1) / shares;
  return per > least ? per : least;
}

// ---- one warp's tiles -------------------------------------------------------
template <int D, bool F8>
struct Warp {
  using S = Shape<D>;
  float acc[D / 16][4];    // O^T: rows 16-byte-piece order, columns 2t, 2t + 1
  float m[2], M[2], l[2];
  uint32_t q[D / 8];       // q^T fragments

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int j = 0; j < D / 16; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    m[0] = m[1] = M[0] = M[1] = kUnset;
    l[0] = l[1] = 0.f;
  }
};

// The lane's V pieces behind the K pieces of its stage (`stage` points at the lane's
// first K piece): 16 bytes of each of four tokens and every 128 values, 8 at D = 64.
template <int D>
__device__ __forceinline__ uint32_t v_pieces(uint32_t stage, int g, int t) {
  return stage + kTile * D - (D == 64 ? 8 * (4 * g + t) : 0);
}

// Issue the copies of one tile: rows 16 * tile .. + 15 of `page`, zeros for rows
// outside [lo, hi) or of no page.
template <int D>
__device__ __forceinline__ void issue_tile(const BlockView& p, uint32_t stage, int tile, int page,
                                           int kvh, int lo, int hi, int g, int t) {
  using S = Shape<D>;
  const int pos = tile * kTile;
  const int slot = pos & ((1 << p.ps_log2) - 1);
  const size_t row = ((((size_t)(page < 0 ? 0 : page) * p.Hkv + kvh) << p.ps_log2) + slot) * D;
  const int a = page < 0 ? 1 << 30 : lo - pos, z = page < 0 ? 0 : hi - pos;   // rows [a, z)
  const uint8_t* k = p.k + row;
  const uint8_t* v = p.v + row;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = g + 8 * r;
    const bool ok = i >= a && i < z;
#pragma unroll
    for (int c = 0; c < S::KP / 2; ++c)
      copy_async<16>(stage + (r * (S::KP / 2) + c) * 512, k + i * D + 64 * c + 16 * t, ok);
  }
  const uint32_t vs = v_pieces<D>(stage, g, t);
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const int i = 2 * t + (n & 1) + 8 * (n >> 1);
    const bool ok = i >= a && i < z;
    if constexpr (D == 64) {
      copy_async<8>(vs + n * 256, v + i * D + 8 * g, ok);
    } else {
#pragma unroll
      for (int c = 0; c < D / 128; ++c)
        copy_async<16>(vs + (n * (D / 128) + c) * 512, v + i * D + 128 * c + 16 * g, ok);
    }
  }
}

// One tile.  f = K scale * softmax scale * log2(e); lv = log2 of the V scale;
// lim[c]: last position that column c attends; masked: whether lim or lo cut the tile.
template <int D, bool F8>
__device__ __forceinline__ void take_tile(Warp<D, F8>& w, uint32_t stage, int pos, float f,
                                          float lv, bool masked, int lo, const int (&lim)[2],
                                          int g, int t) {
  using S = Shape<D>;
  float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < S::KP / 2; ++c) {
    const uint4 x = ptx::lds128(stage + c * 512);
    const uint4 y = ptx::lds128(stage + (S::KP / 2 + c) * 512);
    const uint32_t* xw = reinterpret_cast<const uint32_t*>(&x);
    const uint32_t* yw = reinterpret_cast<const uint32_t*>(&y);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t a[4] = {codes_to_h2<F8>(xw[u]), codes_to_h2<F8>(yw[u]),
                             codes_to_h2<F8>(codes_behind<F8>(xw[u])),
                             codes_to_h2<F8>(codes_behind<F8>(yw[u]))};
      ptx::mma_f16(u & 1 ? s1 : s0, a, w.q[8 * c + 2 * u], w.q[8 * c + 2 * u + 1]);
    }
  }
  // z[2r + c]: row g + 8 r, column 2 t + c
  float z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) z[i] = (s0[i] + s1[i]) * f;
  if (masked) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = pos + g + 8 * (i >> 1);
      if (at < lo || at > lim[i & 1]) z[i] = -INFINITY;
    }
  }
  const float top0 = fmaxf(z[0], z[2]), top1 = fmaxf(z[1], z[3]);
  const bool over = top0 > w.m[0] + kLazy || top1 > w.m[1] + kLazy ||
                    top0 + lv > w.M[0] + kLazy || top1 + lv > w.M[1] + kLazy;
  if (__any_sync(0xffffffffu, over)) {
    float top[2] = {top0, top1};
    float r[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1)
        top[c] = fmaxf(top[c], __shfl_xor_sync(0xffffffffu, top[c], off));
      const float nm = fmaxf(w.m[c], top[c]), nM = fmaxf(w.M[c], top[c] + lv);
      w.l[c] *= ptx::ex2(w.m[c] - nm);
      r[c] = ptx::ex2(w.M[c] - nM);
      w.m[c] = nm;
      w.M[c] = nM;
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      w.acc[j][0] *= r[0];
      w.acc[j][1] *= r[1];
      w.acc[j][2] *= r[0];
      w.acc[j][3] *= r[1];
    }
  }
  float wt[4];
  const float u0 = lv + kWeightShift - w.M[0], u1 = lv + kWeightShift - w.M[1];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w.l[i & 1] += ptx::ex2(z[i] - w.m[i & 1]);
    wt[i] = ptx::ex2(z[i] + (i & 1 ? u1 : u0));
  }
  uint32_t hi[2], lo2[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t h = ptx::pack_f16x2(wt[2 * r], wt[2 * r + 1]);
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h));
    hi[r] = ptx::movmatrix_trans(h);
    lo2[r] = ptx::movmatrix_trans(ptx::pack_f16x2(wt[2 * r] - b.x, wt[2 * r + 1] - b.y));
  }
  // V words: the first half of a token's words in the lane are rows g, the others rows g + 8
  const uint32_t vs = v_pieces<D>(stage, g, t);
#pragma unroll
  for (int h = 0; h < (D == 256 ? 2 : 1); ++h) {    // D = 256: eight words in two halves
    uint32_t a[4][4], b[4][4];                       // [token][word] of rows g and g + 8
    constexpr int N = D == 64 ? 1 : (D == 128 ? 2 : 2);   // words taken per half
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      if constexpr (D == 64) {
        const uint2 x = ptx::lds64(vs + n * 256);
        a[n][0] = x.x;
        b[n][0] = x.y;
      } else if constexpr (D == 128) {
        const uint4 x = ptx::lds128(vs + n * 512);
        a[n][0] = x.x;
        a[n][1] = x.y;
        b[n][0] = x.z;
        b[n][1] = x.w;
      } else {
        const uint2 x = ptx::lds64(vs + n * 1024 + h * 8);
        const uint2 y = ptx::lds64(vs + n * 1024 + 512 + h * 8);
        a[n][0] = x.x;
        a[n][1] = x.y;
        b[n][0] = y.x;
        b[n][1] = y.y;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t pa[2][2], pb[2][2];      // [k half][first / second pair word]
#pragma unroll
      for (int kh = 0; kh < 2; ++kh) {
        pair_words<F8>(a[2 * kh][i], a[2 * kh + 1][i], pa[kh][0], pa[kh][1]);
        pair_words<F8>(b[2 * kh][i], b[2 * kh + 1][i], pb[kh][0], pb[kh][1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t fr[4];
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          const uint32_t wa = pa[kh][e >> 1], wb = pb[kh][e >> 1];
          fr[2 * kh] = codes_to_h2<F8>(e & 1 ? codes_behind<F8>(wa) : wa);
          fr[2 * kh + 1] = codes_to_h2<F8>(e & 1 ? codes_behind<F8>(wb) : wb);
        }
        float(&o)[4] = w.acc[(h * N + i) * 4 + e];
        ptx::mma_f16(o, fr, hi[0], hi[1]);
        ptx::mma_f16(o, fr, lo2[0], lo2[1]);
      }
    }
  }
}

// d index of row (g + 8 r) of O^T tile j.
template <int D>
__device__ __forceinline__ int out_dim(int j, int r, int g) {
  if constexpr (D == 64) return 8 * g + 4 * r + j;
  if constexpr (D == 128) return 16 * g + 8 * r + j;
  return 128 * r + 16 * g + j;
}

template <int D, bool F8>
__global__ void __launch_bounds__(Shape<D>::NW * 32, Shape<D>::BLOCKS)
    decode_block_kernel(const BlockDecodeArgs a) {
  using S = Shape<D>;
  constexpr int NT = S::NW * 32;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long warp_sums[S::NW];
  __shared__ long long place_start;
  __shared__ int place_b;
  __shared__ float stat[3][S::NW][8];     // m, M, l of each warp and column
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = ptx::smem_u32(smem) + warp * S::NS * S::STAGE + lane * 16;
  const BlockView& p = a.pool;
  const int per_seq = p.Hkv * a.n_cg;      // units of a sequence
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();

  long long at, end, seq_start;
  int b;
  if (a.shares == 0) {
    b = blockIdx.x / per_seq;
    int lo, hi;
    unit_range(a, b, lo, hi);
    const int nt = unit_tiles(lo, hi), u = blockIdx.x % per_seq;
    seq_start = 0;
    at = (long long)u * nt;
    end = at + nt;
    if (nt == 0) end = at + 1;    // run the unit's (empty) segment once: zero rows
  } else {
    long long mine;
    const long long total = batch_tiles<NT>(a, per_seq, warp_sums, mine);
    const long long per = share_tiles(total, a.shares, S::NW);
    at = per * blockIdx.x;
    end = min(at + per, total);
    if (at >= end) return;
    const int run = (a.B + NT - 1) / NT;
    for (int i = 0; i < run; ++i) {
      const int s = threadIdx.x * run + i;
      if (s >= a.B) break;
      int lo, hi;
      unit_range(a, s, lo, hi);
      const long long n = (long long)unit_tiles(lo, hi) * per_seq;
      if (at >= mine && at < mine + n) {
        place_b = s;
        place_start = mine;
      }
      mine += n;
    }
    __syncthreads();
    b = place_b;
    seq_start = place_start;
  }

  Warp<D, F8> w;
  while (at < end) {
    int lo, hi;
    unit_range(a, b, lo, hi);
    const int nt = unit_tiles(lo, hi);
    const int u = a.shares == 0 ? blockIdx.x % per_seq : (nt ? (int)((at - seq_start) / nt) : per_seq);
    if (u >= per_seq) {           // past this sequence's units
      seq_start += (long long)nt * per_seq;
      ++b;
      continue;
    }
    const int kvh = u / a.n_cg, cg = u % a.n_cg;
    const int first = nt ? (int)(at - seq_start - (long long)u * nt) : 0;   // tiles of the unit: [first, last)
    const int last = (int)min((long long)nt, first + (end - at));
    const int tile0 = lo / kTile;

    // columns 2t, 2t + 1 of the fragments and the lane's q row (column g)
    const int cols = min(a.width, a.G * a.Q - cg * a.width);
    int lim[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int col = 2 * t + c;
      lim[c] = col < cols ? hi - a.Q + (cg * a.width + col) / a.G : -1;
    }
    const int least = hi - a.Q + (cg * a.width) / a.G;   // positions <= least: no column masks
    {
      const int col = cg * a.width + min(g, cols - 1);
      const uint16_t* q =
          a.q + (((size_t)b * a.Q + col / a.G) * a.H + kvh * a.G + col % a.G) * D + 16 * t;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const uint4 x = ptx::ldg128(q + 64 * c), y = ptx::ldg128(q + 64 * c + 8);
        const uint32_t v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {     // pieces 4k .. 4k + 3 of the lane's 16 values
          uint32_t lo2 = v[2 * k], hi2 = v[2 * k + 1];
          if (g >= cols) lo2 = hi2 = 0;
          w.q[8 * c + 2 * k] = F8 ? lo2 : ptx::prmt(lo2, hi2, 0x5410);
          w.q[8 * c + 2 * k + 1] = F8 ? hi2 : ptx::prmt(lo2, hi2, 0x7632);
        }
      }
    }
    w.reset();

    // the warp's tiles of the segment: first + warp, + NW, ...
    const int n = last - first > warp ? (last - first - warp + S::NW - 1) / S::NW : 0;
    const int32_t* table = a.page_table + (size_t)b * a.max_pages;
    int pages = -1;             // lane i: page and scales of tile (issue index & ~31) + i
    float fs = 0.f, ls = 0.f;
    int pages_now = -1;         // the same for the tile being taken
    float fs_now = 0.f, ls_now = 0.f;
    auto issue = [&](int i) {
      if ((i & 31) == 0) {
        const int mine = i + lane;
        pages = -1;
        if (mine < n) {
          const int pos = (tile0 + first + warp + mine * S::NW) * kTile;
          pages = block_page(table, pos >> p.ps_log2, p);
          if (pages >= 0) {
            const size_t blk = (((size_t)pages * p.Hkv + kvh) << (p.ps_log2 - p.t_log2)) +
                               ((pos & ((1 << p.ps_log2) - 1)) >> p.t_log2);
            fs = __ldg(p.ks + blk) * a.scale_log2;
            ls = log2f(__ldg(p.vs + blk));
          }
        }
      }
      if (i < n) {
        const int tile = tile0 + first + warp + i * S::NW;
        const int page = __shfl_sync(0xffffffffu, pages, i & 31);
        issue_tile<D>(p, ring + (i % S::NS) * S::STAGE, tile, page, kvh, lo, hi, g, t);
      }
      commit_copies();
    };
#pragma unroll
    for (int i = 0; i < S::NS - 1; ++i) issue(i);
    for (int i = 0; i < n; ++i) {
      if ((i & 31) == 0) {
        pages_now = pages;
        fs_now = fs;
        ls_now = ls;
      }
      issue(i + S::NS - 1);
      wait_copies<S::NS - 1>();
      const int page = __shfl_sync(0xffffffffu, pages_now, i & 31);
      const float f = __shfl_sync(0xffffffffu, fs_now, i & 31);
      const float lv = __shfl_sync(0xffffffffu, ls_now, i & 31);
      if (page < 0) continue;     // no such page: its keys are left out
      const int pos = (tile0 + first + warp + i * S::NW) * kTile;
      const bool masked = pos < lo || pos + kTile - 1 > least;
      take_tile<D, F8>(w, ring + (i % S::NS) * S::STAGE, pos, f, lv, masked, lo, lim, g, t);
    }
    wait_copies<0>();

    // join the warps
    __syncthreads();
    float* merge = reinterpret_cast<float*>(smem);
    if (n > 0) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < D / 16; j += 4)
            *reinterpret_cast<float4*>(merge + (warp * 8 + 2 * t + c) * (D + 4) +
                                       out_dim<D>(j, r, g)) =
                make_float4(w.acc[j][2 * r + c], w.acc[j + 1][2 * r + c], w.acc[j + 2][2 * r + c],
                            w.acc[j + 3][2 * r + c]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float l = w.l[c];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      if (g == 0) {
        stat[0][warp][2 * t + c] = w.m[c];
        stat[1][warp][2 * t + c] = w.M[c];
        stat[2][warp][2 * t + c] = l;
      }
    }
    __syncthreads();
    const bool whole = first == 0 && last == nt;
    const int live = min(S::NW, last - first);     // warps that had tiles
    const long long slot = (long long)b * per_seq + u + blockIdx.x;
    for (int i = threadIdx.x; i < cols * (D / 4); i += NT) {
      const int col = i / (D / 4), d = i % (D / 4) * 4;
      float m = kUnset, M = kUnset;
      for (int k = 0; k < live; ++k) {
        m = fmaxf(m, stat[0][k][col]);
        M = fmaxf(M, stat[1][k][col]);
      }
      float l = 0.f;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < live; ++k) {
        l += stat[2][k][col] * ptx::ex2(stat[0][k][col] - m);
        const float r = ptx::ex2(stat[1][k][col] - M);
        const float4 x = *reinterpret_cast<const float4*>(merge + (k * 8 + col) * (D + 4) + d);
        o.x = fmaf(r, x.x, o.x);
        o.y = fmaf(r, x.y, o.y);
        o.z = fmaf(r, x.z, o.z);
        o.w = fmaf(r, x.w, o.w);
      }
      const float inv = l > 0.f ? ptx::ex2(M - m - kWeightShift) / l : 0.f;
      o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      if (whole) {
        const int gc = cg * a.width + col;
        float* out = a.out + (((size_t)b * a.Q + gc / a.G) * a.H + kvh * a.G + gc % a.G) * D + d;
        *reinterpret_cast<float4*>(out) = o;
      } else {
        *reinterpret_cast<float4*>(a.part_o + (slot * a.width + col) * D + d) = o;
        if (d == 0) a.part_lse[slot * a.width + col] = l > 0.f ? m + log2f(l) : -INFINITY;
      }
    }
    if (a.shares == 0) return;
    at += last - first;
    __syncthreads();      // the next segment's copies overwrite the merge buffer
  }
}

// Join the partials of units that a share boundary cut; zero rows of empty units.
// One block per (sequence, query, head).
__global__ void __launch_bounds__(128) decode_block_combine_kernel(const BlockDecodeArgs a, int D,
                                                                   int least) {
  __shared__ long long warp_sums[4];
  __shared__ long long place;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int row = blockIdx.x, h = row % a.H, bq = row / a.H, b = bq / a.Q;
  const int kvh = h / a.G, gc = (bq % a.Q) * a.G + h % a.G, cg = gc / a.width, col = gc % a.width;
  const int per_seq = a.pool.Hkv * a.n_cg;
  long long mine;
  const long long total = batch_tiles<128>(a, per_seq, warp_sums, mine);
  int lo, hi;
  const int run = (a.B + 127) / 128;
  if (b / run == (int)threadIdx.x) {
    for (int s = threadIdx.x * run; s < b; ++s) {
      unit_range(a, s, lo, hi);
      mine += (long long)unit_tiles(lo, hi) * per_seq;
    }
    place = mine;
  }
  __syncthreads();
  unit_range(a, b, lo, hi);
  const int nt = unit_tiles(lo, hi), u = kvh * a.n_cg + cg;
  float* out = a.out + (size_t)row * D;
  if (nt == 0) {
    for (int d = threadIdx.x; d < D; d += 128) out[d] = 0.f;
    return;
  }
  const long long per = share_tiles(total, a.shares, least);
  const long long start = place + (long long)u * nt;
  const long long c0 = start / per, c1 = (start + nt - 1) / per;
  if (c0 == c1) return;      // one block had the whole unit and wrote it
  const long long slot = (long long)b * per_seq + u;
  const float* lse = a.part_lse + (slot + c0) * a.width + col;
  const float* o = a.part_o + ((slot + c0) * a.width + col) * D;
  const int n = (int)(c1 - c0 + 1);
  float M = -INFINITY;
  for (int i = 0; i < n; ++i) M = fmaxf(M, lse[(size_t)i * a.width]);
  for (int d = threadIdx.x; d < D; d += 128) {
    float x = 0.f, l = 0.f;
    for (int i = 0; i < n; ++i) {
      const float r = M > -INFINITY ? ptx::ex2(lse[(size_t)i * a.width] - M) : 0.f;
      l += r;
      x = fmaf(r, o[(size_t)i * a.width * D + d], x);
    }
    out[d] = l > 0.f ? x / l : 0.f;
  }
}

template <int D, bool F8>
cudaError_t launch(const BlockDecodeArgs& a, cudaStream_t stream) {
  using S = Shape<D>;
  const long long units = (long long)a.B * a.pool.Hkv * a.n_cg;
  const long long rows = (long long)a.B * a.Q * a.H;
  const long long grid = a.shares ? a.shares : units;
  if (grid > 0x7fffffffLL || rows > 0x7fffffffLL) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(S::NW * 32);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, decode_block_kernel<D, F8>, a);
  if (e != cudaSuccess || a.shares == 0) return e;
  cfg.gridDim = dim3((unsigned)rows);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, decode_block_combine_kernel, a, D, (int)S::NW);
}

template <int D, bool F8>
int resident() {
  using S = Shape<D>;
  int per_sm = 0, dev = 0, sms = 0;
  if (cudaFuncSetAttribute(decode_block_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           S::SMEM) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, decode_block_kernel<D, F8>,
                                                    S::NW * 32, S::SMEM) != cudaSuccess ||
      cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  return per_sm * sms;
}

}  // namespace

int block_decode_resident(int head_dim, bool f8) {
  switch (head_dim) {
    case 64: return f8 ? resident<64, true>() : resident<64, false>();
    case 128: return f8 ? resident<128, true>() : resident<128, false>();
    case 256: return f8 ? resident<256, true>() : resident<256, false>();
    default: return -1;
  }
}

cudaError_t launch_block_decode(const BlockDecodeArgs& a, int head_dim, bool f8,
                                cudaStream_t stream) {
  switch (head_dim) {
    case 64: return f8 ? launch<64, true>(a, stream) : launch<64, false>(a, stream);
    case 128: return f8 ? launch<128, true>(a, stream) : launch<128, false>(a, stream);
    case 256: return f8 ? launch<256, true>(a, stream) : launch<256, false>(a, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace int8kv
