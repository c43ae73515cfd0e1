// The decode kernel over block-scaled pools (one fp32 scale per T positions and kv
// head; int8 or e4m3 codes), for the translation units that instantiate it.
//
//   z_i = (q . ck_i) sk(block of i) scale,  o = sum_i 2^(z_i) sv(block of i) cv_i / sum_i 2^(z_i)
// in base-2 exponents, ck and cv the codes: a scale multiplies 16 scores at once
// instead of every row's, so dequantizing is a bare conversion of codes to fp16,
// which is exact.
//
// Tiles of 16 positions (T and the page size are multiples of 16, so a tile has
// one page and one scale of each store).  A warp owns its tiles alone:
//   S^T[16 x 8] = K[16 x D] q^T[D x 8]            mma.sync m16n8k16, heads on N
//   O^T[D x 8] += V^T[D x 16] W^T[16 x 8]         W = 2^(z - m - e) sv, as fp16 hi + lo
// A tile's rows are contiguous in the pool; the warp copies them with cp.async, whole
// 128-byte lines at a time, into a ring of its own (no barrier but the warp's), with
// zeros in place of rows outside the context.  (Lanes that fetched just the 64 bytes of
// a row that they use read HBM at 5.5 TB/s, whole lines at 7.4: requests of half a line
// halve what the L2 can ask for.)  The D index of the first product, the row order of
// the second and the order of a tile's positions are permuted, and 16-byte pieces
// swizzled, so that an operand is a 16-byte shared-memory load without bank conflicts
// (D = 64: V two-way).
//
// Two references per head: m for the softmax sum and m + e for the weights times their
// V scales, both the running maximum of what they scale (moved only when exceeded by
// 2^8), so the fp16 pair of W keeps ~22 bits of the largest weight whatever
// the scales' range.  A score meets nothing but m, in a difference of near numbers that is
// exact; e and the V scales' logarithms are small.  (One reference of the scores' own size
// for the weights would round each tile's exponents to its last place: 2^-9 off
// at scores of 4e4, and past fp16's range at 4e7.)
//
// A column is a (query, head) pair of the kv head.  With at most four of them
// (kPair) columns 4 - 7 hold the same queries again: there W is the lo part, and one
// product brings both (the halves are added at the end).  More than eight take two
// groups of columns per pass (NC = 2), so that a page is read and converted once for
// 16 columns; at D 256 their queries' fragments lie in shared memory, the sums alone
// taking 128 registers.
//
// Schedule: all (sequence, kv head, column group) units in one line, each as long as
// its tiles plus a start of kStart (what a block spends on a unit besides its tiles:
// fetching q, the first wait, joining its warps), cut into equal shares, one per
// resident block (a.shares).  A unit that a share boundary cuts leaves partials,
// numbered unit + share, which the combine kernel joins.  The first copies of a
// block's next unit are under way while its warps are joined for the last one.  With
// a.shares = 0 every block takes one whole unit and writes it out, or, for few units of
// middling length, the blocks of a cluster share a unit's tiles and join their outputs
// through distributed shared memory: no partials, no combine kernel.
//
// Behind an append of the same call (a.appended) the kernel starts under it: only the
// blocks that the append writes, the last of every sequence, wait for it.  Lengths, page
// table, queries and the other blocks are read without a wait of this kernel's own.  What that
// rests on is an order: every block of the append has waited, so that all kernels before it
// are complete and their results in global memory, before it lets this one start, and nothing
// writes them while this one runs.  That a kernel two launches on sees such results without
// waiting is documented nowhere; steps back to back with forks of their rows, with nothing
// between them but these launches, bear it out (test_forks_and_fused_steps_back_to_back).
// Reading them past L1, the one place where older copies could be, cost 3 % of a fused step
// (8K 11.8 -> 12.1 us) and 1 to 4 % of the calls without an append.
//
// Bound by HBM: 2 D bytes per position and kv head.
#pragma once

#include <algorithm>
#include <climits>

#include <cooperative_groups.h>

#include "block_common.cuh"
#include "decode_common.cuh"

namespace int8kv {
namespace block {

constexpr int kTile = 16;
constexpr float kUnset = -1e30f;      // reference of a head that has seen nothing
constexpr float kLazy = 8.f;          // a reference moves when exceeded by 2^8
constexpr float kWeightShift = 6.f;   // W is scaled by 2^6: at most 2^14 in fp16

template <int D>
struct Shape {
  // Warps per block, eight to an SM.  D 256: one block of eight halves the partials
  // (128K 31.6 -> 29.8 us; an 8K step 11.3 -> 12.0 us; with sums rounded tile by tile, as they
  // are now, 31.1 and 12.5, and e4m3 30.0 and 11.6); below, two blocks of four
  // keep more units apart (64 sequences at D 128: 314 us against 318).
  static constexpr int NW = D == 256 ? 8 : 4;
  static constexpr int TPI = 256 / D;                 // tiles a warp takes at a time
  static constexpr int NS = 3;                        // ring stages per warp
  static constexpr int BLOCKS = 8 / NW;               // per SM
  static constexpr int START = 2 * NW * TPI;          // a unit's start, in tiles
  static constexpr int LEAST = NW * TPI * (NS - 1);   // a share at least: its rings' first fill
  static constexpr int KP = D / 64;                   // 16-byte K pieces per lane and row
  static constexpr int ROWS = kTile * D;              // bytes of a tile's K rows, or V rows
  static constexpr int TILE = 2 * ROWS;               // bytes of a tile in the ring: K, then V
  static constexpr int STAGE = TPI * TILE;
  static constexpr int RING = NW * NS * STAGE;
};

// Variants of the kernel by columns of a unit.
enum Columns { kPair = 0, kEight = 1, kSixteen = 2 };
template <int V>
struct Cols {
  static constexpr int NC = V == kSixteen ? 2 : 1;
  static constexpr int N = 8 * NC;                    // columns of the products
};

// Whether the queries' fragments lie in shared memory, behind the rings, and its size.
template <int D, int V>
constexpr bool kSharedQ = D == 256 && V == kSixteen;
template <int D, int V>
constexpr int kSmem = Shape<D>::RING + (kSharedQ<D, V> ? 16 * D * 2 : 0);

template <bool FULL>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool valid) {
  if constexpr (FULL) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  } else {
    const int n = valid ? 16 : 0;    // 0: zeros
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
  }
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ int length_of(const BlockDecodeArgs& a, int b) {
  return a.seq_lens ? __ldg(a.seq_lens + b) : a.length;
}

// The positions of sequence b that some query of it attends: [lo, hi).
__device__ __forceinline__ void unit_range(const BlockDecodeArgs& a, int b, int& lo, int& hi) {
  hi = block_length(length_of(a, b), a.max_pages, a.pool);
  lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
}
__device__ __forceinline__ int unit_tiles(int lo, int hi) {
  return hi > lo ? (hi - 1) / kTile - lo / kTile + 1 : 0;
}

// Length in the line of the units of a sequence of length `len`.
__device__ __forceinline__ int line_length(const BlockDecodeArgs& a, int len, int per_seq,
                                           int start) {
  const int cap = a.max_pages << a.pool.ps_log2;
  const int hi = len < cap ? len : cap;
  const int nt = unit_tiles(a.window > 0 && hi > a.window ? hi - a.window : 0, hi);
  return nt ? (nt + start) * per_seq : 0;
}

// What a share's place in the line is made of: sequence b's units begin at `base`.
// Every warp finds it by itself: a lane sums a run of sequences, and the lane whose
// run holds the place walks it.  (The whole line is shorter than 2^31.)
struct Place {
  int at, end, b, base, per;
};
__device__ __forceinline__ Place find_share(const BlockDecodeArgs& a, int per_seq, int start,
                                            int least) {
  const int lane = threadIdx.x & 31, run = (a.B + 31) / 32;
  int sum = 0;
  for (int i = 0; i < run; i += 8) {      // (eight lengths under way)
    int len[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      len[k] = i + k < run && lane * run + i + k < a.B ? length_of(a, lane * run + i + k) : 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) sum += line_length(a, len[k], per_seq, start);
  }
  int inc = sum;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += o;
  }
  const int total = __shfl_sync(0xffffffffu, inc, 31);
  const int even = (int)(((unsigned)total + a.shares - 1) / (unsigned)a.shares);
  const int per = even > least ? even : least;
  Place p;
  p.per = per;
  const long long at = (long long)per * blockIdx.x;
  if (at >= total) {
    p.at = p.end = total;
    p.b = a.B;
    p.base = total;
    return p;
  }
  p.at = (int)at;
  p.end = (int)min(at + per, (long long)total);
  int base = inc - sum, b = lane * run;
  const bool mine = p.at >= base && p.at < inc;
  if (mine && run > 1)
    for (;;) {
      const int n = line_length(a, length_of(a, b), per_seq, start);
      if (p.at < base + n) break;
      base += n;
      ++b;
    }
  const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  p.b = __shfl_sync(0xffffffffu, b, from);
  p.base = __shfl_sync(0xffffffffu, base, from);
  return p;
}

// The part of a unit that one block takes: tiles [first, last) of unit u of sequence b.
// pieces: how many shares the unit lies in, from this one on.
struct Segment {
  int b, u, lo, hi, nt, first, last, pieces;
};

// The segment at p.at, and p behind it; false at the share's end.
__device__ __forceinline__ bool next_segment(const BlockDecodeArgs& a, Place& p, int per_seq,
                                             int start, Segment& s) {
  while (p.at < p.end) {
    unit_range(a, p.b, s.lo, s.hi);
    s.nt = unit_tiles(s.lo, s.hi);
    const int len = s.nt + start;
    s.u = s.nt ? (int)((unsigned)(p.at - p.base) / (unsigned)len) : per_seq;
    if (s.u >= per_seq) {     // past this sequence's units
      p.base += s.nt ? len * per_seq : 0;
      ++p.b;
      continue;
    }
    s.b = p.b;
    const int unit = p.base + s.u * len + start;      // where its tiles begin
    s.first = max(0, p.at - unit);
    s.last = min(s.nt, p.end - unit);
    p.at = min(p.end, unit + s.nt);
    s.pieces = (int)((unsigned)(unit + s.nt - 1) / (unsigned)p.per) - blockIdx.x + 1;
    if (s.last > s.first) return true;                // (else the share ends in the unit's start)
  }
  return false;
}

// ---- one warp's tiles -------------------------------------------------------
template <int D, int V>
struct Warp {
  static constexpr int NC = Cols<V>::NC;
  float acc[NC][D / 16][4];    // O^T: rows in out_dim's order, columns 2t, 2t + 1
  float m[NC][2], e[NC][2], l[NC][2];
  uint32_t q[NC][kSharedQ<D, V> ? 1 : D / 8];       // q^T fragments

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        acc[n][j][0] = acc[n][j][1] = acc[n][j][2] = acc[n][j][3] = 0.f;
      m[n][0] = m[n][1] = e[n][0] = e[n][1] = kUnset;
      l[n][0] = l[n][1] = 0.f;
    }
  }
};

// A tile in shared memory: rows of D bytes, the 16-byte pieces of row r permuted by an
// xor with bits of r so that the loads below meet no bank twice.
template <int D>
__device__ __forceinline__ int piece(int r, int c) {
  return r * D + ((D == 64 ? c ^ (r >> 1 & 3) : c ^ (r & 7)) << 4);
}

// Position of a tile that row x of the fragments stands for (x and x + 8 alike): rows
// 2i and 2i + 1 differ in bits 0 and 2 of it, which the K loads need, and the even (odd)
// rows take all values of bits 1 and 2, which the V loads need.
__device__ __forceinline__ int position_of(int x) { return x ^ ((x & 1) << 2); }

// What of a tile a lane copies and loads: byte offsets within K or V rows.
template <int D>
struct Lane {
  uint32_t to;        // its first copied piece
  uint32_t k;         // row g, piece t
  uint32_t v[2];      // rows 2t and 2t + 1, its piece (D = 64: half a piece)
  __device__ __forceinline__ Lane(int lane) {
    const int g = lane >> 2, t = lane & 3;
    to = piece<D>(lane * 16 / D, lane * 16 % D / 16);
    k = piece<D>(position_of(g), t);
#pragma unroll
    for (int n = 0; n < 2; ++n)
      v[n] = D == 64 ? piece<D>(position_of(2 * t + n), g >> 1) + 8 * (g & 1)
                     : piece<D>(position_of(2 * t + n), g);
  }
};

// Issue the copies of one tile from its rows at k and v (at the lane's 16 bytes):
// zeros for rows outside [a, z).  Copy i takes bytes 512 i + 16 lane of the rows.
template <int D, bool FULL>
__device__ __forceinline__ void copy_tile(const uint8_t* k, const uint8_t* v, uint32_t tile,
                                          const Lane<D>& ln, int a, int z, int lane) {
  using S = Shape<D>;
#pragma unroll
  for (int i = 0; i < S::ROWS / 512; ++i) {
    const int r = (512 * i + 16 * lane) / D;
    const bool ok = r >= a && r < z;
    // rows 512 i / D further: their low bits flip bits of the piece
    const uint32_t to = 512 * i + (D == 64 ? ln.to : ln.to ^ ((512 * i / D & 7) << 4));
    copy_async<FULL>(tile + to, k + 512 * i, ok);
    copy_async<FULL>(tile + S::ROWS + to, v + 512 * i, ok);
  }
}

// The lane's words of its four V tokens and 16 values (D = 64: 8), of O^T rows g (a) and
// g + 8 (b); h: which 128 of D = 256.
template <int D>
__device__ __forceinline__ void v_words(uint32_t tile, const Lane<D>& ln, int h,
                                        uint32_t (&a)[4][2], uint32_t (&b)[4][2]) {
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    const uint32_t at = tile + Shape<D>::ROWS + ln.v[n & 1] + (n >> 1) * 8 * D + h * 128;
    if constexpr (D == 64) {
      const uint2 x = ptx::lds64(at);
      a[n][0] = x.x;
      b[n][0] = x.y;
    } else {
      const uint4 x = ptx::lds128(at);
      a[n][0] = x.x;
      a[n][1] = x.y;
      b[n][0] = x.z;
      b[n][1] = x.w;
    }
  }
}

// D = A * B, as ptx::mma_f16 with no sum to add to.
__device__ __forceinline__ void mma_from_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// S^T of one tile: z[n][2r + c] is row g + 8r, column 2t + c of group n.
template <int D, bool F8, int V>
__device__ __forceinline__ void score_tile(const Warp<D, V>& w, uint32_t tile, const Lane<D>& ln,
                                           uint32_t shared_q, float (&z)[Cols<V>::NC][4]) {
  using S = Shape<D>;
  constexpr int NC = Cols<V>::NC;
  float s[2][NC][4];
#pragma unroll
  for (int c = 0; c < S::KP; ++c) {
    // piece 4c + t of rows g and g + 8
    const uint32_t at = tile + (ln.k ^ ((c & 1) << 6)) + (c >> 1) * 128;
    const uint4 x = ptx::lds128(at), y = ptx::lds128(at + 8 * D);
    const uint32_t* xw = reinterpret_cast<const uint32_t*>(&x);
    const uint32_t* yw = reinterpret_cast<const uint32_t*>(&y);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t a[4] = {codes_to_h2<F8>(xw[u]), codes_to_h2<F8>(yw[u]),
                             codes_behind_to_h2<F8>(xw[u]), codes_behind_to_h2<F8>(yw[u])};
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        uint2 q;
        if constexpr (kSharedQ<D, V>)
          q = ptx::lds64(shared_q + (n * (D / 16) + 4 * c + u) * 256);
        else
          q = make_uint2(w.q[n][8 * c + 2 * u], w.q[n][8 * c + 2 * u + 1]);
        if (c == 0 && u < 2)
          mma_from_zero(s[u][n], a, q.x, q.y);
        else
          ptx::mma_f16(s[u & 1][n], a, q.x, q.y);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) z[n][i] = s[0][n][i] + s[1][n][i];
}

// The TPI tiles of one stage.  f: K scale * softmax scale * log2(e) of each tile; lv: log2 of
// its V scale; lim: last position that each column attends; masked: whether lim, lo
// or a tile that is not there (bit i of `none`) cut the stage.
template <int D, bool F8, int V>
__device__ __forceinline__ void take_stage(Warp<D, V>& w, uint32_t stage, int pos,
                                           const float (&f)[Shape<D>::TPI],
                                           const float (&lv)[Shape<D>::TPI], bool masked,
                                           uint32_t none, int lo, const int (&lim)[Cols<V>::NC][2],
                                           const Lane<D>& ln, uint32_t shared_q, int g, int t) {
  using S = Shape<D>;
  constexpr int NC = Cols<V>::NC, TPI = S::TPI;
  float z[TPI][NC][4];
  float top[NC][2];
#pragma unroll
  for (int i = 0; i < TPI; ++i) {
    score_tile<D, F8, V>(w, stage + i * S::TILE, ln, shared_q, z[i]);
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) z[i][n][k] *= f[i];
  }
  if (masked) {
#pragma unroll
    for (int i = 0; i < TPI; ++i)
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = pos + i * kTile + position_of(g) + 8 * (k >> 1);
          if (at < lo || at > lim[n][k & 1] || (none >> i & 1)) z[i][n][k] = -INFINITY;
        }
  }
  bool over = false;
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int i = 0; i < TPI; ++i) {
        const float x = fmaxf(z[i][n][c], z[i][n][2 + c]);
        top[n][c] = i ? fmaxf(top[n][c], x) : x;
        over |= (x - w.m[n][c]) + lv[i] > w.e[n][c] + kLazy;
      }
      over |= top[n][c] > w.m[n][c] + kLazy;
    }
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      float r[2];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float nm = fmaxf(w.m[n][c], top[n][c]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, off));
        const float e = w.e[n][c] + (w.m[n][c] - nm);      // (the same reference, from the new m)
        float ne = e;
#pragma unroll
        for (int i = 0; i < TPI; ++i)
          ne = fmaxf(ne, (fmaxf(z[i][n][c], z[i][n][2 + c]) - nm) + lv[i]);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          ne = fmaxf(ne, __shfl_xor_sync(0xffffffffu, ne, off));
        w.l[n][c] *= ptx::ex2(w.m[n][c] - nm);
        r[c] = ptx::ex2(e - ne);
        w.m[n][c] = nm;
        w.e[n][c] = ne;
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        w.acc[n][j][0] *= r[0];
        w.acc[n][j][1] *= r[1];
        w.acc[n][j][2] *= r[0];
        w.acc[n][j][3] *= r[1];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < TPI; ++i) {
    uint32_t hi[NC][2], lw[NC][2];      // W^T fragments, hi and lo parts
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      float wt[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float d = z[i][n][k] - w.m[n][k & 1];
        w.l[n][k & 1] += ptx::ex2(d);
        wt[k] = ptx::ex2(d + (lv[i] + kWeightShift - w.e[n][k & 1]));
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t h = ptx::pack_f16x2(wt[2 * r], wt[2 * r + 1]);
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
        const uint32_t o = ptx::pack_f16x2(wt[2 * r] - x.x, wt[2 * r + 1] - x.y);
        if constexpr (V == kPair) {
          hi[n][r] = ptx::movmatrix_trans(t < 2 ? h : o);
        } else {
          hi[n][r] = ptx::movmatrix_trans(h);
          lw[n][r] = ptx::movmatrix_trans(o);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < (D == 256 ? 2 : 1); ++h) {
      constexpr int N = D == 64 ? 1 : 2;              // words
      uint32_t a[4][2], b[4][2];
      v_words<D>(stage + i * S::TILE, ln, h, a, b);
#pragma unroll
      for (int x = 0; x < N; ++x) {
        uint32_t pa[2][2], pb[2][2];      // [k half][first / second pair word]
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          pair_words<F8>(a[2 * kh][x], a[2 * kh + 1][x], pa[kh][0], pa[kh][1]);
          pair_words<F8>(b[2 * kh][x], b[2 * kh + 1][x], pb[kh][0], pb[kh][1]);
        }
        // E rows' fragments at a time: as many as the registers hold beside the sums
        constexpr int E = V == kSixteen || (D == 256 && V == kEight) ? 2 : 4;
#pragma unroll
        for (int e0 = 0; e0 < 4; e0 += E) {
          uint32_t fr[E][4];
#pragma unroll
          for (int e = 0; e < E; ++e)
#pragma unroll
            for (int kh = 0; kh < 2; ++kh) {
              const uint32_t wa = pa[kh][(e0 + e) >> 1], wb = pb[kh][(e0 + e) >> 1];
              fr[e][2 * kh] = e & 1 ? codes_behind_to_h2<F8>(wa) : codes_to_h2<F8>(wa);
              fr[e][2 * kh + 1] = e & 1 ? codes_behind_to_h2<F8>(wb) : codes_to_h2<F8>(wb);
            }
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            // The products' own sum drops the bits below its last place instead of rounding:
            // over a long chain that is a drift (512 tiles: 2e-5 of the result).  So a tile's
            // products start from zero and are added, rounded, to the lane's sums.
            float part[E][4];
#pragma unroll
            for (int e = 0; e < E; ++e) mma_from_zero(part[e], fr[e], hi[n][0], hi[n][1]);
            if constexpr (V != kPair)
#pragma unroll
              for (int e = 0; e < E; ++e) ptx::mma_f16(part[e], fr[e], lw[n][0], lw[n][1]);
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
              for (int k = 0; k < 4; ++k) w.acc[n][(h * N + x) * 4 + e0 + e][k] += part[e][k];
          }
        }
      }
    }
  }
}

// d index of row (g + 8 r) of O^T tile j.
template <int D>
__device__ __forceinline__ int out_dim(int j, int r, int g) {
  if constexpr (D == 64) return 8 * g + 4 * r + j;
  return (j >> 3) * 128 + 16 * g + 8 * r + (j & 7);
}

// The lane's pieces of the queries of a unit's columns, 16 values of every 64: requested
// before the unit's copies, which would delay them ...
template <int D, int V>
__device__ __forceinline__ void load_queries(Warp<D, V>& w, const BlockDecodeArgs& a,
                                             const Segment& s, int g, int t) {
  const int kvh = s.u / a.n_cg, cg = s.u % a.n_cg, cols = min(a.width, a.G * a.Q - cg * a.width);
#pragma unroll
  for (int n = 0; n < Cols<V>::NC; ++n) {
    const int mine = V == kPair ? g & 3 : 8 * n + g;
    const int col = cg * a.width + min(mine, cols - 1);
    const uint16_t* q =
        a.q + (((size_t)s.b * a.Q + col / a.G) * a.H + kvh * a.G + col % a.G) * D + 16 * t;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const uint4 x = ptx::ldg128(q + 64 * (c >> 1) + 8 * (c & 1));
      w.q[n][4 * c] = x.x;
      w.q[n][4 * c + 1] = x.y;
      w.q[n][4 * c + 2] = x.z;
      w.q[n][4 * c + 3] = x.w;
    }
  }
}

// ... and as fragments: columns that are none get zeros, int8 the order of codes_to_h2.
template <int D, bool F8, int V>
__device__ __forceinline__ void order_queries(Warp<D, V>& w, int cols, int g) {
#pragma unroll
  for (int n = 0; n < Cols<V>::NC; ++n) {
    const bool none = (V == kPair ? g & 3 : 8 * n + g) >= cols;
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {     // four values each
      const uint32_t x = none ? 0 : w.q[n][2 * k], y = none ? 0 : w.q[n][2 * k + 1];
      w.q[n][2 * k] = F8 ? x : ptx::prmt(x, y, 0x5410);
      w.q[n][2 * k + 1] = F8 ? y : ptx::prmt(x, y, 0x7632);
    }
  }
}

// The fragments of a unit's queries in shared memory (kSharedQ), a block's threads
// together: lane's two words of group n and 16 values ks at ((n * D / 16 + ks) * 32 + lane) * 8.
template <int D, bool F8, int V>
__device__ __forceinline__ void share_queries(unsigned char* shared, const BlockDecodeArgs& a,
                                              const Segment& s) {
  const int kvh = s.u / a.n_cg, cg = s.u % a.n_cg, cols = min(a.width, a.G * a.Q - cg * a.width);
  for (int i = threadIdx.x; i < Cols<V>::NC * (D / 16) * 32; i += Shape<D>::NW * 32) {
    const int lane = i & 31, ks = i / 32 % (D / 16), n = i / 32 / (D / 16);
    const int mine = 8 * n + (lane >> 2), t = lane & 3;
    uint2 x = make_uint2(0, 0);
    if (mine < cols) {
      const int col = cg * a.width + mine;
      const uint16_t* q = a.q + (((size_t)s.b * a.Q + col / a.G) * a.H + kvh * a.G + col % a.G) * D;
      const uint2 v = *reinterpret_cast<const uint2*>(q + 64 * (ks / 4) + 16 * t + 4 * (ks % 4));
      x = F8 ? v : make_uint2(ptx::prmt(v.x, v.y, 0x5410), ptx::prmt(v.x, v.y, 0x7632));
    }
    *reinterpret_cast<uint2*>(shared + i * 8) = x;
  }
}

// Joining the warps: where a warp's output (column, d) lies in its region of D * N floats.
// The xor spreads the four columns and the pieces of 16 that a warp writes at once.
template <int D>
__device__ __forceinline__ int joined(int col, int d) {
  return col * D + (d ^ ((col >> 1 & 3) << 2));
}

template <int D, bool F8, int V>
__global__ void __launch_bounds__(Shape<D>::NW * 32, Shape<D>::BLOCKS)
    decode_block_kernel(const BlockDecodeArgs a) {
  using S = Shape<D>;
  constexpr int NC = Cols<V>::NC, N = Cols<V>::N, TPI = S::TPI;
  constexpr bool EARLY = N * D * 4 <= S::STAGE;
  static_assert(N * D * 4 <= S::NS * S::STAGE, "a warp's output fits its ring");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float stat[3][S::NW][N];     // m, e, l of each warp and column
  __shared__ float2 block_ml[N];          // of a cluster's block, whose outputs are in warp 0's stage 1
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = ptx::smem_u32(smem) + warp * S::NS * S::STAGE;
  const Lane<D> ln(lane);
  const BlockView& p = a.pool;
  const int per_seq = p.Hkv * a.n_cg;      // units of a sequence
  ptx::grid_launch_dependents();
  if (!a.appended) ptx::grid_dependency_wait();

  Place place;
  Segment seg;
  if (a.shares == 0) {
    const int unit = blockIdx.x / a.cluster;
    seg.b = unit / per_seq;
    seg.u = unit % per_seq;
    unit_range(a, seg.b, seg.lo, seg.hi);
    seg.nt = unit_tiles(seg.lo, seg.hi);               // (none: zero rows)
    const int per = (seg.nt + a.cluster - 1) / a.cluster;
    seg.first = min(seg.nt, blockIdx.x % a.cluster * per);
    seg.last = min(seg.nt, seg.first + per);
    seg.pieces = 1;
    place.at = place.end = 0;
  } else {
    place = find_share(a, per_seq, S::START, S::LEAST);
    if (!next_segment(a, place, per_seq, S::START, seg)) {
      ptx::grid_dependency_wait();    // (the grid is not complete before the append is)
      return;
    }
  }

  // The warp's stages of a segment: TPI tiles each, from first + TPI * (warp + NW * i).
  constexpr int BATCH = 32 / TPI;       // stages whose pages and scales the lanes hold
  int pages = -1;                       // lane TPI * i + j: tile j of stage (issue index & ~(BATCH - 1)) + i
  float ks = 0.f, vs = 0.f;
  int slot_in = 0, slot_out = 0;        // stages' bytes in the ring
  int mine0, n, fresh;        // fresh: positions from here on are waited for
  auto issue = [&](int i) {
    const int kvh = seg.u / a.n_cg;
    const int tile = mine0 + ((i & ~(BATCH - 1)) + lane / TPI) * (S::NW * TPI) + lane % TPI;
    const int at = (seg.lo / kTile + tile) * kTile;
    auto block_of = [&](int page) {
      return (((size_t)page * p.Hkv + kvh) << (p.ps_log2 - p.t_log2)) +
             ((at & ((1 << p.ps_log2) - 1)) >> p.t_log2);
    };
    if ((i & (BATCH - 1)) == 0) {
      pages = tile < seg.last ? block_page(a.page_table + (size_t)seg.b * a.max_pages,
                                           at >> p.ps_log2, p)
                              : -1;
      if (pages >= 0 && at < fresh) {
        ks = __ldg(p.ks + block_of(pages));
        vs = __ldg(p.vs + block_of(pages));
      }
    }
    bool late = false;
    if (i < n) {
      late = (seg.lo / kTile + mine0 + i * (S::NW * TPI) + TPI) * kTile > fresh;
      if (late) {
        ptx::grid_dependency_wait();
        if (pages >= 0 && at >= fresh) {      // (written while this kernel may run: not through L1)
          ks = __ldcg(p.ks + block_of(pages));
          vs = __ldcg(p.vs + block_of(pages));
        }
      }
#pragma unroll
      for (int j = 0; j < TPI; ++j) {
        const int page = __shfl_sync(0xffffffffu, pages, (i & (BATCH - 1)) * TPI + j);
        const int pos = (seg.lo / kTile + mine0 + i * (S::NW * TPI) + j) * kTile;
        const size_t row = ((((size_t)(page < 0 ? 0 : page) * p.Hkv + kvh) << p.ps_log2) +
                            (pos & ((1 << p.ps_log2) - 1))) * D + 16 * lane;
        const uint32_t to = ring + slot_in + j * S::TILE;
        if (page >= 0 && pos >= seg.lo && pos + kTile <= seg.hi)
          copy_tile<D, true>(p.k + row, p.v + row, to, ln, 0, kTile, lane);
        else      // rows behind the context, or of no page, become zeros
          copy_tile<D, false>(p.k + row, p.v + row, to, ln, page < 0 ? kTile : seg.lo - pos,
                              seg.hi - pos, lane);
      }
    }
    commit_copies();
    slot_in = slot_in == (S::NS - 1) * S::STAGE ? 0 : slot_in + S::STAGE;
    return late;
  };
  auto begin = [&]() {       // the first copies of a segment
    mine0 = seg.first + warp * TPI;
    fresh = a.appended ? (seg.hi - 1) >> p.t_log2 << p.t_log2 : INT_MAX;
    n = seg.last > mine0 ? (seg.last - mine0 + S::NW * TPI - 1) / (S::NW * TPI) : 0;
#pragma unroll
    for (int i = 0; i < S::NS - 1; ++i) issue(i);
  };

  Warp<D, V> w;
  const uint32_t shared_q = ptx::smem_u32(smem) + S::RING + 8 * lane;
  if constexpr (!kSharedQ<D, V>) load_queries(w, a, seg, g, t);
  begin();
  if constexpr (kSharedQ<D, V>) {
    share_queries<D, F8, V>(smem + S::RING, a, seg);
    __syncthreads();
  }
  for (;;) {
    const int kvh = seg.u / a.n_cg, cg = seg.u % a.n_cg;
    const int cols = min(a.width, a.G * a.Q - cg * a.width);
    if constexpr (!kSharedQ<D, V>) order_queries<D, F8, V>(w, cols, g);
    w.reset();
    int lim[NC][2];           // columns 2t, 2t + 1 of the fragments
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = V == kPair ? (2 * t + c) & 3 : 8 * k + 2 * t + c;
        lim[k][c] = col < cols ? seg.hi - a.Q + (cg * a.width + col) / a.G : -1;
      }
    const int least = seg.hi - a.Q + (cg * a.width) / a.G;   // positions <= least: no column masks
    int pages_now = -1;       // pages and scales of the stage being taken
    float fs_now = 0.f, ls_now = 0.f;
    for (int i = 0; i < n; ++i) {
      if ((i & (BATCH - 1)) == 0) {
        pages_now = pages;
        fs_now = pages < 0 ? 0.f : ks * a.scale_log2;
        ls_now = pages < 0 ? 0.f : log2f(vs);
      }
      wait_copies<S::NS - 2>();
      __syncwarp();     // stage i is there for all lanes, and none still reads the one before
      if (issue(i + S::NS - 1) && ((i + S::NS - 1) & (BATCH - 1)) >= S::NS - 1) {
        fs_now = pages < 0 ? 0.f : ks * a.scale_log2;     // scales that came late, of the same batch
        ls_now = pages < 0 ? 0.f : log2f(vs);
      }
      float f[TPI], lv[TPI];
      const uint32_t none =
          __ballot_sync(0xffffffffu, pages_now < 0) >> ((i & (BATCH - 1)) * TPI) & ((1u << TPI) - 1);
#pragma unroll
      for (int j = 0; j < TPI; ++j) {
        f[j] = __shfl_sync(0xffffffffu, fs_now, (i & (BATCH - 1)) * TPI + j);
        lv[j] = __shfl_sync(0xffffffffu, ls_now, (i & (BATCH - 1)) * TPI + j);
      }
      const int pos = (seg.lo / kTile + mine0 + i * (S::NW * TPI)) * kTile;
      const bool masked = none || pos < seg.lo || pos + TPI * kTile - 1 > least;
      take_stage<D, F8, V>(w, ring + slot_out, pos, f, lv, masked, none, seg.lo, lim, ln, shared_q, g, t);
      slot_out = slot_out == (S::NS - 1) * S::STAGE ? 0 : slot_out + S::STAGE;
    }
    __syncwarp();

    // the next segment's first copies, into stages 1 and on: stage 0 joins the warps (where it
    // holds their outputs; else the copies wait)
    const Segment done = seg;
    const bool more = next_segment(a, place, per_seq, S::START, seg);
    slot_in = slot_out = S::STAGE;
    if (more) {
      if constexpr (!kSharedQ<D, V>) load_queries(w, a, seg, g, t);
      if constexpr (EARLY) begin();
    }

    const int live = min(S::NW, (done.last - done.first + TPI - 1) / TPI);     // warps that had tiles
    float* mine = reinterpret_cast<float*>(smem + warp * S::NS * S::STAGE);
#pragma unroll
    for (int k = 0; k < NC; ++k)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col = 8 * k + 2 * t + c;
        if (warp < live)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int j = 0; j < D / 16; j += 4)
              *reinterpret_cast<float4*>(mine + joined<D>(col, out_dim<D>(j, r, g))) =
                  make_float4(w.acc[k][j][2 * r + c], w.acc[k][j + 1][2 * r + c],
                              w.acc[k][j + 2][2 * r + c], w.acc[k][j + 3][2 * r + c]);
        float l = w.l[k][c];
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        if (g == 0) {
          stat[0][warp][col] = w.m[k][c];
          stat[1][warp][col] = w.e[k][c];
          stat[2][warp][col] = l;
        }
      }
    __syncthreads();
    if constexpr (kSharedQ<D, V>)      // (no warp needs the last ones any more)
      if (more) share_queries<D, F8, V>(smem + S::RING, a, seg);
    const bool joins = V != kSixteen && a.cluster > 1;     // with the cluster's other blocks
    const bool whole = !joins && done.first == 0 && done.last == done.nt;
    const int unit = done.b * per_seq + done.u, slot = unit + blockIdx.x;
    if (a.shares && done.first == 0 && threadIdx.x == 0)     // for the combine
      a.part_units[unit] = make_int2(slot, done.pieces);
    for (int col = warp; col < cols; col += S::NW) {
      float m = kUnset, e = -INFINITY, l = 0.f, r[S::NW];
#pragma unroll
      for (int k = 0; k < S::NW; ++k)
        if (k < live) m = fmaxf(m, stat[0][k][col]);
#pragma unroll
      for (int k = 0; k < S::NW; ++k) {
        r[k] = -INFINITY;
        if (k < live) {
          const float d = stat[0][k][col] - m;
          l += stat[2][k][col] * ptx::ex2(d);
          r[k] = stat[1][k][col] + d;
          e = fmaxf(e, r[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < S::NW; ++k) r[k] = k < live ? ptx::ex2(r[k] - e) : 0.f;
      const float inv = l > 0.f ? __fdividef(ptx::ex2(e - kWeightShift), l) : 0.f;
      const int gc = cg * a.width + col;
      float* out = a.out + (((size_t)done.b * a.Q + gc / a.G) * a.H + kvh * a.G + gc % a.G) * D;
      if (joins) out = reinterpret_cast<float*>(smem + S::STAGE) + col * D;
      else if (!whole) out = a.part_o + ((size_t)slot * a.width + col) * D;
#pragma unroll
      for (int d = 4 * lane; d < D; d += 128) {
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < S::NW; ++k)
          if (k < live) {
            const float* from = reinterpret_cast<const float*>(smem + k * S::NS * S::STAGE);
            float4 x = *reinterpret_cast<const float4*>(from + joined<D>(col, d));
            if constexpr (V == kPair) {      // hi and lo parts
              const float4 y = *reinterpret_cast<const float4*>(from + joined<D>(col + 4, d));
              x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            }
            o = make_float4(fmaf(r[k], x.x, o.x), fmaf(r[k], x.y, o.y), fmaf(r[k], x.z, o.z),
                            fmaf(r[k], x.w, o.w));
          }
        *reinterpret_cast<float4*>(out + d) =
            make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
      }
      if (!whole && lane == 0) {
        const float2 ml = make_float2(l > 0.f ? m : -INFINITY, l);
        if (joins) block_ml[col] = ml;
        else a.part_ml[(size_t)slot * a.width + col] = ml;
      }
    }
    if constexpr (V != kSixteen) {
      if (joins) {        // (the last segment: no copies are under way)
        static_assert(EARLY && N * D * 4 <= (S::NS - 1) * S::STAGE, "outputs behind stage 0");
        const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
        cluster.sync();
        float* part = reinterpret_cast<float*>(smem + S::STAGE);
        for (int i = blockIdx.x % kBlockCluster * S::NW * 32 + threadIdx.x; i < cols * (D / 4);
             i += kBlockCluster * S::NW * 32) {
          const int col = i / (D / 4), d = i % (D / 4) * 4;
          float2 ml[kBlockCluster];
          float m = kUnset, l = 0.f;
          float4 x[kBlockCluster], o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int r = 0; r < kBlockCluster; ++r) {
            ml[r] = *cluster.map_shared_rank(block_ml + col, r);
            x[r] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(part + col * D + d, r));
            m = fmaxf(m, ml[r].x);
          }
#pragma unroll
          for (int r = 0; r < kBlockCluster; ++r) {
            const float wt = ml[r].y * ptx::ex2(ml[r].x - m);
            l += wt;
            o = make_float4(fmaf(wt, x[r].x, o.x), fmaf(wt, x[r].y, o.y), fmaf(wt, x[r].z, o.z),
                            fmaf(wt, x[r].w, o.w));
          }
          const float inv = l > 0.f ? 1.f / l : 0.f;
          const int gc = cg * a.width + col;
          *reinterpret_cast<float4*>(
              a.out + (((size_t)done.b * a.Q + gc / a.G) * a.H + kvh * a.G + gc % a.G) * D + d) =
              make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        }
        cluster.sync();      // others may still read this block's outputs
      }
    }
    if (!more) break;
    __syncthreads();      // the next segment's copies reach stage 0
    if constexpr (!EARLY) begin();
  }
  ptx::grid_dependency_wait();    // (the grid is not complete before the append is)
}

template <int D, bool F8, int V>
cudaError_t launch_variant(const BlockDecodeArgs& a, cudaStream_t stream) {
  const long long units = (long long)a.B * a.pool.Hkv * a.n_cg;
  const long long grid = a.shares ? a.shares : units * a.cluster;
  if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(Shape<D>::NW * 32);
  cfg.dynamicSmemBytes = kSmem<D, V>;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kBlockCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, decode_block_kernel<D, F8, V>, a);
}

// Blocks per SM of one variant, with its shared-memory attribute set.
template <int D, bool F8, int V>
int variant_blocks() {
  int per_sm = 0;
  if (cudaFuncSetAttribute(decode_block_kernel<D, F8, V>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSmem<D, V>) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, decode_block_kernel<D, F8, V>,
                                                    Shape<D>::NW * 32, kSmem<D, V>) != cudaSuccess)
    return -1;
  return per_sm;
}

// Clusters of one variant that run at once, after variant_blocks.
template <int D, bool F8, int V>
int variant_clusters() {
  int n = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kBlockCluster);
  cfg.blockDim = dim3(Shape<D>::NW * 32);
  cfg.dynamicSmemBytes = kSmem<D, V>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kBlockCluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaOccupancyMaxActiveClusters(&n, decode_block_kernel<D, F8, V>, &cfg) == cudaSuccess ? n : -1;
}

template <int D, bool F8>
cudaError_t launch_codes(const BlockDecodeArgs& a, cudaStream_t stream) {
  if (a.width <= 4) return launch_variant<D, F8, kPair>(a, stream);
  if (a.width <= 8) return launch_variant<D, F8, kEight>(a, stream);
  return launch_variant<D, F8, kSixteen>(a, stream);
}

template <int D, bool F8>
int codes_blocks() {
  return std::min({variant_blocks<D, F8, kPair>(), variant_blocks<D, F8, kEight>(),
                   variant_blocks<D, F8, kSixteen>()});
}

template <int D, bool F8>
int codes_clusters() {
  return std::min(variant_clusters<D, F8, kPair>(), variant_clusters<D, F8, kEight>());
}

}  // namespace block

// One head_dim's kernels, each in a translation unit of its own.
#define INT8KV_DECODE_BLOCK_INSTANCE(D)                                                          \
  cudaError_t launch_block_decode_##D(const BlockDecodeArgs& a, bool f8, cudaStream_t stream) {  \
    return f8 ? block::launch_codes<D, true>(a, stream) : block::launch_codes<D, false>(a, stream); \
  }                                                                                              \
  int block_decode_blocks_##D(bool f8) {                                                         \
    return f8 ? block::codes_blocks<D, true>() : block::codes_blocks<D, false>();                \
  }                                                                                              \
  int block_decode_clusters_##D(bool f8) {                                                       \
    return f8 ? block::codes_clusters<D, true>() : block::codes_clusters<D, false>();            \
  }

cudaError_t launch_block_decode_64(const BlockDecodeArgs& a, bool f8, cudaStream_t stream);
cudaError_t launch_block_decode_128(const BlockDecodeArgs& a, bool f8, cudaStream_t stream);
cudaError_t launch_block_decode_256(const BlockDecodeArgs& a, bool f8, cudaStream_t stream);
int block_decode_blocks_64(bool f8);
int block_decode_blocks_128(bool f8);
int block_decode_blocks_256(bool f8);
int block_decode_clusters_64(bool f8);
int block_decode_clusters_128(bool f8);
int block_decode_clusters_256(bool f8);

}  // namespace int8kv
