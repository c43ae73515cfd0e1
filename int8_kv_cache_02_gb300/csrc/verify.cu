// kv_verify_drafts: how many drafted tokens of each sequence the target's probabilities accept, and
// the token behind them, from given random numbers.
//
//   draft i is taken while u_i q_i(x_i) < p_i(x_i); with r the first that is not,
//   weight w(v) = max(p_r(v) - q_r(v), 0), or p_n(v) where all n are taken;
//   the token is the lowest v with sum_{w <= v} w > u sum w.
//
// Products of two fp32 numbers are exact in fp64.  Probabilities become whole multiples of
// 2^-60 (exactly, from 2^-37 on), so sums and differences are exact in 64-bit integers: the
// token depends neither on how a row is cut nor on the order of the additions.
//
// Such a multiple is made of three numbers of 20 bits: p + 1.5 * 2^3, in fp32, has p's multiple of
// 2^-20 as its lowest bits, and what that leaves of p is exact; so twice more.  The bits are added as
// they are, in 32-bit integers, and joined after eight values.  Two values at a time go through the
// same additions (for max(p - q, 0) the two of a place, whose constants cancel): 13 operations for
// two rows, where shifting mantissas into place took 26, of the slower kind (64 sequences of
// 131072 tokens 23.0 us with that, 22.1 with this).
//
// One cluster of kCluster blocks per sequence.  Each finds r by itself (three short dependent
// loads), sums its slice of the row (or of the two), a run of consecutive values for each
// warp, and writes its sum to the others' shared memory.  The warp whose run holds the place looks it
// up there: 32 equal parts of the run, then 32 of the part, their values from L2.  So a row is
// read once and nothing is written but the results.
//
// 64 sequences of 131072 tokens, 63 MB: 19.7 us (47 % of the copy rate); one of 32000: 5.1 us.  What
// stands beside the stream is a sequence's own chain: the launch, three dependent loads, eight
// batches of a block's slice one after another, the cluster's barriers and two look-ups.  One
// sequence of 131072 takes 9.8 us with two rows (7.8 with one), 19 (a block an SM) 11.8, 38 14.4, 76
// 20.7, 128 33.5: all blocks of a wave are at the same point of the chain, so that none hides
// another's.  Whether sequences read one row or two is not what costs: all drafts refused takes
// 19.9, all taken 12.3.  Clusters of 16 blocks of 128 threads: 19.6 and 4.9, and a size that not
// every device grants; of 4 blocks of 512: 29.0 (without loads ahead, 8 x 256 took 23.2).
#include <utility>

#include <cooperative_groups.h>

#include "common.cuh"
#include "packed.cuh"
#include "ptx.cuh"

namespace int8kv {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct VerifyArgs {
  const float* target;          // rows target_stride apart, n_draft + 1 for each sequence
  const float* draft;           // rows draft_stride apart, n_draft for each sequence; or null
  long long target_stride, draft_stride;
  const int32_t* x;             // [batch][n_draft]
  const int32_t* n_drafts;      // [batch], or null
  const float* u;               // [batch][n_draft]
  const float* sample_u;        // [batch]
  int32_t* tokens;              // [batch][n_draft + 1]
  int32_t* n_accepted;          // [batch]
  const int32_t* seq_lens;      // [batch], or null
  int32_t* seq_lens_out;
  int n_draft, vocab;
};

using u64 = unsigned long long;

__device__ __forceinline__ uint64_t minus2(uint64_t a, uint64_t b) {      // a - b
  return fma2(b, pack2(-1.f, -1.f), a);
}

// Sums of values in units of 2^-20, 2^-40 and 2^-60, in 32 bits, wrapping.
__device__ constexpr float top_of(int k) { return k == 0 ? 0x1.8p3f : k == 1 ? 0x1.8p-17f : 0x1.8p-37f; }
struct Limbs {
  uint32_t n[3] = {0, 0, 0};
  // TWO: p - q where that is positive; else p + q.  Both in [0, 1].
  template <bool TWO>
  __device__ __forceinline__ void add(float p, float q) {
    uint64_t x = pack2(p, q);
    const bool counts = !TWO || p > q;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint64_t m = pack2(top_of(k), top_of(k)), t = add2(x, m);
      if (counts) n[k] += TWO ? (uint32_t)t - (uint32_t)(t >> 32) : (uint32_t)t + (uint32_t)(t >> 32);
      if (k < 2) x = add2(x, minus2(m, t));
    }
  }
  // the sum, of `values` values that were added (not of differences: 0)
  __device__ __forceinline__ u64 sum(uint32_t values) const {
    u64 w = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      w += (u64)(long long)(int)(n[k] - values * __float_as_uint(top_of(k))) << (40 - 20 * k);
    return w;
  }
};

// A probability in units of 2^-60, to the nearest; outside [0, 1] the nearest of the two, NaN 0.
__device__ __forceinline__ u64 fixed60(float p) {
  Limbs l;
  l.add<false>(__saturatef(p), 0.f);
  return l.sum(2);
}

// The weights of a row: what the draft's probabilities leave of the target's.
struct Row {
  const float *p, *q;      // q null: p alone
  int without;             // this value's weight is 0 (a draft without probabilities); or -1
};
__device__ __forceinline__ u64 warp_sum64(u64 x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// Values of a row, or of two, that a lane takes at a time.
template <bool TWO, int VEC, int K>
struct Batch {
  float p[K][VEC], q[K][VEC];
  __device__ __forceinline__ void load(const Row& r, int v0, int step, int z) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = v0 + step * k;
#pragma unroll
      for (int e = 0; e < VEC; ++e) p[k][e] = q[k][e] = 0.f;
      if (v < z) {      // (VEC 4: z and the rows are multiples of 4)
        if constexpr (VEC == 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(r.p + v));
          p[k][0] = x.x, p[k][1] = x.y, p[k][2] = x.z, p[k][3] = x.w;
          if constexpr (TWO) {
            const float4 y = __ldg(reinterpret_cast<const float4*>(r.q + v));
            q[k][0] = y.x, q[k][1] = y.y, q[k][2] = y.z, q[k][3] = y.w;
          }
        } else {
          p[k][0] = __ldg(r.p + v);
          if constexpr (TWO) q[k][0] = __ldg(r.q + v);
        }
      }
    }
  }
  __device__ __forceinline__ u64 sum() const {
    Limbs l;
    if constexpr (TWO) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) l.add<true>(__saturatef(p[k][e]), __saturatef(q[k][e]));
    } else {
#pragma unroll
      for (int n = 0; n < K * VEC; n += 2)
        l.add<false>(__saturatef(p[n / VEC][n % VEC]), __saturatef(p[(n + 1) / VEC][(n + 1) % VEC]));
    }
    return l.sum(TWO ? 0 : K * VEC);
  }
};

// The sum of the weights of values [a, z) that fall to a lane of `lanes`, each taking VEC together; the
// next ones are under way while it adds (64 sequences of 131072 tokens 22.1 -> 19.7 us).
template <bool TWO, int VEC>
__device__ __forceinline__ u64 sum_lane(const Row& r, int a, int z, int lane, int lanes) {
  constexpr int K = VEC == 4 ? 2 : 4;
  const int step = lanes * VEC;
  u64 sum = 0;
  Batch<TWO, VEC, K> now, next;
  int v0 = a + lane * VEC;
  now.load(r, v0, step, z);
  while (v0 < z) {
    v0 += step * K;
    next.load(r, v0, step, z);
    sum += now.sum();
    now = next;
  }
  return sum;
}

// The weight that the sum of [a, z) has too much: that of `without`, if it is among them.
__device__ __forceinline__ u64 left_out(const Row& r, int a, int z) {
  return r.without >= a && r.without < z ? fixed60(__ldg(r.p + r.without)) : 0;
}

// The place-th unit of the weights of [a, z) (fewer than they sum to) is this value's; a warp together.
template <bool TWO, int VEC>
__device__ __forceinline__ int look_up(const Row& r, int a, int z, u64 place, int lane) {
  for (;;) {
    const bool last = z - a <= 32;      // (else a part is a multiple of VEC)
    const int per = last ? 1 : ((z - a + 31) / 32 + VEC - 1) / VEC * VEC;
    const int from = min(z, a + lane * per), to = min(z, from + per);
    u64 inc = (last ? sum_lane<TWO, 1>(r, from, to, 0, 1) : sum_lane<TWO, VEC>(r, from, to, 0, 1)) -
              left_out(r, from, to);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const u64 o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    // (a row that sums to 16 and more wraps, and may have no such place: some value then)
    const int at = (__ffs(__ballot_sync(0xffffffffu, inc > place)) - 1) & 31;
    const u64 before = __shfl_sync(0xffffffffu, inc, at ? at - 1 : 0);
    if (at > 0) place -= before;
    a = a + at * per;
    z = min(z, a + per);
    if (last) return a;
  }
}

// VEC: rows are read 16 bytes at a time, where every row begins at such a boundary (64 sequences of
// 131072 values: 19.8 us; of 131071, 4 bytes at a time: 25.8).
template <int VEC>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    verify_kernel(const VerifyArgs a) {
  namespace cg = cooperative_groups;
  __shared__ u64 runs[kWarps], totals[2][kCluster];
  const cg::cluster_group cluster = cg::this_cluster();
  auto started = cluster.barrier_arrive();      // (all blocks run before one writes to another)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = blockIdx.x % kCluster;
  const size_t b = blockIdx.x / kCluster;
  ptx::grid_dependency_wait();
  ptx::grid_launch_dependents();

  // drafts that are taken: every warp by itself
  const int given = a.n_drafts ? __ldg(a.n_drafts + b) : a.n_draft;
  const int count = min(given, a.n_draft);
  int taken = max(count, 0);
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int i = i0 + lane;
    bool refused = false;
    if (i < count) {
      const int x = __ldg(a.x + b * a.n_draft + i);
      const float u = __ldg(a.u + b * a.n_draft + i);
      refused = true;
      if (x >= 0 && x < a.vocab) {
        const float p = __saturatef(__ldg(a.target + (b * (a.n_draft + 1) + i) * a.target_stride + x));
        const float q =      // (both as the weights take them: NaN is 0)
            a.draft ? __saturatef(__ldg(a.draft + (b * a.n_draft + i) * a.draft_stride + x)) : 1.f;
        refused = !((double)u * (double)q < (double)p);
      }
    }
    const unsigned any = __ballot_sync(0xffffffffu, refused);
    if (any) {
      taken = i0 + __ffs(any) - 1;
      break;
    }
  }
  if (rank == 0) {
    for (int i = threadIdx.x; i <= a.n_draft; i += kThreads)
      // (the place behind the drafts too: -1, where no weight is found below)
      a.tokens[b * (a.n_draft + 1) + i] = i < taken ? __ldg(a.x + b * a.n_draft + i) : -1;
    if (threadIdx.x == 0) {
      a.n_accepted[b] = taken;
      if (a.seq_lens_out) a.seq_lens_out[b] = a.seq_lens[b] - (max(count, 0) - taken);
    }
  }
  const float sample = __ldg(a.sample_u + b);
  const bool refused = taken < count;
  Row row;
  row.p = a.target + (b * (a.n_draft + 1) + taken) * a.target_stride;
  row.q = refused && a.draft ? a.draft + (b * a.n_draft + taken) * a.draft_stride : nullptr;
  row.without = refused && !a.draft ? __ldg(a.x + b * a.n_draft + taken) : -1;
  // runs of consecutive values: warp `rank * kWarps + warp` has [from, to)
  const int per = (int)(((long long)a.vocab + kCluster * kWarps - 1) / (kCluster * kWarps) + 31) & ~31;
  const int from = given < 0 ? 0 : (int)min((long long)a.vocab, (long long)(rank * kWarps + warp) * per);
  const int to = given < 0 ? 0 : min(a.vocab, from + per);
  u64 total = 0, before = 0, mine = 0;
  cluster.barrier_wait(std::move(started));
  for (int round = 0; round < 2; ++round) {
    mine = warp_sum64(row.q ? sum_lane<true, VEC>(row, from, to, lane, 32)
                            : sum_lane<false, VEC>(row, from, to, lane, 32)) -
           left_out(row, from, to);
    if (lane == 0) runs[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      const u64 t = warp_sum64(lane < kWarps ? runs[lane] : 0);
      if (lane < kCluster) *cluster.map_shared_rank(&totals[round][rank], lane) = t;
    }
    cluster.sync();
    total = before = 0;
#pragma unroll
    for (int k = 0; k < kCluster; ++k) {
      const u64 t = totals[round][k];
      before += k < rank ? t : 0;
      total += t;
    }
    if (total || !(row.q || row.without >= 0)) break;
    row.q = nullptr;      // nothing is left of the target's: its own probabilities
    row.without = -1;
  }
  if (total == 0) return;
  // u in units of 2^-64; the place is the first whose sum is above u * total
  const u64 u = fixed60(fminf(fmaxf(sample, 0.f), 0x1.fffffep-1f)) << 4;
  const u64 place = __umul64hi(u, total);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) before += w < warp ? runs[w] : 0;
  if (place < before || place - before >= mine) return;
  const int token = row.q ? look_up<true, VEC>(row, from, to, place - before, lane)
                          : look_up<false, VEC>(row, from, to, place - before, lane);
  if (lane == 0) a.tokens[b * (a.n_draft + 1) + taken] = token;
}

}  // namespace
}  // namespace int8kv

using namespace int8kv;

extern "C" int kv_verify_drafts(int batch, int n_draft, int vocab, const float* target_probs,
                                long long target_stride, const float* draft_probs,
                                long long draft_stride, const int32_t* draft_tokens,
                                const int32_t* n_drafts, const float* accept_u,
                                const float* sample_u, int32_t* tokens, int32_t* n_accepted,
                                const int32_t* seq_lens, int32_t* seq_lens_out, void* stream) {
  // (the kernel counts drafts and values in 32 bits, by steps of a block's threads)
  if (batch < 0 || n_draft < 0 || n_draft > (1 << 30) || vocab <= 0 || vocab > (1 << 30) ||
      target_stride < vocab || (draft_probs && draft_stride < vocab))
    return INT8KV_ERR_INVALID_ARG;
  if (batch == 0) return INT8KV_OK;
  if (!target_probs || !sample_u || !tokens || !n_accepted || !seq_lens != !seq_lens_out ||
      (n_draft > 0 && (!draft_tokens || !accept_u)))
    return INT8KV_ERR_NULL_PTR;
  if ((long long)batch * kCluster > 0x7fffffffLL) return INT8KV_ERR_UNSUPPORTED;
  VerifyArgs a;
  a.target = target_probs;
  a.draft = draft_probs;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.x = draft_tokens;
  a.n_drafts = n_drafts;
  a.u = accept_u;
  a.sample_u = sample_u;
  a.tokens = tokens;
  a.n_accepted = n_accepted;
  a.seq_lens = seq_lens;
  a.seq_lens_out = seq_lens_out;
  a.n_draft = n_draft;
  a.vocab = vocab;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(batch * kCluster);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto fits = [&](const float* p, long long stride) {
    return ((uintptr_t)p & 15u) == 0 && stride % 4 == 0;
  };
  const bool vec = vocab % 4 == 0 && fits(target_probs, target_stride) &&
                   (!draft_probs || fits(draft_probs, draft_stride));
  const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, verify_kernel<4>, a)
                            : cudaLaunchKernelEx(&cfg, verify_kernel<1>, a);
  return e == cudaSuccess ? INT8KV_OK : INT8KV_ERR_CUDA;
}
