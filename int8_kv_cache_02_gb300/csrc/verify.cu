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
// One cluster of kCluster blocks per sequence.  Each finds r by itself (three short dependent
// loads), sums its slice of the row (or of the two), a run of consecutive values for each
// warp, and reads the others' sums from their shared memory.  The warp whose run holds the place looks
// it up there; its values come from L2 the second time.  So a row is read once and nothing
// is written but the results.
#include <cooperative_groups.h>

#include "common.cuh"
#include "ptx.cuh"

namespace int8kv {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 512;
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

// A probability in units of 2^-60, rounded down; outside [0, 1] the nearest of the two, NaN 0.
__device__ __forceinline__ unsigned long long fixed60(float p) {
  const uint32_t b = __float_as_uint(fminf(fmaxf(p, 0.f), 1.f));
  // 24 bits of mantissa at the top of 61, down by the exponent (a subnormal is below 2^-60)
  const unsigned long long m = (unsigned long long)((b & 0x7fffffu) | 0x800000u) << 37;
  return m >> min(127 - (int)(b >> 23), 63);
}

// The weight of a value: what the draft's probability leaves of the target's.
struct Row {
  const float *p, *q;      // q null: p alone
  int without;             // this value's weight is 0 (a draft without probabilities); or -1
  __device__ __forceinline__ unsigned long long weight(int v, float pv, float qv) const {
    unsigned long long w = fixed60(pv);
    if (q) {
      const unsigned long long o = fixed60(qv);
      w = w > o ? w - o : 0;
    }
    return v == without ? 0 : w;
  }
};

__device__ __forceinline__ unsigned long long warp_sum64(unsigned long long x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// The sum of a lane's weights of values [a, z), a warp's lanes 4 bytes apart, 32 * K at a time.
template <bool TWO>
__device__ __forceinline__ unsigned long long sum_run(const Row& r, int a, int z, int lane) {
  constexpr int K = 8;
  unsigned long long sum = 0;
  for (int v0 = a + lane; v0 < z; v0 += 32 * K) {
    float p[K], q[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = v0 + 32 * k;
      p[k] = v < z ? __ldg(r.p + v) : 0.f;
      q[k] = TWO && v < z ? __ldg(r.q + v) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) sum += r.weight(v0 + 32 * k, p[k], q[k]);
  }
  return sum;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    verify_kernel(const VerifyArgs a) {
  namespace cg = cooperative_groups;
  __shared__ unsigned long long runs[kWarps], total_s;
  const cg::cluster_group cluster = cg::this_cluster();
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
      refused = true;
      if (x >= 0 && x < a.vocab) {
        const float p = __ldg(a.target + (b * (a.n_draft + 1) + i) * a.target_stride + x);
        const float q = a.draft ? __ldg(a.draft + (b * a.n_draft + i) * a.draft_stride + x) : 1.f;
        refused = !((double)__ldg(a.u + b * a.n_draft + i) * (double)q < (double)p);
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
      if (given < 0 || i != taken)
        a.tokens[b * (a.n_draft + 1) + i] = i < taken ? __ldg(a.x + b * a.n_draft + i) : -1;
    if (threadIdx.x == 0) {
      a.n_accepted[b] = taken;
      if (a.seq_lens_out) a.seq_lens_out[b] = a.seq_lens[b] - (max(count, 0) - taken);
    }
  }
  if (given < 0) return;      // (the cluster's blocks all do)

  const bool refused = taken < count;
  Row row;
  row.p = a.target + (b * (a.n_draft + 1) + taken) * a.target_stride;
  row.q = refused && a.draft ? a.draft + (b * a.n_draft + taken) * a.draft_stride : nullptr;
  row.without = refused && !a.draft ? __ldg(a.x + b * a.n_draft + taken) : -1;
  // runs of consecutive values: warp `rank * kWarps + warp` has [from, to)
  const int per = ((a.vocab + kCluster * kWarps - 1) / (kCluster * kWarps) + 31) & ~31;
  const int from = (int)min((long long)a.vocab, (long long)(rank * kWarps + warp) * per);
  const int to = min(a.vocab, from + per);
  unsigned long long total = 0, before = 0, mine = 0;
  for (int round = 0; round < 2; ++round) {
    mine = warp_sum64(row.q ? sum_run<true>(row, from, to, lane) : sum_run<false>(row, from, to, lane));
    if (lane == 0) runs[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long t = 0;
      for (int w = 0; w < kWarps; ++w) t += runs[w];
      total_s = t;
    }
    cluster.sync();
    total = before = 0;
    for (int k = 0; k < kCluster; ++k) {
      const unsigned long long t = *cluster.map_shared_rank(&total_s, k);
      before += k < rank ? t : 0;
      total += t;
    }
    cluster.sync();      // (others' sums have been read)
    if (total || !(row.q || row.without >= 0)) break;
    row.q = nullptr;      // nothing is left of the target's: its own probabilities
    row.without = -1;
  }
  if (total == 0) {
    if (rank == 0 && threadIdx.x == 0) a.tokens[b * (a.n_draft + 1) + taken] = -1;
    return;
  }
  // u in units of 2^-64; the place is the first whose sum is above u * total
  const unsigned long long u64 = fixed60(fminf(fmaxf(__ldg(a.sample_u + b), 0.f), 0x1.fffffep-1f)) << 4;
  const unsigned long long place = __umul64hi(u64, total);
  for (int w = 0; w < warp; ++w) before += runs[w];
  if (place < before || place - before >= mine) return;
  for (int v0 = from; v0 < to; v0 += 32) {
    const int v = v0 + lane;
    unsigned long long inc =
        v < to ? row.weight(v, __ldg(row.p + v), row.q ? __ldg(row.q + v) : 0.f) : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const unsigned long long o = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += o;
    }
    const unsigned above = __ballot_sync(0xffffffffu, before + inc > place);
    if (above) {
      if (lane == 0) a.tokens[b * (a.n_draft + 1) + taken] = v0 + __ffs(above) - 1;
      return;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
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
  if (batch < 0 || n_draft < 0 || vocab <= 0 || vocab > (1 << 30) || target_stride < vocab ||
      (draft_probs && draft_stride < vocab))
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
  return cudaLaunchKernelEx(&cfg, verify_kernel, a) == cudaSuccess ? INT8KV_OK : INT8KV_ERR_CUDA;
}
