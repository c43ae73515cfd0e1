// Block-scaled decode: the dispatch over head_dim, and the combine of partials (shaped scores
// included: an empty unit is one of length 0 there, too).
#include "decode_block.cuh"

namespace int8kv {
namespace {

using namespace block;

// Join the partials of units that a share boundary cut; zero rows of empty units:
//   out = sum_i o_i l_i 2^(m_i - M) / sum_i l_i 2^(m_i - M).
// One block per (sequence, query, head) and 128 values of it; a warp takes every 16th
// partial, a lane four values (D = 64: two).  The decode blocks left each unit's first
// partial and their number.  The first kAhead rows of each warp are requested before
// the weights are known, so that the two trips to L2 overlap.
constexpr int kJoinWarps = 16;
constexpr int kAhead = 6;

template <int PER>
__device__ __forceinline__ void load_row(const float* from, float (&x)[PER]) {
  if constexpr (PER == 4) {
    const float4 v = from ? *reinterpret_cast<const float4*>(from) : make_float4(0.f, 0.f, 0.f, 0.f);
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  } else {
    const float2 v = from ? *reinterpret_cast<const float2*>(from) : make_float2(0.f, 0.f);
    x[0] = v.x;
    x[1] = v.y;
  }
}

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) decode_block_combine_kernel(
    const BlockDecodeArgs a) {
  constexpr int NT = kJoinWarps * 32, DIMS = D < 128 ? D : 128, PER = DIMS / 32;
  extern __shared__ float2 ml[];            // [partials of the unit]
  __shared__ float red[kJoinWarps];
  __shared__ float sums[kJoinWarps][DIMS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_launch_dependents();
  const int row = blockIdx.x, h = row % a.H, bq = row / a.H, b = bq / a.Q;
  const int kvh = h / a.G, gc = (bq % a.Q) * a.G + h % a.G, cg = gc / a.width, col = gc % a.width;
  const int per_seq = a.pool.Hkv * a.n_cg, u = kvh * a.n_cg + cg;
  const int d = blockIdx.y * DIMS + PER * lane;
  float* out = a.out + (size_t)row * D + d;
  ptx::grid_dependency_wait();
  const int2 unit = a.part_units[b * per_seq + u];      // (of no meaning where the unit is empty)
  Seen seen;
  if (unit_range(a, b, seen) == 0) {
    if (warp == 0)
#pragma unroll
      for (int k = 0; k < PER; ++k) out[k] = 0.f;
    return;
  }
  const int n = unit.y;
  if (n == 1) return;      // one block had the whole unit and wrote it
  const size_t first = (size_t)unit.x * a.width + col, stride = (size_t)a.width * D;
  const float* o = a.part_o + first * D + d;
  float x[kAhead][PER];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = warp + k * kJoinWarps;
    load_row<PER>(i < n ? o + i * stride : nullptr, x[k]);
  }
  float M = -INFINITY;
  for (int i = threadIdx.x; i < n; i += NT) {
    const float2 v = a.part_ml[first + (size_t)i * a.width];
    ml[i] = v;
    M = fmaxf(M, v.x);
  }
  M = warp_max(M);
  if (lane == 0) red[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, red[w]);
  if (M == -INFINITY) M = 0.f;      // nothing attended: all weights are 0
  float l = 0.f;
  for (int i = lane; i < n; i += 32) l += ml[i].y * ptx::ex2(ml[i].x - M);
  l = warp_sum(l);       // every warp the same sum
  float acc[PER] = {};
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = warp + k * kJoinWarps;
    if (i < n) {
      const float r = ml[i].y * ptx::ex2(ml[i].x - M);
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = fmaf(r, x[k][e], acc[e]);
    }
  }
#pragma unroll 4
  for (int i = warp + kAhead * kJoinWarps; i < n; i += kJoinWarps) {
    float y[PER];
    load_row<PER>(o + i * stride, y);
    const float r = ml[i].y * ptx::ex2(ml[i].x - M);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(r, y[e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) sums[warp][PER * lane + e] = acc[e];
  __syncthreads();
  if (threadIdx.x < DIMS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) v += sums[w][threadIdx.x];
    a.out[(size_t)row * D + blockIdx.y * DIMS + threadIdx.x] = l > 0.f ? v / l : 0.f;
  }
}

// The same for units of few partials: one warp per row and 128 values.
constexpr int kFewWarps = 4;
template <int D>
__global__ void __launch_bounds__(kFewWarps * 32) decode_block_combine_few_kernel(
    const BlockDecodeArgs a, int rows) {
  constexpr int DIMS = D < 128 ? D : 128, PER = DIMS / 32, CHUNKS = D / DIMS, K = 4;
  const int lane = threadIdx.x & 31;
  const int job = blockIdx.x * kFewWarps + (threadIdx.x >> 5);
  const int row = job / CHUNKS, d = job % CHUNKS * DIMS + PER * lane;
  ptx::grid_launch_dependents();
  const int h = row % a.H, bq = row / a.H, b = bq / a.Q;
  const int kvh = h / a.G, gc = (bq % a.Q) * a.G + h % a.G, cg = gc / a.width, col = gc % a.width;
  ptx::grid_dependency_wait();
  if (row >= rows) return;
  const int2 unit = a.part_units[(b * a.pool.Hkv + kvh) * a.n_cg + cg];
  Seen seen;
  const bool empty = unit_range(a, b, seen) == 0;
  const int n = empty ? 0 : unit.y;
  if (n == 1) return;      // one block had the whole unit and wrote it
  const size_t first = (size_t)unit.x * a.width + col, stride = (size_t)a.width * D;
  float M = kUnset, l = 0.f, acc[PER] = {};
  for (int i0 = 0; i0 < n; i0 += K) {
    float2 v[K];
    float x[K][PER], top = M;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = i0 + k < n;
      v[k] = in ? a.part_ml[first + (size_t)(i0 + k) * a.width] : make_float2(-INFINITY, 0.f);
      load_row<PER>(in ? a.part_o + first * D + (i0 + k) * stride + d : nullptr, x[k]);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) top = fmaxf(top, v[k].x);
    const float r = ptx::ex2(M - top);
    M = top;
    l *= r;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= r;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const float f = v[k].y * ptx::ex2(v[k].x - M);
      l += f;
#pragma unroll
      for (int e = 0; e < PER; ++e) acc[e] = fmaf(f, x[k][e], acc[e]);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) a.out[(size_t)row * D + d + e] = acc[e] * inv;
}

template <int D>
cudaError_t launch_combine(const BlockDecodeArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const int rows = a.B * a.Q * a.H, chunks = D > 128 ? D / 128 : 1;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Up to 8 shares a unit: most rows have one to nine partials, and blocks of 16 warps
  // mostly start to find nothing to do (1536 rows of 12 query windows: 13 us of a call of
  // 42 us, which takes 33 us with a warp a row).
  if (a.shares <= 8LL * a.B * a.pool.Hkv * a.n_cg) {
    cfg.gridDim = dim3((unsigned)(((long long)rows * chunks + kFewWarps - 1) / kFewWarps));
    cfg.blockDim = dim3(kFewWarps * 32);
    return cudaLaunchKernelEx(&cfg, decode_block_combine_few_kernel<D>, a, rows);
  }
  cfg.gridDim = dim3(rows, chunks);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = a.shares * sizeof(float2);    // a unit has at most a piece in every share
  return cudaLaunchKernelEx(&cfg, decode_block_combine_kernel<D>, a);
}

}  // namespace

// (Both kinds are compiled for as many blocks an SM; the least, should one not be.)
int block_decode_resident(int head_dim, bool f8) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  switch (head_dim) {
    case 64: return sms * std::min(block_decode_blocks_64(f8), block_scored_blocks_64(f8));
    case 128: return sms * std::min(block_decode_blocks_128(f8), block_scored_blocks_128(f8));
    case 256: return sms * std::min(block_decode_blocks_256(f8), block_scored_blocks_256(f8));
    default: return -1;
  }
}

int block_decode_clusters(int head_dim, bool f8) {
  switch (head_dim) {
    case 64: return std::min(block_decode_clusters_64(f8), block_scored_clusters_64(f8));
    case 128: return std::min(block_decode_clusters_128(f8), block_scored_clusters_128(f8));
    case 256: return std::min(block_decode_clusters_256(f8), block_scored_clusters_256(f8));
    default: return 0;
  }
}

template <int D, class A>
static cudaError_t launch_joined(cudaError_t (*launch)(const A&, bool, cudaStream_t), const A& a,
                                 bool f8, cudaStream_t stream) {
  if ((long long)a.B * a.Q * a.H > 0x3fffffffLL) return cudaErrorNotSupported;
  const cudaError_t e = launch(a, f8, stream);
  return e != cudaSuccess || a.shares == 0 ? e : launch_combine<D>(a, stream);
}

cudaError_t launch_block_decode(const BlockDecodeArgs& a, int head_dim, bool f8,
                                cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_joined<64>(launch_block_decode_64, a, f8, stream);
    case 128: return launch_joined<128>(launch_block_decode_128, a, f8, stream);
    case 256: return launch_joined<256>(launch_block_decode_256, a, f8, stream);
    default: return cudaErrorNotSupported;
  }
}

cudaError_t launch_block_decode_scored(const BlockScoredArgs& a, int head_dim, bool f8,
                                       cudaStream_t stream) {
  switch (head_dim) {
    case 64: return launch_joined<64>(launch_block_scored_64, a, f8, stream);
    case 128: return launch_joined<128>(launch_block_scored_128, a, f8, stream);
    case 256: return launch_joined<256>(launch_block_scored_256, a, f8, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace int8kv
