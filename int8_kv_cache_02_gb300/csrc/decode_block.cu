// Block-scaled decode: the dispatch over head_dim, and the combine of partials.
#include "decode_block.cuh"

namespace int8kv {
namespace {

using namespace block;

// Join the partials of units that a share boundary cut; zero rows of empty units:
//   out = sum_i o_i 2^(lse_i - M) / sum_i 2^(lse_i - M).
// One block per (sequence, query, head) and 64 values of it; its warps share the
// partials, a lane two values.  The first kAhead rows of each warp are requested
// before the weights are known, so that the two trips to L2 overlap.
constexpr int kJoinWarps = 8;
constexpr int kAhead = 8;

__global__ void __launch_bounds__(kJoinWarps * 32) decode_block_combine_kernel(
    const BlockDecodeArgs a, int D, int least) {
  constexpr int NT = kJoinWarps * 32;
  extern __shared__ float weight[];         // [partials of the unit]
  __shared__ long long warp_sums[kJoinWarps];
  __shared__ long long place;
  __shared__ float red[kJoinWarps];
  __shared__ float2 sums[kJoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int row = blockIdx.x, h = row % a.H, bq = row / a.H, b = bq / a.Q;
  const int kvh = h / a.G, gc = (bq % a.Q) * a.G + h % a.G, cg = gc / a.width, col = gc % a.width;
  const int per_seq = a.pool.Hkv * a.n_cg;
  const int d = blockIdx.y * 64 + 2 * lane;
  long long mine;
  const long long total = batch_tiles<NT>(a, per_seq, warp_sums, mine);
  int lo, hi;
  const int run = (a.B + NT - 1) / NT;
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
  float* out = a.out + (size_t)row * D + d;
  if (nt == 0) {
    if (warp == 0) *reinterpret_cast<float2*>(out) = make_float2(0.f, 0.f);
    return;
  }
  const long long per = share_tiles(total, a.shares, least);
  const long long start = place + (long long)u * nt;
  const long long c0 = start / per, c1 = (start + nt - 1) / per;
  if (c0 == c1) return;      // one block had the whole unit and wrote it
  const int n = (int)(c1 - c0 + 1);
  const size_t first = ((size_t)b * per_seq + u + c0) * a.width + col;
  const float* o = a.part_o + first * D + d;
  const size_t stride = (size_t)a.width * D;
  float2 x[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = warp + k * kJoinWarps;
    x[k] = i < n ? *reinterpret_cast<const float2*>(o + i * stride) : make_float2(0.f, 0.f);
  }
  float M = -INFINITY;
  for (int i = threadIdx.x; i < n; i += NT) {
    const float v = a.part_lse[first + (size_t)i * a.width];
    weight[i] = v;
    M = fmaxf(M, v);
  }
  M = warp_max(M);
  if (lane == 0) red[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, red[w]);
  float l = 0.f;
  for (int i = lane; i < n; i += 32) l += M > -INFINITY ? ptx::ex2(weight[i] - M) : 0.f;
  l = warp_sum(l);       // every warp the same sum
  float2 acc = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = warp + k * kJoinWarps;
    if (i < n && l > 0.f) {
      const float r = ptx::ex2(weight[i] - M);
      acc.x = fmaf(r, x[k].x, acc.x);
      acc.y = fmaf(r, x[k].y, acc.y);
    }
  }
#pragma unroll 4
  for (int i = warp + kAhead * kJoinWarps; i < n; i += kJoinWarps) {
    const float2 y = *reinterpret_cast<const float2*>(o + i * stride);
    const float r = l > 0.f ? ptx::ex2(weight[i] - M) : 0.f;
    acc.x = fmaf(r, y.x, acc.x);
    acc.y = fmaf(r, y.y, acc.y);
  }
  sums[warp][lane] = acc;
  __syncthreads();
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < kJoinWarps; ++w) {
      acc.x += sums[w][lane].x;
      acc.y += sums[w][lane].y;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    *reinterpret_cast<float2*>(out) = make_float2(acc.x * inv, acc.y * inv);
  }
}

}  // namespace

int block_decode_resident(int head_dim, bool f8) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return -1;
  switch (head_dim) {
    case 64: return sms * block_decode_blocks_64(f8);
    case 128: return sms * block_decode_blocks_128(f8);
    case 256: return sms * block_decode_blocks_256(f8);
    default: return -1;
  }
}

cudaError_t launch_block_decode(const BlockDecodeArgs& a, int head_dim, bool f8,
                                cudaStream_t stream) {
  const long long rows = (long long)a.B * a.Q * a.H;
  if (rows > 0x7fffffffLL) return cudaErrorNotSupported;
  cudaError_t e;
  int least;      // as the decode kernel's
  switch (head_dim) {
    case 64: e = launch_block_decode_64(a, f8, stream); least = Shape<64>::LEAST; break;
    case 128: e = launch_block_decode_128(a, f8, stream); least = Shape<128>::LEAST; break;
    case 256: e = launch_block_decode_256(a, f8, stream); least = Shape<256>::LEAST; break;
    default: return cudaErrorNotSupported;
  }
  if (e != cudaSuccess || a.shares == 0) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows, head_dim / 64);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = a.shares * sizeof(float);     // a unit has at most a piece in every share
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_block_combine_kernel, a, head_dim, least);
}

}  // namespace int8kv
