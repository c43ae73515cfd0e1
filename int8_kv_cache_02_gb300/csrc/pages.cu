// Pages of a pool on the device: copying them, forking sequences, giving rows of a
// page table the pages their lengths need, and compacting the pool.
//
// page_refs[p] counts the page-table entries that name page p; 0 is a free page.
// Pages are taken in ascending order of id by the rows (forks) in ascending order,
// so results do not depend on timing: counts change by integer atomics whose order
// does not matter, everything that is ranked is ranked by prefix sums.
//
// The bookkeeping of one call runs in one cluster of thread blocks (the calls read
// a few hundred KB: a grid-wide barrier would cost more than the other SMs bring).
// A range of entries or pages is cut into one contiguous run per warp; a rank is the
// prefix sum over the runs before it, exchanged through distributed shared memory.  The bytes of pages move in a second, grid-wide kernel, which reads its
// list of (source, destination) pairs from device memory.
#include <cooperative_groups.h>

#include "block_common.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace int8kv {
namespace {

constexpr int kBlocks = 8;        // blocks of the bookkeeping cluster
constexpr int kThreads = 1024;    // threads of each
constexpr int kWarps = kBlocks * kThreads / 32;

// ---- copies -----------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kPieces = 4;                                   // 16-byte pieces a thread has in flight
constexpr int kChunk = kCopyThreads * kPieces * 16;          // bytes a block copies at a time

struct Regions {
  char* store[2];            // K and V, all layers
  char* scales[2];           // theirs, or null
  unsigned bytes[2];         // of a page of one layer
  unsigned scale_bytes[2];
  int k_chunks, chunks;      // chunks of a page's K store, and of both stores
  int n_layers, n_pages;
  int32_t* err;
};

// Pages (src[i], dst[i]) of every layer, i < n (or *n_dev).  A negative entry on either
// side is no copy.  One block per chunk of a store (a block per chunk balances better
// than blocks that stay: 134 MB copied in 43 against 47 us); the first chunk of a store
// brings its scales.
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(const Regions r, const int32_t* src,
                                                                 const int32_t* dst, int n,
                                                                 const int32_t* n_dev) {
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  if (n_dev) n = *n_dev;
  const unsigned total = (unsigned)n * r.n_layers * r.chunks;      // (fewer than 2^31)
  for (unsigned w = blockIdx.x; w < total; w += gridDim.x) {
    const int c = w % (unsigned)r.chunks;
    const unsigned il = w / (unsigned)r.chunks;
    const int layer = il % (unsigned)r.n_layers, i = il / (unsigned)r.n_layers;
    const int s = src[i], d = dst[i];
    if (s < 0 || d < 0 || s >= r.n_pages || d >= r.n_pages) {
      if (threadIdx.x == 0 && s >= 0 && d >= 0) flag_error(r.err, INT8KV_DEVERR_PAGE_ID);
      continue;
    }
    if (s == d) continue;
    const int k = c >= r.k_chunks;
    const unsigned at = (unsigned)(k ? c - r.k_chunks : c) * kChunk;
    const unsigned len = min(r.bytes[k] - at, (unsigned)kChunk);
    const size_t from = (size_t)layer * r.n_pages + s, to = (size_t)layer * r.n_pages + d;
    const char* in = r.store[k] + from * r.bytes[k] + at;
    char* out = r.store[k] + to * r.bytes[k] + at;
    uint4 x[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const unsigned o = (threadIdx.x + j * kCopyThreads) * 16;
      if (o < len) x[j] = *reinterpret_cast<const uint4*>(in + o);
    }
    if (at == 0 && r.scales[k]) {      // a multiple of 4 bytes
      const unsigned bytes = r.scale_bytes[k];
      const char* f = r.scales[k] + from * bytes;
      char* t = r.scales[k] + to * bytes;
      for (unsigned o = threadIdx.x * 4; o < bytes; o += kCopyThreads * 4)
        *reinterpret_cast<uint32_t*>(t + o) = *reinterpret_cast<const uint32_t*>(f + o);
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const unsigned o = (threadIdx.x + j * kCopyThreads) * 16;
      if (o < len) *reinterpret_cast<uint4*>(out + o) = x[j];
    }
  }
}

// ---- bookkeeping ------------------------------------------------------------
// Each warp of the cluster owns a contiguous run of items, which its lanes read side by
// side, kAhead loads in flight; ranks within 32 items come from a ballot.
constexpr int kAhead = 8;
constexpr unsigned kAll = 0xffffffffu;

struct Ranks {
  int warp[kThreads / 32];
  int block[2];       // this block's sum, double-buffered over calls
};

// Exclusive prefix sum of v (the same in all lanes) over the cluster's warps, in order;
// *total its sum.  Every warp of the cluster calls it the same number of times, and the
// cluster meets at a barrier in it.
__device__ __forceinline__ int cluster_rank(int v, int& total, Ranks& sh, int& phase) {
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  if (lane == 0) sh.warp[wid] = v;
  __syncthreads();
  const int mine = lane < kThreads / 32 ? sh.warp[lane] : 0;
  int before = lane < wid ? mine : 0, sum = mine;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    before += __shfl_xor_sync(kAll, before, off);
    sum += __shfl_xor_sync(kAll, sum, off);
  }
  if (threadIdx.x == 0) sh.block[phase] = sum;
  cl.sync();     // (also: sh.warp may be written again)
  total = 0;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    const int o = *cl.map_shared_rank(&sh.block[phase], b);
    if (b < (int)cl.block_rank()) before += o;
    total += o;
  }
  phase ^= 1;    // the other slot was read before the last cluster barrier
  return before;
}

// This warp's run [a, z) of n items, whole groups of `group`.
__device__ __forceinline__ void run_of(int n, int group, int& a, int& z) {
  const long long per = (((long long)n + group - 1) / group + kWarps - 1) / kWarps * group;
  const long long at = per * (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5));
  a = (int)(at < n ? at : n);
  z = (int)(at + per < n ? at + per : n);
}

// One reference less.  A page that has none stays at 0 (flagged).
__device__ __forceinline__ void give_back(int32_t* refs, int page, int32_t* err) {
  if (atomicAdd(refs + page, -1) <= 0) {
    atomicAdd(refs + page, 1);
    flag_error(err, INT8KV_DEVERR_PAGE_ID);
  }
}

// The `want` first free pages in ascending order -> list; returns how many there are of
// them (fewer than `want` when the pool runs out).  Pools are searched a span at a time.
__device__ __forceinline__ int free_pages(const int32_t* refs, int n_pages, int want, int32_t* list,
                                          Ranks& sh, int& phase) {
  constexpr int SPAN = kWarps * 32 * kAhead;
  const int lane = threadIdx.x & 31;
  int got = 0;
  for (int base = 0; base < n_pages && got < want; base += SPAN) {
    const int first = base + (blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * 32 * kAhead;
    unsigned free[kAhead];
    int mine = 0;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = first + 32 * k + lane;
      free[k] = i < n_pages ? __ldcg(refs + i) : 1;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      free[k] = __ballot_sync(kAll, free[k] == 0);
      mine += __popc(free[k]);
    }
    int found;
    int at = got + cluster_rank(mine, found, sh, phase);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int rank = at + __popc(free[k] & ((1u << lane) - 1));
      if ((free[k] >> lane & 1) && rank < want) list[rank] = first + 32 * k + lane;
      at += __popc(free[k]);
    }
    got += found;
  }
  cg::this_cluster().sync();
  return got < want ? got : want;
}

struct PagesArgs {
  int32_t* refs;
  int32_t* table;          // [n_seqs][max_pages]
  int n_seqs, max_pages, n_pages, page_size, ps_log2;
  int32_t* err;
  int32_t* list;           // workspace: free pages, [n_pages]
  int32_t* src;            // workspace: pages to copy, [max(n_pages, n_seqs)] each
  int32_t* dst;
  int32_t* map;            // workspace: [max(n_pages, 2 n_seqs)]
  int32_t* count;          // workspace: pairs to copy
};

// The table in pieces of 32 entries of a row: a warp reads its run of them kBatch at a
// time and only looks for work; the few pieces that have some are read again.  (Kernels
// like this run their code once: unrolled handling of every piece took longer to fetch
// than to execute.)
constexpr int kBatch = 8;

__global__ void __launch_bounds__(kThreads) resize_kernel(const PagesArgs a,
                                                          const int32_t* __restrict__ lens) {
  __shared__ Ranks sh;
  int phase = 0;
  const int lane = threadIdx.x & 31;
  const int per_row = (a.max_pages + 31) / 32;      // pieces of a row
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  int lo, hi;
  run_of(a.n_seqs * per_row, 1, lo, hi);
  int missing = 0, first_missing = hi, row = lo / per_row, c = lo % per_row;
  for (int base = lo; base < hi; base += kBatch) {
    int e[kBatch];
    bool need[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int p = c * 32 + lane;
      const bool in = base + k < hi && p < a.max_pages;
      need[k] = in && __ldg(lens + row) > p << a.ps_log2;
      e[k] = in ? a.table[(size_t)row * a.max_pages + p] : -1;
      if (++c == per_row) {
        c = 0;
        ++row;
      }
    }
    unsigned work = 0;      // bit k: this lane's entry of piece k goes back, or is no page
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const bool none = e[k] < 0 || e[k] >= a.n_pages;
      missing += __popc(__ballot_sync(kAll, need[k] && none));
      if (e[k] >= a.n_pages || (!need[k] && !none)) work |= 1u << k;
    }
    if (missing && first_missing == hi) first_missing = base;
    while (work) {
      const int k = __ffs(work) - 1, w = base + k;
      work &= work - 1;
      int32_t* at = a.table + (size_t)(w / per_row) * a.max_pages + w % per_row * 32 + lane;
      if (*at >= a.n_pages) flag_error(a.err, INT8KV_DEVERR_PAGE_ID);
      else give_back(a.refs, *at, a.err);
      *at = -1;
    }
  }
  for (int r = blockIdx.x * kThreads + threadIdx.x; r < a.n_seqs; r += kBlocks * kThreads)
    if (__ldg(lens + r) > (long long)a.max_pages << a.ps_log2) flag_error(a.err, INT8KV_DEVERR_LENGTH);
  int want;
  int rank = cluster_rank(missing, want, sh, phase);
  if (want == 0) {            // the same for the whole cluster
    cg::this_cluster().sync();   // the others may still read this block's sum
    return;
  }
  const int n = free_pages(a.refs, a.n_pages, want, a.list, sh, phase);
#pragma unroll 1
  for (int w = first_missing; w < hi && missing > 0; ++w) {
    const int r = w / per_row, p = w % per_row * 32 + lane;
    int32_t* at = a.table + (size_t)r * a.max_pages + p;
    const bool miss = p < a.max_pages && __ldg(lens + r) > p << a.ps_log2 && *at < 0;
    const unsigned all = __ballot_sync(kAll, miss);
    const int mine = rank + __popc(all & ((1u << lane) - 1));
    if (miss) {
      if (mine < n) {
        const int page = __ldcg(a.list + mine);
        *at = page;
        a.refs[page] = 1;
      } else {
        flag_error(a.err, INT8KV_DEVERR_NO_PAGE);
      }
    }
    rank += __popc(all);
    missing -= __popc(all);
  }
}

// Which forks take place.  Up to kRows rows every block keeps its own marks in shared
// memory; beyond, the cluster shares marks in the workspace.
constexpr int kRows = 4096;
struct Marks {
  int* first;      // lowest fork that names a row as its child
  int* parent;     // whether a row is some fork's parent
  bool shared;
  // one that names no two rows (-1) is left out silently
  __device__ __forceinline__ bool take(const PagesArgs& a, int i, int p, int c) const {
    if (p < 0 || c < 0 || p >= a.n_seqs || c >= a.n_seqs) return false;
    return shared ? first[c] == i && parent[c] == 0
                  : __ldcg(first + c) == i && __ldcg(parent + c) == 0;
  }
};

__global__ void __launch_bounds__(kThreads) fork_kernel(const PagesArgs a, int32_t* lens, int n,
                                                        const int32_t* __restrict__ parents,
                                                        const int32_t* __restrict__ children) {
  __shared__ Ranks sh;
  __shared__ int marks[2 * kRows];
  int phase = 0;
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  Marks m;
  m.shared = a.n_seqs <= kRows;
  m.first = m.shared ? marks : a.map;
  m.parent = m.first + a.n_seqs;
  const int me = m.shared ? threadIdx.x : blockIdx.x * kThreads + threadIdx.x;
  const int step = m.shared ? kThreads : kBlocks * kThreads;
  auto meet = [&]() {
    if (m.shared) __syncthreads();
    else cl.sync();
  };
  for (int i = me; i < a.n_seqs; i += step) {
    m.first[i] = INT32_MAX;
    m.parent[i] = 0;
  }
  meet();
  for (int i = me; i < n; i += step) {
    const int p = parents[i], c = children[i];
    if (p < 0 || c < 0 || p >= a.n_seqs || c >= a.n_seqs) continue;
    atomicMin(m.first + c, i);
    atomicExch(m.parent + p, 1);
  }
  meet();
  const long long cap = (long long)a.max_pages * a.page_size;
  // children's rows: what they held goes back, the parent's full pages are shared
  const long long entries = (long long)n * a.max_pages;
  for (long long w = blockIdx.x * kThreads + threadIdx.x; w < entries; w += kBlocks * kThreads) {
    const int i = (int)(w / a.max_pages), k = (int)(w % a.max_pages);
    const int p = parents[i], c = children[i];
    if (!m.take(a, i, p, c)) {
      if (k == 0 && p >= 0 && c >= 0) flag_error(a.err, INT8KV_DEVERR_FORK);
      continue;
    }
    const int len = lens[p];
    if (k == 0 && len > cap) flag_error(a.err, INT8KV_DEVERR_LENGTH);
    int32_t* mine = a.table + (size_t)c * a.max_pages + k;
    const int was = *mine;
    int e = -1;
    if (k < min((long long)max(len, 0), cap) / a.page_size) {
      e = a.table[(size_t)p * a.max_pages + k];
      if (e < 0 || e >= a.n_pages) {
        flag_error(a.err, INT8KV_DEVERR_PAGE_ID);
        e = -1;
      } else {
        atomicAdd(a.refs + e, 1);
      }
    }
    if (was >= 0) {
      if (was < a.n_pages) give_back(a.refs, was, a.err);
      else flag_error(a.err, INT8KV_DEVERR_PAGE_ID);
    }
    *mine = e;
  }
  // forks whose parent ends inside a page need a page of their own for its copy
  int lo, hi;
  run_of(n, 32, lo, hi);
  int need = 0;
  for (int base = lo; base < hi; base += 32) {
    const int i = base + lane;
    int page = -1;
    if (i < hi) {
      const int p = parents[i], c = children[i];
      if (m.take(a, i, p, c)) {
        const long long len = min((long long)max(lens[p], 0), cap);
        if (len % a.page_size) {
          page = a.table[(size_t)p * a.max_pages + len / a.page_size];
          if (page < 0 || page >= a.n_pages) {
            flag_error(a.err, INT8KV_DEVERR_PAGE_ID);
            page = -1;
          }
        }
      }
      a.src[i] = page;
    }
    need += __popc(__ballot_sync(kAll, page >= 0));
  }
  int want;
  int at = cluster_rank(need, want, sh, phase);
  int got = 0;
  if (want) got = free_pages(a.refs, a.n_pages, want, a.list, sh, phase);
  else cl.sync();     // the others may still read this block's sum
  for (int base = lo; base < hi; base += 32) {
    const int i = base + lane;
    const bool copies = i < hi && a.src[i] >= 0;
    const unsigned all = __ballot_sync(kAll, copies);
    const int rank = at + __popc(all & ((1u << lane) - 1));
    at += __popc(all);
    if (i >= hi) continue;
    const int p = parents[i], c = children[i];
    int page = -1;
    if (m.take(a, i, p, c)) {
      int len = (int)min((long long)max(lens[p], 0), cap);
      if (copies) {
        if (rank < got) {
          page = __ldcg(a.list + rank);
          a.refs[page] = 1;
          a.table[(size_t)c * a.max_pages + len / a.page_size] = page;
        } else {     // no page for the rest: the child ends with the shared ones
          flag_error(a.err, INT8KV_DEVERR_NO_PAGE);
          len -= len % a.page_size;
        }
      }
      lens[c] = len;
    }
    a.dst[i] = page;
  }
}

// Ids [0, used) are to be the used ones.  Free ids there (holes) are filled, in order, with
// the used pages from `used` on (movers).  A free id i < used is hole number i - (used
// pages before i); a used id i >= used is mover number (used pages before i) - (used
// pages below `used`), and those are `used` less the holes.
__global__ void __launch_bounds__(kThreads) compact_kernel(const PagesArgs a, int32_t* refs_out,
                                                           int32_t* table_out, int32_t* n_used) {
  __shared__ Ranks sh;
  int phase = 0;
  cg::cluster_group cl = cg::this_cluster();
  const int lane = threadIdx.x & 31;
  const unsigned before_me = (1u << lane) - 1;
  ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  int lo, hi;
  run_of(a.n_pages, 32, lo, hi);
  int mine = 0;
  for (int base = lo; base < hi; base += 32 * kAhead) {
    int r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = base + 32 * k + lane;
      r[k] = i < hi ? a.refs[i] : 0;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) mine += __popc(__ballot_sync(kAll, r[k] > 0));
  }
  int used;
  const int before = cluster_rank(mine, used, sh, phase);     // used pages before the run
  int holes = 0, at = before;
  for (int base = lo; base < hi && base < used; base += 32) {
    const int i = base + lane;
    const int r = i < hi && i < used ? a.refs[i] : 0;
    const unsigned all = __ballot_sync(kAll, r > 0);
    if (i < hi && i < used) {
      a.map[i] = r > 0 ? i : -1;
      if (r > 0) refs_out[i] = r;      // (a hole's count comes with the page that fills it)
      else a.dst[i - (at + __popc(all & before_me))] = i;
      holes += r <= 0;
    }
    at += __popc(all);
  }
  int n;
  holes = __reduce_add_sync(kAll, holes);
  cluster_rank(holes, n, sh, phase);       // n: pages to move (and a.dst is there)
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *n_used = used;
    *a.count = n;
  }
  // the run's pages from `used` on: `at` counts the used ones before them
  const int from = lo > used ? lo : used;
  if (lo >= used) at = before;
  for (int base = from; base < hi; base += 32) {
    const int i = base + lane;
    const int r = i < hi ? a.refs[i] : 0;
    const unsigned all = __ballot_sync(kAll, r > 0);
    if (i < hi) {
      int to = -1;
      if (r > 0) {
        const int rank = at + __popc(all & before_me) - (used - n);
        to = __ldcg(a.dst + rank);
        a.src[rank] = i;
        refs_out[to] = r;
      }
      a.map[i] = to;
      refs_out[i] = 0;
    }
    at += __popc(all);
  }
  cl.sync();
  const long long entries = (long long)a.n_seqs * a.max_pages;
  for (long long i = blockIdx.x * kThreads + threadIdx.x; i < entries; i += kBlocks * kThreads) {
    int e = a.table[i];
    if (e >= 0) {
      e = e < a.n_pages ? __ldcg(a.map + e) : -1;
      if (e < 0) flag_error(a.err, INT8KV_DEVERR_PAGE_ID);
    }
    table_out[i] = e;
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

size_t workspace(const int8kv_pool* p, int n_seqs, PagesArgs* a, void* base) {
  const size_t pages = p->n_pages, seqs = n_seqs;
  const size_t list = up256(pages * 4), pair = up256((pages > seqs ? pages : seqs) * 4),
               map = up256((pages > 2 * seqs ? pages : 2 * seqs) * 4);
  if (a) {
    char* w = (char*)base;
    a->count = (int32_t*)w;
    a->list = (int32_t*)(w + 256);
    a->src = (int32_t*)(w + 256 + list);
    a->dst = (int32_t*)(w + 256 + list + pair);
    a->map = (int32_t*)(w + 256 + list + 2 * pair);
  }
  return 256 + list + 2 * pair + map;
}

template <class... A>
cudaError_t launch_cluster(void (*kernel)(A...), cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kBlocks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kBlocks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A copy of at most `most` pairs: what its kernel gets, and its blocks' number.  n_dev: the number
// of pairs on the device, or null.  Made before a call launches anything, so that one that
// cannot copy changes nothing.
struct Copy {
  Regions r;
  unsigned grid;
  int most;
  const int32_t* n_dev;
};

cudaError_t plan_copy(const int8kv_pool* p, int most, const int32_t* n_dev, Copy* c) {
  Regions& r = c->r;
  const auto bytes = [&](int region, unsigned* out) {
    size_t b = 0;
    int8kv_pool_region_bytes(1, p->n_kv_heads, p->head_dim, p->group_size, p->page_size, 1,
                             p->variant, region, &b);
    *out = (unsigned)b;
    return b <= 0x7fffffff;
  };
  if (!bytes(INT8KV_REGION_K_STORE, &r.bytes[0]) || !bytes(INT8KV_REGION_V_STORE, &r.bytes[1]) ||
      !bytes(INT8KV_REGION_K_SCALES, &r.scale_bytes[0]) ||
      !bytes(INT8KV_REGION_V_SCALES, &r.scale_bytes[1]))
    return cudaErrorNotSupported;
  r.store[0] = (char*)p->k_store;
  r.store[1] = (char*)p->v_store;
  r.scales[0] = (char*)p->k_scales;
  r.scales[1] = (char*)p->v_scales;
  r.k_chunks = (int)((r.bytes[0] + kChunk - 1) / kChunk);
  r.chunks = r.k_chunks + (int)((r.bytes[1] + kChunk - 1) / kChunk);
  r.n_layers = p->n_layers;
  r.n_pages = p->n_pages;
  r.err = p->dev_error;
  const long long total = (long long)most * p->n_layers * r.chunks;
  if (total > 0x7fffffffLL) return cudaErrorNotSupported;
  // a number of pairs known on the device only: at most four blocks a slot, which stride
  const long long cap = n_dev ? 32LL * p->num_sms : 0x7fffffffLL;
  c->grid = (unsigned)(total < cap ? total : cap);
  c->most = most;
  c->n_dev = n_dev;
  return cudaSuccess;
}

cudaError_t launch_copy(const Copy& c, const int32_t* src, const int32_t* dst, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(c.grid);
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, copy_pages_kernel, c.r, src, dst, c.most, c.n_dev);
}

// The checks that the bookkeeping calls share, and their kernels' arguments.
int prepare(const int8kv_pool* pool, const int32_t* refs, const int32_t* table, int n_seqs,
            int max_pages, void* ws, size_t ws_bytes, PagesArgs* a) {
  if (!pool) return INT8KV_ERR_NULL_PTR;
  if (n_seqs < 0 || max_pages <= 0) return INT8KV_ERR_INVALID_ARG;
  if ((long long)n_seqs * (max_pages / 32 + 1) > INT32_MAX / 2 ||
      (long long)max_pages * pool->page_size > INT32_MAX)     // pieces and positions count in 32 bits
    return INT8KV_ERR_UNSUPPORTED;
  if (!refs || (n_seqs > 0 && !table)) return INT8KV_ERR_NULL_PTR;
  if (!ws || ws_bytes < workspace(pool, n_seqs, nullptr, nullptr)) return INT8KV_ERR_WORKSPACE;
  if (((uintptr_t)ws & 15) != 0) return INT8KV_ERR_ALIGNMENT;
  if (!on_current_device(pool)) return INT8KV_ERR_INVALID_ARG;
  a->refs = const_cast<int32_t*>(refs);
  a->table = const_cast<int32_t*>(table);
  a->n_seqs = n_seqs;
  a->max_pages = max_pages;
  a->n_pages = pool->n_pages;
  a->page_size = pool->page_size;
  for (a->ps_log2 = 0; 1 << a->ps_log2 < pool->page_size;) ++a->ps_log2;
  a->err = pool->dev_error;
  workspace(pool, n_seqs, a, ws);
  return INT8KV_OK;
}

int status(cudaError_t e) {
  if (e == cudaErrorNotSupported) return INT8KV_ERR_UNSUPPORTED;
  return e == cudaSuccess ? INT8KV_OK : INT8KV_ERR_CUDA;
}

}  // namespace
}  // namespace int8kv

using namespace int8kv;

extern "C" {

int kv_pages_workspace_bytes(const int8kv_pool* pool, int n_seqs, size_t* out_bytes) {
  if (!pool || !out_bytes) return INT8KV_ERR_NULL_PTR;
  if (n_seqs < 0) return INT8KV_ERR_INVALID_ARG;
  *out_bytes = workspace(pool, n_seqs, nullptr, nullptr);
  return INT8KV_OK;
}

int kv_pages_copy(const int8kv_pool* pool, int n, const int32_t* src, const int32_t* dst,
                  void* stream) {
  if (!pool) return INT8KV_ERR_NULL_PTR;
  if (n < 0) return INT8KV_ERR_INVALID_ARG;
  if (n == 0) return INT8KV_OK;
  if (!src || !dst) return INT8KV_ERR_NULL_PTR;
  if (!on_current_device(pool)) return INT8KV_ERR_INVALID_ARG;
  Copy c;
  const cudaError_t e = plan_copy(pool, n, nullptr, &c);
  return status(e != cudaSuccess ? e : launch_copy(c, src, dst, (cudaStream_t)stream));
}

int kv_pages_resize(const int8kv_pool* pool, int32_t* page_refs, int32_t* page_table, int n_seqs,
                    int max_pages_per_seq, const int32_t* seq_lens, void* workspace,
                    size_t workspace_bytes, void* stream) {
  PagesArgs a;
  const int st = prepare(pool, page_refs, page_table, n_seqs, max_pages_per_seq, workspace,
                         workspace_bytes, &a);
  if (st != INT8KV_OK) return st;
  if (n_seqs == 0) return INT8KV_OK;
  if (!seq_lens) return INT8KV_ERR_NULL_PTR;
  return status(launch_cluster(resize_kernel, (cudaStream_t)stream, (const PagesArgs)a, seq_lens));
}

int kv_pages_fork(const int8kv_pool* pool, int32_t* page_refs, int32_t* page_table, int n_seqs,
                  int max_pages_per_seq, int32_t* seq_lens, int n_forks, const int32_t* parents,
                  const int32_t* children, void* workspace, size_t workspace_bytes, void* stream) {
  PagesArgs a;
  const int st = prepare(pool, page_refs, page_table, n_seqs, max_pages_per_seq, workspace,
                         workspace_bytes, &a);
  if (st != INT8KV_OK) return st;
  if (n_forks < 0 || n_forks > n_seqs) return INT8KV_ERR_INVALID_ARG;
  if (n_forks == 0) return INT8KV_OK;
  if (!seq_lens || !parents || !children) return INT8KV_ERR_NULL_PTR;
  const cudaStream_t s = (cudaStream_t)stream;
  Copy c;
  cudaError_t e = plan_copy(pool, n_forks, nullptr, &c);
  if (e == cudaSuccess)
    e = launch_cluster(fork_kernel, s, (const PagesArgs)a, seq_lens, n_forks, parents, children);
  return status(e != cudaSuccess ? e : launch_copy(c, a.src, a.dst, s));
}

int kv_pages_compact(const int8kv_pool* pool, const int32_t* page_refs, const int32_t* page_table,
                     int n_seqs, int max_pages_per_seq, int32_t* page_refs_out,
                     int32_t* page_table_out, int32_t* n_used, void* workspace,
                     size_t workspace_bytes, void* stream) {
  PagesArgs a;
  const int st = prepare(pool, page_refs, page_table, n_seqs, max_pages_per_seq, workspace,
                         workspace_bytes, &a);
  if (st != INT8KV_OK) return st;
  if (!page_refs_out || (n_seqs > 0 && !page_table_out) || !n_used) return INT8KV_ERR_NULL_PTR;
  const cudaStream_t s = (cudaStream_t)stream;
  Copy c;
  cudaError_t e = plan_copy(pool, pool->n_pages / 2 + 1, a.count, &c);
  if (e == cudaSuccess)
    e = launch_cluster(compact_kernel, s, (const PagesArgs)a, page_refs_out, page_table_out, n_used);
  return status(e != cudaSuccess ? e : launch_copy(c, a.src, a.dst, s));
}

}  // extern "C"
