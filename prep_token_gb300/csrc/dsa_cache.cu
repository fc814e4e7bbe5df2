// Upkeep of a paged cache's pages: copy, fork, free and compact.
//
// A pool of num_pages pages is described by three caller-owned arrays on the
// device: page_refs[p], how many block-table entries hold page p (0 = free);
// block_table[row][j], the page of tokens [j * page_size, (j + 1) *
// page_size) of a row, and context_lens[row].  A page is opaque bytes, so one
// pool serves any number of caches at once (every layer's index-K, K and V):
// each is a base pointer and a page size in bytes.
//
// There is no free list: a new page is always the lowest free one, found by a
// scan of page_refs.  The state then has one truth that cannot disagree with
// itself, releases are commutative decrements (atomics whose order leaves no
// trace), and the pool stays packed towards its start.
//
// Bound: the page bytes (2 per byte moved) for large calls, launch and one or
// two dependent memory round trips for small ones.  Measured (6.78 TB/s): 1024
// pages of 128 KB in 4 caches, 1.07 GB, copied in 162 us (6.64 TB/s); 600 live of
// 2048 such pages packed in 8 caches in 135 us in a graph; a fork of 4 rows with 21
// caches and the free of the children 9 us, the release of half of 64 rows of 512
// blocks behind a window 3.3 us, both in a graph.
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "dsa_common.cuh"
#include "dsa_prep.h"

namespace {

using namespace dsa_dev;

constexpr int kMaxCaches = DSA_MAX_CACHES;
constexpr int kMaxForks = DSA_MAX_FORKS;
constexpr int kCopyThreads = 256;
constexpr int kCopyBytes = 32768;  // of a page per CTA: 8 16-byte loads in flight per thread
constexpr int kPlanThreads = 1024;
constexpr int kMaxCompactPages = 1 << 20;  // the plan holds one bit per page in shared memory

struct Caches {
  char* base[kMaxCaches];
  long long page_bytes[kMaxCaches];
};

// `bytes` from src to dst by one CTA, in units of V (uint4 where the pages are
// 16-byte aligned, else uint32): kUnroll loads of a thread are in flight.
template <class V>
__device__ __forceinline__ void copy_bytes(char* dst, const char* src, int bytes) {
  constexpr int kUnroll = 8;
  const int n = bytes / static_cast<int>(sizeof(V));
  V* d = reinterpret_cast<V*>(dst);
  const V* s = reinterpret_cast<const V*>(src);
  for (int i0 = threadIdx.x; i0 < n; i0 += kUnroll * kCopyThreads) {
    V v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i0 + u * kCopyThreads < n) v[u] = __ldcs(s + i0 + u * kCopyThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (i0 + u * kCopyThreads < n) d[i0 + u * kCopyThreads] = v[u];
  }
}

// Piece `chunk` of page src of cache c to page dst of it.
__device__ __forceinline__ void copy_page_chunk(const Caches& cs, int c, long long src,
                                                long long dst, int chunk) {
  const long long pb = cs.page_bytes[c];
  const long long at = static_cast<long long>(chunk) * kCopyBytes;
  if (at >= pb) return;
  const int bytes = static_cast<int>(pb - at < kCopyBytes ? pb - at : kCopyBytes);
  char* d = cs.base[c] + dst * pb + at;
  const char* s = cs.base[c] + src * pb + at;
  if (((reinterpret_cast<uintptr_t>(cs.base[c]) | static_cast<uintptr_t>(pb)) & 15) == 0)
    copy_bytes<uint4>(d, s, bytes);
  else
    copy_bytes<uint32_t>(d, s, bytes);
}

__device__ __forceinline__ void report(int* err, int bit) {
  if (err) atomicOr(err, bit);
}

__device__ __forceinline__ bool in_pool(int p, int num_pages) {
  return p >= 0 && p < num_pages;
}

// ---------------------------------------------------------------- copy

__global__ void __launch_bounds__(kCopyThreads)
    dsa_copy_pages_kernel(const __grid_constant__ Caches cs, int num_pages, const int* src,
                          const int* dst, int* err) {
  const int s = __ldg(src + blockIdx.x), d = __ldg(dst + blockIdx.x);
  if (!in_pool(s, num_pages) || !in_pool(d, num_pages)) {
    if (threadIdx.x == 0) report(err, DSA_DEVERR_SLOT);
    return;
  }
  if (s != d) copy_page_chunk(cs, blockIdx.y, s, d, blockIdx.z);
}

// ---------------------------------------------------------------- block scans

// Exclusive sum over the CTA's kPlanThreads values; *total gets the sum.
// `part` is 33 ints of shared memory, free again on return.
__device__ __forceinline__ int block_scan(int v, int* part, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = part[lane];
    int s = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += y;
    }
    part[lane] = s - w;
    if (lane == 31) part[32] = s;
  }
  __syncthreads();
  const int before = part[warp] + x - v;
  *total = part[32];
  __syncthreads();
  return before;
}

// ---------------------------------------------------------------- fork

struct ForkParams {
  int* refs;
  int* table;
  int* lens;
  const int* parents;
  const int* children;
  int2* plan;  // [n]: (fresh page, or kNoPage / kRefused; the parent's length)
  long long bt_stride;
  int bt_cols, rows, num_pages, page_size, n;
  int* err;
};
constexpr int kNoPage = -1;   // the parent ends on a page boundary: nothing to copy
constexpr int kRefused = -2;  // this fork does not happen

// One CTA: checks every fork and hands the lowest free pages, in the order of
// the forks, to those whose parent ends inside a page.
__global__ void __launch_bounds__(kPlanThreads) dsa_fork_plan_kernel(const ForkParams p) {
  __shared__ int child_of[kMaxForks];
  __shared__ int fresh[kMaxForks];
  __shared__ int part[33];
  const int i = threadIdx.x;
  int parent = 0, child = -1, len = 0;
  bool ok = false;
  if (i < p.n) {
    parent = __ldg(p.parents + i);
    child = __ldg(p.children + i);
    child_of[i] = child;
    ok = parent >= 0 && parent < p.rows && child >= 0 && child < p.rows;
    if (ok) {
      len = p.lens[parent];
      ok = len >= 0 && (static_cast<long long>(len) + p.page_size - 1) / p.page_size <= p.bt_cols &&
           p.lens[child] == 0;
    }
  }
  __syncthreads();
  if (i < p.n) {  // a child named before belongs to the earlier fork
    for (int j = 0; j < i; ++j) ok = ok && child_of[j] != child;
    if (ok && len == 0)  // parents are read as they were: one that this call makes is not there yet
      for (int j = 0; j < p.n; ++j) ok = ok && child_of[j] != parent;
  }
  if (i < p.n && !ok) report(p.err, DSA_DEVERR_ROW);
  const bool need = ok && len % p.page_size != 0;
  int total = 0;
  const int rank = block_scan(need ? 1 : 0, part, &total);

  // The lowest `total` free pages: 16 consecutive counts per thread and step.
  constexpr int kPer = 16;
  int found = 0;
  for (long long base = 0; base < p.num_pages && found < total; base += kPer * kPlanThreads) {
    const long long first = base + static_cast<long long>(i) * kPer;
    unsigned free_bits = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (first + k < p.num_pages && p.refs[first + k] == 0) free_bits |= 1u << k;
    int here = 0;
    int at = found + block_scan(__popc(free_bits), part, &here);
    for (; free_bits && at < total; free_bits &= free_bits - 1)
      fresh[at++] = static_cast<int>(first) + __ffs(free_bits) - 1;
    found += here;
  }
  __syncthreads();
  if (i < p.n) {
    int page = ok ? kNoPage : kRefused;
    if (need) {
      if (rank < found) {
        page = fresh[rank];
        p.refs[page] = 1;
      } else {
        page = kRefused;
        report(p.err, DSA_DEVERR_POOL);
      }
    }
    p.plan[i] = make_int2(page, len);
  }
}

// blockIdx.z = fork; blockIdx.x == 0, y == 0: the child's table row and the
// counts of the pages it shares; blockIdx.x >= 1: the copy of the parent's
// last page, chunk x - 1 of cache y.
__global__ void __launch_bounds__(kCopyThreads)
    dsa_fork_kernel(const __grid_constant__ Caches cs, const ForkParams p) {
  grid_dependency_wait();
  const int f = blockIdx.z;
  const int2 plan = p.plan[f];
  if (plan.x == kRefused) return;
  const int len = plan.y;
  const int whole = len / p.page_size;
  const int* from = p.table + __ldg(p.parents + f) * p.bt_stride;
  if (blockIdx.x == 0) {
    if (blockIdx.y != 0) return;
    const int child = __ldg(p.children + f);
    int* to = p.table + child * p.bt_stride;
    for (int j = threadIdx.x; j < whole; j += kCopyThreads) {
      int e = from[j];
      if (e >= p.num_pages) {
        report(p.err, DSA_DEVERR_SLOT);
        e = -1;
      }
      if (e >= 0) atomicAdd(p.refs + e, 1);
      to[j] = e < 0 ? -1 : e;  // a page that a window left behind stays absent
    }
    if (threadIdx.x == 0) {
      if (plan.x >= 0) to[whole] = plan.x;
      p.lens[child] = len;
    }
  } else if (plan.x >= 0) {
    const int src = from[whole];
    if (!in_pool(src, p.num_pages)) {
      if (threadIdx.x == 0) report(p.err, DSA_DEVERR_SLOT);
      return;
    }
    copy_page_chunk(cs, blockIdx.y, src, plan.x, blockIdx.x - 1);
  }
}

// ---------------------------------------------------------------- free

// One CTA per listed row.  An entry is taken out of the table by an exchange,
// so a row listed twice still gives every page back once.
__global__ void __launch_bounds__(kCopyThreads)
    dsa_free_kernel(int* refs, int* table, long long bt_stride, int bt_cols, int* lens, int rows,
                    int num_pages, int page_size, const int* which, int window, int sinks,
                    int* err) {
  const int row = __ldg(which + blockIdx.x);
  if (row < 0 || row >= rows) {
    if (threadIdx.x == 0) report(err, DSA_DEVERR_ROW);
    return;
  }
  const int len = lens[row];
  long long blocks = len > 0 ? (static_cast<long long>(len) + page_size - 1) / page_size : 0;
  if (len < 0 || blocks > bt_cols) {
    if (threadIdx.x == 0) report(err, DSA_DEVERR_ROW);
    blocks = blocks < bt_cols ? blocks : bt_cols;
  }
  int first = 0, last = static_cast<int>(blocks);
  if (window > 0) {  // the pages with neither a sink nor one of the last `window` tokens
    first = static_cast<int>((static_cast<long long>(sinks) + page_size - 1) / page_size);
    const int gone = len > window ? (len - window) / page_size : 0;
    last = gone < last ? gone : last;
  }
  int* entry = table + row * bt_stride;
  for (int j = first + threadIdx.x; j < last; j += kCopyThreads) {
    if (entry[j] < 0) continue;
    const int e = atomicExch(entry + j, -1);
    if (e < 0) continue;
    if (e >= num_pages) {
      report(err, DSA_DEVERR_SLOT);
    } else if (atomicSub(refs + e, 1) <= 0) {
      atomicAdd(refs + e, 1);
      report(err, DSA_DEVERR_REFS);
    }
  }
  if (window == 0) {
    __syncthreads();  // every thread has read the length
    if (threadIdx.x == 0) lens[row] = 0;
  }
}

// ---------------------------------------------------------------- compact

struct CompactParams {
  int* refs;
  int* table;
  const int* lens;
  long long bt_stride;
  int bt_cols, rows, num_pages, page_size;
  int* live;
  int* moves;  // workspace: count, then src[num_pages / 2 + 1], dst[the same], and
               // to[num_pages]: where a page's entries point afterwards, -1 if it was free
  int* err;
};

__host__ __device__ __forceinline__ long long compact_half(long long num_pages) {
  return num_pages / 2 + 1;
}

// One CTA: the live pages at or above the number of live pages, ascending,
// pair with the holes below it, ascending.  The sources are all above that
// border and the targets all below it, so the copies cannot collide.
__global__ void __launch_bounds__(kPlanThreads) dsa_compact_plan_kernel(const CompactParams p) {
  extern __shared__ unsigned used[];  // one bit per page
  __shared__ int part[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int words = (p.num_pages + 31) / 32;
  constexpr int kWarps = kPlanThreads / 32, kUnroll = 8;
  int mine = 0;
  for (int w0 = warp; w0 < words; w0 += kWarps * kUnroll) {
    int r[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int at = (w0 + u * kWarps) * 32 + lane;
      r[u] = at < p.num_pages ? p.refs[at] : 0;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const unsigned bits = __ballot_sync(kFull, r[u] > 0);
      const int w = w0 + u * kWarps;
      if (lane == 0 && w < words) {
        used[w] = bits;
        mine += __popc(bits);
      }
    }
  }
  int live = 0;
  block_scan(mine, part, &live);  // its barriers also publish used[]

  // this thread's run of words; `below` masks the pages under the border
  const int per = (words + kPlanThreads - 1) / kPlanThreads;
  const int w_begin = min(static_cast<int>(threadIdx.x) * per, words);
  const int w_end = min(w_begin + per, words);
  auto below = [&](int w) {
    const int n = live - 32 * w;
    return n >= 32 ? kFull : n <= 0 ? 0u : (1u << n) - 1u;
  };
  int holes = 0, movers = 0;
  for (int w = w_begin; w < w_end; ++w) {
    holes += __popc(~used[w] & below(w));
    movers += __popc(used[w] & ~below(w));
  }
  int count = 0;
  int hole_at = block_scan(holes, part, &count);
  int mover_at = block_scan(movers, part, &count);
  int* src = p.moves + 1;
  int* dst = src + compact_half(p.num_pages);
  int* to = dst + compact_half(p.num_pages);
  for (int w = w_begin; w < w_end; ++w) {
    for (unsigned b = ~used[w] & below(w); b; b &= b - 1) dst[hole_at++] = 32 * w + __ffs(b) - 1;
    for (unsigned b = used[w] & ~below(w); b; b &= b - 1) src[mover_at++] = 32 * w + __ffs(b) - 1;
  }
  __syncthreads();
  for (int page = threadIdx.x; page < p.num_pages; page += kPlanThreads) {
    const bool in_use = used[page >> 5] >> (page & 31) & 1;
    if (!in_use || page < live) to[page] = in_use ? page : -1;
  }
  for (int k = threadIdx.x; k < count; k += kPlanThreads) {
    const int s = src[k], d = dst[k];
    to[s] = d;
    p.refs[d] = p.refs[s];
    p.refs[s] = 0;
  }
  if (threadIdx.x == 0) {
    p.moves[0] = count;
    *p.live = live;
  }
}

// blockIdx.y < n_caches: the moves of cache y, chunk z, moves x, x + gridDim.x,
// ...; blockIdx.y == n_caches: the block table's entries.
__global__ void __launch_bounds__(kCopyThreads)
    dsa_compact_kernel(const __grid_constant__ Caches cs, int n_caches, const CompactParams p) {
  grid_dependency_wait();
  const int* src = p.moves + 1;
  const int* dst = src + compact_half(p.num_pages);
  const int* to = dst + compact_half(p.num_pages);
  if (static_cast<int>(blockIdx.y) < n_caches) {
    const int count = p.moves[0];
    for (int k = blockIdx.x; k < count; k += gridDim.x)
      copy_page_chunk(cs, blockIdx.y, src[k], dst[k], blockIdx.z);
    return;
  }
  if (blockIdx.z != 0) return;
  for (int row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const int len = p.lens[row];
    long long blocks = len > 0 ? (static_cast<long long>(len) + p.page_size - 1) / p.page_size : 0;
    if (len < 0 || blocks > p.bt_cols) {
      if (threadIdx.x == 0) report(p.err, DSA_DEVERR_ROW);
      blocks = blocks < p.bt_cols ? blocks : p.bt_cols;
    }
    int* entry = p.table + row * p.bt_stride;
    for (int j = threadIdx.x; j < blocks; j += kCopyThreads) {
      const int e = entry[j];
      if (e < 0) continue;
      if (e >= p.num_pages) {
        report(p.err, DSA_DEVERR_SLOT);
        continue;
      }
      const int moved = to[e];
      // an entry that held a free page: another row's page may be there by now
      if (moved < 0) report(p.err, DSA_DEVERR_REFS);
      if (moved != e) entry[j] = moved;
    }
  }
}

// ---------------------------------------------------------------- host side

bool misaligned(const void* ptr, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
}

// Fills `out` and the largest page's number of kCopyBytes pieces.
dsa_status read_caches(void* const* caches, const int64_t* page_bytes, int32_t n_caches,
                       int64_t num_pages, Caches* out, int* chunks) {
  if (n_caches < 0 || n_caches > kMaxCaches || num_pages < 1 || num_pages > 0x7fffffffLL)
    return DSA_ERR_SHAPE;
  if (n_caches > 0 && (!caches || !page_bytes)) return DSA_ERR_NULL;
  *chunks = 0;
  for (int c = 0; c < n_caches; ++c) {
    if (!caches[c]) return DSA_ERR_NULL;
    if (page_bytes[c] < 1 || page_bytes[c] > (1LL << 30)) return DSA_ERR_SHAPE;
    if (misaligned(caches[c], 4) || page_bytes[c] % 4) return DSA_ERR_ALIGN;
    out->base[c] = static_cast<char*>(caches[c]);
    out->page_bytes[c] = page_bytes[c];
    const int k = static_cast<int>((page_bytes[c] + kCopyBytes - 1) / kCopyBytes);
    *chunks = k > *chunks ? k : *chunks;
  }
  return DSA_OK;
}

dsa_status check_tables(const int32_t* page_refs, const int32_t* block_table, int32_t bt_cols,
                        int64_t bt_stride, const int32_t* context_lens, int32_t rows,
                        int32_t page_size) {
  if (rows < 0 || bt_cols < 0 || bt_stride < bt_cols || page_size < 1) return DSA_ERR_SHAPE;
  if (!page_refs || !block_table || !context_lens) return DSA_ERR_NULL;
  if (misaligned(page_refs, 4) || misaligned(block_table, 4) || misaligned(context_lens, 4))
    return DSA_ERR_ALIGN;
  return DSA_OK;
}

// The launch of a call's second kernel, which waits for the first one's memory
// before it reads anything.  The first does not announce it early, so what the
// attribute may overlap is the first kernel's very end.
template <class... P, class... A>
cudaError_t launch_second(void (*k)(P...), dim3 grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

std::mutex g_compact_mu;
bool g_compact_ready[64];

// Once per device: the plan's bits may take 128 KB of shared memory.
cudaError_t prepare_compact() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_compact_mu);
  if (g_compact_ready[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(dsa_compact_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMaxCompactPages / 8);
  g_compact_ready[dev] = e == cudaSuccess;
  return e;
}

}  // namespace

extern "C" {

dsa_status dsa_cache_copy_pages(void* const* caches, const int64_t* page_bytes, int32_t n_caches,
                                int64_t num_pages, const int32_t* src_pages,
                                const int32_t* dst_pages, int32_t n, uint32_t flags,
                                int32_t* err_flags, void* stream) {
  Caches cs;
  int chunks = 0;
  const dsa_status st = read_caches(caches, page_bytes, n_caches, num_pages, &cs, &chunks);
  if (st != DSA_OK) return st;
  if (n < 0) return DSA_ERR_SHAPE;
  if (flags) return DSA_ERR_UNSUPPORTED;
  if (n == 0 || n_caches == 0) return DSA_OK;
  if (!src_pages || !dst_pages) return DSA_ERR_NULL;
  if (misaligned(src_pages, 4) || misaligned(dst_pages, 4) || misaligned(err_flags, 4))
    return DSA_ERR_ALIGN;
  const dim3 grid(static_cast<unsigned>(n), static_cast<unsigned>(n_caches),
                  static_cast<unsigned>(chunks));
  dsa_copy_pages_kernel<<<grid, kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      cs, static_cast<int>(num_pages), src_pages, dst_pages, err_flags);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}

size_t dsa_cache_fork_workspace_bytes(int32_t n) {
  return n > 0 ? static_cast<size_t>(n) * sizeof(int2) : 0;
}

dsa_status dsa_cache_fork(void* const* caches, const int64_t* page_bytes, int32_t n_caches,
                          int64_t num_pages, int32_t* page_refs, int32_t* block_table,
                          int32_t bt_cols, int64_t bt_stride, int32_t* context_lens, int32_t rows,
                          int32_t page_size, const int32_t* parents, const int32_t* children,
                          int32_t n, uint32_t flags, void* workspace, size_t workspace_bytes,
                          int32_t* err_flags, void* stream) {
  Caches cs;
  int chunks = 0;
  dsa_status st = read_caches(caches, page_bytes, n_caches, num_pages, &cs, &chunks);
  if (st != DSA_OK) return st;
  if (n < 0 || n > kMaxForks) return DSA_ERR_SHAPE;
  if (flags) return DSA_ERR_UNSUPPORTED;
  if (n == 0) return DSA_OK;
  st = check_tables(page_refs, block_table, bt_cols, bt_stride, context_lens, rows, page_size);
  if (st != DSA_OK) return st;
  if (!parents || !children || !workspace) return DSA_ERR_NULL;
  if (misaligned(parents, 4) || misaligned(children, 4) || misaligned(workspace, 8) ||
      misaligned(err_flags, 4))
    return DSA_ERR_ALIGN;
  if (workspace_bytes < dsa_cache_fork_workspace_bytes(n)) return DSA_ERR_SHAPE;
  ForkParams p = {};
  p.refs = page_refs;
  p.table = block_table;
  p.lens = context_lens;
  p.parents = parents;
  p.children = children;
  p.plan = static_cast<int2*>(workspace);
  p.bt_stride = bt_stride;
  p.bt_cols = bt_cols;
  p.rows = rows;
  p.num_pages = static_cast<int>(num_pages);
  p.page_size = page_size;
  p.n = n;
  p.err = err_flags;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  dsa_fork_plan_kernel<<<1, kPlanThreads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_LAUNCH;
  const dim3 grid(static_cast<unsigned>(1 + chunks), static_cast<unsigned>(n_caches ? n_caches : 1),
                  static_cast<unsigned>(n));
  return launch_second(dsa_fork_kernel, grid, kCopyThreads, s, cs, p) == cudaSuccess
             ? DSA_OK : DSA_ERR_LAUNCH;
}

dsa_status dsa_cache_free(int64_t num_pages, int32_t* page_refs, int32_t* block_table,
                          int32_t bt_cols, int64_t bt_stride, int32_t* context_lens, int32_t rows,
                          int32_t page_size, const int32_t* which, int32_t n, int32_t window,
                          int32_t sinks, uint32_t flags, int32_t* err_flags, void* stream) {
  if (num_pages < 1 || num_pages > 0x7fffffffLL || n < 0 || window < 0 || sinks < 0)
    return DSA_ERR_SHAPE;
  if (flags) return DSA_ERR_UNSUPPORTED;
  if (n == 0) return DSA_OK;
  const dsa_status st =
      check_tables(page_refs, block_table, bt_cols, bt_stride, context_lens, rows, page_size);
  if (st != DSA_OK) return st;
  if (!which) return DSA_ERR_NULL;
  if (misaligned(which, 4) || misaligned(err_flags, 4)) return DSA_ERR_ALIGN;
  dsa_free_kernel<<<static_cast<unsigned>(n), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      page_refs, block_table, bt_stride, bt_cols, context_lens, rows, static_cast<int>(num_pages),
      page_size, which, window, sinks, err_flags);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}

size_t dsa_cache_compact_workspace_bytes(int64_t num_pages) {
  return num_pages > 0
             ? static_cast<size_t>(1 + 2 * compact_half(num_pages) + num_pages) * sizeof(int)
             : 0;
}

dsa_status dsa_cache_compact(void* const* caches, const int64_t* page_bytes, int32_t n_caches,
                             int64_t num_pages, int32_t* page_refs, int32_t* block_table,
                             int32_t bt_cols, int64_t bt_stride, const int32_t* context_lens,
                             int32_t rows, int32_t page_size, int32_t* live_pages, uint32_t flags,
                             void* workspace, size_t workspace_bytes, int32_t* err_flags,
                             void* stream) {
  Caches cs;
  int chunks = 0;
  dsa_status st = read_caches(caches, page_bytes, n_caches, num_pages, &cs, &chunks);
  if (st != DSA_OK) return st;
  if (num_pages > kMaxCompactPages) return DSA_ERR_SHAPE;
  if (flags) return DSA_ERR_UNSUPPORTED;
  st = check_tables(page_refs, block_table, bt_cols, bt_stride, context_lens, rows, page_size);
  if (st != DSA_OK) return st;
  if (!live_pages || !workspace) return DSA_ERR_NULL;
  if (misaligned(live_pages, 4) || misaligned(workspace, 4) || misaligned(err_flags, 4))
    return DSA_ERR_ALIGN;
  if (workspace_bytes < dsa_cache_compact_workspace_bytes(num_pages)) return DSA_ERR_SHAPE;
  if (prepare_compact() != cudaSuccess) return DSA_ERR_LAUNCH;
  CompactParams p = {};
  p.refs = page_refs;
  p.table = block_table;
  p.lens = context_lens;
  p.bt_stride = bt_stride;
  p.bt_cols = bt_cols;
  p.rows = rows;
  p.num_pages = static_cast<int>(num_pages);
  p.page_size = page_size;
  p.live = live_pages;
  p.moves = static_cast<int*>(workspace);
  p.err = err_flags;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = static_cast<size_t>((num_pages + 31) / 32) * sizeof(unsigned);
  dsa_compact_plan_kernel<<<1, kPlanThreads, smem, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_LAUNCH;
  // enough CTAs for several waves; the moves are taken with the grid's stride
  const long long per_move = static_cast<long long>(n_caches + 1) * (chunks ? chunks : 1);
  long long gx = 16384 / per_move;
  const long long most = num_pages / 2 > rows ? num_pages / 2 : rows;
  gx = gx > most ? most : gx;
  gx = gx < 1 ? 1 : gx;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(n_caches + 1),
                  static_cast<unsigned>(chunks ? chunks : 1));
  return launch_second(dsa_compact_kernel, grid, kCopyThreads, s, cs, static_cast<int>(n_caches), p)
             == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}

}  // extern "C"
