// The accepted ones of a row's drafted tokens kept: their entries move to the
// front of the drafts' place in every cache, the row's length shrinks to them,
// and the pages behind it go back to the pool.
//
// A row of length L whose last d tokens were drafts has them at tokens
// [L - d, L); with the accepted ones at a_0 < a_1 < ... among them, entry
// L - d + a_j moves to token L - d + j.  As a_j >= j, an entry's new place is
// the old one of an earlier entry of the list or of none: each byte column is
// moved by one thread, in the order of the list, and no copy is needed between.
//
// A cache is described by the addresses of its entries: token t of page p at
// base + p * page + t * token + h * head for each of its heads, `bytes` each.
//
// Bound: the moved bytes where rows and layers are many, two launches and their
// chains of dependent reads (row, list, table, entry) where they are few.
#include <cuda_runtime.h>

#include <cstdint>

#include "dsa_common.cuh"
#include "dsa_prep.h"

namespace {

using namespace dsa_dev;

constexpr int kMaxViews = DSA_MAX_VIEWS;
constexpr int kThreads = 128;
constexpr int kStep = 128;  // entries whose addresses a CTA has in shared memory
constexpr int kBatch = 4;   // entries that a thread has in flight

struct Views {
  char* base[kMaxViews];
  long long page[kMaxViews], token[kMaxViews], head[kMaxViews];  // strides in bytes
  int heads[kMaxViews], bytes[kMaxViews];
};

struct KeepParams {
  int* refs;
  int* table;
  int* lens;
  const int *which, *drafted, *kept, *n_kept;
  long long bt_stride, kept_stride;
  int bt_cols, rows, num_pages, page_size, n, max_kept;
  int* err;
};

__device__ __forceinline__ void report(int* err, int bit) {
  if (err) atomicOr(err, bit);
}

struct Kept {
  int row, before, count, length;  // the row's length before the drafts, and with them
};

// Entry i of the list; false if it may not be carried out.  A whole CTA calls it.
__device__ __forceinline__ bool read_kept(const KeepParams& p, int i, Kept& k) {
  k.row = __ldg(p.which + i);
  const int d = __ldg(p.drafted + i);
  k.count = __ldg(p.n_kept + i);
  const int* list = p.kept + i * p.kept_stride;
  bool bad = k.row < 0 || k.row >= p.rows || d < 0 || k.count < 0 || k.count > p.max_kept ||
             k.count > d;
  if (!bad) {
    k.length = p.lens[k.row];
    k.before = k.length - d;
    bad = k.before < 0 ||
          (static_cast<long long>(k.length) + p.page_size - 1) / p.page_size > p.bt_cols;
    for (int j = threadIdx.x; j < k.count; j += kThreads) {
      const int a = __ldg(list + j);
      bad = bad || a >= d || a <= (j > 0 ? __ldg(list + j - 1) : -1);
    }
    for (int j = threadIdx.x; j < i; j += kThreads)  // a row named before
      bad = bad || __ldg(p.which + j) == k.row;
  }
  return !__syncthreads_or(bad);
}

template <class V>
__device__ __forceinline__ void move_columns(const Views& vs, int v, const longlong2* at, int n) {
  const int pieces = vs.bytes[v] / static_cast<int>(sizeof(V));  // of a head
  const int columns = vs.heads[v] * pieces;
  for (int c = threadIdx.x; c < columns; c += kThreads) {
    const int h = c / pieces;
    char* const base = vs.base[v] + h * vs.head[v] + (c - h * pieces) * sizeof(V);
    for (int j = 0; j < n; j += kBatch) {
      V x[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j + b < n && at[j + b].x >= 0) x[b] = *reinterpret_cast<const V*>(base + at[j + b].x);
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (j + b < n && at[j + b].x >= 0) *reinterpret_cast<V*>(base + at[j + b].y) = x[b];
    }
  }
}

// blockIdx.x: the cache; blockIdx.y: the entry of the list.
__global__ void __launch_bounds__(kThreads)
    dsa_cache_keep_kernel(const __grid_constant__ Views vs, const KeepParams p) {
  __shared__ longlong2 at[kStep];  // from and to, in bytes; from < 0: not moved
  const int v = blockIdx.x;
  Kept k;
  if (!read_kept(p, blockIdx.y, k)) return;
  const int* list = p.kept + blockIdx.y * p.kept_stride;
  const int* table = p.table + k.row * p.bt_stride;
  for (int j0 = 0; j0 < k.count; j0 += kStep) {
    const int n = min(kStep, k.count - j0);
    __syncthreads();  // the step before is done with `at`
    bool moves = false;
    if (static_cast<int>(threadIdx.x) < n) {
      const int j = j0 + threadIdx.x;
      const int a = __ldg(list + j);
      longlong2 x = make_longlong2(-1, -1);
      if (a != j) {
        const int from = k.before + a, to = k.before + j;
        const int fp = table[from / p.page_size], tp = table[to / p.page_size];
        if (fp < 0 || fp >= p.num_pages || tp < 0 || tp >= p.num_pages) {
          report(p.err, DSA_DEVERR_SLOT);
        } else {
          x.x = fp * vs.page[v] + from % p.page_size * vs.token[v];
          x.y = tp * vs.page[v] + to % p.page_size * vs.token[v];
          moves = true;
        }
      }
      at[threadIdx.x] = x;
    }
    if (!__syncthreads_or(moves)) continue;
    const long long bits = reinterpret_cast<long long>(vs.base[v]) | vs.page[v] | vs.token[v] |
                           vs.head[v] | vs.bytes[v];
    if ((bits & 15) == 0)
      move_columns<uint4>(vs, v, at, n);
    else
      move_columns<uint32_t>(vs, v, at, n);
  }
}

// One CTA per entry of the list: the row's length, and its pages behind that.
__global__ void __launch_bounds__(kThreads) dsa_cache_keep_tables_kernel(const KeepParams p) {
  grid_dependency_wait();
  Kept k;
  if (!read_kept(p, blockIdx.x, k)) {
    if (threadIdx.x == 0) report(p.err, DSA_DEVERR_ROW);
    return;
  }
  const int length = k.before + k.count;
  auto blocks = [&](int tokens) {
    return static_cast<int>((static_cast<long long>(tokens) + p.page_size - 1) / p.page_size);
  };
  int* entry = p.table + k.row * p.bt_stride;
  for (int j = blocks(length) + threadIdx.x; j < blocks(k.length); j += kThreads) {
    const int e = entry[j];
    if (e < 0) continue;
    entry[j] = -1;
    if (e >= p.num_pages) {
      report(p.err, DSA_DEVERR_SLOT);
    } else if (atomicSub(p.refs + e, 1) <= 0) {
      atomicAdd(p.refs + e, 1);
      report(p.err, DSA_DEVERR_REFS);
    }
  }
  if (threadIdx.x == 0) p.lens[k.row] = length;  // read by all before read_kept's barrier
}

bool misaligned(const void* ptr, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
}

// views[i] as page, token and head stride, heads and bytes; strides of one entry
// are never used and become 0.
dsa_status read_views(void* const* bases, const int64_t* shapes, int32_t n_views,
                      int64_t num_pages, int32_t page_size, Views* out) {
  if (n_views < 0 || n_views > kMaxViews || num_pages < 1 || num_pages > 0x7fffffffLL ||
      page_size < 1)
    return DSA_ERR_SHAPE;
  if (n_views > 0 && (!bases || !shapes)) return DSA_ERR_NULL;
  for (int i = 0; i < n_views; ++i) {
    const int64_t* s = shapes + 5 * i;
    if (!bases[i]) return DSA_ERR_NULL;
    if (s[3] < 1 || s[4] < 1 || s[3] > 0x7fffffffLL || s[4] > 0x7fffffffLL ||
        static_cast<__int128>(s[3]) * s[4] > 0x7fffffffLL)
      return DSA_ERR_SHAPE;
    const int64_t extent[3] = {num_pages, page_size, s[3]};
    int64_t stride[3];
    for (int d = 0; d < 3; ++d) {
      stride[d] = extent[d] > 1 ? s[d] : 0;
      if (extent[d] > 1 && (s[d] < s[4] || s[d] >= (1LL << 40))) return DSA_ERR_SHAPE;
      if (stride[d] % 4) return DSA_ERR_ALIGN;
    }
    if (misaligned(bases[i], 4) || s[4] % 4) return DSA_ERR_ALIGN;
    out->base[i] = static_cast<char*>(bases[i]);
    out->page[i] = stride[0];
    out->token[i] = stride[1];
    out->head[i] = stride[2];
    out->heads[i] = static_cast<int>(s[3]);
    out->bytes[i] = static_cast<int>(s[4]);
  }
  return DSA_OK;
}

}  // namespace

extern "C" dsa_status dsa_cache_keep(
    void* const* bases, const int64_t* shapes, int32_t n_views, int64_t num_pages,
    int32_t* page_refs, int32_t* block_table, int32_t bt_cols, int64_t bt_stride,
    int32_t* context_lens, int32_t rows, int32_t page_size, const int32_t* which,
    const int32_t* drafted, const int32_t* kept, int64_t kept_stride, int32_t max_kept,
    const int32_t* n_kept, int32_t n, uint32_t flags, int32_t* err_flags, void* stream) {
  Views vs;
  const dsa_status st = read_views(bases, shapes, n_views, num_pages, page_size, &vs);
  if (st != DSA_OK) return st;
  if (n < 0 || n > DSA_MAX_KEEPS || max_kept < 0 || kept_stride < max_kept || rows < 0 ||
      bt_cols < 0 || bt_stride < bt_cols)
    return DSA_ERR_SHAPE;
  if (flags) return DSA_ERR_UNSUPPORTED;
  if (n == 0) return DSA_OK;
  if (!page_refs || !block_table || !context_lens || !which || !drafted || !n_kept ||
      (!kept && max_kept > 0))
    return DSA_ERR_NULL;
  if (misaligned(page_refs, 4) || misaligned(block_table, 4) || misaligned(context_lens, 4) ||
      misaligned(which, 4) || misaligned(drafted, 4) || misaligned(kept, 4) ||
      misaligned(n_kept, 4) || misaligned(err_flags, 4))
    return DSA_ERR_ALIGN;
  KeepParams p = {};
  p.refs = page_refs;
  p.table = block_table;
  p.lens = context_lens;
  p.which = which;
  p.drafted = drafted;
  p.kept = kept;
  p.n_kept = n_kept;
  p.bt_stride = bt_stride;
  p.kept_stride = kept_stride;
  p.bt_cols = bt_cols;
  p.rows = rows;
  p.num_pages = static_cast<int>(num_pages);
  p.page_size = page_size;
  p.n = n;
  p.max_kept = max_kept;
  p.err = err_flags;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (n_views > 0 && max_kept > 0) {
    const dim3 grid(static_cast<unsigned>(n_views), static_cast<unsigned>(n));
    dsa_cache_keep_kernel<<<grid, kThreads, 0, s>>>(vs, p);
    if (cudaGetLastError() != cudaSuccess) return DSA_ERR_LAUNCH;
  }
  // the tables change only once every entry has moved
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = n_views > 0 && max_kept > 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, dsa_cache_keep_tables_kernel, p) == cudaSuccess ? DSA_OK
                                                                                  : DSA_ERR_LAUNCH;
}
