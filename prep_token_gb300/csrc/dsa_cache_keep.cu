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
// The first kernel, a CTA to a row, checks the list and the counts of the pages
// that entries move to, and writes where they move to the workspace.  The second,
// a CTA to a row and a cache, moves: what it waits for is one read of the workspace
// and one of the entries.  One CTA more per row changes its table, counts and
// length: behind the first kernel, so that no row's check depends on which pages
// another row of the list has given back by then, and none is found its own while
// that row's entries still move.  Without caches the first kernel does it.
//
// Bound: the moved bytes where rows and layers are many, two launches and their
// chains of dependent reads where they are few.  Measured: up to 8 of up to 32
// drafts of 48 rows in the K and V caches of 40 layers (2 KB entries, 59 MB) 15.8 us,
// of which the second kernel's 3888 CTAs, two rounds of two round trips each, take 12
// (59 MB at 6.78 TB/s: 8.7); one row in 21 layers 4.3 us.  With the table changed in
// the first kernel 16.3 and 4.5.  One launch, a cluster of CTAs to a row with the
// tables changed behind its barrier, took 23 and 6 us; a kernel that read the lists per
// cache 17.  Moves read by every thread instead of through
// shared memory: the same time at twice the registers.
#include <cuda_runtime.h>

#include <cstdint>

#include "dsa_common.cuh"
#include "dsa_prep.h"
#include "dsa_rows.cuh"

namespace {

using namespace dsa_dev;

constexpr int kThreads = 128;
constexpr int kBatch = 4;  // entries that a thread has in flight

struct View {
  char* base;
  long long page, token, head;  // strides in bytes
  int heads, bytes;
};
// CAP: what a launch carries for; a call of few caches takes the small one.
template <int CAP>
struct Views {
  View v[CAP];
};
constexpr int kFewViews = 64;

struct KeepParams {
  int* refs;
  int* table;
  int* lens;
  const int *which, *drafted, *kept, *n_kept;
  long long bt_stride, kept_stride;
  int bt_cols, rows, num_pages, page_size, n, max_kept;
  int4* moves;  // workspace [n, max_kept]: page and token of an entry and of its new place; page
                // -1: none
  int* runs;    // workspace [n]: how many moves a row has; -1: it stays as it is
  int* err;
};

__device__ __forceinline__ void report(int* err, int bit) {
  if (err) atomicOr(err, bit);
}

// A row's length becomes `shorter`, and its pages behind that go back; all threads of a
// CTA call it.
__device__ __forceinline__ void shrink(const KeepParams& p, int row, int length, int shorter) {
  int* const entry = p.table + row * p.bt_stride;
  auto blocks = [&](int tokens) {
    return static_cast<int>((static_cast<long long>(tokens) + p.page_size - 1) / p.page_size);
  };
  for (int j = blocks(shorter) + threadIdx.x; j < blocks(length); j += kThreads) {
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
  if (threadIdx.x == 0) p.lens[row] = shorter;
}

// One CTA per entry of the list.  MOVES: the second kernel follows; else there is
// nothing to move, and the row shrinks here.
template <bool MOVES>
__global__ void __launch_bounds__(kThreads) dsa_cache_keep_plan_kernel(const KeepParams p) {
  const int i = blockIdx.x;
  if (MOVES) grid_launch_dependents();  // the second kernel's CTAs start, and wait for this one's end
  const int row = __ldg(p.which + i), d = __ldg(p.drafted + i), count = __ldg(p.n_kept + i);
  const int* const list = p.kept + i * p.kept_stride;
  bool bad = row < 0 || row >= p.rows || d < 0 || count < 0 || count > p.max_kept || count > d;
  int length = 0;
  if (!bad) {
    length = p.lens[row];
    bad = length < d ||
          (static_cast<long long>(length) + p.page_size - 1) / p.page_size > p.bt_cols;
    for (int j = threadIdx.x; j < count; j += kThreads) {
      const int a = __ldg(list + j);
      bad = bad || a >= d || a <= (j > 0 ? __ldg(list + j - 1) : -1);
    }
    for (int j = threadIdx.x; j < i; j += kThreads)  // a row named before
      bad = bad || __ldg(p.which + j) == row;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) {
      report(p.err, DSA_DEVERR_ROW);
      if (MOVES) p.runs[i] = -1;
    }
    return;
  }
  const int before = length - d;
  if (!MOVES) {
    shrink(p, row, length, before + count);
    return;
  }
  const int* const entry = p.table + row * p.bt_stride;
  int still = 0;  // entries that stay, all of them in front
  bool shared = false;  // an entry would go to a page that is not the row's own
  int4* const moves = p.moves + static_cast<long long>(i) * p.max_kept;
  for (int j0 = 0; j0 < count; j0 += kThreads) {
    const int j = j0 + threadIdx.x;
    const int a = j < count ? __ldg(list + j) : -1;
    still += __syncthreads_count(j < count && a == j);
    if (j < count && a != j) {
      const int from = before + a, to = before + j;
      const int fp = entry[from / p.page_size], tp = entry[to / p.page_size];
      const bool ok = fp >= 0 && fp < p.num_pages && tp >= 0 && tp < p.num_pages;
      if (!ok)
        report(p.err, DSA_DEVERR_SLOT);
      else
        shared = shared || p.refs[tp] != 1;
      moves[j - still] = make_int4(ok ? fp : -1, from % p.page_size, tp, to % p.page_size);
    }
  }
  shared = __syncthreads_or(shared);
  if (threadIdx.x == 0) {
    if (shared) report(p.err, DSA_DEVERR_REFS);
    p.runs[i] = shared ? -1 : count - still;
  }
}

template <class V>
__device__ __forceinline__ void move_columns(const View& view, const longlong2* at, int n) {
  const int pieces = view.bytes / static_cast<int>(sizeof(V));  // of a head
  const int columns = view.heads * pieces;
  for (int c = threadIdx.x; c < columns; c += kThreads) {
    const int h = c / pieces;
    char* const base = view.base + h * view.head + (c - h * pieces) * sizeof(V);
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

// blockIdx.x: the cache, and behind the caches the row's table; blockIdx.y: the entry
// of the list.  The first moves are read beside their number.
template <int CAP>
__global__ void __launch_bounds__(kThreads)
    dsa_cache_keep_kernel(const __grid_constant__ Views<CAP> vs, const KeepParams p) {
  __shared__ longlong2 at[kThreads];  // from and to, in bytes; from < 0: not moved
  const int i = blockIdx.y;
  if (blockIdx.x + 1 == gridDim.x) {
    // the lists are older than the first kernel, which changes nothing that is read here
    const int row = __ldg(p.which + i), d = __ldg(p.drafted + i), count = __ldg(p.n_kept + i);
    grid_dependency_wait();
    if (p.runs[i] < 0) return;
    const int length = p.lens[row];
    __syncthreads();  // before one thread changes it
    shrink(p, row, length, length - d + count);
    return;
  }
  const View view = vs.v[blockIdx.x];
  const long long bits = reinterpret_cast<long long>(view.base) | view.page | view.token |
                         view.head | view.bytes;
  const int4* const moves = p.moves + static_cast<long long>(i) * p.max_kept;
  grid_dependency_wait();
  const int n = p.runs[i];
  for (int j0 = 0; j0 == 0 || j0 < n; j0 += kThreads) {
    if (j0 > 0) __syncthreads();  // the step before is done with `at`
    const int j = j0 + threadIdx.x;
    if (j < p.max_kept) {
      const int4 m = moves[j];
      at[threadIdx.x] =
          m.x < 0 ? make_longlong2(-1, -1)
                  : make_longlong2(m.x * view.page + m.y * view.token,
                                   m.z * view.page + m.w * view.token);
    }
    __syncthreads();
    if ((bits & 15) == 0)
      move_columns<uint4>(view, at, min(kThreads, n - j0));
    else
      move_columns<uint32_t>(view, at, min(kThreads, n - j0));
  }
}

using dsa_rows::misaligned;

// shapes[5 i ..]: page, token and head stride, heads and bytes; strides of one
// entry are never used and become 0.
template <int CAP>
dsa_status read_views(void* const* bases, const int64_t* shapes, int32_t n_views,
                      int64_t num_pages, int32_t page_size, Views<CAP>* out) {
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
    if (!dsa_rows::rows_apart(s[4], extent, stride)) return DSA_ERR_SHAPE;
    if (misaligned(bases[i], 4) || s[4] % 4) return DSA_ERR_ALIGN;
    out->v[i] = {static_cast<char*>(bases[i]), stride[0], stride[1], stride[2],
                 static_cast<int>(s[3]), static_cast<int>(s[4])};
  }
  return DSA_OK;
}

// The runs in front, 16 bytes aligned behind them the moves.
size_t runs_bytes(int32_t n) { return (static_cast<size_t>(n) * sizeof(int) + 15) / 16 * 16; }

template <int CAP>
dsa_status keep(void* const* bases, const int64_t* shapes, int32_t n_views, int64_t num_pages,
                KeepParams p, bool checked, cudaStream_t s) {
  Views<CAP> vs;
  const dsa_status st = read_views<CAP>(bases, shapes, n_views, num_pages, p.page_size, &vs);
  if (st != DSA_OK || checked) return st;
  const unsigned rows = static_cast<unsigned>(p.n);
  const bool moves = n_views > 0 && p.max_kept > 0;
  if (moves)
    dsa_cache_keep_plan_kernel<true><<<rows, kThreads, 0, s>>>(p);
  else
    dsa_cache_keep_plan_kernel<false><<<rows, kThreads, 0, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return DSA_ERR_LAUNCH;
  if (!moves) return DSA_OK;
  // waits for the first one's memory before it reads anything
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_views) + 1, rows);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, dsa_cache_keep_kernel<CAP>, vs, p);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}

}  // namespace

extern "C" {

size_t dsa_cache_keep_workspace_bytes(int32_t n, int32_t max_kept) {
  if (n < 1 || max_kept < 0) return 0;
  return runs_bytes(n) + static_cast<size_t>(n) * max_kept * sizeof(int4);
}

dsa_status dsa_cache_keep(
    void* const* bases, const int64_t* shapes, int32_t n_views, int64_t num_pages,
    int32_t* page_refs, int32_t* block_table, int32_t bt_cols, int64_t bt_stride,
    int32_t* context_lens, int32_t rows, int32_t page_size, const int32_t* which,
    const int32_t* drafted, const int32_t* kept, int64_t kept_stride, int32_t max_kept,
    const int32_t* n_kept, int32_t n, uint32_t flags, void* workspace, size_t workspace_bytes,
    int32_t* err_flags, void* stream) {
  if (n_views < 0 || n_views > DSA_MAX_VIEWS || num_pages < 1 || num_pages > 0x7fffffffLL ||
      page_size < 1)
    return DSA_ERR_SHAPE;
  if (n_views > 0 && (!bases || !shapes)) return DSA_ERR_NULL;
  KeepParams p = {};
  p.page_size = page_size;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto call = [&](bool checked) {
    return n_views <= kFewViews
               ? keep<kFewViews>(bases, shapes, n_views, num_pages, p, checked, s)
               : keep<DSA_MAX_VIEWS>(bases, shapes, n_views, num_pages, p, checked, s);
  };
  if (n < 0 || n > DSA_MAX_KEEPS || max_kept < 0 || (kept_stride != 0 && kept_stride < max_kept) ||
      rows < 0 || bt_cols < 0 || bt_stride < bt_cols)
    return DSA_ERR_SHAPE;
  if (flags) return DSA_ERR_UNSUPPORTED;
  if (n == 0) return call(true);
  if (!page_refs || !block_table || !context_lens || !which || !drafted || !n_kept ||
      (!kept && max_kept > 0) || !workspace)
    return DSA_ERR_NULL;
  if (misaligned(page_refs, 4) || misaligned(block_table, 4) || misaligned(context_lens, 4) ||
      misaligned(which, 4) || misaligned(drafted, 4) || misaligned(kept, 4) ||
      misaligned(n_kept, 4) || misaligned(workspace, 16) || misaligned(err_flags, 4))
    return DSA_ERR_ALIGN;
  if (workspace_bytes < dsa_cache_keep_workspace_bytes(n, max_kept)) return DSA_ERR_SHAPE;
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
  p.n = n;
  p.max_kept = max_kept;
  p.runs = static_cast<int*>(workspace);
  p.moves = reinterpret_cast<int4*>(static_cast<char*>(workspace) + runs_bytes(n));
  p.err = err_flags;
  return call(false);
}

}  // extern "C"
