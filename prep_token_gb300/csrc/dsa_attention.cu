// Attention of new tokens over a paged K/V cache on the 5th-generation tensor
// cores: a chunk of a prompt, single tokens, or both in one call, over the
// whole context or a sliding window with the first tokens kept visible.
//
// With G = H / Hkv query heads per kv head, query i of sequence b is the token
// at pos = context_lens[b] - n_b + i, and for each of its heads
//   s_j = scale * q . k_j,  out = sum_j e^(s_j) v_j / sum_j e^(s_j),
//   lse = log(sum_j e^(s_j)),
// over the visible keys: j <= pos and (no window, or j > pos - window, or
// j < sinks).  The keys are taken in blocks of 128 with the running maximum m
// and sum l of a softmax, so S never leaves the chip:
//   p_j = 2^(c s_j - c m) with c = scale * log2(e);  O += P V;  l += sum p.
//
// A query tile is 128 rows: floor(128 / G) tokens, their G heads of one kv head
// packed token by token; a single token fills G of them.  A work item is one or
// two query tiles of one sequence, which share the loaded keys (make_plan says
// when two).
//   * warps 0 and 2 load: the query tiles, then per key block the 16 KB units of
//     K (128 keys x 64 dims) and V (8192 / D keys x D dims) into one ring, by
//     4-D TMA boxes of min(page, 64) keys with the 128-byte swizzle; lane l
//     looks up and issues box l of the block.
//   * warp 1 (one lane) issues S = Q K^T (M = N = 128, both operands in shared
//     memory) and O += P V (A = P in TMEM over the columns of S, B = V in
//     shared memory, read MN-major), and commits them to the mbarriers.
//   * one warpgroup per query tile owns one row per thread: S from TMEM, the
//     masks (in blocks at an edge only), the exponentials, P back to TMEM.  m
//     need not be the maximum, only near enough for fp32 and P's type to hold
//     p: the row's first maximum serves until a sum of P passes a limit, so
//     that most blocks form no maximum and rescale nothing.  P is rounded to
//     the values' type for the matrix product (at most 2^-8 of it in bf16,
//     2^-11 in fp16); the sum l takes it unrounded.  In fp16 P, O and l carry a
//     factor of 2^7: a p down to 2^-21 of the largest keeps all its bits.
// An SM holds two query tiles, in one CTA or two: one's softmax runs beside the
// other's products.
//
// Bound, and what was measured (152 SMs, 6.78 TB/s, 1892 TFLOP/s of bf16):
//   * a chunk by the tensor cores, 4 D flops per row and visible key.  A
//     128 x 128 x 16 product with both operands in shared memory takes 105
//     cycles (64 at the nominal rate), with A in TMEM 75: a block of a tile 1445
//     for D = 128, where the nominal rate has 1024.  2048 tokens over 16384, 64
//     heads: 665 us, 1550 TFLOP/s.  For D = 64 the softmax is as long as the
//     products, and the hand-overs between them count: 520 us.
//   * single tokens by the cache's bytes: 64 over 8192, 8 kv heads: 325 us, 6.6
//     TB/s.  About 12 us of a call are its start, its first loads and the second
//     kernel: 1 token over 1000 takes 13 us, 2 over 65536 55 us (40 at 6.78 TB/s).
//   * short items (a window) by what each begins and ends with, about 5 us of
//     code that the instruction cache does not keep: so code is small before it
//     is unrolled here.
// The key blocks of all items are laid end to end and cut into equal shares, one
// per CTA; an item that a cut divides leaves partial (O, m, l) in the workspace,
// which a second kernel joins in a fixed order.  (make_plan and may_split say when
// CTAs take whole items instead: then in the order of the batch, so that unequal
// ones leave CTAs idle at the end.)
//
// Every wait is bounded in time; TMEM is always released before exit.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "dsa_common.cuh"
#include "dsa_prep.h"

namespace {

using namespace dsa_dev;

constexpr int kRows = 128;          // MMA M: rows of a query tile
constexpr int kKeys = 128;          // keys of a block
constexpr int kUnitBytes = 16384;   // of the K/V ring
constexpr int kSms = 152;
// A CTA works on QT query tiles of 128 rows that share the loaded keys: one
// tile and two CTAs per SM, or two tiles and one CTA.  Either way an SM holds
// 256 rows.
template <int QT>
struct Shape {
  static constexpr int kThreads = (1 + QT) * 128;  // loads, MMA, 2 idle warps; softmax
  // Registers: the launch's share per thread is 128 (two CTAs of 256 threads)
  // or 168 (one of 384); the first warpgroup gives some to the others.  ptxas
  // allots by the launch's share: with one tile it spills 140 (D 128) and 88 (D
  // 64) bytes of a thread, with two none.
  static constexpr int kRegsFew = QT == 1 ? 64 : 88;
  static constexpr int kRegsMany = QT == 1 ? 192 : 208;
  static_assert(kRegsFew + QT * kRegsMany <= (1 + QT) * (QT == 1 ? 128 : 168), "registers");
  static constexpr int kCtas = 2 / QT * kSms;
  static constexpr int kTmemCols = 256 * QT;          // per tile: S / P 128, O D
};
// A half block's sum of P above which a row's reference is renewed.  P in
// bf16 has fp32's range; in fp16 no p may pass 65504.
template <bool BF16>
constexpr float kSumLimit = BF16 ? 0x1p20f : 0x1p15f;
constexpr float kLn2 = 0.693147180559945309f;

struct AParams {
  const int* block_table;
  const int* query_start;
  const int* context_lens;
  void* out;
  float* lse;
  long long bt_stride, out_stride_t, out_stride_h;
  int num_pages, page, box;  // box: keys per TMA box, min(page, 64)
  int T, B, Hkv, G;
  int q_tokens;     // tokens of a query tile, floor(128 / G)
  int tile_tokens;  // tokens of a work item, QT * q_tokens
  int max_context;
  int window, sinks;  // window 0: none
  float c;            // scale * log2(e)
  int split;          // 1: equal shares of the key blocks; 0: whole items, gridDim.x apart
  int4* meta;         // split: [CTAs] the item that CTA leaves to later ones
  float2* ml;         // split: [2 * CTAs][QT * kRows] (log2 of the scale, l) of a part
  float* part;        // split: [2 * CTAs][QT * kRows][D] O of a part
  int* err;
};

// ---------------------------------------------------------------- PTX wrappers

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// mbar_wait, with probes that the hardware ends early (the softmax and the
// matrix products hand over to each other three times per key block, and a
// thread that asked for a long sleep wakes late) and without a function call,
// across which the registers of a row would have to be saved.
__device__ __forceinline__ bool wait_soon(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  unsigned long long t0 = 0;
  for (unsigned i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n"
        " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    if (ok) return true;
    if (i % 64 == 0) {
      const unsigned long long t = global_ns();
      if (t0 == 0) t0 = t;
      if (*abort_flag || t - t0 > kWaitLimitNs) return false;
    }
  }
}

// Shared-memory matrix descriptor of 128-byte-swizzled rows: 8-row groups of
// 1024 bytes (the stride offset).  `lead` is the distance of 64-element panels
// of an MN-major operand (unused K-major).
// The low word moves with the address, 16 bytes to a step; the high one does not.
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr, uint32_t lead) {
  return ((smem_addr >> 4) & 0x3FFFu) | ((lead >> 4) & 0x3FFFu) << 16;
}
__device__ __forceinline__ uint64_t make_desc(uint32_t lo) {
  constexpr uint32_t hi = (1024 >> 4) | 1u << 14 /* version */ | 2u << 29 /* swizzle */;
  return static_cast<uint64_t>(hi) << 32 | lo;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}"
               : "=r"(is));
  return is != 0;
}

// Instruction descriptor: D fp32, A and B fp16 or bf16, A K-major.
__host__ __device__ constexpr uint32_t mma_idesc(bool bf16, bool b_mn_major, int n) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn_major ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
               ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Nothing may use values that a tcgen05.ld brings before its wait: an empty
// statement that seems to change them keeps the compiler to that order.
template <int N>
__device__ __forceinline__ void tmem_wait_ld(float (&v)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// 32 consecutive fp32 columns of this warp's 32 TMEM lanes; the values may be
// used after tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr) : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr) : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0],"
      " {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
        "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// c + 0 * v for two values of the 16-bit type: NaN where v is not finite.
template <bool BF16>
__device__ __forceinline__ uint32_t fma0(uint32_t v, uint32_t c) {
  uint32_t r;
  if (BF16)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0), "r"(c));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0), "r"(c));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The n lowest of 32 bits.
__device__ __forceinline__ uint32_t below(int n) {
  return n <= 0 ? 0u : n >= 32 ? kFull : (1u << n) - 1u;
}

// ---------------------------------------------------------------- work items

// One work item of a sequence and the key blocks that some row of it sees.
struct Tile {
  int token0, tokens;  // in q; tokens of the tile
  int pos0;            // position of its first token
  int hi, lo;          // keys seen by some row: [lo, hi) and [0, min(sinks, hi))
  int sink_blocks, main_block, blocks;  // blocks [0, sink_blocks), then from main_block on
};

__device__ __forceinline__ Tile make_tile(const AParams& p, int q0, int n, int ctx, int t) {
  Tile r;
  const int i0 = t * p.tile_tokens;
  r.token0 = q0 + i0;
  r.tokens = min(p.tile_tokens, n - i0);
  r.pos0 = ctx - n + i0;
  r.hi = max(0, r.pos0 + r.tokens);
  r.lo = p.window ? max(0, r.pos0 - p.window + 1) : 0;
  r.main_block = r.lo / kKeys;
  r.sink_blocks = min((min(p.sinks, r.hi) + kKeys - 1) / kKeys, r.main_block);
  // a tile that sees nothing still has one block, all masked: its rows are 0
  r.blocks = max(1, r.sink_blocks + (r.hi + kKeys - 1) / kKeys - r.main_block);
  return r;
}

struct Seq {
  int q0, n, ctx, tiles;
};

// Sequence b, its numbers held to the tensors' sizes.
__device__ __forceinline__ Seq load_seq(const AParams& p, int b) {
  Seq s;
  s.q0 = max(0, min(__ldg(p.query_start + b), p.T));
  s.n = max(0, min(__ldg(p.query_start + b + 1), p.T) - s.q0);
  s.ctx = max(0, min(__ldg(p.context_lens + b), p.max_context));
  s.tiles = (s.n + p.tile_tokens - 1) / p.tile_tokens;
  return s;
}

// 64-bit only where it has to be; out of line, as it is long and rarely run.
__device__ __noinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Key blocks of all tiles of a sequence, for one kv head.  A whole warp calls
// it with each lane's own sequence.
__device__ __noinline__ long long seq_blocks(const AParams& p, int n, int ctx, int tiles) {
  const int lane = threadIdx.x & 31;
  long long mine = tiles > 0 ? make_tile(p, 0, n, ctx, 0).blocks : 0;
  for (unsigned todo = __ballot_sync(kFull, tiles > 1); todo; todo &= todo - 1) {
    const int src = __ffs(todo) - 1;
    const int n1 = __shfl_sync(kFull, n, src), ctx1 = __shfl_sync(kFull, ctx, src);
    const int tiles1 = __shfl_sync(kFull, tiles, src);
    long long sum = 0;
#pragma unroll 1
    for (int t = lane; t < tiles1; t += 32) sum += make_tile(p, 0, n1, ctx1, t).blocks;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if (lane == src) mine = sum;
  }
  return mine;
}

__device__ __forceinline__ long long warp_inclusive(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// Split work: key blocks in the order sequence, kv head, tile.  Each of `ctas`
// CTAs takes `each` of them, the first `extra` CTAs one more.
struct Share {
  long long each, extra, begin, end;
};

// A whole warp calls it.
__device__ __forceinline__ Share my_share(const AParams& p) {
  const int lane = threadIdx.x & 31;
  long long total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    Seq s = {0, 0, 0, 0};
    if (b0 + lane < p.B) s = load_seq(p, b0 + lane);
    total += seq_blocks(p, s.n, s.ctx, s.tiles);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(kFull, total, o);
  total *= p.Hkv;
  Share r;
  r.each = divide(total, gridDim.x);
  r.extra = total - r.each * gridDim.x;
  const long long g = blockIdx.x;
  r.begin = g * r.each + min(g, r.extra);
  r.end = r.begin + r.each + (g < r.extra ? 1 : 0);
  return r;
}

// The CTA that has key block `at`.
__device__ __forceinline__ int cta_of(const Share& s, long long at) {
  const long long longer = s.extra * (s.each + 1);  // blocks of the CTAs with one more
  return static_cast<int>(at < longer ? divide(at, s.each + 1)
                                      : s.extra + divide(at - longer, s.each));
}

// Where a CTA is in its work: the tile, and the key blocks [begin, end) of it.
struct Cursor {
  int b, h, t;
  Seq s;
  Tile tile;
  int begin, end;
  long long left;  // split: key blocks after this segment
};

__device__ __forceinline__ void take_tile(const AParams& p, Cursor& c, int begin, long long budget) {
  c.tile = make_tile(p, c.s.q0, c.s.n, c.s.ctx, c.t);
  c.begin = begin;
  c.end = static_cast<int>(min(static_cast<long long>(c.tile.blocks), begin + budget));
  c.left = budget - (c.end - c.begin);
}

// Puts the cursor at key block `want` (split; `budget` of them are taken) or at
// item `want`.  A whole warp calls it; every lane gets the same.
__device__ __forceinline__ bool seek(const AParams& p, Cursor& c, long long want, long long budget) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    Seq s = {0, 0, 0, 0};
    if (b0 + lane < p.B) s = load_seq(p, b0 + lane);
    const long long per_head = p.split ? seq_blocks(p, s.n, s.ctx, s.tiles) : s.tiles;
    const long long upto = before + warp_inclusive(per_head * p.Hkv);
    const unsigned past = __ballot_sync(kFull, upto > want);
    if (past) {
      const int src = __ffs(past) - 1;
      const long long one = __shfl_sync(kFull, per_head, src);
      const long long rest = want - (__shfl_sync(kFull, upto, src) - one * p.Hkv);
      c.b = b0 + src;
      c.s.q0 = __shfl_sync(kFull, s.q0, src);
      c.s.n = __shfl_sync(kFull, s.n, src);
      c.s.ctx = __shfl_sync(kFull, s.ctx, src);
      c.s.tiles = __shfl_sync(kFull, s.tiles, src);
      c.h = static_cast<int>(divide(rest, one));
      int r = static_cast<int>(rest - c.h * one);
      c.t = c.s.tiles - 1 - r;  // whole items: the last tiles of a chunk see the most keys
      if (p.split) {
        int seen = 0;  // key blocks of the tiles before
#pragma unroll 1
        for (int t0 = 0;; t0 += 32) {
          const int t = t0 + lane;
          const int n = t < c.s.tiles ? make_tile(p, 0, c.s.n, c.s.ctx, t).blocks : 0;
          const int up = seen + static_cast<int>(warp_inclusive(n));
          const unsigned over = __ballot_sync(kFull, up > r);
          if (over) {
            const int at = __ffs(over) - 1;
            c.t = t0 + at;
            r -= __shfl_sync(kFull, up - n, at);
            break;
          }
          seen = __shfl_sync(kFull, up, 31);
        }
      }
      take_tile(p, c, p.split ? r : 0, budget);
      return true;
    }
    before = __shfl_sync(kFull, upto, 31);
  }
  return false;
}

// The next tile, kv head or sequence with tokens, while key blocks are left.
__device__ __forceinline__ bool next_segment(const AParams& p, Cursor& c) {
  if (c.left <= 0) return false;
  if (++c.t == c.s.tiles) {
    c.t = 0;
    if (++c.h == p.Hkv) {
      c.h = 0;
      do {
        if (++c.b >= p.B) return false;
        c.s = load_seq(p, c.b);
      } while (c.s.tiles == 0);
    }
  }
  take_tile(p, c, 0, c.left);
  return true;
}

// ---------------------------------------------------------------- the kernel

// What the load warp tells the others about a segment, in shared memory.
struct Segment {
  int begin, end;  // key blocks of the tile; end -1: there is no more work
  int sink_blocks, main_block, blocks;
  int hi, lo;
  int pos0, tokens, token0, h, b;
  int last_cta;    // of an item that starts here and goes on, else -1
};
// The load warp is at most two segments ahead of the slowest reader: it
// passes on when the last scores of a segment are done, and those of the next
// one wait for the softmax of this one.
constexpr int kSegments = 4;

template <int D, int QT>
struct ASmem {
  static constexpr int kPanels = D / 64;                    // 128-byte panels of a row
  static constexpr int kTileBytes = kRows * D * 2;          // a query tile
  static constexpr int kQBytes = QT * kTileBytes;
  // Places for S in TMEM.  With three for two tiles (where O leaves the room)
  // a tile's next scores are formed while its softmax is still at this block;
  // with one per tile they follow the block's P V.
  static constexpr int kLook = QT == 1 ? 1 : D == 64 ? 3 : 2;
  // two tiles: 2 KB per softmax warp through which rows are turned for stores
  static constexpr int kTurnBytes = QT == 1 ? 0 : 16384;
  // units of the ring: 5 or 6 with two CTAs per SM, 9 or 11 with one
  static constexpr int kStages = ((QT == 1 ? 114688 : 229376) - kQBytes - kTurnBytes) / kUnitBytes;
  static constexpr int kVKeys = kKeys / kPanels;            // keys of a V unit
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffTurn = kOffRing + kStages * kUnitBytes;
  static constexpr int kOffSeg = kOffTurn + kTurnBytes;
  static constexpr int kOffOdd = kOffSeg + kSegments * static_cast<int>(sizeof(Segment));
  static constexpr int kOffBar = kOffOdd + 4 * 4 * 4;
  // barriers: full[S], empty[S], qfull, qempty, drain, segment[4], then per
  // query tile sfull[2], pready[2][2], ohalf, oblock, ofull; checked[4]
  static constexpr int kBars = 2 * kStages + 3 + kSegments + 9 * QT + 4;
  static constexpr int kOffTmem = kOffBar + 8 * kBars;
  static constexpr int kOffAbort = kOffTmem + 4;
  static constexpr int kBytes = kOffAbort + 4;
  static_assert(kBytes <= (QT == 1 ? 115712 : 232448), "shared memory of an SM");
};

// `rows` shared-memory rows of 128 bytes from `at` set to `word` by a warp.
__device__ __forceinline__ void fill_rows(uint32_t at, int rows, uint32_t word) {
#pragma unroll 1
  for (int i = threadIdx.x & 31; i < rows * 8; i += 32)
    asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at + 16 * i), "r"(word)
                 : "memory");
}

template <int D, bool BF16, int QT>
__global__ void __launch_bounds__(Shape<QT>::kThreads, 2 / QT)
    dsa_paged_attention_kernel(const __grid_constant__ CUtensorMap tq,
                               const __grid_constant__ CUtensorMap tk,
                               const __grid_constant__ CUtensorMap tv,
                               const __grid_constant__ AParams p) {
  using L = ASmem<D, QT>;
  constexpr int S = L::kStages;
  constexpr int kP = L::kPanels;
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // the swizzled tiles need this alignment
    if (threadIdx.x == 0 && p.err) atomicOr(p.err, DSA_DEVERR_INTERNAL);
    return;
  }
  const uint32_t bar0 = sbase + L::kOffBar;
  auto full = [&](int s) { return bar0 + 8 * s; };
  auto empty = [&](int s) { return bar0 + 8 * (S + s); };
  const uint32_t qfull = bar0 + 8 * (2 * S), qempty = bar0 + 8 * (2 * S + 1);
  const uint32_t drain = bar0 + 8 * (2 * S + 2);
  auto segment_ready = [&](int i) { return bar0 + 8 * (2 * S + 3 + i % kSegments); };
  constexpr int kB = 2 * S + 3 + kSegments;
  // Of the n-th block.  With three places for S the scores of a tile's next
  // block may be there while some warp of it is still at this one: the others
  // go on, so two blocks take turns at these barriers.
  constexpr int kLook = L::kLook, kTurns = kLook == 3 ? 2 : 1;
  auto turn = [](int n) { return static_cast<uint32_t>(n / kTurns) & 1u; };  // its parity
  auto sfull = [&](int j, int n) { return bar0 + 8 * (kB + 9 * j + n % kTurns); };
  auto pready = [&](int j, int half, int n) {
    return bar0 + 8 * (kB + 2 + 9 * j + 2 * half + n % kTurns);
  };
  // O with the first half of a block's keys; with all; with a segment's last
  auto ohalf = [&](int j) { return bar0 + 8 * (kB + 6 + 9 * j); };
  auto oblock = [&](int j) { return bar0 + 8 * (kB + 7 + 9 * j); };
  auto ofull = [&](int j) { return bar0 + 8 * (kB + 8 + 9 * j); };
  // V of the n-th block at an edge has been looked at; its keys that are odd.
  // The tiles are never four such blocks apart.
  auto checked = [&](int n) { return bar0 + 8 * (kB + 9 * QT + (n & 3)); };
  volatile uint32_t* const odd_keys = reinterpret_cast<volatile uint32_t*>(smem + L::kOffOdd);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
  Segment* const segments = reinterpret_cast<Segment*>(smem + L::kOffSeg);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 32) {
    prefetch_map(&tq);
    prefetch_map(&tk);
    prefetch_map(&tv);
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(qfull, 1);
    mbar_init(qempty, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < kSegments; ++i) mbar_init(segment_ready(i), 1);
    for (int i = 0; i < 4; ++i) mbar_init(checked(i), 4);  // tile 0's warps
    for (int j = 0; j < QT; ++j) {
      for (int n = 0; n < kTurns; ++n) {
        mbar_init(sfull(j, n), 1);
        for (int h = 0; h < 2; ++h) mbar_init(pready(j, h, n), 4);  // the tile's softmax warps
      }
      mbar_init(oblock(j), 1);
      mbar_init(ohalf(j), 1);
      mbar_init(ofull(j), 1);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(sbase + L::kOffTmem), "n"(Shape<QT>::kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(smem + L::kOffTmem);
  auto tmem_s = [&](int i) { return tmem + i * kKeys; };  // the i-th place for S
  auto tmem_o = [&](int j) { return tmem + kLook * kKeys + j * D; };

  grid_dependency_wait();
  grid_launch_dependents();

  auto give_up = [&]() {  // a wait ran out of time
    *abort_flag = 1;
    if (p.err) atomicOr(p.err, DSA_DEVERR_TIMEOUT);
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Shape<QT>::kRegsFew));
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------- loads
      // Warp 0 divides the work and loads Q and K, warp 2 loads V: with pages
      // of 16 keys a block takes 32 copies, which one warp issues too slowly.
      const bool keys = warp == 0;
      Cursor c = {};
      Share share = {0, 0, 0, 0};
      long long want = blockIdx.x;  // an item, or a key block
      bool more = true, placed = false;
      if (keys && p.split) {
        share = my_share(p);
        want = share.begin;
        more = share.begin < share.end;
        if (lane == 0) p.meta[blockIdx.x].x = -1;
      }
      const int boxes = kKeys / p.box;
      const uint32_t box_bytes = static_cast<uint32_t>(p.box) * 128u;  // of one panel
      const int per = L::kVKeys / p.box;     // boxes of a V unit
      int unit = keys ? 0 : kP;              // the ring's units alternate: kP of K, kP of V
      int slot = unit, loads = 0, queries = 0;
      uint32_t phase = 1;                    // parity of the place's last release
      bool ok = true;
      for (int seg = 0; ok; ++seg) {
        if (keys) {
          if (seg > 0) ok = __all_sync(kFull, wait_soon(qempty, (seg & 1) ^ 1, abort_flag));
          if (!ok) break;
          if (more && !placed) {
            more = seek(p, c, want, p.split ? share.end - share.begin : 1LL << 40);
            placed = p.split;
          }
          if (lane == 0) {
            const Tile& tile = c.tile;
            Segment& g = segments[seg % kSegments];
            g.begin = c.begin;
            g.end = more ? c.end : -1;
            g.sink_blocks = tile.sink_blocks;
            g.main_block = tile.main_block;
            g.blocks = tile.blocks;
            g.hi = tile.hi;
            g.lo = tile.lo;
            g.pos0 = tile.pos0;
            g.tokens = tile.tokens;
            g.token0 = tile.token0;
            g.h = c.h;
            g.b = c.b;
            g.last_cta = -1;
            if (more && p.split && c.begin == 0 && c.end < tile.blocks)
              g.last_cta = cta_of(share, share.end - 1 + (tile.blocks - c.end));
            mbar_arrive(segment_ready(seg));
            if (more) {
              mbar_arrive_expect_tx(qfull, QT * kP * p.G * p.q_tokens * 128);
              for (int j = 0; j < QT; ++j)
                for (int pn = 0; pn < kP; ++pn)
                  tma_load_3d(sbase + j * L::kTileBytes + pn * kRows * 128, &tq, pn * 64,
                              c.h * p.G, tile.token0 + j * p.q_tokens, qfull);
            }
          }
          __syncwarp();
          queries += more ? 1 : 0;
        } else {
          ok = __all_sync(kFull, wait_soon(segment_ready(seg), (seg / kSegments) & 1, abort_flag));
          if (!ok) break;
        }
        const Segment& g = segments[seg % kSegments];
        const int begin = g.begin, end = g.end, hi = g.hi, lo = g.lo, h = g.h;
        const int sink_blocks = g.sink_blocks, skip = g.main_block - sink_blocks;
        if (end < 0) break;
        const int* table = p.block_table + g.b * p.bt_stride;
        // box l of a block: its page, -1 if no row sees any of its keys, -2 if
        // the table names no page of the pool for it
        auto lookup = [&](int key0) {
          const int key = key0 + lane * p.box;
          if (lane >= boxes || key >= hi || (key + p.box <= lo && key >= p.sinks)) return -1;
          const int page = __ldg(table + key / p.page);
          return page >= 0 && page < p.num_pages ? page : -2;
        };
        auto first_key = [&](int k) { return (k < sink_blocks ? k : k + skip) * kKeys; };
        int page = lookup(first_key(begin));
        for (int k = begin; k < end; ++k) {
          const int in_page = (first_key(k) + lane * p.box) % p.page;
          const int next = k + 1 < end ? lookup(first_key(k + 1)) : -1;
          const unsigned loaded = __ballot_sync(kFull, page >= 0);
          const unsigned bad = __ballot_sync(kFull, page == -2);
          const unsigned gone = ~loaded & ((1u << boxes) - 1u);
          if (keys && bad && lane == 0 && p.err) atomicOr(p.err, DSA_DEVERR_SLOT);
          for (int i = 0; i < kP; ++i) {
            // the ring's next unit, once it may be written
            ok = unit < S || wait_soon(empty(slot), phase, abort_flag);
            ok = __all_sync(kFull, ok);
            if (!ok) break;
            const uint32_t at = sbase + L::kOffRing + slot * kUnitBytes, bar = full(slot);
            if (keys) {  // 64 dims of all 128 keys
              if (bad && i == 0) {  // NaN keys, so the rows that see them become NaN
                for (unsigned m = bad; m; m &= m - 1)
                  fill_rows(at + (__ffs(m) - 1) * box_bytes, p.box, 0x7fff7fffu);
                fence_async_shared();
                __syncwarp();
              }
              if (lane == 0) mbar_arrive_expect_tx(bar, __popc(loaded) * box_bytes);
              __syncwarp();
              if (page >= 0) tma_load_4d(at + lane * box_bytes, &tk, i * 64, in_page, h, page, bar);
            } else {  // all dims of kVKeys keys
              const unsigned here = ((1u << per) - 1u) << (i * per);
              if (gone & here) {  // P is 0 there, and 0 * V must not be NaN
                for (unsigned m = gone & here; m; m &= m - 1)
                  for (int pn = 0; pn < kP; ++pn)
                    fill_rows(at + pn * L::kVKeys * 128 + (__ffs(m) - 1 - i * per) * box_bytes,
                              p.box, 0u);
                fence_async_shared();
                __syncwarp();
              }
              if (lane == 0) mbar_arrive_expect_tx(bar, kP * __popc(loaded & here) * box_bytes);
              __syncwarp();
              if (page >= 0 && lane / per == i)
                for (int pn = 0; pn < kP; ++pn)
                  tma_load_4d(at + pn * L::kVKeys * 128 + (lane - i * per) * box_bytes, &tv,
                              pn * 64, in_page, h, page, bar);
            }
            ++unit, ++loads;
            if (++slot == S) slot = 0, phase ^= 1;
          }
          if (!ok) break;
          unit += kP, slot += kP;  // the other warp's
          if (slot >= S) slot -= S, phase ^= 1;
          page = next;
        }
        if (!ok || !keys) continue;
        if (p.split)
          more = next_segment(p, c);
        else
          want += gridDim.x;
      }
      if (!ok) {
        if (lane == 0) give_up();
        // Stay until the loads issued have landed (else the MMA warp has waited
        // for each of them).
        volatile int never = 0;
        for (int n = 0, d = unit; n < loads && n < S / 2; ++n) {
          d -= d % (2 * kP) == (keys ? 0 : kP) ? kP + 1 : 1;
          wait_soon(full(d % S), (d / S) & 1, &never);
        }
        if (queries > 0) wait_soon(qfull, (queries - 1) & 1, &never);
      }
    } else if (warp == 1) {
      // ---------------------------------------------- MMA issuer
      // The steps go from block to block and tile to tile.  Behind the P V of
      // step n come the scores of step n + kLook, into the same place of TMEM:
      // products issued by one thread are carried out in their order.  The warp
      // stays together, one lane issues, and the ring's places are counted, not
      // divided: at three hand-overs a step this code's own time counts.
      constexpr uint32_t idesc_s = mma_idesc(BF16, false, kKeys);
      constexpr uint32_t idesc_o = mma_idesc(BF16, true, D);
      const bool leader = elect_one();
      const uint32_t q_lo = desc_lo(sbase, 0);
      const uint32_t k_lo = desc_lo(sbase + L::kOffRing, 0);
      const uint32_t v_lo = desc_lo(sbase + L::kOffRing, L::kVKeys * 128);
      int slot = 0;                        // ring place of the block's first K unit
      uint32_t phase = 0;                  // its parity
      int block = 0, first = 0;            // blocks done; place for S of tile 0's block
      bool ok = true;
      auto place = [&](int unit) {         // of the unit-th one from the block's first
        const int s = slot + unit;
        return s >= S ? s - S : s;
      };
      auto arrived = [&](int unit) {
        const int s = slot + unit;
        ok = wait_soon(full(s >= S ? s - S : s), s >= S ? phase ^ 1 : phase, abort_flag) && ok;
      };
      // S = Q_j K^T of the block `ahead` of this one
      auto scores = [&](int j, int ahead, int at) {
        if (leader && ok) {
#pragma unroll
          for (int pn = 0; pn < kP; ++pn) {
            const int s = place(2 * kP * ahead + pn);
            const uint32_t a = q_lo + ((j * L::kTileBytes + pn * kRows * 128) >> 4);
            const uint32_t b = k_lo + s * (kUnitBytes >> 4);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_ss(tmem_s(at), make_desc(a + 2 * ks), make_desc(b + 2 * ks), idesc_s,
                     pn + ks > 0 ? 1u : 0u);
            if (j + 1 == QT) mma_commit(empty(s));
          }
          mma_commit(sfull(j, block + ahead));
        }
      };
      auto keys_arrived = [&](int ahead) {
#pragma unroll
        for (int pn = 0; pn < kP; ++pn) arrived(2 * kP * ahead + pn);
      };
      auto place_of = [&](int j) {  // for S of tile j's block
        return kLook < 3 ? j : first + j < 3 ? first + j : first + j - 3;
      };
      for (int seg = 0; ok; ++seg) {
        ok = __all_sync(kFull, wait_soon(segment_ready(seg), (seg / kSegments) & 1, abort_flag));
        const int begin = segments[seg % kSegments].begin, end = segments[seg % kSegments].end;
        if (!ok || end < 0) break;
        ok = wait_soon(qfull, seg & 1, abort_flag);
        keys_arrived(0);
        if (kLook == 3 && begin + 1 < end) keys_arrived(1);
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < QT; ++j) scores(j, 0, place_of(j));
        if (kLook == 3 && begin + 1 < end) scores(0, 1, place_of(2));
        if (leader && ok && begin + 1 == end) mma_commit(qempty);
        for (int k = begin; k < end; ++k) {
          // O += P V of half a block, then the scores of kLook steps on
          auto values = [&](int j, int half) {
            const int u = half * kP / 2;           // its V unit of the block
            const int ahead = (j + kLook) / QT, then = (j + kLook) % QT;
            const bool more = half == 1 && k + ahead < end;
            // the loads first, at their first use: they are there before P is
            if (j == 0 && (half == 0 || kP == 2)) arrived(kP + u);
            if (more && then == 0) keys_arrived(ahead);
            ok = wait_soon(pready(j, half, block), turn(block), abort_flag) && ok;
            const int s = place(kP + u), at = place_of(j);
            tc_fence_after();
            if (leader && ok) {
              const int row = half * (kKeys / 2) - u * L::kVKeys;  // its first key in the unit
              const uint32_t b = v_lo + s * (kUnitBytes >> 4) + (row * 128 >> 4);
#pragma unroll
              for (int ks = 0; ks < kKeys / 32; ++ks)
                mma_ts(tmem_o(j), tmem_s(at) + half * (kKeys / 4) + ks * 8,
                       make_desc(b + ks * (2048 >> 4)), idesc_o,
                       (k > begin || half + ks > 0) ? 1u : 0u);
              if (j + 1 == QT && (kP == 2 || half == 1)) mma_commit(empty(s));
              if (half == 0) mma_commit(ohalf(j));
              if (half == 1 && kLook == 3) mma_commit(oblock(j));
              if (half == 1 && k + 1 == end) mma_commit(ofull(j));
            }
            if (more) scores(then, ahead, at);
          };
#pragma unroll
          for (int i = 0; i < 2 * QT; ++i) values(i / 2, i % 2);
          if (leader && ok && k + 2 == end) mma_commit(qempty);
          ++block;
          if (kLook == 3) first = first == 0 ? 2 : first - 1;  // two steps on
          slot += 2 * kP;
          if (slot >= S) slot -= S, phase ^= 1;
          ok = __all_sync(kFull, ok);
          if (!ok) break;
        }
      }
      if (!ok && lane == 0) give_up();
      if (leader) mma_commit(drain);  // every MMA issued must finish before TMEM is released
      volatile int never = 0;
      wait_soon(drain, 0, &never);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Shape<QT>::kRegsMany));
    // ------------------------------------------------ softmax
    const int j = QT == 1 ? 0 : (warp - 4) >> 2;  // the query tile
    const int sub = warp & 3;           // the TMEM lanes this warp may touch
    const int row = 32 * sub + lane;    // of the query tile
    const uint32_t lanes = static_cast<uint32_t>(32 * sub) << 16;
    const uint32_t t_o = tmem_o(j) + lanes;
    // what the exponents are taken against, in powers of two
    auto reference = [&](float m) { return (m == -INFINITY ? 0.0f : m * p.c) - (BF16 ? 0.0f : 7.0f); };
    const int tok = j * p.q_tokens + row / p.G;   // of the item
    int slot = kP;                      // ring place of the block's first V unit
    uint32_t phase = 0;                 // its parity
    int block = 0, at_s = j;            // blocks done; place of S
    int edges = 0;                      // blocks that not every row saw whole
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      ok = __all_sync(kFull, wait_soon(segment_ready(seg), (seg / kSegments) & 1, abort_flag));
      const Segment& g = segments[seg % kSegments];
      if (!ok || g.end < 0) break;
      const int tokens = min(p.q_tokens, g.tokens - j * p.q_tokens);  // of the query tile
      const bool mine = row < tokens * p.G;                // this row exists
      const bool busy = 32 * sub < tokens * p.G;           // some row of the warp does
      const int pos = g.pos0 + tok;
      const int hi = mine ? pos + 1 : 0;                   // keys [lo, hi) and [0, sinks)
      const int lo = p.window ? max(0, pos - p.window + 1) : 0;
      // keys that every existing row of the warp sees
      const int hi_all = __reduce_min_sync(kFull, mine ? hi : 0x7fffffff);
      const int lo_all = __reduce_max_sync(kFull, mine ? lo : 0);
      float m = -INFINITY, l = 0.0f;  // m is the maximum that P and O are scaled by
      bool spoiled = false;  // this row sees a value, zeroed below, that was not finite
      const int begin = g.begin, end = g.end;
      const int sink_blocks = g.sink_blocks, skip = g.main_block - sink_blocks;
      const int seen_hi = g.hi, seen_lo = g.lo;  // by some row of the item
      const int every_hi = g.pos0 + 1;           // by every row
      const int every_lo = p.window ? g.pos0 + g.tokens - p.window : 0;
      for (int k = begin; k < end; ++k) {
        const int key0 = (k < sink_blocks ? k : k + skip) * kKeys;
        auto scores_done = [&]() {
          ok = __all_sync(kFull, wait_soon(sfull(j, block), turn(block), abort_flag));
          tc_fence_after();
          return ok;
        };
        if (QT == 1 && !scores_done()) break;
        // Where some row of the item does not see some key of the block, 0 *
        // its V must be 0 whatever V holds.  Tile 0's thread r looks at key
        // r's row: it zeroes what no row sees (behind the context, before the
        // window) and what is not finite.  In the latter case out of the rows that
        // do see the key becomes NaN; their lse, which no value enters, does not.
        // Tile 0's P V comes first, and waits.  With two
        // tiles all of it is done before S is waited for, as V comes sooner.
        // That takes a ring so long that the unit before V's in its place has
        // landed by now: a barrier's parity tells only its last two phases apart.
        static_assert(QT == 1 || S >= 4 * kP, "a place of V is looked at too early");
        if (!(key0 + kKeys <= every_hi && (key0 >= every_lo || key0 + kKeys <= p.sinks))) {
          if (j == 0) {
            const int key = key0 + row;
            bool odd = false;
            if (!(key < every_hi && (key >= every_lo || key < p.sinks))) {
              int s = slot + row / L::kVKeys;
              uint32_t ph = phase;
              if (s >= S) s -= S, ph ^= 1;
              ok = wait_soon(full(s), ph, abort_flag);
              const uint32_t at = sbase + L::kOffRing + s * kUnitBytes + (row % L::kVKeys) * 128;
              auto piece = [&](int i) {  // 16 bytes; lanes apart, for the banks
                return at + (i >> 3) * (L::kVKeys * 128) + 16 * ((i + lane) & 7);
              };
              const bool some = key < seen_hi && (key >= seen_lo || key < p.sinks);
              if (some) {
                uint32_t zero = 0;  // += 0 * V: stays 0 if all of V is finite
#pragma unroll 4
                for (int i = 0; i < 8 * kP; ++i) {
                  uint32_t v[4];
                  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                               : "r"(piece(i)) : "memory");
#pragma unroll
                  for (int q = 0; q < 4; ++q) zero = fma0<BF16>(v[q], zero);
                }
                odd = (zero & 0x7fff7fffu) != 0;
              }
              if (!some || odd) {
#pragma unroll 1
                for (int i = 0; i < 8 * kP; ++i)
                  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};"
                               ::"r"(piece(i)), "r"(0) : "memory");
                fence_async_shared();
              }
            }
            const unsigned mask = __ballot_sync(kFull, odd);
            if (lane == 0) {
              odd_keys[4 * (edges & 3) + sub] = mask;
              mbar_arrive(checked(edges));
            }
          }
          ok = __all_sync(kFull, ok && wait_soon(checked(edges), (edges >> 2) & 1, abort_flag));
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = key0 + 32 * i;
            const uint32_t mask = odd_keys[4 * (edges & 3) + i];
            if (mask & below(hi - at) & (~below(lo - at) | below(p.sinks - at))) spoiled = true;
          }
          ++edges;
        }
        if (QT == 2 && !scores_done()) break;
        const uint32_t t_s = tmem_s(at_s) + lanes;
        const bool edge = !(key0 + kKeys <= hi_all && (key0 >= lo_all || key0 + kKeys <= p.sinks));
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          if (busy) {
            float s[kKeys / 2];
            tmem_ld32(t_s + 64 * half, s);
            tmem_ld32(t_s + 64 * half + 32, s + 32);
            tmem_wait_ld(s);
            if (edge) {
#pragma unroll
              for (int part = 0; part < 2; ++part) {  // masks only at an edge
                const int at = key0 + 64 * half + part * 32;
                if (at + 32 <= hi_all && (at >= lo_all || at + 32 <= p.sinks)) continue;
                const uint32_t seen = below(hi - at) & (~below(lo - at) | below(p.sinks - at));
#pragma unroll
                for (int i = 0; i < 32; ++i)
                  s[32 * part + i] = seen & (1u << i) ? s[32 * part + i] : -INFINITY;
              }
            }
            float sum;
            uint32_t w[kKeys / 4];
            auto exponentials = [&](float mc) {
              const float2 c2 = make_float2(p.c, p.c), mc2 = make_float2(-mc, -mc);
              float2 add[2] = {};
#pragma unroll
              for (int i = 0; i < kKeys / 4; ++i) {
                const float2 e = __ffma2_rn(make_float2(s[2 * i], s[2 * i + 1]), c2, mc2);
                const float2 f = make_float2(exp2_approx(e.x), exp2_approx(e.y));
                add[i % 2] = __fadd2_rn(add[i % 2], f);
                w[i] = pack2<BF16>(f.x, f.y);
              }
              sum = (add[0].x + add[0].y) + (add[1].x + add[1].y);
            };
            // a segment's first half takes its maximum at once
            bool renew = mine, again = k == begin && half == 0;
#pragma unroll 1
            for (;;) {
              if (again) {
                float mx[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx[i] = s[i];
#pragma unroll
                for (int i = 4; i < kKeys / 2; i += 8)
#pragma unroll
                  for (int q = 0; q < 4; ++q)
                    mx[q] = i + 4 < kKeys / 2 ? max3f(mx[q], s[i + q], s[i + 4 + q])
                                              : fmaxf(mx[q], s[i + q]);
                const float m_new = max3f(m, fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                if (k > begin || half == 1) {  // O exists
                  // and has to be complete up to the half before.  With one place
                  // for S per tile sfull followed the products of the block
                  // before; else they are waited for, before ohalf, whose
                  // parity would else not tell this block from the last but one.
                  if (kLook == 3)
                    ok = __all_sync(kFull, wait_soon(oblock(j), (block + 1) & 1, abort_flag));
                  if (half == 1)
                    ok = __all_sync(kFull, wait_soon(ohalf(j), block & 1, abort_flag) && ok);
                  tc_fence_after();
                  // a first maximum meets O and l that are still 0
                  const float f = renew && m != -INFINITY ? exp2_approx((m - m_new) * p.c) : 1.0f;
                  l *= f;
#pragma unroll 1
                  for (int i = 0; i < D / 16; ++i) {
                    float o[16];
                    tmem_ld16(t_o + 16 * i, o);
                    tmem_wait_ld(o);
#pragma unroll
                    for (int q = 0; q < 16; ++q) o[q] *= f;
                    tmem_st16(t_o + 16 * i, reinterpret_cast<uint32_t*>(o));
                  }
                }
                m = renew ? m_new : m;
              }
              exponentials(reference(m));
              if (again) break;
              renew = mine && (m == -INFINITY || !(sum <= kSumLimit<BF16>));
              if (!__any_sync(kFull, renew)) break;
              again = true;
            }
            l += sum;
            tmem_st16(t_s + 32 * half, w);  // over S of the keys read before
            tmem_st16(t_s + 32 * half + 16, w + 16);
            tmem_wait_st();
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(pready(j, half, block));
        }
        ++block;
        if (kLook == 3) at_s = at_s == 0 ? 2 : at_s - 1;
        slot += 2 * kP;
        if (slot >= S) slot -= S, phase ^= 1;
      }
      if (ok) ok = __all_sync(kFull, wait_soon(ofull(j), seg & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const bool whole = begin == 0 && end == g.blocks;
      if (busy) {
        const int head = row % p.G;
        const int slot_of = 2 * blockIdx.x + (begin == 0 ? 1 : 0);
        float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;  // of O
        if (spoiled) inv = __int_as_float(0x7fc00000);
        const long long token = g.token0 + tok;
        const int h = g.h * p.G + head;
        const long long at = static_cast<long long>(slot_of) * (QT * kRows) + tok * p.G + head;
        // this row in out or in the workspace; both are whole 16-byte pieces
        char* const to = whole ? static_cast<char*>(p.out) +
                                     2 * (token * p.out_stride_t + h * p.out_stride_h)
                               : reinterpret_cast<char*>(p.part + at * D);
        const unsigned rows = __ballot_sync(kFull, mine);
        char* row_to[4];  // QT 2: where this lane writes a quarter of 64 bytes
        if (QT == 2) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            row_to[q] = reinterpret_cast<char*>(__shfl_sync(
                            kFull, reinterpret_cast<unsigned long long>(to), 8 * q + (lane >> 2))) +
                        16 * (lane & 3);
        }
        // 64 bytes of every row of the warp: v holds this lane's.  A lane's
        // own row would go out 16 bytes at a time to 32 places; turned through
        // shared memory (pieces swizzled against bank conflicts) four lanes
        // write 64 bytes of one row.
        auto store64 = [&](const uint4(&v)[4], int offset) {
          if (QT == 1) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (mine) *reinterpret_cast<uint4*>(to + offset + 16 * q) = v[q];
            return;
          }
          uint4* turn = reinterpret_cast<uint4*>(smem + L::kOffTurn) + (warp - 4) * 128;
#pragma unroll
          for (int q = 0; q < 4; ++q) turn[lane * 4 + (q ^ (lane >> 1 & 3))] = v[q];
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 8 * q + (lane >> 2);
            const uint4 u = turn[r * 4 + ((lane & 3) ^ (r >> 1 & 3))];
            if (rows >> r & 1) *reinterpret_cast<uint4*>(row_to[q] + offset) = u;
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          tmem_ld32(t_o + 32 * i, o);
          tmem_wait_ld(o);
#pragma unroll
          for (int q = 0; q < 32; ++q) o[q] *= inv;
          if (whole) {
            uint4 v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              v[q].x = pack2<BF16>(o[8 * q], o[8 * q + 1]);
              v[q].y = pack2<BF16>(o[8 * q + 2], o[8 * q + 3]);
              v[q].z = pack2<BF16>(o[8 * q + 4], o[8 * q + 5]);
              v[q].w = pack2<BF16>(o[8 * q + 6], o[8 * q + 7]);
              if (l == 0.0f) v[q] = make_uint4(0, 0, 0, 0);
            }
            store64(v, 64 * i);
          } else {
            store64(*reinterpret_cast<const uint4(*)[4]>(o), 128 * i);
            store64(*reinterpret_cast<const uint4(*)[4]>(o + 16), 128 * i + 64);
          }
        }
        if (mine) {
          if (!whole)
            p.ml[at] = make_float2(l == 0.0f ? -INFINITY : reference(m), l);
          else if (p.lse)
            p.lse[token * (p.Hkv * p.G) + h] = l == 0.0f ? -INFINITY : reference(m) * kLn2 + logf(l);
        }
      }
      // the item starts here and goes on in later CTAs: the second kernel
      // joins the parts, this CTA's first
      if (g.last_cta >= 0 && threadIdx.x == 128)
        p.meta[blockIdx.x] = make_int4(g.last_cta, g.token0, g.h, g.tokens);
      __syncwarp();  // the segment's numbers have been read
    }
    if (!ok && lane == 0) give_up();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;"
                 ::"r"(tmem), "n"(Shape<QT>::kTmemCols) : "memory");
}

// Joins the parts of the items that a cut divides: with M the largest m of a
// row's parts, out = sum 2^(m - M) O / sum 2^(m - M) l.  Which items those are
// stands in meta; every CTA counts their rows and the rows are dealt out
// evenly, one to a warp at a time, or where they are fewer than the CTAs and
// have many parts one to a CTA, whose warps take an eighth of the parts each.  Bound: the waits
// for meta, (m, l) and O, one behind the other.  Every sum has a fixed order.
constexpr int kJoinWarps = 8;
constexpr int kJoinCtas = 8 * kSms;

template <int N>
struct Vec;
template <>
struct Vec<2> {
  using type = float2;
};
template <>
struct Vec<4> {
  using type = float4;
};

template <int D, bool BF16, int QT>
__global__ void __launch_bounds__(32 * kJoinWarps)
    dsa_attention_join_kernel(const __grid_constant__ AParams p) {
  constexpr int kMost = Shape<QT>::kCtas;  // entries of meta, two to a thread
  static_assert(kMost <= 64 * kJoinWarps && kMost % 2 == 0, "entries");
  __shared__ int4 metas[kMost];
  __shared__ int before[kMost];  // rows of the items before
  __shared__ int warp_rows[kJoinWarps];
  __shared__ float sums[kJoinWarps][D + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_launch_dependents();
  int rows[2] = {0, 0}, most = 0;
  const int e = 2 * threadIdx.x;
  if (e < kMost) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      metas[e + i] = p.meta[e + i];
      rows[i] = metas[e + i].x < 0 ? 0 : metas[e + i].w * p.G;
      most = max(most, metas[e + i].x - (e + i) + 1);  // parts
    }
  }
  int upto = rows[0] + rows[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warp_rows[warp] = upto;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (w < warp) upto += warp_rows[w];
    total += warp_rows[w];
  }
  if (e < kMost) {
    before[e] = upto - rows[0] - rows[1];
    before[e + 1] = upto - rows[1];
  }
  const bool long_rows = __syncthreads_or(most > kJoinWarps);

  constexpr int kV = D / 32;  // values of a row per lane
  using V = typename Vec<kV>::type;
  const bool alone = !long_rows || total > static_cast<int>(gridDim.x);  // a row to a warp
  const int step = gridDim.x * (alone ? kJoinWarps : 1);
  for (int n = alone ? blockIdx.x * kJoinWarps + warp : blockIdx.x; n < total; n += step) {
    int first = 0;  // the last entry with before <= n: the CTA in which the item starts
#pragma unroll
    for (int o = 256; o; o >>= 1)
      if (first + o < kMost && before[first + o] <= n) first += o;
    const int4 meta = metas[first];
    const int row = n - before[first], parts = meta.x - first + 1;
    auto at = [&](int i) {  // the row's part i in ml and part
      return (i == 0 ? 2LL * first + 1 : 2LL * (first + i)) * (QT * kRows) + row;
    };
    float top = -INFINITY;
    for (int i = lane; i < parts; i += 32) top = fmaxf(top, p.ml[at(i)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    const float ref = top == -INFINITY ? 0.0f : top;
    float acc[kV] = {};
    float l = 0.0f;
#pragma unroll 8
    for (int i = alone ? 0 : warp; i < parts; i += alone ? 1 : kJoinWarps) {
      const float2 ml = p.ml[at(i)];
      const V o = *reinterpret_cast<const V*>(p.part + at(i) * D + lane * kV);
      const float f = exp2_approx(ml.x - ref);
      l = fmaf(f, ml.y, l);
#pragma unroll
      for (int j = 0; j < kV; ++j) acc[j] = fmaf(f, reinterpret_cast<const float*>(&o)[j], acc[j]);
    }
    if (!alone) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kV; ++j) sums[warp][lane * kV + j] = acc[j];
      if (lane == 0) sums[warp][D] = l;
      __syncthreads();
      if (warp != 0) continue;
      l = 0.0f;
#pragma unroll
      for (int j = 0; j < kV; ++j) acc[j] = 0.0f;
      for (int w = 0; w < kJoinWarps; ++w) {
        l += sums[w][D];
#pragma unroll
        for (int j = 0; j < kV; ++j) acc[j] += sums[w][lane * kV + j];
      }
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const long long token = meta.y + row / p.G;
    const int h = meta.z * p.G + row % p.G;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) +
                                                token * p.out_stride_t + h * p.out_stride_h) +
                    lane * (kV / 2);
#pragma unroll
    for (int j = 0; j < kV; j += 2)
      out[j / 2] = l == 0.0f ? 0u : pack2<BF16>(acc[j] * inv, acc[j + 1] * inv);
    if (lane == 0 && p.lse)
      p.lse[token * (p.Hkv * p.G) + h] = l == 0.0f ? -INFINITY : ref * kLn2 + logf(l);
  }
}

// ---------------------------------------------------------------- host side

bool misaligned(const void* ptr, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
}

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  std::call_once(g_encode_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  return g_encode;
}

std::mutex g_ready_mu;
bool g_ready[64];

template <int D, bool BF16, int QT>
cudaError_t prepare_one() {
  cudaError_t e = cudaFuncSetAttribute(dsa_paged_attention_kernel<D, BF16, QT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       ASmem<D, QT>::kBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(dsa_paged_attention_kernel<D, BF16, QT>,
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  return e;
}

// Once per device.
cudaError_t prepare_device() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_ready_mu);
  if (g_ready[dev]) return cudaSuccess;
  e = prepare_one<64, false, 1>();
  if (e == cudaSuccess) e = prepare_one<64, true, 1>();
  if (e == cudaSuccess) e = prepare_one<128, false, 1>();
  if (e == cudaSuccess) e = prepare_one<128, true, 1>();
  if (e == cudaSuccess) e = prepare_one<64, false, 2>();
  if (e == cudaSuccess) e = prepare_one<64, true, 2>();
  if (e == cudaSuccess) e = prepare_one<128, false, 2>();
  if (e == cudaSuccess) e = prepare_one<128, true, 2>();
  g_ready[dev] = e == cudaSuccess;
  return e;
}

long long max_items(int T, int B, int Hkv, int tile_tokens) {
  return (static_cast<long long>(T) / tile_tokens + B) * Hkv;
}

// Items of about equal lengths.
long long mean_items(int T, int B, int Hkv, int tile_tokens) {
  const long long per_head = static_cast<long long>(T) / tile_tokens + (B + 1) / 2;
  return (per_head > B ? per_head : B) * Hkv;
}

// Calls that may be cut and need a workspace for it.  Not those of one key
// block, nor four rounds of items of two tiles over keys that L2 cannot hold: a
// cut's place in the keys differs from CTA to CTA, so all keys are in use at
// once, while items in order keep the CTAs on one kv head (4096 tokens over
// 65536 with 8 kv heads, 268 MB: 5.35 ms whole, 5.59 cut).  Any other call needs
// it, cut or not; its size is that of the CTAs, whatever the call's.  The rule
// goes by capacities, as the lengths are on the device: a batch of that kind with
// one long context among short ones ends with the CTAs that have it (2048 tokens
// over 4000 beside 31 single tokens over 3000 and one over 100,000, 64 heads on 8:
// 1277 us; the chunk and the single tokens as calls of their own 181 + 136).
bool may_split(int T, int B, int Hkv, int D, int q_tokens, int max_context) {
  if (max_context <= kKeys) return false;
  // seek counts the key blocks of a sequence and kv head in 32 bits: 116,000 rows
  // over 2^30 keys would pass them
  const long long blocks = (max_context + kKeys - 1LL) / kKeys;
  if ((static_cast<long long>(T) / q_tokens + 1) * blocks > 0x7fffffffLL) return false;
  return mean_items(T, B, Hkv, 2 * q_tokens) <= 3 * kSms || 4.0 * D * Hkv * max_context * B <= 2e8 ||
         2LL * T < static_cast<long long>(q_tokens) * B;
}

// How a call is carried out: 1 or 2 query tiles per CTA, and whether the key
// blocks are cut into equal shares or CTAs take whole items.  Two tiles load
// the keys once for 256 rows, but leave more rows empty where sequences end.
// Cutting balances any lengths, but its parts are written, joined by a second
// kernel and read, and one more item is begun per CTA.  The times of both are
// estimated in us for sequences of equal lengths at max_context (the lengths
// are on the device), with
//   block   a key block of a CTA at D = 128 / 64: 2.6 / 1.6 us with one tile
//           (two CTAs share the SM), 1.7 / 1.1 with two;
//   item    what an item begins and ends with: 3.5 us, with two tiles 5;
//   cut     parts and join: 12 us, with two tiles 15;
//   ragged  a twentieth of an item, by which whole items of unequal lengths
//           end later.
// What is cut has two tiles where sequences have half a tile of new tokens.
// Over 880 random calls (1 to 4096 new tokens, contexts to 40000, 1 to 128
// sequences, of equal lengths, ragged, or one long context among short ones)
// the choice takes 2.2% more than the best of the four on average; the rule
// that it replaces, which cut nearly everything, 11%.  In us:
//                                        whole, 1 and 2 tiles; cut, 1 and 2
//   12 x 350 over 2000, 16 on 16, D 64        61    78    88    88
//   32 x 64 over 1000, 32 on 8, D 128         48    42    97    66
//   2048 over 2048, 32 on 8                   59    56    87    79
//   64 x 8 over 500, 32 on 32                 99   133   102   146
//   8 x 64 over 30000, 32 on 8               352   365   319   196
//   256 over 8192, 64 on 8                   101   106    81    70
struct Plan {
  int tiles;
  bool split;
};

Plan make_plan(int T, int B, int Hkv, int D, int q_tokens, int max_context, int window, int sinks,
               bool may) {
  constexpr double kItem[2] = {3.5, 5.0}, kCut[2] = {12.0, 15.0}, kRagged = 0.05;
  const double block[2] = {D == 64 ? 1.6 : 2.6, D == 64 ? 1.1 : 1.7};
  const int most_tiles = 2LL * T < static_cast<long long>(q_tokens) * B ? 1 : 2;
  Plan best = {1, false};
  double best_us = 0;
  for (int tiles = 1; tiles <= most_tiles; ++tiles) {
    const int tile_tokens = tiles * q_tokens;
    const double items = static_cast<double>(mean_items(T, B, Hkv, tile_tokens));
    double keys = max_context;  // of an item on average
    if (window) {
      const double most = static_cast<double>(window) + sinks + tile_tokens;
      keys = most < keys ? most : keys;
    } else {
      const double new_tokens = static_cast<double>(T) / B;
      keys -= (new_tokens < keys ? new_tokens : keys) / 2;
      keys = keys < kKeys ? kKeys : keys;
    }
    const double ctas = 2 / tiles * kSms, one = keys / kKeys * block[tiles - 1];
    const double whole = std::ceil(items / ctas) * (one + kItem[tiles - 1]) + kRagged * one;
    if (tiles == 1 || whole < best_us) best = {tiles, false}, best_us = whole;
    if (!may || tiles < most_tiles) continue;
    const double cut = items / ctas * one + (items / ctas + 1) * kItem[tiles - 1] + kCut[tiles - 1];
    if (cut < best_us) best = {tiles, true}, best_us = cut;
  }
  return best;
}

bool encode_map(CUtensorMap* map, bool bf16, const void* base, int rank, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box) {
  PFN_cuTensorMapEncodeTiled_v12000 encode = tensor_map_encoder();
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return encode && encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                          rank, const_cast<void*>(base), dims, strides, box, estr,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16, int QT>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const AParams& p, bool pdl, cudaStream_t s) {
  const long long items = max_items(p.T, p.B, p.Hkv, p.tile_tokens);
  const int ctas = p.split || items > Shape<QT>::kCtas ? Shape<QT>::kCtas : static_cast<int>(items);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(Shape<QT>::kThreads);
  cfg.dynamicSmemBytes = ASmem<D, QT>::kBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, dsa_paged_attention_kernel<D, BF16, QT>, tq, tk, tv, p);
  if (e != cudaSuccess || !p.split) return e;
  cfg.gridDim = dim3(kJoinCtas);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, dsa_attention_join_kernel<D, BF16, QT>, p);
}

template <int D, bool BF16>
cudaError_t launch_tiles(int tiles, const CUtensorMap& tq, const CUtensorMap& tk,
                         const CUtensorMap& tv, const AParams& p, bool pdl, cudaStream_t s) {
  return tiles == 2 ? launch<D, BF16, 2>(tq, tk, tv, p, pdl, s)
                    : launch<D, BF16, 1>(tq, tk, tv, p, pdl, s);
}

// Whether two of T x H rows of D elements, at t * stride_t + h * stride_h, share
// an element: rows (t, h) and (t + a, h - b) with |a * stride_t - b * stride_h| < D.
// Strides are at least D (so rows of one t or one h do not).
bool rows_overlap(int64_t T, int64_t stride_t, int64_t H, int64_t stride_h, int64_t D) {
  using Wide = __int128;
  if (T < 2 || H < 2 || stride_t >= static_cast<Wide>(H - 1) * stride_h + D ||
      stride_h >= static_cast<Wide>(T - 1) * stride_t + D)
    return false;
  if (T < H) return rows_overlap(H, stride_h, T, stride_t, D);
  for (int64_t b = 1; b < H; ++b) {
    const Wide x = static_cast<Wide>(b) * stride_h;
    const Wide a = x / stride_t;  // the nearest multiples are a and a + 1
    if (a >= 1 && a < T && x - a * stride_t < D) return true;
    if (a + 1 < T && (a + 1) * stride_t - x < D) return true;
  }
  return false;
}

// the same for one and two query tiles
constexpr size_t kMetaBytes = 2 * kSms * sizeof(int4);
constexpr size_t kPartRows = 2 * 2 * kSms * kRows;
constexpr size_t kMlBytes = kPartRows * sizeof(float2);

size_t workspace_bytes_of(int32_t head_dim) {
  return kMetaBytes + kMlBytes + kPartRows * static_cast<size_t>(head_dim) * sizeof(float);
}

}  // namespace

extern "C" {

size_t dsa_paged_attention_workspace_bytes(int32_t T, int32_t B, int32_t H, int32_t Hkv,
                                           int32_t head_dim, int32_t max_context) {
  if (T < 1 || B < 1 || Hkv < 1 || H < Hkv || H % Hkv || H / Hkv > kRows || head_dim < 1) return 0;
  if (!may_split(T, B, Hkv, head_dim, kRows / (H / Hkv), max_context)) return 0;
  return workspace_bytes_of(head_dim);
}

size_t dsa_paged_attention_max_workspace_bytes(int32_t head_dim) {
  return head_dim < 1 ? 0 : workspace_bytes_of(head_dim);
}

dsa_status dsa_paged_attention(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k_cache,
    const void* v_cache, int64_t k_stride_page, int64_t k_stride_token, int64_t k_stride_head,
    int64_t v_stride_page, int64_t v_stride_token, int64_t v_stride_head, int64_t num_pages,
    int32_t page_size, const int32_t* block_table, int64_t bt_stride, const int32_t* query_start,
    const int32_t* context_lens, int32_t max_context, float scale, int32_t window, int32_t sinks,
    void* out, int64_t out_stride_t, int64_t out_stride_h, float* lse, int32_t T, int32_t B,
    int32_t H, int32_t Hkv, int32_t head_dim, int32_t dtype, uint32_t flags, void* workspace,
    size_t workspace_bytes, int32_t* err_flags, void* stream) {
  if (T < 0 || B < 0 || H < 1 || Hkv < 1 || H % Hkv || max_context < 0 || bt_stride < 0 ||
      num_pages < 1 || num_pages > 0x7fffffffLL || window < 0 || sinks < 0)
    return DSA_ERR_SHAPE;
  const int G = H / Hkv;
  if (head_dim != 64 && head_dim != 128) return DSA_ERR_UNSUPPORTED;
  if (dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_FP16) return DSA_ERR_UNSUPPORTED;
  if (G > kRows) return DSA_ERR_UNSUPPORTED;
  if (page_size < 8 || (page_size < 64 ? 64 % page_size : page_size % 64) != 0)
    return DSA_ERR_UNSUPPORTED;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return DSA_ERR_UNSUPPORTED;
  if (flags & ~static_cast<uint32_t>(DSA_FLAG_PDL)) return DSA_ERR_UNSUPPORTED;
  // every row of the table covers max_context keys
  if (bt_stride < (static_cast<long long>(max_context) + page_size - 1) / page_size)
    return DSA_ERR_SHAPE;
  // positions and grids are 32-bit
  if (max_context > (1 << 30) || T > (1 << 30) || static_cast<long long>(T) * H > 0x7fffffffLL)
    return DSA_ERR_SHAPE;
  const int q_tokens = kRows / G;
  if (max_items(T, B, Hkv, q_tokens) > 0x7fffffffLL) return DSA_ERR_SHAPE;
  if (T == 0 || B == 0) return DSA_OK;
  if (!q || !k_cache || !v_cache || !query_start || !context_lens || !out ||
      (!block_table && max_context > 0))
    return DSA_ERR_NULL;
  // TMA: 16-byte aligned bases, strides that are multiples of 16 bytes, below 2^40
  auto bad_stride = [](int64_t stride, int64_t extent) {
    return extent > 1 && (stride % 8 != 0);
  };
  if ((T > 1 && out_stride_t < head_dim) || (H > 1 && out_stride_h < head_dim))
    return DSA_ERR_SHAPE;
  auto bad_size = [](int64_t stride, int64_t extent) {
    return extent > 1 && (stride < 1 || stride >= (1LL << 39));
  };
  if (bad_size(q_stride_t, T) || bad_size(q_stride_h, H) || bad_size(k_stride_page, num_pages) ||
      bad_size(k_stride_token, page_size) || bad_size(k_stride_head, Hkv) ||
      bad_size(v_stride_page, num_pages) || bad_size(v_stride_token, page_size) ||
      bad_size(v_stride_head, Hkv) || bad_size(out_stride_t, T) || bad_size(out_stride_h, H))
    return DSA_ERR_SHAPE;
  if (bad_stride(q_stride_t, T) || bad_stride(q_stride_h, H) ||
      bad_stride(k_stride_page, num_pages) || bad_stride(k_stride_token, page_size) ||
      bad_stride(k_stride_head, Hkv) || bad_stride(v_stride_page, num_pages) ||
      bad_stride(v_stride_token, page_size) || bad_stride(v_stride_head, Hkv) ||
      bad_stride(out_stride_t, T) || bad_stride(out_stride_h, H))
    return DSA_ERR_ALIGN;
  if (rows_overlap(T, out_stride_t, H, out_stride_h, head_dim)) return DSA_ERR_SHAPE;
  if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
      misaligned(out, 16) || misaligned(block_table, 4) || misaligned(query_start, 4) ||
      misaligned(context_lens, 4) || misaligned(lse, 4) || misaligned(err_flags, 4))
    return DSA_ERR_ALIGN;
  const size_t need = dsa_paged_attention_workspace_bytes(T, B, H, Hkv, head_dim, max_context);
  if (need) {
    if (!workspace) return DSA_ERR_NULL;
    if (misaligned(workspace, 16)) return DSA_ERR_ALIGN;
    if (workspace_bytes < need) return DSA_ERR_SHAPE;
  }
  if (prepare_device() != cudaSuccess) return DSA_ERR_LAUNCH;

  const bool bf16 = dtype == DSA_DTYPE_BF16;
  const cuuint64_t D = static_cast<cuuint64_t>(head_dim);
  // the stride of a dimension of one entry is never used, but has to be valid
  auto bytes = [&](int64_t stride, int64_t extent) {
    return static_cast<cuuint64_t>(extent > 1 ? stride : head_dim) * 2;
  };
  alignas(64) CUtensorMap tq, tk, tv;
  const int box = page_size < 64 ? page_size : 64;
  {
    const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
    const cuuint64_t strides[2] = {bytes(q_stride_h, H), bytes(q_stride_t, T)};
    const cuuint32_t b[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(q_tokens)};
    if (!encode_map(&tq, bf16, q, 3, dims, strides, b)) return DSA_ERR_LAUNCH;
  }
  auto cache_map = [&](CUtensorMap* map, const void* base, int64_t sp, int64_t st, int64_t sh) {
    const cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(page_size),
                                static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(num_pages)};
    const cuuint64_t strides[3] = {bytes(st, page_size), bytes(sh, Hkv), bytes(sp, num_pages)};
    const cuuint32_t b[4] = {64, static_cast<cuuint32_t>(box), 1, 1};
    return encode_map(map, bf16, base, 4, dims, strides, b);
  };
  if (!cache_map(&tk, k_cache, k_stride_page, k_stride_token, k_stride_head) ||
      !cache_map(&tv, v_cache, v_stride_page, v_stride_token, v_stride_head))
    return DSA_ERR_LAUNCH;

  AParams p = {};
  p.block_table = block_table;
  p.query_start = query_start;
  p.context_lens = context_lens;
  p.out = out;
  p.lse = lse;
  p.bt_stride = bt_stride;
  p.out_stride_t = out_stride_t;
  p.out_stride_h = out_stride_h;
  p.num_pages = static_cast<int>(num_pages);
  p.page = page_size;
  p.box = box;
  p.T = T;
  p.B = B;
  p.Hkv = Hkv;
  p.G = G;
  p.window = window < max_context ? window : 0;  // such a window hides nothing
  p.sinks = p.window ? (sinks < max_context ? sinks : max_context) : 0;
  const Plan plan = make_plan(T, B, Hkv, head_dim, q_tokens, max_context, p.window, p.sinks, need > 0);
  const int tiles = plan.tiles;
  p.q_tokens = q_tokens;
  p.tile_tokens = tiles * q_tokens;
  p.max_context = max_context;
  p.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  p.split = plan.split ? 1 : 0;
  p.meta = static_cast<int4*>(workspace);
  p.ml = reinterpret_cast<float2*>(static_cast<char*>(workspace) + kMetaBytes);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + kMetaBytes + kMlBytes);
  p.err = err_flags;
  const bool pdl = (flags & DSA_FLAG_PDL) != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (head_dim == 64)
    e = bf16 ? launch_tiles<64, true>(tiles, tq, tk, tv, p, pdl, s)
             : launch_tiles<64, false>(tiles, tq, tk, tv, p, pdl, s);
  else
    e = bf16 ? launch_tiles<128, true>(tiles, tq, tk, tv, p, pdl, s)
             : launch_tiles<128, false>(tiles, tq, tk, tv, p, pdl, s);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}

}  // extern "C"
