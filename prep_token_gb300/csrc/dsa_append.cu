// New tokens' K and V into the paged cache that dsa_paged_attention reads, with
// an optional RMS norm of every q and k head and the position rotation (RoPE)
// on the way; q goes out rotated in the same launch.
//
//   x = q or k of a head, in fp32
//   x *= gamma / sqrt(mean(x^2) + eps)             (where gamma is given)
//   (a, b) -> (a c - b s, b c + a s) on x[0:rope_dim)
//   rounded once; k and v to slot out_cache_loc[t] of their caches, q to q_out
//
// A head's row of D values is D / 16 lanes wide, two 16-byte pieces to a lane.  A
// pair is in one lane and needs no shuffle; a norm's sum takes log2(D / 16) of them.  c, s and gamma
// are the same for all heads of a token's q (or k): their products are four
// factors per pair, formed once, and the root is multiplied in at the end.
//
// Two kernels: few tokens take a warp to every pass of 512 / D rows, so that all
// is in flight at once, or nearly (1500 tokens of 72 heads of 64 are 1.85 rounds of
// its CTAs); many take warps that stay and load ahead.
//
// Bound: HBM for many tokens, each row read and written once; measured (6.78 TB/s):
// 8192 tokens of 32 + 16 heads of 128, 206 MB, 36.3 us with both norms (5.7 TB/s),
// 35.6 without; 16384 67.7 us (6.1 TB/s).  With nothing to compute the same rows
// take 32 (direct) to 35: what is missing is the start (three round trips: position,
// cos/sin, first store) and the mix of reads and writes in rows of 256 bytes.  The
// first form of the stream kernel, with addresses formed anew for each row, took 55
// us with norms, one pass to a warp takes 56.  16 tokens of 64 + 16 heads take 2.1
// us, launch and two dependent reads.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dsa_prep.h"
#include "dsa_rows.cuh"

namespace {

using namespace dsa_rows;

constexpr int kSms = 152;
constexpr int kWarps = 4;  // of a CTA of the direct kernel
constexpr int kStreamWarps = 8, kStreamCtas = 2;  // of the stream kernel, per CTA and per SM
// Passes per SM from which on it is the faster one (us, direct and stream): 1500
// tokens of 24 + 48 heads of 64, 88 passes, 6.2 and 6.7; 8192 of 8 + 2 of 128, 161,
// 11.0 and 12.6; 4096 of 64 + 16, 539, 31.0 and 29.7; 8192 of 32 + 16, 647, 37.5
// and 35.6.  A norm's longer arithmetic is worth overlapping earlier: 256 tokens of
// 32 + 16 heads, 20 passes, 3.3 and 4.0; 1000, 79, 8.0 and 6.6; 8192, 647, 56 and 36.
constexpr int stream_passes(bool norm) { return norm ? 40 : 250; }

struct AppendParams {
  const uint16_t *q, *k, *v;
  uint16_t *q_out, *k_cache, *v_cache;
  const long long *positions, *slots;
  const float *cos, *sin;
  const float *q_gamma, *k_gamma;
  long long q_t, q_h, k_t, k_h, v_t, v_h, out_t, out_h;  // strides
  long long kc_page, kc_token, kc_head, vc_page, vc_token, vc_head;
  long long cs_stride, max_position, num_slots;
  float eps;
  int T, H, Hkv;
  int turns;        // lanes of a row that rotate: rope_dim / 16
  int page_size, page_shift;
  int passes;       // of a token: its q, k and v rows, 512 / D at a time
  int q_passes, kv_passes;
  int merged;       // k and v rows are few enough to share a pass, k's first
  int* err;
};

// Two pieces of neighbouring pairs as the pairs' first values and their second ones.
__device__ __forceinline__ void split_pairs(float2 (&x)[4], float2 (&y)[4]) {
  const float2 a[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = make_float2(a[2 * i].x, a[2 * i + 1].x);
    y[i] = make_float2(a[2 * i].y, a[2 * i + 1].y);
  }
}

// Where a lane's values are in a row: the pieces of eight at `first` and `second`.
// Whatever pieces a lane has, neighbouring lanes have neighbouring ones, so that a
// load or store of the warp covers whole sectors (with a lane's two side by side
// each took all sectors of the rows, twice: 8192 tokens of 32 + 16 heads, nothing
// to rotate, 50 us instead of 36).  NeoX: the lanes that rotate have the two
// halves of their pairs, piece l and l + rope_dim / 16; the others share the rest.
// GPT-J: pieces l and l + D / 16, whose pairs are within them.
template <int D, int STYLE>
struct Lane {
  static constexpr int kLanes = D / 16;        // of a row
  static constexpr int kRowsOf = 32 / kLanes;  // rows that a warp takes at a time
  int l, sub, first, second;
  bool turns_first, turns_second;
  __device__ __forceinline__ explicit Lane(const AppendParams& p) {
    const int lane = threadIdx.x & 31;
    l = lane % kLanes, sub = lane / kLanes;
    if (STYLE == DSA_ROPE_NEOX) {
      turns_first = turns_second = l < p.turns;
      first = 8 * (l < p.turns ? l : l + p.turns);
      second = 8 * (l < p.turns ? l + p.turns : l + kLanes);
    } else {
      turns_first = l < 2 * p.turns;
      turns_second = l + kLanes < 2 * p.turns;
      first = 8 * l;
      second = 8 * (l + kLanes);
    }
  }
};

__device__ __forceinline__ void load4(const float* p, float2& a, float2& b) {
  const float4 x = *reinterpret_cast<const float4*>(p);
  a = make_float2(x.x, x.y), b = make_float2(x.z, x.w);
}
// Eight floats of a row as four pairs.
__device__ __forceinline__ void load8(const float* p, float2 (&v)[4]) {
  load4(p, v[0], v[1]);
  load4(p + 4, v[2], v[3]);
}

// x' = xx x + xy y, y' = yy y + yx x for a lane's pairs: the rotation and gamma,
// which are the same for every row of a token's q (or k).
struct Turn {
  float2 xx[4], xy[4], yy[4], yx[4];
};

// cos, sin: the token's rows.
template <int STYLE, bool NORM, class L>
__device__ __forceinline__ void make_turn(Turn& r, const L& at, const float* cos, const float* sin,
                                          const float* gamma) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.xx[i] = make_float2(1.0f, 1.0f), r.yx[i] = make_float2(0.0f, 0.0f);
  if (STYLE == DSA_ROPE_NEOX) {
    if (at.turns_first) {
      load8(cos + 8 * at.l, r.xx);
      load8(sin + 8 * at.l, r.yx);
    }
  } else {
    if (at.turns_first) {
      load4(cos + at.first / 2, r.xx[0], r.xx[1]);
      load4(sin + at.first / 2, r.yx[0], r.yx[1]);
    }
    if (at.turns_second) {
      load4(cos + at.second / 2, r.xx[2], r.xx[3]);
      load4(sin + at.second / 2, r.yx[2], r.yx[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r.yy[i] = r.xx[i], r.xy[i] = make_float2(-r.yx[i].x, -r.yx[i].y);
  if (NORM && gamma) {
    float2 gx[4], gy[4];
    load8(gamma + at.first, gx);
    load8(gamma + at.second, gy);
    if (STYLE == DSA_ROPE_GPTJ) split_pairs(gx, gy);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.xx[i] = __fmul2_rn(r.xx[i], gx[i]), r.yx[i] = __fmul2_rn(r.yx[i], gx[i]);
      r.yy[i] = __fmul2_rn(r.yy[i], gy[i]), r.xy[i] = __fmul2_rn(r.xy[i], gy[i]);
    }
  }
}

// A lane's two pieces of a row, turned if it is `active`; a whole warp calls it.
template <bool BF16, int D, int STYLE, bool NORM>
__device__ __forceinline__ void turn_row(uint4& u, uint4& w, const Turn& r,
                                         const Lane<D, STYLE>& at, bool active, bool norm,
                                         float eps) {
  float2 x[4], y[4];
  unpack8<BF16>(u, x);
  unpack8<BF16>(w, y);
  if (STYLE == DSA_ROPE_GPTJ) split_pairs(x, y);
  float2 rs = make_float2(1.0f, 1.0f);
  if (NORM && norm) {
    float2 sum = __fmul2_rn(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sum = __ffma2_rn(x[i], x[i], sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = __ffma2_rn(y[i], y[i], sum);
    float all = sum.x + sum.y;
#pragma unroll
    for (int o = D / 32; o; o >>= 1) all += __shfl_xor_sync(kFull, all, o);
    rs.x = rs.y = rsqrtf(fmaf(all, 1.0f / D, eps));
  }
  // a piece with neither stays as it is, NaN and all
  const bool first = at.turns_first || (NORM && norm), second = at.turns_second || (NORM && norm);
  if (!first || !active) return;  // without the first nor does the second
  if (NORM && rs.x == 0.0f) {
    // The row holds an infinity (or its squares pass fp32): that becomes NaN, what is
    // finite 0.  Places that do not turn are no pairs: there b * -0 would make a finite
    // value NaN beside an infinite one.
    const float2 none = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __fmul2_rn(x[i], rs), b = __fmul2_rn(y[i], rs);
      const bool pair = i < 2 || STYLE == DSA_ROPE_NEOX ? at.turns_first : at.turns_second;
      x[i] = __ffma2_rn(a, r.xx[i], pair ? __fmul2_rn(b, r.xy[i]) : none);
      y[i] = __ffma2_rn(b, r.yy[i], pair ? __fmul2_rn(a, r.yx[i]) : none);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = x[i], b = y[i];
      x[i] = __ffma2_rn(a, r.xx[i], __fmul2_rn(b, r.xy[i]));
      y[i] = __ffma2_rn(b, r.yy[i], __fmul2_rn(a, r.yx[i]));
      if (NORM) x[i] = __fmul2_rn(x[i], rs), y[i] = __fmul2_rn(y[i], rs);
    }
  }
  if (STYLE == DSA_ROPE_NEOX) {
    u = pack8<BF16>(x);
    w = pack8<BF16>(y);
  } else {
    u = make_uint4(pack2<BF16>(x[0].x, y[0].x), pack2<BF16>(x[0].y, y[0].y),
                   pack2<BF16>(x[1].x, y[1].x), pack2<BF16>(x[1].y, y[1].y));
    if (second)
      w = make_uint4(pack2<BF16>(x[2].x, y[2].x), pack2<BF16>(x[2].y, y[2].y),
                     pack2<BF16>(x[3].x, y[3].x), pack2<BF16>(x[3].y, y[3].y));
  }
}

// The token's place in a cache.
__device__ __forceinline__ long long place_of(const AppendParams& p, long long slot,
                                              long long page_stride, long long token_stride) {
  long long page, in_page;
  if (p.page_shift >= 0) {
    page = slot >> p.page_shift;
    in_page = slot & (p.page_size - 1);
  } else {
    page = slot / p.page_size;
    in_page = slot - page * p.page_size;
  }
  return page * page_stride + in_page * token_stride;
}

// The rows of a kind: q (0), k (1) and v (2), or k and v (1).
__device__ __forceinline__ int rows_of(const AppendParams& p, int kind) {
  return kind == 0 ? p.H : kind == 1 && p.merged ? 2 * p.Hkv : p.Hkv;
}
__device__ __forceinline__ bool is_value(const AppendParams& p, int kind, int row) {
  return kind == 2 || (kind == 1 && p.merged && row >= p.Hkv);
}

// Few tokens: a warp to each pass of a token (512 / D rows of q, k or v).
template <bool BF16, int D, int STYLE, bool NORM>
__global__ void __launch_bounds__(32 * kWarps)
    dsa_kv_append_kernel(const __grid_constant__ AppendParams p) {
  const int item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = item / p.passes, pass = item - t * p.passes;
  grid_dependency_wait();
  grid_launch_dependents();
  if (t >= p.T) return;
  const Lane<D, STYLE> at(p);
  const int kind = pass < p.q_passes ? 0 : pass < p.q_passes + p.kv_passes ? 1 : 2;
  const bool is_q = kind == 0;
  int row = (pass - (is_q ? 0 : kind == 1 ? p.q_passes : p.q_passes + p.kv_passes)) * at.kRowsOf +
            at.sub;
  const bool some = row < rows_of(p, kind), is_v = is_value(p, kind, row);
  if (kind == 1 && is_v) row -= p.Hkv;
  const uint16_t* const from = is_q   ? p.q + t * p.q_t + row * p.q_h
                               : is_v ? p.v + t * p.v_t + row * p.v_h
                                      : p.k + t * p.k_t + row * p.k_h;
  // the rows travel beside the position and the slot that they wait for
  const long long pos = __ldg(p.positions + t), slot = __ldg(p.slots + t);
  uint4 u = make_uint4(0, 0, 0, 0), w = u;
  if (some) {
    u = load_piece(from + at.first);
    w = load_piece(from + at.second);
  }
  const bool first_lane = (threadIdx.x & 31) == 0 && pass == 0;
  if (pos < 0 || pos >= p.max_position) {
    if (first_lane && p.err) atomicOr(p.err, DSA_DEVERR_POSITION);
    return;
  }
  const bool keep = slot >= 0 && slot < p.num_slots;
  if (!keep && first_lane && p.err) atomicOr(p.err, DSA_DEVERR_SLOT);
  if (!is_q && !keep) return;
  if (kind < 2) {
    const float* const gamma = is_q ? p.q_gamma : p.k_gamma;
    Turn r;
    make_turn<STYLE, NORM>(r, at, p.cos + pos * p.cs_stride, p.sin + pos * p.cs_stride, gamma);
    turn_row<BF16, D, STYLE, NORM>(u, w, r, at, !is_v, gamma != nullptr, p.eps);
  }
  if (some) {
    uint16_t* const to =
        is_q   ? p.q_out + t * p.out_t + row * p.out_h
        : is_v ? p.v_cache + place_of(p, slot, p.vc_page, p.vc_token) + row * p.vc_head
               : p.k_cache + place_of(p, slot, p.kc_page, p.kc_token) + row * p.kc_head;
    store_piece(to + at.first, u);
    store_piece(to + at.second, w);
  }
}

// Many tokens: warps that stay, each on an equal run of all tokens' passes.  A
// lane's pieces of the passes ahead travel into its own places of a ring in
// shared memory (cp.async; nobody else reads them), a token's cos/sin row into
// one of two places of the warp while the token before is worked on.
constexpr int kDepth = 3;                          // passes in flight, and this one
constexpr int kWarpBytes = kDepth * 1024 + 2 * 512;  // the ring; cos and sin of two tokens

template <bool BF16, int D, int STYLE, bool NORM>
__global__ void __launch_bounds__(32 * kStreamWarps, kStreamCtas)
    dsa_kv_append_stream_kernel(const __grid_constant__ AppendParams p) {
  __shared__ __align__(16) unsigned char smem[kStreamWarps * kWarpBytes];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Lane<D, STYLE> at(p);
  unsigned char* const ring = smem + warp * kWarpBytes;
  float* const angles = reinterpret_cast<float*>(ring + kDepth * 1024);
  const long long total = static_cast<long long>(p.T) * p.passes;
  const int warps = gridDim.x * kStreamWarps, me = blockIdx.x * kStreamWarps + warp;
  const int begin = static_cast<int>(total * me / warps);
  const int n = static_cast<int>(total * (me + 1) / warps) - begin;
  if (n == 0) return;
  int t = begin / p.passes;
  const int pass = begin - t * p.passes;
  const int last = (begin + n - 1) / p.passes;  // this warp's last token
  grid_dependency_wait();
  grid_launch_dependents();

  // Where the loads are: so many passes of q (0), k (1) or v (2) of a token are
  // left, the next one's row and place; addresses move by the pass within a kind.
  const int last_kind = p.merged ? 1 : 2;
  int fetch_t = t, fetch_kind, fetch_left, fetch_rows, fetch_n = n;
  uint32_t fetch_to = smem_u32(ring + 16 * lane);
  const uint32_t ring_end = fetch_to + kDepth * 1024;
  const uint16_t* fetch_from;
  long long fetch_step;
  auto enter = [&](int kind, int skip) {  // `skip` passes of it are done
    fetch_kind = kind;
    fetch_left = (kind == 0 ? p.q_passes : p.kv_passes) - skip;
    int row = skip * at.kRowsOf + at.sub;
    fetch_rows = rows_of(p, kind) - row;
    const bool value = is_value(p, kind, row);
    if (kind == 1 && value) row -= p.Hkv;
    fetch_step = kind == 0 ? p.q_h : value ? p.v_h : p.k_h;
    fetch_from = (kind == 0 ? p.q + fetch_t * p.q_t
                  : value   ? p.v + fetch_t * p.v_t
                            : p.k + fetch_t * p.k_t) + row * fetch_step + at.first;
    fetch_step *= at.kRowsOf;
  };
  const int apart = at.second - at.first;
  auto fetch = [&]() {  // the next pass, if there is one
    if (fetch_left == 0) {
      const bool done = fetch_kind == last_kind;
      if (done) ++fetch_t;
      enter(done ? (p.q_passes > 0 ? 0 : 1) : fetch_kind + 1, 0);
    }
    if (fetch_n > 0 && fetch_rows > 0) {
      cp_async16_cg(fetch_to, fetch_from);
      cp_async16_cg(fetch_to + 512, fetch_from + apart);
    }
    cp_async_commit();
    --fetch_n, --fetch_left;
    fetch_rows -= at.kRowsOf;
    fetch_from += fetch_step;
    fetch_to += 1024;
    if (fetch_to == ring_end) fetch_to -= kDepth * 1024;
  };
  auto position = [&](int token) { return token <= last ? __ldg(p.positions + token) : -1; };
  auto slot_of = [&](int token) { return token <= last ? __ldg(p.slots + token) : -1; };
  auto valid = [&](long long pos) { return pos >= 0 && pos < p.max_position; };
  auto fetch_angles = [&](int token, long long pos) {  // 2 * turns pieces each of cos and sin
    const int piece = lane & 15;
    if (valid(pos) && piece < 2 * p.turns)
      cp_async16_ca(smem_u32(angles + (token & 1) * 128 + 4 * lane),
                    (lane < 16 ? p.cos : p.sin) + pos * p.cs_stride + 4 * piece);
  };
  long long slot = slot_of(t), next_slot = slot_of(t + 1), pos = position(t + 1);
  const long long pos0 = position(t);
  bool ok = valid(pos0), next_ok = valid(pos);
  fetch_angles(t, pos0);
  fetch_angles(t + 1, pos);
  pos = position(t + 2);  // that of the token behind the next one
  int kind = pass < p.q_passes ? 0 : pass < p.q_passes + p.kv_passes ? 1 : 2;
  int skip = pass - (kind == 0 ? 0 : kind == 1 ? p.q_passes : p.q_passes + p.kv_passes);
  enter(kind, skip);
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch();
  cp_async_wait<kDepth - 2>();
  int stage = 0;
  Turn r;  // without a norm k's is q's
  // one kind of a token's rows after the other
#pragma unroll 1
  for (int left = n;;) {
    __syncwarp();  // this token's cos and sin have landed for every lane of the warp
    const bool keep = slot >= 0 && slot < p.num_slots;
    if (lane == 0 && p.err && !(ok && keep))
      atomicOr(p.err, ok ? DSA_DEVERR_SLOT : DSA_DEVERR_POSITION);
    int row = skip * at.kRowsOf + at.sub;
    int rows = ok && (kind == 0 || keep) ? rows_of(p, kind) - row : 0;
    const bool value = is_value(p, kind, row);
    if (kind == 1 && value) row -= p.Hkv;
    long long step = kind == 0 ? p.out_h : value ? p.vc_head : p.kc_head;
    uint16_t* to = kind == 0 ? p.q_out + t * p.out_t
                   : value   ? p.v_cache + place_of(p, keep ? slot : 0, p.vc_page, p.vc_token)
                             : p.k_cache + place_of(p, keep ? slot : 0, p.kc_page, p.kc_token);
    to += row * step + at.first;
    step *= at.kRowsOf;
    const float* const gamma = kind == 0 ? p.q_gamma : p.k_gamma;
    if (kind < 2 && (NORM || kind == 0 || p.q_passes == 0 || left == n)) {
      const float* const cos = angles + (t & 1) * 128;
      make_turn<STYLE, NORM>(r, at, cos, cos + 64, gamma);
    }
    int m = min(left, (kind == 0 ? p.q_passes : p.kv_passes) - skip);
    left -= m;
#pragma unroll 1
    for (; m > 0; --m) {
      fetch();
      cp_async_wait<kDepth - 1>();
      const unsigned char* const from = ring + stage * 1024 + 16 * lane;
      uint4 u = *reinterpret_cast<const uint4*>(from);
      uint4 w = *reinterpret_cast<const uint4*>(from + 512);
      if (kind < 2)
        turn_row<BF16, D, STYLE, NORM>(u, w, r, at, !value, gamma != nullptr, p.eps);
      if (rows > 0) {
        store_piece(to, u);
        store_piece(to + apart, w);
      }
      rows -= at.kRowsOf;
      to += step;
      stage = stage + 1 == kDepth ? 0 : stage + 1;
    }
    if (left == 0) break;
    skip = 0;
    if (kind++ == last_kind) {
      // the next token: the one behind it takes the last one's place for cos and sin
      kind = p.q_passes > 0 ? 0 : 1;
      __syncwarp();  // which every lane has read
      ++t;
      slot = next_slot, ok = next_ok;
      next_slot = slot_of(t + 1), next_ok = valid(pos);
      fetch_angles(t + 1, pos);
      pos = position(t + 2);
    }
  }
}

template <bool BF16, int D, int STYLE, bool NORM>
cudaError_t launch_one(const AppendParams& p, bool stream, const cudaLaunchConfig_t& cfg) {
  return stream ? cudaLaunchKernelEx(&cfg, dsa_kv_append_stream_kernel<BF16, D, STYLE, NORM>, p)
                : cudaLaunchKernelEx(&cfg, dsa_kv_append_kernel<BF16, D, STYLE, NORM>, p);
}

template <bool BF16, int D>
cudaError_t launch(const AppendParams& p, int style, bool stream, const cudaLaunchConfig_t& cfg) {
  if (p.q_gamma || p.k_gamma)
    return style == DSA_ROPE_NEOX ? launch_one<BF16, D, DSA_ROPE_NEOX, true>(p, stream, cfg)
                                  : launch_one<BF16, D, DSA_ROPE_GPTJ, true>(p, stream, cfg);
  return style == DSA_ROPE_NEOX ? launch_one<BF16, D, DSA_ROPE_NEOX, false>(p, stream, cfg)
                                : launch_one<BF16, D, DSA_ROPE_GPTJ, false>(p, stream, cfg);
}

}  // namespace

extern "C" dsa_status dsa_kv_append(
    const void* q, int64_t q_stride_t, int64_t q_stride_h, const void* k, int64_t k_stride_t,
    int64_t k_stride_h, const void* v, int64_t v_stride_t, int64_t v_stride_h,
    const int64_t* positions, const int64_t* out_cache_loc, const float* cos_cache,
    const float* sin_cache, int64_t cs_stride, int64_t max_position, const float* q_gamma,
    const float* k_gamma, float norm_eps, void* q_out, int64_t q_out_stride_t,
    int64_t q_out_stride_h, void* k_cache, void* v_cache, int64_t kc_stride_page,
    int64_t kc_stride_token, int64_t kc_stride_head, int64_t vc_stride_page,
    int64_t vc_stride_token, int64_t vc_stride_head, int64_t num_pages, int32_t page_size,
    int32_t T, int32_t H, int32_t Hkv, int32_t head_dim, int32_t rope_dim, int32_t rope_style,
    int32_t dtype, uint32_t flags, int32_t* err_flags, void* stream) {
  if (T < 0 || H < 0 || Hkv < 1 || page_size < 1 || num_pages < 1 || max_position < 0 ||
      static_cast<__int128>(T) * (static_cast<int64_t>(H) + 2LL * Hkv) > (1 << 30) ||
      num_pages > 0x7fffffffLL)
    return DSA_ERR_SHAPE;
  if (head_dim != 64 && head_dim != 128) return DSA_ERR_UNSUPPORTED;
  if (dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_FP16) return DSA_ERR_UNSUPPORTED;
  if (rope_dim < 0 || rope_dim > head_dim || rope_dim % 16) return DSA_ERR_UNSUPPORTED;
  if (rope_style != DSA_ROPE_NEOX && rope_style != DSA_ROPE_GPTJ) return DSA_ERR_UNSUPPORTED;
  if (flags & ~static_cast<uint32_t>(DSA_FLAG_PDL)) return DSA_ERR_UNSUPPORTED;
  if ((q_gamma || k_gamma) && !(norm_eps > 0.0f && std::isfinite(norm_eps)))
    return DSA_ERR_UNSUPPORTED;
  if (T == 0) return DSA_OK;
  if (!k || !v || !positions || !out_cache_loc || !k_cache || !v_cache || (H > 0 && (!q || !q_out)))
    return DSA_ERR_NULL;
  if (rope_dim > 0 && (!cos_cache || !sin_cache)) return DSA_ERR_NULL;
  if (rope_dim > 0 && max_position > 1 && cs_stride < rope_dim / 2) return DSA_ERR_SHAPE;
  if (stride_short(q_stride_t, H > 0 ? T : 0, 1) || stride_short(q_stride_h, H, 1) ||
      stride_short(k_stride_t, T, 1) || stride_short(k_stride_h, Hkv, 1) ||
      stride_short(v_stride_t, T, 1) || stride_short(v_stride_h, Hkv, 1) ||
      stride_short(q_out_stride_t, H > 0 ? T : 0, 1) || stride_short(q_out_stride_h, H, 1) ||
      stride_short(kc_stride_page, num_pages, 1) || stride_short(kc_stride_token, page_size, 1) ||
      stride_short(kc_stride_head, Hkv, 1) || stride_short(vc_stride_page, num_pages, 1) ||
      stride_short(vc_stride_token, page_size, 1) || stride_short(vc_stride_head, Hkv, 1))
    return DSA_ERR_SHAPE;
  if (!rows_apart(head_dim, {num_pages, page_size, Hkv},
                  {kc_stride_page, kc_stride_token, kc_stride_head}) ||
      !rows_apart(head_dim, {num_pages, page_size, Hkv},
                  {vc_stride_page, vc_stride_token, vc_stride_head}) ||
      (H > 0 && !rows_apart(head_dim, {T, H, 1}, {q_out_stride_t, q_out_stride_h, 0})))
    return DSA_ERR_SHAPE;
  if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_cache, 16) ||
      misaligned(v_cache, 16) || misaligned(positions, 8) || misaligned(out_cache_loc, 8) ||
      misaligned(q_gamma, 16) || misaligned(k_gamma, 16) || misaligned(err_flags, 4) ||
      (H > 0 && (misaligned(q, 16) || misaligned(q_out, 16) || stride_odd(q_stride_t, T) ||
                 stride_odd(q_stride_h, H) || stride_odd(q_out_stride_t, T) ||
                 stride_odd(q_out_stride_h, H))) ||
      stride_odd(k_stride_t, T) || stride_odd(k_stride_h, Hkv) || stride_odd(v_stride_t, T) ||
      stride_odd(v_stride_h, Hkv) || stride_odd(kc_stride_page, num_pages) ||
      stride_odd(kc_stride_token, page_size) || stride_odd(kc_stride_head, Hkv) ||
      stride_odd(vc_stride_page, num_pages) || stride_odd(vc_stride_token, page_size) ||
      stride_odd(vc_stride_head, Hkv))
    return DSA_ERR_ALIGN;
  if (rope_dim > 0 && (misaligned(cos_cache, 16) || misaligned(sin_cache, 16) || cs_stride % 4))
    return DSA_ERR_ALIGN;
  AppendParams p = {};
  p.q = static_cast<const uint16_t*>(q);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_cache = static_cast<uint16_t*>(k_cache);
  p.v_cache = static_cast<uint16_t*>(v_cache);
  p.positions = reinterpret_cast<const long long*>(positions);
  p.slots = reinterpret_cast<const long long*>(out_cache_loc);
  p.cos = cos_cache;
  p.sin = sin_cache;
  p.q_gamma = q_gamma;
  p.k_gamma = k_gamma;
  p.q_t = q_stride_t, p.q_h = q_stride_h;
  p.k_t = k_stride_t, p.k_h = k_stride_h;
  p.v_t = v_stride_t, p.v_h = v_stride_h;
  p.out_t = q_out_stride_t, p.out_h = q_out_stride_h;
  p.kc_page = kc_stride_page, p.kc_token = kc_stride_token, p.kc_head = kc_stride_head;
  p.vc_page = vc_stride_page, p.vc_token = vc_stride_token, p.vc_head = vc_stride_head;
  p.cs_stride = cs_stride;
  p.max_position = max_position;
  p.num_slots = num_pages * page_size;
  p.eps = norm_eps;
  p.T = T, p.H = H, p.Hkv = Hkv;
  p.turns = rope_dim / 16;
  p.page_size = page_size;
  p.page_shift = page_shift_of(page_size);
  const int at_once = 512 / head_dim;  // rows that a warp takes at a time
  p.q_passes = (H + at_once - 1) / at_once;
  p.kv_passes = (Hkv + at_once - 1) / at_once;
  p.merged = 2 * Hkv <= at_once;
  p.passes = p.q_passes + (p.merged ? 1 : 2 * p.kv_passes);
  p.err = err_flags;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const bool norm = q_gamma || k_gamma;
  const long long all = static_cast<long long>(T) * p.passes;
  // a token's cos/sin are fetched a token ahead, which has to be kDepth passes at least
  const bool stream_kernel = all >= stream_passes(norm) * kSms && p.passes >= kDepth;
  cfg.gridDim = dim3(stream_kernel ? kSms * kStreamCtas
                                   : static_cast<unsigned>((all + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(32 * (stream_kernel ? kStreamWarps : kWarps));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = flags & DSA_FLAG_PDL ? 1 : 0;
  const bool bf16 = dtype == DSA_DTYPE_BF16;
  cudaError_t e;
  if (head_dim == 64)
    e = bf16 ? launch<true, 64>(p, rope_style, stream_kernel, cfg)
             : launch<false, 64>(p, rope_style, stream_kernel, cfg);
  else
    e = bf16 ? launch<true, 128>(p, rope_style, stream_kernel, cfg)
             : launch<false, 128>(p, rope_style, stream_kernel, cfg);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}
