// RMS norm of token rows, with the residual's addition in front and an output
// in 16 bits, in e4m3 with one power-of-two scale per group, or both.
//
//   z = x + residual (fp32; residual_out = z rounded once)
//   y = z * gamma / sqrt(mean(z^2) + eps)
//   out = y rounded once;  e = the smallest integer with max(amax, 1e-4) <=
//   448 * 2^e over a group's y, codes = e4m3_rne(y * 2^-e), scale 2^e
//
// The norm takes z unrounded, so y is one rounding from the definition.
//
// A row belongs to the threads of one CTA, which hold it in registers between
// the sum and the outputs: every byte moves once.  A thread has up to four
// 16-byte pieces of eight values, `threads of the row` pieces apart, so that
// a group's pieces (16 of 128 values, 4 of 32) sit in neighbouring lanes and
// its amax takes shuffles only.
//
// Bound: HBM.  Measured (6.78 TB/s): 16384 rows of 7168 with a residual, to e4m3,
// 823 MB, 125.5 us (6.56 TB/s, 0.97); 4096 of them 35.6 us (0.85); one row 2.8 us, launch
// and one round trip.  No ring and no rows ahead: CTAs that stay and load the next
// row with cp.async took 141 us, as what counts is how many rows are resident (56
// registers: five CTAs of 224 threads per SM; 64 registers, four, 131 us).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dsa_prep.h"
#include "dsa_rows.cuh"

namespace {

using namespace dsa_rows;

constexpr int kSms = 152;
constexpr int kMaxPieces = 4;   // of a thread
constexpr int kMaxRowThreads = 1024;

struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;
  uint16_t* residual_out;
  uint16_t* out;
  uint8_t* codes;
  void* scales;
  const float* gamma;
  long long x_stride, residual_stride, residual_out_stride, out_stride, codes_stride,
      scales_stride;
  float eps, inv_n;
  int T, pieces;      // pieces of a row: N / 8
  int group_lanes;    // lanes of a group: 4 or 16
  int scale_bytes;    // 1: the byte e + 127; 4: fp32 2^e
};

// blockDim.x threads for a row, blockDim.y rows.
template <bool BF16, int PIECES, bool RES>
__global__ void __maxnreg__(PIECES == 4 ? 56 : 40) dsa_rms_norm_kernel(const NormParams p) {
  __shared__ float part[32];
  const int lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5, first_warp = threadIdx.y * warps;
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const bool mine = row < p.T;
  grid_dependency_wait();
  grid_launch_dependents();
  uint4 a[PIECES], b[PIECES];
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (mine && at < p.pieces) {
      a[i] = load_piece(p.x + row * p.x_stride + 8 * at);
      if (RES) b[i] = load_piece(p.residual + row * p.residual_stride + 8 * at);
    }
  }
  float2 z[PIECES][4];
  float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    unpack8<BF16>(a[i], z[i]);
    if (RES) {
      float2 r[4];
      unpack8<BF16>(b[i], r);
#pragma unroll
      for (int j = 0; j < 4; ++j) z[i][j] = __fadd2_rn(z[i][j], r[j]);
      if (p.residual_out && mine && at < p.pieces)
        store_piece(p.residual_out + row * p.residual_out_stride + 8 * at, pack8<BF16>(z[i]));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) sum2 = __ffma2_rn(z[i][j], z[i][j], sum2);
  }
  float sum = sum2.x + sum2.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (warps > 1) {
    if (lane == 0) part[first_warp + (threadIdx.x >> 5)] = sum;
    __syncthreads();
    sum = lane < warps ? part[first_warp + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  const float rs = 1.0f / sqrtf(fmaf(sum, p.inv_n, p.eps));
  const float2 rs2 = make_float2(rs, rs);
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    const bool some = mine && at < p.pieces;
    float amax = 0.0f;
    if (some) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 g = __ldg(reinterpret_cast<const float4*>(p.gamma + 8 * at) + j);
        z[i][2 * j] = __fmul2_rn(__fmul2_rn(z[i][2 * j], rs2), make_float2(g.x, g.y));
        z[i][2 * j + 1] = __fmul2_rn(__fmul2_rn(z[i][2 * j + 1], rs2), make_float2(g.z, g.w));
      }
      if (p.out) store_piece(p.out + row * p.out_stride + 8 * at, pack8<BF16>(z[i]));
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = max3f(amax, fabsf(z[i][j].x), fabsf(z[i][j].y));
    }
    if (p.codes) {
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
      if (p.group_lanes == 16) {
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 4));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 8));
      }
      const int e = exponent_of_amax(amax);
      const float2 down = make_float2(pow2f(-e), pow2f(-e));
      if (some) {
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 x = __fmul2_rn(z[i][j], down);
          c[j] = cvt_e4m3x2(x.x, x.y);
        }
        *reinterpret_cast<uint2*>(p.codes + row * p.codes_stride + 8 * at) =
            make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
        if (lane % p.group_lanes == 0) {
          const long long s = row * p.scales_stride + at / p.group_lanes;
          if (p.scale_bytes == 1)
            static_cast<uint8_t*>(p.scales)[s] = static_cast<uint8_t>(e + 127);
          else
            static_cast<float*>(p.scales)[s] = pow2f(e);
        }
      }
    }
  }
}

template <bool BF16, bool RES>
cudaError_t launch(const NormParams& p, int pieces, const cudaLaunchConfig_t& cfg) {
  switch (pieces) {
    case 1: return cudaLaunchKernelEx(&cfg, dsa_rms_norm_kernel<BF16, 1, RES>, p);
    case 2: return cudaLaunchKernelEx(&cfg, dsa_rms_norm_kernel<BF16, 2, RES>, p);
    default: return cudaLaunchKernelEx(&cfg, dsa_rms_norm_kernel<BF16, 4, RES>, p);
  }
}

// Pieces of a thread: one where all rows are resident at once with it (least
// latency), four where they are many times that (most bytes in flight for the
// instructions), two between, unless that makes large CTAs.  In us with 1, 2 and 4
// pieces, rows x N: 304 x 7168 4.5 4.4 5.2; 608 x 5120 6.7 5.6 6.0; 1216 x 4096 8.8
// 8.5 8.4; 4096 x 4096 22.5 19.7 20.6; 4096 x 7168 44.7 37.7 35.7; 304 x 16384 - 10.2
// 8.5; 16384 x 2048 42 38 40; 16384 x 7168 166 137 125.5.
template <class F>
int choose_pieces(int T, F row_threads) {
  auto per_sm = [&](int n) { return static_cast<double>(T) * row_threads(n) / kSms; };
  if (row_threads(1) <= kMaxRowThreads && per_sm(1) <= 1750) return 1;
  if (row_threads(2) <= kMaxRowThreads && per_sm(2) <= (row_threads(2) <= 512 ? 4096 : 1750))
    return 2;
  return 4;
}

}  // namespace

extern "C" dsa_status dsa_rms_norm(
    const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
    void* residual_out, int64_t residual_out_stride, const float* gamma, float eps, void* out,
    int64_t out_stride, void* codes, int64_t codes_stride, void* scales, int64_t scales_stride,
    int32_t scale_format, int32_t group, int32_t T, int32_t N, int32_t dtype, uint32_t flags,
    void* stream) {
  if (T < 0 || T > (1 << 30) || N < 1 || N % 8 || N > 8 * kMaxPieces * kMaxRowThreads)
    return DSA_ERR_SHAPE;
  if (dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_FP16) return DSA_ERR_UNSUPPORTED;
  if (flags & ~static_cast<uint32_t>(DSA_FLAG_PDL)) return DSA_ERR_UNSUPPORTED;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return DSA_ERR_UNSUPPORTED;
  if (codes && group != 32 && group != 128) return DSA_ERR_UNSUPPORTED;
  if (codes && scale_format != DSA_SCALE_FP32 && scale_format != DSA_SCALE_UE8M0)
    return DSA_ERR_UNSUPPORTED;
  const int groups = codes ? (N + group - 1) / group : 0;
  if (stride_short(x_stride, T, N) || (residual && stride_short(residual_stride, T, N)) ||
      (residual_out && stride_short(residual_out_stride, T, N)) ||
      (out && stride_short(out_stride, T, N)) ||
      (codes && (stride_short(codes_stride, T, N) || stride_short(scales_stride, T, groups))))
    return DSA_ERR_SHAPE;
  if (T == 0) return DSA_OK;
  if (!x || !gamma || (!out && !codes) || (codes && !scales) || (!residual && residual_out))
    return DSA_ERR_NULL;
  if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(residual_out, 16) ||
      misaligned(gamma, 16) || misaligned(out, 16) || misaligned(codes, 8) ||
      (codes && scale_format == DSA_SCALE_FP32 && misaligned(scales, 4)) ||
      stride_odd(x_stride, T) || (residual && stride_odd(residual_stride, T)) ||
      (residual_out && stride_odd(residual_out_stride, T)) || (out && stride_odd(out_stride, T)) ||
      (codes && stride_odd(codes_stride, T)))
    return DSA_ERR_ALIGN;
  NormParams p = {};
  p.x = static_cast<const uint16_t*>(x);
  p.residual = static_cast<const uint16_t*>(residual);
  p.residual_out = static_cast<uint16_t*>(residual_out);
  p.out = static_cast<uint16_t*>(out);
  p.codes = static_cast<uint8_t*>(codes);
  p.scales = scales;
  p.gamma = gamma;
  p.x_stride = x_stride;
  p.residual_stride = residual_stride;
  p.residual_out_stride = residual_out_stride;
  p.out_stride = out_stride;
  p.codes_stride = codes_stride;
  p.scales_stride = scales_stride;
  p.eps = eps;
  p.inv_n = 1.0f / static_cast<float>(N);
  p.T = T;
  p.pieces = N / 8;
  p.group_lanes = group / 8;
  p.scale_bytes = scale_format == DSA_SCALE_UE8M0 ? 1 : 4;
  auto row_threads = [&](int n) { return ((p.pieces + n - 1) / n + 31) / 32 * 32; };
  const int pieces = choose_pieces(T, row_threads);
  const int threads = row_threads(pieces);
  const int rows = threads < 128 && T > kSms ? 128 / threads : 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((T + rows - 1) / rows));
  cfg.blockDim = dim3(static_cast<unsigned>(threads), static_cast<unsigned>(rows));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = flags & DSA_FLAG_PDL ? 1 : 0;
  cudaError_t e;
  if (dtype == DSA_DTYPE_BF16)
    e = residual ? launch<true, true>(p, pieces, cfg) : launch<true, false>(p, pieces, cfg);
  else
    e = residual ? launch<false, true>(p, pieces, cfg)
                 : launch<false, false>(p, pieces, cfg);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}
