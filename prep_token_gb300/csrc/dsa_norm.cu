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
template <bool BF16, int PIECES>
__global__ void __launch_bounds__(kMaxRowThreads) dsa_rms_norm_kernel(const NormParams p) {
  __shared__ float sums[32];
  const int row = blockIdx.x * blockDim.y + threadIdx.y;
  const bool mine = row < p.T;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  float z[PIECES][8];
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    const bool some = mine && at < p.pieces;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (some) {
      a = load_piece(p.x + row * p.x_stride + 8 * at);
      if (p.residual) b = load_piece(p.residual + row * p.residual_stride + 8 * at);
    }
    unpack8<BF16>(a, z[i]);
    if (p.residual) {
      float r[8];
      unpack8<BF16>(b, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] += r[j];
    }
    if (p.residual_out && some)
      store_piece(p.residual_out + row * p.residual_out_stride + 8 * at, pack8<BF16>(z[i]));
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(z[i][j], z[i][j], sum);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  const int warps = blockDim.x >> 5;
  if (warps > 1) {
    const int first = threadIdx.y * warps;
    if (lane == 0) sums[first + (threadIdx.x >> 5)] = sum;
    __syncthreads();
    sum = lane < warps ? sums[first + lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  }
  const float rs = 1.0f / sqrtf(fmaf(sum, p.inv_n, p.eps));
#pragma unroll
  for (int i = 0; i < PIECES; ++i) {
    const int at = threadIdx.x + i * blockDim.x;
    const bool some = mine && at < p.pieces;
    float g[8] = {};
    if (some) {
      const float4 lo = __ldg(reinterpret_cast<const float4*>(p.gamma + 8 * at));
      const float4 hi = __ldg(reinterpret_cast<const float4*>(p.gamma + 8 * at + 4));
      g[0] = lo.x, g[1] = lo.y, g[2] = lo.z, g[3] = lo.w;
      g[4] = hi.x, g[5] = hi.y, g[6] = hi.z, g[7] = hi.w;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) z[i][j] = z[i][j] * rs * g[j];
    if (p.out && some) store_piece(p.out + row * p.out_stride + 8 * at, pack8<BF16>(z[i]));
    if (p.codes) {
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(z[i][j]));
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
      if (p.group_lanes == 16) {
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 4));
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 8));
      }
      const int e = exponent_of_amax(amax);
      const float down = pow2f(-e);
      if (some) {
        uint2 c;
        c.x = cvt_e4m3x2(z[i][0] * down, z[i][1] * down) |
              cvt_e4m3x2(z[i][2] * down, z[i][3] * down) << 16;
        c.y = cvt_e4m3x2(z[i][4] * down, z[i][5] * down) |
              cvt_e4m3x2(z[i][6] * down, z[i][7] * down) << 16;
        *reinterpret_cast<uint2*>(p.codes + row * p.codes_stride + 8 * at) = c;
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

template <bool BF16>
cudaError_t launch(const NormParams& p, int pieces, cudaLaunchConfig_t& cfg) {
  switch (pieces) {
    case 1: return cudaLaunchKernelEx(&cfg, dsa_rms_norm_kernel<BF16, 1>, p);
    case 2: return cudaLaunchKernelEx(&cfg, dsa_rms_norm_kernel<BF16, 2>, p);
    default: return cudaLaunchKernelEx(&cfg, dsa_rms_norm_kernel<BF16, 4>, p);
  }
}

}  // namespace

extern "C" dsa_status dsa_rms_norm(
    const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
    void* residual_out, int64_t residual_out_stride, const float* gamma, float eps, void* out,
    int64_t out_stride, void* codes, int64_t codes_stride, void* scales, int64_t scales_stride,
    int32_t scale_format, int32_t group, int32_t T, int32_t N, int32_t dtype, uint32_t flags,
    void* stream) {
  if (T < 0 || N < 1 || N % 8 || N > 8 * kMaxPieces * kMaxRowThreads) return DSA_ERR_SHAPE;
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
  // Few rows: a piece a thread, for the shortest way through.  Many: four, so
  // that the bytes in flight come from few warps.
  int pieces = T <= 2 * kSms ? 1 : kMaxPieces;
  auto row_threads = [&](int n) { return ((p.pieces + n - 1) / n + 31) / 32 * 32; };
  while (row_threads(pieces) > kMaxRowThreads) pieces *= 2;
  const int threads = row_threads(pieces);
  const int rows = T > 2 * kSms && threads < 256 ? 256 / threads : 1;
  while (pieces > 1 && (pieces / 2) * threads >= p.pieces) pieces /= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((T + rows - 1) / rows));
  cfg.blockDim = dim3(static_cast<unsigned>(threads), static_cast<unsigned>(rows));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = flags & DSA_FLAG_PDL ? 1 : 0;
  const cudaError_t e = dtype == DSA_DTYPE_BF16 ? launch<true>(p, pieces, cfg)
                                                : launch<false>(p, pieces, cfg);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}
