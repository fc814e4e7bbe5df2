// Rows of 16-bit values (bf16 or fp16) in 16-byte pieces of eight: loads that
// leave L1 alone, conversions to fp32 and back.  Shared by the kernels that
// stream rows (norm, append).
#ifndef DSA_ROWS_CUH
#define DSA_ROWS_CUH

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "dsa_common.cuh"

namespace dsa_rows {

using namespace dsa_dev;

// Eight values that are read once.  Not the read-only path: a row may be
// written where it was read (by the thread that read it).
__device__ __forceinline__ uint4 load_piece(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void store_piece(uint16_t* p, const uint4& v) {
  *reinterpret_cast<uint4*>(p) = v;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF16) return make_float2(bf16_lo(w), bf16_hi(w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Two values rounded to nearest, ties to even.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&x)[4]) {
  x[0] = unpack2<BF16>(v.x), x[1] = unpack2<BF16>(v.y);
  x[2] = unpack2<BF16>(v.z), x[3] = unpack2<BF16>(v.w);
}

template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float2 (&x)[4]) {
  return make_uint4(pack2<BF16>(x[0].x, x[0].y), pack2<BF16>(x[1].x, x[1].y),
                    pack2<BF16>(x[2].x, x[2].y), pack2<BF16>(x[3].x, x[3].y));
}

// Host side: the checks that these rows' pointers and strides share.
inline bool misaligned(const void* ptr, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) != 0;
}

// A stride of rows of `width` values, `extent` of them: apart, and 16-byte pieces stay aligned.
inline bool stride_short(int64_t stride, int64_t extent, int64_t width) {
  return extent > 1 && (stride < width || stride >= (1LL << 39));
}
inline bool stride_odd(int64_t stride, int64_t extent) { return extent > 1 && stride % 8 != 0; }

// Whether rows of `width` values at i * stride[0] + j * stride[1] + k * stride[2]
// are apart: in the order of the strides, each passes what the smaller ones span.
inline bool rows_apart(int64_t width, const int64_t (&extent)[3], const int64_t (&stride)[3]) {
  bool done[3] = {extent[0] < 2, extent[1] < 2, extent[2] < 2};
  __int128 span = width;
  for (int step = 0; step < 3; ++step) {
    int next = -1;
    for (int i = 0; i < 3; ++i)
      if (!done[i] && (next < 0 || stride[i] < stride[next])) next = i;
    if (next < 0) break;
    if (stride[next] < span) return false;
    span += static_cast<__int128>(stride[next]) * (extent[next] - 1);
    done[next] = true;
  }
  return true;
}

}  // namespace dsa_rows

#endif  // DSA_ROWS_CUH
