// New tokens' K and V into the paged cache that dsa_paged_attention reads, with
// an optional RMS norm of every q and k head and the position rotation (RoPE)
// on the way; q goes out rotated in the same launch.
//
//   x = q or k of a head, in fp32
//   x *= gamma / sqrt(mean(x^2) + eps)                    (where gamma is given)
//   RoPE on x[0:rope_dim): a' = fma(a, c, -(b s)), b' = fma(b, c, a s)
//   rounded once; k and v to slot out_cache_loc[t] of their caches, q to q_out
//
// A head's row of D values is D / 16 lanes wide, two 16-byte pieces to a lane:
// the pieces of a lane that rotates are the two halves of its pairs (NeoX), or
// neighbours (GPT-J and the values that pass through).  A pair is in one lane
// and needs no shuffle; a norm's sum takes log2(D / 16) of them.  A warp works
// on one token, whose cos/sin row it reads once, and 512 / D heads at a time.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "dsa_prep.h"
#include "dsa_rows.cuh"

namespace {

using namespace dsa_rows;

constexpr int kSms = 152;
constexpr int kWarps = 8;  // of a CTA

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
  int passes;       // of a warp: it takes passes * (512 / D) heads of a token
  int chunks;       // warps of a token
  int* err;
};

template <bool BF16, int D, int STYLE>
__global__ void __launch_bounds__(32 * kWarps)
    dsa_kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 16;        // of a row
  constexpr int kRowsOf = 32 / kLanes;  // rows that a warp takes at a time
  const int lane = threadIdx.x & 31;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int t = item / p.chunks, chunk = item - t * p.chunks;
  grid_dependency_wait();
  grid_launch_dependents();
  if (t >= p.T) return;
  const long long pos = p.positions[t], slot = p.slots[t];
  if (pos < 0 || pos >= p.max_position) {
    if (lane == 0 && chunk == 0 && p.err) atomicOr(p.err, DSA_DEVERR_POSITION);
    return;
  }
  const bool keep = slot >= 0 && slot < p.num_slots;
  if (!keep && lane == 0 && chunk == 0 && p.err) atomicOr(p.err, DSA_DEVERR_SLOT);
  long long page = 0, in_page = 0;
  if (keep) {
    if (p.page_shift >= 0) {
      page = slot >> p.page_shift;
      in_page = slot & (p.page_size - 1);
    } else {
      page = slot / p.page_size;
      in_page = slot - page * p.page_size;
    }
  }
  const bool turns = l < p.turns;
  const int first = STYLE == DSA_ROPE_NEOX && turns ? l : 2 * l;  // the lane's pieces
  const int second = STYLE == DSA_ROPE_NEOX && turns ? l + p.turns : 2 * l + 1;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.0f, s[i] = 0.0f;
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(p.cos + pos * p.cs_stride + 8 * l + i));
      const float4 w = __ldg(reinterpret_cast<const float4*>(p.sin + pos * p.cs_stride + 8 * l + i));
      c[i] = u.x, c[i + 1] = u.y, c[i + 2] = u.z, c[i + 3] = u.w;
      s[i] = w.x, s[i + 1] = w.y, s[i + 2] = w.z, s[i + 3] = w.w;
    }
  }
  const int rows = p.H + 2 * p.Hkv;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int row = (chunk * p.passes + pass) * kRowsOf + sub;
    const bool is_q = row < p.H, is_v = row >= p.H + p.Hkv;
    const int h = is_q ? row : is_v ? row - p.H - p.Hkv : row - p.H;
    const bool some = row < rows && (is_q || keep);
    const uint16_t* from = is_q ? p.q + t * p.q_t + h * p.q_h
                         : is_v ? p.v + t * p.v_t + h * p.v_h : p.k + t * p.k_t + h * p.k_h;
    uint16_t* to = is_q ? p.q_out + t * p.out_t + h * p.out_h
                 : is_v ? p.v_cache + page * p.vc_page + in_page * p.vc_token + h * p.vc_head
                        : p.k_cache + page * p.kc_page + in_page * p.kc_token + h * p.kc_head;
    uint4 u = make_uint4(0, 0, 0, 0), w = u;
    if (some) {
      u = load_piece(from + 8 * first);
      w = load_piece(from + 8 * second);
    }
    float a[8], b[8];
    unpack8<BF16>(u, a);
    unpack8<BF16>(w, b);
    const float* gamma = is_v ? nullptr : is_q ? p.q_gamma : p.k_gamma;
    if (p.q_gamma || p.k_gamma) {  // the whole warp: its rows may be of more than one kind
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(a[i], a[i], fmaf(b[i], b[i], sum));
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (gamma) {
        const float rs = 1.0f / sqrtf(fmaf(sum, 1.0f / D, p.eps));
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
          const float4 g = __ldg(reinterpret_cast<const float4*>(gamma + 8 * first + i));
          const float4 f = __ldg(reinterpret_cast<const float4*>(gamma + 8 * second + i));
          a[i] *= rs * g.x, a[i + 1] *= rs * g.y, a[i + 2] *= rs * g.z, a[i + 3] *= rs * g.w;
          b[i] *= rs * f.x, b[i + 1] *= rs * f.y, b[i + 2] *= rs * f.z, b[i + 3] *= rs * f.w;
        }
      }
    }
    if (turns && !is_v) {
      if (STYLE == DSA_ROPE_NEOX) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = a[i], y = b[i];
          a[i] = fmaf(x, c[i], -__fmul_rn(y, s[i]));
          b[i] = fmaf(y, c[i], __fmul_rn(x, s[i]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x = a[2 * i], y = a[2 * i + 1];
          a[2 * i] = fmaf(x, c[i], -__fmul_rn(y, s[i]));
          a[2 * i + 1] = fmaf(y, c[i], __fmul_rn(x, s[i]));
          x = b[2 * i], y = b[2 * i + 1];
          b[2 * i] = fmaf(x, c[4 + i], -__fmul_rn(y, s[4 + i]));
          b[2 * i + 1] = fmaf(y, c[4 + i], __fmul_rn(x, s[4 + i]));
        }
      }
    }
    if (gamma || (turns && !is_v)) {
      u = pack8<BF16>(a);
      w = pack8<BF16>(b);
    }
    if (some) {
      store_piece(to + 8 * first, u);
      store_piece(to + 8 * second, w);
    }
  }
}

template <bool BF16, int D>
cudaError_t launch(const AppendParams& p, int style, const cudaLaunchConfig_t& cfg) {
  return style == DSA_ROPE_NEOX
             ? cudaLaunchKernelEx(&cfg, dsa_kv_append_kernel<BF16, D, DSA_ROPE_NEOX>, p)
             : cudaLaunchKernelEx(&cfg, dsa_kv_append_kernel<BF16, D, DSA_ROPE_GPTJ>, p);
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
  const int passes = (H + 2 * Hkv + 512 / head_dim - 1) / (512 / head_dim);  // of a token
  p.passes = 1;
  p.chunks = (passes + p.passes - 1) / p.passes;
  p.err = err_flags;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const long long warps = static_cast<long long>(T) * p.chunks;
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = flags & DSA_FLAG_PDL ? 1 : 0;
  const bool bf16 = dtype == DSA_DTYPE_BF16;
  cudaError_t e;
  if (head_dim == 64)
    e = bf16 ? launch<true, 64>(p, rope_style, cfg) : launch<false, 64>(p, rope_style, cfg);
  else
    e = bf16 ? launch<true, 128>(p, rope_style, cfg) : launch<false, 128>(p, rope_style, cfg);
  return e == cudaSuccess ? DSA_OK : DSA_ERR_LAUNCH;
}
