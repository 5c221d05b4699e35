// RMSNorm with the residual's addition or the gated activation in front and
// the per-row int8 quantisation behind it: the input of every int8 product of
// a layer (QORA-LLM-2B page, "SubLN Pattern (4 norms per layer)"), for many
// rows. The values are those of the decode step's normalisations:
//   f = fl32(1 / sqrt(mean(v^2) + eps)), the sum and the root in fp64 (each
//   v^2 is exact there, so the order of the sum does not show in f);
//   y = fl32(fl32(v f) gain); a = max |y|; q = clamp(rint(fl32(y fl32(127 / a))), -127, 127).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tern_internal.h"

namespace tern {
namespace {

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

template <int MODE, typename RT>
__device__ __forceinline__ float combine(float x, float r) {
  if constexpr (MODE == TERN_NORM_ADD) return round_to(__fadd_rn(x, r), static_cast<const RT*>(nullptr));
  if constexpr (MODE == TERN_NORM_RELU2) {
    const float g = fmaxf(x, 0.f);
    return __fmul_rn(__fmul_rn(g, g), r);
  }
  return x;
}

__device__ __forceinline__ int8_t quant(float y, float inv) {
  return (int8_t)max(-127, min(127, __float2int_rn(__fmul_rn(y, inv))));
}

// The row's factor f from every thread's part of the sum of squares, and the
// largest |y|; one call of each per row by all threads.
__device__ __forceinline__ float row_factor(double ss, int k, float eps, double* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
  __syncthreads();
  if (threadIdx.x < 32) {
    double s = (int)threadIdx.x < warps ? red[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (threadIdx.x == 0) red[32] = 1.0 / sqrt(s / (double)k + (double)eps);
  }
  __syncthreads();
  return (float)red[32];
}
__device__ __forceinline__ float row_max(float a, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  a = (int)(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// One row per block, any k, stride and alignment: the row is read again for
// each of the three steps.
template <int MODE, typename XT, typename RT>
__global__ void __launch_bounds__(256) norm_any_kernel(const NormParams p) {
  __shared__ double red[33];
  __shared__ float redf[32];
  const int row = blockIdx.x, k = p.k;
  const XT* x = static_cast<const XT*>(p.x) + (int64_t)row * p.ldx;
  const RT* r = MODE == TERN_NORM_PLAIN ? nullptr : static_cast<const RT*>(p.r) + (int64_t)row * p.ldr;
  RT* sum = MODE == TERN_NORM_ADD ? static_cast<RT*>(p.sum) + (int64_t)row * p.ldsum : nullptr;
  double ss = 0.0;
  for (int i = threadIdx.x; i < k; i += blockDim.x) {
    const float v = combine<MODE, RT>(ld1(x + i), r ? ld1(r + i) : 0.f);
    if (sum) st1(sum + i, v);
    ss += (double)v * (double)v;
  }
  // from here on a residual sum is read back from where this thread wrote it (it may stand where r stood)
  const float f = row_factor(ss, k, p.eps, red);
  auto y = [&](int i) {
    const float v = sum ? ld1(sum + i) : combine<MODE, RT>(ld1(x + i), r ? ld1(r + i) : 0.f);
    return __fmul_rn(__fmul_rn(v, f), p.gain[i]);
  };
  float a = 0.f;
  for (int i = threadIdx.x; i < k; i += blockDim.x) a = fmaxf(a, fabsf(y(i)));
  a = row_max(a, redf);
  const float inv = a > 0.f ? __fdiv_rn(127.0f, a) : 0.f;
  int8_t* q = p.xq + (int64_t)row * p.ldq;
  for (int i = threadIdx.x; i < k; i += blockDim.x) {
    const float v = y(i);
    q[i] = v != 0.f ? quant(v, inv) : (int8_t)0;
  }
  if (threadIdx.x == 0) p.xscale[row] = a > 0.f ? __fdiv_rn(a, 127.0f) : 0.f;
}

template <int MODE, typename XT, typename RT>
int launch_mode(const NormParams& p, cudaStream_t s) {
  norm_any_kernel<MODE, XT, RT><<<p.m, 256, 0, s>>>(p);
  return (int)cudaGetLastError();
}

template <int MODE>
int launch_types(const NormParams& p, cudaStream_t s) {
  if constexpr (MODE == TERN_NORM_PLAIN) {
    return p.x_bf16 ? launch_mode<MODE, __nv_bfloat16, float>(p, s) : launch_mode<MODE, float, float>(p, s);
  } else {
    if (p.x_bf16)
      return p.r_bf16 ? launch_mode<MODE, __nv_bfloat16, __nv_bfloat16>(p, s)
                      : launch_mode<MODE, __nv_bfloat16, float>(p, s);
    return p.r_bf16 ? launch_mode<MODE, float, __nv_bfloat16>(p, s) : launch_mode<MODE, float, float>(p, s);
  }
}

bool aligned_to(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }

}  // namespace

int launch_norm(const NormParams& p, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (p.mode) {
    case TERN_NORM_PLAIN: return launch_types<TERN_NORM_PLAIN>(p, s);
    case TERN_NORM_ADD: return launch_types<TERN_NORM_ADD>(p, s);
    default: return launch_types<TERN_NORM_RELU2>(p, s);
  }
}

}  // namespace tern

extern "C" tern_status tern_norm_quantize(tern_norm mode, int32_t m, int32_t k, tern_out x_type, const void* d_x,
                                          int64_t ldx, tern_out r_type, const void* d_r, int64_t ldr,
                                          const float* d_gain, float eps, void* d_sum, int64_t ldsum, int8_t* d_xq,
                                          int64_t ldq, float* d_xscale, void* stream) {
  using namespace tern;
  if (mode != TERN_NORM_PLAIN && mode != TERN_NORM_ADD && mode != TERN_NORM_RELU2) return TERN_EINVAL;
  if (x_type != TERN_OUT_F32 && x_type != TERN_OUT_BF16) return TERN_EINVAL;
  const bool two = mode != TERN_NORM_PLAIN, add = mode == TERN_NORM_ADD;
  if (two && r_type != TERN_OUT_F32 && r_type != TERN_OUT_BF16) return TERN_EINVAL;
  if (m < 0 || k < 1 || !(eps > 0.f) || ldx < k || ldq < k || (two && ldr < k) || (add && ldsum < k))
    return TERN_EINVAL;
  if (m == 0) return TERN_OK;
  if (!d_x || !d_gain || !d_xq || !d_xscale || (two && !d_r) || (add && !d_sum)) return TERN_EINVAL;
  if (add && d_sum == d_r && ldsum != ldr) return TERN_EINVAL;
  const int xb = x_type == TERN_OUT_BF16 ? 2 : 4, rb = r_type == TERN_OUT_BF16 ? 2 : 4;
  if (!aligned_to(d_x, xb) || !aligned_to(d_gain, 4) || !aligned_to(d_xscale, 4) || (two && !aligned_to(d_r, rb)) ||
      (add && !aligned_to(d_sum, rb)))
    return TERN_EALIGN;
  NormParams p{};
  p.x = d_x;
  p.r = two ? d_r : nullptr;
  p.gain = d_gain;
  p.sum = add ? d_sum : nullptr;
  p.xq = d_xq;
  p.xscale = d_xscale;
  p.ldx = ldx;
  p.ldr = ldr;
  p.ldsum = ldsum;
  p.ldq = ldq;
  p.m = m;
  p.k = k;
  p.mode = mode;
  p.x_bf16 = xb == 2;
  p.r_bf16 = rb == 2;
  p.eps = eps;
  return launch_norm(p, stream) == 0 ? TERN_OK : TERN_ECUDA;
}
