// 8-bit product with a scale per token and output channel:
//   y[m][n] = fl(fl(fl(acc) w_scale[n]) x_scale[m]), acc = sum_k w[n][k] x[m][k] exactly.
//
// Each warp takes four output channels and up to eight tokens; its lanes
// stride over k in 16-byte pieces with byte dot products.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "tern_internal.h"
#include "tern_ptx.cuh"

namespace tern {

int read_clear_dev_error_gemm_i8(void* stream, unsigned* out) { return read_clear_dev_error_tu(stream, out); }

namespace {

constexpr int kRows = 4, kTok = 8;

// 16 bytes of a row, zero from `left` bytes on
__device__ __forceinline__ int4 mask16(int4 v, int left) {
  if (left >= 16) return v;
  int w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int b = left - 4 * i;
    w[i] = b >= 4 ? w[i] : (b <= 0 ? 0 : w[i] & (int)((1u << (8 * b)) - 1u));
  }
  return make_int4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(256) dot_kernel(const GemmI8Params p) {
  const int lane = threadIdx.x & 31;
  const int n0 = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)) * kRows, m0 = (int)blockIdx.y * kTok;
  if (n0 >= p.n) return;
  int acc[kRows][kTok] = {};
  for (int k = lane * 16; k < p.k; k += 512) {
    int4 w[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      w[i] = mask16(*reinterpret_cast<const int4*>(p.w + (int64_t)min(n0 + i, p.n - 1) * p.ldw + k), p.k - k);
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (m0 + j >= p.m) break;
      const int4 x = *reinterpret_cast<const int4*>(p.x + (int64_t)(m0 + j) * p.ldx + k);
#pragma unroll
      for (int i = 0; i < kRows; ++i)
        acc[i][j] = __dp4a(w[i].x, x.x, __dp4a(w[i].y, x.y, __dp4a(w[i].z, x.z, __dp4a(w[i].w, x.w, acc[i][j]))));
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      const int v = __reduce_add_sync(0xffffffffu, acc[i][j]);
      if (lane == i * kTok + j && n0 + i < p.n && m0 + j < p.m) {
        const float y = __fmul_rn(__fmul_rn(__int2float_rn(v), p.wscale[n0 + i]), p.xscale[m0 + j]);
        const int64_t at = (int64_t)(m0 + j) * p.ldy + n0 + i;
        if (p.out_bf16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(y);
        else static_cast<float*>(p.y)[at] = y;
      }
    }
  }
}

}  // namespace

int launch_gemm_i8(const GemmI8Params& p, int sms, void* stream) {
  (void)sms;
  const dim3 grid((unsigned)((p.n + 8 * kRows - 1) / (8 * kRows)), (unsigned)((p.m + kTok - 1) / kTok));
  dot_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace tern

extern "C" tern_status tern_gemm_i8(int32_t m, int32_t n, int32_t k, const int8_t* d_x, int64_t ldx,
                                    const float* d_xscale, const int8_t* d_w, int64_t ldw, const float* d_wscale,
                                    tern_out out, void* d_y, int64_t ldy, void* stream) {
  using namespace tern;
  if (m < 0 || n < 1 || k < 1 || k > 131071 || ldx < k || ldw < k || ldy < n || ((ldx | ldw) & 15) != 0)
    return TERN_EINVAL;
  if (out != TERN_OUT_F32 && out != TERN_OUT_BF16) return TERN_EINVAL;
  if (m > 65535 * 8) return TERN_EINVAL;
  if (m == 0) return TERN_OK;
  if (!d_x || !d_xscale || !d_w || !d_wscale || !d_y) return TERN_EINVAL;
  if (((reinterpret_cast<uintptr_t>(d_x) | reinterpret_cast<uintptr_t>(d_w)) & 15u) != 0) return TERN_EALIGN;
  const uintptr_t esize = out == TERN_OUT_F32 ? 3u : 1u;
  if (((reinterpret_cast<uintptr_t>(d_xscale) | reinterpret_cast<uintptr_t>(d_wscale)) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(d_y) & esize) != 0)
    return TERN_EALIGN;
  GemmI8Params p{};
  p.x = d_x;
  p.w = d_w;
  p.xscale = d_xscale;
  p.wscale = d_wscale;
  p.y = d_y;
  p.ldx = ldx;
  p.ldw = ldw;
  p.ldy = ldy;
  p.m = m;
  p.n = n;
  p.k = k;
  p.out_bf16 = out == TERN_OUT_BF16;
  return launch_gemm_i8(p, sm_count(), stream) == 0 ? TERN_OK : TERN_ECUDA;
}
