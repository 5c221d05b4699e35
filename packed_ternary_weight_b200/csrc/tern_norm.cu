// RMSNorm with the residual's addition or the gated activation in front and
// the per-row int8 quantisation behind it: the input of every int8 product of
// a layer (QORA-LLM-2B page, "SubLN Pattern (4 norms per layer)"), for many
// rows. The values are those of the decode step's normalisations:
//   f = fl32(1 / sqrt(mean(v^2) + eps)), the sum and the root in fp64 (each
//   v^2 is exact there, and sums in any order agree far below f's own rounding);
//   y = fl32(fl32(v f) gain); a = max |y|; q = clamp(rint(fl32(y fl32(127 / a))), -127, 127).
// A row in which some v, f or y is not finite has a scale that is not finite, and codes 0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "tern_internal.h"
#include "tern_launch.cuh"
#include "tern_ptx.cuh"

namespace tern {
namespace {

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
// The larger one, not a number if either is not: a row's maximum must show what stands in the row.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) {
  return __bfloat162float(__float2bfloat16_rn(v));
}

template <int MODE, typename RT>
__device__ __forceinline__ float combine(float x, float r) {
  if constexpr (MODE == TERN_NORM_ADD) return round_to(__fadd_rn(x, r), static_cast<const RT*>(nullptr));
  if constexpr (MODE == TERN_NORM_RELU2) {
    const float g = max_nan(x, 0.f);
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
  for (int o = 16; o; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  a = (int)(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// One row per block, any k, stride and alignment (rows that do not fit or align): the row is read again for
// each of the three steps.
template <int MODE, typename XT, typename RT>
__global__ void __launch_bounds__(256) norm_any_kernel(const NormParams p) {
  __shared__ double red[33];
  __shared__ float redf[32];
  pdl_launch_dependents();
  pdl_wait();
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
  for (int i = threadIdx.x; i < k; i += blockDim.x) a = max_nan(a, fabsf(y(i)));
  a = row_max(a, redf);
  const float inv = a > 0.f ? __fdiv_rn(127.0f, a) : 0.f;
  int8_t* q = p.xq + (int64_t)row * p.ldq;
  for (int i = threadIdx.x; i < k; i += blockDim.x) {
    const float v = y(i);
    q[i] = v != 0.f ? quant(v, inv) : (int8_t)0;
  }
  if (threadIdx.x == 0) p.xscale[row] = a > 0.f ? __fdiv_rn(a, 127.0f) : a;
}

// Two fp32 operations in one instruction, each rounded as its own (only where no
// product meets a sum: the compiler makes one rounding of such a packed pair).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// Eight elements as they stand in memory, and their values.
template <typename T>
struct Raw8 {
  uint4 u, w;
  __device__ __forceinline__ void load(const T* p) {
    u = reinterpret_cast<const uint4*>(p)[0];
    w = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { u = w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void values(float2 (&v)[4]) const {
    v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    v[2] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
    v[3] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { u = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void values(float2 (&v)[4]) const {
    const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float2(__uint_as_float(e[i] << 16), __uint_as_float(e[i] & 0xFFFF0000u));
  }
};
__device__ __forceinline__ void st8(float* p, const float2 (&v)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float2 (&v)[4]) {
  uint32_t e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[i].x, v[i].y);
    e[i] = *reinterpret_cast<const uint32_t*>(&a);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(e[0], e[1], e[2], e[3]);
}
template <int MODE, typename RT>
__device__ __forceinline__ float2 combine2(float2 x, float2 r) {
  if constexpr (MODE == TERN_NORM_ADD) {
    const float2 v = add2(x, r);
    return make_float2(round_to(v.x, static_cast<const RT*>(nullptr)), round_to(v.y, static_cast<const RT*>(nullptr)));
  }
  if constexpr (MODE == TERN_NORM_RELU2) {
    const float2 g = make_float2(max_nan(x.x, 0.f), max_nan(x.y, 0.f));
    return mul2(mul2(g, g), r);
  }
  return x;
}

// Rows read once: thread i holds the vectors of eight i, i + T, .. (NV of them) in
// registers through all three steps, and the next row's are on their way meanwhile
// (a block takes the rows blockIdx, blockIdx + grid, ..): the kernel is bound by
// memory once the three block-wide steps of a row are hidden behind the next row's loads.
template <int MODE, typename XT, typename RT, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_row_kernel(const NormParams p) {
  __shared__ double red[33];
  __shared__ float redf[2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int k = p.k, T = blockDim.x, first = 8 * (int)threadIdx.x, step = 8 * T;
  Raw8<XT> xw[NV];
  Raw8<RT> rw[NV];
  auto load = [&](int row) {
    const XT* x = static_cast<const XT*>(p.x) + (int64_t)row * p.ldx + first;
    const RT* r = static_cast<const RT*>(p.r) + (int64_t)row * p.ldr + first;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xw[j].zero();
      rw[j].zero();
      if (row < p.m && first + j * step < k) {
        xw[j].load(x + j * step);
        if (MODE != TERN_NORM_PLAIN) rw[j].load(r + j * step);
      }
    }
  };
  // eight gains of the vector at j; a thread with one vector holds them from the start, ahead of the row's three steps (1 x
  // 4096: 2.7 us, 2.85 us with the gains read behind the factor; with two vectors the registers are worth more)
  float4 held[2];
  auto gains = [&](int j, float4 (&g)[2]) {
    const float4* src = reinterpret_cast<const float4*>(p.gain + first + j * step);
    g[0] = src[0], g[1] = src[1];
  };
  if (NV == 1 && first < k) gains(0, held);
  load(blockIdx.x);
  int turn = 0;
  for (int row = blockIdx.x; row < p.m; row += gridDim.x, turn ^= 1) {
    float2 v[NV][4];
    double s0 = 0.0, s1 = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float2 r[4];
      xw[j].values(v[j]);
      rw[j].values(r);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[j][e] = combine2<MODE, RT>(v[j][e], r[e]);
        s0 = fma((double)v[j][e].x, (double)v[j][e].x, s0);
        s1 = fma((double)v[j][e].y, (double)v[j][e].y, s1);
      }
      if (MODE == TERN_NORM_ADD && first + j * step < k)
        st8(static_cast<RT*>(p.sum) + (int64_t)row * p.ldsum + first + j * step, v[j]);
    }
    load(row + gridDim.x);
    const float f = row_factor(s0 + s1, k, p.eps, red);
    const float2 f2 = make_float2(f, f);
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (first + j * step < k) {
        float4 g[2];
        if (NV == 1)
          g[0] = held[0], g[1] = held[1];
        else
          gains(j, g);
        const float2 gain[4] = {make_float2(g[0].x, g[0].y), make_float2(g[0].z, g[0].w), make_float2(g[1].x, g[1].y),
                                make_float2(g[1].z, g[1].w)};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[j][e] = mul2(mul2(v[j][e], f2), gain[e]);
          a = max_nan(a, max_nan(fabsf(v[j][e].x), fabsf(v[j][e].y)));
        }
      }
    }
    a = row_max(a, redf[turn]);
    const float inv = a > 0.f ? __fdiv_rn(127.0f, a) : 0.f;
    int8_t* out = p.xq + (int64_t)row * p.ldq + first;
    auto store = [&](auto word) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (first + j * step < k)
          *reinterpret_cast<uint2*>(out + j * step) = make_uint2(word(v[j][0], v[j][1]), word(v[j][2], v[j][3]));
    };
    if (inv > 0.f && inv != INFINITY) {
      // |y| <= a, so |y inv| is at most 127 (1 + 2^-22): the sum with 1.5 * 2^23 rounds it to the integer (ties to
      // even) that its low byte holds, and no clamp is needed
      // (one by one: the packed product and sum are contracted into one rounding)
      auto low = [&](float y) { return __float_as_uint(__fadd_rn(__fmul_rn(y, inv), 12582912.f)); };
      store([&](float2 x, float2 y) {
        return __byte_perm(__byte_perm(low(x.x), low(x.y), 0x0040), __byte_perm(low(y.x), low(y.y), 0x0040), 0x5410);
      });
    } else {  // a tiny row takes the definition's steps, and one that is empty or not finite gets zeros
      auto q = [&](float y) { return (uint32_t)(y != 0.f ? quant(y, inv) : 0) & 0xFFu; };
      store([&](float2 x, float2 y) { return q(x.x) | (q(x.y) << 8) | (q(y.x) << 16) | (q(y.y) << 24); });
    }
    if (threadIdx.x == 0) p.xscale[row] = a > 0.f ? __fdiv_rn(a, 127.0f) : a;
  }
}

// Whether a row can be read in vectors of eight.
bool vectors(const NormParams& p) {
  auto ok = [](const void* q, int64_t ld, int bytes) {  // 16-byte pieces; 8 bytes of codes
    const int unit = bytes == 1 ? 8 : 16;
    return !q || ((reinterpret_cast<uintptr_t>(q) & (uintptr_t)(unit - 1)) == 0 && ld * bytes % unit == 0);
  };
  return p.k % 8 == 0 && ok(p.x, p.ldx, p.x_bf16 ? 2 : 4) && ok(p.r, p.ldr, p.r_bf16 ? 2 : 4) &&
         ok(p.sum, p.ldsum, p.r_bf16 ? 2 : 4) && ok(p.xq, p.ldq, 1) && ok(p.gain, 4, 4);
}

// Vectors per thread: two where there are rows enough to fill the device, one
// where a row's latency counts (1 x 2560: 2.4 us, 6.6 us with the row read three
// times by 256 threads) and a block's threads suffice. About 1024 threads per
// multiprocessor, the registers of the next row included: 8192 x 4096 with the
// residual 62 us (0.92 of the measured copy rate; 76 us with 640 threads), 4096 x
// 2560 28 us, 2043 x 6912 gated 19 us (0.57 of the copy rate: DRAM 31 %, issue 51 %, fp64
// 7 %; warps wait for each other and for shared memory in the three block-wide steps,
// which 28 warps per multiprocessor do not hide). Rows read three times, element by
// element: 2043 x 6911 fp32 with the residual 76 us, where 6912 columns take 36.
template <int MODE, typename XT, typename RT>
int launch_mode(const NormParams& p, cudaStream_t s) {
  const int nv = p.k / 8;
  if (nv > 2048 || !vectors(p)) return launch_dependent(norm_any_kernel<MODE, XT, RT>, p.m, 256, 0, 1, s, p);
  const bool few = p.m < 2 * sm_count();
  const int per = nv > 1024 || !few ? 2 : 1;
  const int threads = std::max(64, ((nv + per - 1) / per + 31) / 32 * 32);
  const int grid = std::min(p.m, std::max(2, 1024 / threads) * sm_count());
  if (per == 1) return launch_dependent(norm_row_kernel<MODE, XT, RT, 1, 1024, 1>, grid, threads, 0, 1, s, p);
  if (threads <= 512) return launch_dependent(norm_row_kernel<MODE, XT, RT, 2, 512, 2>, grid, threads, 0, 1, s, p);
  return launch_dependent(norm_row_kernel<MODE, XT, RT, 2, 1024, 1>, grid, threads, 0, 1, s, p);
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
  if (m < 0 || m > kMaxExtent || k < 1 || k > kMaxExtent || !(eps > 0.f) || ldx < k || ldq < k ||
      (two && ldr < k) || (add && ldsum < k))
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
