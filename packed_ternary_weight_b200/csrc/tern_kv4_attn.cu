// Attention of a step's new tokens over the paged 4-bit cache, for few query
// rows per sequence and kv head: single tokens, or a few at a time.
//
// Mathematics. A key of the cache is k = m + s c with codes c in 0..15 and one
// (s, m) per token and head, so q k = s (q c) + m sum(q): the tensor cores
// multiply q by the codes alone and the scales enter once per score. In the
// same way sum_j p_j v_j = sum_j (p_j s_j) c_j + sum_j p_j m_j, where the second
// sum is one number per query row. A code becomes a bf16 operand with one
// logic operation: the bit pattern 0x4300 | c is the bf16 number 128 + c, and
// the 128s leave by 128 sum(q) per score and 128 sum_j bf16(p_j s_j) per row.
// Softmax in base 2 with a running maximum; sums and statistics in fp32. The
// probabilities times value scales are rounded to bf16 (half a step, 2^-9
// relative, is below the bf16 rounding of the output), and the 128 sum uses the
// rounded ones.
//
// Layout. The scores are computed transposed, tokens x query rows
// (m16n8k16): sixteen tokens of codes fill the A operand and eight query rows
// the B operand, so one sequence's group of up to eight heads costs no padding
// in the large dimension. The contraction may run over the dimensions in any
// order, so lane 4 r + t takes the D/4 consecutive dimensions of token r that
// are one 16-byte load (D = 128), and q is loaded in the same order. The
// second product is transposed too, dimensions x rows: its A operand pairs the
// same dimension of two tokens by byte permutation, and its B operand is the
// bf16 probability matrix transposed in registers by movmatrix.
//
// Split. A CTA takes (sequence, kv head, tile of query rows, chunk of
// positions); its eight warps take 32 positions in turn with softmax states of
// their own, joined in shared memory. Chunks of one tile are joined by the last
// CTA to arrive, in chunk order, so results do not depend on timing.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "tern_kv4.cuh"

namespace tern {

int read_clear_dev_error_kv4_attn(void* stream, unsigned* out) { return read_clear_dev_error_tu(stream, out); }

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 32;  // positions a warp takes at a time

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
// Codes at bits 4 I .. + 3 of both halves as the bf16 pair 128 + c.
template <int I>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  return ((w >> (4 * I)) & 0x000F000Fu) | 0x43004300u;
}
__device__ __forceinline__ uint32_t lo16(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi16(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
__device__ __forceinline__ float2 half2_at(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

template <int WORDS>
__device__ __forceinline__ void ldg_words(uint32_t (&v)[WORDS], const uint8_t* p) {
  if constexpr (WORDS == 4) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else if constexpr (WORDS == 2) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = u.x, v[1] = u.y;
  } else {
    v[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}

template <int D, int NT>
struct Shared {
  static constexpr int kRows = 8 * NT, kPitch = D + 4;
  float m[kWarps][kRows], l[kWarps][kRows];
  float o[kWarps][kRows][kPitch];
  int last;
};

// Joins `n` softmax states (m_i, l_i, o_i[4]) in order; the factor of each is 2^(m_i - max).
struct Join {
  float mx = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(float m, float li, float4 v) {
    const float w = m == -INFINITY ? 0.f : ex2(m - mx);
    l = fmaf(w, li, l);
    o[0] = fmaf(w, v.x, o[0]);
    o[1] = fmaf(w, v.y, o[1]);
    o[2] = fmaf(w, v.z, o[2]);
    o[3] = fmaf(w, v.w, o[3]);
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) attn_kernel(const Kv4AttnParams p) {
  constexpr int R = 8 * NT;          // query rows of the tile
  constexpr int KW = D / 32;         // words of K codes per lane and token
  constexpr int VW = D / 64;         // words of V codes per lane and token
  constexpr int MT = D / 16;         // 16-dimension tiles of the output
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared<D, NT>& sm = *reinterpret_cast<Shared<D, NT>*>(smem_raw);
  const Kv4Params& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const int unit = blockIdx.x / p.splits, sp = blockIdx.x - unit * p.splits;
  const int tile = unit % p.tiles, sh = unit / p.tiles;
  const int h = sh % c.kv_heads, s = sh / c.kv_heads;
  const kv4::Seq q = kv4::load_seq(c, s);
  if (!q.ok) {
    if (sp == 0 && threadIdx.x == 0) kv4::report_bad();
    return;
  }
  const int G = p.group, rows = q.n * G, row_first = tile * R;
  if (row_first >= rows) return;
  const int row_last = min(rows, row_first + R) - 1;
  const int limit_max = q.len - q.n + row_last / G + 1;  // positions that the tile's last token sees
  const int ns = limit_max > 0 ? (limit_max + p.chunk - 1) / p.chunk : 1;
  if (sp >= ns) return;
  const int begin = sp * p.chunk, end = min(limit_max, begin + p.chunk);

  // q in the order of the key words; sums of its rows
  uint32_t qf[NT][2 * KW][2];
  float sumq[NT][2];
  int lim[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int row = row_first + 8 * j + r, tok = row / G;
    float sum = 0.f;
    if (row < rows) {
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + ((size_t)(q.row0 + tok) * c.heads + (size_t)h * G + (row - tok * G)) * D + t * (D / 4));
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const uint4 u = src[w];
        qf[j][2 * w][0] = lo16(u.x, u.z);
        qf[j][2 * w][1] = hi16(u.x, u.z);
        qf[j][2 * w + 1][0] = lo16(u.y, u.w);
        qf[j][2 * w + 1][1] = hi16(u.y, u.w);
        const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += __uint_as_float(e[i] << 16) + __uint_as_float(e[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int w = 0; w < 2 * KW; ++w) qf[j][w][0] = qf[j][w][1] = 0u;
    }
    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sumq[j][e] = __shfl_sync(0xffffffffu, sum, (2 * t + e) * 4);
      const int rw = row_first + 8 * j + 2 * t + e;
      lim[j][e] = rw < rows ? min(end, q.len - q.n + rw / G + 1) : 0;
    }
  }

  float o[NT][MT][4], m[NT][2], l[NT][2], corr[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < MT; ++i) o[j][i][0] = o[j][i][1] = o[j][i][2] = o[j][i][3] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) m[j][e] = -INFINITY, l[j][e] = 0.f, corr[j][e] = 0.f;
  }
  const size_t vofs = (size_t)c.page * (D / 2), pofs = (size_t)c.page * D;

  for (int t0 = begin + kStep * warp; t0 < end; t0 += kStep * kWarps) {
    float sc[2][NT][4];
    uint32_t vw[2][4][VW];
    float2 vs[2][2];
    bool good[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int pos = t0 + 16 * g;
      int page = -1;
      if (pos < end) {  // the same in all lanes
        page = kv4::page_of(c, s, pos);
        if (page < 0 && lane == 0) kv4::report_bad();
      }
      good[g] = page >= 0;
      // a group that is masked as a whole reads page 0 instead (in bounds, unused)
      const uint8_t* blk = c.pages + kv4::block_offset(c, good[g] ? page : 0, h);
      const int slot = pos & (c.page - 1);
      uint32_t ka[KW], kb[KW];
      ldg_words<KW>(ka, blk + (size_t)(slot + r) * (D / 2) + t * (D / 8));
      ldg_words<KW>(kb, blk + (size_t)(slot + r + 8) * (D / 2) + t * (D / 8));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        ldg_words<VW>(vw[g][i], blk + vofs + (size_t)(slot + 2 * t + (i & 1) + 8 * (i >> 1)) * (D / 2) + r * (D / 16));
      const uint2 pa = __ldg(reinterpret_cast<const uint2*>(blk + pofs + (size_t)(slot + r) * 8));
      const uint2 pb = __ldg(reinterpret_cast<const uint2*>(blk + pofs + (size_t)(slot + r + 8) * 8));
      vs[g][0] = half2_at(pa.y);
      vs[g][1] = half2_at(pb.y);
#pragma unroll
      for (int j = 0; j < NT; ++j) sc[g][j][0] = sc[g][j][1] = sc[g][j][2] = sc[g][j][3] = 0.f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_bf16(sc[g][j], codes<0>(ka[w]), codes<0>(kb[w]), codes<1>(ka[w]), codes<1>(kb[w]), qf[j][2 * w][0],
                   qf[j][2 * w][1]);
          mma_bf16(sc[g][j], codes<2>(ka[w]), codes<2>(kb[w]), codes<3>(ka[w]), codes<3>(kb[w]), qf[j][2 * w + 1][0],
                   qf[j][2 * w + 1][1]);
        }
      }
      const float2 ks0 = half2_at(pa.x), ks1 = half2_at(pb.x);
      const float s0 = ks0.x * p.scale_log2, b0 = fmaf(-128.f, ks0.x, ks0.y) * p.scale_log2;
      const float s1 = ks1.x * p.scale_log2, b1 = fmaf(-128.f, ks1.x, ks1.y) * p.scale_log2;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int seen = good[g] ? lim[j][e] : 0;
          sc[g][j][e] = pos + r < seen ? fmaf(s0, sc[g][j][e], b0 * sumq[j][e]) : -INFINITY;
          sc[g][j][2 + e] = pos + r + 8 < seen ? fmaf(s1, sc[g][j][2 + e], b1 * sumq[j][e]) : -INFINITY;
        }
      }
    }
    // running maxima; the accumulators are scaled only when one has grown
    float ref[NT][2];
    bool grown = false;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(sc[0][j][e], sc[0][j][2 + e]), fmaxf(sc[1][j][e], sc[1][j][2 + e]));
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
        grown |= x > m[j][e];
        ref[j][e] = fmaxf(x, m[j][e]);
      }
    }
    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[e] = m[j][e] == -INFINITY ? 0.f : ex2(m[j][e] - ref[j][e]);
          m[j][e] = ref[j][e];
          l[j][e] *= f[e];
          corr[j][e] *= f[e];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          o[j][i][0] *= f[0];
          o[j][i][1] *= f[1];
          o[j][i][2] *= f[0];
          o[j][i][3] *= f[1];
        }
      }
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t pb[NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float w[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = sc[g][j][2 * k + e];
            const bool in = x != -INFINITY;  // a masked place takes no part, whatever its scales hold
            const float pr = in ? ex2(x - m[j][e]) : 0.f;
            l[j][e] += pr;
            w[e] = in ? pr * vs[g][k].x : 0.f;
            if (in) corr[j][e] = fmaf(pr, vs[g][k].y, corr[j][e]);
          }
          const __nv_bfloat162 wb = __floats2bfloat162_rn(w[0], w[1]);
          const float2 wr = __bfloat1622float2(wb);
          corr[j][0] = fmaf(-128.f, wr.x, corr[j][0]);
          corr[j][1] = fmaf(-128.f, wr.y, corr[j][1]);
          pb[j][k] = transpose8x8(*reinterpret_cast<const uint32_t*>(&wb));
        }
      }
#pragma unroll
      for (int w = 0; w < VW; ++w) {
        const uint32_t a[2] = {lo16(vw[g][0][w], vw[g][1][w]), hi16(vw[g][0][w], vw[g][1][w])};
        const uint32_t b[2] = {lo16(vw[g][2][w], vw[g][3][w]), hi16(vw[g][2][w], vw[g][3][w])};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma_bf16(o[j][4 * w + 2 * i], codes<0>(a[i]), codes<1>(a[i]), codes<0>(b[i]), codes<1>(b[i]), pb[j][0],
                     pb[j][1]);
            mma_bf16(o[j][4 * w + 2 * i + 1], codes<2>(a[i]), codes<3>(a[i]), codes<2>(b[i]), codes<3>(b[i]),
                     pb[j][0], pb[j][1]);
          }
        }
      }
    }
  }

  // the warps' states
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) {
        l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], k);
        corr[j][e] += __shfl_xor_sync(0xffffffffu, corr[j][e], k);
      }
      const int n = 8 * j + 2 * t + e;
      if (r == 0) sm.m[warp][n] = m[j][e], sm.l[warp][n] = l[j][e];
#pragma unroll
      for (int i = 0; i < MT; ++i)
        *reinterpret_cast<float2*>(&sm.o[warp][n][r * (D / 8) + 2 * i]) =
            make_float2(o[j][i][e] + corr[j][e], o[j][i][2 + e] + corr[j][e]);
    }
  }
  __syncthreads();
  float* part = p.part + ((size_t)unit * p.splits + sp) * (R * (D + 2));
  for (int item = threadIdx.x; item < R * (D / 4); item += kThreads) {
    const int n = item / (D / 4), d = (item - n * (D / 4)) * 4;
    const int row = row_first + n;
    if (row >= rows) continue;
    Join a;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) a.mx = fmaxf(a.mx, sm.m[w][n]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) a.add(sm.m[w][n], sm.l[w][n], *reinterpret_cast<const float4*>(&sm.o[w][n][d]));
    if (ns == 1) {
      const float inv = a.l > 0.f ? 1.0f / a.l : (a.l == 0.f ? 0.f : a.l);  // no position: zero; NaN stays
      const int tok = row / G;
      __nv_bfloat162 v[2] = {__floats2bfloat162_rn(a.o[0] * inv, a.o[1] * inv),
                             __floats2bfloat162_rn(a.o[2] * inv, a.o[3] * inv)};
      *reinterpret_cast<uint2*>(p.out + ((size_t)(q.row0 + tok) * c.heads + (size_t)h * G + (row - tok * G)) * D + d) =
          *reinterpret_cast<const uint2*>(v);
    } else {
      float* dst = part + (size_t)n * (D + 2);
      *reinterpret_cast<float2*>(dst + d) = make_float2(a.o[0], a.o[1]);
      *reinterpret_cast<float2*>(dst + d + 2) = make_float2(a.o[2], a.o[3]);
      if (d == 0) *reinterpret_cast<float2*>(dst + D) = make_float2(a.mx, a.l);
    }
  }
  if (ns == 1) return;

  // the last chunk of the tile to arrive joins all of them
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    sm.last = atomicAdd(p.cnt + unit, 1u) == (unsigned)(ns - 1);
    if (sm.last) p.cnt[unit] = 0u;
  }
  __syncthreads();
  if (!sm.last) return;
  __threadfence();
  const float* first = p.part + (size_t)unit * p.splits * (R * (D + 2));
  for (int item = threadIdx.x; item < R * (D / 4); item += kThreads) {
    const int n = item / (D / 4), d = (item - n * (D / 4)) * 4;
    const int row = row_first + n;
    if (row >= rows) continue;
    const float* src = first + (size_t)n * (D + 2);
    Join a;
    for (int i = 0; i < ns; ++i) a.mx = fmaxf(a.mx, __ldcg(src + (size_t)i * (R * (D + 2)) + D));
    for (int i = 0; i < ns; ++i) {
      const float* e = src + (size_t)i * (R * (D + 2));
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(e + D));
      const float2 x = __ldcg(reinterpret_cast<const float2*>(e + d)), y = __ldcg(reinterpret_cast<const float2*>(e + d + 2));
      a.add(ml.x, ml.y, make_float4(x.x, x.y, y.x, y.y));
    }
    const float inv = a.l > 0.f ? 1.0f / a.l : (a.l == 0.f ? 0.f : a.l);
    const int tok = row / G;
    __nv_bfloat162 v[2] = {__floats2bfloat162_rn(a.o[0] * inv, a.o[1] * inv),
                           __floats2bfloat162_rn(a.o[2] * inv, a.o[3] * inv)};
    *reinterpret_cast<uint2*>(p.out + ((size_t)(q.row0 + tok) * c.heads + (size_t)h * G + (row - tok * G)) * D + d) =
        *reinterpret_cast<const uint2*>(v);
  }
}

template <int D, int NT>
int launch_one(const Kv4AttnParams& p, long long blocks, cudaStream_t s) {
  constexpr int bytes = (int)sizeof(Shared<D, NT>);
  const cudaError_t e =
      cudaFuncSetAttribute(attn_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return (int)e;
  attn_kernel<D, NT><<<(unsigned)blocks, kThreads, bytes, s>>>(p);
  return (int)cudaGetLastError();
}

// Rows per CTA: the smallest of 8, 16, 32 that holds a sequence's rows of one
// kv head, else tiles of 32. Chunks: enough CTAs for about eight per
// multiprocessor at the batch's largest length, whole rounds of the eight warps.
constexpr int kRound = kStep * kWarps;
long long target_ctas(int sms) { return 8ll * sms; }
// A batch is split only while it has fewer tiles than the target, so the
// counters, one per tile, have a place whose size no batch changes.
size_t counter_bytes(int sms) { return ((size_t)target_ctas(sms) * 4 + 255) / 256 * 256; }

tern_status plan_attn(const Kv4Params& c, int heads, int seqs, int max_new, int max_len, int sms, Kv4AttnPlan* pl) {
  const long long rows = (long long)max_new * (heads / c.kv_heads);
  if (rows > (1 << 30)) return TERN_EUNSUPPORTED;
  pl->rows = rows <= 8 ? 8 : (rows <= 16 ? 16 : 32);
  const long long tiles = (rows + pl->rows - 1) / pl->rows;
  pl->tiles = (int)tiles;
  pl->units = (long long)seqs * c.kv_heads * tiles;
  const long long target = target_ctas(sms);
  long long splits = pl->units > 0 ? (target + pl->units - 1) / pl->units : 1;
  splits = std::max(1ll, std::min(splits, ((long long)max_len + kRound - 1) / kRound));
  long long chunk = (max_len + splits - 1) / splits;
  chunk = std::max((long long)kRound, (chunk + kRound - 1) / kRound * kRound);
  pl->chunk = (int)std::min(chunk, 1ll << 30);
  pl->splits = std::max(1, (int)(((long long)max_len + pl->chunk - 1) / pl->chunk));
  if (pl->units * pl->splits > 0x7FFFFFFFll) return TERN_EUNSUPPORTED;
  pl->cnt_bytes = counter_bytes(sms);
  pl->ws_bytes = pl->splits > 1
                     ? pl->cnt_bytes + (size_t)pl->units * pl->splits * pl->rows * (size_t)(c.dim + 2) * 4
                     : 0;
  return TERN_OK;
}

}  // namespace

int launch_kv4_attn(const Kv4AttnParams& p, const Kv4AttnPlan& pl, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const long long blocks = pl.units * pl.splits;
  if (p.c.dim == 128) {
    if (pl.rows == 8) return launch_one<128, 1>(p, blocks, s);
    if (pl.rows == 16) return launch_one<128, 2>(p, blocks, s);
    return launch_one<128, 4>(p, blocks, s);
  }
  if (pl.rows == 8) return launch_one<64, 1>(p, blocks, s);
  if (pl.rows == 16) return launch_one<64, 2>(p, blocks, s);
  return launch_one<64, 4>(p, blocks, s);
}

}  // namespace tern

using namespace tern;

extern "C" tern_status tern_kv4_attention_workspace_size(const tern_kv4_cache* cache, int32_t seqs, int32_t max_new,
                                                         int32_t max_len, int32_t heads, size_t* bytes) {
  if (!bytes) return TERN_EINVAL;
  Kv4Params c{};
  const tern_status st = kv4_check(cache, nullptr, &c);
  if (st != TERN_OK) return st;
  if (seqs < 0 || seqs > 65535 || max_new < 0 || max_len < 0 || heads < 1 || heads % c.kv_heads != 0)
    return TERN_EINVAL;
  const int sms = sm_count();
  Kv4AttnPlan pl{};
  const tern_status sp = plan_attn(c, heads, seqs, max_new, max_len, sms, &pl);
  if (sp != TERN_OK) return sp;
  // tiles x chunks of any batch within the bounds that is split at all: fewer
  // tiles than the target, and one chunk more per tile than divides it
  *bytes = seqs > 0 && max_new > 0 && max_len > kRound
               ? pl.cnt_bytes + 2 * (size_t)target_ctas(sms) * pl.rows * (size_t)(c.dim + 2) * 4
               : 0;
  return TERN_OK;
}

extern "C" tern_status tern_kv4_attention(const tern_kv4_cache* cache, const tern_kv4_batch* batch, int32_t heads,
                                          float scale, const uint16_t* d_q, uint16_t* d_out, void* d_ws,
                                          size_t ws_bytes, void* stream) {
  Kv4AttnParams p{};
  if (!batch) return TERN_EINVAL;
  tern_status st = kv4_check(cache, batch, &p.c);
  if (st != TERN_OK) return st;
  if (heads < 1 || heads > 65535 || heads % p.c.kv_heads != 0 || !std::isfinite(scale)) return TERN_EINVAL;
  if (p.c.seqs == 0 || p.c.tokens == 0 || p.c.max_new == 0) return TERN_OK;
  if (!d_q || !d_out) return TERN_EINVAL;
  if (((reinterpret_cast<uintptr_t>(d_q) | reinterpret_cast<uintptr_t>(d_out)) & 15u) != 0) return TERN_EALIGN;
  Kv4AttnPlan pl{};
  st = plan_attn(p.c, heads, p.c.seqs, p.c.max_new, p.c.max_len, sm_count(), &pl);
  if (st != TERN_OK) return st;
  if (pl.ws_bytes > 0) {
    if (!d_ws || ws_bytes < pl.ws_bytes) return TERN_ENOSPACE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return TERN_EALIGN;
  }
  p.c.heads = heads;
  p.q = d_q;
  p.out = d_out;
  p.scale_log2 = scale * 1.44269504088896340736f;
  p.group = heads / p.c.kv_heads;
  p.tiles = pl.tiles;
  p.chunk = pl.chunk;
  p.splits = pl.splits;
  p.cnt = static_cast<unsigned*>(d_ws);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(d_ws) + pl.cnt_bytes);
  return launch_kv4_attn(p, pl, stream) == 0 ? TERN_OK : TERN_ECUDA;
}
