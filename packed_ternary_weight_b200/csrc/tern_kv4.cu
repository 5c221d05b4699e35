// The paged 4-bit cache: rotation and append of new tokens in one launch, and
// the values read back. A key or value head of a token is D codes of 4 bits
// with one fp16 (scale, min) pair: 4.25 bits per value at D = 128, against 16
// of the decode step's bf16 cache.
//
// A group of D / 16 lanes takes one (token, head) at a time: lane l holds the
// dimensions 8l .. 8l + 7 and D/2 + 8l .. + 7, the pairs that rotate_half combines,
// so the rotation needs no exchange, bf16 rows are read in 16-byte pieces and each
// lane's codes are two whole words. Minimum and maximum go over the group by
// shuffles. A warp takes one head per group of a few tokens and up to three of each
// of many: the search for the token's sequence, its rotation row and its page are
// then shared by them, and the heads' loads are issued together, ahead of that search.
// 8813 prompt tokens (32 heads on 8 kv heads, D = 128, bf16): append 41 us, 4.8 TB/s of
// the bytes it has to move (0.74 of the measured copy rate), with 60 % of the issue slots
// in use; read 13.5 us, the integer pipe at 65 % (codes to fp32: shift, mask, conversion).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tern_kv4.cuh"
#include "tern_launch.cuh"

namespace tern {

int read_clear_dev_error_kv4(void* stream, unsigned* out) { return read_clear_dev_error_tu(stream, out); }

namespace {

constexpr int kThreads = 256;

// The sequence that row t belongs to: the last s with start[s] <= t, found by
// all lanes of a warp together, 32 candidates a round; -1 for a row outside.
__device__ __forceinline__ int seq_of(const Kv4Params& c, int t) {
  int lo = 0, n = c.seqs + 1;  // candidates lo .. lo + n - 1 among start[0 .. seqs]
  if (c.start[0] > t) return -1;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lo + (int)(threadIdx.x & 31) * step;
    const bool le = i < lo + n && c.start[i] <= t;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    const int next = lo + last * step;
    n = min(step, lo + n - next);
    lo = next;
  }
  return lo < c.seqs ? lo : -1;
}

// Eight elements as they stand in memory.
template <typename T>
struct Raw8 {
  uint4 u, w;
  __device__ __forceinline__ void load(const T* p) {
    u = reinterpret_cast<const uint4*>(p)[0];
    w = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t e[8] = {u.x, u.y, u.z, u.w, w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(e[i]);
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(e[i] << 16);
      v[2 * i + 1] = __uint_as_float(e[i] & 0xFFFF0000u);
    }
  }
};
__device__ __forceinline__ void st8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void st8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    e[i] = *reinterpret_cast<const uint32_t*>(&a);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(e[0], e[1], e[2], e[3]);
}

// The smaller and the larger one, not a number if either is not: a head's scales must show what stands in it.
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

constexpr int kMaxHeads = 3;  // of a token that a group of lanes takes

// A warp's token and the heads of its groups: first, first + step, .. (count of them, the same in both groups).
template <int D>
struct Place {
  static constexpr int L = D / 16, kGroups = 32 / L;
  int t, first, step, gl;
  __device__ __forceinline__ bool find(const Kv4Params& c, int warps_per_token) {
    const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long tl = w / warps_per_token;
    if (tl >= c.tokens) return false;  // whole warps
    t = (int)tl;
    gl = threadIdx.x & (L - 1);
    first = (int)(w - tl * warps_per_token) * kGroups + (int)((threadIdx.x & 31) / L);
    step = warps_per_token * kGroups;
    return true;
  }
};

template <int D, typename T, int HEADS>
__global__ void __launch_bounds__(kThreads) append_kernel(const Kv4AppendParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const Kv4Params& c = p.c;
  const int total = c.heads + 2 * c.kv_heads;  // of a token: q heads, k heads, v heads
  Place<D> pl;
  if (!pl.find(c, p.warps_per_token)) return;
  const int t = pl.t, gl = pl.gl;
  Raw8<T> lo[HEADS], hi[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int g = min(pl.first + i * pl.step, total - 1);
    const T* src = g < c.heads ? static_cast<const T*>(p.q) + (int64_t)t * p.ldq + (size_t)g * D
                   : g < c.heads + c.kv_heads
                       ? static_cast<const T*>(p.k) + (int64_t)t * p.ldk + (size_t)(g - c.heads) * D
                       : static_cast<const T*>(p.v) + (int64_t)t * p.ldv + (size_t)(g - c.heads - c.kv_heads) * D;
    lo[i].load(src + 8 * gl);
    hi[i].load(src + D / 2 + 8 * gl);
  }
  const int s = seq_of(c, t);
  if (s < 0) return;
  const kv4::Seq q = kv4::load_seq(c, s);
  if (!q.ok || t < q.row0 || t - q.row0 >= q.n) {
    kv4::report_bad();
    return;
  }
  const int pos = q.len - q.n + (t - q.row0);
  const bool skip = pos < 0 || pos >= p.max_pos;  // not stored, its query is zero
  if (pos >= p.max_pos) kv4::report_bad();
  int page = -1;
  float co[8], si[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) co[k] = si[k] = 0.f;
  if (!skip) {
    page = kv4::page_of(c, s, pos);
    if (page < 0) kv4::report_bad();
    const float4* row = reinterpret_cast<const float4*>(p.rope + ((size_t)pos * (D / 2) + 8 * gl) * 2);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 cs = row[k];
      co[2 * k] = cs.x, si[2 * k] = cs.y, co[2 * k + 1] = cs.z, si[2 * k + 1] = cs.w;
    }
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int g = pl.first + i * pl.step;
    const bool is_q = g < c.heads, is_k = !is_q && g < c.heads + c.kv_heads;
    float a[8], b[8];
    lo[i].values(a);
    hi[i].values(b);
    if (is_q || is_k) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float x = a[k], y = b[k];
        a[k] = __fsub_rn(__fmul_rn(x, co[k]), __fmul_rn(y, si[k]));
        b[k] = __fadd_rn(__fmul_rn(y, co[k]), __fmul_rn(x, si[k]));
      }
    }
    if (is_q) {
      __nv_bfloat16* qo = reinterpret_cast<__nv_bfloat16*>(p.q_out) + ((size_t)t * c.heads + g) * D + 8 * gl;
      if (skip) {
#pragma unroll
        for (int k = 0; k < 8; ++k) a[k] = b[k] = 0.f;
      }
      st8(qo, a);
      st8(qo + D / 2, b);
    }
    // a warp whose groups all hold queries skips the rest
    if (__all_sync(0xffffffffu, is_q || g >= total)) continue;
    float mn = a[0], mx = a[0];
#pragma unroll
    for (int k = 0; k < 8; ++k) mn = min_nan(mn, min_nan(a[k], b[k])), mx = max_nan(mx, max_nan(a[k], b[k]));
#pragma unroll
    for (int o = Place<D>::L / 2; o; o >>= 1) {
      mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, o));
      mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if (is_q || g >= total || page < 0) continue;
    const int head = is_k ? g - c.heads : g - c.heads - c.kv_heads;
    const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.0f)), hm = __float2half_rn(mn);
    const float sc = __half2float(hs), m = __half2float(hm);
    const float inv = sc > 0.f ? __fdiv_rn(1.0f, sc) : 0.f;
    auto code = [&](float v) {
      return (unsigned)max(0, min(15, __float2int_rn(__fmul_rn(__fsub_rn(v, m), inv))));
    };
    auto eight = [&](const float (&v)[8]) {
      unsigned w = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) w |= code(v[k]) << (4 * k);
      return w;
    };
    uint8_t* blk = c.pages + kv4::block_offset(c, page, head);
    const int slot = pos & (c.page - 1);
    uint32_t* row = reinterpret_cast<uint32_t*>(blk + (size_t)(is_k ? 0 : c.page * (D / 2)) + (size_t)slot * (D / 2));
    row[gl] = eight(a);
    row[D / 16 + gl] = eight(b);
    if (gl == 0)
      *reinterpret_cast<__half2*>(blk + (size_t)c.page * D + (size_t)slot * 8 + (is_k ? 0 : 4)) =
          __halves2half2(hs, hm);
  }
}

template <int D, typename T, int HEADS>
__global__ void __launch_bounds__(kThreads) read_kernel(const Kv4ReadParams p) {
  pdl_launch_dependents();
  pdl_wait();
  const Kv4Params& c = p.c;
  const int total = 2 * c.kv_heads;
  Place<D> pl;
  if (!pl.find(c, p.warps_per_token)) return;
  const int t = pl.t, gl = pl.gl;
  const int s = seq_of(c, t);
  if (s < 0) return;
  const kv4::Seq q = kv4::load_seq(c, s);
  if (!q.ok || t < q.row0 || t - q.row0 >= q.n) {
    kv4::report_bad();
    return;
  }
  const int pos = q.len - q.n + (t - q.row0);
  const int page = pos < 0 ? -1 : kv4::page_of(c, s, pos);
  if (page < 0 && pos >= 0) kv4::report_bad();
  const int slot = pos & (c.page - 1);
  uint32_t u[HEADS], v[HEADS], pair[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int g = min(pl.first + i * pl.step, total - 1);
    const bool is_k = g < c.kv_heads;
    u[i] = v[i] = pair[i] = 0u;
    if (page >= 0) {
      const uint8_t* blk = c.pages + kv4::block_offset(c, page, is_k ? g : g - c.kv_heads);
      const uint32_t* row =
          reinterpret_cast<const uint32_t*>(blk + (size_t)(is_k ? 0 : c.page * (D / 2)) + (size_t)slot * (D / 2));
      u[i] = row[gl];
      v[i] = row[D / 16 + gl];
      pair[i] = *reinterpret_cast<const uint32_t*>(blk + (size_t)c.page * D + (size_t)slot * 8 + (is_k ? 0 : 4));
    }
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int g = pl.first + i * pl.step;
    if (g >= total) break;
    const bool is_k = g < c.kv_heads;
    void* dst = is_k ? p.k : p.v;
    if (!dst) continue;
    const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&pair[i]));
    T* out = static_cast<T*>(dst) + (int64_t)t * (is_k ? p.ldk : p.ldv) + (size_t)(is_k ? g : g - c.kv_heads) * D +
             8 * gl;
    // scale * code is exact in fp32 (11 + 4 bits), so the fused form rounds once, as the definition
    float a[8], b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = page < 0 ? 0.f : __fmaf_rn(sm.x, (float)((u[i] >> (4 * k)) & 15u), sm.y);
      b[k] = page < 0 ? 0.f : __fmaf_rn(sm.x, (float)((v[i] >> (4 * k)) & 15u), sm.y);
    }
    st8(out, a);
    st8(out + D / 2, b);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Heads per group of lanes: three where about 24 warps per multiprocessor are left
// (8500 prompt tokens of 32 + 16 heads: append and read 51 us, with one head 63 us),
// one below (64 tokens: 6.1 and 6.6 us; 1000 tokens the same); and the warps of a token.
struct Spread {
  int heads, warps_per_token;
  long long blocks;
};
Spread spread(const Kv4Params& c, int total) {
  const int groups = 32 / (c.dim / 16);
  const long long warps = (long long)c.tokens * ((total + groups - 1) / groups);  // with one head each
  const long long many = warps / (24ll * sm_count());
  Spread s;
  s.heads = many >= kMaxHeads ? kMaxHeads : 1;
  s.warps_per_token = (total + s.heads * groups - 1) / (s.heads * groups);
  s.blocks = ((long long)c.tokens * s.warps_per_token + kThreads / 32 - 1) / (kThreads / 32);
  return s;
}

template <int D, typename T>
int append_any(const Kv4AppendParams& p, const Spread& sp, cudaStream_t s) {
  return launch_dependent(sp.heads == kMaxHeads ? append_kernel<D, T, kMaxHeads> : append_kernel<D, T, 1>,
                          (int)sp.blocks, kThreads, 0, 1, s, p);
}
template <int D, typename T>
int read_any(const Kv4ReadParams& p, const Spread& sp, cudaStream_t s) {
  return launch_dependent(sp.heads == kMaxHeads ? read_kernel<D, T, kMaxHeads> : read_kernel<D, T, 1>,
                          (int)sp.blocks, kThreads, 0, 1, s, p);
}

}  // namespace

int launch_kv4_append(Kv4AppendParams p, void* stream) {
  const Spread sp = spread(p.c, p.c.heads + 2 * p.c.kv_heads);
  p.warps_per_token = sp.warps_per_token;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.c.dim == 128) return p.bf16 ? append_any<128, __nv_bfloat16>(p, sp, s) : append_any<128, float>(p, sp, s);
  return p.bf16 ? append_any<64, __nv_bfloat16>(p, sp, s) : append_any<64, float>(p, sp, s);
}

int launch_kv4_read(Kv4ReadParams p, void* stream) {
  const Spread sp = spread(p.c, 2 * p.c.kv_heads);
  p.warps_per_token = sp.warps_per_token;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.c.dim == 128) return p.bf16 ? read_any<128, __nv_bfloat16>(p, sp, s) : read_any<128, float>(p, sp, s);
  return p.bf16 ? read_any<64, __nv_bfloat16>(p, sp, s) : read_any<64, float>(p, sp, s);
}

tern_status kv4_check(const tern_kv4_cache* cache, const tern_kv4_batch* batch, Kv4Params* c) {
  if (!cache) return TERN_EINVAL;
  if (cache->kv_heads < 1 || cache->kv_heads > 1024 || cache->num_pages < 1) return TERN_EINVAL;
  if (cache->head_dim != 64 && cache->head_dim != 128) return TERN_EUNSUPPORTED;
  const int page = cache->page_size;
  if (page < 16 || page > 256 || (page & (page - 1)) != 0) return TERN_EUNSUPPORTED;
  c->kv_heads = cache->kv_heads;
  c->dim = cache->head_dim;
  c->page = page;
  c->log_page = page == 16 ? 4 : (page == 32 ? 5 : (page == 64 ? 6 : (page == 128 ? 7 : 8)));
  c->num_pages = cache->num_pages;
  c->pages = static_cast<uint8_t*>(cache->d_pages);
  if (!batch) return TERN_OK;
  if (batch->seqs < 0 || batch->seqs > 65535 || batch->tokens < 0 || batch->max_new < 0 || batch->max_len < 0 ||
      batch->max_pages < 0)
    return TERN_EINVAL;
  c->seqs = batch->seqs;
  c->tokens = batch->tokens;
  c->max_new = batch->max_new;
  c->max_len = batch->max_len;
  c->max_pages = batch->max_pages;
  c->start = batch->d_start;
  c->len = batch->d_len;
  c->table = batch->d_table;
  if (batch->seqs == 0 || batch->tokens == 0 || batch->max_new == 0) return TERN_OK;  // nothing to do
  if (!cache->d_pages || !batch->d_start || !batch->d_len || !batch->d_table) return TERN_EINVAL;
  if (!aligned16(cache->d_pages)) return TERN_EALIGN;
  if (((reinterpret_cast<uintptr_t>(batch->d_start) | reinterpret_cast<uintptr_t>(batch->d_len) |
        reinterpret_cast<uintptr_t>(batch->d_table)) & 3u) != 0)
    return TERN_EALIGN;
  return TERN_OK;
}

}  // namespace tern

using namespace tern;

extern "C" tern_status tern_kv4_cache_size(const tern_kv4_cache* cache, size_t* bytes) {
  if (!bytes) return TERN_EINVAL;
  Kv4Params c{};
  const tern_status st = kv4_check(cache, nullptr, &c);
  if (st != TERN_OK) return st;
  *bytes = (size_t)c.num_pages * (size_t)c.kv_heads * kv4_block_bytes(c.page, c.dim);
  return TERN_OK;
}

extern "C" tern_status tern_kv4_append(const tern_kv4_cache* cache, const tern_kv4_batch* batch, int32_t heads,
                                       tern_out type, const void* d_q, int64_t ldq, const void* d_k, int64_t ldk,
                                       const void* d_v, int64_t ldv, const float* d_rope, int32_t max_pos,
                                       uint16_t* d_q_out, void* stream) {
  Kv4AppendParams p{};
  if (!batch) return TERN_EINVAL;
  const tern_status st = kv4_check(cache, batch, &p.c);
  if (st != TERN_OK) return st;
  if (type != TERN_OUT_F32 && type != TERN_OUT_BF16) return TERN_EINVAL;
  const int64_t kvw = (int64_t)p.c.kv_heads * p.c.dim, qw = (int64_t)heads * p.c.dim;
  if (heads < 0 || heads > 65535 || max_pos < 1 || ldk < kvw || ldv < kvw || (heads > 0 && ldq < qw) ||
      ((ldk | ldv | (heads > 0 ? ldq : 0)) & 7) != 0)
    return TERN_EINVAL;
  if (p.c.seqs == 0 || p.c.tokens == 0 || p.c.max_new == 0) return TERN_OK;
  if (!d_k || !d_v || !d_rope || (heads > 0 && (!d_q || !d_q_out))) return TERN_EINVAL;
  if (!aligned16(d_k) || !aligned16(d_v) || !aligned16(d_rope) ||
      (heads > 0 && (!aligned16(d_q) || !aligned16(d_q_out))))
    return TERN_EALIGN;
  p.c.heads = heads;
  if (spread(p.c, heads + 2 * p.c.kv_heads).blocks > 0x7FFFFFFFll) return TERN_EINVAL;
  p.q = d_q;
  p.k = d_k;
  p.v = d_v;
  p.rope = d_rope;
  p.q_out = d_q_out;
  p.ldq = ldq;
  p.ldk = ldk;
  p.ldv = ldv;
  p.max_pos = max_pos;
  p.bf16 = type == TERN_OUT_BF16;
  return launch_kv4_append(p, stream) == 0 ? TERN_OK : TERN_ECUDA;
}

extern "C" tern_status tern_kv4_read(const tern_kv4_cache* cache, const tern_kv4_batch* batch, tern_out type,
                                     void* d_k, int64_t ldk, void* d_v, int64_t ldv, void* stream) {
  Kv4ReadParams p{};
  if (!batch) return TERN_EINVAL;
  const tern_status st = kv4_check(cache, batch, &p.c);
  if (st != TERN_OK) return st;
  if (type != TERN_OUT_F32 && type != TERN_OUT_BF16) return TERN_EINVAL;
  const int64_t kvw = (int64_t)p.c.kv_heads * p.c.dim;
  if ((d_k && (ldk < kvw || (ldk & 7) != 0)) || (d_v && (ldv < kvw || (ldv & 7) != 0))) return TERN_EINVAL;
  if ((d_k && !aligned16(d_k)) || (d_v && !aligned16(d_v))) return TERN_EALIGN;
  if (p.c.seqs == 0 || p.c.tokens == 0 || p.c.max_new == 0 || (!d_k && !d_v)) return TERN_OK;
  if (spread(p.c, 2 * p.c.kv_heads).blocks > 0x7FFFFFFFll) return TERN_EINVAL;
  p.k = d_k;
  p.v = d_v;
  p.ldk = ldk;
  p.ldv = ldv;
  p.bf16 = type == TERN_OUT_BF16;
  return launch_kv4_read(p, stream) == 0 ? TERN_OK : TERN_ECUDA;
}
