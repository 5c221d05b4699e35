// The paged 4-bit cache: rotation and append of new tokens in one launch, and
// the values read back. A key or value head of a token is D codes of 4 bits
// with one fp16 (scale, min) pair: 4.25 bits per value at D = 128, against 16
// of the decode step's bf16 cache.
//
// One group of D / 4 lanes takes one (token, head): lane l holds the
// dimensions 2l, 2l+1 and D/2 + 2l, D/2 + 2l + 1, the two pairs that
// rotate_half combines, so the rotation needs no exchange and each lane's two
// code pairs are two whole bytes. Minimum and maximum go over the group by
// shuffles.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "tern_kv4.cuh"

namespace tern {

int read_clear_dev_error_kv4(void* stream, unsigned* out) { return read_clear_dev_error_tu(stream, out); }

namespace {

constexpr int kThreads = 256;

// The sequence that row t belongs to: the last s with start[s] <= t, found by
// all lanes of a warp together, 32 candidates a round; -1 for a row outside.
__device__ __forceinline__ int seq_of(const Kv4Params& c, int t) {
  int lo = 0, n = c.seqs + 1;  // candidates lo .. lo + n - 1 among start[0 .. seqs]
  if (__ldg(c.start) > t) return -1;
  while (n > 1) {
    const int step = (n + 31) >> 5;
    const int i = lo + (int)(threadIdx.x & 31) * step;
    const bool le = i < lo + n && __ldg(c.start + i) <= t;
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, le) | 1u);
    const int next = lo + last * step;
    n = min(step, lo + n - next);
    lo = next;
  }
  return lo < c.seqs ? lo : -1;
}

__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 ld2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ void st2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void st2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const Kv4AppendParams p) {
  constexpr int L = D / 4;  // lanes of a group
  const Kv4Params& c = p.c;
  const int groups = c.heads + 2 * c.kv_heads;  // of a token: q heads, k heads, v heads
  const int gl = threadIdx.x & (L - 1);
  // a warp's groups are of one token: groups rounded up to whole warps
  const int wpt = (groups * L + 31) >> 5;  // warps per token
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long tl = w / wpt;
  if (tl >= c.tokens) return;  // whole warps
  const int t = (int)tl;
  const int s = seq_of(c, t);
  if (s < 0) return;
  const kv4::Seq q = kv4::load_seq(c, s);
  if (!q.ok || t < q.row0 || t - q.row0 >= q.n) {
    kv4::report_bad();
    return;
  }
  const int g = (int)(w - tl * wpt) * (32 / L) + (int)((threadIdx.x & 31) / L);
  const bool active = g < groups;
  const int pos = q.len - q.n + (t - q.row0);
  const bool is_q = g < c.heads, is_k = !is_q && g < c.heads + c.kv_heads;
  const int head = is_q ? g : (is_k ? g - c.heads : g - c.heads - c.kv_heads);
  __nv_bfloat16* qo = reinterpret_cast<__nv_bfloat16*>(p.q_out) + ((size_t)t * c.heads + head) * D + 2 * gl;
  if (pos < 0 || pos >= p.max_pos) {
    if (pos >= 0) kv4::report_bad();
    if (active && is_q) {
      st2(qo, 0.f, 0.f);
      st2(qo + D / 2, 0.f, 0.f);
    }
    return;
  }
  const T* src = is_q ? static_cast<const T*>(p.q) + (int64_t)t * p.ldq
                      : (is_k ? static_cast<const T*>(p.k) + (int64_t)t * p.ldk
                              : static_cast<const T*>(p.v) + (int64_t)t * p.ldv);
  float2 a = make_float2(0.f, 0.f), b = a;
  if (active) {
    a = ld2(src + (size_t)head * D + 2 * gl);
    b = ld2(src + (size_t)head * D + D / 2 + 2 * gl);
    if (is_q || is_k) {
      const float4 cs = __ldg(reinterpret_cast<const float4*>(p.rope + ((size_t)pos * (D / 2) + 2 * gl) * 2));
      const float2 x = a, y = b;
      a.x = __fsub_rn(__fmul_rn(x.x, cs.x), __fmul_rn(y.x, cs.y));
      b.x = __fadd_rn(__fmul_rn(y.x, cs.x), __fmul_rn(x.x, cs.y));
      a.y = __fsub_rn(__fmul_rn(x.y, cs.z), __fmul_rn(y.y, cs.w));
      b.y = __fadd_rn(__fmul_rn(y.y, cs.z), __fmul_rn(x.y, cs.w));
    }
  }
  float lo = fminf(fminf(a.x, a.y), fminf(b.x, b.y)), hi = fmaxf(fmaxf(a.x, a.y), fmaxf(b.x, b.y));
#pragma unroll
  for (int o = L / 2; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
  }
  if (!active) return;
  if (is_q) {
    st2(qo, a.x, a.y);
    st2(qo + D / 2, b.x, b.y);
    return;
  }
  const int page = kv4::page_of(c, s, pos);
  if (page < 0) {
    kv4::report_bad();
    return;
  }
  const __half hs = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f)), hm = __float2half_rn(lo);
  const float sc = __half2float(hs), mn = __half2float(hm);
  const float inv = sc > 0.f ? __fdiv_rn(1.0f, sc) : 0.f;
  auto code = [&](float v) {
    return (unsigned)max(0, min(15, __float2int_rn(__fmul_rn(__fsub_rn(v, mn), inv))));
  };
  uint8_t* blk = c.pages + kv4::block_offset(c, page, head);
  const int slot = pos & (c.page - 1);
  uint8_t* row = blk + (size_t)(is_k ? 0 : c.page * (D / 2)) + (size_t)slot * (D / 2);
  row[gl] = (uint8_t)(code(a.x) | (code(a.y) << 4));
  row[D / 4 + gl] = (uint8_t)(code(b.x) | (code(b.y) << 4));
  if (gl == 0)
    *reinterpret_cast<__half2*>(blk + (size_t)c.page * D + (size_t)slot * 8 + (is_k ? 0 : 4)) = __halves2half2(hs, hm);
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const Kv4ReadParams p) {
  constexpr int L = D / 4;
  const Kv4Params& c = p.c;
  const int groups = 2 * c.kv_heads;
  const int gl = threadIdx.x & (L - 1);
  const int wpt = (groups * L + 31) >> 5;
  const long long w = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const long long tl = w / wpt;
  if (tl >= c.tokens) return;
  const int t = (int)tl;
  const int s = seq_of(c, t);
  if (s < 0) return;
  const kv4::Seq q = kv4::load_seq(c, s);
  if (!q.ok || t < q.row0 || t - q.row0 >= q.n) {
    kv4::report_bad();
    return;
  }
  const int g = (int)(w - tl * wpt) * (32 / L) + (int)((threadIdx.x & 31) / L);
  if (g >= groups) return;
  const bool is_k = g < c.kv_heads;
  const int head = is_k ? g : g - c.kv_heads;
  void* dst = is_k ? p.k : p.v;
  if (!dst) return;
  T* out = static_cast<T*>(dst) + (int64_t)t * (is_k ? p.ldk : p.ldv) + (size_t)head * D + 2 * gl;
  const int pos = q.len - q.n + (t - q.row0);
  const int page = pos < 0 ? -1 : kv4::page_of(c, s, pos);
  if (page < 0) {
    if (pos >= 0) kv4::report_bad();
    st2(out, 0.f, 0.f);
    st2(out + D / 2, 0.f, 0.f);
    return;
  }
  const uint8_t* blk = c.pages + kv4::block_offset(c, page, head);
  const int slot = pos & (c.page - 1);
  const uint8_t* row = blk + (size_t)(is_k ? 0 : c.page * (D / 2)) + (size_t)slot * (D / 2);
  const float2 sm = __half22float2(
      *reinterpret_cast<const __half2*>(blk + (size_t)c.page * D + (size_t)slot * 8 + (is_k ? 0 : 4)));
  // scale * code is exact in fp32 (11 + 4 bits), so the fused form rounds once, as the definition
  auto val = [&](unsigned code) { return __fmaf_rn(sm.x, (float)code, sm.y); };
  const unsigned u = row[gl], v = row[D / 4 + gl];
  st2(out, val(u & 15u), val(u >> 4));
  st2(out + D / 2, val(v & 15u), val(v >> 4));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

long long blocks_for(const Kv4Params& c, int groups) {
  const long long warps = (long long)c.tokens * ((groups * (c.dim / 4) + 31) / 32);
  return (warps + kThreads / 32 - 1) / (kThreads / 32);
}

}  // namespace

int launch_kv4_append(const Kv4AppendParams& p, void* stream) {
  const unsigned grid = (unsigned)blocks_for(p.c, p.c.heads + 2 * p.c.kv_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.c.dim == 128) {
    if (p.bf16) append_kernel<128, __nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else append_kernel<128, float><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (p.bf16) append_kernel<64, __nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else append_kernel<64, float><<<grid, kThreads, 0, s>>>(p);
  }
  return (int)cudaGetLastError();
}

int launch_kv4_read(const Kv4ReadParams& p, void* stream) {
  const unsigned grid = (unsigned)blocks_for(p.c, 2 * p.c.kv_heads);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.c.dim == 128) {
    if (p.bf16) read_kernel<128, __nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else read_kernel<128, float><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (p.bf16) read_kernel<64, __nv_bfloat16><<<grid, kThreads, 0, s>>>(p);
    else read_kernel<64, float><<<grid, kThreads, 0, s>>>(p);
  }
  return (int)cudaGetLastError();
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
  if (blocks_for(p.c, heads + 2 * p.c.kv_heads) > 0x7FFFFFFFll) return TERN_EINVAL;
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
  if (blocks_for(p.c, 2 * p.c.kv_heads) > 0x7FFFFFFFll) return TERN_EINVAL;
  p.k = d_k;
  p.v = d_v;
  p.ldk = ldk;
  p.ldv = ldv;
  p.bf16 = type == TERN_OUT_BF16;
  return launch_kv4_read(p, stream) == 0 ? TERN_OK : TERN_ECUDA;
}
