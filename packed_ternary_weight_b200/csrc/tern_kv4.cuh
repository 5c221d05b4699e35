// Device helpers of the 4-bit paged cache: a sequence's rows and length with
// their checks, block addresses, fp16 scale pairs.
#pragma once
#include <cuda_fp16.h>

#include "tern_ptx.cuh"

namespace tern {
namespace kv4 {

struct Seq {
  int row0, n, len;  // first row, new tokens, tokens in all
  bool ok;
};

// What the batch says of sequence s; a description that cannot be right is
// reported in the device error word and the sequence left out.
__device__ __forceinline__ Seq load_seq(const Kv4Params& c, int s) {
  Seq q;
  const int a = c.start[s], b = c.start[s + 1];
  q.len = c.len[s];
  q.row0 = a;
  q.n = b - a;
  q.ok = a >= 0 && b >= a && b <= c.tokens && q.n <= c.max_new && q.len >= 0 && q.len <= c.max_len &&
         (long long)q.len <= (long long)c.max_pages << c.log_page;
  return q;
}
__device__ __forceinline__ void report_bad() { atomicOr(&g_dev_error, TERN_DEVERR_FORMAT); }

__device__ __forceinline__ size_t block_offset(const Kv4Params& c, int page, int head) {
  return ((size_t)page * (size_t)c.kv_heads + (size_t)head) * kv4_block_bytes(c.page, c.dim);
}
// The page of a position, or -1 where the table names none of the cache.
__device__ __forceinline__ int page_of(const Kv4Params& c, int s, int pos) {
  const int id = c.table[(size_t)s * c.max_pages + (pos >> c.log_page)];
  return (unsigned)id < (unsigned)c.num_pages ? id : -1;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// The batch's work as one line of rounds, sequence after sequence; CTA c of
// `ctas` takes the rounds [total c / ctas, total (c + 1) / ctas), at least
// min_share of them where there are as many. Every thread of the CTA calls
// find_share; weight(s, report) is the number of rounds of sequence s.
struct Share {
  long long total, ctas, at, stop;
  int s;             // the sequence of round `at`
  long long in_seq;  // rounds of it before `at`
  // the CTA that holds round x
  __device__ __forceinline__ int cta_of(long long x) const { return (int)(((x + 1) * ctas - 1) / total); }
};
template <int WARPS>
struct ShareScratch {
  long long scan[WARPS], off;
  int found;
};
template <int WARPS, typename Weight>
__device__ __forceinline__ bool find_share(int seqs, long long min_share, Weight weight, ShareScratch<WARPS>& sm,
                                           Share* out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // sums over the CTA of v, of this thread's and of the earlier threads' v
  auto scan = [&](long long v, long long* incl) {
    *incl = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, *incl, k);
      if (lane >= k) *incl += u;
    }
    if (lane == 31) sm.scan[warp] = *incl;
    __syncthreads();
    long long all = 0;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      if (k < warp) *incl += sm.scan[k];
      all += sm.scan[k];
    }
    return all;
  };
  // up to as many sequences as threads: one of them each, scanned once; more: their sum first
  const bool one_pass = seqs <= 32 * WARPS;
  long long total = 0, w = 0, incl = 0;
  if (seqs == 1) {
    total = weight(0, blockIdx.x == 0 && threadIdx.x == 0);
  } else if (one_pass) {
    w = (int)threadIdx.x < seqs ? weight(threadIdx.x, blockIdx.x == 0) : 0;
    total = scan(w, &incl);
  } else {
    for (int i = threadIdx.x; i < seqs; i += 32 * WARPS) w += weight(i, blockIdx.x == 0);
    total = scan(w, &incl);
    __syncthreads();
  }
  long long ctas = min((long long)gridDim.x, max(min(total, 1ll), total / min_share));
  if (total > ctas && total <= 4 * ctas) {
    // small shares: as few CTAs as leave the largest one as it is, so that fewer units are cut (8 sequences of 1000
    // positions with 48 rows: 192 rounds on 96 CTAs 14 us, on 148 22 us; with shares of 14 rounds it cost 7 %)
    const long long most = (total + ctas - 1) / ctas;
    ctas = (total + most - 1) / most;
  }
  if (blockIdx.x >= ctas) return false;
  out->total = total;
  out->ctas = ctas;
  out->at = total * blockIdx.x / ctas;
  out->stop = total * (blockIdx.x + 1) / ctas;
  out->s = 0;
  out->in_seq = out->at;
  if (seqs == 1) return true;
  long long before = 0;
  for (int base = 0; base < seqs; base += 32 * WARPS) {
    const int i = base + threadIdx.x;
    if (threadIdx.x == 0) sm.found = -1;
    if (one_pass) {
      __syncthreads();
    } else {
      w = i < seqs ? weight(i, false) : 0;
      const long long all = scan(w, &incl);
      incl += before;
      before += all;
    }
    if (out->at >= incl - w && out->at < incl) {
      sm.found = i;
      sm.off = out->at - (incl - w);
    }
    __syncthreads();
    if (sm.found >= 0) break;
  }
  out->s = sm.found;
  out->in_seq = sm.off;
  return out->s >= 0;  // not found: the lengths changed meanwhile
}

}  // namespace kv4

// Host: argument checks that every call on the cache shares (batch may be NULL).
tern_status kv4_check(const tern_kv4_cache* cache, const tern_kv4_batch* batch, Kv4Params* c);

}  // namespace tern
