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
  const int a = __ldg(c.start + s), b = __ldg(c.start + s + 1);
  q.len = __ldg(c.len + s);
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
  const int id = __ldg(c.table + (size_t)s * c.max_pages + (pos >> c.log_page));
  return (unsigned)id < (unsigned)c.num_pages ? id : -1;
}

}  // namespace kv4

// Host: argument checks that every call on the cache shares (batch may be NULL).
tern_status kv4_check(const tern_kv4_cache* cache, const tern_kv4_batch* batch, Kv4Params* c);

}  // namespace tern
