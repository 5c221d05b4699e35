// Attention of prompts and chunks of prompts over the paged 4-bit cache, on the
// 5th-generation tensor cores: sequences with more than a few query rows per kv
// head (a row is one token's one query head).
//
// Mathematics. out = softmax(scale q k^T) v in the usual one pass over the keys
// with a running reference maximum. A block of 128 keys and values is turned into
// fp16 operands once, fl16(min + scale * code), for up to 256 query rows; that
// rounding, half a step of 2^-11 of each element, is far below the bf16 rounding
// of the output. q is bf16; its row is multiplied by a power of two that puts its
// largest element at 2^14..2^15 of fp16 (and by the sign of `scale`), which keeps
// all its bits. Probabilities go to fp16 as 2^(x - reference + 7); the
// accumulator is rescaled only when a row's maximum has passed its reference by 2^8,
// so they stay below 2^15 and the smallest keep their bits. Sums in fp32.
//
// Work of a CTA: up to two tiles of 128 query rows (the group of heads that reads
// one kv head, times consecutive tokens) over a range of blocks of 128 positions.
//   warps 0-3, 4-7   softmax of the first and second tile, a thread per row:
//                    scores from tensor memory, probabilities back into the columns
//                    that the scores held;
//   warps 8-11       codes -> fp16 in shared memory, a thread per position (128-byte
//                    swizzle; dimensions in the order 0 4 1 5 2 6 3 7 of every eight, as
//                    the masks leave them: q is stored in the same order and the
//                    output's columns are put back when they are written);
//   warp 12          one thread issues S = Q K^T (both operands in shared memory)
//                    and O += P V (P in tensor memory, V with its dimensions
//                    contiguous); the two tiles alternate, so that the tensor cores
//                    work on one while the softmax of the other runs.
// Tensor memory: S of the tiles in columns 0 and 128, O in 256 and 384.
//
// Split. The blocks that each tile sees are laid end to end and dealt in equal
// shares, as in the kernel for few rows; causal tiles cost what they see. A unit cut
// between CTAs is joined by the last of them, in position order.
// Every wait is bounded; on expiry the device error word records a timeout and the
// CTA runs to its end without waiting further.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "tern_kv4.cuh"
#include "tern_tc.cuh"

namespace tern {

int read_clear_dev_error_kv4_prompt(void* stream, unsigned* out) { return read_clear_dev_error_tu(stream, out); }

namespace {

using kv4::ex2;
using kv4::exp2i;

constexpr int kWarps = 13;
constexpr int kThreads = 32 * kWarps;
constexpr int kBlock = 128;             // positions
constexpr int kRows = 256;              // query rows of a unit
constexpr int kHalf = 128;              // of a tile
constexpr int kSub = kBlock * 128;      // bytes of 128 rows by 64 fp16
constexpr float kShift = 7.f;           // probabilities are 2^(x - reference + 7)
constexpr float kGrowth = 8.f;          // a maximum may pass its reference by this much

struct Ctl {
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_free[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], fin;
  uint32_t misc[4];
  alignas(16) uint32_t absent[4][4];  // positions of block (its number mod 4) that a bad page leaves out, a bit each
  alignas(16) uint32_t poison[4][4];  // positions whose values are not finite
  kv4::ShareScratch<kWarps> share;
  int last;
};
constexpr int kCtlBytes = 1024;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

// One stretch of blocks [b0, b1) of a unit (sequence, tile of 256 rows, kv head).
struct Segment {
  kv4::Seq q;
  int s, h, row_first, rows, b0, b1, blocks;
  long long unit_first;  // the unit's first block among all
};

__device__ __forceinline__ int unit_blocks(const Kv4PromptParams& p, const kv4::Seq& q, int tile) {
  const int row_last = min(q.n * p.group, (tile + 1) * kRows) - 1;
  const int seen = q.len - q.n + row_last / p.group + 1;
  return max(1, (seen + kBlock - 1) / kBlock);
}
__device__ __forceinline__ int seq_tiles(const Kv4PromptParams& p, const kv4::Seq& q) {
  return (q.n * p.group + kRows - 1) / kRows;
}
__device__ __forceinline__ long long seq_blocks(const Kv4PromptParams& p, const kv4::Seq& q) {
  if (!q.ok || q.n * p.group < p.min_rows) return 0;
  long long v = 0;
  for (int t = 0; t < seq_tiles(p, q); ++t) v += unit_blocks(p, q, t);
  return v * p.c.kv_heads;
}

// Walks a CTA's share, segment by segment; every role has its own.
struct Walk {
  long long at, stop, in_tile;
  int s, tile;
  kv4::Seq q;
  __device__ __forceinline__ Walk(const Kv4PromptParams& p, const kv4::Share& sh)
      : at(sh.at), stop(sh.stop), in_tile(sh.in_seq), s(sh.s), tile(0), q(kv4::load_seq(p.c, sh.s)) {
    skip(p);
  }
  // past the tiles that end before the place
  __device__ __forceinline__ void skip(const Kv4PromptParams& p) {
    const int tiles = seq_tiles(p, q);
    while (tile < tiles) {
      const long long span = (long long)unit_blocks(p, q, tile) * p.c.kv_heads;
      if (in_tile < span) return;
      in_tile -= span;
      ++tile;
    }
  }
  __device__ __forceinline__ bool next(const Kv4PromptParams& p, Segment* g) {
    if (at >= stop) return false;
    while (!q.ok || q.n * p.group < p.min_rows || tile >= seq_tiles(p, q)) {
      if (++s >= p.c.seqs) return false;
      q = kv4::load_seq(p.c, s);
      tile = 0;
      in_tile = 0;
    }
    const int blocks = unit_blocks(p, q, tile);
    g->q = q;
    g->s = s;
    g->h = (int)(in_tile / blocks);
    g->b0 = (int)(in_tile - (long long)g->h * blocks);
    g->b1 = (int)min((long long)blocks, g->b0 + (stop - at));
    g->blocks = blocks;
    g->row_first = tile * kRows;
    g->rows = min(kRows, q.n * p.group - g->row_first);
    g->unit_first = at - g->b0;
    at += g->b1 - g->b0;
    in_tile += g->b1 - g->b0;
    if (in_tile >= (long long)blocks * p.c.kv_heads) {
      in_tile = 0;
      ++tile;
    }
    return true;
  }
};

__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<const __half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<const uint32_t*>(&v); }
// 16-byte piece `c` of row `r` within 128 rows of 128 bytes, 128-byte swizzle
__device__ __forceinline__ uint32_t piece(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

// A token's head of D codes as fp16 min + scale * code in shared memory. The
// bits 0x6400 | c are the fp16 number 1024 + c, 0x6400 | 16 c is 1024 + 16 c: both
// give c exactly, and the last step rounds once.
template <int D>
__device__ __forceinline__ void expand(uint32_t dst, int row, const uint4 (&w)[D / 32], uint32_t pair) {
  const __half2 sm = as_half2(pair);
  const __half2 s2 = __low2half2(sm), m2 = __high2half2(sm);
  const __half2 k1024 = as_half2(0x64006400u), k16th = as_half2(0x2C002C00u), k64 = as_half2(0xD400D400u);
  auto even = [&](uint32_t x) {
    return as_u32(__hfma2(__hsub2(as_half2((x & 0x000F000Fu) | 0x64006400u), k1024), s2, m2));
  };
  auto odd = [&](uint32_t x) {
    return as_u32(__hfma2(__hfma2(as_half2((x & 0x00F000F0u) | 0x64006400u), k16th, k64), s2, m2));
  };
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint4 v = w[i / 4];
    const uint32_t x = i % 4 == 0 ? v.x : (i % 4 == 1 ? v.y : (i % 4 == 2 ? v.z : v.w));
    tc::sts128(dst + (uint32_t)(i / 8) * kSub + piece(row, i % 8), even(x), odd(x), even(x >> 8), odd(x >> 8));
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const Kv4PromptParams p) {
  constexpr int SUBS = D / 64;            // 64-dimension parts of an operand
  constexpr int kOperand = SUBS * kSub;   // bytes of 128 rows
  constexpr uint32_t kTmemCols = 512;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem), pad = (1024u - (base & 1023u)) & 1023u;
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + pad);
  const uint32_t qs = base + pad + kCtlBytes, ks = qs + 2 * kOperand, vs = ks + 2 * kOperand;
  const Kv4Params& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile uint32_t* misc = ctl.misc;

  kv4::Share sh;
  auto weight = [&](int i, bool report) -> long long {
    const kv4::Seq q = kv4::load_seq(c, i);
    if (!q.ok && report) kv4::report_bad();
    return seq_blocks(p, q);
  };
  if (!kv4::find_share<kWarps>(c.seqs, p.min_share, weight, ctl.share, &sh)) return;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.q_full[i], 4);
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i], 4);
      mbar_init(&ctl.o_full[i], 1);
      mbar_init(&ctl.o_free[i], 4);
      mbar_init(&ctl.k_full[i], 4);
      mbar_init(&ctl.k_empty[i], 1);
      mbar_init(&ctl.v_full[i], 4);
      mbar_init(&ctl.v_empty[i], 1);
    }
    mbar_init(&ctl.fin, 1);
    ctl.misc[tc::kMiscAbort] = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tc::tmem_alloc(smem_u32(&ctl.misc[tc::kMiscTmem]), kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = ctl.misc[tc::kMiscTmem];
  Walk walk(p, sh);
  Segment g;

  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    const int x = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + (uint32_t)(128 * x), o_col = tmem + lanes + 256u + (uint32_t)(128 * x);
    uint32_t s_ph = 0, o_ph = 0;
    int block = 0;  // blocks this CTA has seen
    while (walk.next(p, &g)) {
      const int nsub = g.rows > kHalf ? 2 : 1;
      const int rr = g.row_first + kHalf * x + row;  // among the sequence's rows of this kv head
      const bool live = kHalf * x + row < g.rows;
      const int tok = rr / p.group;
      const size_t at = ((size_t)(g.q.row0 + tok) * c.heads + (size_t)g.h * p.group + (rr - tok * p.group)) * D;
      const int limit = live ? g.q.len - g.q.n + tok + 1 : 1 << 30;  // positions the row sees
      float ref = -INFINITY, l = 0.f, rowf = 0.f;
      const bool here = x < nsub;
      if (here) {
        // q, times a power of two, in the swizzled layout
        auto load = [&](int i) {
          return live ? reinterpret_cast<const uint4*>(p.q + at)[i] : make_uint4(0, 0, 0, 0);
        };
        float big = 0.f;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 u = load(i);
          const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(e[k] << 16)), fabsf(__uint_as_float(e[k] & 0xFFFF0000u))));
        }
        const int ex = max(-100, (__float_as_int(big) >> 23) - 127);
        const float f = p.scale_log2 < 0.f ? -exp2i(14 - ex) : exp2i(14 - ex);
        rowf = exp2i(min(127, ex - 14)) * fabsf(p.scale_log2);
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          const uint4 u = load(i);
          const uint32_t e[4] = {u.x, u.y, u.z, u.w};
          auto lo = [&](int k) { return __uint_as_float(e[k] << 16) * f; };
          auto hi = [&](int k) { return __uint_as_float(e[k] & 0xFFFF0000u) * f; };
          tc::sts128(qs + (uint32_t)(x * kOperand + (i / 8) * kSub) + piece(row, i % 8), pack_half2(lo(0), lo(2)),
                     pack_half2(hi(0), hi(2)), pack_half2(lo(1), lo(3)), pack_half2(hi(1), hi(3)));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.q_full[x]);
      }
      for (int b = g.b0; b < g.b1; ++b, ++block) {
        if (!here) continue;
        tc::tc_wait_many(&ctl.s_full[x], s_ph, misc);
        s_ph ^= 1u;
        tc::fence_after_sync();
        const int seen = limit - b * kBlock;  // of this block's positions
        const uint4 ab = *reinterpret_cast<const uint4*>(ctl.absent[block & 3]),
                    po = *reinterpret_cast<const uint4*>(ctl.poison[block & 3]);
        const bool odd = (ab.x | ab.y | ab.z | ab.w | po.x | po.y | po.z | po.w) != 0u;
        const bool plain = __all_sync(0xffffffffu, seen >= kBlock && !odd);
        auto hidden = [&](int j) {  // of a masked block: is position j hidden from the row?
          const uint32_t w = j < 32 ? ab.x : (j < 64 ? ab.y : (j < 96 ? ab.z : ab.w));
          return j >= seen || ((w >> (j & 31)) & 1u);
        };
        float mx = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v[32];
          tc::ld_x32_sync(s_col + 32 * q, v);
          if (plain) {
#pragma unroll
            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(v[i]));
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!hidden(32 * q + i)) mx = fmaxf(mx, __uint_as_float(v[i]));
          }
        }
        const float top = mx == -INFINITY ? -INFINITY : mx * rowf;
        const bool grow = top > ref + kGrowth || (ref == -INFINITY && top > -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float next = fmaxf(ref, top);
          const float f = ref == -INFINITY ? 0.f : ex2(ref - next);
          ref = next;
          l *= f;
          if (b > g.b0) {  // the last block's product is complete: the scores came after it
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t v[16];
              tc::ld_x16_sync(o_col + 16 * q, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
              tc::st_x16(o_col + 16 * q, v);
            }
          }
        }
        const float bias = kShift - (ref == -INFINITY ? 0.f : ref);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v[32], w[16];
          tc::ld_x32_sync(s_col + 32 * q, v);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float e0 = ex2(fmaf(__uint_as_float(v[i]), rowf, bias)), e1 = ex2(fmaf(__uint_as_float(v[i + 1]), rowf, bias));
            if (!plain) {
              if (hidden(32 * q + i)) e0 = 0.f;
              if (hidden(32 * q + i + 1)) e1 = 0.f;
            }
            l += e0 + e1;
            w[i / 2] = pack_half2(e0, e1);
          }
          tc::st_x16(s_col + 16 * q, w);
        }
        if (odd) {  // a visible value that is not finite makes the row so
          for (int j = 0; j < kBlock; ++j) {
            const uint32_t w = j < 32 ? po.x : (j < 64 ? po.y : (j < 96 ? po.z : po.w));
            if (((w >> (j & 31)) & 1u) && !hidden(j)) l = NAN;
          }
        }
        tc::st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.p_full[x]);
      }
      // ---- the segment's end: the output, or a part of it
      const int first_cta = sh.cta_of(g.unit_first), last_cta = sh.cta_of(g.unit_first + g.blocks - 1);
      const bool whole = first_cta == last_cta;
      constexpr size_t kSlot = (size_t)kRows * (D + 2);  // floats: [D / 4][256][4], then (reference, sum) [256]
      float* part = p.part + (size_t)(2 * blockIdx.x + (g.b0 == 0 ? 1 : 0)) * kSlot;
      const int prow = kHalf * x + row;
      auto write = [&](int i, const float (&o)[8], float sum) {  // columns 8 i .. + 7
        const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
        auto two = [&](int a, int b) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(o[a] * inv, o[b] * inv);
          return *reinterpret_cast<const uint32_t*>(&v);
        };
        *reinterpret_cast<uint4*>(p.out + at + 8 * i) = make_uint4(two(0, 2), two(4, 6), two(1, 3), two(5, 7));
      };
      if (here) {
        tc::tc_wait_many(&ctl.o_full[x], o_ph, misc);
        tc::fence_after_sync();
#pragma unroll 1
        for (int q = 0; q < D / 16; ++q) {
          uint32_t v[16];
          tc::ld_x16_sync(o_col + 16 * q, v);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __uint_as_float(v[8 * i + k]);
            if (whole) {
              if (live) write(2 * q + i, o, l);
            } else {
              float4* dst = reinterpret_cast<float4*>(part);
              dst[(4 * q + 2 * i) * kRows + prow] = make_float4(o[0], o[1], o[2], o[3]);
              dst[(4 * q + 2 * i + 1) * kRows + prow] = make_float4(o[4], o[5], o[6], o[7]);
            }
          }
        }
        if (!whole) reinterpret_cast<float2*>(part + (size_t)kRows * D)[prow] = make_float2(ref, l);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.o_free[x]);
        o_ph ^= 1u;
      }
      if (!whole) {
        const int ns = last_cta - first_cta + 1;
        __threadfence();
        sync_softmax();
        if (threadIdx.x == 0) {
          ctl.last = atomicAdd(p.cnt + first_cta, 1u) == (unsigned)(ns - 1);
          if (ctl.last) p.cnt[first_cta] = 0u;
        }
        sync_softmax();
        if (ctl.last && live) {
          __threadfence();
          const float* parts = p.part + (size_t)2 * first_cta * kSlot;
          auto slot = [&](int i) { return parts + (size_t)(i == 0 ? 1 : 2 * i) * kSlot; };
          float top = -INFINITY, sum = 0.f;
          for (int i = 0; i < ns; ++i)
            top = fmaxf(top, __ldcg(reinterpret_cast<const float2*>(slot(i) + (size_t)kRows * D) + prow).x);
          for (int i = 0; i < ns; ++i) {
            const float2 e = __ldcg(reinterpret_cast<const float2*>(slot(i) + (size_t)kRows * D) + prow);
            sum = fmaf(e.x == -INFINITY ? 0.f : ex2(e.x - top), e.y, sum);
          }
#pragma unroll 1
          for (int q = 0; q < D / 8; ++q) {
            float o[8] = {};
#pragma unroll 4
            for (int i = 0; i < ns; ++i) {
              const float e = __ldcg(reinterpret_cast<const float2*>(slot(i) + (size_t)kRows * D) + prow).x;
              const float f = e == -INFINITY ? 0.f : ex2(e - top);
              const float4* src = reinterpret_cast<const float4*>(slot(i));
              const float4 a = __ldcg(src + (2 * q) * kRows + prow), d = __ldcg(src + (2 * q + 1) * kRows + prow);
              o[0] = fmaf(f, a.x, o[0]), o[1] = fmaf(f, a.y, o[1]), o[2] = fmaf(f, a.z, o[2]), o[3] = fmaf(f, a.w, o[3]);
              o[4] = fmaf(f, d.x, o[4]), o[5] = fmaf(f, d.y, o[5]), o[6] = fmaf(f, d.z, o[6]), o[7] = fmaf(f, d.w, o[7]);
            }
            write(q, o, sum);
          }
        }
        sync_softmax();
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------- codes -> operands
    const int tid = threadIdx.x - 256;  // position within a block
    int block = 0;
    while (walk.next(p, &g)) {
      for (int b = g.b0; b < g.b1; ++b, ++block) {
        const int pos = b * kBlock + tid, stage = block & 1;
        const bool inside = pos < g.q.len;
        int page = -1;
        if (inside) {
          page = kv4::page_of(c, g.s, pos);
          if (page < 0) kv4::report_bad();
        }
        uint4 kw[D / 32], vw[D / 32];
        uint2 pair = make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) kw[i] = vw[i] = make_uint4(0, 0, 0, 0);
        if (page >= 0) {
          const uint8_t* blk = c.pages + kv4::block_offset(c, page, g.h);
          const int slot = pos & (c.page - 1);
          const uint4* kr = reinterpret_cast<const uint4*>(blk + (size_t)slot * (D / 2));
          const uint4* vr = reinterpret_cast<const uint4*>(blk + (size_t)(c.page + slot) * (D / 2));
#pragma unroll
          for (int i = 0; i < D / 32; ++i) kw[i] = __ldg(kr + i), vw[i] = __ldg(vr + i);
          pair = __ldg(reinterpret_cast<const uint2*>(blk + (size_t)c.page * D + (size_t)slot * 8));
        }
        const float2 vp = __half22float2(as_half2(pair.y));
        const bool bad_value = !(fabsf(vp.y) + 15.f * fabsf(vp.x) < 65520.f);  // as fp16, or not a number
        const uint32_t ab = __ballot_sync(0xffffffffu, inside && page < 0);
        const uint32_t po = __ballot_sync(0xffffffffu, bad_value);
        if (block >= 2) tc::tc_wait_many(&ctl.k_empty[stage], (uint32_t)(block / 2 - 1) & 1u, misc);
        if (lane == 0) {
          ctl.absent[block & 3][tid >> 5] = ab;
          ctl.poison[block & 3][tid >> 5] = po;
        }
        expand<D>(ks + (uint32_t)(stage * kOperand), tid, kw, pair.x);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.k_full[stage]);
        if (block >= 2) tc::tc_wait_many(&ctl.v_empty[stage], (uint32_t)(block / 2 - 1) & 1u, misc);
        expand<D>(vs + (uint32_t)(stage * kOperand), tid, vw, bad_value ? 0u : pair.y);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.v_full[stage]);
      }
    }
  } else {
    // ------------------------------------------------------------------ MMA
    if (lane == 0) {
      constexpr uint32_t id_s = tc::idesc_f16_f32(kBlock, false), id_o = tc::idesc_f16_f32(D, true);
      int block = 0;
      uint32_t p_ph[2] = {0, 0}, q_ph[2] = {0, 0}, o_uses[2] = {0, 0};
      auto scores = [&](int x, int stage) {
        const uint32_t a = qs + (uint32_t)(x * kOperand), b = ks + (uint32_t)(stage * kOperand);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t o = (uint32_t)((i / 4) * kSub + (i % 4) * 32);
          tc::mma_f16_ss(tmem + (uint32_t)(128 * x), tc::smem_desc_sw128(a + o), tc::smem_desc_sw128(b + o), id_s,
                         i > 0 ? 1u : 0u);
        }
        tc::commit(&ctl.s_full[x]);
      };
      while (walk.next(p, &g) && !misc[tc::kMiscAbort]) {
        const int nsub = g.rows > kHalf ? 2 : 1;
        tc::tc_wait(&ctl.k_full[block & 1], (uint32_t)(block / 2) & 1u, misc);
        for (int x = 0; x < nsub; ++x) {
          tc::tc_wait(&ctl.q_full[x], q_ph[x], misc);
          q_ph[x] ^= 1u;
          tc::fence_after_sync();
          scores(x, block & 1);
        }
        tc::commit(&ctl.k_empty[block & 1]);
        for (int b = g.b0; b < g.b1; ++b, ++block) {
          if (misc[tc::kMiscAbort]) break;
          const bool more = b + 1 < g.b1;
          tc::tc_wait(&ctl.v_full[block & 1], (uint32_t)(block / 2) & 1u, misc);
          for (int x = 0; x < nsub; ++x) {
            tc::tc_wait(&ctl.p_full[x], p_ph[x], misc);
            p_ph[x] ^= 1u;
            // the accumulator's last user has read it
            if (b == g.b0 && o_uses[x] > 0) tc::tc_wait(&ctl.o_free[x], (o_uses[x] - 1) & 1u, misc);
            tc::fence_after_sync();
            const uint32_t v = vs + (uint32_t)((block & 1) * kOperand);
#pragma unroll
            for (int i = 0; i < kBlock / 16; ++i)
              tc::mma_f16_ts(tmem + 256u + (uint32_t)(128 * x), tmem + (uint32_t)(128 * x + 8 * i),
                             tc::smem_desc_sw128_mn(v + (uint32_t)(i * 16 * 128), kSub), id_o,
                             b > g.b0 || i > 0 ? 1u : 0u);
            if (more) {
              if (x == 0) {
                tc::tc_wait(&ctl.k_full[(block + 1) & 1], (uint32_t)((block + 1) / 2) & 1u, misc);
                tc::fence_after_sync();
              }
              scores(x, (block + 1) & 1);
            } else {
              tc::commit(&ctl.o_full[x]);
              ++o_uses[x];
            }
          }
          tc::commit(&ctl.v_empty[block & 1]);
          if (more) tc::commit(&ctl.k_empty[(block + 1) & 1]);
        }
      }
      // every MMA issued has completed before tensor memory is released
      tc::commit(&ctl.fin);
      mbar_wait_bounded(&ctl.fin, 0u);
    }
  }
  __syncthreads();
  if (warp == 12) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D>
int launch_dim(const Kv4PromptParams& p, int ctas, cudaStream_t s) {
  constexpr int bytes = 1024 + kCtlBytes + 6 * (D / 64) * kSub;
  const cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return (int)e;
  prompt_kernel<D><<<ctas, kThreads, bytes, s>>>(p);
  return (int)cudaGetLastError();
}

}  // namespace

size_t kv4_prompt_part_bytes(int dim, int ctas) { return (size_t)ctas * 2 * kRows * (size_t)(dim + 2) * 4; }

int launch_kv4_prompt(const Kv4PromptParams& p, int ctas, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p.c.dim == 128 ? launch_dim<128>(p, ctas, s) : launch_dim<64>(p, ctas, s);
}

}  // namespace tern
