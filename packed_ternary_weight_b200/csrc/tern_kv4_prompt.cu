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

constexpr int kWarps = 16;  // of them 13-15 idle: register shares move between groups of four warps
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
  kv4::Share mine;  // this CTA's share
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
  long long at, stop;
  int s, tile, h, b;  // where the next segment begins
  kv4::Seq q;
  __device__ __forceinline__ Walk(const Kv4PromptParams& p, const kv4::Share& sh)
      : at(sh.at), stop(sh.stop), s(sh.s), tile(0), h(0), b(0), q(kv4::load_seq(p.c, sh.s)) {
    long long left = sh.in_seq;  // blocks of the sequence before the place
    const int tiles = seq_tiles(p, q);
    for (; tile < tiles; ++tile) {
      const int blocks = unit_blocks(p, q, tile);
      const long long span = (long long)blocks * p.c.kv_heads;
      if (left < span) {
        h = (int)(left / blocks);
        b = (int)(left - (long long)h * blocks);
        break;
      }
      left -= span;
    }
  }
  __device__ __forceinline__ bool next(const Kv4PromptParams& p, Segment* g) {
    if (at >= stop) return false;
    while (!q.ok || q.n * p.group < p.min_rows || tile >= seq_tiles(p, q)) {
      if (++s >= p.c.seqs) return false;
      q = kv4::load_seq(p.c, s);
      tile = h = b = 0;
    }
    const int blocks = unit_blocks(p, q, tile);
    g->q = q;
    g->s = s;
    g->h = h;
    g->b0 = b;
    g->b1 = (int)min((long long)blocks, b + (stop - at));
    g->blocks = blocks;
    g->row_first = tile * kRows;
    g->rows = min(kRows, q.n * p.group - g->row_first);
    g->unit_first = at - b;
    at += g->b1 - b;
    b = g->b1;
    if (b >= blocks) {
      b = 0;
      if (++h >= p.c.kv_heads) {
        h = 0;
        ++tile;
      }
    }
    return true;
  }
};

__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
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

// Multiplies what a row has so far by f: `parts` times 32 probabilities at s_col
// and the accumulator at o_col (0: there is none yet).
template <int D>
__device__ __noinline__ void rescale(uint32_t s_col, int parts, float f, uint32_t o_col) {
  const __half2 f2 = __float2half2_rn(f);
  uint32_t h[16];
#pragma unroll 1
  for (int i = 0; i < parts; ++i) {
    tc::ld_x16_sync(s_col + 16 * i, h);
#pragma unroll
    for (int k = 0; k < 16; ++k) h[k] = as_u32(__hmul2(as_half2(h[k]), f2));
    tc::st_x16(s_col + 16 * i, h);
  }
#pragma unroll 1
  for (int i = 0; o_col != 0u && i < D / 16; ++i) {
    tc::ld_x16_sync(o_col + 16 * i, h);
#pragma unroll
    for (int k = 0; k < 16; ++k) h[k] = __float_as_uint(__uint_as_float(h[k]) * f);
    tc::st_x16(o_col + 16 * i, h);
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
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
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
    ctl.mine = sh;
    fence_mbar_init();
  }
  if (warp == 12) {
    tc::tmem_alloc(smem_u32(&ctl.misc[tc::kMiscTmem]), kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.misc[tc::kMiscTmem], 0);
  Walk walk(p, sh);
  Segment g;
  // the waits of whole warps: suspended by the hardware, bounded, given up at once after another's expiry
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!misc[tc::kMiscAbort] && !mbar_wait_bounded(bar, parity)) misc[tc::kMiscAbort] = 1u;
  };

  // The 512 threads start with 128 registers each, the whole file. Shares per
  // group of four warps: 152 + 152 (softmax) + 112 + 96 = 4 x 128.
  if (warp < 8) {
    // -------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
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
        uint4 u[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          u[i] = live ? reinterpret_cast<const uint4*>(p.q + at)[i] : make_uint4(0, 0, 0, 0);
        float big = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t e[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(e[k] << 16)), fabsf(__uint_as_float(e[k] & 0xFFFF0000u))));
        }
        const int ex = max(-100, (__float_as_int(big) >> 23) - 127);
        const float f = p.scale_log2 < 0.f ? -exp2i(14 - ex) : exp2i(14 - ex);
        rowf = fmaxf(exp2i(min(127, ex - 14)) * fabsf(p.scale_log2), 1e-30f);  // above zero: masked scores stay -inf
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t e[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
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
        wait(&ctl.s_full[x], s_ph);
        s_ph ^= 1u;
        tc::fence_after_sync();
        const int seen = limit - b * kBlock;  // of this block's positions
        const uint32_t* ab = ctl.absent[block & 3];
        const uint32_t* po = ctl.poison[block & 3];
        const bool odd = (ab[0] | ab[1] | ab[2] | ab[3] | po[0] | po[1] | po[2] | po[3]) != 0u;
        const bool plain = __all_sync(0xffffffffu, seen >= kBlock && !odd);
        auto visible = [&](int q) {  // a bit for each of the positions 32 q .. 32 q + 31
          const int n = seen - 32 * q;
          return (n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u)) & ~ab[q];
        };
        // 32 positions at a time, each score read once, the next ones on their way; a row whose maximum has passed
        // its reference by too much (the first block, hardly ever later) is rescaled
        const float2 rowf2 = make_float2(rowf, rowf);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t v[2][32];
        tc::ld_x32(s_col, v[0]);
#pragma unroll 1  // a short loop: four roles share the instruction caches
        for (int q = 0; q < 4; q += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t(&u)[32] = v[h];
            tc::ld_wait_x32(u);
            // after the last columns the first ones again, into registers that nothing reads
            tc::ld_x32(s_col + 32 * ((q + h + 1) & 3), v[h ^ 1]);
            if (!plain) {
              const uint32_t vis = visible(q + h);
#pragma unroll
              for (int i = 0; i < 32; ++i) u[i] = (vis >> i) & 1u ? u[i] : 0xFF800000u;  // minus infinity
            }
            float mx[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(__uint_as_float(u[k]), __uint_as_float(u[4 + k]));
#pragma unroll
            for (int i = 8; i < 32; i += 8) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(u[i + k])), __uint_as_float(u[i + 4 + k]));
            }
            const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
            const float top = most == -INFINITY ? -INFINITY : most * rowf;
            const bool grow = top > ref + kGrowth || (ref == -INFINITY && top > -INFINITY);
            if (__any_sync(0xffffffffu, grow)) {
              const float next = fmaxf(ref, top);
              const float f = ref == -INFINITY ? 0.f : ex2(ref - next);
              ref = next;
              l *= f;
#pragma unroll
              for (int k = 0; k < 2; ++k) sum[k] = make_float2(sum[k].x * f, sum[k].y * f);
              rescale<D>(s_col, q + h, f, b > g.b0 ? o_col : 0u);
            }
            const float bias = kShift - (ref == -INFINITY ? 0.f : ref);
            const float2 bias2 = make_float2(bias, bias);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 x = fma2(make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), rowf2, bias2);
              const float2 e = make_float2(ex2(x.x), ex2(x.y));
              sum[(i / 2) & 1] = add2(sum[(i / 2) & 1], e);
              w[i / 2] = pack_half2(e.x, e.y);
            }
            tc::st_x16(s_col + 16 * (q + h), w);
          }
        }
        tc::ld_wait_x32(v[0]);
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if (odd) {  // a visible value that is not finite makes the row so
          for (int q = 0; q < 4; ++q)
            if (po[q] & visible(q)) l = NAN;
        }
        tc::st_wait();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.p_full[x]);
      }
      // ---- the segment's end: the output, or a part of it
      const int first_cta = ctl.mine.cta_of(g.unit_first), last_cta = ctl.mine.cta_of(g.unit_first + g.blocks - 1);
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
        wait(&ctl.o_full[x], o_ph);
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
          for (int q = 0; q < D / 32; ++q) {  // 32 columns, eight loads in flight
            float o[4][8] = {};
#pragma unroll 1
            for (int i = 0; i < ns; ++i) {
              const float4* src = reinterpret_cast<const float4*>(slot(i)) + (8 * q) * kRows + prow;
              const float e = __ldcg(reinterpret_cast<const float2*>(slot(i) + (size_t)kRows * D) + prow).x;
              float4 a[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) a[k] = __ldcg(src + k * kRows);
              const float f = e == -INFINITY ? 0.f : ex2(e - top);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                float* d = o[k / 2] + 4 * (k & 1);
                d[0] = fmaf(f, a[k].x, d[0]), d[1] = fmaf(f, a[k].y, d[1]);
                d[2] = fmaf(f, a[k].z, d[2]), d[3] = fmaf(f, a[k].w, d[3]);
              }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) write(4 * q + k, o[k], sum);
          }
        }
        sync_softmax();
      }
    }
  } else if (warp < 12) {
    // ------------------------------------------------- codes -> operands
    asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
    // Three steps in flight: the page of block i + 2, the codes of block i + 1, block i into shared memory.
    const int tid = threadIdx.x - 256;  // position within a block
    struct {
      bool valid, inside;
      int page, slot, h;
    } ahead;
    int b = 0, b1 = 0;
    auto look_up = [&] {  // the next block of the share
      if (b == b1) {
        ahead.valid = walk.next(p, &g);
        if (!ahead.valid) return;
        b = g.b0;
        b1 = g.b1;
      }
      const int pos = b * kBlock + tid;
      ahead.valid = true;
      ahead.inside = pos < g.q.len;
      ahead.page = ahead.inside ? __ldg(c.table + (size_t)g.s * c.max_pages + (pos >> c.log_page)) : -1;
      ahead.slot = pos & (c.page - 1);
      ahead.h = g.h;
      ++b;
    };
    uint4 kn[D / 32], vn[D / 32];
    uint2 pn = make_uint2(0, 0);
    bool valid, absent = false;
    auto load = [&] {
      valid = ahead.valid;
      if (!valid) return;
      const bool there = (unsigned)ahead.page < (unsigned)c.num_pages;
      absent = ahead.inside && !there;
      if (absent) kv4::report_bad();
      pn = make_uint2(0, 0);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) kn[i] = vn[i] = make_uint4(0, 0, 0, 0);
      if (there) {
        const uint8_t* blk = c.pages + kv4::block_offset(c, ahead.page, ahead.h);
        const uint4* kr = reinterpret_cast<const uint4*>(blk + (size_t)ahead.slot * (D / 2));
        const uint4* vr = reinterpret_cast<const uint4*>(blk + (size_t)(c.page + ahead.slot) * (D / 2));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) kn[i] = __ldg(kr + i), vn[i] = __ldg(vr + i);
        pn = __ldg(reinterpret_cast<const uint2*>(blk + (size_t)c.page * D + (size_t)ahead.slot * 8));
      }
    };
    look_up();
    load();
    if (valid) look_up();
    for (int block = 0; valid; ++block) {
      const int stage = block & 1;
      uint4 kw[D / 32], vw[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) kw[i] = kn[i], vw[i] = vn[i];
      const uint2 pair = pn;
      const float2 vp = __half22float2(as_half2(pair.y));
      const bool bad_value = !(fabsf(vp.y) + 15.f * fabsf(vp.x) < 65520.f);  // as fp16, or not a number
      const uint32_t ab = __ballot_sync(0xffffffffu, absent), po = __ballot_sync(0xffffffffu, bad_value);
      load();
      if (valid) look_up();
#pragma unroll 1  // keys, then values: one copy of the code
      for (int which = 0; which < 2; ++which) {
        if (block >= 2)
          wait(which == 0 ? &ctl.k_empty[stage] : &ctl.v_empty[stage], (uint32_t)(block / 2 - 1) & 1u);
        if (which == 0) {
          if (lane == 0) {
            ctl.absent[block & 3][tid >> 5] = ab;
            ctl.poison[block & 3][tid >> 5] = po;
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 32; ++i) kw[i] = vw[i];
        }
        expand<D>((which == 0 ? ks : vs) + (uint32_t)(stage * kOperand), tid, kw,
                  which == 0 ? pair.x : (bad_value ? 0u : pair.y));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(which == 0 ? &ctl.k_full[stage] : &ctl.v_full[stage]);
      }
    }
  } else {
    // ------------------------------------------------------------------ MMA
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 12) {
      // the whole warp in step, one lane of it issuing
      constexpr uint32_t id_s = tc::idesc_f16_f32(kBlock, false), id_o = tc::idesc_f16_f32(D, true);
      const uint32_t lead = lane == 0 ? 1u : 0u;
      bool ok = true;
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, tc::tc_wait(bar, parity, misc)) && ok;
      };
      uint32_t block = 0, p_ph[2] = {0, 0}, q_ph[2] = {0, 0}, o_uses[2] = {0, 0};
      // descriptors: an address offset adds to the field in units of 16 bytes
      const uint64_t dq = tc::smem_desc_sw128(qs), dk = tc::smem_desc_sw128(ks), dv = tc::smem_desc_sw128_mn(vs, kSub);
      auto scores = [&](int x, uint32_t stage) {
        const uint64_t a = dq + (uint32_t)(x * (kOperand >> 4)), k = dk + stage * (uint32_t)(kOperand >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t o = (uint32_t)(((i / 4) * kSub + (i % 4) * 32) >> 4);
          tc::mma_f16_ss(tmem + (uint32_t)(128 * x), a + o, k + o, id_s, i > 0 ? 1u : 0u, lead);
        }
        tc::commit_lead(&ctl.s_full[x], lead);
      };
      auto values = [&](int x, uint32_t stage, uint32_t more) {
        const uint64_t v = dv + stage * (uint32_t)(kOperand >> 4);
#pragma unroll
        for (int i = 0; i < kBlock / 16; ++i)
          tc::mma_f16_ts(tmem + 256u + (uint32_t)(128 * x), tmem + (uint32_t)(128 * x + 8 * i), v + (uint32_t)(i * 128),
                         id_o, i > 0 ? 1u : more, lead);
      };
      while (walk.next(p, &g)) {
        const int nsub = __shfl_sync(0xffffffffu, g.rows > kHalf ? 2 : 1, 0);
        const int blocks = __shfl_sync(0xffffffffu, g.b1 - g.b0, 0);
        wait_all(&ctl.k_full[block & 1], (block / 2) & 1u);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x < nsub) {
            wait_all(&ctl.q_full[x], q_ph[x]);
            q_ph[x] ^= 1u;
            tc::fence_after_sync();
            if (!ok) break;
            scores(x, block & 1);
          }
        }
        tc::commit_lead(&ctl.k_empty[block & 1], lead);
        for (int b = 0; b < blocks && ok; ++b, ++block) {
          const bool more = b + 1 < blocks;
          wait_all(&ctl.v_full[block & 1], (block / 2) & 1u);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            if (x >= nsub) break;
            wait_all(&ctl.p_full[x], p_ph[x]);
            p_ph[x] ^= 1u;
            // the accumulator's last user has read it
            if (b == 0 && o_uses[x] > 0) wait_all(&ctl.o_free[x], (o_uses[x] - 1) & 1u);
            tc::fence_after_sync();
            if (!ok) break;
            values(x, block & 1, b > 0 ? 1u : 0u);
            if (more) {
              if (x == 0) {
                wait_all(&ctl.k_full[(block + 1) & 1], ((block + 1) / 2) & 1u);
                tc::fence_after_sync();
                if (!ok) break;
              }
              scores(x, (block + 1) & 1);
            } else {
              tc::commit_lead(&ctl.o_full[x], lead);
              ++o_uses[x];
            }
          }
          tc::commit_lead(&ctl.v_empty[block & 1], lead);
          if (more) tc::commit_lead(&ctl.k_empty[(block + 1) & 1], lead);
        }
        if (!ok) break;
      }
      // every MMA issued has completed before tensor memory is released
      tc::commit_lead(&ctl.fin, lead);
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
