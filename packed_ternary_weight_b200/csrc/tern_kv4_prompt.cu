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
//   warps 0-7, 8-15  softmax of the first and second tile, two threads per row, one
//                    for each half of a block's positions: scores from tensor memory,
//                    probabilities back into columns that the same half's scores held.
//                    With one thread per row the softmax of a block took 3000 cycles
//                    (two warps per scheduler cannot hide its latencies);
//   warps 16-19      codes -> fp16 in shared memory, a thread per position (128-byte
//                    swizzle; dimensions in the order 0 4 1 5 2 6 3 7 of every eight, as
//                    the masks leave them: q is stored in the same order and the
//                    output's columns are put back when they are written);
//   warp 20          issues S = Q K^T (both operands in shared memory) and O += P V (P
//                    in tensor memory, V with its dimensions contiguous); the two
//                    tiles alternate, so that the tensor cores work on one while the
//                    softmax of the other runs.
// Tensor memory: S of the tiles in columns 0 and 128, O in 256 and 384.
//
// Split. The blocks that each tile sees are laid end to end and dealt in equal
// shares, as in the kernel for few rows; causal tiles cost what they see. A unit cut
// between CTAs is joined by the last of them, in position order.
//
// Measured: 2048-token chunks behind 6142 positions and shorter ones (32 heads on 8 kv
// heads, D = 128) 0.44-0.45 ms in a replayed graph, 0.85 PFLOP/s, half of the measured bf16
// rate (0.46 ms as calls; 0.47 ms over seconds, at the power cap's 1.79 GHz); the same at D
// = 64 0.33 ms (the exponentials are the same, the products half). A unit of one block
// takes 9 us by itself, so a prompt of 2048 without history takes 140 us, as long as one
// behind 2048 positions: shares count blocks, and the first tiles, of one or two blocks
// each, go to a few CTAs. A block of both
// tiles takes about 4800 cycles, 2050 of them of tensor work at the full rate; the limit is
// each tile's own chain, which nothing shortens by overlap: softmax 2700 (its exponentials
// alone 2050 of the special-function pipe, shared with the other tile), O += P V and the
// next S 1400 (S takes 95 instead of 64 cycles per instruction: both operands come from
// shared memory), and the signals between the roles 700. Without gain were: 64-position
// halves with two score buffers, probabilities handed over in halves, one reading of the
// scores, a polynomial for a part of the exponentials, eight instead of four expanding
// warps; three idle warps for register shares of 88 (softmax, expansion) and 40 cost 2 %.
// Every wait is bounded; on expiry the device error word records a timeout and the
// CTA runs to its end without waiting further.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "tern_kv4.cuh"
#include "tern_launch.cuh"
#include "tern_tc.cuh"

namespace tern {

int read_clear_dev_error_kv4_prompt(void* stream, unsigned* out) { return read_clear_dev_error_tu(stream, out); }

namespace {

using kv4::ex2;
using kv4::exp2i;

constexpr int kWarps = 21;
constexpr int kExpandWarp = 16, kMmaWarp = 20;
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
  float top[2][2][128], sum[2][2][128];  // rows' maxima and sums that the two threads of a row exchange
  float rowf[2][128];                    // what turns a row's scores into exponents
  alignas(16) uint32_t absent[4][4];  // positions of block (its number mod 4) that a bad page leaves out, a bit each
  alignas(16) uint32_t poison[4][4];  // positions whose values are not finite
  kv4::ShareScratch<kWarps> share;
  kv4::Share mine;  // this CTA's share
  int last;
};
constexpr int kCtlBytes = 6 * 1024;
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

__device__ __forceinline__ void sync_softmax() { asm volatile("bar.sync 9, 512;" ::: "memory"); }
// One tile's eight warps (barriers 10 and 11).
__device__ __forceinline__ void sync_tile(int x) { asm volatile("bar.sync %0, 256;" ::"r"(10 + x) : "memory"); }
// The two warps that share 32 rows (barriers 1-8): a barrier, and the OR of a predicate over it.
__device__ __forceinline__ void sync_pair(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool any_pair(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbar.red.or.pred q, %1, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(v ? 1u : 0u)
      : "memory");
  return r != 0u;
}
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
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
  pdl_launch_dependents();
  pdl_wait();

  kv4::Share sh;
  auto weight = [&](int i, bool report) -> long long {
    const kv4::Seq q = kv4::load_seq(c, i);
    if (!q.ok && report) kv4::report_bad();
    return seq_blocks(p, q);
  };
  if (!kv4::find_share<kWarps>(c.seqs, p.min_share, weight, ctl.share, &sh)) return;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.q_full[i], 8);
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i], 8);
      mbar_init(&ctl.o_full[i], 1);
      mbar_init(&ctl.o_free[i], 8);
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
  if (warp == kMmaWarp) {
    tc::tmem_alloc(smem_u32(&ctl.misc[tc::kMiscTmem]), kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.misc[tc::kMiscTmem], 0);
  Walk walk(p, sh);
  Segment g;
  auto wait = [&](uint64_t* bar, uint32_t parity) { tc::tc_wait_late<true>(bar, parity, misc); };

  if (warp < kExpandWarp) {
    // -------------------------------------------------------------- softmax
    const int x = warp >> 3, half = (warp >> 2) & 1, row = threadIdx.x & 127, pair = 1 + 4 * x + (warp & 3);
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_col = tmem + lanes + (uint32_t)(128 * x + 64 * half),
                   o_col = tmem + lanes + 256u + (uint32_t)(128 * x + (D / 2) * half);
    uint32_t s_ph = 0, o_ph = 0;
    int block = 0;  // blocks this CTA has seen
    while (walk.next(p, &g)) {
      const int nsub = g.rows > kHalf ? 2 : 1;
      const int rr = g.row_first + kHalf * x + row;  // among the sequence's rows of this kv head
      const bool live = kHalf * x + row < g.rows;
      // element offset of one of the sequence's rows of this kv head
      auto place = [&](int i) {
        const int t = i / p.group;
        return ((size_t)(g.q.row0 + t) * c.heads + (size_t)g.h * p.group + (i - t * p.group)) * D;
      };
      const int limit = live ? g.q.len - g.q.n + rr / p.group + 1 : 1 << 30;  // positions the row sees
      float ref = -INFINITY, l = 0.f, rowf = 0.f;
      const bool here = x < nsub;
      if (here) {
        // q, times a power of two, in the swizzled layout: D / 8 lanes take a row, 16 bytes each
        constexpr int kPieces = D / 8, kTurns = 128 * kPieces / 256;
        const int tt = threadIdx.x & 255, pc = tt % kPieces;
        uint4 u[kTurns];
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
          const int r = j * (256 / kPieces) + tt / kPieces;
          u[j] = make_uint4(0, 0, 0, 0);
          if (kHalf * x + r < g.rows)
            u[j] = *reinterpret_cast<const uint4*>(p.q + place(g.row_first + kHalf * x + r) + 8 * pc);
        }
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
          const int r = j * (256 / kPieces) + tt / kPieces;
          const uint32_t e[4] = {u[j].x, u[j].y, u[j].z, u[j].w};
          float big = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(e[k] << 16)), fabsf(__uint_as_float(e[k] & 0xFFFF0000u))));
#pragma unroll
          for (int k = kPieces / 2; k; k >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, k));
          const int ex = max(-100, (__float_as_int(big) >> 23) - 127);
          const float f = p.scale_log2 < 0.f ? -exp2i(14 - ex) : exp2i(14 - ex);
          // above zero: masked scores stay -inf
          if (pc == 0) ctl.rowf[x][r] = fmaxf(exp2i(min(127, ex - 14)) * fabsf(p.scale_log2), 1e-30f);
          auto lo = [&](int k) { return __uint_as_float(e[k] << 16) * f; };
          auto hi = [&](int k) { return __uint_as_float(e[k] & 0xFFFF0000u) * f; };
          tc::sts128(qs + (uint32_t)(x * kOperand + (pc / 8) * kSub) + piece(r, pc % 8), pack_half2(lo(0), lo(2)),
                     pack_half2(hi(0), hi(2)), pack_half2(lo(1), lo(3)), pack_half2(hi(1), hi(3)));
        }
        fence_proxy_async_smem();
        sync_tile(x);
        if (lane == 0) tc::mbar_arrive(&ctl.q_full[x]);
        rowf = ctl.rowf[x][row];
      }
      for (int b = g.b0; b < g.b1; ++b, ++block) {
        if (!here) continue;
        wait(&ctl.s_full[x], s_ph);
        s_ph ^= 1u;
        tc::fence_after_sync();
        const int seen = limit - b * kBlock - 64 * half;  // of this half of the block's positions
        const uint32_t* ab = ctl.absent[block & 3] + 2 * half;
        const uint32_t* po = ctl.poison[block & 3] + 2 * half;
        const bool odd = (ab[0] | ab[1] | po[0] | po[1]) != 0u;
        const bool plain = __all_sync(0xffffffffu, seen >= 64 && !odd);
        auto visible = [&](int q) {  // a bit for each of the positions 32 q .. 32 q + 31 of the half
          const int n = seen - 32 * q;
          return (n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u)) & ~ab[q];
        };
        auto scores = [&](int q, uint32_t (&u)[32]) {
          tc::ld_x32_sync(s_col + 32 * q, u);
          if (!plain) {
            const uint32_t vis = visible(q);
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = (vis >> i) & 1u ? u[i] : 0xFF800000u;  // minus infinity
          }
        };
        // the half's maximum; where a row's has passed its reference by too much (the first block, hardly ever
        // later), both threads of the row take a new one and rescale
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1  // short loops: the roles share the instruction caches
        for (int q = 0; q < 2; ++q) {
          uint32_t u[32];
          scores(q, u);
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = max3(mx[k], __uint_as_float(u[i + k]), __uint_as_float(u[i + 4 + k]));
          }
        }
        const float most = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        float top = most == -INFINITY ? -INFINITY : most * rowf;
        if (any_pair(pair, top > ref + kGrowth || (ref == -INFINITY && top > -INFINITY))) {
          ctl.top[x][half][row] = top;
          sync_pair(pair);
          const float next = fmaxf(ref, fmaxf(top, ctl.top[x][half ^ 1][row]));
          sync_pair(pair);
          const float f = ref == -INFINITY ? 0.f : ex2(ref - next);
          ref = next;
          l *= f;
          if (b > g.b0) {  // the last block's product is complete: the scores came after it
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              uint32_t h[16];
              tc::ld_x16_sync(o_col + 16 * i, h);
#pragma unroll
              for (int k = 0; k < 16; ++k) h[k] = __float_as_uint(__uint_as_float(h[k]) * f);
              tc::st_x16(o_col + 16 * i, h);
            }
          }
        }
        // then the probabilities
        const float bias = kShift - (ref == -INFINITY ? 0.f : ref);
        const float2 rowf2 = make_float2(rowf, rowf), bias2 = make_float2(bias, bias);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
        for (int q = 0; q < 2; ++q) {
          uint32_t u[32], w[16];
          scores(q, u);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 y = fma2(make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), rowf2, bias2);
            const float2 e = make_float2(ex2(y.x), ex2(y.y));
            sum[(i / 2) & 1] = add2(sum[(i / 2) & 1], e);
            w[i / 2] = pack_half2(e.x, e.y);
          }
          tc::st_x16(s_col + 16 * q, w);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if (odd) {  // a visible value that is not finite makes the row so
          for (int q = 0; q < 2; ++q)
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
      // the output's rows are gathered in the tile's part of the q area, which no MMA reads any more, and leave from
      // there as whole lines
      const uint32_t gather = qs + (uint32_t)(x * kOperand);
      auto write = [&](int i, const float (&o)[8], float sum) {  // columns 8 i .. + 7
        const float inv = sum > 0.f ? 1.0f / sum : (sum == 0.f ? 0.f : sum);
        auto two = [&](int a, int b) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(o[a] * inv, o[b] * inv);
          return *reinterpret_cast<const uint32_t*>(&v);
        };
        tc::sts128(gather + (uint32_t)((i / 8) * kSub) + piece(row, i % 8), two(0, 2), two(4, 6), two(1, 3), two(5, 7));
      };
      auto flush = [&] {
        sync_tile(x);
        constexpr int kPieces = D / 8, kTurns = 128 * kPieces / 256;
        const int tt = threadIdx.x & 255, pc = tt % kPieces;
#pragma unroll
        for (int j = 0; j < kTurns; ++j) {
          const int r = j * (256 / kPieces) + tt / kPieces;
          if (kHalf * x + r < g.rows) {
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(gather + (uint32_t)((pc / 8) * kSub) + piece(r, pc % 8)));
            *reinterpret_cast<uint4*>(p.out + place(g.row_first + kHalf * x + r) + 8 * pc) = v;
          }
        }
        sync_tile(x);  // the area takes q again
      };
      if (here) {
        ctl.sum[x][half][row] = l;
        sync_pair(pair);
        l = ctl.sum[x][0][row] + ctl.sum[x][1][row];
        sync_pair(pair);
        wait(&ctl.o_full[x], o_ph);
        tc::fence_after_sync();
#pragma unroll 1
        for (int j = 0; j < D / 32; ++j) {
          const int q = half * (D / 32) + j;  // columns 16 q .. + 15
          uint32_t v[16];
          tc::ld_x16_sync(o_col + 16 * j, v);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __uint_as_float(v[8 * i + k]);
            if (whole) {
              write(2 * q + i, o, l);
            } else {
              float4* dst = reinterpret_cast<float4*>(part);
              dst[(4 * q + 2 * i) * kRows + prow] = make_float4(o[0], o[1], o[2], o[3]);
              dst[(4 * q + 2 * i + 1) * kRows + prow] = make_float4(o[4], o[5], o[6], o[7]);
            }
          }
        }
        if (!whole && half == 0) reinterpret_cast<float2*>(part + (size_t)kRows * D)[prow] = make_float2(ref, l);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&ctl.o_free[x]);
        o_ph ^= 1u;
        if (whole) flush();
      }
      if (!whole) {
        const int ns = last_cta - first_cta + 1;
        sync_softmax();
        if (threadIdx.x == 0) {
          __threadfence();  // of all these warps' stores, which the barrier has put before it
          ctl.last = atomicAdd(p.cnt + first_cta, 1u) == (unsigned)(ns - 1);
          if (ctl.last) p.cnt[first_cta] = 0u;
          __threadfence();
        }
        sync_softmax();
        if (ctl.last && here) {
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
          for (int j = 0; j < D / 32; ++j) {  // this half's columns, 16 at a time
            const int q = half * (D / 32) + j;
            float o[2][8] = {};
#pragma unroll 2
            for (int i = 0; i < ns; ++i) {
              const float4* src = reinterpret_cast<const float4*>(slot(i)) + (4 * q) * kRows + prow;
              const float e = __ldcg(reinterpret_cast<const float2*>(slot(i) + (size_t)kRows * D) + prow).x;
              float4 a[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) a[k] = __ldcg(src + k * kRows);
              const float f = e == -INFINITY ? 0.f : ex2(e - top);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float* d = o[k / 2] + 4 * (k & 1);
                d[0] = fmaf(f, a[k].x, d[0]), d[1] = fmaf(f, a[k].y, d[1]);
                d[2] = fmaf(f, a[k].z, d[2]), d[3] = fmaf(f, a[k].w, d[3]);
              }
            }
            write(2 * q, o[0], sum);
            write(2 * q + 1, o[1], sum);
          }
          flush();
        }
        sync_softmax();
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------- codes -> operands
    // Three steps in flight: the page of block i + 2, the codes of block i + 1, block i into shared memory.
    const int tid = threadIdx.x - 32 * kExpandWarp;  // position within a block
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
      ahead.page = ahead.inside ? c.table[(size_t)g.s * c.max_pages + (pos >> c.log_page)] : -1;
      ahead.slot = pos & (c.page - 1);
      ahead.h = g.h;
      ++b;
    };
    // a block's keys, then its values; each operand's registers take the next block's codes as soon as they are free
    struct Block {
      bool valid, there, absent;
      const uint8_t* row;  // of the keys
    } cur, nxt;
    auto place = [&](Block* n) {
      n->valid = ahead.valid;
      if (!n->valid) return;
      n->there = (unsigned)ahead.page < (unsigned)c.num_pages;
      n->absent = ahead.inside && !n->there;
      if (n->absent) kv4::report_bad();
      n->row = n->there ? c.pages + kv4::block_offset(c, ahead.page, ahead.h) + (size_t)ahead.slot * (D / 2) : nullptr;
    };
    const size_t v_off = (size_t)c.page * (D / 2), p_off = (size_t)c.page * D;
    uint4 kw[D / 32], vw[D / 32];
    uint2 pair;
    int slot = 0;
    auto load = [&](uint4 (&w)[D / 32], const Block& n, size_t off) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        w[i] = n.valid && n.there ? reinterpret_cast<const uint4*>(n.row + off)[i] : make_uint4(0, 0, 0, 0);
    };
    auto load_pair = [&](const Block& n) {  // the scale pairs stand behind the values, 8 bytes a token
      pair = make_uint2(0, 0);
      if (n.valid && n.there)
        pair = *reinterpret_cast<const uint2*>(n.row - (size_t)slot * (D / 2) + p_off + (size_t)slot * 8);
    };
    look_up();
    place(&cur);
    slot = ahead.slot;
    load(kw, cur, 0);
    load(vw, cur, v_off);
    load_pair(cur);
    if (cur.valid) look_up();
    for (int block = 0; cur.valid; ++block) {
      const int stage = block & 1;
      const uint2 sp = pair;
      const float2 vp = __half22float2(as_half2(sp.y));
      const bool bad_value = !(fabsf(fmaf(15.f, vp.x, vp.y)) < 65520.f);  // beyond fp16, or not a number
      const uint32_t ab = __ballot_sync(0xffffffffu, cur.absent), po = __ballot_sync(0xffffffffu, bad_value);
      place(&nxt);
      slot = ahead.slot;
      if (block >= 2) wait(&ctl.k_empty[stage], (uint32_t)(block / 2 - 1) & 1u);
      if (lane == 0) {
        ctl.absent[block & 3][tid >> 5] = ab;
        ctl.poison[block & 3][tid >> 5] = po;
      }
      expand<D>(ks + (uint32_t)(stage * kOperand), tid, kw, sp.x);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ctl.k_full[stage]);
      load(kw, nxt, 0);
      load_pair(nxt);
      if (nxt.valid) look_up();
      if (block >= 2) wait(&ctl.v_empty[stage], (uint32_t)(block / 2 - 1) & 1u);
      expand<D>(vs + (uint32_t)(stage * kOperand), tid, vw, bad_value ? 0u : sp.y);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&ctl.v_full[stage]);
      load(vw, nxt, v_off);
      cur = nxt;
    }
  } else {
    // ------------------------------------------------------------------ MMA
    if (warp == kMmaWarp) {
      // the whole warp in step, one lane of it issuing
      constexpr uint32_t id_s = tc::idesc_f16_f32(kBlock, false), id_o = tc::idesc_f16_f32(D, true);
      const uint32_t lead = lane == 0 ? 1u : 0u;
      bool ok = true;
      auto wait_all = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, tc::tc_wait_late<false>(bar, parity, misc)) && ok;
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
          tc::mma_f16_ts(tmem + 256u + (uint32_t)(128 * x), tmem + (uint32_t)(128 * x + 64 * (i / 4) + 8 * (i % 4)),
                         v + (uint32_t)(i * 128),
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
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

template <int D>
int launch_dim(const Kv4PromptParams& p, int ctas, cudaStream_t s) {
  constexpr int bytes = 1024 + kCtlBytes + 6 * (D / 64) * kSub;
  const int rc = allow_smem(reinterpret_cast<const void*>(prompt_kernel<D>), bytes);
  if (rc != 0) return rc;
  return launch_dependent(prompt_kernel<D>, ctas, kThreads, bytes, 1, s, p);
}

}  // namespace

size_t kv4_prompt_part_bytes(int dim, int ctas) { return (size_t)ctas * 2 * kRows * (size_t)(dim + 2) * 4; }

int launch_kv4_prompt(const Kv4PromptParams& p, int ctas, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return p.c.dim == 128 ? launch_dim<128>(p, ctas, s) : launch_dim<64>(p, ctas, s);
}

}  // namespace tern
