// Attention of a step's new tokens over the paged 4-bit cache, for few query
// rows per sequence and kv head: single tokens, or a few at a time.
//
// Mathematics. A key of the cache is k = m + s c with codes c in 0..15 and one
// (s, m) per token and head, so q k = s (q c) + m sum(q): the tensor cores
// multiply q by the codes alone and the scales enter once per score. In the
// same way sum_j p_j v_j = sum_j w_j c_j + sum_j (p_j (m_j + 7.5 s_j) - 7.5 w_j)
// with w_j = p_j s_j, where the second sum is one number per query row. Softmax in
// base 2 with a running maximum; sums and statistics in fp32.
//
// Operands are fp16. A code needs no conversion: the four bits at the bottom of
// an fp16 are the subnormal c 2^-24, and at bits 4-7 c 2^-20, both exact
// operands, so one mask per two codes makes them (and a shift by 8 per four);
// the factors 2^24 and 2^20 are powers of two that go into q and into the
// output. q is bf16: its row is multiplied by a power of two that puts its
// largest element at 2^14..2^15, so that all its bits are kept for every
// element within 2^27 of the largest. The weights p_j s_j are rounded to fp16 (half a step, 2^-11
// relative; bf16 weights would add an error three times the output's own
// rounding), scaled by a power of two that follows the largest s seen so far, so
// that the largest is near 2^14 and small ones keep their bits. Both sums take the
// rounded w_j, so that a rounding weighs c_j - 7.5, not c_j: against fp64, before the
// output's rounding, 2e-4 of the output's size at 64 to 65536 positions, where the
// plain sum of p_j m_j left 4e-4 to 1.3e-3 (the offset's part grows with the length).
//
// Layout. The scores are computed transposed, tokens x query rows
// (m16n8k16): sixteen tokens of codes fill the A operand and eight query rows
// the B operand, so one sequence's group of up to eight heads costs no padding
// in the large dimension. The contraction may run over the dimensions in any
// order, so lane 4 r + t takes D/4 consecutive dimensions of a token, 16 bytes
// at D = 128, and q is loaded in the same order. The second product is
// transposed too, dimensions x rows: its A operand pairs the same dimension of
// two tokens by byte permutation, and its B operand is the probability matrix
// transposed in registers by movmatrix. Row x of a score block stands for token
// x ^ (x >> 1 & 1): four lanes then read two even and two odd tokens together
// in the second product, whose shared-memory reads meet in two instead of four
// ways, and the first product's reads stay free of conflicts.
//
// Memory. A page's block of one head is contiguous, so a round of 256 positions
// arrives in 256 / page_size bulk copies, into a ring of three stages of a round
// each; two CTAs per multiprocessor keep 139 KB in flight. The warp that requests a
// round changes with every round. Neither memory nor a pipe is full (64 sequences up
// to 8192: DRAM 42 %, issue 55 %, integer pipe 49 % with about 90 masks, shifts and byte
// permutations per lane and 16 tokens): sixteen warps per multiprocessor do not hide
// the latencies of a step, which is one chain from scores to weights to values. Rounds
// that every row sees as a whole take a path without masks.
//
// Split. The work is one line of rounds, 256 positions of a (sequence, kv head,
// tile of query rows), laid end to end over the whole batch; CTA c of G takes
// the rounds [W c / G, W (c + 1) / G), so every CTA reads the same number of
// positions whatever the lengths are, in one resident wave. Inside a CTA the
// eight warps take 32 positions in turn with softmax states of their own, joined
// in shared memory. A tile that CTA boundaries cut is joined by the last of its
// CTAs to arrive, in position order, so results do not depend on timing. A CTA
// holds at most one tile that it begins and does not end and one that it ends
// or passes through, so two slots of the workspace per CTA are enough.
//
// Measured (D = 128, heads : kv heads = 4; device times of replayed graphs, a call through
// the binding takes up to 1 us more): one token of 64 sequences of up to 8192 positions 58
// us, 3.7 TB/s (0.58 of the measured copy rate); of one sequence of 131072 40 us, 3.6
// TB/s; of one of 1024 8.5 us, mostly the fixed part: launch, search, the latency of page
// table and pages, join. Sixteen rows (64 x 4000 positions, 4 tokens of 4 heads): 38 us, 1.8
// TB/s, with 242 registers and one CTA of eight warps per multiprocessor.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "tern_kv4.cuh"
#include "tern_launch.cuh"
#include "tern_tc.cuh"

namespace tern {

int read_clear_dev_error_kv4_attn(void* stream, unsigned* out) { return read_clear_dev_error_tu(stream, out); }

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 32;   // positions a warp takes at a time
constexpr int kStages = 3;  // rounds in the ring
constexpr int kRound = kStep * kWarps;  // positions of a CTA's round
constexpr int kMaxCtas = 512;           // of a launch

using kv4::ex2;
using kv4::exp2i;

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}
__device__ __forceinline__ uint32_t lo16(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi16(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
__device__ __forceinline__ uint32_t even4(uint32_t w) { return w & 0x000F000Fu; }  // codes at bits 0-3: c 2^-24
__device__ __forceinline__ uint32_t odd4(uint32_t w) { return w & 0x00F000F0u; }   // codes at bits 4-7: c 2^-20
__device__ __forceinline__ float2 half2_at(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int WORDS>
__device__ __forceinline__ void lds_words(uint32_t (&v)[WORDS], uint32_t a) {
  if constexpr (WORDS == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(a));
  else if constexpr (WORDS == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
  else
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a));
}

template <int D, int NT>
struct Shared {
  static constexpr int kRows = 8 * NT, kPitch = D + 4;
  union {
    uint8_t ring[kStages][kRound * (D + 8)];
    struct {
      float m[kWarps][kRows], l[kWarps][kRows];
      float o[kWarps][kRows][kPitch];
    };
    struct {
      float sum[kRows];                    // of a join: the rows' sums,
      float2 ml[kMaxCtas][kRows];          // maxima and sums of the parts, then (factor, -)
    };
  };
  uint64_t full[kStages], empty[kStages];
  uint32_t there[kStages];                 // pages of a stage that are in the cache, one bit each
  uint32_t phase[kStages];                 // of a stage's last request; 2: none yet
  uint32_t abort;                          // a bounded wait has given up
  kv4::ShareScratch<kWarps> share;
  int last;
};

// Rounds of a sequence: kv heads x row tiles x rounds of its positions.
__device__ __forceinline__ long long rounds_of(const Kv4AttnParams& p, const kv4::Seq& q, int R, int* tiles,
                                               int* rounds) {
  *tiles = (q.n * p.group + R - 1) / R;
  *rounds = max(1, (q.len + kRound - 1) / kRound);
  return q.ok && q.n * p.group <= p.max_rows ? (long long)p.c.kv_heads * *tiles * *rounds : 0;
}

// The exchanges hold a row's dimensions in the order that the accumulators have
// them, two at a time: place 16 i + 2 r + e is dimension r D/8 + 2 i + e (lanes then
// write without bank conflicts). store_row puts four places back.
template <int D>
__device__ __forceinline__ void store_row(const Kv4AttnParams& p, const kv4::Seq& q, int h, int row, int place,
                                          const float (&o)[4], float l) {
  const float inv = l > 0.f ? 1.0f / l : (l == 0.f ? 0.f : l);  // no position: zero; NaN stays
  const int tok = row / p.group, i = place >> 4, r = (place & 15) >> 1;
  uint16_t* out = p.out + ((size_t)(q.row0 + tok) * p.c.heads + (size_t)h * p.group + (row - tok * p.group)) * D;
  *reinterpret_cast<__nv_bfloat162*>(out + r * (D / 8) + 2 * i) = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
  *reinterpret_cast<__nv_bfloat162*>(out + (r + 1) * (D / 8) + 2 * i) = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
}

// A warp's softmax state and queries: NT tiles of eight rows; the lane holds
// rows 2t, 2t + 1 of each and, of the output, dimensions r D/8 .. + D/8 - 1.
template <int D, int NT>
struct State {
  uint32_t qf[NT][D / 16][2];
  float sumq[NT][2], rowf[NT][2];
  int lim[NT][2];  // positions that a row sees
  float o[NT][D / 16][4], m[NT][2], l[NT][2], corr[NT][2];
  int ve;          // exponent field of the largest value scale so far; weights carry 2^(28 - ve)
};

// 32 positions from pos0 on. kb, pb: shared addresses of the keys' codes and
// of the scale pairs of each group of 16, already moved to the lane's place;
// the values' codes at vb. FULL: every row sees all of them; otherwise
// positions from stop[g] on are masked.
template <int D, int NT, bool FULL>
__device__ __forceinline__ void step(State<D, NT>& S, int pos0, const uint32_t (&kb)[2], const uint32_t (&vb)[2],
                                     const uint32_t (&pb)[2], const int (&stop)[2], int tr, int tx) {
  constexpr int KW = D / 32, VW = D / 64, MT = D / 16;
  float sc[2][NT][4];
  float2 vs[2][2];
  unsigned vbig = 0;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int pos = pos0 + 16 * g;
    uint32_t ka[KW], kc[KW], pa[2], pc[2];
    lds_words<KW>(ka, kb[g]);
    lds_words<KW>(kc, kb[g] + 8 * (D / 2));
    lds_words<2>(pa, pb[g]);
    lds_words<2>(pc, pb[g] + 64);
    vs[g][0] = half2_at(pa[1]);
    vs[g][1] = half2_at(pc[1]);
    if (FULL || pos + tr < stop[g]) vbig = max(vbig, pa[1] & 0xFFFFu);
    if (FULL || pos + tr + 8 < stop[g]) vbig = max(vbig, pc[1] & 0xFFFFu);
#pragma unroll
    for (int j = 0; j < NT; ++j) sc[g][j][0] = sc[g][j][1] = sc[g][j][2] = sc[g][j][3] = 0.f;
#pragma unroll
    for (int w = 0; w < KW; ++w) {
      const uint32_t a8 = ka[w] >> 8, c8 = kc[w] >> 8;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_f16(sc[g][j], even4(ka[w]), even4(kc[w]), odd4(ka[w]), odd4(kc[w]), S.qf[j][2 * w][0], S.qf[j][2 * w][1]);
        mma_f16(sc[g][j], even4(a8), even4(c8), odd4(a8), odd4(c8), S.qf[j][2 * w + 1][0], S.qf[j][2 * w + 1][1]);
      }
    }
    const float2 k0 = half2_at(pa[0]), k1 = half2_at(pc[0]);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float x = fmaf(k0.x * sc[g][j][e], S.rowf[j][e], k0.y * S.sumq[j][e]);
        const float y = fmaf(k1.x * sc[g][j][2 + e], S.rowf[j][e], k1.y * S.sumq[j][e]);
        const int seen = FULL ? 0 : min(stop[g], S.lim[j][e]);
        sc[g][j][e] = FULL || pos + tr < seen ? x : -INFINITY;
        sc[g][j][2 + e] = FULL || pos + tr + 8 < seen ? y : -INFINITY;
      }
    }
  }
  // running maxima; the accumulators are scaled only when one has grown
  const int ve2 = max(S.ve, (int)(__reduce_max_sync(0xffffffffu, vbig) >> 10));
  float ref[NT][2];
  bool grown = ve2 > S.ve;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = fmaxf(fmaxf(sc[0][j][e], sc[0][j][2 + e]), fmaxf(sc[1][j][e], sc[1][j][2 + e]));
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, k));
      grown |= x > S.m[j][e];
      ref[j][e] = fmaxf(x, S.m[j][e]);
    }
  }
  if (__any_sync(0xffffffffu, grown)) {
    const float fv = exp2i(S.ve - ve2);
    S.ve = ve2;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[e] = S.m[j][e] == -INFINITY ? 0.f : ex2(S.m[j][e] - ref[j][e]);
        S.m[j][e] = ref[j][e];
        S.l[j][e] *= f[e];
        S.corr[j][e] *= f[e];
        f[e] *= fv;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        S.o[j][i][0] *= f[0];
        S.o[j][i][1] *= f[1];
        S.o[j][i][2] *= f[0];
        S.o[j][i][3] *= f[1];
      }
    }
  }
  const float vf = exp2i(28 - S.ve), middle = -7.5f * exp2i(S.ve - 28);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    uint32_t pw[NT][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float vsc = vs[g][k].x * vf, mid = fmaf(7.5f, vs[g][k].x, vs[g][k].y);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = sc[g][j][2 * k + e];
          const bool in = FULL || x != -INFINITY;  // a masked place takes no part, whatever its scales hold
          const float pr = in ? ex2(x - S.m[j][e]) : 0.f;
          S.l[j][e] += pr;
          w[e] = in ? pr * vsc : 0.f;
          if (in) S.corr[j][e] = fmaf(pr, mid, S.corr[j][e]);
        }
        const uint32_t rounded = pack_half2(w[0], w[1]);
        const float2 wr = half2_at(rounded);
        S.corr[j][0] = fmaf(wr.x, middle, S.corr[j][0]);
        S.corr[j][1] = fmaf(wr.y, middle, S.corr[j][1]);
        pw[j][k] = transpose8x8(rounded);
      }
    }
    // the lane's tokens of the second product: rows 2t and 2t + 1, and eight on
    uint32_t va[VW], vc[VW], vd[VW], ve[VW];
    const uint32_t first = vb[g] + (tx ? D / 2 : 0), second = vb[g] + (tx ? 0 : D / 2);
    lds_words<VW>(va, first);
    lds_words<VW>(vc, second);
    lds_words<VW>(vd, first + 8 * (D / 2));
    lds_words<VW>(ve, second + 8 * (D / 2));
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t a[2] = {lo16(va[w], vc[w]), hi16(va[w], vc[w])};
      const uint32_t b[2] = {lo16(vd[w], ve[w]), hi16(vd[w], ve[w])};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t a8 = a[i] >> 8, b8 = b[i] >> 8;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_f16(S.o[j][4 * w + 2 * i], even4(a[i]), odd4(a[i]), even4(b[i]), odd4(b[i]), pw[j][0], pw[j][1]);
          mma_f16(S.o[j][4 * w + 2 * i + 1], even4(a8), odd4(a8), even4(b8), odd4(b8), pw[j][0], pw[j][1]);
        }
      }
    }
  }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 2 : 1) attn_kernel(const Kv4AttnParams p) {
  constexpr int R = 8 * NT;          // query rows of the tile
  constexpr int KW = D / 32;         // words of K codes per lane and token
  constexpr int MT = D / 16;         // 16-dimension tiles of the output
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Shared<D, NT>& sm = *reinterpret_cast<Shared<D, NT>*>(smem_raw);
  const Kv4Params& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
  const int G = p.group;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kWarps);
      sm.phase[i] = 2;
    }
    sm.abort = 0;
    fence_mbar_init();
  }
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  volatile uint32_t* abort = &sm.abort;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!*abort && !mbar_wait_bounded(bar, parity)) *abort = 1;
  };
  // Whether a wait of the CTA has given up, the same to all lanes of a warp: what follows takes whole warps.
  auto gave_up = [&] { return __any_sync(0xffffffffu, *abort != 0u) != 0; };

  // where the warp's two groups of 16 tokens stand in a stage: their page's
  // block, then keys, values and scale pairs at the lane's token and dimensions
  const int tr = r ^ ((r >> 1) & 1), tx = t & 1;
  const uint32_t block_bytes = (uint32_t)c.page * (D + 8);
  uint32_t okb[2], ovb[2], opb[2];
  int page_bit[2];
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int tau = kStep * warp + 16 * g, slot = tau & (c.page - 1);
    page_bit[g] = tau >> c.log_page;
    const uint32_t blk = smem_u32(sm.ring) + (uint32_t)page_bit[g] * block_bytes;
    okb[g] = blk + (uint32_t)(slot + tr) * (D / 2) + t * (D / 8);
    ovb[g] = blk + (uint32_t)(c.page + slot + 2 * t) * (D / 2) + r * (D / 16);
    opb[g] = blk + (uint32_t)c.page * D + (uint32_t)(slot + tr) * 8;
  }

  kv4::Share sh;
  auto weight = [&](int i, bool report) -> long long {
    const kv4::Seq q = kv4::load_seq(c, i);
    if (!q.ok && report) kv4::report_bad();
    int tiles, rounds;
    return rounds_of(p, q, R, &tiles, &rounds);
  };
  if (!kv4::find_share<kWarps>(c.seqs, 1, weight, sm.share, &sh)) return;
  int s = sh.s;
  long long at = sh.at, in_seq = sh.in_seq;
  const long long stop_at = sh.stop;

  const uint64_t policy = policy_evict_first();
  int use = 0;  // rounds this CTA has taken
  for (; at < stop_at && s < c.seqs; ++s, in_seq = 0) {  // sequences
    const kv4::Seq q = kv4::load_seq(c, s);
    int tiles, rounds;
    const long long seq_rounds = rounds_of(p, q, R, &tiles, &rounds);
    const int rows = q.n * G;
    while (in_seq < seq_rounds && at < stop_at) {  // the (kv head, tile) ranges of one sequence
      const int unit = (int)(in_seq / rounds), round0 = (int)(in_seq - (long long)unit * rounds);
      const int take = (int)min((long long)(rounds - round0), stop_at - at);
      const long long unit_first = at - round0;  // the unit's first round among all
      at += take;
      in_seq += take;
      const int h = unit / tiles, tile = unit - h * tiles, row_first = tile * R;
      const int row_last = min(rows, row_first + R) - 1;
      const int limit_max = q.len - q.n + row_last / G + 1;  // positions that the tile's last token sees
      const int begin = round0 * kRound, end = (int)min((long long)limit_max, (long long)(round0 + take) * kRound);

      // Rounds of this range arrive in the ring in turn; round number `use` counts
      // over the CTA's whole life. The pages of a round are looked up by one warp,
      // a lane a page, and requested when the stage's last round has been read.
      const int n_rounds = end > begin ? (end - begin + kRound - 1) / kRound : 0;
      auto look_up = [&](int i) {  // page of this lane in the range's round i; -1: not there, -2: beyond the end
        const int pos = begin + i * kRound + (lane << c.log_page);
        if ((lane << c.log_page) >= kRound || pos >= end) return -2;
        const int page = kv4::page_of(c, s, pos);
        if (page < 0) kv4::report_bad();
        return page;
      };
      auto request = [&](int page, int n) {  // the CTA's round number n
        const int stage = n % kStages;
        if (n >= kStages) wait(&sm.empty[stage], (uint32_t)(n / kStages - 1) & 1u);
        const uint32_t there = __ballot_sync(0xffffffffu, page >= 0);
        if (gave_up()) return;
        if (lane == 0) {
          sm.there[stage] = there;
          sm.phase[stage] = (uint32_t)(n / kStages) & 1u;
          mbar_arrive_expect_tx(&sm.full[stage], (uint32_t)__popc(there) * block_bytes);
        }
        __syncwarp();
        if (page >= 0)
          bulk_g2s(sm.ring[stage] + (uint32_t)lane * block_bytes, c.pages + kv4::block_offset(c, page, h), block_bytes,
                   &sm.full[stage], policy);
      };
#pragma unroll
      for (int i = 0; i < kStages - 1; ++i)
        if (warp == i && i < n_rounds) request(look_up(i), use + i);

      // q in the order of the key words, times a power of two per row; sums of its rows
      State<D, NT> S;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int row = row_first + 8 * j + r, tok = row / G;
        uint4 u[KW];
        float sum = 0.f, big = 0.f;  // the sum of the scaled row, which stays in range whatever its size
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          u[w] = make_uint4(0, 0, 0, 0);
          if (row < rows)
            u[w] = reinterpret_cast<const uint4*>(
                p.q + ((size_t)(q.row0 + tok) * c.heads + (size_t)h * G + (row - tok * G)) * D + t * (D / 4))[w];
          const uint32_t e[4] = {u[w].x, u[w].y, u[w].z, u[w].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float x = __uint_as_float(e[i] << 16), y = __uint_as_float(e[i] & 0xFFFF0000u);
            big = fmaxf(big, fmaxf(fabsf(x), fabsf(y)));
          }
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int ex = max(-100, (__float_as_int(big) >> 23) - 127);  // exponent of the largest element
        const float fe = exp2i(14 - ex), fo = fe * 0.0625f;
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          // dimensions i and i + 4 of a word's eight together, as the masks leave them
          const uint32_t e[4] = {u[w].x, u[w].y, u[w].z, u[w].w};
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(e[i] << 16);
            v[2 * i + 1] = __uint_as_float(e[i] & 0xFFFF0000u);
            sum += v[2 * i] * fe + v[2 * i + 1] * fe;
          }
          S.qf[j][2 * w][0] = pack_half2(v[0] * fe, v[4] * fe);
          S.qf[j][2 * w][1] = pack_half2(v[1] * fo, v[5] * fo);
          S.qf[j][2 * w + 1][0] = pack_half2(v[2] * fe, v[6] * fe);
          S.qf[j][2 * w + 1][1] = pack_half2(v[3] * fo, v[7] * fo);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        // the row's exponent meets the scale first: a large row has a small scale, and neither product leaves fp32
        const float unit = exp2i(ex) * p.scale_log2, back = unit * 1024.f;  // 2^(ex - 14 + 24) scale
        sum *= unit * 0x1p-14f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          S.sumq[j][e] = __shfl_sync(0xffffffffu, sum, (2 * t + e) * 4);
          S.rowf[j][e] = __shfl_sync(0xffffffffu, back, (2 * t + e) * 4);
          const int rw = row_first + 8 * j + 2 * t + e;
          S.lim[j][e] = rw < rows ? min(end, q.len - q.n + rw / G + 1) : 0;
        }
      }

#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int i = 0; i < MT; ++i) S.o[j][i][0] = S.o[j][i][1] = S.o[j][i][2] = S.o[j][i][3] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) S.m[j][e] = -INFINITY, S.l[j][e] = 0.f, S.corr[j][e] = 0.f;
      }
      const int lim_all = min(end, q.len - q.n + row_first / G + 1);  // positions that every row of the tile sees
      S.ve = 1;

      for (int i = 0; i < n_rounds; ++i, ++use) {
        const int stage = use % kStages;
        const bool duty = i + kStages - 1 < n_rounds && (use + kStages - 1) % kWarps == warp;
        int page = -2;
        if (duty) page = look_up(i + kStages - 1);
        wait(&sm.full[stage], (uint32_t)(use / kStages) & 1u);
        const int pos0 = begin + i * kRound + kStep * warp;
        if (!gave_up() && pos0 < end) {
          const uint32_t at_stage = (uint32_t)stage * (uint32_t)sizeof(sm.ring[0]), there = sm.there[stage];
          const uint32_t kb[2] = {okb[0] + at_stage, okb[1] + at_stage}, vb[2] = {ovb[0] + at_stage, ovb[1] + at_stage},
                         pb[2] = {opb[0] + at_stage, opb[1] + at_stage};
          const bool g0 = (there >> page_bit[0]) & 1u, g1 = (there >> page_bit[1]) & 1u;
          const int stop[2] = {g0 ? end : 0, g1 ? end : 0};
          if (g0 && g1 && pos0 + kStep <= lim_all)
            step<D, NT, true>(S, pos0, kb, vb, pb, stop, tr, tx);
          else
            step<D, NT, false>(S, pos0, kb, vb, pb, stop, tr, tx);
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.empty[stage]);
        if (duty) request(page, use + kStages - 1);
      }
      __syncthreads();  // the ring becomes the exchange of the states

      // the warps' states: codes were c 2^-24 and c 2^-20, weights carried 2^(28 - ve)
      const float back_even = exp2i(24 - 28 + S.ve), back_odd = exp2i(20 - 28 + S.ve);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) {
            S.l[j][e] += __shfl_xor_sync(0xffffffffu, S.l[j][e], k);
            S.corr[j][e] += __shfl_xor_sync(0xffffffffu, S.corr[j][e], k);
          }
          const int n = 8 * j + 2 * t + e;
          if (r == 0) sm.m[warp][n] = S.m[j][e], sm.l[warp][n] = S.l[j][e];
#pragma unroll
          for (int i = 0; i < MT; ++i)
            *reinterpret_cast<float2*>(&sm.o[warp][n][16 * i + 2 * r]) =
                make_float2(fmaf(S.o[j][i][e], back_even, S.corr[j][e]),
                            fmaf(S.o[j][i][2 + e], back_odd, S.corr[j][e]));
        }
      }
      __syncthreads();
      // the tile's CTAs: the first holds its first round, the last its last
      const int first_cta = sh.cta_of(unit_first), last_cta = sh.cta_of(unit_first + rounds - 1);
      const bool whole = first_cta == last_cta;
      constexpr int kSlot = R * (D + 2);  // floats: weighted values [R][D], then (maximum, sum) [R]
      float* part = p.part + (size_t)(2 * blockIdx.x + (round0 == 0 ? 1 : 0)) * kSlot;
      for (int item = threadIdx.x; item < R * (D / 4); item += kThreads) {
        const int n = item / (D / 4), d = (item - n * (D / 4)) * 4;
        if (row_first + n >= rows) continue;
        float mx = -INFINITY, sum = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][n]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = sm.m[w][n] == -INFINITY ? 0.f : ex2(sm.m[w][n] - mx);
          const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][n][d]);
          sum = fmaf(f, sm.l[w][n], sum);
          v[0] = fmaf(f, x.x, v[0]);
          v[1] = fmaf(f, x.y, v[1]);
          v[2] = fmaf(f, x.z, v[2]);
          v[3] = fmaf(f, x.w, v[3]);
        }
        if (whole) {
          store_row<D>(p, q, h, row_first + n, d, v, sum);
        } else {
          *reinterpret_cast<float4*>(part + n * D + d) = make_float4(v[0], v[1], v[2], v[3]);
          if (d == 0) *reinterpret_cast<float2*>(part + R * D + 2 * n) = make_float2(mx, sum);
        }
      }
      if (!whole) {
        // the last CTA of the tile to arrive joins its parts
        const int ns = last_cta - first_cta + 1;
        __syncthreads();
        if (threadIdx.x == 0) {
          __threadfence();  // of the whole CTA's stores, which the barrier has put before it
          sm.last = atomicAdd(p.cnt + first_cta, 1u) == (unsigned)(ns - 1);
          if (sm.last) p.cnt[first_cta] = 0u;
          __threadfence();
        }
        __syncthreads();
        if (sm.last) {
          const float* parts = p.part + (size_t)2 * first_cta * kSlot;
          auto slot = [&](int i) { return parts + (size_t)(i == 0 ? 1 : 2 * i) * kSlot; };
          for (int i = threadIdx.x; i < ns * R; i += kThreads)
            sm.ml[i / R][i % R] = __ldcg(reinterpret_cast<const float2*>(slot(i / R) + R * D + 2 * (i % R)));
          __syncthreads();
          for (int n = warp; n < R; n += kWarps) {  // a warp per row: every part's factor, and the sum
            if (row_first + n >= rows) continue;    // unwritten
            float mx = -INFINITY, sum = 0.f;
            for (int i = lane; i < ns; i += 32) mx = fmaxf(mx, sm.ml[i][n].x);
#pragma unroll
            for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
            for (int i = lane; i < ns; i += 32) {
              const float2 e = sm.ml[i][n];
              const float f = e.x == -INFINITY ? 0.f : ex2(e.x - mx);
              sum = fmaf(f, e.y, sum);
              sm.ml[i][n].x = f;
            }
#pragma unroll
            for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
            if (lane == 0) sm.sum[n] = sum;
          }
          __syncthreads();
          // `fan` neighbouring threads share an item's parts where the tile has fewer rows than threads for them
          const int live = min(R, rows - row_first), items = live * (D / 4);
          int fan = 1;
          while (fan < 8 && 2 * fan * items <= kThreads) fan *= 2;
          for (int base = 0; base < items * fan; base += kThreads) {  // whole warps
            const int w = base + (int)threadIdx.x, item = w / fan, part0 = w % fan;
            const bool in = item < items;
            const int n = in ? item / (D / 4) : 0, d = in ? (item - n * (D / 4)) * 4 : 0;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 10
            for (int i = part0; i < ns; i += fan) {
              const float4 x = __ldcg(reinterpret_cast<const float4*>(slot(i) + n * D + d));
              const float f = sm.ml[i][n].x;
              v[0] = fmaf(f, x.x, v[0]);
              v[1] = fmaf(f, x.y, v[1]);
              v[2] = fmaf(f, x.z, v[2]);
              v[3] = fmaf(f, x.w, v[3]);
            }
            for (int k = 1; k < fan; k <<= 1) {
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], k);
            }
            if (in && part0 == 0) store_row<D>(p, q, h, row_first + n, d, v, sm.sum[n]);
          }
        }
      }
      fence_proxy_async_smem();
      __syncthreads();  // the exchange becomes the ring again
    }
  }
  if (*abort && threadIdx.x == 0)  // no copy of this CTA's may be under way when it ends
    for (int i = 0; i < kStages; ++i)
      if (sm.phase[i] < 2) mbar_wait_bounded(&sm.full[i], sm.phase[i]);
}

template <int D, int NT>
int launch_one(const Kv4AttnParams& p, int ctas, cudaStream_t s) {
  constexpr int bytes = (int)sizeof(Shared<D, NT>);
  const int rc = allow_smem(reinterpret_cast<const void*>(attn_kernel<D, NT>), bytes);
  if (rc != 0) return rc;
  return launch_dependent(attn_kernel<D, NT>, ctas, kThreads, bytes, 1, s, p);
}

// How a batch within these bounds runs. Sequences of up to 48 query rows per kv
// head take this file's kernel, 8 rows per CTA if no sequence has more, else 16
// (up to three tiles that read the codes anew, from L2); longer ones the prompt
// kernel, whose time does not depend on the rows up to 256. At D = 128 with two kv
// heads, this kernel with 16 / 32 / 48 rows and the prompt kernel: 64 sequences of
// 4000 positions 38 / 63 / 87 and 94 us, one of 30000 23 / 23 / 26 and 59 us, 8 of 1000
// 14 / 14 / 19 and 26 us; a fourth tile would lose.
// Workspace: the CTAs' counters of both kernels, then their parts, at places that
// only the device and the cache's shape decide, so that batches of any size share it.
struct Plan {
  int rows, ctas;           // few rows: rows per CTA, CTAs; 0 if the batch has none
  int prompt_ctas;          // 0 if no sequence may have more than kMaxRows rows
  long long min_share;
  size_t part_off, prompt_off, total;
};
constexpr int kMaxRows = 48;

tern_status plan_attn(const Kv4Params& c, int heads, int seqs, int max_new, int max_len, int sms, Plan* pl) {
  const long long rows = (long long)max_new * (heads / c.kv_heads);
  if (rows > (1 << 30) || max_len > (1 << 30)) return TERN_EUNSUPPORTED;
  const long long rounds = std::max(1, (max_len - 1) / kRound + 1), blocks = std::max(1, (max_len - 1) / 128 + 1);
  // the kernels count rounds times CTAs in 64 bits
  if ((double)seqs * c.kv_heads * (double)((rows + 7) / 8) * (double)blocks > 1e15) return TERN_EUNSUPPORTED;
  pl->rows = rows <= 8 ? 8 : 16;
  // one resident wave: two CTAs per multiprocessor with 8 rows, one with 16 (registers); no more than rounds
  const int wave = std::min(kMaxCtas, (pl->rows == 8 ? 2 : 1) * sms), prompt_wave = std::min(kMaxCtas, sms);
  pl->ctas = (int)std::min<double>(wave, std::max(1.0, (double)seqs * c.kv_heads * (kMaxRows / 16) * (double)rounds));
  pl->prompt_ctas = 0;
  if (rows > kMaxRows) {
    pl->prompt_ctas = prompt_wave;
    if (seqs == 1) pl->ctas = 0;  // the prompt kernel takes the one sequence whatever its length
  }
  // Blocks that a CTA of the prompt kernel takes at least: a unit's last CTA reads all its parts, so up to 8 parts
  // of fewer than four blocks and 16 of more. 64 tokens, 4 kv heads, of 64 / 4000 / 16000 / 60000 positions: 13 / 33 /
  // 63 / 112 us (never fewer than four blocks: 39 us at 64; up to 8 parts always: 175 us at 60000; up to 32: 62, 78 and
  // 107 us at the last three)
  pl->min_share = std::max({1ll, std::min(4ll, blocks / 8), blocks / 16});
  const size_t slot8 = (size_t)8 * (size_t)(c.dim + 2) * 4;
  pl->part_off = 2 * kMaxCtas * sizeof(unsigned);
  // 2 wave slots of 8 rows or wave slots of 16: the same size
  pl->prompt_off = pl->part_off + ((size_t)std::min(kMaxCtas, 2 * sms) * 2 * slot8 + 255) / 256 * 256;
  pl->total = pl->prompt_ctas ? pl->prompt_off + kv4_prompt_part_bytes(c.dim, prompt_wave)
                              : (rounds > 1 ? pl->prompt_off : 0);
  return TERN_OK;
}

}  // namespace

int launch_kv4_attn(const Kv4AttnParams& p, int rows, int ctas, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.c.dim == 128) return rows == 8 ? launch_one<128, 1>(p, ctas, s) : launch_one<128, 2>(p, ctas, s);
  return rows == 8 ? launch_one<64, 1>(p, ctas, s) : launch_one<64, 2>(p, ctas, s);
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
  Plan pl{};
  const tern_status sp = plan_attn(c, heads, seqs, max_new, max_len, sm_count(), &pl);
  if (sp != TERN_OK) return sp;
  *bytes = seqs > 0 && max_new > 0 ? pl.total : 0;
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
  Plan pl{};
  // no sequence has more new tokens than the buffers have rows, however generous the bound is
  st = plan_attn(p.c, heads, p.c.seqs, std::min(p.c.max_new, p.c.tokens), p.c.max_len, sm_count(), &pl);
  if (st != TERN_OK) return st;
  if (pl.total > 0) {
    if (!d_ws || ws_bytes < pl.total) return TERN_ENOSPACE;
    if ((reinterpret_cast<uintptr_t>(d_ws) & 255u) != 0) return TERN_EALIGN;
  }
  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  p.c.heads = heads;
  p.q = d_q;
  p.out = d_out;
  p.scale_log2 = scale * 1.44269504088896340736f;
  p.group = heads / p.c.kv_heads;
  p.max_rows = kMaxRows;
  p.cnt = reinterpret_cast<unsigned*>(ws);
  p.part = reinterpret_cast<float*>(ws + pl.part_off);
  if (pl.prompt_ctas) {
    Kv4PromptParams r{};
    r.c = p.c;
    r.q = p.q;
    r.out = p.out;
    r.scale_log2 = p.scale_log2;
    r.group = p.group;
    r.min_rows = pl.ctas ? kMaxRows + 1 : 1;
    r.min_share = pl.min_share;
    r.cnt = p.cnt + kMaxCtas;
    r.part = reinterpret_cast<float*>(ws + pl.prompt_off);
    if (launch_kv4_prompt(r, pl.prompt_ctas, stream) != 0) return TERN_ECUDA;
  }
  if (pl.ctas && launch_kv4_attn(p, pl.rows, pl.ctas, stream) != 0) return TERN_ECUDA;
  return TERN_OK;
}
