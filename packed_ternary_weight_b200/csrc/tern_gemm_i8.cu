// 8-bit product with a scale per token and output channel:
//   y[m][n] = fl(fl(fl(acc) w_scale[n]) x_scale[m]), acc = sum_k w[n][k] x[m][k] exactly,
// on the 5th-generation tensor cores (tcgen05 kind::i8, int32 accumulators in
// tensor memory).
//
// The weights are the A operand (128 channels per tile) and the tokens the B
// operand (N = 16..256 of them per tile, the count padded to 16), so that one
// kernel serves a single token, where it streams weights, and a prompt, where it
// is bound by the tensor cores; and so that a thread of the epilogue holds one
// channel and a warp writes 32 consecutive channels of a token.
//
// One persistent CTA per SM:
//   warp 0     tensor-map loads of A and B steps (128 bytes of K, 128-byte
//              swizzle) into a ring as deep as shared memory allows; K, rows and
//              tokens beyond the ends arrive as zeros;
//   warp 1     one thread issues the MMAs and commits them to mbarriers;
//   warps 4-7  read the accumulators (two buffers, so that the next tile's MMAs
//              run meanwhile), scale and store.
// Enough tiles for every pair of SMs: pairs of CTAs (cta_group::2) take 256
// channels by up to 256 tokens, each loading its own 128 channels and half of the
// tokens, which is 32 KB instead of 48 KB per SM and step (one CTA per tile was
// held up by these loads: tensor pipe 67 % active, 74 % with pairs). 4095 x 14336 x
// 4096 then takes 195-205 us in a replayed graph, 2.4 POP/s (213 us over seconds, at the
// power cap's 1.44 GHz); a token's 65536 x 2560 head 31 us, 5.5 TB/s (0.85 of the
// measured copy rate).
// Fewer tiles than SMs: the steps of a tile are dealt to a cluster of up to eight
// CTAs, whose exact int32 partial sums meet in distributed shared memory; each
// CTA of the cluster finishes a share of the tokens. Integer sums: the result
// does not depend on the split.
// Every wait is bounded; on expiry the device error word records a timeout and
// the CTA runs to its end without waiting further.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "tern_launch.cuh"
#include "tern_tc.cuh"

namespace tern {

int read_clear_dev_error_gemm_i8(void* stream, unsigned* out) { return read_clear_dev_error_tu(stream, out); }

namespace {

constexpr int kThreads = 256;
constexpr int kRowsA = 128;               // channels per tile
constexpr int kStepK = 128;               // bytes of K per step
constexpr int kBytesA = kRowsA * kStepK;  // 16 KB
constexpr int kMaxStages = 12;
constexpr int kMaxSplit = 8;
constexpr int kMinSteps = 4;              // of K for each CTA of a split tile
constexpr int kTileCost = 64, kPairCost = 32;  // of a tile beyond its tokens, in tokens
constexpr int kSmemTop = 227 * 1024;

struct Plan {
  int tn, tiles_n, tiles_m, tiles;  // tokens per tile; tiles of channels, of tokens
  int steps, split;                 // of K; CTAs that share a tile
  int pair;                         // pairs of CTAs, 256 channels per tile
  int stages, stage_bytes, grid;
  uint32_t tmem_cols;
};

struct Args {
  GemmI8Params p;
  Plan pl;
};

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], fin;
  uint32_t misc[4];  // tensor-memory base, abort flag
  float sx[2][256];
};
constexpr int kCtlBytes = 3 * 1024;
static_assert(sizeof(Ctl) <= kCtlBytes, "control block");

__device__ __forceinline__ void named_sync_epilogue() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ int4 ld_dsmem(uint32_t addr) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void store_one(const GemmI8Params& p, int m, int n, int acc, float sw, float sx) {
  const float v = __fmul_rn(__fmul_rn(__int2float_rn(acc), sw), sx);
  const int64_t at = (int64_t)m * p.ldy + n;
  if (p.out_bf16)
    static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p.y)[at] = v;
}

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_i8_kernel(const Args a, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const GemmI8Params& p = a.p;
  const Plan& pl = a.pl;
  // the dynamic block need not start on a swizzle atom
  const uint32_t base = smem_u32(smem), pad = (1024u - (base & 1023u)) & 1023u;
  Ctl& ctl = *reinterpret_cast<Ctl*>(smem + pad);
  const uint32_t ring = base + pad + kCtlBytes;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  volatile uint32_t* misc = ctl.misc;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.acc_full[i], 1);
      mbar_init(&ctl.acc_empty[i], PAIR ? 8 : 4);
    }
    mbar_init(&ctl.fin, 1);
    ctl.misc[tc::kMiscAbort] = 0;
    fence_mbar_init();
  }
  if (warp == 2 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(&map_x) : "memory");
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tc::tmem_alloc_pair(smem_u32(&ctl.misc[tc::kMiscTmem]), pl.tmem_cols);
    } else {
      tc::tmem_alloc(smem_u32(&ctl.misc[tc::kMiscTmem]), pl.tmem_cols);
      tc::tmem_relinquish();
    }
  }
  tc::fence_before_sync();
  pdl_launch_dependents();
  pdl_wait();
  __syncthreads();
  if constexpr (PAIR) {  // both CTAs' barriers exist before either signals the other's
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    cluster_wait_acquire();
  }
  tc::fence_after_sync();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.misc[tc::kMiscTmem], 0);
  // a tile's CTAs are a cluster of consecutive ones: a pair, or pl.split that share K
  const int ctas = PAIR ? 2 : pl.split, rank = (int)(blockIdx.x % ctas);
  const int first = (int)blockIdx.x / ctas, stride = (int)gridDim.x / ctas;
  const int k0 = PAIR ? 0 : pl.steps * rank / pl.split;  // at least one step each
  const int k1 = PAIR ? pl.steps : pl.steps * (rank + 1) / pl.split;
  constexpr int kRowsTile = PAIR ? 2 * kRowsA : kRowsA;
  const int n_off = PAIR ? rank * kRowsA : 0;             // this CTA's channels of a tile
  const int b_rows = PAIR ? pl.tn / 2 : pl.tn;            // tokens that it loads

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t ph = 0;
      for (int tile = first; tile < pl.tiles && !misc[tc::kMiscAbort]; tile += stride) {
        const int n0 = (tile % pl.tiles_n) * kRowsTile + n_off;
        const int m0 = (tile / pl.tiles_n) * pl.tn + (PAIR ? rank * b_rows : 0);
        for (int k = k0; k < k1; ++k) {
          if (issued >= pl.stages && !tc::tc_wait(&ctl.empty[stage], ph ^ 1u, misc)) break;
          const uint32_t st = ring + (uint32_t)(stage * pl.stage_bytes);
          if constexpr (PAIR) {  // both CTAs' loads complete on the even one's barrier
            const uint32_t bar = map_cluster_rank(smem_u32(&ctl.full[stage]), 0);
            if (rank == 0) mbar_arrive_expect_tx(&ctl.full[stage], 2u * (uint32_t)pl.stage_bytes);
            tc::tma_load_2d_pair(st, &map_w, k * kStepK, n0, bar);
            tc::tma_load_2d_pair(st + kBytesA, &map_x, k * kStepK, m0, bar);
          } else {
            mbar_arrive_expect_tx(&ctl.full[stage], (uint32_t)pl.stage_bytes);
            tc::tma_load_2d(st, &map_w, k * kStepK, n0, &ctl.full[stage]);
            tc::tma_load_2d(st + kBytesA, &map_x, k * kStepK, m0, &ctl.full[stage]);
          }
          ++issued;
          if (++stage == pl.stages) {
            stage = 0;
            ph ^= 1u;
          }
        }
      }
      // When the CTA ends, no load may be under way (the odd CTA of a pair waits for the even one below), and in the odd
      // CTA no signal of the even one's MMAs, which may come after its last thread has nothing left to do.
      const bool gave_up = misc[tc::kMiscAbort], odd = PAIR && rank == 1;
      for (int i = 0; gave_up != odd && i < min(issued, pl.stages); ++i) {
        if (--stage < 0) {
          stage = pl.stages - 1;
          ph ^= 1u;
        }
        if (!mbar_wait_bounded(odd ? &ctl.empty[stage] : &ctl.full[stage], ph) && odd) break;
      }
    }
  } else if (warp == 1 && (!PAIR || rank == 0)) {
    // the whole warp in step, one lane of it issuing
    const uint32_t idesc = PAIR ? tc::idesc_i8_s32_pair(pl.tn) : tc::idesc_i8_s32(pl.tn), lead = lane == 0 ? 1u : 0u;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, tc::tc_wait(bar, parity, misc)); };
    int stage = 0, seg = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int tile = first; tile < pl.tiles && ok; tile += stride, ++seg) {
      const int buf = seg & 1;
      if (seg >= 2)
        ok = PAIR ? __all_sync(0xffffffffu, tc::tc_wait_cluster(&ctl.acc_empty[buf], (uint32_t)(seg / 2 - 1) & 1u, misc))
                  : wait(&ctl.acc_empty[buf], (uint32_t)(seg / 2 - 1) & 1u);
      tc::fence_after_sync();
      const uint32_t acc = tmem + (uint32_t)(buf * pl.tn);
      for (int k = k0; k < k1 && ok; ++k) {
        ok = wait(&ctl.full[stage], ph);
        tc::fence_after_sync();
        const uint32_t st = ring + (uint32_t)(stage * pl.stage_bytes);
        const uint64_t ad = tc::smem_desc_sw128(st), bd = tc::smem_desc_sw128(st + kBytesA);
#pragma unroll
        for (int i = 0; i < kStepK / 32; ++i)  // 32 bytes of K: two 16-byte units of the start address
          if constexpr (PAIR)
            tc::mma_i8_pair(acc, ad + 2 * i, bd + 2 * i, idesc, k > k0 || i > 0 ? 1u : 0u, ok ? lead : 0u);
          else
            tc::mma_i8_lead(acc, ad + 2 * i, bd + 2 * i, idesc, k > k0 || i > 0 ? 1u : 0u, ok ? lead : 0u);
        PAIR ? tc::commit_pair(&ctl.empty[stage], lead) : tc::commit_lead(&ctl.empty[stage], lead);
        if (++stage == pl.stages) {
          stage = 0;
          ph ^= 1u;
        }
      }
      PAIR ? tc::commit_pair(&ctl.acc_full[buf], lead) : tc::commit_lead(&ctl.acc_full[buf], lead);
    }
    // every MMA issued has completed before tensor memory is released
    PAIR ? tc::commit_pair(&ctl.fin, lead) : tc::commit_lead(&ctl.fin, lead);
    mbar_wait_bounded(&ctl.fin, 0u);
  } else if (warp == 1) {
    mbar_wait_bounded(&ctl.fin, 0u);  // the odd CTA's copy: all that the even one sends here has come
  } else if (warp >= 4) {
    const int q4 = warp & 3, et = threadIdx.x - 128;
    const uint32_t lanes = (uint32_t)(32 * q4) << 16;
    int seg = 0;
    for (int tile = first; tile < pl.tiles; tile += stride, ++seg) {
      const int buf = seg & 1;
      const int n = (tile % pl.tiles_n) * kRowsTile + n_off + 32 * q4 + lane, m0 = (tile / pl.tiles_n) * pl.tn;
      const int cols = min(pl.tn, p.m - m0);
      float* sx = ctl.sx[buf];
      for (int i = et; i < cols; i += 128) sx[i] = p.xscale[m0 + i];
      const float sw = n < p.n ? p.wscale[n] : 0.f;
      named_sync_epilogue();
      tc::tc_wait_many(&ctl.acc_full[buf], (uint32_t)(seg / 2) & 1u, misc);
      tc::fence_after_sync();
      const uint32_t acc = tmem + (uint32_t)(buf * pl.tn) + lanes;
      for (int c = 0; c < pl.tn; c += 16) {
        uint32_t v[16];
        tc::ld_x16_sync(acc + (uint32_t)c, v);
        if (!PAIR && pl.split > 1) {  // [token][channel] at the ring's start: the loads are all in, and read
#pragma unroll
          for (int i = 0; i < 16; ++i)
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(ring + (uint32_t)((c + i) * kRowsA + 32 * q4 + lane) * 4u),
                         "r"(v[i])
                         : "memory");
        } else if (n < p.n) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (c + i < cols) store_one(p, m0 + c + i, n, (int)v[i], sw, sx[c + i]);
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR)
          tc::mbar_arrive_cluster(map_cluster_rank(smem_u32(&ctl.acc_empty[buf]), 0));
        else
          tc::mbar_arrive(&ctl.acc_empty[buf]);
      }
    }
  }
  __syncthreads();
  if constexpr (PAIR) {  // neither CTA's shared memory, barriers or tensor memory go before the other is done: its
                         // arrivals on them are released here, and the MMAs' have been waited for above
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    cluster_wait_acquire();
  }
  if (!PAIR && pl.split > 1) {
    // the cluster's partial sums, a share of the tokens per CTA
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    cluster_wait_acquire();
    const int n0 = (first % pl.tiles_n) * kRowsA, m0 = (first / pl.tiles_n) * pl.tn;
    const int cols = min(pl.tn, p.m - m0);
    // four channels of a token per thread and turn, every CTA's sums in one go
    const int n = n0 + 4 * (int)(threadIdx.x & 31);
    if (n < p.n) {
      float sw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) sw[i] = n + i < p.n ? p.wscale[n + i] : 0.f;
      for (int c = rank + pl.split * (int)(threadIdx.x >> 5); c < cols; c += 8 * pl.split) {
        const uint32_t at = ring + (uint32_t)(c * kRowsA + 4 * (int)(threadIdx.x & 31)) * 4u;
        const float sx = p.xscale[m0 + c];
        int4 v[kMaxSplit];
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r)
          v[r] = r < pl.split ? ld_dsmem(map_cluster_rank(at, (uint32_t)r)) : make_int4(0, 0, 0, 0);
        int acc[4] = {0, 0, 0, 0};
#pragma unroll
        for (int r = 0; r < kMaxSplit; ++r) acc[0] += v[r].x, acc[1] += v[r].y, acc[2] += v[r].z, acc[3] += v[r].w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < p.n) store_one(p, m0 + c, n + i, acc[i], sw[i], sx);
      }
    }
    __syncwarp();
    cluster_arrive_relaxed();  // a CTA's shared memory stays until its peers have read it
    cluster_wait_acquire();
  }
  if (warp == 1) {
    if constexpr (PAIR)
      tc::tmem_dealloc_pair(tmem, pl.tmem_cols);
    else
      tc::tmem_dealloc(tmem, pl.tmem_cols);
  }
}

// Clusters of each size that the device holds at once (whole clusters fit into a
// group of multiprocessors: 20 clusters of seven took two waves of 16, 8.7 us for 1
// x 2560 x 2560, where 20 of five took one, 5.1 us). Asked once per device.
const int* resident_clusters(int sms) {
  constexpr int kDevices = 64;
  static int table[kDevices][kMaxSplit + 1];
  static std::mutex lock;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) {
    cudaGetLastError();
    dev = 0;
  }
  const std::lock_guard<std::mutex> hold(lock);
  int* t = table[dev];
  if (t[1] == 0) {
    for (int s = 2; s <= kMaxSplit; ++s) {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3((unsigned)(s * (sms / s)));
      cfg.blockDim = dim3(kThreads);
      cfg.dynamicSmemBytes = kSmemTop;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim = {(unsigned)s, 1, 1};
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaFuncSetAttribute(gemm_i8_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemTop) !=
              cudaSuccess ||
          cudaOccupancyMaxActiveClusters(&n, gemm_i8_kernel<false>, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = 0;
      }
      t[s] = n;
    }
    t[1] = sms;
  }
  return t;
}

// Tokens per tile: up to 256, so that the waves of tiles cost least, a tile its
// tokens and a constant for its weights (2000 x 2560 x 2560: 13 times 160 tokens,
// two waves, 19 us; the fewest tiles, 8 of 256, 27 us. 4095 x 2560 x 2560 33 and 40 us.
// Constants from 64 to 160 differ by 3 %). Pairs of CTAs from one 256-channel tile
// per pair of SMs on and with wide tiles (256 x 32768 x 2560: pairs 31.5, single CTAs
// 33.4 us; 4095 x 14336 x 4096 8 % less than single CTAs; 128 x 32768 x 2560 22.7 and 21.7).
// Fewer tiles than half the SMs: the fewest, and K split over a cluster, as long as
// every CTA keeps four steps; of the cluster sizes the one with the least steps in a
// row, where meeting costs about four (61 x 2560 x 6912: 7 us, unsplit 16 us).
Plan make_plan(int m, int n, int k, int sms) {
  Plan pl{};
  pl.steps = (k + kStepK - 1) / kStepK;
  // one CTA per tile, then pairs; from the fewest tiles to twice as many
  double best = 0;
  auto consider = [&](int pair) {
    const int unit = pair ? 32 : 16, rows = pair ? 2 * kRowsA : kRowsA, units = pair ? sms / 2 : sms;
    const int tiles_n = (n + rows - 1) / rows, fewest = (m + 255) / 256;
    for (int t = fewest; t <= fewest + std::min(fewest, 16); ++t) {
      const int tn = ((m + t - 1) / t + unit - 1) / unit * unit;
      if (tn > 256) continue;
      const long long tiles = (long long)tiles_n * ((m + tn - 1) / tn);
      if (pair ? tn <= 208 || tiles < units : t > fewest && tiles <= units / 2) continue;
      const double cost = (double)((tiles + units - 1) / units) * (tn + (pair ? kPairCost : kTileCost));
      if (best != 0 && cost >= best) continue;
      best = cost;
      pl.pair = pair;
      pl.tn = tn;
      pl.tiles_n = tiles_n;
      pl.tiles_m = (m + tn - 1) / tn;
      if (!pair && t == fewest && tiles <= units / 2) return;  // K is split instead
    }
  };
  consider(0);
  consider(1);
  const long long tiles = (long long)pl.tiles_n * pl.tiles_m;
  pl.tiles = (int)tiles;
  pl.split = 1;
  if (!pl.pair && tiles <= sms / 2) {
    const int* fit = resident_clusters(sms);
    long long best = pl.steps;
    for (int s = 2; s <= kMaxSplit && s * kMinSteps <= pl.steps; ++s) {
      if (fit[s] < 1) continue;
      const long long cost = (tiles + fit[s] - 1) / fit[s] * ((pl.steps + s - 1) / s + kMinSteps);
      if (cost < best) best = cost, pl.split = s;
    }
  }
  pl.stage_bytes = kBytesA + (pl.pair ? pl.tn / 2 : pl.tn) * kStepK;
  pl.stages = std::min(kMaxStages, (kSmemTop - 1024 - kCtlBytes) / pl.stage_bytes);
  pl.grid = pl.pair ? 2 * (int)std::min<long long>(tiles, sms / 2)
                    : (int)std::min<long long>(tiles * pl.split, pl.split > 1 ? tiles * pl.split : sms);
  pl.tmem_cols = 32;
  while (pl.tmem_cols < 2u * (uint32_t)pl.tn) pl.tmem_cols *= 2;
  return pl;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult st;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &st) != cudaSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

bool encode(CUtensorMap* map, const int8_t* base, int k, int rows, int64_t ld, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)k, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)ld};
  const cuuint32_t box[2] = {(cuuint32_t)kStepK, (cuuint32_t)box_rows}, one[2] = {1, 1};
  EncodeTiled fn = encoder();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(base), dims, strides, box, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

int launch_gemm_i8(const GemmI8Params& p, int sms, void* stream) {
  Args a{p, make_plan(p.m, p.n, p.k, sms)};
  CUtensorMap mw, mx;
  if (!encode(&mw, p.w, p.k, p.n, p.ldw, kRowsA) ||
      !encode(&mx, p.x, p.k, p.m, p.ldx, a.pl.pair ? a.pl.tn / 2 : a.pl.tn))
    return -1;
  auto kernel = a.pl.pair ? gemm_i8_kernel<true> : gemm_i8_kernel<false>;
  const int bytes = kSmemTop, cluster = a.pl.pair ? 2 : a.pl.split;
  const int rc = allow_smem(reinterpret_cast<const void*>(kernel), bytes);
  if (rc != 0) return rc;
  return launch_dependent(kernel, a.pl.grid, kThreads, (size_t)bytes, cluster, static_cast<cudaStream_t>(stream), a, mw,
                          mx);
}

}  // namespace tern

extern "C" tern_status tern_gemm_i8(int32_t m, int32_t n, int32_t k, const int8_t* d_x, int64_t ldx,
                                    const float* d_xscale, const int8_t* d_w, int64_t ldw, const float* d_wscale,
                                    tern_out out, void* d_y, int64_t ldy, void* stream) {
  using namespace tern;
  if (m < 0 || m > kMaxExtent || n < 1 || n > kMaxExtent || k < 1 || k > 131071 || ldx < k || ldw < k || ldy < n ||
      ((ldx | ldw) & 15) != 0)
    return TERN_EINVAL;
  if (out != TERN_OUT_F32 && out != TERN_OUT_BF16) return TERN_EINVAL;
  if ((int64_t)((m + 15) / 16) * ((n + 127) / 128) > kMaxExtent) return TERN_EINVAL;
  if (m == 0) return TERN_OK;
  if (!d_x || !d_xscale || !d_w || !d_wscale || !d_y) return TERN_EINVAL;
  if (((reinterpret_cast<uintptr_t>(d_x) | reinterpret_cast<uintptr_t>(d_w)) & 15u) != 0) return TERN_EALIGN;
  const uintptr_t esize = out == TERN_OUT_F32 ? 3u : 1u;
  if (((reinterpret_cast<uintptr_t>(d_xscale) | reinterpret_cast<uintptr_t>(d_wscale)) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(d_y) & esize) != 0)
    return TERN_EALIGN;
  GemmI8Params p{};
  p.x = d_x;
  p.w = d_w;
  p.xscale = d_xscale;
  p.wscale = d_wscale;
  p.y = d_y;
  p.ldx = ldx;
  p.ldw = ldw;
  p.ldy = ldy;
  p.m = m;
  p.n = n;
  p.k = k;
  p.out_bf16 = out == TERN_OUT_BF16;
  const int rc = launch_gemm_i8(p, sm_count(), stream);
  return rc == 0 ? TERN_OK : TERN_ECUDA;
}
