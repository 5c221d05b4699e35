// Inline-PTX wrappers for the 5th-generation tensor cores of sm_100a
// (tcgen05): tensor-memory allocation, shared-memory matrix descriptors, the
// 8-bit integer MMA with its completion commit, and tensor-memory loads.
// Field layouts follow the PTX ISA's tcgen05 descriptor definitions.
#pragma once
#include <cstdint>

#include "tern_ptx.cuh"

namespace tern {
namespace tc {

// Allocate `ncols` tensor-memory columns (power of two >= 32) for this CTA; the
// base address is written to shared memory at `dst`. Executed by one whole warp.
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// Ordering of tcgen05 operations across thread synchronisation.
__device__ __forceinline__ void fence_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Shared-memory matrix descriptor, no swizzle (canonical K-major layout of
// 8-row x 16-byte core matrices): start address, leading byte offset (between
// core matrices adjacent along K), stride byte offset (between core matrices
// adjacent along M or N), descriptor version 1 at bits 46-47, swizzle mode 0.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}

// Shared-memory matrix descriptor, 64-byte swizzle, K-major: rows of 64 bytes,
// 8-row atoms of 512 bytes (16-byte chunk c of row r stored at chunk
// c ^ ((r >> 1) & 3)); stride byte offset between 8-row groups, leading byte
// offset unused (1), swizzle mode 4 at bits 61-63. The atom base must be
// 512-byte aligned; a K offset inside the 64-byte row is added to the start.
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t addr, uint32_t sbo) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) |
         (4ull << 61);
}

// Shared-memory matrix descriptor, 128-byte swizzle, K-major: rows of 128
// bytes, 8-row atoms of 1024 bytes (16-byte chunk c of row r stored at chunk
// c ^ (r & 7)), as a tensor-map load with the same swizzle writes them; swizzle
// mode 2 at bits 61-63. The atom base must be 1024-byte aligned; a K offset
// inside the 128-byte row is added to the start.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) |
         (2ull << 61);
}

// Instruction descriptor of kind::i8 with signed A and B, int32 accumulator,
// both operands K-major, M = 128 rows, N columns (16..256, multiple of 16).
__host__ __device__ constexpr uint32_t idesc_i8_s32(int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T, issued by one thread.
__device__ __forceinline__ void mma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Instruction descriptor of kind::f16 with fp16 A and B, fp32 accumulator, M =
// 128 rows, N columns; A K-major, B K-major or (b_mn) with N contiguous.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int n, bool b_mn) {
  return (1u << 4) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

// Shared-memory matrix descriptor, 128-byte swizzle, N contiguous: atoms of 8
// rows of K by 64 16-bit elements of N (128 bytes a row, swizzled as above);
// `n_stride` bytes from 64 columns to the next 64, 1024 bytes from 8 rows of K to
// the next 8.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t addr, uint32_t n_stride) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((n_stride >> 4) & 0x3FFFu) << 16) |
         ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// MMAs issued by a whole warp in convergent code, of which the lane with `lead`
// set takes part. The instruction takes its operands from uniform registers:
// inside a one-thread branch every descriptor is moved there for every MMA,
// about 120 cycles each, which is twice what the tensor cores take for 128 x
// 128 x 16; computed by the whole warp they stay there.
__device__ __forceinline__ void mma_i8_lead(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// D[tmem] (+)= A[smem] * B[smem], 16-bit operands.
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// ... with A in tensor memory: row i in lane i, two 16-bit elements of K per column.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// commit (below) by the lane with `lead` set.
__device__ __forceinline__ void commit_lead(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// Arrive once on `bar` when every tcgen05 operation this thread issued so far
// has completed.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

// Eight consecutive 32-bit columns of this warp's 32 lanes (lane quarter
// warp_id % 4); thread i receives lane 32 * (warp_id % 4) + i. The load and
// its completion wait are one statement, so no use of the registers can be
// scheduled before the data has arrived.
__device__ __forceinline__ void ld_x8_sync(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
      : "r"(taddr)
      : "memory");
}

// Sixteen consecutive 32-bit columns of this warp's lane quarter, as ld_x8_sync.
__device__ __forceinline__ void ld_x16_sync(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// Thirty-two consecutive 32-bit columns of this warp's lane quarter, as ld_x8_sync.
__device__ __forceinline__ void ld_x32_sync(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
// Sixteen consecutive columns written; st_wait ends when they are.
__device__ __forceinline__ void st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
      "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four consecutive 32-bit columns of this warp's lane quarter, as ld_x8_sync.
__device__ __forceinline__ void ld_x4_sync(uint32_t taddr, uint32_t (&v)[4]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(taddr)
      : "memory");
}

// ---- pairs of CTAs (cta_group::2): one MMA over both CTAs' shared memory, M =
// 256 rows of which each CTA holds 128, accumulators in both tensor memories;
// issued by the CTA of even rank. Both CTAs execute allocation and release.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// As idesc_i8_s32 with M = 256; N a multiple of 32.
__host__ __device__ constexpr uint32_t idesc_i8_s32_pair(int n) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(256 >> 4) << 24);
}
__device__ __forceinline__ void mma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
// commit_lead on the barrier at this place in both CTAs of the pair.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b16 m;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "mov.b16 m, 3;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// tma_load_2d into this CTA, completing on a barrier of either CTA of the pair
// (its address in the cluster's window).
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst_smem, const void* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
      "%3}], [%4];" ::"r"(dst_smem),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Words after the mbarriers of a tensor-core kernel: the tensor-memory base
// address, the abort flag of its bounded waits, the last-arrival flag.
constexpr int kMiscTmem = 0, kMiscAbort = 1, kMiscLast = 2;

// Non-blocking test of a phase.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Bounded wait by polling (a suspended try_wait resumes too late for the
// one-thread roles on the critical path). Gives up at once when another thread
// of the CTA has already given up (misc[kMiscAbort]), so that a failure costs
// about one time limit, not one per wait.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* misc) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_test(bar, parity)) return true;
    if ((it & 255u) == 0u) {
      if (misc[kMiscAbort]) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        atomicOr(&g_dev_error, TERN_DEVERR_TIMEOUT);
        misc[kMiscAbort] = 1u;
        return false;
      }
    }
  }
}

// The same bounded wait for roles of many warps: they sleep between tests, so
// that hundreds of waiting threads do not crowd the issue slots and the
// shared-memory pipe that the single-thread producer and MMA roles need.
__device__ __forceinline__ bool tc_wait_many(uint64_t* bar, uint32_t parity, volatile uint32_t* misc) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    __nanosleep(64);
    if (mbar_test(bar, parity)) return true;
    if ((it & 63u) == 0u) {
      if (misc[kMiscAbort]) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        atomicOr(&g_dev_error, TERN_DEVERR_TIMEOUT);
        misc[kMiscAbort] = 1u;
        return false;
      }
    }
  }
}

// Bounded wait that reads the clock only after many tests: that read takes longer than most waits last. Polling, or
// (kSuspend, for roles of many warps) suspended by the hardware between tests.
template <bool kSuspend>
__device__ __forceinline__ bool tc_wait_late(uint64_t* bar, uint32_t parity, volatile uint32_t* misc) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (kSuspend ? mbar_try_wait(bar, parity) : mbar_test(bar, parity)) return true;
    if ((it & 255u) == 0u) {
      if (misc[kMiscAbort]) return false;
      if (it == 0u) continue;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitLimitNs) {
        atomicOr(&g_dev_error, TERN_DEVERR_TIMEOUT);
        misc[kMiscAbort] = 1u;
        return false;
      }
    }
  }
}

// tc_wait for phases that the other CTA's threads complete.
__device__ __forceinline__ bool tc_wait_cluster(uint64_t* bar, uint32_t parity, volatile uint32_t* misc) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait<true>(bar, parity)) return true;
    if ((it & 255u) == 0u || global_timer_ns() - t0 > kWaitLimitNs) {
      if (misc[kMiscAbort]) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        atomicOr(&g_dev_error, TERN_DEVERR_TIMEOUT);
        misc[kMiscAbort] = 1u;
        return false;
      }
    }
  }
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Bulk copy without a cache-policy hint (a tile's weights are read again by
// its next token pass, so they should stay in L2).
__device__ __forceinline__ void bulk_g2s_plain(uint32_t dst_smem, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst_smem),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Two-dimensional tensor-map load: the box at (x, y), x a multiple of 16 bytes;
// places outside the tensor arrive as zeros and count.
__device__ __forceinline__ void tma_load_2d(uint32_t dst_smem, const void* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst_smem),
      "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

}  // namespace tc
}  // namespace tern
