// fk_mm.cuh -- sm_100a plumbing of the 8-bit matrix product that fk_tc.cuh
// does not hold: instruction descriptors and issue of the 8-bit MMAs, raw
// 32-bit TMEM loads, cluster helpers, and the kernel's bounded waits.
#pragma once

#include <stdint.h>

#include "fk_gelu.cuh"
#include "fk_mm_host.h"
#include "fk_q8.h"
#include "fk_sync.cuh"
#include "fk_tc.cuh"

namespace fk {
namespace mm {

// Threads of this source file's kernels whose bounded wait gave up.
static __device__ unsigned g_mm_wait_timeouts;

// Bounded mbarrier wait: gives up after `limit` (0: at once, for the
// self-test), is counted, and raises the block's abort flag, on which its
// other waits return at once.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit = kWaitNs) {
  if (limit != 0) {
    if (mbar_test_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    do {
      if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;  // suspended up to 20 us per try
      if (*abort) return false;
    } while (global_ns() - t0 <= limit);
  }
  atomicAdd(&g_mm_wait_timeouts, 1u);
  *abort = 1;
  return false;
}

// Bounded wait that ignores the abort flag: copies and MMAs in flight land
// before the block goes on.  False if it gave up: then they may still run, and
// the caller raises the abort flag.
__device__ __forceinline__ bool drain(uint64_t* bar, uint32_t parity, uint64_t limit = kWaitNs) {
  if (limit != 0) {
    const uint64_t t0 = global_ns();
    do {
      if (mbar_try_wait_sleep(bar, parity, 20000u)) return true;
    } while (global_ns() - t0 <= limit);
  }
  atomicAdd(&g_mm_wait_timeouts, 1u);
  return false;
}

// Instruction descriptor of a dense 8-bit MMA, both operands K-major, M x N:
// kind::i8 (signed codes, 32-bit integer accumulator) or kind::f8f6f4 (e4m3,
// fp32 accumulator).  One instruction covers 32 codes of k for either.
template <int Q8>
__host__ __device__ constexpr uint32_t idesc(int m, int n) {
  constexpr uint32_t fmt = Q8 == FK_I8 ? 1u : 0u;  // A and B: signed integer / e4m3
  constexpr uint32_t acc = Q8 == FK_I8 ? 2u : 1u;  // accumulator: s32 / f32
  return (acc << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// D (M x N, tensor memory) = A B^T (+ D when accumulate != 0), operands in
// shared memory.  Issued by one thread.
template <int Q8>
__device__ __forceinline__ void mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                    uint32_t accumulate) {
  if constexpr (Q8 == FK_I8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same on the pair of SMs (M = 256: each block of the pair holds half the
// rows of either operand and half the accumulator), issued by its leader.
template <int Q8>
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (Q8 == FK_I8)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One arrival on the barrier at this offset in both blocks of the pair when
// every MMA issued before by this thread has completed.  `leader`: the
// issuing block's rank in its cluster (even).
__device__ __forceinline__ void commit_pair(uint64_t* bar, int leader) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_addr(bar)),
      "h"(static_cast<uint16_t>(3 << leader))
      : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// 2-D tiled load into this block's shared memory, counted on a barrier of
// either block of the pair (its cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* tmap, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
      "[%2];" ::"r"(smem_addr(dst)),
      "l"(tmap), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// One arrival on a barrier of another block of the cluster.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// 16 consecutive 32-bit TMEM columns of this thread's lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// The same of 32 columns.  (Load and wait in one statement: nothing else ties
// the registers' first use to the wait.)
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// All threads of the cluster: arrive with release, wait with acquire.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The arrival alone, with release (cluster_wait() completes it).
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
}

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}

// Accumulator word to fp32: the exact integer sum rounded once, or the sum.
template <int Q8>
__device__ __forceinline__ float acc_value(uint32_t w) {
  return Q8 == FK_I8 ? static_cast<float>(static_cast<int>(w)) : __uint_as_float(w);
}
template <int Q8>
__device__ __forceinline__ uint32_t acc_add(uint32_t a, uint32_t b) {
  return Q8 == FK_I8 ? a + b : __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}

template <int EPI>
__device__ __forceinline__ float act(float x) {
  if constexpr (EPI == FK_EPILOGUE_GELU_TANH) return gelu_tanh_f<float>(x);
  if constexpr (EPI == FK_EPILOGUE_GELU_ERF) return gelu_erf_f<float>(x);
  return x;
}

// act(acc * sa * sb + bias) of one channel for two tokens, packed: each lane
// rounds as the scalar operations would.
template <int Q8, int EPI>
__device__ __forceinline__ float2 finish2(uint32_t w0, uint32_t w1, float sa0, float sa1, float sb, float bias) {
  const float2 v = fma2(mul2(make_float2(acc_value<Q8>(w0), acc_value<Q8>(w1)), make_float2(sa0, sa1)), splat2(sb),
                        splat2(bias));
  if constexpr (EPI == FK_EPILOGUE_GELU_TANH) return gelu_tanh_f2<float>(v);
  if constexpr (EPI == FK_EPILOGUE_GELU_ERF) return gelu_erf_f2<float>(v);
  return v;
}

}  // namespace mm
}  // namespace fk
