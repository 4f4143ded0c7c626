// fk_q8.cuh -- 8-bit codes and per-row scales: the conversions and the row
// reductions shared by RMSNorm and the row quantiser (sm_100a).
//
// A row v becomes scale = max(max |v_j|, 2^-100) * (1 / Q) and code_j =
// round(v_j / scale), nearest even (Q = 127 or 448; 1 / Q rounded to fp32, as
// torch divides a tensor by a number on the GPU).  The lower limit on the
// maximum keeps 1 / scale finite, so a row of zeros needs no special case.
// v_j / scale exceeds Q by at most a rounding, which rounds back to Q.
//
// The quotient is that of the stored fp32 scale, rounded once: values of bf16
// rows stand often exactly on a border between two codes of max / Q, and go
// the way that v / scale takes them in any fp32 arithmetic.  With 1 / scale in
// two fp32 terms, hi = rounded and lo = hi (1 - scale hi) (the remainder comes
// out of one fused multiply-add without error), v hi + v lo in one FMA is
// within 2^-46 of v / scale before its rounding.  One packed instruction a
// pair more than v hi alone; correcting v hi by its own remainder takes two
// (8192 x 16384 bf16 through GELU to e4m3, against v hi alone: 3.9% and 7.5%
// more time; without GELU, and in the norm, under 2%).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "fk_common.cuh"
#include "fk_f32x2.cuh"
#include "fk_q8.h"

namespace fk {
namespace {

constexpr float kTinyAmax = 0x1p-100f;

// Programmatic dependent launch: a kernel launched with overlap allowed
// (launch_overlapped) may start while its predecessor in the stream still
// runs.  after_previous() returns once the predecessor has completed and its
// writes are visible; nothing in global memory is touched before it.
// let_next_start() allows the same to the successor, from the moment when one
// thread of every block has called it (measured on B200: a block's first call
// counts).  A kernel that takes tensor memory calls it from the warp that
// allocates, after it has: otherwise the successor's blocks could hold the
// columns, waiting for this kernel's end, that a block of it still waits for.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// What a kernel launched this way reads with, in place of __ldg and the
// non-coherent loads of fk_common.cuh: their data must not change while the
// kernel lives, and the predecessor may still be writing it when this one
// starts.
__device__ __forceinline__ float ld_param(const float* p) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ float4 ld_param4(const float* p) {
  float4 v;
  asm volatile("ld.global.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
  return v;
}
// 16 bytes of a row that is read once, zeros when !pred (nothing is read then).
// RELAXED: as a relaxed access, which clusters of bf16 rows take faster (norm,
// 1024 x 49152 82 us against 92) and one block per row does not (4096 x 16384
// 84.3 against 82.7).
template <bool RELAXED>
__device__ __forceinline__ uint4 ld_row_v4_if(const void* p, bool pred) {
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (RELAXED)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q ld.relaxed.gpu.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"(static_cast<unsigned>(pred))
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
        "@q ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
        : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w)
        : "l"(p), "r"(static_cast<unsigned>(pred))
        : "memory");
  return v;
}

// max(a, |b|), NaN if either is.
__device__ __forceinline__ float absmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

// What a row's codes are made with: the stored scale, and its reciprocal in two
// terms; a row that is not finite gets the scale NaN and codes 0 (`ok`).
struct RowScale {
  float scale, hi, lo;
  bool ok;
};

// v / scale, rounded once.
__device__ __forceinline__ float over_scale(float v, const RowScale& q) { return fmaf(v, q.hi, v * q.lo); }
__device__ __forceinline__ float2 over_scale2(float2 v, const RowScale& q) {
  return fma2(v, splat2(q.hi), mul2(v, splat2(q.lo)));
}

template <int Q8>
struct Code8;

template <>
struct Code8<FK_I8> {
  static constexpr float kMax = 127.0f;
  // 1.5 * 2^23 + t has unit spacing, so the sum rounds t to the nearest
  // integer, ties to even, and leaves it in two's complement in the low
  // mantissa bits.
  static constexpr float kUnits = 12582912.0f;
  __device__ __forceinline__ static uint32_t pack4(const float* v, const RowScale& q) {
    const float2 a = add2(over_scale2(make_float2(v[0], v[1]), q), splat2(kUnits));
    const float2 b = add2(over_scale2(make_float2(v[2], v[3]), q), splat2(kUnits));
    const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
    const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
    return __byte_perm(lo, hi, 0x5410);
  }
  __device__ __forceinline__ static uint8_t pack1(float v, const RowScale& q) {
    return static_cast<uint8_t>(__float_as_uint(over_scale(v, q) + kUnits));
  }
};

template <>
struct Code8<FK_E4M3> {
  static constexpr float kMax = 448.0f;
  // Two values to two codes (the first in the low byte), nearest even.
  __device__ __forceinline__ static uint16_t pair(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ __forceinline__ static uint32_t pack4(const float* v, const RowScale& q) {
    const float2 a = over_scale2(make_float2(v[0], v[1]), q), b = over_scale2(make_float2(v[2], v[3]), q);
    return pair(a.x, a.y) | (static_cast<uint32_t>(pair(b.x, b.y)) << 16);
  }
  __device__ __forceinline__ static uint8_t pack1(float v, const RowScale& q) {
    return static_cast<uint8_t>(pair(over_scale(v, q), 0.0f));
  }
};

template <int Q8>
__device__ __forceinline__ RowScale row_scale(float amax) {
  RowScale r;
  r.ok = amax <= 3.402823466e38f;  // neither NaN nor infinite
  r.scale = r.ok ? fmaxf(amax, kTinyAmax) * (1.0f / Code8<Q8>::kMax) : __int_as_float(0x7fffffff);
  r.hi = __frcp_rn(r.scale);  // (rcp_approx spills: 8192 x 16384 through GELU 83.2 us against 81.7)
  r.lo = r.hi * fmaf(-r.scale, r.hi, 1.0f);
  return r;
}

// Sum of `s` and NaN-propagating maximum of `m` over a warp.
__device__ __forceinline__ void warp_sum_max(float& s, float& m) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = absmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
}

// The same over a block of NW warps; `red` holds NW pairs.  The caller puts a
// __syncthreads() between two uses of `red`.
template <int NW>
__device__ __forceinline__ void block_sum_max(float& s, float& m, float2* red) {
  warp_sum_max(s, m);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(s, m);
    __syncthreads();
    s = red[0].x;
    m = red[0].y;
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      s += red[w].x;
      m = absmax_nan(m, red[w].y);
    }
  }
}

// A pair of values into a block's shared memory at cluster address `dst`.
__device__ __forceinline__ void st_cluster_f2(uint32_t dst, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(dst), "f"(a), "f"(b) : "memory");
}

// Every thread of the cluster: what was stored before it is seen after it.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// 1 / sqrt(sum / n + eps); NaN for a sum that is not finite, so that a row
// holding an infinity (or overflowing) is NaN throughout, not zero.
__device__ __forceinline__ float rms_rstd(float sum, float inv_n, float eps) {
  return sum <= 3.402823466e38f ? rsqrtf(fmaf(sum, inv_n, eps)) : __int_as_float(0x7fffffff);
}

}  // namespace
}  // namespace fk
