// fk_quantize.cu -- rows to 8 bits with one scale each, optionally through
// GELU (sm_100a).
#include <cuda_bf16.h>

#include "fk_common.cuh"
#include "fk_gelu.cuh"
#include "fk_q8.cuh"
#include "fk_q8_internal.h"
#include "fk_q8_rows.cuh"

namespace fk {
namespace {

constexpr int kStreamThreads = 512;
constexpr size_t kMaxGrid = 0x7fffffffu;

// Inputs are raised to kGeluFloor first, as in fk_gelu: both forms give -0
// there, and -inf no longer meets inf * 0.  The floor has to lie where GELU is
// 0 as fp32: a row of far negative values has a scale as small as its GELU, so
// that no magnitude above 2^-119 (half a code of the smallest scale) is small
// against it.  The tanh form's reciprocal flushes to 0 from -10 on, the erf
// form's exponential from -13.1 on, GELU there being under 2^-122.
constexpr uint32_t kGeluFloorPair = 0xc1f0c1f0u;  // two bf16 -30

// GELU of a pair to fp32 accuracy, as gelu_tanh_f2 / gelu_erf_f2, of values
// not below kGeluFloor.  (The reciprocal on the FMA pipes instead of MUFU,
// for all pairs or every other one: 46 and 39.6 us against 38.2 for
// 16384 x 4096.)
template <int EPI>
__device__ __forceinline__ float2 act2(float2 x) {
  if constexpr (EPI == FK_EPILOGUE_GELU_TANH) {
    const float2 a = mul2(x, fma2(splat2(kB), mul2(x, x), splat2(kA)));
    const float2 s = add2(make_float2(ex2_ftz(a.x), ex2_ftz(a.y)), splat2(1.0f));
    return mul2(x, make_float2(rcp_approx(s.x), rcp_approx(s.y)));
  }
  if constexpr (EPI == FK_EPILOGUE_GELU_ERF) {
    const float2 w = mul2(make_float2(fabsf(x.x), fabsf(x.y)), splat2(kRsqrt2));
    const float2 s = fma2(splat2(0.5f), w, splat2(1.0f));
    const float2 t = make_float2(rcp_approx(s.x), rcp_approx(s.y));
    const float2 e = mul2(fma2(make_float2(-w.x, -w.y), w, erfc_poly(t)), splat2(kLog2e));
    const float2 h = mul2(mul2(splat2(0.5f), t), make_float2(ex2_ftz(e.x), ex2_ftz(e.y)));
    const float2 sg = make_float2(phi_sign(x.x), phi_sign(x.y));
    return mul2(x, fma2(sg, h, fma2(sg, splat2(-0.5f), splat2(0.5f))));
  }
  return x;
}

// GELU of a pair with one reciprocal for both: 1 / s_x = s_y / (s_x s_y).
// For values of at least kLowFloor, where the product stays in range.
template <int EPI>
__device__ __forceinline__ float2 act2_joint(float2 x) {
  if constexpr (EPI == FK_EPILOGUE_GELU_TANH) {
    const float2 a = mul2(x, fma2(splat2(kB), mul2(x, x), splat2(kA)));
    const float2 s = add2(make_float2(ex2_ftz(a.y), ex2_ftz(a.x)), splat2(1.0f));  // the other's
    return mul2(x, mul2(s, splat2(rcp_approx(s.x * s.y))));  // (x s could overflow)
  }
  if constexpr (EPI == FK_EPILOGUE_GELU_ERF) {
    const float2 w = mul2(make_float2(fabsf(x.x), fabsf(x.y)), splat2(kRsqrt2));
    const float2 s = fma2(splat2(0.5f), make_float2(w.y, w.x), splat2(1.0f));
    const float2 t = mul2(s, splat2(rcp_approx(s.x * s.y)));
    const float2 e = mul2(fma2(make_float2(-w.x, -w.y), w, erfc_poly(t)), splat2(kLog2e));
    const float2 h = mul2(mul2(splat2(0.5f), t), make_float2(ex2_ftz(e.x), ex2_ftz(e.y)));
    const float2 sg = make_float2(phi_sign(x.x), phi_sign(x.y));
    return mul2(x, fma2(sg, h, fma2(sg, splat2(-0.5f), splat2(0.5f))));
  }
  return x;
}

// A packed word's values raised to a floor (NaN stays), where GELU follows.
template <typename T, int EPI>
__device__ __forceinline__ uint4 raised(uint4 w, float floor = kGeluFloor, uint32_t floor_pair = kGeluFloorPair) {
  if constexpr (EPI != FK_EPILOGUE_NONE && sizeof(T) == 4) {
    w.x = __float_as_uint(max_nan(__uint_as_float(w.x), floor));
    w.y = __float_as_uint(max_nan(__uint_as_float(w.y), floor));
    w.z = __float_as_uint(max_nan(__uint_as_float(w.z), floor));
    w.w = __float_as_uint(max_nan(__uint_as_float(w.w), floor));
  } else if constexpr (EPI != FK_EPILOGUE_NONE) {
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.x) : "r"(floor_pair));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.y) : "r"(floor_pair));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.z) : "r"(floor_pair));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w.w) : "r"(floor_pair));
  }
  return w;
}
template <int EPI>
__device__ __forceinline__ float act(float x) {
  return act2<EPI>(splat2(EPI == FK_EPILOGUE_NONE ? x : max_nan(x, kGeluFloor))).x;
}

// The largest |GELU(x)| of negative x is 0.1701 (either form), and GELU rises
// from there on: where GELU of a row's largest value is above this, it is the
// row's largest magnitude, and no other value's GELU is needed for the scale.
constexpr float kGeluDip = 0.1725f;
// In such a row every value below this has the code 0 (|GELU| there is under
// 4e-13, the smallest scale 0.1725 / 448): values are raised to it, which
// bounds what two of them exponentiate together (2^61 each, tanh form).
// Exact in bf16.
constexpr float kLowFloor = -7.5f;
constexpr uint32_t kLowFloorPair = 0xc0f0c0f0u;

// Largest value (not magnitude) among m and a vector's, NaN if one is.
template <typename T>
__device__ __forceinline__ float max_words(float m, const uint4& w) {
  if constexpr (sizeof(T) == 4) {
    m = max_nan(max_nan(m, __uint_as_float(w.x)), __uint_as_float(w.y));
    return max_nan(max_nan(m, __uint_as_float(w.z)), __uint_as_float(w.w));
  } else {
    uint32_t a, b;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(w.x), "r"(w.y));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(w.z), "r"(w.w));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
    return max_nan(max_nan(m, __uint_as_float(a << 16)), __uint_as_float(a & 0xffff0000u));
  }
}

// ---------------------------------------------------------------- rows held in registers

// One team per row (fk_q8_rows.cuh): read, activation, largest magnitude,
// codes.  Bound by HBM without GELU; measured on B200: 16384 x 4096 bf16 to
// e4m3 30.9 us (6.5 TB/s), through the tanh form 37.7 (two MUFU operations a
// value take 30), through the erf form 64; 8192 x 8192 fp32 49 / 52 / 64.
// MAXT, MINB as in fk_rmsnorm.cu.
template <typename T, int OUT, int EPI, int EPT, bool ALIGNED, int LANES, int MAXT, int MINB, int CL = 1>
__global__ void __launch_bounds__(MAXT, MINB) quantize_row_kernel(const __grid_constant__ QuantizeArgs a) {
  constexpr int VEC = Elem<T>::VEC, VPT = EPT / VEC;
  __shared__ __align__(16) float red[LANES ? 1 : MAXT / 32];
  __shared__ float2 pairs[CL > 1 ? CL * (MAXT / 32) : 1];
  let_next_start();
  after_previous();
  for_rows<LANES, CL>(a.rows, static_cast<int>(a.cols), [&](size_t row, int t, int team, int cols) {
    const size_t base = row * a.cols;
    const T* const x = static_cast<const T*>(a.x) + base;
    uint8_t* const o = static_cast<uint8_t*>(a.q) + base;
    const Place p = place_of<T, ALIGNED>(t, team, cols, x);
    const int edge = ALIGNED ? -1 : edge_col<VEC>(p);
    uint4 raw[VPT];
    load_vecs<T, VPT>(x, p, raw);
    float ev = 0.0f;  // this thread's value outside the vectors
    if (!ALIGNED && edge >= 0) ev = load_one(x + edge);
    float v[EPT], m = 0.0f;
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      Elem<T>::unpack(raised<T, EPI>(raw[c]), v + c * VEC);
#pragma unroll
      for (int k = 0; k < VEC; k += 2) {
        const float2 x2 = make_float2(v[c * VEC + k], v[c * VEC + k + 1]);
        const float2 z = act2<EPI>(x2);
        v[c * VEC + k] = z.x;
        v[c * VEC + k + 1] = z.y;
        m = absmax_nan(absmax_nan(m, z.x), z.y);
      }
    }
    if (!ALIGNED && edge >= 0) {
      ev = act<EPI>(ev);
      m = absmax_nan(m, ev);
    }
    if constexpr (CL > 1) {
      float none = 0.0f;
      cluster_sum_max<CL>(none, m, pairs);
    } else {
      team_max<LANES>(m, red);
    }
    const RowScale q = row_scale<OUT>(m);
    if (t == 0 && cols > 0) a.scales[row] = q.scale;
#pragma unroll
    for (int c = 0; c < VPT; ++c) store_codes<T, OUT, ALIGNED>(o, p, c, v + c * VEC, q);
    if (!ALIGNED && edge >= 0) o[edge] = q.ok ? Code8<OUT>::pack1(ev, q) : 0;
  });
}

// Wide bf16 rows: blocks that stay and walk the rows, the next row loaded
// before the current one is computed.  Measured on B200 (8192 x 16384 to
// e4m3): 63 us plain (6.4 TB/s), 82 through the tanh form (with the quotient
// left unrounded, v (Q / max), 80; and 93 with a reciprocal for each value,
// one read a warp of the row's maxima and the scale applied to single values),
// 138 through the erf form (26 instructions a value: issue).  The tanh form's
// rest: MUFU, with 1.5 operations a value at least 46 us, and issue, at 15
// instructions a value 56, in turns between barriers.
// Rows whose largest value does not decide the scale (all below about 0.28)
// take GELU of their packed values twice: 159 and 230 us (rows of 0.05
// deviation; 553 and 617 when they were read again, value by value).
// Rows of up to 8192 columns do not gain (4096: 38.4 against 37.5 with one
// row per block), nor do shifted ones (16383: 112 against 96).
template <typename T, int OUT, int EPI, int EPT, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) quantize_walk_kernel(const __grid_constant__ QuantizeArgs a) {
  constexpr int VEC = Elem<T>::VEC, VPT = EPT / VEC;
  __shared__ __align__(16) float red[2][MAXT / 32], dip[MAXT / 32];
  const int cols = static_cast<int>(a.cols), t = static_cast<int>(threadIdx.x), team = static_cast<int>(blockDim.x);
  const T* const x = static_cast<const T*>(a.x);
  let_next_start();
  after_previous();
  uint4 raw[VPT];
  const Place p = place_of<T, true>(t, team, cols, x);
  if (blockIdx.x < a.rows) load_vecs<T, VPT>(x + blockIdx.x * a.cols, p, raw);
  int turn = 0;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const size_t base = row * a.cols;
    uint4 next[VPT];
    if (row + gridDim.x < a.rows) load_vecs<T, VPT>(x + base + gridDim.x * a.cols, p, next);
    // the row's largest magnitude: for GELU, from its largest value alone
    // where that decides, so that the values stay packed until their codes
    // are made
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      if constexpr (EPI == FK_EPILOGUE_NONE) {
        float f[VEC];
        Elem<T>::unpack(raw[c], f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) m = absmax_nan(m, f[k]);
      } else {
        m = max_words<T>(m, raw[c]);
      }
    }
    team_max<0>(m, red[turn]);
    bool rises = false;
    if constexpr (EPI != FK_EPILOGUE_NONE) {
      m = act<EPI>(m);
      rises = m > kGeluDip;
      if (!rises) {  // small or negative values only, or a NaN: the same for the whole block
        m = 0.0f;
#pragma unroll
        for (int c = 0; c < VPT; ++c) {
          float f[VEC];
          Elem<T>::unpack(raised<T, EPI>(raw[c]), f);
#pragma unroll
          for (int k = 0; k < VEC; k += 2) {
            const float2 z = act2<EPI>(make_float2(f[k], f[k + 1]));
            m = absmax_nan(absmax_nan(m, z.x), z.y);
          }
        }
        team_max<0>(m, dip);
        __syncthreads();  // dip may be used by the next row
      }
    }
    turn ^= 1;
    const RowScale q = row_scale<OUT>(m);
    uint8_t* const o = static_cast<uint8_t*>(a.q) + base;
    if (t == 0) a.scales[row] = q.scale;
    if (rises) {
#pragma unroll
      for (int c = 0; c < VPT; ++c) {
        float f[VEC];
        Elem<T>::unpack(raised<T, EPI>(raw[c], kLowFloor, kLowFloorPair), f);
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
          const float2 z = act2_joint<EPI>(make_float2(f[k], f[k + 1]));
          f[k] = z.x;
          f[k + 1] = z.y;
        }
        store_codes<T, OUT, true>(o, p, c, f, q);
      }
    } else {
#pragma unroll
      for (int c = 0; c < VPT; ++c) {
        float f[VEC];
        Elem<T>::unpack(raised<T, EPI>(raw[c]), f);
#pragma unroll
        for (int k = 0; k < VEC; k += 2) {
          const float2 z = act2<EPI>(make_float2(f[k], f[k + 1]));
          f[k] = z.x;
          f[k + 1] = z.y;
        }
        store_codes<T, OUT, true>(o, p, c, f, q);
      }
    }
#pragma unroll
    for (int c = 0; c < VPT; ++c) raw[c] = next[c];
  }
}

// ---------------------------------------------------------------- streaming path

// One 512-thread block per row, which reads the row twice: the largest
// magnitude, then the codes.  Any length and alignment; value by value, for
// rows past 131072 columns (1024 x 140000 bf16 to e4m3: 339 us; 960 x 131072 in
// clusters 130).
template <typename T, int OUT, int EPI>
__global__ void __launch_bounds__(kStreamThreads) quantize_stream_kernel(QuantizeArgs a) {
  __shared__ float2 red[kStreamThreads / 32];
  const size_t cols = a.cols;
  let_next_start();
  after_previous();
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * cols;
    uint8_t* o = static_cast<uint8_t*>(a.q) + row * cols;
    float s = 0.0f, m = 0.0f;
    for (size_t j = threadIdx.x; j < cols; j += kStreamThreads) m = absmax_nan(m, act<EPI>(static_cast<float>(x[j])));
    block_sum_max<kStreamThreads / 32>(s, m, red);
    const RowScale q = row_scale<OUT>(m);
    if (threadIdx.x == 0) a.scales[row] = q.scale;
    for (size_t j = threadIdx.x; j < cols; j += kStreamThreads)
      o[j] = q.ok ? Code8<OUT>::pack1(act<EPI>(static_cast<float>(x[j])), q) : 0;
    __syncthreads();  // red is rewritten by the next row
  }
}

template <typename T, int OUT, int EPI, bool ALIGNED>
cudaError_t launch_rows(const QuantizeArgs& a, cudaStream_t s) {
  if (a.cols <= kRowWarpCols) {
    const int lanes = row_lanes(a.cols, ALIGNED, Elem<T>::VEC);
    const RowLaunch l = warp_launch(a.rows, lanes);
    if (lanes == 8)
      return launch_overlapped(quantize_row_kernel<T, OUT, EPI, kRowLaneEpt, ALIGNED, 8, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    if (lanes == 16)
      return launch_overlapped(quantize_row_kernel<T, OUT, EPI, kRowLaneEpt, ALIGNED, 16, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    if (a.cols <= kRowWarpCols / 4)
      return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 8, ALIGNED, 32, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    if (a.cols <= kRowWarpCols / 2)
      return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 16, ALIGNED, 32, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, 32, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
  }
  const RowLaunch l = block_launch(a.rows, a.cols, 32);
  if constexpr (sizeof(T) == 2 && ALIGNED) {
    if (a.cols > kRowBlockCols && a.cols <= kRowLargeCols) {
      // as many blocks as stay resident: 1024 threads an SM at 64 registers
      const unsigned fit = 148u * (1024u / l.threads);
      return launch_overlapped(quantize_walk_kernel<T, OUT, EPI, 32, 512, 2>, l.grid < fit ? l.grid : fit,
                               l.threads, 0, 1, s, a);
    }
  }
  if (a.cols <= kRowLargeCols)
    return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, 0, 512, 2>, l.grid, l.threads, 0, 1, s, a);
  if constexpr (sizeof(T) == 2 && EPI != FK_EPILOGUE_NONE) {
    // two blocks of 512 threads to a row compute one row while another loads
    // (4096 rows, tanh form, us against one block of 1024: 20000 columns 67
    // and 92, 24576 95 and 103, 32768 113 and 130, before codes were those of
    // the rounded quotient, with which they take 70, 97 and 116; without GELU,
    // 32768: 89 and 87)
    if (a.cols <= kRowMaxCols) {
      const RowLaunch c = cluster_launch(a.rows, a.cols, 2);
      return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, 0, 512, 2, 2>, c.grid, c.threads, 0, 2, s, a);
    }
  } else if (a.cols <= kRowMaxCols) {
    return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, 0, 1024, 1>, l.grid, l.threads, 0, 1, s, a);
  }
  // 4 or 8 blocks of 512 threads (1024 x 65536 bf16 54 us; 2 or 4 of 1024: 60)
  const int cl = a.cols <= kRowClusterCols / 2 ? 4 : 8;
  const RowLaunch c = cluster_launch(a.rows, a.cols, cl);
  return cl == 4 ? launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, 0, 512, 2, 4>, c.grid, c.threads, 0, 4, s, a)
                 : launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, 0, 512, 2, 8>, c.grid, c.threads, 0, 8, s, a);
}

template <typename T, int OUT, int EPI>
cudaError_t launch_epi(const QuantizeArgs& a, cudaStream_t s) {
  if (a.cols > kRowClusterCols) {
    const unsigned g = static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid);
    return launch_overlapped(quantize_stream_kernel<T, OUT, EPI>, g, kStreamThreads, 0, 1, s, a);
  }
  return a.mode == kRowsAligned ? launch_rows<T, OUT, EPI, true>(a, s) : launch_rows<T, OUT, EPI, false>(a, s);
}

template <typename T, int OUT>
cudaError_t launch_out(const QuantizeArgs& a, cudaStream_t s) {
  switch (a.epilogue) {
    case FK_EPILOGUE_GELU_TANH: return launch_epi<T, OUT, FK_EPILOGUE_GELU_TANH>(a, s);
    case FK_EPILOGUE_GELU_ERF: return launch_epi<T, OUT, FK_EPILOGUE_GELU_ERF>(a, s);
    default: return launch_epi<T, OUT, FK_EPILOGUE_NONE>(a, s);
  }
}

template <typename T>
cudaError_t launch_type(const QuantizeArgs& a, cudaStream_t s) {
  return a.out_dtype == FK_I8 ? launch_out<T, FK_I8>(a, s) : launch_out<T, FK_E4M3>(a, s);
}

}  // namespace

cudaError_t launch_quantize(const QuantizeArgs& a, cudaStream_t stream) {
  return a.dtype == FK_F32 ? launch_type<float>(a, stream) : launch_type<__nv_bfloat16>(a, stream);
}

}  // namespace fk
