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

template <int EPI>
__device__ __forceinline__ float act(float x) {
  if constexpr (EPI == FK_EPILOGUE_GELU_TANH) return gelu_tanh_f<float>(x);
  if constexpr (EPI == FK_EPILOGUE_GELU_ERF) return gelu_erf_f<float>(x);
  return x;
}

// ---------------------------------------------------------------- rows held in registers

// Two values at a time (packed fp32 arithmetic).
template <int EPI>
__device__ __forceinline__ float2 act2(float2 x) {
  if constexpr (EPI == FK_EPILOGUE_GELU_TANH) return gelu_tanh_f2<float>(x);
  if constexpr (EPI == FK_EPILOGUE_GELU_ERF) return gelu_erf_f2<float>(x);
  return x;
}

template <typename T, int OUT, int EPI, int EPT, bool ALIGNED, bool WARP, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) quantize_row_kernel(const __grid_constant__ QuantizeArgs a) {
  constexpr int VEC = Elem<T>::VEC, VPT = EPT / VEC;
  __shared__ float2 red[WARP ? 1 : MAXT / 32];
  let_next_start();
  after_previous();
  for_rows<WARP>(a.rows, static_cast<int>(a.cols), [&](size_t row, Place p) {
    const size_t base = row * a.cols;
    if (!ALIGNED) p.lead = lead_of(static_cast<const T*>(a.x) + base);
    uint4 raw[VPT];
    load_place<T, VPT, ALIGNED>(row_of(static_cast<const T*>(a.x), base, a.rows * a.cols), p, raw);
    mask_place<T, VPT, ALIGNED>(p, raw);
    float v[EPT], s = 0.0f, m = 0.0f;
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      Elem<T>::unpack(raw[c], v + c * VEC);
#pragma unroll
      for (int k = 0; k < VEC; k += 2) {
        const float2 z = act2<EPI>(make_float2(v[c * VEC + k], v[c * VEC + k + 1]));
        v[c * VEC + k] = z.x;
        v[c * VEC + k + 1] = z.y;
        m = absmax_nan(absmax_nan(m, z.x), z.y);
      }
    }
    team_sum_max<WARP>(s, m, red);
    const RowScale q = row_scale<OUT>(m);
    if (p.t == 0) a.scales[row] = q.scale;
#pragma unroll
    for (int c = 0; c < VPT; ++c)
      store_codes<T, OUT, ALIGNED>(static_cast<uint8_t*>(a.q) + base, p, c, v + c * VEC, q);
  });
}

// ---------------------------------------------------------------- streaming path

// One 512-thread block per row, which reads the row twice: the largest
// magnitude, then the codes.  Any length and alignment.
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
      o[j] = q.ok ? Code8<OUT>::pack1(act<EPI>(static_cast<float>(x[j])), q.inv) : 0;
    __syncthreads();  // red is rewritten by the next row
  }
}

template <typename T, int OUT, int EPI, bool ALIGNED>
cudaError_t launch_rows(const QuantizeArgs& a, cudaStream_t s) {
  const size_t span = row_span(a.cols, ALIGNED, Elem<T>::VEC);
  if (span <= kRowWarpCols) {
    const RowLaunch l = warp_launch(a.rows);
    if (span <= kRowWarpCols / 4)
      return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 8, ALIGNED, true, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    else if (span <= kRowWarpCols / 2)
      return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 16, ALIGNED, true, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    else
      return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, true, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
  } else if (span <= kRowSmallCols) {
    constexpr int EPT = 4 * Elem<T>::VEC;
    const RowLaunch l = block_launch(a.rows, span, EPT);
    return launch_overlapped(quantize_row_kernel<T, OUT, EPI, EPT, ALIGNED, false, 512, 2>, l.grid, l.threads, 0, 1, s, a);
  } else if (span <= kRowLargeCols) {
    const RowLaunch l = block_launch(a.rows, span, 32);
    return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, false, 512, 2>, l.grid, l.threads, 0, 1, s, a);
  } else {
    const RowLaunch l = block_launch(a.rows, span, 32);
    return launch_overlapped(quantize_row_kernel<T, OUT, EPI, 32, ALIGNED, false, 1024, 1>, l.grid, l.threads, 0, 1, s, a);
  }
}

template <typename T, int OUT, int EPI>
cudaError_t launch_epi(const QuantizeArgs& a, cudaStream_t s) {
  if (row_span(a.cols, a.mode == kRowsAligned, Elem<T>::VEC) > kRowMaxCols) {
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
