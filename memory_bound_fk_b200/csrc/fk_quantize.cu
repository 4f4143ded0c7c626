// fk_quantize.cu -- rows to 8 bits with one scale each, optionally through
// GELU (sm_100a).
#include <cuda_bf16.h>

#include "fk_common.cuh"
#include "fk_gelu.cuh"
#include "fk_q8.cuh"
#include "fk_q8_internal.h"

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

// ---------------------------------------------------------------- streaming path

// One 512-thread block per row, which reads the row twice: the largest
// magnitude, then the codes.  Any length and alignment.
template <typename T, int OUT, int EPI>
__global__ void __launch_bounds__(kStreamThreads) quantize_stream_kernel(QuantizeArgs a) {
  __shared__ float2 red[kStreamThreads / 32];
  const size_t cols = a.cols;
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

template <typename T, int OUT, int EPI>
cudaError_t launch_epi(const QuantizeArgs& a, cudaStream_t s) {
  const unsigned g = static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid);
  quantize_stream_kernel<T, OUT, EPI><<<g, kStreamThreads, 0, s>>>(a);
  return cudaGetLastError();
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
