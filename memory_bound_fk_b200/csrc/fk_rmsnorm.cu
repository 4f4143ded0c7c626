// fk_rmsnorm.cu -- residual addition and root-mean-square norm over rows,
// the result in the input's type or in 8 bits with a scale per row (sm_100a).
//
//     h = x + residual (rounded to the rows' type),
//     v_j = h_j rstd gamma_j,  rstd = 1 / sqrt(sum h^2 / cols + eps).
// For 8-bit outputs max_j |v_j| = rstd max_j |h_j gamma_j|, so the sum of
// squares and that maximum come out of one pass and one reduction.
#include <cuda_bf16.h>

#include "fk_common.cuh"
#include "fk_q8.cuh"
#include "fk_q8_internal.h"

namespace fk {
namespace {

constexpr int kStreamThreads = 512;
constexpr size_t kMaxGrid = 0x7fffffffu;

// One value of the sum, rounded to the rows' type.
template <typename T>
__device__ __forceinline__ float round_to(float v) {
  if constexpr (sizeof(T) == 4) return v;
  return __bfloat162float(__float2bfloat16_rn(v));
}

// ---------------------------------------------------------------- streaming path

// One 512-thread block per row, which reads the row twice: statistics (and
// h stored), then the outputs.  Any length and alignment.  Plain loads: the
// second pass re-reads h where it was stored, which may be x or residual.
template <typename T, int OUT>
__global__ void __launch_bounds__(kStreamThreads) rmsnorm_stream_kernel(RmsnormArgs a) {
  constexpr bool Q8 = OUT == FK_I8 || OUT == FK_E4M3;
  __shared__ float2 red[kStreamThreads / 32];
  const size_t cols = a.cols;
  const float inv_n = 1.0f / static_cast<float>(cols);
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * cols;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * cols : nullptr;
    T* h = a.h ? static_cast<T*>(a.h) + row * cols : nullptr;
    float s = 0.0f, m = 0.0f;
    for (size_t j = threadIdx.x; j < cols; j += kStreamThreads) {
      float f = static_cast<float>(x[j]);
      if (r) f = round_to<T>(f + static_cast<float>(r[j]));
      if (h) h[j] = static_cast<T>(f);
      s = fmaf(f, f, s);
      if (Q8) m = absmax_nan(m, a.gamma ? f * a.gamma[j] : f);
    }
    block_sum_max<kStreamThreads / 32>(s, m, red);
    const float rstd = rms_rstd(s, inv_n, a.eps);
    RowScale q;
    if constexpr (Q8) {
      q = row_scale<OUT>(m * rstd);
      if (threadIdx.x == 0) a.scales[row] = q.scale;
    }
    // a thread re-reads only what it wrote itself
    for (size_t j = threadIdx.x; j < cols; j += kStreamThreads) {
      float f;
      if (h) {
        f = static_cast<float>(h[j]);
      } else {
        f = static_cast<float>(x[j]);
        if (r) f = round_to<T>(f + static_cast<float>(r[j]));
      }
      const float v = (a.gamma ? f * a.gamma[j] : f) * rstd;
      if constexpr (Q8) {
        static_cast<uint8_t*>(a.y)[row * cols + j] = q.ok ? Code8<OUT>::pack1(v, q.inv) : 0;
      } else {
        static_cast<T*>(a.y)[row * cols + j] = static_cast<T>(v);
      }
    }
    __syncthreads();  // red is rewritten by the next row
  }
}

template <typename T, int OUT>
cudaError_t launch_out(const RmsnormArgs& a, cudaStream_t s) {
  const unsigned g = static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid);
  rmsnorm_stream_kernel<T, OUT><<<g, kStreamThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_type(const RmsnormArgs& a, cudaStream_t s) {
  switch (a.out_dtype) {
    case FK_I8: return launch_out<T, FK_I8>(a, s);
    case FK_E4M3: return launch_out<T, FK_E4M3>(a, s);
    default: return launch_out<T, FK_F32>(a, s);  // the rows' own type
  }
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsnormArgs& a, cudaStream_t stream) {
  return a.dtype == FK_F32 ? launch_type<float>(a, stream) : launch_type<__nv_bfloat16>(a, stream);
}

}  // namespace fk
