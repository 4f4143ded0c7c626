// fk_rmsnorm_bwd.cu -- gradients of the root-mean-square norm (sm_100a).
//
// With r = 1 / sqrt(sum h^2 / cols + eps) and s = sum dy gamma h / cols:
//     dx_j     = r dy_j gamma_j - r^3 s h_j (+ dres_j),
//     dgamma_j = sum_rows dy_j h_j r.
// dgamma is summed in two steps whose order depends on the shape alone:
// partial sums over groups of rows into workspace, then over the groups.
#include <cuda_bf16.h>

#include "fk_common.cuh"
#include "fk_q8.cuh"
#include "fk_q8_internal.h"

namespace fk {
namespace {

constexpr int kStreamThreads = 512;
constexpr size_t kMaxGrid = 0x7fffffffu;
constexpr int kColThreads = 128;      // columns per block of the column sums
constexpr size_t kStreamGroups = 64;  // groups of rows on the streaming path

// ---------------------------------------------------------------- streaming path

// Row statistics: (r, r^3 s) of every row, one block per row.
template <typename T>
__global__ void __launch_bounds__(kStreamThreads) rmsnorm_bwd_stats_kernel(RmsnormBwdArgs a, float2* stats) {
  __shared__ float2 red[kStreamThreads / 32];
  const size_t cols = a.cols;
  const float inv_n = 1.0f / static_cast<float>(cols);
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(a.dy) + row * cols;
    const T* h = static_cast<const T*>(a.h) + row * cols;
    float s = 0.0f, d = 0.0f;
    for (size_t j = threadIdx.x; j < cols; j += kStreamThreads) {
      const float f = static_cast<float>(h[j]), g = static_cast<float>(dy[j]);
      s = fmaf(f, f, s);
      d = fmaf(a.gamma ? g * a.gamma[j] : g, f, d);
    }
    s = warp_sum(s);
    d = warp_sum(d);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(s, d);
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kStreamThreads / 32; ++w) {
        s += red[w].x;
        d += red[w].y;
      }
      const float r = rms_rstd(s, inv_n, a.eps);
      stats[row] = make_float2(r, r * r * r * (d * inv_n));
    }
    __syncthreads();  // red is rewritten by the next row
  }
}

// Partial column sums of dy h r over one group of rows (blockIdx.y).
template <typename T>
__global__ void __launch_bounds__(kColThreads)
    rmsnorm_bwd_cols_kernel(RmsnormBwdArgs a, const float2* stats, float* partial, size_t group_rows) {
  const size_t j = static_cast<size_t>(blockIdx.x) * kColThreads + threadIdx.x;
  if (j >= a.cols) return;
  const size_t r0 = blockIdx.y * group_rows;
  const size_t r1 = r0 + group_rows < a.rows ? r0 + group_rows : a.rows;
  float acc = 0.0f;
  for (size_t r = r0; r < r1; ++r) {
    const size_t i = r * a.cols + j;
    acc = fmaf(static_cast<float>(static_cast<const T*>(a.dy)[i]) * static_cast<float>(static_cast<const T*>(a.h)[i]),
               stats[r].x, acc);
  }
  partial[blockIdx.y * a.cols + j] = acc;
}

// dgamma_j = sum of the groups' partial sums, in order.
__global__ void __launch_bounds__(kColThreads)
    rmsnorm_bwd_join_kernel(const float* partial, float* dgamma, size_t cols, size_t groups) {
  const size_t j = static_cast<size_t>(blockIdx.x) * kColThreads + threadIdx.x;
  if (j >= cols) return;
  float acc = 0.0f;
  for (size_t g = 0; g < groups; ++g) acc += partial[g * cols + j];
  dgamma[j] = acc;
}

// dx, elementwise once the statistics stand (after the column sums have read
// dy and h: dx may be either).
template <typename T>
__global__ void __launch_bounds__(kStreamThreads) rmsnorm_bwd_dx_kernel(RmsnormBwdArgs a, const float2* stats) {
  const size_t cols = a.cols;
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float2 st = stats[row];
    const size_t base = row * cols;
    for (size_t j = threadIdx.x; j < cols; j += kStreamThreads) {
      const size_t i = base + j;
      const float f = static_cast<float>(static_cast<const T*>(a.h)[i]);
      float g = static_cast<float>(static_cast<const T*>(a.dy)[i]);
      if (a.gamma) g *= a.gamma[j];
      float v = fmaf(st.x, g, -st.y * f);
      if (a.dres) v += static_cast<float>(static_cast<const T*>(a.dres)[i]);
      static_cast<T*>(a.dx)[i] = static_cast<T>(v);
    }
  }
}

size_t stream_groups(size_t rows) { return rows < kStreamGroups ? rows : kStreamGroups; }
size_t stats_bytes(size_t rows) { return (rows * sizeof(float2) + 15) / 16 * 16; }

template <typename T>
cudaError_t launch_stream(const RmsnormBwdArgs& a, void* ws, cudaStream_t s) {
  float2* stats = static_cast<float2*>(ws);
  float* partial = reinterpret_cast<float*>(static_cast<char*>(ws) + stats_bytes(a.rows));
  const unsigned g = static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid);
  rmsnorm_bwd_stats_kernel<T><<<g, kStreamThreads, 0, s>>>(a, stats);
  if (a.dgamma) {
    const size_t groups = stream_groups(a.rows), per = (a.rows + groups - 1) / groups;
    const size_t used = (a.rows + per - 1) / per;
    const size_t blocks = (a.cols + kColThreads - 1) / kColThreads;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(used));
    rmsnorm_bwd_cols_kernel<T><<<grid, kColThreads, 0, s>>>(a, stats, partial, per);
    rmsnorm_bwd_join_kernel<<<grid.x, kColThreads, 0, s>>>(partial, a.dgamma, a.cols, used);
  }
  rmsnorm_bwd_dx_kernel<T><<<g, kStreamThreads, 0, s>>>(a, stats);
  return cudaGetLastError();
}

}  // namespace

size_t rmsnorm_bwd_workspace(size_t rows, size_t cols, int dtype, bool want_dgamma) {
  (void)dtype;
  return stats_bytes(rows) + (want_dgamma ? stream_groups(rows) * cols * sizeof(float) : 0);
}

cudaError_t launch_rmsnorm_bwd(const RmsnormBwdArgs& a, void* ws, cudaStream_t stream) {
  return a.dtype == FK_F32 ? launch_stream<float>(a, ws, stream) : launch_stream<__nv_bfloat16>(a, ws, stream);
}

}  // namespace fk
