// fk_q8_internal.h -- host-side interfaces between the C ABI of the 8-bit
// linear layer (fk_q8_api.cu) and its kernel launchers.  Not installed.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "fk_internal.h"
#include "fk_q8.h"

namespace fk {

// Is [p, p + bytes) memory that the current device may access, wholly inside
// one allocation (or the mapped part of one reservation)?  (p not NULL, aligned to `align`; also checks that the
// device is a B200.)
fk_status validate_span(const void* p, size_t bytes, size_t align);

// Keep a CUDA error for fk_last_cuda_error and answer FK_ERR_CUDA (FK_OK for
// cudaSuccess).
fk_status report_cuda(cudaError_t e);

// Launch a kernel that calls after_previous() before it touches global
// memory: its start (launch latency, barriers, tensor memory) overlaps the
// end of the kernel before it in the stream.  cluster: blocks per cluster.
template <typename... KArgs, typename... Args>
cudaError_t launch_overlapped(void (*kernel)(KArgs...), unsigned grid, unsigned threads, size_t smem,
                              unsigned cluster, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- RMSNorm ---------------------------------------------------------------
// How rows lie in memory: every row on a 16-byte boundary; rows shifted
// against such boundaries, but alike in every buffer of their type; or
// anything else (streamed one value at a time).
enum RowMode { kRowsAligned, kRowsShifted, kRowsAny };

// Validated arguments of fk_rmsnorm_rows.
struct RmsnormArgs {
  const void* x;
  const void* residual;  // or nullptr
  const float* gamma;    // or nullptr
  void* y;
  float* scales;  // 8-bit outputs only
  void* h;        // or nullptr
  size_t rows, cols;
  int dtype, out_dtype;
  float eps;
  RowMode mode;
};
cudaError_t launch_rmsnorm(const RmsnormArgs& a, cudaStream_t stream);

struct RmsnormBwdArgs {
  const void* dy;
  const void* h;
  const float* gamma;
  const void* dres;
  void* dx;
  float* dgamma;
  size_t rows, cols;
  int dtype;
  float eps;
  RowMode mode;
};
size_t rmsnorm_bwd_workspace(size_t rows, size_t cols, int dtype, bool want_dgamma, RowMode mode);
size_t rmsnorm_bwd_workspace(size_t rows, size_t cols, int dtype, bool want_dgamma);  // the most of any mode
cudaError_t launch_rmsnorm_bwd(const RmsnormBwdArgs& a, void* ws, cudaStream_t stream);

// ---- rows to 8 bits ----------------------------------------------------------
struct QuantizeArgs {
  const void* x;
  void* q;
  float* scales;
  size_t rows, cols;
  int dtype, out_dtype, epilogue;
  RowMode mode;
};
cudaError_t launch_quantize(const QuantizeArgs& a, cudaStream_t stream);

// ---- 8-bit matrix product ----------------------------------------------------
struct MatmulQ8Args {
  const void* a;
  const void* b;
  const float* a_scales;
  const float* b_scales;
  const float* bias;  // or nullptr
  void* c;
  size_t m, n, k;
  int dtype, out_dtype, epilogue;
  bool give_up;  // self-test: the wait for the finished product gives up at once
};
// `aligned`: a and b on 16-byte boundaries.
size_t matmul_q8_workspace(size_t m, size_t n, size_t k, bool aligned);
cudaError_t launch_matmul_q8(const MatmulQ8Args& a, void* ws, int sm_count, cudaStream_t stream);
cudaError_t read_matmul_wait_timeouts(unsigned* out, bool reset);

}  // namespace fk
