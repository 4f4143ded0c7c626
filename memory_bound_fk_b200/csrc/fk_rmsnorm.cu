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
#include "fk_q8_rows.cuh"

namespace fk {
namespace {

constexpr int kStreamThreads = 512;
constexpr size_t kMaxGrid = 0x7fffffffu;

// ---------------------------------------------------------------- rows held in registers

// One team per row: it is read, kept, reduced and written (fk_q8_rows.cuh).
// Bound by HBM; measured on B200, event overhead taken off: 16384 x 4096
// bf16 + residual to e4m3 and h 73 us (6.4 TB/s), to bf16 82 (6.6 TB/s), the
// same in fp32 159 (6.8 TB/s); 4096 x 16384 bf16 to e4m3 77; one row of 4096
// 2.7 us.  Clusters that share a row, and 16 values a thread in place of 32,
// were slower.
// MAXT, MINB: threads and blocks per SM the registers are sized for (64 a
// thread for 1024 threads on an SM).
template <typename T, int OUT, int EPT, bool ALIGNED, int LANES, int MAXT, int MINB, int CL = 1>
__global__ void __launch_bounds__(MAXT, MINB) rmsnorm_row_kernel(const __grid_constant__ RmsnormArgs a) {
  constexpr bool Q8 = OUT == FK_I8 || OUT == FK_E4M3;
  constexpr int VEC = Elem<T>::VEC, VPT = EPT / VEC;
  constexpr bool RELAXED = CL > 1 && sizeof(T) == 2;
  __shared__ float2 red[LANES ? 1 : CL * (MAXT / 32)];
  const float inv_n = 1.0f / static_cast<float>(a.cols);
  let_next_start();
  after_previous();
  for_rows<LANES, CL>(a.rows, static_cast<int>(a.cols), [&](size_t row, int t, int team, int cols) {
    const size_t base = row * a.cols;
    const T* const x = static_cast<const T*>(a.x) + base;
    const T* const res = static_cast<const T*>(a.residual) + base;
    T* const h = static_cast<T*>(a.h) + base;
    const Place p = place_of<T, ALIGNED>(t, team, cols, x);
    const int edge = ALIGNED ? -1 : edge_col<VEC>(p);
    uint4 raw[VPT];
    load_vecs<T, VPT, RELAXED>(x, p, raw);
    float ev = 0.0f, er = 0.0f;  // this thread's value outside the vectors
    if (!ALIGNED && edge >= 0) ev = load_one(x + edge);
    if (a.residual) {
      // at most 16 fp32 values of the residual at a time: with all 32 beside
      // those of x a thread spills
      constexpr int PART = sizeof(T) == 4 && EPT == 32 ? VPT / 2 : VPT;
      if (!ALIGNED && edge >= 0) er = load_one(res + edge);
#pragma unroll
      for (int from = 0; from < VPT; from += PART) {
        uint4 add[PART];
        load_vecs<T, PART, RELAXED>(res, p, add, from);
#pragma unroll
        for (int c = from; c < from + PART; ++c) {
          float f[VEC], r[VEC];
          Elem<T>::unpack(raw[c], f);
          Elem<T>::unpack(add[c - from], r);
#pragma unroll
          for (int k = 0; k < VEC; ++k) f[k] += r[k];
          raw[c] = Elem<T>::pack(f);  // h, rounded to the rows' type: what is normalised is what is stored
          if (a.h) store_vec(h, p, c, raw[c]);
        }
      }
      if (!ALIGNED && edge >= 0) {
        ev = round_one<T>(ev + er);
        if (a.h) Elem<T>::store1(h + edge, ev);
      }
    }
    float v[EPT], s = 0.0f, m = 0.0f;
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      float g[VEC];
      Elem<T>::unpack(raw[c], v + c * VEC);
      load_params<VEC, ALIGNED>(a.gamma, p, c, g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        float& f = v[c * VEC + k];
        s = fmaf(f, f, s);
        f *= g[k];
        if (Q8) m = absmax_nan(m, f);
      }
    }
    if (!ALIGNED && edge >= 0) {
      s = fmaf(ev, ev, s);
      if (a.gamma) ev *= ld_param(a.gamma + edge);
      if (Q8) m = absmax_nan(m, ev);
    }
    if constexpr (CL > 1)
      cluster_sum_max<CL>(s, m, red);
    else
      team_sum_max<LANES>(s, m, red);
    const float rstd = rms_rstd(s, inv_n, a.eps);
    RowScale q;
    if constexpr (Q8) {
      q = row_scale<OUT>(m * rstd);
      if (t == 0 && cols > 0) a.scales[row] = q.scale;
    }
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      float o[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) o[k] = v[c * VEC + k] * rstd;
      if constexpr (Q8)
        store_codes<T, OUT, ALIGNED>(static_cast<uint8_t*>(a.y) + base, p, c, o, q);
      else
        store_vec(static_cast<T*>(a.y) + base, p, c, Elem<T>::pack(o));
    }
    if (!ALIGNED && edge >= 0) {
      if constexpr (Q8)
        (static_cast<uint8_t*>(a.y) + base)[edge] = q.ok ? Code8<OUT>::pack1(ev * rstd, q) : 0;
      else
        Elem<T>::store1(static_cast<T*>(a.y) + base + edge, ev * rstd);
    }
  });
}

// ---------------------------------------------------------------- streaming path

// One 512-thread block per row, which reads the row twice: statistics (and
// h stored), then the outputs.  Any length and alignment.  Plain loads: the
// second pass re-reads h where it was stored, which may be x or residual.
// Value by value, for rows past 131072 columns and buffers that lie
// differently to 16 bytes: 1024 x 49152 bf16 + residual to bf16 220 us.
template <typename T, int OUT>
__global__ void __launch_bounds__(kStreamThreads) rmsnorm_stream_kernel(RmsnormArgs a) {
  constexpr bool Q8 = OUT == FK_I8 || OUT == FK_E4M3;
  __shared__ float2 red[kStreamThreads / 32];
  const size_t cols = a.cols;
  const float inv_n = 1.0f / static_cast<float>(cols);
  let_next_start();
  after_previous();
  for (size_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * cols;
    const T* r = a.residual ? static_cast<const T*>(a.residual) + row * cols : nullptr;
    T* h = a.h ? static_cast<T*>(a.h) + row * cols : nullptr;
    float s = 0.0f, m = 0.0f;
    for (size_t j = threadIdx.x; j < cols; j += kStreamThreads) {
      float f = static_cast<float>(x[j]);
      if (r) f = round_one<T>(f + static_cast<float>(r[j]));
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
        if (r) f = round_one<T>(f + static_cast<float>(r[j]));
      }
      const float v = (a.gamma ? f * a.gamma[j] : f) * rstd;
      if constexpr (Q8) {
        static_cast<uint8_t*>(a.y)[row * cols + j] = q.ok ? Code8<OUT>::pack1(v, q) : 0;
      } else {
        static_cast<T*>(a.y)[row * cols + j] = static_cast<T>(v);
      }
    }
    __syncthreads();  // red is rewritten by the next row
  }
}

template <typename T, int OUT, bool ALIGNED>
cudaError_t launch_rows(const RmsnormArgs& a, cudaStream_t s) {
  if (a.cols <= kRowWarpCols) {
    const int lanes = row_lanes(a.cols, ALIGNED, Elem<T>::VEC);
    const RowLaunch l = warp_launch(a.rows, lanes);
    if (lanes == 8)
      return launch_overlapped(rmsnorm_row_kernel<T, OUT, kRowLaneEpt, ALIGNED, 8, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    if (lanes == 16)
      return launch_overlapped(rmsnorm_row_kernel<T, OUT, kRowLaneEpt, ALIGNED, 16, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    if (a.cols <= kRowWarpCols / 4)
      return launch_overlapped(rmsnorm_row_kernel<T, OUT, 8, ALIGNED, 32, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    if (a.cols <= kRowWarpCols / 2)
      return launch_overlapped(rmsnorm_row_kernel<T, OUT, 16, ALIGNED, 32, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
    return launch_overlapped(rmsnorm_row_kernel<T, OUT, 32, ALIGNED, 32, 32 * kRowWarps, 4>, l.grid, l.threads, 0, 1, s, a);
  }
  if (a.cols <= kRowBlockCols) {
    constexpr int EPT = 4 * Elem<T>::VEC;
    const RowLaunch l = block_launch(a.rows, a.cols, EPT);
    return launch_overlapped(rmsnorm_row_kernel<T, OUT, EPT, ALIGNED, 0, 512, 2>, l.grid, l.threads, 0, 1, s, a);
  }
  const RowLaunch l = block_launch(a.rows, a.cols, 32);
  if (a.cols <= kRowLargeCols)
    return launch_overlapped(rmsnorm_row_kernel<T, OUT, 32, ALIGNED, 0, 512, 2>, l.grid, l.threads, 0, 1, s, a);
  if (a.cols <= kRowMaxCols)
    return launch_overlapped(rmsnorm_row_kernel<T, OUT, 32, ALIGNED, 0, 1024, 1>, l.grid, l.threads, 0, 1, s, a);
  // 4 or 8 blocks of 512 threads (1024 x 65536 bf16 + residual to bf16 104 us,
  // 1024 x 131072 236; 2 or 4 of 1024: 115 and 265)
  const int cl = a.cols <= kRowClusterCols / 2 ? 4 : 8;
  const RowLaunch c = cluster_launch(a.rows, a.cols, cl);
  return cl == 4 ? launch_overlapped(rmsnorm_row_kernel<T, OUT, 32, ALIGNED, 0, 512, 2, 4>, c.grid, c.threads, 0, 4, s, a)
                 : launch_overlapped(rmsnorm_row_kernel<T, OUT, 32, ALIGNED, 0, 512, 2, 8>, c.grid, c.threads, 0, 8, s, a);
}

template <typename T, int OUT>
cudaError_t launch_out(const RmsnormArgs& a, cudaStream_t s) {
  if (a.mode == kRowsAny || a.cols > kRowClusterCols) {
    const unsigned g = static_cast<unsigned>(a.rows < kMaxGrid ? a.rows : kMaxGrid);
    return launch_overlapped(rmsnorm_stream_kernel<T, OUT>, g, kStreamThreads, 0, 1, s, a);
  }
  return a.mode == kRowsAligned ? launch_rows<T, OUT, true>(a, s) : launch_rows<T, OUT, false>(a, s);
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
