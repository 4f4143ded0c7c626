// fk_rmsnorm_bwd.cu -- gradients of the root-mean-square norm (sm_100a).
//
// With r = 1 / sqrt(sum h^2 / cols + eps) and s = sum dy gamma h / cols:
//     dx_j     = r dy_j gamma_j - r^3 s h_j (+ dres_j)
//              = r (dy_j gamma_j - (r^2 s) h_j) (+ dres_j),
//     dgamma_j = sum_rows dy_j h_j r.
// The second form is what is computed: r^3 leaves fp32's range for rows of
// about 1e-13 (with eps as small), r (r s) stays of the size of dy / h.
// dgamma is summed in two steps whose order depends on the shape alone:
// partial sums over groups of rows into workspace, then over the groups.
#include <cuda_bf16.h>

#include "fk_common.cuh"
#include "fk_q8.cuh"
#include "fk_q8_internal.h"
#include "fk_q8_rows.cuh"
#include "fk_sync.cuh"

namespace fk {
namespace {

constexpr int kStreamThreads = 512;
constexpr size_t kMaxGrid = 0x7fffffffu;
constexpr int kColThreads = 128;      // columns per block of the column sums
constexpr int kJoinCols = 32, kJoinWays = 32;
constexpr int kBwdThreads = 512;      // of a block whose rows are staged, at most
constexpr int kBwdMaxCols = 65536;    // longer rows are streamed
// Blocks per SM of warp teams with 8 values a lane (registers follow): 200000 x
// 64 fp32 29 us at three and 35 at four, 100000 x 128 bf16 27 and 25.
constexpr int small_blocks(int vec) { return vec == 8 ? 4 : 3; }
constexpr int kSmCount = 148;
constexpr size_t kStreamGroups = 64;  // groups of rows on the streaming path

// ---------------------------------------------------------------- rows held in registers

// Rows of up to 1024 columns: blocks that stay on the GPU and walk the rows,
// LANES lanes of a warp to a row, so that a thread's columns never change:
// gamma and the running dgamma sums live in its registers.  The next row's h
// and dy are loaded before the current one is reduced, which keeps HBM busy
// through the reduction.  At the end each block adds its warps' sums in order
// and writes them, one row of workspace per block.  Bound by HBM; measured
// on B200: 200000 x 64 fp32 with dres 37 us (5.6 TB/s), 20000 x 1024 fp32 55
// (5.9), 20000 x 1024 bf16 32 (5.2).
template <typename T, int EPT, bool ALIGNED, int LANES>
__global__ void __launch_bounds__(32 * kRowWarps, EPT == 32 ? 1 : EPT == 16 ? 2 : small_blocks(Elem<T>::VEC))
    rmsnorm_bwd_row_kernel(const __grid_constant__ RmsnormBwdArgs a, float* partial) {
  constexpr int VEC = Elem<T>::VEC, VPT = EPT / VEC;
  constexpr int PER = 32 / LANES;  // rows a warp takes at a time
  const int cols = static_cast<int>(a.cols);
  const float inv_n = 1.0f / static_cast<float>(cols);
  const int warps = static_cast<int>(blockDim.x >> 5), warp = static_cast<int>(threadIdx.x >> 5);
  const int lane = static_cast<int>(threadIdx.x & 31);
  const size_t team = (static_cast<size_t>(blockIdx.x) * warps + warp) * PER + lane / LANES;
  const size_t stride = static_cast<size_t>(gridDim.x) * warps * PER;
  const T* const h = static_cast<const T*>(a.h);
  const T* const dy = static_cast<const T*>(a.dy);
  const T* const dres = static_cast<const T*>(a.dres);
  // shifted rows: a team's rows are a multiple of eight apart (or it has one),
  // so that all of them start alike
  const Place p = place_of<T, ALIGNED>(lane % LANES, LANES, cols, h + team * a.cols);
  const int edge = ALIGNED ? -1 : edge_col<VEC>(p);
  let_next_start();
  after_previous();
  float gam[EPT], acc[EPT];
  float eg = 1.0f, ea = 0.0f, eh = 0.0f, ed = 0.0f;  // gamma, sum, h and dy of this thread's column outside the vectors
  if (!ALIGNED && edge >= 0 && a.gamma) eg = ld_param(a.gamma + edge);
#pragma unroll
  for (int c = 0; c < VPT; ++c) load_params<VEC, ALIGNED>(a.gamma, p, c, gam + c * VEC);
#pragma unroll
  for (int i = 0; i < EPT; ++i) acc[i] = 0.0f;
  uint4 rh[VPT], rd[VPT];
#pragma unroll
  for (int c = 0; c < VPT; ++c) rh[c] = rd[c] = make_uint4(0u, 0u, 0u, 0u);
  if (team < a.rows) {
    load_vecs<T, VPT>(h + team * a.cols, p, rh);
    load_vecs<T, VPT>(dy + team * a.cols, p, rd);
    if (!ALIGNED && edge >= 0) {
      eh = load_one(h + team * a.cols + edge);
      ed = load_one(dy + team * a.cols + edge);
    }
  }
  // (a warp's teams go on together until the last of them has no row left)
  for (size_t row = team; row - lane / LANES < a.rows; row += stride) {
    const size_t base = row * a.cols, next = base + stride * a.cols;
    const bool live = row < a.rows;
    uint4 nh[VPT], nd[VPT], rr[VPT];
    float neh = 0.0f, ned = 0.0f, er = 0.0f;
    if (a.dres && live) {
      load_vecs<T, VPT>(dres + base, p, rr);
      if (!ALIGNED && edge >= 0) er = load_one(dres + base + edge);
    }
    if (row + stride < a.rows) {
      load_vecs<T, VPT>(h + next, p, nh);
      load_vecs<T, VPT>(dy + next, p, nd);
      if (!ALIGNED && edge >= 0) {
        neh = load_one(h + next + edge);
        ned = load_one(dy + next + edge);
      }
    }
    float s = 0.0f, d = 0.0f;
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      float f[VEC], g[VEC];
      Elem<T>::unpack(rh[c], f);
      Elem<T>::unpack(rd[c], g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        s = fmaf(f[k], f[k], s);
        d = fmaf(g[k] * gam[c * VEC + k], f[k], d);
      }
    }
    if (!ALIGNED && edge >= 0) {
      s = fmaf(eh, eh, s);
      d = fmaf(ed * eg, eh, d);
    }
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      d += __shfl_xor_sync(0xffffffffu, d, o);
    }
    const float r = rms_rstd(s, inv_n, a.eps);
    const float r2s = r * (r * (d * inv_n));
    if (!live) break;
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      float f[VEC], g[VEC], o[VEC];
      Elem<T>::unpack(rh[c], f);
      Elem<T>::unpack(rd[c], g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        acc[c * VEC + k] = fmaf(g[k] * f[k], r, acc[c * VEC + k]);
        o[k] = r * fmaf(-r2s, f[k], g[k] * gam[c * VEC + k]);
      }
      if (a.dres) {
        float q[VEC];
        Elem<T>::unpack(rr[c], q);
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] += q[k];
      }
      store_vec(static_cast<T*>(a.dx) + base, p, c, Elem<T>::pack(o));
      rh[c] = nh[c];
      rd[c] = nd[c];
    }
    if (!ALIGNED && edge >= 0) {
      ea = fmaf(ed * eh, r, ea);
      Elem<T>::store1(static_cast<T*>(a.dx) + base + edge, r * fmaf(-r2s, eh, ed * eg) + er);
      eh = neh;
      ed = ned;
    }
  }
  if (partial == nullptr) return;
  float* out = partial + static_cast<size_t>(blockIdx.x) * a.cols;
  __shared__ float sums[kRowWarps * PER][LANES * EPT];
  float* const mine = sums[threadIdx.x / LANES];
#pragma unroll
  for (int c = 0; c < VPT; ++c)
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (has_vec(p, c)) mine[col_of_vec<VEC>(p, c) + k] = acc[c * VEC + k];
  if (!ALIGNED && edge >= 0) mine[edge] = ea;
  __syncthreads();
  for (int e = threadIdx.x; e < cols; e += blockDim.x) {
    float v = sums[0][e];
    for (int w = 1; w < warps * PER; ++w) v += sums[w][e];
    out[e] = v;
  }
}

// ---------------------------------------------------------------- rows staged in shared memory

// 16 bytes from global to shared memory without registers (past L1 where
// ALIGNED); zeros when !on (nothing is read then).
template <bool ALIGNED>
__device__ __forceinline__ void copy16_async(uint4* dst, const void* src, bool on) {
  if constexpr (ALIGNED)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(on ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last committed group of this thread's copies have landed (or all).
__device__ __forceinline__ void copies_wait_but_one() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }


// Longer rows: blocks that stay and walk the rows, as above, a row's h, dy
// and dres waiting in shared memory, two rows at a time.  A thread fills and
// reads only its own slots (copies that pass the registers by, two rows
// ahead), so the one barrier of a row is that of its sums.  CL blocks of a
// cluster share a row.
//
// Bound by HBM.  Measured on B200 (64M values, h, dy and dres in, dx out,
// event overhead and the second step of dgamma included): bf16 4096 columns
// 85.5 us (6.3 TB/s; with the next row prefetched into registers instead
// 90.5), 8192 columns 90 (93), 16384 columns 100 (147, two blocks of a
// cluster); fp32 64M values of 8192 columns 167 (191: spills).  Shifted rows
// copy through L1 (.ca): past it, the boundaries between lanes' 16 bytes
// that are no sector boundaries are read twice (8191 columns fp32: 194 us
// against 207); bf16 4095 columns 112, 16383 146.
template <typename T, int EPT, bool ALIGNED, int CL>
__global__ void __launch_bounds__(kBwdThreads, 1)
    rmsnorm_bwd_staged_kernel(const __grid_constant__ RmsnormBwdArgs a, float* partial) {
  constexpr int VEC = Elem<T>::VEC, VPT = EPT / VEC;
  extern __shared__ uint4 slots[];  // [2 rows][h, dy (, dres)][vector][thread]
  __shared__ float2 red[2][CL * (kBwdThreads / 32)];
  const int cols = static_cast<int>(a.cols);
  const float inv_n = 1.0f / static_cast<float>(cols);
  const int warps = static_cast<int>(blockDim.x >> 5), warp = static_cast<int>(threadIdx.x >> 5);
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int rank = CL > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const size_t team = blockIdx.x / CL, stride = gridDim.x / CL;
  const T* const h = static_cast<const T*>(a.h);
  const T* const dy = static_cast<const T*>(a.dy);
  const T* const dres = static_cast<const T*>(a.dres);
  const int bufs = dres ? 3 : 2;
  // shifted rows: a team's rows are a multiple of eight apart (or it has one),
  // so that all of them start alike
  const Place p = place_of<T, ALIGNED>(static_cast<int>(rank * blockDim.x + threadIdx.x),
                                       static_cast<int>(CL * blockDim.x), cols, h + team * a.cols);
  const int edge = ALIGNED ? -1 : edge_col<VEC>(p);
  auto slot = [&](int st, int buf, int c) {
    return slots + ((st * bufs + buf) * VPT + c) * static_cast<int>(blockDim.x) + threadIdx.x;
  };
  auto fetch = [&](int st, size_t row, int c) {
    const bool on = row < a.rows && has_vec(p, c);
    const size_t at = on ? row * a.cols + col_of_vec<VEC>(p, c) : 0;
    copy16_async<ALIGNED>(slot(st, 0, c), h + at, on);
    copy16_async<ALIGNED>(slot(st, 1, c), dy + at, on);
    if (dres) copy16_async<ALIGNED>(slot(st, 2, c), dres + at, on);
  };
  let_next_start();
  after_previous();
  if constexpr (CL > 1) cluster_arrive_relaxed();  // every block has started: waited for before the first push
#pragma unroll
  for (int st = 0; st < 2; ++st) {
#pragma unroll
    for (int c = 0; c < VPT; ++c) fetch(st, team + st * stride, c);
    copies_commit();
  }
  float gam[EPT], acc[EPT];
  float eg = 1.0f, ea = 0.0f, eh = 0.0f, ed = 0.0f;  // gamma, sum, h and dy of this thread's column outside the vectors
  if (!ALIGNED && edge >= 0) {
    if (a.gamma) eg = ld_param(a.gamma + edge);
    if (team < a.rows) {
      eh = load_one(h + team * a.cols + edge);
      ed = load_one(dy + team * a.cols + edge);
    }
  }
#pragma unroll
  for (int c = 0; c < VPT; ++c) load_params<VEC, ALIGNED>(a.gamma, p, c, gam + c * VEC);
#pragma unroll
  for (int i = 0; i < EPT; ++i) acc[i] = 0.0f;
  if constexpr (CL > 1) cluster_wait();
  int st = 0;
  for (size_t row = team; row < a.rows; row += stride, st ^= 1) {
    const size_t base = row * a.cols, next = base + stride * a.cols;
    float neh = 0.0f, ned = 0.0f, er = 0.0f;
    if (!ALIGNED && edge >= 0) {
      if (dres) er = load_one(dres + base + edge);
      if (row + stride < a.rows) {
        neh = load_one(h + next + edge);
        ned = load_one(dy + next + edge);
      }
    }
    copies_wait_but_one();
    float s = 0.0f, d = 0.0f;
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      float f[VEC], g[VEC];
      Elem<T>::unpack(*slot(st, 0, c), f);
      Elem<T>::unpack(*slot(st, 1, c), g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        s = fmaf(f[k], f[k], s);
        d = fmaf(g[k] * gam[c * VEC + k], f[k], d);
      }
    }
    if (!ALIGNED && edge >= 0) {
      s = fmaf(eh, eh, s);
      d = fmaf(ed * eg, eh, d);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      d += __shfl_xor_sync(0xffffffffu, d, o);
    }
    if constexpr (CL > 1) {
      if (lane < CL) st_cluster_f2(cluster_addr(&red[st][rank * warps + warp], lane), s, d);
      cluster_barrier();
    } else {
      if (lane == 0) red[st][warp] = make_float2(s, d);
      __syncthreads();
    }
    s = red[st][0].x;
    d = red[st][0].y;
    for (int w = 1; w < CL * warps; ++w) {
      s += red[st][w].x;
      d += red[st][w].y;
    }
    const float r = rms_rstd(s, inv_n, a.eps);
    const float r2s = r * (r * (d * inv_n));
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      float f[VEC], g[VEC], o[VEC];
      Elem<T>::unpack(*slot(st, 0, c), f);
      Elem<T>::unpack(*slot(st, 1, c), g);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        acc[c * VEC + k] = fmaf(g[k] * f[k], r, acc[c * VEC + k]);
        o[k] = r * fmaf(-r2s, f[k], g[k] * gam[c * VEC + k]);
      }
      if (dres) {
        float q[VEC];
        Elem<T>::unpack(*slot(st, 2, c), q);
#pragma unroll
        for (int k = 0; k < VEC; ++k) o[k] += q[k];
      }
      store_vec(static_cast<T*>(a.dx) + base, p, c, Elem<T>::pack(o));
      fetch(st, row + 2 * stride, c);  // the slots have been read: what was stored came from them
    }
    copies_commit();
    if (!ALIGNED && edge >= 0) {
      ea = fmaf(ed * eh, r, ea);
      Elem<T>::store1(static_cast<T*>(a.dx) + base + edge, r * fmaf(-r2s, eh, ed * eg) + er);
      eh = neh;
      ed = ned;
    }
  }
  copies_wait();
  if (partial == nullptr) return;
  float* const out = partial + team * a.cols;
#pragma unroll
  for (int c = 0; c < VPT; ++c)
#pragma unroll
    for (int k = 0; k < VEC; ++k)
      if (has_vec(p, c)) out[col_of_vec<VEC>(p, c) + k] = acc[c * VEC + k];
  if (!ALIGNED && edge >= 0) out[edge] = ea;
}

// ---------------------------------------------------------------- streaming path

// Value by value, for rows past 65536 columns and buffers that lie
// differently to 16 bytes, in four kernels: dy and h are read three times
// (1024 x 49152 bf16 with dres: 315 us).
// Row statistics: (r, r^2 s) of every row, one block per row.
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
      stats[row] = make_float2(r, r * (r * (d * inv_n)));
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

// dgamma_j = sum of the groups' partial sums: 32 columns per block, every
// 32nd group to each of its 32 warps, the warps' sums added in order.  About
// 3 us behind the first step (4.8 MB of partial sums from L2 for 4096 columns).
__global__ void __launch_bounds__(kJoinCols* kJoinWays)
    rmsnorm_bwd_join_kernel(const float* partial, float* dgamma, size_t cols, size_t groups) {
  __shared__ float part[kJoinWays][kJoinCols];
  const int lane = threadIdx.x % kJoinCols, way = threadIdx.x / kJoinCols;
  const size_t j = static_cast<size_t>(blockIdx.x) * kJoinCols + lane;
  float acc = 0.0f;
  let_next_start();
  after_previous();
  if (j < cols) {
#pragma unroll 8
    for (size_t g = way; g < groups; g += kJoinWays) acc += partial[g * cols + j];
  }
  part[way][lane] = acc;
  __syncthreads();
  if (way == 0 && j < cols) {
#pragma unroll
    for (int w = 1; w < kJoinWays; ++w) acc += part[w][lane];
    dgamma[j] = acc;
  }
}

cudaError_t launch_join(const float* partial, float* dgamma, size_t cols, size_t groups, cudaStream_t s) {
  const size_t blocks = (cols + kJoinCols - 1) / kJoinCols;
  if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
  return launch_overlapped(rmsnorm_bwd_join_kernel, static_cast<unsigned>(blocks), kJoinCols * kJoinWays, 0, 1, s,
                           partial, dgamma, cols, groups);
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
      float v = st.x * fmaf(-st.y, f, g);
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
    const cudaError_t e = launch_join(partial, a.dgamma, a.cols, used, s);
    if (e != cudaSuccess) return e;
  }
  rmsnorm_bwd_dx_kernel<T><<<g, kStreamThreads, 0, s>>>(a, stats);
  return cudaGetLastError();
}

// How the kernel of resident teams is launched for a shape: blocks, threads,
// blocks per team, rows of partial sums.
struct BwdLaunch {
  int lanes, ept, cluster, threads;  // cluster: 0 for warp teams
  size_t blocks, groups;
};

// Teams stay resident: as many blocks as fit the registers.  Shifted rows:
// teams walk rows a multiple of eight apart.
BwdLaunch bwd_launch(size_t rows, size_t cols, int vec, bool shifted) {
  BwdLaunch l;
  if (cols <= static_cast<size_t>(kRowWarpCols)) {
    // a warp or less per row, 8 / 16 / 32 values a lane
    l.lanes = row_lanes(cols, !shifted, vec);
    l.ept = cols <= 256 ? 8 : cols <= 512 ? 16 : 32;
    l.cluster = 0;
    l.threads = 32 * kRowWarps;
    const size_t per = static_cast<size_t>(kRowWarps) * (32 / l.lanes);
    const size_t fit = kSmCount * (l.ept == 8 ? small_blocks(vec) : l.ept == 16 ? 2 : 1), want = (rows + per - 1) / per;
    l.blocks = l.groups = want < fit ? want : fit;
    return l;
  }
  // Values a thread: 16, or for bf16 32 where one block of 16 a thread would
  // leave its SM half empty (8192 rows, us for 16 / 32: 5120 columns 58 / 63,
  // 6144 75 / 68, 7168 80 / 80, 8192 90 / 97) and past 8192 columns (4096
  // rows: 10240 119 / 62, two blocks of a cluster against one).
  l.lanes = 0;
  l.cluster = 1;
  l.ept = vec == 4 || cols <= 5120 || (cols > 7168 && cols <= 8192) ? 16 : 32;
  while (static_cast<size_t>(l.cluster) * kBwdThreads * l.ept < cols) l.cluster *= 2;
  const size_t per = static_cast<size_t>(l.ept) * l.cluster;
  l.threads = static_cast<int>(((cols + per - 1) / per + 31) / 32 * 32);
  // 128 registers a thread leave 512 threads on an SM, the 96 of aligned bf16
  // at 16 values 640 (1088 columns: 33.6 us against 38.7 with 512)
  const int resident = vec == 8 && l.ept == 16 && !shifted ? 640 : 512;
  // (of the clusters of four 33 run at a time, of those of eight 15: a second wave took 180 us for
  // 1024 x 32768 fp32)
  const size_t fit = l.cluster == 1   ? kSmCount * (resident / l.threads)
                     : l.cluster == 2 ? kSmCount / 2
                     : l.cluster == 4 ? 33
                                      : 15;
  l.groups = rows < fit ? rows : shifted ? fit / 8 * 8 : fit;
  l.blocks = l.groups * l.cluster;
  return l;
}

template <typename T, int EPT, bool ALIGNED, int LANES>
cudaError_t launch_row_kernel(const RmsnormBwdArgs& a, float* partial, const BwdLaunch& l, cudaStream_t s) {
  return launch_overlapped(rmsnorm_bwd_row_kernel<T, EPT, ALIGNED, LANES>, static_cast<unsigned>(l.blocks),
                           static_cast<unsigned>(l.threads), 0, 1, s, a, partial);
}

template <typename T, int EPT, bool ALIGNED, int CL>
cudaError_t launch_staged_kernel(const RmsnormBwdArgs& a, float* partial, const BwdLaunch& l, cudaStream_t s) {
  auto kernel = rmsnorm_bwd_staged_kernel<T, EPT, ALIGNED, CL>;
  // the limit is the kernel's, not the call's: it may not fall under another
  // thread's launch
  constexpr size_t per_thread = 2 * EPT * sizeof(T);
  const size_t smem = per_thread * (a.dres ? 3 : 2) * l.threads;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(per_thread * 3 * kBwdThreads));
  if (e != cudaSuccess) return e;
  return launch_overlapped(kernel, static_cast<unsigned>(l.blocks), static_cast<unsigned>(l.threads), smem, CL, s, a,
                           partial);
}

template <typename T, bool ALIGNED>
cudaError_t launch_rows(const RmsnormBwdArgs& a, void* ws, cudaStream_t s) {
  const BwdLaunch l = bwd_launch(a.rows, a.cols, Elem<T>::VEC, !ALIGNED);
  float* partial = a.dgamma ? static_cast<float*>(ws) : nullptr;
  cudaError_t e = cudaErrorInvalidValue;
  if (l.lanes > 0) {
    if (l.lanes == 8) e = launch_row_kernel<T, 8, ALIGNED, 8>(a, partial, l, s);
    if (l.lanes == 16) e = launch_row_kernel<T, 8, ALIGNED, 16>(a, partial, l, s);
    if (l.lanes == 32 && l.ept == 8) e = launch_row_kernel<T, 8, ALIGNED, 32>(a, partial, l, s);
    if (l.lanes == 32 && l.ept == 16) e = launch_row_kernel<T, 16, ALIGNED, 32>(a, partial, l, s);
    if (l.lanes == 32 && l.ept == 32) e = launch_row_kernel<T, 32, ALIGNED, 32>(a, partial, l, s);
  } else {
    if constexpr (sizeof(T) == 2) {
      if (l.ept == 32 && l.cluster == 1) e = launch_staged_kernel<T, 32, ALIGNED, 1>(a, partial, l, s);
      if (l.ept == 32 && l.cluster == 2) e = launch_staged_kernel<T, 32, ALIGNED, 2>(a, partial, l, s);
      if (l.ept == 32 && l.cluster == 4) e = launch_staged_kernel<T, 32, ALIGNED, 4>(a, partial, l, s);
      if (l.ept == 16 && l.cluster == 1) e = launch_staged_kernel<T, 16, ALIGNED, 1>(a, partial, l, s);
    } else {
      if (l.cluster == 1) e = launch_staged_kernel<T, 16, ALIGNED, 1>(a, partial, l, s);
      if (l.cluster == 2) e = launch_staged_kernel<T, 16, ALIGNED, 2>(a, partial, l, s);
      if (l.cluster == 4) e = launch_staged_kernel<T, 16, ALIGNED, 4>(a, partial, l, s);
      if (l.cluster == 8) e = launch_staged_kernel<T, 16, ALIGNED, 8>(a, partial, l, s);
    }
  }
  if (e != cudaSuccess || partial == nullptr) return e;
  return launch_join(partial, a.dgamma, a.cols, l.groups, s);
}

template <typename T>
cudaError_t launch_type(const RmsnormBwdArgs& a, void* ws, cudaStream_t s) {
  // rows too long for a cluster's shared memory, or buffers that lie differently
  if (a.mode == kRowsAny || a.cols > kBwdMaxCols)
    return launch_stream<T>(a, ws, s);
  return a.mode == kRowsAligned ? launch_rows<T, true>(a, ws, s) : launch_rows<T, false>(a, ws, s);
}

}  // namespace

// What the kernels of this way of lying use.
size_t rmsnorm_bwd_workspace(size_t rows, size_t cols, int dtype, bool want_dgamma, RowMode mode) {
  if (mode == kRowsAny || cols > kBwdMaxCols)
    return stats_bytes(rows) + (want_dgamma ? stream_groups(rows) * cols * sizeof(float) : 0);
  return want_dgamma ? bwd_launch(rows, cols, vec_elems(dtype), mode != kRowsAligned).groups * cols * sizeof(float) : 0;
}

// Enough for every way the buffers may lie.
size_t rmsnorm_bwd_workspace(size_t rows, size_t cols, int dtype, bool want_dgamma) {
  size_t most = 0;
  for (RowMode mode : {kRowsAligned, kRowsShifted, kRowsAny}) {
    const size_t need = rmsnorm_bwd_workspace(rows, cols, dtype, want_dgamma, mode);
    most = need > most ? need : most;
  }
  return most;
}

cudaError_t launch_rmsnorm_bwd(const RmsnormBwdArgs& a, void* ws, cudaStream_t stream) {
  return a.dtype == FK_F32 ? launch_type<float>(a, ws, stream) : launch_type<__nv_bfloat16>(a, ws, stream);
}

}  // namespace fk
