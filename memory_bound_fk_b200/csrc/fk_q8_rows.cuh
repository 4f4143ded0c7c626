// fk_q8_rows.cuh -- the register-resident row pass shared by RMSNorm and the
// row quantiser (sm_100a): a team of threads (a warp, or a block of as many
// warps as the row needs) reads a row once, keeps its values in registers as
// fp32, reduces them once, and writes the outputs.
//
// Placement: with 16-byte vectors (aligned rows) thread t of the team holds
// vectors t, team + t, 2 team + t, ...; otherwise values t, team + t, ...,
// one at a time.  Either way a warp's accesses are contiguous.
//
// Bound by HBM.  A thread holds 16 values (rows up to 4096 columns) or 32:
// the loads of both inputs are all in flight before the first is used.
// Blocks are as wide as the row needs, not the next power of two, so that
// few lanes idle: 2560 columns take 160 threads.  Measured on B200 (64M
// bf16 values, x + residual in, h and e4m3 codes out, L2 flushed, 2.6 us of
// event overhead taken off): 4096 columns 6.08 TB/s at 16 values a thread,
// 6.25 at 32 with 64 registers, 5.4 at 32 without a register limit, 4.8 at
// 8; 8192 columns 5.63 / 5.92 / 5.12; 2048 columns 6.42 / 6.24 / 5.63; fp32
// rows 6.1-6.6 at either.
#pragma once

#include "fk_common.cuh"
#include "fk_q8.cuh"
#include "fk_rows.cuh"

namespace fk {
namespace {

constexpr int kRowWarps = 8;           // rows (warps) per block on the warp path, at most
constexpr int kRowWarpCols = 1024;     // rows up to here take one warp
constexpr int kRowSmallCols = 4096;    // up to here 16 values a thread
constexpr int kRowLargeCols = 16384;   // up to here 32 values a thread, at most 512 threads
constexpr int kRowMaxCols = 32768;     // the same, at most 1024 threads; longer rows are streamed
constexpr size_t kRowMaxGrid = 0x7fffffffu;

// A thread's place in its team.
struct Place {
  int t, team, cols;
};

// Is value k of chunk c one of the row's, and which.
template <int VEC, bool ALIGNED>
__device__ __forceinline__ int col_at(const Place& p, int c, int k) {
  return ALIGNED ? (c * p.team + p.t) * VEC + k : (c * VEC + k) * p.team + p.t;
}

// The thread's VPT chunks of a row, as packed 16-byte words; zeros outside.
template <typename T, int VPT, bool ALIGNED>
__device__ __forceinline__ void load_place(const T* row, const Place& p, uint4* raw) {
  constexpr int VEC = Elem<T>::VEC;
#pragma unroll
  for (int c = 0; c < VPT; ++c) {
    if constexpr (ALIGNED) {
      const int e = col_at<VEC, true>(p, c, 0);
      raw[c] = ld_stream_v4_if(row + e, e < p.cols, 0u);
    } else {
      float f[VEC];
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        const int e = col_at<VEC, false>(p, c, k);
        f[k] = e < p.cols ? Elem<T>::load1(row + e) : 0.0f;
      }
      raw[c] = Elem<T>::pack(f);  // exact
    }
  }
}

// One chunk stored in the rows' own type from its packed words.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_place(T* row, const Place& p, int c, uint4 w) {
  constexpr int VEC = Elem<T>::VEC;
  if constexpr (ALIGNED) {
    const int e = col_at<VEC, true>(p, c, 0);
    if (e < p.cols) *reinterpret_cast<uint4*>(row + e) = w;
  } else {
    float f[VEC];
    Elem<T>::unpack(w, f);
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int e = col_at<VEC, false>(p, c, k);
      if (e < p.cols) Elem<T>::store1(row + e, f[k]);  // exact
    }
  }
}

// One chunk stored as codes (zeros for a row that is not finite).
template <typename T, int OUT, bool ALIGNED>
__device__ __forceinline__ void store_codes(uint8_t* row, const Place& p, int c, const float* v, const RowScale& q) {
  constexpr int VEC = Elem<T>::VEC;
  if constexpr (ALIGNED) {
    const int e = col_at<VEC, true>(p, c, 0);
    uint32_t w[VEC / 4];
#pragma unroll
    for (int k = 0; k < VEC / 4; ++k) w[k] = q.ok ? Code8<OUT>::pack4(v + 4 * k, q.inv) : 0u;
    if (e < p.cols) {
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(row + e) = make_uint2(w[0], w[1]);
      else
        *reinterpret_cast<uint32_t*>(row + e) = w[0];
    }
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int e = col_at<VEC, false>(p, c, k);
      if (e < p.cols) row[e] = q.ok ? Code8<OUT>::pack1(v[k], q.inv) : 0;
    }
  }
}

// VEC fp32 parameters of chunk c (nullptr: ones).  The same for every row,
// so they come from L1 and L2.
template <int VEC, bool ALIGNED>
__device__ __forceinline__ void load_params(const float* g, const Place& p, int c, float* out) {
#pragma unroll
  for (int k = 0; k < VEC; ++k) out[k] = 1.0f;
  if (g == nullptr) return;
  if constexpr (ALIGNED) {
    const int e = col_at<VEC, true>(p, c, 0);
    if (e < p.cols) {
#pragma unroll
      for (int k = 0; k < VEC; k += 4) {
        const float4 z = __ldg(reinterpret_cast<const float4*>(g + e + k));
        out[k] = z.x;
        out[k + 1] = z.y;
        out[k + 2] = z.z;
        out[k + 3] = z.w;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) {
      const int e = col_at<VEC, false>(p, c, k);
      if (e < p.cols) out[k] = __ldg(g + e);
    }
  }
}

// Sum of s and NaN-propagating maximum of m over the team: a warp, or a block
// of any number of warps (`red`: one pair per warp; one barrier).
template <bool WARP>
__device__ __forceinline__ void team_sum_max(float& s, float& m, float2* red) {
  warp_sum_max(s, m);
  if constexpr (!WARP) {
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(s, m);
    __syncthreads();
    s = red[0].x;
    m = red[0].y;
    for (int w = 1; w < warps; ++w) {
      s += red[w].x;
      m = absmax_nan(m, red[w].y);
    }
  }
}

// Calls fn(row, place) for the rows of this block: one row per warp, or one
// per block at a time.
template <bool WARP, typename F>
__device__ __forceinline__ void for_rows(size_t rows, int cols, F fn) {
  if constexpr (WARP) {
    const size_t per = blockDim.x >> 5, stride = gridDim.x * per;
    const Place p = {static_cast<int>(threadIdx.x & 31), 32, cols};
    for (size_t row = blockIdx.x * per + (threadIdx.x >> 5); row < rows; row += stride) fn(row, p);
  } else {
    const Place p = {static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), cols};
    for (size_t row = blockIdx.x; row < rows; row += gridDim.x) {
      fn(row, p);
      if (row + gridDim.x < rows) __syncthreads();  // the reduction's scratch is used again
    }
  }
}

// Shape of a launch: threads per block, blocks.
struct RowLaunch {
  unsigned grid, threads;
};

// One warp per row: eight rows per block, halved down to two while blocks
// would leave multiprocessors idle (as the softmax's warp path does).
inline RowLaunch warp_launch(size_t rows) {
  size_t per = kRowWarps;
  while (per > 2 && (rows + per - 1) / per < 148) per /= 2;
  const size_t blocks = (rows + per - 1) / per;
  return {static_cast<unsigned>(blocks < kRowMaxGrid ? blocks : kRowMaxGrid), static_cast<unsigned>(32 * per)};
}

// One block per row, as many warps as hold it at ept values a thread.
inline RowLaunch block_launch(size_t rows, size_t cols, int ept) {
  const size_t threads = ((cols + ept - 1) / ept + 31) / 32 * 32;
  return {static_cast<unsigned>(rows < kRowMaxGrid ? rows : kRowMaxGrid), static_cast<unsigned>(threads)};
}

}  // namespace
}  // namespace fk
