// fk_q8_rows.cuh -- the register-resident row pass shared by RMSNorm and the
// row quantiser (sm_100a): a team of threads (a warp, or a block of as many
// warps as the row needs) reads a row once, keeps its values in registers as
// fp32, reduces them once, and writes the outputs.
//
// Placement: 16-byte vectors of VEC values; thread t of the team holds vectors
// t, team + t, 2 team + t, ..., so a warp's accesses are contiguous.  Rows
// whose pitch is not a multiple of 16 bytes (ALIGNED = false) start `lead`
// values past a 16-byte boundary, another lead for every row: there vector 0
// is the one that holds the boundary, the first and the last vector of a row
// are accessed value by value (only what belongs to the row), and parameters
// and codes are shifted in registers.  Inputs and outputs of the rows' type
// then have to sit alike to 16 bytes; other buffers are streamed.  4099 rows
// of 1001 fp32: XXX us against YYY one value at a time.
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
constexpr int kRowSmallCols = 8192;    // up to here four vectors a thread
constexpr int kRowLargeCols = 16384;   // up to here 32 values a thread, at most 512 threads
constexpr int kRowMaxCols = 32768;     // the same, at most 1024 threads; longer rows are streamed
// Columns a shifted row may take besides its own: up to VEC - 1 before it.
constexpr size_t row_span(size_t cols, bool aligned, int vec) { return aligned ? cols : cols + vec - 1; }
constexpr size_t kRowMaxGrid = 0x7fffffffu;

// A thread's place in its team, and the row's offset from a 16-byte boundary
// in values (0 when ALIGNED).
struct Place {
  int t, team, cols, lead;
};

// Column of value k of chunk c (outside [0, cols): not one of the row's).
template <int VEC>
__device__ __forceinline__ int col_at(const Place& p, int c, int k) {
  return (c * p.team + p.t) * VEC + k - p.lead;
}

// Values between `p` and the 16-byte boundary before it.
template <typename T>
__device__ __forceinline__ int lead_of(const T* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
}

// The rows of one buffer: where the row at hand starts, and the buffer's ends.
template <typename T>
struct RowOf {
  T* row;
  const T* begin;
  const T* end;
};
template <typename T>
__device__ __forceinline__ RowOf<T> row_of(T* buffer, size_t first, size_t count) {
  return RowOf<T>{buffer + first, buffer, buffer + count};
}

// Values outside columns [0, cols) of the vector at column e set to zero.
template <typename T>
__device__ __forceinline__ uint4 mask_edge(uint4 w, int e, int cols) {
  constexpr int VEC = Elem<T>::VEC;
  float f[VEC];
  Elem<T>::unpack(w, f);
#pragma unroll
  for (int k = 0; k < VEC; ++k) f[k] = e + k >= 0 && e + k < cols ? f[k] : 0.0f;
  return Elem<T>::pack(f);  // exact
}

// The thread's VPT chunks of a row, as packed 16-byte words; zeros outside.
// Shifted rows: a vector that crosses a row's end is loaded whole (its other
// values belong to the neighbouring rows; mask_place() takes them out once
// the loads are used, so that nothing waits here); only where that would
// leave the buffer, at its first and last vector, are values loaded one at a
// time.
template <typename T, int VPT, bool ALIGNED>
__device__ __forceinline__ void load_place(const RowOf<const T>& r, const Place& p, uint4* raw) {
  constexpr int VEC = Elem<T>::VEC;
#pragma unroll
  for (int c = 0; c < VPT; ++c) {
    const int e = col_at<VEC>(p, c, 0);
    const T* const at = r.row + e;
    if constexpr (ALIGNED) {
      raw[c] = ld_stream_v4_if(at, e < p.cols, 0u);
    } else {
      const bool any = e + VEC > 0 && e < p.cols, inside = at >= r.begin && at + VEC <= r.end;
      raw[c] = ld_stream_v4_if(at, any && inside, 0u);
      if (any && !inside) {
        float f[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k)
          f[k] = e + k >= 0 && e + k < p.cols ? static_cast<float>(at[k]) : 0.0f;
        raw[c] = Elem<T>::pack(f);  // exact
      }
    }
  }
}

// Zeros in place of what a shifted row's first and last vector hold of other
// rows.
template <typename T, int VPT, bool ALIGNED>
__device__ __forceinline__ void mask_place(const Place& p, uint4* raw) {
  if constexpr (!ALIGNED) {
#pragma unroll
    for (int c = 0; c < VPT; ++c) {
      const int e = col_at<Elem<T>::VEC>(p, c, 0);
      if (e < 0 || e + Elem<T>::VEC > p.cols) raw[c] = mask_edge<T>(raw[c], e, p.cols);
    }
  }
}

// Stores that stay where they are written in program order: left to itself
// the compiler gathers a row's stores at its end, and 16384 x 4096 bf16 (x +
// residual in, h and y out) goes from 94 us to 107.
__device__ __forceinline__ void st_v4(void* p, uint4 v) {
  asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void st_v2(void* p, uint32_t x, uint32_t y) {
  asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void st_v1(void* p, uint32_t x) {
  asm volatile("st.global.u32 [%0], %1;" ::"l"(p), "r"(x) : "memory");
}

// One chunk stored in the rows' own type from its packed words.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_place(T* row, const Place& p, int c, uint4 w) {
  constexpr int VEC = Elem<T>::VEC;
  const int e = col_at<VEC>(p, c, 0);
  if constexpr (ALIGNED) {
    if (e < p.cols) st_v4(row + e, w);
  } else {
    if (e >= 0 && e + VEC <= p.cols) {
      st_v4(row + e, w);
    } else if (e + VEC > 0 && e < p.cols) {
      float f[VEC];
      Elem<T>::unpack(w, f);
#pragma unroll
      for (int k = 0; k < VEC; ++k)
        if (e + k >= 0 && e + k < p.cols) Elem<T>::store1(row + e + k, f[k]);  // exact
    }
  }
}

// Bytes first .. 3 of a word of codes whose first byte is column e.
__device__ __forceinline__ void store_code_edge(uint8_t* row, int e, int cols, int first, uint32_t w) {
#pragma unroll
  for (int b = 0; b < 4; ++b)
    if (b >= first && e + b >= 0 && e + b < cols) row[e + b] = static_cast<uint8_t>(w >> (8 * b));
}

// One chunk stored as codes (zeros for a row that is not finite).  Every lane
// of the warp takes part.  Shifted rows: a lane's codes start s bytes past a
// 4-byte boundary, the same s for the whole row; each lane writes the aligned
// words that end in its own codes, the first of them completed by the last
// codes of the lane before it.
template <typename T, int OUT, bool ALIGNED>
__device__ __forceinline__ void store_codes(uint8_t* row, const Place& p, int c, const float* v, const RowScale& q) {
  constexpr int VEC = Elem<T>::VEC, W = VEC / 4;
  const int e = col_at<VEC>(p, c, 0);
  uint32_t w[W];
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = q.ok ? Code8<OUT>::pack4(v + 4 * k, q.inv) : 0u;
  if constexpr (ALIGNED) {
    if (e < p.cols) {
      if constexpr (W == 2)
        st_v2(row + e, w[0], w[1]);
      else
        st_v1(row + e, w[0]);
    }
  } else {
    const int s = static_cast<int>(reinterpret_cast<uintptr_t>(row + e) & 3), lane = threadIdx.x & 31;
    uint32_t before = __shfl_up_sync(0xffffffffu, w[W - 1], 1);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const uint32_t word = __funnelshift_l(before, w[k], 8 * s);
      const int at = e - s + 4 * k;                     // column of the word's first byte
      const int first = k == 0 && lane == 0 ? s : 0;    // the warp before wrote those
      if (first == 0 && at >= 0 && at + 4 <= p.cols)
        st_v1(row + at, word);
      else if (at + 4 > 0 && at < p.cols)
        store_code_edge(row, at, p.cols, first, word);
      before = w[k];
    }
    if (lane == 31 && s != 0 && e + VEC - s < p.cols && e + VEC > 0)
      store_code_edge(row, e + VEC - s, p.cols < e + VEC ? p.cols : e + VEC, 0, w[W - 1] >> (8 * (4 - s)));
  }
}

// VEC fp32 parameters of chunk c (nullptr: ones), 16-byte aligned at column
// 0.  The same for every row, so they come from L1 and L2.
template <int VEC, bool ALIGNED>
__device__ __forceinline__ void load_params(const float* g, const Place& p, int c, float* out) {
  const int e = col_at<VEC>(p, c, 0);
#pragma unroll
  for (int k = 0; k < VEC; ++k) out[k] = 1.0f;
  if (g == nullptr) return;
  if constexpr (ALIGNED) {
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
    // the aligned groups of four around e, then a shift by r = e mod 4 (the
    // same for the whole row)
    const int r = e & 3, from = e - r;
    float a[VEC + 4];
#pragma unroll
    for (int k = 0; k < VEC + 4; k += 4) {
      float4 z = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
      const int i = from + k;  // a multiple of 4: a group before column 0 holds none of the row's
      if (i >= 0 && i + 4 <= p.cols) {
        z = __ldg(reinterpret_cast<const float4*>(g + i));
      } else if (i >= 0 && i < p.cols) {
        z.x = __ldg(g + i);
        if (i + 1 < p.cols) z.y = __ldg(g + i + 1);
        if (i + 2 < p.cols) z.z = __ldg(g + i + 2);
      }
      a[k] = z.x;
      a[k + 1] = z.y;
      a[k + 2] = z.z;
      a[k + 3] = z.w;
    }
#pragma unroll
    for (int k = 0; k < VEC + 2; ++k) a[k] = (r & 1) ? a[k + 1] : a[k];
#pragma unroll
    for (int k = 0; k < VEC; ++k) out[k] = (r & 2) ? a[k + 2] : a[k];
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
    const Place p = {static_cast<int>(threadIdx.x & 31), 32, cols, 0};
    for (size_t row = blockIdx.x * per + (threadIdx.x >> 5); row < rows; row += stride) fn(row, p);
  } else {
    const Place p = {static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), cols, 0};
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

// One block per row, as many warps as hold it at ept values a thread (`span`:
// the columns, and the lead where rows are shifted).
inline RowLaunch block_launch(size_t rows, size_t span, int ept) {
  const size_t threads = ((span + ept - 1) / ept + 31) / 32 * 32;
  return {static_cast<unsigned>(rows < kRowMaxGrid ? rows : kRowMaxGrid), static_cast<unsigned>(threads)};
}

}  // namespace
}  // namespace fk
