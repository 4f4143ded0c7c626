// fk_q8_rows.cuh -- the register-resident row pass shared by RMSNorm and the
// row quantiser (sm_100a): a team of threads (part of a warp, a warp, a block
// of as many warps as the row needs, or a cluster of them) reads a row once,
// keeps its values in registers as fp32, reduces them once, and writes the
// outputs.
//
// Placement: 16-byte vectors of VEC values; thread t of the team holds vectors
// t, team + t, 2 team + t, ..., so a warp's accesses are contiguous.  Rows
// whose pitch is not a multiple of 16 bytes (ALIGNED = false) start anywhere:
// their vectors are those that lie on 16-byte boundaries inside the row, and
// the at most 2 (VEC - 1) values before the first and behind the last belong
// to the team's first threads, one each.  Inputs and outputs of the rows' type
// then have to sit alike to 16 bytes; other buffers are streamed.
//
// Bound by HBM.  A thread holds four vectors (16 fp32 or 32 bf16 values): the
// loads of both inputs are all in flight before the first is used, and 64
// registers a thread keep 1024 threads on an SM.  Blocks are as wide as the
// row needs, not the next power of two, so that few lanes idle: 2560 columns
// take 96 threads of bf16.  Kernel arguments are __grid_constant__: copied to
// the stack for the row's lambda, they cost 180 us against 158 (16384 x 4096
// fp32, x + residual in, h and y out) and 108 against 81 (the same in bf16).
#pragma once

#include "fk_common.cuh"
#include "fk_q8.cuh"
#include "fk_sync.cuh"

namespace fk {
namespace {

constexpr int kRowWarps = 8;           // warps per block where a row takes a warp or less, at most
constexpr int kRowLaneEpt = 8;         // values a thread where a row takes 8 or 16 lanes
constexpr int kRowWarpCols = 1024;     // rows up to here take one warp
constexpr int kRowBlockCols = 8192;    // RMSNorm: up to here four vectors a thread (fp32: 512 threads)
constexpr int kRowLargeCols = 16384;   // up to here 32 values a thread, at most 512 threads
constexpr int kRowMaxCols = 32768;     // the same, at most 1024 threads
constexpr int kRowClusterCols = 131072;  // clusters of 4 or 8 such blocks of 512 threads; longer rows are streamed
constexpr size_t kRowMaxGrid = 0x7fffffffu;

// A thread's place in its team; the row's columns, how many of them come
// before the first vector, and how many vectors there are.
struct Place {
  int t, team, cols, head, vecs;
};

// Place of an aligned row (cols a multiple of VEC), or of the one at `row`.
template <typename T, bool ALIGNED>
__device__ __forceinline__ Place place_of(int t, int team, int cols, const T* row) {
  constexpr int VEC = Elem<T>::VEC;
  if constexpr (ALIGNED) return Place{t, team, cols, 0, cols / VEC};
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  int head = off == 0 ? 0 : VEC - off;
  head = head < cols ? head : cols;
  return Place{t, team, cols, head, (cols - head) / VEC};
}

// Is chunk c one of the row's vectors, and the column of its first value.
__device__ __forceinline__ bool has_vec(const Place& p, int c) { return c * p.team + p.t < p.vecs; }
template <int VEC>
__device__ __forceinline__ int col_of_vec(const Place& p, int c) {
  return p.head + (c * p.team + p.t) * VEC;
}

// The column outside the vectors that is this thread's, or -1.
template <int VEC>
__device__ __forceinline__ int edge_col(const Place& p) {
  const int in = p.vecs * VEC;
  return p.t < p.cols - in ? (p.t < p.head ? p.t : in + p.t) : -1;
}

// VPT of the thread's vectors of a row, the first of them its vector `from`,
// as packed 16-byte words; zeros where there is none.
template <typename T, int VPT, bool RELAXED = false>
__device__ __forceinline__ void load_vecs(const T* row, const Place& p, uint4* raw, int from = 0) {
#pragma unroll
  for (int c = 0; c < VPT; ++c)
    raw[c] = ld_row_v4_if<RELAXED>(row + col_of_vec<Elem<T>::VEC>(p, from + c), has_vec(p, from + c));
}

// One value of the rows' type, and the rounding to it.
template <typename T>
__device__ __forceinline__ float load_one(const T* p) {
  return static_cast<float>(*p);
}
template <typename T>
__device__ __forceinline__ float round_one(float v) {
  if constexpr (sizeof(T) == 4) return v;
  return __bfloat162float(__float2bfloat16_rn(v));
}

// Stores of a fixed width, write-back: the next operator of the chain reads
// them, from L2 where they fit.
__device__ __forceinline__ void st_v4(void* p, uint4 v) {
  asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void st_v2(void* p, uint32_t x, uint32_t y) {
  asm volatile("st.global.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void st_v1(void* p, uint32_t x) {
  asm volatile("st.global.u32 [%0], %1;" ::"l"(p), "r"(x) : "memory");
}
__device__ __forceinline__ void st_u16(void* p, uint32_t x) {
  asm volatile("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tst.global.u16 [%0], h;\n\t}" ::"l"(p), "r"(x) : "memory");
}
__device__ __forceinline__ void st_u8(void* p, uint32_t x) {
  asm volatile("st.global.u8 [%0], %1;" ::"l"(p), "r"(x) : "memory");
}

// Vector c stored in the rows' own type.
template <typename T>
__device__ __forceinline__ void store_vec(T* row, const Place& p, int c, uint4 w) {
  if (has_vec(p, c)) st_v4(row + col_of_vec<Elem<T>::VEC>(p, c), w);
}

// Four or eight codes to any address, in the widest aligned pieces: s is the
// address modulo 4 (the same for the whole row, so no lane waits for another).
template <int W>
__device__ __forceinline__ void store_unaligned(uint8_t* at, int s, const uint32_t* w) {
  if (s == 0) {
#pragma unroll
    for (int k = 0; k < W; ++k) st_v1(at + 4 * k, w[k]);
  } else if (s == 2) {
    st_u16(at, w[0]);
    if (W == 2) st_v1(at + 2, __funnelshift_r(w[0], w[W - 1], 16));
    st_u16(at + 4 * W - 2, w[W - 1] >> 16);
  } else if (s == 1) {
    st_u8(at, w[0]);
    st_u16(at + 1, w[0] >> 8);
    if (W == 2) st_v1(at + 3, __funnelshift_r(w[0], w[W - 1], 24));
    st_u8(at + 4 * W - 1, w[W - 1] >> 24);
  } else {
    st_u8(at, w[0]);
    if (W == 2) st_v1(at + 1, __funnelshift_r(w[0], w[W - 1], 8));
    st_u16(at + 4 * W - 3, w[W - 1] >> 8);
    st_u8(at + 4 * W - 1, w[W - 1] >> 24);
  }
}

// Vector c stored as codes (zeros for a row that is not finite).
template <typename T, int OUT, bool ALIGNED>
__device__ __forceinline__ void store_codes(uint8_t* row, const Place& p, int c, const float* v, const RowScale& q) {
  constexpr int VEC = Elem<T>::VEC, W = VEC / 4;
  uint8_t* const at = row + col_of_vec<VEC>(p, c);
  uint32_t w[W];
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = q.ok ? Code8<OUT>::pack4(v + 4 * k, q) : 0u;
  if (!has_vec(p, c)) return;
  if constexpr (!ALIGNED)
    store_unaligned<W>(at, static_cast<int>(reinterpret_cast<uintptr_t>(at) & 3), w);
  else if constexpr (W == 2)
    st_v2(at, w[0], w[1]);
  else
    st_v1(at, w[0]);
}

// VEC fp32 parameters of vector c (nullptr: ones), 16-byte aligned at column
// 0.  The same for every row, so they come from L1 and L2.
template <int VEC, bool ALIGNED>
__device__ __forceinline__ void load_params(const float* g, const Place& p, int c, float* out) {
  const int e = col_of_vec<VEC>(p, c);
#pragma unroll
  for (int k = 0; k < VEC; ++k) out[k] = 1.0f;
  if (g == nullptr || !has_vec(p, c)) return;
  // Shifted rows: the aligned groups of four around the vector, then a shift
  // by r = e mod 4 (the same for the whole row): one of four copies runs.
  const int r = ALIGNED ? 0 : e & 3, from = e - r;
  float a[VEC + 4];
#pragma unroll
  for (int k = 0; k < (ALIGNED ? VEC : VEC + 4); k += 4) {
    float4 z = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    const int i = from + k;
    if (ALIGNED || i + 4 <= p.cols) {
      z = ld_param4(g + i);
    } else if (i < p.cols) {
      z.x = ld_param(g + i);
      if (i + 1 < p.cols) z.y = ld_param(g + i + 1);
      if (i + 2 < p.cols) z.z = ld_param(g + i + 2);
    }
    a[k] = z.x;
    a[k + 1] = z.y;
    a[k + 2] = z.z;
    a[k + 3] = z.w;
  }
  if (r == 0) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) out[k] = a[k];
  } else if (r == 1) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) out[k] = a[k + 1];
  } else if (r == 2) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) out[k] = a[k + 2];
  } else {
#pragma unroll
    for (int k = 0; k < VEC; ++k) out[k] = a[k + 3];
  }
}

// Sum of s and NaN-propagating maximum of m over the team: LANES lanes of a
// warp, or (LANES = 0) a block of any number of warps (`red`: one pair per
// warp; one barrier).
template <int LANES>
__device__ __forceinline__ void team_sum_max(float& s, float& m, float2* red) {
#pragma unroll
  for (int o = (LANES == 0 ? 32 : LANES) / 2; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    m = absmax_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if constexpr (LANES == 0) {
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

// The same over the CL blocks of a cluster (`red`: one pair per warp of the
// cluster).  Every block has started (cluster_wait()); used once.
template <int CL>
__device__ __forceinline__ void cluster_sum_max(float& s, float& m, float2* red) {
  warp_sum_max(s, m);
  const int warps = static_cast<int>(blockDim.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
  if (lane < CL)
    st_cluster_f2(cluster_addr(&red[static_cast<int>(cluster_ctarank()) * warps + static_cast<int>(threadIdx.x >> 5)], lane),
                  s, m);
  cluster_barrier();
  s = red[0].x;
  m = red[0].y;
  for (int w = 1; w < CL * warps; ++w) {
    s += red[w].x;
    m = absmax_nan(m, red[w].y);
  }
}

// The maximum alone (of values: NaN if one is; at least 0 over a block).
// `red`: 16-byte aligned, one word per warp, their number rounded up to four.
template <int LANES>
__device__ __forceinline__ void team_max(float& m, float* red) {
  auto larger = [](float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
  };
#pragma unroll
  for (int o = (LANES == 0 ? 32 : LANES) / 2; o > 0; o >>= 1) m = larger(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (LANES == 0) {
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
    if (threadIdx.x < (-warps & 3)) red[warps + threadIdx.x] = 0.0f;
    __syncthreads();
    m = 0.0f;
    for (int w = 0; w < warps; w += 4) {
      const float4 z = *reinterpret_cast<const float4*>(red + w);
      m = larger(m, larger(larger(z.x, z.y), larger(z.z, z.w)));
    }
  }
}

// Calls fn(row, t, team, cols) for the rows of this block: 32 / LANES rows per
// warp, or (LANES = 0) one per block at a time.  Lanes of a warp that have no
// row left take part with no columns.  CL > 1: one row per cluster of CL
// blocks (their number is that of the rows times CL).
template <int LANES, int CL, typename F>
__device__ __forceinline__ void for_rows(size_t rows, int cols, F fn) {
  if constexpr (CL > 1) {
    cluster_arrive_relaxed();
    cluster_wait();  // every block has started
    fn(blockIdx.x / CL, static_cast<int>(cluster_ctarank() * blockDim.x + threadIdx.x),
       static_cast<int>(CL * blockDim.x), cols);
  } else if constexpr (LANES > 0) {
    constexpr int PER = 32 / LANES;
    const size_t per = (blockDim.x >> 5) * PER, stride = gridDim.x * per;
    const int lane = threadIdx.x & 31;
    for (size_t first = blockIdx.x * per + (threadIdx.x >> 5) * PER; first < rows; first += stride) {
      const size_t row = first + lane / LANES;
      fn(row, lane % LANES, LANES, row < rows ? cols : 0);
    }
  } else {
    for (size_t row = blockIdx.x; row < rows; row += gridDim.x) {
      fn(row, static_cast<int>(threadIdx.x), static_cast<int>(blockDim.x), cols);
      if (row + gridDim.x < rows) __syncthreads();  // the reduction's scratch is used again
    }
  }
}

// Lanes a row of up to kRowWarpCols columns takes: eight values a lane where
// that leaves lanes for another row (and, for shifted rows, a lane for each
// value outside the vectors), else the whole warp.
inline int row_lanes(size_t cols, bool aligned, int vec) {
  if (cols <= 8 * kRowLaneEpt && (aligned || 2 * (vec - 1) <= 8)) return 8;
  return cols <= 16 * kRowLaneEpt ? 16 : 32;
}

// Shape of a launch: threads per block, blocks.
struct RowLaunch {
  unsigned grid, threads;
};

// `lanes` lanes per row: eight warps per block, halved down to two while
// blocks would leave multiprocessors idle (as the softmax's warp path does).
inline RowLaunch warp_launch(size_t rows, int lanes) {
  const size_t per_warp = 32 / lanes;
  size_t warps = kRowWarps;
  while (warps > 2 && (rows + warps * per_warp - 1) / (warps * per_warp) < 148) warps /= 2;
  const size_t blocks = (rows + warps * per_warp - 1) / (warps * per_warp);
  return {static_cast<unsigned>(blocks < kRowMaxGrid ? blocks : kRowMaxGrid), static_cast<unsigned>(32 * warps)};
}

// One block per row, as many warps as hold it at ept values a thread.
inline RowLaunch block_launch(size_t rows, size_t cols, int ept) {
  const size_t threads = ((cols + ept - 1) / ept + 31) / 32 * 32;
  return {static_cast<unsigned>(rows < kRowMaxGrid ? rows : kRowMaxGrid), static_cast<unsigned>(threads)};
}

// One cluster of `cl` blocks per row at 32 values a thread (no blocks, which
// the launch refuses, past the largest grid).
inline RowLaunch cluster_launch(size_t rows, size_t cols, int cl) {
  const size_t per = size_t{32} * cl, threads = ((cols + per - 1) / per + 31) / 32 * 32;
  return {static_cast<unsigned>(rows <= kRowMaxGrid / cl ? rows * cl : 0), static_cast<unsigned>(threads)};
}

}  // namespace
}  // namespace fk
