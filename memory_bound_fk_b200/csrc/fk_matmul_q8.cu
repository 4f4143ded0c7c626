// fk_matmul_q8.cu -- C = act(A B^T * a_scale * b_scale + bias) with A [m, k]
// and B [n, k] in 8 bits, on the tcgen05 tensor cores (sm_100a).
//
// Orientation: the MMA's M side is B (128 output channels), its N side is A
// (tokens), so that an accumulator's lane is a channel and its column a
// token.  One token's outputs then lie across the lanes of a warp: they are
// stored straight from registers as contiguous runs whatever n and the
// alignment of C, and few tokens make a narrow MMA, not an empty one.
//
// Operands come by TMA in boxes of 128 codes of k (one 128-byte swizzled row)
// and the tensor maps fill what lies outside [m, k] and [n, k] with zeros, so
// ragged edges need no code in the main loop.
//
// This file: up to 64 tokens, one tile per block with k split over a cluster.
// More tokens: fk_matmul_q8_pair.cu.
//
// The product is bound by reading B once while m is below about 250 (B at
// 6.5 TB/s against 2 m ops a byte at 3.4 POP/s), by the tensor cores above.
// Measured on B200 in a captured chain (int8 to bf16): 1 x 16384 x 4096 13.3
// us with B from HBM each time (5.0 TB/s; alone 10.3 at the copy's rate, the
// rest is the start and the last blocks), 10.0 with the same B call after
// call, which L2 holds; 48 x 32001 x 4096 to fp32 25 us (5.5 TB/s).
#include <cuda.h>
#include <cuda_bf16.h>

#include "fk_common.cuh"
#include "fk_mm.cuh"
#include "fk_mm_host.h"
#include "fk_q8.cuh"
#include "fk_q8_internal.h"

namespace fk {
namespace {

constexpr int kChan = 128;   // channels per tile (MMA M)
using mm::kKBlock;
constexpr int kMmThreads = 192;  // four epilogue warps, the load warp, the MMA warp
constexpr size_t kMaxTokens = 64;  // more go to the pairs of SMs (fk_matmul_q8_pair.cu)
constexpr size_t kMaxGrid = 0x7fffffffu;

// ---------------------------------------------------------------- one tile per block, k split over a cluster

// A block takes 128 channels x TN tokens over a share of k; the SPLIT blocks
// of a cluster share one tile, push their partial accumulators into the
// shared memory of the block that owns the tokens, and each finishes TN /
// SPLIT tokens.  int32 partials add exactly; fp32 ones are added in block
// order, so results do not depend on timing.
template <int TN>
struct SplitShape {
  static constexpr uint32_t kStageBytes = (kChan + TN) * kKBlock;
  static constexpr uint32_t kRedBytes = TN * kChan * 4;
  // stages and partials together stay below half an SM's shared memory, so
  // that two blocks fit and one's start and end hide under the other's loads
  // (2 x 72 to 96 KB in flight; covering HBM latency at full rate takes 54)
  static constexpr int kStages = TN >= 64 ? 3 : TN >= 32 ? 4 : 5;
  static constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + kRedBytes;
  static constexpr uint32_t kTmemCols = TN < 32 ? 32 : TN;
  static_assert(kSmem >= mm::kSplitSmemLeast, "a pair of SMs would fit beside");
};

template <int Q8, int TN, int SPLIT, typename T, int EPI>
__global__ void __launch_bounds__(kMmThreads)
    matmul_split_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                        mm::Params p) {
  using S = SplitShape<TN>;
  constexpr int ST = S::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[ST], empty[ST], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ uint32_t part_bad[SPLIT];  // whether a block of the cluster gave up on a wait
  __shared__ float s_sa[TN];
  // stages of [128 channels | TN tokens] x 128 codes, 1024-byte aligned
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  uint32_t* red = reinterpret_cast<uint32_t*>(base + ST * S::kStageBytes);  // [SPLIT][TN / SPLIT][128]

  const int tid = threadIdx.x, warp = tid >> 5;
  const int part = SPLIT > 1 ? static_cast<int>(blockIdx.x % SPLIT) : 0;
  const unsigned tile = blockIdx.x / SPLIT;
  const int n0 = static_cast<int>(tile % p.tiles_n) * kChan, m0 = static_cast<int>(tile / p.tiles_n) * TN;
  const int kb0 = static_cast<int>(static_cast<long long>(p.kblocks) * part / SPLIT);
  const int kb1 = static_cast<int>(static_cast<long long>(p.kblocks) * (part + 1) / SPLIT);
  volatile int* abort = &abort_flag;

  if (warp == 5) {
    tc::tmem_alloc(&tmem_slot, S::kTmemCols);
    let_next_start();
  }
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  after_previous();
  if constexpr (SPLIT > 1) cluster_arrive_relaxed();  // every block of the cluster has started: waited for below
  const uint32_t tmem = tmem_slot;

  if (warp == 4) {
    if ((tid & 31) == 0) {
      int i = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int st = i % ST;
        if (i >= ST && !mm::wait(&empty[st], (i / ST - 1) & 1, abort)) break;
        uint8_t* dst = base + st * S::kStageBytes;
        mbar_arrive_expect_tx(&full[st], S::kStageBytes);
        tc::tma_load_2d(dst, &tma_b, &full[st], kb * kKBlock, n0);
        tc::tma_load_2d(dst + kChan * kKBlock, &tma_a, &full[st], kb * kKBlock, m0);
      }
      // copies in flight land before the block exits (all have, unless a wait gave up)
      for (int j = i > ST ? i - ST : 0; j < i; ++j)
        if (!mm::drain(&full[j % ST], (j / ST) & 1)) {
          *abort = 1;
          break;
        }
    }
    __syncwarp();
  } else if (warp == 5) {
    if ((tid & 31) == 0) {
      constexpr uint32_t HI = tc::smem_desc_hi(1024);
      constexpr uint32_t ID = mm::idesc<Q8>(kChan, TN);
      for (int i = 0; i < kb1 - kb0; ++i) {
        const int st = i % ST;
        if (!mm::wait(&full[st], (i / ST) & 1, abort)) break;
        tc::fence_after_sync();
        const uint32_t a = tc::smem_desc_lo(smem_addr(base + st * S::kStageBytes), 16);
        const uint32_t b = a + kChan * kKBlock / 16;
#pragma unroll
        for (int q = 0; q < kKBlock / 32; ++q)
          mm::mma<Q8>(tmem, tc::desc_join(a + 2 * q, HI), tc::desc_join(b + 2 * q, HI), ID, (i | q) != 0);
        tc::mma_commit(&empty[st]);
      }
      tc::mma_commit(&done);
    }
    __syncwarp();
  }
  // ---- epilogue: warp w reads lanes 32 w .. 32 w + 31, lane = channel; the
  // scales are fetched while the MMAs run
  const int chan = n0 + tid;
  float sb = 0.0f, bias = 0.0f;
  if (warp < 4) {
    if (tid < TN) s_sa[tid] = m0 + tid < p.m ? p.sa[m0 + tid] : 0.0f;
    if (chan < p.n) {
      sb = p.sb[chan];
      bias = p.bias ? p.bias[chan] : 0.0f;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");  // s_sa stands
    if (!mm::drain(&done, 0, p.done_ns)) {
      *abort = 1;
      mm::drain(&done, 0);  // MMAs that still run end before their memory goes
    }
    tc::fence_after_sync();
  }
  __syncthreads();  // one verdict for the block
  if constexpr (SPLIT > 1) cluster_wait();
  const bool good = *abort == 0;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(warp & 3) << 21);
  T* c = static_cast<T*>(p.c);
  auto finish = [&](uint32_t w, int t) {
    const float v = mm::act<EPI>(fmaf(mm::acc_value<Q8>(w) * s_sa[t], sb, bias));
    if (chan < p.n && m0 + t < p.m) c[static_cast<size_t>(m0 + t) * p.n + chan] = static_cast<T>(v);
  };
  if constexpr (SPLIT == 1) {
    if (warp < 4 && good) {
#pragma unroll 1
      for (int t = 0; t < TN && m0 + t < p.m; t += 16) {
        uint32_t r[16];
        mm::tmem_ld16(lane_base + t, r);
#pragma unroll
        for (int q = 0; q < 16; ++q) finish(r[q], t + q);
      }
    }
  } else {
    constexpr int OWN = TN / SPLIT;  // tokens this block finishes
    if (warp < 4 && good) {
#pragma unroll 1
      for (int t = 0; t < TN && m0 + t < p.m; t += 16) {
        uint32_t r[16];
        mm::tmem_ld16(lane_base + t, r);
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const int owner = (t + q) / OWN, slot = (t + q) % OWN;
          mm::st_cluster(cluster_addr(red + (part * OWN + slot) * kChan + tid, owner), r[q]);
        }
      }
    }
    if (tid < SPLIT) mm::st_cluster(cluster_addr(&part_bad[part], tid), good ? 0u : 1u);
    mm::cluster_sync();
    bool all_good = true;
#pragma unroll
    for (int o = 0; o < SPLIT; ++o) all_good = all_good && part_bad[o] == 0;
    if (warp < 4 && all_good) {
#pragma unroll
      for (int s = 0; s < OWN; ++s) {
        const int t = part * OWN + s;
        if (m0 + t >= p.m) break;
        uint32_t w = red[s * kChan + tid];
#pragma unroll
        for (int o = 1; o < SPLIT; ++o) w = mm::acc_add<Q8>(w, red[(o * OWN + s) * kChan + tid]);
        finish(w, t);
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 5) tc::tmem_dealloc(tmem, S::kTmemCols);
}

// ---------------------------------------------------------------- rows padded to 16 bytes

// For operands TMA cannot read (a pitch that is no multiple of 16 bytes, or a
// base that is off one): both are copied in one launch to rows of k codes
// rounded up to 16, with zeros past k, `pitch` 16-byte pieces apart.  One thread per 16 bytes of the result:
// five aligned words and a funnel shift, or single bytes next to the ends of
// the source.  (Four pieces a lane from pairs of 16-byte loads: 45 us against
// 36 for 1 x 16384 x 4097 with its product.)  One more write and read of the
// operands, which a caller avoids by keeping k a multiple of 16.
struct PadJob {
  const uint8_t* src;
  uint4* dst;
  size_t rows;  // 0: nothing to do
};

__global__ void __launch_bounds__(256)
    matmul_pad_kernel(const __grid_constant__ PadJob a, const __grid_constant__ PadJob b, size_t k, size_t chunks,
                      size_t pitch) {
  let_next_start();
  after_previous();
  const size_t total_a = a.rows * chunks, total = total_a + b.rows * chunks;
  for (size_t i = static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * 256) {
    const bool first = i < total_a;
    const uint8_t* const src = first ? a.src : b.src;
    const size_t piece = first ? i : i - total_a, end = (first ? a.rows : b.rows) * k;
    const size_t row = total <= 0xffffffffu ? static_cast<uint32_t>(piece) / static_cast<uint32_t>(chunks) : piece / chunks;
    const size_t l = (piece - row * chunks) * 16, at = row * k + l;
    uint32_t w[4];
    const size_t shift = (reinterpret_cast<uintptr_t>(src) + at) & 3;
    if (at >= shift && at - shift + 20 <= end) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(src + at - shift);
      uint32_t v[5];
#pragma unroll
      for (int j = 0; j < 5; ++j) v[j] = q[j];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(v[j], v[j + 1], static_cast<unsigned>(shift) * 8);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (at + 4 * j + e < end) w[j] |= static_cast<uint32_t>(src[at + 4 * j + e]) << (8 * e);
      }
    }
    const size_t left = k - l;  // codes of this row from here on
    if (left < 16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int keep = static_cast<int>(left) - 4 * j;
        w[j] = keep <= 0 ? 0u : keep >= 4 ? w[j] : w[j] & ((1u << (8 * keep)) - 1u);
      }
    }
    (first ? a.dst : b.dst)[row * pitch + l / 16] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------- host side

using PFN_encodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                     const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                     CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

PFN_encodeTiled encode_fn() {
  static PFN_encodeTiled fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return static_cast<PFN_encodeTiled>(nullptr);
    }
    return reinterpret_cast<PFN_encodeTiled>(p);
  }();
  return fn;
}

template <int Q8, int TN, int SPLIT, typename T, int EPI>
cudaError_t launch_split(const mm::Call& c) {
  using S = SplitShape<TN>;
  const size_t tiles_n = (c.p.n + kChan - 1) / kChan, tiles_m = (c.p.m + TN - 1) / TN;
  if (tiles_m > kMaxGrid / SPLIT / tiles_n) return cudaErrorInvalidConfiguration;
  CUtensorMap ma, mb;
  if (!mm::make_map(&ma, c.a, c.p.m, c.k, c.pitch_a, TN) || !mm::make_map(&mb, c.b, c.p.n, c.k, c.pitch_b, kChan))
    return cudaErrorInvalidValue;
  const size_t smem = S::kSmem;
  auto kernel = matmul_split_kernel<Q8, TN, SPLIT, T, EPI>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const mm::Params p = mm::make_params(c, tiles_n, tiles_m);
  return launch_overlapped(kernel, static_cast<unsigned>(tiles_n * tiles_m * SPLIT), kMmThreads, smem, SPLIT, c.stream,
                           ma, mb, p);
}

// Blocks of a cluster that share a tile: doubled while the grid still fits
// two blocks per SM at once and each keeps two 128-code steps of k.  Measured
// on B200 in a captured chain (one token, int8, us for 1 / 2 / 4 / 8 blocks a
// tile): 1024 x 1024 4.3 / 3.5 / 3.0 / 2.8; 4096 x 4096 12.4 / 7.9 / 6.3 / 6.3;
// 8192 x 8192 22.3 / 14.7 / 14.1 / 16.6; 16384 x 4096 14.6 / 14.4 / 16.0 / 20.7.
template <int Q8, int TN, typename T, int EPI>
cudaError_t launch_tokens(const mm::Call& c) {
  const size_t tiles = ((c.p.n + kChan - 1) / kChan) * ((c.p.m + TN - 1) / TN);
  const size_t kblocks = (c.k + kKBlock - 1) / kKBlock, room = 2 * static_cast<size_t>(c.sm_count);
  int split = 1;
  while (split < 8 && tiles * split * 2 <= room && kblocks >= static_cast<size_t>(split) * 4) split *= 2;
  switch (split) {
    case 1: return launch_split<Q8, TN, 1, T, EPI>(c);
    case 2: return launch_split<Q8, TN, 2, T, EPI>(c);
    case 4: return launch_split<Q8, TN, 4, T, EPI>(c);
    default: return launch_split<Q8, TN, 8, T, EPI>(c);
  }
}

template <int Q8, typename T, int EPI>
cudaError_t launch_epi(const mm::Call& c) {
  if (c.p.m <= 16) return launch_tokens<Q8, 16, T, EPI>(c);
  if (c.p.m <= 32) return launch_tokens<Q8, 32, T, EPI>(c);
  return launch_tokens<Q8, 64, T, EPI>(c);
}

template <int Q8, typename T>
cudaError_t launch_out(const mm::Call& c) {
  switch (c.p.epilogue) {
    case FK_EPILOGUE_GELU_TANH: return launch_epi<Q8, T, FK_EPILOGUE_GELU_TANH>(c);
    case FK_EPILOGUE_GELU_ERF: return launch_epi<Q8, T, FK_EPILOGUE_GELU_ERF>(c);
    default: return launch_epi<Q8, T, FK_EPILOGUE_NONE>(c);
  }
}

template <int Q8>
cudaError_t launch_type(const mm::Call& c) {
  return c.p.out_dtype == FK_F32 ? launch_out<Q8, float>(c) : launch_out<Q8, __nv_bfloat16>(c);
}

size_t round16(size_t v) { return (v + 15) / 16 * 16; }

// Bytes from row to row of the copies: whole 128-byte lines for all but short
// rows, so that a box's rows lie in one line each (2000 x 16384 x 4097: 122
// us against 169 with rows 4112 bytes apart).
size_t pad_pitch(size_t k) { return k <= 128 ? round16(k) : (k + 127) / 128 * 128; }

cudaError_t launch_pad(const PadJob& a, const PadJob& b, size_t k, size_t pitch, cudaStream_t s) {
  const size_t chunks = round16(k) / 16, blocks = ((a.rows + b.rows) * chunks + 255) / 256;
  return launch_overlapped(matmul_pad_kernel, static_cast<unsigned>(blocks < 148 * 16 ? blocks : 148 * 16), 256, 0, 1, s,
                           a, b, k, chunks, pitch / 16);
}

}  // namespace

namespace mm {
bool make_map(CUtensorMap* m, const void* ptr, size_t rows, size_t k, size_t pitch, int box_rows) {
  PFN_encodeTiled f = encode_fn();
  if (f == nullptr) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(k), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
  const cuuint32_t box[2] = {kKBlock, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace mm

size_t matmul_q8_workspace(size_t m, size_t n, size_t k, bool aligned) {
  return aligned && k % 16 == 0 ? 0 : (m + n) * pad_pitch(k);
}

cudaError_t launch_matmul_q8(const MatmulQ8Args& p, void* ws, int sm_count, cudaStream_t s) {
  mm::Call c = {p.a, p.b, p.k, p.k, p.k, p, sm_count > 0 ? sm_count : 1, s};
  if (ws != nullptr) {
    // operands that TMA cannot read as they are, or (where one of them has to
    // be copied anyway for its base) only that one: the pitches may differ
    const size_t pitch = pad_pitch(p.k);
    uint8_t* w = static_cast<uint8_t*>(ws);
    const bool pad_a = p.k % 16 != 0 || reinterpret_cast<uintptr_t>(p.a) % 16 != 0;
    const bool pad_b = p.k % 16 != 0 || reinterpret_cast<uintptr_t>(p.b) % 16 != 0;
    const cudaError_t e = launch_pad(
        {static_cast<const uint8_t*>(p.a), reinterpret_cast<uint4*>(w), pad_a ? p.m : 0},
        {static_cast<const uint8_t*>(p.b), reinterpret_cast<uint4*>(w + p.m * pitch), pad_b ? p.n : 0}, p.k, pitch, s);
    if (e != cudaSuccess) return e;
    if (pad_a) c.a = w, c.pitch_a = pitch;
    if (pad_b) c.b = w + p.m * pitch, c.pitch_b = pitch;
    c.k = round16(p.k);
  }
  // Past 64 tokens the pairs of SMs win (128 tokens, 4096 x 4096: 10.9 us
  // against 12.6 with 128-token tiles here).  At 64 and below it depends on the
  // channels: 64 tokens of 4096 x 4096 took 8.5 here against 10.9, of 16384 x
  // 4096 17.4 against 16.2, and the few channels decide the trade.
  if (p.m > kMaxTokens) return mm::launch_pair(c);
  return p.dtype == FK_I8 ? launch_type<FK_I8>(c) : launch_type<FK_E4M3>(c);
}

cudaError_t read_matmul_wait_timeouts(unsigned* out, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(out, mm::g_mm_wait_timeouts, sizeof(unsigned));
  if (e == cudaSuccess && reset) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(mm::g_mm_wait_timeouts, &zero, sizeof(unsigned));
  }
  unsigned pair = 0;
  if (e == cudaSuccess) e = mm::read_pair_wait_timeouts(&pair, reset);
  *out += pair;
  return e;
}

}  // namespace fk
