// fk_matmul_q8_pair.cu -- the 8-bit product for many tokens: persistent pairs
// of SMs on 256 x 256 tiles (sm_100a).
//
// Orientation as in fk_matmul_q8.cu: the MMA's M side is B (256 output
// channels, 128 to each block of the pair), its N side A (256 tokens).  With
// cta_group::2 a block keeps only its own 128 channels and half of the
// tokens in shared memory, and the pair's tensor cores read both halves of
// the tokens: 32 KB a stage and block for 256 x 256 x 128 codes, half of what
// two separate blocks would fill and read.  That matters because operand
// reads of a 128 x 128 tile (8 KB per 64 cycles and SM) already take the whole
// shared-memory bandwidth, and TMA writes come on top.
//
// Each SM's tensor memory holds two accumulators, so the epilogue of one tile
// runs under the MMAs of the next.  Warps: eight for the epilogue (two per
// quarter of the lanes, halves of the tokens), one for the loads, one that
// issues MMAs (in the pair's leader).
#include <cuda.h>
#include <cuda_bf16.h>

#include "fk_mm.cuh"
#include "fk_mm_host.h"

namespace fk {
namespace mm {
namespace {

constexpr int kChan = 128;           // channels per block (256 per pair)
constexpr int kTok = 256;            // tokens per tile
constexpr int kStages = 6;
constexpr uint32_t kHalfBytes = 128 * kKBlock;  // one operand of one block and stage
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 2);
constexpr uint32_t kTmemCols = 2 * kTok;
// Tiles go to pairs in groups of this many channel tiles by all token tiles,
// channels fastest, so that concurrent pairs share operands through L2.
constexpr int kGroup = 8;

struct Tile {
  int n0, m0;  // first channel of the pair's tile, first token
};
__device__ __forceinline__ Tile tile_at(const Params& p, int t) {
  const int per = kGroup * p.tiles_m, g = t / per, r = t - g * per;
  const int first = g * kGroup, width = p.tiles_n - first < kGroup ? p.tiles_n - first : kGroup;
  return Tile{(first + r % width) * 2 * kChan, r / width * kTok};
}

template <int Q8, typename T, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_pair_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b, Params p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int tiles = p.tiles_n * p.tiles_m, pairs = static_cast<int>(gridDim.x) / 2;
  const int pair = static_cast<int>(blockIdx.x) / 2;
  volatile int* abort = &abort_flag;

  if (warp == kEpiWarps + 1) tmem_alloc_pair(&tmem_slot, kTmemCols);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * kEpiWarps);
    }
    abort_flag = 0;
    fence_mbarrier_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();  // both blocks' barriers stand
  tc::fence_after_sync();
  const uint32_t tmem = tmem_slot;

  if (warp == kEpiWarps) {
    // ---- loads: a block's channels and its half of the tokens, counted on the leader's barrier
    if (lane == 0) {
      int i = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const Tile tl = tile_at(p, t);
        for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
          const int st = i % kStages;
          if (i >= kStages && !wait(&empty[st], (i / kStages - 1) & 1, abort)) {
            ok = false;
            break;
          }
          uint8_t* dst = base + st * kStageBytes;
          const uint32_t bar = cluster_addr(&full[st], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * kStageBytes);
          tma_load_2d_pair(dst, &tma_b, bar, kb * kKBlock, tl.n0 + rank * kChan);
          tma_load_2d_pair(dst + kHalfBytes, &tma_a, bar, kb * kKBlock, tl.m0 + rank * (kTok / 2));
        }
      }
      // what was loaded has been read by the MMAs before the block exits
      for (int j = i > kStages ? i - kStages : 0; j < i; ++j) drain(&empty[j % kStages], (j / kStages) & 1);
    }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    // ---- MMAs, issued by the leader for both blocks
    if (rank == 0 && lane == 0) {
      constexpr uint32_t HI = tc::smem_desc_hi(1024);
      constexpr uint32_t ID = idesc<Q8>(2 * kChan, kTok);
      const uint32_t a0 = tc::smem_desc_lo(smem_addr(base), 16);
      int i = 0, u = 0;  // stages consumed, tiles begun
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++u) {
        const int buf = u & 1;
        if (u >= 2 && !wait(&acc_empty[buf], (u / 2 - 1) & 1, abort)) break;
        tc::fence_after_sync();
        for (int kb = 0; kb < p.kblocks; ++kb, ++i) {
          const int st = i % kStages;
          if (!wait(&full[st], (i / kStages) & 1, abort)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint32_t a = a0 + st * (kStageBytes / 16), b = a + kHalfBytes / 16;
#pragma unroll
          for (int q = 0; q < kKBlock / 32; ++q)
            mma_pair<Q8>(tmem + buf * kTok, tc::desc_join(a + 2 * q, HI), tc::desc_join(b + 2 * q, HI), ID,
                         (kb | q) != 0);
          commit_pair(&empty[st]);
        }
        if (ok) commit_pair(&acc_full[buf]);
      }
    }
    __syncwarp();
  } else {
    // ---- epilogue: lane = channel, column = token
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter) << 21);
    T* const c = static_cast<T*>(p.c);
    int u = 0;
    for (int t = pair; t < tiles; t += pairs, ++u) {
      const Tile tl = tile_at(p, t);
      const int buf = u & 1;
      const int chan = tl.n0 + rank * kChan + quarter * 32 + lane;
      const bool in = chan < p.n;
      const float sb = in ? __ldg(p.sb + chan) : 0.0f;
      const float bias = in && p.bias ? __ldg(p.bias + chan) : 0.0f;
      const bool got = wait(&acc_full[buf], (u / 2) & 1, abort);
      if (!__all_sync(0xffffffffu, got)) break;
      tc::fence_after_sync();
#pragma unroll 1
      for (int s = 0; s < kTok / 2; s += 32) {
        const int col = half * (kTok / 2) + s, tok = tl.m0 + col;
        if (tok >= p.m) break;
        const float sa = tok + lane < p.m ? __ldg(p.sa + tok + lane) : 0.0f;
        uint32_t r[32];
        tc::tmem_ld32_async(lane_base + buf * kTok + col, r);
        tc::tmem_wait_ld();
        T* out = c + static_cast<size_t>(tok) * p.n + chan;
        const int left = p.m - tok;
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          const float v = act<EPI>(acc_value<Q8>(r[q]) * __shfl_sync(0xffffffffu, sa, q) * sb + bias);
          if (in && q < left) *out = static_cast<T>(v);
          out += p.n;
        }
      }
      // the accumulator may be overwritten once every warp of the pair has read it
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_cluster(cluster_addr(&acc_empty[buf], 0));
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  cluster_sync();  // no arrival of either block is under way any more
  if (warp == kEpiWarps + 1) tmem_dealloc_pair(tmem, kTmemCols);
}

template <int Q8, typename T, int EPI>
cudaError_t launch_epi(const Call& c) {
  const size_t tiles_n = (c.p.n + 2 * kChan - 1) / (2 * kChan), tiles_m = (c.p.m + kTok - 1) / kTok;
  if (tiles_m > 0x7fffffffu / kGroup / 2 / tiles_n) return cudaErrorInvalidConfiguration;
  CUtensorMap ma, mb;
  if (!make_map(&ma, c.a, c.p.m, c.k, c.pitch, kTok / 2) || !make_map(&mb, c.b, c.p.n, c.k, c.pitch, kChan))
    return cudaErrorInvalidValue;
  const size_t smem = kStages * kStageBytes + 1024;
  auto kernel = matmul_pair_kernel<Q8, T, EPI>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const Params p = {c.p.a_scales, c.p.b_scales, c.p.bias, c.p.c, static_cast<int>(c.p.m), static_cast<int>(c.p.n),
                    static_cast<int>((c.k + kKBlock - 1) / kKBlock), static_cast<int>(tiles_n),
                    static_cast<int>(tiles_m)};
  const size_t pairs = static_cast<size_t>(c.sm_count) / 2, tiles = tiles_n * tiles_m;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (tiles < pairs ? tiles : pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, ma, mb, p);
}

template <int Q8, typename T>
cudaError_t launch_out(const Call& c) {
  switch (c.p.epilogue) {
    case FK_EPILOGUE_GELU_TANH: return launch_epi<Q8, T, FK_EPILOGUE_GELU_TANH>(c);
    case FK_EPILOGUE_GELU_ERF: return launch_epi<Q8, T, FK_EPILOGUE_GELU_ERF>(c);
    default: return launch_epi<Q8, T, FK_EPILOGUE_NONE>(c);
  }
}

template <int Q8>
cudaError_t launch_type(const Call& c) {
  return c.p.out_dtype == FK_F32 ? launch_out<Q8, float>(c) : launch_out<Q8, __nv_bfloat16>(c);
}

}  // namespace

cudaError_t launch_pair(const Call& c) {
  return c.p.dtype == FK_I8 ? launch_type<FK_I8>(c) : launch_type<FK_E4M3>(c);
}

cudaError_t read_pair_wait_timeouts(unsigned* out, bool reset) {
  cudaError_t e = cudaMemcpyFromSymbol(out, g_mm_wait_timeouts, sizeof(unsigned));
  if (e == cudaSuccess && reset) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(g_mm_wait_timeouts, &zero, sizeof(unsigned));
  }
  return e;
}

}  // namespace mm
}  // namespace fk
