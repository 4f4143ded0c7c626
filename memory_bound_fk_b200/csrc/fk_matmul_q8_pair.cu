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
// Bound by the tensor cores and what feeds them: 8192 x 16384 x 4096 int8
// takes 318 us at 1965 MHz with operands of zeros (the MMAs alone 233; 64 B a
// clock and SM would have to come from L2 for that, 46 do, 13.5 TB/s), 334
// through tanh GELU; with random operands the GPU's power limit lowers the
// clock to about 1500 MHz, and it is 383 to 409 (2.7 to 2.9 POP/s), 395 to
// 425 through GELU.
//
// Each SM's tensor memory holds two accumulators, so the epilogue of one tile
// runs under the MMAs of the next.  Warps: eight for the epilogue (two per
// quarter of the lanes, halves of the tokens), one for the loads, one that
// issues MMAs (in the pair's leader).
#include <cuda.h>
#include <cuda_bf16.h>

#include "fk_mm.cuh"
#include "fk_mm_host.h"
#include "fk_q8.cuh"

namespace fk {
namespace mm {
namespace {

constexpr int kChan = 128;           // channels per block (256 per pair)
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (kEpiWarps + 2);
// TOK tokens per tile: a stage of one block holds its 128 channels and half
// of the tokens; 192 KB of stages either way.
template <int TOK>
struct Shape {
  static constexpr uint32_t kChanBytes = kChan * kKBlock;
  static constexpr uint32_t kStageBytes = kChanBytes + TOK / 2 * kKBlock;
  static constexpr int kStages = TOK == 256 ? 6 : 8;
  static constexpr uint32_t kSmem = kStages * kStageBytes + 1024;
  static_assert(kSmem + kSplitSmemLeast > kSmemOfSm, "clusters for few tokens would fit beside");
};
// Tiles go to pairs in groups of this many channel tiles by all token tiles,
// channels fastest, so that concurrent pairs share operands through L2.
constexpr int kGroup = 8;

struct Tile {
  int n0, m0;  // first channel of the pair's tile, first token
};
template <int TOK>
__device__ __forceinline__ Tile tile_at(const Params& p, int t) {
  const int per = kGroup * p.tiles_m, g = t / per, r = t - g * per;
  const int first = g * kGroup, width = p.tiles_n - first < kGroup ? p.tiles_n - first : kGroup;
  return Tile{(first + r % width) * 2 * kChan, r / width * TOK};
}

// ---------------------------------------------------------------- persistent

template <int Q8, int TOK, typename T, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_pair_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b, Params p) {
  constexpr int kStages = Shape<TOK>::kStages;
  constexpr uint32_t kStageBytes = Shape<TOK>::kStageBytes, kChanBytes = Shape<TOK>::kChanBytes;
  constexpr uint32_t kTmemCols = 2 * TOK;
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
  cluster_sync();  // every block's barriers stand
  if (warp == kEpiWarps + 1) {
    tmem_alloc_pair(&tmem_slot, kTmemCols);
    let_next_start();
  }
  tc::fence_before_sync();
  cluster_arrive();  // the pair's tensor memory: waited for by all but the load warp, which does that at its end
  after_previous();

  if (warp == kEpiWarps) {
    // ---- loads: a block's channels and its half of the tokens, counted on the leader's barrier
    int i = 0;
    if (lane == 0) {
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const Tile tl = tile_at<TOK>(p, t);
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
          tma_load_2d_pair(dst + kChanBytes, &tma_a, bar, kb * kKBlock, tl.m0 + rank * (TOK / 2));
        }
      }
    }
    __syncwarp();
    cluster_wait();
    // what was loaded has been read by the MMAs before the block exits
    for (int j = i > kStages ? i - kStages : 0; j < i; ++j)
      if (!drain(&empty[j % kStages], (j / kStages) & 1)) break;
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    // ---- MMAs, issued by the leader for both blocks
    cluster_wait();
    tc::fence_after_sync();
    if (rank == 0 && lane == 0) {
      const uint32_t tmem = tmem_slot;
      constexpr uint32_t HI = tc::smem_desc_hi(1024);
      constexpr uint32_t ID = idesc<Q8>(2 * kChan, TOK);
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
          const uint32_t a = a0 + st * (kStageBytes / 16), b = a + kChanBytes / 16;
#pragma unroll
          for (int q = 0; q < kKBlock / 32; ++q)
            mma_pair<Q8>(tmem + buf * TOK, tc::desc_join(a + 2 * q, HI), tc::desc_join(b + 2 * q, HI), ID,
                         (kb | q) != 0);
          commit_pair(&empty[st], 0);
        }
        if (ok) commit_pair(&acc_full[buf], 0);
      }
    }
    __syncwarp();
  } else {
    // ---- epilogue: lane = channel, column = token
    cluster_wait();
    tc::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    const int quarter = warp & 3, half = warp >> 2;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter) << 21);
    T* const c = static_cast<T*>(p.c);
    int u = 0;
    for (int t = pair; t < tiles; t += pairs, ++u) {
      const Tile tl = tile_at<TOK>(p, t);
      const int buf = u & 1;
      const int chan = tl.n0 + rank * kChan + quarter * 32 + lane;
      const bool in = chan < p.n;
      const float sb = in ? ld_param(p.sb + chan) : 0.0f;
      const float bias = in && p.bias ? ld_param(p.bias + chan) : 0.0f;
      // this warp's token scales, one token of each 32 per lane, fetched before the wait
      float sas[TOK / 64];
#pragma unroll
      for (int s = 0; s < TOK / 64; ++s) {
        const int tok = tl.m0 + half * (TOK / 2) + 32 * s + lane;
        sas[s] = tok < p.m ? ld_param(p.sa + tok) : 0.0f;
      }
      const bool got = wait(&acc_full[buf], (u / 2) & 1, abort, p.done_ns);
      if (!__all_sync(0xffffffffu, got)) {
        // what may have been issued for this tile and the next ends before the block does
        if (lane == 0 && drain(&acc_full[buf], (u / 2) & 1) && t + pairs < tiles)
          drain(&acc_full[buf ^ 1], ((u + 1) / 2) & 1);
        __syncwarp();
        break;
      }
      tc::fence_after_sync();
#pragma unroll
      for (int s = 0; s < TOK / 2; s += 32) {
        const int col = half * (TOK / 2) + s, tok = tl.m0 + col;
        if (tok >= p.m) break;
        const float sa = sas[s / 32];
        uint32_t r[32];
        tmem_ld32(lane_base + buf * TOK + col, r);
        T* out = c + static_cast<size_t>(tok) * p.n + chan;
        const int left = p.m - tok;
#pragma unroll
        for (int q = 0; q < 32; q += 2) {
          const float2 v = finish2<Q8, EPI>(r[q], r[q + 1], __shfl_sync(0xffffffffu, sa, q),
                                            __shfl_sync(0xffffffffu, sa, q + 1), sb, bias);
          if (in && q < left) *out = static_cast<T>(v.x);
          out += p.n;
          if (in && q + 1 < left) *out = static_cast<T>(v.y);
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
  cluster_sync();  // no arrival of either block is under way any more, and the other has read its accumulators
  if (warp == kEpiWarps + 1) tmem_dealloc_pair(tmem_slot, kTmemCols);
}

// ---------------------------------------------------------------- one tile per cluster, k split over its pairs

// When there are too few tiles to fill the GPU: the SPLIT pairs of a cluster
// take a share of k each, then every block keeps the sums of TOK / SPLIT of
// the tile's tokens for its 128 channels and pushes the rest of its
// accumulator into the shared memory of the blocks that own it (the stages,
// free once every pair's MMAs are done).  Added in the order of k.
template <int Q8, int TOK, int SPLIT, typename T, int EPI>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_pair_split_kernel(const __grid_constant__ CUtensorMap tma_a, const __grid_constant__ CUtensorMap tma_b,
                             Params p) {
  constexpr int kStages = Shape<TOK>::kStages, OWN = TOK / SPLIT;
  constexpr uint32_t kStageBytes = Shape<TOK>::kStageBytes, kChanBytes = Shape<TOK>::kChanBytes;
  static_assert(TOK * kChan * 4 <= kStages * kStageBytes, "the partial sums must fit the stages");
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t full[kStages], empty[kStages], done;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ uint32_t part_bad[2 * SPLIT];  // whether a block of the cluster gave up on a wait
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  uint32_t* red = reinterpret_cast<uint32_t*>(base);  // [SPLIT][OWN / 4][128 channels][4 tokens]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = static_cast<int>(cluster_ctarank()), side = rank & 1, leader = rank - side, part = rank >> 1;
  const Tile tl = tile_at<TOK>(p, static_cast<int>(blockIdx.x) / (2 * SPLIT));
  const int kb0 = static_cast<int>(static_cast<long long>(p.kblocks) * part / SPLIT);
  const int steps = static_cast<int>(static_cast<long long>(p.kblocks) * (part + 1) / SPLIT) - kb0;
  volatile int* abort = &abort_flag;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  cluster_sync();  // every block's barriers stand
  if (warp == kEpiWarps + 1) {
    tmem_alloc_pair(&tmem_slot, TOK);
    let_next_start();
  }
  tc::fence_before_sync();
  cluster_arrive();  // the pairs' tensor memory, as in the persistent kernel
  after_previous();

  const int quarter = warp & 3, half = (warp >> 2) & 1;
  const int cl = quarter * 32 + lane;  // channel within the block
  const int chan = tl.n0 + side * kChan + cl;
  const bool in = chan < p.n;
  float sb = 0.0f, bias = 0.0f, sas[OWN / 32];  // scales of this warp's channels and runs of 16 tokens
  if (warp == kEpiWarps) {
    int i = 0;
    if (lane == 0) {
      for (; i < steps; ++i) {
        const int st = i % kStages;
        if (i >= kStages && !wait(&empty[st], (i / kStages - 1) & 1, abort)) break;
        uint8_t* dst = base + st * kStageBytes;
        const uint32_t bar = cluster_addr(&full[st], leader);
        if (side == 0) mbar_arrive_expect_tx(&full[st], 2 * kStageBytes);
        tma_load_2d_pair(dst, &tma_b, bar, (kb0 + i) * kKBlock, tl.n0 + side * kChan);
        tma_load_2d_pair(dst + kChanBytes, &tma_a, bar, (kb0 + i) * kKBlock, tl.m0 + side * (TOK / 2));
      }
    }
    __syncwarp();
    cluster_wait();
    // what was loaded has been read by the MMAs before the stages are used again
    for (int j = i > kStages ? i - kStages : 0; j < i; ++j)
      if (!drain(&empty[j % kStages], (j / kStages) & 1)) {
        *abort = 1;
        break;
      }
    __syncwarp();
  } else if (warp == kEpiWarps + 1) {
    cluster_wait();
    tc::fence_after_sync();
    if (side == 0 && lane == 0) {
      const uint32_t tmem = tmem_slot;
      constexpr uint32_t HI = tc::smem_desc_hi(1024);
      constexpr uint32_t ID = idesc<Q8>(2 * kChan, TOK);
      const uint32_t a0 = tc::smem_desc_lo(smem_addr(base), 16);
      for (int i = 0; i < steps; ++i) {
        const int st = i % kStages;
        if (!wait(&full[st], (i / kStages) & 1, abort)) break;
        tc::fence_after_sync();
        const uint32_t a = a0 + st * (kStageBytes / 16), b = a + kChanBytes / 16;
#pragma unroll
        for (int q = 0; q < kKBlock / 32; ++q)
          mma_pair<Q8>(tmem, tc::desc_join(a + 2 * q, HI), tc::desc_join(b + 2 * q, HI), ID, (i | q) != 0);
        commit_pair(&empty[st], leader);
      }
      commit_pair(&done, leader);
    }
    __syncwarp();
  } else {
    cluster_wait();
    sb = in ? ld_param(p.sb + chan) : 0.0f;
    bias = in && p.bias ? ld_param(p.bias + chan) : 0.0f;
#pragma unroll
    for (int s = 0; s < OWN / 32; ++s) {
      const int tok = tl.m0 + part * OWN + 32 * s + half * 16 + (lane & 15);
      sas[s] = tok < p.m ? ld_param(p.sa + tok) : 0.0f;
    }
    if (!drain(&done, 0, p.done_ns)) {
      *abort = 1;
      drain(&done, 0);  // MMAs that still run end before their memory goes
    }
    tc::fence_after_sync();
  }
  __syncthreads();  // one verdict for the block
  if (tid < 2 * SPLIT) st_cluster(cluster_addr(&part_bad[rank], tid), *abort ? 1u : 0u);
  cluster_sync();  // all MMAs of the cluster are done: the stages may be overwritten, unless a block gave up
  bool good = true;
#pragma unroll
  for (int o = 0; o < 2 * SPLIT; ++o) good = good && part_bad[o] == 0;

  const uint32_t lane_base = tmem_slot + (static_cast<uint32_t>(quarter) << 21);
  if (warp < kEpiWarps && good) {
#pragma unroll 1
    for (int t = half * (TOK / 2); t < (half + 1) * (TOK / 2) && tl.m0 + t < p.m; t += 16) {
      if (t / OWN == part) continue;  // OWN is a multiple of 16: a run of 16 has one owner
      uint32_t r[16];
      tmem_ld16(lane_base + t, r);
      const uint32_t dst = cluster_addr(red + ((part * (OWN / 4) + t % OWN / 4) * kChan + cl) * 4, 2 * (t / OWN) + side);
#pragma unroll
      for (int q = 0; q < 4; ++q) st_cluster_v4(dst + q * kChan * 16, r + 4 * q);
    }
  }
  tc::fence_before_sync();
  cluster_sync();  // every partial sum has arrived
  tc::fence_after_sync();
  if (warp < kEpiWarps && good) {
#pragma unroll
    for (int i = 0; i < OWN / 32; ++i) {
      const int s = 32 * i + half * 16, t = part * OWN + s, tok = tl.m0 + t;
      if (tok >= p.m) break;
      uint32_t r[16];
      tmem_ld16(lane_base + t, r);
      const float sa = sas[i];
      T* out = static_cast<T*>(p.c) + static_cast<size_t>(tok) * p.n + chan;
      const int left = p.m - tok;
#pragma unroll
      for (int q = 0; q < 16; q += 4) {
        uint32_t sum[4];
#pragma unroll
        for (int o = 0; o < SPLIT; ++o) {
          uint32_t w[4];
          if (o == part) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = r[q + e];
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(red + ((o * (OWN / 4) + (s + q) / 4) * kChan + cl) * 4);
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = o == 0 ? w[e] : acc_add<Q8>(sum[e], w[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const float2 v = finish2<Q8, EPI>(sum[e], sum[e + 1], __shfl_sync(0xffffffffu, sa, q + e),
                                            __shfl_sync(0xffffffffu, sa, q + e + 1), sb, bias);
          if (in && q + e < left) *out = static_cast<T>(v.x);
          out += p.n;
          if (in && q + e + 1 < left) *out = static_cast<T>(v.y);
          out += p.n;
        }
      }
    }
  }
  tc::fence_before_sync();
  cluster_sync();  // the pair frees its tensor memory together: the other block has read its half too
  if (warp == kEpiWarps + 1) tmem_dealloc_pair(tmem_slot, TOK);
}

// ---------------------------------------------------------------- host side

// SPLIT = 0: the persistent kernel.
template <int Q8, int TOK, int SPLIT, typename T, int EPI>
cudaError_t launch_shape(const Call& c) {
  const size_t tiles_n = (c.p.n + 2 * kChan - 1) / (2 * kChan), tiles_m = (c.p.m + TOK - 1) / TOK;
  if (tiles_m > 0x7fffffffu / kGroup / 2 / tiles_n) return cudaErrorInvalidConfiguration;
  CUtensorMap ma, mb;
  if (!make_map(&ma, c.a, c.p.m, c.k, c.pitch_a, TOK / 2) || !make_map(&mb, c.b, c.p.n, c.k, c.pitch_b, kChan))
    return cudaErrorInvalidValue;
  void (*kernel)(CUtensorMap, CUtensorMap, Params);
  if constexpr (SPLIT == 0)
    kernel = matmul_pair_kernel<Q8, TOK, T, EPI>;
  else
    kernel = matmul_pair_split_kernel<Q8, TOK, SPLIT, T, EPI>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(Shape<TOK>::kSmem));
  if (e != cudaSuccess) return e;
  const Params p = make_params(c, tiles_n, tiles_m);
  const size_t pairs = static_cast<size_t>(c.sm_count) / 2, tiles = tiles_n * tiles_m;
  return launch_overlapped(kernel, static_cast<unsigned>(SPLIT > 0 ? 2 * SPLIT * tiles : 2 * (tiles < pairs ? tiles : pairs)),
                           kThreads, Shape<TOK>::kSmem, SPLIT > 0 ? 2 * SPLIT : 2, c.stream, ma, mb, p);
}

// How a product is cut: tokens per tile, pairs that share a tile's k (0: the
// persistent kernel).  The time of each cut is estimated as
//     persistent  fixed + waves * steps * step
//     split       waves * (fixed + steps / split * step)
// with `waves` the tiles over what runs at once, `steps` the 128-code steps
// of k, and constants fitted to B200 runs in a captured chain (us; fixed:
// launch, prologue, first loads, epilogue, and the exchange of partial sums;
// step: one 128-code step, of which the MMAs take 0.27 for 256 tokens and
// 0.15 for 128).  The fit and what was measured, tokens x channels x k:
//     100 x 1024 x 1024   128/4  5.6 (5.7)    128/0  6.6 (6.5)   256/2  7.5 (7.6)
//     256 x 4096 x 4096   128/2  9.9 (12.0)   256/2 11.6 (13.1)  256/0 15.6 (16.3)
//     512 x 4096 x 4096   256/2 11.6 (14.5)   128/0 14.2 (15.7)  256/0 15.6 (16.7)
//     768 x 1024 x 8192   256/4 12.0 (14.7)   128/2 15.0 (16.4)  256/0 26.3 (25.9)
//     1024 x 4096 x 4096  256/0 15.6 (17.4)   128/0 24.5 (27.0)  256/2 23.1 (27.8)
// Weights that come from HBM add to every cut alike and are left out.
struct Cut {
  int tok, split;
  double fixed, step;
  size_t at_once;  // tiles that run at the same time (cudaOccupancyMaxActiveClusters: clusters of 2, 4, 8)
};
constexpr Cut kCuts[] = {{256, 0, 4.9, 0.335, 74}, {128, 0, 4.0, 0.320, 74}, {256, 2, 6.2, 0.335, 33},
                         {128, 2, 4.8, 0.320, 33}, {256, 4, 6.6, 0.335, 15}, {128, 4, 5.0, 0.320, 15}};

int best_cut(size_t m, size_t n, size_t kblocks) {
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 6; ++i) {
    const Cut& c = kCuts[i];
    const size_t tiles = ((n + 2 * kChan - 1) / (2 * kChan)) * ((m + c.tok - 1) / c.tok);
    const double waves = static_cast<double>((tiles + c.at_once - 1) / c.at_once);
    if (c.split > 0 && kblocks < static_cast<size_t>(c.split)) continue;
    const double steps = c.split > 0 ? static_cast<double>((kblocks + c.split - 1) / c.split)
                                     : static_cast<double>(kblocks);
    const double t = c.split > 0 ? waves * (c.fixed + steps * c.step) : c.fixed + waves * steps * c.step;
    if (i == 0 || t < least) {
      least = t;
      best = i;
    }
  }
  return best;
}

template <int Q8, typename T, int EPI>
cudaError_t launch_epi(const Call& c) {
  switch (best_cut(c.p.m, c.p.n, (c.k + kKBlock - 1) / kKBlock)) {
    case 1: return launch_shape<Q8, 128, 0, T, EPI>(c);
    case 2: return launch_shape<Q8, 256, 2, T, EPI>(c);
    case 3: return launch_shape<Q8, 128, 2, T, EPI>(c);
    case 4: return launch_shape<Q8, 256, 4, T, EPI>(c);
    case 5: return launch_shape<Q8, 128, 4, T, EPI>(c);
    default: return launch_shape<Q8, 256, 0, T, EPI>(c);
  }
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
