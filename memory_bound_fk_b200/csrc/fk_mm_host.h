// fk_mm_host.h -- host side shared by the kernels of the 8-bit product: the
// launch parameters and the TMA tensor maps.  Not installed.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "fk_q8_internal.h"

namespace fk {
namespace mm {

constexpr int kKBlock = 128;  // codes of k per stage (one swizzled row)

// Limits of the kernels' waits, ns: for a stage or an accumulator; and what the
// wait for a finished product has more for each 128-code step of k (a step
// takes 0.3 us alone).
constexpr uint64_t kWaitNs = 1000000000ull, kStepNs = 2000;

// Shared memory that a block of the kernels for few tokens takes at the least.
// A pair of SMs takes tensor memory on both at once: it must not find another
// cluster's block there whose fellow waits for columns that the pair holds.
// No two such blocks fit an SM together.
constexpr unsigned kSmemOfSm = 228 * 1024, kSplitSmemLeast = 96 * 1024;

struct Params {
  const float* sa;
  const float* sb;
  const float* bias;
  void* c;
  int m, n;
  int kblocks;  // ceil(k / 128)
  int tiles_n, tiles_m;
  uint64_t done_ns;  // limit of the wait for a finished product
};

// A product whose operands TMA can read: [m, k] and [n, k] with row pitches
// that are multiples of 16 bytes.
struct Call {
  const void *a, *b;
  size_t k, pitch_a, pitch_b;
  MatmulQ8Args p;
  int sm_count;
  cudaStream_t stream;
};

inline Params make_params(const Call& c, size_t tiles_n, size_t tiles_m) {
  const size_t kblocks = (c.k + kKBlock - 1) / kKBlock;
  return {c.p.a_scales, c.p.b_scales, c.p.bias, c.p.c, static_cast<int>(c.p.m), static_cast<int>(c.p.n),
          static_cast<int>(kblocks), static_cast<int>(tiles_n), static_cast<int>(tiles_m),
          c.p.give_up ? 0 : kWaitNs + kStepNs * kblocks};
}

// [rows, k] codes in boxes of 128 codes x box_rows rows, 128-byte swizzle;
// outside reads 0.
bool make_map(CUtensorMap* m, const void* ptr, size_t rows, size_t k, size_t pitch, int box_rows);

// The kernel for many tokens (fk_matmul_q8_pair.cu).
cudaError_t launch_pair(const Call& c);
cudaError_t read_pair_wait_timeouts(unsigned* out, bool reset);

}  // namespace mm
}  // namespace fk
