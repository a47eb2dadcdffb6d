// How the tensor-core engine cuts a long reduction into parts.
// Plain C++ beside the kernels' code, so that it can be checked without a GPU.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

// The tensor core adds to its fp32 accumulator with truncation, an error that
// grows with the number of additions: 1e-6 of the result after 1024 products,
// 1.6e-5 after 14,336, and six times that where all products have one sign (1e-7
// of the result an addition of 16). A longer reduction is therefore cut into
// parts, which are added up in memory, rounded to nearest, in order.
// fp32 outputs: parts of at most F32_STEPS k-steps of 64, added in the output
// (14,336: 9e-7; 8 groups of 512 rows, N = 1024: 118 us, 95 with BF16 outputs in
// one part). BF16 outputs: the rounding of the output, half a step of 2e-3 to
// 4e-3, hides what BF16_STEPS lose (1e-4 for 16,384 products of one sign); longer
// ones are added in the workspace (a gradient of a million rows of one sign: off
// by up to 6.5e-3 beyond its rounding in one part).
constexpr int F32_WHOLE = 16, F32_STEPS = 14;
constexpr int BF16_WHOLE = 256, BF16_STEPS = 256;

// Parts of a reduction of `steps` k-steps.
template <bool F32>
MOE_HOST_DEVICE int reduction_parts(int steps) {
  constexpr int WHOLE = F32 ? F32_WHOLE : BF16_WHOLE, STEPS = F32 ? F32_STEPS : BF16_STEPS;
  return steps <= WHOLE ? 1 : (steps + STEPS - 1) / STEPS;
}

// The first k-step of part p; the end of the last for p = parts. (The product
// passes 32 bits from 173,000 k-steps on: a group of 11 million rows.)
MOE_HOST_DEVICE int part_start(int steps, int parts, int p) { return int(int64_t(steps) * p / parts); }

}  // namespace moe
