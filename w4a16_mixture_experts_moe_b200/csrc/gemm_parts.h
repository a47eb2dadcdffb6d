// How the tensor-core engine cuts a long reduction of an fp32 output into parts.
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
// 1.6e-5 after 14,336. For fp32 outputs a longer reduction is therefore cut into
// parts of at most F32_STEPS k-steps, which are added up in memory, rounded to
// nearest, in order (14,336: 9e-7; 8 groups of 512 rows, N = 1024: 118 us, 95
// with BF16 outputs in one part).
constexpr int F32_WHOLE = 16, F32_STEPS = 14;

// Parts of a reduction of `steps` k-steps.
template <bool F32>
MOE_HOST_DEVICE int reduction_parts(int steps) {
  return !F32 || steps <= F32_WHOLE ? 1 : (steps + F32_STEPS - 1) / F32_STEPS;
}

// The first k-step of part p; the end of the last for p = parts. (The product
// passes 32 bits from 173,000 k-steps on: a group of 11 million rows.)
MOE_HOST_DEVICE int part_start(int steps, int parts, int p) { return int(int64_t(steps) * p / parts); }

}  // namespace moe
