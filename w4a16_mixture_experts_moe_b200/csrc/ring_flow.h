// Control flow that the consumers of a ring of loads have to follow alike. Plain
// C++ beside the kernels' code, so that it can be checked without a GPU.
#pragma once

#ifdef __CUDACC__
#define MOE_FLOW __device__ __forceinline__
#else
#define MOE_FLOW inline
#endif

namespace moe {

// Takes a group's stages from the ring. wait(): the rows of the next stage, 0
// at the group's end, below 0 if the wait gave up. products(rows): takes the
// stage. all(ok): a meeting of all consumers; whether each of them passed true.
// Returns 1, 0 for a group without rows, or -1 if any consumer gave up: the same
// for all, because what follows holds barriers, which a consumer that went
// another way would leave the others waiting at.
template <class Wait, class Products, class All>
MOE_FLOW int take_group(Wait wait, Products products, All all) {
  int any = 0, rows;
  while ((rows = wait()) > 0) {
    products(rows);
    any = 1;
  }
  return all(rows == 0) ? any : -1;
}

}  // namespace moe
