// Control flow around a ring of loads: what its consumers have to follow alike,
// and what its producer waits for before it ends. Plain C++ beside the kernels' code, so that it can be checked without a GPU.
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

// wait(slot, parity) for the last use of each slot of a ring that has been used:
// the loads that may be in flight when use `round` of `slot` comes next.
template <class Wait>
MOE_FLOW void last_uses(int stages, int slot, int round, Wait wait) {
  for (int q = 0; q < stages; ++q) {
    const int uses = round + (q < slot ? 1 : 0);
    if (uses > 0) wait(q, (uses - 1) & 1);
  }
}

}  // namespace moe
