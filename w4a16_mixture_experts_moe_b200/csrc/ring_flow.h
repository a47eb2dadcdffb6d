// Control flow around a ring of loads: what its consumers have to follow alike,
// and what its producer waits for before it ends. Plain C++ beside the kernels' code, so that it can be checked without a GPU.
#pragma once

#ifdef __CUDACC__
#define MOE_FLOW __device__ __forceinline__
#else
#define MOE_FLOW inline
#endif

namespace moe {

// Takes a group's stages from the ring, all or the next of them. wait(): the rows
// of the next stage, 0 at the group's end, below 0 if the wait gave up.
// products(rows): takes the stage, (rows + 15) / 16 additions to the consumer's
// sums. all(ok): a meeting of all consumers; whether each of them passed true.
// Returns how the sums stand, the same for all consumers, because what follows
// holds barriers, which one that went another way would leave the others waiting
// at: more of the group follows (behind `most` additions), its end, its end
// without further rows, or some consumer gave up.
enum { TAKEN_MORE, TAKEN_END, TAKEN_NOTHING, TAKEN_GAVE_UP };
template <class Wait, class Products, class All>
MOE_FLOW int take_stages(int most, Wait wait, Products products, All all) {
  int sums = 0, rows;
  while ((rows = wait()) > 0) {
    products(rows);
    if ((sums += (rows + 15) / 16) >= most) break;
  }
  return !all(rows >= 0) ? TAKEN_GAVE_UP : rows > 0 ? TAKEN_MORE : sums ? TAKEN_END : TAKEN_NOTHING;
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
