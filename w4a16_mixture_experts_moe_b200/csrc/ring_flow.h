// Control flow around a ring of loads: what its consumers have to follow alike,
// and what its producer waits for before it ends. Plain C++ beside the kernels' code, so that it can be checked without a GPU.
#pragma once

#ifdef __CUDACC__
#define MOE_FLOW __device__ __forceinline__
#else
#define MOE_FLOW inline
#endif

namespace moe {

// Sums up one group's stages from the ring. wait(): the rows of the next stage, 0
// at the group's end, below 0 if the wait gave up. clear(): sets the consumer's
// sums to zero. products(rows): takes the stage, (rows + 15) / 16 additions to
// them. Behind `most` additions (LONG; else there are no more) and at the end the sums pass on: put(first) for
// the consumers that write theirs to the group's sums first (over what is there
// if `first`), all(ok), a meeting of all consumers that says whether each of them
// passed true, add() for the others', and sync(), a plain meeting. Returns 1, 0
// for a group without rows, or -1 if any consumer gave up.
// A consumer that gives up goes to its next all(), where the others meet it,
// whichever group they are in by then; so each has to come to one more all()
// behind its last group.
template <bool LONG, class Wait, class Clear, class Products, class Put, class All, class Add, class Sync>
MOE_FLOW int sum_group(int most, Wait wait, Clear clear, Products products, Put put, All all, Add add, Sync sync) {
  int any = 0, rows;
  do {
    int sums = 0;
    clear();
    while ((rows = wait()) > 0) {
      products(rows);
      sums += (rows + 15) / 16;
      if (LONG && sums >= most) break;
    }
    if (rows == 0 && sums == 0 && !any) break;
    if (rows >= 0) put(!any);
    if (!all(rows >= 0)) return -1;
    add();
    sync();
    any = 1;
  } while (LONG && rows > 0);
  return any;
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
