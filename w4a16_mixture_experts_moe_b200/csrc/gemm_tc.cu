// BF16 products over ragged row groups on the 5th-generation tensor cores
// (tcgen05.mma, fp32 accumulators in tensor memory). Three directions of one
// weight matrix W_e [N][K] per group e of rows:
//   fwd    y[r]  = x[r] W_e^T           dgrad  dx[r] = dy[r] W_e
//   wgrad  dW_e[n] = sum_r dy[r][n] x[r]
// and, for a single group, low-rank adapters added inside the same sums
// (fwd: + u[r] B_a^T, dgrad: + du[r] A_a for the adapter a of row r's segment).
//
// Every direction puts the output's contiguous dimension on the MMA's M side
// (lanes of tensor memory: a warp then stores neighbouring addresses) and the
// output's rows on its N side, whose width follows the group: a group of 40
// rows runs N = 48, so ragged groups cost little padding. A pair of CTAs
// (cta_group::2) shares one tile of 256 output columns x up to 256 rows: each
// CTA loads its own 128 columns of A and half of the rows of B, so a k-step of
// 64 brings 32 KB into each SM for 2 x 128 x 256 x 64 multiply-adds. A tile
// owned by one CTA would load 48 KB for the same work per SM.
//
// Operand layouts: a dimension that is contiguous in memory is contiguous in
// shared memory too (128-byte swizzle), so dgrad and wgrad need no transposed
// copies: the matrix descriptors name the operand MN-major where the reduction
// runs over memory rows (W in dgrad, both operands in wgrad).
//
// Adapters ride on the reduction: after the k-steps over W, each segment that
// covers whole 16-row blocks of the tile adds ceil(rank / 64) k-steps over
// just those accumulator columns, whose A is the adapter's B_a (A_a) and whose
// B is the segment's rows of u (du): the sums never leave tensor memory. The
// blocks that several segments share get their part in the epilogue, from fp32
// sums that a small launch before this one has made row by row (lora.cu). No
// row is ever multiplied by another request's adapter, not even as a zero: an
// adapter that holds infinities or NaN spoils its own rows only.
//
// wgrad's last k-step ends inside a block of 64 rows: the rows of the next
// group, whatever they hold, are set to zero in shared memory (both operands).
//
// Per CTA: warps 0-7 epilogue (two accumulators of 256 columns, so it overlaps
// the next tile's MMAs), warps 8 and 12 issue the TMA loads of A and B into a
// six-deep ring, warp 9 zeroes the tail of wgrad's last k-steps, and in the
// pair's first CTA warp 11 waits for each k-step and hands it over a named
// barrier to warp 10, which issues the MMAs of both CTAs and touches no memory
// between them (a warp's shared-memory operations behind its MMAs are held
// until those finish, which would drain the tensor core at every k-step). The
// loads of both CTAs count their bytes on the first CTA's barrier (a load of a
// pair may name its peer's), so a k-step costs no message between the CTAs.
// All waits are bounded (see tma.cuh).
#include "gemm.cuh"
#include "gemm_parts.h"

namespace moe {
namespace gt {

using namespace tma;

constexpr int BK = 64;             // reduction per k-step (128 bytes: one swizzle row)
constexpr int BMC = 128;           // output columns per CTA (256 per pair)
constexpr int BN = 256;            // rows per tile
constexpr int STAGES = 6;
constexpr int A_BYTES = BMC * BK * 2;
constexpr int B_BYTES = BN / 2 * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int A_WARP = 8, FIX_WARP = 9, MMA_WARP = 10, WAIT_WARP = 11, B_WARP = 12;
constexpr int THREADS = 416;
constexpr int HANDOFF_BAR = 1;  // named barrier of the waiter and the MMA warp
// A k-step's first handoff: its MMAs (0-4), bits below, or HAND_STOP. With
// HAND_SET two more follow: the width / 16, then the first column / 16 or
// HAND_FIRST (a tile's first k-step, which overwrites the accumulator).
constexpr int HAND_KK = 7, HAND_LAST = 8, HAND_SET = 16, HAND_STOP = 31, HAND_FIRST = 31;
constexpr int ROW_BLOCK = 16;      // row tiles that share a sweep over the output columns
constexpr int OUT_ROWS = 32;       // output rows per staged store
constexpr int OUT_F32_ROWS = 16;   // fp32: per staged store of a warp's 32 columns
constexpr int OUT_BYTES = OUT_ROWS * BMC * 2;  // of the four epilogue warps of a half
// Each half has two staging buffers: with one, every 32 rows wait for the store
// before them to have been read (BF16 gradients of 8 experts of 64 rows, K = 4096,
// N = 14336: 238 -> 189 us; 64 experts of 256 rows, K = 2048, N = 1024: 94 -> 76).
constexpr int SMEM = STAGES * STAGE_BYTES + 4 * OUT_BYTES + 3 * 1024 /*Shared*/;
constexpr int OUT_BAR = 2;         // named barriers 2, 3: the four epilogue warps that share a staging buffer

// One k-step, written by the first CTA's producer for its waiter.
struct Step {
  int kk;      // MMAs of K = 16 (0: none)
  int flags;   // STEP_*
  int n16;     // MMA width / 16
  int col;     // first accumulator column
};
constexpr int STEP_FIRST = 1, STEP_LAST = 2, STEP_STOP = 4;
constexpr int STEP_EXT = 16;      // an adapter's k-step: its own width and first column
constexpr int STEP_FIX_TAIL = 8;  // wgrad: the reduction ends inside the last MMA's 16 rows; warp 9 zeroes the rest

struct Shared {
  uint64_t full[STAGES], empty[STAGES];        // full: the first CTA's counts both CTAs' loads
  uint64_t landed[STAGES], fixed[STAGES];      // k-steps with a tail to zero: this CTA's loads / both CTAs' zeroing
  uint64_t tmem_full[2], tmem_empty[2];
  Step step[STAGES];
  uint32_t tmem_base;
  int32_t abort;
  int32_t total;
  int32_t lo[MAX_E + 1];        // the groups' first rows
  union {
    int32_t tstart[MAX_E + 1];  // first tile of each group (fwd, dgrad)
    int16_t order[MAX_E];       // groups by falling row count (wgrad)
  };
  __device__ __forceinline__ int cnt(int e) const { return max(0, lo[e + 1] - lo[e]); }  // rows of group e
};
static_assert(sizeof(Shared) <= 3 * 1024, "shared tables budget");
static_assert(EPI_WARPS * 2 * OUT_F32_ROWS * 128 <= 4 * OUT_BYTES, "staging buffers of fp32 outputs");
static_assert(SMEM <= 227 * 1024, "shared memory budget");

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Arrives on the barrier at `bar`'s offset in the pair's first CTA. What has to
// be ordered before it here is not generic memory traffic: reads of tensor
// memory (tcgen05.wait, tcgen05.fence) and shared memory handed to the tensor
// core (fence.proxy.async), both completed by their own instructions. So the
// arrive carries no cluster-scope release, which would wait for every global
// store in flight: 1700 cycles a tile in the epilogue, 1000 to 3700 behind a
// zeroed tail.
__device__ __forceinline__ void arrive_leader(uint64_t *bar) {
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, 0;\n"
      " mbarrier.arrive.shared::cluster.b64 _, [a];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}
// TMA tile loads whose bytes are counted on a barrier of the pair's first CTA
// (`bar`: its shared::cluster address).
__device__ __forceinline__ void pair_load_2d(void *dst, const CUtensorMap *tm, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(void *dst, const CUtensorMap *tm, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_4d(void *dst, const CUtensorMap *tm, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
      "%4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t leader_addr(uint64_t *bar) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(bar)));
  return a;
}

// Bounded wait (see tma::wait_bounded), its first poll inline.
__device__ __forceinline__ bool wait(Shared &sh, uint64_t *bar, uint32_t parity, int32_t *err, bool drain = false) {
  return mbar_try(bar, parity) || wait_bounded(&sh.abort, bar, parity, err, drain);
}

// Waiter and MMA warp meet: returns how many of the 64 threads voted.
__device__ __forceinline__ int handoff(bool vote) {
  uint32_t cnt;
  asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n bar.red.popc.u32 %0, %2, 64, p;\n}\n"
               : "=r"(cnt)
               : "r"(uint32_t(vote)), "n"(HANDOFF_BAR)
               : "memory");
  return int(cnt);
}

// Shared-memory matrix descriptor, 128-byte swizzle, version 1. K-major: rows
// of 128 bytes, 8-row atoms 1024 bytes apart (stride offset). MN-major: rows
// are reduction indices of 64 output indices each; 8-row atoms 1024 bytes
// apart along the reduction (stride offset), the next 64 output indices `lbo`
// bytes away (leading offset).
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= uint64_t((saddr >> 4) & 0x3FFF);
  d |= uint64_t((lbo >> 4) & 0x3FFF) << 16;
  d |= uint64_t(1024 >> 4) << 32;
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}

// Instruction descriptor: fp32 sums, BF16 A and B, their major-ness, N and M = 256.
__device__ __forceinline__ constexpr uint32_t idesc_bf16(bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (uint32_t(256 >> 4) << 24);
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
// Arrives on `bar` in both CTAs of the pair once the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(uint16_t(3))
      : "memory");
}
// 16 accumulator columns of the warp's 32 lanes; the wait is part of the
// statement, so no use of the registers can be scheduled before it.
__device__ __forceinline__ void tmem_ld16(uint32_t ta, uint32_t (&a)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
        "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15])
      : "r"(ta)
      : "memory");
}

// Tensor maps of one launch. A k-step's operand is one load where the layout
// allows it: each load instruction costs the TMA unit time of its own (five
// loads a k-step instead of two took the wide product from 1.54 to 1.77 ms).
struct Maps {
  CUtensorMap a;   // fwd: 128 rows of W. dgrad, wgrad: 64 reduction rows x 64 columns (x 2 blocks if a_wide)
  CUtensorMap b[3];   // fwd, dgrad: 32, 64, 128 rows (the first that holds the tile's half: rows behind it are read
                      // for nothing, which costs less than a second load). wgrad: 64 reduction rows x 64 columns,
                      // x 2 blocks (if b_wide)
  CUtensorMap ea, eb[3];  // adapters: like a and b
  CUtensorMap out;     // output: 32 rows x 64 columns (BF16), 16 rows x 32 columns (fp32)
  int a_wide, b_wide;
};

// 32 accumulator columns of lanes ta .. ta + 15, as 8-column fragments: thread
// t holds, of columns 8 i .. 8 i + 7, a[4 i], a[4 i + 1] = lane t / 4, columns
// 2 (t % 4) and the next, a[4 i + 2], a[4 i + 3] = the same of lane t / 4 + 8.
__device__ __forceinline__ void tmem_ld_frag(uint32_t ta, uint32_t (&a)[16], uint32_t (&b)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(a[8]),
        "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]), "=r"(b[0]),
        "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]), "=r"(b[8]), "=r"(b[9]),
        "=r"(b[10]), "=r"(b[11]), "=r"(b[12]), "=r"(b[13]), "=r"(b[14]), "=r"(b[15])
      : "r"(ta), "r"(ta + (16u << 16))
      : "memory");
}
// Four 8 x 8 matrices, stored transposed: lane 8 m + r gives the address of row r of matrix m.
__device__ __forceinline__ void stmatrix_trans(uint32_t saddr, uint32_t r0, uint32_t r1, uint32_t r2, uint32_t r3) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(r0), "r"(r1),
               "r"(r2), "r"(r3)
               : "memory");
}
// A box from shared memory, stored or (F32, add) added to what is there, rounded to nearest.
template <bool F32>
__device__ __forceinline__ void store_2d(const CUtensorMap *tm, uint32_t src, int c0, int c1, bool add = false) {
  if (F32 && add)
    asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(c0), "r"(c1), "r"(src)
                 : "memory");
}
template <bool F32>
__device__ __forceinline__ void store_3d(const CUtensorMap *tm, uint32_t src, int c0, int c1, int c2, bool add = false) {
  if (F32 && add)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(tm)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
}

struct Tile {
  int e;       // group
  int row;     // first row of the output tile (fwd, dgrad: row of x / dy; wgrad: row n of dW_e)
  int nvalid;  // output rows of the tile
  int f0;      // first output column of the pair
};

// Tile t of the list. fwd and dgrad: group by group; a group's rows are cut
// into equal tiles of at most bn (a multiple of 16), and up to ROW_BLOCK row
// tiles run over one 256-column slab of W before the next slab, so W streams
// from HBM once per ROW_BLOCK row tiles while the rows stay in L2. wgrad:
// groups by falling row count, so the longest reductions start first.
template <int MODE>
__device__ __forceinline__ Tile decode_tile(const Shared &sh, const TcGemmArgs &a, int t) {
  Tile x;
  const int FT = (a.M + 2 * BMC - 1) / (2 * BMC);
  if (MODE == GEMM_WGRAD) {
    const int NT = (a.NC + BN - 1) / BN;
    const int g = t / (FT * NT), rem = t - g * FT * NT;
    x.e = sh.order[g];
    x.f0 = rem % FT * 2 * BMC;
    x.row = rem / FT * BN;
    x.nvalid = min(BN, a.NC - x.row);
  } else {
    int lo_e = 0, hi_e = a.groups;  // largest e with tstart[e] <= t
    while (hi_e - lo_e > 1) {
      const int mid = (lo_e + hi_e) >> 1;
      if (sh.tstart[mid] <= t) lo_e = mid; else hi_e = mid;
    }
    const int cnt = sh.cnt(lo_e), idx = t - sh.tstart[lo_e];
    const int rt = (cnt + a.bn - 1) / a.bn;
    const int w = ((cnt + rt - 1) / rt + 15) & ~15;
    const int blk = idx / (ROW_BLOCK * FT), rem = idx - blk * ROW_BLOCK * FT;
    const int nr = min(ROW_BLOCK, rt - blk * ROW_BLOCK);
    const int f = rem / nr, r = blk * ROW_BLOCK + rem - f * nr;
    x.e = lo_e;
    x.f0 = f * 2 * BMC;
    x.row = sh.lo[lo_e] + r * w;
    x.nvalid = min(w, cnt - r * w);
  }
  return x;
}

// Whether several segments share the n <= 16 rows from `row`; *first: the
// segment of the first of them.
__device__ __forceinline__ bool shared_block(const TcGemmArgs &a, int row, int n, int *first = nullptr) {
  const int s0 = a.row_seg[row];
  if (first) *first = s0;
  return s0 != a.row_seg[row + n - 1];
}

// The adapters' part of a 16-row block that several segments share (a block
// of one segment has it in its sums already): n <= 16 rows from `row`.
__device__ __forceinline__ void add_shared_block(const TcGemmArgs &a, int row, int n, int f, uint32_t (&v)[16]) {
  int s0;
  if (!shared_block(a, row, n, &s0)) return;
  const int64_t r0 = a.delta_by_seg ? int64_t(min(max(s0, 0), a.segs - 2) + 1) * 16 : row;
  const float *d = a.delta + r0 * a.M + min(f, a.M - 1);
  float add[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) add[j] = j < n ? d[int64_t(j) * a.M] : 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + add[j]);
}

// Part p of a long reduction: adds what the parts before it left in the workspace
// to 16 accumulator rows of one column, and leaves them there itself unless it
// is the last (true: nothing to store yet). A thread meets its own values only.
__device__ __forceinline__ bool add_part(const TcGemmArgs &a, int p, int parts, int row, int col, uint32_t (&v)[16]) {
  float *s = a.sums + (int64_t(blockIdx.x) * BN + row) * BMC + col;
  if (p > 0) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) + s[j * BMC]);
  }
  if (p + 1 == parts) return false;
#pragma unroll
  for (int j = 0; j < 16; ++j) s[j * BMC] = __uint_as_float(v[j]);
  return true;
}

__device__ __forceinline__ void out_sync(int part) {
  asm volatile("bar.sync %0, 128;" ::"r"(OUT_BAR + part) : "memory");
}
__device__ __forceinline__ uint32_t pack_acc(uint32_t lo, uint32_t hi) {
  return pack_bf16x2(__uint_as_float(lo), __uint_as_float(hi));
}

// Stores n <= 16 output rows of column f (rows a.ldo elements apart from
// element `at`), or adds to them (fp32): a thread adds to its own values only,
// in order, without waiting for what they held. `whole`: all of the warp's
// columns exist. BF16 values go two rows per store: neighbouring lanes swap one
// value each, so an even lane holds columns f, f + 1 of row j and an odd lane
// f - 1, f of row j + 1.
template <bool F32>
__device__ __forceinline__ void store_block(const TcGemmArgs &a, int64_t at, int n, int f, bool whole, bool add,
                                            const uint32_t (&v)[16]) {
  if (F32) {
    float *o = static_cast<float *>(a.out) + at;
    const bool full = n == 16 && whole;
    if (add) {
#pragma unroll
      for (int j = 0; j < 16; ++j, o += a.ldo)
        if (full || (j < n && f < a.M)) asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(o), "f"(__uint_as_float(v[j])) : "memory");
    } else if (full) {
#pragma unroll
      for (int j = 0; j < 16; ++j, o += a.ldo) *o = __uint_as_float(v[j]);
    } else if (f < a.M) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < n) o[j * a.ldo] = __uint_as_float(v[j]);
    }
  } else {
    const int odd = threadIdx.x & 1;
    uint16_t *o = static_cast<uint16_t *>(a.out) + at + odd * a.ldo - odd;
    const int64_t two = 2 * a.ldo;
    const bool full = n == 16 && whole;
#pragma unroll
    for (int j = 0; j < 16; j += 2, o += two) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
      const uint32_t pk = pack_bf16x2(__uint_as_float(odd ? got : v[j]), __uint_as_float(odd ? v[j + 1] : got));
      if (full || (j + odd < n && f < a.M)) *reinterpret_cast<uint32_t *>(o) = pk;
    }
  }
}

// The map of B for `half` rows per CTA: boxes of 32, 64, 128 rows.
__device__ __forceinline__ int row_box(int half) { return half <= 32 ? 0 : half <= 64 ? 1 : 2; }

// Adapters join the two directions of a projection, whose outputs are BF16.
template <int MODE, bool F32>
constexpr bool ADAPTERS = MODE != GEMM_WGRAD && !F32;

// The pair's i-th tile, in a snake over the pairs.
__device__ __forceinline__ int sched_pos(int i) {
  const int G = int(gridDim.x) >> 1, c = int(blockIdx.x) >> 1;
  return i * G + ((i & 1) ? G - 1 - c : c);
}

// One producer warp: A_SIDE issues the loads of A, announces each k-step's
// bytes and describes it to the waiter; the other issues the loads of B. (One
// warp issuing both took 490 cycles a k-step, as long as its MMAs.) The warp
// stays converged and elects the issuing lane, which keeps the loads' operands
// in uniform registers.
template <int MODE, bool F32, bool LONG, bool A_SIDE>
__device__ __forceinline__ void produce(Shared &sh, const TcGemmArgs &a, const Maps &m, uint8_t *smem, uint32_t rank,
                                        int total) {
  int s = 0, round = 0;  // ring slot and its use
  bool ok = true;
  const uint32_t full0 = leader_addr(&sh.full[0]);
  auto slot = [&]() {  // waits until the ring's next slot is free
    ok = __all_sync(0xffffffffu, wait(sh, &sh.empty[s], (round & 1) ^ 1, a.err));
    return ok;
  };
  auto next = [&]() {
    if (++s == STAGES) { s = 0; ++round; }
  };
  for (int i = 0; ok; ++i) {
    const int t = sched_pos(i);
    if (t >= total) break;
    const Tile tl = decode_tile<MODE>(sh, a, t);
    const int n16 = (tl.nvalid + 15) >> 4, half = n16 * 8;  // rows (wgrad: columns of dy) per CTA
    const int f = tl.f0 + int(rank) * BMC, r0 = tl.row + int(rank) * half;
    const int red = MODE == GEMM_WGRAD ? sh.cnt(tl.e) : a.KD;
    const int nsteps = MODE == GEMM_WGRAD && red == 0 ? 1 : (red + BK - 1) / BK;
    const int box = row_box(half), nb = (half + 63) >> 6;  // B's map; wgrad: 64-column blocks of B
    const int b_bytes = MODE == GEMM_WGRAD ? nb * 8192 : (32 << box) * BK * 2;
    // adapters: the next segment that has one and covers whole 16-row blocks of
    // the tile; the lanes look at 32 segments at a time
    const int lane = threadIdx.x & 31, tile_end = tl.row + tl.nvalid;
    int sg = ADAPTERS<MODE, F32> && a.adapter ? first_segment(a.offsets, a.segs, tl.row) : 0;
    int my_lo = 0, my_hi = 0, my_a = -1, seg_lo = 0, seg_hi = 0, seg_a = -1;
    uint32_t found = 0;
    bool end = !ADAPTERS<MODE, F32> || !a.adapter;
    auto next_seg = [&]() {
      while (found == 0) {
        if (end) return false;
        const bool in = sg + lane < a.segs;
        const int o0 = in ? a.offsets[sg + lane] : INT32_MAX, o1 = in ? a.offsets[sg + lane + 1] : 0;
        my_a = in ? a.adapter[sg + lane] : -1;
        my_lo = o0 < tile_end ? (max(o0, tl.row) - tl.row + 15) & ~15 : 0;
        my_hi = o1 >= tile_end ? n16 * 16 : (max(o1, tl.row) - tl.row) & ~15;
        found = __ballot_sync(0xffffffffu, o0 < tile_end && my_hi > my_lo && my_a >= 0 && my_a < a.n_adapters);
        end = __any_sync(0xffffffffu, o0 >= tile_end);
        sg += 32;
      }
      const int l = __ffs(found) - 1;
      found &= found - 1;
      seg_lo = __shfl_sync(0xffffffffu, my_lo, l);
      seg_hi = __shfl_sync(0xffffffffu, my_hi, l);
      seg_a = __shfl_sync(0xffffffffu, my_a, l);
      return true;
    };
    bool more = false, known = false;  // another adapter step follows (looked up behind the first loads)
    const int parts = LONG ? reduction_parts<F32>(nsteps) : 1;
    int part = 0, part_end = parts == 1 ? nsteps : part_start(nsteps, parts, 1);
    bool part_first = true;
    for (int ks = 0; ks < nsteps && slot(); ++ks) {
      if (ADAPTERS<MODE, F32> && ks + 1 == nsteps) { more = next_seg(); known = true; }
      const bool part_last = ks + 1 == (LONG ? part_end : nsteps);
      uint8_t *sa = smem + s * STAGE_BYTES, *sb = sa + A_BYTES;
      const int left = min(BK, red - ks * BK);
      const bool fix = MODE == GEMM_WGRAD && (left & 15);
      // a k-step with a tail to zero: the zeroing warp sees this CTA's loads
      // through, and the waiter waits for both CTAs' zeroing
      const uint32_t bar = fix ? smem_u32(&sh.landed[s]) : full0 + s * 8;
      if (elect_one()) {
        if (A_SIDE) {
          sh.step[s] = Step{max(0, (left + 15) >> 4),
                            (part_first ? STEP_FIRST : 0) | (part_last && !more ? STEP_LAST : 0) | (fix ? STEP_FIX_TAIL : 0),
                            n16, 0};
          if (fix) mbar_arrive_expect_tx(&sh.landed[s], A_BYTES + b_bytes);
          if (rank == 0) {
            if (fix || left <= 0) mbar_arrive(&sh.full[s]);
            else mbar_arrive_expect_tx(&sh.full[s], 2 * (A_BYTES + b_bytes));
          }
        }
        if (MODE == GEMM_WGRAD) {
          const int row = sh.lo[tl.e] + ks * BK;
          if (left <= 0) {  // an empty group: no loads
          } else if (A_SIDE) {
            if (m.a_wide) {
              pair_load_3d(sa, &m.a, 0, row, f >> 6, bar);
            } else {
              pair_load_2d(sa, &m.a, f, row, bar);
              pair_load_2d(sa + 8192, &m.a, f + 64, row, bar);
            }
          } else if (m.b_wide && half == BN / 2) {
            pair_load_3d(sb, &m.b[1], 0, row, r0 >> 6, bar);
          } else {
            for (int j = 0; j < nb; ++j) pair_load_2d(sb + j * 8192, &m.b[0], r0 + j * 64, row, bar);
          }
        } else if (A_SIDE) {
          if (MODE == GEMM_FWD) {
            pair_load_3d(sa, &m.a, ks * BK, f, tl.e, bar);
          } else if (m.a_wide) {
            pair_load_4d(sa, &m.a, 0, ks * BK, f >> 6, tl.e, bar);
          } else {
            pair_load_3d(sa, &m.a, f, ks * BK, tl.e, bar);
            pair_load_3d(sa + 8192, &m.a, f + 64, ks * BK, tl.e, bar);
          }
        } else {
          pair_load_2d(sb, &m.b[box], ks * BK, r0, bar);
        }
      }
      __syncwarp();
      next();
      part_first = LONG && part_last;
      if (LONG && part_last && parts > 1) part_end = part_start(nsteps, parts, ++part + 1);
    }
    if constexpr (ADAPTERS<MODE, F32>) {
      if (more && a.late) pdl_wait();  // u is there; returns at once when the launches before are done
      while (known && more && ok) {
        const int col = seg_lo, w16 = (seg_hi - seg_lo) >> 4, whalf = w16 * 8, ad = seg_a;
        const int er0 = tl.row + col + int(rank) * whalf;  // this CTA's half of the segment's rows
        const int ebox = row_box(whalf);
        more = next_seg();
        for (int j0 = 0; j0 < a.rank && slot(); j0 += BK) {
          uint8_t *sa = smem + s * STAGE_BYTES, *sb = sa + A_BYTES;
          const uint32_t bar = full0 + s * 8;
          if (elect_one()) {
            if (A_SIDE) {
              sh.step[s] = Step{(min(BK, a.rank - j0) + 15) >> 4, STEP_EXT | (j0 + BK >= a.rank && !more ? STEP_LAST : 0),
                                w16, col};
              if (rank == 0) mbar_arrive_expect_tx(&sh.full[s], 2 * (A_BYTES + (32 << ebox) * BK * 2));
              if (MODE == GEMM_FWD) {
                pair_load_3d(sa, &m.ea, j0, f, ad, bar);
              } else {
                pair_load_3d(sa, &m.ea, f, j0, ad, bar);
                pair_load_3d(sa + 8192, &m.ea, f + 64, j0, ad, bar);
              }
            } else {
              pair_load_2d(sb, &m.eb[ebox], j0, er0, bar);
            }
          }
          __syncwarp();
          next();
        }
      }
    }
  }
  if (A_SIDE && ok && slot()) {
    if (elect_one()) {
      sh.step[s] = Step{0, STEP_STOP, 0, 0};
      if (rank == 0) mbar_arrive(&sh.full[s]);
    }
    __syncwarp();
  }
  // Every MMA that reads shared memory (in either CTA) is done, so every load
  // has landed, before shared memory is given up: the last use of each slot.
  // (The stop's own slot is not released; slot() saw its use before through.)
  for (int j = 1; j < STAGES; ++j) {
    const int q = (s + j) % STAGES, uses = round + (q < s ? 1 : 0);
    if (uses > 0) wait(sh, &sh.empty[q], (uses - 1) & 1, a.err, true);
  }
  if (!A_SIDE && round > 0) wait(sh, &sh.empty[s], (round - 1) & 1, a.err, true);
  __syncwarp();
}

// LONG: some reduction may be longer than one part (fp32 outputs: always taken to be).
template <int MODE, bool F32, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    gemm_kernel(const TcGemmArgs a, const __grid_constant__ Maps m) {
  extern __shared__ __align__(1024) uint8_t smem[];  // all of the block's shared memory: swizzled tiles first
  Shared &sh = *reinterpret_cast<Shared *>(smem + STAGES * STAGE_BYTES + 4 * OUT_BYTES);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int FT = (a.M + 2 * BMC - 1) / (2 * BMC);
  // ---- prologue: barriers, tensor memory, tile table
  if (tid == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.empty[s], 1);
      mbar_init(&sh.landed[s], 1);
      mbar_init(&sh.fixed[s], 2);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh.tmem_full[b], 1);
      mbar_init(&sh.tmem_empty[b], 2 * EPI_WARPS);
    }
    sh.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem_base)),
                 "r"(512));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  pdl_trigger();
  // With adapters (`late`) only their k-steps and the epilogue need the launches
  // before this one; those wait, before they let this kernel start, for all that
  // it reads until then.
  if (!ADAPTERS<MODE, F32> || !a.late) pdl_wait();
  if (warp == 0) {
    int v[8], local = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      v[i] = 0;
      if (e < a.groups) {
        const bool segs = ADAPTERS<MODE, F32> && a.adapter;
        const int o0 = segs ? 0 : a.offsets[e], o1 = a.offsets[segs ? a.segs : e + 1];
        bad |= o0 < 0 || o1 < o0 || o1 > a.R;
        const int lo = min(max(o0, 0), a.R), hi = min(max(o1, 0), a.R);
        sh.lo[e] = lo;
        if (e == a.groups - 1) sh.lo[e + 1] = hi;
        v[i] = (max(0, hi - lo) + a.bn - 1) / a.bn * FT;
      }
      local += v[i];
    }
    if (bad) flag_error(a.err, MOE_DEVERR_OFFSETS);
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    int run = incl - local;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane * 8 + i;
      if (MODE != GEMM_WGRAD && e < a.groups) sh.tstart[e] = run;
      run += v[i];
    }
    if (lane == 31) {
      if (MODE != GEMM_WGRAD) sh.tstart[a.groups] = incl;
      sh.total = MODE == GEMM_WGRAD ? a.groups * FT * ((a.NC + BN - 1) / BN) : incl;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (MODE == GEMM_WGRAD && tid < a.groups) {
    const int mine = sh.cnt(tid);
    int r = 0;
    for (int e = 0; e < a.groups; ++e) r += sh.cnt(e) > mine || (sh.cnt(e) == mine && e < tid);
    sh.order[r] = int16_t(tid);
  }
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;
  const int total = sh.total;

  if (warp < EPI_WARPS) {
    // ================================================================ epilogue
    const int q = warp & 3, part = warp >> 2;
    const bool issuer = q == 0 && lane == 0;
    const uint32_t out_bufs = smem_u32(smem + STAGES * STAGE_BYTES + part * 2 * OUT_BYTES);
    const uint32_t warp_bufs = smem_u32(smem + STAGES * STAGE_BYTES + warp * 2 * OUT_F32_ROWS * 128);
    uint32_t stores = 0;
    if (ADAPTERS<MODE, F32> && a.late) pdl_wait();
    bool ok = true;
    for (int i = 0, unit = 0; ok; ++i) {  // unit & 1: the accumulator
      const int t = sched_pos(i);
      if (t >= total) break;
      const Tile tl = decode_tile<MODE>(sh, a, t);
      const int parts = LONG ? reduction_parts<F32>(((MODE == GEMM_WGRAD ? sh.cnt(tl.e) : a.KD) + BK - 1) / BK) : 1;
      for (int p = 0; p < parts; ++p, ++unit) {
        const bool add = F32 && (p > 0 || a.accumulate);
        // what this warp has stored of the tile is there before more is added to it
        if (F32 && p > 0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        const int b = unit & 1;
        ok = __all_sync(0xffffffffu, wait(sh, &sh.tmem_full[b], (unit >> 1) & 1, a.err));
        if (!ok) break;
        tc_fence_after();
        const int fw = tl.f0 + int(rank) * BMC + q * 32, f = fw + lane;
        const bool zero = MODE == GEMM_WGRAD && sh.cnt(tl.e) == 0;  // no rows: the gradient is zero, no MMA ran
        const int64_t base = (MODE == GEMM_WGRAD ? int64_t(tl.e) * a.out_gstride : 0) + int64_t(tl.row) * a.ldo + f;
        const uint32_t tb = tmem + (uint32_t(q * 32) << 16) + b * BN;
        // accumulator columns j0 .. j0 + 15, row by row from registers
        auto direct = [&](int j0) {
          uint32_t v[16];
          tmem_ld16(tb + j0, v);
          if (zero) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0;
          }
          if (LONG && !F32 && parts > 1 && add_part(a, p, parts, j0, q * 32 + lane, v)) return;
          const int n = min(16, tl.nvalid - j0);
          if (ADAPTERS<MODE, F32> && a.delta) add_shared_block(a, tl.row + j0, n, f, v);
          store_block<F32>(a, base + int64_t(j0) * a.ldo, n, f, fw + 32 <= a.M, add, v);
        };
        if (zero && add) {
          // nothing to add
        } else if (F32)
          for (int j0 = part * 16; j0 < tl.nvalid; j0 += 32) {
            if (MODE != GEMM_WGRAD && tl.nvalid - j0 < OUT_F32_ROWS) {
              direct(j0);
              continue;
            }
            // 16 rows of the warp's 32 columns, through two buffers of its own (stores
            // straight from the registers, a row of 32 columns each, cost the epilogue
            // 8 cycles apiece and twice that where rows are not multiples of 128
            // bytes: wgrad of 64 experts x 10 rows, N = 3592, K = 968, 262 -> 165 us;
            // dgrad of 64 x 256 rows, K = 2048, N = 1024, 92 -> 76)
            uint32_t v[16];
            tmem_ld16(tb + j0, v);
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            __syncwarp();
            const uint32_t buf = warp_bufs + (stores++ & 1) * (OUT_F32_ROWS * 128);
#pragma unroll
            for (int j = 0; j < OUT_F32_ROWS; ++j)
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(buf + j * 128 + (((lane >> 2) ^ (j & 7)) << 4) + (lane & 3) * 4),
                           "r"(zero ? 0u : v[j])
                           : "memory");
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              if (fw < a.M) {
                if (MODE == GEMM_WGRAD) store_3d<F32>(&m.out, buf, fw, tl.row + j0, tl.e, add);
                else store_2d<F32>(&m.out, buf, fw, tl.row + j0, add);
              }
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
          }
        else for (int j0 = part * OUT_ROWS; j0 < tl.nvalid; j0 += 2 * OUT_ROWS) {
          const int rows = min(OUT_ROWS, tl.nvalid - j0);
          if ((!LONG || parts == 1) && (MODE == GEMM_WGRAD || rows == OUT_ROWS) &&
              !(ADAPTERS<MODE, F32> && a.delta && (shared_block(a, tl.row + j0, 16) || shared_block(a, tl.row + j0 + 16, 16)))) {
            // BF16, 32 rows (wgrad: the map cuts them at the matrix's end): four
            // warps write 128 columns of them to shared memory, one thread sends
            // them off
            uint32_t x[16], y[16];
            tmem_ld_frag(tb + j0, x, y);
            if (zero) {
#pragma unroll
              for (int j = 0; j < 16; ++j) x[j] = y[j] = 0;
            }
            // (the store before the last one has been read)
            if (issuer) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
            const uint32_t out_buf = out_bufs + (stores++ & 1) * OUT_BYTES;
            out_sync(part);
            const int piece = q * 4 + (lane >> 3);  // 8 columns
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + (lane & 7);
              stmatrix_trans(out_buf + (piece >> 3) * (OUT_ROWS * 128) + r * 128 + (((piece & 7) ^ (r & 7)) << 4),
                             pack_acc(x[4 * i], x[4 * i + 1]), pack_acc(x[4 * i + 2], x[4 * i + 3]),
                             pack_acc(y[4 * i], y[4 * i + 1]), pack_acc(y[4 * i + 2], y[4 * i + 3]));
            }
            fence_proxy_async();
            out_sync(part);
            if (issuer) {
              const int fc = tl.f0 + int(rank) * BMC;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (fc + 64 * h >= a.M) break;
                if (MODE == GEMM_WGRAD) store_3d<false>(&m.out, out_buf + h * (OUT_ROWS * 128), fc + 64 * h, tl.row + j0, tl.e);
                else store_2d<false>(&m.out, out_buf + h * (OUT_ROWS * 128), fc + 64 * h, tl.row + j0);
              }
              asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
            continue;
          }
          for (int j1 = j0; j1 < j0 + rows; j1 += 16) direct(j1);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(&sh.tmem_empty[b]);
      }
    }
    if (F32 ? lane == 0 : issuer) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  } else if (warp == A_WARP) {
    produce<MODE, F32, LONG, true>(sh, a, m, smem, rank, total);
  } else if (warp == B_WARP) {
    produce<MODE, F32, LONG, false>(sh, a, m, smem, rank, total);
  } else if (warp == FIX_WARP) {
    // ================================================================ tails
    if (MODE == GEMM_WGRAD) {
      int it = 0;
      uint32_t phase = 0;  // of landed[], one bit per slot
      for (int i = 0;; ++i) {
        const int t = sched_pos(i);
        if (t >= total) break;
        const Tile tl = decode_tile<MODE>(sh, a, t);
        const int red = sh.cnt(tl.e), left = red & 15;
        it += red > 0 ? (red + BK - 1) / BK : 1;
        if (left == 0) continue;
        const int s = (it - 1) % STAGES;
        if (!__all_sync(0xffffffffu, wait(sh, &sh.landed[s], (phase >> s) & 1, a.err))) break;
        phase ^= 1u << s;
        // 64-column blocks of 64 rows x 128 bytes: two of A, up to two of B
        uint8_t *sa = smem + s * STAGE_BYTES;
        const int end = ((red - 1) % BK | 15) + 1;  // the last MMA's last row
        const int nblk = 2 + ((((tl.nvalid + 15) >> 4) * 8 + 63) >> 6);
        for (int blk = 0; blk < nblk; ++blk)
          for (int r = end - 16 + left + (lane >> 3); r < end; r += 4)
            *reinterpret_cast<uint4 *>(sa + blk * 8192 + r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_leader(&sh.fixed[s]);
      }
    }
  } else if (warp == WAIT_WARP && rank == 0) {
    // ================================================================ waiter
    int tl = 0, s = 0;
    uint32_t round = 0, phase = 0;  // phase: of fixed[], one bit per slot
    for (;;) {
      bool ok = wait(sh, &sh.full[s], round, a.err);
      const Step st = sh.step[s];
      if (ok && !(st.flags & STEP_STOP)) {
        if (MODE == GEMM_WGRAD && (st.flags & STEP_FIX_TAIL)) {
          ok = wait(sh, &sh.fixed[s], (phase >> s) & 1, a.err);
          phase ^= 1u << s;
        }
        if (ok && (st.flags & STEP_FIRST)) ok = wait(sh, &sh.tmem_empty[tl & 1], ((tl >> 1) & 1) ^ 1, a.err);
      }
      ok = __all_sync(0xffffffffu, ok);
      const bool stop = !ok || (st.flags & STEP_STOP);
      const bool set = st.flags & (STEP_FIRST | STEP_EXT);
      handoff(lane < (stop ? HAND_STOP : st.kk | (st.flags & STEP_LAST ? HAND_LAST : 0) | (set ? HAND_SET : 0)));
      if (stop) break;
      if (set) {
        handoff(lane < st.n16);
        handoff(lane < (st.flags & STEP_FIRST ? HAND_FIRST : st.col >> 4));
      }
      if (st.flags & STEP_LAST) ++tl;
      if (++s == STAGES) { s = 0; round ^= 1; }
    }
  } else if (warp == MMA_WARP && rank == 0) {
    // ================================================================ MMA issuer
    constexpr bool A_MN = MODE != GEMM_FWD, B_MN = MODE == GEMM_WGRAD;
    constexpr uint32_t KA = A_MN ? 2048 >> 4 : 32 >> 4, KB = B_MN ? 2048 >> 4 : 32 >> 4;  // 16 reduction indices on
    constexpr uint32_t idesc = idesc_bf16(A_MN, B_MN);
    const uint64_t ring = sw128_desc(smem_u32(smem), 8192);  // the start address is the descriptor's low field
    int tl = 0, n16 = 0, s = 0;
    for (;;) {
      const int v = handoff(0);
      if (v >= HAND_STOP) break;
      int col = 0;
      bool first = false;
      if (v & HAND_SET) {
        n16 = handoff(0);
        const int aux = handoff(0);
        first = aux == HAND_FIRST;
        if (!first) col = aux * 16;
      }
      tc_fence_after();
      const uint64_t da = ring + uint64_t(s) * (STAGE_BYTES >> 4), db = da + (A_BYTES >> 4);
      const uint32_t id = idesc | uint32_t(n16 * 2) << 17, d = tmem + (tl & 1) * BN + col;
      if (elect_one()) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < (v & HAND_KK)) mma_pair(d, da + q * KA, db + q * KB, id, !first || q > 0);
        commit_pair(&sh.empty[s]);
        if (v & HAND_LAST) commit_pair(&sh.tmem_full[tl & 1]);
      }
      __syncwarp();
      if (v & HAND_LAST) ++tl;
      if (++s == STAGES) s = 0;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
  }
}

}  // namespace gt

// Every CTA of the grid keeps one tile's sums.
size_t long_sums_bytes(int length) {
  return length > BF16_WHOLE * gt::BK ? size_t(sm_count() & ~1) * gt::BN * gt::BMC * 4 : 0;
}

int check_device(const char *what) {
  int dev = 0, major = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
  if (major != 10) return set_error(MOE_ERR_UNSUPPORTED, "%s: needs sm_100", what);
  if (!tensor_map_encoder()) return set_error(MOE_ERR_UNSUPPORTED, "%s: cuTensorMapEncodeTiled is not available", what);
  return MOE_OK;
}

static bool encode_map(CUtensorMap *m, CUtensorMapDataType type, int size, const void *base, int nd, const int64_t (&dim)[4],
                       const int64_t (&stride)[3], const int (&box)[4]) {
  cuuint64_t d[4], st[3];
  cuuint32_t bx[4], es[4];
  for (int i = 0; i < nd; ++i) {
    d[i] = cuuint64_t(dim[i]);
    bx[i] = cuuint32_t(box[i]);
    es[i] = 1;
    if (i) st[i - 1] = cuuint64_t(stride[i - 1]) * size;
  }
  return tensor_map_encoder()(m, type, cuuint32_t(nd), const_cast<void *>(base), d, st, bx, es,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_bf16(CUtensorMap *m, const void *base, int nd, const int64_t (&dim)[4], const int64_t (&stride)[3],
              const int (&box)[4]) {
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, nd, dim, stride, box);
}

template <int MODE, bool F32>
static int launch_mode(const TcGemmArgs &a, const TcGemmOperands &op, cudaStream_t s, const char *what) {
  gt::Maps m = {};
  bool ok = true;
  const int N = MODE == GEMM_FWD ? a.M : MODE == GEMM_DGRAD ? a.KD : a.NC;
  const int K = MODE == GEMM_FWD ? a.KD : a.M;
  // Columns in whole blocks of 64 can be a dimension of their own, so that one
  // load brings two blocks (the last block of another width would reach into
  // the next row, and behind the last one).
  m.a_wide = MODE != GEMM_FWD && K % 64 == 0;
  m.b_wide = MODE == GEMM_WGRAD && N % 64 == 0;
  if (MODE == GEMM_FWD)
    ok &= map_bf16(&m.a, op.a, 3, {K, N, a.groups, 1}, {K, op.a_gstride, 0}, {64, gt::BMC, 1, 1});
  else if (MODE == GEMM_DGRAD)
    ok &= m.a_wide ? map_bf16(&m.a, op.a, 4, {64, N, K / 64, a.groups}, {K, 64, op.a_gstride}, {64, 64, 2, 1})
                   : map_bf16(&m.a, op.a, 3, {K, N, a.groups, 1}, {K, op.a_gstride, 0}, {64, 64, 1, 1});
  else
    ok &= m.a_wide ? map_bf16(&m.a, op.a, 3, {64, a.R, K / 64, 1}, {op.lda, 64, 0}, {64, 64, 2, 1})
                   : map_bf16(&m.a, op.a, 2, {K, a.R, 1, 1}, {op.lda, 0, 0}, {64, 64, 1, 1});
  const int64_t width = MODE == GEMM_FWD ? K : N;
  if (MODE == GEMM_WGRAD) {
    ok &= map_bf16(&m.b[0], op.b, 2, {N, a.R, 1, 1}, {op.ldb, 0, 0}, {64, 64, 1, 1});
    if (m.b_wide) ok &= map_bf16(&m.b[1], op.b, 3, {64, a.R, N / 64, 1}, {op.ldb, 64, 0}, {64, 64, 2, 1});
  } else {
    for (int i = 0; i < 3; ++i) ok &= map_bf16(&m.b[i], op.b, 2, {width, a.R, 1, 1}, {op.ldb, 0, 0}, {64, 32 << i, 1, 1});
  }
  if (F32)
    ok &= MODE == GEMM_WGRAD ? encode_map(&m.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.out, 3, {K, N, a.groups, 1},
                                          {a.ldo, a.out_gstride, 0}, {32, gt::OUT_F32_ROWS, 1, 1})
                             : encode_map(&m.out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.out, 2, {a.M, a.R, 1, 1},
                                          {a.ldo, 0, 0}, {32, gt::OUT_F32_ROWS, 1, 1});
  else
    ok &= MODE == GEMM_WGRAD
              ? map_bf16(&m.out, a.out, 3, {K, N, a.groups, 1}, {a.ldo, a.out_gstride, 0}, {64, gt::OUT_ROWS, 1, 1})
              : map_bf16(&m.out, a.out, 2, {a.M, a.R, 1, 1}, {a.ldo, 0, 0}, {64, gt::OUT_ROWS, 1, 1});
  if (a.adapter) {
    if (MODE == GEMM_FWD)
      ok &= map_bf16(&m.ea, a.ext_a, 3, {a.rank, N, a.n_adapters, 1}, {a.rank, int64_t(N) * a.rank, 0},
                     {64, gt::BMC, 1, 1});
    else
      ok &= map_bf16(&m.ea, a.ext_a, 3, {K, a.rank, a.n_adapters, 1}, {K, int64_t(K) * a.rank, 0}, {64, 64, 1, 1});
    for (int i = 0; i < 3; ++i)
      ok &= map_bf16(&m.eb[i], a.ext_b, 2, {a.rank, a.R, 1, 1}, {a.rank, 0, 0}, {64, 32 << i, 1, 1});
  }
  if (!ok) return set_error(MOE_ERR_INVALID_ARG, "%s: tensor map encoding failed (pointers or strides)", what);
  // (the parts' code costs calls that need none 1 us: 18 -> 19 us of a projection of 512 rows, K = N = 2048)
  const bool is_long = F32 || (MODE == GEMM_WGRAD ? a.R : a.KD) > BF16_WHOLE * gt::BK;
  auto *kernel = is_long ? gt::gemm_kernel<MODE, F32, true> : gt::gemm_kernel<MODE, F32, F32>;
  int st = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), gt::SMEM, what);
  if (st != MOE_OK) return st;
  const int grid = sm_count() & ~1;
  const cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(gt::THREADS), gt::SMEM, s, a, m);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

int launch_gemm_tc(GemmMode mode, const TcGemmArgs &a, const TcGemmOperands &op, cudaStream_t s, const char *what) {
  const int st = check_device(what);
  if (st != MOE_OK) return st;
  // the tile list is counted in 32 bits
  const int64_t cols = (int64_t(a.M) + 255) / 256;
  const int64_t rows = mode == GEMM_WGRAD ? int64_t(a.groups) * ((int64_t(a.NC) + 255) / 256) : int64_t(a.R) / a.bn + a.groups;
  if (cols * rows > (int64_t(1) << 30))
    return set_error(MOE_ERR_SHAPE, "%s: too many tiles (%lld)", what, (long long)(cols * rows));
  switch (mode) {
    case GEMM_FWD: return a.out_f32 ? launch_mode<GEMM_FWD, true>(a, op, s, what) : launch_mode<GEMM_FWD, false>(a, op, s, what);
    case GEMM_DGRAD: return a.out_f32 ? launch_mode<GEMM_DGRAD, true>(a, op, s, what) : launch_mode<GEMM_DGRAD, false>(a, op, s, what);
    default: return a.out_f32 ? launch_mode<GEMM_WGRAD, true>(a, op, s, what) : launch_mode<GEMM_WGRAD, false>(a, op, s, what);
  }
}

}  // namespace moe
