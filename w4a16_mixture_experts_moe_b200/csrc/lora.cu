// Low-rank adapters of many requests beside a shared BF16 projection:
//   u[t]  = scale_a x[t] A_a^T     y[t]  = x[t] W^T + u[t] B_a^T
//   du[t] = scale_a dy[t] B_a      dx[t] = dy[t] W + du[t] A_a
//   dA_a  = sum_t du[t]^T x[t]     dB_a  = sum_t dy[t]^T u[t]
// for row t of a segment with adapter a. This file holds the entry points and
// the products of small rank (u, du; dA, dB); the projection with the adapters
// folded into its sums is gemm_tc.cu's (batches), proj_kernel's below (decode) or
// gemm_gemv.cu's (a few rows).
//
// u and du are rounded to BF16 once: they are operands of the BF16 matrix
// instructions that follow, and the adapter's part is a small share of y and dx,
// so the rounding (at most 2^-8 relative, independent from value to value) stays
// below their own. dA is made of du alone: it takes du as two BF16 values, the
// rounded one and what the rounding cut off (16 bits of fraction in all), since
// one would cost dA 1.4 times the error of its own rounding. dB takes u as the
// caller kept it.
//
// The small-rank products read each row of x (dy) once and do 2 rank
// operations per value: at rank 64 that is 64 operations a byte, far below the
// tensor cores' balance point, so they are bound by memory: mma.sync from
// shared memory that TMA fills, a ring of stages deep enough to keep the loads
// in flight.
#include <cooperative_groups.h>

#include <type_traits>

#include "gemm.cuh"
#include "ring_flow.h"

namespace cg = cooperative_groups;

namespace moe {
namespace lora {

constexpr int MAX_RANK = 128;
constexpr int MAX_SEGS = 65535;  // a grid dimension of the decode form

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float dot8(const uint4 &a, const uint4 &b, float d) {
  d = fmaf(bf16_lo(a.x), bf16_lo(b.x), d); d = fmaf(bf16_hi(a.x), bf16_hi(b.x), d);
  d = fmaf(bf16_lo(a.y), bf16_lo(b.y), d); d = fmaf(bf16_hi(a.y), bf16_hi(b.y), d);
  d = fmaf(bf16_lo(a.z), bf16_lo(b.z), d); d = fmaf(bf16_hi(a.z), bf16_hi(b.z), d);
  d = fmaf(bf16_lo(a.w), bf16_lo(b.w), d); d = fmaf(bf16_hi(a.w), bf16_hi(b.w), d);
  return d;
}

// 16-byte piece c of row r in a 128-byte-swizzled tile.
__device__ __forceinline__ uint32_t sw128(uint32_t tile, int r, int c) {
  return tile + r * 128 + ((c ^ (r & 7)) << 4);
}

constexpr int CONSUMERS = 256;  // warps 0-7; warp 8 issues the loads
constexpr int RING_MAX = 12;
constexpr int CONSUMER_BAR = 1;
__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync %0, %1;" ::"n"(CONSUMER_BAR), "n"(CONSUMERS) : "memory"); }
// The consumers meet: whether all of them passed true.
__device__ __forceinline__ bool consumer_all(bool ok) {
  uint32_t all;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}\n"
               : "=r"(all)
               : "r"(uint32_t(ok)), "n"(CONSUMER_BAR), "n"(CONSUMERS)
               : "memory");
  return all != 0;
}

struct Ring {
  uint64_t full[RING_MAX], empty[RING_MAX];
  int rows[RING_MAX];  // valid rows of the stage (adapter gradients; 0: no further stage)
  int32_t abort;
};

__device__ __forceinline__ void ring_init(Ring &ring, int stages) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      tma::mbar_init(&ring.full[s], 1);
      tma::mbar_init(&ring.empty[s], CONSUMERS / 32);
    }
    ring.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}
__device__ __forceinline__ bool ring_wait(Ring &ring, uint64_t *bar, uint32_t parity, int32_t *err, bool drain = false) {
  const bool ok = tma::mbar_try(bar, parity) || tma::wait_bounded(&ring.abort, bar, parity, err, drain);
  return __all_sync(0xffffffffu, ok);
}

// The producer's end: its loads have landed. A block whose waits gave up would
// otherwise leave shared memory while copies are still on their way into it.
__device__ __forceinline__ void ring_drain(Ring &ring, int stages, int slot, int round, int32_t *err) {
  last_uses(stages, slot, round, [&](int q, int parity) { ring_wait(ring, &ring.full[q], uint32_t(parity), err, true); });
}

struct ShrinkArgs {
  const int32_t *seg_offsets, *seg_adapter;
  const float *scale;
  int segs, n_adapters, T, C, rank;
  uint16_t *out;      // [T][rank]
  uint16_t *split;    // [T][2 rank]: the same, and what the rounding cut off, rounded (or nullptr)
  int32_t *row_seg;   // [T] the rows' segments, written for the launches behind (or nullptr)
  int32_t *err;
};

// A tile of ROWS rows and BJ ranks; RW x KW = 8 warps: RW of MT 16-row tiles
// each, and KW that split each stage's CC reduction columns. (Two row tiles a
// warp halve the reads of P from shared memory, which bound the wide tile.)
template <int BJ, bool TRANS, int ROWS>
struct ShrinkCfg {
  static constexpr int MT = ROWS == 64 ? 2 : 1, RW = ROWS / 16 / MT, KW = 8 / RW, CC = ROWS == 16 ? 256 : 128;
  static constexpr int Z = ROWS * CC * 2;              // bytes: boxes of 64 columns
  static constexpr int P = TRANS ? CC * 128 : BJ * CC * 2;  // TRANS: CC rows of 64 ranks
  static constexpr int STAGE = Z + P;
  static constexpr int RED = KW * ROWS * (BJ + 1) * 4;
  static constexpr int STAGES = 128 * 1024 / STAGE < RING_MAX ? 128 * 1024 / STAGE : RING_MAX;
  static constexpr int SMEM = 1024 + STAGES * STAGE + RED + int(sizeof(Ring));
  static_assert(KW * 16 <= CC && CC % (KW * 16) == 0 && SMEM <= 227 * 1024, "tile shape");
};

// One stage's products for a warp: acc += z [16 MT rows][CC / KW] P^T. z: boxes of
// ROWS rows x 64 columns; P behind it: boxes of BJ rows (ranks, or columns of W)
// x 64, or CC rows of 64 (TRANS).
template <class Cfg, int BJ, bool TRANS, int ROWS>
__device__ __forceinline__ void stage_mma(float (&acc)[Cfg::MT][BJ / 8][4], uint32_t z, int rw, int kw) {
  const uint32_t p = z + Cfg::Z;
  const int lane = threadIdx.x & 31, lo = lane & 7, m8 = (lane >> 3) & 1, hi = lane >> 4;
#pragma unroll
  for (int i = 0; i < Cfg::CC / (16 * Cfg::KW); ++i) {
    const int kk = kw * (Cfg::CC / (16 * Cfg::KW)) + i;  // 16 columns of the stage
    uint32_t af[Cfg::MT][4];
#pragma unroll
    for (int m = 0; m < Cfg::MT; ++m)
      ldsm4<false>(af[m], sw128(z + (kk >> 2) * ROWS * 128, (rw * Cfg::MT + m) * 16 + lo + m8 * 8, (kk & 3) * 2 + hi));
#pragma unroll
    for (int jp = 0; jp < BJ / 16; ++jp) {
      uint32_t bf[4];
      if (TRANS)
        ldsm4<true>(bf, sw128(p, kk * 16 + lo + m8 * 8, jp * 2 + hi));
      else
        ldsm4<false>(bf, sw128(p + (kk >> 2) * BJ * 128, jp * 16 + lo + hi * 8, (kk & 3) * 2 + m8));
#pragma unroll
      for (int m = 0; m < Cfg::MT; ++m) {
        mma_16816(acc[m][2 * jp], af[m], bf[0], bf[1]);
        mma_16816(acc[m][2 * jp + 1], af[m], bf[2], bf[3]);
      }
    }
  }
}

// The unit-th piece of the rows that tiles of `rows` rows and segments cut out:
// tile and segment starts, merged in order (equal ones: segments first), each
// begin a piece, so there are at most tiles + segs of them and some are empty.
// Returns the segment; the piece is rows [lo, hi) of one tile, whatever the
// offsets hold.
__device__ __forceinline__ int find_piece(const int32_t *off, int segs, int T, int rows, int unit, int &lo, int &hi) {
  const int tiles = (T + rows - 1) / rows;
  int s = max(0, unit - tiles), e = min(unit, segs);  // segment starts among the first `unit`
  while (s < e) {
    const int mid = (s + e) >> 1;
    if (off[mid] <= (unit - 1 - mid) * rows) s = mid + 1; else e = mid;
  }
  int t = unit - s;
  if (s < segs && (t >= tiles || off[s] <= t * rows)) {
    lo = off[s++];
  } else {
    lo = t++ * rows;
  }
  lo = max(lo, (t - 1) * rows);
  hi = min(min(off[s], t * rows), T);  // off[segs]: the end of the last
  if (s < 1 || t < 1 || t > tiles) hi = lo;
  return s - 1;
}

// What a rounding of v to `rounded` cut off (0 behind infinities and NaN).
__device__ __forceinline__ float cut_off(float v, float rounded) { return isfinite(rounded) ? v - rounded : 0.f; }

// out[t][j] = bf16(scale_a sum_c z[t][c] P_a[j][c]), z = x and P = lora_a, or
// z = dy and P_a[j][c] = lora_b[a][c][j] (TRANS). A CTA takes one segment's rows
// of one tile: it runs the whole tile through that segment's adapter (rows are
// independent) and stores the segment's rows. (A CTA per tile that went through
// the tile's segments one by one took 192 us where 200 single rows precede 8000
// of one segment, K = 4096, rank 16; this 32.)
template <int BJ, bool TRANS, int ROWS>
__global__ void __launch_bounds__(CONSUMERS + 32)
    shrink_kernel(const ShrinkArgs a, const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_p) {
  using Cfg = ShrinkCfg<BJ, TRANS, ROWS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *red = reinterpret_cast<float *>(sm + Cfg::STAGES * Cfg::STAGE);
  Ring &ring = *reinterpret_cast<Ring *>(sm + Cfg::STAGES * Cfg::STAGE + Cfg::RED);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring0 = tma::smem_u32(sm);
  ring_init(ring, Cfg::STAGES);
  pdl_wait();     // in this order: the launches behind this one may start before u is there, but
  pdl_trigger();  // not before what this launch itself waits for
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    for (int s = tid; s < a.segs; s += CONSUMERS + 32) {
      const int o0 = a.seg_offsets[s], o1 = a.seg_offsets[s + 1], ad = a.seg_adapter[s];
      if (o0 < 0 || o1 < o0 || o1 > a.T || (s == 0 && o0 != 0)) flag_error(a.err, MOE_DEVERR_OFFSETS);
      if (ad < -1 || ad >= a.n_adapters) flag_error(a.err, MOE_DEVERR_EXPERT_ID);
    }
  }
  const int j0 = blockIdx.y * BJ;
  int lo, hi;
  const int sg = find_piece(a.seg_offsets, a.segs, a.T, ROWS, blockIdx.x, lo, hi);
  if (hi <= lo) return;
  const int row0 = lo / ROWS * ROWS, ad = a.seg_adapter[sg];
  if (a.row_seg && blockIdx.y == 0)
    for (int p = tid; p < hi - lo; p += CONSUMERS + 32) a.row_seg[lo + p] = sg;
  const int nc = (a.C + Cfg::CC - 1) / Cfg::CC;
  int slot = 0, round = 0;
  bool ok = true;
  if (ad < 0 || ad >= a.n_adapters) {  // no adapter: nothing is added to these rows
    if (warp < 8)
      for (int p = tid; p < (hi - lo) * BJ; p += CONSUMERS)
        if (j0 + p % BJ < a.rank) a.out[int64_t(lo + p / BJ) * a.rank + j0 + p % BJ] = 0;
    return;
  }
  if (warp == 8) {
    for (int c = 0; c < nc; ++c) {
      ok = ring_wait(ring, &ring.empty[slot], (round & 1) ^ 1, a.err);
      if (!ok) break;
      if (tma::elect_one()) {
        uint8_t *z = sm + slot * Cfg::STAGE, *p = z + Cfg::Z;
        tma::mbar_arrive_expect_tx(&ring.full[slot], Cfg::STAGE);
#pragma unroll
        for (int b = 0; b < Cfg::CC / 64; ++b)
          tma::tma_load_2d(z + b * ROWS * 128, &tm_z, c * Cfg::CC + b * 64, row0, &ring.full[slot]);
        if (TRANS) {
          tma::tma_load_3d(p, &tm_p, j0, c * Cfg::CC, ad, &ring.full[slot]);
        } else {
#pragma unroll
          for (int b = 0; b < Cfg::CC / 64; ++b)
            tma::tma_load_3d(p + b * BJ * 128, &tm_p, c * Cfg::CC + b * 64, j0, ad, &ring.full[slot]);
        }
      }
      __syncwarp();
      if (++slot == Cfg::STAGES) { slot = 0; ++round; }
    }
    ring_drain(ring, Cfg::STAGES, slot, round, a.err);
    return;
  }
  const int rw = warp % Cfg::RW, kw = warp / Cfg::RW, g = lane >> 2, t4 = lane & 3;
  float acc[Cfg::MT][BJ / 8][4];
#pragma unroll
  for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
    for (int j = 0; j < BJ / 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.f;
  for (int c = 0; c < nc; ++c) {
    ok = ring_wait(ring, &ring.full[slot], round & 1, a.err);
    if (!ok) break;
    stage_mma<Cfg, BJ, TRANS, ROWS>(acc, ring0 + slot * Cfg::STAGE, rw, kw);
    __syncwarp();
    if (lane == 0) tma::mbar_arrive(&ring.empty[slot]);
    if (++slot == Cfg::STAGES) { slot = 0; ++round; }
  }
  // the KW partial sums, added in a fixed order
#pragma unroll
  for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
    for (int j = 0; j < BJ / 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(kw * ROWS + (rw * Cfg::MT + i) * 16 + g + (q >> 1) * 8) * (BJ + 1) + j * 8 + 2 * t4 + (q & 1)] = acc[i][j][q];
  consumer_sync();
  const float sc = a.scale ? a.scale[ad] : 1.f;
  for (int p = tid; p < (hi - lo) * (BJ / 2); p += CONSUMERS) {
    const int r = lo - row0 + p / (BJ / 2), jj = p % (BJ / 2) * 2;
    if (j0 + jj >= a.rank) continue;
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int k = 0; k < Cfg::KW; ++k) {
      v0 += red[(k * ROWS + r) * (BJ + 1) + jj];
      v1 += red[(k * ROWS + r) * (BJ + 1) + jj + 1];
    }
    v0 *= sc;
    v1 *= sc;
    const uint32_t hi = pack_bf16x2(v0, v1);
    *reinterpret_cast<uint32_t *>(a.out + int64_t(row0 + r) * a.rank + j0 + jj) = hi;
    if (a.split) {
      uint16_t *o = a.split + int64_t(row0 + r) * 2 * a.rank + j0 + jj;
      *reinterpret_cast<uint32_t *>(o) = hi;
      *reinterpret_cast<uint32_t *>(o + a.rank) = pack_bf16x2(cut_off(v0, bf16_lo(hi)), cut_off(v1, bf16_hi(hi)));
    }
  }
}

struct DeltaArgs {
  const int32_t *seg_offsets, *seg_adapter, *row_seg;
  const uint16_t *u, *w;  // u / du [T][rank]; lora_b [n][M][rank], or lora_a [n][rank][M] (COLS)
  int segs, n_adapters, T, rank, M, by_seg;
  float *delta;
};

// The adapters' part of the 16-row blocks that several segments share, as fp32
// rows for the projection's epilogue: delta[j][f] = u[row j] . w_a[f], row j's
// own adapter a. A CTA does 128 threads' columns of one block, which it finds by
// the block's owning segment where segments are few, or by its number.
// Latency bounds it, not the bytes: the rows' segments come as a list from the
// launch before (a search in the offsets takes log2(segs) loads, one after the
// other, in every CTA), and a thread has the loads of two or four rows, each another
// request's perhaps, in flight at once; rows of one segment share them. (200
// single rows before 8000 of one segment, rank 64, N = 4096: 27 us, 50 with a
// search and one row's loads at a time; 256 single rows, rank 16: 22 -> 9.)
//
// lora_a's columns f are neighbours in memory: a thread takes two, all ranks.
// lora_b has a column's ranks in a row: G lanes (G 8 >= rank) take 8 each, G
// loads fetch 32 columns a warp, and the lanes' sums are exchanged so that each
// lane ends with one column's.
constexpr int DELTA_COLS = 128;  // columns a CTA, twice as many of lora_a

template <int G>
__device__ __forceinline__ void delta_rows(const DeltaArgs &a, const float (*us)[MAX_RANK], const int *ads, int n, float *out) {
  constexpr int CW = 32 / G, RB = G <= 4 ? 4 : 2;  // columns a load; rows in flight
  const int lane = threadIdx.x & 31, gl = lane % G, c0 = blockIdx.x * DELTA_COLS + (threadIdx.x >> 5) * 32, own = c0 + gl * CW + lane / G;
  const bool in_rank = gl * 8 < a.rank;
  for (int g = 0; g < n; g += RB) {
    uint4 q[RB][G];
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      const int ad = ads[g + j];
      if (ad < 0 || (j > 0 && ad == ads[g + j - 1])) continue;
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const int col = c0 + i * CW + lane / G;
        q[j][i] = in_rank && col < a.M
                      ? *reinterpret_cast<const uint4 *>(a.w + (int64_t(ad) * a.M + col) * a.rank + gl * 8)
                      : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < RB; ++j) {
      if (g + j >= n) break;
      float v[G];
#pragma unroll
      for (int i = 0; i < G; ++i) v[i] = 0.f;
      if (ads[g + j] >= 0) {
        if (j > 0 && ads[g + j] == ads[g + j - 1]) {
#pragma unroll
          for (int i = 0; i < G; ++i) q[j][i] = q[j - 1][i];
        }
        const float4 y0 = *reinterpret_cast<const float4 *>(&us[g + j][gl * 8]);
        const float4 y1 = *reinterpret_cast<const float4 *>(&us[g + j][gl * 8 + 4]);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const uint4 w = q[j][i];
          float d = bf16_lo(w.x) * y0.x;
          d = fmaf(bf16_hi(w.x), y0.y, d); d = fmaf(bf16_lo(w.y), y0.z, d); d = fmaf(bf16_hi(w.y), y0.w, d);
          d = fmaf(bf16_lo(w.z), y1.x, d); d = fmaf(bf16_hi(w.z), y1.y, d);
          d = fmaf(bf16_lo(w.w), y1.z, d); d = fmaf(bf16_hi(w.w), y1.w, d);
          v[i] = d;
        }
#pragma unroll
        for (int h = G / 2; h > 0; h >>= 1)
#pragma unroll
          for (int k = 0; k < h; ++k) {
            const bool up = gl & h;
            const float got = __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + h], h);
            v[k] = (up ? v[k + h] : v[k]) + got;
          }
      }
      if (own < a.M) out[int64_t(g + j) * a.M + own] = v[0];
    }
  }
}

__device__ __forceinline__ void delta_cols(const DeltaArgs &a, const float (*us)[MAX_RANK], const int *ads, int n, float *out) {
  constexpr int CH = 16;  // ranks a pass
  const int f = (blockIdx.x * DELTA_COLS + threadIdx.x) * 2;
  if (f >= a.M) return;
  for (int g = 0; g < n; g += 4) {
    float acc[4][2];
    int ad[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ad[j] = ads[g + j];  // -1 behind the rows
      acc[j][0] = acc[j][1] = 0.f;
    }
    for (int i0 = 0; i0 < a.rank; i0 += CH) {
      uint32_t q[4][CH];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (ad[j] < 0 || (j > 0 && ad[j] == ad[j - 1])) continue;
#pragma unroll
        for (int i = 0; i < CH; i += 8) {
          const bool in = i0 + i < a.rank;
          const uint16_t *c = a.w + (int64_t(ad[j]) * a.rank + i0 + i) * a.M + f;
#pragma unroll
          for (int k = 0; k < 8; ++k) q[j][i + k] = in ? *reinterpret_cast<const uint32_t *>(c + int64_t(k) * a.M) : 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (ad[j] < 0) continue;
        if (j > 0 && ad[j] == ad[j - 1]) {
#pragma unroll
          for (int i = 0; i < CH; ++i) q[j][i] = q[j - 1][i];
        }
#pragma unroll
        for (int i = 0; i < CH; i += 4) {
          const float4 y = *reinterpret_cast<const float4 *>(&us[g + j][i0 + i]);
          const float yv[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc[j][0] = fmaf(bf16_lo(q[j][i + k]), yv[k], acc[j][0]);
            acc[j][1] = fmaf(bf16_hi(q[j][i + k]), yv[k], acc[j][1]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (g + j < n) *reinterpret_cast<float2 *>(out + int64_t(g + j) * a.M + f) = make_float2(acc[j][0], acc[j][1]);
  }
}

// G: see delta_rows; 0: lora_a.
template <int G>
__global__ void __launch_bounds__(128) delta_kernel(const DeltaArgs a) {
  __shared__ __align__(16) float us[16][MAX_RANK];
  __shared__ int ads[16];
  pdl_wait();
  pdl_trigger();  // behind the wait, as in shrink_kernel
  const int end = min(a.seg_offsets[a.segs], a.T), tid = threadIdx.x;
  int row;  // the block's first row
  if (a.by_seg) {
    const int s = blockIdx.y, o = a.seg_offsets[s];
    row = o & ~15;
    if (o <= 0 || o == row || o >= end || (s > 0 && a.seg_offsets[s - 1] > row)) return;
  } else {
    row = blockIdx.y * 16;
    if (row >= end || a.row_seg[row] == a.row_seg[min(row + 15, end - 1)]) return;
  }
  const int per = 16 / gridDim.z, j0 = blockIdx.z * per, n = min(per, end - row - j0);  // this CTA's rows: row + j0 ...
  if (n <= 0) return;
  float *out = a.delta + (a.by_seg ? int64_t(blockIdx.y) * 16 : int64_t(row)) * a.M + int64_t(j0) * a.M;
  row += j0;
  if (tid < 16) {
    const int sg = tid < n ? a.row_seg[row + tid] : -1;
    const int ad = sg >= 0 && sg < a.segs ? a.seg_adapter[sg] : -1;
    ads[tid] = ad < a.n_adapters ? ad : -1;
  }
  const int width = G ? G * 8 : (a.rank + 15) & ~15;  // whole passes, zeros behind the rank
  for (int p = tid; p < n * width; p += 128) {
    const int j = p / width, i = p % width;
    us[j][i] = i < a.rank ? bf16_to_f(a.u[int64_t(row + j) * a.rank + i]) : 0.f;
  }
  __syncthreads();
  if constexpr (G == 0) delta_cols(a, us, ads, n, out);
  else delta_rows<G>(a, us, ads, n, out);
}

struct ProjArgs {
  const int32_t *seg_offsets, *seg_adapter;
  int segs, n_adapters, T, C, M, rank;  // C: reduction, M: output columns
  const uint16_t *u, *ext;              // u / du [T][rank]; lora_b [n][M][rank], or lora_a [n][rank][M] (TRANS)
  uint16_t *out;
  int64_t ldo;
  int32_t *err;
};

template <bool TRANS, int ROWS>
struct ProjCfg {
  static constexpr int BJ = 64, MT = ROWS == 64 ? 2 : 1, RW = ROWS / 16 / MT, KW = 8 / RW, CC = ROWS == 16 ? 256 : 128;
  static constexpr int Z = ROWS * CC * 2, P = BJ * CC * 2;  // bytes; TRANS: CC rows of 64 columns
  static constexpr int STAGE = Z + P, LD = BJ + 1;
  static constexpr int RED = KW * ROWS * LD * 4;
  static constexpr int STAGES = 120 * 1024 / STAGE < RING_MAX ? 120 * 1024 / STAGE : RING_MAX;
  static constexpr int SMEM = 1024 + STAGES * STAGE + RED + int(sizeof(Ring));
  static_assert(SMEM <= 200 * 1024, "shared memory budget");
};

// The projection of a decode-sized batch with its adapters: out = z W^T + u B_a^T
// (z = x), or z W + du A_a (z = dy, TRANS). W is read once per ROWS rows, so W's
// bytes bound it and the SMs have to share them: a cluster of CTAs takes the
// same ROWS x 64 outputs and splits the reduction; the partial sums meet through
// distributed shared memory, each CTA adding and finishing its share of the
// rows in a fixed order. W and the rows stream before u is there (the launch
// before computes it); the epilogue waits for it.
template <bool TRANS, int ROWS>
__global__ void __launch_bounds__(CONSUMERS + 32)
    proj_kernel(const ProjArgs a, const __grid_constant__ CUtensorMap tm_z, const __grid_constant__ CUtensorMap tm_w) {
  using Cfg = ProjCfg<TRANS, ROWS>;
  constexpr int BJ = Cfg::BJ, LD = Cfg::LD;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int ads[ROWS];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *red = reinterpret_cast<float *>(sm + Cfg::STAGES * Cfg::STAGE);
  Ring &ring = *reinterpret_cast<Ring *>(sm + Cfg::STAGES * Cfg::STAGE + Cfg::RED);
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = int(cluster.num_blocks()), part = int(cluster.block_rank());
  const uint32_t ring0 = tma::smem_u32(sm);
  ring_init(ring, Cfg::STAGES);
  pdl_trigger();
  const int row0 = blockIdx.y * ROWS, j0 = int(blockIdx.x) / parts * BJ;
  const int end = min(max(a.seg_offsets[a.segs], 0), a.T);
  const int nc = (a.C + Cfg::CC - 1) / Cfg::CC, c_lo = nc * part / parts, c_hi = nc * (part + 1) / parts;
  int slot = 0, round = 0;
  bool ok = true;
  if (warp == 8) {
    for (int c = c_lo; c < c_hi && ok; ++c) {
      ok = ring_wait(ring, &ring.empty[slot], (round & 1) ^ 1, a.err);
      if (!ok) break;
      if (tma::elect_one()) {
        uint8_t *z = sm + slot * Cfg::STAGE, *p = z + Cfg::Z;
        tma::mbar_arrive_expect_tx(&ring.full[slot], Cfg::STAGE);
        if (TRANS) tma::tma_load_2d(p, &tm_w, j0, c * Cfg::CC, &ring.full[slot]);
#pragma unroll
        for (int b = 0; b < Cfg::CC / 64; ++b) {
          if (!TRANS) tma::tma_load_2d(p + b * BJ * 128, &tm_w, c * Cfg::CC + b * 64, j0, &ring.full[slot]);
          tma::tma_load_2d(z + b * ROWS * 128, &tm_z, c * Cfg::CC + b * 64, row0, &ring.full[slot]);
        }
      }
      __syncwarp();
      if (++slot == Cfg::STAGES) { slot = 0; ++round; }
    }
    ring_drain(ring, Cfg::STAGES, slot, round, a.err);
  } else {
    if (tid < ROWS) {  // the rows' adapters
      const int row = row0 + tid;
      int ad = -1;
      if (row < end) {
        const int sg = first_segment(a.seg_offsets, a.segs, row);
        if (sg < a.segs && a.seg_offsets[sg] <= row) ad = a.seg_adapter[sg];
        if (ad >= a.n_adapters) ad = -1;
      }
      ads[tid] = ad;
    }
    const int rw = warp % Cfg::RW, kw = warp / Cfg::RW, g = lane >> 2, t4 = lane & 3;
    float acc[Cfg::MT][BJ / 8][4];
#pragma unroll
    for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
      for (int j = 0; j < BJ / 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = 0.f;
    for (int c = c_lo; c < c_hi; ++c) {
      ok = ring_wait(ring, &ring.full[slot], round & 1, a.err);
      if (!ok) break;
      stage_mma<Cfg, BJ, TRANS, ROWS>(acc, ring0 + slot * Cfg::STAGE, rw, kw);
      __syncwarp();
      if (lane == 0) tma::mbar_arrive(&ring.empty[slot]);
      if (++slot == Cfg::STAGES) { slot = 0; ++round; }
    }
#pragma unroll
    for (int i = 0; i < Cfg::MT; ++i)
#pragma unroll
      for (int j = 0; j < BJ / 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          red[(kw * ROWS + (rw * Cfg::MT + i) * 16 + g + (q >> 1) * 8) * LD + j * 8 + 2 * t4 + (q & 1)] = acc[i][j][q];
    consumer_sync();
    if (Cfg::KW > 1) {  // this CTA's sums, into the first warp's place
      for (int p = tid; p < ROWS * BJ; p += CONSUMERS) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < Cfg::KW; ++k) v += red[(k * ROWS + p / BJ) * LD + p % BJ];
        red[p / BJ * LD + p % BJ] = v;
      }
    }
  }
  cluster.sync();  // every CTA's sums are in its shared memory
  if (warp < 8) {
    pdl_wait();
    const int r_lo = ROWS * part / parts, r_hi = ROWS * (part + 1) / parts;
    for (int p = tid; p < (r_hi - r_lo) * (BJ / 2); p += CONSUMERS) {
      const int r = r_lo + p / (BJ / 2), j = p % (BJ / 2) * 2, row = row0 + r, n = j0 + j;
      if (row >= end || n >= a.M) continue;
      float v0 = 0.f, v1 = 0.f;
      for (int q = 0; q < parts; ++q) {
        const float *o = cluster.map_shared_rank(red, q) + r * LD + j;
        v0 += o[0];
        v1 += o[1];
      }
      const int ad = ads[r];
      if (ad >= 0) {
        float d0 = 0.f, d1 = 0.f;
        const uint4 *u = reinterpret_cast<const uint4 *>(a.u + int64_t(row) * a.rank);
        if (TRANS) {
          const uint16_t *w = a.ext + int64_t(ad) * a.rank * a.M + n;
#pragma unroll 2
          for (int i = 0; i < a.rank / 8; ++i) {
            const uint4 y = u[i];
            const uint32_t yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t w2 = *reinterpret_cast<const uint32_t *>(w + int64_t(8 * i + k) * a.M);
              const float f = (k & 1) ? bf16_hi(yw[k >> 1]) : bf16_lo(yw[k >> 1]);
              d0 = fmaf(bf16_lo(w2), f, d0);
              d1 = fmaf(bf16_hi(w2), f, d1);
            }
          }
        } else {
          const uint4 *w0 = reinterpret_cast<const uint4 *>(a.ext + (int64_t(ad) * a.M + n) * a.rank);
          const uint4 *w1 = w0 + a.rank / 8;
#pragma unroll 2
          for (int i = 0; i < a.rank / 8; ++i) {
            const uint4 y = u[i], x0 = w0[i], x1 = w1[i];
            d0 = dot8(x0, y, d0);
            d1 = dot8(x1, y, d1);
          }
        }
        v0 += d0;
        v1 += d1;
      }
      *reinterpret_cast<uint32_t *>(a.out + int64_t(row) * a.ldo + n) = pack_bf16x2(v0, v1);
    }
  }
  cluster.sync();  // no CTA leaves while its sums are read
}

__device__ __forceinline__ void add_shared(float *p, float v) {
  asm volatile("{\n .reg .f32 s;\n ld.shared.f32 s, [%0];\n add.rn.f32 s, s, %1;\n st.shared.f32 [%0], s;\n}\n" ::"r"(tma::smem_u32(p)),
               "f"(v)
               : "memory");
}

struct AdapterGradArgs {
  const int32_t *seg_offsets, *seg_adapter;
  int segs, n_adapters, T, N, K, rank;
  int slabs_a;        // 64-column slabs of x; the others are dy's
  int stages;
  int batch;          // adapters of a CTA whose segments are looked up together; 0: each by itself
  uint16_t *da, *db;  // [n][rank][K], [n][N][rank]
  int32_t *err;
};

constexpr int AG_COLS = 64;
// The matrix unit adds with truncation: its sums pass on to fp32 sums in shared
// memory, rounded to nearest, behind this many additions of 16 rows' products
// (gradients of one adapter with a million rows, all products of one sign: off by
// up to 3.3e-3 of the value beyond the BF16 rounding without, 4e-6 with it).
constexpr int AG_ADDITIONS = 256;

template <int RJ, int AG_ROWS>
struct AdapterGradCfg {
  static constexpr int BOX = AG_ROWS * 128;              // bytes of 64 columns
  // boxes of u, and of du beside what its rounding cut off (twice the columns)
  static constexpr int U_BOXES = RJ == 128 ? 2 : 1, DU_BOXES = RJ <= 32 ? 1 : RJ / 32;
  static constexpr int Z = BOX, P = DU_BOXES * BOX;
  static constexpr int STAGE = Z + P;
  static constexpr int LD = AG_COLS + 2;                 // fp32 partial sums [RJ][LD]
  static constexpr int RED = RJ * LD * 4;
  static constexpr int DEEP = 160 * 1024 / STAGE < RING_MAX ? 160 * 1024 / STAGE : RING_MAX;
  static constexpr int SHALLOW = DEEP / 2 < 2 ? 2 : DEEP / 2;
  static constexpr int smem(int stages) { return 1024 + stages * STAGE + RED + int(sizeof(Ring)); }
};

// The operands' maps: boxes of AG_ROWS rows, and of AG_SHORT for a chunk that
// holds no more (what the stage holds behind them is cleared in the fragments as
// well): the time of a box goes by its rows (dA and dB of 9 adapters, rank 8, 68
// single rows, K = 1832, N = 280: 23 -> 11 us).
constexpr int AG_SHORT = 8;
struct AdapterGradMaps {
  CUtensorMap x[2], dy[2], u[2], du[2];
};

// Which groups of 32 segments hold one of the next a.batch adapters ad, ad + step,
// ...: bit g of an adapter's words. A warp marks them with eight segments a lane
// in flight. Where a CTA would look at more than AG_LOOKS groups for its adapters
// one by one, each a load's latency, this is faster (backward, K = N = 2048, rank
// 16: 4096 segments of one row, 1024 adapters 5.3 -> 1.0 ms, 256 and 64 74 -> 67
// us), with fewer slower (58 and 48: 43 us, 44 with the marks).
constexpr int AG_LOOKS = 48, AG_WORDS = 1024;
__device__ __forceinline__ void mark_segments(const AdapterGradArgs &a, int ad, int step, int words, uint32_t *bits) {
  const int lane = threadIdx.x & 31;
  for (int p = lane; p < a.batch * words; p += 32) bits[p] = 0;
  __syncwarp();
  for (int s0 = 0; s0 < a.segs; s0 += 8 * 32) {
    uint32_t q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      q[k] = s0 + 32 * k + lane < a.segs ? uint32_t(a.seg_adapter[s0 + 32 * k + lane]) - uint32_t(ad) : 0xffffffffu;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = int(min(q[k], 0x7fffffffu)) / step, g = (s0 >> 5) + k;
      if (i < a.batch && i * step == int(q[k])) atomicOr(&bits[i * words + (g >> 5)], 1u << (g & 31));
    }
  }
  __syncwarp();
}

// The gradients of one adapter for a slab of 64 columns c of x (dA) or dy (dB):
// G[j][c] = sum over the rows t of the adapter's segments of p[t][j] z[t][c],
// with p = du (both of its values), z = x or p = u, z = dy. Rows pass AG_ROWS at a
// time through shared memory, read transposed (ldmatrix.trans): M = columns (16
// per warp), N = ranks, K = rows (two warps share a chunk's). The rows behind a
// segment's end are cleared in the fragments. The segments are taken in order by
// one CTA, so the sum's order is fixed. An adapter without rows gets zeros.
// LONG: some adapter may need more additions than AG_ADDITIONS. MARK: see
// mark_segments. (The least CTAs an SM are what its shared memory holds, set where
// the compiler by itself spills or takes registers for fewer: backward at T =
// 4096, K = N = 2048, 256 segments, rank 16, 100 -> 88 us.)
template <int RJ, int AG_ROWS, bool LONG, bool MARK>
__global__ void __launch_bounds__(CONSUMERS + 32, RJ == 64 ? 2 : RJ == 32 ? 3 : RJ == 16 && LONG ? (AG_ROWS == 32 ? 4 : 3) : 0)
    adapter_grad_kernel(const AdapterGradArgs a, const __grid_constant__ AdapterGradMaps maps) {
  using Cfg = AdapterGradCfg<RJ, AG_ROWS>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float *red = reinterpret_cast<float *>(sm + a.stages * Cfg::STAGE);
  Ring &ring = *reinterpret_cast<Ring *>(sm + a.stages * Cfg::STAGE + Cfg::RED);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring0 = tma::smem_u32(sm);
  ring_init(ring, a.stages);
  pdl_wait();
  pdl_trigger();  // behind the wait, as in shrink_kernel
  const bool is_a = int(blockIdx.x) < a.slabs_a;
  const int c0 = (is_a ? blockIdx.x : blockIdx.x - a.slabs_a) * AG_COLS, C = is_a ? a.K : a.N;
  int slot = 0, round = 0;
  bool ok = true;
  if (warp == 8) {
    const CUtensorMap *tz = is_a ? maps.x : maps.dy, *tp = is_a ? maps.du : maps.u;
    uint32_t *bits = reinterpret_cast<uint32_t *>(&ring + 1);  // [batch][words]
    const int words = (a.segs + 1023) >> 10;
    int in_batch = 0;
    for (int ad = blockIdx.y; ad < a.n_adapters && ok; ad += gridDim.y) {
      if (MARK && in_batch == 0) mark_segments(a, ad, gridDim.y, words, bits);
      auto look = [&](int s) {  // at 32 segments, one a lane
        int lo = 0, hi = 0;
        if (s < a.segs && a.seg_adapter[s] == ad) {
          lo = max(a.seg_offsets[s], 0);
          hi = min(a.seg_offsets[s + 1], a.T);
        }
        for (uint32_t m = __ballot_sync(0xffffffffu, hi > lo); m && ok; m &= m - 1) {
          const int l = __ffs(m) - 1, e = __shfl_sync(0xffffffffu, hi, l);
          for (int r = __shfl_sync(0xffffffffu, lo, l); r < e && ok; r += AG_ROWS) {
            ok = ring_wait(ring, &ring.empty[slot], (round & 1) ^ 1, a.err);
            if (ok && tma::elect_one()) {
              uint8_t *z = sm + slot * Cfg::STAGE, *p = z + Cfg::Z;
              const int few = e - r <= AG_SHORT;
              ring.rows[slot] = min(AG_ROWS, e - r);
              const int boxes = is_a ? Cfg::DU_BOXES : Cfg::U_BOXES, bytes = Cfg::BOX * (1 + boxes);
              tma::mbar_arrive_expect_tx(&ring.full[slot], few ? bytes / AG_ROWS * AG_SHORT : bytes);
              tma::tma_load_2d(z, tz + few, c0, r, &ring.full[slot]);
              for (int q = 0; q < boxes; ++q) tma::tma_load_2d(p + q * Cfg::BOX, tp + few, 64 * q, r, &ring.full[slot]);
            }
            __syncwarp();
            if (++slot == a.stages) { slot = 0; ++round; }
          }
        }
      };
      if constexpr (!MARK) {
        for (int s0 = 0; s0 < a.segs && ok; s0 += 32) look(s0 + lane);
      } else {
        for (int h = 0; h < words && ok; h += 32) {  // the lanes' words: 32 times 32 such groups
          const uint32_t word = h + lane < words ? bits[in_batch * words + h + lane] : 0u;
          for (uint32_t nz = __ballot_sync(0xffffffffu, word != 0); nz && ok; nz &= nz - 1) {
            const int l = __ffs(nz) - 1;
            for (uint32_t m = __shfl_sync(0xffffffffu, word, l); m && ok; m &= m - 1)
              look((32 * (h + l) + __ffs(m) - 1) * 32 + lane);
          }
        }
        if (++in_batch == a.batch) in_batch = 0;
      }
      if (!ok) break;
      ok = ring_wait(ring, &ring.empty[slot], (round & 1) ^ 1, a.err);  // the adapter's end: a stage without rows
      if (ok && tma::elect_one()) {
        ring.rows[slot] = 0;
        tma::mbar_arrive(&ring.full[slot]);
      }
      __syncwarp();
      if (++slot == a.stages) { slot = 0; ++round; }
    }
    ring_drain(ring, a.stages, slot, round, a.err);
    return;
  }
  const int cg = warp & 3, kg = warp >> 2, g = lane >> 2, t4 = lane & 3;
  const int lo = lane & 7, m8 = (lane >> 3) & 1, hi = lane >> 4;
  for (int ad = blockIdx.y; ad < a.n_adapters; ad += gridDim.y) {
    float acc[RJ / 8][4];
    auto release = [&]() {
      __syncwarp();
      if (lane == 0) tma::mbar_arrive(&ring.empty[slot]);
      if (++slot == a.stages) { slot = 0; ++round; }
    };
    auto next = [&]() {
      if (!ring_wait(ring, &ring.full[slot], round & 1, a.err)) return -1;
      const int rows = ring.rows[slot];
      if (rows == 0) release();
      return rows;
    };
    auto stage = [&](int rows) {
      const uint32_t z = ring0 + slot * Cfg::STAGE, p = z + Cfg::Z;
      auto products = [&](auto cut) {  // cut: the stage ends inside this warp's rows
#pragma unroll
        for (int i = 0; i < AG_ROWS / 32; ++i) {
          const int kk = kg * (AG_ROWS / 32) + i;
          uint32_t m0 = 0xffffffffu, m1 = 0xffffffffu;  // this lane's reduction rows 2t, 2t+1 and 2t+8, 2t+9
          if (cut) {
            const int left = rows - kk * 16 - 2 * t4;
            if (left + 2 * t4 <= 0) break;
            m0 = left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
            m1 = left >= 10 ? 0xffffffffu : left == 9 ? 0xffffu : 0u;
          }
          uint32_t af[4];
          ldsm4<true>(af, sw128(z, kk * 16 + lo + hi * 8, cg * 2 + m8));
          if (cut) { af[0] &= m0; af[1] &= m0; af[2] &= m1; af[3] &= m1; }
#pragma unroll
          for (int jp = 0; jp < RJ / 16; ++jp) {
            auto ranks = [&](int piece) {  // 16 ranks from the piece-th 8 columns of P on
              uint32_t bf[4];
              ldsm4<true>(bf, sw128(p + (piece >> 3) * Cfg::BOX, kk * 16 + lo + m8 * 8, piece & 7));
              if (cut) { bf[0] &= m0; bf[1] &= m1; bf[2] &= m0; bf[3] &= m1; }
              mma_16816(acc[2 * jp], af, bf[0], bf[1]);
              mma_16816(acc[2 * jp + 1], af, bf[2], bf[3]);
            };
            ranks(2 * jp + hi);
            if (is_a) ranks((a.rank >> 3) + 2 * jp + hi);  // (behind a rank that fills no 16, into sums that nobody stores)
          }
        }
      };
      if (rows >= (kg + 1) * (AG_ROWS / 2)) products(std::false_type{});
      else if (rows > kg * (AG_ROWS / 2)) products(std::true_type{});
      release();
    };
    // accumulator (c0, c1) = column g, ranks 2t, 2t+1; (c2, c3) = column g + 8
    auto at = [&](int j, int q) -> float & {
      return red[(j * 8 + 2 * t4 + (q & 1)) * Cfg::LD + cg * 16 + g + (q >> 1) * 8];
    };
    auto clear = [&]() {
#pragma unroll
      for (int j = 0; j < RJ / 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;
    };
    auto put = [&](bool first) {
      if (kg != 1) return;
      if (!LONG || first) {
#pragma unroll
        for (int j = 0; j < RJ / 8; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) at(j, q) = acc[j][q];
      } else {  // (one after the other: this path is rare, and must not cost the others registers)
#pragma unroll
        for (int j = 0; j < RJ / 8; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) add_shared(&at(j, q), acc[j][q]);
      }
    };
    auto add = [&]() {
      if (kg != 0) return;
#pragma unroll
      for (int j = 0; j < RJ / 8; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) at(j, q) += acc[j][q];
    };
    const int got = sum_group<LONG>(is_a ? AG_ADDITIONS / 2 : AG_ADDITIONS, next, clear, stage, put, consumer_all, add, consumer_sync);
    if (got < 0) return;
    if (got == 0) {  // no rows: zeros
      const uint4 zero = make_uint4(0, 0, 0, 0);
      for (int p = tid; p < AG_COLS * a.rank / 8; p += CONSUMERS) {
        if (is_a) {
          const int j = p / (AG_COLS / 8), c = c0 + p % (AG_COLS / 8) * 8;
          if (c < C) *reinterpret_cast<uint4 *>(a.da + (int64_t(ad) * a.rank + j) * a.K + c) = zero;
        } else if (c0 + p / (a.rank / 8) < C) {
          *reinterpret_cast<uint4 *>(a.db + (int64_t(ad) * a.N + c0) * a.rank + p * 8) = zero;
        }
      }
      continue;
    }
    if (is_a) {  // [rank][K]: 64 columns of each row
      for (int p = tid; p < a.rank * (AG_COLS / 2); p += CONSUMERS) {
        const int j = p / (AG_COLS / 2), c = p % (AG_COLS / 2) * 2;
        if (c0 + c < C)
          *reinterpret_cast<uint32_t *>(a.da + (int64_t(ad) * a.rank + j) * a.K + c0 + c) =
              pack_bf16x2(red[j * Cfg::LD + c], red[j * Cfg::LD + c + 1]);
      }
    } else {     // [N][rank]: 64 whole rows
      for (int p = tid; p < AG_COLS * (a.rank / 2); p += CONSUMERS) {
        const int c = p / (a.rank / 2), j = p % (a.rank / 2) * 2;
        if (c0 + c < C)
          *reinterpret_cast<uint32_t *>(a.db + (int64_t(ad) * a.N + c0 + c) * a.rank + j) =
              pack_bf16x2(red[j * Cfg::LD + c], red[(j + 1) * Cfg::LD + c]);
      }
    }
    consumer_sync();  // the sums are read
  }
  consumer_all(true);
}

// Small-rank operands of one call, for the tensor maps.
struct Rows {
  const uint16_t *p;
  int64_t ld;
  int width;
};

template <int BJ, bool TRANS, int ROWS>
static int launch_shrink_as(const ShrinkArgs &a, const Rows &z, const uint16_t *p, cudaStream_t s, const char *what) {
  using Cfg = ShrinkCfg<BJ, TRANS, ROWS>;
  int st = check_device(what);
  if (st != MOE_OK) return st;
  CUtensorMap tz, tp;
  bool ok = map_bf16(&tz, z.p, 2, {z.width, a.T, 1, 1}, {z.ld, 0, 0}, {64, ROWS, 1, 1});
  if (TRANS)
    ok &= map_bf16(&tp, p, 3, {a.rank, a.C, a.n_adapters, 1}, {a.rank, int64_t(a.C) * a.rank, 0}, {64, Cfg::CC, 1, 1});
  else
    ok &= map_bf16(&tp, p, 3, {a.C, a.rank, a.n_adapters, 1}, {a.C, int64_t(a.C) * a.rank, 0}, {64, BJ, 1, 1});
  if (!ok) return set_error(MOE_ERR_INVALID_ARG, "%s: tensor map encoding failed (pointers or strides)", what);
  st = allow_dynamic_smem(reinterpret_cast<const void *>(shrink_kernel<BJ, TRANS, ROWS>), Cfg::SMEM, what);
  if (st != MOE_OK) return st;
  const dim3 grid(unsigned((a.T + ROWS - 1) / ROWS) + unsigned(a.segs), unsigned((a.rank + BJ - 1) / BJ));
  const cudaError_t e = launch_pdl(shrink_kernel<BJ, TRANS, ROWS>, grid, dim3(CONSUMERS + 32), Cfg::SMEM, s, a, tz, tp);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

// 16-row tiles until they fill the SMs about twice over; then 64-row tiles,
// which read each adapter a quarter as often (whole forward, K = N = 2048, rank 16,
// 4 segments: T = 2048 26.8 us against 28.5 with the high tiles, 4096 40.7 and
// 41.3; K = N = 4096, rank 64, 13 segments: 4096 126.9 and 124.6, 8192 251 and 228).
constexpr int SHRINK_WIDE_T = 4096;

template <bool TRANS>
static int launch_shrink(const ShrinkArgs &a, const Rows &z, const uint16_t *p, cudaStream_t s, const char *what) {
  if (a.T < SHRINK_WIDE_T)
    return a.rank <= 16   ? launch_shrink_as<16, TRANS, 16>(a, z, p, s, what)
           : a.rank <= 32 ? launch_shrink_as<32, TRANS, 16>(a, z, p, s, what)
                          : launch_shrink_as<64, TRANS, 16>(a, z, p, s, what);
  return a.rank <= 16   ? launch_shrink_as<16, TRANS, 64>(a, z, p, s, what)
         : a.rank <= 32 ? launch_shrink_as<32, TRANS, 64>(a, z, p, s, what)
                        : launch_shrink_as<64, TRANS, 64>(a, z, p, s, what);
}

static int proj_parts(int tiles, int nc);

template <bool TRANS, int ROWS>
static int launch_proj_as(const ProjArgs &a, const Rows &z, const uint16_t *w, cudaStream_t s, const char *what) {
  using Cfg = ProjCfg<TRANS, ROWS>;
  int st = check_device(what);
  if (st != MOE_OK) return st;
  CUtensorMap tz, tw;
  bool ok = map_bf16(&tz, z.p, 2, {z.width, a.T, 1, 1}, {z.ld, 0, 0}, {64, ROWS, 1, 1});
  if (TRANS)
    ok &= map_bf16(&tw, w, 2, {a.M, a.C, 1, 1}, {a.M, 0, 0}, {64, Cfg::CC, 1, 1});
  else
    ok &= map_bf16(&tw, w, 2, {a.C, a.M, 1, 1}, {a.C, 0, 0}, {64, Cfg::BJ, 1, 1});
  if (!ok) return set_error(MOE_ERR_INVALID_ARG, "%s: tensor map encoding failed (pointers or strides)", what);
  auto *kernel = proj_kernel<TRANS, ROWS>;
  st = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), Cfg::SMEM, what);
  if (st != MOE_OK) return st;
  const int tiles = (a.M + Cfg::BJ - 1) / Cfg::BJ, row_tiles = (a.T + ROWS - 1) / ROWS;
  const int parts = proj_parts(tiles * row_tiles, (a.C + Cfg::CC - 1) / Cfg::CC);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles * parts), unsigned(row_tiles));
  cfg.blockDim = dim3(CONSUMERS + 32);
  cfg.dynamicSmemBytes = Cfg::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(parts);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, tz, tw);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

template <bool TRANS>
static int launch_proj(const ProjArgs &a, const Rows &z, const uint16_t *w, cudaStream_t s, const char *what) {
  return a.T <= 16   ? launch_proj_as<TRANS, 16>(a, z, w, s, what)
         : a.T <= 32 ? launch_proj_as<TRANS, 32>(a, z, w, s, what)
                     : launch_proj_as<TRANS, 64>(a, z, w, s, what);
}

template <int G>
static int launch_delta_as(const DeltaArgs &a, cudaStream_t s, const char *what) {
  constexpr int cols = G ? DELTA_COLS : 2 * DELTA_COLS;
  // Four CTAs a block, unless lora_b's blocks alone are eight rounds of the SMs,
  // most of them owned by no segment (forward, rank 16, N = 4096, T = 8000: 400
  // segments 278 us with four, 248 with one; rank 128, 16 segments 223 and 230).
  const unsigned x = unsigned((a.M + cols - 1) / cols), y = unsigned(a.by_seg ? a.segs : (a.T + 15) / 16);
  const dim3 grid(x, y, a.by_seg && G && int64_t(x) * y > 8 * sm_count() ? 1u : 4u);
  const cudaError_t e = launch_pdl(delta_kernel<G>, grid, dim3(128), 0, s, a);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

template <bool COLS>
static int launch_delta(const DeltaArgs &a, cudaStream_t s, const char *what) {
  return COLS            ? launch_delta_as<0>(a, s, what)
         : a.rank <= 8   ? launch_delta_as<1>(a, s, what)
         : a.rank <= 16  ? launch_delta_as<2>(a, s, what)
         : a.rank <= 32  ? launch_delta_as<4>(a, s, what)
         : a.rank <= 64  ? launch_delta_as<8>(a, s, what)
                         : launch_delta_as<16>(a, s, what);
}

template <int RJ, int AG_ROWS>
static int launch_adapter_grad_as(AdapterGradArgs a, const Rows &x, const Rows &dy, const Rows &u,
                                  const Rows &du, cudaStream_t s, const char *what) {
  using Cfg = AdapterGradCfg<RJ, AG_ROWS>;
  int st = check_device(what);
  if (st != MOE_OK) return st;
  AdapterGradMaps maps;
  bool ok = true;
  const Rows *r[4] = {&x, &dy, &u, &du};
  CUtensorMap *m[4] = {maps.x, maps.dy, maps.u, maps.du};
  for (int i = 0; i < 8; ++i)
    ok &= map_bf16(m[i >> 1] + (i & 1), r[i >> 1]->p, 2, {r[i >> 1]->width, a.T, 1, 1}, {r[i >> 1]->ld, 0, 0},
                   {64, i & 1 ? AG_SHORT : AG_ROWS, 1, 1});
  if (!ok) return set_error(MOE_ERR_INVALID_ARG, "%s: tensor map encoding failed (pointers or strides)", what);
  // Up to four CTAs per SM, each going through every grid.y-th adapter: an
  // adapter's end (sums joined and stored) hides behind the other CTAs. A grid
  // of less than one CTA per SM gets deep rings instead.
  const int slabs = a.slabs_a + (a.N + AG_COLS - 1) / AG_COLS;
  int ny = (4 * sm_count() + slabs - 1) / slabs;
  ny = ny > a.n_adapters ? a.n_adapters : ny;
  a.stages = slabs * ny <= sm_count() ? Cfg::DEEP : Cfg::SHALLOW;
  const int per = (a.n_adapters + ny - 1) / ny, words = (a.segs + 1023) / 1024;  // adapters a CTA; words an adapter
  a.batch = int64_t(per) * ((a.segs + 31) / 32) <= AG_LOOKS ? 0 : per < AG_WORDS / words ? per : AG_WORDS / words;
  const size_t smem = Cfg::smem(a.stages) + size_t(a.batch) * words * 4;
  const dim3 grid{unsigned(slabs), unsigned(ny)};
  // additions of the longest adapter: 16 rows each, and one more for each chunk; dA's twice
  const bool far = int64_t(a.T) / 16 + a.T / AG_ROWS + a.segs > AG_ADDITIONS / 2;
  auto *kernel = a.batch ? adapter_grad_kernel<RJ, AG_ROWS, true, true>
                 : far   ? adapter_grad_kernel<RJ, AG_ROWS, true, false>
                         : adapter_grad_kernel<RJ, AG_ROWS, false, false>;
  st = allow_dynamic_smem(reinterpret_cast<const void *>(kernel), Cfg::smem(Cfg::DEEP) + AG_WORDS * 4, what);
  if (st != MOE_OK) return st;
  const cudaError_t e = launch_pdl(kernel, grid, dim3(CONSUMERS + 32), smem, s, a, maps);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

// WIDE: long loads, 128 rows or, at ranks whose stages would leave no room for a
// second one, 64.
template <bool WIDE>
static int launch_adapter_grad(const AdapterGradArgs &a, const Rows &x, const Rows &dy, const Rows &u,
                               const Rows &du, cudaStream_t s, const char *what) {
  constexpr int ROWS = WIDE ? 128 : 32, HIGH = WIDE ? 64 : 32;
  return a.rank <= 16   ? launch_adapter_grad_as<16, ROWS>(a, x, dy, u, du, s, what)
         : a.rank <= 32 ? launch_adapter_grad_as<32, ROWS>(a, x, dy, u, du, s, what)
         : a.rank <= 64 ? launch_adapter_grad_as<64, HIGH>(a, x, dy, u, du, s, what)
                        : launch_adapter_grad_as<128, HIGH>(a, x, dy, u, du, s, what);
}

// Rows of the fp32 sums for shared 16-row blocks: 16 per segment, or one per
// row if that is less.
static size_t delta_rows(int T, int S) {
  if (T < 1 || S < 2) return 0;
  const size_t by_seg = size_t(S) * 16, by_row = (size_t(T) + 15) / 16 * 16;
  return by_seg < by_row ? by_seg : by_row;
}

// du beside what its rounding cut off, [T][2 rank]. A megabyte at least, so that
// calls of a few rows ask for one size.
static size_t split_bytes(int T, int rank) {
  const size_t need = T < 1 ? 0 : (size_t(T) * rank * 4 + 255) / 256 * 256;
  return need < (size_t(1) << 20) ? size_t(1) << 20 : need;
}

// The workspace: the error word, what long reductions of the engine add up in,
// the shared blocks' sums, the rows' segments, and the split du, which only calls
// that ask for the adapters' gradients need.
struct Workspace {
  char *sums;
  float *delta;
  int32_t *row_seg;
  uint16_t *split;
  size_t plain, whole;  // bytes without and with the split du
};
static Workspace workspace(int T, int S, int rank, int N, int K, void *ws) {
  const int most = N > K ? N : K;
  const size_t delta = WS_HEADER + long_sums_bytes(most), seg = delta + delta_rows(T, S) * size_t(most) * 4;
  const size_t plain = seg + (T < 1 || S < 2 ? 0 : size_t(T) * 4), split = (plain + 15) / 16 * 16;
  char *p = static_cast<char *>(ws);
  return {p + WS_HEADER, reinterpret_cast<float *>(p + delta), reinterpret_cast<int32_t *>(p + seg),
          reinterpret_cast<uint16_t *>(p + split), plain, split + split_bytes(T, rank)};
}

// The arguments both entry points share; `grads`: the adapters' gradients are asked for.
static int check_common(const char *who, const void *w, const void *seg_offsets, const void *seg_adapter,
                        const void *lora_a, const void *lora_b, int T, int S, int n_adapters, int rank, int N, int K,
                        bool grads, const void *ws, size_t ws_bytes) {
  if (T < 0 || T > (1 << 30) || S < 0 || S > MAX_SEGS || n_adapters < 1 || n_adapters > MAX_SEGS)
    return set_error(MOE_ERR_SHAPE, "%s: T=%d S=%d n_adapters=%d (need 0<=T<=2^30, 0<=S<=65535, 1<=n_adapters<=65535)",
                     who, T, S, n_adapters);
  if (rank < 8 || rank > MAX_RANK || rank % 8)
    return set_error(MOE_ERR_SHAPE, "%s: rank=%d must be a multiple of 8 from 8 to 128", who, rank);
  if (N < 8 || K < 8 || N % 8 || K % 8 || N > MAX_COLS || K > MAX_COLS)
    return set_error(MOE_ERR_SHAPE, "%s: N=%d K=%d must be multiples of 8 from 8 to 2^30", who, N, K);
  if (!ws || !w || !lora_a || !lora_b || !seg_offsets || (S > 0 && !seg_adapter))
    return set_error(MOE_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned(ws, 256) || !aligned(w, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16))
    return set_error(MOE_ERR_INVALID_ARG, "%s: ws needs 256-byte, w, lora_a and lora_b 16-byte alignment", who);
  const Workspace space = workspace(T, S, rank, N, K, nullptr);
  const size_t need = grads ? space.whole : space.plain;
  if (ws_bytes < need) return set_error(MOE_ERR_INVALID_ARG, "%s: workspace %zu B < %zu B", who, ws_bytes, need);
  return MOE_OK;
}

static int check_rows(const char *who, const char *name, const void *p, int64_t ld, int width) {
  if (!p || !aligned(p, 16) || ld < width || ld % 8)
    return set_error(MOE_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned, its row stride (%lld) a multiple of 8 and at least %d",
                     who, name, (long long)ld, width);
  return MOE_OK;
}

// The forward pass of the fewest rows runs in gemm_gemv.cu.
constexpr int GEMV_MAX_T = 8;

// CTAs of proj_kernel that split one tile's reduction (a cluster): doubled until
// the CTAs cover the SMs, each with two stages of work at least.
static int proj_parts(int tiles, int nc) {
  int parts = 1;
  while (parts < 8 && tiles * parts * 2 <= sm_count() && nc >= parts * 4) parts *= 2;
  return parts;
}

// Whether M columns of T rows, reduced over C, run as a weight stream
// (proj_kernel) rather than on the tensor-core engine. Its 64 x 64 tiles have to
// fit the SMs at once (K = N = 1024, four requests of rank 16: T = 512 14 us
// against the engine's 15, T = 768, two rounds, 25 against 16) and a CTA's share
// of the reduction has to be short: 128 columns cost it 0.9 us and the engine
// 0.55, but the engine starts 7 us behind (N = 2048, T = 192: K = 2048 16 us
// against 20, K = 4096 42 against 31).
static bool use_proj(int T, int M, int C) {
  if (T <= 32) return true;  // a tile is one or two rows of MMAs: bound by W's bytes
  const int64_t tiles = int64_t((T + 63) / 64) * ((M + 63) / 64);
  const int nc = (C + 127) / 128;
  return tiles <= sm_count() && nc <= 18 * proj_parts(int(tiles), nc);
}

static TcGemmArgs projection(GemmMode mode, const int32_t *seg_offsets, const int32_t *seg_adapter, int T, int S,
                             int n_adapters, int rank, int N, int K, void *out, int64_t ldo, const Workspace &ws,
                             int32_t *err) {
  TcGemmArgs g = {};
  g.offsets = seg_offsets;
  g.adapter = seg_adapter;
  g.groups = 1;
  g.segs = S;
  g.n_adapters = n_adapters;
  g.rank = rank;
  g.R = T;
  g.M = mode == GEMM_FWD ? N : K;
  g.KD = mode == GEMM_FWD ? K : N;
  // The row tile width with the least time by the loads that bound a k-step: each
  // CTA loads 128 rows of W and bn / 2 rows of x in every round of tiles.
  const int pairs = sm_count() / 2;
  int bn = 256;
  int64_t best = INT64_MAX;
  for (int w = 256; w >= 64; w -= 16) {
    const int64_t tiles = int64_t((T + w - 1) / w) * ((g.M + 255) / 256);
    const int64_t cost = (tiles + pairs - 1) / pairs * (128 + w / 2);
    if (cost < best) { best = cost; bn = w; }
  }
  g.bn = bn;
  g.out = out;
  g.ldo = ldo;
  g.late = 1;
  g.err = err;
  g.sums = reinterpret_cast<float *>(ws.sums);  // there if N or K is long
  return g;
}

// Launches the sums of the blocks that several segments share and points the
// projection at them (one segment shares no block).
template <bool COLS>
static int shared_blocks(TcGemmArgs &g, int T, int S, const Workspace &ws, cudaStream_t s, const char *what) {
  if (S < 2) return MOE_OK;
  g.delta = ws.delta;
  g.delta_by_seg = int64_t(S) * 16 < (int64_t(T) + 15) / 16 * 16;
  g.row_seg = ws.row_seg;
  const DeltaArgs d = {g.offsets, g.adapter, g.row_seg, g.ext_b, g.ext_a, S, g.n_adapters, T, g.rank, g.M, g.delta_by_seg,
                       ws.delta};
  return launch_delta<COLS>(d, s, what);
}

}  // namespace lora
}  // namespace moe

extern "C" size_t moe_lora_workspace_size(int T, int S, int n_adapters, int rank, int N, int K) {
  (void)n_adapters;
  return moe::lora::workspace(T, S, rank, N, K, nullptr).whole;
}

extern "C" int moe_lora_linear(const moe_bf16 *x, int64_t ldx, const moe_bf16 *w, const int32_t *seg_offsets,
                               const int32_t *seg_adapter, const moe_bf16 *lora_a, const moe_bf16 *lora_b,
                               const float *scale, int T, int S, int n_adapters, int rank, int N, int K, moe_bf16 *u,
                               moe_bf16 *y, int64_t ldy, void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe::NvtxScope nvtx_scope("moe_lora_linear");
  using namespace moe;
  const char *who = "moe_lora_linear";
  int st = lora::check_common(who, w, seg_offsets, seg_adapter, lora_a, lora_b, T, S, n_adapters, rank, N, K, false, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (T == 0 || S == 0) return MOE_OK;
  if ((st = lora::check_rows(who, "x", x, ldx, K)) != MOE_OK || (st = lora::check_rows(who, "y", y, ldy, N)) != MOE_OK ||
      (st = lora::check_rows(who, "u", u, rank, rank)) != MOE_OK)
    return st;
  cudaStream_t s = as_stream(stream);
  int32_t *err = static_cast<int32_t *>(ws);
  const lora::Workspace space = lora::workspace(T, S, rank, N, K, ws);
  const bool engine = T > lora::GEMV_MAX_T && !lora::use_proj(T, N, K);
  int32_t *row_seg = engine && S > 1 ? space.row_seg : nullptr;

  if (T <= lora::GEMV_MAX_T || (rank <= 16 && T < 4 * int64_t(S))) {
    // short segments of small rank: each streams its adapter's A (whole call,
    // 256 single rows, K = N = 2048: rank 16 21 us against the shrink kernel's
    // 23.5, rank 64 39; 250 rows behind 99 single ones, rank 64: 36 against 27)
    GemvArgs v = {};
    v.in = x; v.ldi = ldx; v.offsets = seg_offsets; v.index = seg_adapter;
    v.w = lora_a; v.w_stride = int64_t(rank) * K;
    v.groups = S; v.n_weights = n_adapters; v.R = T; v.N = rank; v.K = K;
    v.scale = scale; v.out = u; v.ldo = rank; v.err = err;
    v.split = GEMV_LATER_PASSES;
    v.row_seg = row_seg;
    st = launch_gemm_gemv(v, s, "moe_lora_linear (adapters)");
  } else {
    const lora::ShrinkArgs h = {seg_offsets, seg_adapter, scale, S, n_adapters, T, K, rank, u, nullptr, row_seg, err};
    st = lora::launch_shrink<false>(h, {x, ldx, K}, lora_a, s, "moe_lora_linear (adapters)");
  }
  if (st != MOE_OK) return st;
  if (T <= lora::GEMV_MAX_T) {
    GemvArgs v = {};
    v.in = x; v.ldi = ldx; v.w = w; v.groups = 1; v.n_weights = 1; v.R = T; v.N = N; v.K = K;
    v.out = y; v.ldo = ldy; v.err = err;
    v.seg_offsets = seg_offsets; v.seg_adapter = seg_adapter; v.segs = S; v.n_adapters = n_adapters; v.rank = rank;
    v.u = u; v.lora_b = lora_b;
    return launch_gemm_gemv(v, s, who);
  }
  if (!engine) {
    const lora::ProjArgs v = {seg_offsets, seg_adapter, S, n_adapters, T, K, N, rank, u, lora_b, y, ldy, err};
    return lora::launch_proj<false>(v, {x, ldx, K}, w, s, who);
  }
  TcGemmArgs g = lora::projection(GEMM_FWD, seg_offsets, seg_adapter, T, S, n_adapters, rank, N, K, y, ldy, space, err);
  g.ext_a = lora_b;
  g.ext_b = u;
  if ((st = lora::shared_blocks<false>(g, T, S, space, s, "moe_lora_linear (shared blocks)")) != MOE_OK) return st;
  const TcGemmOperands op = {w, x, K, int64_t(N) * K, ldx};
  return launch_gemm_tc(GEMM_FWD, g, op, s, who);
}

extern "C" int moe_lora_linear_backward(const moe_bf16 *dy, int64_t lddy, const moe_bf16 *x, int64_t ldx,
                                        const moe_bf16 *w, const moe_bf16 *u, const int32_t *seg_offsets,
                                        const int32_t *seg_adapter, const moe_bf16 *lora_a, const moe_bf16 *lora_b,
                                        const float *scale, int T, int S, int n_adapters, int rank, int N, int K,
                                        moe_bf16 *du, moe_bf16 *dx, int64_t lddx, moe_bf16 *d_lora_a,
                                        moe_bf16 *d_lora_b, void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe::NvtxScope nvtx_scope("moe_lora_linear_backward");
  using namespace moe;
  const char *who = "moe_lora_linear_backward";
  int st = lora::check_common(who, w, seg_offsets, seg_adapter, lora_a, lora_b, T, S, n_adapters, rank, N, K, d_lora_a && T > 0 && S > 0, ws,
                              ws_bytes);
  if (st != MOE_OK) return st;
  if (!d_lora_a != !d_lora_b)
    return set_error(MOE_ERR_INVALID_ARG, "%s: d_lora_a and d_lora_b are given together or not at all", who);
  if (d_lora_a && (!aligned(d_lora_a, 16) || !aligned(d_lora_b, 16)))
    return set_error(MOE_ERR_INVALID_ARG, "%s: d_lora_a and d_lora_b must be 16-byte aligned", who);
  cudaStream_t s = as_stream(stream);
  if (T == 0 || S == 0) {
    cudaError_t e = cudaSuccess;
    if (d_lora_a) e = cudaMemsetAsync(d_lora_a, 0, size_t(n_adapters) * rank * K * 2, s);
    if (d_lora_b && e == cudaSuccess) e = cudaMemsetAsync(d_lora_b, 0, size_t(n_adapters) * rank * N * 2, s);
    return e == cudaSuccess ? MOE_OK : set_error(MOE_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  }
  if ((st = lora::check_rows(who, "dy", dy, lddy, N)) != MOE_OK ||
      (st = lora::check_rows(who, "du", du, rank, rank)) != MOE_OK ||
      (dx && (st = lora::check_rows(who, "dx", dx, lddx, K)) != MOE_OK) ||
      (d_lora_a && ((st = lora::check_rows(who, "x", x, ldx, K)) != MOE_OK ||
                    (st = lora::check_rows(who, "u", u, rank, rank)) != MOE_OK)))
    return st;
  int32_t *err = static_cast<int32_t *>(ws);
  const bool engine = dx && !lora::use_proj(T, K, N);
  const lora::Workspace space = lora::workspace(T, S, rank, N, K, ws);
  const lora::ShrinkArgs h = {seg_offsets, seg_adapter, scale, S, n_adapters, T, N, rank, du,
                              d_lora_a ? space.split : nullptr, engine && S > 1 ? space.row_seg : nullptr, err};
  if ((st = lora::launch_shrink<true>(h, {dy, lddy, N}, lora_b, s, "moe_lora_linear_backward (du)")) != MOE_OK) return st;
  TcGemmArgs g = {};
  if (engine) {
    g = lora::projection(GEMM_DGRAD, seg_offsets, seg_adapter, T, S, n_adapters, rank, N, K, dx, lddx, space, err);
    g.ext_a = lora_a;
    g.ext_b = du;
    if ((st = lora::shared_blocks<true>(g, T, S, space, s, "moe_lora_linear_backward (shared blocks)")) != MOE_OK) return st;
  }
  // The engine goes behind the adapters' gradients: it starts while they end and
  // waits for them only in its epilogue (six adapters of rank 16 at T = 2041, one
  // segment: 38.5 -> 35.1 us). The decode form overlaps du instead (T = 200, K = N
  // = 1024: 14.1 us, behind the gradients 16.2).
  if (dx && !engine) {
    const lora::ProjArgs v = {seg_offsets, seg_adapter, S, n_adapters, T, N, K, rank, du, lora_a, dx, lddx, err};
    if ((st = lora::launch_proj<true>(v, {dy, lddy, N}, w, s, who)) != MOE_OK) return st;
  }
  if (d_lora_a) {
    const int slabs_a = (K + lora::AG_COLS - 1) / lora::AG_COLS;
    const lora::AdapterGradArgs q = {seg_offsets, seg_adapter, S, n_adapters, T, N, K, rank, slabs_a, 0, 0, d_lora_a, d_lora_b, err};
    const char *what = "moe_lora_linear_backward (adapters)";
    const lora::Rows rx = {x, ldx, K}, rdy = {dy, lddy, N}, ru = {u, rank, rank}, rdu = {space.split, 2 * rank, 2 * rank};
    // long loads, or loads of 32 rows where segments are short on average (backward,
    // K = N = 2048, with 32 rows against long ones: rank 16, segments of 128 rows 37.3
    // and 37.7 us, of 64 38.6 and 40.6, of 32 28.6 and 32.6; rank 64, of 128 72.0 and
    // 68.9, of 64 74.9 and 71.6, of 32 81.8 and 82.6)
    st = T >= 64 * int64_t(S) ? lora::launch_adapter_grad<true>(q, rx, rdy, ru, rdu, s, what)
                              : lora::launch_adapter_grad<false>(q, rx, rdy, ru, rdu, s, what);
    if (st != MOE_OK) return st;
  }
  return engine ? launch_gemm_tc(GEMM_DGRAD, g, TcGemmOperands{w, dy, K, int64_t(N) * K, lddy}, s, who) : MOE_OK;
}
