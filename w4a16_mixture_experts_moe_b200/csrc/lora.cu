// Low-rank adapters of many requests beside a shared BF16 projection:
//   u[t]  = scale_a x[t] A_a^T     y[t]  = x[t] W^T + u[t] B_a^T
//   du[t] = scale_a dy[t] B_a      dx[t] = dy[t] W + du[t] A_a
//   dA_a  = sum_t du[t]^T x[t]     dB_a  = sum_t dy[t]^T u[t]
// for row t of a segment with adapter a. This file holds the entry points and
// the products of small rank (u, du; dA, dB); the projection with the adapters
// folded into its sums is gemm_tc.cu's (batches) or gemm_gemv.cu's (decode).
//
// u and du are rounded to BF16 once: they are operands of the BF16 matrix
// instructions that follow, and the adapter's part is a small share of y, so
// the rounding (2^-9 relative, independent from value to value) stays below
// y's own.
//
// The small-rank products read each row of x (dy) once and do 2 rank
// operations per value: at rank 64 that is 64 operations a byte, far below the
// tensor cores' balance point, so they are bound by memory and run on
// mma.sync from shared memory filled by cp.async.
#include "gemm.cuh"
#include "tma.cuh"

namespace moe {
namespace lora {

constexpr int MAX_RANK = 128;
constexpr int MAX_SEGS = 65535;  // a grid dimension of the decode form

__device__ __forceinline__ void cp16(void *dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void *p) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))));
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))));
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

struct ShrinkArgs {
  const uint16_t *z;  // [T][C] rows of x or dy
  int64_t ldz;
  const uint16_t *p;  // [n][rank][C] (lora_a), or [n][C][rank] (lora_b, TRANS)
  const int32_t *seg_offsets, *seg_adapter;
  const float *scale;
  int segs, n_adapters, T, C, rank;
  int split;          // CTAs that share a row tile's segments
  uint16_t *out;      // [T][rank]
  int32_t *err;
};

// RW x KW warps: RW 16-row tiles, and KW warps that split each stage's
// reduction (64 wide each).
template <int BJ, bool TRANS, int RW, int KW>
struct ShrinkCfg {
  static constexpr int ROWS = 16 * RW, C = 64 * KW, THREADS = 32 * RW * KW;
  static constexpr int STAGES = 4;
  static constexpr int ZLD = C + 8;                      // 8 elements of padding: no bank conflicts
  static constexpr int Z = ROWS * ZLD;                   // elements per stage
  static constexpr int PLD = TRANS ? BJ + 8 : C + 8;
  static constexpr int P = TRANS ? C * PLD : BJ * PLD;
  static constexpr int SMEM = STAGES * (Z + P) * 2;
  static_assert(KW * ROWS * (BJ + 1) * 4 <= SMEM, "the partial sums reuse the stages");
  static_assert(SMEM <= 200 * 1024, "shared memory budget");
};

// out[t][j] = bf16(scale_a sum_c z[t][c] P_a[j][c]) for a tile of 16 RW rows and
// BJ ranks. A tile may hold several segments: each CTA of the tile (blockIdx.y
// of `split`) takes every split-th of them, reads that segment's rows only
// (the others enter as zeros) and stores them.
template <int BJ, bool TRANS, int RW, int KW>
__global__ void __launch_bounds__(32 * RW * KW) shrink_kernel(const ShrinkArgs a) {
  using Cfg = ShrinkCfg<BJ, TRANS, RW, KW>;
  extern __shared__ __align__(16) uint16_t sm[];
  pdl_wait();     // in this order: the projection may start before u is there (gemm_gemv.cu), but
  pdl_trigger();  // not before what this launch itself waits for
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int rw = warp % RW, kw = warp / RW;
  if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
    for (int s = tid; s < a.segs; s += Cfg::THREADS) {
      const int o0 = a.seg_offsets[s], o1 = a.seg_offsets[s + 1], ad = a.seg_adapter[s];
      if (o0 < 0 || o1 < o0 || o1 > a.T || (s == 0 && o0 != 0)) flag_error(a.err, MOE_DEVERR_OFFSETS);
      if (ad < -1 || ad >= a.n_adapters) flag_error(a.err, MOE_DEVERR_EXPERT_ID);
    }
  }
  const int row0 = blockIdx.x * Cfg::ROWS, row1 = min(row0 + Cfg::ROWS, a.T), j0 = blockIdx.z * BJ;
  const int nc = (a.C + Cfg::C - 1) / Cfg::C;
  int turn = 0;
  for (int sg = first_segment(a.seg_offsets, a.segs, row0); sg < a.segs; ++sg) {
    const int o0 = a.seg_offsets[sg];
    if (o0 >= row1) break;
    const int lo = max(o0, row0), hi = min(a.seg_offsets[sg + 1], row1), ad = a.seg_adapter[sg];
    if (hi <= lo || turn++ % a.split != int(blockIdx.y)) continue;
    if (ad < 0 || ad >= a.n_adapters) {  // no adapter: nothing is added to these rows
      for (int p = tid; p < (hi - lo) * BJ; p += Cfg::THREADS)
        if (j0 + p % BJ < a.rank) a.out[int64_t(lo + p / BJ) * a.rank + j0 + p % BJ] = 0;
      continue;
    }
    const uint16_t *pa = a.p + int64_t(ad) * a.rank * a.C;
    auto load = [&](int c) {
      uint16_t *zs = sm + (c % Cfg::STAGES) * (Cfg::Z + Cfg::P), *ps = zs + Cfg::Z;
      const int c0 = c * Cfg::C;
      constexpr int CP = Cfg::C / 8;  // 16-byte pieces of a row
#pragma unroll
      for (int i = tid; i < Cfg::ROWS * CP; i += Cfg::THREADS) {
        const int r = i / CP, cc = i % CP * 8;
        const bool ok = row0 + r >= lo && row0 + r < hi && c0 + cc < a.C;
        cp16(zs + r * Cfg::ZLD + cc, a.z + (ok ? int64_t(row0 + r) * a.ldz + c0 + cc : 0), ok);
      }
      if (TRANS) {
#pragma unroll
        for (int i = tid; i < Cfg::C * (BJ / 8); i += Cfg::THREADS) {
          const int r = i / (BJ / 8), jj = i % (BJ / 8) * 8;
          const bool ok = c0 + r < a.C && j0 + jj < a.rank;
          cp16(ps + r * Cfg::PLD + jj, pa + (ok ? int64_t(c0 + r) * a.rank + j0 + jj : 0), ok);
        }
      } else {
#pragma unroll
        for (int i = tid; i < BJ * CP; i += Cfg::THREADS) {
          const int r = i / CP, cc = i % CP * 8;
          const bool ok = j0 + r < a.rank && c0 + cc < a.C;
          cp16(ps + r * Cfg::PLD + cc, pa + (ok ? int64_t(j0 + r) * a.C + c0 + cc : 0), ok);
        }
      }
    };
    float acc[BJ / 8][4];
#pragma unroll
    for (int j = 0; j < BJ / 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;
    const bool mine = row0 + rw * 16 < hi && row0 + rw * 16 + 16 > lo;  // rows of the segment in this warp
    __syncthreads();  // the previous segment's sums are read
#pragma unroll
    for (int c = 0; c < Cfg::STAGES - 1; ++c) {
      if (c < nc) load(c);
      cp_commit();
    }
    for (int c = 0; c < nc; ++c) {
      cp_wait<Cfg::STAGES - 2>();
      __syncthreads();
      if (c + Cfg::STAGES - 1 < nc) load(c + Cfg::STAGES - 1);
      cp_commit();
      const uint16_t *zs = sm + (c % Cfg::STAGES) * (Cfg::Z + Cfg::P), *ps = zs + Cfg::Z;
      if (!mine) continue;
#pragma unroll
      for (int kk = kw * 64; kk < kw * 64 + 64; kk += 16) {
        uint32_t af[4];
        ldsm4<false>(af, zs + (rw * 16 + (lane & 15)) * Cfg::ZLD + kk + (lane >> 4) * 8);
#pragma unroll
        for (int jp = 0; jp < BJ / 16; ++jp) {
          uint32_t bf[4];
          if (TRANS)  // stored [c][j]
            ldsm4<true>(bf, ps + (kk + (lane & 7) + ((lane >> 3) & 1) * 8) * Cfg::PLD + jp * 16 + (lane >> 4) * 8);
          else        // stored [j][c]
            ldsm4<false>(bf, ps + (jp * 16 + (lane & 7) + (lane >> 4) * 8) * Cfg::PLD + kk + ((lane >> 3) & 1) * 8);
          mma_16816(acc[2 * jp], af, bf[0], bf[1]);
          mma_16816(acc[2 * jp + 1], af, bf[2], bf[3]);
        }
      }
    }
    cp_wait<0>();
    __syncthreads();
    float *red = reinterpret_cast<float *>(sm);  // [KW][ROWS][BJ + 1]
#pragma unroll
    for (int j = 0; j < BJ / 8; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(kw * Cfg::ROWS + rw * 16 + g + (q >> 1) * 8) * (BJ + 1) + j * 8 + 2 * t4 + (q & 1)] = acc[j][q];
    __syncthreads();
    const float sc = a.scale ? a.scale[ad] : 1.f;
    for (int p = tid; p < (hi - lo) * (BJ / 2); p += Cfg::THREADS) {
      const int r = lo - row0 + p / (BJ / 2), jj = p % (BJ / 2) * 2;
      if (j0 + jj >= a.rank) continue;
      float v0 = 0.f, v1 = 0.f;
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        v0 += red[(k * Cfg::ROWS + r) * (BJ + 1) + jj];
        v1 += red[(k * Cfg::ROWS + r) * (BJ + 1) + jj + 1];
      }
      *reinterpret_cast<uint32_t *>(a.out + int64_t(row0 + r) * a.rank + j0 + jj) = pack_bf16x2(v0 * sc, v1 * sc);
    }
  }
}

struct AdapterGradArgs {
  const uint16_t *x, *dy, *u, *du;
  int64_t ldx, lddy;
  const int32_t *seg_offsets, *seg_adapter;
  int segs, n_adapters, T, N, K, rank;
  int slabs_a;        // 64-column slabs of x; the others are dy's
  uint16_t *da, *db;  // [n][rank][K], [n][N][rank]
};

constexpr int AG_COLS = 64, AG_ROWS = 64, AG_LD = 72, AG_STAGES = 4;

template <int RJ>
struct AdapterGradCfg {
  static constexpr int PLD = RJ + 8;
  static constexpr int STAGE = AG_ROWS * (AG_LD + PLD);
  static constexpr int SMEM = AG_STAGES * STAGE * 2;
};

// The gradients of one adapter for a slab of 64 columns c of x (dA) or dy (dB):
// G[j][c] = sum over the rows t of the adapter's segments of p[t][j] z[t][c],
// with p = du, z = x or p = u, z = dy. Rows pass 64 at a time through shared
// memory, read transposed (ldmatrix.trans): M = columns (16 per warp), N =
// ranks, K = rows. The segments are taken in order by one CTA, so the sum's
// order is fixed. An adapter without rows gets zeros.
template <int RJ>
__global__ void __launch_bounds__(128) adapter_grad_kernel(const AdapterGradArgs a) {
  using Cfg = AdapterGradCfg<RJ>;
  extern __shared__ __align__(16) uint16_t sm[];
  __shared__ int seg_lo[128], seg_hi[128], first[128], wsum[4];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
  const int ad = blockIdx.y;
  const bool is_a = int(blockIdx.x) < a.slabs_a;
  const int c0 = (is_a ? blockIdx.x : blockIdx.x - a.slabs_a) * AG_COLS, C = is_a ? a.K : a.N;
  const uint16_t *z = is_a ? a.x : a.dy, *p = is_a ? a.du : a.u;
  const int64_t ldz = is_a ? a.ldx : a.lddy;
  float acc[RJ / 8][4];
#pragma unroll
  for (int j = 0; j < RJ / 8; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[j][q] = 0.f;

  // A window of the segment list at a time: this adapter's segments in order,
  // as one sequence of 64-row chunks, so the loads run on across segments.
  for (int s0 = 0; s0 < a.segs; s0 += 128) {
    const int s = s0 + tid;
    int lo = 0, nch = 0;
    if (s < a.segs && a.seg_adapter[s] == ad) {
      lo = max(a.seg_offsets[s], 0);
      nch = max(0, min(a.seg_offsets[s + 1], a.T) - lo);
      seg_hi[tid] = lo + nch;
      nch = (nch + AG_ROWS - 1) / AG_ROWS;
    }
    int incl = nch;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += wsum[w];
    const int total = wsum[0] + wsum[1] + wsum[2] + wsum[3];
    seg_lo[tid] = lo;
    first[tid] = incl - nch;  // the segment's first chunk
    __syncthreads();
    auto load = [&](int c) {
      int l = 0, h = 128;  // the last segment whose first chunk is at most c (it has chunks: c lies in it)
      while (h - l > 1) {
        const int mid = (l + h) >> 1;
        if (first[mid] <= c) l = mid; else h = mid;
      }
      const int r0 = seg_lo[l] + (c - first[l]) * AG_ROWS, hi = seg_hi[l];
      uint16_t *zs = sm + (c % AG_STAGES) * Cfg::STAGE, *ps = zs + AG_ROWS * AG_LD;
#pragma unroll
      for (int i = tid; i < AG_ROWS * 8; i += 128) {
        const int r = i >> 3, cc = (i & 7) * 8;
        const bool ok = r0 + r < hi && c0 + cc < C;
        cp16(zs + r * AG_LD + cc, z + (ok ? int64_t(r0 + r) * ldz + c0 + cc : 0), ok);
      }
#pragma unroll
      for (int i = tid; i < AG_ROWS * (RJ / 8); i += 128) {
        const int r = i / (RJ / 8), jj = i % (RJ / 8) * 8;
        const bool ok = r0 + r < hi && jj < a.rank;
        cp16(ps + r * Cfg::PLD + jj, p + (ok ? int64_t(r0 + r) * a.rank + jj : 0), ok);
      }
    };
#pragma unroll
    for (int c = 0; c < AG_STAGES - 1; ++c) {
      if (c < total) load(c);
      cp_commit();
    }
    for (int c = 0; c < total; ++c) {
      cp_wait<AG_STAGES - 2>();
      __syncthreads();
      if (c + AG_STAGES - 1 < total) load(c + AG_STAGES - 1);
      cp_commit();
      const uint16_t *zs = sm + (c % AG_STAGES) * Cfg::STAGE, *ps = zs + AG_ROWS * AG_LD;
#pragma unroll
      for (int kk = 0; kk < AG_ROWS / 16; ++kk) {
        uint32_t af[4];
        ldsm4<true>(af, zs + (kk * 16 + (lane & 7) + (lane >> 4) * 8) * AG_LD + warp * 16 + ((lane >> 3) & 1) * 8);
#pragma unroll
        for (int jp = 0; jp < RJ / 16; ++jp) {
          uint32_t bf[4];
          ldsm4<true>(bf, ps + (kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8) * Cfg::PLD + jp * 16 + (lane >> 4) * 8);
          mma_16816(acc[2 * jp], af, bf[0], bf[1]);
          mma_16816(acc[2 * jp + 1], af, bf[2], bf[3]);
        }
      }
    }
    cp_wait<0>();
    __syncthreads();
  }
  // accumulator (c0, c1) = column g, ranks 2t, 2t+1; (c2, c3) = column g + 8
#pragma unroll
  for (int j = 0; j < RJ / 8; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = c0 + warp * 16 + g + h * 8, jj = j * 8 + 2 * t4;
      if (c >= C || jj >= a.rank) continue;
      if (is_a) {
        uint16_t *o = a.da + (int64_t(ad) * a.rank + jj) * a.K + c;
        o[0] = f_to_bf16(acc[j][2 * h]);
        o[a.K] = f_to_bf16(acc[j][2 * h + 1]);
      } else {
        *reinterpret_cast<uint32_t *>(a.db + (int64_t(ad) * a.N + c) * a.rank + jj) =
            pack_bf16x2(acc[j][2 * h], acc[j][2 * h + 1]);
      }
    }
}

template <int BJ, bool TRANS, int RW, int KW>
static int launch_shrink_as(ShrinkArgs a, cudaStream_t s, const char *what) {
  using Cfg = ShrinkCfg<BJ, TRANS, RW, KW>;
  int st = allow_dynamic_smem(reinterpret_cast<const void *>(shrink_kernel<BJ, TRANS, RW, KW>), Cfg::SMEM, what);
  if (st != MOE_OK) return st;
  // as many CTAs per row tile as it holds segments on average
  const int64_t per = (int64_t(a.segs) * Cfg::ROWS + a.T - 1) / a.T;
  a.split = int(per < 1 ? 1 : per > Cfg::ROWS ? Cfg::ROWS : per);
  const dim3 grid(unsigned((a.T + Cfg::ROWS - 1) / Cfg::ROWS), unsigned(a.split), unsigned((a.rank + BJ - 1) / BJ));
  const cudaError_t e = launch_pdl(shrink_kernel<BJ, TRANS, RW, KW>, grid, dim3(Cfg::THREADS), Cfg::SMEM, s, a);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

// 16-row tiles until they fill the SMs about twice over; then 64-row tiles,
// which read each adapter a quarter as often.
constexpr int SHRINK_WIDE_T = 4096;

template <bool TRANS>
static int launch_shrink(const ShrinkArgs &a, cudaStream_t s, const char *what) {
  if (a.T < SHRINK_WIDE_T)
    return a.rank <= 16   ? launch_shrink_as<16, TRANS, 1, 4>(a, s, what)
           : a.rank <= 32 ? launch_shrink_as<32, TRANS, 1, 4>(a, s, what)
                          : launch_shrink_as<64, TRANS, 1, 4>(a, s, what);
  return a.rank <= 16   ? launch_shrink_as<16, TRANS, 4, 2>(a, s, what)
         : a.rank <= 32 ? launch_shrink_as<32, TRANS, 4, 2>(a, s, what)
                        : launch_shrink_as<64, TRANS, 4, 2>(a, s, what);
}

template <int RJ>
static int launch_adapter_grad_as(const AdapterGradArgs &a, cudaStream_t s, const char *what) {
  const size_t smem = AdapterGradCfg<RJ>::SMEM;
  int st = allow_dynamic_smem(reinterpret_cast<const void *>(adapter_grad_kernel<RJ>), smem, what);
  if (st != MOE_OK) return st;
  const dim3 grid(unsigned(a.slabs_a + (a.N + AG_COLS - 1) / AG_COLS), unsigned(a.n_adapters));
  const cudaError_t e = launch_pdl(adapter_grad_kernel<RJ>, grid, dim3(128), smem, s, a);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

// The arguments both entry points share.
static int check_common(const char *who, const void *w, const void *seg_offsets, const void *seg_adapter,
                        const void *lora_a, const void *lora_b, int T, int S, int n_adapters, int rank, int N, int K,
                        const void *ws, size_t ws_bytes) {
  if (T < 0 || T > (1 << 30) || S < 0 || S > MAX_SEGS || n_adapters < 1 || n_adapters > MAX_SEGS)
    return set_error(MOE_ERR_SHAPE, "%s: T=%d S=%d n_adapters=%d (need 0<=T<=2^30, 0<=S<=65535, 1<=n_adapters<=65535)",
                     who, T, S, n_adapters);
  if (rank < 8 || rank > MAX_RANK || rank % 8)
    return set_error(MOE_ERR_SHAPE, "%s: rank=%d must be a multiple of 8 from 8 to 128", who, rank);
  if (N < 8 || K < 8 || N % 8 || K % 8)
    return set_error(MOE_ERR_SHAPE, "%s: N=%d K=%d must be positive multiples of 8", who, N, K);
  if (!ws || !w || !lora_a || !lora_b || !seg_offsets || (S > 0 && !seg_adapter))
    return set_error(MOE_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned(ws, 256) || !aligned(w, 16) || !aligned(lora_a, 16) || !aligned(lora_b, 16))
    return set_error(MOE_ERR_INVALID_ARG, "%s: ws needs 256-byte, w, lora_a and lora_b 16-byte alignment", who);
  const size_t need = moe_lora_workspace_size(T, S, n_adapters, rank, N, K);
  if (ws_bytes < need) return set_error(MOE_ERR_INVALID_ARG, "%s: workspace %zu B < %zu B", who, ws_bytes, need);
  return MOE_OK;
}

static int check_rows(const char *who, const char *name, const void *p, int64_t ld, int width) {
  if (!p || !aligned(p, 16) || ld < width || ld % 8)
    return set_error(MOE_ERR_INVALID_ARG, "%s: %s must be 16-byte aligned, its row stride (%lld) a multiple of 8 and at least %d",
                     who, name, (long long)ld, width);
  return MOE_OK;
}

// Up to this many rows the projection runs as a weight stream, all rows in one
// pass over W.
constexpr int GEMV_MAX_T = 64;

static TcGemmArgs projection(GemmMode mode, const int32_t *seg_offsets, const int32_t *seg_adapter, int T, int S,
                             int n_adapters, int rank, int N, int K, void *out, int64_t ldo, int32_t *err) {
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
  g.err = err;
  return g;
}

}  // namespace lora
}  // namespace moe

extern "C" size_t moe_lora_workspace_size(int T, int S, int n_adapters, int rank, int N, int K) {
  (void)T; (void)S; (void)n_adapters; (void)rank; (void)N; (void)K;
  return moe::WS_HEADER;
}

extern "C" int moe_lora_linear(const moe_bf16 *x, int64_t ldx, const moe_bf16 *w, const int32_t *seg_offsets,
                               const int32_t *seg_adapter, const moe_bf16 *lora_a, const moe_bf16 *lora_b,
                               const float *scale, int T, int S, int n_adapters, int rank, int N, int K, moe_bf16 *u,
                               moe_bf16 *y, int64_t ldy, void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe::NvtxScope nvtx_scope("moe_lora_linear");
  using namespace moe;
  const char *who = "moe_lora_linear";
  int st = lora::check_common(who, w, seg_offsets, seg_adapter, lora_a, lora_b, T, S, n_adapters, rank, N, K, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if (T == 0 || S == 0) return MOE_OK;
  if ((st = lora::check_rows(who, "x", x, ldx, K)) != MOE_OK || (st = lora::check_rows(who, "y", y, ldy, N)) != MOE_OK ||
      (st = lora::check_rows(who, "u", u, rank, rank)) != MOE_OK)
    return st;
  cudaStream_t s = as_stream(stream);
  int32_t *err = static_cast<int32_t *>(ws);

  if (T <= lora::GEMV_MAX_T || T < 16 * S) {
    // short segments: each streams its adapter's A
    GemvArgs v = {};
    v.in = x; v.ldi = ldx; v.offsets = seg_offsets; v.index = seg_adapter;
    v.w = lora_a; v.w_stride = int64_t(rank) * K;
    v.groups = S; v.n_weights = n_adapters; v.R = T; v.N = rank; v.K = K;
    v.scale = scale; v.out = u; v.ldo = rank; v.err = err;
    st = launch_gemm_gemv(v, S, s, "moe_lora_linear (adapters)");
  } else {
    lora::ShrinkArgs h = {x, ldx, lora_a, seg_offsets, seg_adapter, scale, S, n_adapters, T, K, rank, 1, u, err};
    st = lora::launch_shrink<false>(h, s, "moe_lora_linear (adapters)");
  }
  if (st != MOE_OK) return st;
  if (T <= lora::GEMV_MAX_T) {
    GemvArgs v = {};
    v.in = x; v.ldi = ldx; v.w = w; v.groups = 1; v.n_weights = 1; v.R = T; v.N = N; v.K = K;
    v.out = y; v.ldo = ldy; v.err = err;
    v.seg_offsets = seg_offsets; v.seg_adapter = seg_adapter; v.segs = S; v.n_adapters = n_adapters; v.rank = rank;
    v.u = u; v.lora_b = lora_b;
    return launch_gemm_gemv(v, 1, s, who);
  }
  TcGemmArgs g = lora::projection(GEMM_FWD, seg_offsets, seg_adapter, T, S, n_adapters, rank, N, K, y, ldy, err);
  g.ext_a = lora_b;
  g.ext_b = u;
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
  int st = lora::check_common(who, w, seg_offsets, seg_adapter, lora_a, lora_b, T, S, n_adapters, rank, N, K, ws, ws_bytes);
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
  lora::ShrinkArgs h = {dy, lddy, lora_b, seg_offsets, seg_adapter, scale, S, n_adapters, T, N, rank, 1, du, err};
  if ((st = lora::launch_shrink<true>(h, s, "moe_lora_linear_backward (du)")) != MOE_OK) return st;
  if (dx) {
    TcGemmArgs g = lora::projection(GEMM_DGRAD, seg_offsets, seg_adapter, T, S, n_adapters, rank, N, K, dx, lddx, err);
    g.ext_a = lora_a;
    g.ext_b = du;
    const TcGemmOperands op = {w, dy, K, int64_t(N) * K, lddy};
    if ((st = launch_gemm_tc(GEMM_DGRAD, g, op, s, who)) != MOE_OK) return st;
  }
  if (!d_lora_a) return MOE_OK;
  lora::AdapterGradArgs q = {x, dy, u, du, ldx, lddy, seg_offsets, seg_adapter, S, n_adapters, T, N, K, rank,
                             (K + lora::AG_COLS - 1) / lora::AG_COLS, d_lora_a, d_lora_b};
  const char *what = "moe_lora_linear_backward (adapters)";
  return rank <= 16   ? lora::launch_adapter_grad_as<16>(q, s, what)
         : rank <= 32 ? lora::launch_adapter_grad_as<32>(q, s, what)
         : rank <= 64 ? lora::launch_adapter_grad_as<64>(q, s, what)
                      : lora::launch_adapter_grad_as<128>(q, s, what);
}
