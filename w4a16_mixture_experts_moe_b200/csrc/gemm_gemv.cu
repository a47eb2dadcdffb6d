// The BF16 product out[r] = in[r] W^T over ragged row groups for the smallest
// groups (decode): the weights are the only large operand, each read once, so
// the kernel is bound by HBM and by how many loads are in flight.
//
// A CTA owns 16 output columns (weight rows) of one group; its warps take K in
// interleaved pieces of 128. Lane (g, t) = (lane / 4, lane % 4) loads 16 bytes
// (8 weights) of rows g and g + 8 at each of a piece's four 32-wide chunks:
// eight independent loads, 4 KB per warp, are in
// flight before the first MMA (mma.sync m16n8k16). A dot product does not depend on the order of its
// terms, so a lane's fragment slots are bound to its own eight consecutive k,
// for the rows of `in` (8 per MMA) as well. The warps' partial sums meet in
// shared memory and are added in a fixed order.
//
// A pass takes 16 rows and reads the weights again (from L2): groups of a few
// rows are one pass. Passes of long groups go to CTAs of their own, which find
// theirs by counting (the whole projection, N = K = 2048, rank 16, of 99 single
// rows and a segment of 1400: 262 -> 46 us; 64 groups of 2 rows 44 -> 45).
//
// Per-request adapters are added where the sums meet: out[r][n] gets the dot
// product of u[r] and row n of its adapter's B (rank values, contiguous), so
// they cost one small read per (row, column). u comes from the launch before:
// this kernel streams W first and waits for that launch only then.
#include "gemm.cuh"

namespace moe {
namespace gv {

constexpr int COLS = 16;     // output columns per CTA
constexpr int LD = COLS + 1; // row stride of the partial sums
constexpr int CH = 4;        // 32-wide chunks of a piece
constexpr int MAXNT = GEMV_PASS / 8;  // 8-row tiles of `in` per pass

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once per pass over the rows: no use for them in L1.
__device__ __forceinline__ uint4 ld_stream(const uint16_t *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// This warp's partial sums for NT * 8 rows of `in` from row r0, into red[row][column].
template <int NT, int WARPS>
__device__ __forceinline__ void rows_pass(const GemvArgs &a, const uint16_t *w, int n0, int64_t r0, int rows, float *red) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint16_t *wr = w + int64_t(n0 + g) * a.K + 8 * t;
  const uint16_t *xr = a.in + (r0 + g) * a.ldi + 8 * t;
  float sum[NT][4];  // each piece's MMAs start from zero: their truncating additions stay few
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) sum[i][q] = 0.f;
#pragma unroll 1
  for (int k0 = warp * CH * 32; k0 < a.K; k0 += WARPS * CH * 32) {
    uint4 wv[2][CH];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < CH; ++c)
        wv[i][c] = k0 + 32 * c + 8 * t < a.K && n0 + g + 8 * i < a.N ? ld_stream(wr + int64_t(8 * i) * a.K + k0 + 32 * c) : zero;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      uint4 xv[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c)
        xv[c] = k0 + 32 * c + 8 * t < a.K && g + 8 * i < rows
                    ? __ldg(reinterpret_cast<const uint4 *>(xr + 8 * i * a.ldi + k0 + 32 * c))
                    : zero;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint4 &wa = wv[0][c], &wb = wv[1][c];
        mma_16816(acc, wa.x, wb.x, wa.y, wb.y, xv[c].x, xv[c].y);
        mma_16816(acc, wa.z, wb.z, wa.w, wb.w, xv[c].z, xv[c].w);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[i][q] += acc[q];
    }
  }
  // (c0, c1) = weight row g, rows 2t, 2t+1 of the 8-row tile; (c2, c3) = weight row g + 8
  float *o = red + warp * NT * 8 * LD;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) o[(8 * i + 2 * t + (q & 1)) * LD + g + (q >> 1) * 8] = sum[i][q];
}

// The dot product of u[row] and row n of the adapter of row's segment.
__device__ __forceinline__ float adapter_dot(const GemvArgs &a, int row, int n) {
  const int lo = first_segment(a.seg_offsets, a.segs, row);
  const int ad = lo < a.segs && a.seg_offsets[lo] <= row ? a.seg_adapter[lo] : -1;
  float d = 0.f;
  if (ad >= 0 && ad < a.n_adapters) {
    const uint4 *b = reinterpret_cast<const uint4 *>(a.lora_b + (int64_t(ad) * a.N + n) * a.rank);
    const uint4 *u = reinterpret_cast<const uint4 *>(a.u + int64_t(row) * a.rank);
#pragma unroll 2
    for (int j = 0; j < a.rank / 8; ++j) {
      const uint4 bv = __ldg(b + j), uv = u[j];
      d = fmaf(bf16_lo(bv.x), bf16_lo(uv.x), d); d = fmaf(bf16_hi(bv.x), bf16_hi(uv.x), d);
      d = fmaf(bf16_lo(bv.y), bf16_lo(uv.y), d); d = fmaf(bf16_hi(bv.y), bf16_hi(uv.y), d);
      d = fmaf(bf16_lo(bv.z), bf16_lo(uv.z), d); d = fmaf(bf16_hi(bv.z), bf16_hi(uv.z), d);
      d = fmaf(bf16_lo(bv.w), bf16_lo(uv.w), d); d = fmaf(bf16_hi(bv.w), bf16_hi(uv.w), d);
    }
  }
  return d;
}

template <int WARPS>
struct Cfg {
  static constexpr int SMEM = WARPS * MAXNT * 8 * LD * 4;
};

template <int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 24 / WARPS) gemv_kernel(const GemvArgs a) {
  extern __shared__ float red[];
  __shared__ int found[32], which, pass;
  const bool late = a.seg_adapter != nullptr;  // the previous launch only writes u
  // A launch that starts early may count on what this one waited for. With
  // adapters the launch before has waited for all of that already, and this one
  // waits for that launch before it ends.
  if (!late) pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int e = blockIdx.y, r_first = 0;
  if (a.split == GEMV_ALL_PASSES || (a.split == GEMV_LATER_PASSES && e >= a.groups)) {
    // the want-th pass of the groups' passes, counted from each group's `from`-th
    const int from = a.split == GEMV_ALL_PASSES ? 0 : 1, want = e - from * a.groups;
    const bool check = want == 0 && from == 0;  // looks at every group
    if (tid == 0) which = -1;
    int base = 0;
    for (int e0 = 0; e0 < a.groups && (base <= want || check); e0 += WARPS * 32) {
      const int q = e0 + tid;
      const int o0 = q < a.groups ? a.offsets[q] : 0, o1 = q < a.groups ? a.offsets[q + 1] : 0;
      if (check && blockIdx.x == 0 && (o0 < 0 || o1 < o0 || o1 > a.R)) flag_error(a.err, MOE_DEVERR_OFFSETS);
      const int rows = min(max(o1, 0), a.R) - min(max(o0, 0), a.R);
      const int n = max(0, (rows + MAXNT * 8 - 1) / (MAXNT * 8) - from);
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int p = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += p;
      }
      __syncthreads();
      if (lane == 31) found[warp] = incl;
      __syncthreads();
      int before = base + incl - n;
      for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += found[w];
        base += found[w];
      }
      if (before <= want && want < before + n) { which = q; pass = want - before + from; }
    }
    __syncthreads();
    e = which;
    if (e < 0) return;
    r_first = pass * MAXNT * 8;
  }
  // with adapters: one group, the rows up to the end of the last segment
  const int o0 = late ? 0 : a.offsets[e], o1 = late ? a.seg_offsets[a.segs] : a.offsets[e + 1];
  // (segments start at row 0, groups anywhere)
  if ((o0 < 0 || o1 < o0 || o1 > a.R || (a.index && e == 0 && o0 != 0)) && blockIdx.x == 0 && tid == 0)
    flag_error(a.err, MOE_DEVERR_OFFSETS);
  const int lo = min(max(o0, 0), a.R), rows_in = min(max(o1, 0), a.R) - lo;
  if (rows_in <= 0) {
    if (late) pdl_wait();  // the launches behind this one wait for it alone
    return;
  }
  const int cnt = a.split == GEMV_WHOLE ? rows_in : min(rows_in, r_first + MAXNT * 8);  // this CTA's: r_first .. cnt - 1
  if (a.row_seg && blockIdx.x == 0)
    for (int r = r_first + tid; r < cnt; r += WARPS * 32) a.row_seg[lo + r] = e;
  const int wi = a.index ? a.index[e] : e;
  const bool none = wi < 0 || wi >= a.n_weights;
  if (none && wi != -1 && blockIdx.x == 0 && tid == 0) flag_error(a.err, MOE_DEVERR_EXPERT_ID);
  const uint16_t *w = a.w + int64_t(none ? 0 : wi) * a.w_stride;
  const float scale = none ? 0.f : a.scale ? a.scale[wi] : 1.f;
  const int n0 = blockIdx.x * COLS;

#pragma unroll 1
  for (int r0 = r_first; r0 < cnt; r0 += MAXNT * 8) {
    const int rows = min(MAXNT * 8, cnt - r0);
    int nt = 1;  // 8-row tiles of this pass, the stride of the partial sums
    if (!none) {
      if (rows <= 8) {
        rows_pass<1, WARPS>(a, w, n0, lo + r0, rows, red);
      } else {
        nt = 2;
        rows_pass<2, WARPS>(a, w, n0, lo + r0, rows, red);
      }
    }
    if (late && r0 == 0) pdl_wait();
    __syncthreads();
    for (int p = tid; p < rows * COLS; p += WARPS * 32) {
      const int r = p / COLS, n = p % COLS, row = lo + r0 + r;
      if (n0 + n >= a.N) continue;
      float v = 0.f;
      if (!none) {
#pragma unroll
        for (int q = 0; q < WARPS; ++q) v += red[(q * nt * 8 + r) * LD + n];
        v *= scale;
      }
      if (late) v += adapter_dot(a, row, n0 + n);
      const int64_t at = int64_t(row) * a.ldo + n0 + n;
      if (a.out_f32) {
        float *o = static_cast<float *>(a.out);
        o[at] = a.accumulate ? o[at] + v : v;
      } else {
        static_cast<uint16_t *>(a.out)[at] = f_to_bf16(v);
      }
    }
    __syncthreads();
  }
}

template <int WARPS>
static int launch_as(const GemvArgs &a, int grid_groups, cudaStream_t s, const char *what) {
  constexpr size_t smem = Cfg<WARPS>::SMEM;
  static_assert(smem <= 48 * 1024, "shared memory without a raised limit");
  const dim3 grid(unsigned((a.N + COLS - 1) / COLS), unsigned(grid_groups));
  const cudaError_t e = launch_pdl(gemv_kernel<WARPS>, grid, dim3(WARPS * 32), smem, s, a);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

}  // namespace gv

int launch_gemm_gemv(GemvArgs a, cudaStream_t s, const char *what) {
  // at most one pass per row; at most (R - 1) / GEMV_PASS behind the groups' first
  const int64_t later = (a.R - 1) / GEMV_PASS;
  if (a.split == GEMV_LATER_PASSES && a.groups + later > 65535) a.split = GEMV_WHOLE;  // a grid dimension's limit
  const int ny = a.split == GEMV_ALL_PASSES ? a.R : a.split == GEMV_LATER_PASSES ? int(a.groups + later) : a.groups;
  if (a.seg_adapter) return gv::launch_as<8>(a, ny, s, what);  // one group of few rows
  // few CTAs: more warps share a CTA's reduction
  const int64_t ctas = int64_t(ny) * ((a.N + 15) / 16);
  if (ctas <= 2 * 148) return gv::launch_as<16>(a, ny, s, what);
  return gv::launch_as<4>(a, ny, s, what);
}

}  // namespace moe
