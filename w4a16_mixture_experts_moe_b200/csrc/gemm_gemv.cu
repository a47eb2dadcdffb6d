// The BF16 product out[r] = in[r] W^T over ragged row groups for the smallest
// groups (decode): the weights are the only large operand, each read once, so
// the kernel is bound by HBM and by how many loads are in flight.
//
// A CTA owns 16 output columns (weight rows) of one group; its eight warps
// take K in interleaved 128-wide pieces. Lane (g, t) = (lane / 4, lane % 4)
// loads 16 bytes (8 weights) of rows g and g + 8 at each of a piece's four
// 32-wide chunks: eight independent 16-byte loads per lane, 4 KB per warp, are
// in flight before the first MMA (mma.sync m16n8k16). A dot product does not
// depend on the order of its terms, so a lane's fragment slots are bound to
// its own eight consecutive k, for the rows of `in` (8 per MMA) as well. The
// eight partial sums meet in shared memory and are added in a fixed order.
//
// Per-request adapters are added where the sums meet: out[r][n] gets the dot
// product of u[r] and row n of its adapter's B (rank values, contiguous), so
// they cost one small read per (row, column) and no launch.
#include "gemm.cuh"

namespace moe {
namespace gv {

constexpr int WARPS = 8;
constexpr int ROWS = 16;  // output columns (weight rows) per CTA
constexpr int MAX_NT = 4; // 8-row tiles of `in` per pass
constexpr int PIECE = 128;

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

// Partial sums of this warp's pieces for 8 * NT rows from row r0, into red.
template <int NT>
__device__ __forceinline__ void rows_pass(const GemvArgs &a, const uint16_t *w, int n0, int r0, int rows,
                                          float (*red)[MAX_NT * 8][ROWS + 1]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const bool ok0 = n0 + g < a.N, ok1 = n0 + g + 8 < a.N;
  const uint16_t *w0 = w + int64_t(n0 + g) * a.K + 8 * t, *w1 = w0 + int64_t(8) * a.K;
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[i][q] = 0.f;
  for (int k0 = warp * PIECE; k0 < a.K; k0 += WARPS * PIECE) {
    uint4 wa[4], wb[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const bool in = k0 + 32 * c + 8 * t < a.K;
      wa[c] = in && ok0 ? ld_stream(w0 + k0 + 32 * c) : zero;
      wb[c] = in && ok1 ? ld_stream(w1 + k0 + 32 * c) : zero;
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int r = 8 * i + g;
      const uint16_t *x = a.in + int64_t(r0 + r) * a.ldi + 8 * t + k0;
      uint4 xv[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        xv[c] = r < rows && k0 + 32 * c + 8 * t < a.K ? *reinterpret_cast<const uint4 *>(x + 32 * c) : zero;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        mma_16816(acc[i], wa[c].x, wb[c].x, wa[c].y, wb[c].y, xv[c].x, xv[c].y);
        mma_16816(acc[i], wa[c].z, wb[c].z, wa[c].w, wb[c].w, xv[c].z, xv[c].w);
      }
    }
  }
  // (c0, c1) = weight row g, rows 2t, 2t+1 of the 8-row tile; (c2, c3) = weight row g + 8
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) red[warp][8 * i + 2 * t + (q & 1)][g + (q >> 1) * 8] = acc[i][q];
}

__global__ void __launch_bounds__(WARPS * 32) gemv_kernel(const GemvArgs a) {
  __shared__ float red[WARPS][MAX_NT * 8][ROWS + 1];
  __shared__ int found[WARPS], which;
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int e = blockIdx.y;
  if (a.compact) {  // the blockIdx.y-th group with rows (groups <= 256: one per thread)
    const bool has = tid < a.groups && a.offsets[tid + 1] > a.offsets[tid];
    const uint32_t m = __ballot_sync(0xffffffffu, has);
    if (lane == 0) found[warp] = __popc(m);
    if (tid == 0) which = -1;
    __syncthreads();
    int before = __popc(m & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) before += found[w];
    if (has && before == int(blockIdx.y)) which = tid;
    __syncthreads();
    e = which;
    if (e < 0) return;
  }
  // with adapters: one group, the rows up to the end of the last segment
  const int o0 = a.seg_adapter ? 0 : a.offsets[e], o1 = a.seg_adapter ? a.seg_offsets[a.segs] : a.offsets[e + 1];
  if ((o0 < 0 || o1 < o0 || o1 > a.R) && blockIdx.x == 0 && tid == 0) flag_error(a.err, MOE_DEVERR_OFFSETS);
  const int lo = min(max(o0, 0), a.R), cnt = min(o1, a.R) - lo;
  if (cnt <= 0) return;
  const int wi = a.index ? a.index[e] : e;
  const bool none = wi < 0 || wi >= a.n_weights;
  if (none && wi != -1 && blockIdx.x == 0 && tid == 0) flag_error(a.err, MOE_DEVERR_EXPERT_ID);
  const uint16_t *w = a.w + int64_t(none ? 0 : wi) * a.w_stride;
  const float scale = none ? 0.f : a.scale ? a.scale[wi] : 1.f;
  const int n0 = blockIdx.x * ROWS;

  for (int r0 = 0; r0 < cnt; r0 += MAX_NT * 8) {
    const int rows = min(MAX_NT * 8, cnt - r0);
    __syncthreads();
    if (!none) {
      if (rows <= 8) rows_pass<1>(a, w, n0, lo + r0, rows, red);
      else if (rows <= 16) rows_pass<2>(a, w, n0, lo + r0, rows, red);
      else rows_pass<4>(a, w, n0, lo + r0, rows, red);
    }
    __syncthreads();
    for (int p = tid; p < rows * ROWS; p += WARPS * 32) {
      const int r = p / ROWS, n = p % ROWS, row = lo + r0 + r;
      if (n0 + n >= a.N) continue;
      float v = 0.f;
      if (!none) {
#pragma unroll
        for (int q = 0; q < WARPS; ++q) v += red[q][r][n];
        v *= scale;
      }
      if (a.seg_adapter) {
        int s_lo = 0, s_hi = a.segs;  // the first segment that ends behind the row
        while (s_lo < s_hi) {
          const int mid = (s_lo + s_hi) >> 1;
          if (a.seg_offsets[mid + 1] > row) s_hi = mid; else s_lo = mid + 1;
        }
        const int ad = s_lo < a.segs && a.seg_offsets[s_lo] <= row ? a.seg_adapter[s_lo] : -1;
        if (ad >= 0 && ad < a.n_adapters) {
          const uint4 *b = reinterpret_cast<const uint4 *>(a.lora_b + (int64_t(ad) * a.N + n0 + n) * a.rank);
          const uint4 *u = reinterpret_cast<const uint4 *>(a.u + int64_t(row) * a.rank);
          float d = 0.f;
          for (int j = 0; j < a.rank / 8; ++j) {
            const uint4 bv = b[j], uv = u[j];
            d = fmaf(bf16_lo(bv.x), bf16_lo(uv.x), d); d = fmaf(bf16_hi(bv.x), bf16_hi(uv.x), d);
            d = fmaf(bf16_lo(bv.y), bf16_lo(uv.y), d); d = fmaf(bf16_hi(bv.y), bf16_hi(uv.y), d);
            d = fmaf(bf16_lo(bv.z), bf16_lo(uv.z), d); d = fmaf(bf16_hi(bv.z), bf16_hi(uv.z), d);
            d = fmaf(bf16_lo(bv.w), bf16_lo(uv.w), d); d = fmaf(bf16_hi(bv.w), bf16_hi(uv.w), d);
          }
          v += d;
        }
      }
      const int64_t at = int64_t(row) * a.ldo + n0 + n;
      if (a.out_f32) {
        float *o = static_cast<float *>(a.out);
        o[at] = a.accumulate ? o[at] + v : v;
      } else {
        static_cast<uint16_t *>(a.out)[at] = f_to_bf16(v);
      }
    }
  }
}

}  // namespace gv

int launch_gemm_gemv(const GemvArgs &a, int grid_groups, cudaStream_t s, const char *what) {
  const dim3 grid(unsigned((a.N + gv::ROWS - 1) / gv::ROWS), unsigned(grid_groups));
  const cudaError_t e = launch_pdl(gv::gemv_kernel, grid, dim3(gv::WARPS * 32), 0, s, a);
  if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

}  // namespace moe
