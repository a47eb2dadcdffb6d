// Shared declarations of the BF16 products over ragged row groups (grouped
// products, many-adapter projection): the tensor-core engine of gemm_tc.cu and
// the weight-streaming kernel of gemm_gemv.cu.
#pragma once

#include "common.cuh"
#include "tma.cuh"

namespace moe {

// The largest N and K: column counts are rounded up to tiles in 32 bits.
constexpr int MAX_COLS = 1 << 30;

enum GemmMode { GEMM_FWD = 0, GEMM_DGRAD = 1, GEMM_WGRAD = 2 };

// One product for the tensor-core engine (gemm_tc.cu), passed by value.
struct TcGemmArgs {
  const int32_t *offsets;  // [groups+1] row starts; with adapters: [segs+1] segment starts, one group
  const int32_t *adapter;  // [segs] adapter of each segment (outside [0, n_adapters): none), or nullptr
  int groups, segs, n_adapters, rank;
  int R;       // rows of x / dy
  int M;       // output columns: N (fwd), K (dgrad, wgrad)
  int NC;      // wgrad: rows of one dW (N)
  int KD;      // reduction length: K (fwd), N (dgrad); wgrad reduces over a group's rows
  int bn;      // widest row tile
  int out_f32, accumulate;
  void *out;
  int64_t ldo, out_gstride;  // elements
  const uint16_t *ext_a, *ext_b;  // with adapters: lora_b [n][N][rank] (fwd) or lora_a [n][rank][K], and u / du [R][rank]
  // adapters: fp32 sums for the 16-row blocks that several segments share, from
  // the launch before (lora.cu); row of block b: 16 b, or 16 owner if delta_by_seg
  const float *delta;
  int delta_by_seg;
  const int32_t *row_seg;  // [R] the rows' segments (with delta)
  float *sums;  // what the parts of a long reduction add up in (long_sums_bytes), BF16 outputs
  int late;  // the launches before this one wait for everything but u / du, delta and the output
  int32_t *err;
};

// Operands in global memory (BF16, elements). a: weights [groups][N][K] with
// stride a_gstride (fwd, dgrad) or x [R][K] (wgrad); b: x or dy rows.
struct TcGemmOperands {
  const uint16_t *a, *b;
  int64_t lda, a_gstride, ldb;
};

// The first segment that ends behind `row` (segs if none does).
__device__ __forceinline__ int first_segment(const int32_t *off, int segs, int row) {
  int lo = 0, hi = segs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (off[mid + 1] > row) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Segments and 16-row blocks: block b holds rows 16 b .. 16 b + 15 (cut at the
// last segment's end). Several segments share it if one starts strictly inside;
// the first that does owns the block.

// MOE_OK, or MOE_ERR_UNSUPPORTED where the current device is not sm_100 or the
// driver encodes no tensor maps (also: there is none).
int check_device(const char *what);

// Workspace of the engine's BF16 outputs for reductions of up to `length` products.
size_t long_sums_bytes(int length);

// A BF16 tensor map with the 128-byte swizzle: dimension 0 contiguous, the
// others with strides in elements; out-of-range elements read as zero.
bool map_bf16(CUtensorMap *m, const void *base, int nd, const int64_t (&dim)[4], const int64_t (&stride)[3],
              const int (&box)[4]);

int launch_gemm_tc(GemmMode mode, const TcGemmArgs &a, const TcGemmOperands &op, cudaStream_t s, const char *what);

// Who does a group's passes of GEMV_PASS rows: one grid row per group all of
// them; grid row y the y-th pass of all groups (few rows, many groups); or grid
// rows [0, groups) the groups' first passes and those behind the later ones.
constexpr int GEMV_PASS = 16;
enum GemvSplit { GEMV_WHOLE = 0, GEMV_ALL_PASSES = 1, GEMV_LATER_PASSES = 2 };

// One product for the weight-streaming kernel (gemm_gemv.cu): out[r] = in[r] W^T
// for the rows of each group, W [N][K] at w + index * w_stride.
struct GemvArgs {
  const uint16_t *in;
  int64_t ldi;
  const int32_t *offsets;  // [groups+1]
  const int32_t *index;    // [groups] weight matrix of each group (outside [0, n_weights): none), or nullptr (the group's own)
  const uint16_t *w;
  int64_t w_stride;
  int groups, n_weights, R, N, K;
  int split;               // GEMV_*
  const float *scale;      // [n_weights] factor of each weight matrix, or nullptr
  void *out;
  int64_t ldo;
  int out_f32, accumulate;
  int32_t *row_seg;        // [R] the rows' groups, written (or nullptr)
  int32_t *err;
  // adapters added to a single group's product: out[r] += u[r] B_a^T
  const int32_t *seg_offsets, *seg_adapter;
  int segs, n_adapters, rank;
  const uint16_t *u, *lora_b;
};

int launch_gemm_gemv(GemvArgs a, cudaStream_t s, const char *what);

}  // namespace moe
