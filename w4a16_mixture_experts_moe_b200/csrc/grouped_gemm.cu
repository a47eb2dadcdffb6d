// Entry points of the grouped BF16 products: argument checks and the choice
// between the weight-streaming kernel (decode-sized groups, forward) and the
// tensor-core engine.
#include "gemm.cuh"

namespace moe {

// Whether the forward product streams the weights (gemm_gemv.cu) or takes the
// tensor-core engine. Streaming reads a group's weights once per 16 rows but
// spreads them over all SMs whatever their number; the engine reads them once
// and gives 256 columns of a group to a pair of SMs. So the rows per group up to
// which streaming is faster fall with the number of the engine's tiles, from
// 32 at a few (8 groups of 16, N = 512, K = 2048: 7.1 against 13.2 us) over 8
// (2 groups of 8, N = K = 4096: 12.9 against 20.0) to 2 at several per pair (64
// groups of 2, N = 2048, K = 1024: 45.5 against 49.6; groups of 12: 67 against
// 50). Rows that are few on average but not in every group cost streaming more
// than the engine, too (64 groups, 256 skewed rows: 41 against 38 us).
static bool use_gemv(int R, int E, int N) {
  const int64_t tiles = int64_t(E) * ((N + 255) / 256), most = 4 * 74 / tiles;
  return int64_t(R) <= int64_t(E) * (most < 2 ? 2 : most > 32 ? 32 : most);
}

// `reduction`: the length of the direction's sums.
static int check_grouped(const char *who, int R, int E, int N, int K, int reduction, int flags, const void *offsets,
                         const void *ws, size_t ws_bytes) {
  if (R < 0 || R > (1 << 30) || E < 1 || E > MAX_E)
    return set_error(MOE_ERR_SHAPE, "%s: R=%d E=%d (need 0<=R<=2^30, 1<=E<=256)", who, R, E);
  if (N < 8 || K < 8 || N % 8 || K % 8 || N > MAX_COLS || K > MAX_COLS)
    return set_error(MOE_ERR_SHAPE, "%s: N=%d K=%d must be multiples of 8 from 8 to 2^30", who, N, K);
  if (flags & ~(MOE_GEMM_OUT_F32 | MOE_GEMM_ACCUMULATE))
    return set_error(MOE_ERR_INVALID_ARG, "%s: unknown flag bits 0x%x", who, flags);
  if ((flags & MOE_GEMM_ACCUMULATE) && !(flags & MOE_GEMM_OUT_F32))
    return set_error(MOE_ERR_INVALID_ARG, "%s: MOE_GEMM_ACCUMULATE needs MOE_GEMM_OUT_F32", who);
  if (!offsets || !ws) return set_error(MOE_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned(ws, 256)) return set_error(MOE_ERR_INVALID_ARG, "%s: ws needs 256-byte alignment", who);
  const size_t need = WS_HEADER + ((flags & MOE_GEMM_OUT_F32) ? 0 : long_sums_bytes(reduction));
  if (ws_bytes < need) return set_error(MOE_ERR_INVALID_ARG, "%s: workspace %zu B < %zu B", who, ws_bytes, need);
  return MOE_OK;
}

// A matrix whose rows (or group blocks) lie `stride` elements apart.
static int check_matrix(const char *who, const char *name, const void *p, int64_t stride, int64_t least) {
  if (!p || !aligned(p, 16))
    return set_error(MOE_ERR_INVALID_ARG, "%s: %s must be a 16-byte aligned device pointer", who, name);
  if (stride < least || stride % 8)
    return set_error(MOE_ERR_INVALID_ARG, "%s: stride of %s (%lld) must be a multiple of 8 and at least %lld", who, name,
                     (long long)stride, (long long)least);
  return MOE_OK;
}

static TcGemmArgs grouped_args(const int32_t *offsets, int R, int E, int flags, void *out, int64_t ldo, void *ws) {
  TcGemmArgs a = {};
  a.offsets = offsets;
  a.groups = E;
  a.R = R;
  a.bn = 256;
  a.out_f32 = (flags & MOE_GEMM_OUT_F32) != 0;
  a.accumulate = (flags & MOE_GEMM_ACCUMULATE) != 0;
  a.out = out;
  a.ldo = ldo;
  a.err = static_cast<int32_t *>(ws);
  a.sums = reinterpret_cast<float *>(static_cast<char *>(ws) + WS_HEADER);  // there if a reduction is long
  return a;
}

}  // namespace moe

extern "C" size_t moe_grouped_gemm_workspace_size(int R, int E, int N, int K) {
  (void)E;
  const int most = R > N ? R : N;  // the longest reduction of the three directions
  return moe::WS_HEADER + moe::long_sums_bytes(most > K ? most : K);
}

extern "C" int moe_grouped_gemm(const moe_bf16 *x, int64_t ldx, const int32_t *offsets, const moe_bf16 *w,
                                int64_t w_stride, int R, int E, int N, int K, int flags, void *y, int64_t ldy, void *ws,
                                size_t ws_bytes, moe_stream_t stream) {
  moe::NvtxScope nvtx_scope("moe_grouped_gemm");
  using namespace moe;
  const char *who = "moe_grouped_gemm";
  int st = check_grouped(who, R, E, N, K, K, flags, offsets, ws, ws_bytes);
  if (st != MOE_OK || R == 0) return st;
  if ((st = check_matrix(who, "x", x, ldx, K)) != MOE_OK || (st = check_matrix(who, "y", y, ldy, N)) != MOE_OK ||
      (st = check_matrix(who, "w", w, w_stride, int64_t(N) * K)) != MOE_OK)
    return st;
  cudaStream_t s = as_stream(stream);
  if (use_gemv(R, E, N)) {
    GemvArgs v = {};
    v.in = x; v.ldi = ldx; v.offsets = offsets; v.w = w; v.w_stride = w_stride;
    v.groups = E; v.n_weights = E; v.R = R; v.N = N; v.K = K;
    v.split = R < E ? GEMV_ALL_PASSES : GEMV_LATER_PASSES;
    v.out = y; v.ldo = ldy;
    v.out_f32 = (flags & MOE_GEMM_OUT_F32) != 0;
    v.accumulate = (flags & MOE_GEMM_ACCUMULATE) != 0;
    v.err = static_cast<int32_t *>(ws);
    return launch_gemm_gemv(v, s, who);
  }
  TcGemmArgs a = grouped_args(offsets, R, E, flags, y, ldy, ws);
  a.M = N;
  a.KD = K;
  return launch_gemm_tc(GEMM_FWD, a, TcGemmOperands{w, x, K, w_stride, ldx}, s, who);
}

extern "C" int moe_grouped_gemm_dgrad(const moe_bf16 *dy, int64_t lddy, const int32_t *offsets, const moe_bf16 *w,
                                      int64_t w_stride, int R, int E, int N, int K, int flags, void *dx, int64_t lddx,
                                      void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe::NvtxScope nvtx_scope("moe_grouped_gemm_dgrad");
  using namespace moe;
  const char *who = "moe_grouped_gemm_dgrad";
  int st = check_grouped(who, R, E, N, K, N, flags, offsets, ws, ws_bytes);
  if (st != MOE_OK || R == 0) return st;
  if ((st = check_matrix(who, "dy", dy, lddy, N)) != MOE_OK || (st = check_matrix(who, "dx", dx, lddx, K)) != MOE_OK ||
      (st = check_matrix(who, "w", w, w_stride, int64_t(N) * K)) != MOE_OK)
    return st;
  TcGemmArgs a = grouped_args(offsets, R, E, flags, dx, lddx, ws);
  a.M = K;
  a.KD = N;
  return launch_gemm_tc(GEMM_DGRAD, a, TcGemmOperands{w, dy, K, w_stride, lddy}, as_stream(stream), who);
}

extern "C" int moe_grouped_gemm_wgrad(const moe_bf16 *dy, int64_t lddy, const moe_bf16 *x, int64_t ldx,
                                      const int32_t *offsets, int R, int E, int N, int K, int flags, void *dw,
                                      int64_t dw_stride, void *ws, size_t ws_bytes, moe_stream_t stream) {
  moe::NvtxScope nvtx_scope("moe_grouped_gemm_wgrad");
  using namespace moe;
  const char *who = "moe_grouped_gemm_wgrad";
  int st = check_grouped(who, R, E, N, K, R, flags, offsets, ws, ws_bytes);
  if (st != MOE_OK) return st;
  if ((st = check_matrix(who, "dw", dw, dw_stride, int64_t(N) * K)) != MOE_OK) return st;
  cudaStream_t s = as_stream(stream);
  if (R == 0) {  // no rows: zero gradients (nothing to add when accumulating)
    const size_t el = (flags & MOE_GEMM_OUT_F32) ? 4 : 2, bytes = size_t(N) * K * el;
    const bool whole = dw_stride == int64_t(N) * K;
    cudaError_t e = cudaSuccess;
    if (!(flags & MOE_GEMM_ACCUMULATE))
      for (int g = 0; g < (whole ? 1 : E) && e == cudaSuccess; ++g)
        e = cudaMemsetAsync(static_cast<uint8_t *>(dw) + size_t(g) * dw_stride * el, 0, whole ? bytes * E : bytes, s);
    return e == cudaSuccess ? MOE_OK : set_error(MOE_ERR_CUDA, "%s: %s", who, cudaGetErrorString(e));
  }
  if ((st = check_matrix(who, "dy", dy, lddy, N)) != MOE_OK || (st = check_matrix(who, "x", x, ldx, K)) != MOE_OK)
    return st;
  TcGemmArgs a = grouped_args(offsets, R, E, flags, dw, K, ws);
  a.M = K;
  a.NC = N;
  a.out_gstride = dw_stride;
  return launch_gemm_tc(GEMM_WGRAD, a, TcGemmOperands{x, dy, ldx, 0, lddy}, s, who);
}
