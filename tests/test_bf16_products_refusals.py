"""Argument checks of the grouped BF16 products and the projection with
adapters: every refusal comes before any CUDA call, so this runs on the CPU.
The addresses are made up (aligned, never dereferenced)."""
import pytest

P = 0x10000  # 256-byte aligned
BIG = 1 << 40


@pytest.fixture(scope="module")
def N():
    from w4a16_mixture_experts_moe_b200 import build
    build.build()
    from w4a16_mixture_experts_moe_b200 import _native
    return _native


def _fwd(N, x=P, ldx=64, off=P, w=P, ws_=64 * 32, R=4, E=2, n=32, k=64, flags=0, y=P, ldy=32, ws=P, size=BIG):
    return N.lib.moe_grouped_gemm(x, ldx, off, w, ws_, R, E, n, k, flags, y, ldy, ws, size, None)


def _dgrad(N, dy=P, lddy=32, off=P, w=P, ws_=64 * 32, R=4, E=2, n=32, k=64, flags=0, dx=P, lddx=64, ws=P, size=BIG):
    return N.lib.moe_grouped_gemm_dgrad(dy, lddy, off, w, ws_, R, E, n, k, flags, dx, lddx, ws, size, None)


def _wgrad(N, dy=P, lddy=32, x=P, ldx=64, off=P, R=4, E=2, n=32, k=64, flags=0, dw=P, dws=64 * 32, ws=P, size=BIG):
    return N.lib.moe_grouped_gemm_wgrad(dy, lddy, x, ldx, off, R, E, n, k, flags, dw, dws, ws, size, None)


def _lora(N, x=P, ldx=64, w=P, so=P, sa=P, a=P, b=P, scale=None, T=4, S=2, n=3, r=16, no=32, k=64, u=P, y=P, ldy=32,
          ws=P, size=BIG):
    return N.lib.moe_lora_linear(x, ldx, w, so, sa, a, b, scale, T, S, n, r, no, k, u, y, ldy, ws, size, None)


def _lora_bwd(N, dy=P, lddy=32, x=P, ldx=64, w=P, u=P, so=P, sa=P, a=P, b=P, scale=None, T=4, S=2, n=3, r=16, no=32,
              k=64, du=P, dx=P, lddx=64, da=P, db=P, ws=P, size=BIG):
    return N.lib.moe_lora_linear_backward(dy, lddy, x, ldx, w, u, so, sa, a, b, scale, T, S, n, r, no, k, du, dx, lddx,
                                          da, db, ws, size, None)


@pytest.mark.parametrize("call", [_fwd, _dgrad, _wgrad])
@pytest.mark.parametrize("bad", [dict(R=-1), dict(R=(1 << 30) + 1), dict(E=0), dict(E=257), dict(n=0), dict(n=36),
                                 dict(k=4), dict(k=-8), dict(k=100)])
def test_grouped_shapes(N, call, bad):
    assert call(N, **bad) == N.MOE_ERR_SHAPE
    assert call.__name__[1:] in ("fwd", "dgrad", "wgrad") and b"moe_grouped_gemm" in N.lib.moe_last_error()


@pytest.mark.parametrize("call", [_fwd, _dgrad, _wgrad])
@pytest.mark.parametrize("bad", [dict(flags=4), dict(flags=2), dict(off=None), dict(ws=None), dict(ws=P + 128), dict(size=8)])
def test_grouped_arguments(N, call, bad):
    assert call(N, **bad) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=P + 8), dict(w=None), dict(w=P + 2), dict(y=None), dict(y=P + 4),
                                 dict(ldx=56), dict(ldx=68), dict(ldy=24), dict(ldy=33), dict(ws_=64 * 32 - 8),
                                 dict(ws_=64 * 32 + 4)])
def test_forward_matrices(N, bad):
    assert _fwd(N, **bad) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(dy=None), dict(dy=P + 8), dict(w=P + 8), dict(dx=None), dict(lddy=24), dict(lddx=60),
                                 dict(ws_=8)])
def test_dgrad_matrices(N, bad):
    assert _dgrad(N, **bad) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(dy=None), dict(x=None), dict(x=P + 8), dict(dw=None), dict(dw=P + 8), dict(lddy=24),
                                 dict(ldx=60), dict(dws=8), dict(dws=64 * 32 + 1)])
def test_wgrad_matrices(N, bad):
    assert _wgrad(N, **bad) == N.MOE_ERR_INVALID_ARG


def test_no_rows_is_a_no_op(N):
    assert _fwd(N, x=None, w=None, y=None, R=0) == N.MOE_OK
    assert _dgrad(N, dy=None, w=None, dx=None, R=0) == N.MOE_OK
    assert _wgrad(N, dy=None, x=None, R=0, flags=N.MOE_GEMM_OUT_F32 | N.MOE_GEMM_ACCUMULATE) == N.MOE_OK
    assert _wgrad(N, R=0, dw=None) == N.MOE_ERR_INVALID_ARG  # the zero gradient needs a place
    assert _lora(N, x=None, u=None, y=None, T=0) == N.MOE_OK
    assert _lora(N, x=None, sa=None, u=None, y=None, S=0) == N.MOE_OK
    assert _lora_bwd(N, dy=None, x=None, u=None, du=None, dx=None, da=None, db=None, T=0) == N.MOE_OK


@pytest.mark.parametrize("call", [_lora, _lora_bwd])
@pytest.mark.parametrize("bad", [dict(T=-1), dict(S=-1), dict(S=65536), dict(n=0), dict(n=65536), dict(r=0), dict(r=12),
                                 dict(r=136), dict(no=20), dict(k=0), dict(k=90)])
def test_adapter_shapes(N, call, bad):
    assert call(N, **bad) == N.MOE_ERR_SHAPE


@pytest.mark.parametrize("call", [_lora, _lora_bwd])
@pytest.mark.parametrize("bad", [dict(w=None), dict(w=P + 8), dict(so=None), dict(sa=None), dict(a=None), dict(a=P + 4),
                                 dict(b=None), dict(b=P + 2), dict(ws=None), dict(ws=P + 16), dict(size=16)])
def test_adapter_arguments(N, call, bad):
    assert call(N, **bad) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=P + 8), dict(ldx=56), dict(ldx=65), dict(y=None), dict(ldy=24),
                                 dict(u=None), dict(u=P + 8)])
def test_adapter_forward_rows(N, bad):
    assert _lora(N, **bad) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", [dict(dy=None), dict(lddy=24), dict(du=None), dict(dx=P + 8), dict(lddx=56), dict(x=None),
                                 dict(ldx=60), dict(u=None), dict(da=None), dict(db=None), dict(da=P + 4)])
def test_adapter_backward_rows(N, bad):
    assert _lora_bwd(N, **bad) == N.MOE_ERR_INVALID_ARG


def test_workspace_sizes(N):
    assert N.moe_grouped_gemm_workspace_size(0, 1, 8, 8) >= 256
    base = N.moe_lora_workspace_size(8192, 1, 4, 16, 4096, 2048)
    # fp32 rows for the 16-row blocks that segments share: 16 per segment, at most one per row; the rows' segments
    assert N.moe_lora_workspace_size(8192, 13, 4, 16, 4096, 2048) == base + 13 * 16 * 4096 * 4 + 8192 * 4
    assert N.moe_lora_workspace_size(40, 40, 4, 16, 2048, 4096) == base + 48 * 4096 * 4 + 40 * 4


def test_names_are_public(N):
    import w4a16_mixture_experts_moe_b200 as moe
    for name in ("moe_grouped_gemm", "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad", "moe_lora_linear",
                 "moe_lora_linear_backward", "moe_grouped_gemm_workspace_size", "moe_lora_workspace_size"):
        assert getattr(moe, name) is getattr(N, name)
    assert (moe.MOE_GEMM_OUT_F32, moe.MOE_GEMM_ACCUMULATE, moe.MOE_DEVERR_OFFSETS) == (1, 2, 5)


def test_host_tensors_are_refused(N):
    """A tensor outside the current device is refused by the binding, before the
    library sees its address."""
    import torch
    t = torch.zeros(64, 64, dtype=torch.bfloat16)
    with pytest.raises(N.MoeError) as ei:
        N.moe_grouped_gemm(t, 64, P, P, 64 * 32, 4, 2, 32, 64, 0, P, 32, P, BIG, 0)
    assert ei.value.status == N.MOE_ERR_INVALID_ARG and "current device" in str(ei.value)
    with pytest.raises(N.MoeError):
        N.moe_lora_linear(P, 64, P, t, P, P, P, None, 4, 2, 3, 16, 32, 64, P, P, 32, P, BIG, 0)


def test_too_many_tiles_are_refused(N):
    # 2^30 rows by 2^24 columns: more tiles than the engine counts (refused before or for want of a GPU)
    st = _fwd(N, R=1 << 30, E=1, n=1 << 24, ldy=1 << 24, ws_=(1 << 24) * 64)
    assert st in (N.MOE_ERR_SHAPE, N.MOE_ERR_UNSUPPORTED)
