"""Edges of the grouped BF16 products and the projection with adapters: calls
close behind one another, long sums, many adapters. Tolerances per element as in
test_gpu_lora: n fp32 additions of products 2^-23 sum|a b|, a BF16 rounding 2^-8
of the value."""
import pytest
import torch

from tests.test_gpu_lora import HALF, SUM, _rand, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    import w4a16_mixture_experts_moe_b200 as m
    assert torch.cuda.is_available()
    return m


def test_launches_behind_a_call_whose_last_segment_is_cut_to_nothing(M):
    """The projection of up to eight rows has no rows to do where the last segment ends at row 0, and u's launch is
    long: the next call, which writes what u is made from, still waits for it."""
    T, N, K, r = 8, 8, 131072, 16
    x, w, a, b = _rand((T, K), 1), _rand((N, K), 2), _rand((1, r, K), 3), _rand((1, N, r), 4)
    off, ad = torch.tensor([0, T, 0], dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    u, y = torch.zeros(T, r, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(M.moe_lora_workspace_size(T, 2, 1, r, N, K), dtype=torch.uint8, device="cuda")
    src, wx = _rand((T, 8), 5), _rand((1, K, 8), 6)
    rows, gws = torch.tensor([0, T], dtype=torch.int32, device="cuda"), torch.zeros(256, dtype=torch.uint8, device="cuda")
    xd, ad64 = x.double(), a[0].double()
    ref, mag = xd @ ad64.T, xd.abs() @ ad64.abs().T
    new = src.double() @ wx[0].double().T
    torch.cuda.synchronize()
    M.moe_lora_linear(x, K, w, off, ad, a, b, None, T, 2, 1, r, N, K, u, y, N, ws, ws.numel())
    M.moe_grouped_gemm(src, 8, rows, wx, K * 8, T, 1, K, 8, 0, x, K, gws, 256)
    assert M.moe_read_device_error(ws) == M.MOE_DEVERR_OFFSETS and M.moe_read_device_error(gws) == 0
    _within(u, ref, K * SUM * mag * (1 + HALF) + HALF * ref.abs(), "u")
    _within(x, new, 8 * SUM * (src.double().abs() @ wx[0].double().abs().T) * (1 + HALF) + HALF * new.abs(), "the next call's rows")
    assert (y == 0).all()
