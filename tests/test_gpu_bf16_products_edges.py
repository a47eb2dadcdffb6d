"""Edges of the grouped BF16 products and the projection with adapters: calls
close behind one another, long sums, many adapters. Tolerances per element as in
test_gpu_lora: n fp32 additions of products 2^-23 sum|a b|, a BF16 rounding 2^-8
of the value."""
import pytest
import torch

from tests.test_gpu_lora import HALF, SUM, Problem, _rand, _within

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


@pytest.mark.parametrize("lens", [[1 << 20], [1 << 19, 0, (1 << 19) - 3, 3]])
def test_gradients_of_an_adapter_with_a_million_rows(M, lens):
    """All products of one sign, so that what additions cut off adds up. A matrix unit's additions may cut off up to
    2^-23 of the running sum each, and there are at most 256 and a stage's before a sum passes on: 2^-14.9. The sums
    passed on, two for each 4096 rows, are rounded to nearest, 2^-24 each: 2^-15. So before its own rounding, half a
    BF16 step of its binade, a value is within 2^-13.9 of the exact sum. A sum never passed on loses up to 3e-3."""
    N = K = 512
    r, S = 64, len(lens)
    off = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    T = int(off[-1])
    x, dy, u, b = (_rand(s, i).abs_().add_(0.5) for i, s in enumerate(((T, K), (T, N), (T, r), (1, N, r))))
    a, w = _rand((1, r, K), 5), _rand((N, K), 6)
    ad = torch.zeros(S, dtype=torch.int32, device="cuda")
    du, da, db = torch.zeros_like(u), torch.zeros_like(a), torch.zeros_like(b)
    ws = torch.zeros(M.moe_lora_workspace_size(T, S, 1, r, N, K), dtype=torch.uint8, device="cuda")
    M.moe_lora_linear_backward(dy, N, x, K, w, u, off, ad, a, b, None, T, S, 1, r, N, K, du, None, K, da, db, ws, ws.numel())
    assert M.moe_read_device_error(ws) == 0
    ra, rb = torch.zeros(r, K, dtype=torch.float64, device="cuda"), torch.zeros(N, r, dtype=torch.float64, device="cuda")
    for i in range(0, T, 1 << 16):
        s = slice(i, i + (1 << 16))
        ra += (dy[s].double() @ b[0].double()).T @ x[s].double()
        rb += dy[s].double().T @ u[s].double()
    for got, ref in ((da[0], ra), (db[0], rb)):
        _within(got, ref, _half_step(ref) + 2.0 ** -13.9 * ref, "gradient")


def _half_step(ref):
    return torch.ldexp(torch.ones_like(ref), torch.frexp(ref.abs()).exponent - 9)


@pytest.mark.parametrize("direction,counts,N,K", [
    ("wgrad", [1 << 20], 256, 264), ("wgrad", [40_000, 0, 32_769, 100, 32_768, 77], 520, 328),
    ("wgrad", [16_384, 16_385, 0, 16_400], 72, 136),
    ("fwd", [300, 0, 45], 264, 80_008), ("dgrad", [300, 17], 32_776, 264), ("dgrad", [5, 40], 16_392, 1032)])
def test_long_reductions_of_bf16_outputs(M, direction, counts, N, K):
    """All products of one sign, so that what additions cut off adds up. A part of a reduction has at most 256 k-steps,
    1024 additions of 16 products. Each cuts the products and the running sum off at the sum's last place, and as the
    sum grows evenly to its end, loses 1e-7 of that end on average, below 2^-23: 2^-13 a part. Parts are added rounded
    to nearest, 2^-24 each for at most 64 parts: 2^-18. So before its own rounding, half a BF16 step of its binade, a
    value is within 2^-12.9 of the exact sum."""
    E, R = len(counts), sum(counts)
    off_l = [sum(counts[:i]) for i in range(E + 1)]
    off = torch.tensor(off_l, dtype=torch.int32, device="cuda")
    x, dy, w = (_rand(s, i).abs_().add_(0.5) for i, s in enumerate(((R, K), (R, N), (E, N, K))))
    ws = torch.zeros(M.moe_grouped_gemm_workspace_size(R, E, N, K), dtype=torch.uint8, device="cuda")
    out = torch.full({"fwd": (R, N), "dgrad": (R, K), "wgrad": (E, N, K)}[direction], 3.0, dtype=torch.bfloat16, device="cuda")
    def call():
        if direction == "fwd":
            M.moe_grouped_gemm(x, K, off, w, N * K, R, E, N, K, 0, out, N, ws, ws.numel())
        elif direction == "dgrad":
            M.moe_grouped_gemm_dgrad(dy, N, off, w, N * K, R, E, N, K, 0, out, K, ws, ws.numel())
        else:
            M.moe_grouped_gemm_wgrad(dy, N, x, K, off, R, E, N, K, 0, out, N * K, ws, ws.numel())
    call()
    assert M.moe_read_device_error(ws) == 0
    for e in range(E):
        r = slice(off_l[e], off_l[e + 1])
        if direction == "wgrad":
            got, ref = out[e], torch.zeros(N, K, dtype=torch.float64, device="cuda")
            for i in range(off_l[e], off_l[e + 1], 1 << 16):
                s = slice(i, min(i + (1 << 16), off_l[e + 1]))
                ref += dy[s].double().T @ x[s].double()
        else:
            got, ref = out[r], x[r].double() @ w[e].double().T if direction == "fwd" else dy[r].double() @ w[e].double()
        _within(got, ref, _half_step(ref) + 2.0 ** -12.9 * ref, f"{direction} {e}")
    first = out.clone()
    call()
    torch.cuda.synchronize()
    assert torch.equal(first, out)


@pytest.mark.parametrize("N,K", [(136, 40_008), (40_008, 136)])
def test_adapters_beside_a_long_projection(M, N, K):
    # the reduction in parts, with adapters' k-steps behind the last and blocks that segments share
    p = Problem([300, 3, 0, 90, 411], [1, 0, -1, -1, 1], 2, 24, N, K, tail=5, seed=3)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_forward()
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_backward()


@pytest.mark.parametrize("S,n,r,N,K,long", [
    (300, 40, 16, 2056, 2048, 0), (700, 300, 8, 2048, 2056, 500), (2100, 700, 32, 1032, 1040, 90), (1024, 4, 64, 136, 72, 0),
    (40, 1200, 16, 264, 136, 3), (5000, 90, 128, 264, 520, 40), (33_000, 5000, 8, 72, 136, 0)])
def test_many_adapters_and_segments(M, S, n, r, N, K, long):
    """More adapters than a block of the gradients' kernel looks up at a time, in no order, some without a segment, some
    with many; segments of one row, of none and long ones."""
    g = torch.Generator().manual_seed(S + n)
    lens = torch.randint(0, 3, (S,), generator=g)
    lens[torch.randint(0, S, (5,), generator=g)] = long + 1
    ads = torch.randint(-1, n, (S,), generator=g)
    ads[::7] = n - 1
    p = Problem(lens.tolist(), ads.tolist(), n, r, N, K, tail=3, seed=S)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_forward()
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_backward()


def test_adapters_out_of_range_among_many(M):
    # values far outside count as none, at any place of a look
    S, n = 600, 200
    ads = [(7 * i) % n for i in range(S)]
    for i, v in ((3, 2 ** 31 - 1), (64, -2 ** 31), (130, n), (255, -2), (511, n + 592), (599, 2 ** 30)):
        ads[i] = v
    p = Problem([1] * S, ads, n, 8, 2048, 2048, seed=4)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    assert M.moe_read_device_error(ws) == M.MOE_DEVERR_EXPERT_ID
    p.check_forward()
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == M.MOE_DEVERR_EXPERT_ID
    p.check_backward()


@pytest.mark.parametrize("lens,r,N,K", [([40, 0, 33, 9], 8, 264, 200), ([1] * 60, 24, 520, 136), ([300, 211], 32, 136, 520),
                                        ([300, 211], 40, 264, 200), ([90, 5, 200], 64, 1032, 264), ([64] * 9, 96, 264, 136),
                                        ([5000, 17], 128, 264, 200), ([4000, 100, 900], 16, 200, 264)])
def test_inner_gradient_enters_dA_unrounded(M, lens, r, N, K):
    """dA within its own rounding, half a BF16 step of its binade, and what precedes it: du's fp32 sums of N products,
    what its two BF16 values leave of it (half a step of the second: 2^-9 of the first's half step, 2^-8 of du: 2^-17
    and less), and dA's own sums."""
    n = 2
    p = Problem(lens, [i % n for i in range(len(lens))], n, r, N, K, tail=3, seed=r)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_forward()
    p.check_backward()
    rows, ads, sc = p.per_row()
    for q in range(n):
        t = rows[ads == q]
        x, g, b = p.x[t].double(), p.dy[t].double(), p.b[q].double()
        s = float(p.scale[q])
        du, mag = s * (g @ b), abs(s) * (g.abs() @ b.abs())
        ref = du.T @ x
        err = (N + 1) * SUM * mag + 2.0 ** -17 * du.abs()
        before = err.T @ x.abs()
        before = before + len(t) * SUM * (du.abs().T @ x.abs() + before)
        _within(p.da[q], ref, _half_step(ref) + (1 + HALF) * before, f"dA[{q}]")


def test_infinite_inner_gradients_stay_infinite(M):
    # what a rounding to infinity cuts off is not a number: dA is infinite where du is, and its neighbours' is as before
    p = Problem([20, 30], [0, 1], 2, 16, 72, 64, seed=6, with_scale=False)
    p.x.abs_()
    p.dy[3] = 3e38
    p.b[0].abs_()
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    assert torch.isinf(p.du[3]).all() and (p.da[0][:, p.x[3] > 0] == float("inf")).all()
    assert torch.isfinite(p.da[1]).all()


def test_long_sums_on_two_streams_and_from_graphs(M):
    """Calls whose sums pass through their workspaces, at once on two streams and replayed: the bits of one call alone."""
    R, N, K, n, r = 40_000, 264, 520, 70, 64
    off = torch.tensor([0, 20_001, 20_001, R], dtype=torch.int32, device="cuda")
    seg = torch.arange(0, R + 1, 400, dtype=torch.int32, device="cuda")
    S = seg.numel() - 1
    ad = (torch.arange(S, device="cuda") * 7 % n).to(torch.int32)
    a, b, w = _rand((n, r, K), 1, 0.1), _rand((n, N, r), 2, 0.1), _rand((N, K), 3)
    jobs = []
    for i in range(2):
        x, dy, u = _rand((R, K), 10 + i), _rand((R, N), 20 + i), _rand((R, r), 30 + i)
        dw = torch.zeros(3, N, K, dtype=torch.bfloat16, device="cuda")
        du, da, db = torch.zeros_like(u), torch.zeros_like(a), torch.zeros_like(b)
        gws = torch.zeros(M.moe_grouped_gemm_workspace_size(R, 3, N, K), dtype=torch.uint8, device="cuda")
        lws = torch.zeros(M.moe_lora_workspace_size(R, S, n, r, N, K), dtype=torch.uint8, device="cuda")

        def job(stream=None, x=x, dy=dy, u=u, dw=dw, du=du, da=da, db=db, gws=gws, lws=lws):
            M.moe_grouped_gemm_wgrad(dy, N, x, K, off, R, 3, N, K, 0, dw, N * K, gws, gws.numel(), stream)
            M.moe_lora_linear_backward(dy, N, x, K, w, u, seg, ad, a, b, None, R, S, n, r, N, K, du, None, K, da, db, lws,
                                       lws.numel(), stream)
        job()
        torch.cuda.synchronize()
        jobs.append((job, (dw, da, db), [t.clone() for t in (dw, da, db)], (gws, lws), torch.cuda.Stream()))

    def check():
        torch.cuda.synchronize()
        for _, out, ref, spaces, _ in jobs:
            assert all(M.moe_read_device_error(ws) == 0 for ws in spaces)
            assert all(torch.equal(t, q) for t, q in zip(out, ref))
            for t in out:
                t.fill_(3.0)
        torch.cuda.synchronize()

    check()
    for _ in range(3):
        for job, _, _, _, s in jobs:
            job(s)
        check()
    graphs = []
    for job, _, _, _, s in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            job(s)
        graphs.append(g)
    for _ in range(3):
        for g, (_, _, _, _, s) in zip(graphs, jobs):
            with torch.cuda.stream(s):
                g.replay()
        check()
