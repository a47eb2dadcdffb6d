"""The grouped BF16 products (forward, rows' gradient, weights' gradient)
against the same sums in 64 bits.

Tolerance, per element: an fp32 sum of n exact products taken in any order (and
with truncating additions, as matrix units may do) is within n 2^-23 sum|a b|
of the exact sum; a BF16 output adds one rounding, 2^-8 of the value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def M():
    import w4a16_mixture_experts_moe_b200 as m
    assert torch.cuda.is_available()
    return m


def _rand(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)


def _strided(t, pad):
    """The same values with `pad` further columns of NaN behind each row."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), NAN, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf


def _check(got, ref, mag, n, bf16, what):
    bound = n * 2.0 ** -23 * mag
    if bf16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} elements beyond the bound, first " \
                          f"{bad.nonzero()[0].tolist()}"


def _run(M, direction, counts, N, K, out="bf16", lead=0, tail=0, pad=0, gap=0, accumulate=False, seed=0):
    """One call on rows [lead | groups | tail], whose outer rows hold NaN; strides
    padded by `pad`, weight matrices `gap` elements apart. Checks every output
    element, and that what lies outside the groups keeps its value."""
    E = len(counts)
    off = [lead]
    for c in counts:
        off.append(off[-1] + c)
    R = off[-1] + tail
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, dy = _rand((R, K), seed + 1), _rand((R, N), seed + 2)
    for t in (x, dy):
        t[:lead] = NAN
        t[off[-1]:] = NAN
    w = _rand((E, N * K + gap), seed + 3, 0.05)
    w3 = w[:, :N * K].reshape(E, N, K)
    if gap:
        w[:, N * K:] = NAN
    xs, dys = _strided(x, pad), _strided(dy, pad)
    dt = torch.float32 if out == "f32" else torch.bfloat16
    flags = (M.MOE_GEMM_OUT_F32 if out == "f32" else 0) | (M.MOE_GEMM_ACCUMULATE if accumulate else 0)
    ws = torch.zeros(M.moe_grouped_gemm_workspace_size(R, E, N, K), dtype=torch.uint8, device="cuda")
    if direction == "wgrad":
        o = torch.full((E, N * K + gap), 3.0, dtype=dt, device="cuda")
        before = o.clone()
        M.moe_grouped_gemm_wgrad(dys, N + pad, xs, K + pad, offsets, R, E, N, K, flags, o, N * K + gap, ws, ws.numel())
        torch.cuda.synchronize()
        assert M.moe_read_device_error(ws) == 0
        assert torch.equal(o[:, N * K:], before[:, N * K:])
        for e in range(E):
            a, b = dy[off[e]:off[e + 1]].double(), x[off[e]:off[e + 1]].double()
            ref, mag = a.T @ b, a.T.abs() @ b.abs()
            n = counts[e]
            if accumulate:
                ref, mag, n = ref + 3.0, mag + 3.0, n + 1
            _check(o[e, :N * K].reshape(N, K), ref, mag, n, out == "bf16", f"dW[{e}]")
        return o
    src, width, n = (x, N, K) if direction == "fwd" else (dy, K, N)
    o = torch.full((R, width + pad), 3.0, dtype=dt, device="cuda")
    before = o.clone()
    if direction == "fwd":
        M.moe_grouped_gemm(xs, K + pad, offsets, w, N * K + gap, R, E, N, K, flags, o, width + pad, ws, ws.numel())
    else:
        M.moe_grouped_gemm_dgrad(dys, N + pad, offsets, w, N * K + gap, R, E, N, K, flags, o, width + pad, ws, ws.numel())
    torch.cuda.synchronize()
    assert M.moe_read_device_error(ws) == 0
    assert torch.equal(o[:lead], before[:lead]) and torch.equal(o[off[-1]:], before[off[-1]:])
    assert torch.equal(o[:, width:], before[:, width:])
    for e in range(E):
        if counts[e] == 0:
            continue
        m = w3[e].double().T if direction == "fwd" else w3[e].double()
        a = src[off[e]:off[e + 1]].double()
        ref, mag, nn = a @ m, a.abs() @ m.abs(), n
        if accumulate:
            ref, mag, nn = ref + 3.0, mag + 3.0, n + 1
        _check(o[off[e]:off[e + 1], :width], ref, mag, nn, out == "bf16", f"group {e}")
    return o


SHAPES = [
    # (rows per group, N, K)
    ([1], 8, 8),                                   # the smallest product
    ([1], 128, 64),
    ([5, 0, 1, 2], 136, 72),                       # fewer rows than groups would fill, odd widths
    ([0, 0, 3], 256, 256),
    ([16, 16, 16], 256, 128),
    ([17, 0, 64, 1, 33], 264, 200),                # just above the streaming kernel's group size
    ([255], 512, 192),
    ([256], 256, 64),
    ([257, 1, 0, 300], 520, 328),
    ([100] * 9, 128, 1024),
    ([2100, 3, 700], 384, 136),                    # more than one block of row tiles
    ([63, 64, 65, 127, 128, 129], 1000, 1032),
    ([300, 257, 40, 512, 0, 511, 700, 1030], 1304, 1416),  # tiles of two MMAs beside tiles of one
    ([513] * 3 + [272] * 40, 1024, 1024),
]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_products(M, direction, shape, out):
    counts, N, K = SHAPES[shape]
    _run(M, direction, counts, N, K, out, seed=shape)


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", [[3, 0, 9], [70, 0, 45, 130]])
def test_strides_and_rows_outside_the_groups(M, direction, counts):
    # outer rows and padding hold NaN and are neither read nor written
    for out in ("bf16", "f32"):
        _run(M, direction, counts, 200, 136, out, lead=5, tail=11, pad=24, gap=40, seed=50)


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", [[2, 0, 1], [90, 0, 40]])
def test_accumulate(M, direction, counts):
    _run(M, direction, counts, 144, 96, "f32", accumulate=True, seed=60)


@pytest.mark.parametrize("counts,N", [
    ([32], 64), ([33], 64), ([0, 64], 264), ([0, 65], 264),     # few wide tiles: up to 32 rows a group stream
    ([1, 0, 0, 15], 4096), ([1, 0, 0, 16], 4096),               # 64 of them: up to 4
    ([2] * 64, 2048), ([2] * 63 + [3], 2048), ([1] * 9 + [0] * 54 + [119], 2048)])  # many: up to 2
def test_both_sides_of_the_streaming_rule(M, counts, N):
    _run(M, "fwd", counts, N, 136, seed=70)
    _run(M, "fwd", counts, N, 136, "f32", lead=3, tail=0, seed=71)


def test_no_rows_with_gaps_between_the_gradients(M):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for dt, flags in ((torch.bfloat16, 0), (torch.float32, M.MOE_GEMM_OUT_F32)):
        dw = torch.full((3, 160), 2.0, dtype=dt, device="cuda")
        M.moe_grouped_gemm_wgrad(None, 16, None, 8, off, 0, 3, 16, 8, flags, dw, 160, ws, 256)
        assert (dw[:, :128] == 0).all() and (dw[:, 128:] == 2).all()


@pytest.mark.parametrize("direction,counts,N,K", [
    ("fwd", [40, 300], 256, 14336), ("fwd", [3, 1, 8, 2], 128, 14336), ("fwd", [130], 320, 1088),
    ("dgrad", [40, 300], 14336, 256), ("dgrad", [2, 7, 1, 4], 14336, 128),
    ("wgrad", [16384, 900, 0, 1025], 256, 320)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_error_of_long_reductions(M, direction, counts, N, K, accumulate):
    """The error of an fp32 output as a whole. A matrix unit may cut the running
    sum off at each addition: half a unit of the last place on average, 2^-24 of
    a sum that grows with the root of the number of terms. 64 additions, which
    are 1024 products at 16 each, lose at most 64 2^-24 of the result on average;
    longer reductions are to lose no more."""
    E, R = len(counts), sum(counts)
    off = [sum(counts[:i]) for i in range(E + 1)]
    offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, dy, w = _rand((R, K), 21), _rand((R, N), 22), _rand((E, N, K), 23)
    flags = M.MOE_GEMM_OUT_F32 | (M.MOE_GEMM_ACCUMULATE if accumulate else 0)
    ws = torch.zeros(M.moe_grouped_gemm_workspace_size(R, E, N, K), dtype=torch.uint8, device="cuda")
    shape = {"fwd": (R, N), "dgrad": (R, K), "wgrad": (E, N, K)}[direction]
    o = torch.full(shape, 1.5, device="cuda")
    if direction == "fwd":
        M.moe_grouped_gemm(x, K, offsets, w, N * K, R, E, N, K, flags, o, N, ws, ws.numel())
    elif direction == "dgrad":
        M.moe_grouped_gemm_dgrad(dy, N, offsets, w, N * K, R, E, N, K, flags, o, K, ws, ws.numel())
    else:
        M.moe_grouped_gemm_wgrad(dy, N, x, K, offsets, R, E, N, K, flags, o, N * K, ws, ws.numel())
    torch.cuda.synchronize()
    assert M.moe_read_device_error(ws) == 0
    err = size = 0.0
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if direction == "fwd":
            ref, got = x[r].double() @ w[e].double().T, o[r]
        elif direction == "dgrad":
            ref, got = dy[r].double() @ w[e].double(), o[r]
        else:
            ref, got = dy[r].double().T @ x[r].double(), o[e]
        ref += 1.5 * accumulate
        err += float((got.double() - ref).square().sum())
        size += float(ref.square().sum())
    assert err ** 0.5 <= 64 * 2.0 ** -24 * size ** 0.5


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("E,rows", [(256, 0), (256, 1), (256, 40), (64, 200)])
def test_many_groups(M, direction, E, rows):
    g = torch.Generator().manual_seed(E + rows)
    counts = torch.randint(0, 2 * rows + 1, (E,), generator=g).tolist() if rows else [0] * (E - 1) + [4]
    _run(M, direction, counts, 128, 136, seed=70)


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
def test_other_groups_values_do_not_enter(M, direction):
    """Infinities and NaN in one group's rows stay in that group's results,
    also where its rows share a tile or a reduction step with a neighbour's."""
    counts, N, K, E = [37, 21, 50], 136, 72, 3
    off = torch.tensor([0, 37, 58, 108], dtype=torch.int32, device="cuda")
    x, dy, w = _rand((108, K), 1), _rand((108, N), 2), _rand((E, N, K), 3)
    x[37:58, ::3], dy[37:58, ::5] = float("inf"), NAN
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    res = []
    for clean in (False, True):
        a, b = x.clone(), dy.clone()
        if clean:
            a[37:58], b[37:58] = 0, 0
        if direction == "wgrad":
            o = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
            M.moe_grouped_gemm_wgrad(b, N, a, K, off, 108, E, N, K, 0, o, N * K, ws, 256)
            res.append(o[[0, 2]])
        else:
            width = N if direction == "fwd" else K
            o = torch.empty(108, width, dtype=torch.bfloat16, device="cuda")
            if direction == "fwd":
                M.moe_grouped_gemm(a, K, off, w, N * K, 108, E, N, K, 0, o, N, ws, 256)
            else:
                M.moe_grouped_gemm_dgrad(b, N, off, w, N * K, 108, E, N, K, 0, o, K, ws, 256)
            res.append(torch.cat([o[:37], o[58:]]))
    assert torch.isfinite(res[1]).all() and torch.equal(res[0], res[1])


def test_no_rows(M):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dw = torch.full((3, 16, 8), 2.0, device="cuda")
    M.moe_grouped_gemm(None, 8, off, None, 128, 0, 3, 16, 8, 0, None, 16, ws, 256)
    M.moe_grouped_gemm_wgrad(None, 16, None, 8, off, 0, 3, 16, 8, M.MOE_GEMM_OUT_F32 | M.MOE_GEMM_ACCUMULATE, dw, 128, ws, 256)
    assert (dw == 2).all()
    M.moe_grouped_gemm_wgrad(None, 16, None, 8, off, 0, 3, 16, 8, M.MOE_GEMM_OUT_F32, dw, 128, ws, 256)
    assert (dw == 0).all()


@pytest.mark.parametrize("R,E", [(6, 4), (300, 3)])
def test_bad_offsets_are_cut_and_flagged(M, R, E):
    N, K = 64, 64
    off = torch.tensor(([0, 4, 2, 5, 900] if E == 4 else [-7, 100, 90, 100000]), dtype=torch.int32, device="cuda")
    x, w = _rand((R, K), 1), _rand((E, N, K), 2)
    y = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.moe_grouped_gemm(x, K, off, w, N * K, R, E, N, K, 0, y, N, ws, 256)
    assert M.moe_read_device_error(ws) == M.MOE_DEVERR_OFFSETS
    assert torch.isfinite(y).all()
    assert M.moe_read_device_error(ws) == 0


LO, HI = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("off", [[0, 3, 1, 2, 3], [0, 2, LO, 2, 3], [HI, LO, HI, LO, HI], [1, LO, 3, LO, 2], [2, 2, 2, 2, HI]])
@pytest.mark.parametrize("R", [3, 90, 2000])  # a pass per grid row, later passes, the tensor cores
def test_extreme_offsets(M, off, R):
    E, N, K = 4, 64, 72
    off = torch.tensor([min(o * (R // 3), HI) if 0 < o < HI else o for o in off], dtype=torch.int32, device="cuda")
    x, dy, w = _rand((R, K), 1), _rand((R, N), 3), _rand((E, N, K), 2)
    guard = 64  # rows before and behind what the calls may write
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for flags, dt in ((0, torch.bfloat16), (M.MOE_GEMM_OUT_F32, torch.float32)):
        y = torch.zeros(R + 2 * guard, N, dtype=dt, device="cuda")
        dx = torch.zeros(R + 2 * guard, K, dtype=dt, device="cuda")
        dw = torch.zeros(E + 2, N, K, dtype=dt, device="cuda")
        M.moe_grouped_gemm(x, K, off, w, N * K, R, E, N, K, flags, y[guard:], N, ws, 256)
        assert M.moe_read_device_error(ws) == M.MOE_DEVERR_OFFSETS
        M.moe_grouped_gemm_dgrad(dy, N, off, w, N * K, R, E, N, K, flags, dx[guard:], K, ws, 256)
        assert M.moe_read_device_error(ws) == M.MOE_DEVERR_OFFSETS
        M.moe_grouped_gemm_wgrad(dy, N, x, K, off, R, E, N, K, flags, dw[1:], N * K, ws, 256)
        assert M.moe_read_device_error(ws) == M.MOE_DEVERR_OFFSETS
        for t in (y, dx):
            assert torch.isfinite(t).all() and (t[:guard] == 0).all() and (t[-guard:] == 0).all()
        assert torch.isfinite(dw).all() and (dw[0] == 0).all() and (dw[-1] == 0).all()


@pytest.mark.parametrize("counts", [[200, 0, 1], [1, 0, 100, 0, 0, 17, 16, 33], [0] * 50 + [49] + [0] * 4, [0] * 30 + [64, 1] + [0] * 32])
def test_passes_of_long_groups_beside_short_ones(M, counts):
    N = 8 if len(counts) < 50 else 264  # narrow: such groups stream
    _run(M, "fwd", counts, N, 200, seed=75)
    _run(M, "fwd", counts, N, 200, "f32", accumulate=True, seed=76)


def test_equal_calls_give_equal_bits(M):
    for d in ("fwd", "dgrad", "wgrad"):
        a = _run(M, d, [300, 0, 511, 40], 512, 456, "f32", seed=80)
        b = _run(M, d, [300, 0, 511, 40], 512, 456, "f32", seed=80)
        assert torch.equal(a, b)


def test_gradients_against_differences(M):
    """d(sum(y * dy)) along random directions of x and W against the product's
    own central difference in 64 bits of the formula's inputs."""
    counts, N, K, E = [30, 0, 45], 72, 88, 3
    off_l = [0, 30, 30, 75]
    off = torch.tensor(off_l, dtype=torch.int32, device="cuda")
    R = 75
    x, dy, w = _rand((R, K), 1), _rand((R, N), 2), _rand((E, N, K), 3)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dx = torch.empty(R, K, device="cuda")
    dw = torch.empty(E, N, K, device="cuda")
    M.moe_grouped_gemm_dgrad(dy, N, off, w, N * K, R, E, N, K, M.MOE_GEMM_OUT_F32, dx, K, ws, 256)
    M.moe_grouped_gemm_wgrad(dy, N, x, K, off, R, E, N, K, M.MOE_GEMM_OUT_F32, dw, N * K, ws, 256)

    def loss(xx, ww):
        return sum((xx[off_l[e]:off_l[e + 1]] @ ww[e].T * dy[off_l[e]:off_l[e + 1]].double()).sum() for e in range(E))

    vx, vw = _rand((R, K), 4).double(), _rand((E, N, K), 5).double()
    xd, wd, h = x.double(), w.double(), 2.0 ** -10
    for got, v, num in ((dx, vx, (loss(xd + h * vx, wd) - loss(xd - h * vx, wd)) / (2 * h)),
                        (dw, vw, (loss(xd, wd + h * vw) - loss(xd, wd - h * vw)) / (2 * h))):
        # the loss is linear in each argument: the difference is exact up to 64-bit rounding
        mag = (got.double() * v).abs().sum()
        assert abs((got.double() * v).sum() - num) <= 2.0 ** -23 * 128 * mag + 1e-9 * loss(xd.abs(), wd.abs()).abs()


def test_captured_and_replayed_on_a_side_stream(M):
    counts, N, K, E = [130, 0, 60], 264, 128, 3
    off = torch.tensor([0, 130, 130, 190], dtype=torch.int32, device="cuda")
    R = 190
    x, dy, w = _rand((R, K), 1), _rand((R, N), 2), _rand((E, N, K), 3)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    y, dx = torch.empty(R, N, device="cuda"), torch.empty(R, K, device="cuda")
    dw = torch.empty(E, N, K, device="cuda")

    def step(s):
        f = M.MOE_GEMM_OUT_F32
        M.moe_grouped_gemm(x, K, off, w, N * K, R, E, N, K, f, y, N, ws, 256, s)
        M.moe_grouped_gemm_dgrad(dy, N, off, w, N * K, R, E, N, K, f, dx, K, ws, 256, s)
        M.moe_grouped_gemm_wgrad(dy, N, x, K, off, R, E, N, K, f, dw, N * K, ws, 256, s)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(s)
    x.copy_(_rand((R, K), 11))
    dy.copy_(_rand((R, N), 12))
    torch.cuda.synchronize()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    ref = [t.clone() for t in (y, dx, dw)]
    step(None)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, (y, dx, dw)))


def test_weights_of_a_bf16_bank(M):
    """The gate matrices of Bf16Bank records, in place, and the whole BF16 FFN
    from grouped products against moe_grouped_bf16_ffn's reading of it."""
    from w4a16_mixture_experts_moe_b200.layer import Bf16Bank
    E, H, I, T, k = 8, 256, 384, 96, 2
    gate, up, down = _rand((E, I, H), 1, 0.1), _rand((E, I, H), 2, 0.1), _rand((E, H, I), 3, 0.1)
    bank = Bf16Bank(E, H, I)
    bank.load(gate, up, down)
    x = _rand((T, H), 4)
    ids = torch.stack([torch.randperm(E)[:k] for _ in range(T)]).to(torch.int32).cuda()
    P = T * k
    i32 = dict(dtype=torch.int32, device="cuda")
    counts, off = torch.empty(E, **i32), torch.empty(E + 1, **i32)
    sp, pp = torch.empty(P, **i32), torch.empty(P, **i32)
    gws = torch.zeros(M.moe_group_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    M.moe_group_tokens(ids, T, k, E, counts, off, sp, pp, gws, gws.numel())
    xs = x[(sp // k).long()].contiguous()
    st = bank.rec // 2
    ws = torch.zeros(M.moe_grouped_gemm_workspace_size(P, E, I, H), dtype=torch.uint8, device="cuda")
    g, u = torch.empty(P, I, device="cuda"), torch.empty(P, I, device="cuda")
    y = torch.empty(P, H, device="cuda")
    f = M.MOE_GEMM_OUT_F32
    M.moe_grouped_gemm(xs, H, off, bank.ptr + bank.layout["gate"], st, P, E, I, H, f, g, I, ws, ws.numel())
    M.moe_grouped_gemm(xs, H, off, bank.ptr + bank.layout["up"], st, P, E, I, H, f, u, I, ws, ws.numel())
    h = (torch.nn.functional.silu(g) * u).to(torch.bfloat16)
    M.moe_grouped_gemm(h, I, off, bank.ptr + bank.layout["down"], st, P, E, H, I, f, y, H, ws, ws.numel())
    ref = torch.empty(P, H, device="cuda")
    fws = torch.zeros(M.moe_bf16_ffn_workspace_size(T, k, E, H, I), dtype=torch.uint8, device="cuda")
    M.moe_grouped_bf16_ffn(x, sp, off, bank.ptr, bank.rec, T, k, E, H, I, ref, fws, fws.numel())
    torch.cuda.synchronize()
    # both round h to BF16 from nearly equal fp32 values: at most one BF16 step
    # (2^-7 of |h|) apart, and each sums I products in fp32
    e = torch.repeat_interleave(torch.arange(E, device="cuda"), counts.long())
    mag = torch.einsum("ri,rhi->rh", h.double().abs(), down.double().abs()[e])
    assert ((y - ref).abs().double() <= (2.0 ** -7 + I * 2.0 ** -22) * mag).all()


def test_training_step_of_a_moe_layer(M):
    """The operators as a training step of one MoE layer uses them, behind a
    projection with adapters: every stage against 64 bits on that stage's own
    inputs, forward and backward."""
    from tests.test_gpu_lora import Problem
    E, H, I, k = 8, 256, 192, 2
    p = Problem([70, 0, 41, 52], [1, 0, -1, 0], 2, 16, H, 264, seed=40)
    p.strided()
    T = p.T
    lws = p.workspace(M)
    p.forward(M, lws)                                               # x = projection(tokens), adapters per request
    p.check_forward()
    x = p.y
    wr = _rand((E, H), 41, 0.1)
    up, down = _rand((E, I, H), 42, 0.1), _rand((E, H, I), 43, 0.1)
    i32 = dict(dtype=torch.int32, device="cuda")
    logits = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    ids, tw = torch.empty(T, k, **i32), torch.empty(T, k, device="cuda")
    M.moe_route_topk(x, wr, T, H, E, k, None, M.MOE_RENORM, logits, ids, tw)
    P = T * k
    counts, off, sp, pp = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(P, **i32), torch.empty(P, **i32)
    gws = torch.zeros(M.moe_group_workspace_size(T, k, E), dtype=torch.uint8, device="cuda")
    M.moe_group_tokens(ids, T, k, E, counts, off, sp, pp, gws, gws.numel())
    tok = (sp // k).long()
    xs = x[tok].contiguous()
    ws = torch.zeros(M.moe_grouped_gemm_workspace_size(P, E, I, H), dtype=torch.uint8, device="cuda")
    f = M.MOE_GEMM_OUT_F32
    a = torch.empty(P, I, device="cuda")
    M.moe_grouped_gemm(xs, H, off, up, I * H, P, E, I, H, f, a, I, ws, ws.numel())
    h = torch.relu(a).to(torch.bfloat16)
    y = torch.empty(P, H, device="cuda")
    M.moe_grouped_gemm(h, I, off, down, H * I, P, E, H, I, f, y, H, ws, ws.numel())
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    M.moe_combine(y, tw, pp, x, T, k, H, out)

    dout = _rand((T, H), 44)
    dys = (dout.float()[tok] * tw.flatten()[sp.long()][:, None]).to(torch.bfloat16)
    d_down, d_up = torch.empty(E, H, I, device="cuda"), torch.zeros(E, I, H, device="cuda")
    dh, dxs = torch.empty(P, I, device="cuda"), torch.empty(P, H, device="cuda")
    M.moe_grouped_gemm_wgrad(dys, H, h, I, off, P, E, H, I, f, d_down, H * I, ws, ws.numel())
    M.moe_grouped_gemm_dgrad(dys, H, off, down, H * I, P, E, H, I, f, dh, I, ws, ws.numel())
    da = (dh * (a > 0)).to(torch.bfloat16)
    M.moe_grouped_gemm_wgrad(da, I, xs, H, off, P, E, I, H, f | M.MOE_GEMM_ACCUMULATE, d_up, I * H, ws, ws.numel())
    M.moe_grouped_gemm_dgrad(da, I, off, up, I * H, P, E, I, H, f, dxs, H, ws, ws.numel())
    ones = torch.ones(T, k, device="cuda")
    p.dy = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")   # a token's experts summed, and the residual
    M.moe_combine(dxs, ones, pp, dout, T, k, H, p.dy)
    p.strided()
    p.backward(M, lws)
    torch.cuda.synchronize()
    p.check_backward()
    assert M.moe_read_device_error(ws) == 0 and M.moe_read_device_error(lws) == 0

    o = off.tolist()
    assert o[-1] == P
    for e in range(E):
        r = slice(o[e], o[e + 1])
        n = o[e + 1] - o[e]
        for got, l, m, terms, what in ((a[r], xs[r], up[e].T, H, "a"), (y[r], h[r], down[e].T, I, "y"),
                                       (dh[r], dys[r], down[e], H, "dh"), (dxs[r], da[r], up[e], I, "dxs"),
                                       (d_down[e], dys[r].T, h[r], n, "d_down"), (d_up[e], da[r].T, xs[r], n + 1, "d_up")):
            l, m = l.double(), m.double()
            _check(got, l @ m, l.abs() @ m.abs(), terms, False, f"{what}[{e}]")
    ref = x.double()
    mag = ref.abs()
    for j in range(k):
        v = y.double()[pp.view(T, k)[:, j].long()] * tw.double()[:, j:j + 1]
        ref, mag = ref + v, mag + v.abs()
    _check(out, ref, mag, k + 1, True, "out")
