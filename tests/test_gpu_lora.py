"""The shared projection with per-request low-rank adapters, forward and
backward, against its formulas in 64 bits.

Tolerances per element. fp32 sums of n exact products: n 2^-23 sum|a b|. The
inner values u and du are rounded to BF16 once (2^-8 of the value), which moves
what they enter by at most 2^-8 sum|u b|. Outputs are BF16: 2^-8 of the value.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

NAN = float("nan")
HALF = 2.0 ** -8    # half a BF16 step
SUM = 2.0 ** -23    # one fp32 addition, truncating


@pytest.fixture(scope="module")
def M():
    import w4a16_mixture_experts_moe_b200 as m
    assert torch.cuda.is_available()
    return m


def _rand(shape, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").mul_(std).to(torch.bfloat16)


def _within(got, ref, bound, what):
    bad = ~((got.double() - ref).abs() <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, first {bad.nonzero()[0].tolist()}"


class Problem:
    def __init__(self, lens, adapters, n, r, N, K, tail=0, pad=0, seed=0, with_scale=True):
        self.n, self.r, self.N, self.K, self.S, self.pad = n, r, N, K, len(lens), pad
        off = [0]
        for c in lens:
            off.append(off[-1] + c)
        self.off, self.ad = off, adapters
        self.T, self.end = off[-1] + tail, off[-1]
        self.x, self.dy = _rand((self.T, K), seed + 1), _rand((self.T, N), seed + 2)
        self.x[self.end:], self.dy[self.end:] = NAN, NAN
        self.w = _rand((N, K), seed + 3, 0.05)
        self.a, self.b = _rand((n, r, K), seed + 4, K ** -0.5), _rand((n, N, r), seed + 5, 0.1)
        g = torch.Generator().manual_seed(seed + 6)
        self.scale = (torch.rand(n, generator=g) * 3 - 1).cuda() if with_scale else None
        self.seg_off = torch.tensor(off, dtype=torch.int32, device="cuda")
        self.seg_ad = torch.tensor(adapters, dtype=torch.int32, device="cuda")
        self.u = torch.full((self.T, r), 3.0, dtype=torch.bfloat16, device="cuda")
        self.y = torch.full((self.T, N + pad), 3.0, dtype=torch.bfloat16, device="cuda")
        self.du = torch.full((self.T, r), 3.0, dtype=torch.bfloat16, device="cuda")
        self.dx = torch.full((self.T, K + pad), 3.0, dtype=torch.bfloat16, device="cuda")
        self.da, self.db = torch.full_like(self.a, 3.0), torch.full_like(self.b, 3.0)

    def wide(self, t):
        buf = torch.full((t.shape[0], t.shape[1] + self.pad), NAN, dtype=t.dtype, device=t.device)
        buf[:, :t.shape[1]] = t
        return buf

    def workspace(self, M):
        return torch.zeros(M.moe_lora_workspace_size(self.T, self.S, self.n, self.r, self.N, self.K),
                           dtype=torch.uint8, device="cuda")

    def forward(self, M, ws, stream=None):
        M.moe_lora_linear(self.xs, self.K + self.pad, self.w, self.seg_off, self.seg_ad, self.a, self.b, self.scale,
                          self.T, self.S, self.n, self.r, self.N, self.K, self.u, self.y, self.N + self.pad, ws,
                          ws.numel(), stream)

    def backward(self, M, ws, stream=None):
        M.moe_lora_linear_backward(self.dys, self.N + self.pad, self.xs, self.K + self.pad, self.w, self.u, self.seg_off,
                                   self.seg_ad, self.a, self.b, self.scale, self.T, self.S, self.n, self.r, self.N,
                                   self.K, self.du, self.dx, self.K + self.pad, self.da, self.db, ws, ws.numel(), stream)

    def strided(self):
        self.xs, self.dys = self.wide(self.x), self.wide(self.dy)

    def per_row(self):
        """(rows with an adapter, their adapter, its scale)."""
        rows, ads = [], []
        for s in range(self.S):
            if 0 <= self.ad[s] < self.n:
                rows += range(self.off[s], self.off[s + 1])
                ads += [self.ad[s]] * (self.off[s + 1] - self.off[s])
        rows, ads = torch.tensor(rows, dtype=torch.long, device="cuda"), torch.tensor(ads, dtype=torch.long, device="cuda")
        sc = self.scale.double()[ads] if self.scale is not None else torch.ones(len(ads), dtype=torch.float64, device="cuda")
        return rows, ads, sc[:, None]

    def _product(self, rows, ads, src, mats):
        """src[row] @ mats[adapter].T and the sum of magnitudes, adapter by adapter."""
        out = torch.zeros(len(rows), mats.shape[1], dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(out)
        for q in range(self.n):
            m = ads == q
            if m.any():
                v, t = src[rows[m]].double(), mats[q].double()
                out[m], mag[m] = v @ t.T, v.abs() @ t.abs().T
        return out, mag

    def check_forward(self):
        rows, ads, sc = self.per_row()
        e, K, r = self.end, self.K, self.r
        x, w = self.x[:e].double(), self.w.double()
        y, ymag = x @ w.T, x.abs() @ w.abs().T
        u, ub = torch.zeros(e, r, dtype=torch.float64, device="cuda"), torch.zeros(e, r, dtype=torch.float64, device="cuda")
        if len(rows):
            p, mag = self._product(rows, ads, self.x, self.a)
            u[rows] = p * sc
            ub[rows] = (K + 1) * SUM * (mag * sc.abs())
        err_u = ub * (1 + HALF) + HALF * u.abs()
        _within(self.u[:e], u, err_u, "u")
        bound = torch.zeros_like(y)
        if len(rows):
            full_u = torch.zeros(self.T, r, dtype=torch.float64, device="cuda")
            full_u[:e] = u
            d, dmag = self._product(rows, ads, full_u, self.b)
            y[rows] += d
            ymag[rows] += dmag
            full_u[:e] = err_u
            bound[rows] = self._product(rows, ads, full_u, self.b.abs())[0]
        bound = bound + (K + r) * SUM * (ymag + bound)
        _within(self.y[:e, :self.N], y, bound * (1 + HALF) + HALF * y.abs(), "y")
        assert (self.y[e:] == 3).all() and (self.y[:, self.N:] == 3).all() and (self.u[e:] == 3).all()

    def check_backward(self):
        rows, ads, sc = self.per_row()
        e, N, K, r = self.end, self.N, self.K, self.r
        dy, w = self.dy[:e].double(), self.w.double()
        dx, mag0 = dy @ w, dy.abs() @ w.abs()
        bound = torch.zeros_like(dx)
        du = torch.zeros(self.T, r, dtype=torch.float64, device="cuda")
        err = torch.zeros_like(du)
        if len(rows):
            p, mag = self._product(rows, ads, self.dy, self.b.transpose(1, 2))
            du[rows] = p * sc
            err[rows] = (N + 1) * SUM * mag * sc.abs() * (1 + HALF) + HALF * du[rows].abs()
            d, dmag = self._product(rows, ads, du, self.a.transpose(1, 2))
            dx[rows] += d
            mag0[rows] += dmag
            bound[rows] = self._product(rows, ads, err, self.a.transpose(1, 2).abs())[0]
        bound = bound + (N + r) * SUM * (mag0 + bound)
        _within(self.dx[:e, :K], dx, bound * (1 + HALF) + HALF * dx.abs(), "dx")
        assert (self.dx[e:] == 3).all() and (self.dx[:, K:] == 3).all()
        for q in range(self.n):
            t = rows[ads == q]
            n = len(t)
            x, g, uu = self.x[t].double(), self.dy[t].double(), self.u[t].double()
            da, db = du[t].T @ x, g.T @ uu
            ea = err[t].T @ x.abs()
            ea = ea + n * SUM * (du[t].abs().T @ x.abs() + ea)
            _within(self.da[q], da, ea * (1 + HALF) + HALF * da.abs(), f"dA[{q}]")
            _within(self.db[q], db, n * SUM * (g.abs().T @ uu.abs()) * (1 + HALF) + HALF * db.abs(), f"dB[{q}]")


CASES = [
    # (segment lengths, adapters, n, rank, N, K, tail rows)
    ([1], [0], 1, 8, 8, 8, 0),
    ([1], [0], 4, 16, 256, 512, 0),
    ([1], [-1], 2, 16, 64, 64, 0),                                # no adapter at all
    ([1] * 7, [2, 0, -1, 2, 1, 1, 0], 3, 16, 136, 200, 2),        # a decode batch, padded
    ([1] * 32, list(range(16)) * 2, 16, 24, 264, 328, 0),
    ([1] * 33, [i % 5 - 1 for i in range(33)], 4, 64, 512, 256, 0),
    ([1] * 127, [i % 9 - 1 for i in range(127)], 9, 16, 520, 136, 3),
    ([1] * 130, [i % 9 - 1 for i in range(130)], 9, 128, 520, 136, 3),
    ([60, 7, 61], [2, 0, 1], 3, 48, 2056, 1032, 0),               # the decode form's largest batch, split reductions
    ([5] * 3, [1, -1, 1], 2, 8, 2048, 2048, 0),
    ([2500, 1700], [0, 1], 2, 16, 136, 264, 0),                   # the wide tile of the inner products
    ([3000, 1300, 8], [1, 2, 0], 3, 128, 264, 136, 0),
    # more tiles than the decode form takes: the tensor-core engine, with blocks that segments share
    ([300, 0, 133, 5, 2, 467], [0, 3, 2, 1, -1, 0], 5, 32, 1032, 1160, 9),
    ([1] * 660, [i % 7 - 1 for i in range(660)], 6, 24, 1032, 1040, 3),
    ([777, 1, 230], [1, -1, 0], 2, 128, 1096, 1032, 0),
    ([40, 0, 3, 90, 1], [1, 0, 1, -1, 0], 2, 16, 256, 192, 0),
    ([300, 0, 45, 0, 171], [0, 3, 2, 1, 0], 5, 32, 384, 520, 9),  # adapters without rows, one with two segments
    ([64, 64, 128, 256], [0, 1, 2, 3], 4, 128, 264, 136, 0),
    ([1000, 777], [1, 0], 2, 72, 512, 648, 0),
    ([0, 0, 70], [0, 1, 1], 2, 40, 72, 1032, 0),
    # the engine's shared blocks by every width of rank, found by number and by owning segment
    ([1] * 200 + [500], [i % 4 - 1 for i in range(201)], 3, 8, 1032, 1040, 5),
    ([3] * 150 + [411, 0], [i % 9 - 1 for i in range(152)], 8, 16, 1040, 1032, 0),
    ([900, 37, 0, 1111, 5], [0, 2, 1, -1, 1], 3, 64, 1032, 1040, 0),
    ([1] * 99 + [901], [i % 3 for i in range(100)], 3, 120, 1032, 1040, 0),
    ([1] * 20 + [1400], [i % 6 - 1 for i in range(21)], 5, 40, 1032, 1160, 2),
    ([17] * 140, [i % 6 - 1 for i in range(140)], 5, 16, 1032, 1040, 2),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_and_backward(M, case):
    lens, ad, n, r, N, K, tail = CASES[case]
    p = Problem(lens, ad, n, r, N, K, tail, seed=10 * case, with_scale=case % 3 != 1)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_forward()
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_backward()


@pytest.mark.parametrize("lens,N,K", [([1, 2, 1, 4], 136, 264), ([50, 3, 80], 136, 264), ([411, 3, 290], 1032, 1064)])
def test_strides(M, lens, N, K):
    p = Problem(lens, [1, -1, 0, 1][:len(lens)], 2, 16, N, K, tail=4, pad=16, seed=3)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_forward()
    p.check_backward()


@pytest.mark.parametrize("lens,N,K", [([1] * 6, 264, 136), ([20, 9, 40], 264, 136), ([70, 33, 61], 264, 136),
                                      ([370, 33, 261], 1032, 1064)])
def test_other_segments_values_do_not_enter(M, lens, N, K):
    """An infinity in one request's row stays out of the other requests' rows
    and gradients, though they share tiles."""
    def run(dirty):
        p = Problem(lens, [i % 3 for i in range(len(lens))], 3, 16, N, K, seed=7)
        lo, hi = p.off[1], p.off[2]
        p.x[lo:hi, ::3] = float("inf") if dirty else 0
        p.dy[lo:hi, ::5] = NAN if dirty else 0
        p.strided()
        ws = p.workspace(M)
        p.forward(M, ws)
        p.backward(M, ws)
        torch.cuda.synchronize()
        keep = [i for i in range(p.T) if not lo <= i < hi]
        other = [q for q in range(3) if q != 1]
        return [p.u[keep], p.y[keep], p.dx[keep], p.da[other], p.db[other]] if len(lens) == 3 else \
               [p.u[keep], p.y[keep], p.dx[keep], p.da[[0, 2]], p.db[[0, 2]]]
    for a, b in zip(run(True), run(False)):
        assert torch.isfinite(b).all() and torch.equal(a, b)


@pytest.mark.parametrize("scale,N,K", [(1, 136, 72), (2, 136, 72), (10, 136, 72), (51, 1032, 1064)])
def test_adapters_that_hold_nan_are_not_read_for_other_rows(M, scale, N, K):
    # every form of the projection; the engine's with shared 16-row blocks
    lens = [4 * scale, 6 * scale, 3 * scale]
    p = Problem(lens, [0, 1, -1], 2, 16, N, K, seed=9)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    p.backward(M, ws)
    y, dx, da = p.y.clone(), p.dx.clone(), p.da.clone()
    p.a[1], p.b[1] = NAN, NAN
    p.forward(M, ws)
    p.backward(M, ws)
    for lo, hi in ((0, p.off[1]), (p.off[2], p.off[3])):
        assert torch.equal(p.y[lo:hi], y[lo:hi]) and torch.equal(p.dx[lo:hi], dx[lo:hi])
    assert torch.equal(p.da[0], da[0])


@pytest.mark.parametrize("T,N,K", [(6, 72, 64), (20, 72, 64), (200, 72, 64), (700, 1032, 1040)])
def test_bad_segments_are_cut_and_flagged(M, T, N, K):
    p = Problem([T // 2, T // 2], [0, 1], 2, 16, N, K, seed=5)
    p.strided()
    ws = p.workspace(M)
    good = p.seg_off.clone()
    p.seg_off.copy_(torch.tensor([0, T + 50, T // 2], dtype=torch.int32))
    p.forward(M, ws)
    assert M.moe_read_device_error(ws) == M.MOE_DEVERR_OFFSETS
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == M.MOE_DEVERR_OFFSETS
    p.seg_off.copy_(good)
    p.seg_ad.copy_(torch.tensor([7, 1], dtype=torch.int32))
    p.ad = [-1, 1]
    p.forward(M, ws)
    assert M.moe_read_device_error(ws) == M.MOE_DEVERR_EXPERT_ID
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) == M.MOE_DEVERR_EXPERT_ID
    p.check_forward()
    p.check_backward()


LO, HI = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("off", [[0, 3, 1, 2, 3], [0, 2, LO, 2, 3], [HI, LO, HI, LO, HI], [1, LO, 3, LO, 2], [2, 2, 2, 2, HI]])
@pytest.mark.parametrize("T,N,K", [(6, 64, 72), (60, 64, 72), (201, 64, 72), (2010, 2048, 2048)])
def test_extreme_segments(M, off, T, N, K):
    p = Problem([T, 0, 0, 0], [0, 1, HI, LO], 2, 16, N, K, seed=7)
    p.xs, p.dys = p.x, p.dy
    p.seg_off.copy_(torch.tensor([min(o * (T // 3), HI) if 0 < o < HI else o for o in off], dtype=torch.int32))
    ws = p.workspace(M)
    p.u.zero_(), p.du.zero_()
    guard = 64  # rows before and behind what the calls may write
    y, dx = (torch.zeros(T + 2 * guard, c, dtype=torch.bfloat16, device="cuda") for c in (N, K))
    p.y, p.dx = y[guard:], dx[guard:]
    p.forward(M, ws)
    assert M.moe_read_device_error(ws) in (M.MOE_DEVERR_OFFSETS, M.MOE_DEVERR_EXPERT_ID)
    p.backward(M, ws)
    assert M.moe_read_device_error(ws) in (M.MOE_DEVERR_OFFSETS, M.MOE_DEVERR_EXPERT_ID)
    for t in (y, dx):
        assert (t[:guard] == 0).all() and (t[-guard:] == 0).all()


@pytest.mark.parametrize("lens", [[1] * 30 + [400], [400] + [1] * 40 + [0, 17, 33, 16], [500] + [0] * 40])
def test_long_segments_among_many_short_ones(M, lens):
    p = Problem(lens, [i % 4 - 1 for i in range(len(lens))], 3, 24, 136, 264, seed=8)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    assert M.moe_read_device_error(ws) == 0
    p.check_forward()
    p.backward(M, ws)
    p.check_backward()


def test_no_rows_and_partial_gradients(M):
    p = Problem([30, 20], [0, 1], 2, 16, 72, 64, seed=6)
    p.strided()
    ws = p.workspace(M)
    M.moe_lora_linear(None, 64, p.w, p.seg_off, p.seg_ad, p.a, p.b, None, 0, 2, 2, 16, 72, 64, None, None, 72, ws, ws.numel())
    M.moe_lora_linear_backward(None, 72, None, 64, p.w, None, p.seg_off, p.seg_ad, p.a, p.b, None, 0, 2, 2, 16, 72, 64,
                               None, None, 64, p.da, p.db, ws, ws.numel())
    assert (p.da == 0).all() and (p.db == 0).all()
    p.forward(M, ws)
    p.backward(M, ws)
    dx, da, db = p.dx.clone(), p.da.clone(), p.db.clone()
    p.dx.fill_(3), p.da.fill_(3), p.db.fill_(3)
    args = (p.dys, 72, None, 64, p.w, None, p.seg_off, p.seg_ad, p.a, p.b, p.scale, 50, 2, 2, 16, 72, 64, p.du)
    M.moe_lora_linear_backward(*args, p.dx, 64, None, None, ws, ws.numel())
    assert torch.equal(p.dx, dx) and (p.da == 3).all()
    args = (p.dys, 72, p.xs, 64, p.w, p.u, p.seg_off, p.seg_ad, p.a, p.b, p.scale, 50, 2, 2, 16, 72, 64, p.du)
    M.moe_lora_linear_backward(*args, None, 64, p.da, p.db, ws, ws.numel())
    assert torch.equal(p.da, da) and torch.equal(p.db, db)


def test_gradients_against_differences(M):
    """Along random directions of x, A and B against central differences of
    the formula in 64 bits (the loss is linear in each)."""
    p = Problem([37, 0, 50], [1, 0, 0], 2, 16, 72, 88, seed=8)
    p.strided()
    ws = p.workspace(M)
    p.forward(M, ws)
    p.backward(M, ws)
    dy, w, sc = p.dy.double(), p.w.double(), p.scale.double()

    def loss(x, a, b):
        t = (x @ w.T * dy).sum()
        for s, q in enumerate(p.ad):
            i, j = p.off[s], p.off[s + 1]
            t = t + (sc[q] * (x[i:j] @ a[q].T) @ b[q].T * dy[i:j]).sum()
        return t

    at = [p.x.double(), p.a.double(), p.b.double()]
    h = 2.0 ** -8
    for i, got in enumerate((p.dx, p.da, p.db)):
        v = _rand(at[i].shape, 20 + i).double()
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * v, at[i] - h * v
        num = (loss(*up) - loss(*down)) / (2 * h)
        # each gradient: one BF16 rounding of the output and one of the inner value, 2^-8 each, and fp32 sums;
        # sum |got v| bounds the first, the inner value's part is bounded by the sum of magnitudes below
        mags = [t.abs() for t in at]
        inner = 0.0
        if i < 2:
            for s, q in enumerate(p.ad):
                lo, hi = p.off[s], p.off[s + 1]
                du = (sc[q].abs() * (dy[lo:hi] @ p.b[q].double())).abs()
                other = (v[lo:hi].abs() @ mags[1][q].T) if i == 0 else (mags[0][lo:hi] @ v[q].abs().T)
                inner += (du * other).sum()
        else:
            for s, q in enumerate(p.ad):
                lo, hi = p.off[s], p.off[s + 1]
                inner += (p.u[lo:hi].double().abs() * (dy[lo:hi].abs() @ v[q].abs())).sum()
        bound = 2 * HALF * (got.double() * v).abs().sum() + 2 * HALF * inner
        assert abs((got.double() * v).sum() - num) <= bound


@pytest.mark.parametrize("lens,N,K", [([1] * 9, 264, 200), ([100, 31, 70], 264, 200), ([401, 31, 270], 1032, 1040)])
def test_captured_replayed_and_equal_bits(M, lens, N, K):
    p = Problem(lens, [i % 3 - 1 for i in range(len(lens))], 2, 16, N, K, seed=12)
    p.strided()
    ws = p.workspace(M)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    p.forward(M, ws, s)
    p.backward(M, ws, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        p.forward(M, ws, s)
        p.backward(M, ws, s)
    p.x.copy_(_rand(p.x.shape, 31))
    p.xs[:, :p.K] = p.x
    torch.cuda.synchronize()
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    p.check_forward()
    p.check_backward()
    keep = [t.clone() for t in (p.u, p.y, p.dx, p.da, p.db)]
    p.forward(M, ws)
    p.backward(M, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, (p.u, p.y, p.dx, p.da, p.db)))


def test_calls_on_several_streams_at_once(M):
    """Calls that overlap, each with a workspace of its own, directly and from
    graphs: the bits of the same calls made one by one."""
    probs = [Problem([1] * 60 + [900], [i % 6 - 1 for i in range(61)], 5, 64, 1032, 1040, seed=1),
             Problem([700, 3, 801], [1, -1, 0], 2, 16, 1040, 1032, seed=2),
             Problem([1] * 40, [i % 8 for i in range(40)], 8, 16, 1032, 1040, seed=3)]
    outs, refs, spaces, streams, graphs = [], [], [], [torch.cuda.Stream() for _ in probs], []

    def step(p, ws, stream=None):
        p.forward(M, ws, stream)
        p.backward(M, ws, stream)

    for p in probs:
        p.strided()
        spaces.append(p.workspace(M))
        step(p, spaces[-1])
        torch.cuda.synchronize()
        outs.append([p.u, p.y, p.du, p.dx, p.da, p.db])
        refs.append([t.clone() for t in outs[-1]])

    def check():
        torch.cuda.synchronize()
        for out, ref, ws in zip(outs, refs, spaces):
            assert M.moe_read_device_error(ws) == 0
            assert all(torch.equal(t, q) for t, q in zip(out, ref))
            for t in out:
                t.fill_(3.0)
        torch.cuda.synchronize()

    check()
    for _ in range(5):
        for p, ws, s in zip(probs, spaces, streams):
            step(p, ws, s.cuda_stream)
        check()
    for p, ws, s in zip(probs, spaces, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step(p, ws, s.cuda_stream)
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        check()
