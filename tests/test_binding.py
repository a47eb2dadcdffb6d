"""The Python binding on a machine without a GPU: how it finds torch's stream,
what it hands on, and what it refuses before the library sees an address."""
import pytest
import torch

P = 0x10000  # made-up address, 256-byte aligned, never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module")
def N():
    from w4a16_mixture_experts_moe_b200 import build
    build.build()
    from w4a16_mixture_experts_moe_b200 import _native
    return _native


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: calls that pass the checks end for want of a device")
@pytest.mark.parametrize("T", [4, 40, 700, 5000])
def test_calls_without_a_device_end_with_an_error(N, T):
    n, k = 1024, 1032
    for f32 in (0, N.MOE_GEMM_OUT_F32):
        calls = [N.lib.moe_grouped_gemm(P, k, P, P, n * k, T, 2, n, k, f32, P, n, P, BIG, None),
                 N.lib.moe_grouped_gemm_dgrad(P, n, P, P, n * k, T, 2, n, k, f32, P, k, P, BIG, None),
                 N.lib.moe_grouped_gemm_wgrad(P, n, P, k, P, T, 2, n, k, f32, P, n * k, P, BIG, None),
                 N.lib.moe_grouped_gemm_wgrad(P, n, P, k, P, 0, 2, n, k, f32, P, n * k, P, BIG, None)]
        assert all(st in (N.MOE_ERR_UNSUPPORTED, N.MOE_ERR_CUDA) for st in calls), calls
    for S in (1, 3):
        for r in (16, 128):
            calls = [N.lib.moe_lora_linear(P, k, P, P, P, P, P, None, T, S, 3, r, n, k, P, P, n, P, BIG, None),
                     N.lib.moe_lora_linear_backward(P, n, P, k, P, P, P, P, P, P, None, T, S, 3, r, n, k, P, P, k, P, P, P, BIG, None),
                     N.lib.moe_lora_linear_backward(P, n, P, k, P, P, P, P, P, P, None, T, S, 3, r, n, k, P, None, k, P, P, P, BIG, None)]
            assert all(st in (N.MOE_ERR_UNSUPPORTED, N.MOE_ERR_CUDA) for st in calls), calls


class _NoCuda:
    """torch's C layer where its CUDA functions are missing or raise."""
    def __init__(self, error):
        self._error = error

    def __getattr__(self, name):
        if self._error is AttributeError:
            raise AttributeError(name)

        def call(*args):
            raise self._error("no device")
        return call


class _Torch:
    def __init__(self, error, stream):
        self._C = _NoCuda(error)
        self.cuda = type("cuda", (), {"current_stream": staticmethod(stream)})


@pytest.mark.parametrize("error", [RuntimeError, AttributeError])
def test_without_a_device_the_public_call_tells_why(N, monkeypatch, error):
    def stream():
        raise AssertionError("Torch not compiled with CUDA enabled")
    monkeypatch.setattr(N, "_torch", _Torch(error, stream))
    assert N._current_device() == -2
    for call in (lambda: N.moe_combine(P, P, P, None, 4, 2, 256, P),              # an entry point of the layer
                 lambda: N.moe_grouped_gemm(P, 64, P, P, 64 * 32, 4, 2, 32, 64, 0, P, 32, P, BIG)):
        with pytest.raises(AssertionError, match="not compiled with CUDA"):
            call()


def test_a_device_that_torch_has_not_started_yet(N, monkeypatch):
    # the public call starts CUDA and finds the stream
    monkeypatch.setattr(N, "_torch", _Torch(RuntimeError, lambda: type("S", (), {"cuda_stream": 77})))
    assert N._stream(None) == 77


def test_a_replaced_name_is_seen(N, monkeypatch):
    import w4a16_mixture_experts_moe_b200 as moe
    from w4a16_mixture_experts_moe_b200 import layer
    assert moe.moe_abi_version is N.moe_abi_version and moe.ExpertBank is layer.ExpertBank
    monkeypatch.setattr(N, "moe_abi_version", lambda: 1234)
    monkeypatch.setattr(layer, "ExpertBank", int)
    assert moe.moe_abi_version() == 1234 and moe.ExpertBank is int
    monkeypatch.undo()
    assert moe.moe_abi_version is N.moe_abi_version and moe.ExpertBank is layer.ExpertBank
    with pytest.raises(AttributeError):
        moe.no_such_name


# ---- what the grouped products and the projection with adapters refuse. The tensors live on the CPU, whose device
# number is -1: with that as the current device, the checks behind the device's are reached.

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture
def cpu(N, monkeypatch):
    current = N._current_device
    monkeypatch.setattr(N, "_current_device", lambda: -1)
    calls = []

    class Lib:  # the library, which only records what it is given
        def __getattr__(self, name):
            return lambda *args: calls.append((name, args)) or 0
    monkeypatch.setattr(N, "lib", Lib())
    current()  # fills in the dtypes
    return calls


R, E, n, k, T, S, A, r = 5, 3, 16, 24, 6, 2, 4, 8


def _grouped(N, direction, **other):
    out = {"fwd": ("y", R, n), "dgrad": ("dx", R, k), "wgrad": ("dw", E, n * k)}[direction]
    t = dict(x=torch.zeros(R, k, dtype=BF), dy=torch.zeros(R, n, dtype=BF), w=torch.zeros(E, n, k, dtype=BF),
             offsets=torch.zeros(E + 1, dtype=I32), ws=torch.zeros(256, dtype=torch.uint8), flags=0, ws_bytes=256)
    t[out[0]] = torch.zeros(out[1], out[2], dtype=BF)
    t.update(other)
    if direction == "fwd":
        N.moe_grouped_gemm(t["x"], t.get("ldx", k), t["offsets"], t["w"], n * k, R, E, n, k, t["flags"], t["y"], n, t["ws"], t["ws_bytes"], 0)
    elif direction == "dgrad":
        N.moe_grouped_gemm_dgrad(t["dy"], n, t["offsets"], t["w"], n * k, R, E, n, k, t["flags"], t["dx"], k, t["ws"], t["ws_bytes"], 0)
    else:
        N.moe_grouped_gemm_wgrad(t["dy"], n, t["x"], t.get("ldx", k), t["offsets"], R, E, n, k, t["flags"], t["dw"], n * k, t["ws"], t["ws_bytes"], 0)


def _lora_args():
    return dict(x=torch.zeros(T, k, dtype=BF), dy=torch.zeros(T, n, dtype=BF), w=torch.zeros(n, k, dtype=BF),
                seg_offsets=torch.zeros(S + 1, dtype=I32), seg_adapter=torch.zeros(S, dtype=I32),
                lora_a=torch.zeros(A, r, k, dtype=BF), lora_b=torch.zeros(A, n, r, dtype=BF), scale=torch.zeros(A, dtype=F32),
                u=torch.zeros(T, r, dtype=BF), y=torch.zeros(T, n, dtype=BF), du=torch.zeros(T, r, dtype=BF),
                dx=torch.zeros(T, k, dtype=BF), d_lora_a=torch.zeros(A, r, k, dtype=BF), d_lora_b=torch.zeros(A, n, r, dtype=BF),
                ws=torch.zeros(256, dtype=torch.uint8))


def _lora(N, back, **other):
    t = {**_lora_args(), **other}
    if back:
        N.moe_lora_linear_backward(t["dy"], n, t["x"], k, t["w"], t["u"], t["seg_offsets"], t["seg_adapter"], t["lora_a"],
                                   t["lora_b"], t["scale"], T, S, A, r, n, k, t["du"], t["dx"], k, t["d_lora_a"],
                                   t["d_lora_b"], t["ws"], 256, 0)
    else:
        N.moe_lora_linear(t["x"], k, t["w"], t["seg_offsets"], t["seg_adapter"], t["lora_a"], t["lora_b"], t["scale"], T, S,
                          A, r, n, k, t["u"], t["y"], n, t["ws"], 256, 0)


def _refused(N, cpu, name, call):
    with pytest.raises(N.MoeError, match=f"^.status {N.MOE_ERR_INVALID_ARG}. {name}: ") as ei:
        call()
    assert not cpu  # the library was not called
    return str(ei.value)


@pytest.mark.parametrize("direction", ["fwd", "dgrad", "wgrad"])
def test_grouped_tensors(N, cpu, direction):
    mine = {"fwd": ["x", "offsets", "w", "y", "ws"], "dgrad": ["dy", "offsets", "w", "dx", "ws"],
            "wgrad": ["dy", "x", "offsets", "dw", "ws"]}[direction]
    _grouped(N, direction)
    assert len(cpu) == 1
    full = dict(x=torch.zeros(R, k, dtype=BF), dy=torch.zeros(R, n, dtype=BF), w=torch.zeros(E, n, k, dtype=BF),
                offsets=torch.zeros(E + 1, dtype=I32), ws=torch.zeros(256, dtype=torch.uint8), y=torch.zeros(R, n, dtype=BF),
                dx=torch.zeros(R, k, dtype=BF), dw=torch.zeros(E, n * k, dtype=BF))
    del cpu[:]
    for name in mine:
        t = full[name]
        assert "reaches" in _refused(N, cpu, name, lambda: _grouped(N, direction, **{name: t.flatten()[:-1].clone()}))
        wide = torch.zeros(1, dtype=t.dtype).expand(t.numel())   # one element under any number of indices
        assert "reaches" in _refused(N, cpu, name, lambda: _grouped(N, direction, **{name: wide}))
        if name != "ws":
            for kind in (torch.float32, torch.float16, torch.int64):
                assert str(kind) in _refused(N, cpu, name, lambda: _grouped(N, direction, **{name: t.to(kind)}))
    out = {"fwd": "y", "dgrad": "dx", "wgrad": "dw"}[direction]
    f32 = dict(flags=N.MOE_GEMM_OUT_F32)
    assert "bfloat16" in _refused(N, cpu, out, lambda: _grouped(N, direction, **f32))
    assert "reaches" in _refused(N, cpu, out, lambda: _grouped(N, direction, **f32, **{out: full[out].float().flatten()[1:].clone()}))
    _grouped(N, direction, **f32, **{out: full[out].float()})
    assert len(cpu) == 1


@pytest.mark.parametrize("back", [False, True])
def test_adapters_tensors(N, cpu, back):
    mine = ["x", "w", "seg_offsets", "seg_adapter", "lora_a", "lora_b", "scale", "u", "ws"]
    mine += ["dy", "du", "dx", "d_lora_a", "d_lora_b"] if back else ["y"]
    _lora(N, back)
    assert len(cpu) == 1
    del cpu[:]
    for name in mine:
        t = _lora_args()[name]
        assert "reaches" in _refused(N, cpu, name, lambda: _lora(N, back, **{name: t.flatten()[:-1].clone()}))
        if name != "ws":
            for kind in (torch.float16, torch.int64, torch.float64):
                assert str(kind) in _refused(N, cpu, name, lambda: _lora(N, back, **{name: t.to(kind)}))


def test_views_that_hold_what_the_call_reaches(N, cpu):
    wide = torch.zeros(R, k + 40, dtype=BF)
    _grouped(N, "fwd", x=wide[:, :k], ldx=k + 40)          # a strided view, its rows' padding in the storage
    _grouped(N, "fwd", x=wide[:, 40:], ldx=k + 40)         # (the last row ends with the storage)
    _grouped(N, "fwd", x=torch.zeros(R, k, dtype=torch.int16))  # 16-bit patterns
    record = torch.zeros(E * n * k * 2 + 64, dtype=torch.uint8)  # the bytes of a bank
    _grouped(N, "fwd", w=record[64:], offsets=record[:4 * E + 4])
    assert len(cpu) == 4
    del cpu[:]
    _refused(N, cpu, "w", lambda: _grouped(N, "fwd", w=record[65:]))
    _refused(N, cpu, "x", lambda: _grouped(N, "fwd", x=wide[:, 41:], ldx=k + 40))
    _refused(N, cpu, "x", lambda: _grouped(N, "fwd", x=wide[1:, :k], ldx=k + 40))
    _refused(N, cpu, "ws", lambda: _grouped(N, "fwd", ws_bytes=257))
    _lora(N, False, scale=None)
    _lora(N, True, scale=None, dx=None, d_lora_a=None, d_lora_b=None, x=None, u=None)
    assert len(cpu) == 2


def test_no_rows_reach_nothing(N, cpu):
    few = torch.zeros(1, dtype=BF)
    off, ws = torch.zeros(E + 1, dtype=I32), torch.zeros(256, dtype=torch.uint8)
    N.moe_grouped_gemm(few, k, off, few, n * k, 0, E, n, k, 0, few, n, ws, 256, 0)
    N.moe_grouped_gemm_dgrad(few, n, off, few, n * k, 0, E, n, k, 0, few, k, ws, 256, 0)
    N.moe_grouped_gemm_wgrad(few, n, few, k, off, 0, E, n, k, 0, torch.zeros(E, n, k, dtype=BF), n * k, ws, 256, 0)
    assert len(cpu) == 3


# ---- the calls by words: the same answers as the calls themselves

WORDS = [
    ("moe_grouped_gemm", (P, 64, P, P, 64 * 32, 4, 2, 32, 64, 0, P, 32, P, BIG, 0)),
    ("moe_grouped_gemm_dgrad", (P, 32, P, P, 64 * 32, 4, 2, 32, 64, 0, P, 64, P, BIG, 0)),
    ("moe_grouped_gemm_wgrad", (P, 32, P, 64, P, 4, 2, 32, 64, 0, P, 64 * 32, P, BIG, 0)),
    ("moe_lora_linear", (P, 64, P, P, P, P, P, 0, 4, 2, 3, 16, 32, 64, P, P, 32, P, BIG, 0)),
    ("moe_lora_linear_backward", (P, 32, P, 64, P, P, P, P, P, P, 0, 4, 2, 3, 16, 32, 64, P, P, 64, P, P, P, BIG, 0)),
]


@pytest.mark.parametrize("name,args", WORDS)
def test_words_give_the_answers_of_the_call(N, name, args):
    import struct
    if torch.cuda.is_available():
        pytest.skip("what is not refused would run on made-up addresses")
    call, words = getattr(N.lib, name), getattr(N.lib, name + "_words")
    refused = 0
    for i in range(len(args) - 1):            # the stream is not looked at
        for value in (0, -1, 4, 12, P + 2, (1 << 31) - 1):
            if i == len(args) - 2 and value < 0:
                continue                      # (bytes)
            a = list(args)
            a[i] = value
            plain = [v or None if t is N._p else v for v, t in zip(a, N.SIGNATURES[name][1])]
            st = call(*plain)
            message = N.lib.moe_last_error() if st else b""
            got = words(struct.pack(f"{len(a)}q", *a))
            assert got == st and (N.lib.moe_last_error() if got else b"") == message, (i, value)
            refused += st in (N.MOE_ERR_SHAPE, N.MOE_ERR_INVALID_ARG)
    assert refused > 2 * len(args)


def test_words_beyond_their_arguments_are_refused(N):
    import struct
    for name, args in WORDS:
        words = getattr(N.lib, name + "_words")
        sizes = [i for i, t in enumerate(N.SIGNATURES[name][1]) if t is N._i]
        for i in sizes:
            a = list(args)
            a[i] += 1 << 32                   # would be the same number in 32 bits
            assert words(struct.pack(f"{len(a)}q", *a)) == N.MOE_ERR_SHAPE
            assert b"32 bits" in N.lib.moe_last_error() and name.encode() in N.lib.moe_last_error()
        a = list(args)
        a[-2] = -1                            # would be the largest workspace there is
        assert words(struct.pack(f"{len(a)}q", *a)) == N.MOE_ERR_SHAPE
        assert words(None) == N.MOE_ERR_INVALID_ARG


def test_workspace_of_long_reductions(N):
    """BF16 sums of more than 16,384 products pass through the workspace; a call whose own sums are short, or whose
    output is fp32, does not ask for that."""
    small = N.moe_grouped_gemm_workspace_size(16384, 8, 16384, 16384)
    assert small == 256
    long = [N.moe_grouped_gemm_workspace_size(*a) for a in ((16385, 8, 64, 64), (8, 8, 16392, 64), (8, 8, 64, 16392))]
    assert long == [long[0]] * 3 and long[0] > small + 100 * 256 * 128 * 4
    L, ok = 16392, (N.MOE_ERR_UNSUPPORTED, N.MOE_ERR_CUDA)
    fwd = lambda n, k, flags, size: N.lib.moe_grouped_gemm(P, k, P, P, n * k, 400, 2, n, k, flags, P, n, P, size, None)
    dgrad = lambda n, k, flags, size: N.lib.moe_grouped_gemm_dgrad(P, n, P, P, n * k, 400, 2, n, k, flags, P, k, P, size, None)
    wgrad = lambda r, flags, size: N.lib.moe_grouped_gemm_wgrad(P, 64, P, 64, P, r, 2, 64, 64, flags, P, 64 * 64, P, size, None)
    f32 = N.MOE_GEMM_OUT_F32
    for call in (lambda s: fwd(64, L, 0, s), lambda s: dgrad(L, 64, 0, s), lambda s: wgrad(L, 0, s)):
        assert call(long[0] - 1) == N.MOE_ERR_INVALID_ARG and b"workspace" in N.lib.moe_last_error()
        assert torch.cuda.is_available() or call(long[0]) in ok
    if not torch.cuda.is_available():
        for call in (lambda s: fwd(L, 64, 0, s), lambda s: dgrad(64, L, 0, s), lambda s: fwd(64, L, f32, s),
                     lambda s: dgrad(L, 64, f32, s), lambda s: wgrad(L, f32, s), lambda s: wgrad(16384, 0, s)):
            assert call(256) in ok
    # the adapters': beside that a megabyte at least for the split inner gradient, 4 bytes for each row and rank
    MB = 1 << 20
    assert N.moe_lora_workspace_size(1, 1, 2, 8, 64, 64) == N.moe_lora_workspace_size(2048, 1, 9, 128, 64, 64) == 256 + MB
    assert N.moe_lora_workspace_size(2049, 1, 9, 128, 64, 64) == 256 + 2049 * 512
    assert N.moe_lora_workspace_size(400, 1, 2, 16, 64, L) == N.moe_lora_workspace_size(400, 1, 2, 16, L, 64) == long[0] + MB
    assert N.moe_lora_workspace_size(400, 3, 2, 16, 64, L) == long[0] + MB + 48 * L * 4 + 1600
    # ... which only a call that asks for the adapters' gradients needs
    T, S, n, r, no, k = 400, 3, 2, 16, 64, 1024
    whole = N.moe_lora_workspace_size(T, S, n, r, no, k)
    fwd = lambda s: N.lib.moe_lora_linear(P, k, P, P, P, P, P, None, T, S, n, r, no, k, P, P, no, P, s, None)
    bwd = lambda d, s: N.lib.moe_lora_linear_backward(P, no, P, k, P, P, P, P, P, P, None, T, S, n, r, no, k, P, P, k, d, d, P, s, None)
    bad = N.MOE_ERR_INVALID_ARG
    assert fwd(whole - MB - 1) == bwd(None, whole - MB - 1) == bwd(P, whole - 1) == bad
    if not torch.cuda.is_available():
        assert fwd(whole - MB) in ok and bwd(None, whole - MB) in ok and bwd(P, whole) in ok


def test_columns_beyond_the_kernels_arithmetic_are_refused(N):
    most = 1 << 30
    for n, k in ((most + 8, 8), (8, most + 8), ((1 << 31) - 8, 8), (8, (1 << 31) - 8)):
        size, st = 1 << 60, N.MOE_ERR_SHAPE
        for R in (1, 400):
            assert N.lib.moe_grouped_gemm(P, k, P, P, n * k, R, 1, n, k, 0, P, n, P, size, None) == st
            assert N.lib.moe_grouped_gemm_dgrad(P, n, P, P, n * k, R, 1, n, k, 0, P, k, P, size, None) == st
            assert N.lib.moe_grouped_gemm_wgrad(P, n, P, k, P, R, 1, n, k, 0, P, n * k, P, size, None) == st
            assert N.lib.moe_lora_linear(P, k, P, P, P, P, P, None, R, 1, 1, 8, n, k, P, P, n, P, size, None) == st
            assert N.lib.moe_lora_linear_backward(P, n, P, k, P, P, P, P, P, P, None, R, 1, 1, 8, n, k, P, P, k, P, P, P, size, None) == st
            assert b"2^30" in N.lib.moe_last_error()
