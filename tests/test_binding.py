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
