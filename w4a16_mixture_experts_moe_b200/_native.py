"""ctypes binding of libexactmoe.so: the C ABI of include/exactmoe.h, same names.

Argument marshalling only. Pointer arguments accept a torch tensor (its
data_ptr), a plain int address, or None (NULL). Stream arguments accept a
torch.cuda.Stream, a raw cudaStream_t int, or None (torch's current stream).
A non-zero status raises MoeError with the library's message. There is no
fallback: if the library is missing the import of this module fails.
"""
from __future__ import annotations

import ctypes as C
import os
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libexactmoe.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m w4a16_mixture_experts_moe_b200.build` "
        "(the MoE layer has no CPU or Python fallback)")

lib = C.CDLL(LIB_PATH)

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_SHAPE, MOE_ERR_CUDA, MOE_ERR_CAPACITY, MOE_ERR_DEVICE, MOE_ERR_UNSUPPORTED = range(7)
MOE_DEVERR_NONE, MOE_DEVERR_EXPERT_ID, MOE_DEVERR_NOT_RESIDENT, MOE_DEVERR_TIMEOUT, MOE_DEVERR_RANGE, MOE_DEVERR_OFFSETS = range(6)
MOE_GEMM_OUT_F32, MOE_GEMM_ACCUMULATE = 1, 2
MOE_RENORM, MOE_LOGITS_GIVEN, MOE_IDS_GIVEN = 1, 2, 4
MOE_PATH_AUTO, MOE_PATH_GEMV, MOE_PATH_TC, MOE_PATH_SEQUENTIAL = 0, 1, 2, 3
MOE_SLOT_SKIP = -2
MOE_FFN_X_F16 = 0x100

_p = C.c_void_p
_i = C.c_int
_i64 = C.c_int64
_sz = C.c_size_t


class moe_record_layout(C.Structure):
    _fields_ = [("gate_q", _i64), ("up_q", _i64), ("down_q", _i64),
                ("gate_s", _i64), ("up_s", _i64), ("down_s", _i64), ("bytes", _i64)]


class moe_bf16_layout(C.Structure):
    _fields_ = [("gate", _i64), ("up", _i64), ("down", _i64), ("bytes", _i64)]


class moe_pool_info(C.Structure):
    _fields_ = [("layers", C.c_int32), ("E", C.c_int32), ("H", C.c_int32), ("I", C.c_int32),
                ("record_bytes", _i64)]


# name -> (restype, argtypes); kept in the order of include/exactmoe.h
SIGNATURES = {
    "moe_last_error": (C.c_char_p, []),
    "moe_abi_version": (_i, []),
    "moe_launch_counter": (C.c_uint64, []),
    "moe_expert_record_layout": (_i, [_i, _i, C.POINTER(moe_record_layout)]),
    "moe_quantize_pack": (_i, [_p, _i, _i, _i, _p, _i64, _p, _i64, _p]),
    "moe_route_topk": (_i, [_p, _p, _i, _i, _i, _i, _p, _i, _p, _p, _p, _p]),
    "moe_route_topk_x16": (_i, [_p, _p, _i, _i, _i, _i, _p, _i, _p, _p, _p, _p, _p, _p]),
    "moe_group_workspace_size": (_sz, [_i, _i, _i]),
    "moe_group_tokens": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _p, _sz, _p]),
    "moe_group_tokens_noalloc": (_i, [_p, _i, _i, _i, _p, _p, _p, _p, _p]),
    "moe_ffn_workspace_size": (_sz, [_i, _i, _i, _i, _i, _i]),
    "moe_grouped_w4a16_ffn": (_i, [_p, _p, _p, _p, _i64, _p, _i, _i, _i, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "moe_bf16_record_layout": (_i, [_i, _i, C.POINTER(moe_bf16_layout)]),
    "moe_bf16_ffn_workspace_size": (_sz, [_i, _i, _i, _i, _i]),
    "moe_grouped_bf16_ffn": (_i, [_p, _p, _p, _p, _i64, _i, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "moe_grouped_gemm_workspace_size": (_sz, [_i, _i, _i, _i]),
    "moe_grouped_gemm": (_i, [_p, _i64, _p, _p, _i64, _i, _i, _i, _i, _i, _p, _i64, _p, _sz, _p]),
    "moe_grouped_gemm_dgrad": (_i, [_p, _i64, _p, _p, _i64, _i, _i, _i, _i, _i, _p, _i64, _p, _sz, _p]),
    "moe_grouped_gemm_wgrad": (_i, [_p, _i64, _p, _i64, _p, _i, _i, _i, _i, _i, _p, _i64, _p, _sz, _p]),
    "moe_lora_workspace_size": (_sz, [_i] * 6),
    "moe_lora_linear": (_i, [_p, _i64] + [_p] * 6 + [_i] * 6 + [_p, _p, _i64, _p, _sz, _p]),
    "moe_lora_linear_backward": (_i, [_p, _i64, _p, _i64] + [_p] * 7 + [_i] * 6 + [_p, _p, _i64, _p, _p, _p, _sz, _p]),
    "moe_grouped_gemm_words": (_i, [C.c_char_p]),
    "moe_grouped_gemm_dgrad_words": (_i, [C.c_char_p]),
    "moe_grouped_gemm_wgrad_words": (_i, [C.c_char_p]),
    "moe_lora_linear_words": (_i, [C.c_char_p]),
    "moe_lora_linear_backward_words": (_i, [C.c_char_p]),
    "moe_debug_stall_next_tc_ffn": (_i, [_i]),
    "moe_combine": (_i, [_p, _p, _p, _p, _i, _i, _i, _p, _p]),
    "moe_read_device_error": (_i, [_p, _p, C.POINTER(C.c_int32)]),
    "slot_cache_create": (_i, [C.POINTER(_p), _i, _i, _i, _i64, _p, _p, _p]),
    "slot_cache_lookup": (_i, [_p, _i, _p, _i, _p, _p, C.POINTER(_i)]),
    "slot_cache_fill": (_i, [_p, _i, _p, _i, _p, _p]),
    "slot_cache_release": (_i, [_p, _i, _p]),
    "slot_cache_plan_waves": (_i, [_p, _i, _p, _i, _p, _p, C.POINTER(_i)]),
    "slot_cache_stats": (_i, [_p, C.POINTER(C.c_uint64), C.POINTER(C.c_uint64), C.POINTER(C.c_uint64)]),
    "slot_cache_inject_fill_failure": (_i, [_p, _i]),
    "slot_cache_destroy": (None, [_p]),
    "moe_pool_save": (_i, [C.c_char_p, C.POINTER(moe_pool_info), _p]),
    "moe_pool_file_info": (_i, [C.c_char_p, C.POINTER(moe_pool_info)]),
    "moe_pool_load": (_i, [C.c_char_p, _p, _sz, C.POINTER(moe_pool_info)]),
}

for _name, (_res, _args) in SIGNATURES.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[status {status}] {message}")
        self.status = status


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _dev(x, cur, name, kinds, need):
    """_ptr of an argument that a kernel dereferences. A tensor has to live on the current device `cur` (an address
    that this device cannot reach would fault it), be of one of `kinds` (its dtype; none: any) and hold `need` bytes
    from its first element on, whatever strides its view of them has; an address is taken as it is."""
    if x is None or isinstance(x, int):
        return x or 0
    if x.get_device() != cur or (kinds and x.dtype not in kinds) or x.nbytes < need or not x.is_contiguous():
        _dev_slow(x, cur, name, kinds, need)
    return x.data_ptr()


def _dev_slow(x, cur, name, kinds, need):
    if x.get_device() != cur:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: tensor on {x.device}, but the current device is cuda:{cur}")
    if kinds and x.dtype not in kinds:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: a tensor of {x.dtype}, not of {' or '.join(map(str, kinds))}")
    have = x.untyped_storage().nbytes() - x.storage_offset() * x.itemsize
    if have < need:
        raise MoeError(MOE_ERR_INVALID_ARG, f"{name}: {have} bytes from the tensor's first element on, but the call "
                                            f"reaches {need}")


_torch = None
_BF16 = _I32 = _F32 = ()  # dtypes of the arguments (filled with torch's): BF16 also as 16-bit patterns, each as plain bytes


def _current_device() -> int:
    """torch's current CUDA device (-2 without one). Asked of torch's C layer:
    the public call costs half a microsecond more on every launch."""
    global _torch, _BF16, _I32, _F32
    if _torch is None:
        import torch
        _torch = torch
        _BF16 = (torch.bfloat16, torch.uint16, torch.int16, torch.uint8)
        _I32, _F32 = (torch.int32, torch.uint8), (torch.float32, torch.uint8)
    try:
        return _torch._C._cuda_getDevice()
    except (RuntimeError, AttributeError):  # no driver or device; a torch built without CUDA has no such function
        return -2


def _addr(arr):
    return C.cast(arr, C.c_void_p).value


def _stream(s, d=None):
    if s is None:  # the raw handle of torch's current stream (on device d), without the Stream object around it
        if d is None:
            d = _current_device()
        if d < 0:
            return _torch.cuda.current_stream().cuda_stream  # says why there is none
        return _torch._C._cuda_getCurrentRawStream(d)
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int):
    if status != MOE_OK:
        raise MoeError(status, lib.moe_last_error().decode())


def moe_last_error() -> str:
    return lib.moe_last_error().decode()


def moe_abi_version() -> int:
    return lib.moe_abi_version()


def moe_launch_counter() -> int:
    return lib.moe_launch_counter()


def moe_expert_record_layout(H: int, I: int) -> dict:
    out = moe_record_layout()
    _check(lib.moe_expert_record_layout(H, I, C.byref(out)))
    return {f: getattr(out, f) for f, _ in moe_record_layout._fields_}


def moe_quantize_pack(w, E, N, K, packed, packed_stride, scales, scales_stride, stream=None):
    _check(lib.moe_quantize_pack(_ptr(w), E, N, K, _ptr(packed), packed_stride, _ptr(scales), scales_stride,
                                 _stream(stream)))


def moe_route_topk(x, w_router, T, H, E, k, bias, flags, logits, topk_ids, topk_w, stream=None):
    _check(lib.moe_route_topk(_ptr(x), _ptr(w_router), T, H, E, k, _ptr(bias), flags, _ptr(logits),
                              _ptr(topk_ids), _ptr(topk_w), _stream(stream)))


def moe_route_topk_x16(x, w_router, T, H, E, k, bias, flags, logits, topk_ids, topk_w, x16, err=None, stream=None):
    _check(lib.moe_route_topk_x16(_ptr(x), _ptr(w_router), T, H, E, k, _ptr(bias), flags, _ptr(logits),
                                  _ptr(topk_ids), _ptr(topk_w), _ptr(x16), _ptr(err), _stream(stream)))


def moe_group_workspace_size(T, k, E) -> int:
    return lib.moe_group_workspace_size(T, k, E)


def moe_group_tokens(topk_ids, T, k, E, counts, offsets, sorted_pair, pair_pos, ws, ws_bytes, stream=None):
    _check(lib.moe_group_tokens(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets), _ptr(sorted_pair),
                                _ptr(pair_pos), _ptr(ws), ws_bytes, _stream(stream)))


def moe_group_tokens_noalloc(topk_ids, T, k, E, counts, offsets, sorted_pair, pair_pos, stream=None):
    """moe_group_tokens with the library's fixed scratch (no workspace); see include/exactmoe.h."""
    _check(lib.moe_group_tokens_noalloc(_ptr(topk_ids), T, k, E, _ptr(counts), _ptr(offsets), _ptr(sorted_pair),
                                        _ptr(pair_pos), _stream(stream)))


MOE_NOALLOC_MAX_PAIRS = 65536


def moe_ffn_workspace_size(T, k, E, H, I, path=MOE_PATH_AUTO) -> int:
    return lib.moe_ffn_workspace_size(T, k, E, H, I, path)


def moe_grouped_w4a16_ffn(x, sorted_pair, offsets, bank, record_bytes, expert_slot, n_slots, T, k, E, H, I, path,
                          y, ws, ws_bytes, stream=None):
    _check(lib.moe_grouped_w4a16_ffn(_ptr(x), _ptr(sorted_pair), _ptr(offsets), _ptr(bank), record_bytes,
                                     _ptr(expert_slot), n_slots, T, k, E, H, I, path, _ptr(y), _ptr(ws), ws_bytes,
                                     _stream(stream)))


def moe_bf16_record_layout(H: int, I: int) -> dict:
    out = moe_bf16_layout()
    _check(lib.moe_bf16_record_layout(H, I, C.byref(out)))
    return {f: getattr(out, f) for f, _ in moe_bf16_layout._fields_}


def moe_bf16_ffn_workspace_size(T, k, E, H, I) -> int:
    return lib.moe_bf16_ffn_workspace_size(T, k, E, H, I)


def moe_grouped_bf16_ffn(x, sorted_pair, offsets, bank, record_bytes, T, k, E, H, I, y, ws, ws_bytes,
                         stream=None):
    _check(lib.moe_grouped_bf16_ffn(_ptr(x), _ptr(sorted_pair), _ptr(offsets), _ptr(bank), record_bytes, T, k, E,
                                    H, I, _ptr(y), _ptr(ws), ws_bytes, _stream(stream)))


def moe_grouped_gemm_workspace_size(R, E, N, K) -> int:
    return lib.moe_grouped_gemm_workspace_size(R, E, N, K)


# Arguments as 64-bit words in one array: ctypes converts an argument in 0.1 us, and these calls have up to 25.
_words15, _words20, _words25 = (struct.Struct(f"{n}q").pack for n in (15, 20, 25))


def moe_grouped_gemm(x, ldx, offsets, w, w_stride, R, E, N, K, flags, y, ldy, ws, ws_bytes, stream=None):
    d = _current_device()
    f32 = flags & MOE_GEMM_OUT_F32
    _check(lib.moe_grouped_gemm_words(_words15(
        _dev(x, d, "x", _BF16, R and 2 * ((R - 1) * ldx + K)), ldx, _dev(offsets, d, "offsets", _I32, 4 * E + 4),
        _dev(w, d, "w", _BF16, R and 2 * ((E - 1) * w_stride + N * K)), w_stride, R, E, N, K, flags,
        _dev(y, d, "y", _F32 if f32 else _BF16, R and (4 if f32 else 2) * ((R - 1) * ldy + N)), ldy,
        _dev(ws, d, "ws", (), ws_bytes), ws_bytes, _stream(stream, d) or 0)))


def moe_grouped_gemm_dgrad(dy, lddy, offsets, w, w_stride, R, E, N, K, flags, dx, lddx, ws, ws_bytes, stream=None):
    d = _current_device()
    f32 = flags & MOE_GEMM_OUT_F32
    _check(lib.moe_grouped_gemm_dgrad_words(_words15(
        _dev(dy, d, "dy", _BF16, R and 2 * ((R - 1) * lddy + N)), lddy, _dev(offsets, d, "offsets", _I32, 4 * E + 4),
        _dev(w, d, "w", _BF16, R and 2 * ((E - 1) * w_stride + N * K)), w_stride, R, E, N, K, flags,
        _dev(dx, d, "dx", _F32 if f32 else _BF16, R and (4 if f32 else 2) * ((R - 1) * lddx + K)), lddx,
        _dev(ws, d, "ws", (), ws_bytes), ws_bytes, _stream(stream, d) or 0)))


def moe_grouped_gemm_wgrad(dy, lddy, x, ldx, offsets, R, E, N, K, flags, dw, dw_stride, ws, ws_bytes, stream=None):
    d = _current_device()
    f32 = flags & MOE_GEMM_OUT_F32
    _check(lib.moe_grouped_gemm_wgrad_words(_words15(
        _dev(dy, d, "dy", _BF16, R and 2 * ((R - 1) * lddy + N)), lddy, _dev(x, d, "x", _BF16, R and 2 * ((R - 1) * ldx + K)), ldx,
        _dev(offsets, d, "offsets", _I32, 4 * E + 4), R, E, N, K, flags,
        _dev(dw, d, "dw", _F32 if f32 else _BF16, E and (4 if f32 else 2) * ((E - 1) * dw_stride + N * K)), dw_stride,
        _dev(ws, d, "ws", (), ws_bytes), ws_bytes, _stream(stream, d) or 0)))


def moe_lora_workspace_size(T, S, n_adapters, rank, N, K) -> int:
    return lib.moe_lora_workspace_size(T, S, n_adapters, rank, N, K)


def moe_lora_linear(x, ldx, w, seg_offsets, seg_adapter, lora_a, lora_b, scale, T, S, n_adapters, rank, N, K, u, y, ldy,
                    ws, ws_bytes, stream=None):
    d = _current_device()
    bf, per = _BF16, 2 * n_adapters * rank
    _check(lib.moe_lora_linear_words(_words20(
        _dev(x, d, "x", bf, T and 2 * ((T - 1) * ldx + K)), ldx, _dev(w, d, "w", bf, 2 * N * K),
        _dev(seg_offsets, d, "seg_offsets", _I32, 4 * S + 4), _dev(seg_adapter, d, "seg_adapter", _I32, 4 * S),
        _dev(lora_a, d, "lora_a", bf, per * K), _dev(lora_b, d, "lora_b", bf, per * N),
        _dev(scale, d, "scale", _F32, 4 * n_adapters), T, S, n_adapters, rank, N, K,
        _dev(u, d, "u", bf, 2 * T * rank), _dev(y, d, "y", bf, T and 2 * ((T - 1) * ldy + N)), ldy,
        _dev(ws, d, "ws", (), ws_bytes), ws_bytes, _stream(stream, d) or 0)))


def moe_lora_linear_backward(dy, lddy, x, ldx, w, u, seg_offsets, seg_adapter, lora_a, lora_b, scale, T, S, n_adapters,
                             rank, N, K, du, dx, lddx, d_lora_a, d_lora_b, ws, ws_bytes, stream=None):
    d = _current_device()
    bf, per = _BF16, 2 * n_adapters * rank
    _check(lib.moe_lora_linear_backward_words(_words25(
        _dev(dy, d, "dy", bf, T and 2 * ((T - 1) * lddy + N)), lddy, _dev(x, d, "x", bf, T and 2 * ((T - 1) * ldx + K)), ldx,
        _dev(w, d, "w", bf, 2 * N * K), _dev(u, d, "u", bf, 2 * T * rank),
        _dev(seg_offsets, d, "seg_offsets", _I32, 4 * S + 4), _dev(seg_adapter, d, "seg_adapter", _I32, 4 * S),
        _dev(lora_a, d, "lora_a", bf, per * K), _dev(lora_b, d, "lora_b", bf, per * N),
        _dev(scale, d, "scale", _F32, 4 * n_adapters), T, S, n_adapters, rank, N, K,
        _dev(du, d, "du", bf, 2 * T * rank), _dev(dx, d, "dx", bf, T and 2 * ((T - 1) * lddx + K)), lddx,
        _dev(d_lora_a, d, "d_lora_a", bf, per * K), _dev(d_lora_b, d, "d_lora_b", bf, per * N),
        _dev(ws, d, "ws", (), ws_bytes), ws_bytes, _stream(stream, d) or 0)))


def moe_debug_stall_next_tc_ffn(calls: int):
    """Test hook: the next `calls` tensor-core FFN launches time out on purpose."""
    _check(lib.moe_debug_stall_next_tc_ffn(calls))


def moe_combine(y, topk_w, pair_pos, residual, T, k, H, out, stream=None):
    _check(lib.moe_combine(_ptr(y), _ptr(topk_w), _ptr(pair_pos), _ptr(residual), T, k, H, _ptr(out),
                           _stream(stream)))


def moe_read_device_error(ws, stream=None) -> int:
    """Synchronises, returns the device error code of the workspace and clears it."""
    code = C.c_int32(0)
    st = lib.moe_read_device_error(_ptr(ws), _stream(stream), C.byref(code))
    if st not in (MOE_OK, MOE_ERR_DEVICE):
        _check(st)
    return code.value


class SlotCache:
    """Owner of a moe_slot_cache handle; methods map 1:1 onto slot_cache_*."""

    def __init__(self, layers, E, slots, record_bytes, pinned_pool, device_slots, expert_slot):
        h = C.c_void_p()
        _check(lib.slot_cache_create(C.byref(h), layers, E, slots, record_bytes, _ptr(pinned_pool),
                                     _ptr(device_slots), _ptr(expert_slot)))
        self.h = h
        self.E = E

    def lookup(self, layer, ids):
        """ids: sequence of ints. Returns (slot_of_id list, miss_ids list)."""
        n = len(ids)
        arr = (C.c_int32 * max(n, 1))(*ids)
        slot = (C.c_int32 * max(n, 1))()
        miss = (C.c_int32 * max(n, 1))()
        nm = C.c_int(0)
        _check(lib.slot_cache_lookup(self.h, layer, _addr(arr), n, _addr(slot), _addr(miss), C.byref(nm)))
        return list(slot[:n]), list(miss[:nm.value])

    def fill(self, layer, miss_ids, side=None, compute=None):
        n = len(miss_ids)
        arr = (C.c_int32 * max(n, 1))(*miss_ids)
        _check(lib.slot_cache_fill(self.h, layer, _addr(arr), n, _stream(side), _stream(compute)))

    def release(self, layer, compute=None):
        _check(lib.slot_cache_release(self.h, layer, _stream(compute)))

    def plan_waves(self, layer, ids):
        """ids: sequence of ints. Returns the waves as lists of distinct ids."""
        n = len(ids)
        arr = (C.c_int32 * max(n, 1))(*ids)
        wid = (C.c_int32 * max(n, 1))()
        wst = (C.c_int32 * (n + 1))()
        nw = C.c_int(0)
        _check(lib.slot_cache_plan_waves(self.h, layer, _addr(arr), n, _addr(wid), _addr(wst), C.byref(nw)))
        return [list(wid[wst[w]:wst[w + 1]]) for w in range(nw.value)]

    def stats(self):
        h, m, b = C.c_uint64(), C.c_uint64(), C.c_uint64()
        _check(lib.slot_cache_stats(self.h, C.byref(h), C.byref(m), C.byref(b)))
        return {"hits": h.value, "misses": m.value, "h2d_bytes": b.value}

    def inject_fill_failure(self, count):
        _check(lib.slot_cache_inject_fill_failure(self.h, count))

    def close(self):
        if self.h:
            lib.slot_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _info_dict(info):
    return {f: getattr(info, f) for f, _ in moe_pool_info._fields_}


def moe_pool_save(path, layers, E, H, I, record_bytes, pool):
    """Writes the host pool (a tensor, numpy array via its address, or int) to path."""
    info = moe_pool_info(layers, E, H, I, record_bytes)
    addr = pool if isinstance(pool, int) else (pool.ctypes.data if hasattr(pool, "ctypes") else pool.data_ptr())
    _check(lib.moe_pool_save(os.fsencode(path), C.byref(info), addr))


def moe_pool_file_info(path) -> dict:
    info = moe_pool_info()
    _check(lib.moe_pool_file_info(os.fsencode(path), C.byref(info)))
    return _info_dict(info)


def moe_pool_load(path, pool, capacity) -> dict:
    """Reads path's records into the host buffer `pool` of `capacity` bytes."""
    info = moe_pool_info()
    addr = pool if isinstance(pool, int) else (pool.ctypes.data if hasattr(pool, "ctypes") else pool.data_ptr())
    _check(lib.moe_pool_load(os.fsencode(path), addr, capacity, C.byref(info)))
    return _info_dict(info)
