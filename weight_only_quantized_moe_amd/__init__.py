"""Python binding of libhmoe, the hybrid-precision W4A16 fused MoE layer for
AMD MI355X (gfx950).

This module only marshals arguments: every step of the layer runs in the HIP
kernels of ``libhmoe.so``, whose C ABI is declared in ``include/hmoe.h``. The
functions carry the C names. Tensors are torch tensors on the GPU (torch is
used for device memory and for the current HIP stream only). Importing works
without a GPU; calling anything that launches kernels needs one. If the shared
library has not been built, every call raises.

Build the library with ``python -m weight_only_quantized_moe_amd.build``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from ctypes import (POINTER, Structure, byref, c_char_p, c_int32, c_int64, c_size_t,
                    c_void_p)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libhmoe.so")

KEPT_NVFP4, KEPT_MXFP4 = 0, 1
DECODE_STAGED, DECODE_SINGLE_LAUNCH = 0, 1
ACT_16BIT, ACT_MXFP4 = 0, 1
DTYPE_BF16, DTYPE_FP16, DTYPE_FP32 = 0, 1, 2
TIER_KEPT, TIER_NF3 = 0, 1
TENSOR_W13, TENSOR_W2 = 0, 1
STAGE_ROUTE, STAGE_W13, STAGE_W2, STAGE_COMBINE = 0, 1, 2, 3
WEIGHT_NVFP4, WEIGHT_MXFP4, WEIGHT_INT4 = 0, 1, 2
DECODE_MAX_M = 8
TOKENS_MAX_M = 16
MAX_GROUPS = 2048

EXPORTED = (
    "moe_layer_create", "moe_layer_destroy", "moe_layer_query", "moe_scratch_bytes",
    "moe_scratch_init",
    "moe_route", "moe_align", "moe_align_view", "moe_decode_view", "moe_topk_view",
    "hybrid_moe_forward", "hybrid_moe_forward_static", "hybrid_moe_forward_stage", "moe_dequant",
    "moe_repack", "moe_quantize_mxfp4",
    "moe_permute_scratch_bytes", "moe_permute", "moe_permute_backward", "moe_unpermute",
    "moe_unpermute_backward", "moe_route_backward",
    "moe_lora_scratch_bytes", "moe_lora", "moe_lora_backward",
    "moe_linear_scratch_bytes", "moe_linear", "moe_linear_backward",
    "moe_tokens_scratch_bytes", "moe_tokens",
    "moe_status_string", "moe_last_error",
)


class HmoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class LayerDesc(Structure):
    _fields_ = [("num_experts", c_int32), ("hidden", c_int32), ("inter", c_int32),
                ("top_k", c_int32), ("max_tokens", c_int32), ("kept_format", c_int32),
                ("bit_map", c_void_p), ("block_m", c_int32), ("decode_launch", c_int32),
                ("act_format", c_int32)]


class LayerInfo(Structure):
    _fields_ = [(n, c_int32) for n in (
        "num_experts", "hidden", "inter", "top_k", "max_tokens", "kept_format",
        "num_kept", "num_nf3", "block_m", "max_distinct", "cap_kept", "cap_nf3",
        "fused_decode", "single_launch_available", "act_format")]


class Weights(Structure):
    _fields_ = [(n, c_void_p) for n in (
        "kept_w13_q", "kept_w13_s", "kept_w13_g", "kept_w2_q", "kept_w2_s", "kept_w2_g",
        "nf3_w13_q", "nf3_w13_s", "nf3_w2_q", "nf3_w2_s")]


class ExpertSrc(Structure):
    _fields_ = [(n, c_void_p) for n in (
        "w13_q", "w13_hi", "w13_s", "w13_g", "w2_q", "w2_hi", "w2_s", "w2_g")]


class AlignView(Structure):
    _fields_ = [("sorted_slots", c_void_p), ("block_expert", c_void_p), ("expert_off", c_void_p),
                ("num_padded", c_void_p), ("capacity", c_int32), ("num_experts_tier", c_int32)]


class DecodeView(Structure):
    _fields_ = [("counts", c_void_p), ("experts", c_void_p), ("num_slots", c_void_p),
                ("slots", c_void_p), ("expert_tier", c_void_p), ("passes", c_void_p),
                ("max_distinct", c_int32), ("sync_timeouts", c_void_p)]


class Packed(Structure):
    _fields_ = [("format", c_int32), ("group", c_int32), ("q", c_void_p), ("s", c_void_p),
                ("z", c_void_p), ("g", c_void_p)]


class TokensDesc(Structure):
    _fields_ = [*((n, c_int32) for n in ("num_experts", "hidden", "inter", "top_k", "shared_inter",
                                         "dtype")),
                ("router", c_void_p), ("shared_gate", c_void_p),
                *((n, Packed) for n in ("w13", "w2", "shared_w13", "shared_w2"))]


_lib = None


def load_library() -> ctypes.CDLL:
    """Load libhmoe.so (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m weight_only_quantized_moe_amd.build`")
    # torch's HIP runtime first: the library then takes it. Loaded before torch, the library would
    # bring the system's, and of two runtimes in one process the library's finds no device.
    with contextlib.suppress(ImportError):
        import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    st = c_int32
    lib.moe_layer_create.argtypes = [POINTER(LayerDesc), POINTER(c_void_p)]
    lib.moe_layer_create.restype = st
    lib.moe_layer_destroy.argtypes = [c_void_p]
    lib.moe_layer_destroy.restype = None
    lib.moe_layer_query.argtypes = [c_void_p, POINTER(LayerInfo)]
    lib.moe_layer_query.restype = st
    lib.moe_scratch_bytes.argtypes = [c_void_p, POINTER(c_size_t)]
    lib.moe_scratch_bytes.restype = st
    lib.moe_scratch_init.argtypes = [c_void_p, c_void_p, c_size_t, c_void_p]
    lib.moe_scratch_init.restype = st
    lib.moe_route.argtypes = [c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_void_p]
    lib.moe_route.restype = st
    lib.moe_align.argtypes = [c_void_p, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]
    lib.moe_align.restype = st
    lib.moe_align_view.argtypes = [c_void_p, c_void_p, c_int32, POINTER(AlignView)]
    lib.moe_align_view.restype = st
    lib.moe_decode_view.argtypes = [c_void_p, c_void_p, POINTER(DecodeView)]
    lib.moe_decode_view.restype = st
    lib.moe_topk_view.argtypes = [c_void_p, c_void_p, POINTER(c_void_p), POINTER(c_void_p)]
    lib.moe_topk_view.restype = st
    lib.hybrid_moe_forward.argtypes = [c_void_p, POINTER(Weights), c_void_p, c_void_p, c_int32,
                                       c_void_p, c_void_p, c_size_t, c_void_p]
    lib.hybrid_moe_forward.restype = st
    lib.hybrid_moe_forward_static.argtypes = [c_void_p, POINTER(Weights), c_void_p, c_void_p,
                                              c_int32, c_void_p, c_void_p]
    lib.hybrid_moe_forward_static.restype = st
    lib.hybrid_moe_forward_stage.argtypes = [c_void_p, POINTER(Weights), c_void_p, c_void_p, c_int32,
                                             c_void_p, c_void_p, c_size_t, c_int32, c_void_p]
    lib.hybrid_moe_forward_stage.restype = st
    lib.moe_dequant.argtypes = [c_void_p, POINTER(Weights), c_int32, c_int32, c_void_p, c_void_p,
                                c_void_p]
    lib.moe_dequant.restype = st
    lib.moe_repack.argtypes = [c_void_p, POINTER(ExpertSrc), POINTER(Weights), c_void_p]
    lib.moe_repack.restype = st
    lib.moe_quantize_mxfp4.argtypes = [c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p]
    lib.moe_quantize_mxfp4.restype = st
    P, I, L = c_void_p, c_int32, c_int64
    for name, args in {
        "moe_permute_scratch_bytes": [I, I, I, POINTER(c_size_t)],
        "moe_permute": [P, L, P, I, I, I, I, I, P, L, P, P, P, P, c_size_t, P],
        "moe_permute_backward": [P, L, P, I, I, I, I, P, L, P],
        "moe_unpermute": [P, L, P, P, I, I, I, I, P, L, P],
        "moe_unpermute_backward": [P, L, P, L, P, P, I, I, I, I, P, L, P, P],
        "moe_route_backward": [P, P, P, I, I, I, P, P],
        "moe_lora_scratch_bytes": [I, I, I, I, I, POINTER(c_size_t), POINTER(c_size_t)],
        "moe_lora": [P, L, P, P, P, P, I, I, I, I, I, P, L, P, L, P, P, c_size_t, P],
        "moe_lora_backward": [P, L, P, L, P, P, P, P, P, I, I, I, I, I, P, L, P, L, P, P, P, c_size_t, P],
        "moe_linear_scratch_bytes": [I, I, I, POINTER(c_size_t), POINTER(c_size_t)],
        "moe_linear": [P, L, P, I, I, I, I, P, L, P, L, P, c_size_t, P],
        "moe_linear_backward": [P, L, P, I, I, I, I, P, L, P, L, P, c_size_t, P],
        "moe_tokens_scratch_bytes": [I, I, I, I, I, I, POINTER(c_size_t)],
        "moe_tokens": [P, P, L, I, P, L, P, L, P, P, P, c_size_t, P],
    }.items():
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = st
    lib.moe_status_string.argtypes = [c_int32]
    lib.moe_status_string.restype = c_char_p
    lib.moe_last_error.argtypes = []
    lib.moe_last_error.restype = c_char_p
    _lib = lib
    return lib


def _check(status: int) -> None:
    if status != 0:
        lib = load_library()
        raise HmoeError(status, f"{lib.moe_status_string(status).decode()}: "
                                f"{lib.moe_last_error().decode()}")


def _stream(stream):
    if stream is not None:
        return c_void_p(stream)
    import torch
    return c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else c_void_p(t.data_ptr())


def moe_status_string(status: int) -> str:
    return load_library().moe_status_string(status).decode()


def moe_last_error() -> str:
    return load_library().moe_last_error().decode()


class Layer:
    """Owns one hmoe_layer handle (host memory only)."""

    def __init__(self, handle: c_void_p, bit_map):
        self.handle = handle
        self._bit_map = bit_map   # keeps the host bytes alive for the descriptor's lifetime

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.moe_layer_destroy(self.handle)
            self.handle = None


def moe_layer_create(num_experts: int, hidden: int, inter: int, top_k: int, max_tokens: int,
                     kept_format: int = KEPT_NVFP4, bit_map=None, block_m: int = 0,
                     decode_launch: int = DECODE_STAGED, act_format: int = ACT_16BIT) -> Layer:
    lib = load_library()
    bm = None
    if bit_map is not None:
        bm = (ctypes.c_uint8 * num_experts)(*[int(v) for v in bit_map])
    d = LayerDesc(num_experts, hidden, inter, top_k, max_tokens, kept_format,
                  ctypes.cast(bm, c_void_p) if bm is not None else None, block_m, decode_launch,
                  act_format)
    h = c_void_p()
    _check(lib.moe_layer_create(byref(d), byref(h)))
    return Layer(h, bm)


def moe_layer_query(layer: Layer) -> dict:
    info = LayerInfo()
    _check(load_library().moe_layer_query(layer.handle, byref(info)))
    return {n: getattr(info, n) for n, _ in LayerInfo._fields_}


def moe_scratch_bytes(layer: Layer) -> int:
    n = c_size_t()
    _check(load_library().moe_scratch_bytes(layer.handle, byref(n)))
    return n.value


def moe_scratch_init(layer: Layer, scratch, stream=None) -> None:
    """Zero-fills the scratch's decode counters (not needed for a zero-filled buffer)."""
    _check(load_library().moe_scratch_init(layer.handle, _ptr(scratch),
                                           scratch.numel() * scratch.element_size(),
                                           _stream(stream)))


def moe_route(logits, top_k: int, topk_ids, topk_w, stream=None) -> None:
    M, E = logits.shape
    _check(load_library().moe_route(_ptr(logits), M, E, top_k, _ptr(topk_ids), _ptr(topk_w),
                                    _stream(stream)))


def moe_align(layer: Layer, topk_ids, M: int, scratch, stream=None) -> None:
    _check(load_library().moe_align(layer.handle, _ptr(topk_ids), M, _ptr(scratch),
                                    scratch.numel() * scratch.element_size(), _stream(stream)))


def _scratch_view(scratch, ptr: int, count: int, dtype):
    import torch
    off = ptr - scratch.data_ptr()
    esz = torch.empty((), dtype=dtype).element_size()
    return scratch.view(torch.uint8)[off:off + count * esz].view(dtype)


def moe_align_view(layer: Layer, scratch, tier: int) -> dict:
    """Tensors viewing one tier's align arrays inside `scratch` (full capacity)."""
    import torch
    v = AlignView()
    _check(load_library().moe_align_view(layer.handle, _ptr(scratch), tier, byref(v)))
    bm = moe_layer_query(layer)["block_m"]
    return {
        "sorted_slots": _scratch_view(scratch, v.sorted_slots, v.capacity, torch.int32),
        "block_expert": _scratch_view(scratch, v.block_expert, v.capacity // bm, torch.int32),
        "expert_off": _scratch_view(scratch, v.expert_off, v.num_experts_tier + 1, torch.int32),
        "num_padded": _scratch_view(scratch, v.num_padded, 1, torch.int32),
        "capacity": v.capacity,
    }


def moe_decode_view(layer: Layer, scratch) -> dict:
    import torch
    v = DecodeView()
    _check(load_library().moe_decode_view(layer.handle, _ptr(scratch), byref(v)))
    info = moe_layer_query(layer)
    E, k = info["num_experts"], info["top_k"]
    D = v.max_distinct
    n_pass = DECODE_MAX_M * k
    return {
        "counts": _scratch_view(scratch, v.counts, 2, torch.int32),
        "experts": _scratch_view(scratch, v.experts, D, torch.int32),
        "num_slots": _scratch_view(scratch, v.num_slots, D, torch.int32),
        "slots": _scratch_view(scratch, v.slots, D * DECODE_MAX_M, torch.int32).view(D, DECODE_MAX_M),
        "expert_tier": _scratch_view(scratch, v.expert_tier, E, torch.int32),
        # pass records of the first M * k slots of the last decode forward
        "passes": _scratch_view(scratch, v.passes, n_pass * 4, torch.int32).view(n_pass, 4),
        "sync_timeouts": _scratch_view(scratch, v.sync_timeouts, 1, torch.int32),
    }


def moe_topk_view(layer: Layer, scratch, M: int) -> tuple:
    import torch
    ids, w = c_void_p(), c_void_p()
    _check(load_library().moe_topk_view(layer.handle, _ptr(scratch), byref(ids), byref(w)))
    k = moe_layer_query(layer)["top_k"]
    return (_scratch_view(scratch, ids.value, M * k, torch.int32).view(M, k),
            _scratch_view(scratch, w.value, M * k, torch.float32).view(M, k))


def hybrid_moe_forward(layer: Layer, weights: "DeviceWeights", x, router_logits, y, scratch,
                       stream=None) -> None:
    """y[M, H] (bf16) = the hybrid MoE layer applied to x[M, H] (bf16) routed by
    router_logits[M, E] (fp32)."""
    M = x.shape[0]
    _check(load_library().hybrid_moe_forward(
        layer.handle, byref(weights.struct), _ptr(x), _ptr(router_logits), M, _ptr(y),
        _ptr(scratch), scratch.numel() * scratch.element_size(), _stream(stream)))


def hybrid_moe_forward_static(layer: Layer, weights: "DeviceWeights", x, router_logits, y,
                              stream=None) -> None:
    """hybrid_moe_forward with the library's static per-GPU scratch: allocates nothing;
    calls that overlap on one GPU race (see include/hmoe.h)."""
    M = x.shape[0]
    _check(load_library().hybrid_moe_forward_static(
        layer.handle, byref(weights.struct), _ptr(x), _ptr(router_logits), M, _ptr(y),
        _stream(stream)))


def hybrid_moe_forward_stage(layer: Layer, weights: "DeviceWeights", x, router_logits, y, scratch,
                             stage: int, stream=None) -> None:
    """One stage of hybrid_moe_forward (STAGE_ROUTE, _W13, _W2, _COMBINE, in order)."""
    M = x.shape[0]
    _check(load_library().hybrid_moe_forward_stage(
        layer.handle, byref(weights.struct), _ptr(x), _ptr(router_logits), M, _ptr(y),
        _ptr(scratch), scratch.numel() * scratch.element_size(), stage, _stream(stream)))


def moe_dequant(layer: Layer, weights: "DeviceWeights", expert: int, tensor: int,
                out_f32=None, out_bf16=None, stream=None) -> None:
    _check(load_library().moe_dequant(layer.handle, byref(weights.struct), expert, tensor,
                                      _ptr(out_f32), _ptr(out_bf16), _stream(stream)))


def moe_repack(layer: Layer, experts, dst: "DeviceWeights", stream=None) -> None:
    """Load-time demux/repack (include/hmoe.h): `experts` is a list of E dicts of device
    tensors in the checkpoint layout (kept tier: w13_q, w13_s, w13_g, w2_q, w2_s, w2_g;
    NF3 tier: w13_lo, w13_hi, w13_s, w2_lo, w2_hi, w2_s), written into the tier-local
    arrays of `dst`."""
    info = moe_layer_query(layer)
    if len(experts) != info["num_experts"]:
        raise ValueError(f"moe_repack: {len(experts)} experts given, the layer has "
                         f"{info['num_experts']}")
    arr = (ExpertSrc * len(experts))()
    for i, ex in enumerate(experts):
        nf3 = "w13_lo" in ex
        arr[i] = ExpertSrc(
            _ptr(ex["w13_lo"] if nf3 else ex["w13_q"]), _ptr(ex.get("w13_hi")), _ptr(ex["w13_s"]),
            _ptr(ex.get("w13_g")), _ptr(ex["w2_lo"] if nf3 else ex["w2_q"]), _ptr(ex.get("w2_hi")),
            _ptr(ex["w2_s"]), _ptr(ex.get("w2_g")))
    _check(load_library().moe_repack(layer.handle, arr, byref(dst.struct), _stream(stream)))


def moe_quantize_mxfp4(x, codes, scales, stream=None) -> None:
    """x fp32 [rows, K] -> MXFP4 codes u8 [rows, K/2] and E8M0 scales u8 [rows, K/32]."""
    rows, K = x.shape
    _check(load_library().moe_quantize_mxfp4(_ptr(x), rows, K, _ptr(codes), _ptr(scales),
                                             _stream(stream)))


# ---- operators around the experts ---------------------------------------------------
#
# Small calls take a few microseconds on the GPU, so the checks below are written to cost
# little on the host: no strings or containers are built unless a check fails.

_torch = None
_CODES = {}
_I32 = _F32 = None
_this_device = _raw_stream = None
_functions = {}


def _load_torch():
    global _torch, _I32, _F32, _this_device, _raw_stream
    import torch
    _I32, _F32 = torch.int32, torch.float32
    _this_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    # int16 holds bf16 bits, as for the layer
    _CODES.update({torch.bfloat16: DTYPE_BF16, torch.int16: DTYPE_BF16, torch.float16: DTYPE_FP16,
                   torch.float32: DTYPE_FP32})
    _torch = torch  # last: a thread that finds it set finds the rest


def _dtype_code(t) -> int:
    """Element type of a rows tensor."""
    if _torch is None:
        _load_torch()
    code = _CODES.get(t.dtype)
    if code is None:
        raise ValueError(f"rows of {t.dtype}: expected bfloat16 (or its bits as int16), float16 "
                         "or float32")
    return code


def _matrix(name: str, t, shape: tuple, code: int) -> int:
    """Checks a matrix of the given shape and element type; returns its row stride."""
    if t.shape != shape or _CODES.get(t.dtype) != code:
        raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)}, expected {list(shape)} of the "
                         "operator's row type")
    if t.is_contiguous():
        return shape[1]
    s = t.stride()
    if s[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return s[0] if shape[0] > 1 else shape[1]


def _refuse(shape: tuple, dtype, **tensors) -> None:
    """Names the first tensor that is not contiguous, of this shape and type."""
    for name, t in tensors.items():
        if t is None:
            raise ValueError(f"{name} is missing")
        if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
            raise ValueError(f"{name} is {t.dtype} {tuple(t.shape)} (strides {t.stride()}), expected "
                             f"contiguous {dtype} {tuple(shape)}")


def _at(t):
    return None if t is None else t.data_ptr()


def _launch(function: str, stream, tensors, *args) -> None:
    """Calls a C function on the tensors' device: its stream argument is the given one, else
    that device's current stream. Tensors on different devices, or not on a GPU, are refused."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("all tensors of a call must be on one GPU")
    if dev < 0:
        raise ValueError("all tensors of a call must be on one GPU")
    fn = _functions.get(function)
    if fn is None:
        fn = _functions[function] = getattr(load_library(), function)
    if _this_device() == dev:
        status = fn(*args, _raw_stream(dev) if stream is None else stream)
    else:
        with _torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev) if stream is None else stream)
    if status:
        _check(status)


def _room(scratch) -> tuple:
    """Address and bytes of an optional scratch tensor."""
    if scratch is None:
        return None, 0
    if not scratch.is_contiguous():
        raise ValueError("scratch must be contiguous")
    return scratch.data_ptr(), scratch.nbytes


def moe_permute_scratch_bytes(M: int, top_k: int, num_experts: int) -> int:
    n = c_size_t()
    _check(load_library().moe_permute_scratch_bytes(M, top_k, num_experts, byref(n)))
    return n.value


def moe_permute(x, topk_ids, num_experts: int, rows, sorted_slots, slot_row, expert_off,
                scratch=None, stream=None) -> None:
    """x[M, H] into expert order: rows[M * k, H], sorted_slots i32 [M * k], slot_row i32
    [M, k] and expert_off i32 [E + 1] (see include/hmoe.h). Ids outside [0, E) are dropped."""
    code = _dtype_code(x)
    shape = topk_ids.shape
    M, k = shape
    n, H = M * k, x.shape[-1]
    xs, rs = _matrix("x", x, (M, H), code), _matrix("rows", rows, (n, H), code)
    if not (topk_ids.dtype is _I32 and topk_ids.is_contiguous() and slot_row.dtype is _I32
            and slot_row.shape == shape and slot_row.is_contiguous()):
        _refuse(shape, _I32, topk_ids=topk_ids, slot_row=slot_row)
    if not (sorted_slots.dtype is _I32 and sorted_slots.shape == (n,) and sorted_slots.is_contiguous()):
        _refuse((n,), _I32, sorted_slots=sorted_slots)
    if not (expert_off.dtype is _I32 and expert_off.shape == (num_experts + 1,)
            and expert_off.is_contiguous()):
        _refuse((num_experts + 1,), _I32, expert_off=expert_off)
    ws, nbytes = _room(scratch)
    _launch("moe_permute", stream, (x, topk_ids, rows, sorted_slots, slot_row, expert_off, scratch),
            x.data_ptr(), xs, topk_ids.data_ptr(), M, k, num_experts, H, code, rows.data_ptr(), rs,
            sorted_slots.data_ptr(), slot_row.data_ptr(), expert_off.data_ptr(), ws, nbytes)


def moe_permute_backward(drows, slot_row, dx, stream=None) -> None:
    """dx[M, H] = for each token the sum of its slots' drows[M * k, H]."""
    code = _dtype_code(drows)
    shape = slot_row.shape
    M, k = shape
    H = drows.shape[-1]
    ds, xs = _matrix("drows", drows, (M * k, H), code), _matrix("dx", dx, (M, H), code)
    if not (slot_row.dtype is _I32 and slot_row.is_contiguous()):
        _refuse(shape, _I32, slot_row=slot_row)
    _launch("moe_permute_backward", stream, (drows, slot_row, dx), drows.data_ptr(), ds,
            slot_row.data_ptr(), M, k, H, code, dx.data_ptr(), xs)


def moe_unpermute(rows, slot_row, topk_w, y, stream=None) -> None:
    """y[M, H] = for each token the sum of its slots' rows[M * k, H] times topk_w f32 [M, k]."""
    code = _dtype_code(rows)
    shape = slot_row.shape
    M, k = shape
    H = rows.shape[-1]
    rs, ys = _matrix("rows", rows, (M * k, H), code), _matrix("y", y, (M, H), code)
    if not (slot_row.dtype is _I32 and slot_row.is_contiguous()):
        _refuse(shape, _I32, slot_row=slot_row)
    if not (topk_w.dtype is _F32 and topk_w.shape == shape and topk_w.is_contiguous()):
        _refuse(shape, _F32, topk_w=topk_w)
    _launch("moe_unpermute", stream, (rows, slot_row, topk_w, y), rows.data_ptr(), rs,
            slot_row.data_ptr(), topk_w.data_ptr(), M, k, H, code, y.data_ptr(), ys)


def moe_unpermute_backward(dy, rows, slot_row, topk_w, drows, dw, stream=None) -> None:
    """Gradients of moe_unpermute: drows[M * k, H] (rows no slot names stay as they were) and
    dw f32 [M, k]."""
    code = _dtype_code(rows)
    shape = slot_row.shape
    M, k = shape
    n, H = M * k, rows.shape[-1]
    ys, rs = _matrix("dy", dy, (M, H), code), _matrix("rows", rows, (n, H), code)
    ds = _matrix("drows", drows, (n, H), code)
    if not (slot_row.dtype is _I32 and slot_row.is_contiguous()):
        _refuse(shape, _I32, slot_row=slot_row)
    if not (topk_w.dtype is _F32 and topk_w.shape == shape and topk_w.is_contiguous()
            and dw.dtype is _F32 and dw.shape == shape and dw.is_contiguous()):
        _refuse(shape, _F32, topk_w=topk_w, dw=dw)
    _launch("moe_unpermute_backward", stream, (dy, rows, slot_row, topk_w, drows, dw), dy.data_ptr(),
            ys, rows.data_ptr(), rs, slot_row.data_ptr(), topk_w.data_ptr(), M, k, H, code,
            drows.data_ptr(), ds, dw.data_ptr())


def moe_route_backward(topk_ids, topk_w, dw, dlogits, stream=None) -> None:
    """dlogits f32 [M, E] (fully overwritten) from moe_route's ids and weights and dw f32 [M, k]."""
    if _torch is None:
        _load_torch()
    shape = topk_ids.shape
    M, k = shape
    E = dlogits.shape[-1]
    if not (topk_ids.dtype is _I32 and topk_ids.is_contiguous()):
        _refuse(shape, _I32, topk_ids=topk_ids)
    if not (topk_w.dtype is _F32 and topk_w.shape == shape and topk_w.is_contiguous()
            and dw.dtype is _F32 and dw.shape == shape and dw.is_contiguous()):
        _refuse(shape, _F32, topk_w=topk_w, dw=dw)
    if not (dlogits.dtype is _F32 and dlogits.shape == (M, E) and dlogits.is_contiguous()):
        _refuse((M, E), _F32, dlogits=dlogits)
    _launch("moe_route_backward", stream, (topk_ids, topk_w, dw, dlogits), topk_ids.data_ptr(),
            topk_w.data_ptr(), dw.data_ptr(), M, E, k, dlogits.data_ptr())


def moe_lora_scratch_bytes(M: int, num_adapters: int, K: int, N: int, rank: int) -> tuple:
    """Scratch bytes of moe_lora and of moe_lora_backward for any call of at most M rows."""
    f, b = c_size_t(), c_size_t()
    _check(load_library().moe_lora_scratch_bytes(M, num_adapters, K, N, rank, byref(f), byref(b)))
    return f.value, b.value


def _adapters(M: int, ids, A, B, scale) -> tuple:
    a, b = A.shape, B.shape
    if len(a) != 3 or len(b) != 3 or a[0] != b[0] or a[1] != b[2]:
        raise ValueError(f"A {tuple(a)} and B {tuple(b)}: expected [G, rank, K] and [G, N, rank]")
    if (_dtype_code(A) != DTYPE_BF16 or _dtype_code(B) != DTYPE_BF16 or not A.is_contiguous()
            or not B.is_contiguous()):
        raise ValueError("A and B must be contiguous bfloat16")
    if not (ids.dtype is _I32 and ids.shape == (M,) and ids.is_contiguous()):
        _refuse((M,), _I32, ids=ids)
    if not (scale.dtype is _F32 and scale.shape == (a[0],) and scale.is_contiguous()):
        _refuse((a[0],), _F32, scale=scale)
    return a[0], a[1], a[2], b[1]


def moe_lora(x, ids, A, B, scale, base, y, z=None, scratch=None, stream=None) -> None:
    """y[M, N] = base + scale[g] * B[g] (A[g] x) with g = ids[m]; A bf16 [G, rank, K], B bf16
    [G, N, rank], scale f32 [G]. base may be None (zeros) or y itself; z f32 [M, rank]
    receives A[g] x for moe_lora_backward. Ids outside [0, G): no adapter."""
    M = x.shape[0]
    G, r, K, N = _adapters(M, ids, A, B, scale)
    xs, ys = _matrix("x", x, (M, K), DTYPE_BF16), _matrix("y", y, (M, N), DTYPE_BF16)
    bs = 0 if base is None else _matrix("base", base, (M, N), DTYPE_BF16)
    if z is not None and not (z.dtype is _F32 and z.shape == (M, r) and z.is_contiguous()):
        _refuse((M, r), _F32, z=z)
    ws, nbytes = _room(scratch)
    _launch("moe_lora", stream, (x, ids, A, B, scale, base, y, z, scratch), x.data_ptr(), xs,
            ids.data_ptr(), A.data_ptr(), B.data_ptr(), scale.data_ptr(), M, G, K, N, r, _at(base),
            bs, y.data_ptr(), ys, _at(z), ws, nbytes)


def moe_lora_backward(dy, x, z, ids, A, B, scale, dbase, dx, dA, dB, scratch=None,
                      stream=None) -> None:
    """Gradients of moe_lora: dx[M, K] = dbase + A[g]^T dz, dA f32 [G, rank, K] and dB f32
    [G, N, rank] (fully overwritten). dbase may be None (zeros) or dx itself."""
    M = x.shape[0]
    G, r, K, N = _adapters(M, ids, A, B, scale)
    ys, xs = _matrix("dy", dy, (M, N), DTYPE_BF16), _matrix("x", x, (M, K), DTYPE_BF16)
    ds = _matrix("dx", dx, (M, K), DTYPE_BF16)
    bs = 0 if dbase is None else _matrix("dbase", dbase, (M, K), DTYPE_BF16)
    _refuse((M, r), _F32, z=z)
    _refuse((G, r, K), _F32, dA=dA)
    _refuse((G, N, r), _F32, dB=dB)
    ws, nbytes = _room(scratch)
    _launch("moe_lora_backward", stream, (dy, x, z, ids, A, B, scale, dbase, dx, dA, dB, scratch),
            dy.data_ptr(), ys, x.data_ptr(), xs, z.data_ptr(), ids.data_ptr(), A.data_ptr(),
            B.data_ptr(), scale.data_ptr(), M, G, K, N, r, _at(dbase), bs, dx.data_ptr(), ds,
            dA.data_ptr(), dB.data_ptr(), ws, nbytes)


# ---- matrices of 4-bit weights with group scales ---------------------------------------

class PackedMatrix:
    """A matrix of 4-bit weights on the GPU, [N, K] or several of them [E, N, K]; keeps its tensors.

    q u8 [..., N, K/2]; s: NVFP4 u8 (or float8_e4m3fn) [..., N, K/16], MXFP4 u8 [..., N, K/32], INT4
    bfloat16 or float16 [..., N, K/group]; z (INT4) u8 of s's shape or None; g (NVFP4) f32 with one
    value per matrix (see include/hmoe.h)."""

    def __init__(self, format: int, q, s, z=None, g=None, group: int = 0):
        if _torch is None:
            _load_torch()
        torch = _torch
        if format not in (WEIGHT_NVFP4, WEIGHT_MXFP4, WEIGHT_INT4):
            raise ValueError(f"unknown format {format}")
        if q.dim() not in (2, 3):
            raise ValueError(f"q is {tuple(q.shape)}, expected [N, K/2] or [E, N, K/2]")
        if format == WEIGHT_INT4 and group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        self.group = {WEIGHT_NVFP4: 16, WEIGHT_MXFP4: 32}.get(format, group)
        self.format, self.lead = format, tuple(q.shape[:-2])
        self.rows, self.cols = q.shape[-2], 2 * q.shape[-1]
        if self.cols % max(32, self.group):
            raise ValueError(f"{self.cols} columns, expected a multiple of {max(32, self.group)}")
        groups = (*q.shape[:-1], self.cols // self.group)
        if q.dtype is not torch.uint8 or not q.is_contiguous():
            _refuse(q.shape, torch.uint8, q=q)
        if format == WEIGHT_INT4:
            if s.dtype not in (torch.bfloat16, torch.float16):
                raise ValueError(f"s is {s.dtype}, expected bfloat16 or float16")
            _refuse(groups, s.dtype, s=s)
            if z is not None:
                _refuse(groups, torch.uint8, z=z)
        else:
            if format == WEIGHT_NVFP4 and s.dtype is torch.float8_e4m3fn:
                s = s.view(torch.uint8)
            _refuse(groups, torch.uint8, s=s)
            z = None
        if format == WEIGHT_NVFP4:
            if g is None or g.dtype is not _F32 or g.numel() != (self.lead[0] if self.lead else 1) \
                    or not g.is_contiguous():
                raise ValueError("g must be contiguous float32 with one value per matrix")
        else:
            g = None
        # the type of activations it takes: INT4's scales fix it
        self.code = _CODES[s.dtype] if format == WEIGHT_INT4 else None
        self.tensors = (q, s, z, g)
        self.struct = Packed(format, self.group, _at(q), _at(s), _at(z), _at(g))
        self._ref = byref(self.struct)

    def _takes(self, name: str, code: int) -> None:
        if code == DTYPE_FP32 or (self.code is not None and self.code != code):
            raise ValueError(f"{name}: activations must be bfloat16 or float16, and of the type of "
                             "INT4 scales")


def _addend(name: str, t, shape: tuple, code: int) -> int:
    """Row stride of an addend, which may be one row for all (expanded)."""
    if t.shape == shape and _CODES.get(t.dtype) == code and t.stride(0) == 0 and shape[0] > 1 \
            and t.stride(1) == 1:
        return 0
    return _matrix(name, t, shape, code)


def moe_linear_scratch_bytes(M: int, K: int, N: int) -> tuple:
    """Bytes of scratch of (moe_linear, moe_linear_backward) for a matrix [N, K]."""
    f, b = c_size_t(), c_size_t()
    _check(load_library().moe_linear_scratch_bytes(M, K, N, byref(f), byref(b)))
    return f.value, b.value


def moe_linear(x, w: PackedMatrix, y, base=None, scratch=None, stream=None) -> None:
    """y[M, N] = base + x[M, K] W^T for a packed W [N, K]; base may be None (zeros), y itself, or
    one row for all (a bias, expanded to [M, N])."""
    code = _dtype_code(x)
    w._takes("moe_linear", code)
    if w.lead:
        raise ValueError("moe_linear takes one matrix")
    M, N, K = x.shape[0], w.rows, w.cols
    xs, ys = _matrix("x", x, (M, K), code), _matrix("y", y, (M, N), code)
    bs = 0 if base is None else _addend("base", base, (M, N), code)
    ws, nbytes = _room(scratch)
    _launch("moe_linear", stream, (x, *w.tensors, base, y, scratch), x.data_ptr(), xs, w._ref, M, K, N,
            code, _at(base), bs, y.data_ptr(), ys, ws, nbytes)


def moe_linear_backward(dy, w: PackedMatrix, dx, dbase=None, scratch=None, stream=None) -> None:
    """Gradient of moe_linear: dx[M, K] = dbase + dy[M, N] W; dbase as base there."""
    code = _dtype_code(dy)
    w._takes("moe_linear_backward", code)
    if w.lead:
        raise ValueError("moe_linear_backward takes one matrix")
    M, N, K = dy.shape[0], w.rows, w.cols
    ys, xs = _matrix("dy", dy, (M, N), code), _matrix("dx", dx, (M, K), code)
    bs = 0 if dbase is None else _addend("dbase", dbase, (M, K), code)
    ws, nbytes = _room(scratch)
    _launch("moe_linear_backward", stream, (dy, *w.tensors, dbase, dx, scratch), dy.data_ptr(), ys,
            w._ref, M, K, N, code, _at(dbase), bs, dx.data_ptr(), xs, ws, nbytes)


def moe_tokens_scratch_bytes(M: int, num_experts: int, hidden: int, inter: int, top_k: int,
                             shared_inter: int = 0) -> int:
    n = c_size_t()
    _check(load_library().moe_tokens_scratch_bytes(M, num_experts, hidden, inter, top_k, shared_inter,
                                                   byref(n)))
    return n.value


def moe_tokens(x, router, w13: PackedMatrix, w2: PackedMatrix, top_k: int, y, base=None, shared=None,
               topk_ids=None, topk_w=None, scratch=None, stream=None) -> None:
    """y[M, H] = base + the layer's output for M <= 16 tokens x[M, H]: router [E, H], experts w13
    [E, 2I, H] and w2 [E, H, I], shared = (w13 [2S, H], w2 [H, S], gate [H] or None) or None.
    topk_ids i32 [M, k] and topk_w f32 [M, k] receive the routing if given."""
    code = _dtype_code(x)
    M, H = x.shape
    if len(w13.lead) != 1 or w2.lead != w13.lead or w13.cols != H or w2.rows != H \
            or w13.rows != 2 * w2.cols:
        raise ValueError("w13 must be [E, 2I, H] and w2 [E, H, I]")
    E, I = w13.lead[0], w2.cols
    s13, s2, gate, S = None, None, None, 0
    mats = (w13, w2)
    if shared is not None:
        s13, s2, gate = shared
        S = s2.cols
        if s13.lead or s2.lead or s13.cols != H or s2.rows != H or s13.rows != 2 * S:
            raise ValueError("the shared expert must be [2S, H] and [H, S]")
        mats = (w13, w2, s13, s2)
    for m in mats:
        m._takes("moe_tokens", code)
    for name, t, shape in (("router", router, (E, H)), ("shared gate", gate, (H,))):
        if (t is not None or name == "router") and (t.shape != shape or _CODES.get(t.dtype) != code
                                                    or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous {list(shape)} of the activations' type")
    xs, ys = _matrix("x", x, (M, H), code), _matrix("y", y, (M, H), code)
    bs = 0 if base is None else _addend("base", base, (M, H), code)
    if topk_ids is not None:
        _refuse((M, top_k), _I32, topk_ids=topk_ids)
    if topk_w is not None:
        _refuse((M, top_k), _F32, topk_w=topk_w)
    none = Packed()
    d = TokensDesc(E, H, I, top_k, S, code, router.data_ptr(), _at(gate), w13.struct, w2.struct,
                   s13.struct if S else none, s2.struct if S else none)
    ws, nbytes = _room(scratch)
    _launch("moe_tokens", stream, (x, router, gate, base, y, topk_ids, topk_w, scratch,
                                   *(t for m in mats for t in m.tensors)),
            byref(d), x.data_ptr(), xs, M, _at(base), bs, y.data_ptr(), ys, _at(topk_ids), _at(topk_w),
            ws, nbytes)


class DeviceWeights:
    """Packed tier weights on the GPU (torch tensors) plus the hmoe_weights struct
    pointing at them. Built from the packed-layer dict layout (see include/hmoe.h)."""

    KEYS = {"kept": ("w13_q", "w13_s", "w13_g", "w2_q", "w2_s", "w2_g"),
            "nf3": ("w13_q", "w13_s", "w2_q", "w2_s")}

    def __init__(self, packed: dict, device="cuda"):
        import numpy as np
        import torch
        self.tensors = {}
        for tier, keys in self.KEYS.items():
            for k in keys:
                arr = packed[tier][k]
                if arr.size == 0:
                    self.tensors[f"{tier}_{k}"] = None
                    continue
                a = np.ascontiguousarray(arr)
                if a.dtype == np.uint16:
                    a = a.view(np.int16)
                self.tensors[f"{tier}_{k}"] = torch.from_numpy(a).to(device)
        self._rebuild()

    def _rebuild(self):
        self.struct = Weights(*[_ptr(self.tensors[n]) for n, _ in Weights._fields_])

    def clone(self) -> "DeviceWeights":
        """A second device copy of the same bytes (for benchmarks that rotate copies)."""
        other = DeviceWeights.__new__(DeviceWeights)
        other.tensors = {k: (None if v is None else v.clone()) for k, v in self.tensors.items()}
        other._rebuild()
        return other

    def nbytes(self) -> int:
        return sum(0 if v is None else v.numel() * v.element_size() for v in self.tensors.values())
