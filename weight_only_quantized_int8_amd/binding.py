"""Thin ctypes binding of libint8w.so (include/int8w.h).

Argument marshalling only: every computation runs in the library's HIP
kernels.  PyTorch provides device memory and the current stream.  If the
library has not been built, loading it raises -- there is no fallback.

The checks in :class:`Int8Weight` follow the rustdoc page "MlxInt8Weight",
method load: the weight must be a 2-D 32-bit tensor, scales and biases BF16
of shape [out_features, in_features / group_size], and group_size must divide
in_features.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libint8w.so")

INT8W_OK = 0
INT8W_ERR_NULL = -1
INT8W_ERR_SHAPE = -2
INT8W_ERR_UNSUPPORTED = -3
INT8W_ERR_ALIGN = -4
INT8W_ERR_ALIAS = -5
INT8W_ERR_HIP = -6
ERROR_NAMES = {
    INT8W_ERR_NULL: "INT8W_ERR_NULL",
    INT8W_ERR_SHAPE: "INT8W_ERR_SHAPE",
    INT8W_ERR_UNSUPPORTED: "INT8W_ERR_UNSUPPORTED",
    INT8W_ERR_ALIGN: "INT8W_ERR_ALIGN",
    INT8W_ERR_ALIAS: "INT8W_ERR_ALIAS",
    INT8W_ERR_HIP: "INT8W_ERR_HIP",
}

EXPORTED = (
    "int8w_validate", "int8w_storage_bytes", "int8_dequantize_to", "int8_gemv", "int8_gemv_silu_gate",
    "int8_gemv_silu_gate_resid", "int8_gemm", "int8_gemv_multi", "int8_quantize", "int8_moe_gemv",
    "int8w_fp8_gemv", "int8w_last_error", "int8_gemm_workspace_bytes", "int8_gemm_ws", "int8_gemm_noalloc",
    "int8w_mxfp4_quantize", "int8w_mxfp4_dequantize_to", "int8w_mxfp4_gemm", "int8w_mxfp4_gemm_mx",
    "int8w_moe_workspace_bytes", "int8_moe_layer", "int8w_mxfp4_moe_layer", "int8w_moe_route",
    "int8_moe_layer_routed", "int8w_mxfp4_moe_layer_routed", "int8w_lora_workspace_bytes", "int8w_lora_add",
)
# calibration streams declared in include/int8w_measure.h
EXPORTED_MEASURE = ("int8w_stream_read", "int8w_stream_copy", "int8w_stream_expand")
FP8_PER_ROW, FP8_BLOCK_BF16, FP8_BLOCK_F32, FP8_SINGLE = 0, 1, 2, 3  # INT8W_FP8_*
VALUES_BF16, VALUES_F32 = 0, 1  # INT8W_VALUES_*
MAX_MOE_EXPERTS, MAX_MOE_TOPK = 512, 16  # INT8W_MAX_MOE_EXPERTS, INT8W_MAX_MOE_TOPK
MAX_MULTI = 4  # INT8W_MAX_MULTI
MAX_MOE_GROUPS = 64  # INT8W_MAX_MOE_GROUPS
MAX_LORA_RANK = 256  # INT8W_MAX_LORA_RANK
MAX_LORA_ROWS = 1 << 20  # of a call
ROUTE_SCORING = {"softmax": 0, "sigmoid": 1}  # INT8W_ROUTE_*
GROUP_SCORES = {"max": 0, "top2": 1}  # INT8W_GROUP_*
MAX_MOE_SLOTS = 65536  # INT8W_MAX_MOE_SLOTS


class Int8wError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"{ERROR_NAMES.get(code, code)}: {message}")
        self.code = code
        self.message = message


class WeightDesc(ctypes.Structure):
    """Mirror of ``int8w_weight`` (include/int8w.h)."""
    _fields_ = [
        ("packed", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("biases", ctypes.c_void_p),
        ("out_features", ctypes.c_uint32),
        ("in_features", ctypes.c_uint32),
        ("group_size", ctypes.c_uint32),
    ]


class Fp8WeightDesc(ctypes.Structure):
    """Mirror of ``int8w_fp8_weight`` (include/int8w.h)."""
    _fields_ = [
        ("weight", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("n", ctypes.c_uint32),
        ("k", ctypes.c_uint32),
        ("scale_format", ctypes.c_uint32),
        ("block_size", ctypes.c_uint32),
        ("single_scale", ctypes.c_float),
    ]


class Mxfp4Desc(ctypes.Structure):
    """Mirror of ``int8w_mxfp4`` (include/int8w.h)."""
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("rows", ctypes.c_uint32),
        ("k", ctypes.c_uint32),
    ]


class MoeCall(ctypes.Structure):
    """Mirror of ``int8w_moe_call`` (include/int8w.h)."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("logits", ctypes.c_void_p),
        ("x_resid", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("tokens", ctypes.c_uint32),
        ("topk", ctypes.c_uint32),
        ("logits_format", ctypes.c_uint32),
        ("renormalize", ctypes.c_uint32),
        ("routed_scale", ctypes.c_float),
    ]


class RouteCall(ctypes.Structure):
    """Mirror of ``int8w_route_call`` (include/int8w.h)."""
    _fields_ = [
        ("logits", ctypes.c_void_p),
        ("bias", ctypes.c_void_p),
        ("ids", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("tokens", ctypes.c_uint32),
        ("num_experts", ctypes.c_uint32),
        ("topk", ctypes.c_uint32),
        ("logits_format", ctypes.c_uint32),
        ("scoring", ctypes.c_uint32),
        ("groups", ctypes.c_uint32),
        ("topk_groups", ctypes.c_uint32),
        ("group_score", ctypes.c_uint32),
        ("renormalize", ctypes.c_uint32),
        ("routed_scale", ctypes.c_float),
    ]


class MoeRoutedCall(ctypes.Structure):
    """Mirror of ``int8w_moe_routed_call`` (include/int8w.h)."""
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("ids", ctypes.c_void_p),
        ("weights", ctypes.c_void_p),
        ("x_resid", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("tokens", ctypes.c_uint32),
        ("topk", ctypes.c_uint32),
    ]


class LoraDesc(ctypes.Structure):
    """Mirror of ``int8w_lora`` (include/int8w.h)."""
    _fields_ = [
        ("a", ctypes.c_void_p),
        ("b", ctypes.c_void_p),
        ("scales", ctypes.c_void_p),
        ("ranks", ctypes.c_void_p),
        ("num_adapters", ctypes.c_uint32),
        ("rank", ctypes.c_uint32),
        ("in_features", ctypes.c_uint32),
        ("out_features", ctypes.c_uint32),
    ]


class LoraOut(ctypes.Structure):
    """Mirror of ``int8w_lora_out`` (include/int8w.h)."""
    _fields_ = [
        ("base", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("base_stride", ctypes.c_uint64),
        ("y_stride", ctypes.c_uint64),
    ]


_ROUTE_CALL = struct.Struct("PPPP9If")  # int8w_route_call
_LORA_OUT = struct.Struct("PPQQ")  # int8w_lora_out
assert _ROUTE_CALL.size == ctypes.sizeof(RouteCall) and _LORA_OUT.size == ctypes.sizeof(LoraOut)

_lib = None


def library_path() -> str:
    return _LIB_PATH


def load_library() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            f"{_LIB_PATH} is not built; run `python -m weight_only_quantized_int8_amd.build` "
            "(the HIP library is required: there is no CPU fallback)")
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.c_void_p
    W = ctypes.POINTER(WeightDesc)
    u64 = ctypes.c_uint64
    lib.int8w_validate.argtypes = [W]
    lib.int8w_validate.restype = ctypes.c_int
    lib.int8w_storage_bytes.argtypes = [ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32]
    lib.int8w_storage_bytes.restype = ctypes.c_uint64
    lib.int8_dequantize_to.argtypes = [W, P, u64]
    lib.int8_dequantize_to.restype = ctypes.c_int
    lib.int8_gemv.argtypes = [W, P, P, u64]
    lib.int8_gemv.restype = ctypes.c_int
    lib.int8_gemv_silu_gate.argtypes = [W, P, P, P, u64]
    lib.int8_gemv_silu_gate.restype = ctypes.c_int
    lib.int8_gemv_silu_gate_resid.argtypes = [W, P, P, P, P, u64]
    lib.int8_gemv_silu_gate_resid.restype = ctypes.c_int
    lib.int8_gemm.argtypes = [W, P, P, ctypes.c_uint32, u64]
    lib.int8_gemm.restype = ctypes.c_int
    lib.int8_gemv_multi.argtypes = [W, ctypes.c_uint32, P, ctypes.POINTER(P), u64]
    lib.int8_gemv_multi.restype = ctypes.c_int
    u32 = ctypes.c_uint32
    lib.int8_quantize.argtypes = [P, u32, u32, u32, P, P, P, u64]
    lib.int8_quantize.restype = ctypes.c_int
    lib.int8_moe_gemv.argtypes = [W, u32, P, u32, P, u32, u32, P, u64]
    lib.int8_moe_gemv.restype = ctypes.c_int
    lib.int8w_fp8_gemv.argtypes = [ctypes.POINTER(Fp8WeightDesc), P, P, u64]
    lib.int8w_fp8_gemv.restype = ctypes.c_int
    lib.int8_gemm_workspace_bytes.argtypes = [W, ctypes.c_uint32]
    lib.int8_gemm_workspace_bytes.restype = ctypes.c_uint64
    lib.int8_gemm_ws.argtypes = [W, P, P, ctypes.c_uint32, P, u64, u64]
    lib.int8_gemm_ws.restype = ctypes.c_int
    lib.int8_gemm_noalloc.argtypes = [W, P, P, ctypes.c_uint32, u64]
    lib.int8_gemm_noalloc.restype = ctypes.c_int
    M = ctypes.POINTER(Mxfp4Desc)
    C = ctypes.POINTER(MoeCall)
    lib.int8w_mxfp4_quantize.argtypes = [P, u32, u32, u32, P, P, u64]
    lib.int8w_mxfp4_quantize.restype = ctypes.c_int
    lib.int8w_mxfp4_dequantize_to.argtypes = [M, P, u64]
    lib.int8w_mxfp4_dequantize_to.restype = ctypes.c_int
    lib.int8w_mxfp4_gemm.argtypes = [M, P, P, u32, u64]
    lib.int8w_mxfp4_gemm.restype = ctypes.c_int
    lib.int8w_mxfp4_gemm_mx.argtypes = [M, M, P, u64]
    lib.int8w_mxfp4_gemm_mx.restype = ctypes.c_int
    lib.int8w_moe_workspace_bytes.argtypes = [u32, u32, u32, u32]
    lib.int8w_moe_workspace_bytes.restype = u64
    lib.int8_moe_layer.argtypes = [W, W, W, u32, C, P, u64, u64]
    lib.int8_moe_layer.restype = ctypes.c_int
    lib.int8w_mxfp4_moe_layer.argtypes = [M, M, M, u32, C, P, u64, u64]
    lib.int8w_mxfp4_moe_layer.restype = ctypes.c_int
    lib.int8w_moe_route.argtypes = [ctypes.POINTER(RouteCall), u64]
    lib.int8w_moe_route.restype = ctypes.c_int
    G = ctypes.POINTER(MoeRoutedCall)
    lib.int8_moe_layer_routed.argtypes = [W, W, W, u32, G, P, u64, u64]
    lib.int8_moe_layer_routed.restype = ctypes.c_int
    lib.int8w_mxfp4_moe_layer_routed.argtypes = [M, M, M, u32, G, P, u64, u64]
    lib.int8w_mxfp4_moe_layer_routed.restype = ctypes.c_int
    L = ctypes.POINTER(LoraDesc)
    lib.int8w_lora_workspace_bytes.argtypes = [L, u32, u32]
    lib.int8w_lora_workspace_bytes.restype = u64
    lib.int8w_lora_add.argtypes = [L, ctypes.POINTER(LoraOut), u32, P, u64, P, u32, P, u64, u64]
    lib.int8w_lora_add.restype = ctypes.c_int
    # The same entries for argument blocks packed as bytes: filling a ctypes structure by its fields took 1.5 us
    # of a routing call's 8, and packing takes 0.4.
    lib.packed_route = lib["int8w_moe_route"]
    lib.packed_route.argtypes, lib.packed_route.restype = [P, u64], ctypes.c_int
    lib.packed_lora_bytes = lib["int8w_lora_workspace_bytes"]
    lib.packed_lora_bytes.argtypes, lib.packed_lora_bytes.restype = [P, u32, u32], u64
    lib.packed_lora_add = lib["int8w_lora_add"]
    lib.packed_lora_add.argtypes = [P, P, u32, P, u64, P, u32, P, u64, u64]
    lib.packed_lora_add.restype = ctypes.c_int
    lib.int8w_stream_read.argtypes = [P, u64, P, u64]
    lib.int8w_stream_read.restype = ctypes.c_int
    lib.int8w_stream_copy.argtypes = [P, P, u64, u64]
    lib.int8w_stream_copy.restype = ctypes.c_int
    lib.int8w_stream_expand.argtypes = [P, P, u64, u64]
    lib.int8w_stream_expand.restype = ctypes.c_int
    lib.int8w_last_error.argtypes = []
    lib.int8w_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int) -> None:
    if rc != INT8W_OK:
        msg = load_library().int8w_last_error().decode(errors="replace")
        raise Int8wError(rc, msg)


def storage_bytes(out_features: int, in_features: int, group_size: int) -> int:
    return int(load_library().int8w_storage_bytes(out_features, in_features, group_size))


# ---- raw C-ABI calls (device addresses as ints, stream as int) --------------------------------

def int8w_validate(desc: WeightDesc) -> int:
    return load_library().int8w_validate(ctypes.byref(desc))


def int8_dequantize_to(desc: WeightDesc, out: int, stream: int) -> int:
    return load_library().int8_dequantize_to(ctypes.byref(desc), out, stream)


def int8_gemv(desc: WeightDesc, x: int, y: int, stream: int) -> int:
    return load_library().int8_gemv(ctypes.byref(desc), x, y, stream)


def int8_gemv_silu_gate(desc: WeightDesc, gate: int, up: int, y: int, stream: int) -> int:
    return load_library().int8_gemv_silu_gate(ctypes.byref(desc), gate, up, y, stream)


def int8_gemv_silu_gate_resid(desc: WeightDesc, gate: int, up: int, x_resid: int, y: int, stream: int) -> int:
    return load_library().int8_gemv_silu_gate_resid(ctypes.byref(desc), gate, up, x_resid, y, stream)


def int8_gemm(desc: WeightDesc, x: int, y: int, m: int, stream: int) -> int:
    return load_library().int8_gemm(ctypes.byref(desc), x, y, m, stream)


def int8_quantize(w: int, out_features: int, in_features: int, group_size: int, packed: int, scales: int,
                  biases: int, stream: int) -> int:
    return load_library().int8_quantize(w, out_features, in_features, group_size, packed, scales, biases, stream)


def int8_moe_gemv(desc: WeightDesc, num_experts: int, x: int, x_rows: int, ids: int, tokens: int, topk: int,
                  y: int, stream: int) -> int:
    return load_library().int8_moe_gemv(ctypes.byref(desc), num_experts, x, x_rows, ids, tokens, topk, y, stream)


def int8w_fp8_gemv(desc: Fp8WeightDesc, x: int, y: int, stream: int) -> int:
    return load_library().int8w_fp8_gemv(ctypes.byref(desc), x, y, stream)


def int8_gemm_workspace_bytes(desc: WeightDesc, m: int) -> int:
    return int(load_library().int8_gemm_workspace_bytes(ctypes.byref(desc), m))


def int8_gemm_ws(desc: WeightDesc, x: int, y: int, m: int, ws: int, ws_bytes: int, stream: int) -> int:
    return load_library().int8_gemm_ws(ctypes.byref(desc), x, y, m, ws, ws_bytes, stream)


def int8_gemm_noalloc(desc: WeightDesc, x: int, y: int, m: int, stream: int) -> int:
    return load_library().int8_gemm_noalloc(ctypes.byref(desc), x, y, m, stream)


NOALLOC_SCRATCH_BYTES = 64 << 20  # INT8W_NOALLOC_SCRATCH_BYTES


def int8w_stream_read(src: int, nbytes: int, sink: int, stream: int) -> int:
    return load_library().int8w_stream_read(src, nbytes, sink, stream)


def int8w_stream_copy(src: int, dst: int, nbytes: int, stream: int) -> int:
    return load_library().int8w_stream_copy(src, dst, nbytes, stream)


def int8w_stream_expand(src: int, dst: int, nbytes: int, stream: int) -> int:
    return load_library().int8w_stream_expand(src, dst, nbytes, stream)


def int8w_mxfp4_quantize(x: int, x_format: int, rows: int, k: int, codes: int, scales: int, stream: int) -> int:
    return load_library().int8w_mxfp4_quantize(x, x_format, rows, k, codes, scales, stream)


def int8w_mxfp4_dequantize_to(desc: Mxfp4Desc, out: int, stream: int) -> int:
    return load_library().int8w_mxfp4_dequantize_to(desc, out, stream)


def int8w_mxfp4_gemm(desc: Mxfp4Desc, x: int, y: int, m: int, stream: int) -> int:
    return load_library().int8w_mxfp4_gemm(desc, x, y, m, stream)


def int8w_mxfp4_gemm_mx(desc: Mxfp4Desc, x: Mxfp4Desc, y: int, stream: int) -> int:
    return load_library().int8w_mxfp4_gemm_mx(desc, x, y, stream)


def int8w_moe_workspace_bytes(tokens: int, topk: int, inner: int, hidden: int) -> int:
    return int(load_library().int8w_moe_workspace_bytes(tokens, topk, inner, hidden))


def int8_moe_layer(gate: WeightDesc, up: WeightDesc, down: WeightDesc, num_experts: int, call: MoeCall, ws: int,
                   ws_bytes: int, stream: int) -> int:
    return load_library().int8_moe_layer(gate, up, down, num_experts, call, ws, ws_bytes, stream)


def int8w_mxfp4_moe_layer(gate: Mxfp4Desc, up: Mxfp4Desc, down: Mxfp4Desc, num_experts: int, call: MoeCall, ws: int,
                          ws_bytes: int, stream: int) -> int:
    return load_library().int8w_mxfp4_moe_layer(gate, up, down, num_experts, call, ws, ws_bytes, stream)


def int8w_moe_route(call: RouteCall, stream: int) -> int:
    return load_library().int8w_moe_route(call, stream)


def int8_moe_layer_routed(gate: WeightDesc, up: WeightDesc, down: WeightDesc, num_experts: int, call: MoeRoutedCall,
                          ws: int, ws_bytes: int, stream: int) -> int:
    return load_library().int8_moe_layer_routed(gate, up, down, num_experts, call, ws, ws_bytes, stream)


def int8w_mxfp4_moe_layer_routed(gate: Mxfp4Desc, up: Mxfp4Desc, down: Mxfp4Desc, num_experts: int,
                                 call: MoeRoutedCall, ws: int, ws_bytes: int, stream: int) -> int:
    return load_library().int8w_mxfp4_moe_layer_routed(gate, up, down, num_experts, call, ws, ws_bytes, stream)


def int8w_lora_workspace_bytes(pools, count: int, m: int) -> int:
    """pools: a LoraDesc, or a ctypes array of them."""
    return load_library().int8w_lora_workspace_bytes(pools, count, m)


def int8w_lora_add(pools, out, count: int, x: int, x_stride: int, ids: int, m: int, ws: int, ws_bytes: int,
                   stream: int) -> int:
    """pools, out: ctypes arrays of count LoraDesc and LoraOut (or one of each)."""
    return load_library().int8w_lora_add(pools, out, count, x, x_stride, ids, m, ws, ws_bytes, stream)


def int8_gemv_multi(descs, x: int, ys, stream: int) -> int:
    """descs: sequence of WeightDesc; ys: sequence of device addresses (same length)."""
    n = len(descs)
    arr = (WeightDesc * max(n, 1))(*descs)
    yarr = (ctypes.c_void_p * max(n, 1))(*ys)
    return load_library().int8_gemv_multi(arr, n, x, yarr, stream)


# ---- tensor-level wrapper -----------------------------------------------------------------------

def _stream_of(device: torch.device) -> int:
    # The handle alone: building a torch.cuda.Stream object took 1.8 us of an 8 us call.  The
    # function is not a public one, so a torch without it takes the public way.
    index = device.index if device.index is not None else torch.cuda.current_device()
    try:
        return torch._C._cuda_getCurrentRawStream(index)
    except AttributeError:
        return torch.cuda.current_stream(index).cuda_stream


def _need_bf16(t: torch.Tensor, name: str, numel: int, device: torch.device) -> None:
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, weight on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")


class Int8Weight:
    """One 8-bit affine group-quantized weight on the GPU (borrowed tensors).

    packed:  int32/uint32 [out_features, in_features/4] (code k in byte k%4 of word k/4)
    scales:  bfloat16 [out_features, in_features/group_size]
    biases:  bfloat16 [out_features, in_features/group_size]
    The tensors stay owned by the caller (this object keeps references).
    """

    def __init__(self, packed: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, group_size: int):
        if packed.dim() != 2 or packed.dtype not in (torch.int32, torch.uint32):
            raise ValueError("weight must be a 2-D 32-bit (U32) tensor")
        if scales.dtype != torch.bfloat16 or biases.dtype != torch.bfloat16:
            raise ValueError("scales and biases must be bfloat16")
        N, kw = packed.shape
        K = 4 * kw
        gs = int(group_size)
        if gs <= 0 or K % gs:
            raise ValueError(f"group_size {gs} does not divide in_features {K}")
        G = K // gs
        if tuple(scales.shape) != (N, G) or tuple(biases.shape) != (N, G):
            raise ValueError(f"scales/biases must be [{N}, {G}] = [out_features, in_features/group_size]")
        for t, name in ((packed, "packed"), (scales, "scales"), (biases, "biases")):
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if not (packed.device == scales.device == biases.device) or packed.device.type != "cuda":
            raise ValueError("packed, scales and biases must be on one GPU")
        self.packed, self.scales, self.biases = packed, scales, biases
        self.out_features, self.in_features, self.group_size = N, K, gs
        self.device = packed.device
        self.desc = WeightDesc(packed.data_ptr(), scales.data_ptr(), biases.data_ptr(), N, K, gs)
        _check(int8w_validate(self.desc))

    @classmethod
    def quantize(cls, w: torch.Tensor, group_size: int) -> "Int8Weight":
        """Encode a BF16 weight [out_features, in_features] on the GPU (int8_quantize)."""
        if w.dtype != torch.bfloat16 or w.dim() != 2 or not w.is_contiguous() or w.device.type != "cuda":
            raise ValueError("w must be a contiguous 2-D bfloat16 GPU tensor")
        N, K = w.shape
        gs = int(group_size)
        if gs <= 0 or K % gs or K % 4:
            raise ValueError(f"group_size {gs} must divide in_features {K} (a multiple of 4)")
        packed = torch.empty((N, K // 4), dtype=torch.int32, device=w.device)
        scales = torch.empty((N, K // gs), dtype=torch.bfloat16, device=w.device)
        biases = torch.empty((N, K // gs), dtype=torch.bfloat16, device=w.device)
        _check(int8_quantize(w.data_ptr(), N, K, gs, packed.data_ptr(), scales.data_ptr(), biases.data_ptr(),
                             _stream_of(w.device)))
        return cls(packed, scales, biases, gs)

    @classmethod
    def from_arrays(cls, packed, scales_bits, biases_bits, group_size: int, device="cuda") -> "Int8Weight":
        """Upload NumPy arrays (uint32 words, uint16 BF16 bit patterns)."""
        import numpy as np
        p = torch.from_numpy(np.ascontiguousarray(packed).view(np.int32)).to(device)
        s = torch.from_numpy(np.ascontiguousarray(scales_bits).view(np.int16)).view(torch.bfloat16).to(device)
        b = torch.from_numpy(np.ascontiguousarray(biases_bits).view(np.int16)).view(torch.bfloat16).to(device)
        return cls(p, s, b, group_size)

    def storage_bytes(self) -> int:
        return storage_bytes(self.out_features, self.in_features, self.group_size)

    def dequantize_to(self, out: torch.Tensor | None = None) -> torch.Tensor:
        N, K = self.out_features, self.in_features
        if out is None:
            out = torch.empty((N, K), dtype=torch.bfloat16, device=self.device)
        _need_bf16(out, "out", N * K, self.device)
        _check(int8_dequantize_to(self.desc, out.data_ptr(), _stream_of(self.device)))
        return out

    def gemv(self, x: torch.Tensor, y: torch.Tensor | None = None) -> torch.Tensor:
        _need_bf16(x, "x", self.in_features, self.device)
        if y is None:
            y = torch.empty(self.out_features, dtype=torch.bfloat16, device=self.device)
        _need_bf16(y, "y", self.out_features, self.device)
        _check(int8_gemv(self.desc, x.data_ptr(), y.data_ptr(), _stream_of(self.device)))
        return y

    def gemv_silu_gate(self, gate: torch.Tensor, up: torch.Tensor, y: torch.Tensor | None = None) -> torch.Tensor:
        _need_bf16(gate, "gate", self.in_features, self.device)
        _need_bf16(up, "up", self.in_features, self.device)
        if y is None:
            y = torch.empty(self.out_features, dtype=torch.bfloat16, device=self.device)
        _need_bf16(y, "y", self.out_features, self.device)
        _check(int8_gemv_silu_gate(self.desc, gate.data_ptr(), up.data_ptr(), y.data_ptr(), _stream_of(self.device)))
        return y

    def gemv_silu_gate_resid(self, gate: torch.Tensor, up: torch.Tensor, x_resid: torch.Tensor,
                             y: torch.Tensor | None = None) -> torch.Tensor:
        _need_bf16(gate, "gate", self.in_features, self.device)
        _need_bf16(up, "up", self.in_features, self.device)
        _need_bf16(x_resid, "x_resid", self.out_features, self.device)
        if y is None:
            y = torch.empty(self.out_features, dtype=torch.bfloat16, device=self.device)
        _need_bf16(y, "y", self.out_features, self.device)
        _check(int8_gemv_silu_gate_resid(self.desc, gate.data_ptr(), up.data_ptr(), x_resid.data_ptr(),
                                         y.data_ptr(), _stream_of(self.device)))
        return y

    def gemm(self, x: torch.Tensor, y: torch.Tensor | None = None, split_k: bool = True) -> torch.Tensor:
        """Y = X W^T.  With split_k (the default) a call whose grid has too few
        tiles runs int8_gemm_ws on a cached per-device workspace (int8_gemm_noalloc
        when that would have to grow during graph capture); otherwise int8_gemm."""
        if x.dim() != 2 or x.shape[1] != self.in_features:
            raise ValueError(f"X must be [m, {self.in_features}]")
        m = x.shape[0]
        _need_bf16(x, "X", m * self.in_features, self.device)
        if y is None:
            y = torch.empty((m, self.out_features), dtype=torch.bfloat16, device=self.device)
        _need_bf16(y, "Y", m * self.out_features, self.device)
        need = int8_gemm_workspace_bytes(self.desc, m) if split_k and m > 16 else 0
        stream = _stream_of(self.device)
        ws = _workspace(self.device, need) if need else None
        if ws is not None:
            _check(int8_gemm_ws(self.desc, x.data_ptr(), y.data_ptr(), m, ws.data_ptr(), ws.numel(), stream))
        elif need and need <= NOALLOC_SCRATCH_BYTES:
            # under graph capture, where the cached workspace may not grow: the
            # library's static scratch, same kernels and bits
            _check(int8_gemm_noalloc(self.desc, x.data_ptr(), y.data_ptr(), m, stream))
        else:
            _check(int8_gemm(self.desc, x.data_ptr(), y.data_ptr(), m, stream))
        return y

    def gemm_lora(self, x: torch.Tensor, adapters: "LoraAdapters", ids: torch.Tensor,
                  y: torch.Tensor | None = None) -> torch.Tensor:
        """gemm with each row's low-rank adapter beside it: lora_add in place on gemm's Y (which gemm has rounded)."""
        _need_pool(adapters, self.in_features, self.out_features, x, ids)
        with _current(self.device):
            y = self.gemm(x, y)
        return _add_in_place(adapters, x, ids, y)


# One gemm workspace per device (scratch for split-K partials), grown on
# demand.  Calls that use it are ordered on the caller's stream; overlapping
# calls on several streams of one device would share it and race.
_workspaces: dict = {}


def _workspace(device: torch.device, nbytes: int):
    """The device's cached workspace of at least nbytes, grown if needed; None
    when it would have to grow while the current stream is being captured into
    a graph (an allocation made then would come from the graph's pool)."""
    key = device.index if device.index is not None else torch.cuda.current_device()
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        if torch.cuda.is_current_stream_capturing():
            return None
        ws = torch.empty(max(nbytes, 64 << 20), dtype=torch.uint8, device=device)
        _workspaces[key] = ws
    return ws


def gemv_multi(weights, x: torch.Tensor, ys=None):
    """y_i = W_i x for up to four Int8Weight sharing in_features and group_size, in one launch."""
    weights = list(weights)
    if not weights:
        raise ValueError("gemv_multi needs at least one weight")
    dev = weights[0].device
    _need_bf16(x, "x", weights[0].in_features, dev)
    if ys is None:
        ys = [torch.empty(w.out_features, dtype=torch.bfloat16, device=dev) for w in weights]
    ys = list(ys)
    if len(ys) != len(weights):
        raise ValueError("gemv_multi: one output per weight")
    for w, y in zip(weights, ys):
        if w.device != dev:
            raise ValueError("gemv_multi: weights on different devices")
        _need_bf16(y, "y", w.out_features, dev)
    _check(int8_gemv_multi([w.desc for w in weights], x.data_ptr(), [y.data_ptr() for y in ys], _stream_of(dev)))
    return ys


def moe_gemv(experts: Int8Weight, num_experts: int, x: torch.Tensor, ids: torch.Tensor, y=None):
    """Expert-indexed gemv (int8_moe_gemv).

    experts: E = num_experts experts of [N, K] stacked along rows (out_features = E*N)
    x:       bfloat16 [tokens, 1 or topk, K]
    ids:     int32/uint32 [tokens, topk] on the GPU (expert of each slot)
    returns  bfloat16 [tokens, topk, N]; a slot whose id is not below E is NaN
    """
    dev = experts.device
    E = int(num_experts)
    if E <= 0 or experts.out_features % E:
        raise ValueError(f"{experts.out_features} rows are not a whole number of {E} experts")
    N, K = experts.out_features // E, experts.in_features
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.uint32) or ids.device != dev or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous 32-bit [tokens, topk] tensor on the weight's GPU")
    T, topk = ids.shape
    if x.dim() != 3 or x.shape[0] != T or x.shape[2] != K or x.shape[1] not in (1, topk):
        raise ValueError(f"x must be [{T}, 1 or {topk}, {K}]")
    _need_bf16(x, "x", x.numel(), dev)
    if y is None:
        y = torch.empty((T, topk, N), dtype=torch.bfloat16, device=dev)
    _need_bf16(y, "y", T * topk * N, dev)
    _check(int8_moe_gemv(experts.desc, E, x.data_ptr(), x.shape[1], ids.data_ptr(), T, topk, y.data_ptr(),
                         _stream_of(dev)))
    return y


class Fp8Weight:
    """An FP8 E4M3 weight on the GPU (borrowed tensors), after the rustdoc page "Fp8Weight".

    weight: uint8 [n, k] E4M3 bytes (k a multiple of 16)
    scale:  float32 [n] (FP8_PER_ROW); bfloat16 or float32 [ceil(n/BS), ceil(k/BS)]
            (FP8_BLOCK_BF16 / FP8_BLOCK_F32); None (FP8_SINGLE, with single_scale)
    """

    def __init__(self, weight: torch.Tensor, scale, scale_format: int, block_size: int = 128,
                 single_scale: float = 1.0):
        if weight.dim() != 2 or weight.dtype != torch.uint8 or not weight.is_contiguous():
            raise ValueError("weight must be a contiguous 2-D uint8 tensor of E4M3 bytes")
        if weight.device.type != "cuda":
            raise ValueError("weight must be on a GPU")
        n, k = weight.shape
        fmt = int(scale_format)
        if fmt == FP8_SINGLE:
            if scale is not None:
                raise ValueError("FP8_SINGLE takes no scale tensor")
        else:
            want = {FP8_PER_ROW: torch.float32, FP8_BLOCK_BF16: torch.bfloat16, FP8_BLOCK_F32: torch.float32}.get(fmt)
            if want is None:
                raise ValueError(f"unknown scale format {fmt}")
            if scale is None or scale.dtype != want or scale.device != weight.device or not scale.is_contiguous():
                raise ValueError(f"scale must be a contiguous {want} tensor on the weight's GPU")
            bs = int(block_size)
            shape = (n,) if fmt == FP8_PER_ROW else (-(-n // bs), -(-k // bs))
            if tuple(scale.shape) != shape:
                raise ValueError(f"scale must have shape {shape}")
        self.weight, self.scale = weight, scale
        self.n, self.k, self.scale_format = n, k, fmt
        self.device = weight.device
        self.desc = Fp8WeightDesc(weight.data_ptr(), scale.data_ptr() if scale is not None else None, n, k, fmt,
                                  int(block_size), float(single_scale))

    def gemv(self, x: torch.Tensor, y: torch.Tensor | None = None) -> torch.Tensor:
        _need_bf16(x, "x", self.k, self.device)
        if y is None:
            y = torch.empty(self.n, dtype=torch.bfloat16, device=self.device)
        _need_bf16(y, "y", self.n, self.device)
        _check(int8w_fp8_gemv(self.desc, x.data_ptr(), y.data_ptr(), _stream_of(self.device)))
        return y


class Mxfp4Weight:
    """A matrix in MXFP4 on the GPU (borrowed tensors): a weight, or quantized activations.

    codes:  uint8 [rows, k/2], element j in the low (j even) or high half of byte j/2
    scales: uint8 [rows, k/32], a block of 32 is worth its codes times 2^(scale - 127)
    """

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dim() != 2 or codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise ValueError("codes and scales must be 2-D uint8 tensors")
        rows, k = codes.shape[0], 2 * codes.shape[1]
        if k == 0 or k % 32:
            raise ValueError(f"k {k} must be a positive multiple of 32")
        if tuple(scales.shape) != (rows, k // 32):
            raise ValueError(f"scales must be [{rows}, {k // 32}] = [rows, k/32]")
        if not codes.is_contiguous() or not scales.is_contiguous():
            raise ValueError("codes and scales must be contiguous")
        if codes.device != scales.device or codes.device.type != "cuda":
            raise ValueError("codes and scales must be on one GPU")
        self._set(codes, scales, rows, k, codes.device, codes.data_ptr(), scales.data_ptr())

    @classmethod
    def quantize(cls, x: torch.Tensor) -> "Mxfp4Weight":
        """Encode BF16 or float32 values [rows, k] on the GPU (int8w_mxfp4_quantize)."""
        if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.float32) or not x.is_contiguous() \
                or x.device.type != "cuda":
            raise ValueError("x must be a contiguous 2-D bfloat16 or float32 GPU tensor")
        rows, k = x.shape
        if k == 0 or k % 32:
            raise ValueError(f"k {k} must be a positive multiple of 32")
        codes = x.new_empty((rows, k // 2), dtype=torch.uint8)
        scales = x.new_empty((rows, k // 32), dtype=torch.uint8)
        c, s, device = codes.data_ptr(), scales.data_ptr(), x.device
        _check(load_library().int8w_mxfp4_quantize(x.data_ptr(), VALUES_F32 if x.dtype == torch.float32 else VALUES_BF16,
                                                   rows, k, c, s, _stream_of(device)))
        q = cls.__new__(cls)  # the tensors are as __init__ wants them
        q._set(codes, scales, rows, k, device, c, s)
        return q

    def _set(self, codes, scales, rows, k, device, codes_ptr, scales_ptr) -> None:
        self.codes, self.scales, self.rows, self.k, self.device = codes, scales, rows, k, device
        self.desc = Mxfp4Desc(codes_ptr, scales_ptr, rows, k)

    def dequantize_to(self, out: torch.Tensor | None = None) -> torch.Tensor:
        if out is None:
            out = torch.empty((self.rows, self.k), dtype=torch.bfloat16, device=self.device)
        else:
            _need_bf16(out, "out", self.rows * self.k, self.device)
        if self.rows == 0:  # as from quantize() on no rows; the C entry wants a matrix
            return out
        _check(load_library().int8w_mxfp4_dequantize_to(self.desc, out.data_ptr(), _stream_of(self.device)))
        return out

    def gemm(self, x: torch.Tensor, y: torch.Tensor | None = None) -> torch.Tensor:
        """Y = X W^T for BF16 X [m, k] (m = 1: one token's decode)."""
        if x.dim() != 2 or x.shape[1] != self.k:
            raise ValueError(f"X must be [m, {self.k}]")
        m = x.shape[0]
        _need_bf16(x, "X", m * self.k, self.device)
        if y is None:
            y = x.new_empty((m, self.rows))
        else:
            _need_bf16(y, "Y", m * self.rows, self.device)
        _check(load_library().int8w_mxfp4_gemm(self.desc, x.data_ptr(), y.data_ptr(), m, _stream_of(self.device)))
        return y

    def gemm_lora(self, x: torch.Tensor, adapters: "LoraAdapters", ids: torch.Tensor,
                  y: torch.Tensor | None = None) -> torch.Tensor:
        """gemm with each row's low-rank adapter beside it: lora_add in place on gemm's Y (which gemm has rounded)."""
        _need_pool(adapters, self.k, self.rows, x, ids)
        with _current(self.device):
            y = self.gemm(x, y)
        return _add_in_place(adapters, x, ids, y)

    def gemm_mx(self, x: "Mxfp4Weight", y: torch.Tensor | None = None) -> torch.Tensor:
        """Y = X W^T with both operands in MXFP4 (x e.g. from Mxfp4Weight.quantize)."""
        if x.k != self.k:
            raise ValueError(f"X must be [m, {self.k}]")
        if x.device != self.device:
            raise ValueError(f"X is on {x.device}, weight on {self.device}")
        if y is None:
            y = torch.empty((x.rows, self.rows), dtype=torch.bfloat16, device=self.device)
        else:
            _need_bf16(y, "Y", x.rows * self.rows, self.device)
        _check(load_library().int8w_mxfp4_gemm_mx(self.desc, x.desc, y.data_ptr(), _stream_of(self.device)))
        return y


def moe_layer(gate, up, down, num_experts: int, x: torch.Tensor, logits: torch.Tensor, topk: int,
              renormalize: bool = True, routed_scale: float = 1.0, x_resid: torch.Tensor | None = None,
              y: torch.Tensor | None = None) -> torch.Tensor:
    """A mixture-of-experts layer for a few tokens (int8_moe_layer, int8w_mxfp4_moe_layer).

    gate, up: num_experts experts of [inner, hidden] stacked along rows, all Int8Weight or all Mxfp4Weight
    down:     num_experts experts of [hidden, inner], of the same kind
    x:        bfloat16 [tokens, hidden]
    logits:   float32 or bfloat16 [tokens, num_experts], the router's scores before the softmax
    returns   bfloat16 [tokens, hidden]: x_resid + the weighted sum over the topk experts of each token.
    Scratch is allocated for the call on the current stream, so calls may overlap on several streams.
    """
    mx = isinstance(gate, Mxfp4Weight)
    kind = Mxfp4Weight if mx else Int8Weight
    if not (isinstance(gate, kind) and isinstance(up, kind) and isinstance(down, kind)):
        raise TypeError("gate, up and down must be three Int8Weight or three Mxfp4Weight")
    dev = gate.device
    if up.device != dev or down.device != dev:
        raise ValueError("moe_layer: weights on different devices")
    hidden, inner = (gate.k, down.k) if mx else (gate.in_features, down.in_features)
    if x.dim() != 2 or x.shape[1] != hidden:
        raise ValueError(f"x must be [tokens, {hidden}]")
    T, E = x.shape[0], int(num_experts)
    _need_bf16(x, "x", T * hidden, dev)
    if logits.dtype not in (torch.float32, torch.bfloat16) or tuple(logits.shape) != (T, E) or logits.device != dev \
            or not logits.is_contiguous():
        raise ValueError(f"logits must be a contiguous float32 or bfloat16 [{T}, {E}] tensor on the weights' GPU")
    if x_resid is not None:
        _need_bf16(x_resid, "x_resid", T * hidden, dev)
    if not 1 <= topk <= min(E, MAX_MOE_TOPK):  # before it sizes the scratch
        raise Int8wError(INT8W_ERR_SHAPE, f"topk {topk} outside 1..min({E} experts, {MAX_MOE_TOPK})")
    if y is None:
        y = torch.empty((T, hidden), dtype=torch.bfloat16, device=dev)
    _need_bf16(y, "y", T * hidden, dev)
    need = int8w_moe_workspace_bytes(T, topk, inner, hidden)
    # A call's own: one kept for the device would be shared by streams, and freed when it grows
    # under a graph that still writes to it.
    ws = x.new_empty(need, dtype=torch.uint8)
    call = MoeCall(x.data_ptr(), logits.data_ptr(), x_resid.data_ptr() if x_resid is not None else None, y.data_ptr(),
                   T, topk, VALUES_F32 if logits.dtype == torch.float32 else VALUES_BF16, int(bool(renormalize)),
                   float(routed_scale))
    layer = int8w_mxfp4_moe_layer if mx else int8_moe_layer
    _check(layer(gate.desc, up.desc, down.desc, E, call, ws.data_ptr(), ws.numel(), _stream_of(dev)))
    return y


def moe_route(logits: torch.Tensor, topk: int, scoring: str = "softmax", bias: torch.Tensor | None = None,
              groups: int = 1, topk_groups: int | None = None, group_score: str = "top2", renormalize: bool = True,
              routed_scale: float = 1.0, ids: torch.Tensor | None = None, weights: torch.Tensor | None = None):
    """The routing to experts (int8w_moe_route): ids int32 and weights float32 [tokens, topk], largest choice first.

    logits:  float32 or bfloat16 [tokens, num_experts]
    scoring: "softmax" or "sigmoid", the scores that make the weights
    bias:    float32 [num_experts], added to the scores for the choice alone
    groups:  the experts in that many equal groups, of which the topk_groups (default: all) with the largest
             group_score stay: "max", a group's largest biased score, or "top2", the sum of its two largest
    A slot that no expert is left for (those at -inf are never taken) holds id -1 and weight 0; a token with NaN
    among its logits has id -1 and weight NaN in all its slots.  ids goes to moe_gemv (which gives NaN for an
    id of -1), both to moe_layer_routed.  There is no backward: an input that requires a gradient is refused
    where gradients are recorded.
    """
    dev, f32 = logits.device, logits.dtype is torch.float32
    if not (f32 or logits.dtype is torch.bfloat16) or logits.dim() != 2 or not logits.is_contiguous() or dev.type != "cuda":
        raise ValueError("logits must be a contiguous float32 or bfloat16 [tokens, num_experts] GPU tensor")
    how, of_group = ROUTE_SCORING.get(scoring), GROUP_SCORES.get(group_score)
    if how is None or of_group is None:
        raise ValueError(f"scoring is one of {sorted(ROUTE_SCORING)}, group_score one of {sorted(GROUP_SCORES)}")
    T, E = logits.shape
    if bias is not None and (bias.dtype is not torch.float32 or bias.shape != (E,) or bias.device != dev
                             or not bias.is_contiguous()):
        raise ValueError(f"bias must be a contiguous float32 [{E}] tensor on the logits' GPU")
    if logits.requires_grad or (bias is not None and bias.requires_grad):
        _no_backward("moe_route")
    topk, groups = int(topk), int(groups)
    topk_groups = groups if topk_groups is None else int(topk_groups)
    if not (1 <= topk <= MAX_MOE_TOPK and 1 <= groups <= MAX_MOE_GROUPS and 1 <= topk_groups <= groups):  # before they size the outputs
        raise Int8wError(INT8W_ERR_SHAPE, f"topk {topk}, groups {groups} or topk_groups {topk_groups} out of range")
    if ids is None:
        ids = logits.new_empty_strided((T, topk), (topk, 1), dtype=torch.int32)  # 0.2 us less than new_empty
    else:
        _need_slots(ids, "ids", (torch.int32, torch.uint32), T, topk, dev)
    if weights is None:
        weights = logits.new_empty_strided((T, topk), (topk, 1), dtype=torch.float32)
    else:
        _need_slots(weights, "weights", (torch.float32,), T, topk, dev)
    _call(dev, load_library().packed_route,
          _ROUTE_CALL.pack(logits.data_ptr(), bias.data_ptr() if bias is not None else 0, ids.data_ptr(), weights.data_ptr(), T, E, topk,
                           VALUES_F32 if f32 else VALUES_BF16, how, groups, topk_groups, of_group, bool(renormalize), routed_scale),
          _stream_of(dev))
    return ids, weights


def moe_layer_routed(gate, up, down, num_experts: int, x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                     x_resid: torch.Tensor | None = None, y: torch.Tensor | None = None) -> torch.Tensor:
    """moe_layer from a given routing, moe_route's or any other (int8_moe_layer_routed, int8w_mxfp4_moe_layer_routed).

    ids:     int32/uint32 [tokens, topk]; a slot whose id is not below num_experts (-1) runs no expert
    weights: float32 [tokens, topk], of the slots' experts in the token's sum; any NaN makes the token's output NaN
    returns  bfloat16 [tokens, hidden]: x_resid + the weighted sum over the slots.  The rest as moe_layer.
    There is no backward: an input that requires a gradient is refused where gradients are recorded.
    """
    mx = isinstance(gate, Mxfp4Weight)
    kind = Mxfp4Weight if mx else Int8Weight
    if not (isinstance(gate, kind) and isinstance(up, kind) and isinstance(down, kind)):
        raise TypeError("gate, up and down must be three Int8Weight or three Mxfp4Weight")
    dev = gate.device
    if up.device != dev or down.device != dev:
        raise ValueError("moe_layer_routed: weights on different devices")
    hidden, inner = (gate.k, down.k) if mx else (gate.in_features, down.in_features)
    if x.dim() != 2 or x.shape[1] != hidden:
        raise ValueError(f"x must be [tokens, {hidden}]")
    T, E = x.shape[0], int(num_experts)
    _need_bf16(x, "x", T * hidden, dev)
    if ids.dim() != 2:
        raise ValueError(f"ids must be [{T}, topk]")
    topk = ids.shape[1]
    _need_slots(ids, "ids", (torch.int32, torch.uint32), T, topk, dev)
    _need_slots(weights, "weights", (torch.float32,), T, topk, dev)
    if x_resid is not None:
        _need_bf16(x_resid, "x_resid", T * hidden, dev)
    if x.requires_grad or weights.requires_grad or (x_resid is not None and x_resid.requires_grad):
        _no_backward("moe_layer_routed")
    if not 1 <= topk <= MAX_MOE_TOPK:  # before it sizes the scratch
        raise Int8wError(INT8W_ERR_SHAPE, f"topk {topk} outside 1..{MAX_MOE_TOPK}")
    if y is None:
        y = torch.empty((T, hidden), dtype=torch.bfloat16, device=dev)
    _need_bf16(y, "y", T * hidden, dev)
    ws = x.new_empty(int8w_moe_workspace_bytes(T, topk, inner, hidden), dtype=torch.uint8)  # the call's own, as in moe_layer
    call = MoeRoutedCall(x.data_ptr(), ids.data_ptr(), weights.data_ptr(),
                         x_resid.data_ptr() if x_resid is not None else None, y.data_ptr(), T, topk)
    lib = load_library()
    layer = lib.int8w_mxfp4_moe_layer_routed if mx else lib.int8_moe_layer_routed
    _call(dev, layer, gate.desc, up.desc, down.desc, E, call, ws.data_ptr(), ws.numel(), _stream_of(dev))
    return y


def _need_slots(t: torch.Tensor, name: str, dtypes, tokens: int, topk: int, device: torch.device) -> None:
    if t.dtype not in dtypes or t.shape != (tokens, topk) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {' or '.join(map(str, dtypes))} [{tokens}, {topk}] tensor on {device}")


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # without a check for initialisation


def _current(device: torch.device):
    """Makes another device than the current one current: kernels go to the current device where the stream is the
    default one (handle 0)."""
    return contextlib.nullcontext() if device.index is None or device.index == _current_device() else torch.cuda.device(device)


def _call(device: torch.device, entry, *args) -> None:
    """Calls a C entry that launches on `device`."""
    if device.index is None or device.index == _current_device():  # mostly: without a context object
        rc = entry(*args)
    else:
        with torch.cuda.device(device):
            rc = entry(*args)
    if rc != INT8W_OK:
        _check(rc)


def _no_backward(what: str) -> None:
    """For a call with an input that requires a gradient: refused where gradients are recorded, as a backward pass would
    stop at it without a word."""
    if torch.is_grad_enabled():
        raise Int8wError(INT8W_ERR_UNSUPPORTED, f"{what} has no backward, and an input requires a gradient: call it under "
                                                "torch.no_grad(), or on detached tensors")


class LoraAdapters:
    """A pool of low-rank adapters of one projection on the GPU (borrowed tensors).

    a:      bfloat16 [num_adapters, rank, in_features]; rank and in_features multiples of 8, rank up to 256
    b:      bfloat16 [num_adapters, out_features, rank]
    scales: float32 [num_adapters], the factor of b (a x); None: 1
    ranks:  int32/uint32 [num_adapters], where adapters of smaller ranks share the pool: beyond an adapter's
            own rank its rows of a and columns of b must hold zeros, which are not always read
    Calls have no backward: a pool made of tensors that require a gradient is refused by them where gradients are recorded.
    """

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scales: torch.Tensor | None = None,
                 ranks: torch.Tensor | None = None):
        if a.dim() != 3 or b.dim() != 3 or a.dtype != torch.bfloat16 or b.dtype != torch.bfloat16:
            raise ValueError("a and b must be 3-D bfloat16 tensors")
        (num, rank, k), n = a.shape, b.shape[1]
        if tuple(b.shape) != (num, n, rank):
            raise ValueError(f"b must be [{num}, out_features, {rank}]")
        if rank == 0 or rank % 8 or rank > MAX_LORA_RANK or k % 8:
            raise ValueError(f"rank {rank} must be a multiple of 8 up to {MAX_LORA_RANK}, in_features {k} a multiple of 8")
        if not a.is_contiguous() or not b.is_contiguous():
            raise ValueError("a and b must be contiguous")
        if a.device != b.device or a.device.type != "cuda":
            raise ValueError("a and b must be on one GPU")
        for t, name, dtypes in ((scales, "scales", (torch.float32,)), (ranks, "ranks", (torch.int32, torch.uint32))):
            if t is not None and (t.dtype not in dtypes or tuple(t.shape) != (num,) or t.device != a.device
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {' or '.join(map(str, dtypes))} [{num}] tensor on {a.device}")
        self.a, self.b, self.scales, self.ranks = a, b, scales, ranks
        self.num_adapters, self.rank, self.in_features, self.out_features = num, rank, k, n
        self.device = a.device
        # once: three tensors asked in each call took 0.7 us of 8
        self.trained = a.requires_grad or b.requires_grad or (scales is not None and scales.requires_grad)
        self.desc = LoraDesc(a.data_ptr(), b.data_ptr(), scales.data_ptr() if scales is not None else None,
                             ranks.data_ptr() if ranks is not None else None, num, rank, k, n)
        self.packed = bytes(self.desc)  # as lora_add passes it
        # what no call would take is refused here: a call of no rows checks the pool and launches nothing
        _check(load_library().packed_lora_add(self.packed, None, 1, None, 0, None, 0, None, 0, 0))

    @classmethod
    def from_list(cls, adapters) -> "LoraAdapters":
        """A pool from (a [r, in_features], b [out_features, r], scale) of any ranks r: copies, padded with zeros."""
        adapters = list(adapters)
        if not adapters:
            raise ValueError("from_list needs at least one adapter")
        a0, b0, _ = adapters[0]
        k, n, dev = a0.shape[-1], b0.shape[0], a0.device
        for a, b, _ in adapters:
            if a.dim() != 2 or b.dim() != 2 or a.shape[1] != k or b.shape[0] != n or b.shape[1] != a.shape[0] or a.shape[0] == 0:
                raise ValueError(f"adapters must be a [r, {k}] and b [{n}, r]")
        ranks = [a.shape[0] for a, _, _ in adapters]
        rank = -(-max(ranks) // 8) * 8
        pa = torch.zeros((len(ranks), rank, k), dtype=torch.bfloat16, device=dev)
        pb = torch.zeros((len(ranks), n, rank), dtype=torch.bfloat16, device=dev)
        for i, (a, b, _) in enumerate(adapters):
            pa[i, :ranks[i]] = a
            pb[i, :, :ranks[i]] = b
        return cls(pa, pb, torch.tensor([float(s) for _, _, s in adapters], dtype=torch.float32, device=dev),
                   torch.tensor(ranks, dtype=torch.int32, device=dev))


def _rows(t: torch.Tensor, name: str, m: int, n: int, device: torch.device) -> int:
    """Checks a [m, n] matrix of bfloat16 whose rows may be apart (columns of a wider one); returns its row stride."""
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, adapters on {device}")
    if t.shape != (m, n):
        raise ValueError(f"{name} must be [{m}, {n}]")
    rs, cs = t.stride()
    if m <= 1:
        rs = n  # one row: whatever the stride says
    if (cs != 1 and n > 1) or rs < n:
        raise ValueError(f"{name}'s rows must be contiguous")
    return rs


def _need_pool(pool: LoraAdapters, k: int, n: int, x: torch.Tensor, ids: torch.Tensor) -> None:
    """What gemm_lora wants before its product is launched."""
    if not isinstance(pool, LoraAdapters) or pool.in_features != k or pool.out_features != n:
        raise ValueError(f"adapters must be LoraAdapters of in_features {k} and out_features {n}")
    if x.dim() != 2 or x.device != pool.device:
        raise ValueError(f"X must be [m, {k}] on {pool.device}")
    if x.shape[0] > MAX_LORA_ROWS:
        raise Int8wError(INT8W_ERR_SHAPE, f"m={x.shape[0]} rows are more than 2^20")
    _need_ids(ids, x.shape[0], pool.device)
    if x.requires_grad or pool.trained:
        _no_backward("gemm_lora")


def _need_ids(ids: torch.Tensor, m: int, device: torch.device) -> None:
    if ids.dtype not in (torch.int32, torch.uint32) or ids.shape != (m,) or ids.device != device or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous 32-bit [{m}] tensor on {device}")


def _add_in_place(pool: LoraAdapters, x: torch.Tensor, ids: torch.Tensor, y: torch.Tensor) -> torch.Tensor:
    m, n = x.shape[0], pool.out_features
    rows = y if tuple(y.shape) == (m, n) else y.view(-1)[:m * n].view(m, n)  # gemm takes any buffer that is large enough
    lora_add(pool, x, ids, rows, rows)
    return y


def lora_add(adapters, x: torch.Tensor, ids: torch.Tensor, base=None, y=None):
    """y[t] = base[t] + scales[e] * b[e] (a[e] x[t]) with e = ids[t] (int8w_lora_add).

    adapters: one LoraAdapters, or up to four with the same num_adapters and in_features (q, k and v) that share
              x and ids in one call: then base and y are sequences, and a list comes back
    x:        bfloat16 [m, in_features]
    ids:      int32/uint32 [m] on the GPU; -1: no adapter, the row gets base itself; another id outside the pool: NaN
    base:     bfloat16 [m, out_features], typically the projection's output; None: zeros
    y:        the output, base itself for in place; None: a new one
    x, base and y may have rows apart (columns of a wider matrix; x's a multiple of 8 values).
    Scratch is allocated for the call on the current stream, so calls may overlap on several streams.
    There is no backward: an input or adapter that requires a gradient is refused where gradients are recorded.
    """
    one = isinstance(adapters, LoraAdapters)
    if one:
        pools, bases, ys = (adapters,), (base,), [y]
    else:
        pools = tuple(adapters)
        bases = (None,) * len(pools) if base is None else tuple(base)
        ys = [None] * len(pools) if y is None else list(y)
    count = len(pools)
    if not 1 <= count <= MAX_MULTI:
        raise Int8wError(INT8W_ERR_SHAPE, f"lora_add takes 1..{MAX_MULTI} pools, got {count}")
    if len(bases) != count or len(ys) != count:
        raise ValueError("lora_add: one base and one output per pool")
    dev, k = pools[0].device, pools[0].in_features
    shape = x.shape  # made anew each time it is asked for
    if len(shape) != 2 or shape[1] != k:
        raise ValueError(f"x must be [m, {k}]")
    m = shape[0]
    xs = _rows(x, "x", m, k, dev)
    _need_ids(ids, m, dev)
    trained = x.requires_grad
    descs = outs = b""
    for i, pool in enumerate(pools):
        if pool.device != dev:
            raise ValueError("lora_add: pools on different devices")
        n, b, o = pool.out_features, bases[i], ys[i]
        if trained or pool.trained or (b is not None and b.requires_grad):
            _no_backward("lora_add")
        if o is None:
            o = ys[i] = x.new_empty_strided((m, n), (n, 1))
            os = n
        else:
            os = _rows(o, "y", m, n, dev)
        descs += pool.packed
        outs += _LORA_OUT.pack(0, o.data_ptr(), 0, os) if b is None else \
            _LORA_OUT.pack(b.data_ptr(), o.data_ptr(), _rows(b, "base", m, n, dev), os)
    lib = load_library()
    need = lib.packed_lora_bytes(descs, count, m)
    ws = x.new_empty(need, dtype=torch.uint8) if need else None  # a call's own: one kept for the device would be shared by streams and graphs
    _call(dev, lib.packed_lora_add, descs, outs, count, x.data_ptr(), xs, ids.data_ptr(), m, ws.data_ptr() if need else 0, need,
          _stream_of(dev))
    return ys[0] if one else ys
