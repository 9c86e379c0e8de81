"""ctypes binding of libcoat_fp8.so (declared in include/coat_fp8.h).

Argument marshalling only: every step of the optimizer runs in the library's
HIP kernels.  Marshalling includes what the C ABI cannot see through raw
pointers: each buffer's dtype, contiguity, size and device are checked
before the call (ValueError).  torch tensors are accepted for convenience (their device pointers
and torch's current HIP stream are passed through); the library never sees a
torch type.  Importing this module loads the library and fails loudly if it is
missing: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass
from typing import List, Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcoat_fp8.so")

ABI_VERSION = 1
GROUP_SIZES = (16, 32, 64, 128)

COAT_OK = 0
COAT_ERR_NULL_POINTER = 1
COAT_ERR_INVALID_VALUE = 2
COAT_ERR_GROUP_SIZE = 3
COAT_ERR_MISALIGNED = 4
COAT_ERR_HIP = 5

EXPORTED_SYMBOLS = (
    "coat_adamw_fp8_step", "coat_fp8_expand_quantize", "coat_fp8_dequantize_expand",
    "coat_e4m3_encode", "coat_e4m3_decode", "coat_fp8_quantize_act",
    "coat_fp8_gemm_group_quant", "coat_fp8_gemm_bf16", "coat_status_string",
    "coat_last_hip_error", "coat_abi_version",
    "coat_fp8_rms_norm", "coat_fp8_rms_norm_bwd", "coat_fp8_rms_norm_bwd_workspace",
    "coat_fp8_swiglu", "coat_fp8_swiglu_bwd", "coat_fp8_qk_norm_rope",
    "coat_fp8_qk_norm_rope_bwd", "coat_fp8_qk_norm_rope_bwd_workspace",
    "coat_fp8_weight_grad", "coat_fp8_weight_grad_workspace",
)


class CoatError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


class FP8State(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("k", ctypes.c_void_p)]


class AdamWTensor(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("m", FP8State), ("v", FP8State), ("n", ctypes.c_int64)]


class AdamWHParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float),
                ("beta2", ctypes.c_float), ("eps", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("step", ctypes.c_int64),
                ("group_size", ctypes.c_int32)]


_vp, _f32, _i32, _i64 = ctypes.c_void_p, ctypes.c_float, ctypes.c_int32, ctypes.c_int64


def _fields(spec: str):
    """(name, type) pairs from "type: name name ..., type: name ..."."""
    types = {"ptr": _vp, "f32": _f32, "i32": _i32, "i64": _i64}
    return [(name, types[kind.strip()]) for part in spec.split(",")
            for kind, names in [part.split(":")] for name in names.split()]


def _packer(structure):
    """A function that packs a structure's values, in the order of its fields,
    into bytes of the same layout (in a quarter of the time that building the
    ctypes structure takes, which a small kernel would wait for)."""
    codes = {_vp: "P", _f32: "f", _i32: "i", _i64: "q"}
    flat = []
    for _, t in structure._fields_:
        flat += [u for _, u in t._fields_] if issubclass(t, ctypes.Structure) else [t]
    pack = struct.Struct("@" + "".join(codes[t] for t in flat)).pack

    def packed(*values):
        try:
            return pack(*values)
        except (struct.error, OverflowError) as e:
            raise ValueError(f"an argument does not fit its C type: {e}") from None

    return packed


class RMSNormArgs(ctypes.Structure):
    _fields_ = _fields("ptr: x residual weight residual_out y y_codes y_amax codes scales rstd, "
                       "i64: rows cols, f32: eps y_scale, i32: group_size")


class RMSNormBwdArgs(ctypes.Structure):
    _fields_ = _fields("ptr: dy codes scales rstd weight d_residual dx dw workspace, "
                       "i64: workspace_bytes rows cols, i32: group_size accumulate")


class SwigluArgs(ctypes.Structure):
    _fields_ = _fields("ptr: gate_up codes scales h h_codes h_amax, i64: rows cols, f32: h_scale, "
                       "i32: group_size")


class QkShape(ctypes.Structure):
    _fields_ = _fields("i64: tokens table_rows, i32: q_heads k_heads head_dim rot_dim interleaved "
                       "group_size")


class QkNormRopeArgs(ctypes.Structure):
    _fields_ = [("shape", QkShape)] + _fields(
        "ptr: q k, i64: q_stride k_stride, ptr: q_weight k_weight cos sin positions q_out k_out, "
        "i64: q_out_stride k_out_stride, ptr: codes scales rstd, f32: eps")


class QkNormRopeBwdArgs(ctypes.Structure):
    _fields_ = [("shape", QkShape)] + _fields(
        "ptr: dq_out dk_out, i64: dq_out_stride dk_out_stride, ptr: codes scales rstd q_weight "
        "k_weight cos sin positions dq dk, i64: dq_stride dk_stride, ptr: dq_weight dk_weight "
        "workspace, i64: workspace_bytes, i32: accumulate")


class WeightGradArgs(ctypes.Structure):
    _fields_ = _fields("ptr: dy x_codes x_scales dw_bf16 dw_f32 workspace, i64: workspace_bytes M N K, "
                       "f32: x_scale, i32: group_size accumulate")


def _load(path: str = LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -c \"import "
            f"__graft_entry__; __graft_entry__.build()\"` (hipcc, gfx950)")
    lib = ctypes.CDLL(path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    lib.coat_adamw_fp8_step.restype = ctypes.c_int
    lib.coat_adamw_fp8_step.argtypes = [vp, i32, ctypes.POINTER(AdamWHParams), vp]
    lib.coat_fp8_expand_quantize.restype = ctypes.c_int
    lib.coat_fp8_expand_quantize.argtypes = [vp, i64, i32, FP8State, vp]
    lib.coat_fp8_dequantize_expand.restype = ctypes.c_int
    lib.coat_fp8_dequantize_expand.argtypes = [vp, vp, vp, i64, i32, vp, vp]
    lib.coat_e4m3_encode.restype = ctypes.c_int
    lib.coat_e4m3_encode.argtypes = [vp, i64, vp, vp]
    lib.coat_e4m3_decode.restype = ctypes.c_int
    lib.coat_e4m3_decode.argtypes = [vp, i64, vp, vp]
    lib.coat_fp8_quantize_act.restype = ctypes.c_int
    lib.coat_fp8_quantize_act.argtypes = [vp, i64, i64, i32, vp, vp, vp, vp]
    f32 = ctypes.c_float
    lib.coat_fp8_gemm_group_quant.restype = ctypes.c_int
    lib.coat_fp8_gemm_group_quant.argtypes = [vp, vp, f32, f32, i64, i64, i64, i32, vp, vp, vp, vp]
    lib.coat_fp8_gemm_bf16.restype = ctypes.c_int
    lib.coat_fp8_gemm_bf16.argtypes = [vp, vp, f32, f32, i64, i64, i64, vp, vp]
    for name in ("rms_norm", "rms_norm_bwd", "swiglu", "qk_norm_rope", "qk_norm_rope_bwd", "weight_grad"):
        fn = getattr(lib, f"coat_fp8_{name}")
        fn.restype = ctypes.c_int
        fn.argtypes = [vp, vp]   # a structure by reference, or its packed bytes
    lib.coat_fp8_swiglu_bwd.restype = ctypes.c_int
    lib.coat_fp8_swiglu_bwd.argtypes = [vp, vp, vp, i64, i64, i32, vp, vp]
    lib.coat_fp8_rms_norm_bwd_workspace.restype = i64
    lib.coat_fp8_rms_norm_bwd_workspace.argtypes = [i64, i64]
    lib.coat_fp8_qk_norm_rope_bwd_workspace.restype = i64
    lib.coat_fp8_qk_norm_rope_bwd_workspace.argtypes = [i64, i64, i64]
    lib.coat_fp8_weight_grad_workspace.restype = i64
    lib.coat_fp8_weight_grad_workspace.argtypes = [i64, i64, i64]
    lib.coat_status_string.restype = ctypes.c_char_p
    lib.coat_status_string.argtypes = [ctypes.c_int]
    lib.coat_last_hip_error.restype = ctypes.c_char_p
    lib.coat_last_hip_error.argtypes = []
    lib.coat_abi_version.restype = ctypes.c_int32
    lib.coat_abi_version.argtypes = []
    if lib.coat_abi_version() != ABI_VERSION:
        raise ImportError(f"{path}: ABI version {lib.coat_abi_version()}, "
                          f"binding expects {ABI_VERSION}")
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.coat_status_string(status).decode()


def _check(status: int):
    if status != COAT_OK:
        msg = status_string(status)
        if status == COAT_ERR_HIP:
            msg += ": " + lib.coat_last_hip_error().decode()
        raise CoatError(status, msg)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


# dtypes accepted for each kind of buffer (bit-pattern views are fine)
CODE_DTYPES = (torch.uint8, torch.int8, torch.float8_e4m3fn)
BF16_DTYPES = (torch.bfloat16, torch.int16)
F32_DTYPES = (torch.float32,)


def _need(t: torch.Tensor, name: str, dtypes, min_numel: int):
    """Marshalling checks the C ABI cannot make: the kernels read and write
    through raw device pointers, so a buffer of the wrong type, layout, size
    or device would be accessed out of bounds.  Raises ValueError."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {min_numel}")


def _on_device(**tensors):
    """Every given buffer is HIP device memory on the current device, where
    the library launches its kernels (after the type and size checks)."""
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA (HIP device) tensor, not {t.device}")
        if dev is None:
            dev = torch.cuda.current_device()
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, but the current device "
                             f"is cuda:{dev}")


# The current device, and torch's current stream on a device as a raw handle.
# torch's own queries cost about 0.1 us per call, its public ones 0.3 and 3 us,
# as long as a small kernel; those are taken where a torch lacks the others.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _raw_stream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        if stream.device_index != torch.cuda.current_device():
            raise ValueError(f"stream is on cuda:{stream.device_index}, but the current device "
                             f"is cuda:{torch.cuda.current_device()}")
        return stream.cuda_stream
    return int(stream)


def _fits_c_int(group_size):
    """ctypes cuts a number to the argument's 32 bits: the size that the
    library would see is then not the one the buffers were checked for."""
    if not -(1 << 31) <= group_size < 1 << 31:
        raise ValueError(f"group_size {group_size} does not fit its C type")


def num_groups(n: int, group_size: int) -> int:
    return (n + group_size - 1) // group_size


@dataclass(frozen=True)
class QuantState:
    """One FP8 moment on the device: codes uint8[n], scale/k float32[ng]."""
    codes: torch.Tensor
    scale: torch.Tensor
    k: torch.Tensor

    @classmethod
    def zeros(cls, n: int, group_size: int, device="cuda") -> "QuantState":
        ng = num_groups(n, group_size)
        return cls(torch.zeros(n, dtype=torch.uint8, device=device),
                   torch.zeros(ng, dtype=torch.float32, device=device),
                   torch.zeros(ng, dtype=torch.float32, device=device))

    def as_c(self) -> FP8State:
        return FP8State(_ptr(self.codes), _ptr(self.scale), _ptr(self.k))

    def check(self, n: int, group_size: int, name: str):
        _fits_c_int(group_size)
        _need(self.codes, f"{name}.codes", CODE_DTYPES, n)
        _need(self.scale, f"{name}.scale", F32_DTYPES, num_groups(n, group_size))
        _need(self.k, f"{name}.k", F32_DTYPES, num_groups(n, group_size))

    def check_device(self, name: str):
        _on_device(**{f"{name}.codes": self.codes, f"{name}.scale": self.scale,
                      f"{name}.k": self.k})


@dataclass(frozen=True)
class ParamSlot:
    """One tensor of an optimizer shard: FP32 weights, BF16 gradient, m, v.
    Frozen, like QuantState: a TensorList copies the tensors' device pointers
    once, so a slot's tensors cannot be swapped after it is built (build a new
    slot, e.g. with dataclasses.replace, and a new TensorList instead)."""
    w: torch.Tensor
    grad: torch.Tensor
    m: QuantState
    v: QuantState

    def as_c(self) -> AdamWTensor:
        return AdamWTensor(_ptr(self.w), _ptr(self.grad), self.m.as_c(),
                           self.v.as_c(), self.w.numel())

    def check(self, group_size: int, name: str = "slot"):
        n = self.w.numel()
        _need(self.w, f"{name}.w", F32_DTYPES, n)
        _need(self.grad, f"{name}.grad", BF16_DTYPES, n)
        self.m.check(n, group_size, f"{name}.m")
        self.v.check(n, group_size, f"{name}.v")
        _on_device(**{f"{name}.w": self.w, f"{name}.grad": self.grad})
        self.m.check_device(f"{name}.m")
        self.v.check_device(f"{name}.v")


class TensorList:
    """Marshalled descriptor array for coat_adamw_fp8_step, built once and
    reused across steps (the pointers stay valid while the tensors live: the
    list holds the slots, and slots are frozen).  The buffer checks run once
    per group size and again whenever the current device differs from the
    one they ran on (the library launches on the current device)."""

    def __init__(self, slots: Sequence[ParamSlot]):
        self.slots = list(slots)
        self.array = (AdamWTensor * max(1, len(self.slots)))(
            *[s.as_c() for s in self.slots])
        self._checked = set()   # (group size, device index) the slots have been checked for

    def check(self, group_size: int):
        key = (group_size, torch.cuda.current_device() if torch.cuda.is_initialized() else -1)
        if key not in self._checked:
            for i, slot in enumerate(self.slots):
                slot.check(group_size, f"tensors[{i}]")
            self._checked.add(key)

    def __len__(self):
        return len(self.slots)


def adamw_fp8_step(tensors, *, lr: float, beta1: float, beta2: float, eps: float,
                   weight_decay: float, step: int, group_size: int = 128, stream=None):
    """One fused FP8 AdamW step over `tensors` (a TensorList or a sequence of
    ParamSlot).  Enqueued on `stream` (torch's current stream by default)."""
    tl = tensors if isinstance(tensors, TensorList) else TensorList(tensors)
    tl.check(group_size)
    hp = AdamWHParams(lr, beta1, beta2, eps, weight_decay, step, group_size)
    _check(lib.coat_adamw_fp8_step(ctypes.addressof(tl.array), len(tl),
                                   ctypes.byref(hp), _stream(stream)))


def adamw_fp8_step_raw(array_ptr: Optional[int], num_tensors: int, hp: AdamWHParams,
                       stream=None) -> int:
    """Direct call with a caller-built descriptor array; returns the status."""
    return lib.coat_adamw_fp8_step(array_ptr, num_tensors,
                                   ctypes.byref(hp) if hp is not None else None,
                                   _stream(stream))


def expand_quantize(x: torch.Tensor, out: QuantState, group_size: int = 128, stream=None):
    _need(x, "x", F32_DTYPES, 0)
    out.check(x.numel(), group_size, "out")
    _on_device(x=x)
    out.check_device("out")
    _check(lib.coat_fp8_expand_quantize(_ptr(x), x.numel(), group_size, out.as_c(),
                                        _stream(stream)))


def dequantize_expand(state: QuantState, out: torch.Tensor, group_size: int = 128,
                      stream=None):
    state.check(state.codes.numel(), group_size, "state")
    _need(out, "out", F32_DTYPES, state.codes.numel())
    state.check_device("state")
    _on_device(out=out)
    _check(lib.coat_fp8_dequantize_expand(
        _ptr(state.codes), _ptr(state.scale), _ptr(state.k), state.codes.numel(),
        group_size, _ptr(out), _stream(stream)))


def e4m3_encode(x: torch.Tensor, codes: torch.Tensor, stream=None):
    _need(x, "x", F32_DTYPES, 0)
    _need(codes, "codes", CODE_DTYPES, x.numel())
    _on_device(x=x, codes=codes)
    _check(lib.coat_e4m3_encode(_ptr(x), x.numel(), _ptr(codes), _stream(stream)))


def e4m3_decode(codes: torch.Tensor, x: torch.Tensor, stream=None):
    _need(codes, "codes", CODE_DTYPES, 0)
    _need(x, "x", F32_DTYPES, codes.numel())
    _on_device(codes=codes, x=x)
    _check(lib.coat_e4m3_decode(_ptr(codes), codes.numel(), _ptr(x), _stream(stream)))


def quantize_act(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                 codes_t: Optional[torch.Tensor] = None, group_size: int = 128,
                 stream=None):
    """Per-group (1 x group_size) E4M3 quantization of a 2-D BF16 matrix x into
    codes (same shape, uint8), scales (rows x cols/group_size, float32) and,
    if given, codes_t (cols x rows, uint8)."""
    if x.dim() != 2:
        raise ValueError("quantize_act expects a 2-D (rows, cols) tensor")
    rows, cols = x.shape
    _fits_c_int(group_size)
    _need(x, "x", BF16_DTYPES, 0)
    _need(codes, "codes", CODE_DTYPES, rows * cols)
    _need(scales, "scales", F32_DTYPES, rows * (cols // max(group_size, 1)))
    if codes_t is not None:
        _need(codes_t, "codes_t", CODE_DTYPES, rows * cols)
    _on_device(x=x, codes=codes, scales=scales, codes_t=codes_t)
    _check(lib.coat_fp8_quantize_act(_ptr(x), rows, cols, group_size, _ptr(codes),
                                     _ptr(scales), _ptr(codes_t), _stream(stream)))


def gemm_group_quant(a: torch.Tensor, b: torch.Tensor, a_scale: float, b_scale: float,
                     codes: torch.Tensor, scales: torch.Tensor, group_size: int = 128,
                     c_f32: Optional[torch.Tensor] = None, stream=None):
    """C = a_scale * b_scale * a @ b.T from E4M3 codes a (M x K) and b (N x K),
    quantized per 1 x group_size group of each row into codes (M x N) and
    scales (M x N/group_size); optionally also writes C in FP32."""
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b disagree on K")
    _fits_c_int(group_size)
    _need(a, "a", CODE_DTYPES, 0)
    _need(b, "b", CODE_DTYPES, 0)
    _need(codes, "codes", CODE_DTYPES, M * N)
    _need(scales, "scales", F32_DTYPES, M * (N // max(group_size, 1)))
    if c_f32 is not None:
        _need(c_f32, "c_f32", F32_DTYPES, M * N)
    _on_device(a=a, b=b, codes=codes, scales=scales, c_f32=c_f32)
    _check(lib.coat_fp8_gemm_group_quant(_ptr(a), _ptr(b), a_scale, b_scale, M, N, K,
                                         group_size, _ptr(codes), _ptr(scales), _ptr(c_f32),
                                         _stream(stream)))


def gemm_bf16(a: torch.Tensor, b: torch.Tensor, a_scale: float, b_scale: float,
              c_bf16: torch.Tensor, stream=None):
    """C = a_scale * b_scale * a @ b.T from E4M3 codes, rounded to BF16."""
    M, K = a.shape
    N = b.shape[0]
    if b.shape[1] != K:
        raise ValueError("a and b disagree on K")
    _need(a, "a", CODE_DTYPES, 0)
    _need(b, "b", CODE_DTYPES, 0)
    _need(c_bf16, "c_bf16", BF16_DTYPES, M * N)
    _on_device(a=a, b=b, c_bf16=c_bf16)
    _check(lib.coat_fp8_gemm_bf16(_ptr(a), _ptr(b), a_scale, b_scale, M, N, K, _ptr(c_bf16),
                                  _stream(stream)))


# ------------------------------------------------- activation checkpoints

_pack_rms_norm, _pack_rms_norm_bwd = _packer(RMSNormArgs), _packer(RMSNormBwdArgs)
_pack_swiglu, _pack_weight_grad = _packer(SwigluArgs), _packer(WeightGradArgs)
_pack_qk, _pack_qk_bwd = _packer(QkNormRopeArgs), _packer(QkNormRopeBwdArgs)
CODES, BF16, F32 = CODE_DTYPES, BF16_DTYPES, F32_DTYPES


def _addresses(buffers, heads=()):
    """Addresses (0 for None) of `buffers`, (tensor, name, dtypes, least number
    of values) each, then of `heads` (checked by _heads but for the device),
    (tensor, name) each, after the checks of _need and _on_device; and the
    raw handle of torch's current stream.  One pass over what is right; what
    is not is gone through again for its message."""
    out = []
    dev = None
    try:
        for t, _, dtypes, n in buffers:
            if t is None:
                out.append(0)
                continue
            d = t.get_device()
            if d != dev:
                if dev is not None or d < 0 or d != _current_device():
                    return _refuse(buffers, heads)
                dev = d
            if t.dtype not in dtypes or not t.is_contiguous() or t.numel() < n:
                return _refuse(buffers, heads)
            out.append(t.data_ptr())
        for t, _ in heads:
            if t.get_device() != dev:
                return _refuse(buffers, heads)
            out.append(t.data_ptr())
    except AttributeError:   # not a tensor
        return _refuse(buffers, heads)
    return out, _raw_stream(dev)


def _refuse(buffers, heads):
    for t, name, dtypes, n in buffers:
        if t is not None:
            _need(t, name, dtypes, n)
    _on_device(**{b[1]: b[0] for b in buffers}, **dict((name, t) for t, name in heads))
    raise ValueError("no buffer on the current device")


def _launch(fn, packed: bytes, stream, current):
    status = fn(packed, current if stream is None else _stream(stream))
    if status != COAT_OK:
        _check(status)


def _shape2(t, name: str):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return t.shape


def _groups(cols: int, group_size: int) -> int:
    return cols // group_size if group_size > 0 else 0


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, *, y: Optional[torch.Tensor] = None,
             y_codes: Optional[torch.Tensor] = None, y_scale: float = 1.0,
             y_amax: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
             scales: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
             group_size: int = 128, stream=None):
    """RMS norm of h = x (+ residual, written to residual_out, which may be
    residual) into y (BF16) and/or y_codes (E4M3 under the one scale y_scale;
    y_amax is raised to the largest |y|).  codes and scales, if given, receive
    h's checkpoint and rstd the rows' reciprocal root mean squares, for
    rms_norm_bwd."""
    rows, cols = _shape2(x, "x")
    n = rows * cols
    p, current = _addresses((
        (x, "x", BF16, 0), (residual, "residual", BF16, n), (weight, "weight", BF16, cols),
        (residual_out, "residual_out", BF16, n), (y, "y", BF16, n), (y_codes, "y_codes", CODES, n),
        (y_amax, "y_amax", F32, 1), (codes, "codes", CODES, n),
        (scales, "scales", F32, rows * _groups(cols, group_size)), (rstd, "rstd", F32, rows)))
    _launch(lib.coat_fp8_rms_norm, _pack_rms_norm(*p, rows, cols, eps, y_scale, group_size), stream, current)


def rms_norm_bwd_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace rms_norm_bwd needs for a weight gradient."""
    return _workspace_bytes(lib.coat_fp8_rms_norm_bwd_workspace, rows, cols)


def _workspace_bytes(fn, *sizes: int) -> int:
    if max(sizes) >= 1 << 63 or min(sizes) < 0:   # (ctypes would cut them to 64 bits)
        _check(COAT_ERR_INVALID_VALUE)
    n = fn(*sizes)
    if n < 0:
        _check(COAT_ERR_INVALID_VALUE)
    return n


def _workspace(workspace, nbytes: int) -> int:
    """The workspace's size in bytes; at least nbytes."""
    if workspace is None:
        if nbytes > 0:
            raise ValueError(f"workspace is required ({nbytes} bytes)")
        return 0
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous torch.Tensor")
    have = workspace.nbytes
    if have < nbytes:
        raise ValueError(f"workspace holds {have} bytes, needs at least {nbytes}")
    return have


class _AnyDtype:
    def __contains__(self, dtype):
        return True


ANY = _AnyDtype()   # the workspace's dtype does not matter


def rms_norm_bwd(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, rstd: torch.Tensor,
                 weight: torch.Tensor, dx: torch.Tensor, dw: Optional[torch.Tensor] = None, *,
                 d_residual: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 accumulate: bool = False, group_size: int = 128, stream=None):
    """Gradient of rms_norm from its checkpoint: dx (BF16, d_residual added if
    given; not dy itself, which other blocks still read) and, if given, dw
    (FP32, written or accumulated; needs rms_norm_bwd_workspace(rows, cols)
    bytes of workspace)."""
    rows, cols = _shape2(dy, "dy")
    n = rows * cols
    ws_bytes = _workspace(workspace, rms_norm_bwd_workspace(rows, cols) if dw is not None else 0)
    p, current = _addresses((
        (dy, "dy", BF16, 0), (codes, "codes", CODES, n),
        (scales, "scales", F32, rows * _groups(cols, group_size)), (rstd, "rstd", F32, rows),
        (weight, "weight", BF16, cols), (d_residual, "d_residual", BF16, n), (dx, "dx", BF16, n),
        (dw, "dw", F32, cols), (workspace, "workspace", ANY, 0)))
    _launch(lib.coat_fp8_rms_norm_bwd,
            _pack_rms_norm_bwd(*p, ws_bytes, rows, cols, group_size, accumulate), stream, current)


def swiglu(codes: Optional[torch.Tensor], scales: Optional[torch.Tensor], *,
           gate_up: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
           h_codes: Optional[torch.Tensor] = None, h_scale: float = 1.0,
           h_amax: Optional[torch.Tensor] = None, group_size: int = 128, stream=None):
    """Gated activation gate * sigmoid(gate) * up of rows that hold the gates,
    then the ups, into h (BF16) or h_codes (E4M3 under the one scale h_scale;
    h_amax is raised to the largest |h|).  The input is the checkpoint codes,
    scales; or gate_up (BF16), whose checkpoint is then written to codes and
    scales if they are given."""
    rows, wide = _shape2(codes, "codes") if gate_up is None else _shape2(gate_up, "gate_up")
    if wide % 2:
        raise ValueError("a row holds the gates and as many ups: its length is even")
    cols = wide // 2
    p, current = _addresses((
        (gate_up, "gate_up", BF16, 0), (codes, "codes", CODES, rows * wide),
        (scales, "scales", F32, 2 * rows * _groups(cols, group_size)), (h, "h", BF16, rows * cols),
        (h_codes, "h_codes", CODES, rows * cols), (h_amax, "h_amax", F32, 1)))
    _launch(lib.coat_fp8_swiglu, _pack_swiglu(*p, rows, cols, h_scale, group_size), stream, current)


def swiglu_bwd(dh: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, d_gate_up: torch.Tensor,
               group_size: int = 128, stream=None):
    """Gradient of swiglu from its checkpoint: d_gate_up (BF16), the gates'
    gradients first in each row."""
    rows, cols = _shape2(dh, "dh")
    _fits_c_int(group_size)
    (a, b, c, d), current = _addresses((
        (dh, "dh", BF16, 0), (codes, "codes", CODES, 2 * rows * cols),
        (scales, "scales", F32, 2 * rows * _groups(cols, group_size)),
        (d_gate_up, "d_gate_up", BF16, 2 * rows * cols)))
    _check(lib.coat_fp8_swiglu_bwd(a, b, c, rows, cols, group_size, d,
                                   current if stream is None else _stream(stream)))


def _heads(t: torch.Tensor, name: str, like=None):
    """(tokens, heads, head_dim, token stride) of a tensor of heads, which may
    be part of a packed projection: only the token stride is free."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D (tokens, heads, head_dim) tensor")
    if t.dtype not in BF16_DTYPES:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {BF16_DTYPES}")
    shape = t.shape
    tokens, heads, dim = shape
    if like is not None and shape != like:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {tuple(like)}")
    s0, s1, s2 = t.stride()
    if tokens <= 1:
        s0 = heads * dim
    if tokens and heads and dim and ((dim > 1 and s2 != 1) or (heads > 1 and s1 != dim) or s0 < heads * dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return tokens, heads, dim, s0


def _qk_sizes(q, k, q_other, k_other, cos, sin, names):
    """Sizes and strides that both passes take from their heads and tables."""
    try:   # the usual case in one look
        qs, ks = q.shape, k.shape
        tokens, q_heads, dim = qs
        k_heads = ks[1]
        a, b, c, d = q.stride(), k.stride(), q_other.stride(), k_other.stride()
        plain = (tokens > 0 and ks[0] == tokens and ks[2] == dim and q_other.shape == qs and k_other.shape == ks
                 and a[1] == b[1] == c[1] == d[1] == dim and a[2] == b[2] == c[2] == d[2] == 1
                 and (tokens == 1 or a[0] >= q_heads * dim <= c[0] and b[0] >= k_heads * dim <= d[0])
                 and q.dtype in BF16 and k.dtype in BF16 and q_other.dtype in BF16 and k_other.dtype in BF16)
    except (AttributeError, ValueError, IndexError):
        plain = False
    if plain:
        strides = (a[0], b[0], c[0], d[0]) if tokens > 1 else (q_heads * dim, k_heads * dim) * 2
    else:
        tokens, q_heads, dim, q_stride = _heads(q, names[0])
        k_tokens, k_heads, k_dim, k_stride = _heads(k, names[1])
        if k_tokens != tokens or k_dim != dim:
            raise ValueError(f"{names[0]} and {names[1]} disagree on tokens or head_dim")
        strides = (q_stride, k_stride, _heads(q_other, names[2], q.shape)[3], _heads(k_other, names[3], k.shape)[3])
    table_rows, half = _shape2(cos, "cos")
    if _shape2(sin, "sin") != cos.shape:
        raise ValueError("cos and sin differ in shape")
    return (tokens, q_heads, k_heads, dim, table_rows, 2 * half, *strides)


I64_DTYPES = (torch.int64,)


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                 eps: float, cos: torch.Tensor, sin: torch.Tensor, positions: torch.Tensor,
                 q_out: torch.Tensor, k_out: torch.Tensor, *, codes: Optional[torch.Tensor] = None,
                 scales: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                 interleaved: bool = False, group_size: int = 128, stream=None):
    """RMS norm of every head of q and k (tokens x heads x head_dim, possibly
    parts of one packed projection) and their rotation by row positions[token]
    of cos and sin (rows x rot_dim/2, FP32) into q_out and k_out, which may be
    q and k.  codes, scales and rstd, if given, receive the checkpoint (the
    query heads of a token, then its key heads).  Tokens whose position is
    outside the tables are padding and get zeros."""
    tokens, q_heads, k_heads, dim, table, rot, qs, ks, qos, kos = _qk_sizes(
        q, k, q_out, k_out, cos, sin, ("q", "k", "q_out", "k_out"))
    rows = tokens * (q_heads + k_heads)
    (wq, wk, c, s, pos, pc, ps, pr, pq, pk, pqo, pko), current = _addresses((
        (q_weight, "q_weight", BF16, dim), (k_weight, "k_weight", BF16, dim), (cos, "cos", F32, 0),
        (sin, "sin", F32, 0), (positions, "positions", I64_DTYPES, tokens), (codes, "codes", CODES, rows * dim),
        (scales, "scales", F32, rows * _groups(dim, group_size)), (rstd, "rstd", F32, rows)),
        ((q, "q"), (k, "k"), (q_out, "q_out"), (k_out, "k_out")))
    _launch(lib.coat_fp8_qk_norm_rope,
            _pack_qk(tokens, table, q_heads, k_heads, dim, rot, interleaved, group_size, pq, pk, qs, ks, wq, wk, c, s,
                     pos, pqo, pko, qos, kos, pc, ps, pr, eps), stream, current)


def qk_norm_rope_bwd_workspace(tokens: int, heads: int, head_dim: int) -> int:
    """Bytes of workspace qk_norm_rope_bwd needs for weight gradients (heads:
    queries and keys)."""
    return _workspace_bytes(lib.coat_fp8_qk_norm_rope_bwd_workspace, tokens, heads, head_dim)


def qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor, codes: torch.Tensor,
                     scales: torch.Tensor, rstd: torch.Tensor, q_weight: torch.Tensor,
                     k_weight: torch.Tensor, cos: torch.Tensor, sin: torch.Tensor,
                     positions: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor,
                     dq_weight: Optional[torch.Tensor] = None, dk_weight: Optional[torch.Tensor] = None,
                     *, workspace: Optional[torch.Tensor] = None, accumulate: bool = False,
                     interleaved: bool = False, group_size: int = 128, stream=None):
    """Gradient of qk_norm_rope from its checkpoint: dq and dk (BF16; they may
    be dq_out and dk_out) and, if given, dq_weight and dk_weight (FP32,
    written or accumulated; need qk_norm_rope_bwd_workspace bytes)."""
    tokens, q_heads, k_heads, dim, table, rot, qos, kos, qs, ks = _qk_sizes(
        dq_out, dk_out, dq, dk, cos, sin, ("dq_out", "dk_out", "dq", "dk"))
    rows = tokens * (q_heads + k_heads)
    ws_bytes = _workspace(workspace, qk_norm_rope_bwd_workspace(tokens, q_heads + k_heads, dim)
                          if dq_weight is not None else 0)
    (pc, ps, pr, wq, wk, c, s, pos, dwq, dwk, ws, pqo, pko, pq, pk), current = _addresses((
        (codes, "codes", CODES, rows * dim), (scales, "scales", F32, rows * _groups(dim, group_size)),
        (rstd, "rstd", F32, rows), (q_weight, "q_weight", BF16, dim), (k_weight, "k_weight", BF16, dim),
        (cos, "cos", F32, 0), (sin, "sin", F32, 0), (positions, "positions", I64_DTYPES, tokens),
        (dq_weight, "dq_weight", F32, dim), (dk_weight, "dk_weight", F32, dim), (workspace, "workspace", ANY, 0)),
        ((dq_out, "dq_out"), (dk_out, "dk_out"), (dq, "dq"), (dk, "dk")))
    _launch(lib.coat_fp8_qk_norm_rope_bwd,
            _pack_qk_bwd(tokens, table, q_heads, k_heads, dim, rot, interleaved, group_size, pqo, pko, qos, kos, pc, ps,
                         pr, wq, wk, c, s, pos, pq, pk, qs, ks, dwq, dwk, ws, ws_bytes, accumulate), stream, current)


def weight_grad_workspace(rows: int, n: int, k: int) -> int:
    """Bytes of workspace weight_grad needs (0: none)."""
    return _workspace_bytes(lib.coat_fp8_weight_grad_workspace, rows, n, k)


def weight_grad(dy: torch.Tensor, codes: torch.Tensor, scales, dw: torch.Tensor, *,
                accumulate: bool = False, workspace: Optional[torch.Tensor] = None,
                group_size: int = 128, stream=None):
    """dw = dy^T X for a linear layer whose input X (rows x K) was kept as E4M3
    codes: with group scales (a float32 tensor, rows x K/group_size) or under
    one scale (a number).  dy is rows x N BF16, dw N x K BF16 or float32; a
    float32 dw can be accumulated into.  Group scales round X to BF16 for a
    BF16 dw; a float32 one holds it to 2^-16, in twice the products.  Needs weight_grad_workspace bytes."""
    rows, n = _shape2(dy, "dy")
    x_rows, k = _shape2(codes, "codes")
    if x_rows != rows:
        raise ValueError("dy and codes disagree on the rows")
    grouped, x_scale = None, 1.0
    if isinstance(scales, torch.Tensor):
        grouped = scales
    elif isinstance(scales, (int, float)):
        x_scale = scales
    else:
        raise ValueError("scales must be a float32 tensor or a number")
    if not isinstance(dw, torch.Tensor):
        raise ValueError("dw must be a torch.Tensor")
    ws_bytes = _workspace(workspace, weight_grad_workspace(rows, n, k))
    (py, px, ps, pw, ws), current = _addresses((
        (dy, "dy", BF16, 0), (codes, "codes", CODES, 0),
        (grouped, "scales", F32, rows * _groups(k, group_size)), (dw, "dw", DW_DTYPES, n * k),
        (workspace, "workspace", ANY, 0)))
    f32 = dw.dtype == torch.float32
    _launch(lib.coat_fp8_weight_grad,
            _pack_weight_grad(py, px, ps, 0 if f32 else pw, pw if f32 else 0, ws, ws_bytes, rows, n, k, x_scale,
                              group_size, accumulate), stream, current)


DW_DTYPES = BF16_DTYPES + F32_DTYPES
