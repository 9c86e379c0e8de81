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
    for name, args in (("rms_norm", RMSNormArgs), ("rms_norm_bwd", RMSNormBwdArgs),
                       ("swiglu", SwigluArgs), ("qk_norm_rope", QkNormRopeArgs),
                       ("qk_norm_rope_bwd", QkNormRopeBwdArgs), ("weight_grad", WeightGradArgs)):
        fn = getattr(lib, f"coat_fp8_{name}")
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.POINTER(args), vp]
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


def _stream(stream) -> Optional[int]:
    if stream is None:
        # torch's current stream on the current device, as a raw handle: this
        # query costs about 0.1 us per call, torch.cuda.current_stream() about
        # 3 us, as long as a small kernel
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


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

def _shape2(t, name: str):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    return t.shape


def _opt(t, name: str, dtypes, min_numel: int):
    if t is not None:
        _need(t, name, dtypes, min_numel)


def _groups(cols: int, group_size: int) -> int:
    return cols // group_size if group_size > 0 else 0


def rms_norm(x: torch.Tensor, weight: torch.Tensor, eps: float, *, y: Optional[torch.Tensor] = None,
             y_codes: Optional[torch.Tensor] = None, y_scale: float = 1.0,
             y_amax: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None, codes: Optional[torch.Tensor] = None,
             scales: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
             group_size: int = 128, stream=None):
    """RMS norm of h = x (+ residual, written to residual_out) into y (BF16)
    and/or y_codes (E4M3 under the one scale y_scale; y_amax is raised to the
    largest |y|).  codes and scales, if given, receive h's checkpoint and rstd
    the rows' reciprocal root mean squares, for rms_norm_bwd."""
    rows, cols = _shape2(x, "x")
    n = rows * cols
    _need(x, "x", BF16_DTYPES, 0)
    _need(weight, "weight", BF16_DTYPES, cols)
    _opt(residual, "residual", BF16_DTYPES, n)
    _opt(residual_out, "residual_out", BF16_DTYPES, n)
    _opt(y, "y", BF16_DTYPES, n)
    _opt(y_codes, "y_codes", CODE_DTYPES, n)
    _opt(y_amax, "y_amax", F32_DTYPES, 1)
    _opt(codes, "codes", CODE_DTYPES, n)
    _opt(scales, "scales", F32_DTYPES, rows * _groups(cols, group_size))
    _opt(rstd, "rstd", F32_DTYPES, rows)
    _on_device(x=x, weight=weight, residual=residual, residual_out=residual_out, y=y, y_codes=y_codes,
               y_amax=y_amax, codes=codes, scales=scales, rstd=rstd)
    a = RMSNormArgs(_ptr(x), _ptr(residual), _ptr(weight), _ptr(residual_out), _ptr(y), _ptr(y_codes),
                    _ptr(y_amax), _ptr(codes), _ptr(scales), _ptr(rstd), rows, cols, eps, y_scale,
                    group_size)
    _check(lib.coat_fp8_rms_norm(ctypes.byref(a), _stream(stream)))


def rms_norm_bwd_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace rms_norm_bwd needs for a weight gradient."""
    return _workspace_bytes(lib.coat_fp8_rms_norm_bwd_workspace(rows, cols))


def _workspace_bytes(n: int) -> int:
    if n < 0:
        _check(COAT_ERR_INVALID_VALUE)
    return n


def _workspace(workspace, need: bool, nbytes: int):
    """Address and size of the workspace: a byte count of `nbytes` is required
    where `need`."""
    if workspace is None:
        if need and nbytes > 0:
            raise ValueError(f"workspace is required ({nbytes} bytes)")
        return None, 0
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous torch.Tensor")
    have = workspace.numel() * workspace.element_size()
    if need and have < nbytes:
        raise ValueError(f"workspace holds {have} bytes, needs at least {nbytes}")
    return workspace.data_ptr(), have


def rms_norm_bwd(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, rstd: torch.Tensor,
                 weight: torch.Tensor, dx: torch.Tensor, dw: Optional[torch.Tensor] = None, *,
                 d_residual: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 accumulate: bool = False, group_size: int = 128, stream=None):
    """Gradient of rms_norm from its checkpoint: dx (BF16, d_residual added if
    given) and, if given, dw (FP32, written or accumulated; needs
    rms_norm_bwd_workspace(rows, cols) bytes of workspace)."""
    rows, cols = _shape2(dy, "dy")
    n = rows * cols
    _need(dy, "dy", BF16_DTYPES, 0)
    _need(codes, "codes", CODE_DTYPES, n)
    _need(scales, "scales", F32_DTYPES, rows * _groups(cols, group_size))
    _need(rstd, "rstd", F32_DTYPES, rows)
    _need(weight, "weight", BF16_DTYPES, cols)
    _need(dx, "dx", BF16_DTYPES, n)
    _opt(dw, "dw", F32_DTYPES, cols)
    _opt(d_residual, "d_residual", BF16_DTYPES, n)
    need = dw is not None
    ws, ws_bytes = _workspace(workspace, need, rms_norm_bwd_workspace(rows, cols) if need else 0)
    _on_device(dy=dy, codes=codes, scales=scales, rstd=rstd, weight=weight, dx=dx, dw=dw,
               d_residual=d_residual, workspace=workspace)
    a = RMSNormBwdArgs(_ptr(dy), _ptr(codes), _ptr(scales), _ptr(rstd), _ptr(weight), _ptr(d_residual),
                       _ptr(dx), _ptr(dw), ws, ws_bytes, rows, cols, group_size, int(accumulate))
    _check(lib.coat_fp8_rms_norm_bwd(ctypes.byref(a), _stream(stream)))


def swiglu(codes: Optional[torch.Tensor], scales: Optional[torch.Tensor], *,
           gate_up: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
           h_codes: Optional[torch.Tensor] = None, h_scale: float = 1.0,
           h_amax: Optional[torch.Tensor] = None, group_size: int = 128, stream=None):
    """Gated activation gate * sigmoid(gate) * up of rows that hold the gates,
    then the ups, into h (BF16) or h_codes (E4M3 under the one scale h_scale;
    h_amax is raised to the largest |h|).  The input is the checkpoint codes,
    scales; or gate_up (BF16), whose checkpoint is then written to codes and
    scales if they are given."""
    rows, wide = _shape2(codes if gate_up is None else gate_up, "codes" if gate_up is None else "gate_up")
    if wide % 2:
        raise ValueError("a row holds the gates and as many ups: its length is even")
    cols = wide // 2
    _opt(gate_up, "gate_up", BF16_DTYPES, 0)
    _opt(codes, "codes", CODE_DTYPES, rows * wide)
    _opt(scales, "scales", F32_DTYPES, 2 * rows * _groups(cols, group_size))
    _opt(h, "h", BF16_DTYPES, rows * cols)
    _opt(h_codes, "h_codes", CODE_DTYPES, rows * cols)
    _opt(h_amax, "h_amax", F32_DTYPES, 1)
    _on_device(gate_up=gate_up, codes=codes, scales=scales, h=h, h_codes=h_codes, h_amax=h_amax)
    a = SwigluArgs(_ptr(gate_up), _ptr(codes), _ptr(scales), _ptr(h), _ptr(h_codes), _ptr(h_amax), rows,
                   cols, h_scale, group_size)
    _check(lib.coat_fp8_swiglu(ctypes.byref(a), _stream(stream)))


def swiglu_bwd(dh: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, d_gate_up: torch.Tensor,
               group_size: int = 128, stream=None):
    """Gradient of swiglu from its checkpoint: d_gate_up (BF16), the gates'
    gradients first in each row."""
    rows, cols = _shape2(dh, "dh")
    _need(dh, "dh", BF16_DTYPES, 0)
    _need(codes, "codes", CODE_DTYPES, 2 * rows * cols)
    _need(scales, "scales", F32_DTYPES, 2 * rows * _groups(cols, group_size))
    _need(d_gate_up, "d_gate_up", BF16_DTYPES, 2 * rows * cols)
    _on_device(dh=dh, codes=codes, scales=scales, d_gate_up=d_gate_up)
    _check(lib.coat_fp8_swiglu_bwd(_ptr(dh), _ptr(codes), _ptr(scales), rows, cols, group_size,
                                   _ptr(d_gate_up), _stream(stream)))


def _heads(t: torch.Tensor, name: str, like=None):
    """(tokens, heads, head_dim, token stride) of a tensor of heads, which may
    be part of a packed projection: only the token stride is free."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D (tokens, heads, head_dim) tensor")
    if t.dtype not in BF16_DTYPES:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {BF16_DTYPES}")
    tokens, heads, dim = t.shape
    if like is not None and tuple(t.shape) != tuple(like.shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape)}")
    stride = t.stride(0) if tokens > 1 else heads * dim
    if t.numel() and ((dim > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != dim)
                      or stride < heads * dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return tokens, heads, dim, stride


def _qk_shape(q, k, q_weight, k_weight, cos, sin, positions, interleaved, group_size, names):
    tokens, q_heads, dim, _ = _heads(q, names[0])
    k_tokens, k_heads, k_dim, _ = _heads(k, names[1])
    if k_tokens != tokens or k_dim != dim:
        raise ValueError(f"{names[0]} and {names[1]} disagree on tokens or head_dim")
    table_rows, half = _shape2(cos, "cos")
    if tuple(_shape2(sin, "sin")) != (table_rows, half):
        raise ValueError("cos and sin differ in shape")
    _need(cos, "cos", F32_DTYPES, 0)
    _need(sin, "sin", F32_DTYPES, 0)
    _need(q_weight, "q_weight", BF16_DTYPES, dim)
    _need(k_weight, "k_weight", BF16_DTYPES, dim)
    _need(positions, "positions", (torch.int64,), tokens)
    return QkShape(tokens, table_rows, q_heads, k_heads, dim, 2 * half, int(interleaved), group_size)


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
    s = _qk_shape(q, k, q_weight, k_weight, cos, sin, positions, interleaved, group_size, ("q", "k"))
    q_stride, k_stride = _heads(q, "q")[3], _heads(k, "k")[3]
    q_out_stride, k_out_stride = _heads(q_out, "q_out", q)[3], _heads(k_out, "k_out", k)[3]
    rows = s.tokens * (s.q_heads + s.k_heads)
    _opt(codes, "codes", CODE_DTYPES, rows * s.head_dim)
    _opt(scales, "scales", F32_DTYPES, rows * _groups(s.head_dim, group_size))
    _opt(rstd, "rstd", F32_DTYPES, rows)
    _on_device(q=q, k=k, q_weight=q_weight, k_weight=k_weight, cos=cos, sin=sin, positions=positions,
               q_out=q_out, k_out=k_out, codes=codes, scales=scales, rstd=rstd)
    a = QkNormRopeArgs(s, _ptr(q), _ptr(k), q_stride, k_stride, _ptr(q_weight), _ptr(k_weight), _ptr(cos),
                       _ptr(sin), _ptr(positions), _ptr(q_out), _ptr(k_out), q_out_stride, k_out_stride,
                       _ptr(codes), _ptr(scales), _ptr(rstd), eps)
    _check(lib.coat_fp8_qk_norm_rope(ctypes.byref(a), _stream(stream)))


def qk_norm_rope_bwd_workspace(tokens: int, heads: int, head_dim: int) -> int:
    """Bytes of workspace qk_norm_rope_bwd needs for weight gradients (heads:
    queries and keys)."""
    return _workspace_bytes(lib.coat_fp8_qk_norm_rope_bwd_workspace(tokens, heads, head_dim))


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
    s = _qk_shape(dq_out, dk_out, q_weight, k_weight, cos, sin, positions, interleaved, group_size,
                  ("dq_out", "dk_out"))
    dq_out_stride, dk_out_stride = _heads(dq_out, "dq_out")[3], _heads(dk_out, "dk_out")[3]
    dq_stride, dk_stride = _heads(dq, "dq", dq_out)[3], _heads(dk, "dk", dk_out)[3]
    heads = s.q_heads + s.k_heads
    _need(codes, "codes", CODE_DTYPES, s.tokens * heads * s.head_dim)
    _need(scales, "scales", F32_DTYPES, s.tokens * heads * _groups(s.head_dim, group_size))
    _need(rstd, "rstd", F32_DTYPES, s.tokens * heads)
    _opt(dq_weight, "dq_weight", F32_DTYPES, s.head_dim)
    _opt(dk_weight, "dk_weight", F32_DTYPES, s.head_dim)
    need = dq_weight is not None
    ws, ws_bytes = _workspace(workspace, need, qk_norm_rope_bwd_workspace(s.tokens, heads, s.head_dim)
                              if need else 0)
    _on_device(dq_out=dq_out, dk_out=dk_out, codes=codes, scales=scales, rstd=rstd, q_weight=q_weight,
               k_weight=k_weight, cos=cos, sin=sin, positions=positions, dq=dq, dk=dk,
               dq_weight=dq_weight, dk_weight=dk_weight, workspace=workspace)
    a = QkNormRopeBwdArgs(s, _ptr(dq_out), _ptr(dk_out), dq_out_stride, dk_out_stride, _ptr(codes),
                          _ptr(scales), _ptr(rstd), _ptr(q_weight), _ptr(k_weight), _ptr(cos), _ptr(sin),
                          _ptr(positions), _ptr(dq), _ptr(dk), dq_stride, dk_stride, _ptr(dq_weight),
                          _ptr(dk_weight), ws, ws_bytes, int(accumulate))
    _check(lib.coat_fp8_qk_norm_rope_bwd(ctypes.byref(a), _stream(stream)))


def weight_grad_workspace(rows: int, n: int, k: int) -> int:
    """Bytes of workspace weight_grad needs (0: none)."""
    return _workspace_bytes(lib.coat_fp8_weight_grad_workspace(rows, n, k))


def weight_grad(dy: torch.Tensor, codes: torch.Tensor, scales, dw: torch.Tensor, *,
                accumulate: bool = False, workspace: Optional[torch.Tensor] = None,
                group_size: int = 128, stream=None):
    """dw = dy^T X for a linear layer whose input X (rows x K) was kept as E4M3
    codes: with group scales (a float32 tensor, rows x K/group_size) or under
    one scale (a number).  dy is rows x N BF16, dw N x K BF16 or float32; a
    float32 dw can be accumulated into.  Needs weight_grad_workspace bytes."""
    rows, n = _shape2(dy, "dy")
    x_rows, k = _shape2(codes, "codes")
    if x_rows != rows:
        raise ValueError("dy and codes disagree on the rows")
    grouped = isinstance(scales, torch.Tensor)
    _need(dy, "dy", BF16_DTYPES, 0)
    _need(codes, "codes", CODE_DTYPES, 0)
    if grouped:
        _need(scales, "scales", F32_DTYPES, rows * _groups(k, group_size))
    elif not isinstance(scales, (int, float)):
        raise ValueError("scales must be a float32 tensor or a number")
    _need(dw, "dw", BF16_DTYPES + F32_DTYPES, n * k)
    ws, ws_bytes = _workspace(workspace, True, weight_grad_workspace(rows, n, k))
    _on_device(dy=dy, codes=codes, scales=scales if grouped else None, dw=dw, workspace=workspace)
    f32 = dw.dtype == torch.float32
    a = WeightGradArgs(_ptr(dy), _ptr(codes), _ptr(scales) if grouped else None, None if f32 else _ptr(dw),
                       _ptr(dw) if f32 else None, ws, ws_bytes, rows, n, k, 1.0 if grouped else scales,
                       group_size, int(accumulate))
    _check(lib.coat_fp8_weight_grad(ctypes.byref(a), _stream(stream)))
