"""Refusals of the activation operators, on the CPU: the C entry points return
their status before any HIP call (the pointers are never dereferenced), and
the binding raises ValueError on buffers the C side cannot see into."""
import ctypes
import os
import re
import subprocess
import tempfile

import pytest
import torch

from test_abi_exports import ROOT, _ensure_built

OK, NULLP, INVAL, GSIZE, MISAL = 0, 1, 2, 3, 4
A = 0x10000   # a fake, 16-byte aligned device address


@pytest.fixture(scope="module")
def coat():
    _ensure_built()
    from adamw_coat_fp8_amd import coat
    return coat


def call(coat, name, cls, base, **change):
    f = dict(base)
    f.update(change)
    shape = f.pop("shape", None)
    a = cls(**f)
    if shape is not None:
        a.shape = coat.QkShape(**shape)
    return getattr(coat.lib, f"coat_fp8_{name}")(ctypes.byref(a), None)


def test_structs_have_the_c_layout(coat):
    structs = {"coat_rms_norm_args_t": coat.RMSNormArgs, "coat_rms_norm_bwd_args_t": coat.RMSNormBwdArgs,
               "coat_swiglu_args_t": coat.SwigluArgs, "coat_qk_shape_t": coat.QkShape,
               "coat_qk_norm_rope_args_t": coat.QkNormRopeArgs,
               "coat_qk_norm_rope_bwd_args_t": coat.QkNormRopeBwdArgs,
               "coat_weight_grad_args_t": coat.WeightGradArgs}
    lines, want = [], []
    for c, py in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({c}));')
        want.append(ctypes.sizeof(py))
        for name, _ in py._fields_:
            lines.append(f'printf("%zu\\n", offsetof({c}, {name}));')
            want.append(getattr(py, name).offset)
    src = '#include <stdio.h>\n#include <stddef.h>\n#include "coat_fp8.h"\nint main(void) {' + "\n".join(lines) + "return 0;}"
    with tempfile.TemporaryDirectory() as d:
        open(os.path.join(d, "l.c"), "w").write(src)
        subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                        "-I", "/opt/rocm/include", os.path.join(d, "l.c"), "-o", os.path.join(d, "l")], check=True)
        got = subprocess.run([os.path.join(d, "l")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in got] == want


NORM = dict(x=A, weight=A, y=A, rows=4, cols=256, eps=1e-5, y_scale=1.0, group_size=128)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVAL), (dict(cols=-16), INVAL), (dict(cols=200), INVAL), (dict(cols=32768 + 128), INVAL),
    (dict(rows=1 << 60), INVAL), (dict(group_size=48), GSIZE), (dict(eps=0.0), INVAL), (dict(eps=-1.0), INVAL),
    (dict(eps=float("nan")), INVAL), (dict(y_codes=A, y_scale=0.0), INVAL), (dict(y_codes=A, y_scale=-1.0), INVAL),
    (dict(y_codes=A, y_scale=float("inf")), INVAL), (dict(y_codes=A, y_scale=1e-45), INVAL),
    (dict(y_amax=A), INVAL), (dict(x=None), NULLP), (dict(weight=None), NULLP), (dict(y=None), NULLP),
    (dict(residual=A), NULLP), (dict(residual_out=A), NULLP), (dict(codes=A), NULLP), (dict(scales=A), NULLP),
    (dict(x=A + 8), MISAL), (dict(weight=A + 2), MISAL), (dict(y=A + 4), MISAL),
    (dict(residual=A + 8, residual_out=A), MISAL), (dict(residual=A, residual_out=A + 8), MISAL),
    (dict(y_codes=A + 1), MISAL), (dict(codes=A + 8, scales=A), MISAL), (dict(codes=A, scales=A + 2), MISAL),
    (dict(rstd=A + 1), MISAL), (dict(rows=0, x=None, weight=None, y=None), OK), (dict(cols=0), OK)])
def test_rms_norm(coat, change, status):
    assert call(coat, "rms_norm", coat.RMSNormArgs, NORM, **change) == status


NORM_BWD = dict(dy=A, codes=A, scales=A, rstd=A, weight=A, dx=A, dw=A, workspace=A, workspace_bytes=4 * 256 * 4,
                rows=4, cols=256, group_size=128)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVAL), (dict(cols=130), INVAL), (dict(cols=65536), INVAL), (dict(group_size=0), GSIZE),
    (dict(workspace_bytes=4 * 256 * 4 - 1), INVAL), (dict(workspace=None), NULLP)] +
    [({n: None}, NULLP) for n in ("dy", "codes", "scales", "rstd", "weight", "dx")] +
    [({n: A + 2}, MISAL) for n in ("dy", "codes", "scales", "rstd", "weight", "dx", "dw", "d_residual", "workspace")] +
    [(dict(rows=0, accumulate=1), OK), (dict(rows=0, dw=None), OK), (dict(cols=0), OK)])
def test_rms_norm_bwd(coat, change, status):
    assert call(coat, "rms_norm_bwd", coat.RMSNormBwdArgs, NORM_BWD, **change) == status


SWIGLU = dict(codes=A, scales=A, h=A, rows=4, cols=256, h_scale=1.0, group_size=128)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVAL), (dict(cols=100), INVAL), (dict(cols=1 << 31), INVAL), (dict(rows=1 << 60), INVAL),
    (dict(group_size=8), GSIZE), (dict(h_codes=A), INVAL), (dict(h=None, h_codes=A, h_scale=0.0), INVAL),
    (dict(h=None, h_codes=A, h_scale=float("nan")), INVAL), (dict(h_amax=A), INVAL), (dict(h=None), NULLP),
    (dict(codes=None), NULLP), (dict(scales=None), NULLP), (dict(codes=None, scales=None), NULLP),
    (dict(gate_up=A, scales=None), NULLP), (dict(gate_up=A + 8), MISAL), (dict(codes=A + 8), MISAL),
    (dict(scales=A + 1), MISAL), (dict(h=A + 2), MISAL), (dict(h=None, h_codes=A + 4), MISAL),
    (dict(h=None, h_codes=A, h_amax=A + 2), MISAL), (dict(rows=0, codes=None, scales=None, h=None), OK)])
def test_swiglu(coat, change, status):
    assert call(coat, "swiglu", coat.SwigluArgs, SWIGLU, **change) == status


def test_swiglu_bwd(coat):
    f = coat.lib.coat_fp8_swiglu_bwd
    assert f(A, A, A, -1, 128, 128, A, None) == INVAL
    assert f(A, A, A, 1, 130, 128, A, None) == INVAL
    assert f(A, A, A, 1, 128, 100, A, None) == GSIZE
    assert f(None, None, None, 0, 128, 128, None, None) == OK
    for i in (0, 1, 2, 6):
        args = [A, A, A, 1, 128, 128, A, None]
        args[i] = None
        assert f(*args) == NULLP
        args[i] = A + 2
        assert f(*args) == MISAL


SHAPE = dict(tokens=4, table_rows=32, q_heads=4, k_heads=2, head_dim=128, rot_dim=128, interleaved=0, group_size=64)
QK = dict(q=A, k=A, q_stride=1024, k_stride=1024, q_weight=A, k_weight=A, cos=A, sin=A, positions=A, q_out=A,
          k_out=A, q_out_stride=512, k_out_stride=256, eps=1e-5)
BAD_SHAPES = [(dict(tokens=-1), INVAL), (dict(q_heads=-1), INVAL), (dict(k_heads=70000), INVAL),
              (dict(table_rows=-1), INVAL), (dict(head_dim=120), INVAL), (dict(head_dim=272, group_size=16), INVAL),
              (dict(head_dim=96), INVAL), (dict(rot_dim=0), INVAL), (dict(rot_dim=24), INVAL),
              (dict(rot_dim=144), INVAL), (dict(group_size=7), GSIZE), (dict(tokens=1 << 40), INVAL)]


@pytest.mark.parametrize("shape,status", BAD_SHAPES + [(dict(tokens=0), OK), (dict(q_heads=0, k_heads=0), OK)])
def test_qk_shapes(coat, shape, status):
    assert call(coat, "qk_norm_rope", coat.QkNormRopeArgs, QK, shape={**SHAPE, **shape}) == status
    if status != OK:
        assert call(coat, "qk_norm_rope_bwd", coat.QkNormRopeBwdArgs, QK_BWD, shape={**SHAPE, **shape}) == status


@pytest.mark.parametrize("change,status", [
    (dict(q_stride=510), INVAL), (dict(q_stride=504), INVAL), (dict(k_stride=-8), INVAL), (dict(q_out_stride=1 << 62), INVAL),
    (dict(eps=0.0), INVAL), (dict(codes=A), NULLP), (dict(scales=A), NULLP)] +
    [({n: None}, NULLP) for n in ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "q_out", "k_out")] +
    [({n: A + 2}, MISAL) for n in ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "q_out", "k_out", "rstd")] +
    [(dict(codes=A + 8, scales=A), MISAL), (dict(codes=A, scales=A + 2), MISAL)])
def test_qk_norm_rope(coat, change, status):
    assert call(coat, "qk_norm_rope", coat.QkNormRopeArgs, QK, shape=SHAPE, **change) == status


QK_BWD = dict(dq_out=A, dk_out=A, dq_out_stride=512, dk_out_stride=256, codes=A, scales=A, rstd=A, q_weight=A,
              k_weight=A, cos=A, sin=A, positions=A, dq=A, dk=A, dq_stride=1024, dk_stride=1024, dq_weight=A,
              dk_weight=A, workspace=A, workspace_bytes=1 << 20)


@pytest.mark.parametrize("change,status", [
    (dict(dq_stride=500), INVAL), (dict(dk_out_stride=8), INVAL), (dict(workspace_bytes=100), INVAL),
    (dict(workspace=None), NULLP), (dict(dq_weight=None), NULLP), (dict(dk_weight=None), NULLP)] +
    [({n: None}, NULLP) for n in ("dq_out", "dk_out", "codes", "scales", "rstd", "q_weight", "k_weight", "cos", "sin",
                                  "positions", "dq", "dk")] +
    [({n: A + 2}, MISAL) for n in ("dq_out", "dk_out", "codes", "scales", "rstd", "q_weight", "k_weight", "cos", "sin",
                                   "positions", "dq", "dk", "dq_weight", "dk_weight", "workspace")])
def test_qk_norm_rope_bwd(coat, change, status):
    assert call(coat, "qk_norm_rope_bwd", coat.QkNormRopeBwdArgs, QK_BWD, shape=SHAPE, **change) == status


WGRAD = dict(dy=A, x_codes=A, x_scales=A, dw_bf16=A, M=4096, N=256, K=256, group_size=128, x_scale=float("nan"),
             workspace=A, workspace_bytes=1 << 40)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVAL), (dict(N=8), INVAL), (dict(K=24), INVAL), (dict(N=1 << 25), INVAL), (dict(K=-16), INVAL),
    (dict(K=144), INVAL), (dict(group_size=256), GSIZE), (dict(x_scales=None), INVAL), (dict(dw_f32=A), INVAL),
    (dict(accumulate=1), INVAL), (dict(workspace_bytes=64), INVAL), (dict(workspace=None), NULLP),
    (dict(dw_bf16=None), NULLP), (dict(dy=None), NULLP), (dict(x_codes=None), NULLP), (dict(M=1 << 50), INVAL),
    (dict(N=1 << 24, K=1 << 24), INVAL), (dict(N=0), OK), (dict(K=0), OK)] +
    [({n: A + 2}, MISAL) for n in ("dy", "x_codes", "x_scales", "dw_bf16", "workspace")] +
    [(dict(dw_bf16=None, dw_f32=A + 8), MISAL), (dict(M=0, accumulate=1, dw_bf16=None, dw_f32=A), OK)])
def test_weight_grad(coat, change, status):
    assert call(coat, "weight_grad", coat.WeightGradArgs, WGRAD, **change) == status


def test_null_arguments(coat):
    for name in ("rms_norm", "rms_norm_bwd", "swiglu", "qk_norm_rope", "qk_norm_rope_bwd", "weight_grad"):
        assert getattr(coat.lib, f"coat_fp8_{name}")(None, None) == NULLP


def test_workspaces(coat):
    assert coat.rms_norm_bwd_workspace(3, 4096) == 3 * 4096 * 4
    assert coat.rms_norm_bwd_workspace(1 << 20, 4096) == coat.rms_norm_bwd_workspace(1 << 21, 4096)
    assert coat.rms_norm_bwd_workspace(0, 4096) == 0
    for bad in ((-1, 16), (1, -1), (1, 40000)):
        with pytest.raises(coat.CoatError):
            coat.rms_norm_bwd_workspace(*bad)
    assert coat.qk_norm_rope_bwd_workspace(1, 1, 128) == 2 * 128 * 4
    for bad in ((-1, 4, 128), (1, -1, 128), (1, 4, 0), (1, 4, 100), (1, 4, 512), (1 << 50, 4, 128)):
        with pytest.raises(coat.CoatError):
            coat.qk_norm_rope_bwd_workspace(*bad)


def test_weight_grad_workspace(coat):
    assert coat.weight_grad_workspace(0, 128, 128) == 0
    assert coat.weight_grad_workspace(8192, 4096, 4096) == 0            # the tiles fill the chip
    need = coat.weight_grad_workspace(1 << 20, 256, 256)                # few tiles, many rows
    assert need % (256 * 256 * 4) == 0 and need >= 2 * 256 * 256 * 4
    assert coat.weight_grad_workspace(1 << 22, 256, 256) == need
    for bad in ((-1, 16, 16), (1, 8, 16), (1, 16, 20), (1, 1 << 25, 16)):
        with pytest.raises(coat.CoatError):
            coat.weight_grad_workspace(*bad)


# ------------------------------------------------------------ the binding

def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def u8(*shape):
    return z(*shape, dtype=torch.uint8)


def f32(*shape):
    return z(*shape, dtype=torch.float32)


def refuses(match, f, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


def test_binding_rms_norm(coat):
    x, w = z(4, 256), z(256)
    refuses("device", coat.rms_norm, x, w, 1e-5, y=z(4, 256))
    refuses("2-D", coat.rms_norm, z(256), w, 1e-5, y=z(256))
    refuses("dtype", coat.rms_norm, x.float(), w, 1e-5, y=z(4, 256))
    refuses("contiguous", coat.rms_norm, z(256, 4).t(), w, 1e-5, y=z(4, 256))
    refuses("weight holds", coat.rms_norm, x, w[:8], 1e-5, y=z(4, 256))
    refuses("residual_out holds", coat.rms_norm, x, w, 1e-5, residual=z(4, 256), residual_out=z(3, 256), y=z(4, 256))
    refuses("y_codes has dtype", coat.rms_norm, x, w, 1e-5, y_codes=z(4, 256))
    refuses("scales holds", coat.rms_norm, x, w, 1e-5, y=z(4, 256), codes=u8(4, 256), scales=f32(4), group_size=128)
    refuses("rstd holds", coat.rms_norm, x, w, 1e-5, y=z(4, 256), rstd=f32(3))
    bwd = lambda **k: coat.rms_norm_bwd(**{**dict(dy=x, codes=u8(4, 256), scales=f32(4, 2), rstd=f32(4), weight=w,  # noqa: E731
                                                  dx=z(4, 256)), **k})
    refuses("device", bwd)
    refuses("workspace is required", bwd, dw=f32(256))
    refuses("workspace holds", bwd, dw=f32(256), workspace=f32(1023))
    refuses("dw has dtype", bwd, dw=z(256), workspace=f32(1024))
    refuses("dx holds", bwd, dx=z(4, 128))
    refuses("codes holds", bwd, codes=u8(4, 255))


def test_binding_values_that_do_not_fit(coat):
    for values in ((0,) * 10 + (1 << 70, 1, 1e-5, 1.0, 128), (0,) * 10 + (1, 1, 1e-5, 1.0, 1 << 40)):
        refuses("does not fit", coat._pack_rms_norm, *values)
    # a number past FP32's range is infinite there, and refused as such
    assert coat.lib.coat_fp8_rms_norm(coat._pack_rms_norm(*(A,) * 10, 4, 256, 1e300, 1.0, 128), None) == INVAL
    assert len(coat._pack_rms_norm(*(0,) * 10, 1, 1, 1e-5, 1.0, 128)) <= ctypes.sizeof(coat.RMSNormArgs)


def test_binding_swiglu(coat):
    refuses("device", coat.swiglu, u8(4, 256), f32(4, 2), h=z(4, 128))
    refuses("even", coat.swiglu, u8(4, 255), f32(4, 2), h=z(4, 128))
    refuses("2-D", coat.swiglu, None, None, h=z(4, 128))
    refuses("scales holds", coat.swiglu, u8(4, 256), f32(4, 2), h=z(4, 128), group_size=16)
    refuses("h holds", coat.swiglu, u8(4, 256), f32(4, 2), h=z(3, 128))
    refuses("h_amax has dtype", coat.swiglu, u8(4, 256), f32(4, 2), h_codes=u8(4, 128), h_amax=z(1))
    refuses("codes holds", coat.swiglu, u8(4, 128), f32(4, 2), gate_up=z(4, 256), h=z(4, 128))
    refuses("d_gate_up holds", coat.swiglu_bwd, z(4, 128), u8(4, 256), f32(4, 2), z(4, 128))
    refuses("device", coat.swiglu_bwd, z(4, 128), u8(4, 256), f32(4, 2), z(4, 256))


def test_binding_qk(coat):
    base = dict(q=z(4, 4, 128), k=z(4, 2, 128), q_weight=z(128), k_weight=z(128), eps=1e-5, cos=f32(16, 64),
                sin=f32(16, 64), positions=z(4, dtype=torch.int64), q_out=z(4, 4, 128), k_out=z(4, 2, 128))
    go = lambda **k: coat.qk_norm_rope(**{**base, **k})  # noqa: E731
    refuses("device", go)
    refuses("3-D", go, q=z(4, 512))
    refuses("dtype", go, k=f32(4, 2, 128))
    refuses("disagree", go, k=z(3, 2, 128))
    refuses("contiguous", go, q=z(4, 128, 4).transpose(1, 2))
    refuses("contiguous", go, q=z(4, 128)[:, None, :].expand(4, 4, 128))
    refuses("expected", go, q_out=z(4, 3, 128))
    refuses("differ", go, sin=f32(16, 32))
    refuses("positions has dtype", go, positions=z(4, dtype=torch.int32))
    refuses("positions holds", go, positions=z(3, dtype=torch.int64))
    refuses("k_weight holds", go, k_weight=z(64))
    refuses("scales holds", go, codes=u8(4, 6, 128), scales=f32(4, 5), group_size=128)
    bwd = dict(dq_out=z(4, 4, 128), dk_out=z(4, 2, 128), codes=u8(4, 6, 128), scales=f32(4, 6), rstd=f32(4, 6),
               q_weight=z(128), k_weight=z(128), cos=f32(16, 64), sin=f32(16, 64),
               positions=z(4, dtype=torch.int64), dq=z(4, 4, 128), dk=z(4, 2, 128))
    go = lambda **k: coat.qk_norm_rope_bwd(**{**bwd, **k})  # noqa: E731
    refuses("device", go)
    refuses("workspace is required", go, dq_weight=f32(128), dk_weight=f32(128))
    refuses("dk has shape", go, dk=z(4, 1, 128))
    refuses("rstd holds", go, rstd=f32(4, 5))


def test_binding_weight_grad(coat):
    go = lambda **k: coat.weight_grad(**{**dict(dy=z(4, 128), codes=u8(4, 256), scales=0.5, dw=f32(128, 256)), **k})  # noqa: E731
    refuses("device", go)
    refuses("disagree", go, codes=u8(3, 256))
    refuses("scales holds", go, scales=f32(4, 1))
    refuses("number", go, scales=None)
    refuses("dw holds", go, dw=f32(128, 255))
    refuses("dw has dtype", go, dw=u8(128, 256))
    refuses("workspace is required", go, dy=z(4096, 128), codes=u8(4096, 256))
    refuses("workspace holds", go, dy=z(4096, 128), codes=u8(4096, 256), workspace=f32(10))


def test_every_argument_struct_is_documented(coat):
    text = open(os.path.join(ROOT, "include", "coat_fp8.h")).read()
    for name in coat.EXPORTED_SYMBOLS:
        assert re.search(rf"\b{name}\s*\(", text)
