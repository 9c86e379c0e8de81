"""Refusals of the vocabulary operators, on the CPU: the C entry points return
their status before any HIP call (the pointers are never dereferenced), and
the binding raises ValueError on buffers the C side cannot see into."""
import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from test_abi_exports import ROOT, _ensure_built
from test_activation_refusals import A, INVAL, MISAL, NULLP, OK, call, f32, refuses, u8, z

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def coat():
    _ensure_built()
    from adamw_coat_fp8_amd import coat
    return coat


def test_structs_have_the_c_layout(coat):
    structs = {"coat_embedding_args_t": coat.EmbeddingArgs, "coat_embedding_bwd_args_t": coat.EmbeddingBwdArgs,
               "coat_cross_entropy_args_t": coat.CrossEntropyArgs,
               "coat_cross_entropy_bwd_args_t": coat.CrossEntropyBwdArgs}
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


LOOKUP = dict(table=A, tokens=A, out=A, rows=4, vocab=100, cols=64, table_scale=1.0, scale=1.0)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVAL), (dict(vocab=-1), INVAL), (dict(cols=-16), INVAL), (dict(cols=24), INVAL),
    (dict(cols=(1 << 16) + 16), INVAL), (dict(vocab=(1 << 22) + 1), INVAL), (dict(rows=(1 << 23) + 1), INVAL),
    (dict(rows=1 << 23, cols=2048), INVAL), (dict(vocab=1 << 22, cols=8192), INVAL), (dict(table_codes=A), INVAL),
    (dict(scale=NAN), INVAL), (dict(table_scale=INF), INVAL), (dict(scale=1e30, table_scale=1e30), INVAL),
    (dict(table=None), NULLP), (dict(tokens=None), NULLP), (dict(out=None), NULLP), (dict(table=A + 8), MISAL),
    (dict(table=None, table_codes=A + 4), MISAL), (dict(tokens=A + 4), MISAL), (dict(out=A + 8), MISAL),
    (dict(rows=0, table=None, tokens=None, out=None), OK), (dict(cols=0), OK)])
def test_embedding(coat, change, status):
    assert call(coat, "embedding", coat.EmbeddingArgs, LOOKUP, **change) == status


LOOKUP_BWD = dict(dy=A, tokens=A, dw_bf16=A, workspace=A, workspace_bytes=1 << 20, rows=4, vocab=100, cols=64, scale=1.0)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), INVAL), (dict(vocab=-1), INVAL), (dict(cols=40), INVAL), (dict(scale=INF), INVAL),
    (dict(dw_f32=A), INVAL), (dict(accumulate=1), INVAL), (dict(workspace_bytes=100), INVAL), (dict(workspace=None), NULLP),
    (dict(dy=None), NULLP), (dict(tokens=None), NULLP), (dict(dw_bf16=None), NULLP), (dict(dy=A + 8), MISAL),
    (dict(tokens=A + 4), MISAL), (dict(dw_bf16=A + 8), MISAL), (dict(dw_bf16=None, dw_f32=A + 4), MISAL),
    (dict(workspace=A + 8), MISAL), (dict(vocab=0, dw_bf16=None), OK), (dict(cols=0), OK),
    (dict(rows=0, dw_bf16=None, dw_f32=A, accumulate=1, workspace=None, dy=None), OK)])
def test_embedding_bwd(coat, change, status):
    assert call(coat, "embedding_bwd", coat.EmbeddingBwdArgs, LOOKUP_BWD, **change) == status


LOSS = dict(x=A, weight=A, targets=A, loss=A, lse=A, workspace=A, workspace_bytes=1 << 30, rows=4, vocab=1000, cols=128,
            x_scale=1.0, weight_scale=1.0, logit_scale=1.0, z_loss=0.0)
CODES = dict(x=None, weight=None, x_codes=A, weight_codes=A)
COMMON = [
    (dict(rows=-1), INVAL), (dict(vocab=-1), INVAL), (dict(cols=-64), INVAL), (dict(cols=96), INVAL),
    (dict(cols=192, **CODES), INVAL), (dict(cols=1 << 17), INVAL), (dict(vocab=(1 << 22) + 1), INVAL),
    (dict(rows=(1 << 23) + 1), INVAL), (dict(rows=1 << 23, cols=2048), INVAL), (dict(vocab=1 << 22, cols=8192), INVAL),
    (dict(rows=1 << 22, vocab=1 << 21), INVAL), (dict(vocab=0), INVAL), (dict(cols=0), INVAL), (dict(x_codes=A), INVAL),
    (dict(x=None, x_codes=A), INVAL), (dict(x_scale=0.0), INVAL), (dict(weight_scale=-1.0), INVAL),
    (dict(logit_scale=NAN), INVAL), (dict(logit_scale=INF), INVAL), (dict(x_scale=1e-30, weight_scale=1e-30), INVAL),
    (dict(x_scale=1e30, logit_scale=1e30), INVAL), (dict(z_loss=NAN), INVAL), (dict(z_loss=INF), INVAL),
    (dict(workspace_bytes=1000), INVAL), (dict(workspace=None), NULLP), (dict(x=None), NULLP), (dict(weight=None), NULLP),
    (dict(targets=None), NULLP), (dict(CODES, x_codes=None), NULLP), (dict(x=A + 8), MISAL), (dict(weight=A + 2), MISAL),
    (dict(CODES, x_codes=A + 8), MISAL), (dict(CODES, weight_codes=A + 8), MISAL), (dict(targets=A + 4), MISAL),
    (dict(lse=A + 2), MISAL), (dict(workspace=A + 8), MISAL)]


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(loss=None), NULLP), (dict(loss=A + 1), MISAL), (dict(rows=0, x=None, weight=None, loss=None, workspace=None), OK)])
def test_cross_entropy(coat, change, status):
    assert call(coat, "cross_entropy", coat.CrossEntropyArgs, LOSS, **change) == status


LOSS_BWD = {k: v for k, v in LOSS.items() if k != "loss"}
LOSS_BWD.update(d_loss=A, dx=A, dw_bf16=A)


@pytest.mark.parametrize("change,status", COMMON + [
    (dict(d_loss=None), NULLP), (dict(lse=None), NULLP), (dict(dx=None, dw_bf16=None), NULLP), (dict(dw_f32=A), INVAL),
    (dict(accumulate=1), INVAL), (dict(d_loss=A + 2), MISAL), (dict(dx=A + 8), MISAL), (dict(dw_bf16=A + 8), MISAL),
    (dict(dw_bf16=None, dw_f32=A + 8), MISAL), (dict(rows=0, dw_bf16=None), OK), (dict(rows=0, vocab=0), OK),
    (dict(rows=0, dw_bf16=None, dw_f32=A, accumulate=1), OK)])
def test_cross_entropy_bwd(coat, change, status):
    assert call(coat, "cross_entropy_bwd", coat.CrossEntropyBwdArgs, LOSS_BWD, **change) == status


@pytest.mark.parametrize("scales", [(1.0, 1.0, 3e38), (1e19, 1e19, 3.0), (3e38, 1.0, 1.0)])
def test_scales_whose_exponents_overflow(coat, scales):
    """Finite, but not in powers of two: 3e38 log2(e) passes 2^128."""
    change = dict(zip(("x_scale", "weight_scale", "logit_scale"), scales))
    assert call(coat, "cross_entropy", coat.CrossEntropyArgs, LOSS, **change) == INVAL
    assert call(coat, "cross_entropy_bwd", coat.CrossEntropyBwdArgs, LOSS_BWD, **change) == INVAL


def test_most_tiles(coat):
    """2^22 tiles of 256 x 256 are taken, one row more is not."""
    assert coat.cross_entropy_workspace(1 << 20, 1 << 18, 64) > 0
    assert coat.cross_entropy_bwd_workspace(1 << 20, 1 << 18, 64) > 0
    for f in (coat.cross_entropy_workspace, coat.cross_entropy_bwd_workspace):
        with pytest.raises(coat.CoatError):
            f((1 << 20) + 1, 1 << 18, 64)


def test_null_arguments(coat):
    for name in ("embedding", "embedding_bwd", "cross_entropy", "cross_entropy_bwd"):
        assert getattr(coat.lib, f"coat_fp8_{name}")(None, None) == NULLP


def test_workspaces(coat):
    assert coat.embedding_bwd_workspace(0, 100, 64) == 0
    assert coat.embedding_bwd_workspace(1000, 100, 64) >= 8 * 1000
    assert coat.cross_entropy_workspace(0, 100, 64) == 0
    assert coat.cross_entropy_workspace(1000, 50000, 64) >= 8 * 1000 * (50000 // 128)
    for bad in ((-1, 16, 64), (1, -1, 64), (1, 16, -64), (1, 16, 24), (1 << 70, 1, 64)):
        for f in (coat.embedding_bwd_workspace, coat.cross_entropy_workspace, coat.cross_entropy_bwd_workspace):
            with pytest.raises(coat.CoatError):
                f(*bad)
    need = lambda **k: coat.cross_entropy_bwd_workspace(5000, 32000, 2048, **k)  # noqa: E731
    assert need(piece=1) <= need(piece=256) < need(piece=8192) < need(piece=32000) == need(piece=1 << 40)
    assert need(piece=8192) < need(piece=8192, f32=True) and need(piece=8192) < need(piece=8192, codes=True)
    for bad in (0, -1, 1 << 70):
        with pytest.raises(ValueError):
            need(piece=bad)


def test_least_workspace_is_taken_and_less_refused(coat):
    for codes in (False, True):
        for extra in (dict(), dict(dw_bf16=None, dw_f32=A)):
            ops = dict(CODES) if codes else {}
            need = coat.cross_entropy_bwd_workspace(70, 1000, 128, piece=1, codes=codes, f32="dw_f32" in extra)
            bad = {**ops, **extra, "rows": 70, "workspace_bytes": need - 256}
            assert call(coat, "cross_entropy_bwd", coat.CrossEntropyBwdArgs, LOSS_BWD, **bad) == INVAL


def i64(*shape):
    return z(*shape, dtype=torch.int64)


def test_binding_embedding(coat):
    go = lambda **k: coat.embedding(**{**dict(table=z(10, 64), tokens=i64(5), out=z(5, 64)), **k})  # noqa: E731
    refuses("device", go)
    refuses("2-D", go, table=z(640))
    refuses("dtype", go, table=f32(10, 64))
    refuses("contiguous", go, table=z(64, 10).t())
    refuses("tokens has dtype", go, tokens=z(5, dtype=torch.int32))
    refuses("tokens must be", go, tokens=[1, 2])
    refuses("out holds", go, out=z(4, 64))
    refuses("out has dtype", go, out=f32(5, 64))
    ws = u8(coat.embedding_bwd_workspace(5, 10, 64))
    go = lambda **k: coat.embedding_bwd(**{**dict(dy=z(5, 64), tokens=i64(5), dw=z(10, 64), workspace=ws), **k})  # noqa: E731
    refuses("device", go)
    refuses("disagree", go, dw=z(10, 48))
    refuses("tokens holds", go, tokens=i64(4))
    refuses("dw has dtype", go, dw=u8(10, 64))
    refuses("workspace is required", go, workspace=None)
    refuses("workspace holds", go, workspace=u8(10))


def test_binding_cross_entropy(coat):
    ws = u8(coat.cross_entropy_workspace(5, 300, 128))
    base = dict(x=z(5, 128), weight=z(300, 128), targets=i64(5), loss=f32(5), lse=f32(5), workspace=ws)
    go = lambda **k: coat.cross_entropy(**{**base, **k})  # noqa: E731
    refuses("device", go)
    refuses("disagree", go, weight=z(300, 64))
    refuses("both BF16 or both", go, weight=u8(300, 128))
    refuses("dtype", go, x=f32(5, 128))
    refuses("contiguous", go, weight=z(128, 300).t())
    refuses("targets holds", go, targets=i64(4))
    refuses("loss holds", go, loss=f32(4))
    refuses("lse has dtype", go, lse=z(5))
    refuses("workspace is required", go, workspace=None)
    refuses("workspace holds", go, workspace=u8(10))
    ws = u8(coat.cross_entropy_bwd_workspace(5, 300, 128, f32=True))
    base = dict(d_loss=f32(5), x=z(5, 128), weight=z(300, 128), targets=i64(5), lse=f32(5), dx=z(5, 128),
                dw=f32(300, 128), workspace=ws)
    go = lambda **k: coat.cross_entropy_bwd(**{**base, **k})  # noqa: E731
    refuses("device", go)
    refuses("d_loss holds", go, d_loss=f32(4))
    refuses("dx has dtype", go, dx=f32(5, 128))
    refuses("dw holds", go, dw=f32(299, 128))
    refuses("dw has dtype", go, dw=u8(300, 128))
    refuses("lse holds", go, lse=f32(4))
    refuses("workspace is required", go, workspace=None)
    refuses("workspace holds", go, workspace=u8(10))
