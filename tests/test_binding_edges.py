"""Calls that the binding has to refuse, or must not trip over, on the CPU."""
import importlib.util
import sys

import pytest
import torch


@pytest.fixture(scope="module")
def coat():
    from test_abi_exports import _ensure_built
    _ensure_built()
    from adamw_coat_fp8_amd import coat
    return coat


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


@pytest.mark.parametrize("G", [(1 << 32) + 128, -(1 << 32) + 16, 1 << 31])
def test_group_size_past_a_c_int(coat, G):
    """Cut to 32 bits it would be a valid one, for which the scales checked
    here are too few."""
    few, n = torch.zeros(1), 1024
    state = coat.QuantState(u8(n), few, few)
    slot = coat.ParamSlot(torch.zeros(n), bf16(n), state, state)
    calls = (lambda: coat.swiglu_bwd(bf16(4, 128), u8(4, 256), few, bf16(4, 256), group_size=G),
             lambda: coat.quantize_act(bf16(4, 128), u8(4, 128), few, group_size=G),
             lambda: coat.gemm_group_quant(u8(8, 128), u8(128, 128), 1.0, 1.0, u8(8, 128), few, group_size=G),
             lambda: coat.expand_quantize(torch.zeros(n), state, group_size=G),
             lambda: coat.dequantize_expand(state, torch.zeros(n), group_size=G),
             lambda: coat.adamw_fp8_step([slot], lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1,
                                         group_size=G))
    for call in calls:
        with pytest.raises(ValueError, match="does not fit"):
            call()


def on_device(monkeypatch, coat):
    """The binding's checks as they go for buffers on the current device:
    every one is taken, at address 0x10000, and the library is not called."""
    calls = []
    monkeypatch.setattr(coat, "_addresses", lambda buffers, heads=(): (
        [0 if b[0] is None else 0x10000 for b in (*buffers, *heads)], 0))
    monkeypatch.setattr(coat, "_launch", lambda fn, packed, stream, current: calls.append(packed))
    return calls


def test_weight_grad_without_dw(monkeypatch, coat):
    calls = on_device(monkeypatch, coat)
    coat.weight_grad(bf16(4, 128), u8(4, 128), 0.5, torch.zeros(128, 128))
    assert len(calls) == 1
    for dw in (None, 3.0):
        with pytest.raises(ValueError, match="dw must be"):
            coat.weight_grad(bf16(4, 128), u8(4, 128), 0.5, dw)
    assert len(calls) == 1


I64 = (1 << 63) - 1


@pytest.mark.parametrize("rows,cols", [(I64, 16), (I64 - 100, 4096), (1 << 60, 32768), (4, 24), (4, 8), (0, 8),
                                       ((1 << 64) + 4, 4096), (4, (1 << 64) + 4096)])
def test_norm_workspace_of_sizes_that_the_call_refuses(coat, rows, cols):
    with pytest.raises((coat.CoatError, ValueError)):
        coat.rms_norm_bwd_workspace(rows, cols)


@pytest.mark.parametrize("tokens,heads,dim", [((1 << 31) - 300000, 8, 128), ((1 << 29), 64, 128), (1 << 20, 1 << 17, 256),
                                              ((1 << 64) + 4, 8, 128), (I64, 1, 16)])
def test_heads_workspace_of_sizes_that_the_call_refuses(coat, tokens, heads, dim):
    """However the heads divide into queries and keys."""
    with pytest.raises((coat.CoatError, ValueError)):
        coat.qk_norm_rope_bwd_workspace(tokens, heads, dim)


def test_weight_grad_workspace_past_64_bits(coat):
    for sizes in (((1 << 64) + 64, 128, 128), (64, (1 << 64) + 128, 128), (64, 128, (1 << 64) + 128)):
        with pytest.raises((coat.CoatError, ValueError)):
            coat.weight_grad_workspace(*sizes)


def test_workspaces_at_the_largest_sizes(coat):
    assert coat.rms_norm_bwd_workspace(I64 // 8 // 32768, 4096) == coat.rms_norm_bwd_workspace(1 << 40, 4096) > 0
    assert coat.qk_norm_rope_bwd_workspace(1 << 26, 64, 128) == 1024 * 2 * 128 * 4


def test_norm_backward_over_its_own_input(coat):
    """Up to 512 rows other blocks read dy after a row's dx is written."""
    import ctypes
    A, B = 0x10000, 0x20000
    base = dict(dy=A, codes=A, scales=A, rstd=A, weight=A, rows=4, cols=256, group_size=128, workspace=B,
                workspace_bytes=1 << 20)
    for change in (dict(dx=A, dw=B), dict(dx=A), dict(dx=A, rows=100000, dw=B, workspace_bytes=1 << 30)):
        a = coat.RMSNormBwdArgs(**{**base, **change})
        assert coat.lib.coat_fp8_rms_norm_bwd(ctypes.byref(a), None) == coat.COAT_ERR_INVALID_VALUE


def test_stream_of_another_device(monkeypatch, coat):
    class Stream:
        def __init__(self, device_index):
            self.device_index, self.cuda_stream = device_index, 77

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert coat._stream(Stream(1)) == 77 and coat._stream(77) == 77
    with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
        coat._stream(Stream(0))


def test_without_torchs_private_queries(monkeypatch, coat):
    """A torch that lacks them is served by its public ones."""
    class Tensor:
        dtype = torch.bfloat16
        get_device, is_contiguous, numel, data_ptr = (lambda s: 1), (lambda s: True), (lambda s: 8), (lambda s: 0x10000)

    class Stream:
        cuda_stream = 71

    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: Stream() if device == 1 else None)
    spec = importlib.util.spec_from_file_location("coat_on_another_torch", coat.__file__)
    other = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(sys.modules, spec.name, other)
    spec.loader.exec_module(other)
    assert other._addresses(((Tensor(), "x", other.BF16, 8), (None, "y", other.F32, 8))) == ([0x10000, 0], 71)
    assert other._stream(None) == 71
