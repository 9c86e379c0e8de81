"""Calls that the binding has to refuse, or must not trip over, on the CPU."""
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
