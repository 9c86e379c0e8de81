"""GPU: the FP32 weight gradient of an input under group scales of any value,
in sums short enough for the operands' own error to show."""
import pytest
import torch

import activation_ref as ref
from activation_ref import F
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu

# few and many rows (split and joined ones too), edges, both sizes of tiles, halves of the large ones
SHAPES = [(1, 16, 128), (3, 144, 256), (64, 128, 384), (130, 272, 640), (1024, 128, 128), (2100, 256, 128),
          (70, 4112, 4096), (333, 2048, 2048), (200, 3328, 3328), (65, 144, 33280)]
TERMS = 12   # rows of dy that are not zero


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("G", [16, 32, 64, 128])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_group_scales_of_any_value(m, n, k, G):
    coat = lib()
    g = torch.Generator().manual_seed(m + n + k + G)
    dy = torch.randn(m, n, generator=g).bfloat16()
    if m > TERMS:   # the products with the others are exact zeros
        rows = torch.randperm(m, generator=g)[:TERMS]
        keep = torch.zeros(m, 1, dtype=torch.bool)
        keep[rows] = True
        dy = torch.where(keep, dy, torch.zeros_like(dy))
    codes = torch.randint(0, 256, (m, k), generator=g).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x7E   # the two NaN codes
    scales = torch.exp(2 * torch.randn(m, k // G, generator=g))
    x = ref.restore(codes, scales, G).to(DEV)
    d = dy.double().to(DEV)
    want, size = (d.t().contiguous() @ x).cpu(), (d.abs().t().contiguous() @ x.abs()).cpu()
    ws = torch.empty(coat.weight_grad_workspace(m, n, k), dtype=torch.uint8, device=DEV)
    dw = torch.full((n, k), 5.0, device=DEV)
    args = dy.to(DEV), codes.to(DEV), scales.to(DEV), dw
    coat.weight_grad(*args, workspace=ws, group_size=G)
    # code * S rounded to FP32: 2^-24 of it; its two BF16 parts: 2^-8 of 2^-8; two products
    # for each term, added one after the other at 2^-23 a step (the matrix cores may truncate)
    slack = (2.0 ** -16 + F + (2 * min(m, TERMS) + 4) * 2 * F) * size
    ref.assert_close(dw.cpu(), want, slack, "dw", F)
    once = dw.clone()
    base = torch.randn(n, k, generator=g).to(DEV)
    dw.copy_(base)
    coat.weight_grad(*args, accumulate=True, workspace=ws, group_size=G)
    assert torch.equal(dw, base + once)
    # codes of zero and scales of zero stay exact zeros
    args[2].zero_()
    coat.weight_grad(*args, workspace=ws, group_size=G)
    assert (dw == 0).all()
