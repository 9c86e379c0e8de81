"""GPU: the checkpoint at the edges of its arithmetic (every finite BF16 value
as a group's maximum, subnormal ones and those near the top among them, with
members at and beside the midpoints between codes), and outputs under one
scale that is no power of two."""
import pytest
import torch

import activation_ref as ref
from activation_ref import F
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu
GROUPS = 32640   # 0x7F7F patterns, and one again to fill 255 rows of 128 groups


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def midpoints():
    """Every quotient at which E4M3 rounding changes its mind, and every value, below 448."""
    codes = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    return torch.cat((codes[1:], (codes[1:] + codes[:-1]) / 2))


def groups(G, seed):
    """GROUPS x G BF16 values; group i's largest magnitude is pattern i + 1."""
    g = torch.Generator().manual_seed(seed)
    top = torch.arange(1, GROUPS + 1).clamp(max=0x7F7F)
    mids = midpoints()
    q = mids[torch.randint(0, len(mids), (GROUPS, G), generator=g)]
    value = top.to(torch.int16).view(torch.bfloat16).double()[:, None] * q / 448.0
    near = value.float().bfloat16().view(torch.int16).long()   # (exactly the midpoint where BF16 has it)
    near = near + torch.randint(-1, 2, near.shape, generator=g)
    any_ = (torch.rand(GROUPS, G, generator=g) * (top[:, None] + 1)).long()   # every pattern up to the maximum
    bits = torch.where(torch.rand(GROUPS, G, generator=g) < 0.8, near, any_)
    bits = torch.minimum(bits.clamp(min=0), top[:, None])
    at = torch.randint(0, G, (GROUPS,), generator=g)
    bits[torch.arange(GROUPS), at] = top
    bits = bits | torch.randint(0, 2, bits.shape, generator=g) << 15
    return torch.where(bits >= 1 << 15, bits - (1 << 16), bits).to(torch.int16).view(torch.bfloat16)


@pytest.mark.parametrize("G", [16, 32, 64, 128])
def test_every_maximum(G):
    coat = lib()
    x = groups(G, G).reshape(-1, 2048)
    rows, cols = x.shape
    codes, scales = ref.quantize(x, G)
    assert (scales > 0).all() and scales.isfinite().all()
    xd = x.to(DEV)

    def empty():
        return (torch.full((rows, cols), 0x55, dtype=torch.uint8, device=DEV), torch.full((rows, cols // G), -1.0, device=DEV))

    def check(got, what):
        # -0 may keep its sign or not: the codes' values
        assert torch.equal(ref.code_values(got[0].cpu().view(rows, cols)), ref.code_values(codes)), what
        assert torch.equal(got[1].cpu().view(scales.shape), scales), what

    by_quantizer = empty()
    coat.quantize_act(xd, *by_quantizer, group_size=G)
    check(by_quantizer, "quantize_act")
    y, w = torch.empty_like(xd), torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    o = empty()
    coat.rms_norm(xd, w, 1e-5, y=y, codes=o[0], scales=o[1], group_size=G)
    check(o, "rms_norm")
    assert torch.equal(o[0], by_quantizer[0]) and torch.equal(o[1], by_quantizer[1])
    o = empty()
    coat.swiglu(o[0], o[1], gate_up=xd, h=torch.empty(rows, cols // 2, dtype=torch.bfloat16, device=DEV), group_size=G)
    check(o, "swiglu")
    assert torch.equal(o[0], by_quantizer[0]) and torch.equal(o[1], by_quantizer[1])
    heads = xd.view(rows, cols // 128, 128)
    table = torch.zeros(1, 64, device=DEV)
    pos = torch.zeros(rows, dtype=torch.int64, device=DEV)
    o = empty()
    out = torch.empty_like(heads)
    coat.qk_norm_rope(heads[:, :5], heads[:, 5:], w[:128], w[:128], 1e-5, table, table, pos, out[:, :5], out[:, 5:],
                      codes=o[0], scales=o[1], group_size=G)
    check(o, "qk_norm_rope")
    assert torch.equal(o[0], by_quantizer[0]) and torch.equal(o[1], by_quantizer[1])


SCALES = [0.0123, 1.0 / 3.0, 7.7e-4, 3.3]


@pytest.mark.parametrize("scale", SCALES)
def test_norm_under_any_scale(scale):
    """The output's codes under a scale as amax / 448 gives it: two roundings
    more (the scale's reciprocal and the product)."""
    coat = lib()
    rows, cols = 300, 4096
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(cols, generator=g))).bfloat16()
    w = (1 + 0.3 * torch.randn(cols, generator=g)).bfloat16()
    codes, amax = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.zeros(1, device=DEV)
    coat.rms_norm(x.to(DEV), w.to(DEV), 1e-5, y_codes=codes, y_scale=scale, y_amax=amax)
    y, _ = ref.norm(x, w, 1e-5)
    # squares: 16 values a thread, 6 lane steps, 16 waves, mean, eps, root; two products; then as above
    ref.assert_codes(codes.cpu(), y / float(torch.tensor(scale)), (16 + 6 + 16 + 4 + 2 + 2) * F, "codes")
    assert abs(float(amax) - y.abs().max()) <= 44 * F * y.abs().max()


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("source", ["fp8", "bf16"])
def test_swiglu_under_any_scale(scale, source):
    coat = lib()
    rows, cols, G = 200, 2048, 64
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(rows, 2 * cols, generator=g) * torch.exp(torch.randn(2 * cols, generator=g))).bfloat16()
    out = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    codes, scales = ref.quantize(x, G)
    if source == "fp8":
        coat.swiglu(codes.to(DEV), scales.to(DEV), h_codes=out, h_scale=scale, group_size=G)
        v = ref.restore(codes, scales, G)
    else:
        coat.swiglu(None, None, gate_up=x.to(DEV), h_codes=out, h_scale=scale, group_size=G)
        v = x.double()
    gate, up = v.chunk(2, 1)
    h = gate * ref.silu_parts(gate)[0] * up
    # exp at |gate| < 89, sum, reciprocal and products (1.5 * 89 + 10), the scale's reciprocal and product 2
    ref.assert_codes(out.cpu(), h / float(torch.tensor(scale)), (1.5 * 89 + 12) * F, "codes")
