"""GPU: the gated activation from E4M3 and from BF16, and its gradient from
the checkpoint, against the formulas in 64 bits."""
import pytest
import torch

import activation_ref as ref
from activation_ref import F
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu

SHAPES = [(1, 16, 16), (1, 128, 128), (3, 48, 16), (7, 11008, 128), (65, 352, 32), (130, 2048, 64), (2, 13824, 128),
          (1, 32768, 128), (5000, 64, 16)]
# exp: 2^-24 (1.5 |g| + 2) relative at |g| < 89 (|g| * 1.4427 rounded before
# it is raised), which silu keeps; the sum, reciprocal (one ulp = 2) and products: 8 more
ACT = (1.5 * 89 + 10) * F
# where the sigmoid lies below 2^-126 (gate < -87.33) the hardware's exp gives 0: s, and for positive gates
# 1 - s, is then off by its own value, at most 2^-126, and a result by that times what it multiplies
FLUSH = 2.0 ** -126


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def data(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(rows, 2 * cols, generator=g) * torch.exp(torch.randn(2 * cols, generator=g))).bfloat16()
    if rows > 2:
        x[1, 0], x[1, 1], x[1, 2], x[1, 3] = 60.0, -60.0, -85.0, 0.0
    return x


def run(rows, cols, G, *, x=None, codes=None, scales=None, fp8=None, ckpt=False):
    coat = lib()
    o = {}
    if fp8 is None:
        o["h"] = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    else:
        o["h_codes"] = torch.full((rows, cols), 0x55, dtype=torch.uint8, device=DEV)
        o["h_amax"] = torch.zeros(1, device=DEV)
    if x is not None and ckpt:
        codes = torch.full((rows, 2 * cols), 0x55, dtype=torch.uint8)
        scales = torch.full((rows, 2 * cols // G), -1.0)
    c, s = (None, None) if codes is None else (codes.to(DEV), scales.to(DEV))
    coat.swiglu(c, s, gate_up=None if x is None else x.to(DEV), h_scale=fp8 or 1.0, group_size=G, **o)
    torch.cuda.synchronize()
    o = {k: v.cpu() for k, v in o.items()}
    if c is not None:
        o.update(codes=c.cpu(), scales=s.cpu())
    return o


@pytest.mark.parametrize("rows,cols,G", SHAPES)
@pytest.mark.parametrize("source", ["fp8", "bf16", "bf16 checkpoint"])
@pytest.mark.parametrize("fp8", [None, 0.125])
def test_forward(rows, cols, G, source, fp8):
    x = data(rows, cols, rows + cols)
    codes, scales = ref.quantize(x, G)
    if source == "fp8":
        o = run(rows, cols, G, codes=codes, scales=scales, fp8=fp8)
        v = ref.restore(codes, scales, G)
    else:
        o = run(rows, cols, G, x=x, fp8=fp8, ckpt=source != "bf16")
        v = x.double()
        if source != "bf16":
            assert torch.equal(ref.code_values(o["codes"]), ref.code_values(codes))
            assert torch.equal(o["scales"], scales)
    gate, up = v.chunk(2, 1)
    h = gate * ref.silu_parts(gate)[0] * up
    if fp8 is None:
        ref.assert_close(o["h"], h, ACT * h.abs() + FLUSH * (gate * up).abs(), "h")
    else:
        ref.assert_codes(o["h_codes"], h * 8.0, ACT + F, "h_codes")
        assert abs(float(o["h_amax"]) - h.abs().max()) <= ACT * h.abs().max()


@pytest.mark.parametrize("rows,cols,G", SHAPES)
def test_backward(rows, cols, G):
    coat = lib()
    x = data(rows, cols, rows * 5 + cols)
    dh = (1e-3 * data(rows, cols, 99)[:, :cols].float()).bfloat16()
    codes, scales = ref.quantize(x, G)
    d = torch.full((rows, 2 * cols), 3.0, dtype=torch.bfloat16, device=DEV)
    coat.swiglu_bwd(dh.to(DEV), codes.to(DEV), scales.to(DEV), d, group_size=G)
    gate, up = ref.restore(codes, scales, G).chunk(2, 1)
    s, rest = ref.silu_parts(gate)
    slope = 1 + gate * rest
    # the slope's two terms cancel near gate = -1.28: its error counts against their size
    size = 1 + (gate * rest).abs()
    d = d.cpu()
    dh = dh.double()
    ref.assert_close(d[:, :cols], dh * up * s * slope,
                     ACT * (dh * up * s).abs() * size + FLUSH * (dh * up).abs() * (1 + gate.abs()), "d_gate")
    ref.assert_close(d[:, cols:], dh * gate * s, ACT * (dh * gate * s).abs() + FLUSH * (dh * gate).abs(), "d_up")


def test_gradient_against_differences():
    """Values E4M3 holds exactly, so the checkpoint loses nothing."""
    coat = lib()
    rows, cols, G, h = 2, 32, 16, 1e-5
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-14, 15, (rows, 2 * cols), generator=g).double() / 8
    x[:, ::G] = 1.75
    codes, scales = ref.quantize(x.bfloat16(), G)
    assert torch.equal(ref.restore(codes, scales, G), x)
    dh = torch.randn(rows, cols, generator=g).bfloat16()
    d = torch.empty(rows, 2 * cols, dtype=torch.bfloat16, device=DEV)
    coat.swiglu_bwd(dh.to(DEV), codes.to(DEV), scales.to(DEV), d, group_size=G)

    def f(v):
        gate, up = v.chunk(2, 1)
        return gate * torch.sigmoid(gate) * up

    want = torch.empty(rows, 2 * cols, dtype=torch.float64)
    for j in range(2 * cols):
        e = torch.zeros(2 * cols, dtype=torch.float64)
        e[j] = h
        want[:, j] = ((f(x + e) - f(x - e)) * dh.double()).sum(1) / (2 * h)
    # the difference: h^2 / 6 of third derivatives below 2, and 2^-53 * 50 / h
    ref.assert_close(d.cpu(), want, torch.full_like(want, 2e-9) + 100 * F, "d_gate_up")


def test_far_gates_and_not_finite():
    """silu tends to the gate and to zero without overflow; a NaN or infinity
    stays with its value."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    x[:, 128:] = 2.0
    x[0, :6] = torch.tensor([300.0, -300.0, 1e30, -1e30, -100.0, 88.0])
    x[1, 3], x[2, 128 + 7] = float("nan"), float("inf")
    o = run(4, 128, 128, x=x)
    h = o["h"].float()
    assert h[0, 0] == 600 and h[0, 1] == 0 and h[0, 3] == 0 and h[0, 5] == 176
    assert h[0, 2] == torch.tensor(2e30).bfloat16().float()
    assert h[1, 3].isnan() and h[1, [0, 1, 2, 4]].eq(0).all() and h[3].eq(0).all()
    assert h[2, 7].isnan()   # 0 * infinity


def test_saturates_and_keeps_the_running_maximum():
    coat = lib()
    x = torch.full((3, 64), 100.0, dtype=torch.bfloat16)
    codes = torch.empty(3, 32, dtype=torch.uint8, device=DEV)
    amax = torch.tensor([2e4], device=DEV)
    coat.swiglu(None, None, gate_up=x.to(DEV), h_codes=codes, h_scale=1.0, h_amax=amax, group_size=16)
    assert (codes == 0x7E).all() and float(amax) == 2e4
    amax.zero_()
    coat.swiglu(None, None, gate_up=x.to(DEV), h_codes=codes, h_scale=1.0, h_amax=amax, group_size=16)
    assert abs(float(amax) - 1e4) <= ACT * 1e4


def test_no_rows_and_graph():
    coat = lib()
    coat.swiglu(torch.empty(0, 256, dtype=torch.uint8, device=DEV), torch.empty(0, 2, device=DEV),
                h=torch.empty(0, 128, dtype=torch.bfloat16, device=DEV))
    rows, cols, G = 300, 2048, 64
    x = data(rows, cols, 1).to(DEV)
    dh = x[:, :cols].contiguous()
    mk = lambda: (torch.zeros(rows, 2 * cols, dtype=torch.uint8, device=DEV),  # noqa: E731
                  torch.zeros(rows, 2 * cols // G, device=DEV), torch.zeros(rows, cols, dtype=torch.uint8, device=DEV),
                  torch.zeros(1, device=DEV), torch.zeros(rows, 2 * cols, dtype=torch.bfloat16, device=DEV))

    def go(o, stream=None):
        coat.swiglu(o[0], o[1], gate_up=x, h_codes=o[2], h_scale=0.25, h_amax=o[3], group_size=G, stream=stream)
        coat.swiglu_bwd(dh, o[0], o[1], o[4], group_size=G, stream=stream)

    eager, other, captured = mk(), mk(), mk()
    go(eager)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    go(other, side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(captured)
    for _ in range(3):
        for t in captured:
            t.zero_()
        go(other)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(captured, eager, other):
            assert torch.equal(a, b) and torch.equal(b, c)
