"""GPU: the running maximum that the calls with codes under one scale raise:
exact from any start, wherever the largest value lies, for few blocks and many."""
import pytest
import torch

from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def places(rows, cols):
    return [(0, 0), (rows - 1, cols - 1), (rows // 2, cols // 3), (rows - 1, 0), (rows // 61, cols - 1)]


# one wave to sixteen a row, one row to many thousands, blocks of four rows with some left over
@pytest.mark.parametrize("rows,cols", [(1, 128), (40, 512), (129, 512), (130, 256), (515, 128), (8193, 512), (20000, 128),
                                       (3000, 1024), (2049, 2048), (7, 4096), (1030, 4096), (300, 8192), (600, 16384),
                                       (257, 32768)])
def test_norm(rows, cols):
    """Against the BF16 output of the same call."""
    coat = lib()
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    codes = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    for r, c in places(rows, cols):
        x = torch.randn(rows, cols, device=DEV, generator=g).bfloat16()
        x[r, c] = -64.0
        amax = torch.zeros(1, device=DEV)
        coat.rms_norm(x, w, 1e-5, y=y, y_codes=codes, y_scale=0.05, y_amax=amax)
        top = float(amax)
        # y is amax rounded to BF16; its place is the one planted
        assert float(y.abs().max()) == float(torch.tensor(top).bfloat16()) == float(y[r, c].abs()) > 0
        coat.rms_norm(x, w, 1e-5, y_codes=codes, y_scale=0.05, y_amax=amax)
        assert float(amax) == top
        for start, want in ((top / 2, top), (2 * top, 2 * top)):
            amax.fill_(start)
            coat.rms_norm(x, w, 1e-5, y_codes=codes, y_scale=0.05, y_amax=amax)
            assert float(amax) == float(torch.tensor(want))


@pytest.mark.parametrize("rows,cols", [(1, 128), (7, 11008), (100, 11008), (1024, 4096), (5000, 2048), (9000, 128)])
@pytest.mark.parametrize("source", ["bf16", "fp8"])
def test_swiglu(rows, cols, source):
    coat = lib()
    g = torch.Generator(device=DEV).manual_seed(rows + cols)
    out = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    for r, c in places(rows, cols):
        x = torch.randn(rows, 2 * cols, device=DEV, generator=g).bfloat16()
        x[r, c], x[r, cols + c] = 32.0, -28.0   # silu(32) = 32 in FP32: 896 (E4M3 holds both: multiples of their group's maximum)
        kw = dict(gate_up=x)
        a = (None, None)
        if source == "fp8":
            a = (torch.empty(rows, 2 * cols, dtype=torch.uint8, device=DEV), torch.empty(rows, 2 * cols // 128, device=DEV))
            coat.quantize_act(x, *a)
            kw = {}
        for start, want in ((0.0, 896.0), (500.0, 896.0), (1e4, 1e4)):
            amax = torch.tensor([start], device=DEV)
            coat.swiglu(*a, h_codes=out, h_scale=2.0, h_amax=amax, **kw)
            assert abs(float(amax) - want) <= 2.0 ** -20 * want, (start, float(amax))


def test_captured_from_zero():
    """The maximum starts anew on every replay that clears it."""
    coat = lib()
    x = torch.randn(5000, 512, device=DEV).bfloat16()
    w = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    codes, amax = torch.empty(5000, 512, dtype=torch.uint8, device=DEV), torch.zeros(1, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        amax.zero_()
        coat.rms_norm(x, w, 1e-5, y_codes=codes, y_scale=0.05, y_amax=amax)
    for scale in (1.0, 4.0, 0.5, 1.0):
        w.fill_(scale)
        graph.replay()
        got = float(amax)
        other = torch.zeros(1, device=DEV)
        coat.rms_norm(x, w, 1e-5, y_codes=codes, y_scale=0.05, y_amax=other)
        assert got == float(other)
