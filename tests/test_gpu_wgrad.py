"""GPU: the weight gradient from an E4M3 input, exactly on small integers and
within bounds on random data, and the activation operators run together."""
import pytest
import torch

import activation_ref as ref
from activation_ref import F
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def run(dy, codes, scales, dtype, G=128, base=None):
    coat = lib()
    (m, n), k = dy.shape, codes.shape[1]
    dw = torch.full((n, k), 5.0, dtype=dtype, device=DEV) if base is None else base.to(DEV).clone()
    ws = torch.full((coat.weight_grad_workspace(m, n, k) // 4,), float("nan"), device=DEV)
    coat.weight_grad(dy.to(DEV), codes.to(DEV), scales.to(DEV) if isinstance(scales, torch.Tensor) else scales, dw,
                     accumulate=base is not None, workspace=ws, group_size=G)
    torch.cuda.synchronize()
    return dw.cpu()


def product(dy, x):
    """dy^T x in 64 bits, on the GPU (float64 matrix product)."""
    return (dy.double().to(DEV).t().contiguous() @ x.double().to(DEV)).cpu()


# rows around the 64-row steps and the three stages; edges of both tile sizes;
# one and several row splits; 256 tiles of 256 x 256 (the large ones) with edges
SHAPES = [(1, 16, 16), (2, 16, 128), (63, 128, 128), (64, 144, 128), (65, 128, 256), (128, 272, 384), (129, 16, 640),
          (193, 400, 128), (256, 128, 128), (511, 48, 256), (700, 512, 640), (1024, 128, 128), (4000, 128, 256),
          (2085, 656, 128), (1, 4096, 4096), (70, 4112, 4096), (200, 3856, 4224), (333, 2048, 2048), (130, 16, 16384),
          (130, 2816, 2816), (70, 2064, 2176), (200, 3328, 3328), (33, 128, 33280), (65, 144, 33280)]


def integers(m, n, k, seed):
    """dy and codes of small integers: every product and sum is exact."""
    g = torch.Generator().manual_seed(seed)
    dy = torch.randint(-8, 9, (m, n), generator=g).bfloat16()
    codes = torch.randint(-8, 9, (m, k), generator=g).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return dy, codes, g


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact_under_one_scale(m, n, k):
    dy, codes, g = integers(m, n, k, m + n + k)
    want = product(dy, ref.code_values(codes)) * 0.5
    assert torch.equal(run(dy, codes, 0.5, torch.float32).double(), want)
    assert torch.equal(run(dy, codes, 0.5, torch.bfloat16), want.float().bfloat16())
    base = torch.randint(-100, 100, (n, k), generator=g).float()
    assert torch.equal(run(dy, codes, 0.5, torch.float32, base=base).double(), base.double() + want)


@pytest.mark.parametrize("G", [16, 32, 64, 128])
@pytest.mark.parametrize("m,n,k", [s for s in SHAPES if s[2] % 128 == 0])
def test_exact_with_group_scales(m, n, k, G):
    """Scales of powers of two keep the sums exact."""
    dy, codes, g = integers(m, n, k, m * 3 + n + k)
    scales = torch.exp2(torch.randint(-1, 3, (m, k // G), generator=g).float())
    want = product(dy, ref.restore(codes, scales, G))
    assert torch.equal(run(dy, codes, scales, torch.float32, G).double(), want)
    assert torch.equal(run(dy, codes, scales, torch.bfloat16, G), want.float().bfloat16())


def test_group_sizes_that_do_not_divide_a_tile():
    dy, codes, g = integers(77, 48, 16 * 21, 4)
    scales = torch.exp2(torch.randint(-1, 3, (77, 21), generator=g).float())
    assert torch.equal(run(dy, codes, scales, torch.float32, 16).double(), product(dy, ref.restore(codes, scales, 16)))


@pytest.mark.parametrize("m,n,k", [(333, 2048, 2048), (700, 512, 640), (4000, 128, 256), (200, 3856, 4224)])
def test_random(m, n, k):
    """Every code and scale: sums of m terms in FP32 (2^-23 a step: the matrix
    cores may truncate), x rounded to BF16 under group scales."""
    g = torch.Generator().manual_seed(m)
    dy = torch.randn(m, n, generator=g).bfloat16()
    codes = torch.randint(0, 256, (m, k), generator=g).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x7E   # the two NaN codes
    x = ref.code_values(codes) * 0.37
    size = product(dy.abs(), x.abs())
    s = float(torch.tensor(0.37))
    ref.assert_close(run(dy, codes, 0.37, torch.float32), product(dy, ref.code_values(codes) * s),
                     (m + 4) * 2 * F * size, "one scale", F)
    scales = torch.rand(m, k // 128, generator=g) + 0.01
    x = ref.restore(codes, scales, 128)
    got = run(dy, codes, scales, torch.bfloat16)
    ref.assert_close(got, product(dy, x), ((m + 4) * 2 * F + ref.BF16) * product(dy.abs(), x.abs()), "groups")
    assert torch.equal(got, run(dy, codes, scales, torch.bfloat16))


def test_no_rows():
    e, c = torch.empty(0, 256, dtype=torch.bfloat16), torch.empty(0, 128, dtype=torch.uint8)
    assert (run(e, c, 1.0, torch.bfloat16) == 0).all() and (run(e, c, 1.0, torch.float32) == 0).all()
    assert (run(e, c, 1.0, torch.float32, base=torch.full((256, 128), 2.0)) == 2).all()


def test_not_finite_stays_in_its_row_and_column():
    """Also in the last row of a ragged step, which the loads past it repeat."""
    for row in (0, 76):
        dy, codes, _ = integers(77, 144, 128, 9)
        clean = run(dy, codes, 1.0, torch.float32)
        bad = dy.clone()
        bad[row, 5] = float("inf")
        codes2 = codes.clone()
        codes2[row, 9] = 0x7F
        got = run(bad, codes2, 1.0, torch.float32)
        assert got[:, 9].isnan().all() and not got[5].isfinite().any()
        keep = torch.ones(144, 128, dtype=torch.bool)
        keep[5], keep[:, 9] = False, False
        assert torch.equal(got[keep], clean[keep])


def test_graph_and_stream():
    coat = lib()
    for m, n, k in ((1500, 256, 384), (300, 4096, 4096)):
        dy, codes, g = [t.to(DEV) if isinstance(t, torch.Tensor) else t for t in integers(m, n, k, 2)]
        scales = torch.ones(m, k // 128, device=DEV)
        mk = lambda: (torch.zeros(n, k, dtype=torch.bfloat16, device=DEV),  # noqa: E731
                      torch.zeros(coat.weight_grad_workspace(m, n, k), dtype=torch.uint8, device=DEV))
        go = lambda o, stream=None: coat.weight_grad(dy, codes, scales, o[0], workspace=o[1], stream=stream)  # noqa: E731
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
            captured[0].zero_()
            go(other)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(captured[0], eager[0]) and torch.equal(other[0], eager[0])
