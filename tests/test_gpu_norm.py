"""GPU: RMS norm with the E4M3 checkpoint of its input, and its gradient from
the checkpoint, against the formulas in 64 bits."""
import pytest
import torch

import activation_ref as ref
from activation_ref import BF16, F
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-5

# one wave a row up to 1024 threads of four chunks; odd rows; more rows than blocks
SHAPES = [(1, 16, 16), (3, 48, 16), (5, 512, 128), (2, 528, 16), (7, 1024, 64), (9, 1040, 16), (4, 2048, 32),
          (1, 4096, 128), (33, 4096, 128), (600, 4064, 32), (5, 4112, 16), (3, 8192, 64), (2, 11008, 128),
          (2, 16384, 128), (2, 16400, 16), (3, 32768, 128), (2100, 256, 64), (128, 512, 64), (129, 512, 16), (500, 2048, 32),
          (513, 4096, 128)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def data(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * torch.exp(torch.randn(cols, generator=g))
    w = 1.0 + 0.3 * torch.randn(cols, generator=g)
    r = torch.randn(rows, cols, generator=g)
    return x.bfloat16(), w.bfloat16(), r.bfloat16()


def forward(x, w, G, residual=None, fp8=None, ckpt=True, both=False):
    coat = lib()
    rows, cols = x.shape
    xd, wd = x.to(DEV), w.to(DEV)
    o = dict(y=torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=DEV) if fp8 is None or both else None,
             y_codes=torch.full((rows, cols), 0x55, dtype=torch.uint8, device=DEV) if fp8 is not None else None,
             y_amax=torch.zeros(1, device=DEV) if fp8 is not None else None,
             residual_out=torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV) if residual is not None else None)
    if ckpt:
        o.update(codes=torch.full((rows, cols), 0x55, dtype=torch.uint8, device=DEV),
                 scales=torch.full((rows, cols // G), -1.0, device=DEV), rstd=torch.full((rows,), -1.0, device=DEV))
    coat.rms_norm(xd, wd, EPS, residual=None if residual is None else residual.to(DEV), y_scale=fp8 or 1.0,
                  group_size=G, **o)
    torch.cuda.synchronize()
    return {k: None if v is None else v.cpu() for k, v in o.items()}


# squares: chains of 8 per chunk (at most 4 chunks), 6 lane steps, up to 16
# waves, and the mean, eps, root, quotient; half of the sum's error reaches rstd
RSTD = (8 * 4 + 6 + 16 + 4) * F


@pytest.mark.parametrize("rows,cols,G", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_forward(rows, cols, G, residual):
    x, w, r = data(rows, cols, rows + cols)
    o = forward(x, w, G, r if residual else None, fp8=2.0 ** -5, both=True)
    h = (x.float() + r.float()).bfloat16() if residual else x
    if residual:
        assert torch.equal(o["residual_out"], h)
    y, rstd = ref.norm(h, w, EPS)
    ref.assert_close(o["rstd"], rstd, RSTD * rstd, "rstd", F)
    ref.assert_close(o["y"], y, (RSTD + 2 * F) * y.abs(), "y")
    ref.assert_codes(o["y_codes"], y * 32.0, RSTD + 3 * F, "y_codes")
    top = y.abs().max()
    assert abs(float(o["y_amax"]) - top) <= (RSTD + 2 * F) * top
    codes, scales = ref.quantize(h, G)
    assert torch.equal(ref.code_values(o["codes"]), ref.code_values(codes))
    assert torch.equal(o["scales"], scales)


def test_checkpoint_is_the_quantizers():
    x, w, _ = data(37, 4096, 5)
    o = forward(x, w, 64)
    coat = lib()
    codes = torch.empty(37, 4096, dtype=torch.uint8, device=DEV)
    scales = torch.empty(37, 64, device=DEV)
    coat.quantize_act(x.to(DEV), codes, scales, group_size=64)
    assert torch.equal(o["codes"], codes.cpu()) and torch.equal(o["scales"], scales.cpu())


def test_zero_row_and_saturation():
    x, w, _ = data(4, 256, 3)
    x[1] = 0
    o = forward(x, w, 128, fp8=2.0 ** -12, both=True)
    assert (o["y"][1] == 0).all() and (o["codes"][1] == 0).all() and (o["scales"][1] == 0).all()
    y, _ = ref.norm(x, w, EPS)
    assert (y.abs() * 4096 > 464).any()
    ref.assert_codes(o["y_codes"], y * 4096.0, RSTD + 3 * F, "saturated codes")


def test_not_finite_stays_in_its_row():
    x, w, _ = data(6, 1024, 4)
    clean = forward(x, w, 128, fp8=0.125, both=True)
    bad = x.clone()
    bad[2, 5], bad[4, 1000] = float("nan"), float("inf")
    o = forward(bad, w, 128, fp8=0.125, both=True)
    keep = [0, 1, 3, 5]
    for k in ("y", "y_codes", "codes", "scales", "rstd"):
        assert torch.equal(o[k][keep], clean[k][keep]), k
    assert o["y"][2].isnan().all()
    assert o["y"][4, 1000].isnan() and o["rstd"][4] == 0   # infinity * 0; the rest of the row is 0
    assert not o["scales"][2, 0].isfinite() and not o["scales"][4, 7].isfinite()
    assert ref.code_values(o["y_codes"][2]).isnan().all()


def backward(dy, codes, scales, rstd, w, G, d_residual=None, dw=True, accumulate=None):
    coat = lib()
    rows, cols = dy.shape
    dx = torch.full((rows, cols), 9.0, dtype=torch.bfloat16, device=DEV)
    out = None
    ws = None
    if dw:
        out = torch.full((cols,), 3.0, device=DEV) if accumulate is None else accumulate.to(DEV).clone()
        ws = torch.full((coat.rms_norm_bwd_workspace(rows, cols) // 4,), float("nan"), device=DEV)
    coat.rms_norm_bwd(dy.to(DEV), codes.to(DEV), scales.to(DEV), rstd.to(DEV), w.to(DEV), dx, out,
                      d_residual=None if d_residual is None else d_residual.to(DEV), workspace=ws,
                      accumulate=accumulate is not None, group_size=G)
    torch.cuda.synchronize()
    return dx.cpu(), None if out is None else out.cpu()


def chain(rows):
    """FP32 additions behind one value of dw: the rows of one of at least 256
    blocks, 8 partial sums of a slice, 6 joins, and the product's roundings; up
    to 512 rows may go in slices of at most 32, and 6 joins."""
    return max(-(-rows // 256) + 8, 32 if rows <= 512 else 0) + 6 + 4


@pytest.mark.parametrize("rows,cols,G", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_backward(rows, cols, G, residual):
    x, w, dr = data(rows, cols, rows * 3 + cols)
    g = torch.Generator().manual_seed(rows)
    dy = (1e-3 * torch.randn(rows, cols, generator=g)).bfloat16()
    codes, scales = ref.quantize(x, G)
    rstd = ref.norm(x, w, EPS)[1].float()
    dx, dw = backward(dy, codes, scales, rstd, w, G, dr if residual else None)
    n = ref.restore(codes, scales, G) * rstd.double().unsqueeze(1)
    want, terms, size = ref.norm_bwd(n, rstd, dy, w)
    # n: 2 roundings, dn: 1, the sum as in the forward pass plus those, dx: 3, the addition: 1
    slack = (8 * 4 + 6 + 16 + 12) * F * size
    if residual:
        want = want + dr.double()
        slack = slack + F * dr.double().abs()
    ref.assert_close(dx, want, slack, "dx")
    ref.assert_close(dw, terms.sum(0), chain(rows) * F * terms.abs().sum(0), "dw", F)
    none, _ = backward(dy, codes, scales, rstd, w, G, dr if residual else None, dw=False)
    assert torch.equal(none, dx)


def test_weight_gradient_accumulates_and_repeats():
    rows, cols, G = 1500, 2048, 128
    x, w, base = data(rows, cols, 8)
    dy = x.flip(0).contiguous()
    codes, scales = ref.quantize(x, G)
    rstd = ref.norm(x, w, EPS)[1].float()
    _, once = backward(dy, codes, scales, rstd, w, G)
    _, again = backward(dy, codes, scales, rstd, w, G)
    assert torch.equal(once, again)
    _, added = backward(dy, codes, scales, rstd, w, G, accumulate=base[0].float())
    assert torch.equal(added, base[0].float() + once)


def test_gradient_against_differences():
    """Inputs that E4M3 holds exactly (small multiples of a power of two, each
    group's maximum 448 * 2^-8): the checkpoint loses nothing, so the gradient
    is the function's own."""
    rows, cols, G, h = 3, 64, 16, 1e-5
    g = torch.Generator().manual_seed(1)
    x = torch.randint(-14, 15, (rows, cols), generator=g).double() / 8
    x[:, ::G] = 1.75
    w = (1 + torch.randint(-4, 5, (cols,), generator=g).double() / 16)
    dy = torch.randn(rows, cols, generator=g).bfloat16()
    o = forward(x.bfloat16(), w.bfloat16(), G)
    assert torch.equal(ref.restore(o["codes"], o["scales"], G), x)
    dx, dw = backward(dy, o["codes"], o["scales"], o["rstd"], w.bfloat16(), G)

    def loss(x, w):
        return (ref.norm(x, w, EPS)[0] * dy.double()).sum()

    want = torch.zeros(rows, cols, dtype=torch.float64)
    for i in range(rows):
        for j in range(cols):
            d = torch.zeros(rows, cols, dtype=torch.float64)
            d[i, j] = h
            want[i, j] = (loss(x + d, w) - loss(x - d, w)) / (2 * h)
    # the difference: h^2 / 6 of a third derivative of about 10, and 2^-53 * |loss| / h
    ref.assert_close(dx, want, torch.full_like(want, 1e-8) + 60 * F, "dx")
    want_w = torch.stack([(loss(x, w + h * torch.eye(cols)[j].double()) - loss(x, w - h * torch.eye(cols)[j].double()))
                          / (2 * h) for j in range(cols)])
    ref.assert_close(dw, want_w, torch.full_like(want_w, 1e-8) + 60 * F, "dw", F)


def test_no_rows():
    coat = lib()
    e = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    coat.rms_norm(e, w, EPS, y=e)
    dw = torch.full((256,), 5.0, device=DEV)
    c, s, r = torch.empty(0, 256, dtype=torch.uint8, device=DEV), torch.empty(0, 2, device=DEV), torch.empty(0, device=DEV)
    coat.rms_norm_bwd(e, c, s, r, w, e, dw, accumulate=True)
    assert (dw == 5).all()
    coat.rms_norm_bwd(e, c, s, r, w, e, dw)
    assert (dw == 0).all()


def test_stream_and_graph():
    """On a stream of its own, and captured: every replay equals the eager
    call, with eager work between the replays."""
    coat = lib()
    rows, cols, G = 700, 4096, 128
    x, w, r = [t.to(DEV) for t in data(rows, cols, 11)]
    mk = lambda: dict(y=torch.zeros_like(x), codes=torch.zeros(rows, cols, dtype=torch.uint8, device=DEV),  # noqa: E731
                      scales=torch.zeros(rows, cols // G, device=DEV), rstd=torch.zeros(rows, device=DEV),
                      residual_out=torch.zeros_like(x), dx=torch.zeros_like(x), dw=torch.zeros(cols, device=DEV),
                      ws=torch.zeros(coat.rms_norm_bwd_workspace(rows, cols) // 4, device=DEV))

    def go(o, stream=None):
        coat.rms_norm(x, w, EPS, residual=r, residual_out=o["residual_out"], y=o["y"], codes=o["codes"],
                      scales=o["scales"], rstd=o["rstd"], group_size=G, stream=stream)
        coat.rms_norm_bwd(o["y"], o["codes"], o["scales"], o["rstd"], w, o["dx"], o["dw"], d_residual=r,
                          workspace=o["ws"], group_size=G, stream=stream)

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
        for k in ("dx", "dw", "y"):
            captured[k].zero_()
        go(other)
        graph.replay()
        torch.cuda.synchronize()
        for k in ("y", "codes", "scales", "rstd", "residual_out", "dx", "dw"):
            assert torch.equal(captured[k], eager[k]) and torch.equal(other[k], eager[k]), k
