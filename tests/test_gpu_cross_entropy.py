"""GPU: softmax cross entropy from the output projection and its gradients
against the formulas in 64 bits, within bounds derived from the roundings."""
import pytest
import torch

import vocabulary_ref as ref
from activation_ref import BF16, F, assert_between, assert_close
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class Case:
    def __init__(self, rows, vocab, cols, kind="bf16", padding=0, seed=0, logit_scale=1.0, z=0.0, spread=1.0):
        g = torch.Generator().manual_seed(rows + 3 * vocab + 7 * cols + seed)
        self.kind, self.logit_scale, self.z = kind, logit_scale, z
        x = spread * torch.randn(rows, cols, generator=g)
        w = torch.randn(vocab, cols, generator=g) / cols ** 0.5
        self.targets = ref.tokens(rows, vocab, g, padding)
        if kind == "fp8":
            self.scales = (2.0 ** -5 * 1.1, 2.0 ** -9 * 0.9)
            self.x, self.w = ((v / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                              for v, s in ((x, self.scales[0]), (w, self.scales[1])))
        else:
            self.scales = (1.0, 1.0)
            self.x, self.w = x.bfloat16(), w.bfloat16()
        self.rows, self.vocab, self.cols = rows, vocab, cols
        self.d_loss = torch.rand(rows, generator=g) + 0.1
        live = ref.live_rows(self.targets, vocab)
        # what padding holds reaches nothing
        self.d_loss[~live] = float("nan")
        if kind == "bf16":
            self.x[~live] = float("nan")
        else:
            self.x[~live] = 0x7F

    def reference(self):
        x = ref.values(self.x, self.scales[0])
        return ref.Entropy(x, ref.values(self.w, self.scales[1]), self.targets, self.logit_scale, self.z,
                           codes=self.kind == "fp8")

    def scale_args(self):
        return dict(x_scale=self.scales[0], weight_scale=self.scales[1], logit_scale=self.logit_scale, z_loss=self.z)

    def forward(self):
        coat = lib()
        loss, lse = (torch.full((self.rows,), 9.0, device=DEV) for _ in range(2))
        ws = torch.full((coat.cross_entropy_workspace(self.rows, self.vocab, self.cols),), 255, dtype=torch.uint8,
                        device=DEV)
        coat.cross_entropy(self.x.to(DEV), self.w.to(DEV), self.targets.to(DEV), loss, lse, workspace=ws,
                           **self.scale_args())
        torch.cuda.synchronize()
        return loss.cpu(), lse.cpu()

    def backward(self, lse, dtype=torch.bfloat16, piece=1 << 22, base=None, dx=True, dw=True):
        coat = lib()
        d_x = torch.full((self.rows, self.cols), 5.0, dtype=torch.bfloat16, device=DEV) if dx else None
        d_w = None
        if dw:
            d_w = torch.full((self.vocab, self.cols), 5.0, dtype=dtype, device=DEV) if base is None else base.to(DEV).clone()
        ws = torch.full((coat.cross_entropy_bwd_workspace(self.rows, self.vocab, self.cols, piece=piece,
                                                          codes=self.kind == "fp8", f32=dtype == torch.float32),),
                        255, dtype=torch.uint8, device=DEV)
        coat.cross_entropy_bwd(self.d_loss.to(DEV), self.x.to(DEV), self.w.to(DEV), self.targets.to(DEV), lse.to(DEV),
                               d_x, d_w, workspace=ws, accumulate=base is not None, **self.scale_args())
        torch.cuda.synchronize()
        return d_x.cpu() if dx else None, d_w.cpu() if dw else None

    def check_forward(self):
        r = self.reference()
        loss, lse = self.forward()
        for got, want, err, what in ((loss, r.loss, r.loss_err, "loss"), (lse, r.lse, r.lse_err, "lse")):
            want, err = r.spread(want), r.spread(err)
            assert_between(got.double(), want - err, want + err, what)   # zeros without a target
        return r, lse

    def check_backward(self, r, lse, **kw):
        parts = 2 if kw.get("dtype") == torch.float32 else 1
        pieces = -(-self.vocab // kw.get("piece", 1 << 22))
        dx, dw, dx_err, dw_err = r.gradients(self.d_loss, lse, parts, pieces)
        got_dx, got_dw = self.backward(lse, **kw)
        if got_dx is not None:
            assert_close(got_dx, dx, dx_err, "dx")
        if got_dw is not None:
            if kw.get("base") is not None:
                dw = dw + kw["base"].double()
            assert_close(got_dw, dw, dw_err, "dw", rounding=BF16 if parts == 1 else F)


# rows around the thin tile (64), the halves (128) and the tiles (256); ragged
# vocabularies around the tiles of 64 and 256; 64 and more columns
BF16_CASES = [(1, 1, 64, 0), (1, 2, 128, 0), (1, 1000, 64, 0), (7, 63, 192, 2), (63, 64, 64, 0), (64, 65, 320, 6),
              (65, 257, 64, 1), (100, 300, 128, 0), (128, 256, 256, 12), (129, 1025, 64, 30), (256, 127, 448, 0),
              (257, 511, 64, 100), (300, 3001, 128, 0), (700, 2049, 192, 333), (1025, 700, 64, 0), (5, 20000, 1024, 1),
              (60, 5000, 2048, 0), (2100, 5000, 64, 900)]
FP8_CASES = [(1, 1, 128, 0), (3, 500, 256, 1), (64, 129, 128, 0), (65, 257, 128, 6), (200, 1000, 384, 0),
             (513, 2049, 128, 100), (61, 7001, 1024, 0)]
CASES = [("bf16",) + c for c in BF16_CASES] + [("fp8",) + c for c in FP8_CASES]


@pytest.mark.parametrize("kind,rows,vocab,cols,padding", CASES)
def test_forward(kind, rows, vocab, cols, padding):
    Case(rows, vocab, cols, kind, padding).check_forward()
    Case(rows, vocab, cols, kind, padding, seed=1, logit_scale=0.37, z=1e-3, spread=6.0).check_forward()


@pytest.mark.parametrize("kind,rows,vocab,cols,padding", CASES)
def test_gradients(kind, rows, vocab, cols, padding):
    c = Case(rows, vocab, cols, kind, padding, z=1e-3, logit_scale=0.8)
    r = c.reference()
    lse = r.spread(r.lse).float()
    c.check_backward(r, lse)
    c.check_backward(r, lse, piece=1)             # the least workspace
    c.check_backward(r, lse, piece=vocab // 3 + 1, dtype=torch.float32)
    base = torch.randn(vocab, cols, generator=torch.Generator().manual_seed(1))
    c.check_backward(r, lse, dtype=torch.float32, base=base)
    c.check_backward(r, lse, dx=False)
    c.check_backward(r, lse, dw=False)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_rounds_of_tiles(kind):
    """More tiles than compute units, with a last round in halves, dead rows among them, and few columns to contract."""
    c = Case(4200, 4500, 128, kind, padding=1300)
    r, lse = c.check_forward()
    c.check_backward(r, lse, piece=2304)
    c.check_backward(r, lse)


@pytest.mark.parametrize("rows", [1, 50, 300])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_no_targets(rows, kind):
    c = Case(rows, 500, 128, kind, padding=rows)
    loss, lse = c.forward()
    assert not loss.any() and not lse.any()
    for piece in (1, 500):
        dx, dw = c.backward(lse, piece=piece)
        assert torch.equal(dx, torch.zeros_like(dx)) and torch.equal(dw, torch.zeros_like(dw))
    base = torch.randn(500, 128)
    assert torch.equal(c.backward(lse, torch.float32, base=base)[1], base)


@pytest.mark.parametrize("kind,rows,vocab,cols", [("bf16", 61, 5000, 1024), ("bf16", 40, 3000, 2112), ("fp8", 33, 4100, 512),
                                                 ("bf16", 64, 2500, 2048), ("bf16", 100, 3000, 1024)])
def test_gradients_apart(kind, rows, vocab, cols):
    """dx and dw are the same bits asked for together or alone (few rows finish dx beside dw's product)."""
    c = Case(rows, vocab, cols, kind, padding=3, z=1e-3)
    lse = c.forward()[1]
    both = c.backward(lse)
    assert torch.equal(c.backward(lse, dw=False)[0], both[0])
    assert torch.equal(c.backward(lse, dx=False)[1], both[1])


def test_no_rows():
    c = Case(0, 300, 64)
    c.forward()
    assert torch.equal(c.backward(torch.zeros(0))[1], torch.zeros(300, 64, dtype=torch.bfloat16))
    assert torch.equal(c.backward(torch.zeros(0), torch.float32, base=torch.ones(300, 64))[1], torch.ones(300, 64))


def test_far_logits():
    """Logits of thousands: the maximum is taken out before the exponentials."""
    c = Case(90, 700, 64, spread=2000.0)
    r, lse = c.check_forward()
    dx, dw = c.backward(lse)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("rows", [20, 200])
def test_rows_do_not_mix(rows):
    """A NaN or infinity in a row's hidden state reaches that row alone (and the weights' gradient)."""
    c = Case(rows, 600, 64)
    loss, lse = c.forward()
    dx, _ = c.backward(lse)
    clean = c.x.clone()
    for bad in (float("nan"), float("inf")):
        c.x = clean.clone()
        c.x[3, 5] = bad
        l2, s2 = c.forward()
        d2, w2 = c.backward(s2)
        others = torch.arange(rows) != 3
        assert torch.equal(l2[others], loss[others]) and torch.equal(s2[others], lse[others])
        assert torch.equal(d2[others], dx[others]) and not torch.isfinite(l2[3]) and torch.isnan(w2).any()


def test_gradient_against_differences():
    """The gradients along random directions against central differences of the loss in 64 bits: the steps lie on
    the BF16 grid, so both sides see the same inputs."""
    c = Case(40, 300, 64, z=1e-2)
    r, lse = c.check_forward()
    dx, dw = c.backward(lse, torch.float32)
    g = torch.Generator().manual_seed(5)
    sx = torch.randn(40, 64, generator=g, dtype=torch.float64)
    sw = torch.randn(300, 64, generator=g, dtype=torch.float64) / 8

    def total(h):
        e = ref.Entropy(c.x.double() + h * sx, c.w.double() + h * sw, c.targets, 1.0, 1e-2)
        return (e.loss * c.d_loss.double()).sum()

    h = 1e-5
    slope = (total(h) - total(-h)) / (2 * h)
    _, _, dx_err, dw_err = r.gradients(c.d_loss, lse, 2)
    slack = ((dx_err + 2 * BF16 * dx.abs().double()) * sx.abs()).sum() + (dw_err * sw.abs()).sum()
    assert abs((dx.double() * sx).sum() + (dw.double() * sw).sum() - slope) <= slack + 1e-6


def test_same_result_again():
    c = Case(500, 1500, 128, padding=99)
    loss, lse = c.forward()
    dx, dw = c.backward(lse, piece=512)
    for _ in range(3):
        a, b = c.forward()
        assert torch.equal(a, loss) and torch.equal(b, lse)
        a, b = c.backward(lse, piece=512)
        assert torch.equal(a, dx) and torch.equal(b, dw)


@pytest.mark.parametrize("rows", [30, 400])
def test_captured(rows):
    """Loss and gradients in one graph, replayed with new targets between eager calls of the same buffers."""
    coat = lib()
    c = Case(rows, 900, 64)
    x, w, d = c.x.to(DEV), c.w.to(DEV), c.d_loss.to(DEV)
    targets = c.targets.to(DEV)
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = torch.empty(max(coat.cross_entropy_workspace(rows, 900, 64),
                         coat.cross_entropy_bwd_workspace(rows, 900, 64, piece=512)), dtype=torch.uint8, device=DEV)

    def step():
        coat.cross_entropy(x, w, targets, loss, lse, workspace=ws)
        coat.cross_entropy_bwd(d, x, w, targets, lse, dx, dw, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(5):
        targets.copy_(ref.tokens(rows, 900, torch.Generator().manual_seed(seed), 7 * seed))
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in (loss, lse, dx, dw)]
        for t in (loss, lse, dx, dw):
            t.fill_(3.0)
        ws.fill_(255)
        step()
        assert all(torch.equal(a, b) for a, b in zip(first, (loss, lse, dx, dw)))


@pytest.mark.parametrize("kind,rows,vocab,cols", [("bf16", 700, 300, 2048), ("bf16", 2049, 1000, 1024), ("fp8", 600, 500, 1024),
                                                  ("bf16", 64, 300, 1024), ("bf16", 1000, 2100, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_workspaces_of_the_size_asked_for(kind, rows, vocab, cols, dtype):
    """Few vocabulary rows beside the columns, where one piece takes less than several (their sums of dx): every
    query's size is taken, and nothing behind it is written."""
    coat = lib()
    c = Case(rows, vocab, cols, kind, padding=rows // 9)
    r = c.reference()
    lse = r.spread(r.lse).float()
    dx, dw, dx_err, dw_err = r.gradients(c.d_loss, lse, 2 if dtype == torch.float32 else 1, -(-vocab // 256))
    done = set()
    for piece in (8192, 1024, 512, 1):
        n = coat.cross_entropy_bwd_workspace(rows, vocab, cols, piece=piece, codes=kind == "fp8", f32=dtype == torch.float32)
        if n in done:
            continue
        done.add(n)
        whole = torch.full((n + 4096,), 77, dtype=torch.uint8, device=DEV)
        d_x = torch.full((rows, cols), 5.0, dtype=torch.bfloat16, device=DEV)
        d_w = torch.full((vocab, cols), 5.0, dtype=dtype, device=DEV)
        coat.cross_entropy_bwd(c.d_loss.to(DEV), c.x.to(DEV), c.w.to(DEV), c.targets.to(DEV), lse.to(DEV), d_x, d_w,
                               workspace=whole[:n], **c.scale_args())
        assert_close(d_x.cpu(), dx, dx_err, "dx")
        assert_close(d_w.cpu(), dw, dw_err, "dw", rounding=BF16 if dtype == torch.bfloat16 else F)
        assert bool((whole[n:] == 77).all())


SIGNS = ("negative", "zeros", "none", "wide", "infinite", "nan", "tiny")


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("rows", [1, 30, 64, 65, 900])
@pytest.mark.parametrize("what", SIGNS)
def test_gradients_of_any_d_loss(kind, rows, what):
    """d_loss of both signs, the largest magnitude negative; zeros among them or alone; from 1e-6 to 1e4; of 2^-100;
    an infinity or a NaN, which stays in its row."""
    c = Case(rows, 700, 128, kind, padding=rows // 10, z=1e-3)
    g = torch.Generator().manual_seed(rows)
    live = torch.nonzero(ref.live_rows(c.targets, c.vocab))[:, 0]
    n = len(live)
    d = torch.rand(n, generator=g) + 0.1
    d[torch.rand(n, generator=g) < 0.5] *= -1.0
    d[0] = -3.0
    if what == "zeros":
        d[::3] = 0.0
    elif what == "none":
        d[:] = 0.0
    elif what == "wide":
        d *= 10.0 ** (torch.rand(n, generator=g) * 10 - 6)
    elif what == "tiny":
        d *= 2.0 ** -100
    bad = live[n // 2]
    c.d_loss[live] = d
    r = c.reference()
    lse = r.spread(r.lse).float()
    if what in ("infinite", "nan"):
        others = torch.arange(rows) != bad
        want = r.gradients(torch.where(others, c.d_loss, torch.zeros(())), lse, 1)
        c.d_loss[bad] = -float(what[:3])
        for dtype in (torch.bfloat16, torch.float32):
            dx, dw = c.backward(lse, dtype)
            assert not torch.isfinite(dx[bad]).any() and not torch.isfinite(dw[c.targets[bad]]).any()
            assert_close(dx[others], want[0][others], want[2][others], "dx")
        return
    c.check_backward(r, lse)
    c.check_backward(r, lse, dtype=torch.float32, piece=256)
    if what == "none":
        dx, dw = c.backward(lse)
        assert not dx.any() and not dw.any()


@pytest.mark.parametrize("kind,cols", [("bf16", 64), ("fp8", 128)])
@pytest.mark.parametrize("rows", [1, 30, 64, 65, 900])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_equal_d_loss_is_not_rounded(kind, cols, rows, sign):
    """Equal d, of either sign, that lie between two BF16 values: g holds their share of the largest |d|, which is
    exact.  All of the probability is on row 0 of the vocabulary, nothing on the target."""
    coat = lib()
    vocab, d = 300, sign * (1.0 + 2.0 ** -8 - 2.0 ** -20)
    x, w = torch.ones(rows, cols), torch.full((vocab, cols), -3.25)
    w[0] = 0.0
    cast = (lambda t: t.bfloat16()) if kind == "bf16" else (lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8))
    x, w = cast(x).to(DEV), cast(w).to(DEV)
    targets = torch.full((rows,), 7, device=DEV)
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    coat.cross_entropy(x, w, targets, loss, lse, workspace=torch.empty(coat.cross_entropy_workspace(rows, vocab, cols),
                                                                     dtype=torch.uint8, device=DEV))
    # the scale in powers of two, a logit, ln 2 and the product with it: four roundings
    assert not lse.any() and bool(((loss.double() - 3.25 * cols).abs() <= 5 * F * 3.25 * cols).all())
    dx, dw = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV), torch.empty(vocab, cols, device=DEV)
    ws = torch.empty(coat.cross_entropy_bwd_workspace(rows, vocab, cols, codes=kind == "fp8", f32=True), dtype=torch.uint8,
                     device=DEV)
    coat.cross_entropy_bwd(torch.full((rows,), d, device=DEV), x, w, targets, lse, dx, dw, workspace=ws)
    assert bool((dx == torch.tensor(3.25 * d, dtype=torch.float64).bfloat16().to(DEV)).all())
    want = torch.zeros(vocab, cols, dtype=torch.float64, device=DEV)
    want[0], want[7] = rows * d, -rows * d
    assert bool(((dw.double() - want).abs() <= F * want.abs()).all())
