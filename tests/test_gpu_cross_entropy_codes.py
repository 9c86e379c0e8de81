"""GPU: cross entropy of E4M3 codes where the matrix cores' cut of small
products beside large ones moves a logit far: the target's logit is formed in
FP32, and neither the loss nor the gradients may take anything of it from the
matrix cores."""
import pytest
import torch

import vocabulary_ref as ref
from activation_ref import BF16, F, assert_between, assert_close
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def codes(v):
    return v.float().to(torch.float8_e4m3fn).view(torch.uint8)


class Cut:
    """All rows of x are alike, and so are all rows of w but the target's.

    The first half of the columns: of eight neighbours the first product is
    448 * 448 in all rows of w (its sign changes from eight to eight, so that
    they add up to nothing), and the 7 others are 15 for the target and 0 else,
    which lies more than 13 bits below: their sum is 13440 `sign`.  The second half:
    one product of eight, 448 * target_w for the target and 448 * other_w else,
    which nothing cuts.

    Products are whole numbers and every partial sum is one of 24 bits (with
    powers of two behind it), so the target's FP32 dot product is exact, and so
    are the other rows' on the matrix cores."""

    def __init__(self, rows, scale, sign=1, target_w=0.0, other_w=0.0, cols=2048, vocab=300, padding=0, seed=0):
        self.rows, self.vocab, self.cols, self.scale = rows, vocab, cols, scale
        g = torch.Generator().manual_seed(seed)
        half = cols // 2
        x, w = torch.zeros(cols), torch.zeros(vocab, cols)
        at = 137 % vocab
        x[:half] = 3.75
        x[:half:8] = 448.0
        w[at, :half] = 4.0 * sign
        w[:, 0:half:8] = 448.0
        w[:, 8:half:16] = -448.0
        x[half::8] = 448.0
        w[:, half::8] = other_w
        w[at, half::8] = target_w
        self.x, self.w = codes(x.expand(rows, cols)).contiguous(), codes(w)
        self.targets = torch.full((rows,), at, dtype=torch.int64)
        self.targets[torch.randperm(rows, generator=g)[:padding]] = -100
        self.d_loss = torch.rand(rows, generator=g) + 0.5
        self.d_loss[torch.rand(rows, generator=g) < 0.5] *= -1.0
        self.reference = ref.Entropy(ref.values(self.x, 1.0), ref.values(self.w, 1.0), self.targets, scale)
        # exact products: what is left is the scale in powers of two and one multiplication
        self.reference.l_err = 6 * F * self.reference.l.abs()
        self.l, self.lse = self.reference.l, self.reference.lse

    def args(self):
        return dict(x_scale=1.0, weight_scale=1.0, logit_scale=self.scale)

    def forward(self):
        coat = lib()
        loss, lse = torch.empty(self.rows, device=DEV), torch.empty(self.rows, device=DEV)
        ws = torch.full((coat.cross_entropy_workspace(self.rows, self.vocab, self.cols),), 255, dtype=torch.uint8, device=DEV)
        coat.cross_entropy(self.x.to(DEV), self.w.to(DEV), self.targets.to(DEV), loss, lse, workspace=ws, **self.args())
        return loss.cpu(), lse.cpu()


# rows: the few that need no list, and more
@pytest.mark.parametrize("rows,padding", [(1, 0), (40, 3), (128, 5), (129, 9), (700, 100)])
@pytest.mark.parametrize("cut,others", [
    (-500.0, -1000.0),    # the target's logit lies 500 below what the matrix cores have, and is the largest
    (-20.0, -1000.0),     # by 20: its exponential beside the other's is less than a rounding
    (500.0, -1000.0),     # 500 above: its exponential against the other's is past FP32
    (500.0, 0.0), (-500.0, 0.0),   # the same beside rows as the matrix cores have the target's
    (-30.0, -2.0), (30.0, -2.0), (0.01, -15.0)])
def test_cut_target(rows, padding, cut, others):
    # the sum of the small products is 13440, that of the second half's 448 * 128 * w
    scale = abs(cut) / 13440.0
    w = float(ref.values(codes(torch.tensor([others / (448.0 * 128 * scale)]).clamp(-448, 448)), 1.0)[0])
    c = Cut(rows, scale, 1 if cut > 0 else -1, other_w=w, padding=padding)
    loss, lse = c.forward()
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(lse).all())
    r = c.reference
    # as the reference has it for a logit that is off by l_err, and no more
    err, size = r.l_err.amax(1), r.l.abs().amax(1) + r.lse.abs() + 24
    sums = (64 + c.vocab / 64 / 16 + 8) * 2 * F
    for got, want, slack, what in ((lse, r.lse, err + sums + 8 * F * size, "lse"),
                                   (loss, r.loss, 2 * err + sums + 12 * F * size, "loss")):
        want, slack = r.spread(want), r.spread(slack)
        assert_between(got.double(), want - slack, want + slack, what)


@pytest.mark.parametrize("rows", [50, 400])
@pytest.mark.parametrize("size", [300.0, 3000.0, 30000.0])
def test_far_logits(rows, size):
    """Logits of up to 30000 with some columns 64 times as large, the target the largest of its row: finite, and
    within the bounds."""
    vocab, cols = 1000, 1024
    g = torch.Generator().manual_seed(rows)
    x, w = torch.randn(rows, cols, generator=g), torch.randn(vocab, cols, generator=g)
    many = torch.randperm(cols, generator=g)[:cols // 16]
    x[:, many] *= 8
    w[:, many] *= 8
    x, w = codes((4 * x).clamp(-448, 448)), codes((4 * w).clamp(-448, 448))
    l = ref.values(x, 1.0) @ ref.values(w, 1.0).t()
    scale = float((size / l.abs().max()).float())
    targets = l.argmax(1)
    targets[::7] = l[::7].argsort(1)[:, -2]
    r = ref.Entropy(ref.values(x, 1.0), ref.values(w, 1.0), targets, scale, codes=True)
    coat = lib()
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ws = torch.empty(coat.cross_entropy_workspace(rows, vocab, cols), dtype=torch.uint8, device=DEV)
    coat.cross_entropy(x.to(DEV), w.to(DEV), targets.to(DEV), loss, lse, workspace=ws, logit_scale=scale)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(lse).all())
    for got, want, err, what in ((loss, r.loss, r.loss_err, "loss"), (lse, r.lse, r.lse_err, "lse")):
        assert_between(got.cpu().double(), want - err, want + err, what)


def test_only_the_target():
    """One row of vocabulary: the loss is nothing, whatever the logit."""
    for scale in (1e-3, 0.3, 7.0):
        c = Cut(70, scale, vocab=1, padding=4)
        loss, lse = c.forward()
        want = c.reference.spread(c.lse)
        assert not loss.any()
        assert_between(lse.double(), want - 8 * F * want.abs(), want + 8 * F * want.abs(), "lse")


@pytest.mark.parametrize("rows,padding", [(1, 0), (40, 3), (64, 0), (65, 2), (400, 30)])
@pytest.mark.parametrize("cut,others", [(0.01, -15.0), (-0.01, -15.0), (0.5, -9.0), (-3.0, -9.0), (30.0, -40.0)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_of_a_likely_target(rows, padding, cut, others, dtype):
    """g of the target is p - 1, a small difference: what the cut takes from its logit may not enter it."""
    coat = lib()
    scale = abs(cut) / 13440.0
    w = float(ref.values(codes(torch.tensor([others / (448.0 * 128 * scale)]).clamp(-448, 448)), 1.0)[0])
    c = Cut(rows, scale, 1 if cut > 0 else -1, other_w=w, padding=padding)
    r = c.reference
    lse = r.spread(r.lse).float()
    for piece in (1, c.vocab):
        dx = torch.full((rows, c.cols), 5.0, dtype=torch.bfloat16, device=DEV)
        dw = torch.full((c.vocab, c.cols), 5.0, dtype=dtype, device=DEV)
        ws = torch.full((coat.cross_entropy_bwd_workspace(rows, c.vocab, c.cols, piece=piece, codes=True,
                                                          f32=dtype == torch.float32),), 255, dtype=torch.uint8, device=DEV)
        coat.cross_entropy_bwd(c.d_loss.to(DEV), c.x.to(DEV), c.w.to(DEV), c.targets.to(DEV), lse.to(DEV), dx, dw,
                               workspace=ws, **c.args())
        parts = 2 if dtype == torch.float32 else 1
        want_dx, want_dw, dx_err, dw_err = r.gradients(c.d_loss, lse, parts, -(-c.vocab // piece))
        assert_close(dx.cpu(), want_dx, dx_err, "dx")
        assert_close(dw.cpu(), want_dw, dw_err, "dw", rounding=BF16 if parts == 1 else F)
