"""GPU: the two ends of a model together, as a training step uses them with one
matrix for both: embedding lookup, residual norm, cross entropy; backward, both
gradients into one; and the FP8 AdamW step that reads it.

Every operator reads what the one before it wrote, and is checked against its
formula in 64 bits on those values."""
import pytest
import torch

import activation_ref as act
import vocabulary_ref as ref
from activation_ref import BF16, F, assert_between, assert_close
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu

TOKENS, VOCAB, D, EPS, SCALE = 333, 1200, 256, 1e-5, 16.0
NORM, SUM = 40 * F, 2 * (TOKENS + 4) * F   # as in the tests of a block's operators


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


class Step:
    """kind: what the norm hands to the projection and the matrix is kept in."""

    def __init__(self, kind):
        coat = lib()
        self.fp8 = kind == "fp8"
        g = torch.Generator().manual_seed(5)
        matrix = 0.06 * torch.randn(VOCAB, D, generator=g)
        self.w_scale, self.y_scale = (2.0 ** -11, 2.0 ** -6) if self.fp8 else (1.0, 1.0)
        self.matrix = ((matrix / self.w_scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if self.fp8 else matrix.bfloat16()).to(DEV)
        self.norm_w = (1 + 0.2 * torch.randn(D, generator=g)).bfloat16().to(DEV)
        ids = ref.tokens(TOKENS + 1, VOCAB, g)
        self.ids, self.targets = ids[:-1].clone().to(DEV), ids[1:].clone().to(DEV)
        self.ids[-9:] = -1          # padding
        self.targets[:40] = -100    # a prompt
        self.targets[-9:] = -100
        live = (self.targets >= 0).float()
        self.d_loss = live / live.sum()
        e = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
        self.h, self.y = e(TOKENS, D), e(TOKENS, D, dtype=torch.uint8 if self.fp8 else torch.bfloat16)
        self.codes, self.scales, self.rstd = e(TOKENS, D, dtype=torch.uint8), e(TOKENS, D // 128, dtype=torch.float32), e(TOKENS, dtype=torch.float32)
        self.loss, self.lse = e(TOKENS, dtype=torch.float32), e(TOKENS, dtype=torch.float32)
        self.dy, self.dh = e(TOKENS, D), e(TOKENS, D)
        self.d_norm_w, self.dw = e(D, dtype=torch.float32), e(VOCAB, D, dtype=torch.float32)
        self.head_dw = e(VOCAB, D, dtype=torch.float32)
        need = max(coat.cross_entropy_workspace(TOKENS, VOCAB, D),
                   coat.cross_entropy_bwd_workspace(TOKENS, VOCAB, D, piece=512, codes=self.fp8, f32=True),
                   coat.rms_norm_bwd_workspace(TOKENS, D), coat.embedding_bwd_workspace(TOKENS, VOCAB, D))
        self.ws = e(need, dtype=torch.uint8)   # one for all: the calls follow each other on one stream

    def run(self):
        coat = lib()
        coat.embedding(self.matrix, self.ids, self.h, table_scale=self.w_scale, scale=SCALE)
        out = dict(y_codes=self.y, y_scale=self.y_scale) if self.fp8 else dict(y=self.y)
        coat.rms_norm(self.h, self.norm_w, EPS, codes=self.codes, scales=self.scales, rstd=self.rstd, **out)
        kw = dict(x_scale=self.y_scale, weight_scale=self.w_scale, z_loss=1e-4, workspace=self.ws)
        coat.cross_entropy(self.y, self.matrix, self.targets, self.loss, self.lse, **kw)
        coat.cross_entropy_bwd(self.d_loss, self.y, self.matrix, self.targets, self.lse, self.dy, self.dw, **kw)
        self.head_dw.copy_(self.dw)
        coat.rms_norm_bwd(self.dy, self.codes, self.scales, self.rstd, self.norm_w, self.dh, self.d_norm_w, workspace=self.ws)
        coat.embedding_bwd(self.dh, self.ids, self.dw, scale=SCALE, workspace=self.ws, accumulate=True)

    def check(self):
        c = lambda t: t.cpu()  # noqa: E731
        ids, targets = c(self.ids), c(self.targets)
        matrix = ref.values(c(self.matrix), self.w_scale)
        want = ref.lookup(matrix, ids, SCALE)
        assert_close(c(self.h), want, 4 * F * want.abs(), "lookup")
        y, _ = act.norm(c(self.h), c(self.norm_w), EPS)
        if self.fp8:
            act.assert_codes(c(self.y), y / self.y_scale, NORM, "norm")
        else:
            assert_close(c(self.y), y, NORM * y.abs(), "norm")
        r = ref.Entropy(ref.values(c(self.y), self.y_scale), matrix, targets, 1.0, 1e-4, codes=self.fp8)
        for got, v, err, what in ((self.loss, r.loss, r.loss_err, "loss"), (self.lse, r.lse, r.lse_err, "lse")):
            v, err = r.spread(v), r.spread(err)
            assert_between(c(got).double(), v - err, v + err, what)
        dx, dw, dx_err, dw_err = r.gradients(c(self.d_loss), c(self.lse), 2, 3)
        assert_close(c(self.dy), dx, dx_err, "dx")
        assert_close(c(self.head_dw), dw, dw_err, "dw of the projection", rounding=F)
        n = act.restore(c(self.codes), c(self.scales), 128) * c(self.rstd).double()[:, None]
        dh, terms, size = act.norm_bwd(n, c(self.rstd), c(self.dy), c(self.norm_w))
        assert_close(c(self.dh), dh, NORM * size, "dh")
        assert_close(c(self.d_norm_w), terms.sum(0), SUM * terms.abs().sum(0), "norm's weight", rounding=F)
        add, size, count = ref.lookup_bwd(c(self.dh), ids, VOCAB, SCALE)
        head = c(self.head_dw).double()
        assert_close(c(self.dw), head + add, (count + 3) * F * (size + head.abs()), "dw of both", rounding=F)

    def outputs(self):
        return [t.clone() for t in (self.h, self.y, self.loss, self.lse, self.dy, self.dh, self.d_norm_w, self.dw)]


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_step(kind):
    s = Step(kind)
    s.run()
    torch.cuda.synchronize()
    s.check()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_captured(kind):
    """The whole step in a graph, replayed with new tokens between eager steps of the same buffers."""
    s = Step(kind)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        s.ids.copy_(ref.tokens(TOKENS, VOCAB, g, 5 * seed))
        s.targets.copy_(ref.tokens(TOKENS, VOCAB, g, 30 * seed))
        graph.replay()
        torch.cuda.synchronize()
        s.check()
        first = s.outputs()
        s.ws.fill_(255)
        for t in (s.dw, s.dy, s.dh, s.h, s.loss, s.lse):
            t.fill_(3.0)
        s.run()
        assert all(torch.equal(a, b) for a, b in zip(first, s.outputs()))


def test_optimizer_takes_the_gradient():
    """The gradient of both ends drives the FP8 AdamW step of the FP32 matrix: it runs, and the rows that were
    looked up move."""
    coat = lib()
    from adamw_coat_fp8_amd.shard import FP8AdamWShard
    s = Step("bf16")
    shard = FP8AdamWShard([VOCAB * D], group_size=128, device=DEV)
    shard.w.copy_(s.matrix.float().view(-1))
    for step in (1, 2):
        s.run()
        shard.grad.copy_(s.dw.bfloat16().view(-1))
        before = shard.w.clone()
        shard.step(step, lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
        s.matrix.copy_(shard.w.view(VOCAB, D))
        moved = (shard.w - before).view(VOCAB, D).abs().amax(1)
        assert bool((moved[s.ids[s.ids >= 0]] > 0).all()) and bool(torch.isfinite(shard.w).all())
    assert coat is not None
