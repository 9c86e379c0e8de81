"""GPU: the vocabulary operators where offsets pass 32 bits, outputs and
workspaces that must not be overrun, and calls on other streams."""
import pytest
import torch

import vocabulary_ref as ref
from activation_ref import BF16, F, assert_between, assert_close
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu
LAST = 96


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    torch.cuda.empty_cache()


def randn(*shape, seed=0, scale=1.0):
    return (scale * torch.randn(*shape, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))).bfloat16()


def test_far_table():
    """A table of 5.7 GB, and its gradient in both types (5.7 and 11.5 GB)."""
    coat = lib()
    vocab, cols, rows = 700_000, 4096, 300
    table = torch.zeros(vocab, cols, dtype=torch.bfloat16, device=DEV)
    table[-LAST:] = randn(LAST, cols)
    ids = torch.randint(vocab - LAST, vocab, (rows,), generator=torch.Generator().manual_seed(1))
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    coat.embedding(table, ids.to(DEV), out)
    assert torch.equal(out, table[ids.to(DEV)])
    dy = torch.randint(-8, 9, (rows, cols), generator=torch.Generator().manual_seed(2)).bfloat16()
    want = ref.lookup_bwd(dy, ids - (vocab - LAST), LAST, 1.0)[0]
    ws = torch.empty(coat.embedding_bwd_workspace(rows, vocab, cols), dtype=torch.uint8, device=DEV)
    for dw in (table.fill_(3.0), torch.full((vocab, cols), 3.0, device=DEV)):
        coat.embedding_bwd(dy.to(DEV), ids.to(DEV), dw, workspace=ws)
        assert torch.equal(dw[-LAST:].cpu().double(), want.to(dw.dtype).double())
        assert not dw[:-LAST].any()


def test_far_rows():
    """4.9 GB of looked-up rows, and their gradient."""
    coat = lib()
    vocab, cols, rows = 50, 4096, 600_000
    table = randn(vocab, cols)
    ids = torch.full((rows,), -1, dtype=torch.int64)
    ids[-LAST:] = torch.randint(0, vocab, (LAST,), generator=torch.Generator().manual_seed(1))
    out = torch.full((rows, cols), 3.0, dtype=torch.bfloat16, device=DEV)
    coat.embedding(table, ids.to(DEV), out)
    assert torch.equal(out[-LAST:], table[ids[-LAST:].to(DEV)]) and not out[:-LAST].any()
    out[-LAST:] = torch.randint(-8, 9, (LAST, cols), generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    out[:-LAST] = float("nan")
    dw = torch.empty(vocab, cols, device=DEV)
    ws = torch.empty(coat.embedding_bwd_workspace(rows, vocab, cols), dtype=torch.uint8, device=DEV)
    coat.embedding_bwd(out, ids.to(DEV), dw, workspace=ws)
    assert torch.equal(dw.cpu().double(), ref.lookup_bwd(out[-LAST:].cpu(), ids[-LAST:], vocab, 1.0)[0])


def test_far_hidden_states():
    """4.5 GB of hidden states, which the forward pass takes in two runs of rows."""
    coat = lib()
    rows, vocab, cols = 275_000, 200, 8192
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-LAST:] = randn(LAST, cols)
    w = randn(vocab, cols, seed=1, scale=cols ** -0.5)
    targets = torch.full((rows,), -100, dtype=torch.int64)
    targets[-LAST:] = torch.randint(0, vocab, (LAST,), generator=torch.Generator().manual_seed(1))
    targets[7] = 11
    loss, lse = torch.full((rows,), 3.0, device=DEV), torch.full((rows,), 3.0, device=DEV)
    ws = torch.empty(coat.cross_entropy_workspace(rows, vocab, cols), dtype=torch.uint8, device=DEV)
    coat.cross_entropy(x, w, targets.to(DEV), loss, lse, workspace=ws)
    pick = torch.cat((torch.tensor([7]), torch.arange(rows - LAST, rows)))
    r = ref.Entropy(x[pick.to(DEV)].cpu().double(), w.cpu().double(), targets[pick])
    got = loss.cpu().double()
    assert_between(got[pick], r.loss - r.loss_err, r.loss + r.loss_err, "loss")
    got[pick] = 0
    assert not got.any()
    d = torch.rand(rows, device=DEV)
    dx, dw = torch.full_like(x, 3.0), torch.empty_like(w)
    ws = torch.empty(coat.cross_entropy_bwd_workspace(rows, vocab, cols, piece=1), dtype=torch.uint8, device=DEV)
    coat.cross_entropy_bwd(d, x, w, targets.to(DEV), lse, dx, dw, workspace=ws)
    want_dx, want_dw, dx_err, dw_err = r.gradients(d[pick.to(DEV)].cpu(), lse[pick.to(DEV)].cpu())
    assert_close(dw.cpu(), want_dw, dw_err, "dw")
    assert_close(dx[pick.to(DEV)].cpu(), want_dx, dx_err, "dx")
    assert not dx[8:-LAST].any()


def test_far_weights():
    """4.9 GB of weights."""
    coat = lib()
    rows, vocab, cols = 70, 300_000, 8192
    x, w = randn(rows, cols), randn(vocab, cols, seed=1, scale=cols ** -0.5)
    targets = torch.randint(vocab - LAST, vocab, (rows,), generator=torch.Generator().manual_seed(1))
    loss, lse = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    ws = torch.empty(coat.cross_entropy_workspace(rows, vocab, cols), dtype=torch.uint8, device=DEV)
    coat.cross_entropy(x, w, targets.to(DEV), loss, lse, workspace=ws)
    logits = torch.cat([x.double() @ w[v:v + 50_000].double().t() for v in range(0, vocab, 50_000)], 1)
    exact = torch.logsumexp(logits, 1)
    mine = logits.gather(1, targets.to(DEV)[:, None])[:, 0]
    # as vocabulary_ref.Entropy, whose sums of magnitudes are below cols here (unit rows, products of size 1/sqrt(cols))
    size = (x.double().abs() @ w[-LAST:].double().abs().t()).amax() * 2
    slack = float(2 * (cols / 16 + 64) * 2 * F * size + (64 + vocab / 1024 + 8) * 2 * F + 60 * F * 24)
    assert (lse.double() - exact).abs().max() <= slack and (loss.double() - (exact - mine)).abs().max() <= slack
    d = torch.rand(rows, device=DEV)
    dx, dw = torch.empty_like(x), torch.full_like(w, 3.0)
    ws = torch.empty(coat.cross_entropy_bwd_workspace(rows, vocab, cols, piece=65536), dtype=torch.uint8, device=DEV)
    coat.cross_entropy_bwd(d, x, w, targets.to(DEV), lse, dx, dw, workspace=ws)
    # the last rows of dw, and some from the middle
    for v in (0, vocab // 2, vocab - LAST):
        g = d.double()[:, None] * torch.exp(logits[:, v:v + LAST] - lse.double()[:, None])
        hot = torch.zeros_like(g)
        here = (targets >= v) & (targets < v + LAST)
        hot[here.to(DEV), (targets[here] - v).to(DEV)] = 1.0
        g = g - d.double()[:, None] * hot
        want = g.t() @ x.double()
        room = (BF16 + slack) * (1 + BF16) * (g.abs().t() @ x.double().abs()) + slack * (d.double() @ x.double().abs())
        assert_close(dw[v:v + LAST].cpu(), want.cpu(), room.cpu(), "dw")


@pytest.mark.parametrize("rows,vocab,cols,kind", [(5, 300, 128, "bf16"), (65, 513, 256, "fp8"), (300, 1000, 64, "bf16"),
                                                  (700, 3001, 128, "fp8"), (2100, 4500, 192, "bf16")])
def test_nothing_else_is_written(rows, vocab, cols, kind):
    """Outputs and workspaces that end where the call's sizes end, with guards on both sides."""
    coat = lib()
    guards = []

    def inside(*shape, dtype):
        n = 1
        for s in shape:
            n *= s
        whole = torch.full((n + 512,), 77, dtype=dtype, device=DEV)
        guards.append((whole, n))
        return whole[256:256 + n].view(*shape)

    fp8 = kind == "fp8"
    x, w = randn(rows, cols), randn(vocab, cols, seed=1, scale=cols ** -0.5)
    scales = dict(x_scale=2.0 ** -5, weight_scale=2.0 ** -9) if fp8 else {}
    if fp8:
        x, w = ((t.float() / s).to(torch.float8_e4m3fn).view(torch.uint8) for t, s in zip((x, w), scales.values()))
    targets = ref.tokens(rows, vocab, torch.Generator().manual_seed(2), rows // 5).to(DEV)
    loss, lse = inside(rows, dtype=torch.float32), inside(rows, dtype=torch.float32)
    ws = inside(coat.cross_entropy_workspace(rows, vocab, cols), dtype=torch.uint8)
    coat.cross_entropy(x, w, targets, loss, lse, workspace=ws, **scales)
    d = torch.rand(rows, device=DEV)
    for dtype in (torch.bfloat16, torch.float32):
        for piece in (1, 600, vocab):
            dx, dw = inside(rows, cols, dtype=torch.bfloat16), inside(vocab, cols, dtype=dtype)
            ws = inside(coat.cross_entropy_bwd_workspace(rows, vocab, cols, piece=piece, codes=fp8,
                                                         f32=dtype == torch.float32), dtype=torch.uint8)
            coat.cross_entropy_bwd(d, x, w, targets, lse, dx, dw, workspace=ws, **scales)
    out = inside(rows, cols, dtype=torch.bfloat16)
    coat.embedding(w, targets, out)
    for dtype in (torch.bfloat16, torch.float32):
        dw = inside(vocab, cols, dtype=dtype)
        coat.embedding_bwd(out, targets, dw,
                           workspace=inside(coat.embedding_bwd_workspace(rows, vocab, cols), dtype=torch.uint8))
    torch.cuda.synchronize()
    for whole, n in guards:
        assert bool((whole[:256] == 77).all()) and bool((whole[256 + n:] == 77).all())


def test_two_streams():
    """Calls at once on two streams, with outputs and workspaces of their own, as one after the other."""
    coat = lib()
    rows, vocab, cols = 600, 2000, 256
    w = randn(vocab, cols, seed=1, scale=cols ** -0.5)
    jobs = []
    for seed in (1, 2):
        jobs.append(dict(x=randn(rows, cols, seed=seed), targets=ref.tokens(rows, vocab, torch.Generator().manual_seed(seed), 9).to(DEV),
                         d=torch.rand(rows, device=DEV), loss=torch.empty(rows, device=DEV), lse=torch.empty(rows, device=DEV),
                         dx=torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV), dw=torch.empty(vocab, cols, device=DEV),
                         ws=torch.empty(coat.cross_entropy_bwd_workspace(rows, vocab, cols, f32=True)
                                        + coat.embedding_bwd_workspace(rows, vocab, cols), dtype=torch.uint8, device=DEV),
                         stream=torch.cuda.Stream()))

    def run(j, stream):
        coat.cross_entropy(j["x"], w, j["targets"], j["loss"], j["lse"], workspace=j["ws"], stream=stream)
        coat.cross_entropy_bwd(j["d"], j["x"], w, j["targets"], j["lse"], j["dx"], j["dw"], workspace=j["ws"], stream=stream)
        coat.embedding_bwd(j["dx"], j["targets"], j["dw"], workspace=j["ws"], accumulate=True, stream=stream)

    want = []
    for j in jobs:
        run(j, None)
        want.append([j[k].clone() for k in ("loss", "lse", "dx", "dw")])
    torch.cuda.synchronize()
    for _ in range(5):
        for j in jobs:
            run(j, j["stream"])
    torch.cuda.synchronize()
    for j, ws in zip(jobs, want):
        assert all(torch.equal(j[k], t) for k, t in zip(("loss", "lse", "dx", "dw"), ws))


def test_far_weights_dx():
    """dx from 4.9 GB of weights, whose last rows lie past 4 GiB, in one piece and in five."""
    coat = lib()
    rows, vocab, cols = 70, 300_000, 8192
    x, w = randn(rows, cols), randn(vocab, cols, seed=1, scale=cols ** -0.5)
    targets = torch.randint(vocab - LAST, vocab, (rows,), generator=torch.Generator().manual_seed(1))
    pieces = [slice(v, v + 25_000) for v in range(0, vocab, 25_000)]
    logits = torch.cat([x.double() @ w[p].double().t() for p in pieces], 1)
    lse = torch.logsumexp(logits, 1)
    d = torch.rand(rows, device=DEV) - 0.5
    # as vocabulary_ref.Entropy has it, with the lse that the call is given
    size = (x.double().abs() @ w[-LAST:].double().abs().t()).amax() * 2
    l_err = float((cols / 16 + 64) * 2 * F * size)
    given = lse.float()
    g = torch.exp(logits - given.double()[:, None])
    rel = l_err + 6 * F * (logits.abs() + given.double().abs()[:, None]) + 8 * F
    err = d.double().abs()[:, None] * g * (1.01 * rel)
    hot = torch.arange(rows, device=DEV), targets.to(DEV)
    g[hot] -= 1.0
    g *= d.double()[:, None]
    err[hot] += 8 * F * d.double().abs()
    want = torch.zeros(rows, cols, dtype=torch.float64, device=DEV)
    room = torch.zeros_like(want)
    for p in pieces:
        wide = w[p].double()
        want += g[:, p] @ wide
        room += (err[:, p] + BF16 * (g[:, p].abs() + err[:, p]) + (vocab / 16 + 128 + 5) * 2 * F * g[:, p].abs()) @ wide.abs()
        del wide
    for piece in (65536, vocab):
        dx = torch.full_like(x, 3.0)
        ws = torch.empty(coat.cross_entropy_bwd_workspace(rows, vocab, cols, piece=piece), dtype=torch.uint8, device=DEV)
        coat.cross_entropy_bwd(d, x, w, targets.to(DEV), given, dx, None, workspace=ws)
        assert_close(dx.cpu(), want.cpu(), room.cpu(), "dx")
