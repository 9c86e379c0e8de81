"""GPU: embedding lookup and its gradient, exactly on small integers and
within bounds on random data, with padding, long runs of a token, odd sizes
and captured graphs."""
import pytest
import torch

import vocabulary_ref as ref
from activation_ref import BF16, F, assert_close, code_values
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("rows,vocab,cols,padding", [
    (1, 1, 16, 0), (1, 32000, 4096, 0), (3, 7, 48, 1), (64, 300, 128, 6), (257, 1000, 1040, 20), (1000, 33, 208, 0),
    (5, 4, 16, 5), (2049, 500, 8208, 100)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_lookup(rows, vocab, cols, padding, kind):
    coat = lib()
    g = torch.Generator().manual_seed(rows + cols)
    ids = ref.tokens(rows, vocab, g, padding)
    if kind == "bf16":
        table, table_scale = torch.randn(vocab, cols, generator=g).bfloat16(), 1.0
    else:
        table = torch.randint(0, 256, (vocab, cols), generator=g, dtype=torch.uint8)
        table[(table & 127) == 127] = 5   # no NaN codes
        table_scale = 0.037
    for scale in (1.0, 45.3):
        out = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=DEV)
        coat.embedding(table.to(DEV), ids.to(DEV), out, table_scale=table_scale, scale=scale)
        want = ref.lookup(ref.values(table, 1.0), ids, float(torch.tensor(table_scale)) * float(torch.tensor(scale)))
        # the scales and their product, and the multiplication, in FP32
        assert_close(out.cpu(), want, 4 * F * want.abs(), "out")


def test_lookup_keeps_bits():
    """A BF16 table under scale 1 is copied; NaN and infinity reach their rows alone; padding reads nothing."""
    coat = lib()
    table = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(64, 1024)
    ids = torch.arange(64).flip(0)
    out = torch.empty(64, 1024, dtype=torch.bfloat16, device=DEV)
    coat.embedding(table.to(DEV), ids.to(DEV), out)
    got, want = out.cpu(), table[ids]
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~torch.isnan(got)].view(torch.int16), want[~torch.isnan(want)].view(torch.int16))
    bad = torch.full((4, 32), float("nan"), dtype=torch.bfloat16, device=DEV)
    out = torch.empty(3, 32, dtype=torch.bfloat16, device=DEV)
    coat.embedding(bad, torch.tensor([-1, 4, 1 << 50], device=DEV), out)
    assert torch.equal(out.cpu(), torch.zeros(3, 32, dtype=torch.bfloat16))


def run_bwd(dy, ids, vocab, dtype, scale=1.0, base=None):
    coat = lib()
    rows, cols = dy.shape
    dw = torch.full((vocab, cols), 5.0, dtype=dtype, device=DEV) if base is None else base.to(DEV).clone()
    ws = torch.full((coat.embedding_bwd_workspace(rows, vocab, cols),), 255, dtype=torch.uint8, device=DEV)
    coat.embedding_bwd(dy.to(DEV), ids.to(DEV), dw, scale=scale, workspace=ws, accumulate=base is not None)
    torch.cuda.synchronize()
    return dw.cpu()


# rows around the 32-row parts, the 64-row blocks and the 16384-row runs of the sort
BWD = [(1, 1, 16, 0), (1, 5000, 4096, 0), (31, 3, 48, 2), (32, 2, 16, 0), (33, 1, 128, 0), (64, 64, 256, 3),
       (65, 9, 2064, 0), (100, 1, 16, 7), (500, 3, 4096, 50), (1024, 100000, 32, 10), (1000, 4, 4112, 0), (4, 7, 64, 4),
       (4096, 30, 128, 400), (16384, 3000, 64, 100), (16385, 50, 32, 5), (40001, 2, 16, 1000), (70000, 5000, 48, 0)]


@pytest.mark.parametrize("rows,vocab,cols,padding", BWD)
def test_gradient_exact(rows, vocab, cols, padding):
    """Small integers: every sum is exact."""
    g = torch.Generator().manual_seed(rows * 7 + vocab)
    ids = ref.tokens(rows, vocab, g, padding)
    dy = torch.randint(-8, 9, (rows, cols), generator=g).bfloat16()
    dy[~ref.live_rows(ids, vocab)] = float("nan")   # padding reaches nothing
    want = ref.lookup_bwd(dy, ids, vocab, 0.5)[0]
    assert torch.equal(run_bwd(dy, ids, vocab, torch.float32, 0.5).double(), want)
    assert torch.equal(run_bwd(dy, ids, vocab, torch.bfloat16, 0.5), want.float().bfloat16())
    base = torch.randint(-100, 100, (vocab, cols), generator=g).float()
    base[vocab // 2] = float("inf")
    got = run_bwd(dy, ids, vocab, torch.float32, 0.5, base=base)
    assert torch.equal(got.double(), base.double() + want)


@pytest.mark.parametrize("rows,vocab,cols", [(700, 40, 512), (5000, 900, 4096), (20000, 12, 256)])
def test_gradient_random(rows, vocab, cols):
    g = torch.Generator().manual_seed(rows)
    ids = ref.tokens(rows, vocab, g, rows // 10)
    dy = torch.randn(rows, cols, generator=g).bfloat16()
    dw, size, count = ref.lookup_bwd(dy, ids, vocab, 45.25)
    slack = (count + 2) * F * size
    assert_close(run_bwd(dy, ids, vocab, torch.float32, 45.25), dw, slack, "dw", rounding=F)
    first = run_bwd(dy, ids, vocab, torch.bfloat16, 45.25)
    assert_close(first, dw, slack, "dw", rounding=BF16)
    for _ in range(3):   # the order of the sums is fixed
        assert torch.equal(run_bwd(dy, ids, vocab, torch.bfloat16, 45.25), first)


def test_gradient_is_the_lookups():
    """<dy, d lookup> = <dw, d table>: against differences of the lookup along random directions."""
    coat = lib()
    g = torch.Generator().manual_seed(3)
    ids = ref.tokens(300, 50, g, 11)
    dy = torch.randn(300, 64, generator=g).bfloat16()
    dw = run_bwd(dy, ids, 50, torch.float32, 2.0).double()
    table = torch.randint(-64, 65, (50, 64), generator=g).float()
    step = torch.randint(-64, 65, (50, 64), generator=g).float()   # exact in BF16, as are the sums
    out = []
    for t in (table + step, table - step):
        o = torch.empty(300, 64, dtype=torch.bfloat16, device=DEV)
        coat.embedding(t.bfloat16().to(DEV), ids.to(DEV), o, scale=2.0)
        out.append(o.cpu().double())
    slope = ((out[0] - out[1]) / 2 * dy.double()).sum()
    _, size, count = ref.lookup_bwd(dy, ids, 50, 2.0)
    assert abs(slope - (dw * step.double()).sum()) <= ((count + 2) * F * size * step.abs().double()).sum()


def test_no_rows():
    dy, ids = torch.empty(0, 64, dtype=torch.bfloat16), torch.empty(0, dtype=torch.int64)
    assert torch.equal(run_bwd(dy, ids, 9, torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16))
    base = torch.ones(9, 64)
    assert torch.equal(run_bwd(dy, ids, 9, torch.float32, base=base), base)


def test_captured_and_on_a_stream():
    """A graph of lookup and gradient, replayed with new tokens between eager calls of the same buffers."""
    coat = lib()
    rows, vocab, cols = 900, 70, 256
    g = torch.Generator().manual_seed(8)
    table = torch.randn(vocab, cols, generator=g).bfloat16().to(DEV)
    dy = torch.randint(-8, 9, (rows, cols), generator=g).bfloat16()
    ids, d_dy = torch.zeros(rows, dtype=torch.int64, device=DEV), dy.to(DEV)
    out = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty(vocab, cols, dtype=torch.float32, device=DEV)
    ws = torch.empty(coat.embedding_bwd_workspace(rows, vocab, cols), dtype=torch.uint8, device=DEV)

    def both():
        coat.embedding(table, ids, out)
        coat.embedding_bwd(d_dy, ids, dw, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for seed in range(5):
        new = ref.tokens(rows, vocab, torch.Generator().manual_seed(seed), 10 * seed)
        ids.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        replayed = (out.cpu(), dw.cpu())
        assert torch.equal(replayed[0].double(), ref.lookup(table.cpu().double(), new, 1.0))
        assert torch.equal(replayed[1].double(), ref.lookup_bwd(dy, new, vocab, 1.0)[0])
        out.zero_(), dw.fill_(3.0), ws.fill_(255)
        both()
        assert torch.equal(out.cpu(), replayed[0]) and torch.equal(dw.cpu(), replayed[1])
