"""GPU: the norm and rotation of query and key heads with their checkpoint,
and the gradient from it, against the formulas in 64 bits."""
import pytest
import torch

import activation_ref as ref
from activation_ref import F
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu
EPS = 1e-5
TABLE = 300

# tokens, query heads, key heads, head_dim, rot_dim, G
SHAPES = [(1, 1, 1, 128, 128, 128), (1, 32, 8, 128, 128, 64), (3, 5, 1, 64, 64, 64), (2, 3, 3, 16, 16, 16),
          (17, 8, 2, 96, 96, 32), (5, 7, 1, 80, 80, 16), (9, 4, 4, 256, 256, 128), (6, 4, 2, 256, 64, 32),
          (11, 6, 6, 128, 32, 16), (4, 2, 2, 96, 48, 16), (7, 3, 0, 128, 128, 128), (7, 0, 3, 64, 32, 32),
          (1200, 32, 32, 128, 128, 128), (4500, 3, 1, 64, 64, 16), (2500, 9, 3, 256, 256, 64), (3, 2, 2, 48, 16, 16)]


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def data(t, hq, hk, d, rot, seed, padding=True):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(t, (hq + 2 * hk) * d, generator=g) * torch.exp(torch.randn((hq + 2 * hk) * d, generator=g))).bfloat16()
    wq, wk = [(1 + 0.3 * torch.randn(d, generator=g)).bfloat16() for _ in range(2)]
    freq = 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    angle = torch.arange(TABLE).double()[:, None] * freq
    pos = torch.randint(0, TABLE, (t,), generator=g)
    pos[0] = TABLE - 1
    if padding and t > 3:
        pos[t // 2], pos[-1], pos[-2] = -1, TABLE, 2 ** 40
    return qkv, wq, wk, angle.cos().float(), angle.sin().float(), pos


def split(qkv, hq, hk, d):
    """Query and key heads as parts of the packed rows."""
    return qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))


def outputs(t, hq, hk, d, G):
    return dict(q_out=torch.full((t, hq, d), 7.0, dtype=torch.bfloat16, device=DEV),
                k_out=torch.full((t, hk, d), 7.0, dtype=torch.bfloat16, device=DEV),
                codes=torch.full((t, hq + hk, d), 0x55, dtype=torch.uint8, device=DEV),
                scales=torch.full((t, hq + hk, d // G), -1.0, device=DEV),
                rstd=torch.full((t, hq + hk), -1.0, device=DEV))


def weights_of(wq, wk, hq, hk):
    return torch.cat((wq.double().expand(hq, -1), wk.double().expand(hk, -1)))


# squares of 8 values, 5 lane steps, mean, eps, root and quotient
RSTD = (8 + 5 + 4) * F


@pytest.mark.parametrize("t,hq,hk,d,rot,G", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_forward(t, hq, hk, d, rot, G, interleaved):
    coat = lib()
    qkv, wq, wk, cos, sin, pos = data(t, hq, hk, d, rot, t + d + rot)
    q, k = split(qkv.to(DEV), hq, hk, d)
    o = outputs(t, hq, hk, d, G)
    args = (wq.to(DEV), wk.to(DEV), EPS, cos.to(DEV), sin.to(DEV), pos.to(DEV))
    coat.qk_norm_rope(q, k, *args, interleaved=interleaved, group_size=G, **o)
    torch.cuda.synchronize()
    live = ((pos >= 0) & (pos < TABLE))[:, None, None]
    x = torch.cat(split(qkv, hq, hk, d), 1)
    x = torch.where(live, x, torch.zeros_like(x))
    y, rstd = ref.norm(x, weights_of(wq, wk, hq, hk), EPS)
    rstd = rstd * live.squeeze(2)
    want = ref.rotate(y, cos, sin, pos, interleaved)
    size = ref.rotate(y.abs(), cos.abs(), -sin.abs(), pos, interleaved)   # |a c| + |b s|, or no less than it
    size = torch.maximum(size, ref.rotate(y.abs(), cos.abs(), sin.abs(), pos, interleaved))
    got = torch.cat((o["q_out"], o["k_out"]), 1).cpu()
    ref.assert_close(got, want, (RSTD + 5 * F) * size, "rotated heads")
    ref.assert_close(o["rstd"].cpu(), rstd, RSTD * rstd, "rstd", F)
    codes, scales = ref.quantize(x, G)
    assert torch.equal(ref.code_values(o["codes"].cpu()), ref.code_values(codes))
    assert torch.equal(o["scales"].cpu(), scales)
    # without a checkpoint, in place in the packed rows: the values beside them stay
    packed = qkv.to(DEV)
    q, k = split(packed, hq, hk, d)
    coat.qk_norm_rope(q, k, *args, q, k, interleaved=interleaved, group_size=G)
    torch.cuda.synchronize()
    assert torch.equal(q, o["q_out"]) and torch.equal(k, o["k_out"])
    assert torch.equal(packed[:, (hq + hk) * d:].cpu(), qkv[:, (hq + hk) * d:])


@pytest.mark.parametrize("t,hq,hk,d,rot,G", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_backward(t, hq, hk, d, rot, G, interleaved):
    coat = lib()
    qkv, wq, wk, cos, sin, pos = data(t, hq, hk, d, rot, 2 * t + d + rot)
    g = torch.Generator().manual_seed(t)
    dy = (1e-3 * torch.randn(t, hq + hk, d, generator=g)).bfloat16()
    live = ((pos >= 0) & (pos < TABLE))[:, None, None]
    x = torch.cat(split(qkv, hq, hk, d), 1)
    codes, scales = ref.quantize(x, G)
    rstd = ref.norm(x, wq, EPS)[1].float()
    dead = ~live.squeeze()
    if t > 1:   # whatever the buffers of padding hold
        scales[dead], rstd[dead], dy[dead] = float("nan"), float("inf"), float("nan")
    dqkv = torch.full((t, (hq + 2 * hk) * d), 3.0, dtype=torch.bfloat16, device=DEV)
    dq, dk = split(dqkv, hq, hk, d)
    dwq, dwk = torch.full((d,), 3.0, device=DEV), torch.full((d,), 3.0, device=DEV)
    ws = torch.full((coat.qk_norm_rope_bwd_workspace(t, hq + hk, d) // 4,), float("nan"), device=DEV)
    args = [v.to(DEV) for v in (codes, scales, rstd, wq, wk, cos, sin, pos)]
    dyd = dy.to(DEV)
    dq_out, dk_out = dyd[:, :hq], dyd[:, hq:]
    coat.qk_norm_rope_bwd(dq_out, dk_out, *args, dq, dk, dwq, dwk, workspace=ws, interleaved=interleaved,
                          group_size=G)
    torch.cuda.synchronize()
    dy, scales, rstd = [torch.where(live.reshape(-1, *[1] * (v.dim() - 1)), v, torch.zeros_like(v))
                        for v in (dy, scales, rstd)]
    turned = ref.rotate(dy.double(), cos, sin, pos, interleaved, -1.0)
    size_t = torch.maximum(ref.rotate(dy.double().abs(), cos.abs(), -sin.abs(), pos, interleaved),
                           ref.rotate(dy.double().abs(), cos.abs(), sin.abs(), pos, interleaved))
    n = ref.restore(codes, scales, G) * rstd.double().unsqueeze(2)
    w = weights_of(wq, wk, hq, hk)
    want, terms, _ = ref.norm_bwd(n, rstd, turned, w)
    _, sizes, size = ref.norm_bwd(n.abs(), rstd, size_t, w.abs())
    # rotation 3, n 2, dn 1, the sum 8 + 5, dx 4
    ref.assert_close(torch.cat((dq, dk), 1).cpu(), want, 24 * F * size, "dx")
    # a wave's units of up to 4 sets, one block in 1024; 32 rows of a block, 16 partial sums, 6 joins, 6 roundings
    units = -(-t * (hq + hk) // 4096) * 4 + 4
    slack = (units + 32 + 16 + 6 + 6) * F
    ref.assert_close(dwq.cpu(), terms[:, :hq].sum((0, 1)), slack * sizes[:, :hq].abs().sum((0, 1)), "dq_weight", F)
    ref.assert_close(dwk.cpu(), terms[:, hq:].sum((0, 1)), slack * sizes[:, hq:].abs().sum((0, 1)), "dk_weight", F)
    assert torch.equal(dqkv[:, (hq + hk) * d:].cpu(), torch.full((t, hk * d), 3.0).bfloat16())
    # in place, accumulating, and the same sums again
    base = dwq.clone(), dwk.clone()
    coat.qk_norm_rope_bwd(dq_out, dk_out, *args, dq_out, dk_out, dwq, dwk, workspace=ws, accumulate=True,
                          interleaved=interleaved, group_size=G)
    torch.cuda.synchronize()
    assert torch.equal(dq_out, dq) and torch.equal(dk_out, dk)
    assert torch.equal(dwq, 2 * base[0]) and torch.equal(dwk, 2 * base[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    """Heads that E4M3 holds exactly, so the checkpoint loses nothing."""
    coat = lib()
    t, hq, hk, d, rot, G, h = 2, 2, 1, 32, 16, 16, 1e-5
    _, wq, wk, cos, sin, pos = data(t, hq, hk, d, rot, 5)
    g = torch.Generator().manual_seed(6)
    x = torch.randint(-14, 15, (t, hq + hk, d), generator=g).double() / 8
    x[..., ::G] = 1.75
    dy = torch.randn(t, hq + hk, d, generator=g).bfloat16()
    o = outputs(t, hq, hk, d, G)
    xd, dyd = x.bfloat16().to(DEV), dy.to(DEV)
    tables = [v.to(DEV) for v in (cos, sin, pos)]
    coat.qk_norm_rope(xd[:, :hq], xd[:, hq:], wq.to(DEV), wk.to(DEV), EPS, *tables, interleaved=interleaved,
                      group_size=G, **o)
    assert torch.equal(ref.restore(o["codes"].cpu(), o["scales"].cpu(), G), x)
    dx = torch.empty_like(dyd)
    dw = torch.empty(2, d, device=DEV)
    ws = torch.empty(coat.qk_norm_rope_bwd_workspace(t, hq + hk, d), dtype=torch.uint8, device=DEV)
    coat.qk_norm_rope_bwd(dyd[:, :hq], dyd[:, hq:], o["codes"], o["scales"], o["rstd"], wq.to(DEV), wk.to(DEV),
                          *tables, dx[:, :hq], dx[:, hq:], dw[0], dw[1], workspace=ws, interleaved=interleaved,
                          group_size=G)
    w0 = torch.stack((wq.double(), wk.double()))

    def loss(x, w):
        y, _ = ref.norm(x, weights_of(w[0], w[1], hq, hk), EPS)
        return (ref.rotate(y, cos, sin, pos, interleaved) * dy.double()).sum()

    def slope(f, at):
        out = torch.empty(at.numel(), dtype=torch.float64)
        for i in range(at.numel()):
            e = torch.zeros(at.numel(), dtype=torch.float64)
            e[i] = h
            out[i] = (f(at + e.view(at.shape)) - f(at - e.view(at.shape))) / (2 * h)
        return out.view(at.shape)

    want = slope(lambda v: loss(v, w0), x)
    # the difference: h^2 / 6 of a third derivative of about 10, and 2^-53 * |loss| / h
    ref.assert_close(dx.cpu(), want, torch.full_like(want, 1e-8) + 60 * F, "dx")
    want = slope(lambda v: loss(x, v), w0)
    ref.assert_close(dw.cpu(), want, torch.full_like(want, 1e-8) + 60 * F, "dw", F)


def test_empty_table_is_all_padding():
    coat = lib()
    t, hq, hk, d = 5, 2, 1, 64
    qkv, wq, wk, cos, sin, _ = data(t, hq, hk, d, d, 3)
    q, k = split(qkv.to(DEV), hq, hk, d)
    o = outputs(t, hq, hk, d, 64)
    none = torch.empty(0, d // 2, device=DEV)
    coat.qk_norm_rope(q, k, wq.to(DEV), wk.to(DEV), EPS, none, none, torch.zeros(t, dtype=torch.int64, device=DEV),
                      group_size=64, **o)
    for v in o.values():
        assert (v == 0).all()


def test_not_finite_stays_in_its_head():
    coat = lib()
    t, hq, hk, d = 6, 4, 2, 128
    qkv, wq, wk, cos, sin, pos = data(t, hq, hk, d, d, 4, padding=False)
    tables = [v.to(DEV) for v in (cos, sin, pos)]

    def go(v):
        q, k = split(v.to(DEV), hq, hk, d)
        o = outputs(t, hq, hk, d, 128)
        coat.qk_norm_rope(q, k, wq.to(DEV), wk.to(DEV), EPS, *tables, **o)
        return {n: x.cpu() for n, x in o.items()}

    clean = go(qkv)
    bad = qkv.clone()
    bad[2, d + 3] = float("nan")   # query head 1 of token 2
    o = go(bad)
    assert o["q_out"][2, 1].isnan().all() and o["scales"][2, 1].isnan().all()
    for n in o:
        keep = torch.ones(o[n].shape[:2], dtype=torch.bool)
        if n != "k_out":
            keep[2, 1] = False
        assert torch.equal(o[n][keep], clean[n][keep]), n


def test_graph_and_stream():
    coat = lib()
    t, hq, hk, d, G = 900, 8, 2, 128, 32
    qkv, wq, wk, cos, sin, pos = [v.to(DEV) for v in data(t, hq, hk, d, d, 9)]
    q, k = split(qkv, hq, hk, d)

    def mk():
        o = outputs(t, hq, hk, d, G)
        o.update(dq=torch.zeros_like(o["q_out"]), dk=torch.zeros_like(o["k_out"]), dwq=torch.zeros(d, device=DEV),
                 dwk=torch.zeros(d, device=DEV),
                 ws=torch.zeros(coat.qk_norm_rope_bwd_workspace(t, hq + hk, d), dtype=torch.uint8, device=DEV))
        return o

    def go(o, stream=None):
        coat.qk_norm_rope(q, k, wq, wk, EPS, cos, sin, pos, o["q_out"], o["k_out"], codes=o["codes"],
                          scales=o["scales"], rstd=o["rstd"], group_size=G, stream=stream)
        coat.qk_norm_rope_bwd(o["q_out"], o["k_out"], o["codes"], o["scales"], o["rstd"], wq, wk, cos, sin, pos,
                              o["dq"], o["dk"], o["dwq"], o["dwk"], workspace=o["ws"], group_size=G, stream=stream)

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
        for n in ("dq", "dk", "dwq", "codes"):
            captured[n].zero_()
        go(other)
        graph.replay()
        torch.cuda.synchronize()
        for n in eager:
            if n != "ws":
                assert torch.equal(captured[n], eager[n]) and torch.equal(other[n], eager[n]), n
