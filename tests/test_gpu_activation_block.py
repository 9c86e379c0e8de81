"""GPU: the activation operators and the FP8 linear layers together, as a
training step of a transformer block uses them: residual norm, 8-bit
projection, gated activation, 8-bit projection back; and norm, projection,
query/key norm and rotation; forward, backward, and captured in a graph.

Every operator reads what the one before it wrote, and is checked against its
formula in 64 bits on those values (the linear layers have tests of their
own)."""
import pytest
import torch

import activation_ref as ref
from activation_ref import BF16, F
from gpu_util import DEV, lib, require_gpu

pytestmark = pytest.mark.gpu

TOKENS, D, FFN, G, EPS = 200, 256, 384, 64, 1e-5
HEADS, KV, HEAD = 4, 2, 64
S_Y, S_H = 2.0 ** -5, 2.0 ** -4
# roundings behind a result: a norm's sum and root; exp of |g| < 89; a sum over TOKENS, steps of 2^-23
NORM, ACT, SUM = 40 * F, 145 * F, 2 * (TOKENS + 4) * F


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def empty(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device=DEV)


def u8(*shape):
    return empty(*shape, dtype=torch.uint8)


def f32(*shape):
    return empty(*shape, dtype=torch.float32)


class Block:
    """Weights, activations, checkpoints and gradients of one block."""

    def __init__(self):
        g = torch.Generator().manual_seed(3)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x, self.res = [r(TOKENS, D).bfloat16().to(DEV) for _ in range(2)]
        self.norm_w = (1 + 0.2 * r(D)).bfloat16().to(DEV)
        code = lambda *s: (r(*s) * 2).to(torch.float8_e4m3fn).view(torch.uint8).to(DEV)  # noqa: E731
        self.w_gate_up, self.w_down, self.w_qkv = code(2 * FFN, D), code(D, FFN), code((HEADS + 2 * KV) * HEAD, D)
        self.w_scale = 0.02
        self.qw, self.kw = [(1 + 0.2 * r(HEAD)).bfloat16().to(DEV) for _ in range(2)]
        pos = torch.arange(TOKENS) % 77
        pos[-9:] = -1
        angle = torch.arange(77).double()[:, None] * 10000.0 ** (-torch.arange(0, HEAD, 2).double() / HEAD)
        self.pos, self.cos, self.sin = pos.to(DEV), angle.cos().float().to(DEV), angle.sin().float().to(DEV)
        self.d_out, self.d_qk = [(1e-2 * r(TOKENS, n)).bfloat16().to(DEV) for n in (D, (HEADS + KV) * HEAD)]
        self.d_h, self.d_y = [(1e-2 * r(TOKENS, n)).bfloat16().to(DEV) for n in (FFN, D)]
        # written by the step
        self.sum, self.y_codes, self.amax, self.rstd = empty(TOKENS, D), u8(TOKENS, D), f32(1), f32(TOKENS)
        self.x_codes, self.x_scales = u8(TOKENS, D), f32(TOKENS, D // G)
        self.gu_codes, self.gu_scales = u8(TOKENS, 2 * FFN), f32(TOKENS, 2 * FFN // G)
        self.h_codes, self.h_amax, self.out = u8(TOKENS, FFN), f32(1), empty(TOKENS, D)
        self.qkv = empty(TOKENS, (HEADS + 2 * KV) * HEAD)
        self.q_rot, self.k_rot = empty(TOKENS, HEADS, HEAD), empty(TOKENS, KV, HEAD)
        self.qk_codes, self.qk_scales = u8(TOKENS, HEADS + KV, HEAD), f32(TOKENS, HEADS + KV, 1)
        self.qk_rstd = f32(TOKENS, HEADS + KV)
        self.dw_down, self.dw_gate_up = empty(D, FFN), f32(2 * FFN, D)
        self.d_gu, self.dx, self.d_norm_w = empty(TOKENS, 2 * FFN), empty(TOKENS, D), f32(D)
        self.d_qkv, self.dqw, self.dkw = empty(TOKENS, (HEADS + 2 * KV) * HEAD), f32(HEAD), f32(HEAD)
        self.dw_qkv = empty((HEADS + 2 * KV) * HEAD, D)
        coat = lib()
        need = max(coat.rms_norm_bwd_workspace(TOKENS, D), coat.weight_grad_workspace(TOKENS, 2 * FFN, D),
                   coat.weight_grad_workspace(TOKENS, D, FFN), coat.weight_grad_workspace(TOKENS, self.qkv.shape[1], D),
                   coat.qk_norm_rope_bwd_workspace(TOKENS, HEADS + KV, HEAD))
        self.ws = u8(need)   # one for all: the calls follow each other on one stream

    def heads(self, t):
        q, k = t[:, :HEADS * HEAD], t[:, HEADS * HEAD:(HEADS + KV) * HEAD]
        return q.unflatten(1, (HEADS, HEAD)), k.unflatten(1, (KV, HEAD))

    def step(self):
        c, s = lib(), self
        # forward
        c.rms_norm(s.x, s.norm_w, EPS, residual=s.res, residual_out=s.sum, y_codes=s.y_codes, y_scale=S_Y,
                   y_amax=s.amax, codes=s.x_codes, scales=s.x_scales, rstd=s.rstd, group_size=G)
        c.gemm_group_quant(s.y_codes, s.w_gate_up, S_Y, s.w_scale, s.gu_codes, s.gu_scales, group_size=G)
        c.swiglu(s.gu_codes, s.gu_scales, h_codes=s.h_codes, h_scale=S_H, h_amax=s.h_amax, group_size=G)
        c.gemm_bf16(s.h_codes, s.w_down, S_H, s.w_scale, s.out)
        c.gemm_bf16(s.y_codes, s.w_qkv, S_Y, s.w_scale, s.qkv)
        c.qk_norm_rope(*s.heads(s.qkv), s.qw, s.kw, EPS, s.cos, s.sin, s.pos, s.q_rot, s.k_rot, codes=s.qk_codes,
                       scales=s.qk_scales, rstd=s.qk_rstd, group_size=G)
        # backward, from the checkpoints alone
        c.weight_grad(s.d_out, s.h_codes, S_H, s.dw_down, workspace=s.ws)
        c.swiglu_bwd(s.d_h, s.gu_codes, s.gu_scales, s.d_gu, group_size=G)
        c.weight_grad(s.d_gu, s.y_codes, S_Y, s.dw_gate_up, workspace=s.ws)
        d_q, d_k = s.heads(s.d_qk)
        c.qk_norm_rope_bwd(d_q, d_k, s.qk_codes, s.qk_scales, s.qk_rstd, s.qw, s.kw, s.cos, s.sin, s.pos,
                           *s.heads(s.d_qkv), s.dqw, s.dkw, workspace=s.ws, group_size=G)
        c.weight_grad(s.d_qkv, s.y_codes, S_Y, s.dw_qkv, workspace=s.ws)
        c.rms_norm_bwd(s.d_y, s.x_codes, s.x_scales, s.rstd, s.norm_w, s.dx, s.d_norm_w, d_residual=s.d_out,
                       workspace=s.ws, group_size=G)

    def results(self):
        return {n: getattr(self, n) for n in
                ("sum", "y_codes", "amax", "rstd", "x_codes", "x_scales", "gu_codes", "gu_scales", "h_codes", "h_amax",
                 "out", "q_rot", "k_rot", "qk_codes", "qk_scales", "qk_rstd", "dw_down", "dw_gate_up", "d_gu", "dx",
                 "d_norm_w", "d_qkv", "dqw", "dkw", "dw_qkv")}


def test_block():
    b = Block()
    b.step()
    torch.cuda.synchronize()
    v = {n: getattr(b, n).cpu() for n in vars(b) if isinstance(getattr(b, n), torch.Tensor)}
    h = (v["x"].float() + v["res"].float()).bfloat16()
    assert torch.equal(v["sum"], h)
    y, rstd = ref.norm(h, v["norm_w"], EPS)
    ref.assert_codes(v["y_codes"], y / S_Y, NORM, "y")
    codes, scales = ref.quantize(h, G)
    assert torch.equal(ref.code_values(v["x_codes"]), ref.code_values(codes)) and torch.equal(v["x_scales"], scales)
    gate, up = ref.restore(v["gu_codes"], v["gu_scales"], G).chunk(2, 1)
    s, rest = ref.silu_parts(gate)
    ref.assert_codes(v["h_codes"], gate * s * up / S_H, ACT, "h")
    assert abs(float(v["h_amax"]) - (gate * s * up).abs().max()) <= ACT * (gate * s * up).abs().max()
    live = (v["pos"] >= 0)[:, None, None]
    x = torch.cat(b.heads(v["qkv"]), 1)
    x = torch.where(live, x, torch.zeros_like(x))
    w = torch.cat((v["qw"].double().expand(HEADS, -1), v["kw"].double().expand(KV, -1)))
    n, _ = ref.norm(x, w, EPS)
    size = ref.rotate(n.abs(), v["cos"].abs(), v["sin"].abs(), v["pos"], False)
    size = torch.maximum(size, ref.rotate(n.abs(), v["cos"].abs(), -v["sin"].abs(), v["pos"], False))
    ref.assert_close(torch.cat((v["q_rot"], v["k_rot"]), 1), ref.rotate(n, v["cos"], v["sin"], v["pos"], False),
                     NORM * size, "rotated")
    # backward
    hv = ref.code_values(v["h_codes"]) * S_H
    ref.assert_close(v["dw_down"], v["d_out"].double().t() @ hv, SUM * (v["d_out"].double().abs().t() @ hv.abs()), "dw_down")
    dh = v["d_h"].double()
    d_gate, d_up = v["d_gu"].chunk(2, 1)
    ref.assert_close(d_gate, dh * up * s * (1 + gate * rest), ACT * (dh * up * s).abs() * (1 + (gate * rest).abs()), "d_gate")
    ref.assert_close(d_up, dh * gate * s, ACT * (dh * gate * s).abs(), "d_up")
    yv = ref.code_values(v["y_codes"]) * S_Y
    for dw, d in (("dw_gate_up", "d_gu"), ("dw_qkv", "d_qkv")):
        ref.assert_close(v[dw], v[d].double().t() @ yv, SUM * (v[d].double().abs().t() @ yv.abs()), dw,
                         F if v[dw].dtype == torch.float32 else BF16)
    assert (v["d_qkv"][-9:] == 0).all() and (v["d_qkv"][:, (HEADS + KV) * HEAD:] == 0).all()
    dy = torch.cat(b.heads(v["d_qk"]), 1).double() * live
    turned = ref.rotate(dy, v["cos"], v["sin"], v["pos"], False, -1.0)
    n = ref.restore(v["qk_codes"], v["qk_scales"], G) * v["qk_rstd"].double().unsqueeze(2)
    dx, terms, _ = ref.norm_bwd(n, v["qk_rstd"], turned, w)
    size_t = ref.rotate(dy.abs(), v["cos"].abs(), v["sin"].abs(), v["pos"], False)
    size_t = torch.maximum(size_t, ref.rotate(dy.abs(), v["cos"].abs(), -v["sin"].abs(), v["pos"], False))
    _, sizes, size = ref.norm_bwd(n.abs(), v["qk_rstd"], size_t, w.abs())
    ref.assert_close(torch.cat(b.heads(v["d_qkv"]), 1), dx, NORM * size, "d_qk")
    ref.assert_close(v["dqw"], terms[:, :HEADS].sum((0, 1)), SUM * sizes[:, :HEADS].sum((0, 1)), "dqw", F)
    ref.assert_close(v["dkw"], terms[:, HEADS:].sum((0, 1)), SUM * sizes[:, HEADS:].sum((0, 1)), "dkw", F)
    n = ref.restore(v["x_codes"], v["x_scales"], G) * v["rstd"].double().unsqueeze(1)
    dx, terms, size = ref.norm_bwd(n, v["rstd"], v["d_y"], v["norm_w"])
    ref.assert_close(v["dx"], dx + v["d_out"].double(), NORM * size + F * v["d_out"].double().abs(), "dx")
    ref.assert_close(v["d_norm_w"], terms.sum(0), SUM * terms.abs().sum(0), "d_norm_w", F)


def test_block_in_a_graph():
    """Three replays of the captured step equal the eager step bit for bit,
    with the eager step run between them."""
    eager, captured = Block(), Block()
    eager.step()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in eager.results().items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step()
    for _ in range(3):
        for t in captured.results().values():
            t.zero_()
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in captured.results().items():
            assert torch.equal(t, want[n]), n
            assert torch.equal(eager.results()[n], want[n]), n
