"""The activation operators measured: 8-bit activation checkpoints and the
backward passes that read them.

  norm      RMS norm of a residual stream, with the residual addition, the
            E4M3 checkpoint of the norm's input and the output in BF16 or in
            E4M3 under one scale per tensor
  norm_bwd  its gradient, from the checkpoint
  act       gated activation silu(gate) * up, from the E4M3 output of a
            group-scaled linear layer or from BF16 (then it writes the
            checkpoint)
  act_bwd   its gradient, from the checkpoint
  qk        RMS norm of every query and key head and the position rotation
            in one pass, with the checkpoint of the heads
  qk_bwd    its gradient, from the checkpoint
  wgrad     weight gradient of a linear layer whose input was kept in E4M3

A checkpoint is an E4M3 code for each value and an FP32 scale for each group
of G values of a row (scale = max|x| / 448); "per tensor" means one scale.

With `own` false, run() computes them from elementary torch operations in 32
bits; with `own` true through the package's entry points.  Both get what
prepare() made from the seed.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-5
F8 = torch.float8_e4m3fn
GROUPS = (16, 32, 64, 128)
ROPE_BASE = 10000.0

_LARGEST_FLOPS = 2 * 8192 * 22016 * 4096


def listed():
    return [
        # one decoded token through a block's norm: latency alone
        dict(name="norm, one token", op="norm", rows=1, cols=4096, G=128, residual=True, out="bf16", ckpt=False),
        # the norm before a block's projections in training, feeding an 8-bit linear layer
        dict(name="norm, training", op="norm", rows=8192, cols=4096, G=128, residual=True, out="fp8", ckpt=True),
        # its backward pass, with the gradient that comes down the residual stream
        dict(name="norm backward", op="norm_bwd", rows=8192, cols=4096, G=128, residual=True),
        # an odd number of tokens of a wider model, smaller groups
        dict(name="norm backward, odd rows", op="norm_bwd", rows=4097, cols=5120, G=32, residual=False),
        # a few decoded tokens through the gated activation, from the 8-bit projection
        dict(name="act, few tokens", op="act", rows=7, cols=11008, G=128, source="fp8", out="bf16", ckpt=False),
        # training: 8-bit linear layer in, 8-bit linear layer out
        dict(name="act, training", op="act", rows=8192, cols=11008, G=128, source="fp8", out="fp8", ckpt=False),
        # its backward pass
        dict(name="act backward", op="act_bwd", rows=8192, cols=11008, G=128),
        # one decoded token, grouped heads
        dict(name="qk, one token", op="qk", tokens=1, q_heads=32, k_heads=8, dim=128, rot=128, G=128,
             interleaved=False, ckpt=False, padding=0),
        # training on packed sequences
        dict(name="qk, training", op="qk", tokens=8192, q_heads=32, k_heads=32, dim=128, rot=128, G=128,
             interleaved=False, ckpt=True, padding=0),
        # its backward pass; the packed batch ends in padding
        dict(name="qk backward, padded", op="qk_bwd", tokens=8191, q_heads=32, k_heads=8, dim=128, rot=128, G=64,
             interleaved=True, padding=61),
        # a short ragged batch of a small model, grouped scales
        dict(name="wgrad, short", op="wgrad", rows=333, n=2048, k=2048, G=32, scale="group", out="bf16"),
        # the gate and up projections of a 7B-shaped model, input kept under one scale
        dict(name="wgrad, largest", op="wgrad", rows=8192, n=22016, k=4096, G=128, scale="tensor", out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "act", "act_bwd", "qk", "qk_bwd", "wgrad"))
    G = rng.choice(GROUPS)
    if op in ("norm", "norm_bwd"):
        cols = G * max(1, _log(rng, 256, 16384) // G)
        rows = min(_log(rng, 1, 16384), (8192 * 16384) // cols)
        c = dict(op=op, rows=rows, cols=cols, G=G, residual=rng.random() < 0.5)
        if op == "norm":
            c.update(out=rng.choice(("bf16", "fp8")), ckpt=rng.random() < 0.7)
        return c
    if op in ("act", "act_bwd"):
        cols = G * max(1, _log(rng, 256, 22016) // G)
        rows = min(_log(rng, 1, 16384), (8192 * 11008) // cols)
        c = dict(op=op, rows=rows, cols=cols, G=G)
        if op == "act":
            source = rng.choice(("fp8", "bf16"))
            c.update(source=source, out=rng.choice(("bf16", "fp8")), ckpt=source == "bf16" and rng.random() < 0.7)
        return c
    if op in ("qk", "qk_bwd"):
        dim = rng.choice((64, 80, 96, 128, 256))
        G = rng.choice([g for g in GROUPS if dim % g == 0])
        k_heads = rng.choice((1, 2, 4, 8, 32))
        q_heads = k_heads * rng.choice((1, 1, 2, 3, 4, 8)) if k_heads < 32 else 32
        tokens = min(_log(rng, 1, 16384), 8192 * 64 * 128 // ((q_heads + k_heads) * dim))
        rot = dim if rng.random() < 0.7 else 16 * max(1, dim // 32)
        c = dict(op=op, tokens=tokens, q_heads=q_heads, k_heads=k_heads, dim=dim, rot=rot, G=G,
                 interleaved=rng.random() < 0.5, padding=rng.choice((0, 0, tokens // 7)))
        if op == "qk":
            c["ckpt"] = rng.random() < 0.7
        return c
    n, k = 16 * max(1, _log(rng, 128, 22016) // 16), G * max(1, _log(rng, 128, 11008) // G)
    rows = max(1, min(_log(rng, 1, 16384), _LARGEST_FLOPS // (2 * n * k)))
    scale = rng.choice(("group", "tensor"))
    return dict(op=op, rows=rows, n=n, k=k, G=G, scale=scale,
                out=rng.choice(("bf16", "fp32")) if scale == "tensor" else "bf16")


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(gen, *shape):
    return torch.randn(*shape, device="cuda", generator=gen)


def _activations(gen, rows, cols):
    """Hidden states: normal values, a few channels much larger than the rest."""
    channel = torch.exp(0.5 * _normal(gen, cols))
    channel = torch.where(torch.rand(cols, device="cuda", generator=gen) < 0.005, 20.0 * channel, channel)
    return (_normal(gen, rows, cols) * channel).to(torch.bfloat16)


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    gen, c, op = _gen(seed), case, case["op"]
    s = dict(c)
    G = c["G"]
    if op in ("norm", "norm_bwd"):
        rows, cols = c["rows"], c["cols"]
        x = _activations(gen, rows, cols)
        s["weight"] = (1.0 + 0.1 * _normal(gen, cols)).to(torch.bfloat16)
        if op == "norm":
            s["x"] = x
            s["residual"] = _activations(gen, rows, cols) if c["residual"] else None
            s["sum"] = _empty(rows, cols, dtype=torch.bfloat16) if c["residual"] else None
            s["y"] = _empty(rows, cols, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.uint8)
            s["y_scale"] = 2.0 ** -5
            s["amax"] = torch.zeros(1, device="cuda")
            if c["ckpt"]:
                s["codes"] = _empty(rows, cols, dtype=torch.uint8)
                s["scales"] = _empty(rows, cols // G, dtype=torch.float32)
                s["rstd"] = _empty(rows, dtype=torch.float32)
        else:
            s["codes"], s["scales"] = _quantize(x.float(), G)
            s["rstd"] = torch.rsqrt(x.float().square().mean(1) + EPS)
            s["dy"] = (1e-3 * _normal(gen, rows, cols)).to(torch.bfloat16)
            s["d_sum"] = (1e-3 * _normal(gen, rows, cols)).to(torch.bfloat16) if c["residual"] else None
            s["dx"] = _empty(rows, cols, dtype=torch.bfloat16)
            s["dw"] = _empty(cols, dtype=torch.float32)
            s["workspace"] = _empty(1024 * cols, dtype=torch.float32)
    elif op in ("act", "act_bwd"):
        rows, cols = c["rows"], c["cols"]
        gate_up = _activations(gen, rows, 2 * cols)
        if op == "act":
            if c["source"] == "fp8":
                s["codes"], s["scales"] = _quantize(gate_up.float(), G)
                s["gate_up"] = None
            else:
                s["gate_up"] = gate_up
                s["codes"] = _empty(rows, 2 * cols, dtype=torch.uint8) if c["ckpt"] else None
                s["scales"] = _empty(rows, 2 * cols // G, dtype=torch.float32) if c["ckpt"] else None
            s["h"] = _empty(rows, cols, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.uint8)
            s["h_scale"] = 2.0 ** -3
            s["amax"] = torch.zeros(1, device="cuda")
        else:
            s["codes"], s["scales"] = _quantize(gate_up.float(), G)
            s["dh"] = (1e-3 * _normal(gen, rows, cols)).to(torch.bfloat16)
            s["d_gate_up"] = _empty(rows, 2 * cols, dtype=torch.bfloat16)
    elif op in ("qk", "qk_bwd"):
        t, hq, hk, d, rot = c["tokens"], c["q_heads"], c["k_heads"], c["dim"], c["rot"]
        # queries, keys and values of a token lie side by side, as the projection leaves them
        qkv = _activations(gen, t, (hq + 2 * hk) * d)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["q_weight"] = (1.0 + 0.1 * _normal(gen, d)).to(torch.bfloat16)
        s["k_weight"] = (1.0 + 0.1 * _normal(gen, d)).to(torch.bfloat16)
        # packed sequences of up to 4096 tokens; padding behind the last one has position -1
        table = 8192
        first = int(torch.randint(0, 4096, (1,), generator=gen, device="cuda"))
        pos = (torch.arange(t, device="cuda") + first) % 4096 + (first % (table - 4096))
        if c["padding"]:
            pos[t - c["padding"]:] = -1
        s["positions"] = pos
        freq = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        angle = torch.arange(table, dtype=torch.float64, device="cuda")[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        if op == "qk":
            s["q_out"] = _empty(t, hq, d, dtype=torch.bfloat16)
            s["k_out"] = _empty(t, hk, d, dtype=torch.bfloat16)
            if c["ckpt"]:
                s["codes"] = _empty(t, hq + hk, d, dtype=torch.uint8)
                s["scales"] = _empty(t, hq + hk, d // G, dtype=torch.float32)
                s["rstd"] = _empty(t, hq + hk, dtype=torch.float32)
        else:
            x = torch.cat((s["q"], s["k"]), 1).float()
            x = torch.where((pos >= 0)[:, None, None], x, torch.zeros_like(x))
            codes, scales = _quantize(x.reshape(-1, d), G)
            s["codes"], s["scales"] = codes.view(t, hq + hk, d), scales.view(t, hq + hk, d // G)
            s["rstd"] = torch.where((pos >= 0)[:, None], torch.rsqrt(x.square().mean(2) + EPS),
                                    torch.zeros((), device="cuda"))
            s["dq_out"] = (1e-3 * _normal(gen, t, hq, d)).to(torch.bfloat16)
            s["dk_out"] = (1e-3 * _normal(gen, t, hk, d)).to(torch.bfloat16)
            dqkv = torch.zeros(t, (hq + 2 * hk) * d, dtype=torch.bfloat16, device="cuda")
            s["dq"] = dqkv[:, :hq * d].unflatten(1, (hq, d))
            s["dk"] = dqkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
            s["dq_weight"] = _empty(d, dtype=torch.float32)
            s["dk_weight"] = _empty(d, dtype=torch.float32)
            s["workspace"] = _empty(2048 * 2 * d, dtype=torch.float32)
    else:
        rows, n, k = c["rows"], c["n"], c["k"]
        s["dy"] = (1e-3 * _normal(gen, rows, n)).to(torch.bfloat16)
        x = _activations(gen, rows, k).float()
        if c["scale"] == "group":
            s["codes"], s["scales"] = _quantize(x, G)
        else:
            s["scales"] = 2.0 ** -3
            s["codes"] = _codes(x / s["scales"])
        s["dw"] = _empty(n, k, dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)
        # room for partial sums where the rows are split among workgroups
        s["workspace"] = _empty(1 << 26, dtype=torch.float32)
    return s


# ------------------------------------------------------------ plain forms

def _codes(v):
    """E4M3 codes of FP32 values, saturating."""
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(F8).view(torch.uint8)


def _quantize(x, G):
    """Codes and scales of the groups of G values of each row of x (FP32)."""
    rows, cols = x.shape
    g = x.view(rows, cols // G, G)
    top = g.abs().amax(2, keepdim=True)
    q = torch.where(top > 0, g * E4M3_MAX / torch.where(top > 0, top, torch.ones_like(top)), torch.zeros_like(g))
    return _codes(q).view(rows, cols), (top / E4M3_MAX).view(rows, cols // G)


def _dequantize(codes, scales, G):
    rows, cols = codes.shape
    v = codes.view(F8).float().view(rows, cols // G, G)
    return (v * scales.view(rows, cols // G, 1)).view(rows, cols)


def _plain_norm(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (s["x"].float() + s["residual"].float()).to(torch.bfloat16)
    x = h.float()
    rstd = 1.0 / torch.sqrt(x.square().mean(1, keepdim=True) + EPS)
    y = x * rstd * s["weight"].float()
    out = {"sum": h} if s["residual"] is not None else {}
    if s["out"] == "bf16":
        out["y"] = y.to(torch.bfloat16)
    else:
        out["y"] = _codes(y * (1.0 / s["y_scale"])).view(F8)
        out["amax"] = y.abs().amax().reshape(1)
    if s["ckpt"]:
        codes, scales = _quantize(x, s["G"])
        out.update(codes=codes.view(F8), scales=scales, rstd=rstd.view(-1))
    return out


def _plain_norm_bwd(s):
    rstd = s["rstd"].view(-1, 1)
    n = _dequantize(s["codes"], s["scales"], s["G"]) * rstd
    dy = s["dy"].float()
    dn = dy * s["weight"].float()
    dx = rstd * (dn - n * (dn * n).mean(1, keepdim=True))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].float()
    return {"dx": dx.to(torch.bfloat16), "dw": (dy * n).sum(0)}


def _gate_up(s):
    v = s["gate_up"].float() if s.get("gate_up") is not None else _dequantize(s["codes"], s["scales"], s["G"])
    return v[:, :s["cols"]], v[:, s["cols"]:]


def _plain_act(s):
    gate, up = _gate_up(s)
    h = gate / (1.0 + torch.exp(-gate)) * up
    out = {}
    if s["out"] == "bf16":
        out["h"] = h.to(torch.bfloat16)
    else:
        out["h"] = _codes(h * (1.0 / s["h_scale"])).view(F8)
        out["amax"] = h.abs().amax().reshape(1)
    if s["ckpt"]:
        codes, scales = _quantize(s["gate_up"].float(), s["G"])
        out.update(codes=codes.view(F8), scales=scales)
    return out


def _plain_act_bwd(s):
    gate, up = _gate_up(s)
    sig = 1.0 / (1.0 + torch.exp(-gate))
    dh = s["dh"].float()
    d_gate = dh * up * sig * (1.0 + gate * (1.0 - sig))
    d_up = dh * gate * sig
    return torch.cat((d_gate, d_up), 1).to(torch.bfloat16)


def _angles(s):
    """cos and sin of every token, spread over the rotated values of a head, and where a value's partner lies."""
    pos, rot = s["positions"].clamp(min=0), s["rot"]
    at = torch.arange(rot, device="cuda")
    pair = at // 2 if s["interleaved"] else at % (rot // 2)
    partner = at ^ 1 if s["interleaved"] else (at + rot // 2) % rot
    second = at % 2 == 1 if s["interleaved"] else at >= rot // 2
    cos, sin = s["cos"][pos][:, pair], s["sin"][pos][:, pair]
    return cos[:, None, :], torch.where(second, sin, -sin)[:, None, :], partner


def _turned(x, cos, sin, partner, rot):
    r = x[..., :rot]
    return torch.cat((r * cos + r[..., partner] * sin, x[..., rot:]), -1)


def _head_weights(s):
    wq, wk = s["q_weight"].float(), s["k_weight"].float()
    return torch.cat((wq.expand(s["q_heads"], -1), wk.expand(s["k_heads"], -1)))


def _plain_qk(s):
    live = (s["positions"] >= 0)[:, None, None]
    x = torch.cat((s["q"], s["k"]), 1).float()
    x = torch.where(live, x, torch.zeros_like(x))
    rstd = 1.0 / torch.sqrt(x.square().mean(2, keepdim=True) + EPS)
    rstd = torch.where(live, rstd, torch.zeros_like(rstd))
    y = x * rstd * _head_weights(s)
    cos, sin, partner = _angles(s)
    y = _turned(y, cos, sin, partner, s["rot"]).to(torch.bfloat16)
    out = {"q": y[:, :s["q_heads"]], "k": y[:, s["q_heads"]:]}
    if s["ckpt"]:
        codes, scales = _quantize(x.view(-1, s["dim"]), s["G"])
        out.update(codes=codes.view(x.shape).view(F8), scales=scales.view(x.shape[0], x.shape[1], -1),
                   rstd=rstd.squeeze(2))
    return out


def _plain_qk_bwd(s):
    live = (s["positions"] >= 0)[:, None, None]
    hq = s["q_heads"]
    d = torch.cat((s["dq_out"], s["dk_out"]), 1).float()
    d = torch.where(live, d, torch.zeros_like(d))
    cos, sin, partner = _angles(s)
    dy = _turned(d, cos, -sin, partner, s["rot"])
    t, heads, dim = dy.shape
    n = _dequantize(s["codes"].view(-1, dim), s["scales"].view(t * heads, -1), s["G"]).view(t, heads, dim)
    rstd = s["rstd"].unsqueeze(2)
    n = n * rstd
    dn = dy * _head_weights(s)
    dx = rstd * (dn - n * (dn * n).mean(2, keepdim=True))
    dw = dy * n
    dx = dx.to(torch.bfloat16)
    return {"dq": dx[:, :hq], "dk": dx[:, hq:], "dq_weight": dw[:, :hq].sum((0, 1)), "dk_weight": dw[:, hq:].sum((0, 1))}


def _plain_wgrad(s):
    if s["scale"] == "group":
        x = _dequantize(s["codes"], s["scales"], s["G"])
    else:
        x = s["codes"].view(F8).float() * s["scales"]
    return (s["dy"].float().t() @ x).to(s["dw"].dtype)


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "act": _plain_act, "act_bwd": _plain_act_bwd,
          "qk": _plain_qk, "qk_bwd": _plain_qk_bwd, "wgrad": _plain_wgrad}


# ------------------------------------------------- the package's own calls

_coat = None


def _package():
    global _coat
    if _coat is None:
        from adamw_coat_fp8_amd import coat
        _coat = coat
    return _coat


def _own_norm(s):
    fp8, ckpt = s["out"] == "fp8", s["ckpt"]
    if fp8:
        s["amax"].zero_()   # the call raises what it holds: a new maximum starts at 0
    _package().rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], residual_out=s["sum"],
                        y=None if fp8 else s["y"], y_codes=s["y"] if fp8 else None, y_scale=s["y_scale"],
                        y_amax=s["amax"] if fp8 else None, codes=s["codes"] if ckpt else None,
                        scales=s["scales"] if ckpt else None, rstd=s["rstd"] if ckpt else None, group_size=s["G"])
    out = {"sum": s["sum"]} if s["residual"] is not None else {}
    out["y"] = s["y"].view(F8) if fp8 else s["y"]
    if fp8:
        out["amax"] = s["amax"]
    if ckpt:
        out.update(codes=s["codes"].view(F8), scales=s["scales"], rstd=s["rstd"])
    return out


def _own_norm_bwd(s):
    _package().rms_norm_bwd(s["dy"], s["codes"], s["scales"], s["rstd"], s["weight"], s["dx"], s["dw"],
                            d_residual=s["d_sum"], workspace=s["workspace"], group_size=s["G"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _own_act(s):
    fp8 = s["out"] == "fp8"
    if fp8:
        s["amax"].zero_()
    _package().swiglu(s["codes"], s["scales"], gate_up=s["gate_up"], h=None if fp8 else s["h"],
                      h_codes=s["h"] if fp8 else None, h_scale=s["h_scale"], h_amax=s["amax"] if fp8 else None,
                      group_size=s["G"])
    out = {"h": s["h"].view(F8) if fp8 else s["h"]}
    if fp8:
        out["amax"] = s["amax"]
    if s["ckpt"]:
        out.update(codes=s["codes"].view(F8), scales=s["scales"])
    return out


def _own_act_bwd(s):
    _package().swiglu_bwd(s["dh"], s["codes"], s["scales"], s["d_gate_up"], group_size=s["G"])
    return s["d_gate_up"]


def _own_qk(s):
    ckpt = s["ckpt"]
    _package().qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], EPS, s["cos"], s["sin"], s["positions"],
                            s["q_out"], s["k_out"], codes=s["codes"] if ckpt else None,
                            scales=s["scales"] if ckpt else None, rstd=s["rstd"] if ckpt else None,
                            interleaved=s["interleaved"], group_size=s["G"])
    out = {"q": s["q_out"], "k": s["k_out"]}
    if ckpt:
        out.update(codes=s["codes"].view(F8), scales=s["scales"], rstd=s["rstd"])
    return out


def _own_qk_bwd(s):
    _package().qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["codes"], s["scales"], s["rstd"], s["q_weight"],
                                s["k_weight"], s["cos"], s["sin"], s["positions"], s["dq"], s["dk"],
                                s["dq_weight"], s["dk_weight"], workspace=s["workspace"],
                                interleaved=s["interleaved"], group_size=s["G"])
    return {"dq": s["dq"], "dk": s["dk"], "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]}


def _own_wgrad(s):
    _package().weight_grad(s["dy"], s["codes"], s["scales"], s["dw"], workspace=s["workspace"], group_size=s["G"])
    return s["dw"]


_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "act": _own_act, "act_bwd": _own_act_bwd,
        "qk": _own_qk, "qk_bwd": _own_qk_bwd, "wgrad": _own_wgrad}


def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


# ------------------------------------------------------------------- work

def work(case):
    c, op, G = case, case["op"], case["G"]
    if op in ("norm", "norm_bwd"):
        e = c["rows"] * c["cols"]
        ckpt = e + 4 * e // G + 4 * c["rows"]
        if op == "norm":
            b = 2 * e + (4 * e if c["residual"] else 0) + (2 * e if c["out"] == "bf16" else e)
            return {"bytes": b + (ckpt if c["ckpt"] else 0) + 2 * c["cols"], "flops": 4 * e}
        return {"bytes": 4 * e + (2 * e if c["residual"] else 0) + ckpt + 6 * c["cols"], "flops": 10 * e}
    if op in ("act", "act_bwd"):
        e = c["rows"] * c["cols"]
        ckpt = 2 * e + 8 * e // G
        if op == "act":
            b = (2 * e if c["out"] == "bf16" else e) + (4 * e if c["source"] == "bf16" else ckpt)
            return {"bytes": b + (ckpt if c["ckpt"] else 0), "flops": 5 * e}
        return {"bytes": ckpt + 6 * e, "flops": 12 * e}
    if op in ("qk", "qk_bwd"):
        heads = c["tokens"] * (c["q_heads"] + c["k_heads"])
        e = heads * c["dim"]
        ckpt = e + 4 * e // G + 4 * heads
        table = 8 * c["tokens"] + 4 * c["rot"] * min(c["tokens"], 4096) + 4 * c["dim"]
        if op == "qk":
            return {"bytes": 4 * e + table + (ckpt if c["ckpt"] else 0), "flops": 7 * e}
        return {"bytes": 4 * e + table + ckpt + 8 * c["dim"], "flops": 13 * e}
    m, n, k = c["rows"], c["n"], c["k"]
    b = 2 * m * n + m * k + (4 * m * k // G if c["scale"] == "group" else 0) + (2 if c["out"] == "bf16" else 4) * n * k
    return {"bytes": b, "flops": 2 * m * n * k}


# ----------------------------------------------- the definitions in 64 bits

def _e4m3_64(v):
    """The nearest E4M3 value (ties to even) of each 64-bit value, saturating at 448."""
    a = v.abs()
    exponent = torch.frexp(a)[1].double() - 1.0
    step = torch.exp2(exponent.clamp(min=-6.0) - 3.0)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _group_64(x, G):
    """E4M3 values and scales of groups of G values along the last axis."""
    g = x.unflatten(-1, (-1, G))
    top = g.abs().amax(-1, keepdim=True)
    values = _e4m3_64(torch.nan_to_num(E4M3_MAX * g / top, nan=0.0))
    return values.flatten(-2), top.squeeze(-1) / E4M3_MAX


def _table_64():
    """The value of each of the 256 codes (the two NaN codes as 0)."""
    code = torch.arange(256, device="cuda")
    e, m = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.double() - 10.0))
    v[[127, 255]] = 0.0
    return torch.where(code >= 128, -v, v)


def _restored_64(s):
    values = _table_64()[s["codes"].long()]
    if not torch.is_tensor(s["scales"]):
        return values * float(s["scales"])
    return values * s["scales"].double().repeat_interleave(s["G"], dim=-1)


def _norm_gradient_64(n, rstd, dy, weight):
    """dx of y = n * weight, n = x * rstd, and dy * n (whose sum is the weight's gradient)."""
    dn = dy * weight
    along = (dn * n).sum(-1, keepdim=True) / n.shape[-1]
    return rstd * (dn - along * n), dy * n


def _rotate_64(y, s, sign):
    """Turns the pairs of the first `rot` values of each head by sign * the token's angle."""
    rot, pos = s["rot"], s["positions"].clamp(min=0)
    c, n = s["cos"].double()[pos].unsqueeze(1), sign * s["sin"].double()[pos].unsqueeze(1)
    z = y.clone()
    first = slice(0, rot, 2) if s["interleaved"] else slice(0, rot // 2)
    other = slice(1, rot, 2) if s["interleaved"] else slice(rot // 2, rot)
    a, b = y[..., first], y[..., other]
    z[..., first], z[..., other] = a * c - b * n, a * n + b * c
    return z


def exact(case, seed):
    s = prepare(case, seed)
    op, G = case["op"], case["G"]
    if op == "norm":
        x, out = s["x"].double(), {}
        if case["residual"]:
            # the sum is rounded to BF16 before anything reads it
            x = (x + s["residual"].double()).to(torch.bfloat16).double()
            out["sum"] = x
        rstd = (x.pow(2).sum(1) / case["cols"] + EPS) ** -0.5
        y = s["weight"].double() * x * rstd[:, None]
        out["y"] = y if case["out"] == "bf16" else _e4m3_64(y / s["y_scale"])
        if case["out"] == "fp8":
            out["amax"] = y.abs().max().reshape(1)
        if case["ckpt"]:
            out["codes"], out["scales"] = _group_64(x, G)
            out["rstd"] = rstd
        return out
    if op == "norm_bwd":
        rstd = s["rstd"].double()[:, None]
        dx, dw = _norm_gradient_64(_restored_64(s) * rstd, rstd, s["dy"].double(), s["weight"].double())
        if case["residual"]:
            dx = dx + s["d_sum"].double()
        return {"dx": dx, "dw": dw.sum(0)}
    if op == "act":
        x = s["gate_up"].double() if case["source"] == "bf16" else _restored_64(s)
        gate, up = x.chunk(2, dim=1)
        h = gate * up * torch.sigmoid(gate)
        out = {"h": h if case["out"] == "bf16" else _e4m3_64(h / s["h_scale"])}
        if case["out"] == "fp8":
            out["amax"] = h.abs().max().reshape(1)
        if case["ckpt"]:
            out["codes"], out["scales"] = _group_64(x, G)
        return out
    if op == "act_bwd":
        gate, up = _restored_64(s).chunk(2, dim=1)
        sig, dh = torch.sigmoid(gate), s["dh"].double()
        return torch.cat((dh * up * (sig + gate * sig * torch.sigmoid(-gate)), dh * gate * sig), 1)
    if op in ("qk", "qk_bwd"):
        hq = case["q_heads"]
        live = (s["positions"] >= 0).double()[:, None, None]
        w = torch.stack([s["q_weight"].double()] * hq + [s["k_weight"].double()] * case["k_heads"])
        if op == "qk":
            x = torch.cat((s["q"].double(), s["k"].double()), 1) * live
            rstd = (x.pow(2).sum(2, keepdim=True) / case["dim"] + EPS) ** -0.5 * live
            y = _rotate_64(w * x * rstd, s, 1.0)
            out = {"q": y[:, :hq], "k": y[:, hq:]}
            if case["ckpt"]:
                out["codes"], out["scales"] = _group_64(x, G)
                out["rstd"] = rstd.squeeze(2)
            return out
        rstd = s["rstd"].double().unsqueeze(2)
        dy = _rotate_64(torch.cat((s["dq_out"].double(), s["dk_out"].double()), 1) * live, s, -1.0)
        dx, dw = _norm_gradient_64(_restored_64(s) * rstd, rstd, dy, w)
        dw = dw.sum(0)
        return {"dq": dx[:, :hq], "dk": dx[:, hq:], "dq_weight": dw[:hq].sum(0), "dk_weight": dw[hq:].sum(0)}
    return s["dy"].double().t().contiguous() @ _restored_64(s)
