"""The activation operators from their formulas in 64 bits (plain torch, on
the CPU), and the error bounds their tests use.

Bounds.  A rounding to BF16 is off by at most 2^-8 of the value (half a step
relative to it), one to FP32 by 2^-24; E4M3 codes are checked as intervals: the code of a value
known to within `rel` lies between the codes of its ends.  `F` counts FP32
roundings: a sum of n products formed in chains and trees of depth d is off
by at most (d + 1) 2^-24 of the sum of the products' magnitudes.
"""
import numpy as np
import torch

BF16, F = 2.0 ** -8, 2.0 ** -24
TINY = 2.0 ** -126   # below it a BF16 or FP32 value rounds by an absolute amount


def e4m3_round(v):
    """Nearest E4M3 value (ties to even) of 64-bit values, saturating."""
    a = v.abs()
    e = torch.frexp(a)[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)


def code_values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def quantize(x, G):
    """Codes (uint8) and FP32 scales of a BF16 matrix: ties decided on the
    exact quotient."""
    g = x.double().unflatten(-1, (-1, G))
    top = g.abs().amax(-1, keepdim=True)
    q = torch.where(top > 0, 448.0 * g / torch.where(top > 0, top, torch.ones_like(top)), torch.zeros_like(g))
    codes = e4m3_round(q).float().to(torch.float8_e4m3fn).view(torch.uint8)
    scales = (top.float() / torch.tensor(448.0)).squeeze(-1)
    return codes.flatten(-2), scales


def restore(codes, scales, G):
    return code_values(codes) * scales.double().repeat_interleave(G, -1)


def assert_between(got, lo, hi, what):
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{np.unravel_index(int(bad.flatten().int().argmax()), bad.shape)}")


def assert_close(got, ref, slack, what, rounding=BF16):
    """|got - ref| <= slack (the FP32 arithmetic) + the last rounding."""
    tol = slack + rounding * (ref.abs() + slack) + TINY * rounding
    assert_between(got.double(), ref - tol, ref + tol, what)


def assert_codes(codes, ref, rel, what):
    """E4M3 codes of values within rel of ref."""
    a = ref.abs() * rel + 2.0 ** -140
    assert_between(code_values(codes), e4m3_round(ref - a), e4m3_round(ref + a), what)


def norm(x, weight, eps):
    x = x.double()
    rstd = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    return x * rstd * weight.double(), rstd.squeeze(-1)


def norm_bwd(n, rstd, dy, weight):
    """dx, the terms of dw, and the magnitudes dx is formed from."""
    r = rstd.double().unsqueeze(-1)
    dn = dy.double() * weight.double()
    mean = (dn * n).mean(-1, keepdim=True)
    dx = r * (dn - n * mean)
    size = r * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True))
    return dx, dy.double() * n, size


def silu_parts(gate):
    s = torch.sigmoid(gate.double())
    return s, torch.sigmoid(-gate.double())


def rotate(y, cos, sin, positions, interleaved, sign=1.0):
    rot = 2 * cos.shape[1]
    pos = positions.clamp(min=0, max=max(cos.shape[0] - 1, 0))
    c, s = cos.double()[pos].unsqueeze(1), sign * sin.double()[pos].unsqueeze(1)
    a_at = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b_at = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    z = y.clone()
    a, b = y[..., a_at], y[..., b_at]
    z[..., a_at], z[..., b_at] = a * c - b * s, b * c + a * s
    return z
