"""Plain 64-bit forms of the experts' operators, and the error bounds that
their GPU results are held to.

Bounds. A product of n terms summed in float32 is off by at most
n * 2^-23 * sum |a_i b_i| (every addition rounds or truncates to 24 bits; the
products of two bf16 values, and of E4M3 and E2M1 values, are exact), and a
final rounding by half a step relative to the value: bf16 2^-8, E4M3 2^-4
(2^-10 absolute below its smallest normal number, in units of the scale).
"""
import torch

BF16 = 2.0 ** -8
SUM = 2.0 ** -23
# exp, reciprocal and the few products of the activation in float32: a step
# or two each, and exp's relative error grows with its argument
ACT = 2.0 ** -20
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def ranges(counts, gap=0, order=None):
    """Row offsets for the counts: one after another in `order`, `gap` rows before each."""
    off, at = [0] * len(counts), 0
    for e in order or range(len(counts)):
        at += gap
        off[e] = at
        at += counts[e]
    return off, at + gap


def sigmoid(v):
    return torch.sigmoid(v)


def product(x, w, off, cnt):
    """z[r] = x[r] @ w[e].T and the bound of its float32 sum; rows of no expert are NaN."""
    z = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64, device=x.device)
    b = z.clone()
    for e, (o, c) in enumerate(zip(off, cnt)):
        if c:
            z[o:o + c] = x[o:o + c] @ w[e].T
            b[o:o + c] = x[o:o + c].abs() @ w[e].abs().T * (SUM * max(1, x.shape[1]))
    return z, b


def glu(z, b):
    """silu(gate) * up and its bound, from the product and the product's bound."""
    N = z.shape[1] // 2
    g, u, bg, bu = z[:, :N], z[:, N:], b[:, :N], b[:, N:]
    s = sigmoid(g)
    out = g * s * u
    # |d silu / d gate| <= 1.1
    return out, 1.1 * bg * (u.abs() + bu) + (g * s).abs() * bu + ACT * (1 + g.abs()) * out.abs()


def glu_backward(d, bd, pre):
    K = d.shape[1]
    g, u = pre[:, :K], pre[:, K:]
    s = sigmoid(g)
    fg, fu = u * s * (1 + g * (1 - s)), g * s
    # the gradient's factor cancels near its zero (gate = -1.28): its float32
    # error is relative to the terms
    eg = ACT * (1 + g.abs()) * u.abs() * s * (1 + (g * (1 - s)).abs())
    eu = ACT * (1 + g.abs()) * fu.abs()
    out = torch.cat((d * fg, d * fu), 1)
    return out, torch.cat((bd * fg.abs() + (d.abs() + bd) * eg, bd * fu.abs() + (d.abs() + bd) * eu), 1)


def close(got, want, bound, rounding, name):
    """|got - want| <= bound + rounding * (|want| + bound), where want is a number (a row of some expert)."""
    live = ~torch.isnan(want)
    g, w, b = got.double()[live], want[live], bound[live]
    over = (g - w).abs() - (b + rounding * (w.abs() + b) + 1e-38)
    bad = ~(over <= 0)
    assert not bad.any(), (name, int(bad.sum()), float(over.max()), g[bad][:4].tolist(), w[bad][:4].tolist())


def fp8_rows(x):
    """Codes (uint8), scales and the 64-bit values of rows quantised per 128 channels."""
    b = x.float().view(x.shape[0], -1, 128)
    s = b.abs().amax(2) / 448.0
    q = (b / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    v = (q.double() * s.double().unsqueeze(2)).view(x.shape)
    return q.view(x.shape).view(torch.uint8), s, v


def mxfp4_values(codes, scales):
    """64-bit values of codes [..., K/2] with scale bytes [..., K/32]."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, float("nan")), s)
    return grid[c] * s.repeat_interleave(32, -1)


def mxfp4_quantize(x):
    """Codes and scale bytes of bf16 rows by the definition, from 64-bit values."""
    b = x.double().view(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    odd = ~torch.isfinite(amax)
    safe = torch.where((amax > 0) & ~odd, amax, torch.ones_like(amax))
    e = (torch.frexp(safe).exponent - 3).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    a = b.abs() / torch.exp2(e.double()).unsqueeze(-1)
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    lo, hi = torch.searchsorted(mid, a.contiguous()), torch.searchsorted(mid, a.contiguous(), right=True)
    c = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
    c = (c | (torch.signbit(b).long() << 3)).view(*x.shape[:-1], -1)
    c = torch.where(odd.repeat_interleave(32, -1), torch.zeros_like(c), c).to(torch.uint8)
    scales = torch.where(odd, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4), scales
