"""Plain 64-bit forms of the 8-bit row formats: int8 rows with a float32 scale
each, and blocks of 32 int8 under a power of two (MXINT8)."""
import torch


def int8_rows(x):
    """Codes and scales of bf16 rows. A quotient of a bf16 number (8 bits) and a float32 number (24 bits) that is not
    on a tie is at least 2^-33 of its value from it, so 64 bits round it as the exact one."""
    v = x.double()
    amax = v.abs().amax(-1)
    odd = ~torch.isfinite(amax)
    s = torch.where(odd, torch.zeros_like(amax), amax / 127).float().clamp(min=2.0 ** -125)
    s = torch.where((amax == 0) | odd, torch.zeros_like(s), s)
    q = torch.where((s > 0).unsqueeze(-1), v, torch.zeros_like(v)) / torch.where(s > 0, s, torch.ones_like(s)).double().unsqueeze(-1)
    codes = torch.round(q).to(torch.int8)   # ties to even
    return codes, torch.where(odd, torch.full_like(s, float("nan")), s)


def mxint8(v):
    """Codes and scale bytes of values [..., 32 n] (float32 or float64 numbers)."""
    b = v.double().view(*v.shape[:-1], v.shape[-1] // 32, 32)
    amax = b.abs().amax(-1)
    odd = ~torch.isfinite(amax)
    safe = torch.where((amax > 0) & ~odd, amax, torch.ones_like(amax))
    e = torch.where(amax > 0, (torch.frexp(safe).exponent - 1).clamp(min=-127), torch.full_like(safe, -127, dtype=torch.int32))
    q = torch.round(b * torch.exp2((6 - e).double()).unsqueeze(-1)).clamp(-127, 127)
    codes = torch.where(odd.unsqueeze(-1), torch.zeros_like(q), q).to(torch.int8).view(v.shape)
    return codes, torch.where(odd, torch.full_like(e, 255), e + 127).to(torch.uint8)


def mxint8_steps(scales):
    """The 64-bit step of each scale byte; NaN for 255."""
    s = torch.exp2(scales.double() - 133)
    return torch.where(scales == 255, torch.full_like(s, float("nan")), s)


def mxint8_values(codes, scales):
    return codes.double() * mxint8_steps(scales).repeat_interleave(32, -1)


def same(got, want, name):
    """Equal, NaN with NaN."""
    a, b = got.double(), want.double()
    bad = ~((a == b) | (torch.isnan(a) & torch.isnan(b)))
    assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4].tolist(), a[bad][:4].tolist(), b[bad][:4].tolist())
