"""Operands whose products' sums are exact in float32, in any order, so that a
result has one right value.

Half of a sum is a_i * b_i with whole numbers from 1 to 32, the other half
-(a_i + e_i) * b_i with a few small whole e_i: partial sums reach some million
(below 2^24, so float32 holds them exactly) and the whole sum is -sum e_i * b_i,
a whole number of at most 256 that bf16 holds too. A term that is left out, or
a partial sum that is held in fewer bits, shows in the result.
"""
import torch


def gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def whole(g, lo, hi, *shape):
    """Whole numbers lo .. hi, float32."""
    return torch.randint(lo, hi + 1, shape, generator=g, device=g.device).float()


def few(g, rows, length, most, values):
    """[rows, length]: at most `most` numbers other than 0 a row, -values .. values."""
    e = torch.zeros(rows, length, device=g.device)
    at = torch.randint(0, length, (rows, most), generator=g, device=g.device)
    return e.scatter_(1, at, whole(g, -values, values, rows, most))


def along_rows(g, rows, length, unit=1.0):
    """Left operand [rows, length] whose rows are summed over."""
    assert length % 2 == 0 and length // 2 * 34 * 32 < 1 << 24
    a = whole(g, 1, 32, rows, length // 2)
    return (torch.cat((a, a + few(g, rows, length // 2, 4, 2)), 1) * unit).to(torch.bfloat16)


def matrices(g, n, rows, length):
    """Right operands [n, rows, length] to go with them."""
    b = whole(g, 1, 32, n, rows, length // 2)
    return torch.cat((b, -b), 2).to(torch.bfloat16)


def down_columns(g, rows, left, right, off, cnt):
    """dy [rows, left] and x [rows, right] whose rows are summed over within each range; 0 elsewhere."""
    dy, x = torch.zeros(rows, left, device=g.device), torch.zeros(rows, right, device=g.device)
    for o, c in zip(off, cnt):
        h = c // 2
        assert h * 33 * 32 < 1 << 24
        if h:
            a, b = whole(g, 1, 32, h, left), whole(g, 1, 32, h, right)
            e = torch.zeros(h, left, device=g.device)
            for r in torch.randint(0, h, (4,), generator=g, device=g.device).tolist():
                e[r] = whole(g, -1, 1, left)
            dy[o:o + h], x[o:o + h] = a, b
            dy[o + h:o + 2 * h], x[o + h:o + 2 * h] = a + e, -b
        if c % 2:
            dy[o + c - 1], x[o + c - 1] = whole(g, -3, 3, left), whole(g, 1, 32, right)
    return dy.to(torch.bfloat16), x.to(torch.bfloat16)


def by_expert(x, w, off, cnt):
    """x[r] @ w[e].T in float64; rows of no expert NaN."""
    z = torch.full((x.shape[0], w.shape[1]), float("nan"), dtype=torch.float64, device=x.device)
    for e, (o, c) in enumerate(zip(off, cnt)):
        if c:
            z[o:o + c] = x[o:o + c].double() @ w[e].double().T
    return z


def fp8_and_4_bit(g, n, columns, rows, length):
    """(codes of x, their float32 scales, codes of w, their scale bytes): E4M3 whole numbers 0 .. 16 under powers of
    two, and E2M1 codes under three neighbouring scales. Inside a group of eight the products lie within 2^9 of each
    other's last bits, so that nothing is cut where they are added."""
    assert length % 128 == 0 and length // 2 * 16 * 48 < 1 << 24
    half = length // 2
    a = whole(g, 1, 15, rows, half)
    e = few(g, rows, half, 4, 1)
    x = torch.cat((a, a + e), 1).to(torch.float8_e4m3fn).view(torch.uint8)
    xs = torch.exp2(whole(g, -2, 2, rows, 1)).expand(rows, length // 128).contiguous()
    b = torch.randint(1, 8, (n, columns, half), generator=g, device=g.device)
    b = torch.cat((b, b | 8), 2).to(torch.uint8)
    ws = torch.randint(127, 130, (n, columns, half // 32), generator=g, device=g.device)
    return x, xs, b[..., 0::2] | (b[..., 1::2] << 4), torch.cat((ws, ws), 2).to(torch.uint8)
