"""4-bit weights on the GPU: quantisation and its inverse bit for bit against
the definition, and the product of fp8 rows with such weights against 64-bit
products."""
import pytest
import torch

from tests import experts_reference as ref
from tests.test_experts_gpu import CASES as BF16_CASES
from tests.test_experts_gpu import GUARD, gen, guard, make_rows, rand, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def epx():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a visible GPU")
    from combine_epx_get_amd import epx as mod
    return mod


def check_quantise(epx, x):
    codes = torch.full((*x.shape[:-1], x.shape[-1] // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((*x.shape[:-1], x.shape[-1] // 32), 0xA5, dtype=torch.uint8, device="cuda")
    epx.epx_mxfp4_quantize(x, codes, scales)
    back = torch.full_like(x, GUARD)
    epx.epx_mxfp4_dequantize(codes, scales, back)
    torch.cuda.synchronize()
    c, s = ref.mxfp4_quantize(x)
    assert torch.equal(scales, s)
    bad = (codes != c).nonzero()
    assert not len(bad), [(x.view(-1, x.shape[-1])[r, 2 * i:2 * i + 2].tolist(), hex(codes.view(c.shape)[tuple(at)]),
                           hex(c[tuple(at)]), int(s[tuple(at[:-1])][at[-1] // 16]))
                          for at in bad[:6].tolist() for r, i in [(at[0], at[-1])]]
    want = ref.mxfp4_values(c, s)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(back), nan)
    assert torch.equal(back.double()[~nan], want[~nan])       # exact
    assert torch.equal(torch.signbit(back)[~nan], torch.signbit(want)[~nan])


def test_every_bf16_pattern_under_every_scale(epx):
    """Every bf16 value v beside every block maximum m >= |v| that has its exponent or up to 6 above (the codes are
    0 further below), in both signs; infinities and NaN among them."""
    bits = torch.arange(1 << 15, dtype=torch.int32, device="cuda")
    for up in range(7):
        top = ((bits >> 7) + up).clamp(max=254) << 7
        for mant in (0, 1, 63, 64, 127):
            m = torch.maximum(top | mant, bits)
            block = torch.zeros(1 << 15, 32, dtype=torch.int32, device="cuda")
            block[:, 0] = m
            block[:, 1] = bits
            block[:, 2] = bits | 0x8000
            block[:, 31] = 0x8000
            x = block.to(torch.int16).view(torch.bfloat16)
            check_quantise(epx, x)


@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (1, 7168), (129, 96), (2, 5, 256), (3, 40, 1056), (4097, 2048)],
                         ids=str)
def test_quantise(epx, shape):
    g = gen(sum(shape))
    x = rand(g, *shape, std=0.02)
    x[0, ..., :32] = 0.0
    check_quantise(epx, x)


def test_extremes(epx):
    """All zeros, negative zeros, subnormals, the largest values, infinities and NaN."""
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    x[1] = -0.0
    x[2, ::3] = 9.2e-41          # bf16's smallest subnormal
    x[2, 5] = 1e-38
    x[3] = 3.3e38
    x[3, ::2] = -1.0
    x[4, 7], x[5, 40], x[6, 0] = float("inf"), float("-inf"), float("nan")
    x[7] = torch.linspace(-6, 6, 64, device="cuda").to(torch.bfloat16)
    check_quantise(epx, x)


def test_dequantise_every_code_and_scale(epx):
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(16, 16).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").repeat_interleave(16).view(-1, 1)
    out = torch.empty(4096, 32, dtype=torch.bfloat16, device="cuda")
    epx.epx_mxfp4_dequantize(codes, scales, out)
    torch.cuda.synchronize()
    want = ref.mxfp4_values(codes, scales).to(torch.float32).to(torch.bfloat16)   # codes 4, 6 of the top scales: infinity
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(out), nan)
    assert torch.equal(out[~nan], want[~nan])


# as for the bf16 products, with inner a multiple of 128 and an inner of one,
# two and an odd number of blocks
CASES = [(n, c, gap, o, N, 128 * (1 + (K // 72) % 9)) for n, c, gap, o, N, K in BF16_CASES] + [
    ("few tiles, 21 blocks", [33, 0, 64, 7], 1, None, 264, 2688),
    ("some tiles, 29 blocks", [100, 0, 60, 150], 0, None, 520, 3712),
    ("more tiles, 23 blocks", [290, 2, 260], 2, [2, 0, 1], 808, 2944),
    ("24 experts, 13 blocks", [(i * 53) % 300 for i in range(24)], 1, None, 1032, 1664),
    ("24 experts, wide, 13 blocks", [(i * 53) % 300 for i in range(24)], 1, None, 2056, 1664)]


def operands(g, n, M, R, K, epx):
    x, xs, xv = ref.fp8_rows(rand(g, R, K, std=3.0))
    w = rand(g, n, M, K, std=K ** -0.5)
    codes = torch.empty(n, M, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n, M, K // 32, dtype=torch.uint8, device="cuda")
    epx.epx_mxfp4_quantize(w, codes, scales)
    return x, xs, xv, codes, scales, ref.mxfp4_values(codes, scales)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_product(epx, case, act):
    name, cnt, gap, order, N, K = case
    off, R = ref.ranges(cnt, gap, order)
    print(f"[mx] {name} R={R} n={len(cnt)} N={N} K={K}", flush=True)
    rows = make_rows(epx, off, cnt, R)
    M = 2 * N if act == "swiglu" else N
    x, xs, xv, codes, scales, wv = operands(gen(20), len(cnt), M, R, K, epx)
    out = guard(R, N)
    epx.epx_expert_gemm_mxfp4(rows, x, xs, codes, scales, out, act=epx.ACT_SWIGLU if act == "swiglu" else epx.ACT_NONE)
    torch.cuda.synchronize()
    z, b = ref.product(xv, wv, off, cnt)
    if act == "swiglu":
        z, b = ref.glu(z, b)
    ref.close(out, z, b, ref.BF16, "out")
    untouched(out, off, cnt, "out")


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("case", [("one", [1], 0, None, 128, 128), ("decode", [0, 3, 17, 1], 2, None, 384, 640),
                                  ("middle", [50, 0, 90, 64], 1, [2, 0, 1, 3], 256, 384),
                                  ("more rows", [130, 257, 3], 0, None, 640, 256),
                                  ("large tiles", [(i * 53) % 300 for i in range(150)], 1, None, 384, 256),
                                  ("few rows, 60 experts", [i % 5 for i in range(60)], 0, None, 256, 640),
                                  ("middle, wide", [40, 64, 0, 130, 200, 61, 150, 55], 0, None, 1536, 384),
                                  ("few tiles, 21 blocks", [70, 3], 1, None, 256, 2688),
                                  ("24 experts, wide", [(i * 53) % 300 for i in range(24)], 1, None, 2176, 1664)],
                         ids=lambda c: c[0])
def test_product_to_fp8_rows(epx, case, act):
    name, cnt, gap, order, N, K = case
    off, R = ref.ranges(cnt, gap, order)
    print(f"[mx fp8] {name} R={R} n={len(cnt)} N={N} K={K}", flush=True)
    rows = make_rows(epx, off, cnt, R)
    M = 2 * N if act == "swiglu" else N
    x, xs, xv, codes, scales, wv = operands(gen(21), len(cnt), M, R, K, epx)
    out = torch.full((R, N), 0xA5, dtype=torch.uint8, device="cuda")
    osc = torch.full((R, N // 128), GUARD, device="cuda")
    epx.epx_expert_gemm_mxfp4(rows, x, xs, codes, scales, out, act=epx.ACT_SWIGLU if act == "swiglu" else epx.ACT_NONE,
                              out_scales=osc)
    torch.cuda.synchronize()
    z, b = ref.product(xv, wv, off, cnt)
    if act == "swiglu":
        z, b = ref.glu(z, b)
    live = ~torch.isnan(z[:, 0])
    zb, bb = z[live].view(-1, N // 128, 128), b[live].view(-1, N // 128, 128)
    # the scale: the largest magnitude, off by at most its bound, over 448 and rounded
    amax, bmax = zb.abs().amax(2), bb.amax(2)
    s = osc[live].double()
    assert bool(((s * 448 - amax).abs() <= bmax + 2.0 ** -22 * amax).all())
    v = out.view(torch.float8_e4m3fn)[live].double().view_as(zb) * s.unsqueeze(2)
    # half a step of E4M3 (2^-10 of the scale below its normal numbers); a
    # quotient that the rounding of the scale puts past 448 is clamped
    tol = bb + 2.0 ** -4 * (zb.abs() + bb) + s.unsqueeze(2) * 2.0 ** -10 + 2.0 ** -21 * zb.abs()
    assert bool(((v - zb).abs() <= tol).all())
    assert bool((out[~live] == 0xA5).all()) and bool((osc[~live] == GUARD).all())


def test_zero_rows_give_zero_scales(epx):
    rows = make_rows(epx, [0], [5], 5)
    x, xs, xv, codes, scales, wv = operands(gen(22), 1, 128, 5, 256, epx)
    x[2], xs[3] = 0, 0.0
    out = torch.full((5, 128), 0xA5, dtype=torch.uint8, device="cuda")
    osc = torch.full((5, 1), GUARD, device="cuda")
    epx.epx_expert_gemm_mxfp4(rows, x, xs, codes, scales, out, out_scales=osc)
    torch.cuda.synchronize()
    assert osc[2].item() == 0.0 and osc[3].item() == 0.0
    assert not (out[2:4] & 0x7F).any()
    assert (osc[[0, 1, 4]] > 0).all()


def test_scale_range(epx):
    """Weights at both ends of the scale bytes, and a NaN block, which stays in its own columns.

    The sums of 128 codes times weights are float32 sums before the row's scale is applied. Under scale byte 250
    they reach 128 * 448 * 6 * 2^123 > 2^128, so there a column is infinite (or NaN, from infinities of both signs)
    although its value times the row's scale may be a number again; it is compared where no sum of magnitudes can
    reach 2^128."""
    rows = make_rows(epx, [0], [20], 20)
    x, xs, xv, codes, scales, wv = operands(gen(23), 1, 64, 20, 384, epx)
    scales[0, 3], scales[0, 7, 1], scales[0, 9, 2] = 20, 250, 255
    scales[0, 11], scales[0, 12, ::2] = 1, 0
    wv = ref.mxfp4_values(codes, scales)
    out = guard(20, 64)
    epx.epx_expert_gemm_mxfp4(rows, x, xs, codes, scales, out)
    torch.cuda.synchronize()
    codes_x = x.view(torch.float8_e4m3fn).double().view(20, 3, 128)
    size = torch.einsum("rbk,nbk->rnb", codes_x.abs(), wv[0].nan_to_num().abs().view(64, 3, 128)).amax(2)
    assert bool((size[:, [c for c in range(64) if c != 7]] < 2.0 ** 127).all())
    total = torch.einsum("rbk,bk->rb", codes_x, wv[0, 7].view(3, 128)).abs().amax(1)
    assert not torch.isfinite(out[:, 7][total > 2.0 ** 129]).any()
    keep = [c for c in range(64) if c not in (7, 9)]
    z, b = ref.product(xv, wv[:, [7]], [0], [20])
    fine = size[:, 7] < 2.0 ** 127
    ref.close(out[fine][:, [7]], z[fine], b[fine], ref.BF16, "out")
    assert torch.isnan(out[:, 9]).all()
    z, b = ref.product(xv, wv[:, keep], [0], [20])
    ref.close(out[:, keep].contiguous(), z, b, ref.BF16, "out")


def test_graph(epx):
    cnt = [40, 0, 9]
    off, R = ref.ranges(cnt)
    rows = make_rows(epx, off, cnt, R)
    g = gen(24)
    x, xs, xv, codes, scales, wv = operands(g, 3, 256, R, 384, epx)
    w = rand(g, 3, 256, 384)
    a, b = guard(R, 128), guard(R, 128)
    graph = torch.cuda.CUDAGraph()
    c2, s2 = torch.empty_like(codes), torch.empty_like(scales)
    with torch.cuda.graph(graph):
        epx.epx_mxfp4_quantize(w, c2, s2)
        epx.epx_expert_gemm_mxfp4(rows, x, xs, c2, s2, b, act=epx.ACT_SWIGLU)
    for _ in range(3):
        w.normal_(0, 0.05)
        epx.epx_mxfp4_quantize(w, codes, scales)
        epx.epx_expert_gemm_mxfp4(rows, x, xs, codes, scales, a, act=epx.ACT_SWIGLU)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b)
