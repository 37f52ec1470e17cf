"""The experts' products of int8 rows, and those that write or read activations
kept in 8 bits, on the GPU against 64-bit products: ragged, empty, single and
scattered row ranges, sizes that end inside tiles, and buffers with guard rows
that must stay as they were.

Tolerances. An int8 product is exact up to three roundings to float32, which
the tests repeat, so its results are equal. What is kept from sums in float32
may be off by half a step of its block and by the sum's own bound; the scale
byte is that of a largest magnitude within the sum's bound. All else as
experts_reference states."""
import pytest
import torch

from tests import experts_reference as ref
from tests import rows8_reference as r8
from tests.test_experts_gpu import CASES as BF16_CASES
from tests.test_experts_gpu import gen, guard, make_rows, rand, untouched

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def epx():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a visible GPU")
    from combine_epx_get_amd import epx as mod
    return mod


def up(v, unit):
    return (v + unit - 1) // unit * unit


# The bf16 products' cases, with sizes that these calls take, and some of their own.
MORE = [
    ("32 gates, one row", [1], 0, None, 32, 32),
    ("uneven blocks", [70, 0, 3], 1, None, 96, 160),
    ("decode of one expert's size", [32] * 8, 0, None, 1024, 2048),
    ("long sum, few rows", [1, 2], 0, None, 64, 8192),
    ("one small matrix, many rows", [3001], 2, None, 136, 256),
    ("two matrices of a few tiles", [700, 0, 529], 1, [2, 0, 1], 376, 640),
    ("a matrix of more tiles", [1300], 0, None, 1024, 992),
]
CASES = BF16_CASES + MORE


def cases(unit_width, unit_inner):
    return [pytest.param((n, c, g, o, up(w, unit_width), up(i, unit_inner)), id=n) for n, c, g, o, w, i in CASES]


def setup(epx, case, seed):
    name, cnt, gap, order, N, K = case
    off, R = ref.ranges(cnt, gap, order)
    print(f"[experts8] {name} R={R} n={len(cnt)} N={N} K={K}", flush=True)
    return gen(seed), off, cnt, R, N, K, make_rows(epx, off, cnt, R)


def int8(g, *shape):
    return torch.randint(-128, 128, shape, device="cuda", generator=g, dtype=torch.int32).to(torch.int8)


def scales32(g, *shape):
    return torch.empty(*shape, device="cuda").uniform_(2.0 ** -9, 2.0 ** -7, generator=g)


def kept_guard(R, M):
    return torch.full((R, M), 77, dtype=torch.int8, device="cuda"), torch.full((R, M // 32), 99, dtype=torch.uint8, device="cuda")


def kept_untouched(codes, scales, off, cnt):
    live = torch.zeros(codes.shape[0], dtype=torch.bool, device="cuda")
    for o, c in zip(off, cnt):
        live[o:o + c] = True
    assert bool((codes[~live] == 77).all()) and bool((scales[~live] == 99).all())


def int8_sums(x, w, sx, sw, off, cnt):
    """The product by its definition, float32 by float32; rows of no expert are NaN."""
    z = torch.full((x.shape[0], w.shape[1]), float("nan"), device="cuda")
    for e, (o, c) in enumerate(zip(off, cnt)):
        if c:
            z[o:o + c] = (x[o:o + c].double() @ w[e].double().T).float() * sx[o:o + c, None] * sw[e]
    return z


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("case", cases(8, 16))
def test_int8(epx, case, act):
    g, off, cnt, R, N, K, rows = setup(epx, case, 11)
    M = 2 * N if act == "swiglu" else N
    x, w = int8(g, R, K), int8(g, len(cnt), M, K)
    sx, sw = scales32(g, R) * K ** -0.5, scales32(g, len(cnt), M)
    z = int8_sums(x, w, sx, sw, off, cnt)
    live = ~torch.isnan(z[:, 0])
    out = guard(R, N)
    if act == "none":
        epx.epx_expert_gemm_int8(rows, x, sx, w, sw, out)
        torch.cuda.synchronize()
        r8.same(out[live], z[live].to(torch.bfloat16), "out")
    else:
        epx.epx_expert_gemm_int8(rows, x, sx, w, sw, out, act=epx.ACT_SWIGLU)
        torch.cuda.synchronize()
        a, b = ref.glu(z.double(), torch.zeros_like(z, dtype=torch.float64))
        ref.close(out, a, b, ref.BF16, "out")
    untouched(out, off, cnt, "out")


@pytest.mark.parametrize("case", cases(32, 16))
def test_int8_keeps_preactivations(epx, case):
    g, off, cnt, R, N, K, rows = setup(epx, case, 12)
    x, w = int8(g, R, K), int8(g, len(cnt), 2 * N, K)
    sx, sw = scales32(g, R) * K ** -0.5, scales32(g, len(cnt), 2 * N)
    z = int8_sums(x, w, sx, sw, off, cnt)
    live = ~torch.isnan(z[:, 0])
    out, plain = guard(R, N), guard(R, N)
    codes, scales = kept_guard(R, 2 * N)
    epx.epx_expert_gemm_int8(rows, x, sx, w, sw, out, act=epx.ACT_SWIGLU, preact_codes=codes, preact_scales=scales)
    epx.epx_expert_gemm_int8(rows, x, sx, w, sw, plain, act=epx.ACT_SWIGLU)
    torch.cuda.synchronize()
    want_codes, want_scales = r8.mxint8(z[live])
    r8.same(scales[live], want_scales, "scales")
    r8.same(codes[live], want_codes, "codes")
    assert torch.equal(out, plain)
    kept_untouched(codes, scales, off, cnt)


def test_int8_largest_sums(epx):
    """The longest sum of the largest products, 2^31 - 2^18, in either sign; and one that cancels to 0."""
    K = (1 << 17) - 16
    rows = make_rows(epx, [0], [3], 3)
    x = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((1, 8, K), -128, dtype=torch.int8, device="cuda")
    x[1] = 127
    x[2, ::2], x[2, 1::2] = 127, -127
    sx, sw = torch.ones(3, device="cuda"), torch.ones(1, 8, device="cuda")
    out = guard(3, 8)
    epx.epx_expert_gemm_int8(rows, x, sx, w, sw, out)
    torch.cuda.synchronize()
    want = torch.tensor([[16384.0 * K], [-127 * 128.0 * K], [0.0]], device="cuda").to(torch.bfloat16).repeat(1, 8)
    assert torch.equal(out, want)


def test_int8_scales_of_any_kind(epx):
    """NaN, infinite, zero and negative scales of a row or a column reach that row or column and no other."""
    g = gen(13)
    rows = make_rows(epx, [0], [40], 40)
    x, w = int8(g, 40, 64), int8(g, 1, 128, 64)
    sx, sw = scales32(g, 40), scales32(g, 1, 128)
    sx[3], sx[7], sx[9], sx[11] = float("nan"), float("inf"), 0.0, -1.0
    sw[0, 5], sw[0, 70], sw[0, 80] = float("nan"), float("inf"), 0.0
    out = guard(40, 128)
    epx.epx_expert_gemm_int8(rows, x, sx, w, sw, out)
    z = int8_sums(x, w, sx, sw, [0], [40])
    codes, scales = kept_guard(40, 128)
    half = guard(40, 64)
    epx.epx_expert_gemm_int8(rows, x, sx, w, sw, half, act=epx.ACT_SWIGLU, preact_codes=codes, preact_scales=scales)
    torch.cuda.synchronize()
    r8.same(out, z.to(torch.bfloat16), "out")
    want_codes, want_scales = r8.mxint8(z)
    r8.same(scales, want_scales, "scales")
    r8.same(codes, want_codes, "codes")


def kept_close(codes, scales, z, b, name):
    """What is kept of z, which float32 sums give within b."""
    live = ~torch.isnan(z[:, 0])
    z, b, codes, scales = z[live], b[live], codes[live], scales[live]
    blocks = lambda t: t.view(t.shape[0], t.shape[1] // 32, 32)   # noqa: E731
    amax, slack = blocks(z.abs()).amax(2), blocks(b).amax(2)
    # b - 127 = floor(log2 of the largest magnitude)
    top = torch.exp2(scales.double() - 126)
    assert bool((amax - slack < top).all()) and bool(((amax + slack >= top / 2) | (scales == 0)).all()), name
    step = r8.mxint8_steps(scales).repeat_interleave(32, 1)
    at_most = torch.where(codes.abs() == 127, step, step / 2)   # 127 stands for up to 128
    over = (codes.double() * step - z).abs() - at_most - b * 1.0001
    assert bool((over <= 0).all()), (name, float(over.max()))


@pytest.mark.parametrize("case", cases(32, 8))
def test_keep8(epx, case):
    g, off, cnt, R, N, K, rows = setup(epx, case, 14)
    x, w = rand(g, R, K), rand(g, len(cnt), 2 * N, K, std=K ** -0.5)
    out = guard(R, N)
    codes, scales = kept_guard(R, 2 * N)
    epx.epx_expert_gemm_keep8(rows, x, w, out, codes, scales)
    torch.cuda.synchronize()
    z, b = ref.product(x.double(), w.double(), off, cnt)
    kept_close(codes, scales, z, b, "preact")
    a, ba = ref.glu(z, b)
    ref.close(out, a, ba, ref.BF16, "out")
    untouched(out, off, cnt, "out")
    kept_untouched(codes, scales, off, cnt)


def test_keep8_of_exact_sums(epx):
    """Small whole operands, whose sums float32 holds: what is kept is equal to the rows' quantisation. A row of zeros,
    of infinities and one with a NaN among them."""
    g = gen(15)
    R, N, K = 300, 96, 264
    rows = make_rows(epx, [0, 100], [100, 200], R)
    x = torch.randint(-8, 9, (R, K), device="cuda", generator=g).to(torch.bfloat16)
    w = torch.randint(-8, 9, (2, 2 * N, K), device="cuda", generator=g).to(torch.bfloat16)
    x[5], x[130, 3], x[131, 7] = 0, float("nan"), float("inf")
    out = guard(R, N)
    codes, scales = kept_guard(R, 2 * N)
    epx.epx_expert_gemm_keep8(rows, x, w, out, codes, scales)
    torch.cuda.synchronize()
    x64 = x.double()
    z = torch.cat((x64[:100] @ w[0].double().T, x64[100:] @ w[1].double().T))
    clean = torch.ones(R, dtype=torch.bool, device="cuda")
    clean[130:132] = False
    want_codes, want_scales = r8.mxint8(z[clean])
    r8.same(scales[clean], want_scales, "scales")
    r8.same(codes[clean], want_codes, "codes")
    assert bool((scales[130:132] == 255).all()) and not codes[130:132].any()
    assert not out[5].any() and bool(torch.isnan(out[130].float()).all())


def kept_values(g, R, M, std=1.0):
    return r8.mxint8(rand(g, R, M, std=std).float())


@pytest.mark.parametrize("case", cases(8, 32))
def test_dgrad_kept8(epx, case):
    g, off, cnt, R, N, K, rows = setup(epx, case, 16)
    dy, w = rand(g, R, N), rand(g, len(cnt), N, K, std=N ** -0.5)
    codes, scales = kept_values(g, R, 2 * K, std=1.5)
    dx, act, only = guard(R, 2 * K), guard(R, K), guard(R, 2 * K)
    epx.epx_expert_gemm_dgrad_kept8(rows, dy, w, codes, scales, dx, act_out=act)
    epx.epx_expert_gemm_dgrad_kept8(rows, dy, w, codes, scales, only)
    torch.cuda.synchronize()
    pre = r8.mxint8_values(codes, scales)
    d, b = ref.product(dy.double(), w.double().transpose(1, 2), off, cnt)
    want, bound = ref.glu_backward(d, b, pre)
    ref.close(dx, want, bound, ref.BF16, "dx")
    a, ba = ref.glu(pre, torch.zeros_like(pre))
    dead = torch.isnan(d[:, 0])
    a[dead] = float("nan")
    ref.close(act, a, ba, ref.BF16, "act")
    assert torch.equal(dx, only)
    untouched(dx, off, cnt, "dx")
    untouched(act, off, cnt, "act")


def test_dgrad_kept8_equals_the_one_from_bf16(epx):
    """Kept values are bf16 numbers: the gradient from them in bf16 is the same bits."""
    g = gen(17)
    for R, n, N, K in ((37, 3, 264, 96), (700, 2, 520, 544), (5000, 4, 1032, 2048)):
        cnt = [R // n] * n
        off, total = ref.ranges(cnt, 1)
        rows = make_rows(epx, off, cnt, total)
        dy, w = rand(g, total, N), rand(g, n, N, K, std=N ** -0.5)
        codes, scales = kept_values(g, total, 2 * K)
        pre = r8.mxint8_values(codes, scales).to(torch.bfloat16)
        dx, plain = guard(total, 2 * K), guard(total, 2 * K)
        epx.epx_expert_gemm_dgrad_kept8(rows, dy, w, codes, scales, dx)
        epx.epx_expert_gemm_dgrad(rows, dy, w, plain, input_act=epx.ACT_SWIGLU, preact=pre)
        torch.cuda.synchronize()
        assert torch.equal(dx, plain)


def test_dgrad_kept8_a_nan_block_reaches_its_columns_only(epx):
    g = gen(18)
    R, N, K = 70, 64, 96
    rows = make_rows(epx, [0], [R], R)
    dy, w = rand(g, R, N), rand(g, 1, N, K, std=0.1)
    codes, scales = kept_values(g, R, 2 * K)
    codes[7, 32:64], scales[7, 1] = 0, 255        # gates 32..63 of a row
    dx, act = guard(R, 2 * K), guard(R, K)
    epx.epx_expert_gemm_dgrad_kept8(rows, dy, w, codes, scales, dx, act_out=act)
    torch.cuda.synchronize()
    odd = torch.zeros(R, K, dtype=torch.bool, device="cuda")
    odd[7, 32:64] = True
    assert torch.equal(torch.isnan(act.float()), odd) and torch.equal(torch.isnan(dx.float()), torch.cat((odd, odd), 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f32 added"])
@pytest.mark.parametrize("case", cases(8, 32))
def test_wgrad_kept8(epx, case, dtype):
    g, off, cnt, R, N, K, rows = setup(epx, case, 19)
    dy = rand(g, R, N)
    codes, scales = kept_values(g, R, K)
    v = r8.mxint8_values(codes, scales)
    n = len(cnt)
    dw = guard(n, N, K, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32)
    before = dw.double() if dtype == "f32 added" else None
    epx.epx_expert_gemm_wgrad_kept8(rows, dy, codes, scales, dw, accumulate=dtype == "f32 added")
    torch.cuda.synchronize()
    for e, (o, c) in enumerate(zip(off, cnt)):
        a, b = dy[o:o + c].double(), v[o:o + c]
        want = a.T @ b
        bound = (a.abs().T @ b.abs()) * (ref.SUM * max(1, c))
        if before is not None:
            want = want + before[e]
            bound = bound + 2.0 ** -24 * (want.abs() + bound)
        ref.close(dw[e], want, bound, ref.BF16 if dtype == "bf16" else 0.0, f"dw[{e}]")


def test_wgrad_kept8_what_lies_outside_the_ranges(epx):
    """Rows of no expert hold NaN codes' scales and NaN gradients, and so do columns' neighbours: nothing of it shows."""
    g = gen(20)
    for N, K, cnt in ((72, 96, [5, 0, 33]), (264, 544, [70, 1, 200]), (520, 1056, [600, 300])):
        off, R = ref.ranges(cnt, 3)
        rows = make_rows(epx, off, cnt, R)
        dy = rand(g, R, N)
        codes, scales = kept_values(g, R, K)
        live = torch.zeros(R, dtype=torch.bool, device="cuda")
        for o, c in zip(off, cnt):
            live[o:o + c] = True
        dy[~live] = float("nan")
        scales[~live] = 255
        dw = guard(len(cnt), N, K, dtype=torch.float32)
        epx.epx_expert_gemm_wgrad_kept8(rows, dy, codes, scales, dw)
        torch.cuda.synchronize()
        v = r8.mxint8_values(codes, scales)
        for e, (o, c) in enumerate(zip(off, cnt)):
            a, b = dy[o:o + c].double(), v[o:o + c]
            ref.close(dw[e], a.T @ b, (a.abs().T @ b.abs()) * (ref.SUM * max(1, c)), 0.0, f"dw[{e}]")


def test_wgrad_kept8_a_nan_block_reaches_its_columns_only(epx):
    g = gen(21)
    for R, N, K in ((40, 64, 128), (900, 1032, 1056)):
        rows = make_rows(epx, [0], [R], R)
        dy = rand(g, R, N)
        codes, scales = kept_values(g, R, K)
        codes[R - 3, 64:96], scales[R - 3, 2] = 0, 255
        dw = guard(1, N, K, dtype=torch.float32)
        epx.epx_expert_gemm_wgrad_kept8(rows, dy, codes, scales, dw)
        torch.cuda.synchronize()
        odd = torch.zeros(1, N, K, dtype=torch.bool, device="cuda")
        odd[:, :, 64:96] = True
        assert torch.equal(torch.isnan(dw), odd)


@pytest.mark.parametrize("f32", [False, True])
def test_wgrad_kept8_without_rows(epx, f32):
    rows = make_rows(epx, [0, 0], [0, 0], 0)
    e8, u8 = torch.empty(0, 64, dtype=torch.int8, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda")
    dy = torch.empty(0, 48, dtype=torch.bfloat16, device="cuda")
    dw = guard(2, 48, 64, dtype=torch.float32 if f32 else torch.bfloat16)
    epx.epx_expert_gemm_wgrad_kept8(rows, dy, e8, u8, dw)
    torch.cuda.synchronize()
    assert not dw.any()


def test_ranges_outside_the_buffers_are_empty(epx):
    """As for the bf16 products: a range that is not inside the buffers is neither read nor written."""
    g = gen(22)
    off, cnt, R, N, K = [0, -1, 60, 20], [10, 5, 5, 8], 64, 64, 96
    good, kept = [0, 0, 0, 20], [10, 0, 0, 8]
    rows = make_rows(epx, off, cnt, R)
    x, w = int8(g, R, K), int8(g, 4, 2 * N, K)
    sx, sw = scales32(g, R), scales32(g, 4, 2 * N)
    out = guard(R, N)
    codes, scales = kept_guard(R, 2 * N)
    epx.epx_expert_gemm_int8(rows, x, sx, w, sw, out, act=epx.ACT_SWIGLU, preact_codes=codes, preact_scales=scales)
    bx, bw = rand(g, R, K), rand(g, 4, 2 * N, K, std=0.1)
    bout = guard(R, N)
    c2, s2 = kept_guard(R, 2 * N)
    epx.epx_expert_gemm_keep8(rows, bx, bw, bout, c2, s2)
    dy = rand(g, R, 2 * N)
    xc, xs = kept_values(g, R, K)
    dw = guard(4, 2 * N, K, dtype=torch.float32)
    epx.epx_expert_gemm_wgrad_kept8(rows, dy, xc, xs, dw)
    torch.cuda.synchronize()
    for t in (out, bout):
        untouched(t, good, kept, "out")
    kept_untouched(codes, scales, good, kept)
    kept_untouched(c2, s2, good, kept)
    assert not dw[1:3].any() and bool(dw[0].any()) and bool(dw[3].any())


def test_binding_refuses(epx):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype, device="cuda")   # noqa: E731
    rows = make_rows(epx, [0], [8], 8)
    i8, u8, f = torch.int8, torch.uint8, torch.float32
    good = dict(x=z(8, 64, dtype=i8), x_scales=z(8, dtype=f), w=z(1, 64, 64, dtype=i8), w_scales=z(1, 64, dtype=f), out=z(8, 32),
                act=epx.ACT_SWIGLU, preact_codes=z(8, 64, dtype=i8), preact_scales=z(8, 2, dtype=u8))
    epx.epx_expert_gemm_int8(rows, **good)
    for name, bad in (("x", z(8, 64)), ("x", z(8, 128, dtype=i8)[:, ::2]), ("x_scales", z(8, 1, dtype=f)), ("x_scales", z(7, dtype=f)),
                      ("w", z(1, 32, 64, dtype=i8)), ("w_scales", z(1, 32, dtype=f)), ("w_scales", z(1, 64)), ("out", z(8, 32, dtype=f)),
                      ("out", z(7, 32)), ("preact_codes", z(8, 32, dtype=i8)), ("preact_codes", None), ("preact_scales", None),
                      ("preact_scales", z(8, 64, dtype=u8)), ("preact_codes", z(8, 64, dtype=u8)), ("x", z(8, 64, dtype=i8).cpu())):
        with pytest.raises(ValueError):
            epx.epx_expert_gemm_int8(rows, **{**good, name: bad})
    with pytest.raises(epx.EpxError):      # without the activation there is nothing to keep
        epx.epx_expert_gemm_int8(rows, **{**good, "act": epx.ACT_NONE, "w": z(1, 32, 64, dtype=i8), "w_scales": z(1, 32, dtype=f),
                                          "preact_codes": z(8, 32, dtype=i8), "preact_scales": z(8, 1, dtype=u8)})
    with pytest.raises(ValueError):
        epx.epx_expert_gemm_keep8(rows, z(8, 64), z(1, 64, 64), z(8, 32), z(8, 64), z(8, 2, dtype=u8))
    with pytest.raises(ValueError):
        epx.epx_expert_gemm_dgrad_kept8(rows, z(8, 64), z(1, 64, 32), z(8, 64, dtype=i8), z(8, 1, dtype=u8), z(8, 64))
    with pytest.raises(ValueError):
        epx.epx_expert_gemm_wgrad_kept8(rows, z(8, 64), z(8, 48, dtype=i8), z(8, 1, dtype=u8), z(1, 64, 48))
    with pytest.raises(ValueError):
        epx.epx_int8_quantize(z(8, 24), z(8, 24, dtype=i8), z(8, dtype=f))
    with pytest.raises(ValueError):
        epx.epx_mxint8_quantize(z(8, 48), z(8, 48, dtype=i8), z(8, 1, dtype=u8))
    torch.cuda.synchronize()


