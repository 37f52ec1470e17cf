"""The experts' products on operands with one right result: every bit of every
sum counts (tests/test_exact_sums.py shows what these operands catch)."""
import pytest
import torch

from tests import exact_sums as ex
from tests import experts_reference as ref
from tests.test_experts_gpu import CASES, GUARD, epx, guard, make_rows, untouched  # noqa: F401
from tests.test_mxfp4_gpu import CASES as MX_CASES

pytestmark = pytest.mark.gpu
LONG = [("one expert, many rows", [15000], 1, None, 136, 264), ("three experts, many rows", [4001, 0, 3998], 2, None, 264, 392),
        ("large tiles, long sum, many rows", [2048, 1500], 0, None, 1032, 4104)]
IDS = [c[0] for c in CASES + LONG]


def setup(epx, case):  # noqa: F811
    name, cnt, gap, order, N, K = case
    off, R = ref.ranges(cnt, gap, order)
    print(f"[exact] {name} R={R} n={len(cnt)} N={N} K={K}", flush=True)
    return ex.gen(R + N + K, "cuda"), off, cnt, R, N, K, make_rows(epx, off, cnt, R)


def same(got, want, name):
    live = ~torch.isnan(want)
    bad = (got.double() != want) & live
    assert not bad.any(), (name, int(bad.sum()), got[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.mark.parametrize("case", CASES + LONG, ids=IDS)
def test_forward(epx, case):  # noqa: F811
    g, off, cnt, R, N, K, rows = setup(epx, case)
    x, w = ex.along_rows(g, R, K), ex.matrices(g, len(cnt), N, K)
    out = guard(R, N)
    epx.epx_expert_gemm(rows, x, w, out)
    torch.cuda.synchronize()
    same(out, ex.by_expert(x, w, off, cnt), "out")
    untouched(out, off, cnt, "out")


@pytest.mark.parametrize("case", CASES + LONG, ids=IDS)
def test_gated_forward(epx, case):  # noqa: F811
    """Rows in sixteenths, so that gates stay within 16."""
    g, off, cnt, R, N, K, rows = setup(epx, case)
    x, w = ex.along_rows(g, R, K, 2.0 ** -4), ex.matrices(g, len(cnt), 2 * N, K)
    out, pre = guard(R, N), guard(R, 2 * N)
    epx.epx_expert_gemm(rows, x, w, out, act=epx.ACT_SWIGLU, preact=pre)
    torch.cuda.synchronize()
    z = ex.by_expert(x, w, off, cnt)
    same(pre, z, "preact")
    ref.close(out, *ref.glu(z, torch.zeros_like(z)), ref.BF16, "out")


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("case", CASES + LONG, ids=IDS)
def test_input_gradient(epx, case, act):  # noqa: F811
    g, off, cnt, R, N, K, rows = setup(epx, case)
    dy, wt = ex.along_rows(g, R, N), ex.matrices(g, len(cnt), K, N)
    w = wt.transpose(1, 2).contiguous()
    d = ex.by_expert(dy, wt, off, cnt)
    if act == "none":
        dx = guard(R, K)
        epx.epx_expert_gemm_dgrad(rows, dy, w, dx)
        torch.cuda.synchronize()
        same(dx, d, "dx")
    else:
        pre = torch.empty(R, 2 * K, dtype=torch.bfloat16, device="cuda").normal_(0, 2, generator=g)
        dx = guard(R, 2 * K)
        epx.epx_expert_gemm_dgrad(rows, dy, w, dx, input_act=epx.ACT_SWIGLU, preact=pre)
        torch.cuda.synchronize()
        ref.close(dx, *ref.glu_backward(d, torch.zeros_like(d), pre.double()), ref.BF16, "dx")
    untouched(dx, off, cnt, "dx")


@pytest.mark.parametrize("kind", ["bf16", "f32", "accumulate"])
@pytest.mark.parametrize("case", CASES + LONG, ids=IDS)
def test_weight_gradient(epx, case, kind):  # noqa: F811
    g, off, cnt, R, N, K, rows = setup(epx, case)
    dy, x = ex.down_columns(g, R, N, K, off, cnt)
    dw = guard(len(cnt), N, K, dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
    base = torch.zeros(len(cnt), N, K, device="cuda")
    if kind == "accumulate":
        base = ex.whole(g, -(1 << 22), 1 << 22, len(cnt), N, K)
        dw.copy_(base)
    epx.epx_expert_gemm_wgrad(rows, dy, x, dw, accumulate=kind == "accumulate")
    torch.cuda.synchronize()
    for e, (o, c) in enumerate(zip(off, cnt)):
        same(dw[e], dy[o:o + c].double().T @ x[o:o + c].double() + base[e].double(), ("dw", e))


def test_rows_of_other_ranges_do_not_enter_a_weight_gradient(epx):  # noqa: F811
    """Rows before, between and behind the ranges hold NaN and infinities."""
    case = ("gaps", [33, 0, 130, 257, 1], 5, None, 264, 136)
    g, off, cnt, R, N, K, rows = setup(epx, case)
    dy, x = ex.down_columns(g, R, N, K, off, cnt)
    live = torch.zeros(R, dtype=torch.bool, device="cuda")
    for o, c in zip(off, cnt):
        live[o:o + c] = True
    dy[~live], x[~live] = float("nan"), float("inf")
    dw, dx, out = guard(5, N, K, dtype=torch.float32), guard(R, K), guard(R, N)
    w = ex.matrices(g, 5, N, K)
    epx.epx_expert_gemm_wgrad(rows, dy, x, dw)
    epx.epx_expert_gemm(rows, x, w, out)
    epx.epx_expert_gemm_dgrad(rows, dy, w, dx)
    torch.cuda.synchronize()
    for e, (o, c) in enumerate(zip(off, cnt)):
        same(dw[e], dy[o:o + c].double().T @ x[o:o + c].double(), ("dw", e))
    assert torch.isfinite(out).all() and torch.isfinite(dx).all()
    untouched(out, off, cnt, "out")
    untouched(dx, off, cnt, "dx")


MX = MX_CASES + [("one expert, long sum", [70], 0, None, 264, 7168), ("large tiles, long sum", [700, 600], 0, None, 1032, 3968)]


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("case", MX, ids=[c[0] for c in MX])
def test_fp8_rows_and_4_bit_weights(epx, case, act):  # noqa: F811
    g, off, cnt, R, N, K, rows = setup(epx, case)
    M = 2 * N if act == "swiglu" else N
    x, xs, w, ws = ex.fp8_and_4_bit(g, len(cnt), M, R, K)
    if act == "swiglu":
        xs = xs * 2.0 ** -3   # gates within some tens
    out = guard(R, N)
    epx.epx_expert_gemm_mxfp4(rows, x, xs, w, ws, out, act=epx.ACT_SWIGLU if act == "swiglu" else epx.ACT_NONE)
    torch.cuda.synchronize()
    v = x.view(torch.float8_e4m3fn).double() * xs[:, :1].double()
    z = ex.by_expert(v, ref.mxfp4_values(w, ws), off, cnt)
    if act == "none":
        same(out, z, "out")
    else:
        ref.close(out, *ref.glu(z, torch.zeros_like(z)), ref.BF16, "out")
    untouched(out, off, cnt, "out")


@pytest.mark.parametrize("case", [c for c in MX if c[4] % 128 == 0] + [
    ("decode", [0, 3, 17, 1], 2, None, 384, 640), ("more rows", [130, 257, 3], 0, None, 640, 256),
    ("large tiles", [(i * 53) % 300 for i in range(150)], 1, None, 384, 256),
    ("few tiles, 21 blocks", [70, 3], 1, None, 256, 2688)], ids=lambda c: c[0])
def test_fp8_rows_out(epx, case):  # noqa: F811
    """Scales are the largest magnitude of 128 over 448, exactly; codes are within half a step."""
    g, off, cnt, R, N, K, rows = setup(epx, case)
    x, xs, w, ws = ex.fp8_and_4_bit(g, len(cnt), N, R, K)
    out = torch.full((R, N), 0xA5, dtype=torch.uint8, device="cuda")
    osc = torch.full((R, N // 128), GUARD, device="cuda")
    epx.epx_expert_gemm_mxfp4(rows, x, xs, w, ws, out, out_scales=osc)
    torch.cuda.synchronize()
    z = ex.by_expert(x.view(torch.float8_e4m3fn).double() * xs[:, :1].double(), ref.mxfp4_values(w, ws), off, cnt)
    live = ~torch.isnan(z[:, 0])
    zb = z[live].view(-1, N // 128, 128)
    # in 64 bits: torch divides a float32 tensor by a number through its reciprocal, a step off at times (and no
    # quotient by 448 = 7 * 64 is near the middle of two float32 numbers: its bits repeat after three)
    s = (zb.abs().amax(2) / 448.0).float()
    assert torch.equal(osc[live], s)
    v = out[live].view(torch.float8_e4m3fn).double().view_as(zb) * s.double().unsqueeze(2)
    # the quotient's rounding to float32, then half a step: 2^-4 of the value, 2^-10 below the normal numbers
    assert bool(((v - zb).abs() <= zb.abs() * (2.0 ** -4 + 2.0 ** -23) + s.double().unsqueeze(2) * 2.0 ** -10).all())


def window(places, values, big):
    """One row and one column of 256 codes: `big` = 4 * x at place 0 and taken off again at place 128, and
    0.5 * values[i] at places[i]; the result without the pair, in float64, and the operands."""
    x, w = torch.zeros(1, 256, device="cuda"), torch.zeros(256, dtype=torch.long, device="cuda")
    x[0, 0], x[0, 128], w[0], w[128] = big / 4, big / 4, 6, 14
    x[0, places], w[places] = torch.tensor(values, device="cuda"), 1
    q = x.to(torch.float8_e4m3fn)
    codes = (w[0::2] | (w[1::2] << 4)).to(torch.uint8).expand(1, 8, 128).contiguous()
    scales = torch.full((1, 8, 8), 127, dtype=torch.uint8, device="cuda")
    return q.view(torch.uint8), torch.ones(1, 2, device="cuda"), codes, scales, 0.5 * q[0, places].double().sum()


@pytest.mark.parametrize("place", [1, 5, 7, 8, 15, 16, 31, 32, 64, 100, 127, 129, 135, 136])
def test_what_the_matrix_instruction_cuts(epx, place):  # noqa: F811
    """Beside 2^10 in the same eight of a sum a product keeps its bits from 2^-3 on; elsewhere all of them that a
    float32 sum of 2^10 holds."""
    rows = make_rows(epx, [0], [1], 1)
    near = place // 8 in (0, 16)
    for value in (2.0 ** -2, 1.75, 2.0 ** -3, 1.125 * 2.0 ** -2, 1.875 * 2.0 ** -5, 2.0 ** -6, 13.0, -(2.0 ** -2), -1.875 * 2.0 ** -3):
        x, xs, w, ws, want = window([place], [value], 1024.0)
        out = guard(1, 8)
        epx.epx_expert_gemm_mxfp4(rows, x, xs, w, ws, out)
        torch.cuda.synchronize()
        unit = 2.0 ** -3 if near else 2.0 ** -13
        assert torch.equal(out[0].double(), (torch.trunc(want / unit) * unit).expand(8)), (place, value)


def test_bound_of_the_cut(epx):  # noqa: F811
    """Any operands: the result is off by less than 7 * 2^-13 of the largest product of every eight, and float32's sums."""
    g = ex.gen(40, "cuda")
    R, N, K = 48, 72, 1024
    rows = make_rows(epx, [0], [R], R)
    far = torch.exp2(torch.randint(-8, 9, (R, K), generator=g, device="cuda").float())
    x = (torch.randn(R, K, generator=g, device="cuda") * far).clamp(-448, 448)
    # the second half takes the first half's sum away: the same products in other eights
    x[:, K // 2:] = x[:, :K // 2].roll(4, 1)
    x = x.to(torch.float8_e4m3fn)
    w = torch.randint(0, 16, (1, N, K // 2), generator=g, device="cuda")
    w = torch.cat((w, w.roll(4, 2) ^ 8), 2)
    codes = (w[..., 0::2] | (w[..., 1::2] << 4)).to(torch.uint8)
    scales = torch.full((1, N, K // 32), 127, dtype=torch.uint8, device="cuda")
    out = guard(R, N)
    epx.epx_expert_gemm_mxfp4(rows, x.view(torch.uint8), torch.ones(R, K // 128, device="cuda"), codes, scales, out)
    torch.cuda.synchronize()
    p = x.double()[:, None, :] * ref.mxfp4_values(codes, scales)[0][None]
    want = p.sum(2)
    largest = p.abs().view(R, N, K // 8, 8).amax(3).sum(2)
    bound = 7 * 2.0 ** -13 * largest + K / 8 * 2.0 ** -24 * p.abs().sum(2)
    assert bool(((out.double() - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)).all())


def test_gates_far_below_zero(epx):  # noqa: F811
    """silu and its gradient for gates down to -400: below -87 the reciprocal is no
    normal float32 number any more and the result is 0, which is off by less than 88 * 2^-126 < 2^-119 times the other factors."""
    gates = -torch.cat((torch.arange(0, 128, device="cuda") * 1.0, 80 + torch.arange(0, 40, device="cuda") * 0.5,
                        torch.tensor([150.0, 200.0, 400.0], device="cuda"))).to(torch.bfloat16)
    R, N, K = gates.numel(), 40, 8
    rows = make_rows(epx, [0], [R], R)
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = gates, 1.0
    ups = (torch.arange(N, device="cuda") - 20.0).to(torch.bfloat16)
    w = torch.zeros(1, 2 * N, K, dtype=torch.bfloat16, device="cuda")
    w[0, :N, 0], w[0, N:, 1] = 1.0, ups
    out, pre = guard(R, N), guard(R, 2 * N)
    epx.epx_expert_gemm(rows, x, w, out, act=epx.ACT_SWIGLU, preact=pre)
    torch.cuda.synchronize()
    same(pre, torch.cat((gates.double()[:, None].expand(R, N), ups.double().expand(R, N)), 1), "preact")
    z = pre.double()
    lost = 2.0 ** -119 * (ups.double().abs() + 1)
    a, b = ref.glu(z, torch.zeros_like(z))
    ref.close(out, a, b + lost, ref.BF16, "out")
    # the gradient of preact for d = 3
    dy, wd = torch.full((R, 8), 3.0, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 8, N, dtype=torch.bfloat16, device="cuda")
    wd[0, 0] = 1.0
    dx = guard(R, 2 * N)
    epx.epx_expert_gemm_dgrad(rows, dy, wd, dx, input_act=epx.ACT_SWIGLU, preact=pre)
    torch.cuda.synchronize()
    d, bd = ref.glu_backward(torch.full((R, N), 3.0, dtype=torch.float64, device="cuda"), torch.zeros(R, N, dtype=torch.float64, device="cuda"), z)
    ref.close(dx, d, bd + 3 * torch.cat((lost, lost)), ref.BF16, "dx")
