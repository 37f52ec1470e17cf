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
