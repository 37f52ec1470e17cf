"""Buffers of more than 2^31 values in the calls on 8-bit rows: the ranges take
a few rows at both ends, so that offsets pass 32 bits."""
import pytest
import torch

from tests import experts_reference as ref
from tests import rows8_reference as r8
from tests.test_experts8_gpu import int8, int8_sums, kept_values, scales32
from tests.test_experts_gpu import epx, gen, make_rows, rand  # noqa: F401

pytestmark = pytest.mark.gpu
WIDE, ROWS = 1 << 15, 70_000   # 2.3 * 10^9 values
CNT = [37, 0, 70]
OFF = [2, 0, ROWS - 72]


@pytest.fixture(autouse=True)
def release():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 30 GB")
    yield
    torch.cuda.empty_cache()


def big(*shape, dtype):
    """Uninitialised: only some of its rows are written and read."""
    return torch.empty(*shape, dtype=dtype, device="cuda")


def parts():
    return [(e, slice(o, o + c)) for e, (o, c) in enumerate(zip(OFF, CNT))]


def test_int8(epx):  # noqa: F811
    g = gen(71)
    rows = make_rows(epx, OFF, CNT, ROWS)
    x, w, sx, sw = big(ROWS, WIDE, dtype=torch.int8), int8(g, 3, 64, WIDE), scales32(g, ROWS), scales32(g, 3, 64)
    for _, r in parts():
        x[r] = int8(g, r.stop - r.start, WIDE)
    out = torch.full((ROWS, 64), 3.5, dtype=torch.bfloat16, device="cuda")
    epx.epx_expert_gemm_int8(rows, x, sx, w, sw, out)
    torch.cuda.synchronize()
    for e, r in parts():
        if CNT[e]:
            want = int8_sums(x[r], w[e:e + 1], sx[r], sw[e:e + 1], [0], [CNT[e]])
            r8.same(out[r], want.to(torch.bfloat16), e)
    assert bool((out[39:ROWS - 72] == 3.5).all())


@pytest.mark.parametrize("form", ["int8", "keep8"])
def test_kept_preactivations(epx, form):  # noqa: F811
    g = gen(72)
    N, K = WIDE // 2, 32
    rows = make_rows(epx, OFF, CNT, ROWS)
    codes, scales = big(ROWS, 2 * N, dtype=torch.int8), big(ROWS, 2 * N // 32, dtype=torch.uint8)
    out = big(ROWS, N, dtype=torch.bfloat16)
    for t in (codes, scales, out):
        t[:2], t[39:41], t[ROWS - 74:ROWS - 72], t[-2:] = 7, 7, 7, 7
    if form == "int8":
        x, w, sx, sw = int8(g, ROWS, K), int8(g, 3, 2 * N, K), scales32(g, ROWS), scales32(g, 3, 2 * N)
        epx.epx_expert_gemm_int8(rows, x, sx, w, sw, out, act=epx.ACT_SWIGLU, preact_codes=codes, preact_scales=scales)
    else:
        # whole operands, whose sums are exact
        x = torch.randint(-8, 9, (ROWS, K), device="cuda", generator=g).to(torch.bfloat16)
        w = torch.randint(-8, 9, (3, 2 * N, K), device="cuda", generator=g).to(torch.bfloat16)
        epx.epx_expert_gemm_keep8(rows, x, w, out, codes, scales)
    torch.cuda.synchronize()
    for e, r in parts():
        if CNT[e]:
            z = (int8_sums(x[r], w[e:e + 1], sx[r], sw[e:e + 1], [0], [CNT[e]]) if form == "int8"
                 else x[r].double() @ w[e].double().T)
            want_codes, want_scales = r8.mxint8(z)
            r8.same(scales[r], want_scales, e)
            r8.same(codes[r], want_codes, e)
    for t in (codes, scales, out):
        for s in (slice(0, 2), slice(39, 41), slice(ROWS - 74, ROWS - 72), slice(ROWS - 2, ROWS)):
            assert bool((t[s] == 7).all())


def test_gradients(epx):  # noqa: F811
    g = gen(73)
    N, K = 32, WIDE
    rows = make_rows(epx, OFF, CNT, ROWS)
    codes, scales = big(ROWS, K, dtype=torch.int8), big(ROWS, K // 32, dtype=torch.uint8)
    dy = rand(g, ROWS, N)
    for _, r in parts():
        codes[r], scales[r] = kept_values(g, r.stop - r.start, K)
    dw = torch.empty(3, N, K, device="cuda")
    epx.epx_expert_gemm_wgrad_kept8(rows, dy, codes, scales, dw)
    # the same buffers as pre-activations of half as many columns
    w, dx = rand(g, 3, N, K // 2, std=0.2), big(ROWS, K, dtype=torch.bfloat16)
    act = big(ROWS, K // 2, dtype=torch.bfloat16)
    epx.epx_expert_gemm_dgrad_kept8(rows, dy, w, codes, scales, dx, act_out=act)
    torch.cuda.synchronize()
    for e, r in parts():
        v, d = r8.mxint8_values(codes[r], scales[r]), dy[r].double()
        ref.close(dw[e], d.T @ v, (d.abs().T @ v.abs()) * (ref.SUM * max(1, CNT[e])), 0.0, e)
        s = d @ w[e].double()
        want, bound = ref.glu_backward(s, (d.abs() @ w[e].double().abs()) * (ref.SUM * N), v)
        ref.close(dx[r], want, bound, ref.BF16, e)
        a, ba = ref.glu(v, torch.zeros_like(v))
        ref.close(act[r], a, ba, ref.BF16, e)


@pytest.mark.parametrize("form", ["int8", "mxint8"])
def test_conversions(epx, form):  # noqa: F811
    g = gen(74)
    x = big(ROWS, WIDE, dtype=torch.bfloat16)
    x.zero_()
    x[-40:] = rand(g, 40, WIDE)
    codes = big(ROWS, WIDE, dtype=torch.int8)
    scales = big(ROWS, dtype=torch.float32) if form == "int8" else big(ROWS, WIDE // 32, dtype=torch.uint8)
    getattr(epx, f"epx_{form}_quantize")(x, codes, scales)
    want_codes, want_scales = (r8.int8_rows if form == "int8" else r8.mxint8)(x[-40:])
    r8.same(codes[-40:], want_codes, "codes")
    r8.same(scales[-40:], want_scales, "scales")
    assert not codes[:-40].any() and not scales[:-40].any()
    x.fill_(3.5)
    getattr(epx, f"epx_{form}_dequantize")(codes, scales, x)
    torch.cuda.synchronize()
    want = ((codes[-40:].float() * scales[-40:].unsqueeze(1)).to(torch.bfloat16) if form == "int8"
            else r8.mxint8_values(codes[-40:], scales[-40:]))
    r8.same(x[-40:], want, "values")
    assert not x[:-40].any()
