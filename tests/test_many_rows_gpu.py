"""Buffers of 10^9 rows and more, of which the ranges take a few at both ends,
and offsets that pass 32 bits in every call."""
import ctypes

import pytest
import torch

from tests import exact_sums as ex
from tests import experts_reference as ref
from tests.test_experts_gpu import epx, make_rows  # noqa: F401

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 4096


def buffer(rows, columns):
    """Uninitialised: only the rows of the ranges are written and read."""
    if torch.cuda.get_device_properties(0).total_memory < 200 << 30:
        pytest.skip("needs 70 GB")
    return torch.empty(rows, columns, dtype=torch.bfloat16, device="cuda")


@pytest.fixture(autouse=True)
def release():
    yield
    torch.cuda.empty_cache()


def test_products_on_2_to_the_30_rows(epx):  # noqa: F811
    R, cnt = 1 << 30, [3, 0, 300, 70]
    off = [5, 0, R - 300, 1 << 29]
    g = ex.gen(61, "cuda")
    x, w = ex.along_rows(g, sum(cnt), 8), ex.matrices(g, 4, 8, 8)
    src, dst = buffer(R, 8), buffer(R, 8)
    at = 0
    for o, c in zip(off, cnt):
        src[o:o + c] = x[at:at + c]
        dst[max(0, o - 2):o + c + 2] = -7.25
        at += c
    rows = make_rows(epx, off, cnt, R)
    for forward in (True, False):
        if forward:
            epx.epx_expert_gemm(rows, src, w, dst)
        else:
            epx.epx_expert_gemm_dgrad(rows, src, w.transpose(1, 2).contiguous(), dst)
        torch.cuda.synchronize()
        at = 0
        for e, (o, c) in enumerate(zip(off, cnt)):
            assert torch.equal(dst[o:o + c].double(), x[at:at + c].double() @ w[e].double().T), (forward, e)
            if c:
                assert bool((dst[o - 2:o] == -7.25).all()) and bool((dst[o + c:o + c + 2] == -7.25).all())
            dst[o:o + c] = 0
            at += c


def test_weight_gradient_on_the_most_rows(epx):  # noqa: F811
    cnt = [2001, 0, 40, 5]
    off = [MOST - 2001, 0, 1 << 30, 3]
    g = ex.gen(62, "cuda")
    rows = make_rows(epx, off, cnt, MOST)
    dy, x = buffer(MOST, 8), buffer(MOST, 8)
    small = ex.down_columns(g, sum(cnt), 8, 8, [0, 0, 2001, 2041], cnt)
    at = 0
    for o, c in zip(off, cnt):
        dy[o:o + c], x[o:o + c] = small[0][at:at + c], small[1][at:at + c]
        at += c
    dw = torch.full((4, 8, 8), -7.25, device="cuda")
    epx.epx_expert_gemm_wgrad(rows, dy, x, dw)
    torch.cuda.synchronize()
    for e, (o, c) in enumerate(zip(off, cnt)):
        assert torch.equal(dw[e].double(), dy[o:o + c].double().T @ x[o:o + c].double()), e


def test_more_tiles_than_a_launch_takes(epx):  # noqa: F811
    """Turned down on the host (the addresses are never read), and the next call is not affected."""
    A = 0x200000
    r = epx.epx_expert_rows(1, MOST, A, A + 0x1000)
    assert epx._lib.epx_expert_gemm(ctypes.byref(r), A, A + 0x10000, 8, 8, 0, None, A + 0x20000, None) == 4
    assert epx._lib.epx_expert_gemm_dgrad(ctypes.byref(r), A, A + 0x10000, 8, 8, 0, None, A + 0x20000, None) == 4
    assert epx._lib.epx_expert_gemm_mxfp4(ctypes.byref(r), A, A + 0x10000, A + 0x20000, A + 0x30000, 8, 128, 0, 0, A + 0x40000,
                                          None, None) == 4
    g = ex.gen(63, "cuda")
    x, w = ex.along_rows(g, 5, 64), ex.matrices(g, 1, 8, 64)
    out = torch.empty(5, 8, dtype=torch.bfloat16, device="cuda")
    epx.epx_expert_gemm(make_rows(epx, [0], [5], 5), x, w, out)
    torch.cuda.synchronize()
    assert torch.equal(out.double(), x.double() @ w[0].double().T)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_router_at_the_most_tokens(epx, dtype):  # noqa: F811
    """2^24 tokens of 260 experts: more than 2^32 logits."""
    T, E, k = 1 << 24, 260, 5
    p = epx.make_problem(T, k, E, 1, 1)
    if torch.cuda.get_device_properties(0).total_memory < 200 << 30:
        pytest.skip("needs 70 GB")
    l, d = torch.empty(T, E, dtype=dtype, device="cuda"), torch.empty(T, E, dtype=dtype, device="cuda")
    l.fill_(-1.0)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    dw = torch.zeros(T, k, device="cuda")
    g = ex.gen(64, "cuda")
    for part in (slice(0, 64), slice(T // 2 - 3, T // 2 + 61), slice(T - 64, T)):
        l[part] = torch.randn(64, E, generator=g, device="cuda").to(dtype)
        dw[part] = torch.randn(64, k, generator=g, device="cuda")
    epx.epx_route(p, l, epx.SCORE_SOFTMAX, idx, w)
    epx.epx_route_backward(p, l, epx.SCORE_SOFTMAX, idx, dw, d)
    torch.cuda.synchronize()
    for part in (slice(0, 64), slice(T // 2 - 3, T // 2 + 61), slice(T - 64, T)):
        x = l[part].double()
        at = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(idx[part].long(), at)
        want = torch.softmax(x.gather(1, at), 1)
        assert float((w[part].double() - want).abs().max()) <= 2.0 ** -20
        grad = want * (dw[part].double() - (want * dw[part].double()).sum(1, keepdim=True))
        got = d[part].double()
        half = ref.BF16 if dtype == torch.bfloat16 else 2.0 ** -24
        # a few float32 steps of the largest |dw| (below 8), and half a step of the type
        assert bool(((got.gather(1, at) - grad).abs() <= 8 * 2.0 ** -19 + half * grad.abs()).all())
        assert not got.scatter(1, at, 0.0).any()


def test_combine_gradient_past_32_bits(epx):  # noqa: F811
    """70000 tokens, top-8, 8200 channels: 4.6 * 10^9 elements of y."""
    T, k, E, h = 70000, 8, 16, 8200
    g = ex.gen(65, "cuda")
    p = epx.make_problem(T, k, E, 1, 1)
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32).contiguous()
    L = epx.Layout(p)
    epx.epx_get_layout(p, idx, L)
    y, dy, dout = buffer(T * k, h), buffer(T * k, h), torch.empty(T, h, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y.normal_(generator=g)
    w, dw = torch.rand(T, k, generator=g, device="cuda"), torch.empty(T, k, device="cuda")
    epx.epx_combine_backward(p, L, dout, y, w, dy, dw)
    torch.cuda.synchronize()
    slot = L["slot"].view(T, k).long()
    assert int(slot.max()) * h > 1 << 32
    for part in (slice(0, 500), slice(T - 500, T)):
        at = slot[part]
        assert torch.equal(dy[at], (w[part].unsqueeze(2) * dout[part].float().unsqueeze(1)).to(torch.bfloat16))
        prod = y[at].double() * dout[part].double().unsqueeze(1)
        assert bool(((dw[part].double() - prod.sum(2)).abs() <= prod.abs().sum(2) * (h * 2.0 ** -24)).all())


def test_4_bit_conversion_past_32_bits(epx):  # noqa: F811
    R, K = (1 << 20) + 5, 4160   # 4.4 * 10^9 values
    x = buffer(R, K)
    x.normal_(generator=ex.gen(66, "cuda"))
    codes, scales = torch.empty(R, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(R, K // 32, dtype=torch.uint8, device="cuda")
    epx.epx_mxfp4_quantize(x, codes, scales)
    back = buffer(R, K)
    epx.epx_mxfp4_dequantize(codes, scales, back)
    torch.cuda.synchronize()
    for part in (slice(0, 700), slice(R - 700, R)):
        c, s = ref.mxfp4_quantize(x[part])
        assert torch.equal(codes[part], c) and torch.equal(scales[part], s)
        assert torch.equal(back[part].double(), ref.mxfp4_values(c, s))


def test_4_bit_product_past_32_bits(epx):  # noqa: F811
    """Rows behind 2^32 bytes of codes, and experts whose weights start there."""
    R, n, N, K = (1 << 20) + 77, 700, 3080, 4096
    cnt, off = [0] * n, [0] * n
    for e, c, o in ((0, 9, 3), (350, 200, 1 << 19), (698, 33, R - 100), (699, 60, R - 60)):
        cnt[e], off[e] = c, o
    g = ex.gen(67, "cuda")
    rows = make_rows(epx, off, cnt, R)
    x, out = torch.empty(R, K, dtype=torch.uint8, device="cuda"), torch.empty(R, N, dtype=torch.bfloat16, device="cuda")
    xs = torch.empty(R, K // 128, device="cuda")
    w, ws = torch.empty(n, N, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(n, N, K // 32, dtype=torch.uint8, device="cuda")
    assert w.numel() > 1 << 32 and x.numel() > 1 << 32
    live = [e for e in range(n) if cnt[e]]
    parts = {e: ex.fp8_and_4_bit(g, 1, N, cnt[e], K) for e in live}
    for e in live:
        at = slice(off[e], off[e] + cnt[e])
        x[at], xs[at], w[e], ws[e] = parts[e][0], parts[e][1], parts[e][2][0], parts[e][3][0]
    epx.epx_expert_gemm_mxfp4(rows, x, xs, w, ws, out)
    torch.cuda.synchronize()
    for e in live:
        cx, cs, cw, cws = parts[e]
        want = (cx.view(torch.float8_e4m3fn).double() * cs[:, :1].double()) @ ref.mxfp4_values(cw, cws)[0].T
        assert torch.equal(out[off[e]:off[e] + cnt[e]].double(), want), e
