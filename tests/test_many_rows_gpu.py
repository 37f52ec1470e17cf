"""Buffers of 10^9 rows and more, of which the ranges take a few at both ends."""
import ctypes

import pytest
import torch

from tests import exact_sums as ex
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
