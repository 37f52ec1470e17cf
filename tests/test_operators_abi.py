"""Refusals of the router, the experts' products, 4-bit conversion and combine's
gradient: every bad argument is turned down on the host, before anything is
launched (so these run without a GPU; the addresses are never read)."""
import ctypes

import pytest
import torch

A = 0x200000   # a 16-byte aligned address


@pytest.fixture(scope="module")
def epx():
    from combine_epx_get_amd import epx as mod
    return mod


@pytest.fixture(scope="module")
def lib(epx):
    return epx._lib


def by(x):
    return ctypes.byref(x)


def rows(epx, n=4, R=64, off=A, cnt=A + 0x1000):
    return epx.epx_expert_rows(n, R, off, cnt)


def layout(epx):
    ptrs = [None if f in epx.RELAY_FIELDS else 0x100000 + 0x1000 * i for i, f in enumerate(epx.LAYOUT_FIELDS)]
    return epx.epx_layout(*ptrs)


def test_route(epx, lib):
    p = epx.make_problem(64, 2, 16, 1, 1)
    ok = dict(logits=A, dtype=2, score=0, bias=None, renorm=1, scale=1.0, idx=A, w=A)

    def call(problem=p, **k):
        a = {**ok, **k}
        return lib.epx_route(by(problem), a["logits"], a["dtype"], a["score"], a["bias"], a["renorm"], a["scale"],
                             a["idx"], a["w"], None)

    for bad in (dict(dtype=1), dict(dtype=3), dict(score=2), dict(score=-1), dict(renorm=2), dict(renorm=-1),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(logits=None), dict(logits=A + 4),
                dict(bias=A), dict(score=1, bias=A + 2), dict(idx=None), dict(w=None), dict(idx=A + 2), dict(w=A + 1)):
        assert call(**bad) == 1, bad
    assert call(problem=epx.make_problem(64, 17, 16, 1, 1)) == 1
    assert call(problem=epx.make_problem(64, 65, 128, 1, 1)) == 1
    assert call(problem=epx.make_problem(64, 2, 4096, 1, 1)) == 1
    assert call(problem=epx.make_problem(-1, 2, 16, 1, 1)) == 1
    assert lib.epx_route(None, A, 2, 0, None, 1, 1.0, A, A, None) == 1
    assert call(problem=epx.make_problem(0, 2, 16, 1, 1), logits=None, idx=None, w=None) == 0


def test_route_backward(epx, lib):
    p = epx.make_problem(64, 2, 16, 1, 1)
    ok = dict(logits=A, dtype=0, score=1, renorm=0, scale=1.0, idx=A, dw=A, d=A + 0x1000)

    def call(problem=p, **k):
        a = {**ok, **k}
        return lib.epx_route_backward(by(problem), a["logits"], a["dtype"], a["score"], a["renorm"], a["scale"],
                                      a["idx"], a["dw"], a["d"], None)

    for bad in (dict(dtype=1), dict(score=2), dict(renorm=3), dict(scale=float("-inf")), dict(logits=None),
                dict(logits=A + 8), dict(idx=None), dict(dw=None), dict(d=None), dict(d=A + 0x1004), dict(d=A)):
        assert call(**bad) == 1, bad
    assert call(problem=epx.make_problem(0, 2, 16, 1, 1), logits=None) == 0


def test_combine_backward(epx, lib):
    p, L = epx.make_problem(64, 2, 16, 1, 1), layout(epx)
    B, C = A + 0x1000, A + 0x2000

    def call(problem=p, lay=L, dout=A, y=B, y_rows=128, w=A, h=256, dy=C, dw=A):
        return lib.epx_combine_backward(by(problem), by(lay) if lay is not None else None, dout, y, y_rows, w, h, dy, dw,
                                        None)

    assert call(y_rows=127) == 3
    for bad in (dict(lay=None), dict(h=252), dict(h=0), dict(dout=None), dict(dout=A + 8), dict(y=None), dict(y=B + 4),
                dict(w=None), dict(w=A + 2), dict(dy=None), dict(dy=C + 8), dict(dw=A + 2), dict(dy=B), dict(dy=A)):
        assert call(**bad) == 1, bad
    assert call(problem=epx.make_problem(64, 2, 16, 3, 1)) == 1
    assert call(problem=epx.make_problem(0, 2, 16, 1, 1), dout=None, y=None, w=None, dy=None) == 0


BAD_ROWS = [dict(n=0), dict(n=-1), dict(n=2049), dict(R=-1), dict(off=None), dict(cnt=None), dict(off=A + 2),
            dict(cnt=A + 1), dict(R=2 ** 31 - 4095), dict(R=2 ** 31 - 1)]
# width, inner (of a product whose matrix has `wide` rows)
BAD_SIZES = [(0, 64), (4, 64), (12, 64), (-8, 64), (64, 0), (64, 12), (64, -8), ((1 << 20) + 8, 8), (8, (1 << 20) + 8),
             (65536, 16392)]


@pytest.mark.parametrize("bad", BAD_ROWS, ids=str)
def test_rows(epx, lib, bad):
    r = rows(epx, **bad)
    assert lib.epx_expert_gemm(by(r), A, A, 64, 64, 0, None, A + 0x1000, None) == 1
    assert lib.epx_expert_gemm_dgrad(by(r), A, A, 64, 64, 0, None, A + 0x1000, None) == 1
    assert lib.epx_expert_gemm_wgrad(by(r), A, A, 64, 64, 0, 0, A, None) == 1
    assert lib.epx_expert_gemm_mxfp4(by(r), A, A, A, A, 128, 128, 0, 0, A + 0x1000, None, None) == 1


@pytest.mark.parametrize("width,inner", BAD_SIZES)
def test_sizes(epx, lib, width, inner):
    r = rows(epx)
    assert lib.epx_expert_gemm(by(r), A, A, width, inner, 0, None, A + 0x1000, None) == 1
    assert lib.epx_expert_gemm_dgrad(by(r), A, A, width, inner, 0, None, A + 0x1000, None) == 1
    assert lib.epx_expert_gemm_wgrad(by(r), A, A, width, inner, 0, 0, A, None) == 1
    assert lib.epx_expert_gemm_mxfp4(by(r), A, A, A, A, width, inner, 0, 0, A + 0x1000, None, None) == 1


def test_products(epx, lib):
    r, O = rows(epx), A + 0x1000

    def fwd(x=A, w=A, act=0, pre=None, out=O, width=64):
        return lib.epx_expert_gemm(by(r), x, w, width, 64, act, pre, out, None)

    for bad in (dict(x=None), dict(x=A + 8), dict(w=None), dict(w=A + 8), dict(out=None), dict(out=O + 8), dict(act=2),
                dict(act=-1), dict(pre=A), dict(act=1, pre=A + 8), dict(out=A), dict(act=1, pre=O)):
        assert fwd(**bad) == 1, bad
    assert lib.epx_expert_gemm(None, A, A, 64, 64, 0, None, O, None) == 1
    # the gated matrix has twice the rows
    assert lib.epx_expert_gemm(by(r), A, A, 32768, 16392, 1, None, O, None) == 1

    def dgrad(dy=A, w=A, act=0, pre=None, dx=O):
        return lib.epx_expert_gemm_dgrad(by(r), dy, w, 64, 64, act, pre, dx, None)

    for bad in (dict(dy=None), dict(dy=A + 4), dict(w=None), dict(dx=None), dict(dx=O + 2), dict(act=1), dict(pre=A),
                dict(act=2, pre=A), dict(act=1, pre=A + 8), dict(dx=A), dict(act=1, pre=O)):
        assert dgrad(**bad) == 1, bad

    def wgrad(dy=A, x=A, dtype=0, acc=0, dw=O):
        return lib.epx_expert_gemm_wgrad(by(r), dy, x, 64, 64, dtype, acc, dw, None)

    for bad in (dict(dy=None), dict(x=None), dict(dw=None), dict(dw=O + 8), dict(dtype=1), dict(dtype=3),
                dict(dtype=0, acc=1), dict(dtype=2, acc=2), dict(dy=A + 8), dict(x=A + 8)):
        assert wgrad(**bad) == 1, bad
    # nothing to do without rows
    none = rows(epx, R=0)
    assert lib.epx_expert_gemm(by(none), None, None, 64, 64, 0, None, None, None) == 0
    assert lib.epx_expert_gemm_dgrad(by(none), None, None, 64, 64, 0, None, None, None) == 0
    assert lib.epx_expert_gemm_mxfp4(by(none), None, None, None, None, 128, 128, 0, 0, None, None, None) == 0


def test_mxfp4(epx, lib):
    for f in (lib.epx_mxfp4_quantize, lambda x, n, k, c, s, st: lib.epx_mxfp4_dequantize(c, s, n, k, x, st)):
        for bad in ((None, 4, 64, A, A), (A + 8, 4, 64, A, A), (A, 4, 64, None, A), (A, 4, 64, A + 8, A),
                    (A, 4, 64, A, None), (A, -1, 64, A, A), (A, 1 << 31, 64, A, A), (A, 4, 0, A, A), (A, 4, 48, A, A),
                    (A, 4, -32, A, A)):
            assert f(*bad, None) == 1, bad
        assert f(None, 0, 64, None, None, None) == 0

    r, O = rows(epx), A + 0x1000

    def mx(x=A, xs=A, w=A, ws=A, width=128, inner=128, act=0, dtype=0, out=O, osc=None):
        return lib.epx_expert_gemm_mxfp4(by(r), x, xs, w, ws, width, inner, act, dtype, out, osc, None)

    for bad in (dict(x=None), dict(x=A + 8), dict(xs=None), dict(xs=A + 2), dict(w=None), dict(w=A + 4), dict(ws=None),
                dict(ws=A + 2), dict(out=None), dict(out=O + 8), dict(act=2), dict(dtype=2), dict(dtype=1),
                dict(dtype=1, osc=A + 2), dict(dtype=1, osc=A, width=136), dict(inner=64), dict(inner=192), dict(out=A)):
        assert mx(**bad) == 1, bad


def test_binding_rejects_wrong_tensors(epx):
    p = epx.make_problem(4, 2, 16, 1, 1)
    cpu = torch.zeros(4, 16)
    with pytest.raises(ValueError):
        epx.epx_route(p, cpu, 0, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        epx.epx_route(p, cpu.to(torch.float16), 0, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        epx.expert_rows(torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), 8)
    with pytest.raises(ValueError):
        epx.epx_mxfp4_quantize(torch.zeros(4, 32, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.uint8),
                               torch.zeros(4, 1, dtype=torch.uint8))
