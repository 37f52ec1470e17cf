"""Refusals of the calls on 8-bit rows: every bad argument, and every output in
place of another buffer, is turned down on the host before anything is launched
(so these run without a GPU; the addresses are never read)."""
import pytest
import torch

from tests.test_operators_abi import A, BAD_ROWS, by, epx, lib, rows  # noqa: F401

O = A + 0x1000   # noqa: E741
C, S = A + 0x2000, A + 0x3000


def fns(lib):  # noqa: F811
    """Each call with good arguments by name, `None` where it writes nothing optional."""
    return {
        "int8": (lib.epx_expert_gemm_int8, dict(x=A, xs=A + 0x100, w=A, ws=A + 0x200, width=64, inner=64, act=0, pc=None,
                                                ps=None, out=O)),
        "keep8": (lib.epx_expert_gemm_keep8, dict(x=A, w=A, width=64, inner=64, pc=C, ps=S, out=O)),
        "dgrad8": (lib.epx_expert_gemm_dgrad_kept8, dict(dy=A, w=A, width=64, inner=64, pc=C, ps=S, act=None, dx=O)),
        "wgrad8": (lib.epx_expert_gemm_wgrad_kept8, dict(dy=A, xc=C, xs=S, width=64, inner=64, dtype=2, acc=0, dw=O)),
    }


def call(lib, name, r, **k):  # noqa: F811
    f, ok = fns(lib)[name]
    assert set(k) <= set(ok), k
    return f(by(r) if r is not None else None, *{**ok, **k}.values(), None)


NAMES = ["int8", "keep8", "dgrad8", "wgrad8"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("bad", BAD_ROWS, ids=str)
def test_rows(epx, lib, name, bad):  # noqa: F811
    assert call(lib, name, rows(epx, **bad)) == 1


@pytest.mark.parametrize("name", NAMES)
def test_no_rows(epx, lib, name):  # noqa: F811
    assert call(lib, name, None) == 1
    if name != "wgrad8":
        assert call(lib, name, rows(epx, R=0), **{k: None for k in ("x", "w", "dy", "out", "dx", "xs", "ws", "pc", "ps")
                                                  if k in fns(lib)[name][1]}) == 0


BAD_SIZES = {
    "int8": [(0, 64), (4, 64), (12, 64), (-8, 64), (64, 0), (64, 8), (64, 24), (64, -16), ((1 << 20) + 8, 16),
             (8, 1 << 17), (16384, 65552), (8, 1 << 20)],
    "keep8": [(0, 64), (16, 64), (40, 64), (-32, 64), (64, 0), (64, 12), ((1 << 20) + 32, 8), (32, (1 << 20) + 8),
              (32768, 16392)],
    "dgrad8": [(0, 64), (4, 64), (12, 64), (64, 0), (64, 16), (64, 40), (64, -32), ((1 << 20) + 8, 32),
               (8, (1 << 20) + 32), (65536, 16416)],
}
BAD_SIZES["wgrad8"] = BAD_SIZES["dgrad8"]


@pytest.mark.parametrize("name,width,inner", [(n, *s) for n in NAMES for s in BAD_SIZES[n]])
def test_sizes(epx, lib, name, width, inner):  # noqa: F811
    assert call(lib, name, rows(epx), width=width, inner=inner) == 1


BAD = {
    "int8": [dict(x=None), dict(x=A + 8), dict(xs=None), dict(xs=A + 2), dict(w=None), dict(w=A + 4), dict(ws=None),
             dict(ws=A + 8), dict(out=None), dict(out=O + 8), dict(act=2), dict(act=-1), dict(pc=C, ps=S),
             dict(act=1, pc=C), dict(act=1, ps=S), dict(act=1, pc=C + 8, ps=S), dict(act=1, pc=C, ps=S, width=40),
             dict(act=1, width=32768, inner=16400)],
    "keep8": [dict(x=None), dict(x=A + 8), dict(w=None), dict(w=A + 8), dict(out=None), dict(out=O + 8), dict(pc=None),
              dict(pc=C + 8), dict(ps=None)],
    "dgrad8": [dict(dy=None), dict(dy=A + 8), dict(w=None), dict(w=A + 8), dict(dx=None), dict(dx=O + 8), dict(pc=None),
               dict(pc=C + 8), dict(ps=None), dict(act=A + 8)],
    "wgrad8": [dict(dy=None), dict(dy=A + 8), dict(xc=None), dict(xc=C + 8), dict(xs=None), dict(dw=None), dict(dw=O + 8),
               dict(dtype=1), dict(dtype=3), dict(dtype=0, acc=1), dict(acc=2), dict(acc=-1)],
}


@pytest.mark.parametrize("name,bad", [(n, b) for n in NAMES for b in BAD[n]], ids=str)
def test_arguments(epx, lib, name, bad):  # noqa: F811
    assert call(lib, name, rows(epx), **bad) == 1


# name: (outputs, everything that is given); argument i stands at its own address
BUFFERS = {
    "int8": (("out", "pc", "ps"), ("x", "xs", "w", "ws", "out", "pc", "ps")),
    "keep8": (("out", "pc", "ps"), ("x", "w", "out", "pc", "ps")),
    "dgrad8": (("dx", "act"), ("dy", "w", "pc", "ps", "dx", "act")),
    "wgrad8": (("dw",), ("dy", "xc", "xs", "dw")),
}


@pytest.mark.parametrize("name,out,other", [(n, o, i) for n in NAMES for o in BUFFERS[n][0] for i in BUFFERS[n][1] if i != o])
def test_in_place(epx, lib, name, out, other):  # noqa: F811
    a = {n: A + i * 0x1000 for i, n in enumerate(BUFFERS[name][1])}
    a[out] = a[other]
    if name == "int8":
        a["act"] = 1
    assert call(lib, name, rows(epx), **a) == 1


@pytest.mark.parametrize("f,unit", [("int8", 16), ("mxint8", 32)])
def test_conversions(lib, f, unit):  # noqa: F811
    q, d = getattr(lib, f"epx_{f}_quantize"), getattr(lib, f"epx_{f}_dequantize")
    for go in (lambda x, n, k, c, s: q(x, n, k, c, s, None), lambda x, n, k, c, s: d(c, s, n, k, x, None)):
        for bad in ((None, 4, 64, C, S), (A + 8, 4, 64, C, S), (A, 4, 64, None, S), (A, 4, 64, C + 8, S), (A, 4, 64, C, None),
                    (A, -1, 64, C, S), (A, 1 << 31, 64, C, S), (A, 4, 0, C, S), (A, 4, unit // 2, C, S),
                    (A, 4, 64 + unit // 2, C, S), (A, 4, -unit, C, S), (A, 4, (1 << 20) + unit, C, S)):
            assert go(*bad) == 1, bad
        assert go(None, 0, 64, None, None) == 0
    for a in ((A, A, S), (A, C, A), (A, C, C)):
        assert q(a[0], 4, 64, a[1], a[2], None) == 1
    for a in ((C, S, C), (C, S, S)):
        assert d(a[0], a[1], 4, 64, a[2], None) == 1
    if f == "int8":
        assert q(A, 4, 64, C, S + 2, None) == 1 and d(C, S + 2, 4, 64, A, None) == 1


def test_binding_rejects_wrong_tensors(epx):  # noqa: F811
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    for f in (epx.epx_int8_quantize, epx.epx_mxint8_quantize):
        with pytest.raises(ValueError):
            f(x, torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4))
    with pytest.raises(ValueError):
        epx.epx_mxint8_dequantize(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 1, dtype=torch.uint8), x)
