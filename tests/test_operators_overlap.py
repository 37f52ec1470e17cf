"""Outputs in place of another buffer: refused on the host, before anything is
launched (so this runs without a GPU; the addresses are never read)."""
import pytest

from tests.test_operators_abi import by, epx, layout, lib, rows  # noqa: F401

BASE = 0x200000   # 16-byte aligned; argument i stands at BASE + i * 0x1000


def calls(epx, lib):  # noqa: F811
    """name: (call of the addresses, their names, the outputs among them)."""
    p, L, r = epx.make_problem(64, 2, 16, 1, 1), layout(epx), rows(epx)
    return {
        "route": (lambda a: lib.epx_route(by(p), a["logits"], 2, 1, a["bias"], 1, 1.0, a["idx"], a["w"], None),
                  ["logits", "bias", "idx", "w"], ["idx", "w"]),
        "route_backward": (lambda a: lib.epx_route_backward(by(p), a["logits"], 2, 1, 1, 1.0, a["idx"], a["dw"], a["d"], None),
                           ["logits", "idx", "dw", "d"], ["d"]),
        "combine_backward": (lambda a: lib.epx_combine_backward(by(p), by(L), a["dout"], a["y"], 128, a["w"], 256, a["dy"],
                                                                a["dw"], None),
                             ["dout", "y", "w", "dy", "dw"], ["dy", "dw"]),
        "gemm": (lambda a: lib.epx_expert_gemm(by(r), a["x"], a["w"], 64, 64, 1, a["pre"], a["out"], None),
                 ["x", "w", "pre", "out"], ["pre", "out"]),
        "dgrad": (lambda a: lib.epx_expert_gemm_dgrad(by(r), a["dy"], a["w"], 64, 64, 1, a["pre"], a["dx"], None),
                  ["dy", "w", "pre", "dx"], ["dx"]),
        "wgrad": (lambda a: lib.epx_expert_gemm_wgrad(by(r), a["dy"], a["x"], 64, 64, 2, 1, a["dw"], None),
                  ["dy", "x", "dw"], ["dw"]),
        "quantize": (lambda a: lib.epx_mxfp4_quantize(a["x"], 4, 64, a["codes"], a["scales"], None),
                     ["x", "codes", "scales"], ["codes", "scales"]),
        "dequantize": (lambda a: lib.epx_mxfp4_dequantize(a["codes"], a["scales"], 4, 64, a["out"], None),
                       ["codes", "scales", "out"], ["out"]),
        "mxfp4": (lambda a: lib.epx_expert_gemm_mxfp4(by(r), a["x"], a["xs"], a["w"], a["ws"], 128, 128, 1, 1, a["out"],
                                                      a["osc"], None),
                  ["x", "xs", "w", "ws", "out", "osc"], ["out", "osc"]),
    }


PAIRS = [("route", o, i) for o in ("idx", "w") for i in ("logits", "bias", "idx", "w") if i != o] + [
    ("route_backward", "d", i) for i in ("logits", "idx", "dw")] + [
    ("combine_backward", o, i) for o in ("dy", "dw") for i in ("dout", "y", "w", "dy", "dw") if i != o] + [
    ("gemm", o, i) for o in ("out", "pre") for i in ("x", "w", "pre", "out") if i != o] + [
    ("dgrad", "dx", i) for i in ("dy", "w", "pre")] + [("wgrad", "dw", i) for i in ("dy", "x")] + [
    ("quantize", o, i) for o in ("codes", "scales") for i in ("x", "codes", "scales") if i != o] + [
    ("dequantize", "out", i) for i in ("codes", "scales")] + [
    ("mxfp4", o, i) for o in ("out", "osc") for i in ("x", "xs", "w", "ws", "out", "osc") if i != o]


@pytest.mark.parametrize("name,out,other", PAIRS)
def test_in_place(epx, lib, name, out, other):  # noqa: F811
    call, names, outs = calls(epx, lib)[name]
    assert out in outs
    a = {n: BASE + i * 0x1000 for i, n in enumerate(names)}
    a[out] = a[other]
    assert call(a) == 1
