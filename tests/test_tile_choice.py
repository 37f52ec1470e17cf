"""Which tiles the experts' products on 8-bit rows take, by the kernels that
the library's own host code launches (no GPU)."""
import re

import pytest

from tests import experts_reference as ref
from tests import test_expert_tiles8_gpu as tiles
from tests import test_experts8_gpu as products
from tests.launches import Recorder, expert_calls


@pytest.fixture(scope="module")
def recorder(tmp_path_factory):
    return Recorder(str(tmp_path_factory.mktemp("launches")))


# call: template arguments of its square (128 x 128) and small (128 x 64) tiles
SQUARE = {c: f"gemm_kernel<{op}, 128, 128, 64, 2, 2, 2, 1>"
          for c, op in (("keep8", 6), ("int8", 7), ("int8 gated", 8), ("int8 kept", 9), ("dgrad8", 10))}


def small(call, buffers):
    op, p = {"keep8": (6, 2), "int8": (7, 4), "int8 gated": (8, 4), "int8 kept": (9, 2), "dgrad8": (10, 4)}[call]
    return f"gemm_kernel<{op}, 128, 64, 64, {buffers}, {p}, {4 // p}, 1>"


# 513 to 768 small tiles, the squares in one round. Sums that take three buffers, two workgroups a CU: two rounds of small tiles.
LONG = [("keep8", 9 * 894, 9, 224, 2760), ("int8", 9 * 1017, 9, 576, 5536), ("int8 gated", 52 * 70, 52, 576, 2592),
        ("int8 kept", 52 * 70, 52, 576, 2592), ("dgrad8", 27 * 127, 27, 3360, 1056), ("dgrad8", 18 * 226, 18, 2176, 1120)]
# ... and sums that take two, three workgroups a CU: one round.
SHORT = [("keep8", 9 * 894, 9, 224, 256), ("int8 gated", 52 * 70, 52, 576, 512), ("dgrad8", 27 * 127, 27, 256, 1056)]


@pytest.mark.parametrize("call,rows,experts,width,inner", LONG)
def test_a_round_of_small_tiles_with_three_buffers_is_512(recorder, call, rows, experts, width, inner):
    assert recorder.launched(expert_calls(rows, experts, width, inner)[call]) == [SQUARE[call]]


@pytest.mark.parametrize("call,rows,experts,width,inner", SHORT)
def test_a_round_of_small_tiles_with_two_buffers_is_768(recorder, call, rows, experts, width, inner):
    assert recorder.launched(expert_calls(rows, experts, width, inner)[call]) == [small(call, 2)]


# call: (its template argument, units of width and inner)
CALLS = {"int8": (7, (8, 16)), "int8 gated": (8, (8, 16)), "int8 kept": (9, (32, 16)), "keep8": (6, (32, 8)), "dgrad8": (10, (8, 32)),
         "wgrad8 bf16": ("false", (8, 32)), "wgrad8 f32": ("true", (8, 32))}


def launched(recorder, call, case):
    name, cnt, gap, order, width, inner = case
    width, inner = (products.up(v, u) for v, u in zip((width, inner), CALLS[call][1]))
    return recorder.launched(expert_calls(ref.ranges(cnt, gap, order)[1], len(cnt), width, inner)[call])


def tile_cases(call):
    return tiles.CASES[call.removesuffix(" bf16").removesuffix(" f32")]


def test_every_tile_has_a_case_with_results(recorder):
    """Each kernel of these calls is launched by a case that the GPU tests hold against 64-bit products."""
    reached = {k for call in CALLS for case in products.CASES + [c for _, c in tile_cases(call)]
               for k in launched(recorder, call, case)}
    kernels = {k for k in recorder.kernels() if re.match(r"gemm_kernel<(6|7|8|9|10),|wgrad_kept", k)}
    assert len(kernels) >= 50 and kernels == reached, sorted(kernels ^ reached)


@pytest.mark.parametrize("call", CALLS)
def test_cases_take_the_tiles_that_they_are_for(recorder, call):
    kernel = "wgrad_kept_kernel" if "wgrad" in call else "gemm_kernel"
    for tile, case in tile_cases(call):
        assert launched(recorder, call, case) == [f"{kernel}<{CALLS[call][0]}, {tile}>"], case[0]
