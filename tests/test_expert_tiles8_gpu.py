"""The experts' products on 8-bit rows at sizes that take the tiles which the
other tests' sizes do not (tests/test_tile_choice.py holds every tile against
the cases here and there): ranges with gaps and empty experts, and ends inside
tiles, fragments and steps."""
import pytest

from tests import test_experts8_gpu as products
from tests.test_experts8_gpu import epx  # noqa: F401

pytestmark = pytest.mark.gpu


def counts(experts, most, step=53):
    """Ragged rows, none for one expert."""
    c = [(i * step + 7) % most for i in range(experts)]
    c[experts // 2] = 0
    return c


SQUARE, TWO_GROUPS = "128, 128, 64, 2, 2, 2, 1", "128, 64, 64, 3, 4, 1, 2"
# call: (template arguments of the tile, (name, counts, gap, order, width, inner))
CASES = {
    "int8": [
        (SQUARE, ("short sums", counts(14, 700), 1, None, 1184, 32)),
        (SQUARE, ("a sum that ends inside a step", counts(14, 1000), 1, None, 1176, 112)),
        ("128, 64, 64, 3, 4, 1, 1", ("three buffers, few rows", counts(33, 70), 1, None, 904, 1296)),
        (TWO_GROUPS, ("two groups of waves", counts(48, 300), 1, None, 80, 2320)),
    ],
    "int8 gated": [
        ("128, 32, 64, 4, 4, 1, 1", ("four buffers, few rows", counts(20, 8), 1, None, 392, 1360)),
        ("128, 32, 64, 4, 4, 1, 1", ("four buffers, 64 experts", counts(64, 32), 1, None, 1024, 2048)),
        (TWO_GROUPS, ("two groups of waves", counts(48, 300), 1, None, 40, 2672)),
    ],
    "int8 kept": [
        ("128, 32, 64, 4, 2, 2, 1", ("four buffers, few rows", counts(20, 8), 1, None, 416, 1360)),
        ("128, 32, 64, 4, 2, 2, 1", ("four buffers, 64 experts", counts(64, 32), 1, None, 1024, 2048)),
        ("128, 64, 64, 3, 2, 2, 2", ("two groups of waves", counts(48, 300), 1, None, 64, 2672)),
    ],
    "keep8": [
        ("128, 32, 64, 4, 2, 2, 1", ("four buffers, few rows", counts(7, 8), 1, None, 1248, 680)),
        (SQUARE, ("long sums", counts(9, 1800, 229), 1, None, 352, 2760)),
    ],
    "dgrad8": [
        (SQUARE, ("short sums", counts(33, 150), 1, None, 40, 1888)),
        (SQUARE, ("a sum that ends inside a step", counts(20, 700), 1, None, 104, 1120)),
        (SQUARE, ("long sums", counts(18, 450), 1, None, 1096, 1120)),
    ],
    "wgrad8": [
        ("64, 128, 32, 1, 2, 4", ("four pairs of waves", counts(12, 1500), 1, None, 656, 96)),
        ("64, 128, 32, 1, 2, 4", ("four pairs of waves, an odd number of columns", counts(11, 1500, 79), 1, None, 648, 160)),
    ],
}


def param(call):
    return pytest.mark.parametrize("case", [c for _, c in CASES[call]], ids=lambda c: c[0])


@param("int8")
def test_int8(epx, case):  # noqa: F811
    products.test_int8(epx, case, "none")


@param("int8 gated")
def test_int8_gated(epx, case):  # noqa: F811
    products.test_int8(epx, case, "swiglu")


@param("int8 kept")
def test_int8_keeps_preactivations(epx, case):  # noqa: F811
    products.test_int8_keeps_preactivations(epx, case)


@param("keep8")
def test_keep8(epx, case):  # noqa: F811
    products.test_keep8(epx, case)


@param("dgrad8")
def test_dgrad_kept8(epx, case):  # noqa: F811
    products.test_dgrad_kept8(epx, case)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "f32 added"])
@param("wgrad8")
def test_wgrad_kept8(epx, case, dtype):  # noqa: F811
    products.test_wgrad_kept8(epx, case, dtype)
