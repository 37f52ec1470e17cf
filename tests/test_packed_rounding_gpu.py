"""The rounding to bf16 of the products on 8-bit rows, on every float32 number:
an int8 product whose sums are 1 and -1 gives the rows' scales, rounded once."""
import pytest
import torch

from tests.test_experts_gpu import epx, make_rows  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = 1 << 25


def test_every_float32(epx):  # noqa: F811
    """Nearest, ties to even, by the integers of the definition; NaN gives NaN."""
    rows = make_rows(epx, [0], [ROWS], ROWS)
    x = torch.zeros(ROWS, 16, dtype=torch.int8, device="cuda")
    w = torch.zeros(1, 8, 16, dtype=torch.int8, device="cuda")
    x[:, 3], w[0, ::2, 3], w[0, 1::2, 3] = 1, 1, -1
    ones = torch.ones(1, 8, device="cuda")
    out = torch.empty(ROWS, 8, dtype=torch.bfloat16, device="cuda")
    index = torch.arange(ROWS, dtype=torch.int64, device="cuda")
    for first in range(0, 1 << 32, ROWS):
        u = index + first
        scales = torch.where(u < 1 << 31, u, u - (1 << 32)).to(torch.int32).view(torch.float32)
        out.fill_(7.0)
        epx.epx_expert_gemm_int8(rows, x, scales, w, ones, out)
        magnitude = u & 0x7FFFFFFF
        nan = magnitude > 0x7F800000
        want = (magnitude + 0x7FFF + ((magnitude >> 16) & 1)) >> 16
        sign = (u >> 31) << 15
        bits = out.view(torch.int16).to(torch.int64) & 0xFFFF
        for column in range(8):
            got = bits[:, column]
            flip = (column % 2) << 15
            # (a zero's sign is that of the product, too)
            wrong = torch.where(nan, (got & 0x7FFF) <= 0x7F80, got != (want | (sign ^ flip)))
            assert not bool(wrong.any()), (hex(first), column, u[wrong][:4].tolist(), got[wrong][:4].tolist())
