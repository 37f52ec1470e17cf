"""That tests/exact_sums.py's operands tell a float32 sum from less (on the CPU,
with the mistakes planted in a plain product)."""
import torch

import pytest

from tests import exact_sums as ex
from tests import experts_reference as ref


def running(x, w, step, hold):
    """The product summed in float32 within `step`, the running sum rounded to `hold` after each."""
    acc = torch.zeros(x.shape[0], w.shape[0])
    for k in range(0, x.shape[1], step):
        acc = (acc + x[:, k:k + step].float() @ w[:, k:k + step].float().T).to(hold).float()
    return acc


@pytest.mark.parametrize("length", [72, 136, 1048, 2056, 16392])
def test_products(length):
    g = ex.gen(length, "cpu")
    x, w = ex.along_rows(g, 12, length), ex.matrices(g, 1, 24, length)[0]
    want = ex.by_expert(x, w[None], [0], [12])
    assert want.abs().max() <= 256 and want.abs().max() > 0
    assert torch.equal(want.to(torch.bfloat16).double(), want)
    for step in (8, 32, 64, length):
        assert torch.equal(running(x, w, step, torch.float32).double(), want)

    def wrong(got):
        return float((got.to(torch.bfloat16).double() != want).double().mean())

    assert wrong(running(x[:, :-8], w[:, :-8], 64, torch.float32)) > 0.95
    assert wrong(running(x[:, 8:], w[:, 8:], 64, torch.float32)) > 0.95
    # the first sum that passes 2^11 or 2^8 loses bits, if there is more than one step
    for hold in (torch.float16, torch.bfloat16):
        for step in (16, 64, 512):
            if step < length // 2:
                assert wrong(running(x, w, step, hold)) > 0.5, (hold, step)


@pytest.mark.parametrize("rows", [1, 2, 7, 33, 300, 2100])
def test_weight_gradients(rows):
    g = ex.gen(rows, "cpu")
    dy, x = ex.down_columns(g, rows + 3, 24, 16, [2], [rows])
    want = dy[2:2 + rows].double().T @ x[2:2 + rows].double()
    assert want.abs().max() <= 256 and torch.equal(want.to(torch.bfloat16).double(), want)
    assert torch.equal(running(dy.T, x.T, 32, torch.float32).double(), want)
    if rows >= 300:
        assert float((running(dy.T, x.T, 64, torch.float16).double() != want).double().mean()) > 0.5
    if rows > 1:
        short = running(dy[:1 + rows].T, x[:1 + rows].T, 32, torch.float32)   # the last row left out
        assert float((short.double() != want).double().mean()) > 0.6


@pytest.mark.parametrize("length", [128, 384, 1664, 7168])
def test_fp8_rows_and_4_bit_weights(length):
    g = ex.gen(length, "cpu")
    x, xs, w, ws = ex.fp8_and_4_bit(g, 1, 24, 12, length)
    xv, wv = x.view(torch.float8_e4m3fn).double(), ref.mxfp4_values(w, ws)[0]
    want = (xv @ wv.T) * xs[:, :1].double()
    assert want.abs().max() > 0 and torch.equal(want.to(torch.bfloat16).double(), want)
    assert torch.equal((running(xv, wv, 128, torch.float32) * xs[:, :1]).double(), want)
    if length > 128:
        for got in (running(xv[:, :-128], wv[:, :-128], 128, torch.float32), running(xv, wv, 128, torch.float16)):
            assert float(((got * xs[:, :1]).double() != want).double().mean()) > 0.5
    # what the matrix instruction cuts (2^-13 of a group's largest power of two) is no bit of any product
    for lo in range(0, length, 8):
        p = (xv[:, None, lo:lo + 8] * wv[None, :, lo:lo + 8]).abs()
        top = torch.exp2(torch.floor(torch.log2(p.amax(2, keepdim=True).clamp(min=2.0 ** -20))))
        assert torch.equal(torch.floor(p / (top * 2.0 ** -13)) * (top * 2.0 ** -13), p)
