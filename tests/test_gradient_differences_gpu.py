"""Differences of the forward calls along their gradients: the step follows the
sign of the gradient, so that what is compared is the sum of magnitudes and not
a sum of terms of both signs that is about as small as its own noise."""
import pytest
import torch

from tests import experts_reference as ref
from tests.test_combine_backward_gpu import setup as combine_setup
from tests.test_experts_gpu import epx, gen, guard, make_rows, rand  # noqa: F401

pytestmark = pytest.mark.gpu


def agree(diff, grad, noise):
    """The difference is the gradient's within the noise, which tells it from none and from its negative."""
    diff, grad, noise = float(diff), float(grad), float(noise)
    print(f"difference {diff:.6g}, gradient {grad:.6g}, noise {noise:.3g}")
    assert noise < 0.25 * abs(grad)
    assert abs(diff - grad) <= noise
    assert abs(diff) > noise and abs(diff + grad) > noise


def output_noise(a, b, dout, sums):
    """Both outputs are off by half a bf16 step of themselves and by `sums` times their size (their float32 sums)."""
    return ((a.abs() + b.abs()) * dout.double().abs()).sum() * (ref.BF16 + 2 * sums)


@pytest.fixture(scope="module")
def layer(epx):  # noqa: F811
    g = gen(51)
    cnt = [20, 0, 9, 133]
    off, R = ref.ranges(cnt)
    N, K = 72, 104
    return dict(rows=make_rows(epx, off, cnt, R), x=rand(g, R, K), w=rand(g, 4, N, K, std=K ** -0.5), dy=rand(g, R, N), R=R, N=N, K=K)


def product(epx, lay, x, w):  # noqa: F811
    out = guard(lay["R"], lay["N"])
    epx.epx_expert_gemm(lay["rows"], x, w, out)
    torch.cuda.synchronize()
    return out.double()


# 104 terms of float32 a sum, against results of about their root's size: the magnitudes' sum is at most some
# tens of times a result's typical size, which 2^-23 * 104 * 100 covers
SUMS = 104 * 100 * 2.0 ** -23


def test_input_gradient(epx, layer):  # noqa: F811
    x, w, dy = layer["x"], layer["w"], layer["dy"]
    dx = guard(layer["R"], layer["K"])
    epx.epx_expert_gemm_dgrad(layer["rows"], dy, w, dx)
    moved = (x.float() + 4.0 * torch.sign(dx.float())).to(torch.bfloat16)
    move = moved.double() - x.double()
    a, b = product(epx, layer, moved, w), product(epx, layer, x, w)
    noise = output_noise(a, b, dy, SUMS) + (move * dx.double()).abs().sum() * (ref.BF16 + SUMS)
    agree(((a - b) * dy.double()).sum(), (move * dx.double()).sum(), noise)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_weight_gradient(epx, layer, dtype):  # noqa: F811
    x, w, dy = layer["x"], layer["w"], layer["dy"]
    dw = guard(4, layer["N"], layer["K"], dtype=dtype)
    epx.epx_expert_gemm_wgrad(layer["rows"], dy, x, dw)
    moved = (w.float() + 0.5 * torch.sign(dw.float())).to(torch.bfloat16)
    move = moved.double() - w.double()
    a, b = product(epx, layer, x, moved), product(epx, layer, x, w)
    half = ref.BF16 if dtype == torch.bfloat16 else 2.0 ** -24
    noise = output_noise(a, b, dy, SUMS) + (move * dw.double()).abs().sum() * (half + 2 * SUMS)
    agree(((a - b) * dy.double()).sum(), (move * dw.double()).sum(), noise)


def test_gated_layer(epx, layer):  # noqa: F811
    """The gradient of the pre-activations: the forward call's activation at two of them, in float64 by autograd's own
    formula and by a central difference."""
    g = gen(52)
    R, K = layer["R"], layer["K"]
    pre, dy = rand(g, R, 2 * K, std=1.5), layer["dy"]
    dpre = guard(R, 2 * K)
    epx.epx_expert_gemm_dgrad(layer["rows"], dy, layer["w"], dpre, input_act=epx.ACT_SWIGLU, preact=pre)
    torch.cuda.synchronize()
    off, cnt = layer["rows"].row_offset.tolist(), layer["rows"].row_count.tolist()

    def loss(z):
        act = ref.glu(z, torch.zeros_like(z))[0]
        return sum(((act[o:o + c] @ layer["w"][e].double().T) * dy[o:o + c].double()).sum() for e, (o, c) in enumerate(zip(off, cnt)))

    h = 2.0 ** -12
    move = h * torch.sign(dpre.double())
    diff = (loss(pre.double() + move) - loss(pre.double() - move)) / 2
    grad = (move * dpre.double()).sum()
    # third derivatives of silu(g) * u along a unit step of both: at most 2 (1 + |u|), times |d| of some units
    third = h ** 3 / 6 * 2 * (1 + pre.double().abs().max()) * 10 * dpre.numel()
    noise = (move * dpre.double()).abs().sum() * (2 * ref.BF16 + SUMS) + third
    agree(diff, grad, noise)


@pytest.fixture(scope="module")
def combined(epx):  # noqa: F811
    p, L, idx, dout, y, w = combine_setup(epx, (33, 5, 16, 1, 1, 136, False, 1), spare=0)
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    epx.epx_combine_backward(p, L, dout, y, w, dy, dw)
    torch.cuda.synchronize()

    def out(yy, ww):
        o = torch.empty_like(dout)
        epx.epx_combine(p, L, yy, ww, o)
        torch.cuda.synchronize()
        return o.double()

    return dict(dout=dout, y=y, w=w, dy=dy, dw=dw, out=out)


def test_combine_weights(combined):
    c = combined
    moved = c["w"] + torch.sign(c["dw"])
    a, b = c["out"](c["y"], moved), c["out"](c["y"], c["w"])
    move = moved.double() - c["w"].double()
    noise = output_noise(a, b, c["dout"], SUMS) + (move * c["dw"].double()).abs().sum() * SUMS
    agree(((a - b) * c["dout"].double()).sum(), (move * c["dw"].double()).sum(), noise)


def test_combine_rows(combined):
    c = combined
    moved = (c["y"].float() + 2.0 * torch.sign(c["dy"].float())).to(torch.bfloat16)
    a, b = c["out"](moved, c["w"]), c["out"](c["y"], c["w"])
    move = moved.double() - c["y"].double()
    noise = output_noise(a, b, c["dout"], SUMS) + (move * c["dy"].double()).abs().sum() * (ref.BF16 + SUMS)
    agree(((a - b) * c["dout"].double()).sum(), (move * c["dy"].double()).sum(), noise)
