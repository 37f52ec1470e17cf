"""Differences of the forward calls along the gradients that the calls on kept
activations give."""
import pytest
import torch

from tests import experts_reference as ref
from tests import rows8_reference as r8
from tests.test_experts8_gpu import kept_values
from tests.test_experts_gpu import epx, gen, guard, make_rows, rand  # noqa: F401
from tests.test_gradient_differences_gpu import agree, output_noise

pytestmark = pytest.mark.gpu
CNT = [20, 0, 9, 133]
# sums of at most 96 terms, against results of about their root's size: see the bf16 products' differences
SUMS = 96 * 100 * 2.0 ** -23


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_weight_gradient(epx, dtype):  # noqa: F811
    """The product of the kept values, which are bf16 numbers, at two weights."""
    g = gen(81)
    off, R = ref.ranges(CNT)
    rows, N, K = make_rows(epx, off, CNT, R), 72, 96
    codes, scales = kept_values(g, R, K)
    x = r8.mxint8_values(codes, scales).to(torch.bfloat16)
    w, dy = rand(g, 4, N, K, std=K ** -0.5), rand(g, R, N)
    dw = guard(4, N, K, dtype=dtype)
    epx.epx_expert_gemm_wgrad_kept8(rows, dy, codes, scales, dw)

    def out(weights):
        o = guard(R, N)
        epx.epx_expert_gemm(rows, x, weights, o)
        torch.cuda.synchronize()
        return o.double()

    moved = (w.float() + 0.5 * torch.sign(dw.float())).to(torch.bfloat16)
    move = moved.double() - w.double()
    a, b = out(moved), out(w)
    half = ref.BF16 if dtype == torch.bfloat16 else 2.0 ** -24
    noise = output_noise(a, b, dy, SUMS) + (move * dw.double()).abs().sum() * (half + 2 * SUMS)
    agree(((a - b) * dy.double()).sum(), (move * dw.double()).sum(), noise)


def test_gated_layer(epx):  # noqa: F811
    """The gradient of kept pre-activations: a central difference of the layer in float64."""
    g = gen(82)
    off, R = ref.ranges(CNT)
    rows, N, K = make_rows(epx, off, CNT, R), 72, 96
    codes, scales = kept_values(g, R, 2 * K, std=1.5)
    pre = r8.mxint8_values(codes, scales)
    w, dy = rand(g, 4, N, K, std=N ** -0.5), rand(g, R, N)
    dpre = guard(R, 2 * K)
    epx.epx_expert_gemm_dgrad_kept8(rows, dy, w, codes, scales, dpre)
    torch.cuda.synchronize()

    def loss(z):
        act = ref.glu(z, torch.zeros_like(z))[0]
        return sum(((act[o:o + c] @ w[e].double().T) * dy[o:o + c].double()).sum() for e, (o, c) in enumerate(zip(off, CNT)))

    h = 2.0 ** -12
    move = h * torch.sign(dpre.double())
    diff = (loss(pre + move) - loss(pre - move)) / 2
    grad = (move * dpre.double()).sum()
    third = h ** 3 / 6 * 2 * (1 + pre.abs().max()) * 10 * dpre.numel()
    noise = (move * dpre.double()).abs().sum() * (2 * ref.BF16 + SUMS) + third
    agree(diff, grad, noise)
