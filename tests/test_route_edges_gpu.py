"""The router and its gradient where masks meet infinite or NaN gradients and
biases, and with more choices than half a wave has lanes."""
import numpy as np
import pytest
import torch

from tests.test_route_gpu import as_input, epx, gradient, run, run_backward, scores  # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = ["softmax", "softmax_all", "sigmoid", "sigmoid_all"]


def backward(epx, p, t, score, idx, dw, renorm, scale=1.0):  # noqa: F811
    d = torch.full_like(t, -9.0)
    epx.epx_route_backward(p, t, score, idx, dw, d, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    return d


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("E,k", [(40, 8), (200, 40), (300, 8), (1500, 40)])
def test_gradients_of_masked_choices_reach_nothing(epx, E, k, kind, dtype):  # noqa: F811
    """Tokens with fewer live experts than k choose masked ones, whose weights are 0: what stands at those places of
    dweights changes nothing, and a masked expert's gradient is 0 whatever the live choices' are."""
    rng = np.random.default_rng(E + k)
    l = rng.standard_normal((9, E))
    l[:, 5:] = -np.inf
    l[1, 2], l[2, :4], l[3, :] = np.nan, -np.inf, np.nan
    t, l = as_input(l, dtype)
    softmax, renorm = kind.startswith("softmax"), not kind.endswith("_all")
    score = epx.SCORE_SOFTMAX if softmax else epx.SCORE_SIGMOID
    p = epx.make_problem(9, k, E, 1, 1)
    idx, w = torch.empty(9, k, dtype=torch.int32, device="cuda"), torch.empty(9, k, device="cuda")
    epx.epx_route(p, t, score, idx, w, renormalize=renorm)
    dead = torch.from_numpy(~(l > -np.inf)).cuda()
    chosen_dead = dead.gather(1, idx.long())
    assert not w[chosen_dead].any() and int(chosen_dead.sum()) >= 9 * (k - 5)
    dw = torch.from_numpy(rng.standard_normal((9, k)).astype(np.float32)).cuda()
    dw[chosen_dead] = 0.0
    want = backward(epx, p, t, score, idx, dw, renorm)
    ref, size = gradient(l, idx.cpu().numpy(), dw.double().cpu().numpy(), softmax, renorm, 1.0)
    # as in the router's other tests: terms of the largest |dw|, and half a step of the type
    tol = 2.0 ** -23 * (16 + 4 * 5 + E) * dw.abs().max(1, keepdim=True).values.double().cpu().numpy()
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    assert np.all(np.abs(want.double().cpu().numpy() - ref) <= tol + half * (np.abs(ref) + tol) + 1e-37)
    for bad in (float("nan"), float("inf"), float("-inf"), 3e38):
        dw2 = dw.clone()
        dw2[chosen_dead] = bad
        assert torch.equal(backward(epx, p, t, score, idx, dw2, renorm, 2.5), backward(epx, p, t, score, idx, dw, renorm, 2.5)), bad
    for bad in (float("nan"), float("inf")):
        dw2 = dw.clone()
        dw2[~chosen_dead] = bad
        assert not backward(epx, p, t, score, idx, dw2, renorm)[dead].any(), bad


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(70, 8), (200, 40), (600, 12)])
def test_bias_of_minus_infinity_or_nan_orders_only(epx, E, k, renorm, dtype):  # noqa: F811
    """Such an expert comes after every other one, with the masked ones in order of id; chosen all the same, it has its
    score's weight and gradient."""
    rng = np.random.default_rng(E * 3 + k)
    t, l = as_input(rng.standard_normal((6, E)), dtype)
    l[2, ::2], l[3, 1::2] = -np.inf, np.nan
    t, l = as_input(l, dtype)
    b = rng.standard_normal(E).astype(np.float32)
    b[6:] = -np.inf
    b[8::3] = np.nan
    b[E - 2] = 0.25
    p = epx.make_problem(6, k, E, 1, 1)
    idx, w = torch.empty(6, k, dtype=torch.int32, device="cuda"), torch.empty(6, k, device="cuda")
    epx.epx_route(p, t, epx.SCORE_SIGMOID, idx, w, bias=torch.from_numpy(b).cuda(), renormalize=renorm, scale=2.5)
    torch.cuda.synchronize()
    sc = scores(l, False)
    key = sc + b.astype(np.float64)
    key = np.where((l > -np.inf) & (key > -np.inf), key, -np.inf)
    want = np.argsort(-key, axis=1, kind="stable")[:, :k]
    assert np.array_equal(idx.cpu().numpy(), want)
    # at most 7 experts have a bias that is a number
    c = np.take_along_axis(sc, want, 1)
    assert (c[:, 7:] > 0).any() and (np.take_along_axis(l, want, 1)[2] == -np.inf).any()
    s = c.sum(1, keepdims=True)
    assert np.all(np.abs(w.cpu().numpy() - 2.5 * (c / s if renorm else c)) <= 2.0 ** -20 * 2.5 * (c / s if renorm else c))
    run_backward(epx, p, t, l, idx, epx.SCORE_SIGMOID, False, renorm, 2.5, E)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS + ["biased"])
@pytest.mark.parametrize("shape", [(4, 40, 40), (5, 33, 33), (7, 64, 64), (3, 65, 34), (9, 100, 40), (6, 128, 33), (11, 256, 64),
                                   (1, 200, 47)], ids=str)
def test_more_than_32_choices_of_up_to_256_experts(epx, shape, kind, dtype):  # noqa: F811
    """Two choices a lane forwards, a whole wave a token backwards; with masked tokens of fewer than k experts."""
    T, E, k = shape
    rng = np.random.default_rng(T * 10007 + E * 101 + k)
    l = 1.5 * rng.standard_normal((T, E))
    l[0, rng.permutation(E)[:E - 20]] = -np.inf
    if T > 3:
        l[1], l[2, 10:] = np.nan, -np.inf
        l[3] = np.round(l[3])   # ties
    softmax, renorm = kind.startswith("softmax"), not kind.endswith("_all")
    bias = 0.2 * rng.standard_normal(E) if kind == "biased" else None
    p, t, l, idx, score = run(epx, l, dtype, k, softmax, bias, renorm, 2.5)
    run_backward(epx, p, t, l, idx, score, softmax, renorm, 2.5, E)
