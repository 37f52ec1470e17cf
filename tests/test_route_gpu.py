"""The router and its gradient on the GPU against 64-bit forms: every width of
row, ties, masked experts, rows with nothing left, infinities, far logits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def epx():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a visible GPU")
    from combine_epx_get_amd import epx as mod
    return mod


def scores(l, softmax):
    """64-bit scores of logits l; masked experts 0."""
    masked = ~(l > -np.inf)
    if softmax:
        m = np.max(np.where(masked, -np.inf, l), axis=1, keepdims=True)
        with np.errstate(invalid="ignore"):
            e = np.where(l == m, 1.0, np.exp(np.where(masked, -np.inf, l) - m))
        e = np.where(masked, 0.0, e)
        s = e.sum(1, keepdims=True)
        return e / np.where(s > 0, s, 1.0)
    with np.errstate(over="ignore"):
        return np.where(masked, 0.0, 1.0 / (1.0 + np.exp(-np.where(masked, 0.0, l))))


def reference(l, k, softmax, bias, renorm, scale):
    masked = ~(l > -np.inf)
    p = scores(l, softmax)
    key = p + bias if bias is not None else l
    # masked ones last, in order of id
    key = np.where(masked, -np.inf, key)
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    rows = np.arange(l.shape[0])[:, None]
    c = p[rows, idx]
    if softmax and renorm:   # over the chosen only: what the others hold plays no part
        c = scores(np.where(masked, -np.inf, l)[rows, idx], True)
    s = c.sum(1, keepdims=True)
    w = scale * (c / np.where(s > 0, s, 1.0) if renorm else c)
    return idx, w


def gradient(l, idx, dw, softmax, renorm, scale):
    T, E = l.shape
    rows = np.arange(T)[:, None]
    ok = (idx >= 0) & (idx < E)
    at = np.where(ok, idx, 0)
    p = scores(l, softmax)
    g = np.where(ok, scale * dw, 0.0)
    c = np.where(ok, p[rows, at], 0.0)
    if softmax and renorm:
        c = scores(np.where(ok, l[rows, at], -np.inf), True)
    q = 1.0
    if not softmax:
        q = np.where(l[rows, at] > -np.inf, 1.0 / (1.0 + np.exp(np.where(l[rows, at] > -np.inf, l[rows, at], 0.0))), 0)
    d = np.zeros_like(l)
    if renorm:
        s = c.sum(1, keepdims=True)
        r = c / np.where(s > 0, s, 1.0)
        part = r * (g - (g * r).sum(1, keepdims=True)) * q
    elif softmax:
        part = g * c
        d -= p * part.sum(1, keepdims=True)
    else:
        part = g * c * q
    np.add.at(d, (rows.repeat(idx.shape[1], 1), at), np.where(ok, part, 0.0))
    return d, np.abs(part).sum(1, keepdims=True)


def as_input(l, dtype):
    t = torch.from_numpy(l.astype(np.float32)).to(dtype).cuda()
    return t, t.float().cpu().numpy().astype(np.float64)


def run(epx, l, dtype, k, softmax, bias=None, renorm=True, scale=1.0):
    t, l = as_input(l, dtype)
    T, E = l.shape
    p = epx.make_problem(T, k, E, 1, 1)
    idx = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -9.0, dtype=torch.float32, device="cuda")
    b = torch.from_numpy(bias.astype(np.float32)).cuda() if bias is not None else None
    score = epx.SCORE_SOFTMAX if softmax else epx.SCORE_SIGMOID
    epx.epx_route(p, t, score, idx, w, bias=b, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    b64 = b.double().cpu().numpy() if b is not None else None
    want_idx, want_w = reference(l, k, softmax, b64, renorm, scale)
    got = idx.cpu().numpy()
    assert np.array_equal(got, want_idx), np.nonzero((got != want_idx).any(1))[0][:5]
    # exp in float32 (a step or two, growing with its argument), up to E additions, a quotient
    m = np.where(np.isfinite(l), np.abs(l), 0).max() if l.size else 0
    tol = 2.0 ** -23 * (8 + 2 * m + E)
    assert np.all(np.abs(w.cpu().numpy() - want_w) <= tol * np.abs(want_w) + 1e-37)
    return p, t, l, idx, score


def run_backward(epx, p, t, l, idx, score, softmax, renorm, scale, seed):
    T, E = l.shape
    dw = torch.from_numpy(np.random.default_rng(seed).standard_normal(tuple(idx.shape)).astype(np.float32)).cuda()
    d = torch.full_like(t, -9.0)
    epx.epx_route_backward(p, t, score, idx, dw, d, renormalize=renorm, scale=scale)
    torch.cuda.synchronize()
    want, size = gradient(l, idx.cpu().numpy(), dw.double().cpu().numpy(), softmax, renorm, scale)
    dws = scale * dw.abs().max(1, keepdim=True).values.double().cpu().numpy() if dw.numel() else size
    m = np.where(np.isfinite(l), np.abs(l), 0).max() if l.size else 0
    # relative to the sizes of the terms that cancel: a token's largest |dw| times its scores (at most 1)
    tol = 2.0 ** -23 * (16 + 4 * m + E) * np.broadcast_to(dws, want.shape)
    half = 2.0 ** -8 if t.dtype == torch.bfloat16 else 2.0 ** -24
    got = d.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol + half * (np.abs(want) + tol) + 1e-37), np.abs(got - want).max()
    assert not got[~(l > -np.inf)].any()


SHAPES = [(1, 1, 1), (1, 2, 1), (3, 5, 5), (7, 7, 3), (9, 16, 4), (5, 33, 8), (70, 64, 6), (13, 65, 2), (6, 100, 16),
          (129, 256, 8), (4, 257, 8), (17, 384, 10), (5, 512, 64), (3, 1000, 7), (6, 1024, 33), (5, 1999, 64),
          (9, 2048, 8)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["softmax", "softmax_all", "sigmoid", "sigmoid_all", "biased"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_route(epx, shape, kind, dtype):
    T, E, k = shape
    rng = np.random.default_rng(T * 10007 + E * 101 + k)
    l = 1.5 * rng.standard_normal((T, E))
    softmax, renorm = kind.startswith("softmax"), not kind.endswith("_all")
    bias = 0.2 * rng.standard_normal(E) if kind == "biased" else None
    scale = 2.5 if kind in ("biased", "softmax_all") else 1.0
    p, t, l, idx, score = run(epx, l, dtype, k, softmax, bias, renorm, scale)
    run_backward(epx, p, t, l, idx, score, softmax, renorm, scale, E)


@pytest.mark.parametrize("softmax", [True, False], ids=["softmax", "sigmoid"])
def test_ties_go_to_the_lowest_id(epx, softmax):
    rng = np.random.default_rng(5)
    l = rng.integers(-2, 3, (40, 200)).astype(np.float64)
    l[0] = 0.0
    l[1, ::2] = -0.0
    l[1, 1::2] = 0.0
    run(epx, l, torch.float32, 12, softmax)
    if not softmax:
        run(epx, l, torch.bfloat16, 12, False, bias=rng.integers(0, 2, 200) * 0.5)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid", "biased"])
def test_masks(epx, kind, renorm):
    """-infinity, NaN and the type's lowest value; rows with fewer experts than k, and with none."""
    rng = np.random.default_rng(6)
    l = rng.standard_normal((12, 70))
    low = float(np.finfo(np.float32).min)
    l[0, :] = -np.inf
    l[1, :] = np.nan
    l[2, 3:] = -np.inf
    l[3, rng.permutation(70)[:67]] = np.nan
    l[4, :] = low
    l[5, 10:] = low
    l[6, ::2] = -np.inf
    l[7, 1::3] = np.nan
    l[8, 69] = np.inf
    l[9, [4, 50]] = np.inf
    l[10, :] = np.inf
    softmax = kind == "softmax"
    bias = rng.standard_normal(70) if kind == "biased" else None
    p, t, l, idx, score = run(epx, l, torch.float32, 8, softmax, bias, renorm)
    finite = np.where(np.isposinf(l), 30.0, l)   # gradients at +infinity are not defined
    t2, l2 = as_input(finite, torch.float32)
    run_backward(epx, p, t2, l2, idx, score, softmax, renorm, 1.0, 6)


def test_far_logits(epx):
    """Scores that float32 loses: sigmoids of logits far below zero, normalised; and close biased keys."""
    l = np.full((3, 20), -200.0)
    l[0, :8] = -150.0 - np.arange(8)
    l[1] = 60.0 + np.arange(20)
    run(epx, l, torch.float32, 4, False)
    # float32 sums of score and bias would tie here; the 64-bit keys do not
    l = np.zeros((2, 64))
    bias = np.full(64, 100.0)
    l[0] = 1e-6 * np.arange(64)
    l[1] = -1e-6 * np.arange(64)
    run(epx, l, torch.float32, 10, False, bias=bias)


def test_backward_of_given_ids(epx):
    """Ids out of range contribute nothing; an id given twice counts twice."""
    rng = np.random.default_rng(8)
    t, l = as_input(rng.standard_normal((5, 30)), torch.float32)
    idx = torch.from_numpy(rng.integers(0, 30, (5, 6)).astype(np.int32)).cuda()
    idx[0, 1], idx[1, 0], idx[2, :] = 30, -1, 7
    idx[3, :] = -5
    p = epx.make_problem(5, 6, 30, 1, 1)
    for softmax in (True, False):
        for renorm in (True, False):
            score = epx.SCORE_SOFTMAX if softmax else epx.SCORE_SIGMOID
            run_backward(epx, p, t, l, idx, score, softmax, renorm, 1.5, 3)


@pytest.mark.parametrize("kind", ["softmax", "softmax_all", "sigmoid", "sigmoid_all"])
def test_gradient_against_differences(epx, kind):
    """Central differences of the 64-bit weights for fixed ids, against the call's gradient."""
    rng = np.random.default_rng(9)
    softmax, renorm = kind.startswith("softmax"), not kind.endswith("_all")
    p, t, l, idx, score = run(epx, rng.standard_normal((4, 24)), torch.float32, 5, softmax, None, renorm)
    at = idx.cpu().numpy()
    dw = rng.standard_normal((4, 5))
    d = torch.empty_like(t)
    epx.epx_route_backward(p, t, score, idx, torch.from_numpy(dw.astype(np.float32)).cuda(), d, renormalize=renorm)
    torch.cuda.synchronize()
    rows = np.arange(4)[:, None]

    def loss(x):
        c = scores(x, softmax)[rows, at]
        return ((c / c.sum(1, keepdims=True) if renorm else c) * dw.astype(np.float32)).sum(1)

    h = 1e-5   # differences: h^2 / 6 times third derivatives (< 1 each), and 1e-16 / h of rounding
    for e in range(24):
        lo, hi = l.copy(), l.copy()
        lo[:, e] -= h
        hi[:, e] += h
        diff = (loss(hi) - loss(lo)) / (2 * h)
        assert np.all(np.abs(d[:, e].double().cpu().numpy() - diff) <= 1e-9 + 2.0 ** -23 * 60 * np.abs(dw).max())


def test_many_tokens_and_graph(epx):
    """More tokens than one grid round; replays of a captured call equal the eager one."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    T, E, k = 70001, 64, 6
    l = torch.empty(T, E, device="cuda").normal_(generator=g)
    p = epx.make_problem(T, k, E, 1, 1)
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    epx.epx_route(p, l, epx.SCORE_SOFTMAX, idx, w)
    want = torch.sort(l, dim=1, descending=True, stable=True)
    assert torch.equal(idx, want.indices[:, :k].to(torch.int32))
    idx2, w2, d2 = torch.empty_like(idx), torch.empty_like(w), torch.empty_like(l)
    dw = torch.empty(T, k, device="cuda").normal_(generator=g)
    d = torch.empty_like(l)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        epx.epx_route(p, l, epx.SCORE_SOFTMAX, idx2, w2)
        epx.epx_route_backward(p, l, epx.SCORE_SOFTMAX, idx2, dw, d2)
    for _ in range(3):
        l.normal_(generator=g)
        epx.epx_route(p, l, epx.SCORE_SOFTMAX, idx, w)
        epx.epx_route_backward(p, l, epx.SCORE_SOFTMAX, idx, dw, d)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, idx2) and torch.equal(w, w2) and torch.equal(d, d2)
