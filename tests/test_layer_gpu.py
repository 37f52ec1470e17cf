"""Whole expert layers through the library's calls: router, layout and
dispatch, the experts' products and combine, forwards and backwards in bf16,
and the serving form with fp8 rows and 4-bit weights; against 64-bit layers."""
import numpy as np
import pytest
import torch

from tests import experts_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def epx():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a visible GPU")
    from combine_epx_get_amd import epx as mod
    return mod


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rand(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0, std, generator=g)


class Layer:
    """One GPU's layer: every buffer and call of a step, as a user holds them."""

    def __init__(self, epx, T, E, k, h, width, seed, groups=1):
        g = gen(seed)
        self.epx, self.T, self.E, self.k, self.h, self.width = epx, T, E, k, h, width
        self.p = epx.make_problem(T, k, E, 1, 1, 0, epx.MODE_PER_EXPERT, groups)
        self.L = epx.Layout(self.p)
        R = T * k
        self.x = rand(g, T, h)
        self.logits = rand(g, T, E, dtype=torch.float32)
        self.w1, self.w2 = rand(g, E, 2 * width, h, std=h ** -0.5), rand(g, E, h, width, std=width ** -0.5)
        self.dout = rand(g, T, h)
        new = lambda *s, dtype=torch.bfloat16: torch.full(s, 3.5, dtype=dtype, device="cuda")   # noqa: E731
        self.idx, self.wt = new(T, k, dtype=torch.int32), new(T, k, dtype=torch.float32)
        self.recv, self.pre, self.a, self.y, self.out = new(R, h), new(R, 2 * width), new(R, width), new(R, h), new(T, h)
        self.dy, self.dpre, self.drecv, self.dx = new(R, h), new(R, 2 * width), new(R, h), new(T, h)
        self.dw1, self.dw2 = new(E, 2 * width, h, dtype=torch.float32), new(E, h, width, dtype=torch.float32)
        self.dwt, self.dlogits = new(T, k, dtype=torch.float32), new(T, E, dtype=torch.float32)
        self.ones = torch.ones(T, k, device="cuda")
        self.rows = epx.expert_rows(self.L["expert_offset"], self.L["expert_count"], R)

    def forward(self):
        epx = self.epx
        epx.epx_route(self.p, self.logits, epx.SCORE_SOFTMAX, self.idx, self.wt)
        epx.epx_layout_dispatch(self.p, self.idx, self.L, self.x, epx.BF16, self.recv)
        epx.epx_expert_gemm(self.rows, self.recv, self.w1, self.a, act=epx.ACT_SWIGLU, preact=self.pre)
        epx.epx_expert_gemm(self.rows, self.a, self.w2, self.y)
        epx.epx_combine(self.p, self.L, self.y, self.wt, self.out)

    def backward(self):
        epx = self.epx
        epx.epx_combine_backward(self.p, self.L, self.dout, self.y, self.wt, self.dy, self.dwt)
        epx.epx_expert_gemm_wgrad(self.rows, self.dy, self.a, self.dw2)
        epx.epx_expert_gemm_dgrad(self.rows, self.dy, self.w2, self.dpre, input_act=epx.ACT_SWIGLU, preact=self.pre)
        epx.epx_expert_gemm_wgrad(self.rows, self.dpre, self.recv, self.dw1)
        epx.epx_expert_gemm_dgrad(self.rows, self.dpre, self.w1, self.drecv)
        epx.epx_combine(self.p, self.L, self.drecv, self.ones, self.dx)
        epx.epx_route_backward(self.p, self.logits, epx.SCORE_SOFTMAX, self.idx, self.dwt, self.dlogits)

    def results(self):
        return [self.idx, self.wt, self.out, self.dx, self.dw1, self.dw2, self.dlogits]


def reference(lay):
    """The layer and its gradients in float64 by autograd, for the routing that the layer chose."""
    leaf = lambda t: t.double().clone().requires_grad_()   # noqa: E731
    x, logits, w1, w2 = leaf(lay.x), leaf(lay.logits), leaf(lay.w1), leaf(lay.w2)
    idx = lay.idx.long()
    chosen = logits.gather(1, idx)
    wt = torch.softmax(chosen, 1)
    out = torch.zeros_like(x)
    for e in range(lay.E):
        t, j = (idx == e).nonzero(as_tuple=True)
        if t.numel() == 0:
            continue
        z = x[t] @ w1[e].T
        a = torch.nn.functional.silu(z[:, :lay.width]) * z[:, lay.width:]
        out = out.index_add(0, t, wt[t, j].unsqueeze(1) * (a @ w2[e].T))
    out.backward(lay.dout.double())
    return out.detach(), x.grad, w1.grad, w2.grad, logits.grad


def near(got, want, steps, name):
    """In the 2-norm: `steps` roundings to bf16 in a row, of at most half a step (2^-8) each relative to the value, whose
    errors are carried on by products that neither enlarge nor shrink them on the whole (random operands of unit gain);
    twice that is allowed."""
    d = float((got.double() - want).norm() / want.norm())
    assert d <= 2 * steps * 2.0 ** -8, (name, d)


@pytest.mark.parametrize("shape", [(1, 8, 2, 64, 40), (33, 16, 4, 264, 136), (300, 24, 6, 520, 264), (64, 64, 8, 1024, 256)],
                         ids=str)
def test_training_step(epx, shape):
    T, E, k, h, width = shape
    print(f"[layer] {shape}", flush=True)
    lay = Layer(epx, T, E, k, h, width, seed=T)
    lay.forward()
    lay.backward()
    torch.cuda.synchronize()
    assert epx.epx_read_error(lay.L) == 0
    want_idx = torch.sort(lay.logits, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(lay.idx.long(), want_idx)
    out, dx, dw1, dw2, dl = reference(lay)
    near(lay.out, out, 3, "out")            # a, y, out
    near(lay.dw2, dw2, 2, "dw2")            # a, dy
    near(lay.dx, dx, 5, "dx")               # pre, dy, dpre, drecv, dx
    near(lay.dw1, dw1, 3, "dw1")            # pre, dy, dpre
    near(lay.dlogits, dl, 3, "dlogits")     # a, y (twice: the mean is taken from each)


def test_training_step_repeats_and_in_a_graph(epx):
    """The same step eagerly, again, and replayed from a graph with eager work between: the same bits."""
    lay = Layer(epx, 128, 32, 4, 264, 136, seed=5)
    lay.forward()
    lay.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in lay.results()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lay.forward()
        lay.backward()
    for i in range(4):
        for t in lay.results():
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(lay.results(), want):
            assert torch.equal(a, b), i
        lay.forward()
        torch.cuda.synchronize()
        assert torch.equal(lay.out, want[2])


def test_expert_groups_one_after_another(epx):
    """Two expert groups: each group's dispatch, products and combine in turn give the ungrouped layer's output."""
    T, E, k, h, width = 96, 16, 4, 264, 136
    plain = Layer(epx, T, E, k, h, width, seed=6)
    plain.forward()
    lay = Layer(epx, T, E, k, h, width, seed=6, groups=2)
    epx.epx_route(lay.p, lay.logits, epx.SCORE_SOFTMAX, lay.idx, lay.wt)
    epx.epx_get_layout(lay.p, lay.idx, lay.L)
    carry = torch.zeros(T, h, device="cuda")
    half = E // 2
    for grp in range(2):
        part = slice(grp * half, (grp + 1) * half)
        rows = epx.expert_rows(lay.L["expert_offset"][part], lay.L["expert_count"][part], T * k)
        epx.epx_dispatch_group(lay.p, lay.L, grp, lay.x, epx.BF16, lay.recv)
        epx.epx_expert_gemm(rows, lay.recv, lay.w1[part], lay.a, act=epx.ACT_SWIGLU)
        epx.epx_expert_gemm(rows, lay.a, lay.w2[part], lay.y)
        epx.epx_combine_group(lay.p, lay.L, grp, lay.y, lay.wt, carry, lay.out)
    torch.cuda.synchronize()
    # the rows' products are the same sums whatever the tile they fall in;
    # combine adds a token's rows group by group
    near(lay.out, plain.out.double(), 1, "out")


@pytest.mark.parametrize("shape", [(1, 8, 2, 256, 128), (40, 16, 4, 512, 256), (700, 8, 4, 1024, 384)], ids=str)
def test_serving_step_fp8_rows_4_bit_weights(epx, shape):
    """fp8 dispatch, two products with 4-bit weights (fp8 rows between them), combine."""
    T, E, k, h, width = shape
    print(f"[serving layer] {shape}", flush=True)
    g = gen(T)
    p = epx.make_problem(T, k, E, 1, 1)
    L = epx.Layout(p)
    R = T * k
    x, logits, bias = rand(g, T, h), rand(g, T, E), rand(g, E, std=0.1, dtype=torch.float32)
    w = [rand(g, E, 2 * width, h, std=h ** -0.5), rand(g, E, h, width, std=width ** -0.5)]
    codes = [torch.empty(*t.shape[:-1], t.shape[-1] // 2, dtype=torch.uint8, device="cuda") for t in w]
    scales = [torch.empty(*t.shape[:-1], t.shape[-1] // 32, dtype=torch.uint8, device="cuda") for t in w]
    for t, c, s in zip(w, codes, scales):
        epx.epx_mxfp4_quantize(t, c, s)
    idx, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    q, qs = torch.empty(R, h, dtype=torch.uint8, device="cuda"), torch.empty(R, h // 128, device="cuda")
    a, as_ = torch.empty(R, width, dtype=torch.uint8, device="cuda"), torch.empty(R, width // 128, device="cuda")
    y, out = torch.empty(R, h, dtype=torch.bfloat16, device="cuda"), torch.empty(T, h, dtype=torch.bfloat16, device="cuda")
    rows = epx.expert_rows(L["expert_offset"], L["expert_count"], R)
    epx.epx_route(p, logits, epx.SCORE_SIGMOID, idx, wt, bias=bias, scale=2.5)
    epx.epx_layout_dispatch(p, idx, L, x, epx.FP8_E4M3, q, qs)
    epx.epx_expert_gemm_mxfp4(rows, q, qs, codes[0], scales[0], a, act=epx.ACT_SWIGLU, out_scales=as_)
    epx.epx_expert_gemm_mxfp4(rows, a, as_, codes[1], scales[1], y)
    epx.epx_combine(p, L, y, wt, out)
    torch.cuda.synchronize()
    # router
    key = torch.sigmoid(logits.double()) + bias.double()
    want_idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(idx.long(), want_idx)
    sc = torch.sigmoid(logits.double()).gather(1, want_idx)
    ww = 2.5 * sc / sc.sum(1, keepdim=True)
    assert float((wt.double() - ww).abs().max()) <= 2.0 ** -20
    # the layer with the same quantised rows, activations and weights
    off, cnt = L["expert_offset"].tolist()[:E], L["expert_count"].tolist()
    v = (q.view(torch.float8_e4m3fn).double().view(R, -1, 128) * qs.double().unsqueeze(2)).view(R, h)
    z, b = ref.product(v, ref.mxfp4_values(codes[0], scales[0]), off, cnt)
    act, bact = ref.glu(z, b)
    av = (a.view(torch.float8_e4m3fn).double().view(R, -1, 128) * as_.double().unsqueeze(2)).view(R, width)
    s = as_.double().repeat_interleave(128, 1)
    assert bool(((av - act).abs() <= bact + 2.0 ** -4 * (act.abs() + bact) + s * 2.0 ** -10 + 2.0 ** -21 * act.abs()).all())
    yv, by = ref.product(av, ref.mxfp4_values(codes[1], scales[1]), off, cnt)
    ref.close(y, yv, by, ref.BF16, "y")
    want = (y.double()[L["slot"].view(T, k).long()] * wt.double().unsqueeze(2)).sum(1)
    size = (y.double()[L["slot"].view(T, k).long()].abs() * wt.double().unsqueeze(2)).sum(1)
    assert bool(((out.double() - want).abs() <= size * k * 2.0 ** -23 + 2.0 ** -8 * (want.abs() + size * k * 2.0 ** -23)).all())


def test_rows_of_an_empty_batch(epx):
    """No tokens: no call launches anything but the weights' gradients, which are zero."""
    p = epx.make_problem(0, 2, 8, 1, 1)
    L = epx.Layout(p)
    z = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")   # noqa: E731
    epx.epx_route(p, z(0, 8), epx.SCORE_SOFTMAX, z(0, 2, dtype=torch.int32), z(0, 2, dtype=torch.float32))
    epx.epx_get_layout(p, z(0, 2, dtype=torch.int32), L)
    rows = epx.expert_rows(L["expert_offset"], L["expert_count"], 0)
    w = rand(gen(1), 8, 64, 64)
    epx.epx_expert_gemm(rows, z(0, 64), w, z(0, 64))
    epx.epx_expert_gemm_dgrad(rows, z(0, 64), w, z(0, 64))
    dw = torch.full((8, 64, 64), 5.0, device="cuda")
    epx.epx_expert_gemm_wgrad(rows, z(0, 64), z(0, 64), dw)
    acc = torch.full((8, 64, 64), 5.0, device="cuda")
    epx.epx_expert_gemm_wgrad(rows, z(0, 64), z(0, 64), acc, accumulate=True)
    epx.epx_combine_backward(p, L, z(0, 64), None, z(0, 2, dtype=torch.float32), z(0, 64))
    torch.cuda.synchronize()
    assert not dw.any() and bool((acc == 5.0).all())
