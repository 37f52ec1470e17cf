"""Whole expert layers in 8-bit integers: a training step that keeps its
activations in 8 bits, a serving step on int8 rows and weights, and both forms
together; against 64-bit layers of the values that were kept."""
import pytest
import torch

from tests import experts_reference as ref
from tests import rows8_reference as r8
from tests.test_experts8_gpu import int8_sums
from tests.test_layer_gpu import Layer, epx, gen, near, rand  # noqa: F401

pytestmark = pytest.mark.gpu


class Kept(Layer):
    """The training step of Layer, which holds its rows and pre-activations in 8 bits between the passes."""

    def __init__(self, epx, T, E, k, h, width, seed, int8=False):  # noqa: F811
        super().__init__(epx, T, E, k, h, width, seed)
        R = T * k
        new = lambda *s, dtype: torch.full(s, 7, dtype=dtype, device="cuda")   # noqa: E731
        self.xc, self.xs = new(R, h, dtype=torch.int8), new(R, h // 32, dtype=torch.uint8)
        self.pc, self.ps = new(R, 2 * width, dtype=torch.int8), new(R, 2 * width // 32, dtype=torch.uint8)
        self.int8 = int8
        if int8:
            self.q, self.qs = new(R, h, dtype=torch.int8), new(R, dtype=torch.float32)
            self.w1c, self.w1s = new(E, 2 * width, h, dtype=torch.int8), new(E, 2 * width, dtype=torch.float32)
            epx.epx_int8_quantize(self.w1, self.w1c, self.w1s)

    def forward(self):
        epx = self.epx  # noqa: F811
        epx.epx_route(self.p, self.logits, epx.SCORE_SOFTMAX, self.idx, self.wt)
        epx.epx_layout_dispatch(self.p, self.idx, self.L, self.x, epx.BF16, self.recv)
        epx.epx_mxint8_quantize(self.recv, self.xc, self.xs)
        if self.int8:
            epx.epx_int8_quantize(self.recv, self.q, self.qs)
            epx.epx_expert_gemm_int8(self.rows, self.q, self.qs, self.w1c, self.w1s, self.a, act=epx.ACT_SWIGLU,
                                     preact_codes=self.pc, preact_scales=self.ps)
        else:
            epx.epx_expert_gemm_keep8(self.rows, self.recv, self.w1, self.a, self.pc, self.ps)
        epx.epx_expert_gemm(self.rows, self.a, self.w2, self.y)
        epx.epx_combine(self.p, self.L, self.y, self.wt, self.out)

    def backward(self):
        epx = self.epx  # noqa: F811
        epx.epx_combine_backward(self.p, self.L, self.dout, self.y, self.wt, self.dy, self.dwt)
        # the activation comes again with the gradient: a is not held between the passes
        epx.epx_expert_gemm_dgrad_kept8(self.rows, self.dy, self.w2, self.pc, self.ps, self.dpre, act_out=self.a)
        epx.epx_expert_gemm_wgrad(self.rows, self.dy, self.a, self.dw2)
        epx.epx_expert_gemm_wgrad_kept8(self.rows, self.dpre, self.xc, self.xs, self.dw1)
        epx.epx_expert_gemm_dgrad(self.rows, self.dpre, self.w1, self.drecv)
        epx.epx_combine(self.p, self.L, self.drecv, self.ones, self.dx)
        epx.epx_route_backward(self.p, self.logits, epx.SCORE_SOFTMAX, self.idx, self.dwt, self.dlogits)

    def results(self):
        return super().results() + [self.xc, self.xs, self.pc, self.ps, self.a]


def check_gradients(lay):
    """Gradients by the formulas in 64 bits from the values that were kept."""
    E, k, T = lay.E, lay.k, lay.T
    slot = lay.L["slot"].view(T, k).long()
    off, cnt = lay.L["expert_offset"].tolist()[:E], lay.L["expert_count"].tolist()
    x, pre = r8.mxint8_values(lay.xc, lay.xs), r8.mxint8_values(lay.pc, lay.ps)
    dy = torch.empty_like(x)
    dy[slot.flatten()] = (lay.wt.double().unsqueeze(2) * lay.dout.double().unsqueeze(1)).view(T * k, -1)
    W = lay.width
    g, u = pre[:, :W], pre[:, W:]
    s = torch.sigmoid(g)
    act = g * s * u
    drecv = torch.empty_like(x)
    dw1, dw2 = torch.zeros_like(lay.w1, dtype=torch.float64), torch.zeros_like(lay.w2, dtype=torch.float64)
    for e, (o, c) in enumerate(zip(off, cnt)):
        r = slice(o, o + c)
        d = dy[r] @ lay.w2[e].double()
        dpre = torch.cat((d * u[r] * s[r] * (1 + g[r] * (1 - s[r])), d * g[r] * s[r]), 1)
        dw2[e], dw1[e] = dy[r].T @ act[r], dpre.T @ x[r]
        drecv[r] = dpre @ lay.w1[e].double()
    dx = drecv[slot].sum(1)
    near(lay.a, act, 1, "act")
    near(lay.dw2, dw2, 2, "dw2")     # dy, a
    near(lay.dw1, dw1, 2, "dw1")     # dy, dpre
    near(lay.dx, dx, 4, "dx")        # dy, dpre, drecv, dx
    return dx, dw1, dw2


SHAPES = [(1, 8, 2, 64, 32), (33, 16, 4, 288, 160), (300, 24, 6, 544, 288), (64, 64, 8, 1024, 256)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_training_step(epx, shape):  # noqa: F811
    T, E, k, h, width = shape
    print(f"[kept layer] {shape}", flush=True)
    lay = Kept(epx, T, E, k, h, width, seed=T)
    lay.forward()
    lay.backward()
    plain = Layer(epx, T, E, k, h, width, seed=T)
    plain.forward()
    plain.backward()
    torch.cuda.synchronize()
    assert epx.epx_read_error(lay.L) == 0
    near(lay.out, plain.out.double(), 6, "out")   # three roundings on either side
    dx, dw1, dw2 = check_gradients(lay)
    # what is kept is off by half a step, 2^-7 of a block's largest magnitude at most, which for blocks of 32 normal
    # values is about twice their root mean square: 2^-6 in the 2-norm of each, for rows and pre-activations; the
    # gradients of the step that keeps bf16 are off by their own roundings
    for name, got, want, kept in (("dx", lay.dx, plain.dx, 1), ("dw1", lay.dw1, plain.dw1, 2), ("dw2", lay.dw2, plain.dw2, 1)):
        d = float((got.double() - want.double()).norm() / want.double().norm())
        assert d <= 2 * (kept * 2.0 ** -6 + 10 * 2.0 ** -8), (name, d)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_training_step_on_int8_rows(epx, shape):  # noqa: F811
    """Forwards on int8, backwards through what that forward kept."""
    T, E, k, h, width = shape
    print(f"[int8 kept layer] {shape}", flush=True)
    lay = Kept(epx, T, E, k, h, width, seed=T + 1, int8=True)
    lay.forward()
    lay.backward()
    torch.cuda.synchronize()
    off, cnt = lay.L["expert_offset"].tolist()[:E], lay.L["expert_count"].tolist()
    codes, scales = r8.int8_rows(lay.recv)
    r8.same(lay.q, codes, "rows")
    r8.same(lay.qs, scales, "scales")
    z = int8_sums(lay.q, lay.w1c, lay.qs, lay.w1s, off, cnt)
    want_codes, want_scales = r8.mxint8(z)
    r8.same(lay.ps, want_scales, "kept scales")
    r8.same(lay.pc, want_codes, "kept")
    check_gradients(lay)


def test_training_step_repeats_and_in_a_graph(epx):  # noqa: F811
    """The same step eagerly, again, and replayed from a graph with eager work between: the same bits."""
    for int8 in (False, True):
        lay = Kept(epx, 128, 32, 4, 288, 160, seed=5, int8=int8)
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
            lay.backward()
            torch.cuda.synchronize()
            for a, b in zip(lay.results(), want):
                assert torch.equal(a, b), i


def test_two_layers_on_two_streams(epx):  # noqa: F811
    """Two steps at once, each on a stream of its own: each one's bits are those it has alone."""
    lays = [Kept(epx, 200, 16, 4, 544, 288, seed=s) for s in (1, 2)]
    want = []
    for lay in lays:
        lay.forward()
        lay.backward()
        torch.cuda.synchronize()
        want.append([t.clone() for t in lay.results()])
    streams = [torch.cuda.Stream() for _ in lays]
    for lay in lays:
        for t in lay.results():
            t.fill_(1)
    torch.cuda.synchronize()
    for _ in range(3):
        for lay, s in zip(lays, streams):
            with torch.cuda.stream(s):
                lay.forward()
                lay.backward()
    torch.cuda.synchronize()
    for lay, w in zip(lays, want):
        for a, b in zip(lay.results(), w):
            assert torch.equal(a, b)


@pytest.mark.parametrize("shape", [(1, 8, 2, 256, 128), (40, 16, 4, 512, 264), (700, 8, 4, 1024, 384)], ids=str)
def test_serving_step(epx, shape):  # noqa: F811
    """Two products on int8 rows and weights, rows to int8 before each; weights converted once."""
    T, E, k, h, width = shape
    width = width // 16 * 16
    print(f"[int8 layer] {shape}", flush=True)
    g = gen(T)
    p = epx.make_problem(T, k, E, 1, 1)
    L = epx.Layout(p)
    R = T * k
    x, logits = rand(g, T, h), rand(g, T, E)
    w = [rand(g, E, 2 * width, h, std=h ** -0.5), rand(g, E, h, width, std=width ** -0.5)]
    i8 = lambda *s: torch.empty(*s, dtype=torch.int8, device="cuda")   # noqa: E731
    f32 = lambda *s: torch.empty(*s, device="cuda")   # noqa: E731
    wc, ws = [i8(*t.shape) for t in w], [f32(*t.shape[:2]) for t in w]
    for t, c, s in zip(w, wc, ws):
        epx.epx_int8_quantize(t, c, s)
    idx, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), f32(T, k)
    recv, a, y = (torch.empty(R, n, dtype=torch.bfloat16, device="cuda") for n in (h, width, h))
    out = torch.empty(T, h, dtype=torch.bfloat16, device="cuda")
    q, qs, aq, aqs = i8(R, h), f32(R), i8(R, width), f32(R)
    rows = epx.expert_rows(L["expert_offset"], L["expert_count"], R)
    epx.epx_route(p, logits, epx.SCORE_SIGMOID, idx, wt, scale=2.5)
    epx.epx_layout_dispatch(p, idx, L, x, epx.BF16, recv)
    epx.epx_int8_quantize(recv, q, qs)
    epx.epx_expert_gemm_int8(rows, q, qs, wc[0], ws[0], a, act=epx.ACT_SWIGLU)
    epx.epx_int8_quantize(a, aq, aqs)
    epx.epx_expert_gemm_int8(rows, aq, aqs, wc[1], ws[1], y)
    epx.epx_combine(p, L, y, wt, out)
    torch.cuda.synchronize()
    off, cnt = L["expert_offset"].tolist()[:E], L["expert_count"].tolist()
    z = int8_sums(q, wc[0], qs, ws[0], off, cnt)
    act, bound = ref.glu(z.double(), torch.zeros_like(z, dtype=torch.float64))
    ref.close(a, act, bound, ref.BF16, "a")
    codes, scales = r8.int8_rows(a)
    r8.same(aq, codes, "rows")
    r8.same(aqs, scales, "scales")
    r8.same(y, int8_sums(aq, wc[1], aqs, ws[1], off, cnt).to(torch.bfloat16), "y")
    parts = y.double()[L["slot"].view(T, k).long()] * wt.double().unsqueeze(2)
    want, slack = parts.sum(1), parts.abs().sum(1) * k * 2.0 ** -23
    assert bool(((out.double() - want).abs() <= slack + 2.0 ** -8 * (want.abs() + slack)).all())


def test_one_expert_group_at_a_time(epx):  # noqa: F811
    """Ranges that are part of a layer's: the halves one after another give the whole call's bits."""
    lay = Kept(epx, 96, 16, 4, 288, 160, seed=6, int8=True)
    lay.forward()
    lay.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in (lay.a, lay.pc, lay.ps, lay.dpre, lay.dw1)]
    for t in (lay.a, lay.pc, lay.ps, lay.dpre, lay.dw1):
        t.fill_(1)
    for part in (slice(8, 16), slice(0, 8)):
        rows = epx.expert_rows(lay.L["expert_offset"][part], lay.L["expert_count"][part], lay.T * lay.k)
        epx.epx_expert_gemm_int8(rows, lay.q, lay.qs, lay.w1c[part], lay.w1s[part], lay.a, act=epx.ACT_SWIGLU,
                                 preact_codes=lay.pc, preact_scales=lay.ps)
        epx.epx_expert_gemm_dgrad_kept8(rows, lay.dy, lay.w2[part], lay.pc, lay.ps, lay.dpre, act_out=lay.a)
        epx.epx_expert_gemm_wgrad_kept8(rows, lay.dpre, lay.xc, lay.xs, lay.dw1[part])
    torch.cuda.synchronize()
    got = [lay.a, lay.pc, lay.ps]
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # other tiles, other orders of float32 sums
    near(lay.dpre, want[3].double(), 2, "dpre")
    near(lay.dw1, want[4].double(), 2, "dw1")


def test_an_empty_batch(epx):  # noqa: F811
    rows = epx.expert_rows(torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"), 0)
    z = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device="cuda")   # noqa: E731
    i8, u8, f = torch.int8, torch.uint8, torch.float32
    epx.epx_expert_gemm_int8(rows, z(0, 64, dtype=i8), z(0, dtype=f), z(2, 64, 64, dtype=i8), z(2, 64, dtype=f), z(0, 32),
                             act=epx.ACT_SWIGLU, preact_codes=z(0, 64, dtype=i8), preact_scales=z(0, 2, dtype=u8))
    epx.epx_expert_gemm_keep8(rows, z(0, 64), z(2, 64, 64), z(0, 32), z(0, 64, dtype=i8), z(0, 2, dtype=u8))
    epx.epx_expert_gemm_dgrad_kept8(rows, z(0, 64), z(2, 64, 32), z(0, 64, dtype=i8), z(0, 2, dtype=u8), z(0, 64))
    acc = torch.full((2, 64, 32), 5.0, device="cuda")
    epx.epx_expert_gemm_wgrad_kept8(rows, z(0, 64), z(0, 32, dtype=i8), z(0, 1, dtype=u8), acc, accumulate=True)
    torch.cuda.synchronize()
    assert bool((acc == 5.0).all())
