"""Combine's gradient on the GPU against 64-bit forms, for layouts of one and
several ranks, expert groups and relay mode, odd widths and many choices."""
import numpy as np
import pytest
import torch

from combine_epx_get_amd import workloads as W

pytestmark = pytest.mark.gpu
GUARD = -7.25


@pytest.fixture(scope="module")
def epx():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a visible GPU")
    from combine_epx_get_amd import epx as mod
    return mod


CASES = [
    # T, k, E, R, H, hidden, relay, groups
    (1, 1, 1, 1, 1, 8, False, 1),
    (1, 8, 16, 1, 1, 7168, False, 1),
    (3, 2, 16, 4, 2, 264, False, 1),
    (64, 2, 16, 4, 2, 256, True, 1),
    (50, 9, 32, 4, 1, 1032, False, 1),
    (7, 64, 128, 4, 2, 40, False, 1),
    (40, 17, 64, 4, 2, 4104, False, 4),
    (300, 8, 256, 16, 2, 520, False, 1),
    (2100, 4, 64, 1, 1, 136, False, 1),
    (2049, 11, 64, 1, 1, 8200, False, 1),
]


def setup(epx, case, seed=1, spare=3):
    T, k, E, R, H, h, relay, m = case
    print(f"[combine backward] {case}", flush=True)
    rng = np.random.Generator(np.random.PCG64(seed))
    idx = torch.from_numpy(W.draw_routing(rng, T, E, k, "uniform")).cuda()
    p = epx.make_problem(T, k, E, R, H, 0, epx.MODE_HOST_RELAY if relay else epx.MODE_PER_EXPERT, m)
    L = epx.Layout(p)
    epx.epx_get_layout(p, idx, L)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dout = torch.empty(T, h, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y = torch.empty(T * k + spare, h, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.from_numpy(W.draw_gate_weights(rng, T, k)).cuda()
    return p, L, idx, dout, y, w


@pytest.mark.parametrize("case", CASES, ids=str)
def test_against_64_bits(epx, case):
    p, L, idx, dout, y, w = setup(epx, case)
    T, k, h = p.num_tokens, p.topk, dout.shape[1]
    dy, only = torch.full_like(y, GUARD), torch.full_like(y, GUARD)
    dw = torch.full((T, k), GUARD, device="cuda")
    epx.epx_combine_backward(p, L, dout, y, w, dy, dw)
    epx.epx_combine_backward(p, L, dout, None, w, only)
    torch.cuda.synchronize()
    slot = L["slot"].view(T, k).long()
    want = w.double().unsqueeze(2) * dout.double().unsqueeze(1)
    got = dy[slot].double()
    # one product, rounded to float32 and to bf16
    assert bool(((got - want).abs() <= (2.0 ** -8 + 2.0 ** -23) * want.abs() + 1e-38).all())
    assert torch.equal(dy[T * k:], torch.full_like(dy[T * k:], GUARD))
    assert torch.equal(dy, only)
    prod = y[slot].double() * dout.double().unsqueeze(1)
    bound = prod.abs().sum(2) * (h * 2.0 ** -24) + 1e-38
    assert bool(((dw.double() - prod.sum(2)).abs() <= bound).all())
    again = torch.empty_like(dw)
    epx.epx_combine_backward(p, L, dout, y, w, dy, again)
    torch.cuda.synchronize()
    assert torch.equal(dw, again)


def test_duplicate_ids(epx):
    """An expert given twice has two rows; each gets its own weight's gradient."""
    T, k, E, h = 5, 4, 8, 64
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    idx[:, 2:] = 3
    p = epx.make_problem(T, k, E, 1, 1)
    L = epx.Layout(p)
    epx.epx_get_layout(p, idx, L)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    dout = torch.empty(T, h, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y = torch.empty(T * k, h, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(T, k, device="cuda", generator=g)
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    epx.epx_combine_backward(p, L, dout, y, w, dy, dw)
    torch.cuda.synchronize()
    slot = L["slot"].view(T, k).long()
    assert slot.unique().numel() == T * k
    assert torch.equal(dy[slot], (w.unsqueeze(2) * dout.float().unsqueeze(1)).to(torch.bfloat16))


def test_bad_ids_write_nothing(epx):
    p, L, idx, dout, y, w = setup(epx, (6, 3, 16, 1, 1, 64, False, 1))
    idx[4, 1] = 16
    epx.epx_get_layout(p, idx, L)
    dy, dw = torch.full_like(y, GUARD), torch.full_like(w, GUARD)
    epx.epx_combine_backward(p, L, dout, y, w, dy, dw)
    torch.cuda.synchronize()
    assert bool((dy == GUARD).all()) and bool((dw == GUARD).all())
    assert epx.epx_read_error(L) == 1


def test_gradient_against_differences(epx):
    """combine is linear in y and in the weights: its differences against the gradient call."""
    p, L, idx, dout, y, w = setup(epx, (33, 5, 16, 1, 1, 136, False, 1), spare=0)
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    epx.epx_combine_backward(p, L, dout, y, w, dy, dw)

    def out(yy, ww):
        o = torch.empty_like(dout)
        epx.epx_combine(p, L, yy, ww, o)
        torch.cuda.synchronize()
        return o.double()

    base = out(y, w)
    step = torch.rand_like(w) - 0.5
    w2 = w + step
    far = out(y, w2)
    noise = float(((base.abs() + far.abs()) * dout.double().abs()).sum()) * 2.0 ** -7
    diff, grad = float(((far - base) * dout.double()).sum()), float(((w2 - w).double() * dw.double()).sum())
    assert abs(diff - grad) <= noise
    y2 = (y.float() + torch.randn_like(y.float())).to(torch.bfloat16)
    far = out(y2, w)
    move = y2.double() - y.double()
    noise = float(((base.abs() + far.abs()) * dout.double().abs()).sum()) * 2.0 ** -7
    noise += float((move * dy.double()).abs().sum()) * 2.0 ** -7
    diff, grad = float(((far - base) * dout.double()).sum()), float((move * dy.double()).sum())
    assert abs(diff - grad) <= noise


def test_graph(epx):
    p, L, idx, dout, y, w = setup(epx, (40, 8, 64, 1, 1, 520, False, 1))
    a, da = torch.empty_like(y), torch.empty_like(w)
    b, db = torch.full_like(y, GUARD), torch.empty_like(w)
    a.fill_(GUARD)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        epx.epx_combine_backward(p, L, dout, y, w, b, db)
    for _ in range(3):
        dout.normal_()
        epx.epx_combine_backward(p, L, dout, y, w, a, da)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(da, db)
