"""The experts' products and their gradients on the GPU against 64-bit
products, at ragged, empty, single and scattered row ranges, sizes that end
inside tiles, and buffers with guard rows that must stay as they were."""
import numpy as np
import pytest
import torch

from tests import experts_reference as ref

pytestmark = pytest.mark.gpu
GUARD = -7.25   # a bf16 value


@pytest.fixture(scope="module")
def epx():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a visible GPU")
    from combine_epx_get_amd import epx as mod
    return mod


def rand(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0, std, generator=g)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make_rows(epx, off, cnt, R):
    return epx.expert_rows(torch.tensor(off, dtype=torch.int32, device="cuda"),
                           torch.tensor(cnt, dtype=torch.int32, device="cuda"), R)


def guard(*shape, dtype=torch.bfloat16):
    return torch.full(shape, GUARD, dtype=dtype, device="cuda")


def untouched(t, off, cnt, name):
    live = torch.zeros(t.shape[0], dtype=torch.bool, device=t.device)
    for o, c in zip(off, cnt):
        live[o:o + c] = True
    assert torch.equal(t[~live], torch.full_like(t[~live], GUARD)), name


# counts, gap between ranges, order of ranges in memory, width, inner. The
# average rows per expert, the number of tiles and the length of the sum choose
# the kernel: few rows or tiles the small ones, the last cases the larger ones.
CASES = [
    ("one row", [1], 0, None, 8, 8),
    ("one row each", [1, 1, 1, 1], 0, None, 40, 72),
    ("no rows at all", [0, 0, 0], 3, None, 64, 64),
    ("few rows, empty experts", [0, 7, 0, 33, 1, 0, 16, 0], 2, None, 264, 200),
    ("decode, long sum", [5, 0, 2, 31], 0, None, 136, 1048),
    ("middle, odd sizes", [17, 90, 0, 64, 65], 1, [3, 0, 4, 1, 2], 520, 328),
    ("middle, one step", [40, 50], 0, None, 256, 64),
    ("large tiles, partial", [130, 257, 511, 1], 0, None, 264, 136),
    ("large tiles, one over", [256, 257], 5, [1, 0], 512, 72),
    ("large tiles, long sum", [300], 0, None, 384, 2056),
    ("skewed", [1200, 3, 0, 1, 700, 2], 0, None, 136, 264),
    ("many experts", [i % 5 for i in range(200)], 0, None, 72, 64),
    ("more experts than lanes, large", [150 + (i * 37) % 90 for i in range(70)], 0, None, 64, 72),
    ("wide", [3, 2], 0, None, 4104, 24),
    ("150 experts, every kind of last tile", [(i * 53) % 300 for i in range(150)], 1, None, 264, 520),
    ("very wide", [700, 300], 0, [1, 0], 16392, 136),
    ("very long sum", [700, 300], 2, None, 136, 16392),
    ("few tiles, a sum that ends inside a group's step", [33, 0, 64, 7], 1, None, 264, 2104),
    ("64 experts", [(i * 53) % 128 for i in range(64)], 0, None, 520, 328),
    ("middle, wide", [40, 0, 64, 65, 90, 31, 2, 130], 0, None, 2056, 2056),
    ("five experts, wide", [100, 0, 60, 200, 64], 0, None, 1032, 1032),
    ("few experts, many rows", [2100, 0, 1900], 0, None, 520, 2056),
    ("four experts, long sums", [900, 0, 33, 700], 0, None, 1096, 1096),
    ("24 experts, large tiles, every kind of last one", [(i * 53) % 300 for i in range(24)], 1, None, 2056, 2056),
    ("square tiles, odd sizes", [1500, 0, 901, 303], 1, None, 1800, 1672),
]
IDS = [c[0] for c in CASES]


def setup(epx, case, seed):
    name, cnt, gap, order, N, K = case
    off, R = ref.ranges(cnt, gap, order)
    print(f"[experts] {name} R={R} n={len(cnt)} N={N} K={K}", flush=True)
    return gen(seed), off, cnt, R, N, K, make_rows(epx, off, cnt, R)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward(epx, case, act):
    g, off, cnt, R, N, K, rows = setup(epx, case, 1)
    M = 2 * N if act == "swiglu" else N
    x, w = rand(g, R, K), rand(g, len(cnt), M, K, std=K ** -0.5)
    out = guard(R, N)
    z, b = ref.product(x.double(), w.double(), off, cnt)
    if act == "none":
        epx.epx_expert_gemm(rows, x, w, out)
        torch.cuda.synchronize()
        ref.close(out, z, b, ref.BF16, "out")
        untouched(out, off, cnt, "out")
        return
    pre = guard(R, M)
    epx.epx_expert_gemm(rows, x, w, out, act=epx.ACT_SWIGLU, preact=pre)
    only = guard(R, N)
    epx.epx_expert_gemm(rows, x, w, only, act=epx.ACT_SWIGLU)
    torch.cuda.synchronize()
    ref.close(pre, z, b, ref.BF16, "preact")
    a, ba = ref.glu(z, b)
    ref.close(out, a, ba, ref.BF16, "out")
    untouched(out, off, cnt, "out")
    untouched(pre, off, cnt, "preact")
    assert torch.equal(out, only)


@pytest.mark.parametrize("act", ["none", "swiglu"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_input_gradient(epx, case, act):
    g, off, cnt, R, N, K, rows = setup(epx, case, 2)
    dy, w = rand(g, R, N), rand(g, len(cnt), N, K, std=N ** -0.5)
    d, b = ref.product(dy.double(), w.double().transpose(1, 2), off, cnt)
    if act == "none":
        dx = guard(R, K)
        epx.epx_expert_gemm_dgrad(rows, dy, w, dx)
        torch.cuda.synchronize()
        ref.close(dx, d, b, ref.BF16, "dx")
    else:
        pre = rand(g, R, 2 * K, std=2.0)
        dx = guard(R, 2 * K)
        epx.epx_expert_gemm_dgrad(rows, dy, w, dx, input_act=epx.ACT_SWIGLU, preact=pre)
        torch.cuda.synchronize()
        ref.close(dx, *ref.glu_backward(d, b, pre.double()), ref.BF16, "dx")
    untouched(dx, off, cnt, "dx")


@pytest.mark.parametrize("kind", ["bf16", "f32", "accumulate"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_weight_gradient(epx, case, kind):
    g, off, cnt, R, N, K, rows = setup(epx, case, 3)
    dy, x = rand(g, R, N), rand(g, R, K)
    dw = guard(len(cnt), N, K, dtype=torch.bfloat16 if kind == "bf16" else torch.float32)
    epx.epx_expert_gemm_wgrad(rows, dy, x, dw, accumulate=kind == "accumulate")
    torch.cuda.synchronize()
    base = GUARD if kind == "accumulate" else 0.0
    for e, (o, c) in enumerate(zip(off, cnt)):
        a, v = dy[o:o + c].double(), x[o:o + c].double()
        want, bound = a.T @ v + base, a.abs().T @ v.abs() * (ref.SUM * max(c, 1))
        if kind == "accumulate":
            bound = bound + ref.SUM * (want.abs() + bound)
        ref.close(dw[e], want, bound, ref.BF16 if kind == "bf16" else 2.0 ** -24, ("dw", e))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_large_tiles_weight_gradient(epx, dtype):
    """The larger weight-gradient tiles (long sums, hundreds of tiles), sizes that end inside them."""
    g = gen(4)
    cnt = [900, 0, 1300, 700, 1005, 5]
    off, R = ref.ranges(cnt, 1)
    N, K = 2056, 2056
    rows = make_rows(epx, off, cnt, R)
    dy, x = rand(g, R, N), rand(g, R, K)
    dw = guard(len(cnt), N, K, dtype=dtype)
    epx.epx_expert_gemm_wgrad(rows, dy, x, dw)
    torch.cuda.synchronize()
    for e, (o, c) in enumerate(zip(off, cnt)):
        a, v = dy[o:o + c].double(), x[o:o + c].double()
        ref.close(dw[e], a.T @ v, a.abs().T @ v.abs() * (ref.SUM * max(c, 1)),
                  ref.BF16 if dtype == torch.bfloat16 else 2.0 ** -24, ("dw", e))


def test_ranges_outside_the_buffers_count_as_empty(epx):
    """Offsets and counts that no buffer holds: negative, past the end, summing past 2^31."""
    g = gen(5)
    R, N, K = 64, 40, 72
    off = [0, -4, 60, 70, 20, 2 ** 31 - 8, 30]
    cnt = [10, 8, 5, 1, -3, 100, 12]
    rows = make_rows(epx, off, cnt, R)
    x, w = rand(g, R, K), rand(g, len(cnt), N, K)
    out, dx = guard(R, N), guard(R, K)
    dw = guard(len(cnt), N, K, dtype=torch.float32)
    dy = rand(g, R, N)
    epx.epx_expert_gemm(rows, x, w, out)
    epx.epx_expert_gemm_dgrad(rows, dy, w, dx)
    epx.epx_expert_gemm_wgrad(rows, dy, x, dw)
    torch.cuda.synchronize()
    good = [c if e in (0, 6) else 0 for e, c in enumerate(cnt)]
    safe = [o if e in (0, 6) else 0 for e, o in enumerate(off)]
    ref.close(out, *ref.product(x.double(), w.double(), safe, good), ref.BF16, "out")
    ref.close(dx, *ref.product(dy.double(), w.double().transpose(1, 2), safe, good), ref.BF16, "dx")
    untouched(out, safe, good, "out")
    untouched(dx, safe, good, "dx")
    assert not dw[[1, 2, 3, 4, 5]].any()


def test_extreme_values(epx):
    """Infinities and NaN stay in their own rows; saturated gates give no NaN."""
    g = gen(6)
    cnt = [6, 5]
    off, R = ref.ranges(cnt)
    N, K = 48, 104
    rows = make_rows(epx, off, cnt, R)
    x, w = rand(g, R, K), rand(g, 2, 2 * N, K)
    want = guard(R, N)
    epx.epx_expert_gemm(rows, x, w, want, act=epx.ACT_SWIGLU)
    x2 = x.clone()
    x2[2, 100], x2[7, 0] = float("nan"), float("inf")
    out = guard(R, N)
    epx.epx_expert_gemm(rows, x2, w, out, act=epx.ACT_SWIGLU)
    torch.cuda.synchronize()
    keep = [r for r in range(R) if r not in (2, 7)]
    assert torch.equal(out[keep], want[keep])
    assert torch.isnan(out[2]).all()
    # gates of +-10^4: silu is the gate, or 0
    big = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    big[:, 0] = 1.0
    w3 = torch.zeros_like(w)
    w3[:, :N, 0] = torch.where(torch.arange(N, device="cuda") % 2 == 0, 1e4, -1e4).to(torch.bfloat16)
    w3[:, N:, 0] = 1.0
    epx.epx_expert_gemm(rows, big, w3, out, act=epx.ACT_SWIGLU)
    torch.cuda.synchronize()
    assert torch.equal(out[0].float(), w3[0, :N, 0].float().clamp(min=0))


def test_repeats_bitwise(epx):
    """The same call twice gives the same bits (fixed order of every sum)."""
    g = gen(7)
    cnt = [300, 0, 77, 5]
    off, R = ref.ranges(cnt)
    rows = make_rows(epx, off, cnt, R)
    x, w, dy = rand(g, R, 520), rand(g, 4, 264, 520), rand(g, R, 264)
    got = []
    for _ in range(2):
        out, dx, dw = guard(R, 264), guard(R, 520), guard(4, 264, 520, dtype=torch.float32)
        epx.epx_expert_gemm(rows, x, w, out)
        epx.epx_expert_gemm_dgrad(rows, dy, w, dx)
        epx.epx_expert_gemm_wgrad(rows, dy, x, dw)
        torch.cuda.synchronize()
        got.append((out, dx, dw))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(epx):
    """Rows whose byte offset passes 2^32, and weights whose expert starts there."""
    g = gen(8)
    N, K = 1024, 8192
    R = 300000                       # x: 4.9e9 bytes
    cnt = [3, 0, 200, 60]
    off = [5, 0, R - 260, R - 60]
    rows = make_rows(epx, off, cnt, R)
    x = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    for o, c in zip(off, cnt):
        x[o:o + c] = rand(g, c, K)
    w = rand(g, 4, N, K, std=K ** -0.5)
    out = guard(R, N)
    epx.epx_expert_gemm(rows, x, w, out)
    torch.cuda.synchronize()
    for e, (o, c) in enumerate(zip(off, cnt)):
        z, b = ref.product(x[o:o + c].double(), w[e:e + 1].double(), [0], [c])
        ref.close(out[o:o + c], z, b, ref.BF16, "out")
    dy = rand(g, R, N)
    dw = guard(4, N, K, dtype=torch.float32)
    epx.epx_expert_gemm_wgrad(rows, dy, x, dw)
    torch.cuda.synchronize()
    for e, (o, c) in enumerate(zip(off, cnt)):
        a, v = dy[o:o + c].double(), x[o:o + c].double()
        ref.close(dw[e], a.T @ v, a.abs().T @ v.abs() * (ref.SUM * max(c, 1)), 2.0 ** -24, ("dw", e))


def test_graph_and_other_stream(epx):
    """Captured and replayed, with eager work between the replays; and on a side stream."""
    g = gen(9)
    cnt = [60, 3, 0, 140]
    off, R = ref.ranges(cnt)
    rows = make_rows(epx, off, cnt, R)
    x, w, dy = rand(g, R, 200), rand(g, 4, 2 * 136, 200), rand(g, R, 136)
    w2 = rand(g, 4, 136, 200)

    def go(out, pre, dx, dw):
        epx.epx_expert_gemm(rows, x, w, out, act=epx.ACT_SWIGLU, preact=pre)
        epx.epx_expert_gemm_dgrad(rows, dy, w2, dx)
        epx.epx_expert_gemm_wgrad(rows, dy, x, dw)

    def bufs():
        return guard(R, 136), guard(R, 272), guard(R, 200), guard(4, 136, 200, dtype=torch.float32)

    want = bufs()
    go(*want)
    side, other = torch.cuda.Stream(), bufs()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(*other)
    torch.cuda.synchronize()
    for a, b in zip(want, other):
        assert torch.equal(a, b)
    cap = bufs()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(*cap)
    for i in range(4):
        for t in cap:
            t.fill_(GUARD)
        x.copy_(rand(g, R, 200))
        go(*want)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, cap):
            assert torch.equal(a, b), i


def test_two_streams_at_once(epx):
    """Calls that overlap on two streams share nothing."""
    g = gen(10)
    sets = []
    for i in range(2):
        cnt = [200 + 50 * i, 0, 33]
        off, R = ref.ranges(cnt)
        rows = make_rows(epx, off, cnt, R)
        x, w = rand(g, R, 1032), rand(g, 3, 520, 1032)
        want, out = guard(R, 520), guard(R, 520)
        epx.epx_expert_gemm(rows, x, w, want)
        sets.append((rows, x, w, want, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for rows, x, w, want, out, s in sets:
            epx.epx_expert_gemm(rows, x, w, out, stream=s)
    torch.cuda.synchronize()
    for rows, x, w, want, out, s in sets:
        assert torch.equal(out, want)


def test_gradient_against_differences(epx):
    """Directional differences of the forward call agree with the gradient calls' results."""
    g = gen(11)
    cnt = [20, 0, 9]
    off, R = ref.ranges(cnt)
    rows = make_rows(epx, off, cnt, R)
    N, K = 72, 104
    x, w, dy = rand(g, R, K), rand(g, 3, N, K, std=K ** -0.5), rand(g, R, N)
    dx, dw = guard(R, K), guard(3, N, K, dtype=torch.float32)
    epx.epx_expert_gemm_dgrad(rows, dy, w, dx)
    epx.epx_expert_gemm_wgrad(rows, dy, x, dw)

    def loss(xx, ww):
        out = guard(R, N)
        epx.epx_expert_gemm(rows, xx, ww, out)
        return out.double()

    # the map is linear in x and in w: f(a + b) - f(a) is exact up to the
    # bf16 rounding of both outputs (half a step each) and of a + b
    step = rand(g, R, K)
    xs = (x.float() + step.float()).to(torch.bfloat16)
    real = xs.double() - x.double()
    a, b = loss(xs, w), loss(x, w)
    diff = ((a - b) * dy.double()).sum()
    grad = (real * dx.double()).sum()
    noise = ((a.abs() + b.abs()) * dy.double().abs()).sum() * ref.BF16 * 2 + (real.abs() * dx.double().abs()).sum() * ref.BF16 * 2
    assert abs(float(diff - grad)) <= float(noise)
    # the noise bound must be able to tell: a wrong sign or factor is larger
    assert float(noise) < 0.5 * float((real.abs() * dx.double().abs()).sum())
    ws = (w.float() + rand(g, 3, N, K, std=K ** -0.5).float()).to(torch.bfloat16)
    real = ws.double() - w.double()
    a = loss(x, ws)
    diff, grad = ((a - b) * dy.double()).sum(), (real * dw.double()).sum()
    noise = ((a.abs() + b.abs()) * dy.double().abs()).sum() * ref.BF16 * 2
    assert abs(float(diff - grad)) <= float(noise)
