"""Rows in 8 bits on the GPU against their definitions in 64 bits: every code,
scale and value equal."""
import pytest
import torch

from tests import rows8_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def epx():
    if not torch.cuda.is_available():
        raise RuntimeError("GPU tests need a visible GPU")
    from combine_epx_get_amd import epx as mod
    return mod


def bits(a):
    """bf16 numbers of these patterns (any integers of 16 bits)."""
    return torch.as_tensor(a, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()


def quantize(epx, form, x):
    lead, inner = tuple(x.shape[:-1]), x.shape[-1]
    codes = torch.full(lead + (inner,), 77, dtype=torch.int8, device="cuda")
    scales = (torch.full(lead, 5.0, device="cuda") if form == "int8"
              else torch.full(lead + (inner // 32,), 99, dtype=torch.uint8, device="cuda"))
    getattr(epx, f"epx_{form}_quantize")(x, codes, scales)
    torch.cuda.synchronize()
    return codes, scales


def check(epx, form, x):
    print(f"[rows8] {form} {tuple(x.shape)}", flush=True)
    codes, scales = quantize(epx, form, x)
    want_codes, want_scales = (ref.int8_rows if form == "int8" else ref.mxint8)(x)
    ref.same(scales, want_scales, "scales")
    ref.same(codes, want_codes, "codes")
    out = torch.full_like(x, 3.5)
    getattr(epx, f"epx_{form}_dequantize")(codes, scales, out)
    torch.cuda.synchronize()
    if form == "int8":
        # the float32 product rounds once more before bf16 does; that is the definition's product in float32
        ref.same(out, (codes.float() * scales.unsqueeze(-1)).to(torch.bfloat16), "values")
        v = codes.double() * scales.double().unsqueeze(-1)
        live = torch.isfinite(v)
        assert bool(((out.double() - v).abs()[live] <= v.abs()[live] * (2.0 ** -8 + 2.0 ** -23) + 2.0 ** -133).all())
    else:
        ref.same(out, ref.mxint8_values(codes, scales), "values")
    return codes, scales, out


def random(shape, seed, std=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)


# every number of lanes that a row of int8 can take, rows that end inside a workgroup, rows longer than it holds
INT8_SHAPES = [(1, 16), (3, 16), (257, 16), (65, 128), (1, 144), (33, 512), (7, 528), (5, 2048), (9, 2064), (3, 7168),
               (130, 8192), (2, 8208), (3, 32768), (2, 32784), (1, 131056), (1, 1 << 20), (0, 64), (4, 3, 48)]
MX_SHAPES = [(1, 32), (3, 32), (257, 32), (65, 96), (33, 544), (5, 2048), (3, 7168), (130, 8224), (1, 1 << 20), (0, 64),
             (4, 3, 64)]


@pytest.mark.parametrize("form,shape", [("int8", s) for s in INT8_SHAPES] + [("mxint8", s) for s in MX_SHAPES], ids=str)
def test_rows(epx, form, shape):
    check(epx, form, random(shape, sum(shape)))


@pytest.mark.parametrize("binade", [0, 1, 7, 8, 9, 14, 15, 16, 127, 253, 254], ids=str)
def test_int8_every_pair(epx, binade):
    """Every bf16 magnitude up to each largest one of a binade, in both signs: quotients next to every tie."""
    x = torch.zeros(128, 1 << 16, dtype=torch.int32)
    for m in range(128):
        top = (binade << 7) | m
        p = torch.arange(1 << 15).clamp(max=top)
        x[m] = torch.cat((p, p | 0x8000))
    check(epx, "int8", bits(x).view(128, 1 << 16))


@pytest.mark.parametrize("binade", [0, 1, 5, 6, 7, 8, 127, 253, 254], ids=str)
def test_mxint8_every_pair(epx, binade):
    """The same for blocks: each holds its largest magnitude and 31 of the smaller ones (those down to 2^-9 of it)."""
    top = torch.arange(128).repeat_interleave(64) | (binade << 7)   # 64 blocks a largest magnitude
    below = (torch.arange(64).view(-1, 1) * 31 + torch.arange(31)).repeat(128, 1)
    p = torch.cat((top.view(-1, 1), (top.view(-1, 1) - below).clamp(min=0)), 1)
    sign = (torch.arange(p.numel()).view(p.shape) * 7 % 3 == 1).int() << 15
    check(epx, "mxint8", bits(p.int() | sign).view(128, 64 * 32))


def test_infinities_nan_and_zeros(epx):
    inf, nan = float("inf"), float("nan")
    x = random((12, 96), 4)
    x[1], x[2], x[3, 5], x[4, 40], x[5, 95], x[6] = 0, -0.0, inf, -inf, nan, nan
    x[7, :64], x[8, 32:] = 0, 0
    x[9] = torch.finfo(torch.bfloat16).max
    x[10] = -torch.finfo(torch.bfloat16).max
    x[11] = 2.0 ** -133
    for form in ("int8", "mxint8"):
        codes, scales, out = check(epx, form, x)
        odd = torch.isnan(out.float())
        if form == "int8":
            assert odd[3:7].all() and not odd[7:].any() and not odd[:3].any()
            assert not codes[3:7].any()
        else:
            blocks = odd.view(12, 3, 32)
            want = torch.zeros(12, 3, dtype=torch.bool, device="cuda")
            want[3, 0] = want[4, 1] = want[5, 2] = True
            want[6] = True
            assert torch.equal(blocks.all(2), want) and torch.equal(blocks.any(2), want)
            assert bool((scales[want] == 255).all())


def test_mxint8_reads_every_code(epx):
    """Every code under every scale byte is read back as what it stands for; 127 * 2^121 is the largest."""
    codes = torch.arange(-128, 128, dtype=torch.int8, device="cuda").repeat(256, 1).contiguous()
    scales = torch.arange(256, device="cuda").to(torch.uint8).view(-1, 1).repeat(1, 8).contiguous()
    out = torch.empty(256, 256, dtype=torch.bfloat16, device="cuda")
    epx.epx_mxint8_dequantize(codes, scales, out)
    torch.cuda.synchronize()
    want = ref.mxint8_values(codes, scales)
    want[254, 0] = -float("inf")   # -128 * 2^121 = -2^128
    ref.same(out, want, "values")


def test_int8_reads_scales_of_any_origin(epx):
    """Scales that the conversion never gives: negative, infinite, NaN, tiny."""
    codes = torch.arange(-128, 128, dtype=torch.int8, device="cuda").repeat(8, 1).contiguous()
    scales = torch.tensor([-2.0, float("inf"), float("nan"), 2.0 ** -149, 0.0, 3.1e38, 1 / 3, -0.0], device="cuda")
    out = torch.empty(8, 256, dtype=torch.bfloat16, device="cuda")
    epx.epx_int8_dequantize(codes, scales, out)
    torch.cuda.synchronize()
    ref.same(out, (codes.float() * scales.unsqueeze(1)).to(torch.bfloat16), "values")


@pytest.mark.parametrize("form", ["int8", "mxint8"])
def test_neighbours_stay(epx, form):
    """What lies before and behind a call's rows is not written."""
    x = random((40, 160), 9)
    codes = torch.full((44, 160), 77, dtype=torch.int8, device="cuda")
    scales = (torch.full((44,), 5.0, device="cuda") if form == "int8"
              else torch.full((44, 5), 99, dtype=torch.uint8, device="cuda"))
    out = torch.full((44, 160), 3.5, dtype=torch.bfloat16, device="cuda")
    part = slice(2, 42)
    getattr(epx, f"epx_{form}_quantize")(x, codes[part], scales[part])
    getattr(epx, f"epx_{form}_dequantize")(codes[part], scales[part], out[part])
    torch.cuda.synchronize()
    for t, v in ((codes, 77), (scales, 5.0 if form == "int8" else 99), (out, 3.5)):
        assert bool((t[:2] == v).all()) and bool((t[42:] == v).all())


@pytest.mark.parametrize("form", ["int8", "mxint8"])
def test_on_another_stream_and_in_a_graph(epx, form):
    x = random((300, 1056), 11)
    codes, scales, out = check(epx, form, x)
    s = torch.cuda.Stream()
    c2, s2, o2 = torch.empty_like(codes), torch.empty_like(scales), torch.empty_like(out)
    q, d = getattr(epx, f"epx_{form}_quantize"), getattr(epx, f"epx_{form}_dequantize")
    s.wait_stream(torch.cuda.current_stream())
    q(x, c2, s2, stream=s)
    d(c2, s2, o2, stream=s)
    s.synchronize()
    assert torch.equal(codes, c2) and torch.equal(scales, s2) and torch.equal(out, o2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q(x, c2, s2)
        d(c2, s2, o2)
    y = random((300, 1056), 12)
    want = None
    for i in range(4):
        x.copy_(y if i % 2 else random((300, 1056), 11))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (c2, s2, o2)]
        want = check(epx, form, x)
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
