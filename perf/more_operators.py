"""Cases for 8-bit integers in the experts' layer: rows and weights in int8 with
a scale for each token and channel and the experts' products on them, and
activations kept in 8 bits (blocks of 32 under a power of two) with the
gradients that use them.

Shapes follow this repository's workloads (hidden 7168, at most 256 rows on a
rank's 8 experts at decode, 4096-token batches of 8 copies on 16 experts) with
an expert width of 2048; the drawn cases spread over odd and ragged sizes
around them.

``run`` computes a case with elementary torch operations, or, where ``own``
is true, with the library's calls. ``exact`` computes the same outputs in 64
bits from the definitions.
"""
import math

import torch

own = False


def listed():
    return [
        # the rows of a decode step to int8 and back
        {"name": "int8_rows_decode", "op": "int8_rows", "rows": 128, "inner": 7168},
        # a batch's dispatched rows to int8 and back
        {"name": "int8_rows_batch", "op": "int8_rows", "rows": 32768, "inner": 7168},
        # decode on one of 32 ranks: 256 rows on 8 local experts, int8 weights are the traffic
        {"name": "int8_decode", "op": "int8", "rows": 256, "experts": 8, "zipf": 0.0, "width": 2048, "inner": 7168,
         "act": "swiglu", "keep": False},
        # the first product of a 4096-token batch on 16 local experts
        {"name": "int8_batch", "op": "int8", "rows": 32768, "experts": 16, "zipf": 0.0, "width": 2048, "inner": 7168,
         "act": "swiglu", "keep": False},
        # the activations of one expert kept in 8 bits, and read back
        {"name": "mxint8_expert", "op": "mxint8", "rows": 2048, "inner": 2048},
        # the dispatched rows of a batch kept in 8 bits, and read back
        {"name": "mxint8_batch", "op": "mxint8", "rows": 32768, "inner": 7168},
        # a small skewed layer of odd sizes, forwards
        {"name": "keep8_ragged", "op": "keep8", "rows": 1999, "experts": 24, "zipf": 1.0, "width": 544, "inner": 1048},
        # the first product of a training batch, keeping its pre-activations in 8 bits
        {"name": "keep8_batch", "op": "keep8", "rows": 32768, "experts": 16, "zipf": 0.0, "width": 2048, "inner": 7168},
        # the small layer backwards through its gated activation
        {"name": "dgrad8_ragged", "op": "dgrad8", "rows": 1999, "experts": 24, "zipf": 1.0, "width": 1048, "inner": 544},
        # the second product's input gradient through the pre-activations kept by the first, and its input again
        {"name": "dgrad8_batch", "op": "dgrad8", "rows": 32768, "experts": 16, "zipf": 0.0, "width": 7168, "inner": 2048},
        # the small layer's weight gradient in float32
        {"name": "wgrad8_ragged", "op": "wgrad8", "rows": 1999, "experts": 24, "zipf": 1.0, "width": 520, "inner": 1056,
         "dw": "f32"},
        # the first product's weight gradient from the dispatched rows kept in 8 bits
        {"name": "wgrad8_batch", "op": "wgrad8", "rows": 32768, "experts": 16, "zipf": 0.0, "width": 4096, "inner": 7168,
         "dw": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["int8_rows", "int8", "mxint8", "keep8", "dgrad8", "wgrad8"])
    if op == "int8_rows":
        return {"op": op, "rows": _log(rng, 1, 32768), "inner": 16 * _log(rng, 1, 448)}
    if op == "mxint8":
        return {"op": op, "rows": _log(rng, 1, 32768), "inner": 32 * _log(rng, 1, 224)}
    rows = _log(rng, 1, 32768)
    case = {"op": op, "rows": rows, "experts": _log(rng, 1, 64 if rows <= 4096 else 16),
            "zipf": rng.choice([0.0, 1.0]) if rows <= 4096 else 0.0}
    if op == "int8":
        case.update(act=rng.choice(["none", "swiglu"]), inner=16 * _log(rng, 4, 448))
        case["keep"] = case["act"] == "swiglu" and rng.random() < 0.4
        # kept blocks hold 32 neighbouring pre-activations
        case["width"] = 32 * _log(rng, 2, 64) if case["keep"] else 8 * _log(rng, 8, 256)
    elif op == "keep8":
        case.update(width=32 * _log(rng, 2, 64), inner=8 * _log(rng, 8, 896))
    elif op == "dgrad8":
        case.update(width=8 * _log(rng, 8, 896), inner=32 * _log(rng, 2, 64))
    else:
        case.update(width=8 * _log(rng, 8, 512), inner=32 * _log(rng, 2, 224), dw=rng.choice(["bf16", "f32"]))
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _ranges(case, g):
    """Rows per expert, one after another: uniform or skewed; small batches leave experts without rows."""
    n, rows = case["experts"], case["rows"]
    p = torch.arange(1, n + 1, device="cuda", dtype=torch.float64).pow(-case["zipf"])
    p = p[torch.randperm(n, device="cuda", generator=g)]
    count = torch.bincount(torch.multinomial(p, rows, replacement=True, generator=g), minlength=n)
    offset = count.cumsum(0) - count
    return offset.to(torch.int32), count.to(torch.int32)


def _rows_int8(x):
    """Rows in int8: a float32 scale max|x| / 127 (at least 2^-125; 0 for a row of zeros) and the nearest integers of
    the quotients, ties to even. A quotient next to a tie needs more than 32 bits; 64 tell all of them."""
    amax = x.float().abs().amax(-1)
    s = torch.where(amax > 0, (amax / 127.0).clamp(min=2.0 ** -125), 0.0)
    q = torch.round(x.double() / torch.where(s > 0, s, 1.0).double().unsqueeze(-1))
    return q.clamp(-127, 127).to(torch.int8), s


def _keep(z):
    """Values in 8 bits: per 32 the byte of 2^floor(log2 max|z|), at least 2^-127, and the nearest integers (ties to
    even) of 64 times the quotients, saturated at 127."""
    b = z.float().view(*z.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, (torch.frexp(amax).exponent - 1).clamp(min=-127), -127)
    q = torch.round(torch.ldexp(b, (6 - e).unsqueeze(-1))).clamp(-127, 127)
    return q.to(torch.int8).view(z.shape), (e + 127).to(torch.uint8)


def _kept(codes, scales):
    """The values kept, in float32 (every one is a bfloat16 number)."""
    b = codes.float().view(*scales.shape, 32)
    return torch.ldexp(b, (scales.to(torch.int32) - 133).unsqueeze(-1)).view(codes.shape)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op in ("int8_rows", "mxint8"):
        R, K = case["rows"], case["inner"]
        st["x"] = _normal(g, R, K)
        st["codes"] = _empty(R, K, dtype=torch.int8)
        st["scales"] = _empty(R, dtype=torch.float32) if op == "int8_rows" else _empty(R, K // 32, dtype=torch.uint8)
        st["out"] = _empty(R, K)
        return st
    n, R, N, K = case["experts"], case["rows"], case["width"], case["inner"]
    st["offset"], st["count"] = _ranges(case, g)
    st["most"] = int(st["count"].max())
    if op in ("int8", "keep8"):
        M = 2 * N if op == "keep8" or case["act"] == "swiglu" else N
        st["x"], st["weight"] = _normal(g, R, K), _normal(g, n, M, K, std=K ** -0.5)
        if op == "int8":
            # rows as the call before left them; weights laid out once
            st["x"], st["x_scales"] = _rows_int8(st["x"])
            codes, scales = zip(*(_rows_int8(w) for w in st["weight"]))
            st["weight"], st["w_scales"] = torch.stack(codes), torch.stack(scales)
        if op == "keep8" or case["keep"]:
            st["codes"], st["scales"] = _empty(R, M, dtype=torch.int8), _empty(R, M // 32, dtype=torch.uint8)
            st["preact"] = _empty(R, M)
        st["out"] = _empty(R, N)
    elif op == "dgrad8":
        st["dy"], st["weight"] = _normal(g, R, N), _normal(g, n, N, K, std=N ** -0.5)
        st["codes"], st["scales"] = _keep(_normal(g, R, 2 * K))
        st["act"], st["dx"] = _empty(R, K), _empty(R, 2 * K)
    else:
        st["dy"] = _normal(g, R, N)
        st["codes"], st["scales"] = _keep(_normal(g, R, K))
        st["dw"] = _empty(n, N, K, dtype=torch.float32 if case["dw"] == "f32" else torch.bfloat16)
    return st


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from combine_epx_get_amd import epx
    case = st["case"]
    op = case["op"]
    if op == "int8_rows":
        epx.epx_int8_quantize(st["x"], st["codes"], st["scales"])
        epx.epx_int8_dequantize(st["codes"], st["scales"], st["out"])
        return {"scales": st["scales"], "values": st["out"]}
    if op == "mxint8":
        epx.epx_mxint8_quantize(st["x"], st["codes"], st["scales"])
        epx.epx_mxint8_dequantize(st["codes"], st["scales"], st["out"])
        return {"values": st["out"]}
    rows = epx.expert_rows(st["offset"], st["count"], case["rows"])
    if op == "dgrad8":
        epx.epx_expert_gemm_dgrad_kept8(rows, st["dy"], st["weight"], st["codes"], st["scales"], st["dx"],
                                        act_out=st["act"])
        return {"dx": st["dx"], "act": st["act"]}
    if op == "wgrad8":
        epx.epx_expert_gemm_wgrad_kept8(rows, st["dy"], st["codes"], st["scales"], st["dw"])
        return {"dw": st["dw"]}
    if op == "keep8":
        epx.epx_expert_gemm_keep8(rows, st["x"], st["weight"], st["out"], st["codes"], st["scales"])
    else:
        epx.epx_expert_gemm_int8(rows, st["x"], st["x_scales"], st["weight"], st["w_scales"], st["out"],
                                 act=epx.ACT_SWIGLU if case["act"] == "swiglu" else epx.ACT_NONE,
                                 preact_codes=st.get("codes"), preact_scales=st.get("scales"))
        if not case["keep"]:
            return {"out": st["out"]}
    epx.epx_mxint8_dequantize(st["codes"], st["scales"], st["preact"])
    return {"out": st["out"], "preact": st["preact"]}


def _pad(x, st):
    """Float32 rows [experts, most, :] of each expert, zero behind its last one."""
    i = torch.arange(max(st["most"], 1), device=x.device)
    live = i < st["count"].long().unsqueeze(1)
    at = (st["offset"].long().unsqueeze(1) + i).clamp(max=x.shape[0] - 1)
    return x[at].float() * live.unsqueeze(2), at[live], live


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _run_plain(st):
    case = st["case"]
    op = case["op"]
    if op == "int8_rows":
        codes, scales = _rows_int8(st["x"])
        return {"scales": scales, "values": (codes.float() * scales.unsqueeze(1)).to(torch.bfloat16)}
    if op == "mxint8":
        return {"values": _kept(*_keep(st["x"])).to(torch.bfloat16)}
    N, K = case["width"], case["inner"]
    if op == "dgrad8":
        dy, at, live = _pad(st["dy"], st)
        d = torch.bmm(dy, st["weight"].float())[live]
        gate, up = _kept(st["codes"][at], st["scales"][at]).split(K, 1)
        s = 1.0 / (1.0 + torch.exp(-gate))
        act, dx = torch.empty_like(st["act"]), torch.empty_like(st["dx"])
        act[at] = (gate * s * up).to(torch.bfloat16)
        dx[at] = torch.cat((d * up * s * (1.0 + gate * (1.0 - s)), d * gate * s), 1).to(torch.bfloat16)
        return {"dx": dx, "act": act}
    if op == "wgrad8":
        dy, _, _ = _pad(st["dy"], st)
        x, _, _ = _pad(_kept(st["codes"], st["scales"]), st)
        return {"dw": torch.bmm(dy.transpose(1, 2).contiguous(), x).to(st["dw"].dtype)}
    # sums of products of int8 numbers are whole and stay below 2^24 here: float32 holds them exactly
    x, at, live = _pad(st["x"], st)
    z = torch.bmm(x, st["weight"].float().transpose(1, 2).contiguous())
    if op == "int8":
        sx, _, _ = _pad(st["x_scales"].unsqueeze(1), st)
        z = z * sx * st["w_scales"].unsqueeze(1)
    z = z[live]
    gated = op == "keep8" or case["act"] == "swiglu"
    out = torch.empty_like(st["out"])
    out[at] = (_silu(z[:, :N]) * z[:, N:] if gated else z).to(torch.bfloat16)
    if op == "int8" and not case["keep"]:
        return {"out": out}
    preact = torch.empty_like(st["preact"])
    preact[at] = _kept(*_keep(z)).to(torch.bfloat16)
    return {"out": out, "preact": preact}


def work(case):
    op = case["op"]
    R, K = case["rows"], case["inner"]
    if op == "int8_rows":
        return {"bytes": 6 * R * K + 8 * R, "flops": 4 * R * K}
    if op == "mxint8":
        return {"bytes": 6 * R * K + 2 * (R * K // 32), "flops": 4 * R * K}
    N, live = case["width"], min(case["experts"], R)   # no more experts have rows than there are rows
    flops = 2 * R * N * K
    if op == "dgrad8":
        return {"bytes": 2 * R * N + 2 * live * N * K + 2 * R * K * 33 // 32 + 6 * R * K, "flops": flops}
    if op == "wgrad8":
        return {"bytes": 2 * R * N + R * K * 33 // 32 + case["experts"] * N * K * (4 if case["dw"] == "f32" else 2),
                "flops": flops}
    M = 2 * N if op == "keep8" or case["act"] == "swiglu" else N
    if op == "keep8":
        moved = 2 * R * K + 2 * live * M * K + 2 * R * N
    else:
        moved = R * K + 4 * R + live * M * (K + 4) + 2 * R * N
    if op == "keep8" or case["keep"]:
        moved += 2 * (R * M * 33 // 32) + 2 * R * M   # kept, read back, and the values
    return {"bytes": moved, "flops": 2 * R * M * K}


def _steps_exact(v):
    """The nearest of the values that a block of 32 numbers can be kept as, from 64 bits; in parts."""
    res = []
    for part in v.split(max(1, (1 << 25) // v.shape[1])):
        b = part.reshape(part.shape[0], -1, 32)
        amax = b.abs().amax(2, keepdim=True)
        power = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0)))
        # a logarithm that rounding took to the next whole number
        power = torch.where(torch.exp2(power) > amax, power - 1, power).clamp(min=-127.0)
        step = torch.exp2(torch.where(amax > 0, power, -127.0) - 6.0)
        a = b.abs() / step
        low = torch.floor(a)
        up = (a - low > 0.5) | ((a - low == 0.5) & (low % 2 == 1))
        res.append((torch.where(up, low + 1, low).clamp(max=127.0) * step * torch.sign(b)).view(part.shape))
    return torch.cat(res)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "mxint8":
        return {"values": _steps_exact(st["x"].double())}
    if op == "int8_rows":
        scales, values = [], []
        for part in st["x"].split(4096):
            v = part.double()
            # the scale is a float32 number by definition
            s = torch.clamp(torch.linalg.vector_norm(v, float("inf"), dim=1) / 127.0, min=2.0 ** -125).float().double()
            s = torch.where((v == 0).all(1), 0.0, s)
            a = v.abs() / torch.where(s > 0, s, 1.0).unsqueeze(1)
            low = torch.floor(a)
            up = (a - low > 0.5) | ((a - low == 0.5) & (low % 2 == 1))
            scales.append(s)
            values.append(torch.where(up, low + 1, low).clamp(max=127.0) * torch.sign(v) * s.unsqueeze(1))
        return {"scales": torch.cat(scales), "values": torch.cat(values)}
    R, N, K = case["rows"], case["width"], case["inner"]
    new = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")   # noqa: E731
    ranges = list(enumerate(zip(st["offset"].tolist(), st["count"].tolist())))
    if op in ("dgrad8", "wgrad8"):
        v = st["codes"].double() * torch.exp2(st["scales"].double() - 133.0).repeat_interleave(32, 1)
        if op == "wgrad8":
            dw = new(*st["dw"].shape)
            for e, (o, c) in ranges:
                dw[e] = st["dy"][o:o + c].double().T @ v[o:o + c]
            return {"dw": dw}
        d = new(R, K)
        for e, (o, c) in ranges:
            d[o:o + c] = st["dy"][o:o + c].double() @ st["weight"][e].double()
        gate, up = v[:, :K], v[:, K:]
        s = torch.sigmoid(gate)
        return {"dx": torch.cat((d * up * (s + gate * s * (1 - s)), d * (gate * s)), 1), "act": up * (gate * s)}
    z = new(R, st["weight"].shape[1])
    for e, (o, c) in ranges:
        z[o:o + c] = st["x"][o:o + c].double() @ st["weight"][e].double().T
        if op == "int8":
            z[o:o + c] *= st["x_scales"][o:o + c].double().unsqueeze(1) * st["w_scales"][e].double()
    gated = op == "keep8" or case["act"] == "swiglu"
    out = z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:] if gated else z
    if op == "int8" and not case["keep"]:
        return {"out": out}
    return {"out": out, "preact": _steps_exact(z)}
