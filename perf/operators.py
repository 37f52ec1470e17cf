"""Cases for the operators around the expert-parallel exchange: the router in
front of dispatch, the experts' products between dispatch and combine, their
gradients, combine's gradient, and expert weights held in microscaled 4-bit
floating point.

Shapes follow this repository's workloads (hidden 7168, 256 experts, top-8,
at most 128 tokens per GPU at decode, 4096-token batches) with an expert
width of 2048; the drawn cases spread over odd and ragged sizes around them.

``run`` computes a case with elementary torch operations, or, where ``own``
is true, with the library's calls. ``exact`` computes the same outputs in 64
bits from the definitions.
"""
import math

import numpy as np
import torch

own = False

# The values of the 4-bit codes 0..7 (E2M1); codes 8..15 are their negatives.
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the router of one decode step: 128 tokens, biased sigmoid scores
        {"name": "route_decode", "op": "route", "tokens": 128, "experts": 256, "topk": 8, "score": "sigmoid",
         "biased": True, "renorm": True, "scale": 2.5, "dtype": "bf16", "grad": False},
        # the router of a training batch with its gradient
        {"name": "route_train", "op": "route", "tokens": 16384, "experts": 256, "topk": 8, "score": "softmax",
         "biased": False, "renorm": True, "scale": 1.0, "dtype": "f32", "grad": True},
        # combine's gradient for the 384 tokens of a loaded source rank
        {"name": "combine_bwd_rank", "op": "combine_bwd", "tokens": 384, "experts": 256, "topk": 8, "hidden": 7168},
        # combine's gradient for the 4096-token batch
        {"name": "combine_bwd_batch", "op": "combine_bwd", "tokens": 4096, "experts": 256, "topk": 8, "hidden": 7168},
        # decode on one of 32 ranks: 32 tokens per GPU, 8 local experts, 256 rows: the weights are the traffic
        {"name": "experts_decode", "op": "experts", "rows": 256, "experts": 8, "zipf": 0.0, "width": 2048,
         "inner": 7168, "act": "swiglu", "train": False},
        # the first product of a 4096-token batch on 16 local experts, keeping what its gradient needs
        {"name": "experts_batch", "op": "experts", "rows": 32768, "experts": 16, "zipf": 0.0, "width": 2048,
         "inner": 7168, "act": "swiglu", "train": True},
        # gradients of a small skewed layer of odd sizes, float32 weight gradients
        {"name": "experts_bwd_ragged", "op": "experts_bwd", "rows": 1999, "experts": 24, "zipf": 1.0, "width": 520,
         "inner": 1048, "act": "none", "dw": "f32"},
        # gradients of the second product through the gated activation of the first
        {"name": "experts_bwd_batch", "op": "experts_bwd", "rows": 16384, "experts": 8, "zipf": 0.0, "width": 7168,
         "inner": 2048, "act": "swiglu", "dw": "bf16"},
        # 4-bit form of one expert's matrix, and back
        {"name": "mxfp4_expert", "op": "mxfp4", "rows": 2048, "inner": 7168},
        # 4-bit form of a rank's first matrices, and back
        {"name": "mxfp4_rank", "op": "mxfp4", "rows": 65536, "inner": 7168},
        # decode rows of the fp8 dispatch against 4-bit weights
        {"name": "mx_experts_decode", "op": "mx_experts", "rows": 64, "experts": 8, "zipf": 0.0, "width": 2048,
         "inner": 7168, "act": "swiglu"},
        # the fp8 dispatch of a 4096-token batch against 4-bit weights
        {"name": "mx_experts_batch", "op": "mx_experts", "rows": 32768, "experts": 16, "zipf": 0.0, "width": 2048,
         "inner": 7168, "act": "swiglu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "combine_bwd", "experts", "experts_bwd", "mxfp4", "mx_experts"])
    if op == "route":
        experts = _log(rng, 2, 512)
        score = rng.choice(["softmax", "sigmoid"])
        topk = rng.randint(1, min(16, experts))
        # a single weight that is normalised is the scale itself, and its gradient nothing
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": experts, "topk": topk, "score": score,
                "biased": score == "sigmoid" and rng.random() < 0.5, "renorm": topk > 1 and rng.random() < 0.7,
                "scale": rng.choice([1.0, 2.5]), "dtype": rng.choice(["bf16", "f32"]), "grad": rng.random() < 0.5}
    if op == "combine_bwd":
        experts = _log(rng, 4, 256)
        return {"op": op, "tokens": _log(rng, 1, 4096), "experts": experts, "topk": rng.randint(1, min(8, experts)),
                "hidden": 8 * _log(rng, 16, 896)}
    if op == "mxfp4":
        return {"op": op, "rows": _log(rng, 1, 65536), "inner": 128 * rng.randint(1, 56)}
    rows = _log(rng, 1, 32768)
    case = {"op": op, "rows": rows, "experts": _log(rng, 1, 64 if rows <= 4096 else 16),
            "zipf": rng.choice([0.0, 1.0]) if rows <= 4096 else 0.0}
    if op == "mx_experts":
        case.update(width=8 * _log(rng, 8, 256), inner=128 * _log(rng, 1, 56), act=rng.choice(["none", "swiglu"]))
    else:
        case.update(width=8 * _log(rng, 8, 256), inner=8 * _log(rng, 8, 896))
        case["act"] = rng.choice(["none", "swiglu"])
        if op == "experts":
            case["train"] = case["act"] == "swiglu" and rng.random() < 0.5
        else:
            case["dw"] = rng.choice(["bf16", "f32"])
            if case["act"] == "swiglu":
                case["width"], case["inner"] = case["inner"], case["width"]
    return case


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _routing(g, tokens, experts, topk):
    """Distinct experts per token, as a router gives them."""
    keys = torch.rand(tokens, experts, device="cuda", generator=g)
    return keys.topk(topk, dim=1).indices.to(torch.int32).contiguous()


def _ranges(case, g):
    """Rows per expert, one after another: uniform or skewed; small batches leave experts without rows."""
    n, rows = case["experts"], case["rows"]
    p = torch.arange(1, n + 1, device="cuda", dtype=torch.float64).pow(-case["zipf"])
    p = p[torch.randperm(n, device="cuda", generator=g)]
    of = torch.multinomial(p, rows, replacement=True, generator=g)
    count = torch.bincount(of, minlength=n)
    offset = count.cumsum(0) - count
    return offset.to(torch.int32), count.to(torch.int32)


def _to_fp8(x):
    """bf16 rows as the fp8 dispatch delivers them: E4M3 codes and a float32 scale per 128 channels."""
    b = x.float().view(x.shape[0], -1, 128)
    s = b.abs().amax(2) / 448.0
    q = (b / torch.where(s > 0, s, 1.0).unsqueeze(2)).clamp(-448.0, 448.0)
    return q.view(x.shape).to(torch.float8_e4m3fn).view(torch.uint8), s


def _to_mxfp4(x):
    """Rows in 4 bits: per 32 values the scale 2^(floor(log2 max) - 2) as a biased exponent byte, and E2M1 codes
    rounded to nearest even, saturated at 6, two to a byte (the even value in the low half)."""
    b = x.float().view(x.shape[0], -1, 32)
    amax = b.abs().amax(2)
    e = (torch.frexp(amax).exponent - 3).clamp(min=-127)
    e = torch.where(amax > 0, e, -127)
    v = torch.ldexp(b, -e.unsqueeze(2))
    a = v.abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    r = (torch.round(a / step) * step).clamp(max=6.0)
    c = torch.where(r < 2.0, 2.0 * r, torch.where(r < 4.0, r + 2.0, r * 0.5 + 4.0)).to(torch.uint8)
    c = (c | torch.where(torch.signbit(b), 8, 0).to(torch.uint8)).view(x.shape[0], -1, 2)
    return (c[..., 0] | (c[..., 1] << 4)).contiguous(), (e + 127).to(torch.uint8)


def _from_mxfp4(codes, scales, dtype):
    """The values that 4-bit codes [..., inner/2] with scales [..., inner/32] stand for."""
    c = torch.stack((codes & 15, codes >> 4), -1).long()
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    v = lut[c].view(*scales.shape, 32)
    return torch.ldexp(v, (scales.to(torch.int32) - 127).unsqueeze(-1)).to(dtype).flatten(-2)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dev = "cuda"
    st = {"case": case}
    if op == "route":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        st["logits"] = _normal(g, case["tokens"], case["experts"], std=1.5, dtype=dt)
        st["bias"] = _normal(g, case["experts"], std=0.1, dtype=torch.float32) if case["biased"] else None
        st["idx"] = torch.empty(case["tokens"], case["topk"], dtype=torch.int32, device=dev)
        st["w"] = torch.empty(case["tokens"], case["topk"], dtype=torch.float32, device=dev)
        st["dw"] = _normal(g, case["tokens"], case["topk"], dtype=torch.float32)
        st["dlogits"] = torch.empty_like(st["logits"])
    elif op == "combine_bwd":
        T, k, h = case["tokens"], case["topk"], case["hidden"]
        idx = _routing(g, T, case["experts"], k)
        # the layout's order: rows by expert, then token, then position
        order = torch.sort(idx.flatten().long(), stable=True).indices
        slot = torch.empty_like(order)
        slot[order] = torch.arange(T * k, device=dev)
        st["idx"], st["slot"] = idx, slot.view(T, k)
        st["w"] = torch.softmax(_normal(g, T, k, dtype=torch.float32), 1)
        st["dout"] = _normal(g, T, h)
        st["y"] = _normal(g, T * k, h)
        st["dy"] = torch.empty(T * k, h, dtype=torch.bfloat16, device=dev)
        st["dw"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        if own:
            # the forward pass made the layout
            from combine_epx_get_amd import epx
            st["problem"] = epx.make_problem(T, k, case["experts"], 1, 1)
            st["layout"] = epx.Layout(st["problem"])
            epx.epx_get_layout(st["problem"], idx, st["layout"])
    elif op == "mxfp4":
        R, K = case["rows"], case["inner"]
        st["x"] = _normal(g, R, K, std=0.02)
        st["codes"] = torch.empty(R, K // 2, dtype=torch.uint8, device=dev)
        st["scales"] = torch.empty(R, K // 32, dtype=torch.uint8, device=dev)
        st["out"] = torch.empty_like(st["x"])
    else:
        n, R, N, K = case["experts"], case["rows"], case["width"], case["inner"]
        gated = case["act"] == "swiglu"
        st["offset"], st["count"] = _ranges(case, g)
        st["most"] = int(st["count"].max())
        if op == "experts":
            M = 2 * N if gated else N
            st["x"] = _normal(g, R, K)
            st["weight"] = _normal(g, n, M, K, std=K ** -0.5)
            st["preact"] = torch.empty(R, M, dtype=torch.bfloat16, device=dev) if case["train"] else None
            st["out"] = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
        elif op == "experts_bwd":
            st["dy"] = _normal(g, R, N)
            st["x"] = _normal(g, R, K)
            st["weight"] = _normal(g, n, N, K, std=N ** -0.5)
            st["preact"] = _normal(g, R, 2 * K) if gated else None
            st["dx"] = torch.empty(R, 2 * K if gated else K, dtype=torch.bfloat16, device=dev)
            st["dw"] = torch.empty(n, N, K, device=dev, dtype=torch.float32 if case["dw"] == "f32" else torch.bfloat16)
        else:
            M = 2 * N if gated else N
            st["x"], st["x_scales"] = _to_fp8(_normal(g, R, K))
            codes, scales = zip(*(_to_mxfp4(_normal(g, M, K, std=K ** -0.5)) for _ in range(n)))
            st["codes"], st["scales"] = torch.stack(codes), torch.stack(scales)
            st["out"] = torch.empty(R, N, dtype=torch.bfloat16, device=dev)
    return st


def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    from combine_epx_get_amd import epx
    case = st["case"]
    op = case["op"]
    if op == "route":
        p = epx.make_problem(case["tokens"], case["topk"], case["experts"], 1, 1)
        score = epx.SCORE_SIGMOID if case["score"] == "sigmoid" else epx.SCORE_SOFTMAX
        epx.epx_route(p, st["logits"], score, st["idx"], st["w"], bias=st["bias"], renormalize=case["renorm"],
                      scale=case["scale"])
        if not case["grad"]:
            return {"idx": st["idx"], "w": st["w"]}
        epx.epx_route_backward(p, st["logits"], score, st["idx"], st["dw"], st["dlogits"],
                               renormalize=case["renorm"], scale=case["scale"])
        return {"idx": st["idx"], "w": st["w"], "dlogits": st["dlogits"]}
    if op == "combine_bwd":
        epx.epx_combine_backward(st["problem"], st["layout"], st["dout"], st["y"], st["w"], st["dy"], st["dw"])
        return {"dy": st["dy"], "dw": st["dw"]}
    if op == "mxfp4":
        epx.epx_mxfp4_quantize(st["x"], st["codes"], st["scales"])
        epx.epx_mxfp4_dequantize(st["codes"], st["scales"], st["out"])
        return {"values": st["out"]}
    act = epx.ACT_SWIGLU if case["act"] == "swiglu" else epx.ACT_NONE
    rows = epx.expert_rows(st["offset"], st["count"], case["rows"])
    if op == "experts":
        epx.epx_expert_gemm(rows, st["x"], st["weight"], st["out"], act=act, preact=st["preact"])
        return {"out": st["out"], "preact": st["preact"]} if case["train"] else {"out": st["out"]}
    if op == "experts_bwd":
        epx.epx_expert_gemm_dgrad(rows, st["dy"], st["weight"], st["dx"], input_act=act, preact=st["preact"])
        epx.epx_expert_gemm_wgrad(rows, st["dy"], st["x"], st["dw"])
        return {"dx": st["dx"], "dw": st["dw"]}
    epx.epx_expert_gemm_mxfp4(rows, st["x"], st["x_scales"], st["codes"], st["scales"], st["out"], act=act)
    return {"out": st["out"]}


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
    if op == "route":
        return _route_plain(st)
    if op == "combine_bwd":
        T, k, h = case["tokens"], case["topk"], case["hidden"]
        dout = st["dout"].float()
        dw = (st["y"][st["slot"]].float() * dout.unsqueeze(1)).sum(2)
        dy = torch.empty(T * k, h, dtype=torch.bfloat16, device=dout.device)
        dy[st["slot"].flatten()] = (st["w"].unsqueeze(2) * dout.unsqueeze(1)).to(torch.bfloat16).view(T * k, h)
        return {"dy": dy, "dw": dw}
    if op == "mxfp4":
        codes, scales = _to_mxfp4(st["x"])
        return {"values": _from_mxfp4(codes, scales, torch.float32).to(torch.bfloat16)}
    N, K = case["width"], case["inner"]
    gated = case["act"] == "swiglu"
    if op == "experts_bwd":
        dy, at, live = _pad(st["dy"], st)
        x, _, _ = _pad(st["x"], st)
        d = torch.bmm(dy, st["weight"].float())[live]
        if gated:
            gate, up = (v.float() for v in st["preact"][at].split(K, 1))
            s = 1.0 / (1.0 + torch.exp(-gate))
            d = torch.cat((d * up * s * (1.0 + gate * (1.0 - s)), d * gate * s), 1)
        dx = torch.empty_like(st["dx"])
        dx[at] = d.to(torch.bfloat16)
        return {"dx": dx, "dw": torch.bmm(dy.transpose(1, 2).contiguous(), x).to(st["dw"].dtype)}
    if op == "experts":
        x, at, live = _pad(st["x"], st)
        w = st["weight"].float()
    else:
        s = st["x_scales"].repeat_interleave(128, 1)
        x, at, live = _pad(st["x"].view(torch.float8_e4m3fn).float() * s, st)
        w = _from_mxfp4(st["codes"], st["scales"], torch.float32)
    z = torch.bmm(x, w.transpose(1, 2).contiguous())[live]
    a = _silu(z[:, :N]) * z[:, N:] if gated else z
    out = torch.empty_like(st["out"])
    out[at] = a.to(torch.bfloat16)
    if not case.get("train"):
        return {"out": out}
    preact = torch.empty_like(st["preact"])
    preact[at] = z.to(torch.bfloat16)
    return {"out": out, "preact": preact}


def _route_plain(st):
    case, l = st["case"], st["logits"].float()
    k, c = case["topk"], case["scale"]
    # the choice is made on 64-bit keys (two scores can be nearer than 32 bits tell), the lowest index first
    key = l.double()
    if case["biased"]:
        key = 1.0 / (1.0 + torch.exp(-key)) + st["bias"].double()
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    if case["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    chosen = p.gather(1, idx)
    total = chosen.sum(1, keepdim=True) if case["renorm"] else 1.0
    w = c * chosen / total
    res = {"idx": idx.to(torch.int32), "w": w}
    if case["grad"]:
        dw = c * st["dw"]
        dp = (dw - (dw * chosen).sum(1, keepdim=True) / total) / total if case["renorm"] else dw
        full = torch.zeros_like(l).scatter(1, idx, dp)
        if case["score"] == "softmax":
            d = p * (full - (full * p).sum(1, keepdim=True))
        else:
            d = full * p * (1.0 - p)
        res["dlogits"] = d.to(st["logits"].dtype)
    return res


def _weight_bytes(case):
    """Experts that can have rows: no more than there are rows."""
    return min(case["experts"], case["rows"])


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["topk"]
        b = 2 if case["dtype"] == "bf16" else 4
        moved = T * E * b + T * k * 8 + (E * 4 if case["biased"] else 0)
        if case["grad"]:
            moved += T * E * b + T * k * 4
        return {"bytes": moved, "flops": T * E * (8 if case["grad"] else 4)}
    if op == "combine_bwd":
        T, k, h = case["tokens"], case["topk"], case["hidden"]
        return {"bytes": T * h * 2 + 2 * T * k * h * 2 + T * k * 12, "flops": 3 * T * k * h}
    if op == "mxfp4":
        n = case["rows"] * case["inner"]
        return {"bytes": 4 * n + 2 * (n // 2 + n // 32), "flops": 4 * n}
    R, N, K = case["rows"], case["width"], case["inner"]
    M = 2 * N if case["act"] == "swiglu" and op != "experts_bwd" else N
    live = _weight_bytes(case)
    if op == "experts":
        return {"bytes": 2 * (R * K + live * M * K + R * N + (R * M if case["train"] else 0)), "flops": 2 * R * M * K}
    if op == "experts_bwd":
        more = 4 * R * K if case["act"] == "swiglu" else 0
        b = 4 if case["dw"] == "f32" else 2
        return {"bytes": 2 * (R * N + 2 * R * K + live * N * K) + more + (more and 2 * R * K) + case["experts"] * N * K * b,
                "flops": 4 * R * N * K}
    return {"bytes": R * K + R * K // 32 + live * M * K * 17 // 32 + 2 * R * N, "flops": 2 * R * M * K}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _route_exact(st)
    if op == "combine_bwd":
        T, k, h = case["tokens"], case["topk"], case["hidden"]
        dout, w = st["dout"].double(), st["w"].double()
        dy = torch.empty(T * k, h, dtype=torch.float64, device="cuda")
        dw = torch.empty(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            at = st["slot"][:, j]
            dy[at] = w[:, j, None] * dout
            dw[:, j] = torch.linalg.vecdot(st["y"][at].double(), dout)
        return {"dy": dy, "dw": dw}
    if op == "mxfp4":
        return {"values": _mxfp4_exact(st["x"])}
    N, K = case["width"], case["inner"]
    gated = case["act"] == "swiglu"
    offset, count = st["offset"].tolist(), st["count"].tolist()
    if op == "experts_bwd":
        dx = torch.zeros(st["dx"].shape, dtype=torch.float64, device="cuda")
        dw = torch.zeros(st["dw"].shape, dtype=torch.float64, device="cuda")
        for e, (o, c) in enumerate(zip(offset, count)):
            dy = st["dy"][o:o + c].double()
            d = dy @ st["weight"][e].double()
            dw[e] = dy.T @ st["x"][o:o + c].double()
            if gated:
                gate, up = st["preact"][o:o + c, :K].double(), st["preact"][o:o + c, K:].double()
                s = torch.sigmoid(gate)
                dx[o:o + c, :K] = d * up * (s + gate * s * (1 - s))
                dx[o:o + c, K:] = d * gate * s
            else:
                dx[o:o + c] = d
        return {"dx": dx, "dw": dw}
    M = 2 * N if gated else N
    z = torch.zeros(case["rows"], M, dtype=torch.float64, device="cuda")
    for e, (o, c) in enumerate(zip(offset, count)):
        if op == "experts":
            x, w = st["x"][o:o + c].double(), st["weight"][e].double()
        else:
            x = st["x"][o:o + c].view(torch.float8_e4m3fn).double().view(c, -1, 128)
            x = (x * st["x_scales"][o:o + c].double().unsqueeze(2)).view(c, K)
            w = _values_exact(st["codes"][e], st["scales"][e])
        z[o:o + c] = x @ w.T
    out = z
    if gated:
        out = z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]
    return {"out": out, "preact": z} if case.get("train") else {"out": out}


def _values_exact(codes, scales):
    """4-bit values from the fields of each code: sign, two exponent bits, one mantissa bit."""
    c = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    sign, ex, man = 1.0 - 2.0 * (c >> 3).double(), (c >> 1) & 3, (c & 1).double()
    mag = torch.where(ex == 0, 0.5 * man, (1.0 + 0.5 * man) * torch.exp2((ex - 1).double()))
    return sign * mag * torch.exp2(scales.double() - 127.0).repeat_interleave(32, 1)


def _mxfp4_exact(x):
    """The nearest 4-bit value of each element under its block's scale, found among all eight magnitudes; in parts."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    # midpoints between neighbours: one on a midpoint goes to the neighbour with the even code
    mid = (grid[1:] + grid[:-1]) / 2
    res = []
    for part in x.split(max(1, (1 << 26) // x.shape[1])):
        b = part.double().view(part.shape[0], -1, 32)
        amax = b.abs().amax(2, keepdim=True)
        unit = torch.exp2(torch.where(amax > 0, torch.floor(torch.log2(amax)) - 2.0, -127.0).clamp(min=-127.0))
        a = (b.abs() / unit).contiguous()
        lo, hi = torch.searchsorted(mid, a, right=False), torch.searchsorted(mid, a, right=True)
        code = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
        res.append((grid[code] * unit * torch.sign(b)).view(part.shape))
    return torch.cat(res)


def _route_exact(st):
    case = st["case"]
    l = st["logits"].double().cpu().numpy()
    T, k, c = case["tokens"], case["topk"], case["scale"]
    if case["score"] == "softmax":
        p = np.exp(l - l.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
    key = p + st["bias"].double().cpu().numpy() if case["biased"] else l
    idx = np.argsort(-key, axis=1, kind="stable")[:, :k]
    rows = np.arange(T)[:, None]
    chosen = p[rows, idx]
    total = chosen.sum(1, keepdims=True)
    w = c * (chosen / total if case["renorm"] else chosen)
    res = {"idx": torch.from_numpy(idx.astype(np.int32)), "w": torch.from_numpy(w)}
    if case["grad"]:
        dw = st["dw"].double().cpu().numpy()
        d = np.zeros_like(l)
        if case["renorm"]:
            # w = c * softmax over the chosen (or c * score / total): the others' logits do not enter
            inner = (dw * w).sum(1, keepdims=True) / c
            d[rows, idx] = w * (dw - inner) * (1.0 if case["score"] == "softmax" else 1.0 - chosen)
        elif case["score"] == "softmax":
            d -= p * (dw * w).sum(1, keepdims=True)
            d[rows, idx] += w * dw
        else:
            d[rows, idx] = w * dw * (1.0 - chosen)
        res["dlogits"] = torch.from_numpy(d)
    return res
