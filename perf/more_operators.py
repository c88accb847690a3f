"""Cases of the 8-bit path of an expert layer and of its training: e4m3 quantisation with one fp32 scale per
block of 128, the products of such matrices (dense, per expert, and the experts' weight gradients), and the
gradients of the steps that sort tokens by expert and bring them back with their weights.

Each case runs in two ways.  Where `own` is true the library's entry points are called as a user calls
them; otherwise the operator is computed in plain torch operations, in fp32, rounded once at the end.
`exact` computes it a third time in fp64 from the definition.
"""
import math

import torch

own = False

TINY = 2.0 ** -100  # the least magnitude that a block's scale is taken from
E4M3 = torch.float8_e4m3fn
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # the hidden state of one token before a projection: latency is all that counts
        dict(name="quant_token", op="quant", kind="rows", m=1, k=7168, dtype="bf16"),
        # a training step's activations: routed to 128 experts, eight copies of each token, quantised along
        # the channels for the product and along the expert's tokens for the weight gradient
        dict(name="quant_experts", op="quant", kind="experts", m=4096, k=2048, dtype="bf16", experts=128, topk=8, skew=0.5),
        # a master weight after an optimiser step: 128 x 128 blocks, for the product and for its transpose
        dict(name="quant_weight", op="quant", kind="weight", m=4096, k=7168, dtype="f32"),
        # one token through a projection: the weight is read once
        dict(name="gemm_token", op="gemm", m=1, n=4096, k=7168, block_b=128, out="bf16"),
        # sizes that fill no tile, both operands scaled by row, fp32 result, as for a small weight gradient
        dict(name="gemm_odd", op="gemm", m=300, n=1001, k=2080, block_b=1, out="f32"),
        # a prefill chunk: bound by the tensor cores
        dict(name="gemm_prefill", op="gemm", m=4096, n=4096, k=7168, block_b=128, out="bf16"),
        # sixteen decoding tokens over 128 experts: the weights of the experts that were hit are read
        dict(name="grouped_decode", op="grouped", tokens=16, topk=8, experts=128, n=1536, k=2048, skew=0.5),
        # a prefill chunk of 4096 tokens through the same gate and up weights
        dict(name="grouped_prefill", op="grouped", tokens=4096, topk=8, experts=128, n=1536, k=2048, skew=0.5),
        # weight gradients of a few experts at sizes that fill no tile, an expert without tokens among them
        dict(name="wgrad_odd", op="wgrad", tokens=333, topk=2, experts=9, n=784, k=1040, skew=2.0, out="f32"),
        # weight gradients of the gate and up projections over a training batch of 4096 tokens
        dict(name="wgrad_train", op="wgrad", tokens=4096, topk=8, experts=128, n=1536, k=2048, skew=0.5, out="bf16"),
        # the routing's gradients of a small batch at an odd width
        dict(name="route_odd", op="route", tokens=37, topk=3, experts=16, h=1000, skew=0.5),
        # the same over a training batch: bound by memory
        dict(name="route_train", op="route", tokens=4096, topk=8, experts=128, h=2048, skew=0.5),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _routed(rng, most):
    topk = rng.choice([1, 2, 4, 6, 8])
    experts = _spread(rng, topk, 128)
    return dict(tokens=_spread(rng, 1, max(1, min(4096, most // topk))), topk=topk, experts=experts,
                skew=round(rng.uniform(0.0, 1.5), 2))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "grouped", "wgrad", "route"])
    if op == "quant":
        kind = rng.choice(["rows", "both", "experts", "weight"])
        k = 16 * _spread(rng, 4, 448)
        c = dict(op=op, kind=kind, k=k, dtype=rng.choice(["bf16", "f32"]))
        if kind == "experts":
            r = _routed(rng, 32768 * 2048 // 2 // k)
            return dict(c, m=r["tokens"], experts=r["experts"], topk=r["topk"], skew=r["skew"])
        m = _spread(rng, 1, min(8192, 4096 * 7168 // 2 // k))
        return dict(c, m=16 * max(1, m // 16) if kind == "weight" else m)
    if op == "gemm":
        k = 16 * _spread(rng, 8, 448)
        n = _spread(rng, 16, 4096)
        n = 16 * max(1, n // 16) if rng.random() < 0.7 else n
        return dict(op=op, m=_spread(rng, 1, min(4096, 4096 * 4096 * 7168 // (n * k))), n=n, k=k,
                    block_b=rng.choice([128, 128, 1]), out=rng.choice(["bf16", "bf16", "f32"]))
    if op == "route":
        h = 8 * _spread(rng, 8, 512)
        return dict(_routed(rng, 32768 * 2048 // h), op=op, h=h)
    n, k = 8 * _spread(rng, 16, 192), 16 * _spread(rng, 8, 128)
    c = dict(_routed(rng, 32768), op=op, n=n, k=k)
    return dict(c, n=16 * (n // 16), out=rng.choice(["bf16", "f32"])) if op == "wgrad" else c


def _rows_of(case):
    return case["tokens"] * case["topk"]


def _blocks(n):
    return -(-n // 128)


def _padded(rows, experts):
    """Columns of a matrix that is scaled along an expert's tokens: each expert begins at a multiple of 128."""
    return _blocks(rows) * 128 + 128 * experts


def work(case):
    op = case["op"]
    if op == "quant":
        m, k, kind, xb = case["m"], case["k"], case["kind"], 2 if case["dtype"] == "bf16" else 4
        r = m * case["topk"] if kind == "experts" else m
        out = r * k + r * _blocks(k) * 4 if kind != "weight" else r * k
        if kind in ("both", "experts"):
            out += r * k + _blocks(r) * k * 4
        if kind == "weight":
            out += r * k
        return {"bytes": m * k * xb + out, "flops": 4 * r * k}
    if op == "gemm":
        m, n, k, ob = case["m"], case["n"], case["k"], 2 if case["out"] == "bf16" else 4
        return {"bytes": m * k + n * k + m * _blocks(k) * 4 + m * n * ob, "flops": 2 * m * n * k}
    r = _rows_of(case)
    if op == "route":
        t, h = case["tokens"], case["h"]
        # output's gradient and expert outputs in, their gradients and the weights' out; then the experts'
        # input gradients in and the tokens' out
        return {"bytes": t * h * 2 + 2 * r * h * 2 + 12 * r + r * h * 2 + t * h * 2, "flops": 4 * r * h}
    n, k, e = case["n"], case["k"], case["experts"]
    if op == "grouped":
        return {"bytes": r * k + min(e, r) * n * k + r * _blocks(k) * 4 + r * n * 2, "flops": 2 * r * n * k}
    return {"bytes": r * (n + k) + e * n * k * (2 if case["out"] == "bf16" else 4), "flops": 2 * r * n * k}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, m, k, dtype=torch.bfloat16):
    x = torch.randn(m, k, generator=g, device="cuda")
    x[:, :: max(1, k // 4)] *= 20.0  # channels with outliers, as in a residual stream
    return x.to(dtype)


def _gradients(g, m, k):
    """Small, and some tokens far larger than others."""
    x = torch.randn(m, k, generator=g, device="cuda") * 1e-4
    return (x * torch.exp(torch.randn(m, 1, generator=g, device="cuda"))).to(torch.bfloat16)


def _divided(amax):
    """(scale, factor to the codes) of blocks with these largest magnitudes."""
    a = amax.clamp(min=TINY)
    top = torch.full_like(a, 448.0)
    return a / top, top / a


def _codes(x, factor):
    return (x * factor).clamp(-448.0, 448.0).to(E4M3)


def _quantised_rows(x):
    """One scale per row and 128 columns: codes [m, k], scales [ceil(k / 128), m]."""
    m, k = x.shape
    b = torch.nn.functional.pad(x.float(), (0, _blocks(k) * 128 - k)).view(m, -1, 128)
    s, f = _divided(b.abs().amax(2))
    return _codes(b, f.unsqueeze(2)).view(m, -1)[:, :k].contiguous(), s.t().contiguous()


def _quantised_columns(x):
    """One scale per column and 128 rows, transposed: codes [k, rows], scales [rows / 128, k]; x with a
    multiple of 128 rows."""
    b = x.float().view(-1, 128, x.shape[1])
    s, f = _divided(b.abs().amax(1))
    return _codes(b, f.unsqueeze(1)).view(x.shape).t().contiguous(), s


def _quantised_blocks(x):
    """One scale per 128 x 128 block of each matrix: codes [.., n, k], scales [.., ceil(n / 128), ceil(k / 128)]."""
    n, k = x.shape[-2:]
    nb, kb = _blocks(n), _blocks(k)
    b = torch.nn.functional.pad(x.float(), (0, kb * 128 - k, 0, nb * 128 - n)).view(-1, nb, 128, kb, 128)
    s, f = _divided(b.abs().amax(dim=(2, 4)))
    q = _codes(b, f.view(-1, nb, 1, kb, 1)).view(-1, nb * 128, kb * 128)[:, :n, :k]
    return q.reshape(x.shape).contiguous(), s.view(x.shape[:-2] + (nb, kb))


def _route(g, tokens, topk, experts, skew):
    """Top-k routing with experts of uneven popularity: what a sort by expert leaves."""
    logits = torch.randn(tokens, experts, generator=g, device="cuda")
    logits += skew * torch.randn(1, experts, generator=g, device="cuda")
    p, ids = torch.topk(torch.softmax(logits, 1), topk, dim=1)
    order = torch.sort(ids.view(-1), stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device="cuda")
    counts = torch.bincount(ids.view(-1), minlength=experts)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts.cumsum(0)
    # the plan of the plain forms: the rows of each expert, one line per expert, and where they lie in a
    # matrix whose experts begin at multiples of 128
    most = max(1, int(counts.max()))
    line = torch.arange(most, device="cuda")
    real = line < counts.view(-1, 1)
    first = ((counts + 127) // 128 * 128).cumsum(0) - (counts + 127) // 128 * 128
    rows = torch.where(real, offsets[:-1].view(-1, 1) + line, 0)
    expert = torch.repeat_interleave(torch.arange(experts, device="cuda"), counts)
    wide = first[expert] + torch.arange(order.numel(), device="cuda") - offsets[expert]
    return dict(offsets=offsets, src=(order // topk).to(torch.int32), pos=pos.view(tokens, topk).to(torch.int32),
                weights=p / p.sum(1, keepdim=True), rows=rows, real=real, wide=wide, padded=_padded(order.numel(), experts))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quant":
        dtype = TYPES[case["dtype"]]
        if case["kind"] == "weight":
            s["x"] = (torch.randn(case["m"], case["k"], generator=g, device="cuda") * 0.02).to(dtype)
        else:
            s["x"] = _activations(g, case["m"], case["k"], dtype)
        if case["kind"] == "experts":
            s.update(_route(g, case["m"], case["topk"], case["experts"], case["skew"]))
        return s
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sfa"] = _quantised_rows(_activations(g, m, k))
        w = torch.randn(n, k, generator=g, device="cuda") * 0.02
        s["b"], s["sfb"] = _quantised_blocks(w) if case["block_b"] == 128 else _quantised_rows(w)
        return s
    s.update(_route(g, case["tokens"], case["topk"], case["experts"], case["skew"]))
    r = _rows_of(case)
    if op == "route":
        s["dout"] = _gradients(g, case["tokens"], case["h"])
        s["y"] = torch.randn(r, case["h"], generator=g, device="cuda").to(torch.bfloat16)
        s["dx"] = _gradients(g, r, case["h"])
        return s
    n, k, e = case["n"], case["k"], case["experts"]
    x = _activations(g, case["tokens"], k)[s["src"].long()]
    if op == "grouped":
        s["a"], s["sfa"] = _quantised_rows(x)
        s["b"], s["sfb"] = _quantised_blocks(torch.randn(e, n, k, generator=g, device="cuda") * 0.02)
        return s
    wide = torch.zeros(s["padded"], k, dtype=torch.bfloat16, device="cuda")
    wide[s["wide"]] = x
    s["b"], s["sfb"] = _quantised_columns(wide)
    wide = torch.zeros(s["padded"], n, dtype=torch.bfloat16, device="cuda")
    wide[s["wide"]] = _gradients(g, r, n)
    s["a"], s["sfa"] = _quantised_columns(wide)
    return s


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import nvfp4_block_scaled_bf16_gb300 as nv
    case = s["case"]
    op = case["op"]
    if op == "quant":
        if case["kind"] == "rows":
            return nv.fp8_quantize(s["x"])
        if case["kind"] == "both":
            return nv.fp8_quantize(s["x"], transpose=True)
        if case["kind"] == "weight":
            return nv.fp8_quantize_weight(s["x"], transpose=True)
        return nv.fp8_quantize(s["x"], src_rows=s["src"], row_offsets=s["offsets"], transpose=True)
    if op == "gemm":
        return nv.fp8_gemm(s["a"], s["sfa"], s["b"], s["sfb"], block_b=case["block_b"], out_dtype=TYPES[case["out"]])
    if op == "grouped":
        return nv.fp8_grouped_gemm(s["a"], s["sfa"], s["offsets"], s["b"], s["sfb"])
    if op == "wgrad":
        return nv.fp8_grouped_weight_grad(s["a"], s["sfa"], s["b"], s["sfb"], s["offsets"], out_dtype=TYPES[case["out"]])
    dy, dw = nv.moe_combine_backward(s["dout"], s["y"], s["pos"], s["weights"])
    return dy, dw, nv.moe_gather_backward(s["dx"], s["pos"])


def _plain(s):
    return {"quant": _quant_plain, "gemm": _gemm_plain, "grouped": _grouped_plain, "wgrad": _wgrad_plain,
            "route": _route_plain}[s["case"]["op"]](s)


def _quant_plain(s):
    kind, x = s["case"]["kind"], s["x"]
    if kind == "weight":
        q, sf = _quantised_blocks(x)
        return q, sf, q.t().contiguous(), sf.t().contiguous()
    if kind == "rows":
        return _quantised_rows(x)
    if kind == "experts":
        x = x[s["src"].long()]
        wide = torch.zeros(s["padded"], x.shape[1], dtype=x.dtype, device=x.device)
        wide[s["wide"]] = x
    else:
        wide = torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % 128))
    return _quantised_rows(x) + _quantised_columns(wide)


def _rows_value(q, sf):
    """fp32 values of codes with one scale per row and 128 columns."""
    k = q.shape[1]
    return q.float() * sf.t().repeat_interleave(128, dim=1)[:, :k]


def _blocks_value(q, sf):
    """fp32 values of codes with one scale per 128 x 128 block."""
    n, k = q.shape[-2:]
    return q.float() * sf.repeat_interleave(128, dim=-2)[..., :n, :].repeat_interleave(128, dim=-1)[..., :k]


def _gemm_plain(s):
    a = _rows_value(s["a"], s["sfa"])
    b = _blocks_value(s["b"], s["sfb"]) if s["case"]["block_b"] == 128 else _rows_value(s["b"], s["sfb"])
    return (a @ b.t()).to(TYPES[s["case"]["out"]])


def _grouped_plain(s):
    a = _rows_value(s["a"], s["sfa"])[s["rows"]]                      # [experts, most, k]
    d = torch.bmm(a, _blocks_value(s["b"], s["sfb"]).transpose(1, 2))
    return d[s["real"]].to(torch.bfloat16)


def _wgrad_plain(s):
    at = s["wide"][s["rows"]]
    real = s["real"].unsqueeze(2)
    a = torch.where(real, _rows_value(s["a"], s["sfa"]).t()[at], 0.0)   # [experts, most, n]
    b = torch.where(real, _rows_value(s["b"], s["sfb"]).t()[at], 0.0)
    return torch.bmm(a.transpose(1, 2), b).to(TYPES[s["case"]["out"]])


def _route_plain(s):
    pos = s["pos"].long()
    dout, w = s["dout"].float(), s["weights"]
    dw = (dout.unsqueeze(1) * s["y"].float()[pos]).sum(2)
    dy = torch.empty_like(s["y"])
    dy[pos.view(-1)] = (w.unsqueeze(2) * dout.unsqueeze(1)).to(torch.bfloat16).view(-1, dout.shape[1])
    return dy, dw, s["dx"].float()[pos].sum(1).to(torch.bfloat16)


# ------------------------------------------------------------------------------------------ in 64 bits
def _value64(q):
    """Values of e4m3 codes from their fields."""
    c = q.view(torch.uint8).int()
    e, m = c >> 3 & 15, (c & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * torch.exp2((e - 7).double()))
    return torch.where(c > 127, -v, v)


def _nearest64(y):
    """The nearest e4m3 value, ties to the even code: a multiple of the step of y's binade."""
    a = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0) - 3.0)
    return torch.copysign(torch.round(a / step) * step, y)


def _by_tiles64(x, br, bc):
    """(codes' values, scales) of blocks of br x bc: the definition's two fp32 roundings of a block's scale
    and of its factor, and the one of each product."""
    m, k = x.shape
    mb, kb = -(-m // br), -(-k // bc)
    full = torch.zeros(mb * br, kb * bc, dtype=torch.float64, device=x.device)
    full[:m, :k] = x.double()
    t = full.view(mb, br, kb, bc)
    amax = t.abs().amax(dim=(1, 3)).clamp(min=TINY)
    f = (448.0 / amax).float().double().view(mb, 1, kb, 1)
    return _nearest64((t * f).float().double()).view(mb * br, kb * bc)[:m, :k], (amax / 448.0).float().double()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        x = s["x"]
        if case["kind"] == "weight":
            q, sf = _by_tiles64(x, 128, 128)
            return q, sf, q.t().contiguous(), sf.t().contiguous()
        if case["kind"] == "experts":
            x = x.index_select(0, s["src"].long())
        q, sf = _by_tiles64(x, 1, 128)
        if case["kind"] == "rows":
            return q, sf.t().contiguous()
        if case["kind"] == "experts":
            wide = torch.zeros(s["padded"], x.shape[1], dtype=torch.float64, device="cuda")
            wide.index_copy_(0, s["wide"], x.double())
        else:
            wide = torch.zeros(_blocks(x.shape[0]) * 128, x.shape[1], dtype=torch.float64, device="cuda")
            wide[: x.shape[0]] = x.double()
        qt, sft = _by_tiles64(wide, 128, 1)
        return q, sf.t().contiguous(), qt.t().contiguous(), sft
    if op == "route":
        dout, y, w = s["dout"].double(), s["y"].double(), s["weights"].double()
        src, pos = s["src"].long(), s["pos"].long()
        slot = torch.empty(src.numel(), dtype=torch.int64, device="cuda")
        slot[pos.view(-1)] = torch.arange(src.numel(), device="cuda")
        dy = dout.index_select(0, src) * w.view(-1).index_select(0, slot).view(-1, 1)
        dots = (y * dout.index_select(0, src)).sum(1)
        dx = torch.zeros_like(dout).index_add_(0, src, s["dx"].double())
        return dy, dots[pos], dx
    k = s["a"].shape[1]
    block = torch.arange(k, device="cuda") // 128
    a = _value64(s["a"]) * s["sfa"].double()[block].t()
    if op == "gemm":
        b = _value64(s["b"])
        if case["block_b"] == 128:
            b *= s["sfb"].double()[torch.arange(b.shape[0], device="cuda") // 128][:, block]
        else:
            b *= s["sfb"].double()[block].t()
        return a @ b.t()
    offsets = s["offsets"].tolist()
    if op == "grouped":
        out = torch.empty(a.shape[0], case["n"], dtype=torch.float64, device="cuda")
        rows = torch.arange(case["n"], device="cuda") // 128
        for e in range(case["experts"]):
            lo, hi = offsets[e], offsets[e + 1]
            if hi > lo:
                out[lo:hi] = a[lo:hi] @ (_value64(s["b"][e]) * s["sfb"][e].double()[rows][:, block]).t()
        return out
    b = _value64(s["b"]) * s["sfb"].double()[block].t()
    out = torch.zeros(case["experts"], case["n"], case["k"], dtype=torch.float64, device="cuda")
    at = 0
    for e in range(case["experts"]):
        n = offsets[e + 1] - offsets[e]
        out[e] = a[:, at : at + n] @ b[:, at : at + n].t()
        at += -(-n // 128) * 128
    return out
