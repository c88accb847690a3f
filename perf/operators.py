"""Cases of the operators around the NVFP4 products of a decoder: the norms before and after a block,
the gated product of a feed-forward block, and the draw of the next token from its logits.

Each case runs in two ways.  Where `own` is true the library's entry points are called as a user calls
them; otherwise the operator is computed in plain torch operations, in fp32, rounded once at the end.
`exact` computes it a third time in fp64 from the definition.
"""
import math

import torch

own = False

# log2(e) in fp32: weights of the draw are powers of two of (logit - max) * (LOG2E / temperature)
LOG2E = 1.4426950408889634
UNIT = 2.0 ** 30  # the largest weight of a row, as an integer
ROWS = 16  # gate rows and up rows of a gated weight alternate in groups of 16


# ------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token between two blocks of a 7168-wide decoder: norm of the block's output, residual
        # sum, norm before the next block; latency is all that counts
        dict(name="norm_token", op="norm", m=1, h=7168, stream="bf16", post=True, gate="none", offset=0.0, scale=1.0),
        # a small batch at an odd width, rows that are not 16-byte aligned, fp32 residual stream,
        # zero-centred weights, one gate per channel
        dict(name="norm_odd", op="norm", m=77, h=2047, stream="f32", post=True, gate="channel", offset=1.0, scale=0.5),
        # a prefill chunk of 4096 tokens, the memory-bound case
        dict(name="norm_prefill", op="norm", m=4096, h=7168, stream="bf16", post=True, gate="channel", offset=0.0, scale=1.0),
        # its backward pass over a training batch, gates that differ from token to token
        dict(name="norm_train", op="norm_grad", m=2048, h=4096, stream="bf16", post=True, gate="token", offset=0.0, scale=0.7),
        # both projections of one token: the packed weight is read once
        dict(name="gated_token", op="gated", m=1, k=4096, i=7168, act="silu"),
        # a batch of decodes on a small block whose sizes fill no tile
        dict(name="gated_ragged", op="gated", m=100, k=2080, i=784, act="gelu_tanh"),
        # a prefill chunk: bound by the tensor cores
        dict(name="gated_prefill", op="gated", m=2048, k=4096, i=7168, act="silu"),
        # the gradient of both projections, recomputed from the packed operands
        dict(name="gated_train", op="gated_grad", m=1024, k=4096, i=7168, act="silu"),
        # one sequence, temperature alone
        dict(name="sample_one", op="sample", b=1, v=32000, dtype="f32", spread=2.5, filters="none", pad=0),
        # seven requests at an odd vocabulary, rows of a wider buffer, min-p
        dict(name="sample_odd", op="sample", b=7, v=50001, dtype="f32", spread=2.0, filters="min_p", pad=15),
        # a serving batch with every filter set, other values for each request
        dict(name="sample_batch", op="sample", b=64, v=131072, dtype="bf16", spread=2.5, filters="all", pad=0),
        # a large batch at flat distributions, where top-p keeps thousands of tokens
        dict(name="sample_flat", op="sample", b=256, v=131072, dtype="bf16", spread=1.0, filters="top_p", pad=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "gated", "gated_grad", "sample", "sample"])
    if op in ("norm", "norm_grad"):
        most = 4096 * 7168 if op == "norm" else 2048 * 4096
        h = _spread(rng, 64, 8192)
        h = h // 8 * 8 if rng.random() < 0.7 else h
        m = _spread(rng, 1, max(1, min(4096, most // h)))
        return dict(op=op, m=m, h=h, stream=rng.choice(["bf16", "f32"]), post=rng.random() < 0.8,
                    gate=rng.choice(["none", "channel", "token"]), offset=rng.choice([0.0, 1.0]),
                    scale=round(rng.uniform(0.2, 1.5), 3))
    if op in ("gated", "gated_grad"):
        most = (2048 if op == "gated" else 1024) * 4096 * 7168
        k = 32 * _spread(rng, 8, 224)
        i = 16 * _spread(rng, 16, 448)
        m = _spread(rng, 1, max(1, min(2048, most // (k * i))))
        return dict(op=op, m=m, k=k, i=i, act=rng.choice(["silu", "gelu_tanh"]))
    v = _spread(rng, 1000, 131072)
    return dict(op=op, b=_spread(rng, 1, 256), v=v, dtype=rng.choice(["bf16", "f32"]) if v <= 65536 else "bf16",
                spread=round(rng.uniform(1.0, 3.0), 2), filters=rng.choice(["none", "top_k", "top_p", "min_p", "all"]),
                pad=rng.choice([0, 0, 8, 15]))


def work(case):
    if case["op"] in ("norm", "norm_grad"):
        m, h, xb = case["m"], case["h"], 2 if case["stream"] == "bf16" else 4
        post, gate = case["post"], case["gate"]
        gates = {"none": 0, "channel": h * 2, "token": m * h * 2}[gate] if post else 0
        if case["op"] == "norm":
            # read the stream, the block's output, its gates and the weights; write the stream and the normed rows
            nbytes = m * h * (2 * xb if post else xb) + m * h * (2 if post else 0) + gates + 4 * h + m * h * 2
            return {"bytes": nbytes, "flops": m * h * (10 if post else 4)}
        # read both incoming gradients, the stream and the block's output; write both outgoing ones
        nbytes = m * h * (2 + xb + xb) + m * h * xb + (m * h * 4 if post else 0) + gates + 4 * h + 8 * h
        nbytes += {"none": 0, "channel": h * 4, "token": m * h * 2}[gate] if post else 0
        return {"bytes": nbytes, "flops": m * h * (24 if post else 10)}
    if case["op"] in ("gated", "gated_grad"):
        m, k, i = case["m"], case["k"], case["i"]
        nbytes = (m + 2 * i) * k * 9 // 16 + m * i * 2
        if case["op"] == "gated_grad":
            nbytes += m * i * 2 + m * 2 * i * 2
        return {"bytes": nbytes, "flops": 2 * m * 2 * i * k}
    b, v = case["b"], case["v"]
    return {"bytes": b * v * (2 if case["dtype"] == "bf16" else 4) + b * 28, "flops": 4 * b * v}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _packed(x):
    """NVFP4 of a [rows, k] matrix: packed e2m1 codes, e4m3 scales per 16 in the 128x4 layout, and the
    global scale 448 * 6 / amax."""
    rows, k = x.shape
    gs = 2688.0 / x.abs().amax()
    blocks = x.view(rows, k // 16, 16)
    sc = (gs * blocks.abs().amax(2) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    y = blocks * (gs / sc.float().clamp(min=2.0 ** -9)).unsqueeze(2)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    codes = torch.bucketize(y.abs(), edges).to(torch.uint8) | (y < 0).to(torch.uint8) << 3
    codes = codes.view(rows, k)
    q = codes[:, 0::2] | codes[:, 1::2] << 4
    rp, cp = -(-rows // 128) * 128, -(-(k // 16) // 4) * 4
    full = torch.zeros(rp, cp, dtype=torch.uint8, device=x.device)
    full[:rows, : k // 16] = sc.view(torch.uint8)
    sf = full.view(rp // 128, 4, 32, cp // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return q.contiguous(), sf, gs


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        m, h = case["m"], case["h"]
        xt = torch.bfloat16 if case["stream"] == "bf16" else torch.float32
        x = torch.randn(m, h, generator=g, device="cuda")
        x[:, :: max(1, h // 4)] *= 20.0  # channels with outliers, as in a residual stream
        s["x"] = x.to(xt)
        off = case["offset"]
        s["w_pre"] = (1.0 - off + torch.randn(h, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
        s["y"] = s["w_post"] = s["gate"] = None
        if case["post"]:
            s["y"] = _normal(g, m, h, std=0.7)
            s["w_post"] = (1.0 - off + torch.randn(h, generator=g, device="cuda") * 0.1).to(torch.bfloat16)
            if case["gate"] == "channel":
                s["gate"] = _normal(g, h, std=0.5)
            elif case["gate"] == "token":
                s["gate"] = _normal(g, m, h, std=0.5)
        if op == "norm_grad":
            s["dh"] = _normal(g, m, h, std=0.02)
            s["dx_out"] = _normal(g, m, h, std=0.02, dtype=xt)
        return s
    if op in ("gated", "gated_grad"):
        m, k, i = case["m"], case["k"], case["i"]
        x = torch.randn(m, k, generator=g, device="cuda")
        x[:, :: max(1, k // 4)] *= 20.0
        s["a"], s["sfa"], gsa = _packed(x.to(torch.bfloat16).float())
        # gate rows and up rows alternate in groups of 16
        w = torch.randn(2 * i, k, generator=g, device="cuda") * 0.02
        s["b"], s["sfb"], gsb = _packed(w.to(torch.bfloat16).float())
        s["alpha"] = torch.stack([1.0 / (gsa * gsb), 1.0 / (gsa * gsb)])
        s["lut"] = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
        if op == "gated_grad":
            s["dh"] = _normal(g, m, i, std=0.02)
        return s
    b, v, kind = case["b"], case["v"], case["filters"]
    z = torch.randn(b, v + case["pad"], generator=g, device="cuda") * case["spread"]
    peaks = torch.randint(0, v, (b, 8), generator=g, device="cuda")
    z.scatter_add_(1, peaks, torch.rand(b, 8, generator=g, device="cuda") * 2.0 * case["spread"])
    s["logits"] = z.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)[:, :v]
    s["uniform"] = torch.rand(b, generator=g, device="cuda")
    s["temperature"] = 0.5 + torch.rand(b, generator=g, device="cuda")
    s["top_k"] = s["top_p"] = s["min_p"] = None
    if kind in ("top_k", "all"):
        s["top_k"] = torch.randint(1, 200, (b,), generator=g, device="cuda", dtype=torch.int32)
    if kind in ("top_p", "all"):
        s["top_p"] = 0.8 + 0.2 * torch.rand(b, generator=g, device="cuda")
    if kind in ("min_p", "all"):
        s["min_p"] = 0.1 * torch.rand(b, generator=g, device="cuda")
    return s


# ------------------------------------------------------------------------------------------ one pass
def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import nvfp4_block_scaled_bf16_gb300 as nv
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return nv.block_norm(s["x"], s["w_pre"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                             residual_scale=case["scale"], eps=1e-6, weight_offset=case["offset"])
    if op == "norm_grad":
        return nv.block_norm_backward(s["dh"], s["dx_out"], s["x"], s["w_pre"], y=s["y"], w_post=s["w_post"],
                                      gate=s["gate"], residual_scale=case["scale"], eps=1e-6,
                                      weight_offset=case["offset"])
    if op == "gated":
        return nv.nvfp4_gated_gemm(s["a"], s["sfa"], s["b"], s["sfb"], s["alpha"], activation=case["act"])
    if op == "gated_grad":
        return nv.nvfp4_gated_gemm_backward(s["a"], s["sfa"], s["b"], s["sfb"], s["alpha"], s["dh"],
                                            activation=case["act"])
    return nv.sample_tokens(s["logits"], s["uniform"], temperature=s["temperature"], top_k=s["top_k"],
                            top_p=s["top_p"], min_p=s["min_p"])


def _plain(s):
    return {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "gated": _gated_plain, "gated_grad": _gated_grad_plain,
            "sample": _sample_plain}[s["case"]["op"]](s)


def _norm_plain(s):
    case = s["case"]
    r = s["x"].float()
    if s["y"] is not None:
        y = s["y"].float()
        n = y * torch.rsqrt((y * y).mean(1, keepdim=True) + 1e-6) * (case["offset"] + s["w_post"].float())
        if s["gate"] is not None:
            n = n * s["gate"].float()
        r = r + case["scale"] * n
    h = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-6) * (case["offset"] + s["w_pre"].float())
    return r.to(s["x"].dtype), h.to(torch.bfloat16)


def _norm_grad_plain(s):
    """x is the stream after the block: the backward pass starts from what the forward pass stored."""
    case = s["case"]
    x, w, dh = s["x"].float(), case["offset"] + s["w_pre"].float(), s["dh"].float()
    rx = torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-6)
    xn = x * rx
    dw_pre = (dh * xn).sum(0)
    d = dh * w
    dx = s["dx_out"].float() + rx * (d - xn * (d * xn).mean(1, keepdim=True))
    if s["y"] is None:
        return dx.to(s["x"].dtype), None, dw_pre, None, None
    y, wp = s["y"].float(), case["offset"] + s["w_post"].float()
    ry = torch.rsqrt((y * y).mean(1, keepdim=True) + 1e-6)
    yn = y * ry
    t = case["scale"] * dx
    dgate = None
    if s["gate"] is not None:
        gate = s["gate"].float()
        dg = t * yn * wp
        dgate = dg.sum(0) if gate.dim() == 1 else dg.to(torch.bfloat16)
        t = t * gate
    dw_post = (t * yn).sum(0)
    e = t * wp
    dy = ry * (e - yn * (e * yn).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), dy.to(torch.bfloat16), dw_pre, dw_post, dgate


def _dequantised(q, sf, lut):
    rows, kb = q.shape
    codes = torch.stack((q & 15, q >> 4), dim=2).view(rows, 2 * kb).int()
    cols = kb // 8
    rp, cp = -(-rows // 128) * 128, -(-cols // 4) * 4
    sc = sf[: rp * cp].view(rp // 128, cp // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rp, cp)[:rows, :cols]
    sc = sc.contiguous().view(torch.float8_e4m3fn).float()
    return (lut[codes].view(rows, cols, 16) * sc.unsqueeze(2)).view(rows, 2 * kb)


def _products(s):
    a = _dequantised(s["a"], s["sfa"], s["lut"])
    b = _dequantised(s["b"], s["sfb"], s["lut"])
    c = (a @ b.t()).view(a.shape[0], -1, 2, ROWS)
    return c[:, :, 0] * s["alpha"][0], c[:, :, 1] * s["alpha"][1]


def _gated_plain(s):
    g, u = _products(s)
    if s["case"]["act"] == "silu":
        f = g / (1.0 + torch.exp(-g))
    else:
        f = 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))
    return (f * u).reshape(g.shape[0], -1).to(torch.bfloat16)


def _gated_grad_plain(s):
    g, u = _products(s)
    m = g.shape[0]
    if s["case"]["act"] == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        f, df = g * sg, sg * (1.0 + g * (1.0 - sg))
    else:
        th = torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))
        f = 0.5 * g * (1.0 + th)
        df = 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * 0.7978845608028654 * (1.0 + 3.0 * 0.044715 * g * g)
    dh = s["dh"].float().view(m, -1, ROWS)
    dgu = torch.stack((dh * u * df, dh * f), dim=2).reshape(m, -1)
    return dgu.to(torch.bfloat16), (f * u).reshape(m, -1).to(torch.bfloat16)


def _sample_plain(s):
    """Weights are whole multiples of 2^-30 of the row's largest, so their sums are exact in any order."""
    z = s["logits"].float()
    b, v = z.shape
    m = z.amax(1, keepdim=True)
    t = s["temperature"].unsqueeze(1)
    x = (z - m) * (torch.full_like(t, LOG2E) / t)
    e = torch.exp2(x)
    w = torch.round(e * UNIT).to(torch.int64)
    wi = w
    if s["top_k"] is not None or s["top_p"] is not None or s["min_p"] is not None:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        ws = w.gather(1, order)
        rank = torch.arange(v, device=z.device).unsqueeze(0)
        keep = torch.ones_like(ws, dtype=torch.bool)
        if s["top_k"] is not None:
            k = s["top_k"].unsqueeze(1)
            keep = (rank < k) | (k <= 0)
        if s["top_p"] is not None:
            p = s["top_p"].unsqueeze(1)
            wk = torch.where(keep, ws, 0)
            before = wk.cumsum(1) - wk
            total = wk.sum(1, keepdim=True)
            keep = keep & ((before.double() < p.double() * total.double()) | (p >= 1.0))
        if s["min_p"] is not None:
            keep = keep & (e.gather(1, order) >= s["min_p"].unsqueeze(1))
        keep = keep | (rank == 0)
        wi = torch.zeros_like(w).scatter(1, order, torch.where(keep, ws, 0))
    cdf = wi.cumsum(1)
    total = cdf[:, -1:]
    target = (s["uniform"].unsqueeze(1).double() * total.double()).to(torch.int64)
    target = torch.minimum(target, total - 1)
    token = (cdf <= target).sum(1)
    drawn = x.gather(1, token.unsqueeze(1)).squeeze(1)
    logprob = drawn * (1.0 / LOG2E) - torch.log(total.squeeze(1).float() * (1.0 / UNIT))
    return token.to(torch.int32), logprob


# ------------------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    if op in ("norm", "norm_grad"):
        # the forward pass as one function; the backward pass by differentiating it, with the stream
        # after the block as the point the second norm is taken at
        off, eps = case["offset"], 1e-6
        names = [n for n in ("x", "y", "gate", "w_pre", "w_post") if d[n] is not None]
        leaf = {n: d[n].clone().requires_grad_(op == "norm_grad") for n in names}

        def rms(v, w):
            return v / torch.sqrt(torch.mean(v ** 2, dim=-1, keepdim=True) + eps) * (w + off)

        def branch():
            n = rms(leaf["y"], leaf["w_post"])
            return case["scale"] * (n * leaf["gate"] if "gate" in leaf else n)

        if op == "norm":
            r = leaf["x"] + branch() if "y" in leaf else leaf["x"]
            return r, rms(r, leaf["w_pre"])
        delta = branch() if "y" in leaf else torch.zeros_like(leaf["x"])
        r = leaf["x"] + delta - delta.detach()
        loss = (rms(r, leaf["w_pre"]) * d["dh"]).sum() + (r * d["dx_out"]).sum()
        got = dict(zip(names, torch.autograd.grad(loss, [leaf[n] for n in names])))
        return tuple(got.get(n) for n in ("x", "y", "w_pre", "w_post", "gate"))
    if op in ("gated", "gated_grad"):
        value = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        value = torch.tensor(value + [-v for v in value], dtype=torch.float64, device="cuda")

        def matrix(q, sf):
            rows, kb = q.shape
            out = torch.empty(rows, 2 * kb, dtype=torch.float64, device="cuda")
            out[:, 0::2] = value[(q % 16).long()]
            out[:, 1::2] = value[(q // 16).long()]
            r = torch.arange(rows, device="cuda").view(-1, 1)
            j = torch.arange(kb // 8, device="cuda").view(1, -1)
            tiles = (kb // 8 + 3) // 4
            at = (r // 128 * tiles + j // 4) * 512 + r % 32 * 16 + r // 32 % 4 * 4 + j % 4
            code = sf[at].long()
            ex, man = code // 8, (code % 8).double()
            scale = torch.where(ex == 0, man * 2.0 ** -9, (1.0 + man / 8.0) * torch.exp2((ex - 7).double()))
            return out * scale.repeat_interleave(16, dim=1)

        a, w = matrix(s["a"], s["sfa"]), matrix(s["b"], s["sfb"])
        r = torch.arange(w.shape[0], device="cuda")
        g = a @ w[r % 32 < 16].t() * d["alpha"][0]
        u = a @ w[r % 32 >= 16].t() * d["alpha"][1]
        g.requires_grad_(op == "gated_grad")
        if case["act"] == "silu":
            f = g * torch.sigmoid(g)
        else:
            f = torch.nn.functional.gelu(g, approximate="tanh")
        if op == "gated":
            return f * u
        (dg,) = torch.autograd.grad((f * u * d["dh"]).sum(), g)
        du = d["dh"] * f.detach()
        m = dg.shape[0]
        dgu = torch.cat((dg.view(m, -1, 16), du.view(m, -1, 16)), dim=2).view(m, -1)
        return dgu, (f * u).detach()
    # the draw from real weights: a token that the whole-number weights draw otherwise is next to it
    z = d["logits"]
    t = d["temperature"].view(-1, 1)
    lp = torch.log_softmax(z / t, dim=1)
    val, order = torch.sort(lp, dim=1, descending=True, stable=True)
    v = z.shape[1]
    rank = torch.arange(v, device="cuda").view(1, -1)
    cut = torch.full((z.shape[0], 1), v, device="cuda")
    if d["top_k"] is not None:
        cut = torch.where(d["top_k"].view(-1, 1) > 0, d["top_k"].view(-1, 1).long(), cut)
    if d["top_p"] is not None:
        p = torch.where(rank < cut, val.exp(), 0.0)
        p = p / p.sum(1, keepdim=True)
        cut = torch.minimum(cut, ((p.cumsum(1) - p) < d["top_p"].view(-1, 1)).sum(1, keepdim=True))
    if d["min_p"] is not None:
        cut = torch.minimum(cut, ((val - val[:, :1]).exp() >= d["min_p"].view(-1, 1)).sum(1, keepdim=True))
    cut = cut.clamp(min=1)
    kept = torch.zeros_like(lp).scatter(1, order, torch.where(rank < cut, val.exp(), 0.0))
    cdf = kept.cumsum(1)
    token = (cdf <= d["uniform"].view(-1, 1) * cdf[:, -1:]).sum(1).clamp(max=v - 1)
    return None, torch.log(kept.gather(1, token.view(-1, 1)).squeeze(1) / cdf[:, -1])
