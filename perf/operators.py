"""Cases of the gate and of the MX4 experts: what a layer of routed experts runs
between its gate projection and its combine.

  gate           scores, biased and group-limited choice, weights, from logits
  gate_backward  the gradient of those weights (and of the scores) at the logits
  mx4            rounding to microscaled 4-bit floating point and back
  ffn            the SwiGLU experts on MX4 weights and MX4 activations

Plain forms are elementary torch operations in 32 bits.  MX4: blocks of 32 values
along a row share a power of two 2^(s - 127), s = exponent field of the block's
largest magnitude minus 2 (at least 0); a value is the nearest of
+-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times that, ties to the even code, larger ones to 6.
A row holds whole runs of 128 values (64 code bytes, low nibble first, and 4 scale
bytes), zeros after the last one.
"""
import math

import torch

own = False

INF = float("inf")
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # serving, one new token: routed to 8 of 256 experts, at most 4 of 8 groups
        dict(name="gate, one token", op="gate", T=1, E=256, G=8, M=4, K=8, score="sigmoid", group="top2", bias=True,
             dtype="fp32", pad=0, renorm=True, scale=1.0, dead=0),
        # a long prompt or a training batch through the same gate
        dict(name="gate, prompt", op="gate", T=16384, E=256, G=8, M=4, K=8, score="sigmoid", group="top2", bias=True,
             dtype="fp32", pad=0, renorm=True, scale=1.0, dead=0),
        # many small experts with softmax scores, bf16 logits in a padded buffer, two experts offline
        dict(name="gate, softmax", op="gate", T=65521, E=64, G=1, M=1, K=6, score="softmax", group="max", bias=False,
             dtype="bf16", pad=16, renorm=False, scale=1.0, dead=2),
        # training: the gate's gradient for that batch
        dict(name="gate gradient, sigmoid", op="gate_backward", T=16384, E=256, G=8, M=4, K=8, score="sigmoid",
             group="top2", bias=True, dtype="fp32", pad=0, renorm=True, scale=2.5, dead=0, aux=False),
        # training: softmax scores that also carry the gradient of a balance loss
        dict(name="gate gradient, softmax", op="gate_backward", T=65521, E=64, G=1, M=1, K=6, score="softmax",
             group="max", bias=False, dtype="bf16", pad=16, renorm=False, scale=1.0, dead=2, aux=True),
        # hidden states of a decode batch on their way into the experts
        dict(name="mx4, decode batch", op="mx4", rows=128, cols=7168, pad=0, dtype="bf16"),
        # hidden states of a long prompt
        dict(name="mx4, prompt", op="mx4", rows=16384, cols=7168, pad=0, dtype="bf16"),
        # serving, one new token: 8 of 256 experts are read
        dict(name="ffn, one token", op="ffn", T=1, E=256, K=8, d=7168, inter=2048, skew=0.0),
        # serving, a decode batch: nearly all experts, a few rows each
        dict(name="ffn, decode batch", op="ffn", T=128, E=256, K=8, d=7168, inter=2048, skew=0.0),
        # a prompt through all experts of one layer
        dict(name="ffn, prompt", op="ffn", T=4096, E=256, K=8, d=7168, inter=2048, skew=0.0),
        # one GPU's share of the experts under expert parallelism, with the rows of a large batch
        dict(name="ffn, expert shard", op="ffn", T=16384, E=32, K=1, d=7168, inter=2048, skew=0.0),
        # a small model of odd sizes with a few popular experts and some idle ones
        dict(name="ffn, odd and skewed", op="ffn", T=777, E=24, K=3, d=1000, inter=360, skew=1.5),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("gate", "gate_backward", "mx4", "ffn", "ffn"))
    if op == "mx4":
        cols = _log(rng, 32, 8192)
        return dict(op=op, rows=_log(rng, 1, 16384 * 7168 // max(cols, 7168)), cols=cols, pad=rng.choice((0, 3, 64)),
                    dtype=rng.choice(("bf16", "fp32")))
    if op == "ffn":
        E = rng.choice((1, 4, 13, 32, 60, 256))
        K = min(E, rng.choice((1, 2, 5, 8)))
        d, inter = _log(rng, 200, 7168), _log(rng, 96, 2048)
        if rng.random() < 0.5:
            d, inter = -(-d // 128) * 128, -(-inter // 128) * 128
        return dict(op=op, T=max(1, _log(rng, 1, 16384) // K), E=E, K=K, d=d, inter=inter,
                    skew=rng.choice((0.0, 1.0)))
    G = rng.choice((1, 1, 4, 8))
    E = G * _log(rng, 16 // G + 2, 512 // G)
    M = rng.randint((G + 1) // 2, G)
    K = min(rng.choice((1, 2, 4, 6, 8, 10)), M * (E // G))
    score = rng.choice(("sigmoid", "softmax"))
    c = dict(op=op, T=_log(rng, 1, 16384 * 256 // max(E, 256)), E=E, G=G, M=M, K=K, score=score,
             group=rng.choice(("top2", "max")), bias=rng.random() < 0.5, dtype=rng.choice(("bf16", "fp32")),
             pad=rng.choice((0, 5, 32)), renorm=K > 1 and rng.random() < 0.5, scale=rng.choice((1.0, 2.5)),
             dead=rng.choice((0, 0, 1)))
    if op == "gate_backward":
        c["aux"] = rng.random() < 0.5
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _padded(v, pad):
    """v's values as the leading columns of a wider buffer."""
    if not pad:
        return v
    wide = v.new_zeros((v.shape[0], v.shape[1] + pad))
    wide[:, : v.shape[1]] = v
    return wide[:, : v.shape[1]]


def prepare(case, seed):
    g = _gen(seed)
    rand = lambda *n: torch.randn(n, device="cuda", generator=g)  # noqa: E731
    s = dict(case=case)
    if case["op"] == "mx4":
        x = rand(case["rows"], case["cols"]) * torch.exp(rand(case["rows"], 1))
        s["x"] = _padded(x.to(_dtype(case)), case["pad"])
        runs = -(-case["cols"] // 128)
        s["codes"] = torch.empty((case["rows"], 64 * runs), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((case["rows"], 4 * runs), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty((case["rows"], case["cols"]), dtype=torch.bfloat16, device="cuda")
        return s
    if case["op"] == "ffn":
        T, E, K, d, inter = (case[k] for k in ("T", "E", "K", "d", "inter"))
        s["x"] = rand(T, d).to(torch.bfloat16)
        like = torch.arange(1, E + 1, device="cuda").float().pow(-case["skew"])[torch.randperm(E, device="cuda", generator=g)]
        noise = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=g).clamp_(1e-6, 1 - 1e-6)))
        experts = torch.topk(like.log() + noise, K, dim=1).indices.reshape(-1)
        order = torch.sort(experts, stable=True).indices
        counts = torch.bincount(experts, minlength=E)
        s["gather"] = (order // K).to(torch.int32)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["used"] = torch.nonzero(counts).reshape(-1)
        s["most"] = int(counts.max())
        s["w"], s["ws"] = [], []
        for n, k in ((inter, d), (inter, d), (d, inter)):
            runs = -(-k // 128)
            codes = torch.empty((E, n, 64 * runs), dtype=torch.uint8, device="cuda")
            scales = torch.empty((E, n, 4 * runs), dtype=torch.uint8, device="cuda")
            step = max(1, (1 << 28) // (n * k))
            for e in range(0, E, step):
                m = min(step, E - e)
                codes[e:e + m], scales[e:e + m] = _to_mx4(rand(m, n, k).mul_(k ** -0.5))
            s["w"].append(codes)
            s["ws"].append(scales)
        runs = -(-d // 128)
        s["codes"] = torch.empty((T, 64 * runs), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((T, 4 * runs), dtype=torch.uint8, device="cuda")
        s["y"] = torch.empty((T * K, d), dtype=torch.bfloat16, device="cuda")
        s["scratch"] = torch.empty(T * K * -(-inter // 128) * 68 + 65536, dtype=torch.uint8, device="cuda")
        return s
    T, E, K = case["T"], case["E"], case["K"]
    z = rand(T, E)
    if case["dead"]:
        z[:, torch.randperm(E, device="cuda", generator=g)[: min(case["dead"], E - K)]] = -INF
    s["logits"] = _padded(z.to(_dtype(case)), case["pad"])
    s["bias"] = torch.rand(E, device="cuda", generator=g) * 0.2 - 0.1 if case["bias"] else None
    s["idx"] = torch.empty((T, K), dtype=torch.int32, device="cuda")
    s["weights"] = torch.empty((T, K), device="cuda")
    if case["op"] == "gate_backward":
        s["idx"], s["weights"] = _gate(s)
        s["dweights"] = rand(T, K)
        s["dscores"] = rand(T, E) * 0.01 if case["aux"] else None
        s["dlogits"] = torch.empty((T, E), dtype=_dtype(case), device="cuda")
    return s


# ---- plain forms ------------------------------------------------------------------------------


def _scores(z, score):
    """Scores of the logits z, and where there is none: at minus infinity and NaN."""
    dead = ~(z > -INF)
    if score == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
    else:
        m = z.masked_fill(dead, -INF).amax(1, keepdim=True)
        e = torch.exp(z - m).masked_fill(z == m, 1.0).masked_fill(dead, 0.0)
        # the sum is rounded once, so that no order of the additions shows in a choice
        s = e * (1.0 / e.sum(1, keepdim=True, dtype=torch.float64).float())
    return s.masked_fill(dead, 0.0), dead


def _gate(st):
    case = st["case"]
    T, E, G = case["T"], case["E"], case["G"]
    s, dead = _scores(st["logits"].float(), case["score"])
    c = s if st["bias"] is None else s + st["bias"]
    c = c.masked_fill(dead | c.isnan(), -INF)
    if G > 1:
        top = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values
        best = top[:, :, 0]
        if case["group"] == "top2" and E > G:
            best = torch.where(top[:, :, 1] > -INF, best + top[:, :, 1], best)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : case["M"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=c.device).scatter_(1, kept, True)
        c = c.view(T, G, E // G).masked_fill(~keep[:, :, None], -INF).view(T, E)
    order = torch.sort(c, dim=1, descending=True, stable=True)
    idx = order.indices[:, : case["K"]]
    w = s.gather(1, idx).masked_fill(order.values[:, : case["K"]] == -INF, 0.0)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = (w / total).masked_fill(total == 0, 0.0)
    return idx.to(torch.int32), w * case["scale"]


def _gate_gradient(st):
    case = st["case"]
    s, dead = _scores(st["logits"].float(), case["score"])
    idx = st["idx"].long()
    live = st["weights"] != 0
    sel, dw = s.gather(1, idx) * live, st["dweights"] * live
    if case["renorm"]:
        total = sel.sum(1, keepdim=True)
        inv = torch.where(total > 0, 1.0 / total, 0.0)
        dw = dw - dw[:, :1]  # the weights' sum is fixed: a common part of their gradients moves nothing
        dsel = (dw - (dw * sel).sum(1, keepdim=True) * inv) * inv * live
    else:
        dsel = dw
    ds = torch.zeros_like(s) if st["dscores"] is None else st["dscores"].masked_fill(dead, 0.0)
    ds = ds.scatter_add(1, idx, dsel * case["scale"])
    if case["score"] == "sigmoid":
        dz = ds * s * (1.0 - s)
    else:
        dz = s * (ds - (ds * s).sum(1, keepdim=True))
    return dz.to(st["logits"].dtype)


def _blocks(x):
    """x with zeros up to a whole number of 128-value runs, as blocks of 32, and the blocks' scale bytes."""
    cols = x.shape[-1]
    runs = -(-cols // 128)
    if cols % 128:
        x = torch.nn.functional.pad(x, (0, runs * 128 - cols))
    x = x.reshape(*x.shape[:-1], runs * 4, 32)
    top = x.abs().amax(-1)
    s = torch.where(top > 0, ((top.view(torch.int32) >> 23) - 2).clamp(min=0), 127)
    return x, s


def _power(e):
    """2^e in 32 bits for whole e from -126 to 127."""
    return ((e + 127) << 23).view(torch.float32)


def _steps(x, s):
    """Magnitudes of the blocks x over their scale, on the grid."""
    y = (x.abs() * _power(127 - s).unsqueeze(-1)).clamp(max=6.0)
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return torch.round(y / step) * step


def _on_grid(x):
    """x's values once they are held in MX4."""
    b, s = _blocks(x)
    # 2^(s - 127) as two factors: s = 0 alone is below the smallest normal number
    v = torch.copysign(_steps(b, s), b) * _power(s.clamp(min=1) - 127).unsqueeze(-1) * torch.where(s > 0, 1.0, 0.5).unsqueeze(-1)
    return v.reshape(*x.shape[:-1], -1)[..., : x.shape[-1]]


def _to_mx4(x):
    """Codes and scale bytes of x."""
    b, s = _blocks(x)
    q = _steps(b, s)
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    code = code + 8 * (torch.signbit(b)).to(torch.uint8)
    code = code.reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), s.reshape(*x.shape[:-1], -1).to(torch.uint8)


def _values(codes, scales):
    """The values that codes and scale bytes stand for, zeros after the last one among them."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    byte = torch.arange(256, device=codes.device)
    pairs = torch.stack([grid[byte & 15], grid[byte >> 4]], 1)
    v = torch.nn.functional.embedding(codes.to(torch.int32), pairs).view(*scales.shape, 32)
    return v.mul_(_power(scales.to(torch.int32) - 127).unsqueeze(-1)).flatten(-2)


def _experts(st):
    case, used = st["case"], st["used"]
    d, inter = case["d"], case["inter"]
    x = _on_grid(st["x"].float())
    row = st["offsets"][used][:, None] + torch.arange(st["most"], device="cuda")
    there = row < st["offsets"][used + 1][:, None]
    x = x[st["gather"][row.clamp(max=case["T"] * case["K"] - 1)].long()]
    x = x.transpose(1, 2).contiguous()
    w = lambda k, n: _values(st["w"][k][used], st["ws"][k][used])[..., :n].contiguous()  # noqa: E731
    a, b = torch.bmm(w(0, d), x), torch.bmm(w(1, d), x)
    h = (a / (1.0 + torch.exp(-a)) * b).transpose(1, 2)
    h = _on_grid(h.contiguous()).transpose(1, 2).contiguous()
    y = torch.bmm(w(2, inter), h).transpose(1, 2)[there]
    return y.to(torch.bfloat16)


# ---- one pass ----------------------------------------------------------------------------------


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "gate":
        return dict(zip(("idx", "weights"), _gate(state)))
    if case["op"] == "gate_backward":
        return _gate_gradient(state)
    if case["op"] == "mx4":
        return _on_grid(state["x"].float()).to(torch.bfloat16)
    return _experts(state)


def _run_own(case, s):
    import mixture_experts_layer_35_amd as moe

    if case["op"] in ("gate", "gate_backward"):
        rule = moe.make_gate_rule(case["T"], case["E"], case["K"], score=case["score"], n_groups=case["G"],
                                  topk_groups=case["M"], group_score=case["group"], renormalize=case["renorm"],
                                  routed_scale=case["scale"], logits=case["dtype"])
        z = s["logits"]
        if case["op"] == "gate":
            moe.moe_gate(rule, z, z.stride(0), s["bias"], None, s["idx"], s["weights"])
            return {"idx": s["idx"], "weights": s["weights"]}
        moe.moe_gate_backward(rule, z, z.stride(0), s["idx"], s["weights"], s["dweights"], s["dscores"], s["dlogits"],
                              s["dlogits"].stride(0))
        return s["dlogits"]
    x = s["x"]
    rows, cols = x.shape
    dtype = moe.MOE_BF16 if x.dtype == torch.bfloat16 else moe.MOE_F32
    moe.moe_quantize_mx4(rows, cols, dtype, x, x.stride(0), s["codes"], s["scales"])
    if case["op"] == "mx4":
        moe.moe_dequantize_mx4(rows, cols, s["codes"], s["scales"], moe.MOE_BF16, s["y"], s["y"].stride(0))
    else:
        moe.moe_grouped_ffn_mx4(case["E"], s["offsets"], s["y"].shape[0], s["gather"], case["d"], case["inter"],
                                s["codes"], s["scales"], s["w"], s["ws"], s["y"], s["scratch"])
    return s["y"]


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    if case["op"] == "mx4":
        n = case["rows"] * case["cols"]
        # in, codes and scales out; the codes and scales in again, the values out
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + 2 * (0.5 + 1 / 32) + 2), "flops": 4 * n}
    if case["op"] == "ffn":
        T, E, K, d, inter = (case[k] for k in ("T", "E", "K", "d", "inter"))
        p = [k ** -case["skew"] for k in range(1, E + 1)]
        touched = sum(1 - (1 - min(1.0, K * v / sum(p))) ** T for v in p)
        return {"bytes": touched * 3 * d * inter * (0.5 + 1 / 32) + T * d * 2 + T * K * d * 2,
                "flops": 6 * T * K * d * inter}
    T, E, K, size = case["T"], case["E"], case["K"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "gate":
        return {"bytes": T * E * size + T * K * 8, "flops": 10 * T * E}
    # sigmoid scores without a gradient of their own need the chosen logits alone
    read = T * E * size if case["score"] == "softmax" or case["aux"] else T * K * size
    return {"bytes": read + T * E * size + (T * E * 4 if case["aux"] else 0) + T * K * 12, "flops": 10 * T * E}


# ---- the definitions in 64 bits -------------------------------------------------------------------


def _unit(e):
    """2^e in 64 bits for whole e."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _nearest(x):
    """x (64 bits) in MX4, by a search of the grid's midpoints; the values."""
    cols = x.shape[-1]
    fill = -cols % 32
    x = torch.cat([x, x.new_zeros(*x.shape[:-1], fill)], -1).reshape(*x.shape[:-1], -1, 32)
    top = x.abs().amax(-1, keepdim=True)
    exponent = torch.frexp(top).exponent - 1
    unit = _unit((exponent - 2).clamp(min=-127))
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    middle = (grid[1:] + grid[:-1]) / 2
    y = x.abs() / unit
    below, above = torch.bucketize(y, middle, right=False), torch.bucketize(y, middle, right=True)
    code = torch.where(below % 2 == 0, below, above)  # they differ at a midpoint alone: the even one of the two
    return (torch.sign(x) * grid[code] * unit).flatten(-2)[..., :cols]


def _gate_64(case, s):
    z = s["logits"].double()
    if case["score"] == "sigmoid":
        p = torch.sigmoid(z)
    else:
        p = torch.softmax(z, 1)
    return z, p


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "mx4":
        return torch.cat([_nearest(part.double()) for part in s["x"].split(1024)])
    if case["op"] == "ffn":
        x = _nearest(s["x"].double())
        y = torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")
        grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device="cuda")

        def weight(k, e, n):
            c = s["w"][k][e].long()
            v = torch.stack([grid[c % 16], grid[c // 16]], -1).flatten(-2)
            return (v * _unit(s["ws"][k][e].long() - 127).repeat_interleave(32, -1))[:, :n].t().contiguous()

        ends = s["offsets"].tolist()
        for e in range(case["E"]):
            lo, hi = ends[e], ends[e + 1]
            if lo == hi:
                continue
            u = x[s["gather"][lo:hi].long()]
            a, b = u @ weight(0, e, case["d"]), u @ weight(1, e, case["d"])
            y[lo:hi] = _nearest(a * torch.sigmoid(a) * b) @ weight(2, e, case["inter"])
        return y
    z, p = _gate_64(case, s)
    T, E, G, K = (case[k] for k in ("T", "E", "G", "K"))
    if case["op"] == "gate":
        c = p + s["bias"].double() if s["bias"] is not None else p.clone()
        c[z == -INF] = -INF
        if G > 1:
            by = c.view(T, G, E // G)
            best = by.amax(2)
            if case["group"] == "top2" and E > G:
                two = by.topk(2, 2).values
                best = two[:, :, 0] + two[:, :, 1].masked_fill(two[:, :, 1] == -INF, 0.0)
            out = best.argsort(dim=1, descending=True, stable=True)[:, case["M"]:]
            c = by.clone().scatter_(1, out[:, :, None].expand(-1, -1, E // G), -INF).view(T, E)
        at = c.argsort(dim=1, descending=True, stable=True)[:, :K]
        w = p.gather(1, at) * (c.gather(1, at) > -INF)
        if case["renorm"]:
            w = torch.nan_to_num(w / w.sum(1, keepdim=True))
        return {"idx": None, "weights": w * case["scale"]}
    # the gradient by the chain rule on the chosen scores: dL/ds, then ds/dz
    idx, live = s["idx"].long(), (s["weights"] != 0).double()
    chosen, dw = p.gather(1, idx) * live, s["dweights"].double() * live
    if case["renorm"]:
        total = chosen.sum(1, keepdim=True).clamp(min=1e-300)
        share = chosen / total
        dchosen = (dw - (dw * share).sum(1, keepdim=True)) / total * live
    else:
        dchosen = dw
    ds = torch.zeros_like(p).scatter_add_(1, idx, dchosen * case["scale"])
    if s["dscores"] is not None:
        ds += s["dscores"].double()
    if case["score"] == "sigmoid":
        return ds * p * (1 - p)
    return p * (ds - (p * ds).sum(1, keepdim=True))
