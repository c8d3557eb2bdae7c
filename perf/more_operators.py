"""Cases of the products of routed experts and of their update: what a user runs who
writes experts of another kind than the SwiGLU ones, trains them and serves them in
8 bits.

  product        y[r] = W[e] x[token of r] for the rows r of each expert e, bf16
  dx             its gradient at x's rows: dx[r] = W[e]^T dy[r]
  dw             its gradient at the weights: dW[e] = sum over r of dy[r] x[token of r]^T
  int8           the same product on 8-bit integers: tokens are rounded with a scale
                 each, weights have a scale for each output channel
  orthogonalize  an update's matrices brought near the nearest orthogonal ones, by
                 Newton-Schulz steps of degree five

Plain forms are elementary torch operations in 32 bits.  8-bit rows: with m the row's
largest magnitude (2^-100 where it is less) the scale is m / 127 and a code is
x (127 / m) rounded to the nearest whole number, ties to even.
"""
import math

import torch

own = False

STEPS = 5
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
FEW = 2.0 ** -100


def listed():
    return [
        # serving, one new token: 8 of 256 experts are read
        dict(name="product, one token", op="product", T=1, E=256, K=8, d=7168, out=2048, skew=0.0, pad=0, dtype="bf16"),
        # a prompt through the first product of all experts of a layer
        dict(name="product, prompt", op="product", T=4096, E=256, K=8, d=7168, out=2048, skew=0.0, pad=0, dtype="bf16"),
        # a small model of odd sizes with a few popular experts and some idle ones
        dict(name="product, odd and skewed", op="product", T=777, E=24, K=3, d=1000, out=360, skew=1.5, pad=0,
             dtype="bf16"),
        # training one GPU's share of the experts with the rows of a large batch
        dict(name="input gradient, expert shard", op="dx", T=16384, E=32, K=1, d=7168, out=2048, skew=0.0, pad=0,
             dtype="bf16"),
        # training a small model of odd sizes, gradients inside a wider buffer
        dict(name="input gradient, odd and skewed", op="dx", T=777, E=24, K=3, d=1001, out=363, skew=1.5, pad=5,
             dtype="fp32"),
        # that share's weight gradients, kept in 32 bits for the optimiser
        dict(name="weight gradient, expert shard", op="dw", T=16384, E=32, K=1, d=7168, out=2048, skew=0.0, pad=0,
             dtype="fp32"),
        # the small model's, in the weights' type
        dict(name="weight gradient, odd and skewed", op="dw", T=777, E=24, K=3, d=1000, out=360, skew=1.5, pad=0,
             dtype="bf16"),
        # serving in 8 bits, one new token
        dict(name="int8, one token", op="int8", T=1, E=256, K=8, d=7168, out=2048, skew=0.0, pad=0, dtype="bf16"),
        # serving in 8 bits, a decode batch: nearly all experts, a few rows each
        dict(name="int8, decode batch", op="int8", T=128, E=256, K=8, d=7168, out=2048, skew=0.0, pad=0, dtype="bf16"),
        # serving in 8 bits, a prompt
        dict(name="int8, prompt", op="int8", T=4096, E=256, K=8, d=7168, out=2048, skew=0.0, pad=0, dtype="bf16"),
        # an optimiser's step on some experts' first matrices
        dict(name="orthogonalize, experts", op="orthogonalize", n=8, rows=2048, cols=7168, dtype="bf16"),
        # on the second matrices of a small model, with more rows than columns, momentum in 32 bits
        dict(name="orthogonalize, small and tall", op="orthogonalize", n=24, rows=1000, cols=360, dtype="fp32"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("product", "product", "dx", "dw", "int8", "int8", "orthogonalize"))
    if op == "orthogonalize":
        a, b = sorted((_log(rng, 24, 2048), _log(rng, 24, 7168)))
        if rng.random() < 0.5:
            a, b = -(-a // 64) * 64, -(-b // 64) * 64
        a = min(a, 2048)
        most = 8 * 2048 * 2048 * (3 * 7168 + 2048) // (a * a * (3 * b + a))
        n = _log(rng, 1, max(1, min(64, most)))
        rows, cols = rng.choice(((a, b), (b, a)))
        return dict(op=op, n=n, rows=rows, cols=cols, dtype=rng.choice(("bf16", "fp32")))
    E = rng.choice((1, 4, 13, 32, 60, 256))
    K = min(E, rng.choice((1, 2, 5, 8)))
    d, out = _log(rng, 200, 7168), _log(rng, 96, 2048)
    if rng.random() < 0.5:
        d, out = -(-d // 128) * 128, -(-out // 128) * 128
    if rng.random() < 0.3:
        d, out = out, d
    return dict(op=op, T=max(1, _log(rng, 1, 16384) // K), E=E, K=K, d=d, out=out, skew=rng.choice((0.0, 1.0)),
                pad=rng.choice((0, 0, 3, 64)), dtype=rng.choice(("bf16", "bf16", "fp32")))


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _padded(v, pad):
    """v's values as the leading columns of a wider buffer."""
    if not pad:
        return v
    wide = v.new_zeros((v.shape[0], v.shape[1] + pad))
    wide[:, : v.shape[1]] = v
    return wide[:, : v.shape[1]]


def _empty(rows, cols, pad, dtype):
    return torch.empty((rows, cols + pad), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *n: torch.randn(n, device="cuda", generator=g)  # noqa: E731
    s = dict(case=case)
    if case["op"] == "orthogonalize":
        n, rows, cols = case["n"], case["rows"], case["cols"]
        # momentum of a gradient: most of its weight in a part of its directions
        G = rand(n, rows, cols)
        G.mul_(torch.exp(0.5 * rand(n, rows, 1))).mul_(torch.exp(0.5 * rand(n, 1, cols)))
        s["g"] = (G * 1e-3).to(_dtype(case))
        s["y"] = torch.empty((n, rows, cols), dtype=torch.bfloat16, device="cuda")
        # room for X and X X^T twice each, in 32 bits a value, with sides of whole 256
        r, c = (-(-v // 256) * 256 for v in sorted((rows, cols)))
        s["scratch"] = torch.empty(n * 8 * r * (r + c) + (1 << 20), dtype=torch.uint8, device="cuda")
        return s
    T, E, K, d, out, pad = (case[k] for k in ("T", "E", "K", "d", "out", "pad"))
    like = torch.arange(1, E + 1, device="cuda").float().pow(-case["skew"])[torch.randperm(E, device="cuda", generator=g)]
    noise = -torch.log(-torch.log(torch.rand((T, E), device="cuda", generator=g).clamp_(1e-6, 1 - 1e-6)))
    experts = torch.topk(like.log() + noise, K, dim=1).indices.reshape(-1)
    order = torch.sort(experts, stable=True).indices
    counts = torch.bincount(experts, minlength=E)
    s["gather"] = (order // K).to(torch.int32)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["used"] = torch.nonzero(counts).reshape(-1)
    s["most"] = int(counts.max())
    if case["op"] != "dx":
        s["x"] = _padded(rand(T, d).to(torch.bfloat16), pad)
    if case["op"] in ("dx", "dw"):
        s["dy"] = _padded(rand(T * K, out).to(torch.bfloat16), pad)
    if case["op"] == "dw":
        s["dw"] = torch.empty((E, out, d), dtype=_dtype(case), device="cuda")
        return s
    w = torch.empty((E, out, d), dtype=torch.bfloat16, device="cuda")
    step = max(1, (1 << 28) // (out * d))
    for e in range(0, E, step):
        w[e:e + step] = rand(min(step, E - e), out, d).mul_(d ** -0.5)
    s["y"] = _empty(T * K, d if case["op"] == "dx" else out, pad, _dtype(case))
    if case["op"] != "int8":
        s["w"] = w
        return s
    # rows of codes are whole runs of 128, zeros behind the last
    run = -(-d // 128) * 128
    s["w"] = torch.zeros((E, out, run), dtype=torch.int8, device="cuda")
    s["ws"] = torch.empty((E, out), device="cuda")
    for e in range(0, E, step):
        q, scale = _to_int8(w[e:e + step].float())
        s["w"][e:e + step, :, :d], s["ws"][e:e + step] = q.to(torch.int8), scale
    s["codes"] = torch.empty((T, run), dtype=torch.int8, device="cuda")
    s["scales"] = torch.empty(T, device="cuda")
    return s


# ---- plain forms ------------------------------------------------------------------------------


def _to_int8(x):
    """Codes (as 32-bit floats) and scales of the rows of x."""
    m = x.abs().amax(-1).clamp(min=FEW)
    return torch.round(x * (127.0 / m).unsqueeze(-1)), m / 127.0


def _places(st):
    """[used expert][place] -> row, and which places hold one."""
    row = st["offsets"][st["used"]][:, None] + torch.arange(st["most"], device="cuda")
    there = row < st["offsets"][st["used"] + 1][:, None]
    return row.clamp(max=st["case"]["T"] * st["case"]["K"] - 1).long(), there


def _product(st, transposed):
    row, there = _places(st)
    w = st["w"][st["used"]].float()
    if transposed:
        return torch.bmm(st["dy"].float()[row], w)[there].to(st["y"].dtype)
    x = st["x"].float()[st["gather"][row].long()]
    return torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2)[there].to(st["y"].dtype)


def _weight_gradient(st):
    row, there = _places(st)
    x = st["x"].float()[st["gather"][row].long()]
    dy = st["dy"].float()[row].masked_fill(~there[:, :, None], 0.0)
    dw = torch.zeros(st["dw"].shape, device="cuda")
    dw[st["used"]] = torch.bmm(dy.transpose(1, 2).contiguous(), x)
    return dw.to(st["dw"].dtype)


def _product_int8(st):
    row, there = _places(st)
    x, scale = _to_int8(st["x"].float())
    token = st["gather"][row].long()
    w = st["w"][st["used"], :, : st["case"]["d"]].float()
    y = torch.bmm(w, x[token].transpose(1, 2).contiguous()).transpose(1, 2)
    y = y * scale[token][:, :, None] * st["ws"][st["used"]][:, None, :]
    return y[there].to(st["y"].dtype)


def _orthogonal(st):
    x = st["g"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    # the squares' sum in 64 bits: it is long, and every value is divided by its root
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()
    x = (x / (norm + EPS)).float()
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        s = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16)


# ---- one pass ----------------------------------------------------------------------------------


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    if op == "product":
        return _product(state, False)
    if op == "dx":
        return _product(state, True)
    if op == "dw":
        return _weight_gradient(state)
    if op == "int8":
        return _product_int8(state)
    return _orthogonal(state)


def _run_own(op, s):
    import mixture_experts_layer_35_amd as moe

    case = s["case"]
    code = moe.MOE_BF16 if case["dtype"] == "bf16" else moe.MOE_F32
    if op == "orthogonalize":
        moe.moe_orthogonalize(case["n"], case["rows"], case["cols"], code, s["g"], STEPS, COEFFICIENTS * STEPS, EPS, 1.0,
                              s["y"], s["scratch"])
        return s["y"]
    E, d, out, rows = case["E"], case["d"], case["out"], case["T"] * case["K"]
    if op == "product":
        moe.moe_grouped_product(E, s["offsets"], rows, s["gather"], d, out, s["x"], s["x"].stride(0), s["w"], code,
                                s["y"], s["y"].stride(0))
        return s["y"]
    if op == "dx":
        moe.moe_grouped_product_dx(E, s["offsets"], rows, d, out, s["dy"], s["dy"].stride(0), s["w"], code, s["y"],
                                   s["y"].stride(0))
        return s["y"]
    if op == "dw":
        moe.moe_grouped_product_dw(E, s["offsets"], rows, s["gather"], d, out, s["x"], s["x"].stride(0), s["dy"],
                                   s["dy"].stride(0), code, s["dw"], False)
        return s["dw"]
    moe.moe_quantize_int8(case["T"], d, moe.MOE_BF16, s["x"], s["x"].stride(0), s["codes"], s["scales"])
    moe.moe_grouped_product_int8(E, s["offsets"], rows, s["gather"], d, out, s["codes"], s["scales"], s["w"], s["ws"],
                                 code, s["y"], s["y"].stride(0))
    return s["y"]


# ---- what a pass cannot do without ---------------------------------------------------------------


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "orthogonalize":
        n, r, c = case["n"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # a step: half of the symmetric X X^T, half of the symmetric square of that, and the product with X
        return {"bytes": n * r * c * (size + 2), "flops": STEPS * n * r * r * (c + r + 2 * c)}
    T, E, K, d, out = (case[k] for k in ("T", "E", "K", "d", "out"))
    flops = 2 * T * K * d * out
    p = [k ** -case["skew"] for k in range(1, E + 1)]
    touched = sum(1 - (1 - min(1.0, K * v / sum(p))) ** T for v in p)
    if case["op"] == "dw":
        return {"bytes": T * d * 2 + T * K * out * 2 + E * d * out * size, "flops": flops}
    if case["op"] == "dx":
        return {"bytes": touched * d * out * 2 + T * K * out * 2 + T * K * d * size, "flops": flops}
    if case["op"] == "int8":
        return {"bytes": touched * (d + 4) * out + T * d * 2 + T * K * out * size, "flops": flops}
    return {"bytes": touched * d * out * 2 + T * d * 2 + T * K * out * size, "flops": flops}


# ---- the definitions in 64 bits -------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonalize":
        a, b, c = COEFFICIENTS
        y = torch.empty(s["g"].shape, dtype=torch.float64, device="cuda")
        for i, m in enumerate(s["g"]):
            m = m.double()
            wide = m if m.shape[0] <= m.shape[1] else m.t().contiguous()
            wide = wide / (torch.linalg.vector_norm(wide) + EPS)
            for _ in range(STEPS):
                # X <- a X + b (X X^T) X + c (X X^T)^2 X, from the right
                first = (wide @ wide.t()) @ wide
                second = (wide @ wide.t()) @ first
                wide = a * wide + b * first + c * second
            y[i] = wide if m.shape[0] <= m.shape[1] else wide.t()
        return y
    ends, token = s["offsets"].tolist(), s["gather"].long()
    out = s["dw"] if case["op"] == "dw" else s["y"]
    y = torch.zeros(out.shape, dtype=torch.float64, device="cuda")
    if case["op"] == "int8":
        x = s["x"].double()
        top = x.abs().amax(1, keepdim=True).clamp(min=FEW)
        # a code as the 32-bit rule gives it: its rounding is what the operator defines, its sums are not
        code = torch.round((x.float() * (127.0 / top.float()))).double()
    for e in range(case["E"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        if case["op"] == "dw":
            y[e] = s["dy"][lo:hi].double().t() @ s["x"][token[lo:hi]].double()
        elif case["op"] == "dx":
            y[lo:hi] = s["dy"][lo:hi].double() @ s["w"][e].double()
        elif case["op"] == "int8":
            w = s["w"][e, :, : case["d"]].double() * (s["ws"][e].double()[:, None])
            y[lo:hi] = (code[token[lo:hi]] * (top[token[lo:hi]] / 127.0)) @ w.t()
        else:
            y[lo:hi] = s["x"][token[lo:hi]].double() @ s["w"][e].double().t()
    return y
