"""moe_orthogonalize's arithmetic on the CPU, with single mistakes to plant in it, and a measure that sees errors well below
the rounding of the result to bf16.

X, S and P in two bf16 parts of 8 bits each, hi and lo; a product of pairs is hi hi + hi lo + lo hi, summed in fp32.  As long as
the steps left multiply by more than 64, a X takes a third part of X, with which it has all of fp32's 24 bits."""
import math

import torch

MUON = (3.4445, -4.7750, 2.0315)
MISTAKES = ["gram hi lo", "gram lo hi", "square hi lo", "square lo hi", "update hi lo", "update lo hi", "lo of the mirrored half",
            "lo of b S", "lo of a X", "bf16 throughout", "last part of X"]


def _bf(v):
    return v.to(torch.bfloat16).float()


def _parts(v):
    hi = _bf(v)
    lo = _bf(v - hi)
    return hi, lo, _bf(v - hi - lo)


def _product(a, b, name, mistake):
    s = a[0] @ b[0]
    if mistake == "bf16 throughout":
        return s
    if mistake != name + " hi lo":
        s = s + a[0] @ b[1]
    if mistake != name + " lo hi":
        s = s + a[1] @ b[0]
    return s


def pairs(g, coeffs=MUON * 5, eps=1e-7, mistake=None):
    """The last X of one matrix in fp32, not yet rounded to bf16."""
    tall = g.shape[0] > g.shape[1]
    x = g.double()
    x = (x * (1 / (x.square().sum().sqrt() + eps))).float()
    x = x.t().contiguous() if tall else x
    for k in range(0, len(coeffs), 3):
        a, b, c = coeffs[k:k + 3]
        hi, lo, rest = _parts(x)
        if mistake in ("bf16 throughout", "last part of X") or math.prod(abs(v) for v in coeffs[k::3]) <= 64:
            rest = torch.zeros_like(rest)
        if mistake == "bf16 throughout":
            lo = torch.zeros_like(lo)
        turned = (hi.t().contiguous(), lo.t().contiguous())
        sh, sl, _ = _parts(_product((hi, lo), turned, "gram", mistake))
        if mistake == "lo of the mirrored half":
            sl = sl.tril()
        if mistake == "bf16 throughout":
            sl = torch.zeros_like(sl)
        p = c * _product((sh, sl), (sh, sl), "square", mistake) + b * (sh + (0 if mistake == "lo of b S" else sl))
        ph, pl, _ = _parts(p)
        if mistake == "bf16 throughout":
            pl = torch.zeros_like(pl)
        ax = hi + rest if mistake == "lo of a X" else hi + lo + rest
        x = a * ax + _product((ph, pl), (hi, lo), "update", mistake)
    return x.t() if tall else x


def exact(g, coeffs=MUON * 5, eps=1e-7):
    """The formula in 64 bits."""
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    x = x / (x.square().sum().sqrt() + eps)
    for k in range(0, len(coeffs), 3):
        a, b, c = coeffs[k:k + 3]
        s = x @ x.t()
        x = a * x + (b * s + c * s @ s) @ x
    return x.t() if tall else x


# n, rows, cols, rank (0: full): between them every tile of every product, the last one's for wide and for tall matrices
PRECISE = [(1, 7, 5, 0), (2, 64, 200, 0), (2, 200, 64, 0), (6, 100, 36, 0), (1, 300, 301, 0), (3, 200, 512, 1), (2, 512, 200, 1),
           (1, 300, 301, 2), (1, 260, 700, 3), (60, 400, 410, 0), (64, 512, 256, 1), (60, 285, 288, 0), (20, 90, 800, 2),
           (60, 410, 400, 0), (64, 256, 511, 3), (20, 799, 90, 0)]


def matrices(n, rows, cols, rank):
    g = torch.Generator().manual_seed(rows * cols + n + rank)
    if rank:
        return torch.randn((n, rows, rank), generator=g) @ torch.randn((n, rank, cols), generator=g)
    return torch.randn((n, rows, cols), generator=g)


# Results are rounded to bf16, 1.7e-3 of their norm, which hides errors of a tenth of that.  The mean over results at many
# scales, each taken back, hides less: a value's rounding is another one at each scale.
SCALES = [2.0 ** float(v) for v in torch.rand(64, generator=torch.Generator().manual_seed(64), dtype=torch.float64)]
SCALES = torch.tensor(SCALES).float().tolist()                       # as fp32 holds them


def mean_of(y_at):
    """The mean of y / scale over SCALES, in 64 bits."""
    return sum(y_at(s).double().cpu() / s for s in SCALES) / len(SCALES)


def allowed(g, want):
    """The largest 2-norm of the mean's error for the arithmetic above with its sums in another order.

    The arithmetic's own error is one of independent roundings that another order of sums draws anew: its norm is the
    emulation's but for its spread, 1 / sqrt(2 N) of N draws (of rank * side draws at low rank), half of it from N = 18 at three
    spreads.  A rounding to bf16 errs by half a step at most, 2^-8 of the value, with a spread of 1 / sqrt(3) of that; the mean of K
    independent ones by 1 / sqrt(3 K), and the norm of N >= 35 such by at most 1.3 times as much at three spreads of sqrt(1 / (2 N))."""
    own = float((pairs(g).double() - want).norm())
    return 1.5 * own + 1.3 * 2.0 ** -8 / (3 * len(SCALES)) ** 0.5 * float(want.norm())
