"""Sizes of the grouped products' tests, and what the products are in 64 bits on the CPU."""
import torch

# rows of each expert, in, out
SHAPES = [
    ([1], 8, 8), ([3], 1, 1), ([0, 1, 0], 7, 5), ([1, 1, 1, 1], 64, 16), ([5, 0, 2, 17], 72, 40), ([33, 1, 0, 64], 136, 264),
    ([130, 2, 31], 200, 304), ([16] * 9, 1000, 360), ([0, 0, 0], 64, 64), ([257, 300, 0, 511], 320, 520),
    ([161, 1, 90], 513, 257), ([700], 192, 136), ([4] * 70, 128, 72), ([40, 65, 100, 129, 170, 200, 231, 256], 96, 280), ([300] * 9, 1536, 1600), ([161, 1, 40] * 20, 256, 1544),
]
# x_ld - in, first element's place, y_ld - out, first element's place
LAYOUTS = [(0, 0, 0, 0), (8, 8, 8, 8), (3, 1, 5, 1)]


def integers(g, *shape):
    """Whole numbers in -3 .. 3: their products and sums are exact in every order."""
    return torch.randint(-3, 4, shape, generator=g).double()


def batch(counts, seed, tokens=None):
    """offsets, gather (or None) and the generator of a batch with `counts` rows an expert."""
    g = torch.Generator().manual_seed(seed)
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32)
    rows = int(offsets[-1])
    gather = None if tokens is None else torch.randint(0, tokens, (rows,), generator=g).to(torch.int32)
    return offsets, gather, g


def spans(counts):
    lo = 0
    for e, n in enumerate(counts):
        yield e, lo, lo + n
        lo += n


def product(counts, x, gather, w):
    xr = x if gather is None else x[gather.long()]
    return torch.cat([xr[lo:hi] @ w[e].t() for e, lo, hi in spans(counts)])


def product_dx(counts, dy, w):
    return torch.cat([dy[lo:hi] @ w[e] for e, lo, hi in spans(counts)])


def product_dw(counts, x, gather, dy):
    xr = x if gather is None else x[gather.long()]
    return torch.stack([dy[lo:hi].t() @ xr[lo:hi] for e, lo, hi in spans(counts)])


def quantize(x):
    """Codes and scales of the rows of x (fp32 values), by fp32 operations."""
    x = x.float()
    m = x.abs().amax(1).clamp(min=2.0 ** -100)
    bad = ~torch.isfinite(x).all(1)
    q = torch.round(x * (torch.tensor(127.0) / m)[:, None])
    s = m / torch.tensor(127.0)
    q[bad], s[bad] = 0.0, float("nan")
    return q, s
