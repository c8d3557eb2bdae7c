"""MX4 and gate definitions in 64 bits on the CPU, for the tests."""
import math

import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
MID = (GRID[1:] + GRID[:-1]) / 2


def runs(cols):
    return -(-cols // 128)


def quantize(x):
    """x [rows, cols] float64 -> codes [rows, 64 R], scales [rows, 4 R] (uint8), and each value's distance to the
    nearest rounding boundary in units of its block's scale."""
    rows, cols = x.shape
    v = torch.zeros((rows, runs(cols) * 128), dtype=torch.float64)
    v[:, :cols] = x
    b = v.view(rows, -1, 32)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(top)
    top = torch.where(bad, torch.ones_like(top), top)
    e = torch.tensor([0 if t == 0 else math.frexp(t)[1] - 1 for t in top.flatten().tolist()]).view(top.shape)
    s = torch.where(top == 0, torch.full_like(e, 127), (e - 2 + 127).clamp(min=0))
    y = (b.abs() / torch.pow(torch.tensor(2.0, dtype=torch.float64), (s - 127).double())[..., None])
    lo, hi = torch.bucketize(y, MID), torch.bucketize(y, MID, right=True)
    code = torch.where(lo % 2 == 0, lo, hi) + 8 * torch.signbit(b).long()
    code = torch.where(bad[..., None], torch.zeros_like(code), code)
    s = torch.where(bad, torch.full_like(s, 255), s)
    near = (y[..., None] - MID).abs().amin(-1).view(rows, -1)[:, :cols]
    pair = code.view(rows, -1, 2)
    return (pair[..., 0] + 16 * pair[..., 1]).to(torch.uint8), s.view(rows, -1).to(torch.uint8), near


def values(codes, scales, cols):
    """The float64 values that codes and scales stand for."""
    rows = codes.shape[0]
    c = codes.long()
    c = torch.stack([c % 16, c // 16], -1).view(rows, -1, 32)
    v = GRID[c % 8] * torch.where(c >= 8, -1.0, 1.0)
    s = scales.long()
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64), (s - 127).double())
    unit = torch.where(s == 255, torch.full_like(unit, float("nan")), unit)
    return (v * unit[..., None]).view(rows, -1)[:, :cols]


def scores(z, softmax):
    """z float64 -> scores; experts out of use (-infinity, NaN) score 0."""
    dead = ~(z > -math.inf)
    if softmax:
        m = torch.where(dead, torch.full_like(z, -math.inf), z).amax(1, keepdim=True)
        e = torch.where(z == m, torch.ones_like(z), torch.exp(z - m))
        e = torch.where(dead, torch.zeros_like(z), e)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1 / (1 + torch.exp(-z))
    return torch.where(dead, torch.zeros_like(z), s), dead


def gate(z, bias, G, M, K, softmax, group_max, renorm, scale):
    """idx, weights, choice values (before the groups are dropped), group scores."""
    T, E = z.shape
    s, dead = scores(z, softmax)
    c = s if bias is None else s + bias
    c = torch.where(dead | c.isnan(), torch.full_like(c, -math.inf), c)
    full = c
    by = c.view(T, G, E // G)
    top = by.sort(dim=2, descending=True).values
    best = top[..., 0].clone()
    if not group_max and E > G:
        best = best + torch.where(top[..., 1] == -math.inf, torch.zeros_like(best), top[..., 1])
    if G > 1:
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :M]
        keep = torch.zeros((T, G), dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), c, torch.full_like(c, -math.inf))
    order = c.sort(dim=1, descending=True, stable=True)
    idx = order.indices[:, :K]
    w = torch.where(order.values[:, :K] == -math.inf, torch.zeros(()).double(), s.gather(1, idx))
    return idx, weigh(w, renorm, scale), full, best


def weigh(w, renorm, scale):
    if renorm:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), torch.zeros_like(w))
    return w * scale
