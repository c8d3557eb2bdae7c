"""SiLU of the MX4 experts to the last bits: values of H a few fp32 roundings beside the middle of two codes."""
import math

import pytest

import _definitions as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

BITS, MARGIN = 24, 2.0 ** -20


def sums_of_powers(v, d):
    """Codes and scales of rows whose product with ones in every 32nd column is v (float64 of 24 bits at most): one
    bit a block, so that no order of the additions rounds."""
    codes = torch.zeros((len(v), d // 2), dtype=torch.uint8)
    scales = torch.full((len(v), d // 32), 127, dtype=torch.uint8)
    for f, x in enumerate(v.tolist()):
        m, e = math.frexp(abs(x))
        m = int(m * 2 ** BITS)
        assert m * 2.0 ** (e - BITS) == abs(x)
        for j in range(BITS):
            if m >> j & 1:
                codes[f, 16 * j] = 0x2 | (0x8 if x < 0 else 0)           # 1
                scales[f, j] = 127 + e - BITS + j
    return codes, scales


def test_silu_beside_the_middle_of_two_codes():
    """Feature f of a block of 32 has the gate value a and an up value b chosen so that silu(a) b lies 2^-20 of itself
    beside a middle of two codes.  A result within fp32's roundings of the formula (the exponential 2 ulp; 1 + exp, the
    quotient and the product half an ulp each, b's own rounding a quarter: below 2^-21) gives the code on its side."""
    import mixture_experts_layer_35_amd as moe
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    d, inter, unit = 768, 640, 2.0 ** -40
    g = torch.Generator().manual_seed(1)
    a = (torch.rand(inter, generator=g, dtype=torch.float64) * 105 - 85).mul(256).round() / 256
    a = torch.where(a == 0, 1.0, a)
    mid = ref.MID[torch.randint(0, 6, (inter,), generator=g)]            # below 5 units
    side = torch.randint(0, 2, (inter,), generator=g).double() * 2 - 1
    h = mid * unit * (1 + side * MARGIN)
    h[::32], a[::32] = 5.5 * unit, 2.0                                   # sets the block's scale
    silu = a / (1 + torch.exp(-a))
    b = (h / silu).float().double()
    h = silu * b
    codes, scales, near = ref.quantize(h[None])
    assert float(near.min()) > 0.2 * MARGIN and (scales == 127 - 40).all()

    w = [sums_of_powers(a, d), sums_of_powers(b, d)]
    down = torch.zeros((d, inter), dtype=torch.float64)
    down[torch.arange(inter), torch.arange(inter)] = 1.0
    w.append(ref.quantize(down)[:2])
    x = torch.zeros((1, d), dtype=torch.float64)
    x[:, : 32 * BITS: 32] = 1.0
    xq, xs, _ = ref.quantize(x)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    y = torch.empty((1, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_ffn_mx4_workspace_bytes(1, inter), dtype=torch.uint8, device="cuda")
    moe.moe_grouped_ffn_mx4(1, off, 1, None, d, inter, xq.cuda(), xs.cuda(), [q.cuda() for q, _ in w],
                            [s.cuda() for _, s in w], y, ws)
    want = ref.values(codes, scales, inter)[0]
    got = y[0, :inter].double().cpu()
    wrong = torch.nonzero(got != want).flatten()
    assert len(wrong) == 0, [(float(a[f]), float(got[f] / unit), float(want[f] / unit)) for f in wrong[:5]]
