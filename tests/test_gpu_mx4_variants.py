"""The MX4 experts in every variant of their kernels, chosen by sizes and alignment, against the definition."""
import pytest

import _definitions as ref
from test_gpu_mx4 import check, ffn, weights

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

MANY = [97, 161, 130, 132, 159, 160, 1, 200] * 2           # averages of 130 rows
VARIANTS = [
    # rows of each expert, d, inter
    (MANY, 2560, 2048),                                    # up to 160 tokens in both passes; scales in 16-byte pieces,
    (MANY, 2600, 2100),                                    # by words with an odd number of runs,
    (MANY, 2690, 2180),                                    # and with an even one
    ([5], 256, 2048),                                      # four waves a tile in the down pass,
    ([3, 2], 300, 1400),                                   # by words
    ([6], 1700, 1664),                                     # and in both passes by words
    ([6, 0, 3], 1600, 1792),
]


@pytest.mark.parametrize("counts,d,inter", VARIANTS, ids=lambda v: str(v)[:24])
def test_every_variant_against_the_definition(counts, d, inter):
    import mixture_experts_layer_35_amd as moe
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rows, n = sum(counts), len(counts)
    torch.manual_seed(rows + d)
    T = max(1, rows // 2)
    x, gather = torch.randn(T, d, dtype=torch.float64), torch.randint(0, T, (rows,))
    w = [weights(n, inter, d, 1), weights(n, inter, d, 2), weights(n, d, inter, 3)]
    y, xv = ffn(moe, counts, d, inter, x, gather, w, max_rows=rows + 3)
    check(y, counts, d, inter, xv, gather, w)


def late(t, by):
    """t's bytes at an address `by` bytes past a 256-byte boundary."""
    flat = torch.empty(t.numel() + 256, dtype=torch.uint8, device="cuda")
    view = flat[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    assert view.data_ptr() % 256 == by
    return view


@pytest.mark.parametrize("counts,d,inter", [([1, 0, 16, 2], 1024, 512), ([2] * 40, 512, 512), ([5], 256, 2048),
                                            ([40] * 40, 1024, 1024)], ids=lambda v: str(v)[:24])
def test_scales_at_4_byte_addresses(counts, d, inter):
    """Where 16-byte pieces of scales are out of reach, words serve the same sizes."""
    import mixture_experts_layer_35_amd as moe
    rows, n = sum(counts), len(counts)
    torch.manual_seed(rows + d)
    x, gather = torch.randn(rows, d, dtype=torch.float64), torch.randperm(rows)
    w = [weights(n, inter, d, 1), weights(n, inter, d, 2), weights(n, d, inter, 3)]
    xq, xs, _ = ref.quantize(x)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    y = torch.full((rows, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_ffn_mx4_workspace_bytes(rows, inter), dtype=torch.uint8, device="cuda")
    moe.moe_grouped_ffn_mx4(n, off, rows, gather.to(torch.int32).cuda(), d, inter, late(xq, 16), late(xs, 4),
                            [late(q, 48) for q, _, _ in w], [late(s, k) for k, (_, s, _) in zip((8, 12, 20), w)], y, ws)
    check(y, counts, d, inter, ref.values(xq, xs, d), gather, w)
