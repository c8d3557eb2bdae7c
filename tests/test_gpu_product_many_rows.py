"""Products of one expert with as many rows as a call takes: 2^31 - 1."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF16 = torch.bfloat16
ROWS = (1 << 31) - 1


@pytest.mark.parametrize("side", [1, 8], ids=["odd", "pieces"])
def test_the_largest_batch(side):
    """side x side times the identity's whole multiples: each row's value is known, and exact in bf16."""
    import mixture_experts_layer_35_amd as moe
    torch.cuda.empty_cache()
    x = torch.empty((ROWS, side), dtype=BF16, device="cuda")
    flat = x.view(-1)
    step = 1 << 28
    for lo in range(0, flat.numel(), step):
        n = min(step, flat.numel() - lo)
        flat[lo:lo + n] = (torch.arange(lo, lo + n, device="cuda") % 29).to(BF16)
    w = (3 * torch.eye(side)).to(BF16).cuda().view(1, side, side)
    offsets = torch.tensor([0, ROWS], dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    for call in (lambda: moe.moe_grouped_product(1, offsets, ROWS, None, side, side, x, side, w, moe.MOE_BF16, y, side),
                 lambda: moe.moe_grouped_product_dx(1, offsets, ROWS, side, side, x, side, w, moe.MOE_BF16, y, side)):
        y.fill_(-1.0)
        call()
        got = y.view(-1)
        for lo in range(0, flat.numel(), step):
            assert torch.equal(got[lo:lo + step], 3 * flat[lo:lo + step]), lo
