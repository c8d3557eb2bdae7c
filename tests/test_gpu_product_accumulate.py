"""Gradients at the weights added to what is there: experts without rows keep theirs to the bit."""
import pytest

import _product_cases as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF16 = torch.bfloat16
KEPT = (-0x80000000, 0x7FA12345, -0x55EDCC, 0x7F800000, 1, 0x3F800000)    # -0, two signalling NaN, infinity, 2^-149, 1


@pytest.mark.parametrize("counts", [[0], [0, 0, 40, 0, 7, 0], [0, 3, 0, 0, 70] * 50], ids=["none", "some", "many"])
@pytest.mark.parametrize("cin,cout", [(264, 272), (261, 259), (8, 8)], ids=["pieces", "odd", "small"])
def test_experts_without_rows(counts, cin, cout):
    import mixture_experts_layer_35_amd as moe
    rows = sum(counts)
    offsets, gather, g = ref.batch(counts, cin, 50)
    x, dy = ref.integers(g, 50, cin), ref.integers(g, rows, cout)
    start = torch.tensor(KEPT, dtype=torch.int64).to(torch.int32).repeat(len(counts) * cout * cin // len(KEPT) + 1)
    start = start[:len(counts) * cout * cin].view(len(counts), cout, cin).clone()
    busy = [e for e, n in enumerate(counts) if n]
    start[busy] = torch.full((1,), 2.0).view(torch.int32)
    dw = start.cuda().view(torch.float32)
    want = ref.product_dw(counts, x, gather, dy) if rows else None
    o, gd, xd, dd = offsets.cuda(), gather.cuda(), x.to(BF16).cuda(), dy.to(BF16).cuda()
    for times in (1, 2):
        moe.moe_grouped_product_dw(len(counts), o, rows, gd, cin, cout, xd, cin, dd, cout, moe.MOE_F32, dw, True)
        got = dw.view(torch.int32).cpu()
        idle = [e for e, n in enumerate(counts) if not n]
        assert (got[idle] == start[idle]).all()
        if busy:
            assert (dw.cpu()[busy].double() == 2 + times * want[busy]).all()
