"""Grouped products and updates of more tiles than workgroups: what passes from a tile to the next."""
import math

import pytest

import _product_cases as ref
from _product_many import GRADIENTS, PRODUCTS, UPDATES

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF16, FP32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_35_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("op,counts,cin,cout,kernel", PRODUCTS, ids=["%s-%d" % (c[0], c[4]) for c in PRODUCTS])
def test_products(moe, op, counts, cin, cout, kernel, dtype):
    """Whole numbers: exact."""
    n, rows, tokens = len(counts), sum(counts), 500
    offsets, gather, g = ref.batch(counts, 31, tokens)
    w, code = ref.integers(g, n, cout, cin), moe.MOE_BF16 if dtype == BF16 else moe.MOE_F32
    out = torch.full((rows + 3, cin if op == "dx" else cout), math.nan, dtype=dtype, device="cuda")
    o, gd = offsets.cuda(), gather.cuda()
    if op == "dx":
        dy = ref.integers(g, rows, cout)
        moe.moe_grouped_product_dx(n, o, rows + 3, cin, cout, dy.to(BF16).cuda(), cout, w.to(BF16).cuda(), code, out, cin)
        want = ref.product_dx(counts, dy, w)
    elif op == "y":
        x = ref.integers(g, tokens, cin)
        moe.moe_grouped_product(n, o, rows + 3, gd, cin, cout, x.to(BF16).cuda(), cin, w.to(BF16).cuda(), code, out, cout)
        want = ref.product(counts, x, gather, w)
    else:
        run = -(-cin // 128) * 128
        x = ref.integers(g, tokens, cin)
        xq, wq = torch.zeros(tokens, run, dtype=torch.int8), torch.zeros(n, cout, run, dtype=torch.int8)
        xq[:, :cin], wq[..., :cin] = x.to(torch.int8), w.to(torch.int8)
        xs, ws = 2.0 ** (torch.arange(tokens) % 5 - 2), 2.0 ** (torch.arange(n * cout).view(n, cout) % 7 - 3)
        moe.moe_grouped_product_int8(n, o, rows + 3, gd, cin, cout, xq.cuda(), xs.float().cuda(), wq.cuda(), ws.float().cuda(),
                                     code, out, cout)
        want = ref.product(counts, x * xs.double()[:, None], gather, w * ws.double()[:, :, None])
    assert torch.equal(out[:rows].double().cpu(), want.to(dtype).double())
    assert out[rows:].isnan().all()


@pytest.mark.parametrize("dtype,add", [(BF16, False), (FP32, False), (FP32, True)], ids=["bf16", "fp32", "added"])
@pytest.mark.parametrize("counts,cin,cout", GRADIENTS, ids=["pieces", "odd"])
def test_gradients_at_the_weights(moe, counts, cin, cout, dtype, add):
    n, rows, tokens = len(counts), sum(counts), 200
    offsets, gather, g = ref.batch(counts, 32, tokens)
    x, dy, start = ref.integers(g, tokens, cin), ref.integers(g, rows, cout), ref.integers(g, n, cout, cin)
    dw = (start if add else torch.full((n, cout, cin), math.nan)).to(dtype).cuda()
    moe.moe_grouped_product_dw(n, offsets.cuda(), rows, gather.cuda(), cin, cout, x.to(BF16).cuda(), cin, dy.to(BF16).cuda(), cout,
                               moe.MOE_BF16 if dtype == BF16 else moe.MOE_F32, dw, add)
    want = ref.product_dw(counts, x, gather, dy) + (start if add else 0)
    assert torch.equal(dw.double().cpu(), want.to(dtype).double())


@pytest.mark.parametrize("tall", [False, True], ids=["wide", "tall"])
@pytest.mark.parametrize("n,a,b", UPDATES)
def test_updates(moe, n, a, b, tall):
    """Seven matrices in turn: every copy of one has the same bits, and the first of each is the formula's."""
    from test_gpu_orthogonalize import MUON, check, exact
    rows, cols = (b, a) if tall else (a, b)
    few = torch.randn((7, rows, cols), generator=torch.Generator().manual_seed(n + rows))
    g = few.cuda()[torch.arange(n, device="cuda") % 7]
    y = torch.full(g.shape, math.nan, dtype=BF16, device="cuda")
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(n, rows, cols), dtype=torch.uint8, device="cuda")
    moe.moe_orthogonalize(n, rows, cols, moe.MOE_F32, g, 5, MUON * 5, 1e-7, 1.0, y, ws)
    for i in range(7):
        check(y[i], *exact(few[i]))
        assert torch.equal(y[i::7], y[i].expand_as(y[i::7]))
