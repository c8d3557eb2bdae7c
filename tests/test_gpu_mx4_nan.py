"""Blocks of NaN (scale 255) and infinities on their way through the MX4 experts: they reach what the formula takes them
to, and nothing beside it."""
import pytest

import _definitions as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

SHAPES = [
    # rows of each expert, d, inter
    ([3, 0, 5, 1], 256, 128),
    ([4, 17, 2], 384, 160),                    # an odd number of runs
    ([2, 9], 100, 40),
    ([40] * 40, 1024, 1024),                   # whole-workgroup tiles
    ([33, 1, 0, 64, 500, 129] * 4, 700, 700),
]


def parts(n, out, k, seed):
    g = torch.Generator().manual_seed(seed)
    q, s, _ = ref.quantize(torch.randn(n * out, k, generator=g, dtype=torch.float64) * k ** -0.5)
    return [q.view(n, out, -1).cuda(), s.view(n, out, -1).cuda()]


@pytest.mark.parametrize("counts,d,inter", SHAPES, ids=lambda v: str(v)[:24])
def test_nan_blocks_reach_their_results_alone(counts, d, inter):
    import mixture_experts_layer_35_amd as moe
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    n, rows = len(counts), sum(counts)
    T = rows // 2 + 1
    torch.manual_seed(d)
    gather = torch.randint(0, T, (rows,))
    ends = torch.tensor([0] + counts).cumsum(0)
    expert = torch.repeat_interleave(torch.arange(n), torch.tensor(counts))
    w = [parts(n, inter, d, 1), parts(n, inter, d, 2), parts(n, d, inter, 3)]
    xq, xs, _ = ref.quantize(torch.randn(T, d, dtype=torch.float64))
    xq, xs, off = xq.cuda(), xs.cuda(), ends.to(torch.int32).cuda()
    gd = gather.to(torch.int32).cuda()
    ws = torch.empty(moe.moe_ffn_mx4_workspace_bytes(rows, inter), dtype=torch.uint8, device="cuda")

    def run(xs=xs, scales=None):
        y = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
        moe.moe_grouped_ffn_mx4(n, off, rows, gd, d, inter, xq, xs, [q for q, _ in w], scales or [s for _, s in w], y, ws)
        return y.float().cpu()

    clean = run()
    assert torch.isfinite(clean).all()

    def check(y, bad):
        assert (y.isnan() == bad).all(), int((y.isnan() != bad).sum())
        assert (y[~bad] == clean[~bad]).all()

    token = int(gather[rows // 2])
    for block in {0, (d - 1) // 32}:
        nan = xs.clone()
        nan[token, block] = 255
        check(run(nan), (gather == token)[:, None].expand(rows, d))
    e = int(expert[rows // 2])
    for k, f in ((0, 0), (0, inter - 1), (1, inter // 2)):     # a value of H is NaN, so its block, so all of y's row
        scales = [s for _, s in w]
        scales[k] = scales[k].clone()
        scales[k][e, f, (d - 1) // 32] = 255
        check(run(scales=scales), (expert == e)[:, None].expand(rows, d))
    for f in (0, d // 2, d - 1):
        scales = [s for _, s in w]
        scales[2] = scales[2].clone()
        scales[2][e, f, (inter - 1) // 32] = 255
        check(run(scales=scales), (expert == e)[:, None] & (torch.arange(d) == f))
    # gate and up values near 2^100 (a block's weights 2^90 and more times what they were): their product is infinite
    scales = [s for _, s in w]
    for k in (0, 1):
        scales[k] = scales[k].clone()
        scales[k][e, 5] += 100
    # a negative gate of this size gives -0 times the up value: finite, as the formula, and another H than before
    a = ref.values(xq.cpu(), xs.cpu(), d)[gather] @ ref.values(w[0][0][e, 5:6].cpu(), w[0][1][e, 5:6].cpu(), d)[0]
    y, hit = run(scales=scales), expert == e
    assert (y.isnan() == (hit & (a > 0))[:, None]).all()
    assert (y[~hit] == clean[~hit]).all()
