"""MX4 rounding, its inverse, and the experts on MX4 operands against the definition in 64 bits."""
import math

import pytest

import _definitions as ref

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_35_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


def code(moe, dtype):
    return moe.MOE_BF16 if dtype == torch.bfloat16 else moe.MOE_F32


def quantize(moe, x, ld=None):
    rows, cols = x.shape
    R = ref.runs(cols)
    q = torch.full((rows, 64 * R), 0xEE, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, 4 * R), 0xEE, dtype=torch.uint8, device="cuda")
    moe.moe_quantize_mx4(rows, cols, code(moe, x.dtype), x, ld or x.stride(0), q, s)
    return q, s


def samples(rows, cols, dtype):
    """Rows of many magnitudes, with exact rounding ties, zeros, and the ends of the range among them."""
    torch.manual_seed(rows * 1000 + cols)
    x = torch.randn(rows, cols) * torch.exp2(torch.randint(-60, 60, (rows, 1)).float())
    if rows > 6:
        x[0] = 0.0
        x[1] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -5.0, 6.0, 0.0]).repeat(-(-cols // 12))[:cols]
        x[2] = torch.randn(cols) * 2.0 ** -130                        # subnormal
        x[3] = torch.randn(cols).sign() * torch.finfo(dtype).max
        x[4] = x[4].sign() * 2.0 ** -126
        x[5, ::2] = 0.0
        x[5, 1::3] = -0.0
    return x.to(dtype)


@pytest.mark.parametrize("rows,cols", [(1, 1), (9, 31), (9, 32), (9, 33), (40, 100), (33, 128), (17, 129), (8, 257),
                                       (5, 1000), (130, 384), (3, 7168)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1), (8, 8)])
def test_rounding_and_back(moe, rows, cols, dtype, pad, offset):
    x = samples(rows, cols, dtype)
    flat = torch.full((offset + rows * (cols + pad),), math.nan, dtype=dtype, device="cuda")
    view = flat[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    q, s = quantize(moe, view, cols + pad)
    rq, rs, _ = ref.quantize(x.double())
    assert (s.cpu() == rs).all()
    assert (q.cpu() == rq).all()
    want = ref.values(rq, rs, cols)
    for ydt in (torch.float32, torch.bfloat16):
        wide = torch.full((offset + rows * (cols + pad),), 5.0, dtype=ydt, device="cuda")
        y = wide[offset:].view(rows, cols + pad)[:, :cols]
        moe.moe_dequantize_mx4(rows, cols, q, s, code(moe, ydt), y, cols + pad)
        assert (y.double().cpu() == want).all()
        if pad:
            assert (wide[offset:].view(rows, cols + pad)[:, cols:] == 5.0).all()


def test_infinities_and_nan_mark_their_block(moe):
    x = torch.randn(4, 256)
    x[0, 5], x[1, 40], x[2, 255] = math.inf, -math.inf, math.nan
    q, s = quantize(moe, x.cuda())
    rq, rs, _ = ref.quantize(x.double())
    assert (s.cpu() == rs).all() and (q.cpu() == rq).all()
    y = torch.empty(4, 256, device="cuda")
    moe.moe_dequantize_mx4(4, 256, q, s, moe.MOE_F32, y, 256)
    bad = y.isnan().cpu().view(4, 8, 32)
    want = torch.zeros(4, 8, dtype=torch.bool)
    want[0, 0] = want[1, 1] = want[2, 7] = True
    assert (bad == want[:, :, None]).all()


def test_every_code_and_scale(moe):
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)[:, :, None].expand(256, 256, 64).reshape(256, -1)
    scales = torch.arange(256, dtype=torch.uint8)[:, None].expand(256, 256 * 4).contiguous()
    cols = 256 * 128
    for dt in (torch.float32, torch.bfloat16):
        y = torch.empty(256, cols, dtype=dt, device="cuda")
        moe.moe_dequantize_mx4(256, cols, codes.cuda(), scales.cuda(), code(moe, dt), y, cols)
        want = ref.values(codes, scales, cols)
        # 2^127 times 3, 4 and 6 lies past the largest number of both types
        want = torch.where(want.abs() >= 2.0 ** 128, want.sign() * math.inf, want)
        got = y.double().cpu()
        assert ((got == want) | (got.isnan() & want.isnan())).all()


# ---- experts --------------------------------------------------------------------------

def weights(n, out, k, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(n * out, k, generator=g, dtype=torch.float64) * k ** -0.5
    q, s, _ = ref.quantize(w)
    return q, s, ref.values(q, s, k).view(n, out, k)


def ffn(moe, counts, d, inter, x, gather, w, stream=None, max_rows=None):
    n = len(counts)
    rows = sum(counts)
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    xq, xs, _ = ref.quantize(x)
    cap = max_rows or rows
    y = torch.full((cap, d), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((moe.moe_ffn_mx4_workspace_bytes(cap, inter),), 0xFF, dtype=torch.uint8, device="cuda")
    args = [t.cuda() for t in (xq, xs)]
    wq, wsc = [q.cuda() for q, _, _ in w], [s.cuda() for _, s, _ in w]
    moe.moe_grouped_ffn_mx4(n, off, cap, None if gather is None else gather.to(torch.int32).cuda(), d, inter, *args, wq,
                            wsc, y, ws, stream)
    torch.cuda.synchronize()
    return y, ref.values(xq, xs, d)


def check(y, counts, d, inter, x, gather, w):
    """y against the definition.  A code of H rounds to its neighbour where fp32 and 64 bits lie on different sides of
    a midpoint: rows with a value within 1e-4 of a midpoint, in units of its block's scale (a block's values are
    sums of up to d products, each of fp32 precision: under 1e-5 of the block's largest value, which is below 8),
    are left out; those are few.  Else a result is fp32 sums of exact products (2^-20 of the sum of magnitudes) and
    one rounding to bf16 (2^-9 of itself)."""
    got = y.double().cpu()
    lo, used, total = 0, 0, 0
    for e, m in enumerate(counts):
        if m == 0:
            continue
        r = torch.arange(lo, lo + m)
        u = x[gather[r]] if gather is not None else x[r]
        a, b = u @ w[0][2][e].t(), u @ w[1][2][e].t()
        hq, hs, near = ref.quantize(a / (1 + torch.exp(-a)) * b)
        h = ref.values(hq, hs, inter)
        want = h @ w[2][2][e].t()
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * (h.abs() @ w[2][2][e].t().abs())
        clear = (near > 1e-4).all(1)
        err = (got[lo:lo + m] - want).abs()
        assert (err[clear] <= tol[clear]).all(), (e, float((err[clear] / tol[clear]).max()))
        # a neighbouring code moves a result by a third of the block's largest value times a weight, at most
        assert (err <= tol + h.abs().max() * w[2][2][e].abs().max()).all()
        used, total, lo = used + int(clear.sum()), total + m, lo + m
    assert total == 0 or used >= 0.3 * total or total < 8
    assert (got[lo:] == 7.0).all(), "rows past the last expert's are not written"


SHAPES = [
    # rows of each expert, d, inter
    ([1], 128, 128),
    ([1], 7168, 64),
    ([3, 0, 5, 1], 256, 128),
    ([0, 0, 0, 7], 100, 33),
    ([16, 17, 1, 15], 384, 96),
    ([33, 0, 64, 2, 31], 1000, 360),
    ([65, 1, 0, 129], 256, 160),
    ([300], 512, 256),
    ([257, 3, 130, 0], 130, 97),
    ([2, 600, 0, 9], 640, 224),
    ([1] * 70, 128, 32),
    ([5] * 40 + [0] * 30, 96, 31),
    ([4, 3], 31, 1),
    ([4, 40], 1, 5),
    # scales in pieces of two segments: waves sharing a tile, waves by themselves, tiles of up to 128 and 160 tokens
    ([1, 0, 16, 2], 1024, 512),
    ([2] * 40, 512, 512),
    ([17, 1, 0, 40, 33], 1024, 512),
    ([3, 500, 129, 2], 512, 512),
    ([120, 140, 160, 129, 161, 31], 512, 512),
    # the same kernels with scales by words
    ([1] * 60, 384, 640),
    ([150, 97], 130, 97),
    ([150, 128, 159, 1, 260], 384, 640),
    # enough tiles for the kernel of whole workgroups: of up to 128 tokens, and (averages of 130) of up to 160
    ([40] * 40, 1024, 1024),
    ([33, 1, 0, 64, 500, 129] * 4, 700, 700),
    ([97, 161, 130, 132, 159, 160, 1, 200] * 2, 2304, 2048),
    ([128, 130, 129, 131, 150, 96, 192, 84] * 2, 2300, 2100),
]


@pytest.mark.parametrize("counts,d,inter", SHAPES, ids=lambda v: str(v)[:24])
@pytest.mark.parametrize("gathered", [True, False])
def test_experts_against_the_definition(moe, counts, d, inter, gathered):
    rows = sum(counts)
    torch.manual_seed(rows + d)
    T = max(1, rows // 2) if gathered else rows
    x = torch.randn(T, d, dtype=torch.float64)
    gather = torch.randint(0, T, (rows,)) if gathered else None
    n = len(counts)
    w = [weights(n, inter, d, 1), weights(n, inter, d, 2), weights(n, d, inter, 3)]
    print("ffn", counts[:8], d, inter, gathered, flush=True)
    y, xv = ffn(moe, counts, d, inter, x, gather, w, max_rows=rows + 3)
    check(y, counts, d, inter, xv, gather, w)


def test_no_rows(moe):
    w = [weights(2, 32, 128, 1), weights(2, 32, 128, 2), weights(2, 128, 32, 3)]
    y, _ = ffn(moe, [0, 0], 128, 32, torch.randn(1, 128, dtype=torch.float64), torch.zeros(0).long(), w, max_rows=4)
    assert (y == 7.0).all()
    assert moe.moe_grouped_ffn_mx4(2, 0, 0, None, 128, 32, 0, 0, None, None, 0, None) == 0


def test_same_bits_each_time(moe):
    counts, d, inter = [40, 0, 3, 90], 512, 192
    torch.manual_seed(9)
    x = torch.randn(133, d, dtype=torch.float64)
    w = [weights(4, inter, d, 1), weights(4, inter, d, 2), weights(4, d, inter, 3)]
    a, _ = ffn(moe, counts, d, inter, x, None, w)
    b, _ = ffn(moe, counts, d, inter, x, None, w)
    assert (a == b).all()


def test_weights_past_4_gib(moe):
    n, d, inter = 1024, 7168, 1280                # 4.7 GB of codes a matrix
    rows = 20
    q = [torch.zeros((n, inter, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    q.append(torch.zeros((n, d, inter // 2), dtype=torch.uint8, device="cuda"))
    s = [torch.full((t.shape[0], t.shape[1], t.shape[2] // 16), 127, dtype=torch.uint8, device="cuda") for t in q]
    q[0][n - 1, :, 0] = 0x02                      # gate: 1 at column 0; up: 2 there; down: 1 at columns 0 and 1
    q[1][n - 1, :, 0] = 0x04
    q[2][n - 1, :, 0] = 0x22
    x = torch.zeros((rows, d))
    x[:, 0] = torch.tensor([0.5, 1, 2, 3, 4] * 4)
    xq, xs = quantize(moe, x.cuda())
    off = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    off[n] = rows
    y = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_ffn_mx4_workspace_bytes(rows, inter), dtype=torch.uint8, device="cuda")
    moe.moe_grouped_ffn_mx4(n, off, rows, None, d, inter, xq, xs, q, s, y, ws)
    v = x[:, 0].double()
    hq, hs, _ = ref.quantize((v / (1 + torch.exp(-v)) * 2 * v)[:, None])
    want = 2 * ref.values(hq, hs, 1)
    assert (y.double().cpu() == want.expand(rows, d)).all()


def test_rows_past_4_gib(moe):
    rows, cols = 700_001, 4096
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    x[rows - 1] = torch.randn(cols, device="cuda").to(torch.bfloat16)
    q, s = quantize(moe, x)
    rq, rs, _ = ref.quantize(x[rows - 1:].double().cpu())
    assert (q[rows - 1:].cpu() == rq).all() and (s[rows - 1:].cpu() == rs).all()
    assert int(q[: rows - 1].max()) == 0 and int(s[: rows - 1].min()) == 127
    x.fill_(9.0)
    moe.moe_dequantize_mx4(rows, cols, q, s, moe.MOE_BF16, x, cols)
    assert (x[rows - 1].double().cpu() == ref.values(rq, rs, cols)[0]).all() and float(x[: rows - 1].abs().max()) == 0.0


def test_streams_and_graph_replays(moe):
    counts, d, inter = [9, 0, 40, 3], 384, 160
    rows = sum(counts)
    torch.manual_seed(2)
    w = [weights(4, inter, d, 1), weights(4, inter, d, 2), weights(4, d, inter, 3)]
    wq, wsc = [q.cuda() for q, _, _ in w], [s.cuda() for _, s, _ in w]
    off = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()
    x = torch.randn(rows, d, device="cuda").to(torch.bfloat16)
    xq, xs = quantize(moe, x)
    y = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_ffn_mx4_workspace_bytes(rows, inter), dtype=torch.uint8, device="cuda")

    def both(stream):
        moe.moe_quantize_mx4(rows, d, moe.MOE_BF16, x, d, xq, xs, stream)
        moe.moe_grouped_ffn_mx4(4, off, rows, None, d, inter, xq, xs, wq, wsc, y, ws, stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both(side)
    for k in range(4):
        x.copy_(torch.randn(rows, d, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.zero_()
        both(None)
        torch.cuda.synchronize()
        assert (got == y).all()
