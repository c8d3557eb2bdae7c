"""moe_orthogonalize's error before the rounding of its result, against the arithmetic it is meant to have."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
from _orth_pairs import MUON, PRECISE, SCALES, allowed, exact, matrices  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_35_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


@pytest.mark.parametrize("size", PRECISE, ids=lambda s: "%dx%dx%d_%d" % s)
def test_error_is_that_of_the_pairs(moe, size):
    n, rows, cols, _ = size
    g = matrices(*size)
    gd, y = g.cuda(), torch.empty((n, rows, cols), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(n, rows, cols), dtype=torch.uint8, device="cuda")
    mean = torch.zeros((n, rows, cols), dtype=torch.float64, device="cuda")
    for s in SCALES:
        moe.moe_orthogonalize(n, rows, cols, moe.MOE_F32, gd, 5, MUON * 5, 1e-7, s, y, ws)
        mean += y.double() / s
    mean = mean.cpu() / len(SCALES)
    for i in {0, n - 1}:
        want = exact(g[i])
        got, most = float((mean[i] - want).norm()), allowed(g[i], want)
        print("%s matrix %d: %.2e of %.2e" % (size, i, got / float(want.norm()), most / float(want.norm())))
        assert got <= most


@pytest.mark.parametrize("n,rows,cols", [(3, 96, 200), (3, 200, 96), (2, 131, 67), (2, 67, 131), (1, 1, 9), (70, 300, 130)])
def test_in_place(moe, n, rows, cols):
    """y is g: the same bits as elsewhere, whichever side is longer."""
    g = matrices(n, rows, cols, 0).to(torch.bfloat16).cuda()
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(n, rows, cols), dtype=torch.uint8, device="cuda")
    y = torch.full_like(g, float("nan"))
    for out in (y, g):
        moe.moe_orthogonalize(n, rows, cols, moe.MOE_BF16, g, 5, MUON * 5, 1e-7, 1.0, out, ws)
    assert torch.equal(y, g) and y.isfinite().all()


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 2), (2, 1), (1, 3), (3, 2), (3, 3), (3, 4), (4, 3), (4, 4), (4, 5), (1, 5), (2, 35)])
def test_few_values(moe, rows, cols):
    """Rows of fewer values than a load takes, and just as many; nothing behind the last one is written."""
    from test_gpu_orthogonalize import check, exact as bounds
    n = 5
    g = torch.randn((n, rows, cols), generator=torch.Generator().manual_seed(7 * rows + cols))
    out = torch.full((n * rows * cols + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(n, rows, cols), dtype=torch.uint8, device="cuda")
    y = out[1:1 + n * rows * cols].view(n, rows, cols)
    moe.moe_orthogonalize(n, rows, cols, moe.MOE_F32, g.cuda(), 5, MUON * 5, 1e-7, 1.0, y, ws)
    for i in range(n):
        check(y[i], *bounds(g[i]))
    assert out[0] == 7 and (out[1 + n * rows * cols:] == 7).all()


@pytest.mark.parametrize("rows,cols", [(300, 130), (130, 300)], ids=["tall", "wide"])
@pytest.mark.parametrize("coeffs", [MUON * 4 + (100.0, -120.0, 21.0), (100.0, -120.0, 21.0) + (0.1, 0.2, 0.1), MUON, (65.0, 0.0, 0.0)],
                         ids=["last", "first", "one", "only"])
def test_steps_that_grow_differently(moe, rows, cols, coeffs):
    """The last step takes all bits of X too where it multiplies by much, or a step in the middle does not: in place and elsewhere
    the same bits, and the formula's values."""
    from test_gpu_orthogonalize import check, exact as bounds
    g = matrices(20, rows, cols, 0).to(torch.bfloat16)
    gd = g.cuda()
    ws = torch.empty(moe.moe_orthogonalize_workspace_bytes(20, rows, cols), dtype=torch.uint8, device="cuda")
    y = torch.full_like(gd, float("nan"))
    for out in (y, gd):
        moe.moe_orthogonalize(20, rows, cols, moe.MOE_BF16, gd, len(coeffs) // 3, coeffs, 1e-7, 1.0, out, ws)
    assert torch.equal(y, gd)
    for i in (0, 19):
        check(y[i], *bounds(g[i], coeffs))
