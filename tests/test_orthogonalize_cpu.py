"""The measure that the update's precision is tested by sees every single mistake in the pairs' arithmetic."""
import pytest

torch = pytest.importorskip("torch")
from _orth_pairs import MISTAKES, PRECISE, allowed, exact, matrices, mean_of, pairs  # noqa: E402
from test_product_cpu import ask  # noqa: E402,F401


def off(g, want, mistake=None):
    x = pairs(g, mistake=mistake)
    return float((mean_of(lambda s: (x * s).to(torch.bfloat16)) - want).norm())


@pytest.mark.parametrize("size", [s for s in PRECISE if s[1] * s[2] <= 200 * 512], ids=lambda s: "%dx%dx%d_%d" % s)
def test_mistakes_are_seen(size):
    """Those of a product's terms at full rank, those of X's last bits where directions are missing."""
    g = matrices(*size)[0]
    want = exact(g)
    most = allowed(g, want)
    assert off(g, want) <= most
    for mistake in (["last part of X", "lo of a X", "bf16 throughout"] if size[3] else MISTAKES[:-1]):
        got = off(g, want, mistake)
        assert got > 1.3 * most, (mistake, got, most)


def test_sizes_reach_every_tile(ask):
    got = {"square": set(), "wide": set(), "tall": set()}
    for n, rows, cols, _ in PRECISE:
        a, b = (-(-v // 32) * 32 for v in sorted((rows, cols)))
        got["square"] |= set(ask([("o", n, a, a, 1)]))
        got["tall" if rows > cols else "wide"] |= set(ask([("o", n, b, a, 0)]))
    assert got["square"] == got["wide"] == got["tall"] == {0, 1, 2, 3}


def test_a_result_over_its_input_is_refused():
    """y holds a part of X between the steps: it may be g itself in bf16 and share nothing else with it."""
    import ctypes

    import mixture_experts_layer_35_amd as moe
    lib, at = moe.lib(), 1 << 20
    c = (ctypes.c_float * 3)(1.5, -0.5, 0.0)

    def call(dt, g, y):
        return lib.moe_orthogonalize(2, 40, 50, dt, g, 1, ctypes.cast(c, ctypes.c_void_p), 1e-7, 1.0, y, 1 << 30, 1 << 28, None)

    for dt, size in ((moe.MOE_F32, 4), (moe.MOE_BF16, 2)):
        for y in (at + 2, at - 2, at + 4000 * size - 2, at - 4000 * 2 + 2) + ((at,) if dt == moe.MOE_F32 else ()):
            assert call(dt, at, y) == moe.MOE_ERR_INVALID_ARG and "overlaps" in moe.moe_last_error(), (dt, y - at)
