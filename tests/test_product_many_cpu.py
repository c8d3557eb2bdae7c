"""The batches of _product_many.py reach every kernel with the tiles that they are meant to have."""
import pytest

pytest.importorskip("torch")
from _product_many import GRADIENTS, PRODUCTS, UPDATES, WORKGROUPS  # noqa: E402
from test_product_cpu import ask  # noqa: E402,F401


def parts(n, unit):
    return -(-n // unit)


def test_products(ask):
    got = {"y": set(), "dx": set(), "int8": set()}
    for op, counts, cin, cout, kernel in PRODUCTS:
        features, pieces = (cin if op == "dx" else cout), op == "int8" or (cin % 8 == 0 and (op == "y" or cout % 8 == 0))
        assert ask([("p", sum(counts) + 3, len(counts), features, int(pieces))]) == [kernel]
        rows, wide = {0: (128, 256), 1: (8, 64), 2: (160, 256), 3: (256, 256)}[kernel]
        tiles = sum(parts(n, rows) for n in counts) * parts(features, wide)
        # few tiles are what the streaming kernel is for: two a workgroup at most
        assert tiles > (1 if kernel == 1 else 2) * WORKGROUPS
        got[op].add(kernel)
    assert got["y"] == got["dx"] == {0, 1, 2, 3} and got["int8"] == {1, 2, 3}
    assert {cin % 8 == 0 and cout % 8 == 0 for _, cin, cout in GRADIENTS} == {True, False}
    for counts, cin, cout in GRADIENTS:
        assert len(counts) * parts(cin, 256) * parts(cout, 256) > 2 * WORKGROUPS


def test_updates(ask):
    got = {True: set(), False: set()}
    for n, a, b in UPDATES:
        a, b = 32 * parts(a, 32), 32 * parts(b, 32)
        square, update = ask([("o", n, a, a, 1), ("o", n, b, a, 0)])
        for symmetric, kernel, long in ((True, square, a), (False, update, b)):
            ta, tb = ((256, 256), (256, 128), (128, 128), (64, 64))[kernel]
            at, bt = parts(long, ta), parts(a, tb)
            tiles = n * (sum(bt - min(bt, i * ta // tb) for i in range(at)) if symmetric else at * bt)
            if tiles > 2 * WORKGROUPS:
                got[symmetric].add(kernel)
    assert got[True] == got[False] == {0, 1, 2, 3}
