"""Which kernel a call takes is decided by csrc/variants.h from sizes alone: the sizes that the GPU tests use reach every
variant, so that a change of a threshold that leaves one without a test shows here."""
import os
import subprocess

import pytest

pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUS = 256
SOURCE = """
#include <cstdio>
#include "variants.h"
int main() {
    long long a, b, c, d;
    char what;
    while (std::scanf(" %c %lld %lld %lld %lld", &what, &a, &b, &c, &d) == 5) {
        if (what == 'm') std::printf("%d\\n", (int)moe::mx4_variant(a, b, c, d, CUS));
        else { const moe::GateWidth w = moe::gate_width(a, (int)b, CUS); std::printf("%d %d\\n", w.lanes, w.values); }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("variants")
    (d / "ask.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "mixture_experts_layer_35_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-DCUS=%d" % CUS, "-I", csrc, str(d / "ask.cpp"), "-o", str(d / "ask")],
                   check=True)

    def lines(queries):
        text = "".join("%s %d %d %d %d\n" % q for q in queries)
        out = subprocess.run([str(d / "ask")], input=text, capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
        assert len(out) == len(queries)
        return [tuple(map(int, line.split())) for line in out]

    return lines


def runs(cols):
    return -(-cols // 128)


def test_gpu_tests_reach_every_expert_kernel(ask):
    from test_gpu_mx4 import SHAPES
    from test_gpu_mx4_variants import VARIANTS
    asked = []
    for counts, d, inter in SHAPES + VARIANTS:
        rows = sum(counts) + 3                              # as those tests call it
        for up, kruns, ftiles in ((True, runs(d), runs(inter) * 4), (False, runs(inter), -(-d // 64))):
            asked.append((up, kruns, ("m", rows, len(counts), kruns, ftiles)))
    variants = ask([q for _, _, q in asked])
    reached = {(up, v, "pieces" if k % 4 == 0 else "odd" if k % 2 else "even") for (up, k, _), (v,) in zip(asked, variants)}
    missing = {(up, v, s) for up in (True, False) for v in range(4) for s in ("pieces", "odd", "even")} - reached
    assert not missing, missing


def test_gpu_tests_reach_every_width_of_the_gate(ask):
    from test_gpu_gate_widths import WIDTHS
    widths = set(ask([("g", c[0], c[1], 0, 0) for c in WIDTHS]))
    sizes = [(T, E) for T in (1, 100, 1000, 10000, 100000) for E in range(1, 1025)]
    every = ask([("g", T, E, 0, 0) for T, E in sizes])
    assert all(lanes * values >= E for (lanes, values), (_, E) in zip(every, sizes))
    assert set(every) == widths and len(widths) == 10


def test_expert_kernels_of_known_sizes(ask):
    """256 experts of 7168 x 2048 at 1, 128 and 4096 tokens of 8 experts each, 32 of them at 512 rows each."""
    up, down = (56, 64), (16, 112)
    queries = [("m", rows, n, k, f) for rows, n in ((8, 256), (1024, 256), (32768, 256), (16384, 32)) for k, f in (up, down)]
    assert [v for (v,) in ask(queries)] == [0, 1, 2, 2, 3, 3, 3, 3]
