"""Rows of an expert counted in tiles and steps, up to the largest batch that the products take (fewer than 2^31 rows)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SOURCE = """
#include <cstdio>
#include "parts.h"
int main() {
    const int units[] = {1, 8, 16, 32, 64, 128, 160, 256}, top = 2147483647;
    for (int unit : units)
        for (int i = -300; i <= 600; ++i) {
            const int n = i <= 300 ? i : top - (600 - i);
            const long long want = n <= 0 ? 0 : ((long long)n + unit - 1) / unit;
            if (moe::parts_of(n, unit) != want) return std::printf("%d by %d\\n", n, unit), 1;
        }
    return 0;
}
"""


def test_parts_of_counts_below_2_31(tmp_path):
    (tmp_path / "ask.cpp").write_text(SOURCE)
    csrc = os.path.join(ROOT, "mixture_experts_layer_35_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", csrc,
                    str(tmp_path / "ask.cpp"), "-o", str(tmp_path / "ask")], check=True)
    run = subprocess.run([str(tmp_path / "ask")], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr

