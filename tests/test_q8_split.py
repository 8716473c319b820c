"""Where the split attention kernel finds its work, on the CPU: the header
online_rank_kv_b200/csrc/q8_split.h is plain C++ and compiled here with the host
compiler; the answers are checked against Python's whole numbers."""

import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "online_rank_kv_b200", "csrc")

DRIVER = r"""
#include <cstdio>
#include "q8_split.h"
int main() {
    long long off; int tiles, steps;
    while (std::scanf("%lld %d %d", &off, &tiles, &steps) == 3) {
        const iskv::q8::StepPlace s = iskv::q8::place_of_step(off, tiles, steps);
        std::printf("%d %d %d\n", s.h, s.tile, s.step);
    }
}
"""


def _places(tmp_path, cases):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, exe = tmp_path / "split.cpp", tmp_path / "split"
    src.write_text(DRIVER)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], input="".join(f"{o} {t} {s}\n" for o, t, s in cases), capture_output=True, text=True,
                         check=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


# (row tiles, 32-token steps) of a request and KV heads: small ones, and ones
# whose steps of a head pass 2^31 (fp32 prompts on long requests; bf16 ones whose
# caller gave too small a largest number of queries) and 2^32
SHAPES = [(1, 1, 3), (5, 7, 4), (150, 40, 8), (185500, 11594, 2), (68500, 31250, 8), (262144, 8192, 1),
          (270000, 8438, 2), (2 ** 20, 2 ** 15, 4)]


@pytest.mark.parametrize("tiles,steps,heads", SHAPES)
def test_a_step_lies_in_its_head_and_tile(tiles, steps, heads, tmp_path):
    per, rng = tiles * steps, np.random.default_rng(tiles)
    offs = [0, steps - 1, steps, per - 1, per * heads - 1, per * (heads - 1), 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5]
    offs += [int(x) for x in rng.integers(0, per * heads, 200)]
    offs = [o for o in offs if o < per * heads]
    got = _places(tmp_path, [(o, tiles, steps) for o in offs])
    assert got == [(o // per, o % per // steps, o % steps) for o in offs]
