"""The rotary angle's integer arithmetic, compiled for the host with the checks for undefined behaviour (CPU only)."""
import os
import random
import shutil
import subprocess

import pytest

import hadamard_incoherence_transforms_b200 as hit

CSRC = os.path.join(os.path.dirname(hit.__file__), "csrc")
MAIN = r"""
#include "kv_turn.h"
#include <cstdio>
int main() {
  int pos;
  unsigned long long turn;
  while (std::scanf("%d %llu", &pos, &turn) == 2) std::printf("%d\n", hit::kv_fraction(pos, turn));
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_fraction_of_a_turn_wraps_without_undefined_behaviour(tmp_path):
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "fraction")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                    str(tmp_path / "main.cpp"), "-o", exe], check=True)
    r = random.Random(7)
    edge = [0, 1, -1, 2, 100, 2 ** 31 - 1, -2 ** 31, 123456789]
    turns = [0, 1, 2 ** 32 - 1, 2 ** 32, 2 ** 63 - 1, 2 ** 63, 2 ** 64 - 1, int(2 ** 64 / 6.283185307179586)]
    cases = [(p, t) for p in edge for t in turns]
    cases += [(r.randrange(-2 ** 31, 2 ** 31), r.getrandbits(64)) for _ in range(2000)]
    done = subprocess.run([exe], input="\n".join(f"{p} {t}" for p, t in cases), capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    want = [((p * t % 2 ** 64 >> 32) + 2 ** 31) % 2 ** 32 - 2 ** 31 for p, t in cases]
    assert [int(x) for x in done.stdout.split()] == want


def test_angles_use_it():
    """Every product of a position and a frequency's fraction goes through it."""
    text = open(os.path.join(CSRC, "kv.cuh")).read()
    assert text.count("kv_fraction(pos, turn)") == 1 and "int64_t(turn)" not in text
