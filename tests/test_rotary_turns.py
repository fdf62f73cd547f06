"""Frequencies as 64-bit fractions of a turn (csrc/lla_turns.h), compiled for the host, against 80 digits: off by half a
unit of 2^-64 turns, and by the roundings of two doubles, 2^-89 turns for the largest frequency."""
import random
import shutil
import subprocess
from decimal import Decimal, getcontext

import pytest

from test_smem_limits import CSRC

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "lla_turns.h"

int main() {
  char line[64];
  while (fgets(line, sizeof line, stdin)) printf("%llu\n", lla::rotary::turns_of(strtod(line, nullptr)));
  return 0;
}
"""
TWO_PI = "6.28318530717958647692528676655900576839433879875021164194988918461563281257241799725606965068423413596"


@pytest.mark.parametrize("flags", [["-O0"], ["-O3", "-ffp-contract=fast"]])
def test_half_a_unit(tmp_path, flags):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    getcontext().prec = 80
    src = tmp_path / "turns.cc"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", *flags, "-I", CSRC, str(src), "-o", str(tmp_path / "turns")], check=True)
    rng = random.Random(1)
    freq = [base ** (-2 * i / rot) / factor for rot in (64, 128) for base in (1e4, 5e5, 1e6) for i in range(rot // 2)
            for factor in (1.0, 8.0)]
    freq += [rng.choice((-1, 1)) * 2.0 ** rng.uniform(-60, 20) for _ in range(3000)]
    freq += [0.0, 2.0 ** 20, -2.0 ** 20, 6.283185307179586, 6.283185307179587, 5e-324, 2.0 ** -64]
    run = subprocess.run([str(tmp_path / "turns")], input="".join(f.hex() + "\n" for f in freq), capture_output=True, text=True,
                         check=True)
    got = [int(x) for x in run.stdout.split()]
    assert len(got) == len(freq)
    for f, x in zip(freq, got):
        off = (Decimal(f) / Decimal(TWO_PI) * 2 ** 64 - x) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= Decimal(0.5 + 2.0 ** -22), f
