"""CPU test of the rotary frequencies (csrc/rope_angle.h), compiled by itself: 64-bit fractions against 60 digits."""
import decimal
import os
import subprocess

import pytest

from lossless_depth_adaptive_gb300 import build

DRIVER = r"""
#include <stdio.h>
#include <stdlib.h>
#include "rope_angle.h"
int main(int argc, char** argv) {
  uint64_t p[6];
  dex::rope_powers(strtof(argv[1], nullptr), atoi(argv[2]), p);
  printf("%llu", (unsigned long long)dex::kTurnPerRadian);
  for (uint64_t x : p) printf(" %llu", (unsigned long long)x);
}
"""
PI = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    d = tmp_path_factory.mktemp("rope")
    (d / "rope.cpp").write_text(DRIVER)
    subprocess.run(["g++", "-O2", "-std=c++17", "-o", str(d / "rope"), str(d / "rope.cpp"), "-I", build.CSRC], check=True)
    return str(d / "rope")


@pytest.mark.parametrize("hd", [64, 128])
def test_powers(driver, hd):
    # 24-bit values, exact in text: powers of two, next to them, the usual ones, the largest of the type
    thetas = [1.0, 1.0 + 2.0 ** -23, 2.0 - 2.0 ** -23, 2.0, 2.0 + 2.0 ** -22, 1.5, 3.0, 4.0, 10.0, 10000.0, 500000.0, 1e6, 2.0 ** 20,
              2.0 ** 63, 2.0 ** 64, 2.0 ** 65, 2.0 ** 127, (2.0 - 2.0 ** -23) * 2.0 ** 127]
    with decimal.localcontext() as ctx:
        ctx.prec = 60
        for theta in thetas:
            got = [int(x) for x in subprocess.run([driver, repr(theta), str(hd)], capture_output=True, text=True, check=True).stdout.split()]
            assert got[0] == int(decimal.Decimal(2 ** 64) / (2 * PI))
            for b in range(6):
                if 2 ** b >= hd // 2:
                    assert got[1 + b] == 0
                    continue
                want = (decimal.Decimal(-2 * 2 ** b) / hd * decimal.Decimal(theta).ln()).exp() * 2 ** 64
                assert abs(got[1 + b] - want) <= 8, (theta, b, got[1 + b], want)
