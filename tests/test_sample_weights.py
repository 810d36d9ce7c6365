"""CPU tests of the sampler's arithmetic, compiled by itself."""
import subprocess

from lossless_depth_adaptive_gb300 import build

HEAD = r"""
#include <initializer_list>
#include <math.h>
#include <stdio.h>
#include <random>
#include "sample_weight.h"
using namespace dex;
std::mt19937_64 gen(11);
double uniform(double lo, double hi) { return std::uniform_real_distribution<double>(lo, hi)(gen); }
"""

LOG_SHARE = r"""
int main() {
  long double worst = 0;
  for (int i = 0; i < 2000000; ++i) {
    const float T = static_cast<float>(exp(uniform(-4, 4))), top = static_cast<float>(uniform(-60, 60));
    const float x = top - static_cast<float>(uniform(0, 1) * exp2(uniform(-20, 5)) * T);
    const uint64_t mass = static_cast<uint64_t>(ldexp(exp2(uniform(0, 18)), kWeightBits)) + (gen() & 0xffffff);
    const long double ref = (static_cast<long double>(x) - top) / T - logl(ldexpl(mass, -kWeightBits));
    if (ref > -0.69L) continue;
    worst = fmaxl(worst, fabsl(log_share(octaves_of(x, top, octaves_per_unit(T)), mass) / ref - 1));
  }
  printf("2^%.2Lf\n", log2l(worst));
  return worst > 0x1p-22L;
}
"""


def run(tmp_path, program):
    (tmp_path / "t.cpp").write_text(HEAD + program)
    subprocess.run(["g++", "-O1", "-std=c++17", "-ffp-contract=off", "-o", str(tmp_path / "t"), str(tmp_path / "t.cpp"),
                    "-I", build.CSRC], check=True)
    r = subprocess.run([str(tmp_path / "t")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_log_share(tmp_path):
    """To 2^-22 of itself down to 46 octaves: a log good to a unit in the last place (2^-23 of it, and it is no larger than the
    result), the product's and the sum's half steps of 2^-24."""
    run(tmp_path, LOG_SHARE)
