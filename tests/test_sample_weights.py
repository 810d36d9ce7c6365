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


# (weight_near on this side takes the exponential of the C library)
ROUGH = r"""
int main() {
  long double one = 0, four = 0;
  for (int i = 0; i < 2000000; ++i) {
    const float T = static_cast<float>(exp(uniform(-4, 4))), top = static_cast<float>(uniform(-60, 60));
    const Pair c = octaves_per_unit(T);
    const double reach = uniform(0, 1) * exp2(uniform(-14, 5.5));
    long double sum = 0, deepest = 0;
    float some = 0;
    for (int k = 0; k < 4; ++k) {
      const float x = top - static_cast<float>(uniform(0.9, 1) * fmin(reach, 31.0) * T);
      const long double y = (static_cast<long double>(x) - top) / T * 1.4426950408889634073599L, w = exp2l(y);
      const float near = weight_near(x, top, c, -128.0f / c.hi);
      one = fmaxl(one, fabsl(near / w - 1) / (0x1.4001p-22L + 0x1p-24L * 0.6931472L * fabsl(y)));
      some += near;
      sum += w;
      deepest = fmaxl(deepest, -y);
    }
    // of a large sum, in which single units do not count
    const uint64_t whole = static_cast<uint64_t>(ldexpl(sum, kWeightBits));
    const long double allowed = ldexpl(static_cast<long double>(rough_slack(whole, deepest) - (uint64_t(1) << 20)), -kWeightBits);
    if (deepest < 20) four = fmaxl(four, fabsl(some - sum) / allowed);
  }
  printf("%.4Lf %.4Lf of the bounds\n", one, four);
  return one > 1 || four > 1;
}
"""


def test_rough_weights_within_their_bound(tmp_path):
    """Each to its own depth, 2^-22 + 2^-24 + 2^-24 |y| ln 2 (and a hundred-thousandth of it for what is of second order), and sums of four floats to
    what the sampler takes them to be worth."""
    run(tmp_path, ROUGH)


SLACK = r"""
int main() {
  // the units: a rounding down, two of weight_of, and half of one below which that is nothing, for each token of the longest row
  const double units = (1 + 2 + 0.5) * (1 << 18);
  int bad = rough_slack(0, 0) < units;
  for (int i = 0; i < 1000000; ++i) {
    const double sum = ldexp(exp2(uniform(0, 18)), kWeightBits);
    const float octaves = static_cast<float>(uniform(0, 45));
    bad += rough_slack(static_cast<uint64_t>(sum), octaves) < sum * (0x1p-21 + octaves * 0x1p-24 * 0.69314718) + units;
  }
  printf("%d\n", bad);
  return bad;
}
"""


def test_slack_covers_every_unit(tmp_path):
    run(tmp_path, SLACK)
