"""GPU test of the sampler's rough weights: the GPU's exponential and fused products, within the bounds that its decisions rest on."""
import subprocess

import pytest

from gpu_util import require_gpu
from lossless_depth_adaptive_gb300 import build

pytestmark = pytest.mark.gpu

PROGRAM = r"""
#include <math.h>
#include <stdio.h>
#include <random>
#include <vector>
#include "sample_weight.h"
using namespace dex;

__global__ void weights(const float* x, const float* top, const float* t, int n, float* near, unsigned long long* whole) {
  __shared__ Pair table[kWeightTable];
  if (threadIdx.x < kWeightTable) table[threadIdx.x] = pair_of(weight_table_entry(threadIdx.x));
  __syncthreads();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= n) return;
  const Pair c = octaves_per_unit(t[i]);
  near[i] = weight_near(x[i], top[i], c, -128.0f / c.hi);
  whole[i] = weight_of(x[i], top[i], c, table);
}

int main() {
  const int n = 1 << 22;
  std::mt19937_64 gen(5);
  auto uniform = [&](double lo, double hi) { return std::uniform_real_distribution<double>(lo, hi)(gen); };
  std::vector<float> x(n), top(n), t(n), near(n);
  std::vector<unsigned long long> whole(n);
  for (int i = 0; i < n; i += 4) {   // four tokens of a row
    const float T = static_cast<float>(exp(uniform(-4, 4))), peak = static_cast<float>(uniform(-60, 60));
    const double reach = i % 8 ? uniform(0, 31) : uniform(0, 1) * exp2(uniform(-14, 5));
    for (int k = 0; k < 4; ++k) {
      t[i + k] = T;
      top[i + k] = peak;
      x[i + k] = peak - static_cast<float>(uniform(0.8, 1) * reach * T);
    }
  }
  float *dx, *dtop, *dt, *dnear;
  unsigned long long* dwhole;
  bool ok = cudaMalloc(&dx, n * 4) == cudaSuccess && cudaMalloc(&dtop, n * 4) == cudaSuccess && cudaMalloc(&dt, n * 4) == cudaSuccess &&
            cudaMalloc(&dnear, n * 4) == cudaSuccess && cudaMalloc(&dwhole, n * 8) == cudaSuccess;
  ok = ok && cudaMemcpy(dx, x.data(), n * 4, cudaMemcpyHostToDevice) == cudaSuccess;
  ok = ok && cudaMemcpy(dtop, top.data(), n * 4, cudaMemcpyHostToDevice) == cudaSuccess;
  ok = ok && cudaMemcpy(dt, t.data(), n * 4, cudaMemcpyHostToDevice) == cudaSuccess;
  if (!ok) return 2;
  weights<<<n / 256, 256>>>(dx, dtop, dt, n, dnear, dwhole);
  ok = cudaGetLastError() == cudaSuccess && cudaMemcpy(near.data(), dnear, n * 4, cudaMemcpyDeviceToHost) == cudaSuccess;
  ok = ok && cudaMemcpy(whole.data(), dwhole, n * 8, cudaMemcpyDeviceToHost) == cudaSuccess;
  if (!ok) return 2;
  double one = 0, four = 0, units = 0;
  int bad = 0;
  for (int i = 0; i < n; i += 4) {
    double sum = 0, deepest = 0;
    float some = 0;
    for (int k = i; k < i + 4; ++k) {
      const double y = (static_cast<double>(x[k]) - top[k]) / t[k] * 1.4426950408889634, w = exp2(y);
      units = fmax(units, fabs(whole[k] - ldexp(w, kWeightBits)));
      if (y < -45) continue;
      one = fmax(one, fabs(near[k] / w - 1) / (0x1.4001p-22 + 0x1p-24 * 0.69314719 * fabs(y)));
      some += near[k];
      sum += w;
      deepest = fmax(deepest, -y);
      bad += in_units(near[k]) != static_cast<uint64_t>(ldexp(near[k], kWeightBits));
    }
    if (deepest > 0 && deepest < 20)   // (further down single units count, which slack has apart)
      four = fmax(four, fabs(some - sum) / ldexp(static_cast<double>(rough_slack(static_cast<uint64_t>(ldexp(sum, kWeightBits)), static_cast<float>(deepest)) - (uint64_t(1) << 20)), -kWeightBits));
  }
  printf("one %.4f four %.4f of the bounds, units %.3f bad %d\n", one, four, units, bad);
  return one > 1 || four > 1 || units > 2 || bad;
}
"""


def test_rough_weights_on_the_gpu(tmp_path):
    """Each within 2^-22 (the exponential's bound) + 2^-24 (a rounding) + 2^-24 |y| ln 2 (the difference) of itself, sums of four as floats within
    what the sampler takes them to be worth, and whole weights within two units as on the CPU."""
    require_gpu()
    (tmp_path / "w.cu").write_text(PROGRAM)
    subprocess.run([build.NVCC, *build.ARCH, "-O3", "-std=c++17", "-o", str(tmp_path / "w"), str(tmp_path / "w.cu"), "-I", build.CSRC],
                   check=True)
    r = subprocess.run([str(tmp_path / "w")], capture_output=True, text=True, timeout=120)
    print(r.stdout)
    assert r.returncode == 0, r.stdout
