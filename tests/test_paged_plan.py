"""CPU test of the shared-prefix attention's host plan (csrc/prefix_plan.h), compiled by itself: what its kernels may
index lies within the workspace."""
import os
import subprocess

import pytest

from lossless_depth_adaptive_gb300 import build

DRIVER = r"""
#include <stdio.h>
#include <stdlib.h>
#include "prefix_plan.h"
using namespace dex;

static PrefixAttnArgs sizes(int batch, int kvh, int G, int hd, int tokens, int max_q, int prefix) {
  PrefixAttnArgs a = {};
  a.kv.batch = batch, a.kv.KVH = kvh, a.kv.hd = hd;
  a.n_tokens = tokens, a.G = G, a.H = kvh * G, a.max_q = max_q, a.prefix_len = prefix;
  return a;
}

// Entries of any value: the ranges that the join follows have their two parts within the workspace.
static int check_parts(const PrefixAttnArgs& a) {
  const Plan p = make_plan(a);
  const size_t row = static_cast<size_t>(a.kv.hd) * 4;
  const int values[] = {-2147483647 - 1, -1, 0, 1, 151, 152, 303, 304, 400, 607, 608, 2147483647};
  for (int pre = 0; pre < 2; ++pre) {
    if (pre && !p.share) continue;
    const bool tile = pre ? p.prefix_tile : p.own_tile;
    const int ranges = pre ? p.pre_ranges() : p.own_ranges(), rt = pre ? p.pre_rt() : p.own_rt();
    const size_t begin = tile ? p.o_tile_part : p.o_rows_part, end = tile ? p.o_tile_ml : p.o_rows_ml;
    for (int x : values)
      for (int y : values) {
        const int n = parts_in(x, y, ranges);
        if (n < 0 || (n > 0 && (x < 0 || x + n - 1 != y))) return printf("entry %d %d gives %d parts\n", x, y, n), 1;
        if (n > 0 && (2 * static_cast<size_t>(y) + 2) * rt * row > end - begin)
          return printf("batch %d kvh %d G %d tokens %d max_q %d prefix %d: entry %d %d is followed out of the workspace\n",
                        a.kv.batch, a.kv.KVH, a.G, a.n_tokens, a.max_q, a.prefix_len, x, y), 1;
      }
  }
  return 0;
}

int main() {
  int bad = 0, shared = 0, tiles = 0;
  for (int batch : {1, 2, 5, 14, 32, 64, 300, 1024})
    for (int kvh : {1, 2, 8, 32})
      for (int G : {1, 3, 4, 8, 40, 128})
        for (int per : {1, 2, 9, 64, 700})
          for (int prefix : {0, 64, 128, 777, 4096, 32768}) {
            const PrefixAttnArgs a = sizes(batch, kvh, G, per % 2 ? 64 : 128, batch * per, per, prefix);
            bad += check_parts(a);
            shared += make_plan(a).share, tiles += make_plan(a).own_tile;
          }
  if (!shared || !tiles) return printf("no such plan\n"), 2;
  return bad != 0;
}
"""


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(DRIVER)
    subprocess.run(["g++", "-O1", "-std=c++17", "-o", str(d / "plan"), str(d / "plan.cpp"), "-I", build.CSRC,
                    "-I", os.path.join(build.ROOT, "include"), "-I", os.path.join(build.CUDA_HOME, "include")], check=True)
    return str(d / "plan")


def test_entries_are_followed_within_the_workspace(driver):
    r = subprocess.run([driver], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout[-2000:]
