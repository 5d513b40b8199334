"""The deal of attention work on the host: its closed sums against sums term by term.  The numbers
come from the kernels' own header, compiled into a small program."""
import os
import subprocess

import pytest

from lossless_kv_compressed_b200.csrc import build

PROGRAM = r"""
#include <cstdio>
#include <random>
#include "paged.cuh"
using namespace vc::paged;

static int bad = 0;
static void check(bool ok, const char* what, long long a, long long b, long long c, long long d) {
  if (!ok && ++bad < 10) printf("%s: %lld %lld %lld %lld\n", what, a, b, c, d);
}

template <int RG, int KT>
static void deal(std::mt19937_64& r, int n) {
  for (int t = 0; t < n; ++t) {
    Deal<RG, KT> d = {};
    d.g = 1 + r() % (t % 3 ? 8 : 300);
    d.Hkv = 1;
    d.rows_upto = INT32_MAX;
    SeqLen q = {0, (int)(r() % (t % 2 ? 40 : 3000)), (int)(r() % (t % 5 ? 5000 : 60))};
    int64_t sum = 0;
    const int ng = d.groups(q);
    for (int rg = 0; rg <= ng; ++rg) {
      check(d.tiles_before(q, rg) == sum, "tiles_before", q.nq, q.len, d.g, rg);
      if (rg < ng) sum += d.tiles(q, rg);
    }
  }
}

int main() {
  std::mt19937_64 r(1);
  for (int t = 0; t < 200000; ++t) {
    const int64_t n = r() % 40, m = 1 + r() % 70, a = r() % 200, b = r() % 200;
    int64_t want = 0;
    for (int64_t i = 0; i < n; ++i) want += (a * i + b) / m;
    check(floor_sum(n, m, a, b) == want, "floor_sum", n, m, a, b);
  }
  for (int t = 0; t < 300; ++t) {                 // lengths up to 2^31, groups of any size
    const int64_t n = 1 + r() % 200000, m = 1 + r() % 40000, a = t % 2 ? 256 : 1 + r() % 100000;
    const int64_t b = (int64_t)(r() % ((1ull << 31) * 64));
    int64_t want = 0;
    for (int64_t i = 0; i < n; ++i) want += (a * i + b) / m;
    check(floor_sum(n, m, a, b) == want, "floor_sum", n, m, a, b);
  }
  check(floor_sum(0, 5, 3, 2) == 0 && floor_sum(7, 1, 0, 0) == 0 && floor_sum(1, 9, 8, 8) == 0,
        "floor_sum edges", 0, 0, 0, 0);
  deal<16, 16>(r, 3000);
  deal<16, 64>(r, 3000);
  deal<256, 64>(r, 3000);
  for (int t = 0; t < 20000; ++t) {
    const int64_t total = 1 + r() % 5000, W = 1 + r() % total;
    const Shares s(total, W);
    check(s.first(0) == 0 && s.first(W) == total, "shares", total, W, 0, 0);
    for (int k = 0; k < 5; ++k) {
      const int64_t p = r() % total, w = s.owner(p);
      check(w >= 0 && w < W && s.first(w) <= p && p < s.first(w + 1), "owner", total, W, p, w);
    }
  }
  printf("%d\n", bad);
  return bad != 0;
}
"""


def test_closed_sums_of_the_deal(tmp_path):
    try:
        nvcc = build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    src, exe = tmp_path / "deal.cu", tmp_path / "deal"
    src.write_text(PROGRAM)
    subprocess.run([nvcc, *build.ARCH, "-O2", "-std=c++17", "-I", build.INCLUDE, "-I", build.HERE,
                    str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True,
                       env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}, timeout=300)
    assert r.returncode == 0, r.stdout
