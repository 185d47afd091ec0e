"""The paged attention's work list (csrc/page_sched.cuh), compiled from the library's own header
for the host and checked against counting the tiles one by one: tiles of a row block and tiles before
a row block."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CXX = shutil.which("g++") or shutil.which("c++")

PROGRAM = r"""
#include <cstdio>
#include "page_sched.cuh"
using namespace salsc;
int main() {
  unsigned long long x = 88172645463325252ull;  // xorshift64
  auto rnd = [&](long long n) { x ^= x << 13; x ^= x >> 7; x ^= x << 17; return (long long)(x % n); };
  for (int trial = 0; trial < 20000; ++trial) {
    const int n = (int)rnd(trial % 3 ? 700 : 40000), m = 1 + (int)rnd(trial % 2 ? 300 : 3000);
    const int tb = 1 + (int)rnd(trial % 5 ? 40 : 256);
    const int w = trial % 4 ? 0 : 1 + (int)rnd(900);
    const int over = (int)rnd(5);
    const PageBlocks p{n, m, tb, w, over};
    if (p.count() != (m + tb - 1) / tb) return 1;
    long long before = 0;
    for (int k = 0; k < p.count(); ++k) {
      // the block's rows, one by one
      int first = -1, last = -1;
      for (int i = k * tb; i < m && i < (k + 1) * tb; ++i) {
        const int pos = n - m + i;
        if (pos < 0) continue;
        const int lo = w && pos - w + 1 > 0 ? pos - w + 1 : 0;
        if (first < 0) first = lo / kPageTile;
        last = pos / kPageTile;
      }
      if (p.before(k) != before) return 2;
      if (first < 0) {  // no row sees anything: one tile
        if (p.tiles(k) != 1) return 3;
      } else {
        if (p.tile0(k) != first || p.tiles(k) != last - first + 1) return 4;
      }
      before += over + p.tiles(k);
    }
    if (p.before(p.count()) != before) return 5;
  }
  // the largest sizes: no 32-bit overflow
  const PageBlocks big{2147483647, 2147483647, 8, 0, 0};
  if (big.tiles(big.count() - 1) != 16777216) return 6;
  long long full = 0;
  for (long long k = 0; k < big.count(); ++k) {
    const long long e = (k + 1) * 8 < 2147483647ll ? (k + 1) * 8 : 2147483647ll;
    full += (e - 1) / 128 + 1;
  }
  if (big.before(big.count()) != full) return 7;
  std::printf("ok\n");
  return 0;
}
"""


@pytest.mark.skipif(CXX is None, reason="no C++ compiler")
def test_page_work_list_host_build(tmp_path):
    src = tmp_path / "sched.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "sched"
    subprocess.run([CXX, "-O2", "-std=c++17", "-I",
                    os.path.join(ROOT, "latent_space_sparse_b200", "csrc"), str(src), "-o",
                    str(exe)], check=True, capture_output=True, timeout=300)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", (r.returncode, r.stdout, r.stderr)
