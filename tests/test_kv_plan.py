"""Host-side check of the prompt kernel's list of row tiles (kv_kernel.cuh,
KvTileList): every tile of the list is found in a request that has it, also where
the offsets of Q name its rows many times over, more often than 32 bits count.

The list is made of __host__ __device__ functions, so a small host program
compiled with nvcc calls the library's own code; no GPU is needed."""
import os
import subprocess

import pytest

from tests.test_raster import BUILD, CSRC, ROOT, _nvcc

HARNESS = r"""
#include <cstdio>
#include <vector>
#include "kv_kernel.cuh"

// requests of n[b] tokens each: the list as the kernel plans it, some tiles looked up
static long check(const std::vector<long long>& n, long long tokens, int group) {
  const int B = static_cast<int>(n.size()), rows = 256;
  const mxk::KvTileList list(tokens, group, rows, B);
  std::vector<int> starts(B);
  long long at = 0;
  for (int b = 0; b < B; ++b) {
    starts[b] = list.start(at);
    at += (n[b] * group + rows - 1) / rows;
  }
  const long long tiles = list.clip(at);
  long bad = 0;
  for (long long i = 0; i <= 4096 && tiles; ++i) {
    const long long f = i == 4096 ? tiles - 1 : tiles / 4096 * i + i % 7 * (tiles > 4096 * 7);
    if (f >= tiles) continue;
    int b = mxk::KvTileList::request(starts.data(), B, f);
    long long rt = f - starts[b];
    while (b < B && rt >= (n[b] * group + rows - 1) / rows) rt = 0, ++b;   // as the kernel's walk
    if (b >= B || rt < 0 || rt > 0x7FFFFFFF / rows) ++bad;
  }
  return bad;
}

int main() {
  long bad = 0;
  // rows that belong to one request each: nothing is clipped
  for (int B : {1, 2, 7, 700, 16384})
    for (int group : {1, 3, 8}) {
      std::vector<long long> n;
      long long tokens = 0, sum = 0;
      for (int b = 0; b < B; ++b) {
        n.push_back((b * 37) % 301);
        tokens += n.back();
        sum += (n.back() * group + 255) / 256;
      }
      const mxk::KvTileList list(tokens, group, 256, B);
      bad += list.clip(sum) != sum;
      bad += check(n, tokens, group);
    }
  // offsets that go from one end of Q to the other and back
  for (int group : {1, 16}) {
    const long long tokens = (0x7FFFFFFFll - 1024) / group;
    std::vector<long long> n;
    for (int b = 0; b < 16384; ++b) n.push_back(b % 2 ? 0 : tokens);
    bad += check(n, tokens, group);
  }
  std::printf("bad %ld\n", bad);
  return bad != 0;
}
"""


def test_the_list_of_row_tiles():
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not available")
    os.makedirs(BUILD, exist_ok=True)
    src, exe = os.path.join(BUILD, "plan_check.cu"), os.path.join(BUILD, "plan_check")
    with open(src, "w") as f:
        f.write(HARNESS)
    subprocess.check_call([nvcc, "-std=c++17", "-O1", "-gencode", "arch=compute_103a,code=sm_103a",
                           "--expt-relaxed-constexpr", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                           src, "-o", exe])
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout
    assert "bad 0" in out.stdout
