"""The paged attends' cut of work (csrc/paged_cut.h, the header that the kernels include),
compiled for the host: sums that pass 32 bits, and calls whose shares would."""
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_scored_kv_gb300", "csrc")

MAIN = r'''
#include <cstdio>
#include <cstdlib>
#include "paged_cut.h"
using namespace kvs::cut;
int main(int argc, char** argv) {
  long long v[5];
  for (int i = 0; i < 5 && i + 2 < argc; ++i) v[i] = atoll(argv[i + 2]);
  if (argv[1][0] == 'c') {            // cost: p0 n window per
    long long sum = 0;
    for (int lane = 0; lane < 32; ++lane) sum += lane_cost((int)v[0], (int)v[1], (int)v[2], (int)v[3], lane, 32);
    std::printf("%lld\n", sum);
  } else {                            // fits: units stride hkv ctas
    std::printf("%d\n", (int)share_fits(v[0], (int)v[1], (int)v[2], (int)v[3]));
  }
}
'''


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    d = tmp_path_factory.mktemp("cut")
    src, exe = d / "main.cpp", d / "main"
    src.write_text(MAIN)
    subprocess.run(["g++", "-O2", "-std=c++17", "-fwrapv", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return lambda *a: int(subprocess.run([str(exe), *map(str, a)], capture_output=True, text=True, check=True).stdout)


def cost(p0, n, window, per):
    i0 = np.arange(0, n, per, dtype=np.int64)
    hi = np.maximum(p0 + np.minimum(i0 + per, n), 0)
    lo = np.maximum(p0 + i0 + 1 - window, 0) if window else np.zeros_like(i0)
    blocks = np.maximum(-(-hi // 16) - lo // 16, 0)
    return int((np.maximum(-(-blocks // 8), 1) + 3).sum())


@pytest.mark.parametrize("p0,n,window,per", [
    (0, 1, 0, 32), (0, 8192, 0, 32), (-3, 5, 0, 16), (1000, 333, 40, 2), (7, 100, 1, 4), (0, 0, 0, 8),
    (0, 1_500_000, 0, 4), (0, 4_100_000, 0, 32), (8_000_000, 131072, 0, 4), (0, 1 << 26, 0, 256), (0, 1 << 26, 1, 4),
    (0, 4_300_000, 0, 32), (8_400_000, 131072, 0, 4),
])
def test_costs(run, p0, n, window, per):
    want = cost(p0, n, window, per)
    assert run("cost", p0, n, window, per) == want
    if (p0, n, per) in ((0, 1_500_000, 4), (0, 4_300_000, 32), (8_400_000, 131072, 4)):
        assert want > 2 ** 31                      # what an int does not hold


def test_shares(run):
    # an 8 M token prompt on 64/8 heads, and a batch of 1024 contexts of 131072 tokens
    assert run("fits", 8_000_000 // 32 + 1, 500_000, 8, 152) == 1
    assert run("fits", 1024, 8192, 8, 304) == 1
    assert run("fits", 1 << 20, 1 << 22, 1, 304) == 1
    assert run("fits", 1 << 20, 1 << 22, 2, 304) == 0
    assert run("fits", 1 << 26, 1 << 22, 1, 152) == 0
