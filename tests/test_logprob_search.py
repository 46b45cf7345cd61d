"""The search for the likeliest groups: the kernel's own steps (sv_logprobs.cuh), compiled
for the host, against sorting."""
import os
import subprocess

import numpy as np
import pytest

from speculative_decoding_verification_63_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "sv_logprobs.cuh"
int main() {  // cases: n, lo, hi, how many keys, the keys
  unsigned n, lo, hi, m;
  while (std::scanf("%u %u %u %u", &n, &lo, &hi, &m) == 4) {
    std::vector<unsigned> keys(m);
    for (unsigned& k : keys) if (std::scanf("%u", &k) != 1) return 1;
    sv::LpSearch s{lo, hi, 0};
    int step = 0;
    for (; s.more(step); ++step) {
      unsigned at[3], reach[3] = {0, 0, 0};
      s.keys(step, at);
      for (unsigned k : keys)
        for (int q = 0; q < 3; ++q) reach[q] += k >= at[q];
      s.narrow(at, reach, n);
    }
    std::printf("%u %u %u %d\n", s.lo, s.hi, s.above, step);
  }
}
"""


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    at = tmp_path_factory.mktemp("search")
    (at / "search.cu").write_text(PROGRAM)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-O1", "-std=c++17", f"-I{_build.CSRC}",
                    f"-I{_build.INCLUDE}", "-o", str(at / "search"), str(at / "search.cu")],
                   check=True)

    def run(cases):
        text = "\n".join(" ".join(map(str, [n, lo, hi, len(keys), *keys]))
                         for n, lo, hi, keys in cases)
        out = subprocess.run([str(at / "search")], input=text, capture_output=True, text=True,
                             check=True).stdout
        return [tuple(map(int, line.split())) for line in out.splitlines()]
    return run


def test_the_kernels_search_finds_the_last_group(search):
    """Keys of 16 and of 32 bits, alone and equal, few and many, from a bound that they all
    reach or that lies far below."""
    rng = np.random.default_rng(3)
    cases = []
    for trial in range(4000):
        hi = 0x10000 if trial % 2 else 0xffffffff
        span = int(rng.choice([0, 1, 2, 3, 4, 5, 100, 5000, hi - 300]))
        base = int(rng.integers(129, hi - 100 - span)) if span < hi - 300 else 129
        n = int(rng.integers(1, 65))
        keys = np.minimum(base + rng.integers(0, span + 1, rng.integers(n, 200)), hi - 1)
        if trial % 3 == 0:  # most of them equal
            keys[rng.random(len(keys)) < 0.9] = keys[0]
        cases.append((n, int(rng.choice([np.sort(keys)[-n], keys.min(), 128])), hi, keys.tolist()))
    for (n, _, _, keys), (lo, hi, above, steps) in zip(cases, search(cases), strict=True):
        last = sorted(keys)[-n]
        assert (lo, hi, above) == (last, last + 1, sum(k > last for k in keys))
        assert steps <= 18


def test_the_search_takes_no_more_steps_than_there_are_counts_for(search):
    """The widest ranges, with the key at their ends and all over them."""
    rng = np.random.default_rng(4)
    cases = []
    for hi in (0x10000, 0xffffffff):
        for lo in (128, 0x7fff, hi // 2, hi - 2):
            for key in [lo, lo + 1, hi - 1, *rng.integers(lo, hi, 300).tolist()]:
                cases.append((1, lo, hi, [min(key, hi - 1)]))
    for (n, _, _, keys), (lo, hi, above, steps) in zip(cases, search(cases), strict=True):
        assert (lo, hi, above) == (keys[0], keys[0] + 1, 0) and steps <= 18
