"""How many clusters shared prefixes get beside the kernel for few rows, on the host: the plan's own arithmetic
(csrc/share_split.h), compiled with the host's compiler."""
import os
import shutil
import subprocess

import pytest

import fp8_mla_latent_gb300 as pkg

CSRC = os.path.join(os.path.dirname(os.path.abspath(pkg.__file__)), "csrc")
SMS = 152

# the plan's search, with one lane for all of them: clusters at most, of those that the device holds at once
PROGRAM = r"""
#include <cstdio>
#include "share_split.h"
int main() {
  float wide, narrow;
  long long apart;
  int most, clusters, always;
  while (std::scanf("%f %f %lld %d %d %d", &wide, &narrow, &apart, &most, &clusters, &always) == 6) {
    int64_t least = INT64_MAX;
    for (int t = 1; t <= most && t < clusters; ++t) {
      const int64_t z = kv8::split_cost(wide, narrow, t, 152);
      least = z < least ? z : least;
    }
    std::printf("%d\n", kv8::split_taken(least, apart, always != 0));
  }
}
"""


@pytest.fixture(scope="module")
def splits(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    d = tmp_path_factory.mktemp("split")
    (d / "split.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I" + CSRC, str(d / "split.cpp"), "-o", str(d / "split")], check=True)

    def run(cases):
        text = "\n".join(" ".join(str(v) for v in c) for c in cases)
        out = subprocess.run([str(d / "split")], input=text, capture_output=True, text=True, check=True).stdout.split()
        assert len(out) == len(cases)
        return [int(v) for v in out]
    return run


WORK = [(1e3, 1e3), (3.1e3 * 300, 3.2e3 * 64), (3.1e3 * 600, 3.2e3 * 6400), (4.3e9, 1e4), (1e4, 4.3e9), (5e13, 5e13)]


def test_one_cluster_at_once_shares_nothing(splits):
    """The prefixes' cluster would be the only one there is: no count is tried, and none is taken, demanded or not."""
    cases = [(w, n, apart, most, clusters, always) for w, n in WORK for apart in (0, 10 ** 5, 10 ** 15) for most in (1, 38)
             for clusters in (0, 1) for always in (0, 1)]
    assert set(splits(cases)) == {0}


def test_a_count_that_leaves_sms_to_both(splits):
    cases = [(w, n, apart, most, clusters, always) for w, n in WORK for apart in (0, 10 ** 5, 10 ** 15)
             for most in (1, 2, 7, 37, 38) for clusters in (2, 3, 36, 37, 38) for always in (0, 1)]
    for c, t in zip(cases, splits(cases)):
        assert 0 <= t <= c[3] and t < c[4] and SMS - 4 * t > 0, c
        assert t > 0 or not c[5], c     # demanded: wherever it can be
        assert t == 0 or c[2] > 0 or c[5], c  # (nothing costs less than nothing)
    some = {t for c, t in zip(cases, splits(cases)) if not c[5]}
    assert 0 in some and len(some) > 3
