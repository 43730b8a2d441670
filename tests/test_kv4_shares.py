"""How the 4-bit attention's warps share out the key tiles and count finished parts: the kernel's own
arithmetic (csrc/sv_kv4_shares.h), compiled for the host, over many batches and SM counts.  Every tile
belongs to one warp, every cut group's parts have places of their own, every counter word belongs to
one group, and each group's runs cover its warps."""

import os
import shutil
import subprocess

import numpy as np
import pytest

from speculative_decoding_verification_47_gb300 import build

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <map>
#include <utility>
#include "sv_kv4_shares.h"
using namespace sv::kv4;
typedef unsigned long long U;

// warps, heads, then the sequences' tiles; prints "ok <cut groups> <runs of one warp>"
int main() {
  unsigned warps, heads, n;
  while (std::scanf("%u %u %u", &warps, &heads, &n) == 3) {
    std::map<std::pair<int, unsigned>, U> words, places;  // (level or place, warp) -> group
    std::map<U, int> groups;
    U total = 0;
    for (unsigned b = 0; b < n; ++b) {
      int tiles;
      if (std::scanf("%d", &tiles) != 1) return 2;
      for (unsigned h = 0; h < heads; ++h) groups[total] = tiles, total += tiles + kGroupCost;
    }
    const U share = share_of(total, warps);
    if (share < (U)kMinShare || share * warps < total) return 3;
    int cut = 0, alone = 0;
    for (auto& g : groups) {
      const U at = g.first + kGroupCost, end = at + g.second;
      const unsigned first = (unsigned)(at / share), last = (unsigned)((end - 1) / share);
      if (last >= warps) return 4;
      if (first == last) continue;
      ++cut;
      unsigned covered = 0, runs = 0;
      for (unsigned w = first; w <= last; ++w) {
        const Run r = run_of(g.first, g.second, share, w);
        if (r.w0 != first || w < r.first || w >= r.first + r.n || r.first + r.n - 1 > last || r.n < 1 || r.n > kJoin) return 5;
        if ((r.first - first) % kJoin != 0 || r.runs != (last - first) / kJoin + 1) return 6;
        if (w == r.first) covered += r.n, ++runs, alone += r.n == 1;
        if (r.n > 1 && words.insert({{0, r.first}, g.first}).first->second != g.first) return 7;
        if (r.runs > 1 && words.insert({{1, r.w0}, g.first}).first->second != g.first) return 8;
        if (!places.insert({{part_place(w, share, g.first), w}, g.first}).second) return 9;
      }
      if (covered != last - first + 1 || runs != run_of(g.first, g.second, share, first).runs) return 10;
    }
    std::printf("ok %d %d\n", cut, alone);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("shares")
    (d / "shares.cpp").write_text(PROGRAM)
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", f"-I{build.CSRC}", str(d / "shares.cpp"), "-o",
           str(d / "shares")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr

    def run(batches):
        text = "".join(f"{w} {h} {len(t)} {' '.join(map(str, t))}\n" for w, h, t in batches)
        r = subprocess.run([str(d / "shares")], input=text, capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, (r.returncode, r.stdout.count("ok"))  # which check failed, in which batch
        return [tuple(map(int, line.split()[1:])) for line in r.stdout.splitlines()]
    return run


def tiles(lens):
    return [max(1, -(-int(n) // 16)) for n in lens]


def test_one_long_sequence_among_short_ones(shares):
    """A last run of one warp in whose share the next cut group begins."""
    lens = ([60464] + [1600] * 63, [126768] + [1000] * 63, [52016] + [100] * 31,
            [32305, 17049, 24541, 20725, 322, 30937, 250, 8225, 32072, 32413, 22325, 4621, 15128, 7244, 26248, 1359])
    for warps in (1824, 1776, 1216):
        got = shares([(warps, 8, tiles(n)) for n in lens])
        assert len(got) == 4 and all(cut > 0 for cut, _ in got)


@pytest.mark.parametrize("sms", [148, 152, 132, 160])
@pytest.mark.parametrize("ctas", [2, 3])
def test_drawn_batches(shares, sms, ctas):
    r = np.random.default_rng(sms * 10 + ctas)
    batches = []
    for _ in range(1500):
        n, kind = int(r.integers(1, 65)), r.integers(3)
        lens = r.integers(0, 1 << int(r.integers(4, 16)), n)
        if kind == 0:
            lens[:] = lens[0]                                 # all alike
        elif kind == 1:
            lens[r.integers(0, n)] = r.integers(20000, 130000)  # a long one among them
        batches.append((min(sms * ctas, 640) * 4, int(r.choice([1, 2, 4, 8, 12])), tiles(lens)))
    got = shares(batches)
    assert len(got) == len(batches) and sum(alone for _, alone in got) > 200  # the runs of one warp occur
