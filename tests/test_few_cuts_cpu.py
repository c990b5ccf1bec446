"""The records of pairs that are cut, without a GPU: what the join makes of them stays inside the pairs and
the slots whatever the workspace holds, and records of a call as it should be stay as they are."""
import subprocess

from jacobi_block_refiner_amd import build

CUTS = r"""
#include "attend_plan.hpp"
#include <climits>
#include <random>
#include <set>
#include <vector>
using namespace xpress;
int inside(const Cut& c, int pairs, int parts) {
  if (c.pair < 0 || c.pair >= pairs || c.slots < 0) return 1;
  for (int own = 0; own < c.slots; ++own) {  // the slots that the join reads
    const int64_t at = own == 0 ? c.slot : 2 * ((int64_t)c.part + own);
    if (at < 0 || at >= 2 * (int64_t)parts) return 2;
  }
  return 0;
}
int main() {
  std::mt19937 rng(1);
  const int odd[] = {INT_MIN, INT_MIN + 1, -1, 0, 1, 2, 7, 511, 512, 1 << 30, INT_MAX - 1, INT_MAX};
  for (int pairs : {1, 5, 290, 1 << 23})
    for (int parts : {1, 2, 512, 2048}) {
      for (int a : odd)
        for (int b : odd)
          for (int c : odd)
            for (int d : odd)
              if (int e = inside(cut_inside(Cut{a, b, c, d}, pairs, parts), pairs, parts)) return e;
      for (int i = 0; i < 20000; ++i) {
        const Cut x{(int)rng(), (int)rng(), (int)rng(), (int)rng()};
        if (int e = inside(cut_inside(x, pairs, parts), pairs, parts)) return e;
      }
    }
  // a sequence of pairs' tiles in equal parts, as the waves walk through it
  for (int round = 0; round < 300; ++round) {
    const int pairs = 1 + rng() % 400, parts = 1 + rng() % 64, least = 1 + rng() % 3;
    std::vector<int64_t> first(pairs + 1, 0);
    for (int p = 0; p < pairs; ++p) first[p + 1] = first[p] + 1 + (rng() % 8 ? rng() % 4 : rng() % 200);
    const int64_t all = first[pairs], each = std::max<int64_t>((all + parts - 1) / parts, least);
    std::set<int> used;
    for (int p = 0; p < pairs; ++p) {
      const int from = (int)(first[p] / each), to = (int)((first[p + 1] - 1) / each);
      if (to >= parts) return 3;
      if (from == to) continue;
      const int slot = 2 * from + (first[p] > from * each ? 1 : 0);  // (behind another pair in its part)
      const Cut c{p, to - from + 1, from, slot}, got = cut_inside(c, pairs, parts);
      if (got.pair != c.pair || got.slots != c.slots || got.part != c.part || got.slot != c.slot) return 4;
      for (int own = 0; own < c.slots; ++own)
        if (!used.insert(own == 0 ? c.slot : 2 * (c.part + own)).second) return 5;  // a slot of two pairs
    }
  }
  return 0;
}
"""


def test_records_of_cut_pairs(tmp_path):
    src = tmp_path / "cuts.cpp"
    src.write_text(CUTS)
    exe = tmp_path / "cuts"
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover",
                    f"-I{build.CSRC}", f"-I{build.INCLUDE}", str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], timeout=60).returncode == 0
