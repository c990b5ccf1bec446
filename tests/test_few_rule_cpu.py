"""Which calls of the attention over 4 bits the register path takes, without a GPU: the rule takes the side
that was measured faster."""
import subprocess

from jacobi_block_refiner_amd import build
from tests import few_plan

# D, requests, own tokens that a table holds (8 heads, 64 rows a head), and whether few_kernel was faster, by
# more than one part in twenty
MEASURED = [
    (64, 64, 4000, 1), (64, 8, 16000, 1), (64, 64, 1000, 0), (64, 4, 16000, 0), (64, 1, 16000, 0), (64, 8, 4000, 0),
    (128, 64, 4000, 1), (128, 64, 1000, 1), (128, 8, 4000, 1), (128, 2, 16000, 1), (128, 32, 2000, 1),
    (128, 64, 300, 0), (128, 1, 16000, 0), (128, 8, 1000, 0), (128, 4, 2000, 0),
    (256, 64, 4000, 1), (256, 64, 300, 1), (256, 8, 2000, 1), (256, 16, 1000, 1), (256, 1, 16000, 1),
    (256, 16, 300, 0), (256, 8, 1000, 0), (256, 1, 4000, 0),
]


def test_the_tests_know_the_plan(tmp_path):
    """few_plan.py, by which tests say which path a call takes, agrees with the library's own plan."""
    src = tmp_path / "plan.cpp"
    src.write_text('''#include "attend_plan.hpp"
#include <cstdio>
using namespace xpress;
int main() {
  for (int D : {64, 128, 256})
    for (int R = 1; R <= kFewRows4; ++R)
      for (int n : {1, 9, 64})
        for (int pages : {1, 40, 700, 3000}) {
          xpress_cache c{};
          c.D = D, c.Hkv = 4, c.page = 64, c.table_ld = pages;
          printf("%d %d %d ", few_waves(D, R), few_parts(D, R), (int)few_rows(c, n, R, 64));
        }
  printf("%d", kFewRequests);
}
''')
    exe = tmp_path / "plan"
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{build.CSRC}", f"-I{build.INCLUDE}", str(src), "-o",
                    str(exe)], check=True)
    want = []
    for D in (64, 128, 256):
        for R in range(1, 65):
            for n in (1, 9, 64):
                for pages in (1, 40, 700, 3000):
                    want += [few_plan.waves(D, R), few_plan.parts(D, R),
                             int(few_plan.taken(D, R, n, 4, pages * 64 - 64))]
    got = subprocess.run([str(exe)], capture_output=True, text=True).stdout
    assert [int(x) for x in got.split()] == want + [few_plan.REQUESTS]


def test_the_rule_against_its_measurements(tmp_path):
    calls = "".join(f"  if (taken({D}, {n}, {own}) != {few}) return {i + 1};\n"
                    for i, (D, n, own, few) in enumerate(MEASURED))
    src = tmp_path / "rule.cpp"
    src.write_text('''#include "attend_plan.hpp"
using namespace xpress;
bool taken(int D, int n, int own, int R = 64) {
  xpress_cache c{};
  c.D = D, c.Hkv = 8, c.page = 64, c.table_ld = (own + 63) / 64 + 1;
  return few_rows(c, n, R, 0);
}
int main() {
''' + calls + '''  for (int D : {64, 128, 256}) {
    if (!taken(D, 1, 1, 1) || !taken(D, 1, 1, 32) || taken(D, 4096, 1 << 20, kFewRows4 + 1)) return 100;
    for (int R = 1; R <= kFewRows4; ++R) {  // the waves of a part hold its rows
      if (few_waves(D, R) * few_row_tiles(D, R) * 16 < R || 4 % few_waves(D, R)) return 101;
      if (few_parts(D, R) < kCUs * 2) return 102;
    }
  }
  return 0;
}
''')
    exe = tmp_path / "rule"
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{build.CSRC}", f"-I{build.INCLUDE}", str(src), "-o",
                    str(exe)], check=True)
    got = subprocess.run([str(exe)], timeout=60).returncode
    assert got == 0, MEASURED[got - 1] if got <= len(MEASURED) else got
