"""The rule for an entry of a path of accepted drafts (csrc/paged_path.h), compiled as it is and gone through on the CPU:
what it lets pass never leads out of a sequence's row of the page table, and every path that increases passes."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_grouped_expert_moe_gb300", "csrc")

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include "paged_path.h"
using bgmoe::paged::path_entry_ok;
int main() {
  const int values[] = {INT_MIN, INT_MIN + 1, -100, -99, -3, -2, -1, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 100, INT_MAX - 1, INT_MAX};
  const long long limits[] = {1, 2, 5, 9, 1ll << 26};
  long passed = 0;
  for (long long limit : limits)
    for (long long s = 0; s <= limit; s = s < 9 ? s + 1 : s < limit - 9 ? limit - 9 : s + 1)
      for (int k = 0; k < 6; ++k)
        for (int before : values)
          for (int from : values) {
            if (k == 0 && before != -1) continue;
            const int start = (int)s;
            const bool ok = path_entry_ok(from, before, k, start, limit);
            passed += ok;
            // both positions of an entry that passes
            if (ok && !(from >= 0 && start + (long long)from < limit && start + (long long)k < limit)) {
              std::printf("entry %d of %d after %d from %d leaves %lld\n", from, k, before, start, limit);
              return 1;
            }
            // an entry of a path that increases within the table: k entries before it, the last of them `before`
            if (!ok && before >= k - 1 && from > before && start + (long long)from < limit) {
              std::printf("entry %d of %d after %d from %d refused\n", from, k, before, start);
              return 1;
            }
          }
  return passed > 100 ? 0 : 2;
}
"""


def test_entries_that_pass_stay_in_the_table(tmp_path):
    src, exe = tmp_path / "path.cpp", tmp_path / "path"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout
