"""The paged cache's index arithmetic (csrc/kv_index.h) on the host, over its whole range."""
import os
import shutil
import subprocess

import pytest

from speculative_decode_verify_gdn_gb300.build import CSRC_DIR

# Each column's first and last unit of 16 tokens, for every page size and up to the longest slot (the
# quotient is monotonic in between, and so is the exact one).
PROGRAM = """
#include <cstdio>
#include "kv_index.h"
int main() {
  for (int m = 1; m <= 64; ++m) {
    const uint32_t inv = gdn::page_units_inv(16 * m);
    const long long units = (1ll << 30) / 16;
    for (long long col = 0; col * m < units; ++col) {
      const long long first = col * m, last = col * m + m - 1 < units ? col * m + m - 1 : units - 1;
      if (gdn::page_column(int(16 * first), inv) != col || gdn::page_column(int(16 * last), inv) != col) {
        printf("page_size %d column %lld\\n", 16 * m, col);
        return 1;
      }
    }
  }
  return 0;
}
"""


def test_page_columns_are_exact_up_to_the_longest_slot(tmp_path):
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "columns.cpp").write_text(PROGRAM)
    subprocess.run([compiler, "-O2", "-std=c++17", f"-I{CSRC_DIR}", "columns.cpp", "-o", "columns"], cwd=tmp_path, check=True)
    r = subprocess.run([os.path.join(tmp_path, "columns")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
