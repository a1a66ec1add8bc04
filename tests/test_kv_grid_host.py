"""CTAs of a call on packed tokens (csrc/kv_index.h) on the host, up to the largest number of tokens that a call takes."""
import os
import shutil
import subprocess

import pytest

from speculative_decode_verify_gdn_gb300.build import CSRC_DIR

PROGRAM = """
#include <cstdio>
#include "kv_index.h"
int main() {
  const long long edges[] = {0, 4096, (1ll << 30), (1ll << 31) - 1};
  for (int each = 1; each <= 8; ++each)
    for (long long edge : edges)
      for (long long n = edge - 40; n <= edge + 40; ++n) {
        if (n < 0 || n >= (1ll << 31)) continue;
        const long long want = n / each + (n % each != 0);
        if (gdn::ctas_of(int(n), each) != want || (want - 1) * each > 0x7fffffffll) {
          printf("%lld tokens, %d a CTA: %u\\n", n, each, gdn::ctas_of(int(n), each));
          return 1;
        }
      }
  return 0;
}
"""


def test_ctas_up_to_the_most_tokens(tmp_path):
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "ctas.cpp").write_text(PROGRAM)
    subprocess.run([compiler, "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", f"-I{CSRC_DIR}", "ctas.cpp", "-o", "ctas"],
                   cwd=tmp_path, check=True)
    r = subprocess.run([os.path.join(tmp_path, "ctas")], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
