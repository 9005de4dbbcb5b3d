"""No signed overflow in the page plan's arithmetic (csrc/pages_sums.h) at the ends of its ranges: compiled with traps for it."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_layer_dsv3_gb300", "csrc")
CODE = """
#include <cstdlib>
#include "pages_sums.h"
using namespace moe::pages;
int main() {
  const int last = 2147483647, most = 1 << 30;
  const int pages[] = {1, 2, 7, 64, 1 << 20, most};
  for (int page : pages) {
    const int top = last - 1 - page;       // the longest length: (max_pages + 1) page_size is below 2^31 - 1
    const int lens[] = {0, 1, page < top ? page : top, top / 2, top - 1, top};
    Sums all{0, 0, 0};
    for (int n : lens)
      for (int m : lens) {
        all += sums_of(n, m, page);
        step_code(all, 0, 1, 0);
        step_code(all, most - 1, most - 1, most - 1);
      }
  }
  // the last of nearly 2^30 new tokens, at the end of the longest sequence, and of nearly 2^30 pages of one token
  if (nth(last - 10, most - 1, most - 4) != last - 7) return 1;
  if (nth(most - 4, last - 10, last - 13) != most - 1) return 2;
  if (nth(0, most - 1, 0) != most - 1) return 3;
  return 0;
}
"""


def test_no_signed_overflow(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    (tmp_path / "ends.cpp").write_text(CODE)
    exe = str(tmp_path / "ends")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=signed-integer-overflow",
                    "-fsanitize-undefined-trap-on-error", "-I", CSRC, "-o", exe, str(tmp_path / "ends.cpp")], check=True)
    assert subprocess.run([exe]).returncode == 0


def test_the_kernel_uses_this_code():
    text = open(os.path.join(CSRC, "k_pages.cu")).read()
    assert "pages::nth(len[b], i, starts[b])" in text and "pages::nth(taken[b], j, old)" in text
