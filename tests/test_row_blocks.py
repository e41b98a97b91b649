"""The copies of a weight gradient's rows, checked on the host for every range of small buffers: each row
of the range exactly once and none beside it, no view that reaches out of its buffer, no negative start."""
import os
import subprocess

from mxfp4_expert_gemm_b200 import build

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "row_blocks.h"
using namespace moe;
static int bad(const char* what, int rows, int c0, int n) {
  std::printf("%s: rows %d, range %d + %d\n", what, rows, c0, n);
  return 1;
}
static int check(int rows, int c0, int n, int most) {
  const int win = window_rows(0, rows), blocks = weight_blocks(win, c0, n);
  if (blocks > most) return bad("too many blocks", rows, c0, n);
  std::vector<int> seen(rows, 0);
  for (int kb = 0; kb < blocks; ++kb) {
    const RowBlock b = weight_block(win, c0, n, kb);
    if (b.map < 0 || b.map > 2) return bad("no such map", rows, c0, n);
    const int w = window_rows(b.map, rows), starts = rows - w + 1;   // the view: [starts][w]
    if (w < 1 || starts < 1 || (starts - 1) + (w - 1) > rows - 1) return bad("the view leaves the buffer", rows, c0, n);
    if (b.d1 < 0 || b.d1 >= w || b.d2 < 0 || b.d2 >= starts) return bad("the copy starts outside the view", rows, c0, n);
    for (int k = 0; k < kBlockRows; ++k)
      if (b.d1 + k < w) ++seen[b.d1 + k + b.d2];   // others read zeros
  }
  for (int r = 0; r < rows; ++r)
    if (seen[r] != (r >= c0 && r < c0 + n)) return bad("a row too often, or too few times", rows, c0, n);
  return 0;
}
int main() {
  for (int rows = 1; rows <= 200; ++rows)
    for (int c0 = 0; c0 <= rows; ++c0)
      for (int n = 0; c0 + n <= rows; ++n)
        if (check(rows, c0, n, c0 + n >= 64 || c0 + n == rows ? (n + 63) / 64 : 14)) return 1;
  for (int c0 : {0, 1, 63, 64, 1000, 16777000})
    for (int n : {0, 1, 7, 63, 64, 65, 200})
      if (check(1 << 24, c0, n, c0 + n >= 64 ? (n + 63) / 64 : 14)) return 1;
  return 0;
}
"""


def test_every_range(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", build.CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout


def test_the_build_watches_the_header():
    assert os.path.join(build.CSRC, "row_blocks.h") in build.dependencies()
