"""The bytes that the staged norm backward's bulk copies read, on the host (CPU only).

The kernel takes them from csrc/row_span.h, which is compiled here as plain C++
and checked row by row: every copy starts and ends on 16 bytes, none reads
outside the matrix, and the columns that a copy leaves out are few, at the end
of the last row.
"""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "row_span.h"

// Copies of a [rows][ld] matrix of `size`-byte elements whose base lies on a unit.
static int check(long rows, long cols, long ld, long size) {
  const long extent = ((rows - 1) * ld + cols) * size;
  for (long r = 0; r < rows; ++r) {
    const long m = r * (ld & 7) & 7, unit = (r * ld - m) * size;       // the unit's first byte
    const sf::CopySpan s = sf::copy_span((uint32_t)m, (uint32_t)cols, (uint32_t)size, r == rows - 1);
    const long from = unit + s.begin, to = unit + s.end, row = r * ld * size, row_end = row + cols * size;
    const char* wrong = unit % (8 * size) ? "unit" : from % 16 || to % 16 ? "alignment" : from < 0 || to > extent ? "outside"
                      : from > row || row - from > 15 ? "start" : r < rows - 1 && to < row_end ? "end"
                      : row_end - to > 15 ? "left out" : to - row_end > 15 ? "beyond" : nullptr;
    if (wrong) {
      std::printf("%s: row %ld of %ld, cols %ld ld %ld size %ld, bytes %ld..%ld of %ld\n", wrong, r, rows, cols, ld, size, from, to, extent);
      return 1;
    }
  }
  return 0;
}

int main() {
  for (long size = 2; size <= 4; size += 2)
    for (long cols = 512; cols < 552; ++cols)
      for (long pad = 0; pad < 18; ++pad)
        for (long rows = 1; rows < 20; ++rows)
          if (check(rows, cols, cols + pad, size)) return 1;
  return 0;
}
"""


def test_bulk_copies_stay_inside_the_matrix(tmp_path):
    src, exe = tmp_path / "span.cpp", tmp_path / "span"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "layer_optimizer_gb300", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
