"""The bulk copies of the norm's ring on the CPU: every row is taken once, by a copy or
in place, and no copy reads outside the matrix."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int4_gemm_gb300", "csrc")
PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "ring_rows.h"

// rows of row_bytes at `at`, pitch bytes apart, by turns of per_block over `blocks` blocks
static bool check(uintptr_t at, int64_t pitch, uint32_t row_bytes, int64_t rows, int per_block, int blocks) {
  using namespace q4;
  const int edge = edge_rows(row_bytes);
  const uintptr_t last = at + (uintptr_t)((rows - 1) * pitch) + row_bytes;
  std::vector<int> taken((size_t)rows, 0);
  for (int b = 0; b < blocks; ++b)
    for (int64_t base = (int64_t)b * per_block; base < rows; base += (int64_t)blocks * per_block) {
      const CopiedRows c = copied_rows(base, per_block, rows, edge);
      for (int64_t r = base + c.begin; r < base + c.end; ++r) {
        if (r < base || r >= base + per_block) return false;
        const uintptr_t begin = at + (uintptr_t)(r * pitch);
        const Window w = window_of(begin, row_bytes);
        if (w.begin % 16 || w.size % 16 || w.begin > begin || w.begin + w.size < begin + row_bytes) return false;
        if (w.begin < at || w.begin + w.size > last || w.size > window_bytes(row_bytes)) return false;
        ++taken[(size_t)r];
      }
      for (int64_t r = base; r < base + per_block && r < rows; ++r)
        if (read_in_place(r, rows, edge)) ++taken[(size_t)r];
    }
  for (int64_t r = 0; r < rows; ++r)
    if (taken[(size_t)r] != 1) return false;
  return true;
}

int main() {
  long checked = 0;
  for (int size : {2, 4})
    for (int H : {1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 129, 501})
      for (int pad : {0, 1, 3, 8})
        for (int offset = 0; offset < 16 / size; ++offset)
          for (int rows : {16, 17, 33, 100, 1000})
            for (int per_block : {1, 2, 3, 16}) {
              const uintptr_t at = 4096 + (uintptr_t)(offset * size);
              if (!check(at, (H + pad) * size, H * size, rows, per_block, 2)) {
                printf("size %d H %d pad %d offset %d rows %d per block %d\n", size, H, pad, offset, rows, per_block);
                return 1;
              }
              ++checked;
            }
  printf("%ld\n", checked);
}
"""


def test_copies_stay_inside_the_matrix(tmp_path):
    cc = shutil.which("g++") or shutil.which("c++")
    if cc is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "rows.cc").write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-O1", "-I", CSRC, "-o", str(tmp_path / "rows"), str(tmp_path / "rows.cc")], check=True)
    r = subprocess.run([str(tmp_path / "rows")], capture_output=True, text=True)
    assert r.returncode == 0 and int(r.stdout) > 10000, r.stdout
