"""Eight elements of a row that starts anywhere, compiled by itself on the CPU with every byte outside of the
rows watched: the values, and nothing read that is not the caller's."""
import os
import subprocess

import pytest

from .test_lm_host import CSRC, ROOT, cuda_include

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include "row_piece.h"
int main() {
  // a matrix whose last row ends the allocation: each piece of each row, rows off 16 bytes by every even number
  for (int ld = 1; ld <= 40; ++ld)
    for (int cols = 1; cols <= ld; ++cols) {
      const int rows = 10, n = (rows - 1) * ld + cols;
      uint16_t* m = static_cast<uint16_t*>(std::malloc(2 * n));  // (16-byte aligned)
      for (int i = 0; i < n; ++i) m[i] = static_cast<uint16_t>(1 + i);
      for (int r = 0; r < rows; ++r)
        for (int c = 0; c < cols; c += 8) {
          const uint4 v = zopt::lm::row_piece8(m + r * ld + c, cols - c);
          uint16_t got[8];
          std::memcpy(got, &v, 16);
          for (int k = 0; k < 8; ++k)
            if (got[k] != (c + k < cols ? 1 + r * ld + c + k : 0)) return std::printf("wrong: %d %d %d %d\n", ld, cols, r, c), 1;
        }
      std::free(m);
    }
  std::printf("right\n");
}
"""


def test_no_byte_outside_the_rows_is_read(tmp_path):
    src, exe = tmp_path / "a.cpp", tmp_path / "a"
    src.write_text("int main() {}\n")
    command = ["g++", "-std=c++17", "-g", "-O0", "-fsanitize=address", "-D__forceinline__=inline", f"-I{CSRC}", f"-I{cuda_include()}",
               f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)]
    if subprocess.run(command, capture_output=True).returncode != 0 or subprocess.run([str(exe)], capture_output=True).returncode != 0:
        pytest.skip("no address sanitizer here")
    src.write_text(SOURCE)
    subprocess.run(command, check=True)
    done = subprocess.run([str(exe)], capture_output=True, text=True)
    assert done.returncode == 0 and done.stdout == "right\n", done.stdout + done.stderr[-3000:]
