"""How the norm kernels spread rows over CTAs (csrc/row_grid.cuh), as plain
C++ on the CPU: within the rows and the workspace's partial rows, and with
rows a multiple of a vector apart, on whole devices and on a few SMs of one
(a partition, or a limited share under MPS)."""
import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_dynamic_quantization_amax_b200", "csrc")

PROGRAM = r"""
#include "row_grid.cuh"
#include <cstdio>
int main() {
  const long long apart[] = {1, 4, 8};
  for (long long a : apart)
    for (long long most = 1; most <= 300; ++most)
      for (long long rows = 1; rows <= 700; ++rows) {
        const long long g = hq::row_grid(rows, most, a);
        const bool one_each = g == rows;
        if (g < 1 || g > rows || g > (most > a ? most : a) || (!one_each && g % a != 0) || (rows <= most && !one_each)) {
          std::printf("rows %lld most %lld apart %lld: %lld\n", rows, most, a, g);
          return 1;
        }
      }
  return hq::row_grid(2147483647, 296, 8) == 296 && hq::row_grid(2147483647, 148, 8) == 144 &&
         hq::row_grid(6, 2, 8) == 6 && hq::row_grid(100, 3, 4) == 4 ? 0 : 2;
}
"""


def test_rows_spread_over_ctas(tmp_path):
    src, exe = tmp_path / "grid.cpp", tmp_path / "grid"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_norm_kernels_take_their_grids_from_it():
    text = open(os.path.join(CSRC, "norm.cu")).read()
    assert text.count("row_grid(") == 4 and "most / vec_elems" not in text
