"""The few-row kernels' index arithmetic at sizes near 2^31 - 1 (CPU: a program
that includes the kernels' header walks the ends)."""

import os
import shutil
import subprocess

import pytest

from tensor_core_dense_fp16_gb300 import build as tcbuild

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "linear_rows.h"
using namespace hg;

// The walk of one lane as the kernel does it, its last steps only: every
// position that passes for inside K is the one that 64 bits give.
static int walk(int K, int warps, int ahead) {
  int bad = 0;
  for (int warp = 0; warp < warps; ++warp)
    for (int t = 0; t < 4; ++t) {
      const long long step = 32ll * warps, round = ahead * step;
      const long long begin = 32ll * warp + 8 * t;
      long long last = K > 3 * round ? (K - 3 * round) / round * round : 0;  // whole rounds ahead
      RowsK k0 = rows_begin(warp, t) + static_cast<RowsK>(last);
      long long wide = begin + last;
      int rounds = 0;
      for (; rows_inside(k0 - 8 * t, K); k0 = rows_on(k0, ahead, warps), wide += round) {
        if (wide - 8 * t >= K || ++rounds > 8) return bad + 1000;  // runs past the end
        for (int u = 0; u < 2 * ahead; ++u) {
          const RowsK k = rows_on(k0, u, warps);
          const long long w = wide + u * step;
          if (rows_inside(k, K) != (w < K) || (w < K && static_cast<long long>(k) != w)) ++bad;
        }
      }
      if (wide - 8 * t < K) ++bad;  // stopped short
    }
  return bad;
}

int main() {
  int bad = 0;
  const int sizes[] = {1, 31, 32, 33, 4096, 0x7FFFFFFF, 0x7FFFFFFF - 1, 0x7FFFFFF8, 0x7FFFFFFF - 3000, 0x7FFFFFFF - 5000};
  for (int n : sizes) {
    for (int warps : {4, 8, 16})
      for (int ahead : {2, 4}) bad += walk(n, warps, ahead);
    if (rows_blocks(n) != (n + 15ll) / 16 || rows_pieces(n) != (n + 31ll) / 32 || rows_lines(n) != (n + 63ll) / 64) ++bad;
    if (tiles_of(n, 128) != (n + 127ll) / 128) ++bad;
  }
  std::printf("%d\n", bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_positions_along_k_near_the_size_limit(tmp_path):
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    csrc = os.path.join(os.path.dirname(tcbuild.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-Wall", "-Wextra", "-Werror", "-I", csrc, str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_the_walk_finds_a_signed_position(tmp_path):
    """The same walk with 32-bit signed positions runs past the end."""
    csrc = os.path.join(os.path.dirname(tcbuild.__file__), "csrc")
    text = open(os.path.join(csrc, "linear_rows.h"), encoding="utf-8").read()
    assert "using RowsK = uint32_t;" in text
    (tmp_path / "linear_rows.h").write_text(text.replace("using RowsK = uint32_t;", "using RowsK = int32_t;"))
    src, exe = tmp_path / "walk.cpp", tmp_path / "walk"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", "-I", str(tmp_path), str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, timeout=120).returncode != 0
