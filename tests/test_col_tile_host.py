"""Where the column tiles' loads read (csrc/col_geom.h), enumerated on the host: every lane of every
load, steps past the end among them, lies inside the matrix or out of the descriptor's range, and what
is valid is read from its place."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "grouped_gemm_moonep_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "col_geom.h"
using namespace moonep;

// One tile: `regions` regions of COLS columns from column n0 of a [T][ld] matrix.  Returns the number
// of wrong loads.
template <int COLS, int WAVES>
static int tile(int regions, int64_t ld, int64_t T, int64_t n0) {
  typedef ColGeom<COLS, WAVES> G;
  int bad = 0;
  const uint32_t ld2 = (uint32_t)(ld * 2);
  const int64_t end = T * ld * 2, steps = (T + 63) / 64;
  for (int w = 0; w < WAVES * regions; ++w) {
    const int64_t c0 = n0 + w / WAVES * COLS;
    const int nv = (int)(ld - c0 < 0 ? 0 : ld - c0 < COLS ? ld - c0 : COLS);
    const int64_t range = G::bytes(ld2, (int)T, nv);
    bad += nv > 0 && T > 0 && c0 * 2 + range > end;
    for (int lane = 0; lane < 64; ++lane) {
      const int k = 64 / WAVES * (w % WAVES) + lane / G::kLanes;
      const int col = 8 * ((lane % G::kLanes) ^ G::swz(k));
      const uint32_t voff = G::lane(w, lane, ld2, nv);
      for (int64_t s = 0; s <= steps; ++s)
        for (int i = 0; i < G::kLoads; ++i) {
          // s == steps: a step past the end
          const uint32_t off = G::load(voff, s < steps ? (uint32_t)(s * 64 * ld2) : kOob, i, ld2);
          const int64_t row = s * 64 + k + G::kRows * i;
          const bool in = (int64_t)off + 16 <= range, part = (int64_t)off < range && !in;
          const bool want = s < steps && row < T && col < nv;
          if (part || (in && c0 * 2 + off + 16 > end)) ++bad;
          if (want && (!in || off != (uint32_t)((row * ld + col) * 2))) ++bad;
          // a step that counts reads zeros outside the matrix's rows and the region's columns
          if (!want && s < steps && in) ++bad;
        }
    }
  }
  return bad;
}

int main() {
  const int64_t lds[] = {64, 128, 192, 256, 320, 384, 448, 832, 2880};
  for (int64_t ld : lds)
    for (int64_t T = 0; T <= 130; ++T)
      for (int64_t n0 = 0; n0 < ld; n0 += 64) {
        const int bad[] = {tile<64, 2>(2, ld, T, n0), tile<128, 2>(2, ld, T, n0),
                           tile<128, 4>(2, ld, T, n0), tile<128, 8>(1, ld, T, n0)};
        for (int g = 0; g < 4; ++g)
          if (bad[g]) {
            printf("geometry %d: %d wrong loads of a %lld x %lld matrix from column %lld\n", g, bad[g],
                   (long long)T, (long long)ld, (long long)n0);
            return 1;
          }
      }
  // the largest matrix: offsets up to 2^31
  if (tile<128, 2>(2, 65536, 16383, 65408) || tile<64, 2>(2, 65536, 16383, 65472)) {
    printf("offsets near 2^31\n");
    return 1;
  }
  printf("ok\n");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_no_load_reads_past_the_matrix(tmp_path):
    src, exe = tmp_path / "col.cpp", tmp_path / "col"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", CSRC, str(src), "-o",
                    str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
