"""The launch of the MXFP4 tile kernel holds every tile that the kernel makes.

mxfp4_tiles.hpp, which both the launch and the kernel include, is compiled for
the host and swept: for every number of row tiles up to the launch's bound, the
kernel's tiles fit the workgroups, rounded up to a multiple of the 8 XCDs, of
which each takes an equal share.
"""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "combine_moe_route_topk_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "mxfp4_tiles.hpp"
using namespace moe::big;
int main() {
  long long checked = 0, tight = 0;
  for (int glu = 0; glu < 2; ++glu)
    for (int any = 0; any < 2; ++any)
      for (int64_t n = 1; n <= 40000; n += n < 700 ? 1 : 127)
        for (int64_t most = 1; most <= 400; most += most < 140 ? 1 : 13) {
          const int64_t blocks = (blocks_for(most, n, glu, any) + 7) / 8 * 8;
          int64_t largest = 0;
          for (int64_t m = 0; m <= most; ++m) {
            // the definition, apart from the header's functions
            const int64_t cols = glu ? 128 : 256, wide = (n + cols - 1) / cols;
            const bool few = any && m * wide <= 128;
            const int64_t tiles = m * (few ? (n + cols / 2 - 1) / (cols / 2) : wide);
            if (tiles != tiles_of(m, n, glu, any) || (tiles + 7) / 8 > blocks / 8) {
              std::printf("glu %d any %d n %lld most %lld m %lld: %lld tiles, %lld workgroups\n", glu, any,
                          (long long)n, (long long)most, (long long)m, (long long)tiles, (long long)blocks);
              return 1;
            }
            if (tiles > largest) largest = tiles;
            ++checked;
          }
          tight += (largest + 7) / 8 * 8 == blocks;
          if ((largest + 7) / 8 * 8 != blocks) {
            std::printf("more workgroups than any number of tiles needs\n");
            return 1;
          }
        }
  std::printf("%lld %lld\n", checked, tight);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_every_tile_has_a_workgroup(tmp_path):
    src, exe = tmp_path / "tiles.cpp", tmp_path / "tiles"
    src.write_text(PROGRAM)
    subprocess.check_call(["g++", "-std=c++17", "-O2", "-I", CSRC, str(src), "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, out.stdout
    assert int(out.stdout.split()[0]) > 1_000_000
