"""The result lanes of skinny.h's tiles, walked on the host over every lane,
number of tokens and turn: the header's own functions, compiled without a
device pass.  A lane that a tile holds reads the columns of its token inside
its row group, no column serves two lanes, and every token's sums are stored
by exactly one lane of one turn."""
import os
import subprocess

import pytest

from sparse_expert_routing_sigmoid_amd import build as B

SOURCE = r"""
#include <cstdio>
#include "skinny.h"
using namespace moe;

template <typename S, bool PK>
int walk(const char* name) {
  for (int toks = 1; toks <= MOE_FEW_TOKENS; ++toks) {
    int stored[4][MOE_FEW_TOKENS] = {};
    for (int j0 = 0; j0 < toks; j0 += S::TOKENS) {
      int used[64] = {};
      for (int lane = 0; lane < 64; ++lane) {
        if (!S::holds(lane, j0, toks)) continue;
        const int group = lane >> 4, columns = PK ? S::XV : 1, at = PK ? sk_packed_at<S::XV>(lane) : lane;
        for (int i = at; i < at + columns; ++i)
          if (i >> 4 != group || used[i]++) {
            printf("%s: toks %d, j0 %d, lane %d reads column %d\n", name, toks, j0, lane, i);
            return 1;
          }
        ++stored[group][j0 + (lane & 15)];
      }
    }
    for (int g = 0; g < 4; ++g)
      for (int t = 0; t < toks; ++t)
        if (stored[g][t] != 1) {
          printf("%s: toks %d, token %d stored %d times\n", name, toks, t, stored[g][t]);
          return 1;
        }
  }
  return 0;
}

int main() {
  return walk<Skinny<MOE_F32, float, 2, 1>, false>("f32") + walk<Skinny<MOE_BF16, uint16_t, 2, 1>, false>("bf16") +
         walk<Skinny<MOE_E4M3, uint16_t, 2, 1>, false>("e4m3") + walk<Skinny<MOE_E2M1, uint16_t, 2, 1>, false>("e2m1") +
         walk<Skinny<MOE_E4M3, uint16_t, 2, 1, false, true>, true>("e4m3 packed") +
         walk<Skinny<MOE_E2M1, uint16_t, 2, 1, false, true>, true>("e2m1 packed") +
         walk<Skinny<MOE_E2M1, uint16_t, 2, 1, true, true>, true>("e2m1 packed, vector scales");
}
"""


def test_tiles_store_each_token_once_and_read_within_their_row_group(tmp_path):
    try:
        hipcc = B.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    src, out = tmp_path / "tiles.hip", tmp_path / "tiles"
    src.write_text(SOURCE)
    done = subprocess.run([hipcc, "--offload-host-only", "-std=c++17", "-O1", "-w", "-I", B.INCLUDE, "-I", B.CSRC,
                           str(src), "-o", str(out)], capture_output=True, text=True)
    assert done.returncode == 0, done.stderr
    done = subprocess.run([str(out)], capture_output=True, text=True, env={**os.environ, "HIP_VISIBLE_DEVICES": ""})
    assert done.returncode == 0, done.stdout
