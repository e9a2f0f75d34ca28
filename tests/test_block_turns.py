"""How the waves of the balance kernels share a chunk of tokens (csrc/dg_turns.h), up to
the last token that a call may have, 2^31 - 2.  The walk runs in the host compiler's
constant evaluation, which refuses signed overflow."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_grouped_gemm_02_amd", "csrc")

SOURCE = """
#define __host__
#define __device__
#include "dg_turns.h"

// Every row of [from, to) once, by the wave that it belongs to, the next row known beforehand.
template <int WAVES>
constexpr bool walks(int from, int to) {
  long long rows = 0;
  for (int wave = 0; wave < WAVES; ++wave) {
    dg::Turns<WAVES> turn(from, to, wave);
    long long want = (long long)from + wave;
    if (turn.here() != (want < to)) return false;
    for (; turn.here(); turn.next()) {
      if (turn.row() != want) return false;
      want += WAVES;
      ++rows;
      if (turn.has_next() != (want < to)) return false;
      if (turn.has_next() && turn.next_row() != want) return false;
    }
    if (want < to) return false;
  }
  return rows == (long long)to - from;
}
template <int WAVES>
constexpr bool walks_everywhere() {
  constexpr int kEnd = 2147483647;
  for (int size = 0; size <= 3 * WAVES + 1; ++size)
    if (!walks<WAVES>(0, size) || !walks<WAVES>(5, 5 + size) || !walks<WAVES>(kEnd - size, kEnd) || !walks<WAVES>(kEnd - 9 - size, kEnd - 9)) return false;
  return true;
}
static_assert(walks_everywhere<16>(), "forward");
static_assert(walks_everywhere<4>(), "gradient");
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_every_token_has_its_turn(tmp_path):
    source = tmp_path / "turns.cpp"
    source.write_text(SOURCE)
    res = subprocess.run(["g++", "-std=c++17", "-fsyntax-only", "-fconstexpr-ops-limit=100000000", "-I", CSRC, str(source)],
                         capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stderr[-4000:]


def test_the_balance_kernels_count_tokens_this_way():
    """No loop over tokens of its own is left in them."""
    text = open(os.path.join(CSRC, "dg_balance.hip")).read()
    assert text.count("Turns<kSumWaves> turn(from, to, wave)") == 1 and text.count("Turns<kWaves> turn(from, to, wave)") == 1
    assert "from + wave" not in text and " t += k" not in text
