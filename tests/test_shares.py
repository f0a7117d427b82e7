"""CPU checks of the launches' shares (csrc/shares.h) over all sizes, compiled by themselves."""

import os
import subprocess

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "split_kv_decode_bsr_gb300", "csrc")


def _run(tmp_path, body):
    """The output of a C++ program whose main is `body`."""
    src, exe = tmp_path / "check.cpp", tmp_path / "check"
    src.write_text('#include <cstdio>\n#include "shares.h"\nusing namespace sta;\nint main() {\n' + body + "\n}\n")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout


def test_the_backward_norms_have_a_row_of_scratch_for_each_cta(tmp_path):
    # pieces of a token: up to 128 query and 64 key heads, one a piece
    out = _run(tmp_path, """
  for (int most : {304, 152})
    for (int p = 0; p <= 128; ++p)
      for (int q = 0; q <= 64; ++q)
        for (long n : {1l, 2l, 5l, 79l, 80l, 81l, 200l, 8192l, 3000000000l}) {
          if (p + q == 0) continue;
          const int pieces[2] = {p, q};
          int c[2];
          norm_ctas(most, pieces, n, 8, c);
          const bool fits = c[0] + c[1] <= most;
          const bool each = (c[0] > 0) == (p > 0) && (c[1] > 0) == (q > 0);
          const bool busy = c[0] <= (n * p + 7) / 8 && c[1] <= (n * q + 7) / 8;
          const bool full = n < 8192 || c[0] + c[1] == most;
          if (!(fits && each && busy && full)) std::printf("%d: %d + %d pieces, %ld tokens: %d + %d\\n", most, p, q, n, c[0], c[1]);
        }
""")
    assert out == "", out[:400]


def test_a_warp_of_few_rows_has_read_a_stage_before_it_waits_for_the_next_tile_there(tmp_path):
    # a wait for phase n of a stage passes while phase n - 1 is still open: a warp may wait for tile t of the run only where it
    # has waited for tile t - stages itself. Each tile by one warp of a head, whatever the pieces' lengths.
    out = _run(tmp_path, """
  unsigned seed = 1;
  for (int d : {64, 128})
    for (int Hkv = 1; Hkv <= 12; ++Hkv) {
      const int turns = row_turns(Hkv), stages = row_stages(d, row_heads(Hkv));
      if (stages < 2 || stages * row_heads(Hkv) * d * 64 > kRowRing) std::printf("%d heads of %d: %d stages\\n", Hkv, d, stages);
      for (int round = 0; round < 200; ++round) {
        int by[4096] = {}, n = 0;  // warp of a tile, + 1
        for (int piece = 0; piece < 20 && n < 3000; ++piece) {
          seed = seed * 1664525u + 1013904223u;
          const int tiles = (seed >> 16) % (round % 3 ? 5 : 40);
          for (int turn = 0; turn < turns; ++turn)
            for (int i = row_first((unsigned)n, turn, turns); i < tiles; i += turns) {
              if (i < 0 || by[n + i]) std::printf("%d heads of %d: tile %d taken twice\\n", Hkv, d, n + i);
              by[n + i] = turn + 1;
            }
          n += tiles;
        }
        for (int t = 0; t < n; ++t) {
          if (!by[t]) std::printf("%d heads of %d: tile %d by none\\n", Hkv, d, t);
          if (t >= stages && by[t] != by[t - stages])
            std::printf("%d heads of %d: tile %d by warp %d, the one before it in its stage by %d\\n", Hkv, d, t, by[t], by[t - stages]);
        }
      }
    }
""")
    assert out == "", out[:400]
