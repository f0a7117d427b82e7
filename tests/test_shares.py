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
