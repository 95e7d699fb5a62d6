"""The join's check of a cut unit's entry (csrc/paged_cut.cuh), on the host:
entries that a chunk CTA never wrote may hold anything, and none may name a
request, head, unit or part that the call does not have."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sink_sliding_window_b200", "csrc")

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include <random>
#include "paged_cut.cuh"

// The tensors of a call, as the join addresses them with an entry; returns false on any index outside.
struct Call {
  int batch, heads, parts, cut, G, tokens, tiles, T, max_parts;
  int cu[6];
  int rows(int b) const { return cu[b + 1] - cu[b]; }
  int units(int b) const { return (rows(b) + tiles * tokens - 1) / (tiles * tokens); }
  bool inside(int i, int b, int group, int head, int n) const {
    if (b < 0 || b >= batch) return false;  // cu, kv_lens
    for (int k = 0; k < n; ++k)             // parts of the workspace
      if (static_cast<long long>(i) * n + k >= max_parts) return false;
    for (int row = 0; row < tiles * 128; ++row) {
      const int r = row & 127, t = r / G;
      const long long it = (static_cast<long long>(tiles) * group + (row >> 7)) * tokens + t;
      if (t >= tokens || it >= cu[b + 1] - cu[b]) continue;
      const long long h = static_cast<long long>(head) * G + r - t * G, at = cu[b] + it;
      if (it < 0 || at < 0 || at >= T || h < 0 || h >= heads * G) return false;
    }
    return true;
  }
};

int main() {
  const Call c = {5, 2, 3, 4, 8, 16, 2, 200, 12, {0, 70, 70, 71, 169, 200}};
  std::mt19937 rng(1);
  const int odd[] = {0, 1, 2, 3, 4, 5, 6, 31, 32, 33, 128, -1, -2, 1 << 24, 1 << 30, INT_MAX, INT_MIN, 0x5A5A5A5A, 0x7FC00000};
  long long taken = 0, refused = 0, wrong = 0, lost = 0;
  auto rows = [&](int b) {
    if (b < 0 || b >= c.batch) ++wrong;  // asked for a request that there is not
    return b >= 0 && b < c.batch ? c.rows(b) : 0;
  };
  for (int x = 0; x < 400000; ++x) {
    int e[4];
    for (int& v : e) v = rng() % 4 ? odd[rng() % (sizeof(odd) / sizeof(int))] : static_cast<int>(rng());
    const bool fits = sa::cut_unit_fits(e[0], e[1], e[2], e[3], c.batch, c.heads, c.parts, 32, rows);
    (fits ? taken : refused) += 1;
    if (fits && !c.inside(c.cut - 1, e[0], e[1], e[2], e[3])) ++wrong;
  }
  for (int b = 0; b < c.batch; ++b)
    for (int u = 0; u < c.units(b); ++u)
      for (int h = 0; h < c.heads; ++h)
        if (!sa::cut_unit_fits(b, u, h, c.parts, c.batch, c.heads, c.parts, 32, rows)) ++lost;
  std::printf("%lld %lld %lld %lld\n", taken, refused, wrong, lost);
}
"""


def test_entries_of_any_content(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not available")
    src, exe = tmp_path / "cut.cpp", tmp_path / "cut"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover", "-Wall", "-Werror", "-I", CSRC,
                    str(src), "-o", str(exe)], check=True)
    taken, refused, wrong, lost = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert taken > 20 and refused > 300000  # both kinds were met
    assert wrong == 0 and lost == 0


def test_the_join_asks_before_it_uses_an_entry():
    """In the kernel: nothing is made from an entry above the check."""
    text = open(os.path.join(CSRC, "paged_join.cuh")).read()
    body = text[text.index("void chunk_join("):]
    check = body.index("cut_unit_fits(")
    for use in ("paged_request(", "u.w;", "p.part_ml", "p.a.sinks"):
        assert body.index(use) > check, use
