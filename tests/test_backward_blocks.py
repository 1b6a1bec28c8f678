"""Which blocks a tile of the backward pass visits: csrc/bwd_blocks.h compiled for the
host, against the pairs that the mask leaves, and the start of every part of a split
list against a walk from the front."""
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "scaled_dot_product_13_b200" / "csrc"

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "bwd_blocks.h"
using namespace sdpa;
struct Params { int L, S, R, off, causal, window; };
static long cases = 0, seeks = 0;
#define EXPECT(x) do { if (!(x)) { printf("%s: L=%d S=%d R=%d off=%d causal=%d window=%d x0=%d BN=%d\n", #x, \
    a.L, a.S, a.R, a.off, a.causal, a.window, x0, BN); exit(1); } } while (0)

static bool sees(const Params &a, int row, int key) {
  const long long at = (long long)(row % a.L) + a.off;
  return !a.causal || (key <= at && (a.window == 0 || at - key < a.window));
}

template <bool KEYS, int BN> void check(const Params &a, int x0) {
  const int xs = KEYS ? a.S : a.R, ys = KEYS ? a.R : a.S;
  std::vector<int> want(ys, 0);  // Y rows that some X row of the tile sees
  for (int y = 0; y < ys; ++y)
    for (int x = x0; x < x0 + 128 && x < xs && !want[y]; ++x) want[y] = KEYS ? sees(a, y, x) : sees(a, x, y);
  std::vector<BwdBlocks<KEYS, BN>> at;
  std::vector<int> visited;
  BwdBlocks<KEYS, BN> w = bwd_blocks<KEYS, BN>(a, x0);
  for (int b = w.at_or_after(w.first); b >= 0; b = w.at_or_after(b + 1)) {
    EXPECT(visited.empty() || b > visited.back());
    EXPECT((long long)b * BN < ys);
    visited.push_back(b);
    at.push_back(w);
    if (KEYS) EXPECT(w.query(b * BN) == b * BN % a.L);
  }
  for (int b = 0, i = 0; b * BN < ys; ++b) {
    bool any = false;
    for (int y = b * BN; y < ys && y < (b + 1) * BN; ++y) any |= want[y] != 0;
    const bool is = i < (int)visited.size() && visited[i] == b;
    i += is;
    EXPECT(is || !any);         // no pair is left out
    if (KEYS) EXPECT(any || !is);  // and no block visited for nothing
  }
  const int n = (int)visited.size();
  for (int k = 0; k <= n + 1; ++k, ++seeks) {
    BwdBlocks<KEYS, BN> s = bwd_blocks<KEYS, BN>(a, x0);
    int total = -1;
    const int b = s.seek(k, total);
    EXPECT(total == n);
    EXPECT(b == (k < n ? visited[k] : -1));
    if (b < 0) continue;
    if (KEYS) EXPECT(s.lo == at[k].lo && s.hi == at[k].hi && s.base == at[k].base);
    const int next = s.at_or_after(b + 1);
    EXPECT(next == (k + 1 < n ? visited[k + 1] : -1));
  }
  ++cases;
}

int main() {
  for (int L : {1, 2, 3, 31, 32, 47, 48, 49, 64, 95, 96, 97, 130, 200, 300})
    for (int g : {1, 2, 3, 7, 40})
      for (int S : {1, 5, 64, 128, 129, 260, 400})
        for (int mask = 0; mask < 12; ++mask) {
          Params a = {L, S, g * L, S - L, mask > 0, 0};
          if (mask >= 4) a.window = mask % 4 == 0 ? 1 : mask % 4 == 1 ? 20 : mask % 4 == 2 ? 128 : 1 << 30;
          if (mask >= 8) a.off = S / 3; else if (mask == 2) a.off = 0; else if (mask == 3) a.off = S + 50;
          if (a.causal && a.off < 0) continue;
          if (a.window > 0 && (long long)a.off + L - a.window > S - 1) continue;
          if ((long long)a.R * S > 400000) continue;
          for (int x0 = 0; x0 < S; x0 += 128) {
            check<true, 32>(a, x0); check<true, 48>(a, x0); check<true, 64>(a, x0);
            check<true, 80>(a, x0); check<true, 96>(a, x0);
          }
          for (int x0 = 0; x0 < a.R; x0 += 128) {
            check<false, 32>(a, x0); check<false, 64>(a, x0); check<false, 80>(a, x0); check<false, 96>(a, x0);
          }
        }
  // the largest sizes: no product or sum leaves 32 bits
  for (int L : {1, 1 << 20, 1 << 30}) {
    Params a = {L, 1 << 30, 1 << 30, (1 << 30) - L, 1, 0};
    const int x0 = 0, BN = 96;
    BwdBlocks<true, 96> w = bwd_blocks<true, 96>(a, x0);
    int total;
    const int last = ((1 << 30) + 95) / 96 - 1;
    EXPECT(w.seek(last, total) == last && total == last + 1);
    EXPECT(w.query(last * 96) == last * 96 % L);
    EXPECT(w.at_or_after(last + 1) == -1);
  }
  printf("%ld cases, %ld parts\n", cases, seeks);
}
"""


def test_blocks_and_where_parts_begin(tmp_path):
    compiler = shutil.which("g++") or shutil.which("c++")
    if compiler is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "blocks.cpp", tmp_path / "blocks"
    src.write_text(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-O2", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover", "-I", str(CSRC),
                    str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout.split()[0]) > 10000, r.stdout
    print(r.stdout)


def test_the_kernel_takes_the_parts_from_it():
    """Each part's start and the length of the list come from seek: a walk over the
    blocks before it makes the last part's start as long as the whole list."""
    text = (CSRC / "bwd_tc.cuh").read_text()
    assert "walk.seek(split * span.per, total)" in text
    assert text.count("at_or_after(") == 2  # the first block, and the next
