"""How the own rows of a shared-prefix decode are cut into ranges
(csrc/own_cut.h, on the host): every tile is in one range, whatever part of the
list the early CTAs take, and a row's partials fit their slots."""

import subprocess

import pytest

from gqa_attention_kv_decode_gb300 import build

PROGRAM = r"""
#include <algorithm>
#include <cstdio>
#include <random>
#include <vector>
#include "own_cut.h"
using namespace gqa;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s (N %u head %u early %u late %u min %u)\n", __LINE__, #x, N, head, early, late, min_tiles); return 1; } } while (0)

int main() {
  std::mt19937 rng(SEED);
  auto upto = [&](unsigned n) { return unsigned(rng() % (n + 1)); };
  for (int n = 0; n < 4000; ++n) {
    // some units of leading and key tiles, the longest of which leaves the ranges their least size
    std::vector<unsigned> units(1 + upto(60));
    const unsigned longest = 1 + upto(n % 3 ? 40 : 3000), capacity = longest + upto(n % 2 ? 5000 : 0);
    unsigned N = 0, most = 1;
    for (unsigned& u : units) u = upto(longest), most = std::max(most, u), N += u ? u + 1 : 0;
    unsigned early = 9 * upto(152), late = 9 * (152 - early / 9), head = 0, min_tiles = 1;
    if (n % 7 == 0) early = 0, late = 1368;
    if (n % 7 == 1) late = 0, early = 1368;
    // slots and least size as own_rows_plan and own_rows have them
    const int cap_min = std::max(1, int(capacity + 31) / 32);
    const int slots = capacity < 2 ? 1 : int(capacity - 2) / cap_min + 3;
    min_tiles = most < 2 ? 1 : (most - 2) / unsigned(slots - 2) + 1;
    // (any number will do: what is estimated for it decides the time alone)
    head = early == 0 ? 0 : late == 0 ? N : n % 5 == 0 ? N : upto(N);
    const unsigned asked = n % 11 == 0 && head == N ? N + 17 : head;  // never past the list
    const OwnCut c = OwnCut::of(N, asked, early, late, min_tiles);
    CHECK(c.head == head);
    CHECK(c.a.n <= std::max(early, 1u) && c.b.n <= std::max(late, 1u));
    std::vector<int> owner(N, -1);
    int next = 0;
    for (int part = 0; part < 2; ++part) {
      const OwnRanges& r = part ? c.b : c.a;
      const unsigned base = part ? c.head : 0, size = part ? N - c.head : c.head;
      CHECK(r.start(0) == 0 && r.start(r.n) == size);
      if (part == 0 && size == 0) continue;  // (its one range, without tiles, is not counted)
      for (unsigned w = 0; w < r.n; ++w, ++next)
        for (unsigned x = r.start(w); x < r.start(w + 1); ++x) {
          CHECK(owner[base + x] == -1);
          owner[base + x] = next;
        }
    }
    for (unsigned x = 0; x < N; ++x) CHECK(owner[x] >= 0 && c.holder(x) == owner[x]);
    unsigned x = 0;
    for (unsigned u : units) {
      if (u == 0) continue;
      CHECK(owner[x + u] - owner[x + 1] + 1 <= slots);
      x += u + 1;
    }
  }
  std::printf("ok\n");
  return 0;
}
"""


@pytest.mark.parametrize("seed", [1, 2, 3])
def test_every_tile_is_in_one_range(tmp_path, seed):
    src, exe = tmp_path / "cut.cpp", tmp_path / "cut"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-DSEED={seed}", "-I", build.CSRC, str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert (out.returncode, out.stdout.strip()) == (0, "ok")
