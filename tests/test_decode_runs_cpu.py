"""Runs of whole strips (csrc/paged.cuh: run_blocks), compiled for the host: a worker's walk over a unit's blocks, as the one-token attention's kernel
makes it, with and without runs, over all small ranges, for every number of warps and both strip lengths the kernel has; and the walk over key ranges
with first keys for 16 warps."""
import os
import subprocess

from test_more_serving_cpu import MAIN

HERE = os.path.dirname(os.path.abspath(__file__))

RUNS = r"""
#include <algorithm>
#include <cstdio>
#include <vector>
#include "%s/../flexible_mask_flashattention_gb300/csrc/paged.cuh"
using namespace ffa;
static int fails = 0;
struct At { int left, key; };
int main() {
  const int stages = 2;
  long long in_runs = 0;
  for (int strip : {16, 32})
    for (int warps : {8, 12, 16}) {
      const int block = strip * warps;
      for (int len = 0; len <= 12 * block; len += 1 + len / 5)
        for (int start : {0, 1, strip - 1, strip, block - 1, block + 5, 3 * block + 7, len - 1})
          for (int first : {0, 1, strip, strip + 3, 2 * block})
            for (int turn : {0, 1, warps / 2, warps - 1}) {
              const KeyRange r = key_range(len, start, first, 1 << 20, 6, strip);
              const int blocks = static_cast<int>(range_blocks(r, block, strip)), end = static_cast<int>(r.end), from = static_cast<int>(r.start);
              auto open = [&](int blk) { return At{blocks - blk, std::min(static_cast<int>(range_first(r, strip)) + (blk * warps + turn) * strip, end)}; };
              auto step = [&](At& a) { --a.left, a.key = end - a.key > block ? a.key + block : end; };
              auto whole = [&](int key) { return end - key >= strip && key >= from; };
              for (int t0 = 0; t0 < blocks; t0 += 1 + blocks / 3)
                for (int more : {0, 1, 5, -1, -3}) {   // blocks of later units in the worker's share, or of this one that are the next worker's
                  if (blocks - t0 + more < 1) continue;
                  At cur = open(t0), ld = cur;
                  int64_t todo = blocks - t0 + more;
                  if (ld.left > 1 && todo > 1) step(ld); else continue;   // the loads are a block ahead, in the same unit
                  std::vector<int> got, want;
                  for (int b = t0; b < blocks + std::min(more, 0); ++b) want.push_back(open(b).key);
                  bool same_unit = true;
                  for (;;) {
                    int run = 0;
                    if (cur.left < blocks - t0 && cur.left > 2 && same_unit)
                      run = run_blocks(from, end, cur.key, cur.left, ld.key, ld.left, todo, block, strip, stages);
                    for (int i = 0; i < run; ++i) {
                      ++in_runs;
                      if (!whole(cur.key) || !whole(ld.key)) ++fails, std::printf("a strip of a run is not whole\n");
                      if (todo - i <= stages - 1) ++fails, std::printf("a load behind the share\n");
                      got.push_back(cur.key);
                      cur.key += block, ld.key += block, --ld.left;
                      if (!whole(ld.key)) ++fails, std::printf("a page is looked up for a strip that is not whole\n");
                      if (key_of(ld.key, r.first, static_cast<int>(r.gap)) + strip > len) ++fails, std::printf("behind the length\n");
                    }
                    if (run > 0) cur.left -= run, todo -= run;
                    if (cur.left < 1 || ld.left < 1 || cur.key != open(blocks - cur.left).key) ++fails, std::printf("a run ends at another block\n");
                    got.push_back(cur.key);
                    if (cur.left == 1 || todo == 1) break;
                    if (todo > stages && ld.left > 1) step(ld); else same_unit = same_unit && ld.left > 1;   // the share's last load leaves the walk where it is
                    step(cur), --todo;
                  }
                  if (got != want) ++fails, std::printf("strip %%d warps %%d len %%d start %%d first %%d turn %%d from %%d: other strips\n", strip, warps, len, start, first, turn, t0);
                  if (fails > 20) return 1;
                }
            }
    }
  std::printf("%%lld blocks in runs, %%d failures\n", in_runs, fails);
  return fails != 0 || in_runs == 0;
}
"""


def build_and_run(tmp_path, source):
    src, exe = tmp_path / "walk.cpp", str(tmp_path / "walk")
    src.write_text(source)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-1500:]


def test_runs_are_whole_strips_inside_the_range(tmp_path):
    build_and_run(tmp_path, RUNS % HERE)


def test_ranges_with_first_keys_for_16_warps(tmp_path):
    assert "warps : {8, 12}" in MAIN
    build_and_run(tmp_path, MAIN.replace("warps : {8, 12}", "warps : {16}") % HERE)
