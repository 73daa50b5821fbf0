"""Which page-table entries a one-token attention looks up, from the index arithmetic its kernel walks (csrc/paged.cuh, compiled for the
host): those that a key of the range lies in, and none for a range without a key."""
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))

MAIN = r"""
#include <cstdio>
#include <set>
#include "%s/../flexible_mask_flashattention_gb300/csrc/paged.cuh"
using namespace ffa;
int main() {
  int fails = 0;
  for (int page_log2 : {4, 5, 7})
    for (int strip : {16, 32})
      for (int warps : {8, 12})
        for (int len = -2; len <= 100; ++len)
          for (int start = -2; start <= 104; ++start) {
            const int max_pages = (100 >> page_log2) + 1, block = strip * warps;
            const KeyRange r = key_range(len, start, max_pages, page_log2);
            std::set<int64_t> want, got;
            for (int64_t j = start < 0 ? 0 : start; j < len; ++j) want.insert(j >> page_log2);
            for (int64_t i = 0; i < range_blocks(r, block, strip) * warps; ++i) {
              const int64_t first = range_first(r, strip) + i * strip, key = first < r.end ? first : r.end;   // a strip behind the end is empty
              if (r.end - key <= 0) continue;                                                                // nothing of it is loaded
              for (int g = 0; g < strip; g += 16)
                if (r.end - key > g && r.start - key < g + 16) got.insert((key + g) >> page_log2);
            }
            if (want.empty() && (r.start != 0 || r.end != 0)) ++fails, std::printf("len %%d start %%d: an empty range is [%%lld, %%lld)\n", len, start, (long long)r.start, (long long)r.end);
            if (want != got) ++fails, std::printf("len %%d start %%d page %%d strip %%d: other entries\n", len, start, 1 << page_log2, strip);
          }
  std::printf("%%d failures\n", fails);
  return fails != 0;
}
"""


def test_page_table_entries_that_are_looked_up(tmp_path):
    src, exe = tmp_path / "ranges.cpp", str(tmp_path / "ranges")
    src.write_text(MAIN % HERE)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-1500:]
