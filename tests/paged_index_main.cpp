// Host build of the paged cache's index arithmetic (csrc/paged.cuh) for tests/test_serving_cpu.py: walks what the
// kernels walk and prints one line a finding.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <vector>

#include "../flexible_mask_flashattention_gb300/csrc/paged.cuh"

using namespace ffa;

static int fails = 0;
#define CHECK(c, ...) do { if (!(c)) { std::printf("FAIL %s: ", #c); std::printf(__VA_ARGS__); std::printf("\n"); ++fails; } } while (0)

static uint64_t state = 1;
static int64_t rnd(int64_t n) { state = state * 6364136223846793005ull + 1442695040888963407ull; return static_cast<int64_t>((state >> 33) % static_cast<uint64_t>(n)); }

// Every group of 16 keys that a strip of any block reads lies in the page that its first key names, inside the cache, and in
// range; every key of the range is read once.
static void walk(int page_log2, int hkv, int64_t num_pages, int max_pages, int32_t len, int32_t start, int warps, int groups) {
  const PageGeom g{num_pages, page_log2, hkv};
  const int strip = 16 * groups, block = strip * warps;
  const KeyRange r = key_range(len, start, max_pages, page_log2);
  const int64_t cap = static_cast<int64_t>(max_pages) << page_log2;
  CHECK(r.bad == (len > cap), "len %d cap %lld", len, static_cast<long long>(cap));
  CHECK(r.start >= 0 && r.start <= r.end && r.end <= cap, "range");
  std::vector<int> seen(static_cast<size_t>(r.end), 0);
  const int64_t n = range_blocks(r, block, strip);
  CHECK(n >= 1, "blocks");
  for (int64_t b = 0; b < n; ++b)
    for (int w = 0; w < warps; ++w)
      for (int i = 0; i < groups; ++i) {
        const int64_t key0 = range_first(r, strip) + (b * warps + w) * strip + 16 * i, have = r.end - key0;
        if (have <= 0 || r.start - key0 >= 16) continue;   // no key of the range: nothing is read, its page not looked up
        const int64_t entry = key0 >> page_log2;
        CHECK(entry >= (r.start >> page_log2) && entry < max_pages, "table entry %lld", static_cast<long long>(entry));
        const int off = static_cast<int>(key0 & ((1 << page_log2) - 1));
        CHECK(off % 16 == 0 && off + 16 <= (1 << page_log2), "a group crosses its page");
        const int lo = static_cast<int>(r.start > key0 ? r.start - key0 : 0), hi = static_cast<int>(have < 16 ? have : 16);
        for (int j = lo; j < hi; ++j) ++seen[static_cast<size_t>(key0 + j)];
        for (int64_t page : {int64_t{0}, num_pages - 1})
          for (int h : {0, hkv - 1}) {
            const int64_t row = cache_row(g, page, h, off);
            CHECK(page_ok(g, page) && row >= 0 && row + 16 <= (num_pages * hkv << page_log2), "row out of the cache");
            CHECK(row % 16 == 0, "exponent bytes are read 16 at a time");
          }
      }
  for (int64_t j = 0; j < r.end; ++j) CHECK(seen[static_cast<size_t>(j)] == (j >= r.start), "key %lld", static_cast<long long>(j));
}

int main() {
  for (int i = 0; i < 4000; ++i) {
    const int pl = 4 + static_cast<int>(rnd(5)), mp = static_cast<int>(rnd(9));
    const int cap = mp << pl;
    const int32_t len = i % 7 == 0 ? cap : static_cast<int32_t>(rnd(cap + 40)) - 10;
    const int32_t start = i % 3 == 0 ? 0 : static_cast<int32_t>(rnd(cap + 40)) - 10;
    walk(pl, 1 + static_cast<int>(rnd(4)), 1 + rnd(20), mp, len, start, i % 2 ? 8 : 12, 1 << (i / 2 % 3));
  }
  walk(4, 2, 3, 2, 2147483647, 0, 8, 2);
  walk(4, 2, 3, 2, -2147483647 - 1, 5, 8, 1);
  walk(10, 2, 3, 5, 4999, 2147483647, 16, 4);
  // pages and slots as a user's arrays may hold them
  const PageGeom g{7, 5, 3};
  for (int64_t p : {int64_t{-1}, int64_t{7}, int64_t{2147483647}, int64_t{-2147483648LL}}) CHECK(!page_ok(g, p), "page %lld", static_cast<long long>(p));
  for (int64_t s : {int64_t{-1}, int64_t{7 * 32}, INT64_MAX, INT64_MIN}) CHECK(!slot_ok(g, s), "slot %lld", static_cast<long long>(s));
  CHECK(slot_ok(g, 7 * 32 - 1) && slot_ok(g, 0) && page_ok(g, 6), "the cache's own");
  // rows past 32 bits
  CHECK(cache_row(PageGeom{int64_t{1} << 27, 6, 8}, (int64_t{1} << 27) - 1, 7, 63) == (int64_t{1} << 36) - 1, "64-bit rows");
  // the shares: contiguous, complete, never empty where parts <= total; share_of is their inverse
  for (int i = 0; i < 3000; ++i) {
    const int64_t total = 1 + rnd(i % 2 ? 400 : 100000), most = 1 + rnd(4096), parts = most < total ? most : total;
    CHECK(share_begin(total, parts, 0) == 0 && share_begin(total, parts, parts) == total, "ends");
    for (int64_t c = 0; c < parts; ++c) {
      const int64_t a = share_begin(total, parts, c), b = share_begin(total, parts, c + 1);
      CHECK(a < b, "an empty share");
      CHECK(share_of(total, parts, a) == c && share_of(total, parts, b - 1) == c, "share_of");
    }
  }
  for (int i = 0; i < 3000; ++i) {   // around the border of the 32-bit form, and far behind it
    const int64_t total = i % 2 ? (int64_t{1} << 19) - 3 + rnd(6) : (int64_t{1} << 19) + (rnd(1 << 30) << (i % 13));
    const int64_t parts = 1 + rnd(4096);
    for (int64_t c : {int64_t{0}, rnd(parts), parts - 1}) {
      const int64_t a = share_begin(total, parts, c), b = share_begin(total, parts, c + 1);
      CHECK(a == static_cast<int64_t>(static_cast<__int128>(total) * c / parts), "share_begin");
      CHECK(a < b && share_of(total, parts, a) == c && share_of(total, parts, b - 1) == c, "share_of, total %lld", static_cast<long long>(total));
    }
  }
  for (uint32_t d : {1u, 2u, 3u, 5u, 7u, 8u, 31u, 32u, 33u, 96u, 1000u, 4095u, 4096u, 4097u, 65536u, 4194303u, 4194304u}) {
    const FastDiv f = fast_div(d);
    for (int i = 0; i < 4000; ++i) {
      const uint32_t n = i < 1000 ? static_cast<uint32_t>(i) : i < 2000 ? 2147483647u - static_cast<uint32_t>(i - 1000) : static_cast<uint32_t>(rnd(2147483648LL));
      CHECK(divide(f, n) == n / d, "%u / %u", n, d);
      const uint32_t k = n / d * d;   // around multiples
      CHECK(divide(f, k) == k / d && (k == 0 || divide(f, k - 1) == (k - 1) / d), "%u / %u", k, d);
    }
  }
  // a strip's chunks: a permutation of its 16-byte places, and no bank conflict in either read pattern
  for (int cpr : {4, 8, 16}) {
    std::set<int> all;
    for (int key = 0; key < 16; ++key)
      for (int c = 0; c < cpr; ++c) all.insert(strip_chunk(key, c, cpr));
    CHECK(static_cast<int>(all.size()) == 16 * cpr && *all.begin() == 0 && *all.rbegin() == 16 * cpr - 1, "cpr %d", cpr);
    const int period = strip_period(cpr);
    for (int lane = 0; lane < 32; ++lane)
      for (int i = 0; i < cpr / 2; ++i) {
        const int j = i % period;
        CHECK(strip_chunk((lane + 32 * i) / cpr, (lane + 32 * i) % cpr, cpr) ==
                  strip_chunk((lane + 32 * j) / cpr, (lane + 32 * j) % cpr, cpr) + i / period * period * 32, "period, cpr %d", cpr);
      }
    for (int i = 0; i < 8; ++i)
      for (int h = 0; h < cpr / 4; ++h) {   // K: rows 2i, 2i + 1, chunks 4h .. 4h + 3
        std::set<int> banks;
        for (int k = 0; k < 2; ++k)
          for (int t = 0; t < 4; ++t) banks.insert(strip_chunk(2 * i + k, t + 4 * h, cpr) % 8);
        CHECK(banks.size() == 8, "K reads, cpr %d", cpr);
      }
    for (int o = 0; o < 4; ++o)             // V: rows 2t + (o & 1) + 8 (o >> 1), two neighbouring chunks
      for (int c = 0; c + 1 < cpr; c += 2) {
        std::set<int> banks;
        for (int t = 0; t < 4; ++t)
          for (int k = 0; k < 2; ++k) banks.insert(strip_chunk(2 * t + (o & 1) + 8 * (o >> 1), c + k, cpr) % 8);
        CHECK(banks.size() == 8, "V reads, cpr %d", cpr);
      }
  }
  std::printf("%d failures\n", fails);
  return fails != 0;
}
