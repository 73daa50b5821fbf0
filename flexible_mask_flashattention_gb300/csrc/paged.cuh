// Index arithmetic of the paged key-value cache, shared by its kernels and, compiled for the host, by its tests.  Nothing
// here reads device memory: what a kernel has read from a page table, a length or a slot list goes through these
// functions before it becomes an address, so that no such value reaches outside the cache.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define FFA_HD __host__ __device__ __forceinline__
#else
#define FFA_HD inline
#endif

namespace ffa {

// A cache [num_pages][hkv][page_size][d]; its exponent bytes are [num_pages][hkv][page_size].
struct PageGeom {
  int64_t num_pages;
  int32_t page_log2;   // page_size is a power of two, 16 at least
  int32_t hkv;
};

// Division of 0 <= n < 2^31 by a constant 1 <= d <= 2^22 as a product: n / d = floor(n m / 2^(31 + s)) with s = ceil(log2 d) and m =
// floor(2^(31 + s) / d) + 1, which is below 2^32.
struct FastDiv {
  uint32_t d, m;
  int32_t shift;   // s - 1; -1 for d = 1
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, -1};
  while ((uint64_t{1} << (f.shift + 1)) < d) ++f.shift;
  f.m = static_cast<uint32_t>((uint64_t{1} << (32 + f.shift)) / d + 1);
  return f;
}
FFA_HD uint32_t divide(const FastDiv& f, uint32_t n) {
  if (f.shift < 0) return n;
#ifdef __CUDA_ARCH__
  return __umulhi(n, f.m) >> f.shift;
#else
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * f.m) >> 32 >> f.shift);
#endif
}

// Row (page, head, offset) of the cache, counted in rows of d values.
FFA_HD int64_t cache_row(const PageGeom& g, int64_t page, int32_t head, int32_t off) {
  return ((page * g.hkv + head) << g.page_log2) + off;
}

// Is `page`, as a page table gives it, one of the cache's?
FFA_HD bool page_ok(const PageGeom& g, int64_t page) { return page >= 0 && page < g.num_pages; }

// Is `slot` (page * page_size + offset) one of the cache's?
FFA_HD bool slot_ok(const PageGeom& g, int64_t slot) { return slot >= 0 && (slot >> g.page_log2) < g.num_pages; }

// The keys [start, end) of one sequence that a one-token attention reads, and [0, first) beside them.  A start below 0 counts as 0; a
// range without a key is [0, 0), so that nothing is loaded for it; a length that the page table's row cannot hold is marked bad and
// reads no key.  Where first keys and a later range both have keys, the whole strips between them are left out: keys are then
// counted without those `gap` keys, start and end among them, and key k of that count is key k + gap from `first` rounded up to a
// strip on (key_of).  Otherwise first and gap are 0.
struct KeyRange {
  int64_t start, end;
  bool bad;
  int32_t first = 0;
  int64_t gap = 0;
};
FFA_HD KeyRange key_range(int32_t len, int32_t start, int64_t max_pages, int32_t page_log2) {
  KeyRange r;
  const int64_t cap = max_pages << page_log2;
  r.bad = len > cap;
  const bool some = !r.bad && len > 0 && start < len;
  r.end = some ? len : 0;
  r.start = some && start > 0 ? start : 0;
  return r;
}
FFA_HD KeyRange key_range(int32_t len, int32_t start, int32_t first, int64_t max_pages, int32_t page_log2, int32_t strip) {
  KeyRange r = key_range(len, start, max_pages, page_log2);
  if (r.bad || first <= 0 || len <= 0) return r;
  if (r.end == 0) {   // no key in the range: the first ones alone
    r.end = first < len ? first : len;
  } else if (first >= r.start) {
    r.start = 0;
  } else {
    const int64_t hop = (static_cast<int64_t>(first) + strip - 1) / strip * strip, lo = r.start / strip * strip;
    r.first = first;
    r.gap = lo > hop ? lo - hop : 0;
    r.start -= r.gap;
    r.end -= r.gap;
  }
  return r;
}

// The key that a strip's first counted key is.
template <typename I>
FFA_HD I key_of(I key, I first, I gap) { return key < first ? key : key + gap; }

// Blocks of `block` keys (a multiple of `strip`, itself one of 16) that cover the range.  Blocks are counted from the range's first key
// rounded down to `strip`, so that a strip's groups of 16 keys never cross a page.  An empty range has one block, which
// writes its empty row.
// Keys are numbers of 31 bits, so that 32 do for the divisions.
FFA_HD uint32_t range_first(const KeyRange& r, uint32_t strip) { return r.first > 0 ? 0 : static_cast<uint32_t>(r.start) / strip * strip; }
FFA_HD int64_t range_blocks(const KeyRange& r, uint32_t block, uint32_t strip) {
  const uint32_t n = (static_cast<uint32_t>(r.end) - range_first(r, strip) + block - 1) / block;
  return n > 0 ? n : 1;
}

// Blocks of a run, <= 0 for none: those from the current one on whose strips, a warp's own (first key `key`, `left` blocks of the unit from it on) and the one that
// is being loaded meanwhile (`ahead`, `ahead_left`; of the same unit, not before it), are whole ones of the range, none of them in the unit's last block nor in
// the last `stages` of the worker's `todo`.  Their walks need no more than a counter: every strip of a run, and the one that the loads then stand at, whose
// page is looked up, lies inside [start, end).
FFA_HD int32_t run_blocks(int32_t start, int32_t end, int32_t key, int32_t left, int32_t ahead, int32_t ahead_left, int64_t todo, int32_t block,
                          int32_t strip, int32_t stages) {
  if (key < start) return 0;
  const int32_t here = (left < ahead_left ? left : ahead_left) - 1, whole = (end - ahead - strip) / block, most = here < whole ? here : whole;
  return static_cast<int32_t>(most < todo - stages ? most : todo - stages);
}

// `total` blocks are dealt to `parts` (4096 at most) workers in equal contiguous shares: worker c has [share_begin(c),
// share_begin(c + 1)).  Few enough blocks take 32-bit divisions, a fifth of the 64-bit ones' time.
FFA_HD int64_t share_begin(int64_t total, int64_t parts, int64_t c) {
  if (total < (int64_t{1} << 19)) return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(parts);
  return total * c / parts;
}
// The worker whose share holds block x.
FFA_HD int64_t share_of(int64_t total, int64_t parts, int64_t x) {
  if (total < (int64_t{1} << 19)) return ((static_cast<uint32_t>(x) + 1) * static_cast<uint32_t>(parts) - 1) / static_cast<uint32_t>(total);
  return ((x + 1) * parts - 1) / total;
}

// 16-byte chunk of a 16-key strip in shared memory: row `key` (0..15), chunk c of `cpr` a row.  Both ways a warp reads
// the strip then touch every bank once: 8 lanes reading 4 neighbouring chunks of rows 2i, 2i + 1 (keys as matrix
// rows), and 8 lanes reading chunks 2i, 2i + 1 of rows 0, 2, 4, 6 or 1, 3, 5, 7 (keys as the contraction).
FFA_HD int32_t strip_chunk(int32_t key, int32_t c, int32_t cpr) {
  if (cpr >= 8) return key * cpr + (c ^ ((((key >> 1) & 3) ^ ((key & 1) << 1)) << 1));
  if (cpr == 2) return (key >> 2) * 8 + (((key ^ (key >> 2 & 1)) & 3) << 1) + c;   // four rows a line, read in 8- and 4-byte pieces
  const int32_t line = key >> 1;   // 4 chunks a row: two rows a 128-byte line
  return line * 8 + ((((key & 1) << 2) | c) ^ ((line & 3) << 1));
}

// A lane's chunks lane + 32 i lie 512 bytes apart in a strip as the cache has it, and 512 * period apart, every `period` of them, as
// shared memory has it: chunk i is at that of chunk i % period plus (i / period) * period * 512 bytes.
FFA_HD constexpr int32_t strip_period(int32_t cpr) { return cpr == 16 ? 4 : cpr == 8 ? 2 : 1; }

}  // namespace ffa
