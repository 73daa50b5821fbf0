// Attention of one new token a sequence over the paged key-value cache, split over the cache's length and joined.
//
// For sequence b, q head h (kv head h / (hq / hkv)) and the keys j in [start_b, len_b):
//   s_j = scale q . k_j,  lse = ln(sum_j e^{s_j} [+ e^{sink_h}]),  out = sum_j e^{s_j - lse} v_j.
//
// Bound by HBM for groups (hq / hkv) of up to 8: every stored key and value is read once, 4 hq / hkv FLOPs a byte (e4m3) or half that (bf16),
// far under what the tensor cores need to be busy.  Groups above 8 take two query tiles a warp, whose registers leave two warps a
// scheduler, and a strip's chain of dependent instructions bounds them (no pipe is above 45 %); groups above 16 walk over the
// cache once for every 16 of their heads.  The design is about keeping loads in flight:
//   - The batch's keys are counted in blocks of a strip (16 or 32 keys) a warp; all (sequence, kv head) units' blocks form
//     one list, dealt to the CTAs, one an SM, in equal contiguous shares (paged.cuh: share_begin).  Ragged lengths and few
//     long sequences balance the same way, and no length has to be known on the host.
//   - A warp streams its own strips (K, V, exponent bytes) through a ring in shared memory with cp.async, across unit
//     borders, and never waits for another warp until a unit's part ends, nor then if the unit was one strip.
//   - Scores are computed transposed, S^T = K Q^T, with 16 keys as the rows and up to 8 q heads of the group as the
//     columns of mma.m16n8k16, and out^T = V^T P^T.  A group rarely has more than 8 heads, and this shape wastes
//     half of what 16 query rows would.  (tcgen05 wants 64 rows at least and its operands in shared
//     memory in their multiplied type; here the codes are widened on the way from shared memory to registers.)
//   - The contraction order of an MMA is free as long as both operands agree: a thread takes 16 consecutive bytes of a K
//     row as the contraction elements of several MMAs, and of V it owns whole column chunks, so both are read by
//     16-byte loads without a transposition; a byte permutation pairs two keys' values.
//
// Types.  bf16 cache: bf16 MMAs; P goes in as a bf16 value plus the bf16 value of its remainder, so that its rounding
// does not add to the output's.  e4m3 cache: codes are exact in f16; q is scaled by a power of two a row to f16's top range (its bf16
// mantissa fits; values below 2^-31 of the row's largest round); the scale of a key's row multiplies its score.  The scale 2^n of a
// value's row goes into its weight, as e^{s_j} 2^{n_j}, which each query has a running reference of its own for: what an f16 weight
// (11 bits) is relative to is the largest that has counted for this query, not the largest row there is.  Weights
// from 2^-24 of that on are rounded to 2^-11 of themselves, smaller ones by at most 2^-35 of it.  11 bits are enough here: the output's error
// against 64 bits is 1.673e-3 of its norm, and 1.661e-3 with a pair of f16 values, which the output's own rounding makes; the
// pair costs nothing at 64 x 16K keys, but 3 % at 32 x 1K, 4 to 5 % at d = 64 and 4 to 12 % in groups above 8.  Scores, maxima,
// sums and the output accumulate in fp32.
//
// Split parts go to the workspace as (m, l, O) and a second kernel joins them in a fixed order.
//
// Measured on the device (of the 6795 GB/s that a copy reaches; the range is that of several GPUs): 1M keys, 16 + 4 heads, d = 128, e4m3:
// 164 to 168 us (95 to 97 %); 64 x 16K keys, 64 + 8 heads, e4m3: 219 to 223 us (93 to 94 %); 24 x 8K keys with a window of 4096, 32
// heads, d = 64, bf16: 115 to 119 us (89 to 92 %), 113 with the products left out; 777 keys, bf16: 6.6 us.  Far from HBM's bound: groups of 16
// (380K keys, e4m3: 41.9 us, 69 %; 32 x 4K keys, d = 64, bf16: 18.7 us, 35 %), 48 heads over one kv head (1M keys, e4m3: 129 us,
// 31 %), and short sequences (32 x 1K keys, e4m3: 12.0 us, 25 %).
#include <cuda_bf16.h>

#include <algorithm>

#include "ffa_internal.h"
#include "kv_cache.h"
#include "launch.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace ffa {
namespace {

// Warps a CTA, and groups of 16 keys a strip.  Warps hide each other's latencies, as far as registers and the ring allow; longer strips
// spread a strip's fixed instructions over more keys.  Measured before later steps (us; 50 x 20K keys, 64 + 8 heads, d = 64, e4m3): 8 warps x 1 group 165,
// 8 x 2 137, 8 x 4 120, 12 x 4 118, 16 x 2 118, and later 12 x 2 114 and 16 x 2 116; (1M keys, 16 + 4 heads, d = 128, e4m3): 8 x 1 181, 12 x 1 170, 8 x 2 169; (24 x 8K
// keys, 32 heads, d = 64, bf16): 8 x 1 119, 8 x 2 122, 12 x 2 117; (380K keys, 32 + 2 heads, d = 128, e4m3): 8 x 1 46, 8 x 2 43.
constexpr int warps_of(int d, int nt) { return nt == 2 || d == 128 ? 8 : 12; }
constexpr int groups_of(int d, bool fp8) { return d == 128 && !fp8 ? 1 : 2; }
constexpr int kMaxCtas = 160;          // CTAs (one an SM) the workspace holds parts for: two a CTA
constexpr int kSmemMax = 226 * 1024;   // of 227 KB
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What a CTA leaves for the join: the unit that begins in its last part and goes on in later CTAs.
struct JoinDesc {
  int32_t parts;   // 0: none
  int32_t batch, unit;
  int32_t first_slot;
  int32_t pad[4];
};

struct DecodeParams {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const void* k;
  const void* v;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  PageGeom geom;
  const int32_t* table;
  int64_t table_stride;
  int32_t max_pages;
  int32_t batch, hq, group, subs;   // group = hq / hkv; subs = units a kv head (group / (8 NT) rounded up)
  const int32_t* lens;
  const int32_t* starts;
  float scale_log2;
  const float* sink;
  __nv_bfloat16* out;
  float* lse;
  JoinDesc* desc;     // [kMaxCtas]
  float2* ml;         // [2 kMaxCtas][8 NT]
  float* part;        // [2 kMaxCtas][8 NT][D]
};

template <int D, bool FP8, int NT>
struct Cfg {
  static constexpr int W = warps_of(D, NT);
  static constexpr int THREADS = 32 * W;
  static constexpr int SK = groups_of(D, FP8);
  static constexpr int KEYS = 16 * SK;                  // keys of a strip
  static constexpr int BLOCK = KEYS * W;                // keys of a block
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int ROW = D * ES;                    // bytes a stored row
  static constexpr int CPR = ROW / 16;                  // 16-byte chunks a row
  static constexpr int STRIP = 16 * ROW;                // bytes of 16 rows
  static constexpr int GROUP = 2 * STRIP + (FP8 ? 32 : 0);   // of 16 keys: K, V, exponents
  static constexpr int STAGE = SK * GROUP;
  static constexpr int JOIN = (W / 2) * 8 * NT * D * 4 + (W + 1) * 8 * NT * 8;   // O buffers; (m, l) of every warp, the rows' factors
  static constexpr int MISC = 1024;
  static constexpr int FIT = (kSmemMax - JOIN - MISC) / (W * STAGE);
  // Two stages, though three would fit e4m3 at d = 128 and groups over 8 at d = 64: more loads in flight are slower (e4m3, 64 x 16K keys
  // 219 and 224 us, 1M keys 164 and 169 us; 16 x 32K keys of 16-head groups, d = 64, bf16 37 and 39 us).  bf16 at d = 128 takes what
  // fits (777 keys 6.6 us with three and 6.8 with two, large batches alike).
  static constexpr int STAGES = FP8 || D == 64 ? 2 : FIT;
  static constexpr int SMEM = MISC + JOIN + W * STAGE * STAGES;
  static constexpr int KSTEPS = D / 16;
  static constexpr int MT = D / 16;                     // 16-column tiles of the output
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ void sts128(uint32_t a, uint32_t v) {   // four times v
  asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {   // transpose of an 8 x 8 matrix of 16-bit values
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 ex2(float2 v) { return make_float2(ex2_approx(v.x), ex2_approx(v.y)); }
__device__ __forceinline__ float pow2i(int e) {   // 2^e, 0 below the normal range; e <= 127
  return e < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Where a walk over the CTA's share of the block list stands: unit (b, u) with u = kv head * subs + sub, `left` blocks of it from
// the current one on, and the first key of this warp's strip in the current block.  Which of a block's strips is a warp's turns with
// every unit, so that units of one strip keep all warps busy.
template <int W, int KEYS>
struct Walk {
  static constexpr int kBlock = KEYS * W;
  int b, u, left, key, start, end, turn;   // turn: of the block's strips, the one that is this warp's
  bool bad;
  // The first of the unit's blocks that is walked is `blk`.
  __device__ __forceinline__ void set(const KeyRange& r, int seq, int unit, int64_t blk) {
    b = seq;
    u = unit;
    start = static_cast<int>(r.start);
    end = static_cast<int>(r.end);
    bad = r.bad;
    left = static_cast<int>(range_blocks(r, kBlock, KEYS) - blk);
    const int64_t k = range_first(r, KEYS) + (blk * W + turn) * KEYS;
    key = static_cast<int>(k < r.end ? k : r.end);   // a strip behind the end is empty
  }
  __device__ __forceinline__ void step() {   // to the unit's next block
    --left;
    key = end - key > kBlock ? key + kBlock : end;
  }
  __device__ __forceinline__ void next_unit(const DecodeParams& p, int units) {
    turn = turn == 0 ? W - 1 : turn - 1;
    const bool wrap = u + 1 == units;
    const int seq = wrap ? b + 1 : b;
    set(key_range(p.lens[seq], p.starts ? p.starts[seq] : 0, p.max_pages, p.geom.page_log2), seq, wrap ? 0 : u + 1, 0);
  }
};

// The first of the two neighbouring columns that a lane's MMA results of tile i are.
template <int D, bool FP8>
__device__ __forceinline__ int column(int i, int n) {
  return FP8 ? (D / 8) * n + 2 * i : (i / 4) * 64 + 8 * n + 2 * (i % 4);
}

// 2^x for factors of the output, down to fp32's smallest values (ex2_approx gives 0 under 2^-126).
__device__ __forceinline__ float ex2_wide(float x) {
  const bool low = x < -64.f;
  return ex2_approx(low ? x + 64.f : x) * (low ? 5.421010862427522e-20f : 1.f);   // 2^-64
}

// The end of a row whose sums are relative to 2^mx: the sink, then what its columns are multiplied by (NaN where the sum is) and
// its lse.
struct RowEnd {
  float inv, lse;
};
__device__ __forceinline__ RowEnd row_end(const DecodeParams& p, int head, float mx, float sum) {
  float f = 1.f;
  if (p.sink) {
    const float s2 = p.sink[head] * kLog2e;
    const float top = fmaxf(mx, s2);
    f = mx == -INFINITY ? 0.f : ex2_approx(mx - top);
    sum = (mx == -INFINITY && sum == 0.f ? 0.f : sum * f) + (s2 == -INFINITY ? 0.f : ex2_approx(s2 - top));
    mx = top;
  }
  RowEnd r;   // the approximations are off by 2^-22 or two steps, far under the rounding of the output
  r.inv = sum == 0.f ? 0.f : __fdividef(f, sum);
  r.lse = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * kLn2;
  return r;
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(32 * warps_of(D, NT), 1) decode_kernel(DecodeParams p) {
  using C = Cfg<D, FP8, NT>;
  constexpr int NQ = 8 * NT, kW = C::W, kThreads = C::THREADS, kBlock = C::BLOCK, SK = C::SK;
  extern __shared__ __align__(128) uint8_t smem[];
  float2* join_o = reinterpret_cast<float2*>(smem + C::MISC);   // [kW / 2][an MMA's result registers in pairs][32 lanes]
  float2* join_ml = join_o + (kW / 2) * NQ * D / 2;             // (m, l) [kW][NQ], then the rows' factors [NQ]
  int64_t* scan = reinterpret_cast<int64_t*>(smem);                               // [kW] warp sums, then the total
  int64_t* kept = scan + 32;                                                      // [3]
  struct Begin { int32_t b; int64_t off; };
  Begin* begin = reinterpret_cast<Begin*>(smem + 512);

  allow_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, t = lane & 3;   // an MMA fragment's row (or column) group and position in it
  const int units = p.geom.hkv * p.subs;

  // ---- this CTA's share of the block list
  auto range_of = [&](int seq) { return key_range(p.lens[seq], p.starts ? p.starts[seq] : 0, p.max_pages, p.geom.page_log2); };
  auto blocks_of = [&](int seq) { return range_blocks(range_of(seq), kBlock, C::KEYS); };
  int64_t total, t0, t1, parts, off;   // off: of the share's first block in its sequence b
  int b;
  KeyRange range;
  const int64_t cta = blockIdx.x;
  if (p.batch <= 32) {   // a sequence a lane, every warp for itself
    KeyRange r{0, 0, false};
    if (lane < p.batch) r = range_of(lane);
    const int64_t mine = lane < p.batch ? range_blocks(r, kBlock, C::KEYS) : 0;
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    total = __shfl_sync(0xffffffffu, incl, 31) * units;
    parts = total < gridDim.x ? total : gridDim.x;
    if (cta >= parts) {
      if (tid == 0) p.desc[cta].parts = 0;
      return;
    }
    t0 = share_begin(total, parts, cta);
    t1 = share_begin(total, parts, cta + 1);
    b = __ffs(__ballot_sync(0xffffffffu, t0 < incl * units)) - 1;
    off = t0 - __shfl_sync(0xffffffffu, incl - mine, b) * units;
    range.start = __shfl_sync(0xffffffffu, static_cast<int>(r.start), b);
    range.end = __shfl_sync(0xffffffffu, static_cast<int>(r.end), b);
    range.bad = __shfl_sync(0xffffffffu, static_cast<int>(r.bad), b) != 0;
  } else {
    const int per = (p.batch + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, p.batch), b1 = min(b0 + per, p.batch);
    int64_t mine = 0;
    for (int i = b0; i < b1; ++i) mine += blocks_of(i);
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int64_t before = incl - mine;
    total = 0;
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    total *= units;
    parts = total < gridDim.x ? total : gridDim.x;
    if (cta >= parts) {
      if (tid == 0) p.desc[cta].parts = 0;
      return;
    }
    t0 = share_begin(total, parts, cta);
    t1 = share_begin(total, parts, cta + 1);
    int64_t x = before * units;
    if (t0 >= x && t0 < x + mine * units) {
      int i = b0;
      for (;; ++i) {
        const int64_t nb = units * blocks_of(i);
        if (t0 < x + nb) break;
        x += nb;
      }
      begin->b = i;
      begin->off = t0 - x;
    }
    __syncthreads();
    b = begin->b;
    off = begin->off;
    range = range_of(b);
  }
  Walk<kW, C::KEYS> cur;
  bool opens_mid;
  {
    const int64_t nb = range_blocks(range, kBlock, C::KEYS);
    int u = 0;
    if (off >= nb) u = off <= 0x7fffffff ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(nb)) : static_cast<int>(off / nb);
    cur.turn = warp;
    cur.set(range, b, u, off - u * nb);
    opens_mid = off != u * nb;
  }

  // ---- loading one strip of this warp; the loads' walk runs ahead of the products'
  const uint32_t ring = smem_u32(smem + C::MISC + C::JOIN) + warp * (C::STAGE * C::STAGES);
  Walk<kW, C::KEYS> ld = cur;
  const int page_rows = p.geom.hkv << p.geom.page_log2, page_mask = (1 << p.geom.page_log2) - 1;
  int head_row;           // the loading unit's head's first row in a page
  int page[SK];           // of the next strip's groups of 16 keys, read a strip ahead; -1 for a group outside the range
  auto read_pages = [&]() {
    const int32_t* row = p.table + ld.b * p.table_stride;
#pragma unroll
    for (int g = 0; g < SK; ++g) {
      const bool in = ld.end - ld.key > 16 * g && ld.start - ld.key < 16 * (g + 1);
      page[g] = in ? __ldg(row + ((ld.key + 16 * g) >> p.geom.page_log2)) : -1;
    }
  };
  auto open_unit = [&]() {
    head_row = (p.subs == 1 ? ld.u : ld.u / p.subs) << p.geom.page_log2;
    read_pages();
  };
  // this lane's chunks of a strip: chunk lane + 32 i, 512 bytes apart in the cache; their places repeat every kPeriod of them
  constexpr int kPeriod = strip_period(C::CPR);
  uint32_t dst_of[kPeriod];
#pragma unroll
  for (int i = 0; i < kPeriod; ++i) dst_of[i] = ring + 16 * strip_chunk((lane + 32 * i) / C::CPR, (lane + 32 * i) % C::CPR, C::CPR);
  auto load_strip = [&](int stage, bool more) {
    const int have = ld.end - ld.key;
    if (have > 0) {
      const bool full = have >= C::KEYS && ld.key >= ld.start;
#pragma unroll
      for (int g = 0; g < SK; ++g) {
        const bool ok = static_cast<uint32_t>(page[g]) < static_cast<uint32_t>(p.geom.num_pages);   // as page_ok, for pages of 32 bits
        const int64_t row = static_cast<int64_t>(ok ? page[g] : 0) * page_rows + (head_row + ((ld.key + 16 * g) & page_mask));
        const int64_t at = row * C::ROW + lane * 16;
        const uint8_t *k = static_cast<const uint8_t*>(p.k) + at, *v = static_cast<const uint8_t*>(p.v) + at;
        const uint32_t base = stage * C::STAGE + g * C::GROUP;
        if (full && ok) {
#pragma unroll
          for (int i = 0; i < C::CPR / 2; ++i) {
            const uint32_t to = base + dst_of[i % kPeriod] + i / kPeriod * (kPeriod * 512);
            cp_async16(to, k + 512 * i);
            cp_async16(to + C::STRIP, v + 512 * i);
          }
        } else {   // rows outside the range are filled with zeros, not read
          const int lo = ld.start - ld.key - 16 * g, hi = min(have - 16 * g, 16);
          const bool none = lo >= 16 || hi <= 0;
#pragma unroll
          for (int i = 0; i < C::CPR / 2; ++i) {
            const uint32_t to = base + dst_of[i % kPeriod] + i / kPeriod * (kPeriod * 512);
            const int key = (lane + 32 * i) / C::CPR, bytes = ok && key >= lo && key < hi ? 16 : 0;
            if (ok || none) cp_async16(to, k + 512 * i, bytes);
            else sts128(to, 0x7fff7fffu);   // no such page: keys of NaN, which make the row NaN
            cp_async16(to + C::STRIP, v + 512 * i, bytes);
          }
        }
        if constexpr (FP8) {
          if (lane < 2) cp_async16(ring + base + 2 * C::STRIP + 16 * lane, (lane ? p.v_exp : p.k_exp) + row);
        }
      }
    }
    if (!more) return;
    if (ld.left > 1) {
      ld.step();
      read_pages();
    } else {
      ld.next_unit(p, units);
      open_unit();
    }
  };

  open_unit();
  int64_t todo = t1 - t0;   // blocks from the current one on; the loads are STAGES - 1 of them ahead
  if (tid == 0) kept[0] = t1, kept[1] = total, kept[2] = parts;   // wanted again at the end: not held in registers meanwhile
#pragma unroll 1
  for (int s = 0; s < C::STAGES - 1; ++s) {
    if (s < todo) load_strip(s, s + 1 < todo);
    cp_async_commit();
  }

  // Exponents (log2 units) are taken against references, which are raised only when passed, then to kLazy above the largest: most strips
  // cost one vote.  l and, for bf16, O are relative to 2^m.  e4m3's O is relative to 2^(m + vr), so that its weights
  // 2^((score - m) + (n - vr)) lie under 2^kTop and the largest over 2^(kTop - kLazy): f16 reaches down to 2^-34 of that one.  vr is
  // counted from m so that a score's own rounding, in the first bracket, is the same in a weight and in l.
  constexpr float kLazy = FP8 ? 5.f : 8.f;
  constexpr float kTop = 15.f;
  constexpr float kNone = -3.402823466e38f;   // a reference that no key has raised

  // ---- per-unit state
  uint32_t qf[NT][C::KSTEPS][2];   // Q^T fragments in the contraction order of the K loads
  float qs[NT][2];                 // per query column: scale_log2, with the e4m3 path's power of two taken back
  float o[NT][C::MT][4];
  float m[NT][2], l[NT][2], vr[NT][2];
  // The query rows of a unit on their way to registers (a warp without a key in the part needs none), and what else begins with it.
  auto load_q = [&](const Walk<kW, C::KEYS>& w) {
    const int kvh = w.u / p.subs, s0 = (w.u - kvh * p.subs) * NQ;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qi = s0 + nt * 8 + n;
      const bool act = qi < p.group && w.key < w.end;
      const __nv_bfloat16* src = p.q + w.b * p.q_stride + static_cast<int64_t>(kvh * p.group + (act ? qi : 0)) * D;
#pragma unroll
      for (int ks = 0; ks < C::KSTEPS; ++ks) {
        const int at = FP8 ? (t + 4 * (ks / 4)) * 16 + 4 * (ks % 4) : (t + 4 * (ks / 2)) * 8 + 4 * (ks % 2);
        const uint2 x = act ? __ldg(reinterpret_cast<const uint2*>(src + at)) : uint2{};
        qf[nt][ks][0] = x.x;
        qf[nt][ks][1] = x.y;
      }
    }
  };
  auto begin_unit = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (FP8) {
        uint32_t top = 0;   // of the magnitudes' bit patterns, which order as integers but for NaN, two at a time
#pragma unroll
        for (int ks = 0; ks < C::KSTEPS; ++ks)
          top = __vmaxu2(top, __vmaxu2(qf[nt][ks][0] & 0x7fff7fffu, qf[nt][ks][1] & 0x7fff7fffu));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^(14 - e) brings the largest to [2^14, 2^15); the exponent kept in range for rows of zeros and of tiny values
        const int e = max(static_cast<int>(max(top & 0xffffu, top >> 16) >> 7) - 127, -100);
        const float f = pow2i(14 - e);
#pragma unroll
        for (int ks = 0; ks < C::KSTEPS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qf[nt][ks][i];
            const float2 x = mul2(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), make_float2(f, f));
            qf[nt][ks][i] = pack_f16x2(x.x, x.y);
          }
        // query columns 2t, 2t + 1 of the scores are rows 2t, 2t + 1 here: lanes 4 (2t), 4 (2t + 1)
        const int e0 = __shfl_sync(0xffffffffu, e, 8 * t), e1 = __shfl_sync(0xffffffffu, e, 8 * t + 4);
        qs[nt][0] = p.scale_log2 * pow2i(e0 - 14);
        qs[nt][1] = p.scale_log2 * pow2i(e1 - 14);
      } else {
        qs[nt][0] = qs[nt][1] = p.scale_log2;
      }
#pragma unroll
      for (int i = 0; i < C::MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      m[nt][0] = m[nt][1] = kNone;
      l[nt][0] = l[nt][1] = vr[nt][0] = vr[nt][1] = 0.f;
    }
  };

  // ---- one strip: all groups' scores, their exponentials, then all groups' values
  auto strip = [&](int stage) {
    const int have = cur.end - cur.key;
    if (have <= 0) return;
    const bool whole = have >= C::KEYS && cur.key >= cur.start;
    const uint32_t sb = ring + stage * C::STAGE;
    constexpr int CH = SK == 1 ? 2 : 1;   // accumulators a score tile: one group alone would be one long chain of MMAs
    float s[SK][NT][CH][4] = {};
#pragma unroll
    for (int h = 0; h < C::CPR / 4; ++h)
#pragma unroll
      for (int g = 0; g < SK; ++g) {
        const uint32_t kb = sb + g * C::GROUP;
        const uint4 x = lds128(kb + 16 * strip_chunk(n, t + 4 * h, C::CPR));
        const uint4 y = lds128(kb + 16 * strip_chunk(n + 8, t + 4 * h, C::CPR));
        const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
        if constexpr (FP8) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x2(xa[j], a0, a2);
            e4m3x4_to_f16x2(ya[j], a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<true>(s[g][nt][j % CH], a0, a1, a2, a3, qf[nt][4 * h + j][0], qf[nt][4 * h + j][1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma<false>(s[g][nt][j % CH], xa[2 * j], ya[2 * j], xa[2 * j + 1], ya[2 * j + 1], qf[nt][2 * h + j][0], qf[nt][2 * h + j][1]);
        }
      }
    // keys n and n + 8 of a group are this lane's; columns 2t, 2t + 1 of each query tile
    auto inside = [&](int key) { return whole || (key >= cur.start - cur.key && key < have); };
    float ks[SK][2], vn[SK][2];   // e4m3: the scale of a key's row, n of its value's (byte 0 stands for a value of 0)
    if constexpr (FP8) {
#pragma unroll
      for (int g = 0; g < SK; ++g)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t eb = sb + g * C::GROUP + 2 * C::STRIP + n + 8 * r;
          ks[g][r] = exp_scale(lds8(eb));
          const uint32_t byte = lds8(eb + 16);
          vn[g][r] = byte ? static_cast<float>(static_cast<int>(byte) - 127) : -INFINITY;
        }
    }
    // scores of a key (n, n + 8 of a group) and the two queries, two an instruction; exponents of the weights: of l (and bf16's O), of e4m3's O
    float2 x[SK][NT][2];
    auto less_m = [&](int g, int nt, int r) { return add2(x[g][nt][r], make_float2(-m[nt][0], -m[nt][1])); };
    auto less_vr = [&](int g, int nt, int r) {
      return add2(less_m(g, nt, r), add2(make_float2(vn[g][r], vn[g][r]), make_float2(-vr[nt][0], -vr[nt][1])));
    };
    bool raise = false;
#pragma unroll
    for (int g = 0; g < SK; ++g)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 q2 = make_float2(qs[nt][0], qs[nt][1]);
          float2 v = make_float2(s[g][nt][0][2 * r], s[g][nt][0][2 * r + 1]);
          if constexpr (CH == 2) v = add2(v, make_float2(s[g][nt][1][2 * r], s[g][nt][1][2 * r + 1]));
          v = mul2(v, FP8 ? mul2(q2, make_float2(ks[g][r], ks[g][r])) : q2);
          if (!whole && !inside(16 * g + n + 8 * r)) v = make_float2(-INFINITY, -INFINITY);
          x[g][nt][r] = v;
          raise |= v.x > m[nt][0] || v.y > m[nt][1];
          if constexpr (FP8) {
            const float2 y = less_vr(g, nt, r);
            raise |= y.x > kTop || y.y > kTop;
          }
        }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          auto score = [&](int g, int r) { return c ? x[g][nt][r].y : x[g][nt][r].x; };
          auto largest = [&](auto value) {   // of this query's keys in the strip
            float mx = -INFINITY;
#pragma unroll
            for (int g = 0; g < SK; ++g) mx = fmaxf(mx, fmaxf(value(g, 0), value(g, 1)));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            return fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          };
          const float mx = fmaxf(largest(score) + kLazy, m[nt][c]);
          const float up = m[nt][c] - mx;
          float f = ex2_approx(up);
          m[nt][c] = mx;
          l[nt][c] *= f;
          if constexpr (FP8) {
            const float top = fmaxf(largest([&](int g, int r) { return (score(g, r) - mx) + vn[g][r]; }) + (kLazy - kTop), vr[nt][c] + up);
            f = ex2_approx(up + (vr[nt][c] - top));
            vr[nt][c] = top;
          }
#pragma unroll
          for (int i = 0; i < C::MT; ++i) {
            o[nt][i][c] *= f;
            o[nt][i][c + 2] *= f;
          }
        }
    }
    uint32_t pf[SK][NT][2], pl[SK][NT][2];
#pragma unroll
    for (int g = 0; g < SK; ++g)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float2 e0 = ex2(less_m(g, nt, 0)), e1 = ex2(less_m(g, nt, 1));
        const float2 sum = add2(make_float2(l[nt][0], l[nt][1]), add2(e0, e1));
        l[nt][0] = sum.x, l[nt][1] = sum.y;
        if constexpr (FP8) {
          e0 = ex2(less_vr(g, nt, 0)), e1 = ex2(less_vr(g, nt, 1));
          pf[g][nt][0] = movmatrix(pack_f16x2(e0.x, e0.y));
          pf[g][nt][1] = movmatrix(pack_f16x2(e1.x, e1.y));
        } else {
          const uint32_t h0 = pack_bf16x2(e0.x, e0.y), h1 = pack_bf16x2(e1.x, e1.y);
          pf[g][nt][0] = movmatrix(h0);
          pf[g][nt][1] = movmatrix(h1);
          pl[g][nt][0] = movmatrix(pack_bf16x2(e0.x - __uint_as_float(h0 << 16), e0.y - __uint_as_float(h0 & 0xffff0000u)));
          pl[g][nt][1] = movmatrix(pack_bf16x2(e1.x - __uint_as_float(h1 << 16), e1.y - __uint_as_float(h1 & 0xffff0000u)));
        }
      }
    // out^T += V^T P^T: this lane's four keys 2t, 2t + 1, 2t + 8, 2t + 9 of each group, and its columns
#pragma unroll
    for (int g = 0; g < SK; ++g) {
      const uint32_t vb = sb + g * C::GROUP + C::STRIP;
      if constexpr (FP8) {
        constexpr int WORDS = C::MT / 2;   // 32-bit words of a row this lane owns: 2 (d = 64) or 4
        uint32_t r[4][WORDS];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = 2 * t + (i & 1) + 8 * (i >> 1);
          if constexpr (D == 128) {
            const uint4 w = lds128(vb + 16 * strip_chunk(key, n, C::CPR));
            r[i][0] = w.x, r[i][1] = w.y, r[i][2] = w.z, r[i][3] = w.w;
          } else {
            const uint2 w = lds64(vb + 16 * strip_chunk(key, n >> 1, C::CPR) + 8 * (n & 1));
            r[i][0] = w.x, r[i][1] = w.y;
          }
        }
#pragma unroll
        for (int i = 0; i < C::MT; ++i) {
          const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;   // columns 2i, 2i + 1 of two keys, paired by column
          const uint32_t w0 = __byte_perm(r[0][i / 2], r[1][i / 2], sel), w1 = __byte_perm(r[2][i / 2], r[3][i / 2], sel);
          uint32_t a0, a1, a2, a3;
          e4m3x4_to_f16x2(w0, a0, a1);
          e4m3x4_to_f16x2(w1, a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma<true>(o[nt][i], a0, a1, a2, a3, pf[g][nt][0], pf[g][nt][1]);
        }
      } else {
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh) {
          uint32_t r[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 w = lds128(vb + 16 * strip_chunk(2 * t + (i & 1) + 8 * (i >> 1), n + 8 * hh, C::CPR));
            r[i][0] = w.x, r[i][1] = w.y, r[i][2] = w.z, r[i][3] = w.w;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t a0 = __byte_perm(r[0][i], r[1][i], 0x5410), a1 = __byte_perm(r[0][i], r[1][i], 0x7632);
            const uint32_t a2 = __byte_perm(r[2][i], r[3][i], 0x5410), a3 = __byte_perm(r[2][i], r[3][i], 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<false>(o[nt][4 * hh + i], a0, a1, a2, a3, pf[g][nt][0], pf[g][nt][1]);
              mma<false>(o[nt][4 * hh + i], a0, a1, a2, a3, pl[g][nt][0], pl[g][nt][1]);
            }
          }
        }
      }
    }
  };

  // ---- the end of a unit's part: join the warps, then write the rows or the part.  The buffers hold the values as the MMAs'
  // results lie in a warp (pair, lane), so that neither side has a bank conflict.
  constexpr int kPairs = NT * C::MT * 2;
  auto end_part = [&](bool whole, int slot) {
    const int h0 = (cur.u / p.subs) * p.group, s0 = (cur.u % p.subs) * NQ;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float s = l[nt][c];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        m[nt][c] = m[nt][c] == kNone ? -INFINITY : m[nt][c];
        if (n == 0) join_ml[warp * NQ + nt * 8 + 2 * t + c] = make_float2(m[nt][c], s);
      }
    __syncthreads();
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kW; ++w) mx = fmaxf(mx, join_ml[w * NQ + nt * 8 + 2 * t + c].x);
        f[nt][c] = m[nt][c] == -INFINITY ? 0.f : FP8 ? ex2_wide(m[nt][c] - mx + vr[nt][c]) : ex2_approx(m[nt][c] - mx);
      }
    if (warp >= kW / 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            join_o[((warp - kW / 2) * kPairs + (nt * C::MT + i) * 2 + c) * 32 + lane] =
                make_float2(o[nt][i][c] * f[nt][c], o[nt][i][c + 2] * f[nt][c]);
    } else if (warp < NT) {   // a row's warps are dealt to 4 lanes
      const int row = warp * 8 + (lane & 7);
      float2 v[(kW + 3) / 4];
      float mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < (kW + 3) / 4; ++i) {
        const int w = (lane >> 3) + 4 * i;
        v[i] = w < kW ? join_ml[w * NQ + row] : make_float2(-INFINITY, 0.f);
        mx = fmaxf(mx, v[i].x);
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
#pragma unroll
      for (int i = 0; i < (kW + 3) / 4; ++i)
        sum += v[i].x == -INFINITY ? v[i].y : v[i].y * ex2_approx(v[i].x - mx);   // v.y is 0 or NaN without a maximum
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (lane < 8) {
        if (whole && s0 + row < p.group) {
          const RowEnd r = row_end(p, h0 + s0 + row, mx, sum);
          p.lse[static_cast<int64_t>(h0 + s0 + row) * p.batch + cur.b] = r.lse;
          join_ml[kW * NQ + row].x = r.inv;
        } else if (!whole) {
          p.ml[static_cast<int64_t>(slot) * NQ + row] = make_float2(mx, sum);
        }
      }
    }
    __syncthreads();
    if (warp < kW / 2) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float2* at = join_o + (warp * kPairs + (nt * C::MT + i) * 2 + c) * 32 + lane;
            const float2 v = *at;
            *at = make_float2(fmaf(o[nt][i][c], f[nt][c], v.x), fmaf(o[nt][i][c + 2], f[nt][c], v.y));
          }
    }
    __syncthreads();
    // what is read from here on (the buffers, the rows' factors) is written again only behind the next part's first barrier
    for (int e = warp; e < kPairs; e += kW) {
      const int i = e / 2 % C::MT, qi = e / (2 * C::MT) * 8 + 2 * t + (e & 1);
      const int col = column<D, FP8>(i, n);
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kW / 2; ++w) {
        const float2 a = join_o[(w * kPairs + e) * 32 + lane];
        v.x += a.x, v.y += a.y;
      }
      if (s0 + qi >= p.group) continue;
      if (!whole) {
        *reinterpret_cast<float2*>(p.part + (static_cast<int64_t>(slot) * NQ + qi) * D + col) = v;
      } else {
        const float inv = join_ml[kW * NQ + qi].x;
        *reinterpret_cast<uint32_t*>(p.out + (static_cast<int64_t>(cur.b) * p.hq + h0 + s0 + qi) * D + col) = pack_bf16x2(v.x * inv, v.y * inv);
      }
    }
  };

  // A unit that was this warp's alone: its rows.  A sequence with a length that its table row cannot hold reads no key and ends here too.
  auto end_alone = [&]() {
    const int h0 = (cur.u / p.subs) * p.group, s0 = (cur.u % p.subs) * NQ;
    const float poison = cur.bad ? __int_as_float(0x7fffffff) : 0.f;   // makes its rows NaN
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[nt][c];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int row = s0 + nt * 8 + 2 * t + c, head = h0 + row;
        if (row >= p.group) continue;
        const float mx = m[nt][c] == kNone ? -INFINITY : m[nt][c];
        const RowEnd r = row_end(p, head, mx, sum + poison);
        const float f = FP8 && mx != -INFINITY ? r.inv * ex2_wide(vr[nt][c]) : r.inv;
        __nv_bfloat16* out = p.out + (static_cast<int64_t>(cur.b) * p.hq + head) * D;
        if (n == 0) p.lse[static_cast<int64_t>(head) * p.batch + cur.b] = r.lse;
#pragma unroll
        for (int i = 0; i < C::MT; ++i)
          *reinterpret_cast<uint32_t*>(out + column<D, FP8>(i, n)) = pack_bf16x2(o[nt][i][c] * f, o[nt][i][c + 2] * f);
      }
  };

  // ---- the share
  load_q(cur);
  bool first_part = true, from_start = !opens_mid;
  int32_t opened = 0;   // parts of the unit this CTA leaves open to later ones
  int stage = 0, fill = C::STAGES - 1;
#pragma unroll 1
  for (;;) {   // a unit's part after the other
    begin_unit();
#pragma unroll 1
    for (;;) {   // its blocks
      if (todo > C::STAGES - 1) load_strip(fill, todo > C::STAGES);
      cp_async_commit();
      fill = fill + 1 == C::STAGES ? 0 : fill + 1;
      cp_async_wait<C::STAGES - 1>();
      __syncwarp();
      strip(stage);
      __syncwarp();   // the stage has been read by every lane before the next iteration refills it
      stage = stage + 1 == C::STAGES ? 0 : stage + 1;
      if (cur.left == 1 || todo == 1) break;
      cur.step();
      --todo;
    }
    const bool last = cur.left == 1, whole = last && from_start;
    const int slot = static_cast<int>(2 * cta) + (first_part ? 0 : 1);
    Walk<kW, C::KEYS> next = cur;
    if (todo > 1) {   // the next unit's queries travel while this one's part ends
      next.next_unit(p, units);
      load_q(next);
    }
    if (whole && cur.end - cur.start / C::KEYS * C::KEYS <= C::KEYS) {   // a unit of one strip: its warp alone
      if (cur.turn == 0) end_alone();
    } else {
      end_part(whole, slot);
    }
    if (!last && from_start) {
      opened = static_cast<int32_t>(share_of(kept[1], kept[2], kept[0] - todo + cur.left - 1) - cta + 1);
      if (tid == 0) {
        JoinDesc d{};
        d.parts = opened;
        d.batch = cur.b;
        d.unit = cur.u;
        d.first_slot = slot;
        p.desc[cta] = d;
      }
    }
    if (--todo == 0) break;
    first_part = false;
    from_start = true;
    cur = next;
  }
  if (opened == 0 && tid == 0) p.desc[cta].parts = 0;
}

// Joins the parts of the unit that CTA blockIdx.x of the main kernel opened: a CTA a q head of the unit (blockIdx.y), D / 4
// threads to a part and as many parts at once as 256 threads hold, then those by the order of their first part.  Every load
// of a round is independent, so a unit of 152 parts takes a few memory latencies.
template <int D, int NT>
__global__ void __launch_bounds__(256) decode_join_kernel(DecodeParams p) {
  constexpr int NQ = 8 * NT, COLS = D / 4, LANES = 256 / COLS, UNROLL = 4;
  __shared__ float4 so[LANES][COLS];
  __shared__ float2 sm[LANES];
  wait_for_primary();
  const JoinDesc d = p.desc[blockIdx.x];
  const int qi = blockIdx.y, row = (d.unit % p.subs) * NQ + qi;
  if (d.parts == 0 || row >= p.group) return;
  const int c = threadIdx.x % COLS, lane = threadIdx.x / COLS;
  float mx = -INFINITY, sum = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  auto merge = [&](float2 ml, float4 a) {
    const float top = fmaxf(mx, ml.x);
    const float fo = mx == -INFINITY ? 0.f : ex2_approx(mx - top), fn = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
    sum = (mx == -INFINITY ? sum : sum * fo) + (ml.x == -INFINITY ? ml.y : ml.y * fn);   // sums without a maximum are 0 or NaN
    v = make_float4(v.x * fo + a.x * fn, v.y * fo + a.y * fn, v.z * fo + a.z * fn, v.w * fo + a.w * fn);
    mx = top;
  };
  for (int k0 = lane; k0 < d.parts; k0 += UNROLL * LANES) {
    float2 ml[UNROLL];
    float4 a[UNROLL];
#pragma unroll
    for (int i = 0; i < UNROLL; ++i) {
      const int k = k0 + i * LANES;
      if (k >= d.parts) continue;
      const int64_t at = (k == 0 ? d.first_slot : 2 * (static_cast<int64_t>(blockIdx.x) + k)) * NQ + qi;
      ml[i] = p.ml[at];
      a[i] = *reinterpret_cast<const float4*>(p.part + at * D + 4 * c);
    }
#pragma unroll
    for (int i = 0; i < UNROLL; ++i)
      if (k0 + i * LANES < d.parts) merge(ml[i], a[i]);
  }
  so[lane][c] = v;
  if (c == 0) sm[lane] = make_float2(mx, sum);
  __syncthreads();
  if (lane != 0) return;
#pragma unroll
  for (int i = 1; i < LANES; ++i) merge(sm[i], so[i][c]);
  const int head = (d.unit / p.subs) * p.group + row;
  const RowEnd r = row_end(p, head, mx, sum);
  *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(d.batch) * p.hq + head) * D + 4 * c) =
      make_uint2(pack_bf16x2(v.x * r.inv, v.y * r.inv), pack_bf16x2(v.z * r.inv, v.w * r.inv));
  if (c == 0) p.lse[static_cast<int64_t>(head) * p.batch + d.batch] = r.lse;
}

constexpr size_t kDescBytes = sizeof(JoinDesc) * kMaxCtas;
size_t ml_bytes(int nt) { return size_t{2} * kMaxCtas * 8 * nt * 2 * sizeof(float); }
size_t part_bytes(int nt, int d) { return size_t{2} * kMaxCtas * 8 * nt * d * sizeof(float); }
int tiles_of(int group) { return group > 8 ? 2 : 1; }   // query tiles of 8 a unit

template <int D, bool FP8, int NT>
ffa_status launch(const DecodeParams& p, int device, int sms, cudaStream_t s) {
  using C = Cfg<D, FP8, NT>;
  static_assert(C::FIT >= C::STAGES && C::STAGES >= 2, "ring");
  static std::atomic<bool> raised[kDevices];
  const int grid = std::min(sms, kMaxCtas);
  const cudaError_t e = launch_large(decode_kernel<D, FP8, NT>, dim3(grid), C::THREADS, C::SMEM, C::SMEM, s, device, raised, p);
  if (e != cudaSuccess) return FFA_ERR_CUDA;
  return cuda_status(launch_after(decode_join_kernel<D, NT>, dim3(grid, std::min(8 * NT, p.group)), 256, s, p));
}

}  // namespace
}  // namespace ffa

using namespace ffa;

extern "C" {

size_t ffa_fwd_decode_workspace_size(int32_t hq, int32_t hkv, int32_t d) {
  if (hq <= 0 || hkv <= 0 || hq % hkv != 0 || (d != 64 && d != 128)) return 0;
  const int nt = tiles_of(hq / hkv);
  return kDescBytes + ml_bytes(nt) + part_bytes(nt, d);
}

ffa_status ffa_fwd_decode(const void* q, int64_t q_stride, const ffa_kv_cache* cache, const int32_t* page_table,
                          int64_t table_stride, int32_t max_pages, int32_t batch, int32_t hq, const int32_t* kv_lens,
                          const int32_t* kv_starts, float scale, const float* sink, void* out, float* lse,
                          void* workspace, size_t workspace_bytes, void* stream) {
  DecodeParams p{};
  const ffa_status st = check_cache(cache, p.geom);
  if (st != FFA_OK) return st;
  if (batch < 0 || max_pages < 0 || hq <= 0 || hq % cache->hkv != 0) return FFA_ERR_INVALID_ARG;
  if (!(scale * kLog2e > -INFINITY && scale * kLog2e < INFINITY)) return FFA_ERR_INVALID_ARG;   // the scale in log2 units
  if (batch > 1 && table_stride < max_pages) return FFA_ERR_INVALID_ARG;
  if (hq > (1 << 16) || batch > (1 << 20)) return FFA_ERR_OVERFLOW;
  if (batch == 0) return FFA_OK;
  const int32_t d = cache->d;
  if (!q || !out || !lse || !kv_lens || !workspace) return FFA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || !aligned16(workspace)) return FFA_ERR_INVALID_ARG;
  if (max_pages > 0 && !page_table) return FFA_ERR_INVALID_ARG;
  for (const void* a : {static_cast<const void*>(page_table), static_cast<const void*>(kv_lens),
                        static_cast<const void*>(kv_starts), static_cast<const void*>(sink)})
    if (reinterpret_cast<uintptr_t>(a) & 3u) return FFA_ERR_INVALID_ARG;
  if (q_stride % 8 != 0 || (batch > 1 && q_stride < static_cast<int64_t>(hq) * d)) return FFA_ERR_INVALID_ARG;
  if (workspace_bytes < ffa_fwd_decode_workspace_size(hq, cache->hkv, d)) return FFA_ERR_INVALID_ARG;
  const int group = hq / cache->hkv, nt = tiles_of(group);
  const CacheSpans at(*cache);
  Span in[9] = {{q, span_bytes(batch, q_stride, hq, d)}, {page_table, 4 * (static_cast<int64_t>(batch - 1) * table_stride + max_pages)},
                {kv_lens, 4 * int64_t{batch}}, {kv_starts, kv_starts ? 4 * int64_t{batch} : 0}, {sink, sink ? 4 * hq : 0}};
  for (int i = 0; i < at.n; ++i) in[5 + i] = at.s[i];
  const Span outs[] = {{out, 2 * int64_t{batch} * hq * d}, {lse, 4 * int64_t{batch} * hq},
                       {workspace, static_cast<int64_t>(ffa_fwd_decode_workspace_size(hq, cache->hkv, d))}};
  if (any_meet(outs, 3, in, 5 + at.n)) return FFA_ERR_INVALID_ARG;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.k = cache->k;
  p.v = cache->v;
  p.k_exp = cache->k_exp;
  p.v_exp = cache->v_exp;
  p.table = page_table;
  p.table_stride = table_stride;
  p.max_pages = max_pages;
  p.batch = batch;
  p.hq = hq;
  p.group = group;
  p.subs = (group + 8 * nt - 1) / (8 * nt);
  p.lens = kv_lens;
  p.starts = kv_starts;
  p.scale_log2 = scale * kLog2e;
  p.sink = sink;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.desc = reinterpret_cast<JoinDesc*>(ws);
  p.ml = reinterpret_cast<float2*>(ws + kDescBytes);
  p.part = reinterpret_cast<float*>(ws + kDescBytes + ml_bytes(nt));
  int device = 0, sms = 0;
  if (!current_device(device, sms)) return FFA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = cache->dtype == FFA_KV_E4M3;
  if (d == 128) {
    if (nt == 1) return fp8 ? launch<128, true, 1>(p, device, sms, s) : launch<128, false, 1>(p, device, sms, s);
    return fp8 ? launch<128, true, 2>(p, device, sms, s) : launch<128, false, 2>(p, device, sms, s);
  }
  if (nt == 1) return fp8 ? launch<64, true, 1>(p, device, sms, s) : launch<64, false, 1>(p, device, sms, s);
  return fp8 ? launch<64, true, 2>(p, device, sms, s) : launch<64, false, 2>(p, device, sms, s);
}

}  // extern "C"
