// Attention of one new token a sequence over the paged key-value cache, split over the cache's length and joined.
//
// For sequence b, q head h (kv head h / (hq / hkv)) and the keys j in [start_b, len_b):
//   s_j = scale q . k_j,  lse = ln(sum_j e^{s_j} [+ e^{sink_h}]),  out = sum_j e^{s_j - lse} v_j.
//
// Bound by HBM: every stored key and value is read once, 4 hq / hkv FLOPs a byte (e4m3) or half that (bf16), far under what the tensor cores need
// to be busy.  So the design is about keeping loads in flight:
//   - The batch's keys are counted in blocks of 16 keys a warp; all (sequence, kv head) units' blocks form one list,
//     dealt to the CTAs in equal contiguous shares (paged.cuh: share_begin).  Ragged lengths and few long sequences
//     balance the same way, and no length has to be known on the host.
//   - A warp streams its own 16-key strips (K, V, exponent bytes) through a ring in shared memory with cp.async, across
//     unit borders, and never waits for another warp until a unit's part ends.
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
// mantissa fits, values 2^-29 of the row's largest and below round); the scale of a key's row multiplies its score, the scale
// of a value's row its weight, relative to the largest seen; P is f16 (11 bits).  Scores, maxima, sums and the output
// accumulate in fp32.
//
// Split parts go to the workspace as (m, l, O) and a second kernel joins them in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>

#include "ffa_internal.h"
#include "kv_cache.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace ffa {
namespace {

constexpr int warps_of(bool fp8, int nt) { return fp8 && nt == 1 ? 12 : 8; }   // warps a CTA
constexpr int kMaxCtas = 512;          // split parts the workspace holds: two a CTA
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
  float* ml;          // [2 kMaxCtas][8 NT][2]
  float* part;        // [2 kMaxCtas][8 NT][D]
};

template <int D, bool FP8, int NT>
struct Cfg {
  static constexpr int W = warps_of(FP8, NT);
  static constexpr int THREADS = 32 * W;
  static constexpr int BLOCK = 16 * W;                  // keys of a block
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int ROW = D * ES;                    // bytes a stored row
  static constexpr int CPR = ROW / 16;                  // 16-byte chunks a row
  static constexpr int STRIP = 16 * ROW;                // bytes of 16 rows
  static constexpr int STAGE = 2 * STRIP + (FP8 ? 32 : 0);
  static constexpr int JOIN = (W / 2) * 8 * NT * D * 4 + (W + 1) * 8 * NT * 8;   // O buffers; (m, l) of every warp and of all
  static constexpr int MISC = 1024;
  static constexpr int STAGES = (kSmemMax - JOIN - MISC) / (W * STAGE) < 8 ? (kSmemMax - JOIN - MISC) / (W * STAGE) : 8;
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
__device__ __forceinline__ float pow2i(int e) {   // 2^e, 0 below the normal range; e <= 127
  return e < -126 ? 0.f : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Where a walk over the CTA's share of the block list stands: unit (b, u) with u = kv head * subs + sub, `left` blocks of it from
// the current one on, and the first key of this warp's strip in the current block.
template <int W>
struct Walk {
  static constexpr int kBlock = 16 * W;
  int b, u, left, key, start, end;
  bool bad;
  // The first of the unit's blocks that is walked is `blk`.
  __device__ __forceinline__ void set(const DecodeParams& p, int seq, int unit, int64_t blk, int warp) {
    const KeyRange r = key_range(p.lens[seq], p.starts ? p.starts[seq] : 0, p.max_pages, p.geom.page_log2);
    b = seq;
    u = unit;
    start = static_cast<int>(r.start);
    end = static_cast<int>(r.end);
    bad = r.bad;
    left = static_cast<int>(range_blocks(r, kBlock) - blk);
    // a warp's strip may lie behind the end, by a block at most: as keys are below 2^31, unsigned arithmetic and a clamp
    const int64_t k = range_first(r) + (blk * W + warp) * 16;
    key = static_cast<int>(k < r.end ? k : r.end);
  }
  __device__ __forceinline__ void step() {   // to the unit's next block
    --left;
    key = end - key > kBlock ? key + kBlock : end;
  }
  __device__ __forceinline__ void next_unit(const DecodeParams& p, int units, int warp) {
    const bool wrap = u + 1 == units;
    set(p, wrap ? b + 1 : b, wrap ? 0 : u + 1, 0, warp);
  }
};

// The end of a row whose sums, times 2^bias, are relative to the maximum mx: the sink, then what its columns are multiplied by
// (NaN where the sum is) and its lse.
struct RowEnd {
  float inv, lse;
};
__device__ __forceinline__ RowEnd row_end(const DecodeParams& p, int head, float mx, float sum, float bias) {
  float f = 1.f;
  mx -= bias;
  if (p.sink) {
    const float s2 = p.sink[head] * kLog2e;
    const float top = fmaxf(mx, s2);
    f = mx == -INFINITY ? 0.f : ex2_approx(mx - top);
    sum = (mx == -INFINITY && sum == 0.f ? 0.f : sum * f) + (s2 == -INFINITY ? 0.f : ex2_approx(s2 - top));
    mx = top;
  }
  RowEnd r;
  r.inv = sum == 0.f ? 0.f : f / sum;
  r.lse = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
  return r;
}

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(32 * warps_of(FP8, NT), 1) decode_kernel(DecodeParams p) {
  using C = Cfg<D, FP8, NT>;
  constexpr int NQ = 8 * NT, kW = C::W, kThreads = C::THREADS, kBlock = C::BLOCK;
  extern __shared__ __align__(128) uint8_t smem[];
  float2* join_o = reinterpret_cast<float2*>(smem + C::MISC);   // [kW / 2][an MMA's result registers in pairs][32 lanes]
  float2* join_ml = join_o + (kW / 2) * NQ * D / 2;             // [kW][NQ], then [NQ] of all warps
  int64_t* scan = reinterpret_cast<int64_t*>(smem);                               // [kW] warp sums, then the total
  struct Begin { int32_t b; int64_t off; };
  Begin* begin = reinterpret_cast<Begin*>(smem + 512);

  allow_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, t = lane & 3;   // an MMA fragment's row (or column) group and position in it
  const int units = p.geom.hkv * p.subs;

  // ---- this CTA's share of the block list
  auto blocks_of = [&](int b) {
    return range_blocks(key_range(p.lens[b], p.starts ? p.starts[b] : 0, p.max_pages, p.geom.page_log2), kBlock);
  };
  int64_t total, t0, t1, parts, off;   // off: of the share's first block in its sequence b
  int b;
  const int64_t cta = blockIdx.x;
  if (p.batch <= 32) {   // a sequence a lane, every warp for itself
    const int64_t mine = lane < p.batch ? blocks_of(lane) : 0;
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
  }
  Walk<kW> cur;
  bool opens_mid;
  {
    const int64_t nb = blocks_of(b);
    const int u = off < nb ? 0 : off <= 0x7fffffff ? static_cast<int>(static_cast<uint32_t>(off) / static_cast<uint32_t>(nb)) : static_cast<int>(off / nb);
    cur.set(p, b, u, off - u * nb, warp);
    opens_mid = off != u * nb;
  }

  // ---- loading one strip of this warp; the loads' walk runs ahead of the products'
  const uint32_t ring = smem_u32(smem + C::MISC + C::JOIN) + warp * (C::STAGE * C::STAGES);
  uint32_t stage_bad = 0;   // stages whose page the cache does not have
  Walk<kW> ld = cur;
  auto page_of = [&]() -> int { return ld.key < ld.end ? __ldg(p.table + ld.b * p.table_stride + (ld.key >> p.geom.page_log2)) : 0; };
  int page = page_of();     // the page of the next strip to load, read one strip ahead
  // this lane's chunks of a strip: chunk lane + 32 i, rows 32 / CPR apart; source and destination offsets
  uint32_t dst_of[C::CPR / 2];
#pragma unroll
  for (int i = 0; i < C::CPR / 2; ++i) dst_of[i] = 16 * strip_chunk((lane + 32 * i) / C::CPR, (lane + 32 * i) % C::CPR, C::CPR);
  auto load_strip = [&](int stage, bool more) {
    const int have = ld.end - ld.key;
    if (have > 0) {
      const int off = ld.key & ((1 << p.geom.page_log2) - 1);
      const bool ok = page_ok(p.geom, page);
      const uint32_t bit = 1u << stage;
      stage_bad = ok ? stage_bad & ~bit : stage_bad | bit;
      const int64_t row = ok ? cache_row(p.geom, page, p.subs == 1 ? ld.u : ld.u / p.subs, off) : 0;
      const uint8_t* ksrc = static_cast<const uint8_t*>(p.k) + row * C::ROW + lane * 16;
      const uint8_t* vsrc = static_cast<const uint8_t*>(p.v) + row * C::ROW + lane * 16;
      const uint32_t dst = ring + stage * C::STAGE;
      if (ok && have >= 16 && ld.key >= ld.start) {
#pragma unroll
        for (int i = 0; i < C::CPR / 2; ++i) {
          cp_async16(dst + dst_of[i], ksrc + 512 * i);
          cp_async16(dst + C::STRIP + dst_of[i], vsrc + 512 * i);
        }
      } else {   // rows outside the range are filled with zeros, not read
        const int lo = max(ld.start - ld.key, 0), hi = ok ? min(have, 16) : 0;
#pragma unroll
        for (int i = 0; i < C::CPR / 2; ++i) {
          const int key = (lane + 32 * i) / C::CPR, bytes = key >= lo && key < hi ? 16 : 0;
          cp_async16(dst + dst_of[i], ksrc + 512 * i, bytes);
          cp_async16(dst + C::STRIP + dst_of[i], vsrc + 512 * i, bytes);
        }
      }
      if constexpr (FP8) {
        if (lane < 2) cp_async16(dst + 2 * C::STRIP + 16 * lane, (lane ? p.v_exp : p.k_exp) + row, ok ? 16 : 0);
      }
    }
    if (!more) return;
    if (ld.left > 1) ld.step(); else ld.next_unit(p, units, warp);
    page = page_of();
  };

  int64_t ahead = t0;
#pragma unroll 1
  for (int s = 0; s < C::STAGES - 1; ++s) {
    if (ahead < t1) {
      ++ahead;
      load_strip(s, ahead < t1);
    }
    cp_async_commit();
  }

  // A row maximum is raised only when a score passes it by kLazy (log2 units): most strips then cost one vote.
  constexpr float kLazy = FP8 ? 5.f : 8.f;
  constexpr float kBias = FP8 ? 10.f : 0.f;   // e4m3: P is held times 2^10, at most 2^15: f16 reaches 2^-34 of the largest

  // ---- per-unit state
  uint32_t qf[NT][C::KSTEPS][2];   // Q^T fragments in the contraction order of the K loads
  float qs[NT][2];                 // per query column: scale_log2, with the e4m3 path's power of two taken back
  float o[NT][C::MT][4];
  float m[NT][2], l[NT][2];
  float mb[NT][2], thr[NT][2];     // what a score's exponent is taken against, and what raises the maximum
  int ev_ref = 0;                  // e4m3: exponent byte that O's unit stands for
  bool bad = false;
  auto begin_unit = [&]() {
    const int h0 = (cur.u / p.subs) * p.group, s0 = (cur.u % p.subs) * NQ;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qi = s0 + nt * 8 + n;
      const bool act = qi < p.group;
      const __nv_bfloat16* src = p.q + cur.b * p.q_stride + static_cast<int64_t>(h0 + (act ? qi : 0)) * D;
      float amax = 0.f;
#pragma unroll
      for (int ks = 0; ks < C::KSTEPS; ++ks) {
        const int at = FP8 ? (t + 4 * (ks / 4)) * 16 + 4 * (ks % 4) : (t + 4 * (ks / 2)) * 8 + 4 * (ks % 2);
        const uint2 w = act ? __ldg(reinterpret_cast<const uint2*>(src + at)) : uint2{};
        qf[nt][ks][0] = w.x;
        qf[nt][ks][1] = w.y;
        if constexpr (FP8) {
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xffff0000u))));
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xffff0000u))));
        }
      }
      if constexpr (FP8) {
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^(14 - e) brings the largest to [2^14, 2^15); the exponent kept in range for rows of zeros and of tiny values
        const int e = max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -100);
        const float f = pow2i(14 - e);
#pragma unroll
        for (int ks = 0; ks < C::KSTEPS; ++ks)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qf[nt][ks][i];
            qf[nt][ks][i] = pack_f16x2(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xffff0000u) * f);
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
      m[nt][0] = m[nt][1] = thr[nt][0] = thr[nt][1] = -INFINITY;
      mb[nt][0] = mb[nt][1] = -kBias;
      l[nt][0] = l[nt][1] = 0.f;
    }
    ev_ref = 0;
    bad = cur.bad;
  };

  // ---- one strip
  auto strip = [&](int stage) {
    const int have = cur.end - cur.key;
    if (have <= 0) return;
    const bool whole = have >= 16 && cur.key >= cur.start;
    const uint32_t kb = ring + stage * C::STAGE, vb = kb + C::STRIP;
    bad |= (stage_bad >> stage & 1u) != 0;
    float s[NT][2][4] = {};
#pragma unroll
    for (int h = 0; h < C::CPR / 4; ++h) {
      const uint4 x = lds128(kb + 16 * strip_chunk(n, t + 4 * h, C::CPR));
      const uint4 y = lds128(kb + 16 * strip_chunk(n + 8, t + 4 * h, C::CPR));
      const uint32_t xa[4] = {x.x, x.y, x.z, x.w}, ya[4] = {y.x, y.y, y.z, y.w};
      if constexpr (FP8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = e4m3x2_to_f16x2(xa[j]), a2 = e4m3x2_to_f16x2(xa[j] >> 16);
          const uint32_t a1 = e4m3x2_to_f16x2(ya[j]), a3 = e4m3x2_to_f16x2(ya[j] >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma<true>(s[nt][j & 1], a0, a1, a2, a3, qf[nt][4 * h + j][0], qf[nt][4 * h + j][1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma<false>(s[nt][j & 1], xa[2 * j], ya[2 * j], xa[2 * j + 1], ya[2 * j + 1], qf[nt][2 * h + j][0], qf[nt][2 * h + j][1]);
      }
    }
    // keys n and n + 8 of the strip are this lane's; columns 2t, 2t + 1 of each query tile
    const int lo = cur.start - cur.key;
    const bool in0 = whole || (n >= lo && n < have), in1 = whole || (n + 8 >= lo && n + 8 < have);
    float ks0 = 1.f, ks1 = 1.f, vs0 = 1.f, vs1 = 1.f;
    if constexpr (FP8) {
      const uint32_t eb = vb + C::STRIP + n;
      ks0 = exp_scale(lds8(eb));
      ks1 = exp_scale(lds8(eb + 8));
      int v0 = lds8(eb + 16), v1 = lds8(eb + 24);
      if (!whole) v0 = in0 ? v0 : 0, v1 = in1 ? v1 : 0;
      const int top = max(v0, v1);
      if (__any_sync(0xffffffffu, top > ev_ref)) {
        const int ref = max(ev_ref, static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(top))));
        const float f = pow2i(ev_ref - ref);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < C::MT; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[nt][i][c] *= f;
        ev_ref = ref;
      }
      vs0 = __uint_as_float(static_cast<uint32_t>(max(v0 - ev_ref + 127, 0)) << 23);   // 2^(v0 - ev_ref), 0 below 2^-126
      vs1 = __uint_as_float(static_cast<uint32_t>(max(v1 - ev_ref + 127, 0)) << 23);
    }
    float x[NT][4];
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[nt][c] = (s[nt][0][c] + s[nt][1][c]) * (qs[nt][c & 1] * (c < 2 ? ks0 : ks1));
        if (!whole) x[nt][c] = (c < 2 ? in0 : in1) ? x[nt][c] : -INFINITY;
        raise |= x[nt][c] > thr[nt][c & 1];
      }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(x[nt][c], x[nt][c + 2]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          mx = fmaxf(mx, m[nt][c]);
          const float f = mx == -INFINITY ? 1.f : ex2_approx(m[nt][c] - mx);
          m[nt][c] = mx;
          thr[nt][c] = mx + kLazy;
          mb[nt][c] = mx == -INFINITY ? -kBias : mx - kBias;
          l[nt][c] *= f;
#pragma unroll
          for (int i = 0; i < C::MT; ++i) {
            o[nt][i][c] *= f;
            o[nt][i][c + 2] *= f;
          }
        }
    }
    uint32_t pf[NT][2], pl[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float e[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) e[c] = ex2_approx(x[nt][c] - mb[nt][c & 1]);
      l[nt][0] += e[0] + e[2];
      l[nt][1] += e[1] + e[3];
      if constexpr (FP8) {
        pf[nt][0] = movmatrix(pack_f16x2(e[0] * vs0, e[1] * vs0));
        pf[nt][1] = movmatrix(pack_f16x2(e[2] * vs1, e[3] * vs1));
      } else {
        const uint32_t h0 = pack_bf16x2(e[0], e[1]), h1 = pack_bf16x2(e[2], e[3]);
        pf[nt][0] = movmatrix(h0);
        pf[nt][1] = movmatrix(h1);
        pl[nt][0] = movmatrix(pack_bf16x2(e[0] - __uint_as_float(h0 << 16), e[1] - __uint_as_float(h0 & 0xffff0000u)));
        pl[nt][1] = movmatrix(pack_bf16x2(e[2] - __uint_as_float(h1 << 16), e[3] - __uint_as_float(h1 & 0xffff0000u)));
      }
    }
    // out^T += V^T P^T: this lane's four keys 2t, 2t + 1, 2t + 8, 2t + 9 and its columns
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
        const uint32_t a0 = e4m3x2_to_f16x2(w0), a1 = e4m3x2_to_f16x2(w0 >> 16);
        const uint32_t a2 = e4m3x2_to_f16x2(w1), a3 = e4m3x2_to_f16x2(w1 >> 16);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma<true>(o[nt][i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
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
            mma<false>(o[nt][4 * hh + i], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
            mma<false>(o[nt][4 * hh + i], a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
          }
        }
      }
    }
  };

  // ---- the end of a unit's part: join the warps, then write the rows or the part.  The buffers hold the values as the MMAs'
  // results lie in a warp (pair, lane), so that neither side has a bank conflict.
  constexpr int kPairs = NT * C::MT * 2;
  auto end_part = [&](bool whole, int slot) {
    const float poison = __any_sync(0xffffffffu, bad) ? __int_as_float(0x7fffffff) : 0.f;   // a bad page or length
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float s = l[nt][c];
        s += __shfl_xor_sync(0xffffffffu, s, 4);
        s += __shfl_xor_sync(0xffffffffu, s, 8);
        s += __shfl_xor_sync(0xffffffffu, s, 16);
        if (n == 0) join_ml[warp * NQ + nt * 8 + 2 * t + c] = make_float2(m[nt][c], s + poison);
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
        f[nt][c] = m[nt][c] == -INFINITY ? 0.f : ex2_approx(m[nt][c] - mx) * (FP8 ? pow2i(ev_ref - 127) : 1.f);
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
    } else if (tid < NQ) {
      float mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kW; ++w) mx = fmaxf(mx, join_ml[w * NQ + tid].x);
#pragma unroll
      for (int w = 0; w < kW; ++w) {
        const float2 v = join_ml[w * NQ + tid];
        sum += v.x == -INFINITY ? v.y : v.y * ex2_approx(v.x - mx);   // v.y is 0 or NaN without a maximum
      }
      join_ml[kW * NQ + tid] = make_float2(mx, sum);
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
    // what is read from here on (the buffers, the joint (m, l)) is written again only behind the next part's first barrier
    const int h0 = (cur.u / p.subs) * p.group, s0 = (cur.u % p.subs) * NQ;
    for (int e = warp; e < kPairs; e += kW) {
      const int i = e / 2 % C::MT, qi = e / (2 * C::MT) * 8 + 2 * t + (e & 1);
      const int col = FP8 ? (D / 8) * n + 2 * i : (i / 4) * 64 + 8 * n + 2 * (i % 4);
      float2 v = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kW / 2; ++w) {
        const float2 a = join_o[(w * kPairs + e) * 32 + lane];
        v.x += a.x, v.y += a.y;
      }
      if (s0 + qi >= p.group) continue;
      const float2 ml = join_ml[kW * NQ + qi];
      const int64_t at = static_cast<int64_t>(slot) * NQ + qi;
      if (!whole) {
        *reinterpret_cast<float2*>(p.part + at * D + col) = v;
        if (col == 0) *reinterpret_cast<float2*>(p.ml + at * 2) = ml;
      } else {
        const RowEnd r = row_end(p, h0 + s0 + qi, ml.x, ml.y, kBias);
        *reinterpret_cast<uint32_t*>(p.out + (static_cast<int64_t>(cur.b) * p.hq + h0 + s0 + qi) * D + col) = pack_bf16x2(v.x * r.inv, v.y * r.inv);
        if (col == 0) p.lse[static_cast<int64_t>(h0 + s0 + qi) * p.batch + cur.b] = r.lse;
      }
    }
  };

  // ---- the share
  bool fresh = true, first_part = true, from_start = !opens_mid;
  int32_t opened = 0;   // parts of the unit this CTA leaves open to later ones
  int stage = 0, fill = C::STAGES - 1;
#pragma unroll 1
  for (int64_t x = t0; x < t1; ++x) {
    if (ahead < t1) {
      ++ahead;
      load_strip(fill, ahead < t1);
    }
    cp_async_commit();
    fill = fill + 1 == C::STAGES ? 0 : fill + 1;
    if (fresh) begin_unit();
    fresh = false;
    cp_async_wait<C::STAGES - 1>();
    __syncwarp();
    strip(stage);
    __syncwarp();   // the stage has been read by every lane before the next iteration refills it
    stage = stage + 1 == C::STAGES ? 0 : stage + 1;
    if (cur.left > 1 && x + 1 < t1) {
      cur.step();
      continue;
    }
    const bool last = cur.left == 1;
    const int slot = static_cast<int>(2 * cta) + (first_part ? 0 : 1);
    end_part(last && from_start, slot);
    if (!last && from_start) {
      opened = static_cast<int32_t>(share_of(total, parts, x + cur.left - 1) - cta + 1);
      if (tid == 0) {
        JoinDesc d{};
        d.parts = opened;
        d.batch = cur.b;
        d.unit = cur.u;
        d.first_slot = slot;
        p.desc[cta] = d;
      }
    }
    first_part = false;
    from_start = fresh = true;
    if (x + 1 < t1) cur.next_unit(p, units, warp);
  }
  if (opened == 0 && tid == 0) p.desc[cta].parts = 0;
}

// Joins the parts of the unit that CTA blockIdx.x of the main kernel opened: a CTA a q head of the unit (blockIdx.y), D / 4
// threads to a part and as many parts at once as 256 threads hold, then those by the order of their first part.  Every load
// of a round is independent, so a unit of 152 parts takes a few memory latencies.
template <int D, int NT>
__global__ void __launch_bounds__(256) decode_join_kernel(DecodeParams p, float bias) {
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
      ml[i] = *reinterpret_cast<const float2*>(p.ml + at * 2);
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
  const RowEnd r = row_end(p, head, mx, sum, bias);
  *reinterpret_cast<uint2*>(p.out + (static_cast<int64_t>(d.batch) * p.hq + head) * D + 4 * c) =
      make_uint2(pack_bf16x2(v.x * r.inv, v.y * r.inv), pack_bf16x2(v.z * r.inv, v.w * r.inv));
  if (c == 0) p.lse[static_cast<int64_t>(head) * p.batch + d.batch] = r.lse;
}

constexpr size_t kDescBytes = sizeof(JoinDesc) * kMaxCtas;
size_t ml_bytes(int nt) { return size_t{2} * kMaxCtas * 8 * nt * 2 * sizeof(float); }
size_t part_bytes(int nt, int d) { return size_t{2} * kMaxCtas * 8 * nt * d * sizeof(float); }
int tiles_of(int group) { return group > 8 ? 2 : 1; }   // query tiles of 8 a unit

template <int D, bool FP8, int NT>
ffa_status launch(const DecodeParams& p, int sms, cudaStream_t s) {
  using C = Cfg<D, FP8, NT>;
  static_assert(C::STAGES >= 2, "ring");
  auto* kernel = decode_kernel<D, FP8, NT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return FFA_ERR_CUDA;
  const int grid = std::min(sms, kMaxCtas);
  kernel<<<grid, C::THREADS, C::SMEM, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FFA_ERR_CUDA;
  return cuda_status(launch_after(decode_join_kernel<D, NT>, dim3(grid, std::min(8 * NT, p.group)), 256, s, p, FP8 ? 10.f : 0.f));
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
  if (!(scale > -INFINITY && scale < INFINITY)) return FFA_ERR_INVALID_ARG;
  if (batch > 1 && table_stride < max_pages) return FFA_ERR_INVALID_ARG;
  if (hq > (1 << 16) || batch > (1 << 20)) return FFA_ERR_OVERFLOW;
  if (batch == 0) return FFA_OK;
  const int32_t d = cache->d;
  if (!q || !out || !lse || !kv_lens || !workspace) return FFA_ERR_INVALID_ARG;
  if (!kv_aligned16(q) || !kv_aligned16(out) || !kv_aligned16(lse) || !kv_aligned16(workspace)) return FFA_ERR_INVALID_ARG;
  if (max_pages > 0 && !page_table) return FFA_ERR_INVALID_ARG;
  for (const void* a : {static_cast<const void*>(page_table), static_cast<const void*>(kv_lens),
                        static_cast<const void*>(kv_starts), static_cast<const void*>(sink)})
    if (reinterpret_cast<uintptr_t>(a) & 3u) return FFA_ERR_INVALID_ARG;
  if (q_stride % 8 != 0 || (batch > 1 && q_stride < static_cast<int64_t>(hq) * d)) return FFA_ERR_INVALID_ARG;
  if (workspace_bytes < ffa_fwd_decode_workspace_size(hq, cache->hkv, d)) return FFA_ERR_INVALID_ARG;
  const int group = hq / cache->hkv, nt = tiles_of(group);
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
  p.ml = reinterpret_cast<float*>(ws + kDescBytes);
  p.part = reinterpret_cast<float*>(ws + kDescBytes + ml_bytes(nt));
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return FFA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = cache->dtype == FFA_KV_E4M3;
  if (d == 128) {
    if (nt == 1) return fp8 ? launch<128, true, 1>(p, sms, s) : launch<128, false, 1>(p, sms, s);
    return fp8 ? launch<128, true, 2>(p, sms, s) : launch<128, false, 2>(p, sms, s);
  }
  if (nt == 1) return fp8 ? launch<64, true, 1>(p, sms, s) : launch<64, false, 1>(p, sms, s);
  return fp8 ? launch<64, true, 2>(p, sms, s) : launch<64, false, 2>(p, sms, s);
}

}  // extern "C"
