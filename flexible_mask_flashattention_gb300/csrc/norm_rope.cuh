// What the kernels that normalise and rotate head rows share: how a warp walks over tokens and heads, its copies to shared memory,
// and a lane's columns and rotation (norm_rope.cu says why they are so), with the host's checks and sizes.
#pragma once

#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "ffa_internal.h"
#include "launch.h"
#include "ptx.cuh"

namespace ffa {
namespace {   // a copy for each file: kernels' templates are the file's own

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBwdCtas = 1024;   // partial weight gradients the workspace holds
constexpr int kStages = 2;          // units in shared memory: one being used, one on its way
// Heads of a unit: as many as keep the bytes in flight where they do best, or, with so few heads in all that they are one unit, kUnitMost
// (365K tokens of 3 + 3 heads, d = 64: 90 us in one unit, 111 in two; 14K tokens of 64 + 8 heads in units of 6: 87 us, of 5: 82).
// Several axes take larger units, as a unit's table rows cost more (unit_heads).
template <bool BWD>
constexpr int kUnitHeads = BWD ? 4 : 5;
template <bool BWD, bool AXES = false>
constexpr int kUnitMost = BWD ? (AXES ? 5 : 4) : 6;

struct NormRopeParams {
  const __nv_bfloat16* x[3];      // q, k (v, on its way to a cache)
  int64_t x_stride[3];            // values between tokens
  const __nv_bfloat16* dout[2];   // backward: gradients of the outputs, contiguous
  __nv_bfloat16* out[2];          // forward: outputs; backward: dx; contiguous
  const float* w[2];              // null (several axes): no norm, the rotation alone
  int32_t heads[3];
  int32_t unit;                   // heads of a unit (q's, then k's)
  int32_t per;                    // units a group of tokens
  int32_t step_units, step_tokens;   // kWarps units in whole groups' tokens and units
  int64_t tokens;
  int64_t units, span;            // all units, and those of a CTA (consecutive ones)
  float eps;
  const float* cos_sin;
  int64_t max_pos;
  int32_t rot;
  const int32_t* pos;             // [tokens], of several axes [axes][tokens]
  float* partial;                 // backward: [CTAs][2][d]
  int32_t axes;                   // several axes: how many, and which one each pair of columns goes by, 2 bits a pair
  uint32_t pair_axis[4];
  bool chunks;                    // the 4 pairs of every 16-byte chunk of a table row go by one axis
  float turn;                     // several axes, forward: 1, or -1 for the rotation back
};

// The 8 columns of a row that a lane holds, in two runs of 4 such that a rotation's pairs lie in one lane: values 0..3 are columns
// from `lo` on, 4..7 those from `hi` on.  Pairs (i, i + rot / 2): run l of the rotated columns' first half and run l of the second, then
// likewise of the columns from rot on; pairs (2i, 2i + 1): 8 neighbouring columns.
template <int D, bool INTER>
struct Columns {
  int lo, hi;
  __device__ __forceinline__ Columns(int l, int rot) {
    if constexpr (INTER) {
      lo = 8 * l, hi = lo + 4;
    } else {
      const bool in = 8 * l < rot;
      lo = in ? 4 * l : rot / 2 + 4 * l;   // rot + 4 (l - rot / 8)
      hi = lo + (in ? rot : D - rot) / 2;
    }
  }
  __device__ __forceinline__ uint4 load(const uint8_t* row, int swap) const {
    if constexpr (INTER) return *reinterpret_cast<const uint4*>(row + ((2 * lo) ^ swap));
    const uint2 a = *reinterpret_cast<const uint2*>(row + ((2 * lo) ^ swap)), b = *reinterpret_cast<const uint2*>(row + ((2 * hi) ^ swap));
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, const uint4& v) const {
    if constexpr (INTER) {
      *reinterpret_cast<uint4*>(row + lo) = v;
    } else {
      *reinterpret_cast<uint2*>(row + lo) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(row + hi) = make_uint2(v.z, v.w);
    }
  }
  __device__ __forceinline__ void store(uint8_t* row, int swap, const uint4& v) const {   // to shared memory, as load reads it
    if constexpr (INTER) {
      *reinterpret_cast<uint4*>(row + ((2 * lo) ^ swap)) = v;
    } else {
      *reinterpret_cast<uint2*>(row + ((2 * lo) ^ swap)) = make_uint2(v.x, v.y);
      *reinterpret_cast<uint2*>(row + ((2 * hi) ^ swap)) = make_uint2(v.z, v.w);
    }
  }
  __device__ __forceinline__ void load(const float* row, float2 (&f)[4]) const {
    const float4 a = *reinterpret_cast<const float4*>(row + lo), b = *reinterpret_cast<const float4*>(row + hi);
    f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w), f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
  }
  __device__ __forceinline__ int column(int j) const { return j < 4 ? lo + j : hi + j - 4; }
};
// The pair partners of the two values f[j].
template <bool INTER>
__device__ __forceinline__ float2 partner(const float2 (&f)[4], int j) {
  return INTER ? make_float2(f[j].y, f[j].x) : f[j ^ 2];
}

__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y), pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
}

// A lane's part of one token's rotation, forward or (BACK) by the negative angle: value j becomes c(j) v + s(j) (its partner's
// value).  Columns behind rot_dim have c = 1, s = 0.
template <bool INTER, bool BACK>
struct Rotation {
  float2 cos[INTER ? 4 : 2], up[INTER ? 4 : 2], down[2];   // sines: of values 0..3 (interleaved: of all), of values 4..7
  __device__ __forceinline__ void load(const float* row, int rot, int l, float turn = 1.f) {   // turn: 1 or -1
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (8 * l < rot) c = *reinterpret_cast<const float4*>(row + 4 * l), s = *reinterpret_cast<const float4*>(row + rot / 2 + 4 * l);
    if constexpr (BACK) s = make_float4(-s.x, -s.y, -s.z, -s.w);
    s = make_float4(s.x * turn, s.y * turn, s.z * turn, s.w * turn);
    if constexpr (INTER) {
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) cos[i] = make_float2(cc[i], cc[i]), up[i] = make_float2(-ss[i], ss[i]);
    } else {
      cos[0] = make_float2(c.x, c.y), cos[1] = make_float2(c.z, c.w);
      up[0] = make_float2(-s.x, -s.y), up[1] = make_float2(-s.z, -s.w);
      down[0] = make_float2(s.x, s.y), down[1] = make_float2(s.z, s.w);
    }
  }
  __device__ __forceinline__ float2 c(int j) const { return INTER ? cos[j] : cos[j & 1]; }
  __device__ __forceinline__ float2 s(int j) const {
    if constexpr (INTER) return up[j];
    else return j < 2 ? up[j] : down[j & 1];
  }
};

// Sums over the D / 8 lanes of a row, of several rows whose chains of exchanges run side by side.
template <int D, int N>
__device__ __forceinline__ void row_sums(float (&v)[N]) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}
// f(count, i) for batches of N = 2 or 3, then fewer, that cover 0 .. n - 1.
template <int N, typename F>
__device__ __forceinline__ void in_batches(int n, F& f) {
  int i = 0;
#pragma unroll 1
  for (; i + N <= n; i += N) f(std::integral_constant<int, N>{}, i);
  if constexpr (N > 2) {
    if (i + 2 <= n) f(std::integral_constant<int, 2>{}, i), i += 2;
  }
  if (i < n) f(std::integral_constant<int, 1>{}, i);
}

// Where a warp stands in its units: unit `c` of its 256 / D tokens' units; this lane's token (behind the last one: has = false) and its
// position.  Of several axes lane l of a token's D / 8 reads the position on axis l % 4, and `pos` says, once all have come (settle), whether
// they are good: negative if one is, behind the table if one is, else any good one.
template <int D, bool AXES = false>
struct UnitWalk {
  static constexpr int kGroup = 256 / D;   // tokens a warp
  int64_t token;
  int left;        // units of the CTA's from this one on
  int c, pos;
  int mine;        // several axes: the position this lane has read
  bool has;
  __device__ __forceinline__ void read_pos(const NormRopeParams& p) {
    has = left > 0 && token < p.tokens;
    if constexpr (AXES) mine = has ? __ldg(p.pos + min(static_cast<int>(threadIdx.x) & 3, p.axes - 1) * p.tokens + token) : -1;
    else pos = has ? __ldg(p.pos + token) : -1;
  }
  __device__ __forceinline__ void settle(const NormRopeParams& p) {   // by all lanes of the warp
    const uint32_t token_lanes = (D == 128 ? 0xffffu : 0xffu) << (threadIdx.x & (32 - D / 8));
    const uint32_t low = __ballot_sync(0xffffffffu, mine < 0), far = __ballot_sync(0xffffffffu, mine >= p.max_pos);
    pos = low & token_lanes ? -1 : far & token_lanes ? 0x7fffffff : 0;
  }
  __device__ __forceinline__ void init(const NormRopeParams& p, int warp, int sub) {
    const int64_t begin = blockIdx.x * p.span, first = begin + warp, group = first / p.per;
    left = static_cast<int>(min(p.span, p.units - begin)) - warp;
    token = group * kGroup + sub;
    c = static_cast<int>(first - group * p.per);
    read_pos(p);
  }
  __device__ __forceinline__ void next(const NormRopeParams& p) {   // the warp's next unit: kWarps further
    left -= kWarps;
    c += p.step_units;
    token += p.step_tokens;
    if (c >= p.per) c -= p.per, token += kGroup;
  }
};

// A warp's stages in shared memory: of every head of a unit its tokens' rows, x [unit][token][D], in the backward dout likewise, then
// the table's rows [token][D] (fp32).  At d = 64 odd tokens have their rows' halves swapped, so that two tokens' neighbouring runs
// of 4 columns lie in different banks.
template <int D, bool BWD>
struct Stages {
  static constexpr int kTokens = 256 / D;
  uint8_t* base;    // this warp's
  int unit;
  static __host__ __device__ constexpr int stage_bytes(int unit) { return kTokens * D * (2 * unit * (BWD ? 2 : 1) + 4); }
  static __host__ __device__ constexpr int bytes(int unit) { return kWarps * kStages * stage_bytes(unit); }
  __device__ __forceinline__ uint8_t* rows(int stage, int sub, int tensor) const {   // tensor 0: x, 1: dout; heads 512 bytes apart
    return base + stage * stage_bytes(unit) + tensor * unit * 512 + sub * (2 * D);
  }
  __device__ __forceinline__ float* table(int stage, int sub) const {
    return reinterpret_cast<float*>(base + stage * stage_bytes(unit) + (BWD ? 2 : 1) * unit * 512) + sub * D;
  }
  static __device__ __forceinline__ int swap(int sub) { return D == 64 && (sub & 1) ? 64 : 0; }   // XORed to a byte's place in its row
};

// The part of a unit in one tensor: `n` heads from `head` on, from place `first` of the unit on.
struct UnitPart {
  int n, first, head;
};
__device__ __forceinline__ UnitPart part_of(const NormRopeParams& p, int c, int t) {
  const int from = t == 0 ? 0 : t == 1 ? p.heads[0] : p.heads[0] + p.heads[1], j0 = c * p.unit, a = max(j0, from), b = min(j0 + p.unit, from + p.heads[t]);
  return UnitPart{b - a, a - j0, a - from};
}

// Copy `n` heads' rows of a unit's part, 16 bytes a lane each, or (bytes 0) fill them with zeros.
template <int D, bool BWD>
__device__ __forceinline__ void copy_rows(uint32_t to, const __nv_bfloat16* x, int n, int bytes) {
#pragma unroll
  for (int i = 0; i < kUnitMost<BWD>; ++i) {
    if (i >= n) break;
    cp_async16(to + i * 512, x + i * D, bytes);
  }
}

// Copy a token's table row, with the lanes of the token: 16-byte chunks l and l + D / 8 of it.  Of several axes lane l takes the cosines
// and the sines of pairs 4l .. 4l + 3, if every such chunk goes by one axis, or of pairs l, l + D / 8, ...: neighbouring lanes then copy
// neighbouring values, as far as they are of one row.
template <int D, bool AXES>
__device__ __forceinline__ void copy_table(const NormRopeParams& p, uint32_t to, const UnitWalk<D, AXES>& w, int l, bool live) {
  constexpr int L = D / 8;
  if constexpr (!AXES) {
    if (!live) return;
    const float* row = p.cos_sin + static_cast<int64_t>(w.pos) * p.rot;
    if (4 * l < p.rot) cp_async16(to + 16 * l, row + 4 * l);
    if (4 * (l + L) < p.rot) cp_async16(to + 16 * (l + L), row + 4 * (l + L));
  } else {
    const int half = p.rot / 2;
    auto axis_of = [&](int pair) {
      const uint32_t lo = pair & 16 ? p.pair_axis[1] : p.pair_axis[0], hi = pair & 16 ? p.pair_axis[3] : p.pair_axis[2];
      return static_cast<int>((pair & 32 ? hi : lo) >> (2 * (pair & 15)) & 3u);
    };
    auto row_of = [&](int pair) {   // of the axis that the pair goes by; shuffled by all lanes
      return p.cos_sin + static_cast<int64_t>(__shfl_sync(0xffffffffu, w.mine, axis_of(pair), L)) * p.rot;
    };
    // through L1: thousands of tokens have one time, so that the rows of a few positions are asked of L2 from all sides (128K tokens of 64 + 8
    // heads: d = 64 367 us, 480 to 546 past L1; d = 128 725 and 734)
    if (p.chunks) {
      const float* row = row_of(4 * l);
      if (live && 4 * l < half) {
        cp_async16_l1(to + 16 * l, row + 4 * l);
        cp_async16_l1(to + 16 * l + 4 * half, row + half + 4 * l);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int pair = l + L * i;
        const float* row = row_of(pair) + pair;
        if (live && pair < half) {
          cp_async4(to + 4 * pair, row);
          cp_async4(to + 4 * (half + pair), row + half);
        }
      }
    }
  }
}

// The rotation alone, of fewer columns than a row has: a kernel of its own (AS_IS) copies the others, since the products would make NaN of what
// stands beside an infinity there, as 0 times it.  In one kernel for all, 128K tokens of 64 + 8 heads with a norm took 738 us for 732, and the append
// of 67K tokens of 16 + 4 into 4 bits, read back, 176 for 171.
inline bool copies_columns(const NormRopeParams& p, int d) { return !p.w[0] && p.rot < d; }

// Start the copies of one unit into `stage`.  The rows of a token without a valid position, and of none, are filled with zeros:
// they are not read, so that nothing in them reaches a sum.
template <int D, bool BWD, bool AXES, typename P>
__device__ __forceinline__ void copy_unit(const P& p, const Stages<D, BWD>& st, int stage, const UnitWalk<D, AXES>& w) {
  const int lane = threadIdx.x & 31, l = lane & (D / 8 - 1), sub = lane / (D / 8);
  const bool live = w.pos >= 0 && w.pos < p.max_pos;
  const int64_t token = live ? w.token : 0;
  const int bytes = live ? 16 : 0, at = (16 * l) ^ Stages<D, BWD>::swap(sub);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const UnitPart r = part_of(p, w.c, t);
    if (r.n <= 0) continue;
    const __nv_bfloat16* x = p.x[t] + token * p.x_stride[t] + r.head * D + 8 * l;
    const __nv_bfloat16* g = BWD ? p.dout[t] + (token * p.heads[t] + r.head) * D + 8 * l : nullptr;
    const uint32_t to = smem_u32(st.rows(stage, sub, 0)) + r.first * 512 + at, to_g = smem_u32(st.rows(stage, sub, 1)) + r.first * 512 + at;
#pragma unroll
    for (int i = 0; i < kUnitMost<BWD, AXES>; ++i) {
      if (i >= r.n) break;
      cp_async16(to + i * 512, x + i * D, bytes);
      if constexpr (BWD) cp_async16(to_g + i * 512, g + i * D, bytes);
    }
  }
  copy_table<D, AXES>(p, smem_u32(st.table(stage, sub)), w, l, live);
}

// Several axes (0: one position a token): how many, and the axis of every pair (null: one axis).
inline ffa_status check_axes(int32_t axes, const uint8_t* pair_axis, int32_t rot, NormRopeParams& p) {
  if (axes < 0 || (axes > 1 && !pair_axis)) return FFA_ERR_INVALID_ARG;
  if (axes > 4) return FFA_ERR_UNSUPPORTED;
  p.axes = axes;
  p.turn = 1.f;
  p.chunks = true;
  for (int i = 0; axes && pair_axis && i < rot / 2; ++i) {
    if (pair_axis[i] >= axes) return FFA_ERR_INVALID_ARG;
    p.pair_axis[i / 16] |= static_cast<uint32_t>(pair_axis[i]) << (2 * (i % 16));
    p.chunks &= pair_axis[i] == pair_axis[i / 4 * 4];
  }
  return FFA_OK;
}

// The checks both directions share; fills what they have in common.
inline ffa_status check_common(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens, int32_t hq,
                        int32_t hkv, int32_t d, const float* qw, const float* kw, float eps, const float* cos_sin,
                        int64_t max_pos, int32_t rot, const int32_t* pos, int32_t axes, const uint8_t* pair_axis,
                        NormRopeParams& p) {
  if (tokens < 0 || hq <= 0 || hkv <= 0 || max_pos <= 0) return FFA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FFA_ERR_UNSUPPORTED;
  if (rot < 16 || rot > d || rot % 16 != 0) return FFA_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || eps > 1e30f) return FFA_ERR_INVALID_ARG;
  if (!cos_sin || (axes ? !qw != !kw : !qw || !kw)) return FFA_ERR_INVALID_ARG;   // of several axes: both weights or none
  if (!aligned16(qw) || !aligned16(kw) || !aligned16(cos_sin)) return FFA_ERR_INVALID_ARG;
  if (tokens > 0) {
    if (!q || !k || !pos || !aligned16(q) || !aligned16(k)) return FFA_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(pos) & 3u) return FFA_ERR_INVALID_ARG;
    if (q_stride % 8 != 0 || k_stride % 8 != 0) return FFA_ERR_INVALID_ARG;
    if (tokens > 1 && (q_stride < static_cast<int64_t>(hq) * d || k_stride < static_cast<int64_t>(hkv) * d))
      return FFA_ERR_INVALID_ARG;
  }
  if (hq > (1 << 16) || hkv > (1 << 16) || tokens > (int64_t{1} << 36)) return FFA_ERR_OVERFLOW;
  p.x[0] = static_cast<const __nv_bfloat16*>(q);
  p.x[1] = static_cast<const __nv_bfloat16*>(k);
  p.x_stride[0] = q_stride;
  p.x_stride[1] = k_stride;
  p.w[0] = qw;
  p.w[1] = kw;
  p.heads[0] = hq;
  p.heads[1] = hkv;
  p.eps = eps;
  p.cos_sin = cos_sin;
  p.max_pos = max_pos;
  p.rot = rot;
  p.pos = pos;
  return check_axes(axes, pair_axis, rot, p);
}

// Cut the heads of a group of tokens into `per` units of `unit` heads at most.
inline void cut_units(NormRopeParams& p, int64_t tokens, int d, int64_t per, int64_t unit) {
  const int group = 256 / d;
  p.tokens = tokens;
  p.unit = static_cast<int32_t>(unit);
  p.per = static_cast<int32_t>(per);
  p.units = (tokens + group - 1) / group * per;
  p.step_units = kWarps % p.per;
  p.step_tokens = kWarps / p.per * group;
}

// Heads of a unit at most where there are several units a token.  Of several axes (us, with kUnitHeads and so): forward 128K
// tokens of 64 + 8 heads, d = 128, sections 759 and 725, axes in turns 812 and 733; backward 32K such tokens 287 and 281, 302 and 296, 128K tokens of
// 12 + 2 heads 250 and 222, 265 and 243; but 64K tokens of 64 + 8 heads, d = 64, in turns, backward 303 and 315.
template <bool BWD>
int64_t unit_heads(const NormRopeParams& p, int d) {
  const bool larger = p.axes > 1 && (!BWD || p.chunks || d == 128);
  return larger ? kUnitMost<BWD, true> : kUnitHeads<BWD>;
}

// Units for `warps` resident warps: equal sizes, unit_heads at most, and smaller ones where there would be fewer units than warps.
template <bool BWD>
void set_units(NormRopeParams& p, int64_t tokens, int d, int64_t warps) {
  const int group = 256 / d;
  const int64_t groups = (tokens + group - 1) / group, all = p.heads[0] + p.heads[1];
  const int64_t most = unit_heads<BWD>(p, d);
  const int64_t fewest = all <= std::max<int64_t>(most, kUnitMost<BWD>) ? 1 : (all + most - 1) / most;
  const int64_t per = std::max(fewest, std::min(all, warps / std::max<int64_t>(groups, 1)));
  const int64_t unit = (all + per - 1) / per;
  cut_units(p, tokens, d, (all + unit - 1) / unit, unit);
}

template <int D, bool BWD>
constexpr int smem_bytes(int unit) {
  return (BWD ? 1 + kWarps : 1) * 2 * D * 4 + Stages<D, BWD>::bytes(unit);
}

// CTAs of `kernel` the whole device holds at its largest shared memory.  The figure depends on the kernel and the device's
// type alone, so it is asked for once a device (`known`, 0 before; two threads would store the same).
template <typename K>
int resident(K* kernel, int smem, int device, int sms, std::atomic<int> (&known)[kDevices]) {
  int n = device < kDevices ? known[device].load(std::memory_order_relaxed) : 0;
  if (n) return n;
  int per = 0;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, smem) != cudaSuccess)
    return 0;
  n = per * sms;
  if (device < kDevices) known[device].store(n, std::memory_order_relaxed);
  return n;
}

// Launch a kernel over all units; P is or extends NormRopeParams.  `known` and `raised` are the kernel's own.
template <int D, bool BWD, bool AXES, typename P>
ffa_status launch_units(void (*kernel)(P), P p, int64_t tokens, cudaStream_t s, int* ctas, std::atomic<int> (&known)[kDevices],
                        std::atomic<bool> (&raised)[kDevices]) {
  constexpr int kMost = smem_bytes<D, BWD>(kUnitMost<BWD, AXES>);
  int device = 0, sms = 0;
  if (!current_device(device, sms)) return FFA_ERR_CUDA;
  const int held = resident(kernel, kMost, device, sms, known);
  if (held == 0) return FFA_ERR_CUDA;
  set_units<BWD>(p, tokens, D, static_cast<int64_t>(held) * kWarps);
  // consecutive units to each CTA, all CTAs resident at once (64K tokens, 16 + 4 heads, d = 128, measured with CTAs of 4 warps: 112
  // us forward and 170 us backward, against 120 to 125 and 180 to 184 us with CTAs of 2 to 32 units a warp)
  const int64_t most = std::min(held, kMaxBwdCtas);
  p.span = std::max<int64_t>((p.units + most - 1) / most, 1);
  p.span = (p.span + kWarps - 1) / kWarps * kWarps;
  if (p.span > 0x40000000) return FFA_ERR_OVERFLOW;
  const int grid = static_cast<int>((p.units + p.span - 1) / p.span);
  *ctas = grid;
  if (grid == 0) return FFA_OK;
  return cuda_status(launch_large(kernel, dim3(grid), kThreads, smem_bytes<D, BWD>(p.unit), kMost, s, device, raised, p));
}

}  // namespace
}  // namespace ffa
