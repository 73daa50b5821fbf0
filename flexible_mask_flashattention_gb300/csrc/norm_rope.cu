// RMS norm of every query and key head row with the position rotation in the same pass, forward and backward.
//
// For a head row x of d values with weight w and position p (r = 1 / sqrt(mean x^2 + eps)):
//   y = r x w,   out = R(p) y,
// R(p) rotating the first rot_dim columns in pairs (a, b) by the table's angle i of position p:
//   out_a = y_a cos_i - y_b sin_i,   out_b = y_b cos_i + y_a sin_i.
// With g = R(p)^T dout and h = w g the gradients are
//   dw = sum over rows of g r x,     dx = r (h - x r^2 mean(h x)).
// r is recomputed in the backward from x, which it reads anyway, so the forward stores nothing for it.
//
// Both are bound by HBM: 4 bytes a value forward (x in, out out), 6 backward (x, dout in, dx out).  A warp takes 2 or 4
// neighbouring tokens, d / 8 lanes a token, one head of each at a time, so that a token's rotation is read once for many heads and
// no head count leaves lanes empty; a lane's 8 columns are two runs of 4 whose values are each other's pair partners, so that the
// rotation exchanges nothing.  The kernels are persistent: a warp walks over units of up to 5 (backward: 4) heads of its
// tokens, and cp.async keeps the next unit's values and table rows on their way to shared memory.  A unit's sums are taken for
// several heads side by side, as one head's exchanges would leave the warp waiting.  Norm statistics, rotation and every gradient sum are
// fp32, two values an instruction (fma.rn.f32x2); the one rounding to bf16 is the store's.
//
// What decides at this bandwidth is how the copies reach memory.  The 8 warps of a CTA take consecutive units and start each round's
// copies together, behind a barrier: 4 tokens (20 KB) then arrive as one run, where warps on their own spread 2.5 KB pieces over the
// memory.  And more in flight is slower: 57 KB an SM does best.  Measured on one GPU at 64K tokens, 16 + 4 heads, d = 128
// (forward and backward): 107 and 157 us (94 and 95 % of a copy's 6795 GB/s); CTAs of 4 warps, as many bytes in flight, 109 and 162, with
// more in flight 127, without the barrier 119 and 176; of 16 warps 110 and 164; units of 4 and 5 heads 110 and 159, of 10 and 7
// 115 and 185.  Bulk copies (cp.async.bulk) took 110 and 164 where these took 109 and 172, and 0.1 to 0.5 us longer for small
// batches.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "ffa_internal.h"
#include "launch.h"
#include "ptx.cuh"

namespace ffa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBwdCtas = 1024;   // partial weight gradients the workspace holds
constexpr int kStages = 2;          // units in shared memory: one being used, one on its way
// Heads of a unit at most, and with so few heads in all that they are one unit (365K tokens of 3 + 3 heads, d = 64: 90 us in one
// unit, 111 in two; 14K tokens of 64 + 8 heads in units of 6: 87 us, of 5: 82).
template <bool BWD>
constexpr int kUnitHeads = BWD ? 4 : 5;
template <bool BWD>
constexpr int kUnitMost = BWD ? 4 : 6;

struct NormRopeParams {
  const __nv_bfloat16* x[2];      // q, k
  int64_t x_stride[2];            // values between tokens
  const __nv_bfloat16* dout[2];   // backward: gradients of the outputs, contiguous
  __nv_bfloat16* out[2];          // forward: outputs; backward: dx; contiguous
  const float* w[2];
  int32_t heads[2];
  int32_t unit;                   // heads of a unit (q's, then k's)
  int32_t per;                    // units a group of tokens
  int32_t step_units, step_tokens;   // kWarps units in whole groups' tokens and units
  int64_t tokens;
  int64_t units, span;            // all units, and those of a CTA (consecutive ones)
  float eps;
  const float* cos_sin;
  int64_t max_pos;
  int32_t rot;
  const int32_t* pos;
  float* partial;                 // backward: [CTAs][2][d]
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
  __device__ __forceinline__ void load(const float* row, int rot, int l) {
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (8 * l < rot) c = *reinterpret_cast<const float4*>(row + 4 * l), s = *reinterpret_cast<const float4*>(row + rot / 2 + 4 * l);
    if constexpr (BACK) s = make_float4(-s.x, -s.y, -s.z, -s.w);
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
// position.
template <int D>
struct UnitWalk {
  static constexpr int kGroup = 256 / D;   // tokens a warp
  int64_t token;
  int left;        // units of the CTA's from this one on
  int c, pos;
  bool has;
  __device__ __forceinline__ void read_pos(const NormRopeParams& p) {
    has = left > 0 && token < p.tokens;
    pos = has ? __ldg(p.pos + token) : -1;
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
  const int from = t ? p.heads[0] : 0, j0 = c * p.unit, a = max(j0, from), b = min(j0 + p.unit, from + p.heads[t]);
  return UnitPart{b - a, a - j0, a - from};
}

// Start the copies of one unit into `stage`.  The rows of a token without a valid position, and of none, are filled with zeros:
// they are not read, so that nothing in them reaches a sum.
template <int D, bool BWD>
__device__ __forceinline__ void copy_unit(const NormRopeParams& p, const Stages<D, BWD>& st, int stage, const UnitWalk<D>& w) {
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
    for (int i = 0; i < kUnitMost<BWD>; ++i) {
      if (i >= r.n) break;
      cp_async16(to + i * 512, x + i * D, bytes);
      if constexpr (BWD) cp_async16(to_g + i * 512, g + i * D, bytes);
    }
  }
  if (live) {
    const float* row = p.cos_sin + static_cast<int64_t>(w.pos) * p.rot;
    const uint32_t to = smem_u32(st.table(stage, sub));
    if (4 * l < p.rot) cp_async16(to + 16 * l, row + 4 * l);
    if (4 * (l + D / 8) < p.rot) cp_async16(to + 16 * (l + D / 8), row + 4 * (l + D / 8));
  }
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(NormRopeParams p) {
  constexpr int L = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  float* weights = reinterpret_cast<float*>(smem);   // [2][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (L - 1), sub = lane / L;
  const Stages<D, false> st{smem + 2 * D * 4 + warp * kStages * Stages<D, false>::stage_bytes(p.unit), p.unit};
  const Columns<D, INTER> cols(l, p.rot);
  const int swap = Stages<D, false>::swap(sub);
  UnitWalk<D> cur, ld;
  cur.init(p, warp, sub);
  ld = cur;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (ld.left > 0) copy_unit<D, false>(p, st, s, ld);
    cp_async_commit();
    ld.next(p);
    ld.read_pos(p);
  }
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) weights[i] = p.w[i / D][i % D];
  __syncthreads();
  int stage = 0, fill = kStages - 1;
  for (int todo = cur.left + warp; todo > 0; todo -= kWarps, cur.next(p)) {
    __syncthreads();   // the warps' copies go out together: one run of memory
    if (cur.left <= 0) continue;
    cur.read_pos(p);   // again: from L1
    if (ld.left > 0) copy_unit<D, false>(p, st, fill, ld);
    cp_async_commit();
    ld.next(p);
    ld.read_pos(p);   // a unit ahead of its use
    cp_async_wait<kStages - 1>();
    __syncwarp();   // lanes read what others copied
    const int pos = cur.pos;
    const bool live = pos >= 0 && pos < p.max_pos;
    // a padded token (negative position) gives zeros, one behind the table NaN
    const uint32_t fill_bits = pos < 0 ? 0u : 0x7fff7fffu;
    const uint4 constant = make_uint4(fill_bits, fill_bits, fill_bits, fill_bits);
    Rotation<INTER, false> rot;
    rot.load(st.table(stage, sub), live ? p.rot : 0, l);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const UnitPart u = part_of(p, cur.c, t);
      if (u.n <= 0) continue;
      __nv_bfloat16* out = p.out[t] + (cur.token * p.heads[t] + u.head) * D;
      const uint8_t* in = st.rows(stage, sub, 0) + u.first * 512;
      // coefficients with the weights: out_j = r (x_j a_j + partner_j b_j)
      float2 w[4], a[4], b[4];
      cols.load(weights + t * D, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = mul2(w[j], rot.c(j)), b[j] = mul2(partner<INTER>(w, j), rot.s(j));
      auto some = [&](auto count, int i) {   // `count` heads from i on, their sums side by side
        constexpr int N = decltype(count)::value;
        float2 f[N][4];
        float r[N];
#pragma unroll
        for (int h = 0; h < N; ++h) {
          unpack8(cols.load(in + (i + h) * 512, swap), f[h]);
          float2 ss = mul2(f[h][0], f[h][0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) ss = fma2(f[h][j], f[h][j], ss);
          r[h] = ss.x + ss.y;
        }
        row_sums<D>(r);
#pragma unroll
        for (int h = 0; h < N; ++h) {
          r[h] = rsqrtf(r[h] * (1.f / D) + p.eps);
          float2 o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = mul2(fma2(f[h][j], a[j], mul2(partner<INTER>(f[h], j), b[j])), make_float2(r[h], r[h]));
          if (live) cols.store(out + (i + h) * D, pack8(o));
          else if (cur.has) cols.store(out + (i + h) * D, constant);
        }
      };
      in_batches<3>(u.n, some);
    }
    __syncwarp();   // the stage's table row has been read by every lane before the next iteration refills it
    stage = stage + 1 == kStages ? 0 : stage + 1;
    fill = fill + 1 == kStages ? 0 : fill + 1;
  }
}

// Each lane keeps its 8 columns' weight-gradient sums for q and k in registers; a CTA adds its warps' in a fixed order and writes
// one partial row pair, which norm_rope_dw_kernel adds up.  The assignment of units to warps is static, so
// the result does not depend on timing.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(NormRopeParams p) {
  constexpr int L = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  float* weights = reinterpret_cast<float*>(smem);   // [2][D]
  float* red = weights + 2 * D;                      // [kWarps][2][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (L - 1), sub = lane / L;
  const Stages<D, true> st{smem + (1 + kWarps) * 2 * D * 4 + warp * kStages * Stages<D, true>::stage_bytes(p.unit), p.unit};
  const Columns<D, INTER> cols(l, p.rot);
  const int swap = Stages<D, true>::swap(sub);
  UnitWalk<D> cur, ld;
  cur.init(p, warp, sub);
  ld = cur;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (ld.left > 0) copy_unit<D, true>(p, st, s, ld);
    cp_async_commit();
    ld.next(p);
    ld.read_pos(p);
  }
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) weights[i] = p.w[i / D][i % D];
  __syncthreads();
  allow_dependents();
  float2 acc[2][4] = {};
  int stage = 0, fill = kStages - 1;
  for (int todo = cur.left + warp; todo > 0; todo -= kWarps, cur.next(p)) {
    __syncthreads();   // the warps' copies go out together: one run of memory
    if (cur.left <= 0) continue;
    cur.read_pos(p);   // again: from L1
    if (ld.left > 0) copy_unit<D, true>(p, st, fill, ld);
    cp_async_commit();
    ld.next(p);
    ld.read_pos(p);
    cp_async_wait<kStages - 1>();
    __syncwarp();   // lanes read what others copied
    const int pos = cur.pos;
    const bool live = pos >= 0 && pos < p.max_pos;
    // a padded token (negative position) gives zeros, one behind the table NaN
    const uint32_t fill_bits = pos < 0 ? 0u : 0x7fff7fffu;
    const uint4 constant = make_uint4(fill_bits, fill_bits, fill_bits, fill_bits);
    Rotation<INTER, true> rot;   // R^T turns by the negative angle
    rot.load(st.table(stage, sub), live ? p.rot : 0, l);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const UnitPart u = part_of(p, cur.c, t);
      if (u.n <= 0) continue;
      __nv_bfloat16* dx = p.out[t] + (cur.token * p.heads[t] + u.head) * D;
      if (!live && pos >= 0)   // a position behind the table makes the weight's gradient NaN too
        acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = make_float2(__int_as_float(0x7fffffff), __int_as_float(0x7fffffff));
      const uint8_t *in = st.rows(stage, sub, 0) + u.first * 512, *in_g = st.rows(stage, sub, 1) + u.first * 512;
      float2 w[4];
      cols.load(weights + t * D, w);
      auto some = [&](auto count, int k) {
        constexpr int N = decltype(count)::value;
        float2 f[N][4], g[N][4];
        float r[N], c[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const uint4 v = cols.load(in + (k + n) * 512, swap), gv = cols.load(in_g + (k + n) * 512, swap);
          float2 d[4], ss = make_float2(0.f, 0.f), hx = make_float2(0.f, 0.f);
          unpack8(v, f[n]);
          unpack8(gv, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[n][i] = fma2(d[i], rot.c(i), mul2(partner<INTER>(d, i), rot.s(i)));
            ss = fma2(f[n][i], f[n][i], ss);
            hx = fma2(mul2(g[n][i], w[i]), f[n][i], hx);
          }
          r[n] = ss.x + ss.y;
          c[n] = hx.x + hx.y;
        }
        row_sums<D>(r);   // by all lanes, live or not
        row_sums<D>(c);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          r[n] = live ? rsqrtf(r[n] * (1.f / D) + p.eps) : 0.f;   // 0: adds nothing
          c[n] = -c[n] * (r[n] * r[n]) * (r[n] * (1.f / D));
          float2 o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[n][i] = mul2(g[n][i], make_float2(r[n], r[n]));
            o[i] = fma2(f[n][i], make_float2(c[n], c[n]), mul2(g[n][i], w[i]));   // dx = r h - x r^3 mean(h x)
            acc[t][i] = fma2(g[n][i], f[n][i], acc[t][i]);
          }
          if (live) cols.store(dx + (k + n) * D, pack8(o));
          else if (cur.has) cols.store(dx + (k + n) * D, constant);
        }
      };
      in_batches<2>(u.n, some);
    }
    __syncwarp();
    stage = stage + 1 == kStages ? 0 : stage + 1;
    fill = fill + 1 == kStages ? 0 : fill + 1;
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float s = j & 1 ? acc[t][j / 2].y : acc[t][j / 2].x;
#pragma unroll
      for (int o = L; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (sub == 0) red[(warp * 2 + t) * D + cols.column(j)] = s;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) s += red[k * 2 * D + i];
    p.partial[blockIdx.x * static_cast<int64_t>(2 * D) + i] = s;
  }
}

// dw = sum of the CTAs' partial rows, in a fixed order: 32 columns a block, 32 partial rows at a time.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* partial, int n, float* dqw, float* dkw) {
  __shared__ float red[32][33];
  wait_for_primary();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  float s = 0.f;
  for (int i = r; i < n; i += 32) s += partial[static_cast<int64_t>(i) * (2 * D) + c];
  red[r][threadIdx.x & 31] = s;
  __syncthreads();
  s = red[threadIdx.x & 31][r];   // column r of the block, partial row by lane
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) {
    const int col = blockIdx.x * 32 + r;
    (col < D ? dqw : dkw)[col % D] = s;
  }
}

// The checks both directions share; fills what they have in common.
ffa_status check_common(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens, int32_t hq,
                        int32_t hkv, int32_t d, const float* qw, const float* kw, float eps, const float* cos_sin,
                        int64_t max_pos, int32_t rot, const int32_t* pos, NormRopeParams& p) {
  if (tokens < 0 || hq <= 0 || hkv <= 0 || max_pos <= 0) return FFA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FFA_ERR_UNSUPPORTED;
  if (rot < 16 || rot > d || rot % 16 != 0) return FFA_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || eps > 1e30f) return FFA_ERR_INVALID_ARG;
  if (!qw || !kw || !cos_sin) return FFA_ERR_INVALID_ARG;
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
  return FFA_OK;
}

// Units for `warps` resident warps: the heads of a group of tokens are cut into units of equal size, kUnitHeads or kUnitMost at
// most, and smaller ones where there would be fewer units than warps.
template <bool BWD>
void set_units(NormRopeParams& p, int64_t tokens, int d, int64_t warps) {
  const int group = 256 / d;
  const int64_t groups = (tokens + group - 1) / group, all = p.heads[0] + p.heads[1];
  const int64_t fewest = all <= kUnitMost<BWD> ? 1 : (all + kUnitHeads<BWD> - 1) / kUnitHeads<BWD>;
  const int64_t per = std::max(fewest, std::min(all, warps / std::max<int64_t>(groups, 1)));
  p.tokens = tokens;
  p.unit = static_cast<int32_t>((all + per - 1) / per);
  p.per = static_cast<int32_t>((all + p.unit - 1) / p.unit);
  p.units = groups * p.per;
  p.step_units = kWarps % p.per;
  p.step_tokens = kWarps / p.per * group;
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

template <int D, bool INTER, bool BWD>
ffa_status launch(NormRopeParams p, int64_t tokens, cudaStream_t s, int* ctas) {
  auto* kernel = [] {
    if constexpr (BWD) return norm_rope_bwd_kernel<D, INTER>;
    else return norm_rope_fwd_kernel<D, INTER>;
  }();
  static std::atomic<int> known[kDevices];
  constexpr int kMost = smem_bytes<D, BWD>(kUnitMost<BWD>);
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
  static std::atomic<bool> raised[kDevices];
  return cuda_status(launch_large(kernel, dim3(grid), kThreads, smem_bytes<D, BWD>(p.unit), kMost, s, device, raised, p));
}

template <bool BWD>
ffa_status launch_any(const NormRopeParams& p, int64_t tokens, int d, bool interleaved, cudaStream_t s, int* ctas) {
  if (d == 128) return interleaved ? launch<128, true, BWD>(p, tokens, s, ctas) : launch<128, false, BWD>(p, tokens, s, ctas);
  return interleaved ? launch<64, true, BWD>(p, tokens, s, ctas) : launch<64, false, BWD>(p, tokens, s, ctas);
}

}  // namespace
}  // namespace ffa

using namespace ffa;

extern "C" {

ffa_status ffa_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                            int32_t hq, int32_t hkv, int32_t d, const float* q_weight, const float* k_weight, float eps,
                            const float* cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                            const int32_t* positions, void* q_out, void* k_out, void* stream) {
  NormRopeParams p{};
  const ffa_status st = check_common(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin,
                                     max_pos, rot_dim, positions, p);
  if (st != FFA_OK) return st;
  if (tokens == 0) return FFA_OK;
  if (!q_out || !k_out || !aligned16(q_out) || !aligned16(k_out)) return FFA_ERR_INVALID_ARG;
  const Span in[] = {{q, span_bytes(tokens, q_stride, hq, d)}, {k, span_bytes(tokens, k_stride, hkv, d)},
                     {q_weight, 4 * d}, {k_weight, 4 * d}, {cos_sin, 4 * max_pos * rot_dim}, {positions, 4 * tokens}};
  const Span outs[] = {{q_out, 2 * tokens * hq * d}, {k_out, 2 * tokens * hkv * d}};
  if (any_meet(outs, 2, in, 6)) return FFA_ERR_INVALID_ARG;
  p.out[0] = static_cast<__nv_bfloat16*>(q_out);
  p.out[1] = static_cast<__nv_bfloat16*>(k_out);
  int ctas = 0;
  return launch_any<false>(p, tokens, d, interleaved != 0, static_cast<cudaStream_t>(stream), &ctas);
}

size_t ffa_qk_norm_rope_bwd_workspace_size(int32_t d) {
  return d == 64 || d == 128 ? static_cast<size_t>(kMaxBwdCtas) * 2 * d * sizeof(float) : 0;
}

ffa_status ffa_qk_norm_rope_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                                int32_t hq, int32_t hkv, int32_t d, const float* q_weight, const float* k_weight,
                                float eps, const float* cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                                const int32_t* positions, const void* dq_out, const void* dk_out, void* dq, void* dk,
                                float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                void* stream) {
  NormRopeParams p{};
  const ffa_status st = check_common(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin,
                                     max_pos, rot_dim, positions, p);
  if (st != FFA_OK) return st;
  if (!dq_weight || !dk_weight || !workspace || !aligned16(dq_weight) || !aligned16(dk_weight) || !aligned16(workspace))
    return FFA_ERR_INVALID_ARG;
  if (workspace_bytes < ffa_qk_norm_rope_bwd_workspace_size(d)) return FFA_ERR_INVALID_ARG;
  if (tokens > 0 && (!dq_out || !dk_out || !dq || !dk || !aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) ||
                     !aligned16(dk)))
    return FFA_ERR_INVALID_ARG;
  const int64_t nq = 2 * tokens * hq * d, nk = 2 * tokens * hkv * d;
  const Span in[] = {{q, span_bytes(tokens, q_stride, hq, d)}, {k, span_bytes(tokens, k_stride, hkv, d)},
                     {q_weight, 4 * d}, {k_weight, 4 * d}, {cos_sin, 4 * max_pos * rot_dim}, {positions, 4 * tokens},
                     {dq_out, nq}, {dk_out, nk}};
  const Span outs[] = {{dq, nq}, {dk, nk}, {dq_weight, 4 * d}, {dk_weight, 4 * d},
                       {workspace, static_cast<int64_t>(ffa_qk_norm_rope_bwd_workspace_size(d))}};
  if (any_meet(outs, 5, in, 8)) return FFA_ERR_INVALID_ARG;
  p.dout[0] = static_cast<const __nv_bfloat16*>(dq_out);
  p.dout[1] = static_cast<const __nv_bfloat16*>(dk_out);
  p.out[0] = static_cast<__nv_bfloat16*>(dq);
  p.out[1] = static_cast<__nv_bfloat16*>(dk);
  p.partial = static_cast<float*>(workspace);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int blocks = 0;
  const ffa_status sl = launch_any<true>(p, tokens, d, interleaved != 0, s, &blocks);
  if (sl != FFA_OK) return sl;
  const cudaError_t e = d == 128 ? launch_after(norm_rope_dw_kernel<128>, 8, 1024, s, p.partial, blocks, dq_weight, dk_weight)
                                 : launch_after(norm_rope_dw_kernel<64>, 4, 1024, s, p.partial, blocks, dq_weight, dk_weight);
  return cuda_status(e);
}

}  // extern "C"
