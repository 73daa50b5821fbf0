// What the kernels over the paged key-value cache share.
#pragma once

#include <cuda_fp16.h>

#include "ffa_internal.h"
#include "launch.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace ffa {

// Host check of a cache description; fills its geometry.
ffa_status check_cache(const ffa_kv_cache* c, PageGeom& g);

// Stored types, as the kernels' template arguments.
constexpr int kBf16 = FFA_KV_BF16, kE4m3 = FFA_KV_E4M3, kE2m1 = FFA_KV_E2M1;

// Bytes of a stored row's values, and of its e2m1 scales.
FFA_HD constexpr int value_bytes(int type, int d) { return type == kBf16 ? 2 * d : type == kE4m3 ? d : d / 2; }
FFA_HD constexpr int scale_bytes(int type, int d) { return type == kE2m1 ? d / 16 : 0; }

// A cache's arrays, of k or of v.
struct CacheRows {
  void* rows;
  uint8_t* exps;
  uint8_t* scales;
};
// Those of a cache, with null for what its type does not have.  The scales' fields are read for their type only: a caller compiled before they were
// there passes a description without them.
inline CacheRows k_rows(const ffa_kv_cache& c) {
  return {c.k, c.dtype == FFA_KV_BF16 ? nullptr : c.k_exp, c.dtype == FFA_KV_E2M1 ? c.k_scale : nullptr};
}
inline CacheRows v_rows(const ffa_kv_cache& c) {
  return {c.v, c.dtype == FFA_KV_BF16 ? nullptr : c.v_exp, c.dtype == FFA_KV_E2M1 ? c.v_scale : nullptr};
}

// The memory of a checked cache.
struct CacheSpans {
  Span s[6];
  int n;
  explicit CacheSpans(const ffa_kv_cache& c) {
    const int64_t rows = c.num_pages * c.hkv * c.page_size, bytes = rows * value_bytes(c.dtype, c.d);
    const CacheRows k = k_rows(c), v = v_rows(c);
    s[0] = {k.rows, bytes};
    s[1] = {v.rows, bytes};
    s[2] = {k.exps, rows};
    s[3] = {v.exps, rows};
    s[4] = {k.scales, rows * scale_bytes(c.dtype, c.d)};
    s[5] = {v.scales, rows * scale_bytes(c.dtype, c.d)};
    n = c.dtype == FFA_KV_E2M1 ? 6 : c.dtype == FFA_KV_E4M3 ? 4 : 2;
  }
};

// 2^(byte - 127), the scale an exponent byte stands for (0 for byte 0, which no write stores).
__device__ __forceinline__ float exp_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two e4m3 codes as two f16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
// Four codes of a word as two pairs.
__device__ __forceinline__ void e4m3x4_to_f16x2(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(codes));
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}


// Eight e2m1 codes of a word as four pairs of f16 values, exactly: values 2i and 2i + 1 in r[i].
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t codes, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(codes));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x2(float2 f) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(f.y), "f"(f.x));
  return r;
}
// The nearest e2m1 codes of 8 values, ties to even, beyond 6 as 6: value i in bits 4i .. 4i + 3.
__device__ __forceinline__ uint32_t e2m1x8(float2 f0, float2 f1, float2 f2, float2 f3) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r) : "f"(f0.x), "f"(f0.y), "f"(f1.x), "f"(f1.y), "f"(f2.x), "f"(f2.y), "f"(f3.x), "f"(f3.y));
  return r;
}

// Quotients y / s of an 8-bit value by a 4-bit one (or by 6), given an approximate 1 / s: corrected by what is left of y, so that one that
// is halfway between two codes is exactly so.  Any other is off every such point by 2^-8 of itself, so that both rounded to codes are the
// exact quotient's.  (y * (1 / s) alone misses 18 % of the halfway points.)  Zeros keep their signs.
__device__ __forceinline__ float2 quotient(float2 y, float s, float over) {
  const float2 z = mul2(y, make_float2(over, over));
  const float2 e = fma2(z, make_float2(s, s), make_float2(-y.x, -y.y));
  return fma2(e, make_float2(-over, -over), z);
}

// A row as a cache stores it, spread over lanes: lane `l` of the D / V that hold it has columns V l .. V l + V - 1.  V is 8, or 16 for e2m1: a
// lane then has all of what one scale is of (168K tokens of 8 heads, d = 128: written in 138 us and read in 140; with 8 a lane 185
// and 150).
template <int T>
constexpr int kLaneValues = T == kE2m1 ? 16 : 8;
template <int T>
using LaneValues = uint4[kLaneValues<T> / 8];   // bf16
struct StoredRow {
  uint4 codes;      // e4m3, e2m1: x, y
  uint32_t scale;   // e2m1
  int byte;
};

// One row of bf16 values in its stored form.  All lanes of the warp take part.
template <int D, int T>
__device__ __forceinline__ StoredRow make_row(const LaneValues<T>& v) {
  StoredRow r{};
  if constexpr (T == kBf16) {
    r.codes = v[0];
  } else {
    // bf16 magnitudes order as 15-bit integers: the lane's largest, then the row's, two at a time
    constexpr int N = kLaneValues<T> / 2;
    uint32_t u[N];
#pragma unroll
    for (int j = 0; j < N / 4; ++j) u[4 * j] = v[j].x, u[4 * j + 1] = v[j].y, u[4 * j + 2] = v[j].z, u[4 * j + 3] = v[j].w;
    uint32_t g = u[0] & 0x7fff7fffu;
#pragma unroll
    for (int j = 1; j < N; ++j) g = __vmaxu2(g, u[j] & 0x7fff7fffu);
    uint32_t m = g;
#pragma unroll
    for (int o = D / kLaneValues<T> / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m & 0xffffu, m >> 16);
    const bool finite = m < 0x7f80u;
    // max|x| = 1.f * 2^(e - 127).  448 = 1.75 * 2^8: the scale's byte is e - 8, one more where 1.f > 1.75 (mantissa 0x60).
    // 6 * 448 = 1.3125 * 2^11: e - 11, one more where 1.f > 1.3125 (mantissa 0x28).
    r.byte = !finite ? 127 : T == kE4m3 ? max(static_cast<int>((m + 0x1fu) >> 7) - 8, 1) : max(static_cast<int>((m + 0x57u) >> 7) - 11, 1);
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - r.byte) << 23);   // 2^-(byte - 127), exact
    auto scaled = [&](int j) {
      return mul2(make_float2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u)), make_float2(inv, inv));
    };
    if constexpr (T == kE4m3) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = e4m3x2(scaled(j));
      r.codes.x = finite ? x[0] | x[1] << 16 : 0x7f7f7f7fu;
      r.codes.y = finite ? x[2] | x[3] << 16 : 0x7f7f7f7fu;
    } else {
      g = max(g & 0xffffu, g >> 16);
      const float top = __uint_as_float(g << 16) * inv;
      const uint32_t code = e4m3x2(quotient(make_float2(top, 0.f), 6.f, 1.f / 6.f)) & 0xffu;
      const float s = e4m3x2_to_float2(code).x, over = s > 0.f ? __fdividef(1.f, s) : 0.f;
      float2 z[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) z[j] = quotient(scaled(j), s, over);
      r.codes.x = finite ? e2m1x8(z[0], z[1], z[2], z[3]) : 0u;
      r.codes.y = finite ? e2m1x8(z[4], z[5], z[6], z[7]) : 0u;
      r.scale = finite ? code : 0x7fu;
    }
  }
  return r;
}

// Write it at `row` of the cache.
template <int D, int T>
__device__ __forceinline__ void put_row(const StoredRow& r, int64_t row, int l, const CacheRows& c) {
  constexpr int L = D / kLaneValues<T>;
  if constexpr (T == kBf16) {
    reinterpret_cast<uint4*>(c.rows)[row * L + l] = r.codes;
  } else {
    reinterpret_cast<uint2*>(c.rows)[row * L + l] = make_uint2(r.codes.x, r.codes.y);
    if constexpr (T == kE2m1) c.scales[row * L + l] = static_cast<uint8_t>(r.scale);
    if (l == 0) c.exps[row] = static_cast<uint8_t>(r.byte);
  }
}

}  // namespace ffa
