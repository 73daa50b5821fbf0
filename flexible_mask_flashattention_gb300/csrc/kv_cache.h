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

// The memory of a checked cache.
struct CacheSpans {
  Span s[6];
  int n;
  explicit CacheSpans(const ffa_kv_cache& c) {
    const int64_t rows = c.num_pages * c.hkv * c.page_size, bytes = rows * value_bytes(c.dtype, c.d);
    s[0] = {c.k, bytes};
    s[1] = {c.v, bytes};
    s[2] = {c.k_exp, rows};
    s[3] = {c.v_exp, rows};
    s[4] = {c.k_scale, rows * scale_bytes(c.dtype, c.d)};
    s[5] = {c.v_scale, rows * scale_bytes(c.dtype, c.d)};
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
__device__ __forceinline__ uint32_t e2m1x8(const float2 (&f)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r) : "f"(f[0].x), "f"(f[0].y), "f"(f[1].x), "f"(f[1].y), "f"(f[2].x), "f"(f[2].y), "f"(f[3].x), "f"(f[3].y));
  return r;
}

// Values rounded to 12 bits (z (2^12 + 1) split in two).  A quotient of an 8-bit value by a 4-bit one (or by 6) that is not halfway between
// two codes is off it by 2^-8 of itself, far over 12 bits, so a quotient from an approximate reciprocal, rounded so, lies on the same
// side of, or exactly on, every border between codes as the exact one.
__device__ __forceinline__ float2 round12(float2 z) {
  const float2 c = mul2(z, make_float2(4097.f, 4097.f));
  const float2 low = fma2(z, make_float2(-1.f, -1.f), c);
  return fma2(low, make_float2(-1.f, -1.f), c);
}

// A cache's arrays, of k or of v.
struct CacheRows {
  void* rows;
  uint8_t* exps;
  uint8_t* scales;
};

// A row as a cache stores it, 8 values a lane: lane `l` of the D / 8 that hold the row has columns 8l .. 8l + 7.
struct StoredRow {
  uint4 codes;      // e4m3: x, y; e2m1: x
  uint32_t scale;   // e2m1: of this lane's 16 columns (lanes 2i and 2i + 1 alike)
  int byte;
};

// One row of bf16 values in its stored form.  All lanes of the warp take part.
template <int D, int T>
__device__ __forceinline__ StoredRow make_row(const uint4& v) {
  constexpr int L = D / 8;
  StoredRow r{};
  if constexpr (T == kBf16) {
    r.codes = v;
  } else {
    // bf16 magnitudes order as 15-bit integers: the row's largest, two at a time
    uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t g = max(m & 0xffffu, m >> 16);   // of 16 columns
#pragma unroll
    for (int o = L / 2; o > 1; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m & 0xffffu, m >> 16);
    const bool finite = m < 0x7f80u;
    // max|x| = 1.f * 2^(e - 127).  448 = 1.75 * 2^8: the scale's byte is e - 8, one more where 1.f > 1.75 (mantissa 0x60).
    // 6 * 448 = 1.3125 * 2^11: e - 11, one more where 1.f > 1.3125 (mantissa 0x28).
    r.byte = !finite ? 127 : T == kE4m3 ? max(static_cast<int>((m + 0x1fu) >> 7) - 8, 1) : max(static_cast<int>((m + 0x57u) >> 7) - 11, 1);
    const float inv = __uint_as_float(static_cast<uint32_t>(254 - r.byte) << 23);   // 2^-(byte - 127), exact
    const uint32_t u4[4] = {v.x, v.y, v.z, v.w};
    float2 y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[j] = mul2(make_float2(__uint_as_float(u4[j] << 16), __uint_as_float(u4[j] & 0xffff0000u)), make_float2(inv, inv));
    if constexpr (T == kE4m3) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = e4m3x2(y[j]);
      r.codes.x = finite ? x[0] | x[1] << 16 : 0x7f7f7f7fu;
      r.codes.y = finite ? x[2] | x[3] << 16 : 0x7f7f7f7fu;
    } else {
      const float sixth = __uint_as_float(g << 16) * inv * (1.f / 6.f);
      const uint32_t code = e4m3x2(round12(make_float2(sixth, 0.f))) & 0xffu;
      const float s = e4m3x2_to_float2(code).x, over = s > 0.f ? __fdividef(1.f, s) : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = round12(mul2(y[j], make_float2(over, over)));
      r.codes.x = finite ? e2m1x8(y) : 0u;
      r.scale = finite ? code : 0x7fu;
    }
  }
  return r;
}

// Write it at `row` of the cache.
template <int D, int T>
__device__ __forceinline__ void put_row(const StoredRow& r, int64_t row, int l, const CacheRows& c) {
  constexpr int L = D / 8;
  if constexpr (T == kBf16) {
    reinterpret_cast<uint4*>(c.rows)[row * L + l] = r.codes;
  } else {
    if constexpr (T == kE4m3) {
      reinterpret_cast<uint2*>(c.rows)[row * L + l] = make_uint2(r.codes.x, r.codes.y);
    } else {
      reinterpret_cast<uint32_t*>(c.rows)[row * L + l] = r.codes.x;
      if (!(l & 1)) c.scales[row * (L / 2) + (l >> 1)] = static_cast<uint8_t>(r.scale);
    }
    if (l == 0) c.exps[row] = static_cast<uint8_t>(r.byte);
  }
}

}  // namespace ffa
