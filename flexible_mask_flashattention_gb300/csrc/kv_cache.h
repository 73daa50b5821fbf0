// What the kernels over the paged key-value cache share.
#pragma once

#include <cuda_fp16.h>

#include "ffa_internal.h"
#include "launch.h"
#include "paged.cuh"

namespace ffa {

// Host check of a cache description; fills its geometry.
ffa_status check_cache(const ffa_kv_cache* c, PageGeom& g);

// The memory of a checked cache.
struct CacheSpans {
  Span s[4];
  int n;
  explicit CacheSpans(const ffa_kv_cache& c) {
    const int64_t rows = c.num_pages * c.hkv * c.page_size, bytes = rows * c.d * (c.dtype == FFA_KV_E4M3 ? 1 : 2);
    s[0] = {c.k, bytes};
    s[1] = {c.v, bytes};
    s[2] = {c.k_exp, rows};
    s[3] = {c.v_exp, rows};
    n = c.dtype == FFA_KV_E4M3 ? 4 : 2;
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

}  // namespace ffa
