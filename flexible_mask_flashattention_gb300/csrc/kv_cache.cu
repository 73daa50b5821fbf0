// Writing rows into a paged key-value cache, quantising them on the way, and reading them back.
//
// The cache is [num_pages][hkv][page_size][d], so that what one kv head holds of a page is contiguous.  Stored types:
//   bf16  the row as it is;
//   e4m3  8-bit codes and one exponent byte a row: value = code * 2^(byte - 127), with 2^n, n >= -126, the smallest power of
//         two for which max|x| <= 448 * 2^n.  A power of two rather than max|x| / 448: codes have an exponent of
//         their own, so the scale's rounding up costs no mantissa bit, the division by it is exact (each value is rounded once),
//         and every stored value is exact in bf16 down to bf16's smallest, so that reading back does not round again.
//         A row that holds a NaN or an infinity is stored as NaN throughout (byte 127).
//
// Both kernels are bound by HBM: 2 d bytes a row on the tensors' side, 2 d or d + 1 on the cache's.  A grid's second
// dimension is k or v; a warp holds 2 or 4 consecutive rows at once (a pass), whatever tokens and heads they are of, 8 values a
// lane, and starts the loads of kUnroll passes before it uses the first (168K tokens of 8 heads, d = 128, e4m3, written, all on one GPU: 147
// us so, 194 us with 8 passes, 167 us with 2).  Measured on another GPU, the same tokens: e4m3 written in 153 us and read in 157 us,
// 101 and 97 % of a copy's 6795 GB/s; bf16 in 199 and 203 us, 102 and 100 %.
#include <cuda_bf16.h>

#include <algorithm>

#include "ffa_internal.h"
#include "kv_cache.h"
#include "launch.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace ffa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;

// A parameter pair's entry by a run-time index, as a select (an indexed one would copy the parameters to local memory).
template <typename T>
__device__ __forceinline__ T pick(T const (&pair)[2], int i) {
  return i ? pair[1] : pair[0];
}

struct WriteParams {
  const __nv_bfloat16* x[2];   // k, v
  int64_t stride[2];
  void* cache[2];
  uint8_t* exps[2];
  const int64_t* slots;
  PageGeom geom;
  FastDiv heads;
  uint32_t rows;               // tokens * hkv
};

__device__ __forceinline__ uint32_t e4m3x2(float2 f) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(f.y), "f"(f.x));
  return r;
}

// FILLED: a token's rows fill the passes of a whole number of warps (hkv a multiple of kUnroll * RW), so that token and page are the
// warp's and addresses a step apart.  Measured (168K tokens of 8 heads, d = 128, e4m3, on the first GPU above): 147 us, and 172 us without; with
// 3 heads of d = 64, which leave most of such a warp empty, 21.6 us for 30K tokens, and 11.8 us without.
template <int D, bool FP8, bool FILLED>
__global__ void __launch_bounds__(kThreads) kv_cache_write_kernel(WriteParams p) {
  constexpr int L = D / 8, RW = 32 / L;
  const int lane = threadIdx.x & 31, l = lane & (L - 1), sub = lane / L, which = blockIdx.y;
  const uint32_t row0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * (kUnroll * RW) + sub;
  if (row0 - sub >= p.rows) return;
  const int page_rows = p.geom.hkv << p.geom.page_log2, page_mask = (1 << p.geom.page_log2) - 1;
  uint4 v[kUnroll];
  int64_t dst[kUnroll];   // cache row; -1: not written
  if constexpr (FILLED) {
    const uint32_t token = divide(p.heads, row0 - sub);
    const int h = static_cast<int>(row0 - token * p.heads.d);
    const int64_t slot = __ldg(p.slots + token);
    const __nv_bfloat16* x = pick(p.x, which) + token * pick(p.stride, which) + h * D + 8 * l;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(x + i * (RW * D)));
    if (!slot_ok(p.geom, slot)) return;   // padding, or no slot of this cache
    dst[0] = (slot >> p.geom.page_log2) * page_rows + (h << p.geom.page_log2) + (slot & page_mask);
#pragma unroll
    for (int i = 1; i < kUnroll; ++i) dst[i] = dst[i - 1] + (RW << p.geom.page_log2);
  } else {
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const uint32_t row = row0 + i * RW, token = divide(p.heads, row);
      const int h = static_cast<int>(row - token * p.heads.d);
      v[i] = uint4{};
      dst[i] = -1;
      if (row < p.rows) {
        v[i] = __ldg(reinterpret_cast<const uint4*>(pick(p.x, which) + token * pick(p.stride, which) + h * D + 8 * l));
        const int64_t slot = __ldg(p.slots + token);
        if (slot_ok(p.geom, slot)) dst[i] = (slot >> p.geom.page_log2) * page_rows + (h << p.geom.page_log2) + (slot & page_mask);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const bool act = FILLED || dst[i] >= 0;
    if constexpr (!FP8) {
      if (act) reinterpret_cast<uint4*>(pick(p.cache, which))[dst[i] * (D / 8) + l] = v[i];
    } else {
      // bf16 magnitudes order as 15-bit integers: the row's largest, two at a time
      uint32_t m = __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu), __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = max(m & 0xffffu, m >> 16);
      // max|x| = 1.f * 2^(e - 127), 448 = 1.75 * 2^8: the scale's byte is e - 8, one more where 1.f > 1.75 (mantissa 0x60)
      const bool finite = m < 0x7f80u;
      const int byte = finite ? max(static_cast<int>((m + 0x1fu) >> 7) - 8, 1) : 127;
      const float inv = __uint_as_float(static_cast<uint32_t>(254 - byte) << 23);   // 2^-(byte - 127), exact
      const uint32_t u4[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        c[j] = e4m3x2(mul2(make_float2(__uint_as_float(u4[j] << 16), __uint_as_float(u4[j] & 0xffff0000u)), make_float2(inv, inv)));
      uint2 codes = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
      if (!finite) codes = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
      if (act) {
        reinterpret_cast<uint2*>(pick(p.cache, which))[dst[i] * (D / 8) + l] = codes;
        if (l == 0) pick(p.exps, which)[dst[i]] = static_cast<uint8_t>(byte);
      }
    }
  }
}

struct ReadParams {
  const void* cache[2];
  const uint8_t* exps[2];
  __nv_bfloat16* out[2];
  const int32_t* table;
  int64_t table_stride;
  int32_t max_pages, batch;
  const int32_t* cu;
  int64_t total;
  PageGeom geom;
  FastDiv heads;
  int32_t tile;   // tokens a CTA
};

constexpr int kReadRows = 256;   // rows a CTA, or those of 8 tokens: so many tokens that a thread each finds their places

// A CTA takes `tile` consecutive tokens of the output; a thread a token finds its sequence and page.
template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) kv_cache_read_kernel(ReadParams p) {
  constexpr int L = D / 8, RW = 32 / L;
  __shared__ int64_t src[kReadRows];   // row of head 0 in the cache; -1: outside the batch, -2: no page of this cache
  const int64_t t0 = blockIdx.x * static_cast<int64_t>(p.tile);
  if (threadIdx.x < p.tile) {
    const int64_t t = t0 + threadIdx.x;
    int64_t at = -1;
    if (t < p.total && t < p.cu[p.batch]) {
      int lo = 0, hi = p.batch;   // the last sequence with cu <= t
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= t) lo = mid + 1; else hi = mid;
      }
      if (lo > 0) {
        const int64_t pos = t - p.cu[lo - 1];
        const int64_t pi = pos >> p.geom.page_log2;
        at = -2;
        if (pi < p.max_pages) {
          const int64_t page = p.table[(lo - 1) * p.table_stride + pi];
          if (page_ok(p.geom, page))
            at = cache_row(p.geom, page, 0, static_cast<int>(pos & ((1 << p.geom.page_log2) - 1)));
        }
      }
    }
    src[threadIdx.x] = at;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, l = lane & (L - 1), sub = lane / L, which = blockIdx.y;
  const uint32_t rows = p.tile * p.geom.hkv;
  __nv_bfloat16* out = pick(p.out, which) + t0 * p.geom.hkv * D + 8 * l;
  for (uint32_t r0 = (threadIdx.x >> 5) * (kUnroll * RW) + sub; r0 - sub < rows; r0 += kWarps * kUnroll * RW) {
    uint4 v[kUnroll];
    uint32_t e[kUnroll];
    int64_t at[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const uint32_t r = r0 + i * RW, token = divide(p.heads, r);
      at[i] = -1;
      if (r >= rows) continue;
      at[i] = src[token];
      if (at[i] < 0) continue;
      const int64_t row = at[i] + (static_cast<int64_t>(r - token * p.heads.d) << p.geom.page_log2);
      if constexpr (FP8) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(pick(p.cache, which)) + row * (D / 8) + l);
        v[i].x = c.x, v[i].y = c.y;
        e[i] = __ldg(pick(p.exps, which) + row);
      } else {
        v[i] = __ldg(reinterpret_cast<const uint4*>(pick(p.cache, which)) + row * (D / 8) + l);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (at[i] == -1) continue;
      uint4 o = v[i];
      if (at[i] == -2) {
        o = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      } else if constexpr (FP8) {
        const float s = exp_scale(e[i]);
        const uint32_t c[4] = {v[i].x & 0xffffu, v[i].x >> 16, v[i].y & 0xffffu, v[i].y >> 16};
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = mul2(e4m3x2_to_float2(c[j]), make_float2(s, s));
          w[j] = pack_bf16x2(f.x, f.y);
        }
        o = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r0 + i * RW) * D) = o;
    }
  }
}

}  // namespace

ffa_status check_cache(const ffa_kv_cache* c, PageGeom& g) {
  if (!c) return FFA_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->hkv <= 0 || c->page_size <= 0) return FFA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FFA_ERR_UNSUPPORTED;
  if (c->dtype != FFA_KV_BF16 && c->dtype != FFA_KV_E4M3) return FFA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return FFA_ERR_UNSUPPORTED;
  // page numbers are int32; a page's rows, and their bytes, fit 32 bits in the kernels' index arithmetic
  if (c->num_pages > (int64_t{1} << 31) || static_cast<int64_t>(c->hkv) * c->page_size > (1 << 22)) return FFA_ERR_OVERFLOW;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return FFA_ERR_INVALID_ARG;
  if (c->dtype == FFA_KV_E4M3 && (!c->k_exp || !c->v_exp || !aligned16(c->k_exp) || !aligned16(c->v_exp)))
    return FFA_ERR_INVALID_ARG;
  g.num_pages = c->num_pages;
  g.hkv = c->hkv;
  g.page_log2 = 0;
  while ((1 << g.page_log2) < c->page_size) ++g.page_log2;
  return FFA_OK;
}

}  // namespace ffa

using namespace ffa;

extern "C" {

ffa_status ffa_kv_cache_write(const void* k, int64_t k_stride, const void* v, int64_t v_stride, int64_t tokens,
                              const int64_t* slots, const ffa_kv_cache* cache, void* stream) {
  WriteParams p{};
  const ffa_status st = check_cache(cache, p.geom);
  if (st != FFA_OK) return st;
  if (tokens < 0) return FFA_ERR_INVALID_ARG;
  if (tokens == 0) return FFA_OK;
  if (!k || !v || !slots || !aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return FFA_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(cache->hkv) * cache->d;
  if (k_stride % 8 != 0 || v_stride % 8 != 0 || (tokens > 1 && (k_stride < row || v_stride < row)))
    return FFA_ERR_INVALID_ARG;
  if (tokens > 0x7fffffff / cache->hkv - 256) return FFA_ERR_OVERFLOW;   // rows are counted in 31 bits
  const CacheSpans at(*cache);
  const Span in[] = {{k, span_bytes(tokens, k_stride, cache->hkv, cache->d)}, {v, span_bytes(tokens, v_stride, cache->hkv, cache->d)},
                     {slots, 8 * tokens}};
  if (any_meet(at.s, at.n, in, 3)) return FFA_ERR_INVALID_ARG;
  p.x[0] = static_cast<const __nv_bfloat16*>(k);
  p.x[1] = static_cast<const __nv_bfloat16*>(v);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.cache[0] = cache->k;
  p.cache[1] = cache->v;
  p.exps[0] = cache->k_exp;
  p.exps[1] = cache->v_exp;
  p.slots = slots;
  p.rows = static_cast<uint32_t>(tokens * cache->hkv);
  p.heads = fast_div(static_cast<uint32_t>(cache->hkv));
  const int per = kWarps * kUnroll * 256 / cache->d;   // rows a CTA
  const unsigned blocks = (p.rows + per - 1) / per;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = cache->dtype == FFA_KV_E4M3;
  const dim3 grid(blocks, 2);
  const bool filled = cache->hkv % (kUnroll * 256 / cache->d) == 0;
  auto* kernel = cache->d == 128 ? fp8 ? filled ? kv_cache_write_kernel<128, true, true> : kv_cache_write_kernel<128, true, false>
                                       : filled ? kv_cache_write_kernel<128, false, true> : kv_cache_write_kernel<128, false, false>
                                 : fp8 ? filled ? kv_cache_write_kernel<64, true, true> : kv_cache_write_kernel<64, true, false>
                                       : filled ? kv_cache_write_kernel<64, false, true> : kv_cache_write_kernel<64, false, false>;
  kernel<<<grid, kThreads, 0, s>>>(p);
  return cuda_status(cudaGetLastError());
}

ffa_status ffa_kv_cache_read(const ffa_kv_cache* cache, const int32_t* page_table, int64_t table_stride,
                             int32_t max_pages, int32_t batch, const int32_t* cu_seqlens, int64_t total, void* k,
                             void* v, void* stream) {
  ReadParams p{};
  const ffa_status st = check_cache(cache, p.geom);
  if (st != FFA_OK) return st;
  if (total < 0 || batch < 0 || max_pages < 0 || (batch > 1 && table_stride < max_pages)) return FFA_ERR_INVALID_ARG;
  if (total == 0 || batch == 0) return FFA_OK;
  if (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return FFA_ERR_INVALID_ARG;
  if (max_pages > 0 && (!page_table || (reinterpret_cast<uintptr_t>(page_table) & 3u))) return FFA_ERR_INVALID_ARG;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FFA_ERR_INVALID_ARG;
  if (total > 0x7fffffff) return FFA_ERR_OVERFLOW;   // cu_seqlens is int32
  const CacheSpans at(*cache);
  Span in[6] = {{page_table, 4 * (static_cast<int64_t>(batch - 1) * table_stride + max_pages)}, {cu_seqlens, 4 * (int64_t{batch} + 1)}};
  for (int i = 0; i < at.n; ++i) in[2 + i] = at.s[i];
  const int64_t bytes = 2 * total * cache->hkv * cache->d;
  const Span out[] = {{k, bytes}, {v, bytes}};
  if (any_meet(out, 2, in, 2 + at.n)) return FFA_ERR_INVALID_ARG;
  p.cache[0] = cache->k;
  p.cache[1] = cache->v;
  p.exps[0] = cache->k_exp;
  p.exps[1] = cache->v_exp;
  p.out[0] = static_cast<__nv_bfloat16*>(k);
  p.out[1] = static_cast<__nv_bfloat16*>(v);
  p.table = page_table;
  p.table_stride = table_stride;
  p.max_pages = max_pages;
  p.batch = batch;
  p.cu = cu_seqlens;
  p.total = total;
  p.heads = fast_div(static_cast<uint32_t>(cache->hkv));
  p.tile = std::max(8, kReadRows / cache->hkv);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp8 = cache->dtype == FFA_KV_E4M3;
  const dim3 grid(static_cast<unsigned>((total + p.tile - 1) / p.tile), 2);
  if (cache->d == 128)
    (fp8 ? kv_cache_read_kernel<128, true> : kv_cache_read_kernel<128, false>)<<<grid, kThreads, 0, s>>>(p);
  else
    (fp8 ? kv_cache_read_kernel<64, true> : kv_cache_read_kernel<64, false>)<<<grid, kThreads, 0, s>>>(p);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
