// Writing rows into a paged key-value cache, quantising them on the way, and reading them back.
//
// The cache is [num_pages][hkv][page_size][d], so that what one kv head holds of a page is contiguous.  Stored types:
//   bf16  the row as it is;
//   e4m3  8-bit codes and one exponent byte a row: value = code * 2^(byte - 127), with 2^n, n >= -126, the smallest power of
//         two for which max|x| <= 448 * 2^n.  A power of two rather than max|x| / 448: codes have an exponent of
//         their own, so the scale's rounding up costs no mantissa bit, the division by it is exact (each value is rounded once),
//         and every stored value is exact in bf16 down to bf16's smallest, so that reading back does not round again.
//         A row that holds a NaN or an infinity is stored as NaN throughout (byte 127);
//   e2m1  4-bit codes, an e4m3 scale every 16 columns and one exponent byte a row: value = code * scale * 2^(byte - 127).  The byte takes
//         the row's range, so that scales need no calibration and no fp32 factor beside the cache; code times scale has 6 bits,
//         exact in f16 and in bf16.  d / 2 + d / 16 + 1 bytes: 4.6 bits a value at d = 128.
//
// Both kernels are bound by HBM: 2 d bytes a row on the tensors' side, 2 d, d + 1 or 9 d / 16 + 1 on the cache's.  A grid's second
// dimension is k or v; a warp holds 2 to 8 consecutive rows at once (a pass), whatever tokens and heads they are of, 8 values a
// lane (e2m1: 16), and starts the loads of its passes, 64 bytes a lane, before it uses the first (168K tokens of 8 heads, d = 128, e4m3,
// written, all on one GPU: 147 us so, 194 us with twice as many, 167 us with half).  Measured, the same tokens: e4m3 written in 150 us and
// read in 161 us, 102 and 95 % of a copy's 6782 GB/s; bf16 in 201 and 206 us, 101 and 99 %; e2m1 in 138 and 140 us, 95 and 94 %, where
// 32-byte stores count: an instruction's 16-byte pieces of the 16 values a lane has lie 32 bytes apart (161 us read so).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

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
  CacheRows cache[2];
  const int64_t* slots;
  PageGeom geom;
  FastDiv heads;
  uint32_t rows;               // tokens * hkv
  bool wide;                   // every row of k and v at a multiple of 32 bytes
};

// FILLED: a token's rows fill the passes of a whole number of warps (hkv a multiple of kUnroll * RW), so that token and page are the
// warp's and addresses a step apart.  Measured (168K tokens of 8 heads, d = 128, e4m3, on the first GPU above): 147 us, and 172 us without; with
// 3 heads of d = 64, which leave most of such a warp empty, 21.6 us for 30K tokens, and 11.8 us without.  (32-byte loads: e2m1 138.3 us for
// 139.8; 72 for 68 where rows are not FILLED.)
template <int D, int T, bool FILLED>
__global__ void __launch_bounds__(kThreads) kv_cache_write_kernel(WriteParams p) {
  constexpr int V = kLaneValues<T>, L = D / V, RW = 32 / L, U = kUnroll * 8 / V;   // passes of RW rows
  const int lane = threadIdx.x & 31, l = lane & (L - 1), sub = lane / L, which = blockIdx.y;
  const uint32_t row0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * (U * RW) + sub;
  if (row0 - sub >= p.rows) return;
  const int page_rows = p.geom.hkv << p.geom.page_log2, page_mask = (1 << p.geom.page_log2) - 1;
  auto read = [&](const __nv_bfloat16* x, LaneValues<T>& to) {
    if (FILLED && V == 16 && p.wide) {
      load32(x, to[0], to[V / 8 - 1]);
    } else {
#pragma unroll
      for (int j = 0; j < V / 8; ++j) to[j] = __ldg(reinterpret_cast<const uint4*>(x) + j);
    }
  };
  LaneValues<T> v[U];
  int64_t dst[U];   // cache row; -1: not written
  if constexpr (FILLED) {
    const uint32_t token = divide(p.heads, row0 - sub);
    const int h = static_cast<int>(row0 - token * p.heads.d);
    const int64_t slot = __ldg(p.slots + token);
    const __nv_bfloat16* x = pick(p.x, which) + token * pick(p.stride, which) + h * D + V * l;
#pragma unroll
    for (int i = 0; i < U; ++i) read(x + i * (RW * D), v[i]);
    if (!slot_ok(p.geom, slot)) return;   // padding, or no slot of this cache
    dst[0] = (slot >> p.geom.page_log2) * page_rows + (h << p.geom.page_log2) + (slot & page_mask);
#pragma unroll
    for (int i = 1; i < U; ++i) dst[i] = dst[i - 1] + (RW << p.geom.page_log2);
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t row = row0 + i * RW, token = divide(p.heads, row);
      const int h = static_cast<int>(row - token * p.heads.d);
#pragma unroll
      for (int j = 0; j < V / 8; ++j) v[i][j] = uint4{};
      dst[i] = -1;
      if (row < p.rows) {
        read(pick(p.x, which) + token * pick(p.stride, which) + h * D + V * l, v[i]);
        const int64_t slot = __ldg(p.slots + token);
        if (slot_ok(p.geom, slot)) dst[i] = (slot >> p.geom.page_log2) * page_rows + (h << p.geom.page_log2) + (slot & page_mask);
      }
    }
  }
  const CacheRows cache = pick(p.cache, which);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const StoredRow r = make_row<D, T>(v[i]);
    if (FILLED || dst[i] >= 0) put_row<D, T>(r, dst[i], l, cache);
  }
}

struct ReadParams {
  void* rows[2];
  uint8_t* exps[2];
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
// What e2m1 has on top is in a type of its own: with larger parameters the compiler gives the other types' kernels fewer registers (1K rows of
// bf16 3.4 us for 3.2, 168K tokens of 8 heads, e4m3, 158.6 for 157.7).
struct ReadParams4 : ReadParams {
  uint8_t* scales[2];
  bool wide;      // both outputs at multiples of 32 bytes
};
template <int T>
using ReadParamsOf = std::conditional_t<T == kE2m1, ReadParams4, ReadParams>;

constexpr int kReadRows = 256;   // rows a CTA, or those of 8 tokens: so many tokens that a thread each finds their places

// A CTA takes `tile` consecutive tokens of the output; a thread a token finds its sequence and page.
template <int D, int T>
__global__ void __launch_bounds__(kThreads) kv_cache_read_kernel(ReadParamsOf<T> p) {
  constexpr int V = kLaneValues<T>, L = D / V, RW = 32 / L, U = kUnroll * 8 / V;   // passes of RW rows
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
  __nv_bfloat16* out = pick(p.out, which) + t0 * p.geom.hkv * D + V * l;
  for (uint32_t r0 = (threadIdx.x >> 5) * (U * RW) + sub; r0 - sub < rows; r0 += kWarps * U * RW) {
    uint4 v[U];
    uint32_t e[U];
    int64_t at[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t r = r0 + i * RW, token = divide(p.heads, r);
      at[i] = -1;
      if (r >= rows) continue;
      at[i] = src[token];
      if (at[i] < 0) continue;
      const int64_t row = at[i] + (static_cast<int64_t>(r - token * p.heads.d) << p.geom.page_log2);
      if constexpr (T == kE2m1) {
        const uint2 c = __ldg(static_cast<const uint2*>(pick(p.rows, which)) + row * L + l);
        v[i].x = c.x, v[i].y = c.y, v[i].z = __ldg(pick(p.scales, which) + row * L + l);
        e[i] = __ldg(pick(p.exps, which) + row);
      } else if constexpr (T == kE4m3) {
        const uint2 c = __ldg(static_cast<const uint2*>(pick(p.rows, which)) + row * L + l);
        v[i].x = c.x, v[i].y = c.y;
        e[i] = __ldg(pick(p.exps, which) + row);
      } else {
        v[i] = __ldg(static_cast<const uint4*>(pick(p.rows, which)) + row * L + l);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (at[i] == -1) continue;
      uint4 o[V / 8];
#pragma unroll
      for (int j = 0; j < V / 8; ++j) {
        o[j] = v[i];
        if (at[i] == -2) {
          o[j] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
        } else if constexpr (T != kBf16) {
          const float s = exp_scale(e[i]);
          uint32_t c[4], w[4];
          if constexpr (T == kE2m1) {
            const uint32_t scale = e4m3x2_to_f16x2(v[i].z | v[i].z << 8);
            e2m1x8_to_f16x2(j ? v[i].y : v[i].x, c);
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = mul_f16x2(c[k], scale);   // exact
          } else {
            e4m3x4_to_f16x2(v[i].x, c[0], c[1]);
            e4m3x4_to_f16x2(v[i].y, c[2], c[3]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = mul2(__half22float2(*reinterpret_cast<const __half2*>(&c[k])), make_float2(s, s));
            w[k] = pack_bf16x2(f.x, f.y);
          }
          o[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __nv_bfloat16* to = out + static_cast<int64_t>(r0 + i * RW) * D;
      if constexpr (T == kE2m1) {
        if (p.wide) {
          store32(to, o[0], o[1]);
          continue;
        }
      }
#pragma unroll
      for (int j = 0; j < V / 8; ++j) reinterpret_cast<uint4*>(to)[j] = o[j];
    }
  }
}

template <int D, int T>
auto* write_kernel_of(bool filled) {
  return filled ? kv_cache_write_kernel<D, T, true> : kv_cache_write_kernel<D, T, false>;
}
template <int D>
auto* write_kernel(int type, bool filled) {
  return type == kE2m1 ? write_kernel_of<D, kE2m1>(filled) : type == kE4m3 ? write_kernel_of<D, kE4m3>(filled) : write_kernel_of<D, kBf16>(filled);
}
template <int D>
void launch_read(int type, const ReadParams4& p, dim3 grid, cudaStream_t s) {
  if (type == kE2m1) kv_cache_read_kernel<D, kE2m1><<<grid, kThreads, 0, s>>>(p);
  else if (type == kE4m3) kv_cache_read_kernel<D, kE4m3><<<grid, kThreads, 0, s>>>(p);
  else kv_cache_read_kernel<D, kBf16><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace

ffa_status check_cache(const ffa_kv_cache* c, PageGeom& g) {
  if (!c) return FFA_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->hkv <= 0 || c->page_size <= 0) return FFA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FFA_ERR_UNSUPPORTED;
  if (c->dtype != FFA_KV_BF16 && c->dtype != FFA_KV_E4M3 && c->dtype != FFA_KV_E2M1) return FFA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return FFA_ERR_UNSUPPORTED;
  // page numbers are int32; a page's rows, and their bytes, fit 32 bits in the kernels' index arithmetic
  if (c->num_pages > (int64_t{1} << 31) || static_cast<int64_t>(c->hkv) * c->page_size > (1 << 22)) return FFA_ERR_OVERFLOW;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return FFA_ERR_INVALID_ARG;
  if (c->dtype != FFA_KV_BF16 && (!c->k_exp || !c->v_exp || !aligned16(c->k_exp) || !aligned16(c->v_exp)))
    return FFA_ERR_INVALID_ARG;
  if (c->dtype == FFA_KV_E2M1 && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)))
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
  p.cache[0] = k_rows(*cache);
  p.cache[1] = v_rows(*cache);
  p.slots = slots;
  p.rows = static_cast<uint32_t>(tokens * cache->hkv);
  p.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0 && k_stride % 16 == 0 && v_stride % 16 == 0;
  p.heads = fast_div(static_cast<uint32_t>(cache->hkv));
  const int per = kWarps * kUnroll * 256 / cache->d;   // rows a CTA
  const unsigned blocks = (p.rows + per - 1) / per;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(blocks, 2);
  const bool filled = cache->hkv % (kUnroll * 256 / cache->d) == 0;
  auto* kernel = cache->d == 128 ? write_kernel<128>(cache->dtype, filled) : write_kernel<64>(cache->dtype, filled);
  kernel<<<grid, kThreads, 0, s>>>(p);
  return cuda_status(cudaGetLastError());
}

ffa_status ffa_kv_cache_read(const ffa_kv_cache* cache, const int32_t* page_table, int64_t table_stride,
                             int32_t max_pages, int32_t batch, const int32_t* cu_seqlens, int64_t total, void* k,
                             void* v, void* stream) {
  ReadParams4 p{};
  const ffa_status st = check_cache(cache, p.geom);
  if (st != FFA_OK) return st;
  if (total < 0 || batch < 0 || max_pages < 0 || (batch > 1 && table_stride < max_pages)) return FFA_ERR_INVALID_ARG;
  if (total == 0 || batch == 0) return FFA_OK;
  if (!cu_seqlens || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u)) return FFA_ERR_INVALID_ARG;
  if (max_pages > 0 && (!page_table || (reinterpret_cast<uintptr_t>(page_table) & 3u))) return FFA_ERR_INVALID_ARG;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return FFA_ERR_INVALID_ARG;
  if (total > 0x7fffffff) return FFA_ERR_OVERFLOW;   // cu_seqlens is int32
  const CacheSpans at(*cache);
  Span in[8] = {{page_table, 4 * (static_cast<int64_t>(batch - 1) * table_stride + max_pages)}, {cu_seqlens, 4 * (int64_t{batch} + 1)}};
  for (int i = 0; i < at.n; ++i) in[2 + i] = at.s[i];
  const int64_t bytes = 2 * total * cache->hkv * cache->d;
  const Span out[] = {{k, bytes}, {v, bytes}};
  if (any_meet(out, 2, in, 2 + at.n)) return FFA_ERR_INVALID_ARG;
  const CacheRows kr = k_rows(*cache), vr = v_rows(*cache);
  p.rows[0] = kr.rows, p.rows[1] = vr.rows;
  p.exps[0] = kr.exps, p.exps[1] = vr.exps;
  p.scales[0] = kr.scales, p.scales[1] = vr.scales;
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
  p.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>((total + p.tile - 1) / p.tile), 2);
  if (cache->d == 128) launch_read<128>(cache->dtype, p, grid, s);
  else launch_read<64>(cache->dtype, p, grid, s);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
