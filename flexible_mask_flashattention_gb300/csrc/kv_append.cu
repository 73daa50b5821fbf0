// Norm and rotation of new tokens' q and k, and their keys and values into the paged key-value cache, in one pass.
//
// What qk_norm_rope (without weights: the rotation alone) and then kv_cache_write compute, rounding for rounding: a key is rounded to bf16
// and then, where the cache is quantised, to its type; the rows in the cache are the same bits as the two calls leave, so that a prompt
// written one way and steps written the other agree.
//
// Bound by HBM: q in and out, k and v in, their stored rows out; the two calls also write k and read it again, 4 d bytes a k row, and are
// two launches.  The walk over tokens and heads, the copies to shared memory and the rotation are norm_rope.cu's, with v as a third tensor
// behind q and k.  A normalised key's columns lie in its lanes as rotation partners; it goes back to its place in shared memory and is
// read from there in the order that kv_cache.h's rows want.
//
// Unlike there, the warps of a CTA do not start their copies together: units of q's, k's and v's heads take different times (67K tokens
// of 16 + 4 heads, d = 128, into 4 bits: 169 us with a barrier a round, 140 without), nor are units cut across tensors (155) or made of
// equal shares of each (206).  Measured since, the same tokens: into bf16 132 us, e4m3 140, e2m1 137 (92, 79 and 78 % of a copy's rate on
// the bytes); 64 + 8 heads, 29K tokens: 183, 185 and 179 (95, 89 and 90 %); 6 + 2 heads, d = 64, 250K tokens: 127, 132 and 132 (74, 64 and
// 61 %, three units of few heads).  What is left is instructions: some 100 for a q head of a warp's tokens, issue slots 57 (bf16) and 62 %
// (e2m1) busy.  48 new tokens take 3 us.
#include "kv_cache.h"
#include "norm_rope.cuh"

namespace ffa {
namespace {

struct AppendParams : NormRopeParams {
  CacheRows cache[2];
  const int64_t* slots;
  PageGeom geom;
  int32_t first[4];   // q's, k's and v's first unit, and behind the last
  int32_t size[3];    // heads of such a unit
};

// Unit c's heads of tensor t.
__device__ __forceinline__ UnitPart part_of(const AppendParams& p, int c, int t) {
  const int head = (c - p.first[t]) * p.size[t];
  return UnitPart{c < p.first[t] || c >= p.first[t + 1] ? 0 : min(p.size[t], p.heads[t] - head), 0, head};
}

// Units of q's, of k's and of v's heads: what a unit begins with (its rotation, coefficients, places) is then of one tensor.  As many as
// fit, since that costs as much as three heads; smaller ones where there would be fewer units than warps.
constexpr int kAppendMost = kUnitMost<false>;
template <bool>   // as launch_units asks: there is no backward
void set_units(AppendParams& p, int64_t tokens, int d, int64_t warps) {
  const int group = 256 / d;
  const int64_t groups = std::max<int64_t>((tokens + group - 1) / group, 1), heads = p.heads[0] + p.heads[1] + p.heads[2];
  for (int t = 0; t < 3; ++t) {
    const int64_t all = p.heads[t], per = std::max((all + kAppendMost - 1) / kAppendMost, std::min(all, warps / groups * all / heads));
    p.size[t] = static_cast<int32_t>((all + per - 1) / per);
    p.first[t + 1] = p.first[t] + static_cast<int32_t>((all + p.size[t] - 1) / p.size[t]);
  }
  cut_units(p, tokens, d, p.first[3], std::max({p.size[0], p.size[1], p.size[2]}));
}

template <int D, bool INTER, int T, bool AS_IS>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(AppendParams p) {
  constexpr int L = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  float* weights = reinterpret_cast<float*>(smem);   // [2][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (L - 1), sub = lane / L;
  const Stages<D, false> st{smem + 2 * D * 4 + warp * kStages * Stages<D, false>::stage_bytes(p.unit), p.unit};
  const Columns<D, INTER> cols(l, p.rot);
  const int swap = Stages<D, false>::swap(sub), natural = (16 * l) ^ swap;
  auto copy = [&](int stage, const UnitWalk<D, true>& w) {
    if (w.c < p.first[2]) {
      copy_unit<D, false, true>(p, st, stage, w);
    } else {   // a value goes into the cache whatever its token's positions
      const UnitPart v = part_of(p, w.c, 2);
      copy_rows<D, false>(smem_u32(st.rows(stage, sub, 0)) + natural, p.x[2] + (w.has ? w.token : 0) * p.x_stride[2] + v.head * D + 8 * l, v.n,
                          w.has ? 16 : 0);
    }
  };
  UnitWalk<D, true> cur, ld;
  int pos_ahead = -1;   // what the copies one unit ahead have found of its positions
  static_assert(kStages == 2, "one unit ahead");
  cur.init(p, warp, sub);
  ld = cur;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    ld.settle(p);
    if (ld.left > 0) copy(s, ld);
    cp_async_commit();
    pos_ahead = ld.pos;
    ld.next(p);
    ld.read_pos(p);
  }
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) weights[i] = p.w[0] ? p.w[i / D][i % D] : 1.f;
  __syncthreads();
  const int page_rows = p.geom.hkv << p.geom.page_log2, page_mask = (1 << p.geom.page_log2) - 1;
  int stage = 0, fill = kStages - 1;
  // cur.left alone ends the loop; without the count beside it the compiler's code is slower (67K tokens into 4 bits, read back: 171.5 and 166.9 us)
  for (int todo = cur.left + warp; todo > 0; todo -= kWarps, cur.next(p)) {
    if (cur.left <= 0) break;
    cur.pos = pos_ahead;
    cur.has = cur.token < p.tokens;
    ld.settle(p);
    pos_ahead = ld.pos;
    const int64_t slot = cur.has ? __ldg(p.slots + cur.token) : -1;
    if (ld.left > 0) copy(fill, ld);
    cp_async_commit();
    ld.next(p);
    ld.read_pos(p);   // a unit ahead of its use
    cp_async_wait<kStages - 1>();
    __syncwarp();   // lanes read what others copied
    const int pos = cur.pos;
    const bool live = pos >= 0 && pos < p.max_pos, keep = slot_ok(p.geom, slot);
    const int64_t base = keep ? (slot >> p.geom.page_log2) * page_rows + (slot & page_mask) : 0;   // head 0's row
    // a padded token (negative position) gives zeros, one behind the table NaN
    const uint32_t fill_bits = pos < 0 ? 0u : 0x7fff7fffu;
    const uint4 constant = make_uint4(fill_bits, fill_bits, fill_bits, fill_bits);
    // the rows of a part's heads into the cache: D / V lanes a row, so that a token's lanes have one head's at once, or (e2m1) two heads'
    auto store_heads = [&](const uint8_t* in, const UnitPart& u, int which) {
      constexpr int V = kLaneValues<T>, kRows = V / 8;
      const int rl = l % (D / V), rh = l / (D / V);
      auto some = [&](auto count, int i) {
        constexpr int N = decltype(count)::value;
        StoredRow row[N];
#pragma unroll
        for (int h = 0; h < N; ++h) {
          const uint8_t* at = in + min((i + h) * kRows + rh, u.n - 1) * 512;
          LaneValues<T> v;
#pragma unroll
          for (int j = 0; j < V / 8; ++j) v[j] = *reinterpret_cast<const uint4*>(at + ((2 * V * rl + 16 * j) ^ swap));
          row[h] = make_row<D, T>(v);
        }
#pragma unroll
        for (int h = 0; h < N; ++h) {
          const int head = (i + h) * kRows + rh;
          if (keep && head < u.n)
            put_row<D, T>(row[h], base + (static_cast<int64_t>(u.head + head) << p.geom.page_log2), rl, which ? p.cache[1] : p.cache[0]);
        }
      };
      in_batches<2>((u.n + kRows - 1) / kRows, some);
    };
    if (cur.c >= p.first[2]) {
      store_heads(st.rows(stage, sub, 0), part_of(p, cur.c, 2), 1);
    } else {
      Rotation<INTER, false> rot;
      rot.load(st.table(stage, sub), live ? p.rot : 0, l);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const UnitPart u = part_of(p, cur.c, t);
        if (u.n <= 0) continue;
        __nv_bfloat16* out = p.out[0] + (cur.token * p.heads[0] + u.head) * D;   // q's
        uint8_t* in = st.rows(stage, sub, 0) + u.first * 512;
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
            r[h] = p.w[0] ? rsqrtf(r[h] * (1.f / D) + p.eps) : 1.f;
            float2 o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              o[j] = mul2(fma2(f[h][j], a[j], mul2(partner<INTER>(f[h], j), b[j])), make_float2(r[h], r[h]));
            const uint4 v = !live ? constant : AS_IS && 8 * l >= p.rot ? cols.load(in + (i + h) * 512, swap) : pack8(o);
            if (t == 1) cols.store(in + (i + h) * 512, swap, v);   // a key's row goes back to its place
            else if (cur.has) cols.store(out + (i + h) * D, v);
          }
        };
        in_batches<2>(u.n, some);
        if (t == 1) {
          __syncwarp();
          store_heads(in, u, 0);
        }
      }
    }
    __syncwarp();   // the stage has been read by every lane before the next iteration refills it
    stage = stage + 1 == kStages ? 0 : stage + 1;
    fill = fill + 1 == kStages ? 0 : fill + 1;
  }
}

template <int D, bool INTER, int T, bool AS_IS>
ffa_status launch(const AppendParams& p, int64_t tokens, cudaStream_t s) {
  static std::atomic<int> known[kDevices];
  static std::atomic<bool> raised[kDevices];
  int ctas = 0;
  return launch_units<D, false, false>(kv_append_kernel<D, INTER, T, AS_IS>, p, tokens, s, &ctas, known, raised);
}
template <int D, bool INTER, bool AS_IS>
ffa_status launch_type(const AppendParams& p, int type, int64_t tokens, cudaStream_t s) {
  if (type == kE2m1) return launch<D, INTER, kE2m1, AS_IS>(p, tokens, s);
  return type == kE4m3 ? launch<D, INTER, kE4m3, AS_IS>(p, tokens, s) : launch<D, INTER, kBf16, AS_IS>(p, tokens, s);
}
template <int D, bool INTER>
ffa_status launch_any(const AppendParams& p, int type, int64_t tokens, cudaStream_t s) {
  return copies_columns(p, D) ? launch_type<D, INTER, true>(p, type, tokens, s) : launch_type<D, INTER, false>(p, type, tokens, s);
}

}  // namespace
}  // namespace ffa

using namespace ffa;

extern "C" {

ffa_status ffa_kv_cache_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                               int64_t tokens, int32_t hq, const float* q_weight, const float* k_weight, float eps,
                               const float* cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                               const int32_t* positions, int32_t n_axes, const uint8_t* pair_axis, const int64_t* slots,
                               const ffa_kv_cache* cache, void* q_out, void* stream) {
  AppendParams p{};
  ffa_status st = check_cache(cache, p.geom);
  if (st != FFA_OK) return st;
  if (n_axes <= 0) return FFA_ERR_INVALID_ARG;
  const int32_t d = cache->d, hkv = cache->hkv;
  st = check_common(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin, max_pos, rot_dim, positions, n_axes,
                    pair_axis, p);
  if (st != FFA_OK) return st;
  if (tokens == 0) return FFA_OK;
  if (!v || !slots || !q_out || !aligned16(v) || !aligned16(q_out) || (reinterpret_cast<uintptr_t>(slots) & 7u)) return FFA_ERR_INVALID_ARG;
  if (v_stride % 8 != 0 || (tokens > 1 && v_stride < static_cast<int64_t>(hkv) * d)) return FFA_ERR_INVALID_ARG;
  const CacheSpans at(*cache);
  Span outs[7] = {{q_out, 2 * tokens * hq * d}};
  for (int i = 0; i < at.n; ++i) outs[1 + i] = at.s[i];
  const Span in[] = {{q, span_bytes(tokens, q_stride, hq, d)}, {k, span_bytes(tokens, k_stride, hkv, d)}, {v, span_bytes(tokens, v_stride, hkv, d)},
                     {q_weight, q_weight ? 4 * d : 0}, {k_weight, k_weight ? 4 * d : 0}, {cos_sin, 4 * max_pos * rot_dim},
                     {positions, 4 * tokens * n_axes}, {slots, 8 * tokens}};
  if (any_meet(outs, 1 + at.n, in, 8)) return FFA_ERR_INVALID_ARG;
  p.x[2] = static_cast<const __nv_bfloat16*>(v);
  p.x_stride[2] = v_stride;
  p.heads[2] = hkv;
  p.out[0] = static_cast<__nv_bfloat16*>(q_out);
  p.cache[0] = k_rows(*cache);
  p.cache[1] = v_rows(*cache);
  p.slots = slots;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d == 128) return interleaved ? launch_any<128, true>(p, cache->dtype, tokens, s) : launch_any<128, false>(p, cache->dtype, tokens, s);
  return interleaved ? launch_any<64, true>(p, cache->dtype, tokens, s) : launch_any<64, false>(p, cache->dtype, tokens, s);
}

}  // extern "C"
