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
//
// Positions of several axes (time, height, width): pair i of a token turns by the angle of the position on its axis, so that a token's cosines and sines
// come from several rows of the table.  A token's lanes read its positions one each and shuffle them to where a row's address is made.  Where
// each 16 bytes of a table row, 4 pairs, go by one axis, they are copied as before; otherwise value by value, neighbouring lanes neighbouring pairs;
// both through L1, as thousands of tokens share a row of the time's.  Units are larger, 6 and 5 heads, as their table rows cost more.  Measured
// (128K tokens, 64 + 8 heads, d = 128; 715 us at a copy's rate): one axis 731 us, sections of 16, 24 and 24 pairs 725, axes in turns
// 733; units of 5 heads 759 and 812, and every lane reading every position 898 and 963.  Backward (32K tokens, 270 us): 279, 281 and 296.  The
// rotation alone (no weights) is the same forward kernel, backward too: the gradients' rotation is the other way round.  Of fewer columns than a
// row has it is one that copies the others (rot_dim 96: 729 us).
#include "norm_rope.cuh"

namespace ffa {
namespace {

template <int D, bool INTER, bool AXES, bool AS_IS>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(NormRopeParams p) {
  constexpr int L = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  float* weights = reinterpret_cast<float*>(smem);   // [2][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (L - 1), sub = lane / L;
  const Stages<D, false> st{smem + 2 * D * 4 + warp * kStages * Stages<D, false>::stage_bytes(p.unit), p.unit};
  const Columns<D, INTER> cols(l, p.rot);
  const int swap = Stages<D, false>::swap(sub);
  UnitWalk<D, AXES> cur, ld;
  [[maybe_unused]] int pos_ahead = -1;   // several axes: what the copies one unit ahead have found of its positions
  static_assert(kStages == 2, "one unit ahead");
  cur.init(p, warp, sub);
  ld = cur;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if constexpr (AXES) ld.settle(p);
    if (ld.left > 0) copy_unit<D, false, AXES>(p, st, s, ld);
    cp_async_commit();
    if constexpr (AXES) pos_ahead = ld.pos;
    ld.next(p);
    ld.read_pos(p);
  }
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) weights[i] = AXES && !p.w[0] ? 1.f : p.w[i / D][i % D];
  __syncthreads();
  int stage = 0, fill = kStages - 1;
  for (int todo = cur.left + warp; todo > 0; todo -= kWarps, cur.next(p)) {
    __syncthreads();   // the warps' copies go out together: one run of memory
    if (cur.left <= 0) continue;
    if constexpr (AXES) {
      cur.pos = pos_ahead;
      cur.has = cur.token < p.tokens;
      ld.settle(p);
      pos_ahead = ld.pos;
    } else {
      cur.read_pos(p);   // again: from L1
    }
    if (ld.left > 0) copy_unit<D, false, AXES>(p, st, fill, ld);
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
    rot.load(st.table(stage, sub), live ? p.rot : 0, l, AXES ? p.turn : 1.f);
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
          r[h] = AXES && !p.w[0] ? 1.f : rsqrtf(r[h] * (1.f / D) + p.eps);
          float2 o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            o[j] = mul2(fma2(f[h][j], a[j], mul2(partner<INTER>(f[h], j), b[j])), make_float2(r[h], r[h]));
          if (live) cols.store(out + (i + h) * D, AS_IS && 8 * l >= p.rot ? cols.load(in + (i + h) * 512, swap) : pack8(o));
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
template <int D, bool INTER, bool AXES>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(NormRopeParams p) {
  constexpr int L = D / 8;
  extern __shared__ __align__(128) uint8_t smem[];
  float* weights = reinterpret_cast<float*>(smem);   // [2][D]
  float* red = weights + 2 * D;                      // [kWarps][2][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (L - 1), sub = lane / L;
  const Stages<D, true> st{smem + (1 + kWarps) * 2 * D * 4 + warp * kStages * Stages<D, true>::stage_bytes(p.unit), p.unit};
  const Columns<D, INTER> cols(l, p.rot);
  const int swap = Stages<D, true>::swap(sub);
  UnitWalk<D, AXES> cur, ld;
  [[maybe_unused]] int pos_ahead = -1;   // several axes: what the copies one unit ahead have found of its positions
  static_assert(kStages == 2, "one unit ahead");
  cur.init(p, warp, sub);
  ld = cur;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if constexpr (AXES) ld.settle(p);
    if (ld.left > 0) copy_unit<D, true, AXES>(p, st, s, ld);
    cp_async_commit();
    if constexpr (AXES) pos_ahead = ld.pos;
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
    if constexpr (AXES) {
      cur.pos = pos_ahead;
      cur.has = cur.token < p.tokens;
      ld.settle(p);
      pos_ahead = ld.pos;
    } else {
      cur.read_pos(p);   // again: from L1
    }
    if (ld.left > 0) copy_unit<D, true, AXES>(p, st, fill, ld);
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

template <int D, bool INTER, bool BWD, bool AXES, bool AS_IS>
ffa_status launch(const NormRopeParams& p, int64_t tokens, cudaStream_t s, int* ctas) {
  static std::atomic<int> known[kDevices];
  static std::atomic<bool> raised[kDevices];
  if constexpr (BWD) return launch_units<D, true, AXES>(norm_rope_bwd_kernel<D, INTER, AXES>, p, tokens, s, ctas, known, raised);
  else return launch_units<D, false, AXES>(norm_rope_fwd_kernel<D, INTER, AXES, AS_IS>, p, tokens, s, ctas, known, raised);
}

template <bool BWD, bool AXES, bool AS_IS = false>
ffa_status launch_of(const NormRopeParams& p, int64_t tokens, int d, bool interleaved, cudaStream_t s, int* ctas) {
  if (d == 128)
    return interleaved ? launch<128, true, BWD, AXES, AS_IS>(p, tokens, s, ctas) : launch<128, false, BWD, AXES, AS_IS>(p, tokens, s, ctas);
  return interleaved ? launch<64, true, BWD, AXES, AS_IS>(p, tokens, s, ctas) : launch<64, false, BWD, AXES, AS_IS>(p, tokens, s, ctas);
}
template <bool BWD>
ffa_status launch_any(const NormRopeParams& p, int64_t tokens, int d, bool interleaved, cudaStream_t s, int* ctas) {
  if constexpr (!BWD) {
    if (p.axes && copies_columns(p, d)) return launch_of<false, true, true>(p, tokens, d, interleaved, s, ctas);
  }
  return p.axes ? launch_of<BWD, true>(p, tokens, d, interleaved, s, ctas) : launch_of<BWD, false>(p, tokens, d, interleaved, s, ctas);
}

ffa_status forward(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens, int32_t hq, int32_t hkv, int32_t d,
                   const float* q_weight, const float* k_weight, float eps, const float* cos_sin, int64_t max_pos, int32_t rot_dim,
                   int32_t interleaved, const int32_t* positions, int32_t n_axes, const uint8_t* pair_axis, float turn, void* q_out,
                   void* k_out, void* stream) {
  NormRopeParams p{};
  const ffa_status st = check_common(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin,
                                     max_pos, rot_dim, positions, n_axes, pair_axis, p);
  if (st != FFA_OK) return st;
  if (tokens == 0) return FFA_OK;
  if (!q_out || !k_out || !aligned16(q_out) || !aligned16(k_out)) return FFA_ERR_INVALID_ARG;
  const Span in[] = {{q, span_bytes(tokens, q_stride, hq, d)}, {k, span_bytes(tokens, k_stride, hkv, d)},
                     {q_weight, q_weight ? 4 * d : 0}, {k_weight, k_weight ? 4 * d : 0}, {cos_sin, 4 * max_pos * rot_dim},
                     {positions, 4 * tokens * std::max(n_axes, 1)}};
  const Span outs[] = {{q_out, 2 * tokens * hq * d}, {k_out, 2 * tokens * hkv * d}};
  if (any_meet(outs, 2, in, 6)) return FFA_ERR_INVALID_ARG;
  p.out[0] = static_cast<__nv_bfloat16*>(q_out);
  p.out[1] = static_cast<__nv_bfloat16*>(k_out);
  p.turn = turn;
  int ctas = 0;
  return launch_any<false>(p, tokens, d, interleaved != 0, static_cast<cudaStream_t>(stream), &ctas);
}

size_t bwd_workspace(int32_t d) { return d == 64 || d == 128 ? static_cast<size_t>(kMaxBwdCtas) * 2 * d * sizeof(float) : 0; }

ffa_status backward(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens, int32_t hq, int32_t hkv, int32_t d,
                    const float* q_weight, const float* k_weight, float eps, const float* cos_sin, int64_t max_pos, int32_t rot_dim,
                    int32_t interleaved, const int32_t* positions, int32_t n_axes, const uint8_t* pair_axis, const void* dq_out,
                    const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                    void* stream) {
  NormRopeParams p{};
  const ffa_status st = check_common(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin,
                                     max_pos, rot_dim, positions, n_axes, pair_axis, p);
  if (st != FFA_OK) return st;
  if (!dq_weight || !dk_weight || !workspace || !aligned16(dq_weight) || !aligned16(dk_weight) || !aligned16(workspace))
    return FFA_ERR_INVALID_ARG;
  if (workspace_bytes < bwd_workspace(d)) return FFA_ERR_INVALID_ARG;
  if (tokens > 0 && (!dq_out || !dk_out || !dq || !dk || !aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) ||
                     !aligned16(dk)))
    return FFA_ERR_INVALID_ARG;
  const int64_t nq = 2 * tokens * hq * d, nk = 2 * tokens * hkv * d;
  const Span in[] = {{q, span_bytes(tokens, q_stride, hq, d)}, {k, span_bytes(tokens, k_stride, hkv, d)},
                     {q_weight, 4 * d}, {k_weight, 4 * d}, {cos_sin, 4 * max_pos * rot_dim}, {positions, 4 * tokens * std::max(n_axes, 1)},
                     {dq_out, nq}, {dk_out, nk}};
  const Span outs[] = {{dq, nq}, {dk, nk}, {dq_weight, 4 * d}, {dk_weight, 4 * d},
                       {workspace, static_cast<int64_t>(bwd_workspace(d))}};
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

}  // namespace
}  // namespace ffa

using namespace ffa;

extern "C" {

ffa_status ffa_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                            int32_t hq, int32_t hkv, int32_t d, const float* q_weight, const float* k_weight, float eps,
                            const float* cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                            const int32_t* positions, void* q_out, void* k_out, void* stream) {
  return forward(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin, max_pos, rot_dim, interleaved, positions,
                 0, nullptr, 1.f, q_out, k_out, stream);
}

ffa_status ffa_qk_norm_rope_axes(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                                 int32_t hq, int32_t hkv, int32_t d, const float* q_weight, const float* k_weight,
                                 float eps, const float* cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                                 const int32_t* positions, int32_t n_axes, const uint8_t* pair_axis, void* q_out,
                                 void* k_out, void* stream) {
  if (n_axes <= 0) return FFA_ERR_INVALID_ARG;
  return forward(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin, max_pos, rot_dim, interleaved, positions,
                 n_axes, pair_axis, 1.f, q_out, k_out, stream);
}

size_t ffa_qk_norm_rope_bwd_workspace_size(int32_t d) { return bwd_workspace(d); }

ffa_status ffa_qk_norm_rope_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                                int32_t hq, int32_t hkv, int32_t d, const float* q_weight, const float* k_weight,
                                float eps, const float* cos_sin, int64_t max_pos, int32_t rot_dim, int32_t interleaved,
                                const int32_t* positions, const void* dq_out, const void* dk_out, void* dq, void* dk,
                                float* dq_weight, float* dk_weight, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return backward(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin, max_pos, rot_dim, interleaved, positions,
                  0, nullptr, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, workspace_bytes, stream);
}

ffa_status ffa_qk_norm_rope_axes_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, int64_t tokens,
                                     int32_t hq, int32_t hkv, int32_t d, const float* q_weight, const float* k_weight,
                                     float eps, const float* cos_sin, int64_t max_pos, int32_t rot_dim,
                                     int32_t interleaved, const int32_t* positions, int32_t n_axes,
                                     const uint8_t* pair_axis, const void* dq_out, const void* dk_out, void* dq,
                                     void* dk, float* dq_weight, float* dk_weight, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (n_axes <= 0) return FFA_ERR_INVALID_ARG;
  if (q_weight || k_weight)
    return backward(q, q_stride, k, k_stride, tokens, hq, hkv, d, q_weight, k_weight, eps, cos_sin, max_pos, rot_dim, interleaved,
                    positions, n_axes, pair_axis, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace, workspace_bytes, stream);
  // the rotation alone: the gradients are the outputs' turned back
  return forward(dq_out, int64_t{hq} * d, dk_out, int64_t{hkv} * d, tokens, hq, hkv, d, nullptr, nullptr, eps, cos_sin, max_pos, rot_dim,
                 interleaved, positions, n_axes, pair_axis, -1.f, dq, dk, stream);
}

}  // extern "C"
