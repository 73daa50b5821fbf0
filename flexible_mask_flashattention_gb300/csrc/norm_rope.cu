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
// Both are bound by HBM: 4 bytes a value forward (x in, out out), 6 backward (x, dout in, dx out).  A lane holds 8
// consecutive values of a row (one 16-byte load), d / 8 lanes a row; a warp takes one token and up to kUnroll passes
// over its heads, all loads issued first, and reads the token's table row once for them.  Norm statistics, rotation
// and every gradient sum are fp32; the one rounding to bf16 is the store's.
#include <cuda_bf16.h>

#include <algorithm>

#include "ffa_internal.h"
#include "ptx.cuh"

namespace ffa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;          // head passes of one warp unit, loaded together
constexpr int kMaxBwdCtas = 1024;   // partial weight gradients the workspace holds

struct NormRopeParams {
  const __nv_bfloat16* x[2];      // q, k
  int64_t x_stride[2];            // values between tokens
  const __nv_bfloat16* dout[2];   // backward: gradients of the outputs, contiguous
  __nv_bfloat16* out[2];          // forward: outputs; backward: dx; contiguous
  const float* w[2];
  int32_t heads[2];
  int32_t chunks[2];              // warp units a token
  int64_t units;
  float eps;
  const float* cos_sin;
  int64_t max_pos;
  int32_t rot;
  const int32_t* pos;
  float* partial;                 // backward: [CTAs][2][d]
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 shfl4(const uint4& v, int src) {
  uint4 r;
  r.x = __shfl_sync(0xffffffffu, v.x, src);
  r.y = __shfl_sync(0xffffffffu, v.y, src);
  r.z = __shfl_sync(0xffffffffu, v.z, src);
  r.w = __shfl_sync(0xffffffffu, v.w, src);
  return r;
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// A lane's part of one token's rotation, for the 8 values it holds of each row: value j becomes
// c[j] v[j] + s[j] (its pair partner's value).  Columns behind rot_dim have c = 1, s = 0.  `src` is the lane that holds
// the partners (itself when pairs are interleaved).
template <int D, bool INTER>
struct Rotation {
  float c[8], s[8];
  int src;
  __device__ __forceinline__ void identity(int lane) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 1.f, s[j] = 0.f;
    src = lane;
  }
  __device__ __forceinline__ void load(const float* row, int rot, int lane) {
    identity(lane);
    const int l = lane & (D / 8 - 1);
    if (8 * l >= rot) return;
    if constexpr (INTER) {
      const float4 c4 = __ldg(reinterpret_cast<const float4*>(row + 4 * l));
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(row + rot / 2 + 4 * l));
      const float cc[4] = {c4.x, c4.y, c4.z, c4.w}, ss[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) c[2 * i] = c[2 * i + 1] = cc[i], s[2 * i] = -ss[i], s[2 * i + 1] = ss[i];
    } else {   // rot_dim is a multiple of 16, so a lane's values are all in one half
      const int half = rot >> 4;   // lanes a half
      const bool lo = l < half;
      const int i = 8 * (lo ? l : l - half);
      load8(row + i, c);
      load8(row + rot / 2 + i, s);
      if (lo) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] = -s[j];
      }
      src = lo ? lane + half : lane - half;
    }
  }
  // The values of f's pair partners; v is f in its packed form.
  __device__ __forceinline__ void partners(const uint4& v, const float (&f)[8], float (&p)[8]) const {
    if constexpr (INTER) {
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = f[j ^ 1];
    } else {
      unpack8(shfl4(v, src), p);
    }
  }
};

// Sum over the D / 8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = D / 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Unit {
  int64_t token;
  int which;    // 0 q, 1 k
  int head0;    // first head of the unit
  int64_t pos;
};
__device__ __forceinline__ Unit unit_of(const NormRopeParams& p, int64_t u, int heads_per_unit) {
  const int per = p.chunks[0] + p.chunks[1];
  Unit r;
  r.token = u / per;
  const int c = static_cast<int>(u - r.token * per);
  r.which = c >= p.chunks[0];
  r.head0 = (r.which ? c - p.chunks[0] : c) * heads_per_unit;
  r.pos = p.pos[r.token];
  return r;
}

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_fwd_kernel(NormRopeParams p) {
  constexpr int L = D / 8, RW = 32 / L;
  const int lane = threadIdx.x & 31, l = lane & (L - 1), sub = lane / L;
  const int64_t u = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5);
  if (u >= p.units) return;
  const Unit un = unit_of(p, u, kUnroll * RW);
  const int heads = p.heads[un.which];
  const __nv_bfloat16* x = p.x[un.which] + un.token * p.x_stride[un.which] + 8 * l;
  uint4 v[kUnroll];
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    const int h = un.head0 + i * RW + sub;
    v[i] = h < heads ? __ldg(reinterpret_cast<const uint4*>(x + h * D)) : uint4{};
  }
  Rotation<D, INTER> rot;
  rot.identity(lane);
  if (un.pos >= 0 && un.pos < p.max_pos) rot.load(p.cos_sin + un.pos * p.rot, p.rot, lane);
  // own and partner coefficients with their weights: out_j = r (x_j a_j + partner_j b_j)
  float a[8], b[8];
  {
    float w[8];
    load8(p.w[un.which] + 8 * l, w);
    const int pl = (rot.src & (L - 1)) * 8;
    float wp[8];
    load8(p.w[un.which] + pl, wp);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      a[j] = rot.c[j] * w[j];
      b[j] = rot.s[j] * (INTER ? w[j ^ 1] : wp[j]);
    }
  }
  // a padded token (negative position) gives zeros, one behind the table NaN
  const float keep = un.pos < 0 ? 0.f : un.pos < p.max_pos ? 1.f : __int_as_float(0x7fffffff);
  __nv_bfloat16* out = p.out[un.which] + un.token * heads * D + 8 * l;
#pragma unroll
  for (int i = 0; i < kUnroll; ++i) {
    float f[8], q[8], o[8], ss = 0.f;
    unpack8(v[i], f);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + p.eps);
    rot.partners(v[i], f, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = r * fmaf(f[j], a[j], q[j] * b[j]);
    if (keep != 1.f) {
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = keep;
    }
    const int h = un.head0 + i * RW + sub;
    if (h < heads) *reinterpret_cast<uint4*>(out + h * D) = pack8(o);
  }
}

// Persistent: each warp strides over the units and keeps its 8 columns' weight-gradient sums for q and k in registers;
// a CTA adds its warps' in a fixed order and writes one partial row pair, which norm_rope_dw_kernel adds up.  The
// assignment of units to warps is static, so the result does not depend on timing.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) norm_rope_bwd_kernel(NormRopeParams p) {
  constexpr int L = D / 8, RW = 32 / L;
  constexpr int kU = 2;   // passes loaded together: x and dout each
  __shared__ float red[kWarps][2][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (L - 1), sub = lane / L;
  float acc[2][8] = {};
  const int64_t stride = gridDim.x * static_cast<int64_t>(kWarps);
  for (int64_t u = blockIdx.x * static_cast<int64_t>(kWarps) + warp; u < p.units; u += stride) {
    const Unit un = unit_of(p, u, kU * RW);
    const int heads = p.heads[un.which];
    const __nv_bfloat16* x = p.x[un.which] + un.token * p.x_stride[un.which] + 8 * l;
    const __nv_bfloat16* dy = p.dout[un.which] + un.token * heads * D + 8 * l;
    uint4 v[kU], g[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int h = un.head0 + i * RW + sub;
      v[i] = h < heads ? __ldg(reinterpret_cast<const uint4*>(x + h * D)) : uint4{};
      g[i] = h < heads ? __ldg(reinterpret_cast<const uint4*>(dy + h * D)) : uint4{};
    }
    Rotation<D, INTER> rot;
    rot.identity(lane);
    if (un.pos >= 0 && un.pos < p.max_pos) rot.load(p.cos_sin + un.pos * p.rot, p.rot, lane);
    float w[8];
    load8(p.w[un.which] + 8 * l, w);
    __nv_bfloat16* dx = p.out[un.which] + un.token * heads * D + 8 * l;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      float f[8], gf[8], gp[8], ss = 0.f, hx = 0.f;
      unpack8(v[i], f);
      unpack8(g[i], gf);
      rot.partners(g[i], gf, gp);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gf[j] = fmaf(gf[j], rot.c[j], -gp[j] * rot.s[j]);   // R^T dout: the transposed rotation turns the sign of s
        ss = fmaf(f[j], f[j], ss);
        hx = fmaf(gf[j] * w[j], f[j], hx);
      }
      const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + p.eps);
      const float c = row_sum<D>(hx) * r * r * (1.f / D);
      const int h = un.head0 + i * RW + sub;
      if (un.pos < 0) {   // padded: no gradient
        if (h < heads) *reinterpret_cast<uint4*>(dx + h * D) = uint4{};
        continue;
      }
      const float bad = un.pos < p.max_pos ? 0.f : __int_as_float(0x7fffffff);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = r * fmaf(gf[j], w[j], -f[j] * c) + bad;
        acc[0][j] += un.which == 0 ? gf[j] * (f[j] * r) + bad : 0.f;
        acc[1][j] += un.which == 1 ? gf[j] * (f[j] * r) + bad : 0.f;
      }
      if (h < heads) *reinterpret_cast<uint4*>(dx + h * D) = pack8(o);
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float s = acc[t][j];
#pragma unroll
      for (int o = L; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (sub == 0) red[warp][t][8 * l + j] = s;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) s += red[k][i / D][i % D];
    p.partial[blockIdx.x * static_cast<int64_t>(2 * D) + i] = s;
  }
}

// dw = sum of the CTAs' partial rows, in a fixed order: 32 columns a block, 32 partial rows at a time.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* partial, int n, float* dqw, float* dkw) {
  __shared__ float red[32][33];
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

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Do the byte ranges [a, a + na) and [b, b + nb) meet?
bool meet(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) && y < x + static_cast<uintptr_t>(na);
}

struct Span {
  const void* p;
  int64_t n;
};

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

void set_units(NormRopeParams& p, int64_t tokens, int heads_per_unit) {
  for (int i = 0; i < 2; ++i) p.chunks[i] = (p.heads[i] + heads_per_unit - 1) / heads_per_unit;
  p.units = tokens * (p.chunks[0] + p.chunks[1]);
}

// Bytes from the first to the last value of a strided [tokens][heads][d] bf16 tensor.
int64_t span_bytes(int64_t tokens, int64_t stride, int64_t heads, int64_t d) {
  return tokens <= 0 ? 0 : 2 * ((tokens - 1) * stride + heads * d);
}

bool any_meet(const Span* out, int n_out, const Span* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (meet(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (meet(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
  }
  return false;
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
  set_units(p, tokens, kUnroll * 256 / d);
  const int64_t blocks = (p.units + kWarps - 1) / kWarps;
  if (blocks > 0x7fffffff) return FFA_ERR_OVERFLOW;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(blocks));
  if (d == 128)
    (interleaved ? norm_rope_fwd_kernel<128, true> : norm_rope_fwd_kernel<128, false>)<<<grid, kThreads, 0, s>>>(p);
  else
    (interleaved ? norm_rope_fwd_kernel<64, true> : norm_rope_fwd_kernel<64, false>)<<<grid, kThreads, 0, s>>>(p);
  return cuda_status(cudaGetLastError());
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
  set_units(p, tokens, 2 * 256 / d);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int device = 0, sms = 0;
  if (cudaGetDevice(&device) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) != cudaSuccess)
    return FFA_ERR_CUDA;
  const int64_t want = (p.units + kWarps - 1) / kWarps;
  const int blocks = static_cast<int>(std::min<int64_t>({want, int64_t{4} * sms, int64_t{kMaxBwdCtas}}));
  if (blocks > 0) {
    if (d == 128)
      (interleaved ? norm_rope_bwd_kernel<128, true> : norm_rope_bwd_kernel<128, false>)<<<blocks, kThreads, 0, s>>>(p);
    else
      (interleaved ? norm_rope_bwd_kernel<64, true> : norm_rope_bwd_kernel<64, false>)<<<blocks, kThreads, 0, s>>>(p);
  }
  if (d == 128)
    norm_rope_dw_kernel<128><<<8, 1024, 0, s>>>(p.partial, blocks, dq_weight, dk_weight);
  else
    norm_rope_dw_kernel<64><<<4, 1024, 0, s>>>(p.partial, blocks, dq_weight, dk_weight);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"
