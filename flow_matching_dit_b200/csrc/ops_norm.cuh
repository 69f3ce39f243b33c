// gdit_norm_residual: h' = residual_scale h + gate * post(y),
// u = pre(h') (1 + scale) + shift, one pass over the rows.
#pragma once

#include "ops_common.cuh"

namespace gdit {

struct NormArgs {
  const void* h;
  const void* y;
  void* out_h;
  void* out_u;
  const float *post_gain, *post_bias, *gate, *pre_gain, *pre_bias, *scale, *shift;
  const int* row_group;
  long long rows, ldh, ldy, ldoh, ldou;
  int dim;
  int h_f32, y_f32, u_f32;
  int post, pre;
  int gate_groups, mod_groups;
  float residual_scale, eps;
};

// Mean and sum of squared deviations of n values, and their union (Chan,
// Golub and LeVeque's pairwise update): no cancellation when the mean is large
// against the deviations.
struct Moments {
  float n, mean, m2;
};

__device__ __forceinline__ Moments merge(Moments a, Moments b) {
  const float n = a.n + b.n;
  if (n == 0.f) return a;
  const float d = b.mean - a.mean, f = b.n / n;
  return {n, a.mean + d * f, a.m2 + b.m2 + d * d * a.n * f};
}

__device__ __forceinline__ float load_elt(const void* p, long long i, int f32) {
  return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void store_elt(void* p, long long i, int f32, float v) {
  if (f32) static_cast<float*>(p)[i] = v;
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// 8 consecutive values; i a multiple of 8 on 16-byte aligned rows.
__device__ __forceinline__ void load8(const void* p, long long i, int f32, float (&v)[8]) {
  if (f32) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = q[0], b = q[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + i);
    const float4 x = bf16x4_to_f32(make_uint2(a.x, a.y)), y = bf16x4_to_f32(make_uint2(a.z, a.w));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
}

__device__ __forceinline__ void store8(void* p, long long i, int f32, const float (&v)[8]) {
  if (f32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + i) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  }
}

// One row is held by a team of `team` threads (whole warps), 8 * NV values a
// thread, all in registers.  VEC: thread t holds the 8-value vectors t, t +
// team, ...; otherwise the values t, t + team, ...
template <bool VEC, int NV>
struct RowTeam {
  int dim, team, t, warps, bar;
  float* red;   // 3 floats per warp of the team

  __device__ __forceinline__ int index(int c, int j) const {   // of value j of vector c
    return VEC ? (c * team + t) * 8 + j : (c * 8 + j) * team + t;
  }

  __device__ __forceinline__ void load(const void* p, long long base, int f32, float (&v)[NV][8]) const {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      if (VEC) {
        if (index(c, 0) < dim) load8(p, base + index(c, 0), f32, v[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (index(c, j) < dim) v[c][j] = load_elt(p, base + index(c, j), f32);
      }
    }
  }

  __device__ __forceinline__ void store(void* p, long long base, int f32, const float (&v)[NV][8]) const {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      if (VEC) {
        if (index(c, 0) < dim) store8(p, base + index(c, 0), f32, v[c]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (index(c, j) < dim) store_elt(p, base + index(c, j), f32, v[c][j]);
      }
    }
  }

  // v = v * a + b with per-channel f32 vectors (NULL: 1 or 0; one: a is 1 + a)
  __device__ __forceinline__ void affine(float (&v)[NV][8], const float* a, const float* b, float one) const {
    if (a == nullptr && b == nullptr) return;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      if (VEC) {
        if (index(c, 0) >= dim) continue;
        float f[8];
        if (a != nullptr) {
          load8(a, index(c, 0), 1, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] *= one + f[j];
        }
        if (b != nullptr) {
          load8(b, index(c, 0), 1, f);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[c][j] += f[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (index(c, j) >= dim) continue;
          if (a != nullptr) v[c][j] *= one + a[index(c, j)];
          if (b != nullptr) v[c][j] += b[index(c, j)];
        }
      }
    }
  }

  // The row's moments, in every thread of the team.
  __device__ __forceinline__ Moments moments(const float (&v)[NV][8]) const {
    float n = 0.f, sum = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (index(c, VEC ? 0 : j) < dim) n += 1.f, sum += v[c][j];
    Moments m = {n, n > 0.f ? sum / n : 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (index(c, VEC ? 0 : j) < dim) m.m2 += (v[c][j] - m.mean) * (v[c][j] - m.mean);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Moments b = {__shfl_xor_sync(~0u, m.n, o), __shfl_xor_sync(~0u, m.mean, o),
                         __shfl_xor_sync(~0u, m.m2, o)};
      // the lower lane's moments first on both sides, so that both get the same bits
      m = (threadIdx.x & o) ? merge(b, m) : merge(m, b);
    }
    if (warps > 1) {
      const int w = t >> 5;
      named_bar_sync(bar, team);   // the previous sums have been read
      if ((t & 31) == 0) red[3 * w] = m.n, red[3 * w + 1] = m.mean, red[3 * w + 2] = m.m2;
      named_bar_sync(bar, team);
      m = {red[0], red[1], red[2]};
      for (int i = 1; i < warps; ++i) m = merge(m, {red[3 * i], red[3 * i + 1], red[3 * i + 2]});
    }
    return m;
  }

  __device__ __forceinline__ float square_sum(const float (&v)[NV][8]) const {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (index(c, VEC ? 0 : j) < dim) s += v[c][j] * v[c][j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (warps > 1) {
      named_bar_sync(bar, team);
      if ((t & 31) == 0) red[t >> 5] = s;
      named_bar_sync(bar, team);
      s = red[0];
      for (int i = 1; i < warps; ++i) s += red[i];
    }
    return s;
  }

  __device__ __forceinline__ void norm(float (&v)[NV][8], int kind, const float* gain, const float* bias,
                                       float eps) const {
    if (kind == GDIT_NORM_NONE) return;
    float mean = 0.f, rs;
    if (kind == GDIT_NORM_LAYER) {
      const Moments m = moments(v);
      mean = m.mean;
      rs = rsqrtf(m.m2 / (float)dim + eps);
    } else {
      rs = rsqrtf(square_sum(v) / (float)dim + eps);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = (v[c][j] - mean) * rs;
    affine(v, gain, bias, 0.f);
  }
};

constexpr int kNormThreads = 512;   // most threads of a CTA

template <bool VEC, int NV>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormArgs a, int team, int teams) {
  __shared__ float red[kNormThreads / 32 * 3];
  const int which = threadIdx.x / team;
  RowTeam<VEC, NV> T;
  T.dim = a.dim;
  T.team = team;
  T.t = threadIdx.x - which * team;
  T.warps = team >> 5;
  T.bar = 1 + which;
  T.red = red + which * T.warps * 3;
  pdl_wait();
  pdl_launch_dependents();
  for (long long r = (long long)blockIdx.x * teams + which; r < a.rows; r += (long long)gridDim.x * teams) {
    float h[NV][8], y[NV][8];
    T.load(a.h, r * a.ldh, a.h_f32, h);
    if (a.y != nullptr) T.load(a.y, r * a.ldy, a.y_f32, y);
    long long g = a.row_group != nullptr ? a.row_group[r] : 0;
    const int groups = max(a.gate_groups, a.mod_groups);
    const bool bad = groups > 1 && (g < 0 || (a.gate_groups > 1 && g >= a.gate_groups) ||
                                    (a.mod_groups > 1 && g >= a.mod_groups));
    if (bad) {
      g = 0;
      if (T.t == 0) atomicOr(&g_op_status, OP_ERR_GROUP);
    }
    const long long go = a.gate_groups > 1 ? g * a.dim : 0, mo = a.mod_groups > 1 ? g * a.dim : 0;
    if (a.y != nullptr) {
      T.norm(y, a.post, a.post_gain, a.post_bias, a.eps);
      T.affine(y, a.gate != nullptr ? a.gate + go : nullptr, nullptr, 0.f);
    }
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h[c][j] = a.y != nullptr ? fmaf(a.residual_scale, h[c][j], y[c][j]) : a.residual_scale * h[c][j];
        if (bad) h[c][j] = __int_as_float(0x7fffffff);
      }
    if (a.out_h != nullptr) T.store(a.out_h, r * a.ldoh, a.h_f32, h);
    if (a.out_u != nullptr) {
      T.norm(h, a.pre, a.pre_gain, a.pre_bias, a.eps);
      T.affine(h, a.scale != nullptr ? a.scale + mo : nullptr, a.shift != nullptr ? a.shift + mo : nullptr, 1.f);
      T.store(a.out_u, r * a.ldou, a.u_f32, h);
    }
  }
}

inline void launch_norm(const NormArgs& a, int sms, cudaStream_t s) {
  auto aligned = [&](const void* p, long long ld, int f32) {
    return p == nullptr || (((uintptr_t)p & 15u) == 0 && (ld * (f32 ? 4 : 2)) % 16 == 0);
  };
  bool vec = a.dim % 8 == 0 && aligned(a.h, a.ldh, a.h_f32) && aligned(a.y, a.ldy, a.y_f32) &&
             aligned(a.out_h, a.ldoh, a.h_f32) && aligned(a.out_u, a.ldou, a.u_f32);
  for (const float* p : {a.post_gain, a.post_bias, a.gate, a.pre_gain, a.pre_bias, a.scale, a.shift})
    vec = vec && ((uintptr_t)p & 15u) == 0;
  int nv = 1;
  while (8 * nv * kNormThreads < a.dim) nv *= 2;
  const int team = ((a.dim + 8 * nv - 1) / (8 * nv) + 31) / 32 * 32;
  const int teams = std::max(1, 256 / team);
  const long long blocks = std::min<long long>((a.rows + teams - 1) / teams, (long long)sms * 8);
  const dim3 grid((unsigned)blocks), block(team * teams);
  if (vec) {
    if (nv == 1) launch_op(s, 1, norm_kernel<true, 1>, grid, block, 0, a, team, teams);
    else if (nv == 2) launch_op(s, 1, norm_kernel<true, 2>, grid, block, 0, a, team, teams);
    else launch_op(s, 1, norm_kernel<true, 4>, grid, block, 0, a, team, teams);
  } else {
    if (nv == 1) launch_op(s, 1, norm_kernel<false, 1>, grid, block, 0, a, team, teams);
    else if (nv == 2) launch_op(s, 1, norm_kernel<false, 2>, grid, block, 0, a, team, teams);
    else launch_op(s, 1, norm_kernel<false, 4>, grid, block, 0, a, team, teams);
  }
}

}  // namespace gdit
