// gdit_norm_residual: h' = residual_scale h + gate * post(y),
// u = pre(h') (1 + scale) + shift, one pass over the rows.
#pragma once

#include <type_traits>

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

// A row is held in registers by a team of whole warps, 4 * NU values a thread,
// and read and written once; a team takes one row at a time, other teams hide its
// latency.  What bounds it: memory (h and y in, h' and u out): 65536 x 2048 in
// 276 us, 5.8 TB/s of the 6.46 that a copy reaches.  Few rows are bound by the
// latency of one (17 x 1024: 3.3 us), odd widths by the vectors of the channels,
// which are then read value by value (2999 x 1337: 19 us, 1.7 TB/s).
// A warp of the team takes 128 * NU neighbouring values, so that a thread's
// addresses differ by constants:
//   kUnits    lane i holds the 4-value units i, i + 32, ...: 16 bytes of f32 or 8 of bf16
//   kShifted  the same for a width or a row stride that is no multiple of 4: the units lie where the addresses are
//             aligned, and those that the row has only a part of, at its ends, are read and written value by value
//   kValues   lane i holds the values i, i + 32, ...: any alignment
// Mean and variance are sums over the registers, the second of squared deviations
// from the first: no cancellation when the mean is large.
enum RowLayout { kUnits, kShifted, kValues };

template <RowLayout LAYOUT, int NU>
struct RowTeam {
  static constexpr bool VEC = LAYOUT != kValues;
  static constexpr int N = 4 * NU;
  int first, left;   // first value of this thread; values of the row from there on
  int warp, warps, bar;
  float* red;        // two times a float per warp of the team
  int which;         // of the two, in turn

  __device__ __forceinline__ static constexpr int offset(int e) {   // of value e from the first
    return VEC ? (e >> 2) * 128 + (e & 3) : e * 32;
  }
  __device__ __forceinline__ bool there(int e) const {
    return offset(e) < left && (LAYOUT != kShifted || first + offset(e) >= 0);
  }
  // the unit of value e, a multiple of 4: all in the row, or at least a part of it
  __device__ __forceinline__ bool whole(int e) const { return LAYOUT != kShifted ? there(e) : there(e) && there(e + 3); }
  __device__ __forceinline__ bool some(int e) const { return offset(e) < left && first + offset(e) > -4; }

  __device__ __forceinline__ void load(const void* p, long long base, int f32, float (&v)[N]) const {
    if (VEC) {
      if (f32) {
        const float* q = static_cast<const float*>(p) + base + first;
#pragma unroll
        for (int c = 0; c < N; c += 4) {
          float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
          if (whole(c)) {
            f = load_f32x4(q + offset(c));
          } else if (LAYOUT == kShifted && some(c)) {
            f.x = there(c) ? q[offset(c)] : 0.f, f.y = there(c + 1) ? q[offset(c + 1)] : 0.f;
            f.z = there(c + 2) ? q[offset(c + 2)] : 0.f, f.w = there(c + 3) ? q[offset(c + 3)] : 0.f;
          }
          v[c] = f.x, v[c + 1] = f.y, v[c + 2] = f.z, v[c + 3] = f.w;
        }
      } else {
        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + base + first;
        uint2 w[NU];
#pragma unroll
        for (int c = 0; c < N; c += 4) {
          w[c >> 2] = make_uint2(0, 0);
          if (whole(c)) {
            w[c >> 2] = load_b16x4(q + offset(c));
          } else if (LAYOUT == kShifted && some(c)) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              b[e] = there(c + e) ? (uint32_t)reinterpret_cast<const unsigned short*>(q)[offset(c + e)] : 0u;
            w[c >> 2] = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
          }
        }
#pragma unroll
        for (int c = 0; c < N; c += 4) {
          const float4 f = bf16x4_to_f32(w[c >> 2]);
          v[c] = f.x, v[c + 1] = f.y, v[c + 2] = f.z, v[c + 3] = f.w;
        }
      }
    } else if (f32) {
      const float* q = static_cast<const float*>(p) + base + first;
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = there(e) ? q[offset(e)] : 0.f;
    } else {
      const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p) + base + first;
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = there(e) ? __bfloat162float(q[offset(e)]) : 0.f;
    }
  }

  __device__ __forceinline__ void store(void* p, long long base, int f32, const float (&v)[N]) const {
    if (f32) {
      float* q = static_cast<float*>(p) + base + first;
#pragma unroll
      for (int e = 0; e < N; e += VEC ? 4 : 1) {
        if (VEC && whole(e)) {
          *reinterpret_cast<float4*>(q + offset(e)) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
        } else if (LAYOUT != kUnits) {
#pragma unroll
          for (int k = 0; k < (VEC ? 4 : 1); ++k)
            if (there(e + k)) q[offset(e + k)] = v[e + k];
        }
      }
    } else {
      __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p) + base + first;
#pragma unroll
      for (int e = 0; e < N; e += VEC ? 4 : 1) {
        if (VEC && whole(e)) {
          *reinterpret_cast<uint2*>(q + offset(e)) = make_uint2(pack_bf16x2(v[e], v[e + 1]), pack_bf16x2(v[e + 2], v[e + 3]));
        } else if (LAYOUT != kUnits) {
#pragma unroll
          for (int k = 0; k < (VEC ? 4 : 1); ++k)
            if (there(e + k)) q[offset(e + k)] = __float2bfloat16_rn(v[e + k]);
        }
      }
    }
  }

  // v = v * (one + a) + b with per-channel f32 vectors (NULL: one = 0, a = 1; b = 0)
  __device__ __forceinline__ void affine(float (&v)[N], const float* a, const float* b, float one) const {
    constexpr int STEP = LAYOUT == kUnits ? 4 : 1;
    if (a != nullptr) {
#pragma unroll
      for (int e = 0; e < N; e += STEP) {
        if (!there(e)) continue;
        if (STEP == 4) {
          const float4 f = *reinterpret_cast<const float4*>(a + first + offset(e));
          v[e] *= one + f.x, v[e + 1] *= one + f.y, v[e + 2] *= one + f.z, v[e + 3] *= one + f.w;
        } else {
          v[e] *= one + a[first + offset(e)];
        }
      }
    }
    if (b != nullptr) {
#pragma unroll
      for (int e = 0; e < N; e += STEP) {
        if (!there(e)) continue;
        if (STEP == 4) {
          const float4 f = *reinterpret_cast<const float4*>(b + first + offset(e));
          v[e] += f.x, v[e + 1] += f.y, v[e + 2] += f.z, v[e + 3] += f.w;
        } else {
          v[e] += b[first + offset(e)];
        }
      }
    }
  }

  // The team's sum, the same bits in every thread.
  __device__ __forceinline__ float total(float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
    if (warps > 1) {
      float* r = red + which * warps;
      which ^= 1;   // so that one barrier is enough: the sum before last has been read
      if ((threadIdx.x & 31) == 0) r[warp] = s;
      named_bar_sync(bar, 32 * warps);
      s = r[0];
      for (int i = 1; i < warps; ++i) s += r[i];
    }
    return s;
  }

  __device__ __forceinline__ void norm(float (&v)[N], int kind, const float* gain, const float* bias, float eps, float dim) {
    if (kind == GDIT_NORM_NONE) return;
    float mean = 0.f, s = 0.f;
    if (kind == GDIT_NORM_LAYER) {
#pragma unroll
      for (int e = 0; e < N; ++e) s += v[e];   // 0 behind the row's end
      mean = total(s) / dim;
      s = 0.f;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      v[e] -= mean;
      if (there(e)) s = fmaf(v[e], v[e], s);
    }
    const float rs = rsqrtf(total(s) / dim + eps);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] *= rs;
    affine(v, gain, bias, 0.f);
  }
};

constexpr int kNormThreads = 512;   // most threads of a row's team

// THREADS: most of a CTA, 256 or, for rows that need a wider team, 512.  As many CTAs an
// SM as the registers of h, y and their addresses allow (2, 3 or 4; of all forms only the one
// value by value with 24 a thread spills, 8 bytes): with all the registers the compiler
// likes, 2999 x 1337 took 24 us instead of 20.
template <RowLayout LAYOUT, int NU, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > 256 ? 1 : NU == 8 ? 2 : NU == 6 ? 3 : 4) norm_kernel(const NormArgs a, int warps, int teams) {
  __shared__ float red[kNormThreads / 32 * 2];
  const int which = threadIdx.x / (32 * warps);
  RowTeam<LAYOUT, NU> T;
  T.warps = warps;
  T.warp = (threadIdx.x >> 5) - which * warps;
  T.first = T.warp * 128 * NU + (threadIdx.x & 31) * (T.VEC ? 4 : 1);
  T.left = a.dim - T.first;
  T.bar = 1 + which;
  T.red = red + which * warps * 2;
  T.which = 0;
  const float dim = (float)a.dim;
  const int first = T.first;
  pdl_wait();
  pdl_launch_dependents();
  for (long long r = (long long)blockIdx.x * teams + which; r < a.rows; r += (long long)gridDim.x * teams) {
    if (LAYOUT == kShifted) {
      T.first = first - (int)((r * a.ldh) & 3);
      T.left = a.dim - T.first;
    }
    float h[4 * NU], y[4 * NU];
    T.load(a.h, r * a.ldh, a.h_f32, h);
    if (a.y != nullptr) T.load(a.y, r * a.ldy, a.y_f32, y);
    long long g = a.row_group != nullptr ? a.row_group[r] : 0;
    const int groups = max(a.gate_groups, a.mod_groups);
    const bool bad = groups > 1 && (g < 0 || (a.gate_groups > 1 && g >= a.gate_groups) ||
                                    (a.mod_groups > 1 && g >= a.mod_groups));
    if (bad) {
      g = 0;
      if (first == 0) atomicOr(&g_op_status, OP_ERR_GROUP);
    }
    const long long go = a.gate_groups > 1 ? g * a.dim : 0, mo = a.mod_groups > 1 ? g * a.dim : 0;
    if (a.y != nullptr) {
      T.norm(y, a.post, a.post_gain, a.post_bias, a.eps, dim);
      T.affine(y, a.gate != nullptr ? a.gate + go : nullptr, nullptr, 0.f);
    }
#pragma unroll
    for (int e = 0; e < 4 * NU; ++e) {
      h[e] = a.y != nullptr ? fmaf(a.residual_scale, h[e], y[e]) : a.residual_scale * h[e];
      if (!T.there(e)) h[e] = 0.f;
      if (bad) h[e] = __int_as_float(0x7fffffff);
    }
    if (a.out_h != nullptr) T.store(a.out_h, r * a.ldoh, a.h_f32, h);
    if (a.out_u != nullptr) {
      T.norm(h, a.pre, a.pre_gain, a.pre_bias, a.eps, dim);
      T.affine(h, a.scale != nullptr ? a.scale + mo : nullptr, a.shift != nullptr ? a.shift + mo : nullptr, 1.f);
      T.store(a.out_u, r * a.ldou, a.u_f32, h);
    }
  }
}

inline void launch_norm(const NormArgs& a, int sms, cudaStream_t s) {
  auto aligned = [&](const void* p, long long ld, int f32) {   // rows that units of 4 values fit, all shifted alike
    return p == nullptr || ((uintptr_t)p % (f32 ? 16 : 8) == 0 && (ld - a.ldh) % 4 == 0);
  };
  const int shift = a.ldh % 4 != 0 ? 3 : 0;   // values that a row's first unit may begin in front of it, at most
  const bool units = aligned(a.h, a.ldh, a.h_f32) && aligned(a.y, a.ldy, a.y_f32) &&
                     aligned(a.out_h, a.ldoh, a.h_f32) && aligned(a.out_u, a.ldou, a.u_f32) &&
                     a.dim + shift <= 32 * kNormThreads;   // (and with the shift the widest team holds them)
  bool vec = units && a.dim % 4 == 0 && shift == 0;
  for (const float* p : {a.post_gain, a.post_bias, a.gate, a.pre_gain, a.pre_bias, a.scale, a.shift})
    vec = vec && ((uintptr_t)p & 15u) == 0;
  const int width = a.dim + (units ? shift : 0);   // with what the shift may add in front
  // Warps of a row: as few as hold it with 32 values a thread, so that a row of
  // up to 1024 needs no barrier; more where the rows would leave an SM fewer than 32
  // (4352 x 1024: 14 us in two warps a row, 20 in one, 19 in four).  Above 8 warps a thread
  // holds 32 values all the same: where 3, 5, 6 or 7 warps were doubled past 8, those that
  // the row does not need only join the barriers.
  int warps = (width + 1023) / 1024;
  while (a.rows * warps < 32ll * sms && 128 * warps < width && warps < 8) warps *= 2;
  const int per = (width + 128 * warps - 1) / (128 * warps);   // units of 4 values a thread
  const int teams = std::max(1, 8 / warps);
  const dim3 grid((unsigned)std::min<long long>((a.rows + teams - 1) / teams, INT32_MAX)), block(32 * warps * teams);
  auto launch = [&](auto kern) { launch_op(s, 1, kern, grid, block, 0, a, warps, teams); };
  auto pick = [&](auto layout) {
    constexpr RowLayout V = decltype(layout)::value;
    if (warps > 8) launch(norm_kernel<V, 8, 512>);
    else if (per == 1) launch(norm_kernel<V, 1, 256>);
    else if (per == 2) launch(norm_kernel<V, 2, 256>);
    else if (per <= 4) launch(norm_kernel<V, 4, 256>);
    else if (per <= 6) launch(norm_kernel<V, 6, 256>);
    else launch(norm_kernel<V, 8, 256>);
  };
  if (vec) pick(std::integral_constant<RowLayout, kUnits>());
  else if (units) pick(std::integral_constant<RowLayout, kShifted>());
  else pick(std::integral_constant<RowLayout, kValues>());
}

}  // namespace gdit
