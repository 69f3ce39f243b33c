// gdit_linear: out[m, n] = act(sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n].
#pragma once

#include "ops_common.cuh"

namespace gdit {

struct LinearArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* w;
  const float* bias;
  const void* residual;
  void* out;
  long long m, ldx, ldw, ldr, ldo;
  int n, k;
  int out_f32;
  int act;
};

__device__ __forceinline__ float act_value(int act, float v) {
  switch (act) {
    case GDIT_ACT_RELU: return v < 0.f ? 0.f : v;   // NaN stays NaN
    case GDIT_ACT_GELU: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case GDIT_ACT_GELU_TANH: return 0.5f * v * (1.f + tanhf(0.79788456080286536f * (v + 0.044715f * v * v * v)));
    case GDIT_ACT_SILU: return v / (1.f + expf(-v));
    default: return v;
  }
}

// 64 x 64 outputs a CTA of 256 threads, 4 x 4 a thread, f32 multiply-adds.
__global__ void __launch_bounds__(256) linear_simple_kernel(const LinearArgs a) {
  __shared__ float sx[16][68], sw[16][68];
  pdl_wait();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long m0 = (long long)blockIdx.y * 64;
  const int n0 = blockIdx.x * 64;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < a.k; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int r = i >> 4, c = i & 15;
      const bool kok = k0 + c < a.k;
      sx[c][r] = kok && m0 + r < a.m ? __bfloat162float(a.x[(m0 + r) * a.ldx + k0 + c]) : 0.f;
      sw[c][r] = kok && n0 + r < a.n ? __bfloat162float(a.w[(long long)(n0 + r) * a.ldw + k0 + c]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 16; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sx[c][ty * 4 + i], sw[c][tx * 4 + j], acc[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i) {
    const long long m = m0 + ty * 4 + i;
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (m >= a.m || n >= a.n) continue;
      float v = act_value(a.act, acc[i][j] + (a.bias ? a.bias[n] : 0.f));
      if (a.out_f32) {
        if (a.residual) v += static_cast<const float*>(a.residual)[m * a.ldr + n];
        static_cast<float*>(a.out)[m * a.ldo + n] = v;
      } else {
        if (a.residual) v += __bfloat162float(static_cast<const __nv_bfloat16*>(a.residual)[m * a.ldr + n]);
        static_cast<__nv_bfloat16*>(a.out)[m * a.ldo + n] = __float2bfloat16_rn(v);
      }
    }
  }
}

inline void launch_linear(const LinearArgs& a, cudaStream_t s) {
  launch_op(s, 1, linear_simple_kernel, dim3((a.n + 63) / 64, (unsigned)((a.m + 63) / 64)), dim3(256), 0, a);
}

}  // namespace gdit
