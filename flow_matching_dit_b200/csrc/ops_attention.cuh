// gdit_attention: softmax attention over packed sequences with grouped heads.
#pragma once

#include "ops_common.cuh"

namespace gdit {

struct AttnArgs {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  __nv_bfloat16* out;
  float* lse;
  const int* cu_q;
  const int* cu_k;
  const int* k_len;
  long long total_q, total_k;
  long long q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;
  int batch, heads, kv_heads, dim;
  int max_q, max_k;
  int causal;
  float scale_log2;   // scale * log2(e)
};

// Sequence b: its queries [q0, q0 + nq) and keys [k0, k0 + nk).
struct Seq {
  int q0, nq, k0, nk;
};

// Reads and checks sequence b.  A sequence whose offsets decrease, leave the
// tensors or exceed max_q / max_k is not followed: ok is false.
__device__ __forceinline__ Seq read_seq(const AttnArgs& a, int b, bool& ok) {
  const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
  ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q && k0 >= 0 && k1 >= k0 && k1 <= a.total_k && q1 - q0 <= a.max_q;
  int nk = k1 - k0;
  if (a.k_len != nullptr) {
    const int n = a.k_len[b];
    ok = ok && n >= 0 && n <= nk;
    nk = n;
  }
  ok = ok && nk <= a.max_k;
  return {q0, q1 - q0, k0, nk};
}

// CTA 0 reports bad sequences, whether or not any tile looks at them.
__device__ __forceinline__ void report_bad_seqs(const AttnArgs& a, int tid, int nthreads) {
  bool bad = false;
  for (int b = tid; b < a.batch; b += nthreads) {
    bool ok;
    read_seq(a, b, ok);
    bad |= !ok;
  }
  if (bad) atomicOr(&g_op_status, OP_ERR_OFFSETS);
}

// One warp per (query, head), keys one after another, 4 values of the head a lane.
__global__ void __launch_bounds__(256) attention_simple_kernel(const AttnArgs a) {
  pdl_wait();
  if (blockIdx.x == 0) report_bad_seqs(a, threadIdx.x, blockDim.x);
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const long long t = item / a.heads;
  const int head = (int)(item - t * a.heads);
  if (t >= a.total_q) return;
  for (int b = 0; b < a.batch; ++b) {
    bool ok;
    const Seq s = read_seq(a, b, ok);
    if (!ok || t < s.q0 || t >= s.q0 + s.nq) continue;
    const int kvh = head / (a.heads / a.kv_heads);
    const int end = a.causal ? min(s.nk, (int)(t - s.q0) + s.nk - s.nq + 1) : s.nk;
    float q[4], o[4] = {}, top = -INFINITY, sum = 0.f;
    for (int i = 0; i < 4; ++i) {
      const int c = lane + 32 * i;
      q[i] = c < a.dim ? __bfloat162float(a.q[t * a.q_t + head * a.q_h + c]) * a.scale_log2 : 0.f;
    }
    for (int j = 0; j < end; ++j) {
      float d = 0.f;
      for (int i = 0; i < 4; ++i) {
        const int c = lane + 32 * i;
        if (c < a.dim) d = fmaf(q[i], __bfloat162float(a.k[(s.k0 + j) * a.k_t + kvh * a.k_h + c]), d);
      }
      for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(~0u, d, x);
      const float m = fmaxf(top, d), f = m == -INFINITY ? 1.f : exp2f(top - m), p = m == -INFINITY ? 0.f : exp2f(d - m);
      sum = sum * f + p;
      top = m;
      for (int i = 0; i < 4; ++i) {
        const int c = lane + 32 * i;
        if (c < a.dim) o[i] = o[i] * f + p * __bfloat162float(a.v[(s.k0 + j) * a.v_t + kvh * a.v_h + c]);
      }
    }
    for (int i = 0; i < 4; ++i) {
      const int c = lane + 32 * i;
      if (c < a.dim) a.out[t * a.o_t + head * a.o_h + c] = __float2bfloat16_rn(sum > 0.f ? o[i] / sum : sum == 0.f ? 0.f : sum);
    }
    if (a.lse != nullptr && lane == 0)
      a.lse[t * a.heads + head] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    return;
  }
}

inline void launch_attention(const AttnArgs& a, cudaStream_t s) {
  launch_op(s, 1, attention_simple_kernel, dim3((unsigned)((a.total_q * a.heads + 7) / 8)), dim3(256), 0, a);
}

}  // namespace gdit
