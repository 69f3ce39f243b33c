// gdit_linear: out[m, n] = act(sum_k x[m, k] w[n, k] + bias[n]) + residual[m, n].
//
// Two kernels, both tcgen05.mma bf16 with f32 accumulators in TMEM, fed by TMA
// boxes of 64 values of K (128-byte swizzle):
//   linear_pair_kernel   256 x BN tiles on pairs of CTAs, persistent: the
//                        epilogue of a tile runs under the products of the next
//   linear_split_kernel  128 x BN tiles, K cut over the CTAs of a cluster, which
//                        add their partial tiles through distributed shared
//                        memory: few rows or few tiles
// 16384 x 8192 x 2048 with GELU: 437 us, 1.26 PFLOP/s of 1.63 measured (of 1.38
// under the power limit, which holds this size to 1.6 GHz).  Middle sizes are bound by
// what the SMs load from L2, about 51 bytes a cycle each, and the epilogue of their one
// or two tiles (1237 x 2056 x 1096: 17 us); one token by latency (4.3 us).
#pragma once

#include <atomic>
#include <type_traits>

#include "gemm_tc.cuh"
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
  int tma;   // pair kernel: TMA addresses out and residual
};

// Activations in f32.  v0 and v1 by 1 / (1 + 2^-a) of theirs, with one reciprocal for
// both: of the product, times the other's denominator (the special function unit is
// what such an epilogue waits for: 16 results a cycle).  So that the product stays
// finite, powers are cut at 2^62, and above that the factor is 0.  Good to a few 2^-22
// of the value otherwise.
__device__ __forceinline__ void sigmoid_times2(float& v0, float& v1, float a0, float a1) {
  const float d0 = 1.f + ex2(fminf(-a0, 62.f)), d1 = 1.f + ex2(fminf(-a1, 62.f));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d0 * d1));
  v0 *= -a0 > 62.f ? 0.f : r * d1;
  v1 *= -a1 > 62.f ? 0.f : r * d0;
}

// v Phi(v) = max(v, 0) - |v| Phi(-|v|), with Phi(-a) = 2^L(a): the logarithm is smooth, so that a polynomial in it is
// good relative to the tail's small values, where 1 + erf would cancel, and one exponential is all that the special
// function unit has to do.  L by a fit of least maximum error on [0, 13.2], weighted: 2^-21 up to a = 1, 2^-17 at 5,
// 2^-12 at 10, 2^-11 at 13, where 2^L leaves the range of f32 (beyond, 0).
__device__ __forceinline__ void gelu2(float& v0, float& v1) {
  const float a0 = fminf(fabsf(v0), 13.2f), a1 = fminf(fabsf(v1), 13.2f);
  const uint64_t a = f2_pack(a0, a1);
  uint64_t l = f2_splat(-1.46768685e-11f);
  l = f2_fma(l, a, f2_splat(1.05980167e-9f));
  l = f2_fma(l, a, f2_splat(-3.32314526e-8f));
  l = f2_fma(l, a, f2_splat(5.91531819e-7f));
  l = f2_fma(l, a, f2_splat(-6.51040364e-6f));
  l = f2_fma(l, a, f2_splat(4.40518648e-5f));
  l = f2_fma(l, a, f2_splat(-1.47657455e-4f));
  l = f2_fma(l, a, f2_splat(-3.19504992e-4f));
  l = f2_fma(l, a, f2_splat(7.40393086e-3f));
  l = f2_fma(l, a, f2_splat(-5.28077180e-2f));
  l = f2_fma(l, a, f2_splat(-4.59074565e-1f));
  l = f2_fma(l, a, f2_splat(-1.15112649f));
  l = f2_fma(l, a, f2_splat(-0.999999447f));
  float l0, l1, t0, t1;
  f2_unpack(l, l0, l1);
  f2_unpack(f2_mul(f2_pack(v0, v1), f2_splat(0.5f)), t0, t1);   // max(v, 0) = v / 2 + |v / 2|, where NaN stays NaN
  v0 = fmaf(-a0, ex2(l0), t0 + fabsf(t0));
  v1 = fmaf(-a1, ex2(l1), t1 + fabsf(t1));
}

template <int N>
__device__ __forceinline__ void apply_act(int act, float (&v)[N]) {
  if (act == GDIT_ACT_RELU) {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = v[j] < 0.f ? 0.f : v[j];   // NaN stays NaN
  } else if (act == GDIT_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < N; j += 2) gelu2(v[j], v[j + 1]);
  } else if (act == GDIT_ACT_GELU_TANH) {
#pragma unroll
    for (int j = 0; j < N; j += 2) {   // 2 sqrt(2 / pi) log2(e) (v + 0.044715 v^3)
      constexpr float c = 2.3022081985104166f;
      sigmoid_times2(v[j], v[j + 1], c * fmaf(0.044715f * v[j] * v[j], v[j], v[j]),
                     c * fmaf(0.044715f * v[j + 1] * v[j + 1], v[j + 1], v[j + 1]));
    }
  } else if (act == GDIT_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < N; j += 2)
      sigmoid_times2(v[j], v[j + 1], 1.4426950408889634f * v[j], 1.4426950408889634f * v[j + 1]);
  }
}

// ------------------------------------------------------------------ CTA pairs
//
// One thread of the even CTA issues the MMAs of both (cta_group::2, 256 x BN x
// 16): each CTA loads its 128 rows of x and half of the tile's rows of w, and
// holds its 128 rows of the accumulator.  Eight epilogue warps a CTA, two per
// 32-lane TMEM quarter, each working through 32-row boxes of 128 bytes of
// output: TMEM -> bias, activation -> residual (brought into the box by TMA
// beforehand) -> box -> TMA store.  The boxes of a warp alternate, so that the
// next residual is on its way while one is used.

constexpr int kLinEpiWarps = 8;
constexpr int kLinThreads = 64 + 32 * kLinEpiWarps;

template <int BN>
struct LinPairCfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = BN / 2 * 128;
  static constexpr int STAGE = A_BYTES + B_BYTES;   // per CTA
  static constexpr int BOXES = kLinEpiWarps * 2 * 4096;
  static constexpr int STAGES = (227 * 1024 - 1024 - BOXES - 512) / STAGE;
  static constexpr int SMEM = 1024 + STAGES * STAGE + BOXES + 512;
  static_assert((2 * STAGES + 4 + 2 * kLinEpiWarps) * 8 + 64 <= 512, "barriers");
};

// Tile t: 256-row block and column tile, row blocks in groups of 8 so that
// neighbouring tiles share rows of x and of w in L2.
__device__ __forceinline__ void lin_pair_tile(int t, int mt, int nt, int& mi, int& ni) {
  const int gs = 8 * nt, g = t / gs, first = g * 8, gm = min(mt - first, 8), r = t - g * gs;
  mi = first + r % gm;
  ni = r / gm;
}

// A warp's box of 32 rows x 128 bytes (128-byte swizzle), from and to a matrix that TMA
// cannot address: rows from `row`, columns from n, a word a lane.  Reads behind the
// matrix' edges are moved onto it (what they give is not stored): a branch around each
// of them costs more than the reads.
__device__ __forceinline__ uint32_t* box_word(uint8_t* box, int r) {
  const int lane = threadIdx.x & 31;
  return reinterpret_cast<uint32_t*>(box + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) + (lane & 3) * 4);
}

__device__ __forceinline__ void box_from(uint8_t* box, const void* p, long long ld, int f32, long long row, long long m,
                                         int n, int cols) {
  const int lane = threadIdx.x & 31, c = n + (f32 ? lane : 2 * lane);
  const int c0 = min(c, cols - 1), c1 = min(c + 1, cols - 1);
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 16) {
    uint32_t v[16];
    if (f32) {
#pragma unroll
      for (int r = 0; r < 16; ++r) v[r] = static_cast<const uint32_t*>(p)[min(row + r0 + r, m - 1) * ld + c0];
    } else {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const unsigned short* q = static_cast<const unsigned short*>(p) + min(row + r0 + r, m - 1) * ld;
        v[r] = q[c0] | (uint32_t)q[c1] << 16;
      }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) *box_word(box, r0 + r) = v[r];
  }
}

__device__ __forceinline__ void box_to(uint8_t* box, void* p, long long ld, int f32, long long row, long long m, int n,
                                       int cols) {
  const int lane = threadIdx.x & 31, c = n + (f32 ? lane : 2 * lane);
  const int rows = (int)min((long long)32, m - row);
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
    const uint32_t v = *box_word(box, r);
    const long long at = (row + r) * ld + c;
    if (f32) {
      if (r < rows && c < cols) static_cast<uint32_t*>(p)[at] = v;
    } else {
      unsigned short* q = static_cast<unsigned short*>(p) + at;
      if (r < rows && c < cols) q[0] = (unsigned short)v;
      if (r < rows && c + 1 < cols) q[1] = (unsigned short)(v >> 16);
    }
  }
}

template <int BN>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                       const __grid_constant__ CUtensorMap tmR, const __grid_constant__ CUtensorMap tmO,
                       const LinearArgs a) {
  using Cfg = LinPairCfg<BN>;
  constexpr int STAGES = Cfg::STAGES;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int s_abort;
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  uint8_t* sA = smem;
  uint8_t* sB = sA + STAGES * Cfg::A_BYTES;
  uint8_t* sBox = sB + STAGES * Cfg::B_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(sBox + Cfg::BOXES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* rfull = tempty + 2;   // 2 a warp

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int b = 0; b < 2; ++b) mbar_init(&tfull[b], 1), mbar_init(&tempty[b], 2 * kLinEpiWarps);
    for (int i = 0; i < 2 * kLinEpiWarps; ++i) mbar_init(&rfull[i], 1);
    fence_mbar_init();
    s_abort = 0;
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmO);
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_holder, 2 * BN);
    tmem_relinquish_pair();
    tc_fence_before();
  }
  cluster_sync();   // both CTAs' barriers exist before either signals the other's
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  const uint32_t full_l = mapa_shared(&full[0], 0), tempty_l = mapa_shared(&tempty[0], 0);
  pdl_wait();
  pdl_launch_dependents();

  const int mt = (int)((a.m + 255) / 256), nt = (a.n + BN - 1) / BN, total = mt * nt;
  const int nkb = (a.k + 63) / 64;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  int mi, ni;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = cid; t < total && ok; t += ncl) {
        lin_pair_tile(t, mt, nt, mi, ni);
        const int xr = mi * 256 + (int)rank * 128, wr = ni * BN + (int)rank * (BN / 2);
        for (int kb = 0; kb < nkb; ++kb) {
          ok = op_wait(&empty[stage], phase ^ 1u, &s_abort);
          if (!ok) break;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * Cfg::STAGE);
          tma_load_2d_pair(sA + stage * Cfg::A_BYTES, &tmX, full_l + 8u * stage, kb * 64, xr);
          tma_load_2d_pair(sB + stage * Cfg::B_BYTES, &tmW, full_l + 8u * stage, kb * 64, wr);
          ++issued;
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
      }
      // every stage has been released by the MMAs' commits, so nothing is pending when the CTA exits
      const unsigned long long t0 = globaltimer_ns();
      for (int i = 0; i < min(issued, STAGES); ++i) {
        while (!mbar_try_wait(&empty[stage], phase ^ 1u) && globaltimer_ns() - t0 < 10000000ull) {
        }
        if (++stage == STAGES) stage = 0, phase ^= 1u;
      }
    }
  } else if (warp == 1) {
    if (leader) {
      const uint32_t acc = uniform(tmem), xa = desc_lo_k(uniform(smem_u32(sA))), wa = desc_lo_k(uniform(smem_u32(sB)));
      const uint32_t empty_u = uniform(smem_u32(empty)), tfull_u = uniform(smem_u32(tfull));
      uint32_t stage = 0, phase = 0;
      int it = 0;
      for (int t = cid; t < total; t += ncl, ++it) {
        const uint32_t buf = it & 1;
        op_wait_through(&tempty[buf], ((it >> 1) & 1) ^ 1u, &s_abort);
        tc_fence_after();
        for (int kb = 0; kb < nkb; ++kb) {
          op_wait_through(&full[stage], phase, &s_abort);
          tc_fence_after();
          const uint32_t xs = xa + stage * (Cfg::A_BYTES >> 4), ws = wa + stage * (Cfg::B_BYTES >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_pair_lo(acc + buf * BN, xs + 2 * k, ws + 2 * k, idesc_bf16_f32(256, BN), kb > 0 || k > 0);
            umma_commit_both_at(empty_u + 8 * stage);
            if (kb == nkb - 1) umma_commit_both_at(tfull_u + 8 * buf);
          }
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2, ew = warp - 2;
    uint8_t* boxes = sBox + ew * 2 * 4096;
    const bool bias_vec = ((uintptr_t)a.bias & 15u) == 0;
    uint64_t* rbar = rfull + 2 * ew;
    const int cols = a.out_f32 ? 32 : 64, chunks = BN / cols / 2;   // columns of a box, boxes of this warp in a tile
    const int sw = lane & 7;
    const bool res = a.residual != nullptr, res_tma = res && a.tma;
    // TMA clips a store at the matrix' last column in units of 16 bytes: where that lies inside a unit, it would write
    // what is beside the output, and the box over the last column is written by words
    const bool ragged = (a.n & (a.out_f32 ? 3 : 7)) != 0;
    int it = 0, seq = 0;
    for (int t = cid; t < total; t += ncl, ++it) {
      lin_pair_tile(t, mt, nt, mi, ni);
      const int buf = it & 1, ym = mi * 256 + (int)rank * 128 + q * 32, n0 = ni * BN + half * cols;
      auto fetch = [&](int s, int n) {   // residual box of chunk s
        if (lane == 0) {
          bulk_wait_read<0>();   // the store of chunk s - 2 has left the box
          mbar_arrive_expect_tx(&rbar[s & 1], 4096);
          tma_load_2d(boxes + (s & 1) * 4096, &tmR, &rbar[s & 1], n, ym);
        }
      };
      auto gather = [&](int s, int n) {   // residual box of chunk s, without TMA
        box_from(boxes + (s & 1) * 4096, a.residual, a.ldr, a.out_f32, ym, a.m, n, a.n);
      };
      if (res_tma) {
        fetch(seq, n0);
      } else if (res && ym < a.m) {
        for (int c = 0; c < min(2, chunks); ++c) gather(seq + c, n0 + c * 2 * cols);
      }
      op_wait_through(&tfull[buf], (it >> 1) & 1, &s_abort);
      tc_fence_after();
      const uint32_t acc = tmem + ((uint32_t)(q * 32) << 16) + buf * BN + half * cols;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c, ++seq) {
        const int n = n0 + c * 2 * cols;
        uint8_t* box = boxes + (seq & 1) * 4096;
        if (!a.tma) {
          __syncwarp();
        } else if (res) {
          op_wait_through(&rbar[seq & 1], (seq >> 1) & 1, &s_abort);
          if (c + 1 < chunks) fetch(seq + 1, n + 2 * cols);
          __syncwarp();
        } else {
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
        }
        uint8_t* brow = box + lane * 128;
        // 32 columns at a time, in a loop: the instructions of a tile's epilogue come from L2 the first time
#pragma unroll 1
        for (int x = 0; x < cols; x += 32) {
          float v[32];
          tmem_ld32(acc + c * 2 * cols + x, reinterpret_cast<uint32_t(&)[32]>(v));
          tmem_ld_wait();
          if (c == chunks - 1 && x == cols - 32) {   // the accumulator is in registers: the next products may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(tempty_l + 8u * buf);
          }
          const int nb = n + x;
          if (a.bias != nullptr) {   // the same addresses on all lanes
            if (bias_vec && nb + 32 <= a.n) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(a.bias + nb + j));
                v[j] += f.x, v[j + 1] += f.y, v[j + 2] += f.z, v[j + 3] += f.w;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += __ldg(a.bias + min(nb + j, a.n - 1));
            }
          }
          apply_act(a.act, v);
          if (a.out_f32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              float4* p = reinterpret_cast<float4*>(brow + ((j ^ sw) << 4));
              float4 o = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
              if (res) {
                const float4 r = *p;
                o.x += r.x, o.y += r.y, o.z += r.z, o.w += r.w;
              }
              *p = o;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint4* p = reinterpret_cast<uint4*>(brow + ((((x >> 3) + j) ^ sw) << 4));
              if (res) {
                const uint4 r = *p;
                const float4 r0 = bf16x4_to_f32(make_uint2(r.x, r.y)), r1 = bf16x4_to_f32(make_uint2(r.z, r.w));
                v[8 * j] += r0.x, v[8 * j + 1] += r0.y, v[8 * j + 2] += r0.z, v[8 * j + 3] += r0.w;
                v[8 * j + 4] += r1.x, v[8 * j + 5] += r1.y, v[8 * j + 6] += r1.z, v[8 * j + 7] += r1.w;
              }
              *p = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                              pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
            }
          }
        }
        const bool words = !a.tma || (ragged && n < a.n && n + cols > a.n);
        if (words) {
          __syncwarp();
          if (ym < a.m) box_to(box, a.out, a.ldo, a.out_f32, ym, a.m, n, a.n);
          __syncwarp();
          if (!a.tma) {
            if (res && ym < a.m && c + 2 < chunks) gather(seq + 2, n + 4 * cols);
            continue;
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (!words && n < a.n && ym < a.m) tma_store_2d(&tmO, box, n, ym);   // clipped at the matrix' edges
          bulk_commit();   // (a group a box, also without a store: the boxes are counted by them)
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
  }
  __syncthreads();
  if (threadIdx.x == 0) op_leave(&s_abort);
  __syncwarp();
  cluster_sync();   // neither CTA leaves while the other may still signal it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * BN);
  }
}

// ------------------------------------------------------------------ split K over a cluster
//
// The CTAs of a cluster share one 128 x BN tile and take a part of K each.
// Every CTA puts its partial tile into its own shared memory (f32, over the
// spent stages); CTA r then adds the rows r, r + S, ... of all S partial tiles
// in the order of the parts, so the result does not depend on timing, and
// writes them with neighbouring columns on neighbouring lanes, by fours where
// alignment and width allow.
// Rows of x that a tile does not have are not loaded: boxes of `xrows` rows; the
// MMA reads whatever the shared memory behind them holds into accumulator rows
// that nobody reads.

constexpr int kSplitThreads = 256;
constexpr int kSplitSmem = 226 * 1024;   // at most: the kernel has some bytes of its own

struct SplitPlan {
  double time;   // microseconds
  int bn, splits, stages, xrows;
  int smem() const { return 1024 + std::max(stages * (xrows + bn) * 128 + (128 - xrows) * 128, 128 * bn * 4) + 512; }
};

template <int BN>
__global__ void __launch_bounds__(kSplitThreads, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                        const LinearArgs a, int splits, int stages, int xrows, int smem_bytes) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int s_abort;
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  const int xbytes = xrows * 128, wbytes = BN * 128;
  uint8_t* sA = smem;
  uint8_t* sB = sA + stages * xbytes;
  float* part = reinterpret_cast<float*>(smem);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + smem_bytes - 1024 - 512);
  uint64_t* empty = full + stages;
  uint64_t* done = empty + stages;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % splits;
  const long long tile = blockIdx.x / splits;
  const int nt = (a.n + BN - 1) / BN;
  const long long m0 = tile / nt * 128;
  const int n0 = (int)(tile % nt) * BN;
  const int nkb = (a.k + 63) / 64;
  const int kb0 = (int)((long long)rank * nkb / splits), kb1 = (int)((long long)(rank + 1) * nkb / splits);
  if (threadIdx.x == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    mbar_init(done, 1);
    fence_mbar_init();
    s_abort = 0;
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, BN);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  pdl_wait();
  pdl_launch_dependents();

  if (warp == 0 && lane == 0) {
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!op_wait(&empty[stage], phase ^ 1u, &s_abort)) break;
      mbar_arrive_expect_tx(&full[stage], xbytes + wbytes);
      tma_load_2d(sB + stage * wbytes, &tmW, &full[stage], kb * 64, n0);
      tma_load_2d(sA + stage * xbytes, &tmX, &full[stage], kb * 64, (int)m0);
      if (++stage == stages) stage = 0, phase ^= 1u;
    }
  } else if (warp == 1) {
    const uint32_t acc = uniform(tmem), xa = desc_lo_k(uniform(smem_u32(sA))), wa = desc_lo_k(uniform(smem_u32(sB)));
    const uint32_t empty_u = uniform(smem_u32(empty)), done_u = uniform(smem_u32(done));
    uint32_t stage = 0, phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      op_wait_through(&full[stage], phase, &s_abort);
      tc_fence_after();
      const uint32_t xs = xa + stage * (xbytes >> 4), ws = wa + stage * (wbytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_bf16_lo(acc, xs + 2 * k, ws + 2 * k, idesc_bf16_f32(128, BN), kb > kb0 || k > 0);
        umma_commit_at(kb == kb1 - 1 ? done_u : empty_u + 8 * stage);
      }
      if (++stage == stages) stage = 0, phase ^= 1u;
    }
  }
  __syncwarp();
  // the products are complete, so every load has landed and every stage has been read
  op_wait_through(done, 0, &s_abort);
  __syncthreads();
  const bool ok = !s_abort;
  tc_fence_after();
  const int rows = (int)min((long long)128, a.m - m0);
  const int q = warp & 3;
  if (ok && q * 32 < rows) {
    const int row = q * 32 + lane;
#pragma unroll 1
    for (int c = (warp >> 2) * 32; c < BN; c += 64) {
      uint32_t r[32];
      tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + c, r);
      tmem_ld_wait();
      if (row < rows) {
#pragma unroll
        for (int j = 0; j < 8; ++j)   // 16-byte pieces of a row in an order of its own: no bank conflicts
          *reinterpret_cast<uint4*>(part + row * BN + ((((c >> 2) + j) ^ (row & 7)) << 2)) =
              make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // given back before the CTAs of the cluster wait for one another: one of them may
  // still be waiting for TMEM that another kernel on its SM holds
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, BN);
  }
  if (splits > 1) cluster_sync();
  if (ok) {
    // lane: 4 columns of a row, BN / 4 lanes a row; its rows are `stride` apart
    constexpr int LANES = BN / 4, PER = 32 / LANES;
    const int col = (lane % LANES) * 4, n = n0 + col, left = a.n - n;   // columns from here on
    const int stride = 8 * PER * splits;
    const int es = a.out_f32 ? 4 : 2;
    // by fours: the tile's columns are all there, rows begin at multiples of four
    const bool vec = n0 + BN <= a.n && ((uintptr_t)a.out % (4 * es) == 0) && a.ldo % 4 == 0 &&
                     (a.residual == nullptr || ((uintptr_t)a.residual % (4 * es) == 0 && a.ldr % 4 == 0));
    int at_col[4];   // (columns behind the last are read as the last and not written: no branches around the reads)
    float bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) at_col[e] = min(n + e, a.n - 1);
#pragma unroll
    for (int e = 0; e < 4; ++e) bias[e] = a.bias != nullptr ? __ldg(a.bias + at_col[e]) : 0.f;
    // R rows at a time: four of a whole tile, so that their reads are under way together; one where the CTAs of a
    // cluster share few rows, since four times the instructions would have to be fetched
    auto write_rows = [&](auto count) {
      constexpr int R = decltype(count)::value;
#pragma unroll 1
      for (int r0 = rank + splits * (warp * PER + lane / LANES); r0 < rows; r0 += R * stride) {
        float v[R][4], res[R][4];
        if (a.residual != nullptr) {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const long long row = (m0 + min(r0 + i * stride, rows - 1)) * a.ldr;
            if (a.out_f32) {
              const float* p = static_cast<const float*>(a.residual) + row;
              if (vec) {
                *reinterpret_cast<float4*>(res[i]) = *reinterpret_cast<const float4*>(p + n);
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) res[i][e] = p[at_col[e]];
              }
            } else {
              const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.residual) + row;
              if (vec) {
                *reinterpret_cast<float4*>(res[i]) = bf16x4_to_f32(*reinterpret_cast<const uint2*>(p + n));
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) res[i][e] = __bfloat162float(p[at_col[e]]);
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int row = min(r0 + i * stride, rows - 1);
          const uint32_t at = smem_u32(part) + (uint32_t)(row * BN + (((col >> 2) ^ (row & 7)) << 2)) * 4u;
          if (R > 1) {
            *reinterpret_cast<float4*>(v[i]) = ld_shared_f4(at);
          } else {
            float4 f[8];
#pragma unroll
            for (int s = 0; s < 8; ++s)
              if (s < splits) f[s] = ld_cluster_f4(mapa_shared_at(at, s));
            *reinterpret_cast<float4*>(v[i]) = f[0];
#pragma unroll
            for (int s = 1; s < 8; ++s)
              if (s < splits) v[i][0] += f[s].x, v[i][1] += f[s].y, v[i][2] += f[s].z, v[i][3] += f[s].w;
          }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[i][e] += bias[e];
          apply_act(a.act, v[i]);
          if (a.residual != nullptr) {
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i][e] += res[i][e];
          }
          const int row = r0 + i * stride;
          const long long at = (m0 + row) * a.ldo + n;
          if (a.out_f32) {
            float* p = static_cast<float*>(a.out) + at;
            if (vec) {
              if (row < rows) *reinterpret_cast<float4*>(p) = *reinterpret_cast<const float4*>(v[i]);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (row < rows && e < left) p[e] = v[i][e];
            }
          } else {
            __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.out) + at;
            if (vec) {
              if (row < rows)
                *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (row < rows && e < left) p[e] = __float2bfloat16_rn(v[i][e]);
            }
          }
        }
      }
    };
    if (splits == 1) write_rows(std::integral_constant<int, 4>());
    else write_rows(std::integral_constant<int, 1>());
  }
  if (threadIdx.x == 0) op_leave(&s_abort);
  if (splits > 1) {
    __syncwarp();
    cluster_sync();   // nobody leaves while its partial tile is read
  }
}

// ------------------------------------------------------------------ planning and launches

// [rows, cols] of the output type, boxes of 32 rows x 128 bytes, 128-byte swizzle.
inline CUtensorMap make_box_tmap(const void* p, int f32, long long rows, long long cols, long long ld) {
  CUtensorMap m;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(ld * (f32 ? 4 : 2))};
  cuuint32_t box[2] = {f32 ? 32u : 64u, 32u};
  cuuint32_t estr[2] = {1u, 1u};
  CUresult r = encode_fn()(&m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                           const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) throw GditError(GDIT_ECUDA, fmt("cuTensorMapEncodeTiled (output) failed (%d)", (int)r));
  return m;
}

template <int BN>
void launch_linear_pair(const LinearArgs& a, int sms, cudaStream_t s) {
  using Cfg = LinPairCfg<BN>;
  const CUtensorMap tx = make_tmap(a.x, a.m, a.k, a.ldx, 128), tw = make_tmap(a.w, a.n, a.k, a.ldw, BN / 2);
  // (without TMA for the output the maps are not used, but they have to be valid)
  const CUtensorMap to = a.tma ? make_box_tmap(a.out, a.out_f32, a.m, a.n, a.ldo) : tx;
  const CUtensorMap tr = a.tma && a.residual != nullptr ? make_box_tmap(a.residual, a.out_f32, a.m, a.n, a.ldr) : to;
  const long long tiles = (a.m + 255) / 256 * ((a.n + BN - 1) / BN);
  REQUIRE(tiles <= INT32_MAX / 2, "m %lld x n %d has too many tiles", a.m, a.n);
  allow_smem(linear_pair_kernel<BN>, Cfg::SMEM);
  launch_op(s, 2, linear_pair_kernel<BN>, dim3((unsigned)(2 * std::min<long long>(tiles, sms / 2))), dim3(kLinThreads),
            Cfg::SMEM, tx, tw, tr, to, a);
}

template <int BN>
void launch_linear_split(const LinearArgs& a, const SplitPlan& p, cudaStream_t s) {
  const CUtensorMap tx = make_tmap(a.x, a.m, a.k, a.ldx, p.xrows), tw = make_tmap(a.w, a.n, a.k, a.ldw, BN);
  const long long tiles = (a.m + 127) / 128 * ((a.n + BN - 1) / BN);
  REQUIRE(tiles * p.splits <= INT32_MAX, "m %lld x n %d has too many tiles", a.m, a.n);
  allow_smem(linear_split_kernel<BN>, kSplitSmem);
  launch_op(s, p.splits, linear_split_kernel<BN>, dim3((unsigned)(tiles * p.splits)), dim3(kSplitThreads), p.smem(), tx,
            tw, a, p.splits, p.stages, p.xrows, p.smem());
}

// CTAs in clusters of 1 to 8 that the current device holds with one an SM, asked once.
struct SplitSlots {
  int of[9];
};
inline const SplitSlots& split_slots(int sms) {
  static std::mutex mu;
  static std::atomic<const SplitSlots*> known[kMaxDevices];
  int dev = 0;
  CUDA_TRY(cudaGetDevice(&dev));
  const SplitSlots* p = known[dev].load(std::memory_order_acquire);
  if (p == nullptr) {
    std::lock_guard<std::mutex> lock(mu);
    p = known[dev].load(std::memory_order_relaxed);
    if (p == nullptr) {
      SplitSlots s = {{0, sms}};
      for (int n = 2; n <= 8; ++n) s.of[n] = n * max_clusters(linear_split_kernel<128>, n, kSplitThreads, kSplitSmem);
      p = new SplitSlots(s);
      known[dev].store(p, std::memory_order_release);
    }
  }
  return *p;
}

// Which kernel, tile width and parts of K: those with the shortest time by this and
// pair_time.  The coefficients fit the times of 80 sizes (1 to 16384 rows, 16 to 8192
// columns, K of 32 to 8192, aligned and odd) in up to 23 plans each; the plan chosen took
// 3 % longer than the best one on average, 24 % at most.
inline SplitPlan plan_split(long long m, int n, int k, const SplitSlots& slots) {
  SplitPlan p = {};
  const int nkb = (k + 63) / 64;
  const long long mt = (m + 127) / 128;
  p.xrows = 8;
  while (p.xrows < 128 && p.xrows < m) p.xrows *= 2;
  // A CTA's own time (its start, its steps along K, the kilobytes it loads, its share of
  // the tile's rows to write), times the CTAs for each place, and the join.
  const int rows = (int)std::min<long long>(m, 128);
  for (int bn = 128; bn >= 32; bn /= 2)
    for (int s = 1; s <= 8 && (s == 1 || 2 * s <= nkb); ++s) {
      const int steps = (nkb + s - 1) / s;
      const double own = 1.63 + 0.120 * steps + 0.0063 * steps * (p.xrows + bn) / 8 + 4.6 * rows * bn / 16384 / s;
      const double places = (double)(mt * ((n + bn - 1) / bn) * s) / slots.of[s];
      const double time = own * std::max(1.0, places) + (s > 1 ? 0.89 + 0.096 * s : 0);
      if (p.bn == 0 || time < p.time) p.time = time, p.bn = bn, p.splits = s;
    }
  const long long ctas = mt * ((n + p.bn - 1) / p.bn) * p.splits;
  const int per = (nkb + p.splits - 1) / p.splits;
  const int budget = (ctas > slots.of[p.splits] ? 110 : 220) * 1024 - 2048 - (128 - p.xrows) * 128;   // two CTAs an SM, or one
  p.stages = std::max(2, std::min({per, 16, budget / ((p.xrows + p.bn) * 128)}));
  return p;
}

// The pair kernel's time in microseconds: rounds of tiles over the pairs, a step along K
// at what its loads take, and an epilogue that runs under the next tile's products.
inline double pair_time(const LinearArgs& a, int bn, int sms) {
  const long long tiles = (a.m + 255) / 256 * ((a.n + bn - 1) / bn), pairs = sms / 2;
  const double rounds = (double)((tiles + pairs - 1) / pairs), products = (a.k + 63) / 64 * 0.33 * (128 + bn / 2) / 256;
  const double epilogue = (a.tma ? 6.8 : 9.8) * bn / 256;
  return 1.2 + std::max(rounds * products + epilogue, rounds * std::max(products, epilogue));
}

struct LinearPlan {
  int pair_bn;       // tile width of the pair kernel, or 0 for the split kernel
  SplitPlan split;
};

// (sets a.tma, too)
inline LinearPlan plan_linear(LinearArgs& a, int sms, const SplitSlots& slots) {
  const int es = a.out_f32 ? 4 : 2;
  auto tma_ok = [&](const void* p, long long ld) { return ((uintptr_t)p & 15u) == 0 && ld * es % 16 == 0; };
  a.tma = tma_ok(a.out, a.ldo) && (a.residual == nullptr || tma_ok(a.residual, a.ldr));
  LinearPlan p = {0, plan_split(a.m, a.n, a.k, slots)};
  const double wide = pair_time(a, 256, sms), narrow = pair_time(a, 128, sms);
  if (std::min(wide, narrow) < p.split.time) p.pair_bn = wide < narrow ? 256 : 128;
  return p;
}

inline void launch_linear(LinearArgs& a, int sms, cudaStream_t s) {
  const LinearPlan p = plan_linear(a, sms, split_slots(sms));
  if (p.pair_bn == 256) launch_linear_pair<256>(a, sms, s);
  else if (p.pair_bn == 128) launch_linear_pair<128>(a, sms, s);
  else if (p.split.bn == 128) launch_linear_split<128>(a, p.split, s);
  else if (p.split.bn == 64) launch_linear_split<64>(a, p.split, s);
  else launch_linear_split<32>(a, p.split, s);
}

}  // namespace gdit
