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
  long long max_tiles;   // tiles of a key head that valid offsets can have at most
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

// ------------------------------------------------------------------ tensor-core kernel
//
// The queries of one key head are taken as packed rows r = position * group +
// head in the group, so that the heads that share keys share a tile: the keys
// are read once for all of them, and a causal tile of 256 rows spans only
// 256 / group positions.  A CTA works on tiles of 256 rows as two halves of
// 128, each with a softmax warpgroup of its own: while one half's scores are
// turned into probabilities, the tensor core multiplies for the other.
//
//   warp 0       K and V tiles of 128 keys by TMA into a ring of SLOTS tiles
//   warp 1       tcgen05.mma: S = Q K^T (f32, TMEM), O += P V (P from TMEM)
//   warps 2, 3   Q rows by cp.async; warp 3 also zeroes the rows of the last V tile that no row of the tile sees
//   warps 4-11   softmax of one half each: thread = row; P (bf16) overwrites S; O is rescaled only when the running maximum
//                has grown by more than 2^8 (the statistics refer to the maximum in use, so nothing is lost), and
//                divided by the sum at the end
//
// The tensor core executes in issue order P V (j), Q K^T (j + 1) of one half,
// then of the other, so a full S (j + 1) also says that O holds the blocks up
// to j.  Tiles are walked in a static order, the longest of a sequence first.

constexpr int kAtBM = 128;       // rows of a half
constexpr int kAtBN = 128;       // keys of a block
constexpr int kAtThreads = 384;

template <int DP>   // head_dim rounded up to 64 or 128
struct AttnCfg {
  static constexpr int BOX = kAtBN * 128;                    // bytes of a [128][64] box
  static constexpr int TILE = BOX * (DP / 64);
  static constexpr int SLOTS = DP == 128 ? 5 : 10;
  static constexpr int SMEM = 1024 + 2 * TILE + SLOTS * TILE + 256;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// A tile: rows [r0, r0 + rows) of sequence s and key head kvh, the first
// `blocks` key blocks, of which the keys below `end` are seen by some row.
struct AttnTile {
  Seq s;
  int r0, rows, kvh, end, blocks;
};

// Walks the tiles t, t + step, ... of the call: all lanes of a warp together.
// A group of 32 sequences at a time, lane i looks after sequence base + i.
struct TileWalk {
  int base;              // first sequence of the group
  long long before;      // tiles in front of it
  int incl;              // lane: tiles of the group up to and with this sequence
  int mine;
  Seq seq;

  __device__ __forceinline__ void load(const AttnArgs& a, int tile_rows) {
    const int lane = threadIdx.x & 31, b = base + lane;
    seq = {0, 0, 0, 0};
    mine = 0;
    if (b < a.batch) {
      bool ok;
      const Seq s = read_seq(a, b, ok);
      if (ok) {
        seq = s;
        mine = (int)(((long long)s.nq * (a.heads / a.kv_heads) + tile_rows - 1) / tile_rows);
      }
    }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(~0u, incl, o);
      if (lane >= o) incl += x;
    }
  }

  __device__ __forceinline__ void start(const AttnArgs& a, int tile_rows) {
    base = 0;
    before = 0;
    load(a, tile_rows);
  }

  // id = tile * kv_heads + key head; false behind the last tile
  __device__ __forceinline__ bool at(const AttnArgs& a, int tile_rows, long long id, AttnTile& t) {
    const int kvh = (int)(id % a.kv_heads);
    const long long n = id / a.kv_heads;
    if (n >= a.max_tiles) return false;
    while (true) {
      const int total = __shfl_sync(~0u, incl, 31);
      if (n < before + total) break;
      before += total;
      base += 32;
      if (base >= a.batch) return false;
      load(a, tile_rows);
    }
    const int rel = (int)(n - before);
    const int src = __popc(__ballot_sync(~0u, incl <= rel));
    t.s.q0 = __shfl_sync(~0u, seq.q0, src);
    t.s.nq = __shfl_sync(~0u, seq.nq, src);
    t.s.k0 = __shfl_sync(~0u, seq.k0, src);
    t.s.nk = __shfl_sync(~0u, seq.nk, src);
    const int last = __shfl_sync(~0u, incl, src) - 1 - rel;   // the last tile of a sequence first
    const int group = a.heads / a.kv_heads;
    t.kvh = kvh;
    t.r0 = last * tile_rows;
    t.rows = min(tile_rows, t.s.nq * group - t.r0);
    t.end = t.s.nk;
    if (a.causal) t.end = max(0, min(t.s.nk, (t.r0 + t.rows - 1) / group + t.s.nk - t.s.nq + 1));
    t.blocks = (t.end + kAtBN - 1) / kAtBN;
    return true;
  }
};

__device__ __forceinline__ void store_out_row(__nv_bfloat16* o, int vec, int c0, int dim, const float (&v)[32]) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < 32; j += 8)
      if (c0 + j < dim)
        *reinterpret_cast<uint4*>(o + c0 + j) =
            make_uint4(pack_bf16x2(v[j], v[j + 1]), pack_bf16x2(v[j + 2], v[j + 3]), pack_bf16x2(v[j + 4], v[j + 5]),
                       pack_bf16x2(v[j + 6], v[j + 7]));
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c0 + j < dim) o[c0 + j] = __float2bfloat16_rn(v[j]);
  }
}

template <int DP>
__global__ void __launch_bounds__(kAtThreads, 1)
    attention_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const AttnArgs a, int tile_rows, int out_vec) {
  using Cfg = AttnCfg<DP>;
  constexpr int SLOTS = Cfg::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int s_abort;
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  uint8_t* sQ = smem;                        // two halves
  uint8_t* sKV = smem + 2 * Cfg::TILE;       // ring
  uint64_t* full = reinterpret_cast<uint64_t*>(sKV + SLOTS * Cfg::TILE);
  uint64_t* empty = full + SLOTS;
  uint64_t* qfull = empty + SLOTS;
  uint64_t* qempty = qfull + 1;
  uint64_t* vfix = qempty + 1;
  uint64_t* vgo = vfix + 1;
  uint64_t* sfull = vgo + 1;                 // [2]
  uint64_t* pfull = sfull + 2;               // [2]
  uint64_t* ofull = pfull + 2;               // [2]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < SLOTS; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    mbar_init(qfull, 64);
    mbar_init(qempty, 1);
    mbar_init(vfix, 1);
    mbar_init(vgo, 1);
    for (int s = 0; s < 2; ++s) mbar_init(&sfull[s], 1), mbar_init(&pfull[s], 4), mbar_init(&ofull[s], 1);
    fence_mbar_init();
    s_abort = 0;
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  pdl_wait();
  pdl_launch_dependents();

  const int group = a.heads / a.kv_heads;
  const int ksteps = (a.dim + 15) / 16;
  TileWalk walk;
  AttnTile t;
  walk.start(a, tile_rows);

  if (warp == 0) {
    int slot = 0;
    uint32_t phase = 0;
    int issued = 0, nfix = 0;
    bool ok = true;
    for (long long id = blockIdx.x; walk.at(a, tile_rows, id, t) && ok; id += gridDim.x) {
      if (lane == 0) {
        for (int j = 0; j < 2 * t.blocks && ok; ++j) {
          ok = op_wait(&empty[slot], phase ^ 1u, &s_abort);
          if (!ok) break;
          uint8_t* dst = sKV + slot * Cfg::TILE;
          const CUtensorMap* map = (j & 1) ? &tmV : &tmK;
          const int boxes = a.dim > 64 ? 2 : 1;
          mbar_arrive_expect_tx(&full[slot], boxes * Cfg::BOX);
          for (int x = 0; x < boxes; ++x)
            tma_load_3d(dst + x * Cfg::BOX, map, &full[slot], x * 64, t.kvh, t.s.k0 + (j >> 1) * kAtBN);
          ++issued;
          if (++slot == SLOTS) slot = 0, phase ^= 1u;
        }
        if (ok && (t.end & 15)) {
          // the last V tile has been asked for: warp 3 may wait for it (the
          // one before it is done, so that vgo is never two phases ahead)
          if (nfix > 0) ok = op_wait(vfix, (nfix - 1) & 1, &s_abort);
          if (ok) mbar_arrive(vgo);
          ++nfix;
        }
      }
      ok = __shfl_sync(~0u, ok, 0);
    }
    // nothing of this CTA's is in flight when it exits, whatever happened
    if (lane == 0) {
      for (int i = 0; i < min(issued, SLOTS); ++i) {
        if (slot == 0) phase ^= 1u;
        slot = slot == 0 ? SLOTS - 1 : slot - 1;
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(&full[slot], phase) && globaltimer_ns() - t0 < 10000000ull) {
        }
      }
    }
  } else if (warp == 1) {
    const uint32_t idesc_qk = idesc_bf16_f32(kAtBM, kAtBN) | (a.scale_log2 < 0.f ? 1u << 13 : 0u);   // -Q for a negative scale
    const uint32_t idesc_pv = idesc_bf16_f32(kAtBM, (a.dim + 15) / 16 * 16) | (1u << 16);            // V: N-major
    int slot = 0, nq = 0, nfix = 0;
    uint32_t phase = 0, pphase[2] = {0, 0};
    bool ok = true;
    for (long long id = blockIdx.x; walk.at(a, tile_rows, id, t) && ok; id += gridDim.x) {
      if (t.blocks == 0) continue;
      if (lane == 0) {
        const int halves = t.rows > kAtBM ? 2 : 1;
        auto qk = [&](int s, int sl) {
          const uint32_t q = smem_u32(sQ + s * Cfg::TILE), k = smem_u32(sKV + sl * Cfg::TILE);
          for (int x = 0; x < ksteps; ++x) {
            const uint32_t o = (x >> 2) * Cfg::BOX + (x & 3) * 32;
            umma_bf16(tmem + s * kAtBN, smem_desc_sw128(q + o), smem_desc_sw128(k + o), idesc_qk, x > 0);
          }
          umma_commit(&sfull[s]);
        };
        auto next = [&] {
          if (++slot == SLOTS) slot = 0, phase ^= 1u;
        };
        ok = op_wait(qfull, nq & 1, &s_abort) && op_wait(&full[slot], phase, &s_abort);
        if (ok) {
          tc_fence_after();
          for (int s = 0; s < halves; ++s) qk(s, slot);
          umma_commit(&empty[slot]);
          next();
        }
        for (int j = 0; j < t.blocks && ok; ++j) {
          const int vslot = slot;
          const uint32_t vphase = phase;
          next();
          const bool more = j + 1 < t.blocks;
          const int keys = min(kAtBN, t.end - j * kAtBN);
          for (int s = 0; s < halves && ok; ++s) {
            ok = op_wait(&pfull[s], pphase[s], &s_abort);
            pphase[s] ^= 1u;
            if (ok && s == 0) {
              ok = op_wait(&full[vslot], vphase, &s_abort);
              if (ok && !more && (keys & 15)) ok = op_wait(vfix, nfix++ & 1, &s_abort);
            }
            if (!ok) break;
            tc_fence_after();
            const uint32_t v = smem_u32(sKV + vslot * Cfg::TILE);
            for (int x = 0; x < (keys + 15) / 16; ++x)
              umma_bf16_ts(tmem + 2 * kAtBN + s * 128, tmem + s * kAtBN + x * 8,
                           smem_desc_mn_sw128(v + x * 2048, Cfg::BOX), idesc_pv, j > 0 || x > 0);
            if (s == halves - 1) umma_commit(&empty[vslot]);
            if (more) {
              if (s == 0) ok = op_wait(&full[slot], phase, &s_abort);
              if (!ok) break;
              tc_fence_after();
              qk(s, slot);
              if (s == halves - 1) umma_commit(&empty[slot]);
            } else {
              umma_commit(&ofull[s]);
            }
          }
          if (more) {
            next();
          }
        }
        umma_commit(qempty);
        ++nq;
      }
      ok = __shfl_sync(~0u, ok, 0);
    }
  } else if (warp < 4) {
    if (blockIdx.x == 0 && warp == 2) report_bad_seqs(a, lane, 32);
    const int tid = threadIdx.x - 64;
    const int chunks = ksteps * 2, dchunks = a.dim / 8;
    int nq = 0, nfix = 0;
    long long it = 0;   // ring position of the tile's first block
    bool ok = true;
    for (long long id = blockIdx.x; walk.at(a, tile_rows, id, t) && ok; id += gridDim.x) {
      if (t.blocks == 0) continue;
      ok = op_wait_warp(qempty, (nq & 1) ^ 1u, &s_abort);
      if (!ok) break;
      ++nq;
      const int rows = t.rows > kAtBM ? 2 * kAtBM : kAtBM;
      // 16 threads (chunks of 8 values) a row
      for (int i = tid >> 4; i < rows; i += 4) {
        const int c = tid & 15;
        const int r = t.r0 + i, pos = r / group, head = t.kvh * group + r - pos * group;
        const bool there = i < t.rows && c < dchunks;
        if (c < chunks)
          cp_async16(sQ + (i >> 7) * Cfg::TILE + (c >> 3) * Cfg::BOX + (i & 127) * 128 + (((c & 7) ^ (i & 7)) << 4),
                     there ? a.q + (t.s.q0 + pos) * a.q_t + head * a.q_h + c * 8 : a.q, there);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async_smem();
      mbar_arrive(qfull);
      const int keys = t.end - (t.blocks - 1) * kAtBN;
      if (warp == 3 && (keys & 15)) {
        const long long p = it + 2 * t.blocks - 1;
        ok = op_wait_warp(vgo, nfix++ & 1, &s_abort) &&
             op_wait_warp(&full[p % SLOTS], (uint32_t)(p / SLOTS) & 1u, &s_abort);
        if (!ok) break;
        uint8_t* v = sKV + (p % SLOTS) * Cfg::TILE;
        for (int i = lane; i < (16 - (keys & 15)) * (DP / 8); i += 32) {
          const int row = keys + i / (DP / 8), c = i % (DP / 8);
          *reinterpret_cast<uint4*>(v + (c >> 3) * Cfg::BOX + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(vfix);
      }
      it += 2 * t.blocks;
    }
  } else {
    const int s = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + s * kAtBN, tO = tmem + lanes + 2 * kAtBN + s * 128;
    const float c = fabsf(a.scale_log2);
    uint32_t sphase = 0, ophase = 0;
    bool ok = true;
    for (long long id = blockIdx.x; walk.at(a, tile_rows, id, t) && ok; id += gridDim.x) {
      if (s * kAtBM >= t.rows) continue;
      const int r = t.r0 + s * kAtBM + row;
      const int pos = r / group;
      const bool valid = s * kAtBM + row < t.rows;
      int limit = valid ? t.s.nk : 0;   // keys that this row sees
      if (a.causal && valid) limit = max(0, min(limit, pos + t.s.nk - t.s.nq + 1));
      float top = -INFINITY, sum = 0.f;
      for (int j = 0; j < t.blocks; ++j) {
        ok = op_wait_warp(&sfull[s], sphase, &s_abort);
        if (!ok) break;
        sphase ^= 1u;
        tc_fence_after();
        float v[128];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32(tS + x * 32, reinterpret_cast<uint32_t(&)[32]>(v[x * 32]));
        tmem_ld_wait();
        const int left = limit - j * kAtBN;   // columns of this block that the row sees
        if (!__all_sync(~0u, left >= kAtBN)) {
#pragma unroll
          for (int x = 0; x < 128; ++x) v[x] = x < left ? v[x] : -INFINITY;
        }
        float m = v[0];
#pragma unroll
        for (int x = 1; x < 128; ++x) m = fmaxf(m, v[x]);
        m = fmaxf(m, top);
        // (an infinite difference included: the first block, or a row that saw nothing so far)
        if (__any_sync(~0u, (m - top) * c > 8.f)) {
          const float f = top == -INFINITY ? 0.f : ex2((top - m) * c);
          if (j > 0) {
#pragma unroll 1
            for (int x = 0; x < a.dim; x += 32) {
              uint32_t o[32];
              tmem_ld32(tO + x, o);
              tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
              tmem_st32(tO + x, o);
            }
          }
          sum *= f;
          top = m;
        }
        const float base = top == -INFINITY ? 0.f : -top * c;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t p[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            const float p0 = ex2(fmaf(v[x * 32 + 2 * y], c, base)), p1 = ex2(fmaf(v[x * 32 + 2 * y + 1], c, base));
            sum += p0;
            sum += p1;
            p[y] = pack_bf16x2(p0, p1);
          }
          tmem_st16(tS + x * 16, p);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[s]);
      }
      if (!ok) break;
      if (t.blocks > 0) {
        ok = op_wait_warp(&ofull[s], ophase, &s_abort);
        if (!ok) break;
        ophase ^= 1u;
        tc_fence_after();
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int head = t.kvh * group + r - pos * group;
      __nv_bfloat16* orow = a.out + (t.s.q0 + pos) * a.o_t + head * a.o_h;
#pragma unroll 1
      for (int x = 0; x < a.dim; x += 32) {
        float v[32] = {};
        if (t.blocks > 0) {
          tmem_ld32(tO + x, reinterpret_cast<uint32_t(&)[32]>(v));
          tmem_ld_wait();
        }
#pragma unroll
        for (int y = 0; y < 32; ++y) v[y] = sum == 0.f ? 0.f : v[y] * inv;
        if (valid) store_out_row(orow, out_vec, x, a.dim, v);
      }
      if (valid && a.lse != nullptr)
        a.lse[(t.s.q0 + pos) * (long long)a.heads + head] =
            sum == 0.f ? -INFINITY : (top * c + log2f(sum)) * 0.69314718055994531f;
      tc_fence_before();   // these reads of O come before what the next tile's first block lets the tensor core write
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// [tokens][kv_heads][dim] bf16 with the given strides, boxes of 128 tokens x 1
// head x 64 values, zeros past dim and past the last token.
inline CUtensorMap make_heads_tmap(const __nv_bfloat16* p, long long tokens, int heads, int dim, long long st,
                                   long long sh) {
  CUtensorMap m;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
  cuuint32_t box[3] = {64u, 1u, (cuuint32_t)kAtBN};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = encode_fn()(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) throw GditError(GDIT_ECUDA, fmt("cuTensorMapEncodeTiled (keys) failed (%d)", (int)r));
  return m;
}

template <int DP>
void launch_attention_tc(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int sms, int out_vec,
                         cudaStream_t s) {
  using Cfg = AttnCfg<DP>;
  allow_smem(attention_tc_kernel<DP>, Cfg::SMEM);
  launch_op(s, 1, attention_tc_kernel<DP>, dim3((unsigned)std::min<long long>(a.max_tiles * a.kv_heads, sms)),
            dim3(kAtThreads), Cfg::SMEM, mk, mv, a, 2 * kAtBM, out_vec);
}

inline void launch_attention(AttnArgs& a, int sms, cudaStream_t s) {
  a.max_tiles = a.total_q * (a.heads / a.kv_heads) / (2 * kAtBM) + a.batch;
  const bool none = a.total_k == 0;   // no key: the maps are not used, but they have to be valid
  const CUtensorMap mk = none ? make_heads_tmap(a.q, 1, 1, a.dim, a.dim, a.dim)
                              : make_heads_tmap(a.k, a.total_k, a.kv_heads, a.dim, a.k_t, a.k_h);
  const CUtensorMap mv = none ? mk : make_heads_tmap(a.v, a.total_k, a.kv_heads, a.dim, a.v_t, a.v_h);
  const int out_vec = ((uintptr_t)a.out & 15u) == 0 && a.o_t % 8 == 0 && a.o_h % 8 == 0;
  if (a.dim > 64) launch_attention_tc<128>(a, mk, mv, sms, out_vec, s);
  else launch_attention_tc<64>(a, mk, mv, sms, out_vec, s);
}

}  // namespace gdit
