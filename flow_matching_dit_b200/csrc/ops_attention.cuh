// gdit_attention: softmax attention over packed sequences with grouped heads.
#pragma once

#include <type_traits>

#include "gemm_tc.cuh"
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

// ------------------------------------------------------------------ the kernel
//
// The queries of one key head are taken as packed rows i = position * group +
// head in the group, so that the heads that share keys share a tile and the
// keys are read once for all of them.  128 rows (128 / group whole positions,
// one 3-D TMA box) make a half; a CTA has two halves, each with a softmax
// warpgroup, scores and an output of its own in TMEM, so that one half's scores
// are turned into probabilities while the tensor core multiplies for the other.
//
//   rows kernel (ROWS = 0)      the halves are neighbouring positions and go over the same keys: prompts
//   keys kernel (ROWS = 64, 16) the halves have the same rows, so many at most, and take turns at the blocks of 128 keys, and the
//                               CTAs of a cluster take a part of the keys each: single tokens and too few tiles for the SMs.
//                               Two warps of each half are left over: they join the partial outputs, in the order of the
//                               parts, through distributed shared memory, while the others go on with the next tile.
//
//   warp 0       Q boxes, K and V tiles of 128 keys by TMA, each kind into a ring of its own
//   warp 1       tcgen05.mma: S = Q K^T (f32, TMEM)
//   warp 2       tcgen05.mma: O += P V (P from TMEM); zeroes the rows of the last V tile that lie behind the tile's last key
//                within 16, since 0 times what they hold may be NaN
//   warp 3       reports bad sequences
//   warps 4-11   softmax of one half each: thread = row; O is rescaled only when the running maximum has grown by more than
//                2^8 (the statistics refer to the maximum in use, so nothing is lost), and divided by the sum at the end;
//                probabilities are rounded to bf16, which is what the tensor core multiplies, their sum is of the unrounded
//                ones in f32
//
// Two causal prompts of 8192 tokens, 16 heads on 8, width 128: 1.1 PFLOP/s of 1.63 measured (417 us in a loop at the
// 1.6 GHz that the power limit leaves, 490 us with inputs that change); bound by the tensor core and the special function
// unit, both needed 2048 cycles for 256 rows x 128 keys, 2850 taken.  Short prompts are bound by what a tile costs beside
// its blocks: about 5000 cycles for its first scores, its last output and its stores.  Single tokens are bound by memory
// where they fill the SMs: 48 sequences x 4096 keys at 4.6 TB/s of 6.46, 64 x 3000 at 6.2.
//
// TMEM is full with two outputs of 128 columns: 256 columns are left for two
// times scores and probabilities.  The scores are a mailbox of 128 columns that
// both halves use in turn, emptied into registers as soon as they are there, and
// each half has 64 columns of P.  So the tensor core computes the next scores of
// a half while it still exponentiates the previous ones (scores in place of P
// would make the chain scores, softmax, P V of each half bound the kernel).  A
// warp's waits, its address arithmetic and the issue of eight multiplications take
// longer than the tensor core needs for them (64 cycles each), so two warps share
// the issuing.  For the same reason nothing in these loops branches on a lane's own
// values: waits are left to run out (op_wait_through), operands are in uniform registers.

constexpr int kAtBM = 128;       // rows of a half
constexpr int kAtBN = 128;       // keys of a block
constexpr int kAtThreads = 384;
constexpr int kAtColS = 0, kAtColP = 128, kAtColO = 256;   // TMEM: S; P of the halves (64 columns each); O of the halves (128)
// Registers of a thread: 168 at launch (64512 in all), then 104 for the first
// warpgroup and 200 for the softmax ones (the same 64512).
constexpr int kAtRegs = 168, kAtRegsIssue = 104, kAtRegsSoftmax = 200;
static_assert(3 * kAtRegs == kAtRegsIssue + 2 * kAtRegsSoftmax, "register split");

// DP: head_dim rounded up to 64 or 128.  ROWS: rows of a tile of the keys kernel
// (64, or 16), of the 128 that the tensor core computes; 0 is the rows kernel.
template <int DP, int ROWS>
struct AttnCfg {
  static constexpr bool KEYS = ROWS > 0;
  static constexpr int BOX = kAtBN * 128;                    // bytes of a [128][64] box
  static constexpr int TILE = BOX * (DP / 64);
  static constexpr int QBOX = KEYS ? ROWS * 128 : BOX;       // of a [rows][64] box of Q
  static constexpr int Q = 2 * QBOX * (DP / 64);             // two halves, or two tiles
  static constexpr int PART = KEYS ? 2 * ROWS * DP * 4 : 0;   // f32 partial outputs of the halves
  static constexpr int STATS = KEYS ? 2 * ROWS * 8 : 0;       // maximum and sum of their rows
  static constexpr int BARS = 384;
  static constexpr int RING = 227 * 1024 - (KEYS ? 384 : 128) - 1024 - Q - PART - STATS - BARS;   // 384, 128: static shared memory
  static constexpr int SLOTS = RING / TILE < 10 ? RING / TILE : 10;
  static constexpr int SMEM = 1024 + Q + PART + STATS + BARS + SLOTS * TILE;
  static constexpr int WARPS = KEYS ? (ROWS + 31) / 32 : 4;   // of a half that have rows
  static_assert((2 * SLOTS + 16) * 8 <= BARS, "barriers");
};

// A tile: positions [p0, p0 + np) of sequence s and the heads of key head kvh.
// Some row sees the keys below `end`; this CTA takes the key blocks [b0, b0 + nb).
struct AttnTile {
  Seq s;
  int p0, np, kvh, end, b0, nb;
};

// Walks tiles in an order that all warps and CTAs agree on: all lanes of a warp
// together.  A group of 32 sequences at a time, one a lane; within a group by
// falling position (the longest tiles of causal prompts first).  Every warp reads every
// group's offsets for itself, so that a CTA's time grows with the batch, also where its
// own tiles are few.
struct TileWalk {
  int base;              // first sequence of the group
  long long before;      // tiles in front of the group
  int level, full;       // tiles `level` and up of the group's sequences: `full` in number, those above `level`: `above`
  int above;
  int mine;              // lane: tiles of its sequence
  Seq seq;
  const uint8_t* order;  // the sequences by falling number of keys, or NULL

  __device__ __forceinline__ void load(const AttnArgs& a, int tile_pos) {
    const int lane = threadIdx.x & 31;
    seq = {0, 0, 0, 0};
    if (base + lane < a.batch) {
      bool ok;
      const Seq s = read_seq(a, order != nullptr ? order[base + lane] : base + lane, ok);
      if (ok) seq = s;
    }
    mine = seq.nq / tile_pos + (seq.nq % tile_pos != 0);
    level = __reduce_max_sync(~0u, mine);
    full = above = 0;
  }

  __device__ __forceinline__ void start(const AttnArgs& a, int tile_pos, const uint8_t* sorted) {
    base = 0;
    before = 0;
    order = sorted;
    load(a, tile_pos);
  }

  // id = tile * kv_heads + key head, growing from call to call; false behind the last tile
  template <bool KEYS>
  __device__ __forceinline__ bool at(const AttnArgs& a, int tile_pos, long long id, int rank, int splits, AttnTile& t) {
    const long long n = id / a.kv_heads;
    t.kvh = (int)(id - n * a.kv_heads);
    if (n >= a.max_tiles) return false;
    const int lane = threadIdx.x & 31;
    while (n - before >= full) {   // the next level, or the next group
      if (level == 0) {
        before += full;
        base += 32;
        if (base >= a.batch) return false;
        load(a, tile_pos);
        continue;
      }
      --level;
      above = full;
      full += __popc(__ballot_sync(~0u, mine > level));
    }
    const unsigned there = __ballot_sync(~0u, mine > level);
    const int nth = (int)(n - before) - above;
    const int src = __ffs(__ballot_sync(~0u, mine > level && __popc(there & ((1u << lane) - 1)) == nth)) - 1;
    t.s.q0 = __shfl_sync(~0u, seq.q0, src);
    t.s.nq = __shfl_sync(~0u, seq.nq, src);
    t.s.k0 = __shfl_sync(~0u, seq.k0, src);
    t.s.nk = __shfl_sync(~0u, seq.nk, src);
    t.p0 = level * tile_pos;
    t.np = min(tile_pos, t.s.nq - t.p0);
    t.end = t.s.nk;
    if (a.causal) t.end = max(0, min(t.s.nk, t.p0 + t.np + (t.s.nk - t.s.nq)));
    const int blocks = (t.end + kAtBN - 1) / kAtBN;
    t.b0 = KEYS ? (int)((long long)rank * blocks / splits) : 0;
    t.nb = KEYS ? (int)((long long)(rank + 1) * blocks / splits) - t.b0 : blocks;
    return true;
  }
};

// The keys kernel, whose sequences mostly have one tile a key head, takes up to
// kAtSorted sequences by falling number of keys, so that the last tiles to be handed
// out are short.
constexpr int kAtSorted = 256;

// Position r of a walk over `count` workers in rounds that run back and forth:
// with tiles of falling length everybody gets as much.
__device__ __forceinline__ long long snake(long long round, int worker, int count) {
  return round * count + ((round & 1) ? count - 1 - worker : worker);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The first `cols` of 32 bf16 of a row, where ok.  mode 2: rows aligned to 32 bytes, 1:
// to 16 bytes, 0: to their elements.  Predicated, without branches on ok.
__device__ __forceinline__ void store_row32(__nv_bfloat16* o, int mode, int cols, const uint32_t (&w)[16], bool ok) {
  if (mode == 2 && cols == 32) {
#pragma unroll
    for (int j = 0; j < 16; j += 8)
      asm volatile(
          "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %9, 0;\n\t"
          "@p st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n\t}" ::"l"(o + 2 * j),
          "r"(w[j]), "r"(w[j + 1]), "r"(w[j + 2]), "r"(w[j + 3]), "r"(w[j + 4]), "r"(w[j + 5]), "r"(w[j + 6]),
          "r"(w[j + 7]), "r"((int)ok)
          : "memory");
  } else if (mode >= 1) {
#pragma unroll
    for (int j = 0; j < 16; j += 4)
      asm volatile(
          "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
          "@p st.global.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(o + 2 * j),
          "r"(w[j]), "r"(w[j + 1]), "r"(w[j + 2]), "r"(w[j + 3]), "r"((int)(ok && 2 * j < cols))
          : "memory");
  } else {
    unsigned short* q = reinterpret_cast<unsigned short*>(o);
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (ok && j < cols) q[j] = (unsigned short)(w[j >> 1] >> (16 * (j & 1)));
  }
}

template <int DP, int ROWS>
__global__ void __launch_bounds__(kAtThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const AttnArgs a, int splits, int out_mode) {
  using Cfg = AttnCfg<DP, ROWS>;
  constexpr bool KEYS = ROWS > 0;
  constexpr int SLOTS = Cfg::SLOTS, KS = (SLOTS + 1) / 2, VS = SLOTS / 2;   // ring of K tiles, ring of V tiles behind it
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t tmem_holder;
  __shared__ volatile int s_abort;
  uint8_t* smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + Cfg::Q;
  float* part = reinterpret_cast<float*>(sKV + SLOTS * Cfg::TILE);
  float2* stats = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(part) + Cfg::PART);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(stats) + Cfg::STATS);
  uint64_t* empty = full + SLOTS;
  uint64_t* qfull = empty + SLOTS;
  uint64_t* qempty = qfull + 2;              // [2] each (the rows kernel has one Q buffer)
  uint64_t* sfull = qempty + 2;              // [2]
  uint64_t* sfree = sfull + 2;               // the scores have been read
  uint64_t* pfull = sfree + 1;               // [2]
  uint64_t* ofull = pfull + 2;               // [2]: P V of a block is done
  uint64_t* jfull = ofull + 2;               // the parts of all CTAs are in their shared memory
  uint64_t* jempty = jfull + 1;              // and have been read by all

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = KEYS ? (int)(blockIdx.x % splits) : 0;
  const int worker = blockIdx.x / splits, workers = gridDim.x / splits;
  if (threadIdx.x == 0) {
    for (int i = 0; i < SLOTS; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&qfull[s], 1), mbar_init(&qempty[s], 1);
      mbar_init(&sfull[s], 1), mbar_init(&pfull[s], Cfg::WARPS), mbar_init(&ofull[s], 1);
    }
    mbar_init(sfree, Cfg::WARPS);
    mbar_init(jfull, 2 * Cfg::WARPS * splits);
    mbar_init(jempty, 4 * splits);
    fence_mbar_init();
    s_abort = 0;
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_holder, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (KEYS && splits > 1) cluster_sync();   // all CTAs' barriers exist before any is signalled from outside
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_holder;
  pdl_wait();
  pdl_launch_dependents();

  const int group = a.heads / a.kv_heads;
  const int half_pos = (KEYS ? ROWS : kAtBM) / group;   // positions of a half
  const int tile_pos = KEYS ? half_pos : 2 * half_pos;
  const uint8_t* sorted = nullptr;
  if constexpr (KEYS) {
    __shared__ uint8_t s_order[kAtSorted];
    if (a.batch <= kAtSorted) {
      int* keys = reinterpret_cast<int*>(part);   // free until the first tile is joined
      bool fine;
      int mine = 0;
      if (threadIdx.x < a.batch) keys[threadIdx.x] = mine = read_seq(a, threadIdx.x, fine).nk;
      __syncthreads();
      if (threadIdx.x < a.batch) {
        int before = 0;
        for (int i = 0; i < a.batch; ++i) before += keys[i] > mine || (keys[i] == mine && i < (int)threadIdx.x);
        s_order[before] = (uint8_t)threadIdx.x;
      }
      __syncthreads();
      sorted = s_order;
    }
  }
  TileWalk walk;
  AttnTile t;
  bool ok = true;

  if (warp < 4) {
    set_max_regs_dec<kAtRegsIssue>();
    if (warp == 0) {
      walk.start(a, tile_pos, sorted);
      int kslot = 0, vslot = 0, nq = 0;
      uint32_t kphase = 0, vphase = 0;
      const int boxes = a.dim > 64 ? 2 : 1;
      for (long long round = 0;
           ok && walk.at<KEYS>(a, tile_pos, snake(round, worker, workers), rank, splits, t); ++round) {
        if (t.nb == 0) continue;
        if (lane == 0) {
          const int qb = KEYS ? nq & 1 : 0;
          ok = op_wait(&qempty[qb], ((KEYS ? nq >> 1 : nq) & 1) ^ 1u, &s_abort);
          if (ok) {
            const int halves = !KEYS && t.np > half_pos ? 2 : 1;
            mbar_arrive_expect_tx(&qfull[qb], halves * boxes * half_pos * group * 128);
            for (int s = 0; s < halves; ++s)
              for (int x = 0; x < boxes; ++x)
                tma_load_3d(sQ + (KEYS ? qb : s) * (Cfg::Q / 2) + x * Cfg::QBOX, &tmQ,
                            &qfull[qb], x * 64, t.kvh * group, t.s.q0 + t.p0 + s * half_pos);
          }
          // the order of use: K of the first blocks, then V of a block and K of a later one in turn
          const int ahead = min(KEYS ? 3 : 2, t.nb), turns = 2 * (t.nb - ahead);
          for (int i = 0; i < 2 * t.nb && ok; ++i) {
            const int u = i - ahead;
            const bool is_v = u >= 0 && (u >= turns || (u & 1) == 0);
            const int j = u < 0 ? i : u >= turns ? t.nb - ahead + u - turns : (u & 1) ? ahead + (u >> 1) : u >> 1;
            const int slot = is_v ? KS + vslot : kslot;
            ok = op_wait(&empty[slot], (is_v ? vphase : kphase) ^ 1u, &s_abort);
            if (!ok) break;
            mbar_arrive_expect_tx(&full[slot], boxes * Cfg::BOX);
            for (int x = 0; x < boxes; ++x)
              tma_load_3d(sKV + slot * Cfg::TILE + x * Cfg::BOX, is_v ? &tmV : &tmK, &full[slot], x * 64, t.kvh,
                          t.s.k0 + (t.b0 + j) * kAtBN);
            if (is_v) {
              if (++vslot == VS) vslot = 0, vphase ^= 1u;
            } else {
              if (++kslot == KS) kslot = 0, kphase ^= 1u;
            }
          }
        }
        ++nq;
        ok = __shfl_sync(~0u, ok, 0);
      }
    } else if (warp == 1) {
      walk.start(a, tile_pos, sorted);
      const uint32_t idesc = idesc_bf16_f32(kAtBM, kAtBN) | (a.scale_log2 < 0.f ? 1u << 13 : 0u);   // -Q for a negative scale
      const int ksteps = (a.dim + 15) / 16;
      const uint32_t d = uniform(tmem) + kAtColS, bars = uniform(smem_u32(full));
      const uint32_t q0 = desc_lo_k(uniform(smem_u32(sQ))), k0 = desc_lo_k(uniform(smem_u32(sKV)));
      auto at = [&](const uint64_t* bar) { return bars + (uint32_t)((bar - full) * 8); };
      uint32_t slot = 0, phase = 0, sphase = 1, nq = 0;
      for (long long round = 0;
           walk.at<KEYS>(a, tile_pos, snake(round, worker, workers), rank, splits, t); ++round) {
        const int nb = (int)uniform(t.nb);
        const bool two = !KEYS && uniform(t.np > half_pos) != 0;   // both halves share each block
        if (nb == 0) continue;
        const uint32_t qb = KEYS ? nq & 1 : 0;
        op_wait_through(&qfull[qb], (KEYS ? nq >> 1 : nq) & 1, &s_abort);
        ++nq;
        for (int j = 0; j < nb; ++j) {
          op_wait_through(&full[slot], phase, &s_abort);
          const uint32_t k = k0 + slot * (Cfg::TILE >> 4);
          auto scores = [&](uint32_t s, bool closes) {
            op_wait_through(sfree, sphase, &s_abort);
            sphase ^= 1u;
            tc_fence_after();
            // (the keys kernel's Q tile has fewer rows; what is read behind them belongs to rows that nobody looks at)
            const uint32_t q = q0 + (KEYS ? qb : s) * (Cfg::Q / 2 >> 4);
            auto step = [&](int x) {
              const uint32_t o = (x & 3) * 32 >> 4, b = x >> 2;
              umma_bf16_lo(d, q + b * (Cfg::QBOX >> 4) + o, k + b * (Cfg::BOX >> 4) + o, idesc, x > 0);
            };
            if (elect_one()) {
              if (ksteps == DP / 16) {
#pragma unroll
                for (int x = 0; x < DP / 16; ++x) step(x);
              } else {
#pragma unroll 1
                for (int x = 0; x < ksteps; ++x) step(x);
              }
              umma_commit_at(at(sfull) + s * 8);
              if (closes) {
                umma_commit_at(at(empty) + slot * 8);
                if (j == nb - 1) umma_commit_at(at(qempty) + qb * 8);   // Q has been used for the last time
              }
            }
          };
          if constexpr (KEYS) {
            scores(j & 1, true);
          } else {
            scores(0, !two);
            if (two) scores(1, true);
          }
          if (++slot == KS) slot = 0, phase ^= 1u;
        }
      }
    } else if (warp == 2) {
      walk.start(a, tile_pos, sorted);
      const uint32_t idesc = idesc_bf16_f32(kAtBM, (a.dim + 15) / 16 * 16) | (1u << 16);   // V: N-major
      const uint32_t acc = uniform(tmem), bars = uniform(smem_u32(full));
      const uint32_t v0 = desc_lo_mn(uniform(smem_u32(sKV)) + KS * Cfg::TILE, Cfg::BOX);
      auto at = [&](const uint64_t* bar) { return bars + (uint32_t)((bar - full) * 8); };
      uint32_t slot = 0, phase = 0, pphase[2] = {0, 0};
      for (long long round = 0;
           walk.at<KEYS>(a, tile_pos, snake(round, worker, workers), rank, splits, t); ++round) {
        const int nb = (int)uniform(t.nb), last_keys = (int)uniform(min(kAtBN, t.end - (t.b0 + t.nb - 1) * kAtBN));
        const bool two = !KEYS && uniform(t.np > half_pos) != 0;
        for (int j = 0; j < nb; ++j) {
          op_wait_through(&full[KS + slot], phase, &s_abort);
          const int keys = j == nb - 1 ? last_keys : kAtBN, steps = (keys + 15) / 16;
          if (keys & 15) {   // zeros where the last 16 keys lie behind the tile's last one
            uint8_t* v = sKV + (KS + slot) * Cfg::TILE;
            for (int e = lane; e < (16 - (keys & 15)) * (DP / 8); e += 32) {
              const int row = keys + e / (DP / 8), c = e % (DP / 8);
              *reinterpret_cast<uint4*>(v + (c >> 3) * Cfg::BOX + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          const uint32_t v = v0 + slot * (Cfg::TILE >> 4);
          auto values = [&](uint32_t s, uint32_t& ph, bool closes) {
            op_wait_through(&pfull[s], ph, &s_abort);
            ph ^= 1u;
            tc_fence_after();
            const uint32_t p = acc + kAtColP + s * 64, o = acc + kAtColO + s * 128;
            const bool first = KEYS ? j < 2 : j == 0;
            auto step = [&](int x) {
              umma_bf16_ts_lo(o, p + x * 8, v + (x * 2048 >> 4), idesc, x > 0 || !first);
            };
            if (elect_one()) {
              if (steps == kAtBN / 16) {
#pragma unroll
                for (int x = 0; x < kAtBN / 16; ++x) step(x);
              } else {
#pragma unroll 1
                for (int x = 0; x < steps; ++x) step(x);
              }
              umma_commit_at(at(ofull) + s * 8);
              if (closes) umma_commit_at(at(empty) + (KS + slot) * 8);
            }
          };
          if constexpr (KEYS) {
            if (j & 1) values(1, pphase[1], true);
            else values(0, pphase[0], true);
          } else {
            values(0, pphase[0], !two);
            if (two) values(1, pphase[1], true);
          }
          if (++slot == VS) slot = 0, phase ^= 1u;
        }
      }
    } else if (blockIdx.x == 0) {
      report_bad_seqs(a, lane, 32);
    }
  } else {
    set_max_regs_inc<kAtRegsSoftmax>();
    walk.start(a, tile_pos, sorted);
    const int s = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int row_pos = row / group, row_head = row - row_pos * group;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + kAtColS, tP = tmem + lanes + kAtColP + s * 64, tO = tmem + lanes + kAtColO + s * 128;
    const float c = fabsf(a.scale_log2);
    const uint64_t c2 = f2_splat(c);
    uint32_t sphase = 0, ophase = 0, tphase = 0;
    auto rescale = [&](float f) {   // row `row` of O times f
#pragma unroll 1
      for (int x = 0; x < a.dim; x += 32) {
        uint32_t o[32];
        tmem_ld32(tO + x, o);
        tmem_ld_wait();
#pragma unroll
        for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
        tmem_st32(tO + x, o);
      }
    };
    if (KEYS && (warp & 2)) {
      // join: the parts (two of each CTA) of some rows, added up in their order
      const int w = s * 2 + (warp & 1), parts = 2 * splits, lparts = 31 - __clz(parts);   // (powers of two)
      for (long long round = 0;
           walk.at<KEYS>(a, tile_pos, snake(round, worker, workers), rank, splits, t); ++round) {
        ok = op_wait_warp_cluster(jfull, tphase, &s_abort);
        if (!ok) break;
        tphase ^= 1u;
        // The warp's rows are rank + splits (w + 4 j).  Item e = j * parts + p is part p of row j, 32 items at most
        // (64 rows over 4 warps and the CTAs, two parts from each of these), and lane e looks after the statistics of item e.
        const int rows = t.np * group;
        auto row_of = [&](int e) { return rank + splits * (w + 4 * (e >> lparts)); };
        const int i = row_of(lane);
        const bool mine = i < rows;
        const int items = __popc(__ballot_sync(~0u, mine));
        float2 st = make_float2(-INFINITY, 0.f);
        if (mine) st = ld_cluster_f2(mapa_shared(stats + (lane & 1) * ROWS + i, (lane & (parts - 1)) >> 1));
        float m = st.x;
        for (int o = 1; o < parts; o <<= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        // A part of which the row sees no key has the sum 0, and what memory holds of it does not count.  Where a score is NaN
        // the sum is: it is kept, also where the maximum, which passes over NaN, is -infinity or far below the others'.
        const unsigned has = __ballot_sync(~0u, st.y != 0.f);
        const float f = st.x == -INFINITY ? st.y : ex2((st.x - m) * c);
        float l = st.y * f;
        for (int o = 1; o < parts; o <<= 1) l += __shfl_xor_sync(~0u, l, o);
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int ip = i / group, head = t.kvh * group + i - ip * group;
        const long long token = t.s.q0 + t.p0 + ip, at = token * a.o_t + head * a.o_h;
        if (mine && (lane & (parts - 1)) == 0 && a.lse != nullptr)
          a.lse[token * a.heads + head] = l == 0.f ? -INFINITY : (m * c + log2f(l)) * 0.69314718055994531f;
        const int nj = (int)uniform(items >> lparts);
        auto add_up = [&](auto lp) {   // for 2, 4, 8, 16 parts: eight reads under way together, no branches between them
          constexpr int LP = decltype(lp)::value, P = 1 << LP, R = P < 8 ? 8 / P : 1, PB = P < 8 ? P : 8;
#pragma unroll 1
          for (int j0 = 0; j0 < nj; j0 += R) {
            float4 o[R];
#pragma unroll
            for (int r = 0; r < R; ++r) o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int p0 = 0; p0 < P; p0 += PB) {
              float4 h[R][PB];
#pragma unroll
              for (int r = 0; r < R; ++r)
#pragma unroll
                for (int p = 0; p < PB; ++p) {
                  const int row = rank + splits * (w + 4 * min(j0 + r, nj - 1));   // (a row again where there are no more)
                  const uint32_t from = smem_u32(part + (((p0 + p) & 1) * ROWS + row) * DP) + (((lane & (DP / 4 - 1)) ^ (row & 7)) << 4);
                  h[r][p] = LP == 1 ? ld_shared_f4(from) : ld_cluster_f4(mapa_shared_at(from, (p0 + p) >> 1));
                }
#pragma unroll
              for (int r = 0; r < R; ++r)
#pragma unroll
                for (int p = 0; p < PB; ++p) {
                  const int e = (min(j0 + r, nj - 1) << LP) + p0 + p;
                  const float fp = __shfl_sync(~0u, f, e);
                  const bool any = has >> e & 1u;
                  o[r].x = fmaf(any ? h[r][p].x : 0.f, fp, o[r].x), o[r].y = fmaf(any ? h[r][p].y : 0.f, fp, o[r].y);
                  o[r].z = fmaf(any ? h[r][p].z : 0.f, fp, o[r].z), o[r].w = fmaf(any ? h[r][p].w : 0.f, fp, o[r].w);
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const int e = min(j0 + r, nj - 1) << LP;
              const float q = __shfl_sync(~0u, inv, e);
              __nv_bfloat16* dst = a.out + __shfl_sync(~0u, at, e) + lane * 4;
              const uint2 both = make_uint2(pack_bf16x2(o[r].x * q, o[r].y * q), pack_bf16x2(o[r].z * q, o[r].w * q));
              if (j0 + r < nj && lane * 4 < a.dim) {
                if (out_mode > 0) {
                  *reinterpret_cast<uint2*>(dst) = both;
                } else {
                  unsigned short* d = reinterpret_cast<unsigned short*>(dst);
                  d[0] = (unsigned short)both.x, d[1] = (unsigned short)(both.x >> 16);
                  d[2] = (unsigned short)both.y, d[3] = (unsigned short)(both.y >> 16);
                }
              }
            }
          }
        };
        if (lparts == 1) add_up(std::integral_constant<int, 1>());
        else if (lparts == 2) add_up(std::integral_constant<int, 2>());
        else if (lparts == 3) add_up(std::integral_constant<int, 3>());
        else add_up(std::integral_constant<int, 4>());
        __syncwarp();
        if (lane < splits) mbar_arrive_cluster(mapa_shared(jempty, lane));
      }
    } else if ((warp & 3) < Cfg::WARPS) for (long long round = 0;
         walk.at<KEYS>(a, tile_pos, snake(round, worker, workers), rank, splits, t); ++round) {
      const int first_pos = KEYS ? 0 : s * half_pos;   // of this half in the tile
      if (first_pos >= t.np) continue;
      const int pos = t.p0 + first_pos + row_pos;
      const bool valid = row_pos < half_pos && first_pos + row_pos < t.np;
      const bool active = __any_sync(~0u, valid);      // a warp without rows only keeps the tensor core going
      int limit = valid ? t.s.nk : 0;                  // keys that this row sees
      if (a.causal && valid) limit = max(0, min(limit, pos + (t.s.nk - t.s.nq) + 1));
      float top = -INFINITY, sum = 0.f;
      int done = 0;                                    // blocks of this half
      // ROWS = 16: a quad of lanes has the rows quad and quad + 8, two neighbouring keys of every eight a lane; in the
      // layout of a thread a row the four rows of a token would cost the exponentials of 32.
      float top2[2] = {-INFINITY, -INFINITY}, sum2[2] = {0.f, 0.f};
      const bool upper = t.np * group > 8;             // rows 8 and up are there
      auto few_rows = [&](int block, int done, auto& wait_o) {
        tc_fence_after();
        float v[64];
        tmem_ld16x256(tS, reinterpret_cast<uint32_t(&)[64]>(v));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree);
        const int lim0 = __shfl_sync(~0u, limit, lane >> 2), lim1 = __shfl_sync(~0u, limit, (lane >> 2) + 8);
        const int left0 = lim0 - block * kAtBN - 2 * (lane & 3), left1 = lim1 - block * kAtBN - 2 * (lane & 3);
        if (!__all_sync(~0u, min(left0, left1) >= kAtBN)) {
#pragma unroll
          for (int x = 0; x < 64; ++x)
            v[x] = (x >> 2) * 8 + (x & 1) < ((x & 2) ? left1 : left0) ? v[x] : -INFINITY;
        }
        float m[2] = {top2[0], top2[1]};
#pragma unroll
        for (int x = 0; x < 64; x += 4) m[0] = max3(m[0], v[x], v[x + 1]), m[1] = max3(m[1], v[x + 2], v[x + 3]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          m[r] = fmaxf(m[r], __shfl_xor_sync(~0u, m[r], 1));
          m[r] = fmaxf(m[r], __shfl_xor_sync(~0u, m[r], 2));
        }
        wait_o();
        tc_fence_after();
        if (__any_sync(~0u, (m[0] - top2[0]) * c > 8.f || (m[1] - top2[1]) * c > 8.f)) {
          float f[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            f[r] = top2[r] == -INFINITY ? 0.f : ex2((top2[r] - m[r]) * c);
            sum2[r] *= f[r];
            top2[r] = m[r];
          }
          const float g0 = __shfl_sync(~0u, f[0], (lane & 7) * 4), g1 = __shfl_sync(~0u, f[1], (lane & 7) * 4);
          if (done > 0) rescale(lane < 8 ? g0 : g1);
        }
        uint32_t p[32];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float base = top2[r] == -INFINITY ? 0.f : -top2[r] * c;
          float part_sum = 0.f;
          if (r == 0 || upper) {
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float e0 = ex2(fmaf(v[4 * x + 2 * r], c, base)), e1 = ex2(fmaf(v[4 * x + 2 * r + 1], c, base));
              part_sum += e0 + e1;
              p[2 * x + r] = pack_bf16x2(e0, e1);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) p[2 * x + r] = 0;
          }
          sum2[r] += part_sum;
        }
        tmem_st16x128(tP, p);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[s]);
      };
      for (int j = KEYS ? s : 0; j < t.nb; j += KEYS ? 2 : 1, ++done) {
        op_wait_through(&sfull[s], sphase, &s_abort);
        sphase ^= 1u;
        // the P V of this half's previous block: it has read P and written O
        auto wait_o = [&] {
          if (done > 0) {
            op_wait_through(&ofull[s], ophase, &s_abort);
            ophase ^= 1u;
          }
        };
        if constexpr (ROWS == 16) {
          few_rows(t.b0 + j, done, wait_o);
          continue;
        }
        if (!active) {
          wait_o();
          __syncwarp();   // every lane has seen its phases: the arrivals let the next ones end
          if (lane == 0) mbar_arrive(sfree), mbar_arrive(&pfull[s]);
          continue;
        }
        tc_fence_after();
        float v[128];
#pragma unroll
        for (int x = 0; x < 4; ++x) tmem_ld32(tS + x * 32, reinterpret_cast<uint32_t(&)[32]>(v[x * 32]));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree);
        const int left = limit - (t.b0 + j) * kAtBN;   // columns of this block that the row sees
        if (!__all_sync(~0u, left >= kAtBN)) {
#pragma unroll
          for (int x = 0; x < 128; ++x) v[x] = x < left ? v[x] : -INFINITY;
        }
        float m4[4] = {top, v[0], v[1], v[2]};
#pragma unroll
        for (int x = 3; x + 1 < 128; x += 2) m4[(x >> 1) & 3] = max3(m4[(x >> 1) & 3], v[x], v[x + 1]);
        const float m = fmaxf(max3(m4[0], m4[1], m4[2]), fmaxf(m4[3], v[127]));
        wait_o();
        tc_fence_after();
        // (an infinite difference included: the first block, or a row that saw nothing so far)
        if (__any_sync(~0u, (m - top) * c > 8.f)) {
          const float f = top == -INFINITY ? 0.f : ex2((top - m) * c);
          if (done > 0) rescale(f);
          sum *= f;
          top = m;
        }
        const uint64_t base2 = f2_splat(top == -INFINITY ? 0.f : -top * c);
        uint64_t sums[2] = {f2_pack(sum, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t p[16];
#pragma unroll
          for (int y = 0; y < 16; ++y) {
            float e0, e1;
            f2_unpack(f2_fma(f2_pack(v[x * 32 + 2 * y], v[x * 32 + 2 * y + 1]), c2, base2), e0, e1);
            e0 = ex2(e0), e1 = ex2(e1);
            sums[y & 1] = f2_add(sums[y & 1], f2_pack(e0, e1));
            p[y] = pack_bf16x2(e0, e1);
          }
          tmem_st16(tP + x * 16, p);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[s]);
        float s0, s1;
        f2_unpack(f2_add(sums[0], sums[1]), s0, s1);
        sum = s0 + s1;
      }
      if (done > 0) {
        op_wait_through(&ofull[s], ophase, &s_abort);
        ophase ^= 1u;
        tc_fence_after();
      }
      if constexpr (!KEYS) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const int head = t.kvh * group + row_head;
        __nv_bfloat16* orow = a.out + (t.s.q0 + pos) * a.o_t + head * a.o_h;
        if (active) {
          const bool nothing = sum == 0.f;   // (what TMEM holds of a row without keys does not matter)
#pragma unroll 1
          for (int x = 0; x < a.dim; x += 32) {
            float v[32];
            tmem_ld32(tO + x, reinterpret_cast<uint32_t(&)[32]>(v));
            tmem_ld_wait();
            uint32_t w[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const uint32_t both = pack_bf16x2(v[2 * y] * inv, v[2 * y + 1] * inv);
              w[y] = nothing ? 0u : both;
            }
            store_row32(orow + x, out_mode, min(32, a.dim - x), w, valid);
          }
        }
        if (valid && a.lse != nullptr)
          a.lse[(t.s.q0 + pos) * (long long)a.heads + head] =
              sum == 0.f ? -INFINITY : (top * c + log2f(sum)) * 0.69314718055994531f;
        tc_fence_before();   // these reads of O come before what the next tile's first block lets the tensor core write
      } else {
        if constexpr (ROWS == 16) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            sum2[r] += __shfl_xor_sync(~0u, sum2[r], 1);
            sum2[r] += __shfl_xor_sync(~0u, sum2[r], 2);
          }
          const float t0 = __shfl_sync(~0u, top2[0], (lane & 7) * 4), t1 = __shfl_sync(~0u, top2[1], (lane & 7) * 4);
          const float s0 = __shfl_sync(~0u, sum2[0], (lane & 7) * 4), s1 = __shfl_sync(~0u, sum2[1], (lane & 7) * 4);
          top = lane < 8 ? t0 : t1, sum = lane < 8 ? s0 : s1;
        }
        // this part of the rows for the join, after all CTAs have read the previous tile's
        ok = op_wait_warp_cluster(jempty, tphase ^ 1u, &s_abort);
        if (!ok) break;
        tphase ^= 1u;
        if (active) {
          float* dst = part + (s * ROWS + row) * DP;
          if (done > 0) {
#pragma unroll 1
            for (int x = 0; x < a.dim; x += 32) {
              float v[32];
              tmem_ld32(tO + x, reinterpret_cast<uint32_t(&)[32]>(v));
              tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 32; y += 4)   // 16-byte pieces of a row in an order of its own: no bank conflicts
                if (row < ROWS) reinterpret_cast<float4*>(dst)[((x + y) >> 2) ^ (row & 7)] = make_float4(v[y], v[y + 1], v[y + 2], v[y + 3]);
            }
          }
          if (row < ROWS) stats[s * ROWS + row] = make_float2(top, sum);
        }
        tc_fence_before();
        __syncwarp();
        if (lane < splits) mbar_arrive_cluster(mapa_shared(jfull, lane));
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) op_leave(&s_abort);
  if (KEYS && splits > 1) {
    __syncwarp();
    cluster_sync();   // nobody leaves while its part is read or its barriers are signalled
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// [tokens][heads][dim] bf16 with the given strides, boxes of `box_tokens`
// tokens x `box_heads` heads x 64 values, zeros past dim and past the last token.
inline CUtensorMap make_heads_tmap(const __nv_bfloat16* p, long long tokens, int heads, int dim, long long st,
                                   long long sh, int box_tokens, int box_heads) {
  CUtensorMap m;
  cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)sh * 2, (cuuint64_t)st * 2};
  cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_tokens};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  CUresult r = encode_fn()(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16*>(p), dims, strides, box,
                           estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) throw GditError(GDIT_ECUDA, fmt("cuTensorMapEncodeTiled (heads) failed (%d)", (int)r));
  return m;
}

// How a kernel would take a call: its time, roughly, in microseconds, the CTAs of a
// cluster, and how many clusters there are.
struct AttnPlan {
  double time;
  int splits, workers;
};

// Tiles of `pos` positions that the sequences can have at most.
inline long long attn_tiles(const AttnArgs& a, int pos) { return std::min(a.total_q, a.total_q / pos + a.batch); }

// The times are those of sequences all as long as the longest: rounds of tiles, a
// time for each block of 128 keys and for a tile's first scores, output and join, and
// for the launch.  Fitted to prompts of 64 to 4000 tokens and pieces of 16 to 300
// queries over up to 8000 keys with 1 to 32 heads: the kernel chosen was the faster
// one of each, or within 3 % of it.
template <int DP, int ROWS>
AttnPlan plan_attention(const AttnArgs& a, int sms) {
  const int group = a.heads / a.kv_heads, pos = ROWS > 0 ? ROWS / group : 2 * (kAtBM / group);
  const long long units = attn_tiles(a, pos) * a.kv_heads, blocks = ((long long)a.max_k + kAtBN - 1) / kAtBN;
  if (ROWS == 0)
    return {5 + 1.75 * (double)((units + sms - 1) / sms) * (double)(blocks + 1), 1, (int)std::min<long long>(units, sms)};
  AttnPlan p = {-1, 1, 0};
  for (int n = 1; n <= 8; n *= 2) {
    const int most = n > 1 ? max_clusters(attention_kernel<DP, ROWS>, n, kAtThreads, AttnCfg<DP, ROWS>::SMEM) : sms;
    const double time = 10 + (double)((units + most - 1) / most) * (0.9 * (double)((blocks + n - 1) / n) + 2);
    if (p.time < 0 || time < p.time) p = {time, n, (int)std::min<long long>(units, most)};
  }
  return p;
}

template <int DP, int ROWS>
void launch_attention_as(AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  using Cfg = AttnCfg<DP, ROWS>;
  auto kern = attention_kernel<DP, ROWS>;
  const int group = a.heads / a.kv_heads, half_pos = (ROWS > 0 ? ROWS : kAtBM) / group;
  a.max_tiles = attn_tiles(a, ROWS > 0 ? half_pos : 2 * half_pos);
  const CUtensorMap mq = make_heads_tmap(a.q, a.total_q, a.heads, a.dim, a.q_t, a.q_h, half_pos, group);
  const bool none = a.total_k == 0;   // no key: the maps are not used, but they have to be valid
  const CUtensorMap mk = none ? mq : make_heads_tmap(a.k, a.total_k, a.kv_heads, a.dim, a.k_t, a.k_h, kAtBN, 1);
  const CUtensorMap mv = none ? mq : make_heads_tmap(a.v, a.total_k, a.kv_heads, a.dim, a.v_t, a.v_h, kAtBN, 1);
  auto rows_aligned = [&](int bytes) {
    return (uintptr_t)a.out % bytes == 0 && a.o_t * 2 % bytes == 0 && a.o_h * 2 % bytes == 0;
  };
  const int out_mode = rows_aligned(32) ? 2 : rows_aligned(16) ? 1 : 0;
  allow_smem(kern, Cfg::SMEM, kAtRegs);
  launch_op(s, p.splits, kern, dim3((unsigned)(p.workers * p.splits)), dim3(kAtThreads), Cfg::SMEM, mq, mk, mv, a,
            p.splits, out_mode);
}

template <int DP>
void launch_attention_dim(AttnArgs& a, int sms, cudaStream_t s) {
  const int group = a.heads / a.kv_heads;
  const AttnPlan rows = plan_attention<DP, 0>(a, sms);
  if (group <= 16 && a.max_q <= 16 / group) {
    const AttnPlan keys = plan_attention<DP, 16>(a, sms);
    if (keys.time < rows.time) return launch_attention_as<DP, 16>(a, keys, s);
  } else if (group <= 64) {
    const AttnPlan keys = plan_attention<DP, 64>(a, sms);
    if (keys.time < rows.time) return launch_attention_as<DP, 64>(a, keys, s);
  }
  launch_attention_as<DP, 0>(a, rows, s);
}

inline void launch_attention(AttnArgs& a, int sms, cudaStream_t s) {
  if (a.dim > 64) launch_attention_dim<128>(a, sms, s);
  else launch_attention_dim<64>(a, sms, s);
}

}  // namespace gdit
