// Attention over packed prompts with grouped heads:
//
//   query i of a sequence with nq queries and nk keys sees keys j <= i + nk - nq (causal) or all,
//   p = softmax(scale q . k),   o = sum_j p_j v_j
//
// 4 D operations per visible (query, key) pair against 2 D bytes of a key for all the queries of a tile:
// bound by the tensor cores and, next to them, by one exp per pair (16 a clock and SM, so that a
// 128 x 128 tile of 128 features takes both of them about 1024 clocks).
//
// A tile is 128 rows of (token, query head), heads of one KV head packed together as far as a power of
// two divides their number, so that few tokens fill it too. A CTA holds two tiles of neighbouring tokens
// (one for 256 features, whose accumulator takes half of tensor memory) and passes the key blocks once:
//
//   S = Q K^T      tcgen05.mma, both operands in shared memory, to tensor memory
//   P = exp2(scale log2(e) (S - m)), rounded to bf16, in tensor memory; fp32 sums before rounding
//   O += P V       tcgen05.mma, P from tensor memory, V as it lies (its features contiguous)
//
// The running maximum m moves only when a row's scores pass it by more than 8 binades of the weights
// (they stay below 2^8), so O is rarely rescaled, by the softmax threads themselves. A thread holds a
// row, so its statistics need no exchange.
//
//   warps 0-3 (4-7)  softmax of the first (second) tile, then its output
//   a warp per tile  an elected lane issues the tile's products from uniform operands (with divergent ones a
//                    product took it 80 to 100 clocks, more than the tensor core). At 128 features the
//                    first warp serves both tiles in turn, see PromptCfg::kOver
//   next warp        TMA copies of Q, then of K and V blocks through a ring. Rows of V behind a sequence's
//                    last key, which may hold anything, are cleared in shared memory (the scores of such
//                    keys are replaced by -inf)
//   last warp        plans: which tile pair comes next
//
// One CTA per SM. The grid has a CTA per (tile pair, head group), the pairs of most keys first, but a running
// CTA takes the places of those that have not started yet (cluster launch control), so that the copies of
// the next pair's Q and its first scores run under the softmax and the output of this one. (A CTA for each
// pair took 9 to 11 us of start and end.) Sizes of sequences are read on the device: the planning warp finds
// a pair's sequence from the borders.
//
// Measured at 128 features: one 8192-token prompt of 32 heads 468 us (1175 TFLOP/s) in single calls, 553 us
// (994 TFLOP/s) in a loop under the power cap; 12 packed prompts of 100 to 2400 tokens, 32 heads on 8, 197
// and 225 us. What is left is the chain scores - softmax - weights - sums of a tile (about 3300 clocks a block
// for 2048 clocks of products of both tiles).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "common.cuh"
#include "drain.cuh"
#include "gemm_swap.cuh"
#include "gemm_tc.cuh"
#include "kv_cache.cuh"

namespace hbl {

constexpr int kPromptMaxB = 4096;  // sequences of one call

struct PromptAttnArgs {
  const uint16_t *Q, *K, *V;  // bf16 rows; head h of token t at t * stride + h * D
  size_t q_stride, k_stride, v_stride;
  const int32_t *cu_q, *cu_k;  // [B + 1]
  int B, total_q, total_k, max_q, Hq, Hkv;
  float scale_log2;  // |scale| log2(e), 1 for a zero scale
  float sign;        // of the scale, 0 for a zero scale
  int causal;
  int pack, groups;  // query heads packed into a tile; such groups per KV head
  uint16_t* O;  // bf16 [total_q][Hq][D]
  float* lse;   // [total_q][Hq] or nullptr
};

// First query and key of sequence b and their numbers; false where its borders are out of order or range.
__device__ __forceinline__ bool prompt_borders(const PromptAttnArgs& a, int b, int& q0, int& nq, int& k0, int& nk) {
  q0 = a.cu_q[b];
  k0 = a.cu_k[b];
  const int q1 = a.cu_q[b + 1], k1 = a.cu_k[b + 1];
  nq = q1 - q0;
  nk = k1 - k0;
  return q0 >= 0 && q0 <= q1 && q1 <= a.total_q && k0 >= 0 && k0 <= k1 && k1 <= a.total_k;
}

template <int D>
struct PromptCfg {
  static constexpr int kTiles = D == 256 ? 1 : 2;
  // Keys of a block. A product with 64 keys was measured at 62 clocks, as long as one with 128 (its rows of Q
  // come from shared memory either way); for 256 features shared memory has no room for 128.
  static constexpr int kKeys = D == 256 ? 64 : 128;
  static constexpr int kParts = kKeys / 64;
  static constexpr int kChunks = D / 64;             // 128-byte columns of a row
  static constexpr int kQBytes = 128 * D * 2;
  static constexpr int kStageBytes = kKeys * D * 2;
  static constexpr int kStages = D == 64 ? 10 : 5;
  static constexpr int kSmem = 1024 + kTiles * kQBytes + kStages * kStageBytes;
  static constexpr int kSoftWarps = 4 * kTiles;
  static constexpr int kThreads = 32 * (kSoftWarps + kTiles + 2);
  // Two tiles: registers of a thread at launch, and after the split between the softmax and the other warps
  static constexpr int kRegisters = 168, kMoreRegisters = 208, kFewerRegisters = 88;
  // Tensor memory, 512 columns: each tile's scores and weights, then the accumulators. With 128 features
  // the weights take the scores' place, and the next scores wait until they have been used; elsewhere the
  // next scores come as soon as these have been read (two buffers of weights for blocks of 64 keys).
  static constexpr bool kOver = D == 128;
  static constexpr int kBuffers = D == 256 ? 2 : 1;
  static constexpr int kTileCols = kOver ? 128 : 192, kWeights = kOver ? 0 : D == 64 ? 128 : 64;
  static constexpr int kAcc = D == 64 ? 384 : 256;
};

__host__ __device__ constexpr uint32_t prompt_idesc(int N, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((128u >> 4) << 24);
}

// V block: features contiguous, 64 of them to a 128-byte swizzled row, keys one row after the other;
// chunks of 64 features lie chunk_bytes apart, groups of eight keys 1024 bytes.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t addr, uint32_t chunk_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3fffu);
  d |= (uint64_t)((chunk_bytes >> 4) & 0x3fffu) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

__device__ __forceinline__ void mma_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// 32 columns of this thread's lane, not waited for; tmem_ld_wait ties the registers to the wait.
__device__ __forceinline__ void tmem_ld_nowait_x32(uint32_t taddr, float* r) {
  uint32_t* u = reinterpret_cast<uint32_t*>(r);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
        "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]),
        "=r"(u[15]), "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]),
        "=r"(u[22]), "=r"(u[23]), "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]),
        "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr));
}
template <int N>
__device__ __forceinline__ void tmem_ld_wait(float (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(r[i]));
}

__device__ __forceinline__ float ex2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A value that is the same in all lanes, told to the compiler.
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// Cluster launch control: takes the place of a CTA of this grid that has not started (16 bytes of answer,
// counted on `bar`).
__device__ __forceinline__ void cancel_next(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
               ::"r"(smem_u32(answer)), "r"(smem_u32(bar))
               : "memory");
}
// The number of the CTA whose place was taken, or -1 if there was none left.
__device__ __forceinline__ int cancelled_cta(const void* answer) {
  uint32_t x, ok;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %0, h;\n\t}"
      : "=r"(x), "=r"(ok)
      : "r"(smem_u32(answer))
      : "memory");
  return ok ? (int)x : -1;
}

// A tile pair of a sequence and a head group, as the scheduling warp hands it out.
struct PromptItem {
  int first;  // first token of the sequence; negative: no more
  int hq;     // head group
  int q0, nq, k0, nk;
  int pad[2];
};

template <int D>
__global__ void __launch_bounds__(PromptCfg<D>::kThreads, 1)
attn_prompt_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                   const __grid_constant__ CUtensorMap mapV, const PromptAttnArgs a) {
  using Cfg = PromptCfg<D>;
  constexpr int NT = Cfg::kTiles, BN = Cfg::kKeys, ST = Cfg::kStages, PARTS = Cfg::kParts, THREADS = Cfg::kThreads;
  constexpr bool OVER = Cfg::kOver;
  constexpr int MMA_WARP = Cfg::kSoftWarps, TMA_WARP = MMA_WARP + NT, PLAN_WARP = TMA_WARP + 1;
  extern __shared__ __align__(1024) uint8_t prompt_smem[];
  __shared__ __align__(8) uint64_t q_full[NT], q_empty[NT], kv_full[ST], kv_empty[ST], s_full[NT], s_free[NT], p_full[NT][2],
      o_done[NT][2], v_raw, drain[NT], item_full[2], item_empty[2], answer_full;
  __shared__ __align__(16) uint8_t answer[16];
  __shared__ __align__(16) PromptItem items[2];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;

  uint8_t* smem = align_shared<1024>(prompt_smem);
  uint8_t* ring = smem + NT * Cfg::kQBytes;
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int hx = a.Hkv * a.groups;      // head groups
  const int per_tile = 128 / a.pack;    // tokens of a tile

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < ST; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], OVER ? 1 : NT);
    }
    for (int t = 0; t < NT; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&p_full[t][i], 4);  // the warps of a tile
        mbar_init(&o_done[t][i], 1);
      }
      mbar_init(&s_full[t], 1);
      mbar_init(&s_free[t], 4);
      mbar_init(&drain[t], 1);
    }
    mbar_init(&v_raw, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], PLAN_WARP);  // every other warp reads it
    }
    mbar_init(&answer_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    tma_prefetch_desc(&mapQ);
    tma_prefetch_desc(&mapK);
    tma_prefetch_desc(&mapV);
  }
  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // ---- the item that the scheduling warp hands out next, the same to every other warp
  bool ok = true;
  int first = 0, q0 = 0, nq_all = 0, nq = 0, k0 = 0, nk = 0, hk = 0, head0 = 0, most = 0, blocks[NT];
  RingPos item_pos;
  auto seen = [&](int token) {
    const int n = a.causal ? token + 1 + nk - nq_all : nk;
    return n < 0 ? 0 : n > nk ? nk : n;
  };
  auto next_item = [&]() {
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&item_full[item_pos.s], item_pos.ph, &abort_flag));
    if (!ok) return false;
    const PromptItem& it = items[item_pos.s];
    first = uniform(it.first);
    q0 = uniform(it.q0);
    nq_all = uniform(it.nq);
    k0 = uniform(it.k0);
    nk = uniform(it.nk);
    const int hq = uniform(it.hq);
    __syncwarp();
    if (lane == 0) mbar_arrive(&item_empty[item_pos.s]);
    item_pos.advance(1, 2);
    if (first < 0) return false;
    nq = nq_all < a.max_q ? nq_all : a.max_q;
    hk = hq / a.groups;
    head0 = hk * (a.Hq / a.Hkv) + hq % a.groups * a.pack;
    most = 0;
#pragma unroll
    for (int t = 0; t < NT; ++t) {  // key blocks that a tile sees
      const int lo = first + t * per_tile, hi = lo + per_tile < nq ? lo + per_tile : nq;
      blocks[t] = lo < nq ? (seen(hi - 1) + BN - 1) / BN : 0;
      most = blocks[t] > most ? blocks[t] : most;
    }
    return true;
  };

  // Two tiles: the softmax threads hold a row of 128 scores, so they take registers from the other warps.
  static_assert(NT == 1 || (THREADS == 384 && MMA_WARP == 8 &&
                            256 * Cfg::kMoreRegisters + 128 * Cfg::kFewerRegisters == 384 * Cfg::kRegisters), "");
  if (warp >= MMA_WARP) {
    if constexpr (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kFewerRegisters));
    if (warp == PLAN_WARP) {
      // ---- a CTA number's tile pair, from where the last search ended (numbers mostly rise). Up to 32
      // sequences, causal: the pairs of most keys first, whatever their sequence (a level is a pair's place
      // counted in pairs from its sequence's first key), so that the last ones are short. Else one sequence
      // after the other, 32 at a time: a lane holds one sequence, and more of them have more pairs to end with.
      // By level and by sequence, 32 heads on 8 of 128, 100 to 2400 tokens, us: 4 sequences 68, 74; 12 254, 259;
      // 24 401, 409; 32 592, 604; of 1 to 600 tokens, 8 sequences 24, 26; 32 67, 73.
      const bool by_level = a.causal && a.B <= 32;
      int base_b = 0, base_tiles = 0;  // sequences and tile pairs before the current 32 (the current level)
      int level = -1, top_level = -1, q_b = 0, n_b = 0, k_b = 0, m_b = 0, low_b = 0, tiles_b = 0;  // of lane b
      if (by_level) {
        if (lane < a.B && prompt_borders(a, lane, q_b, n_b, k_b, m_b))
          tiles_b = ((n_b < a.max_q ? n_b : a.max_q) + NT * per_tile - 1) / (NT * per_tile);
        low_b = m_b > n_b ? (m_b - n_b) / (NT * per_tile) : 0;
        top_level = __reduce_max_sync(0xffffffffu, tiles_b > 0 ? low_b + tiles_b - 1 : -1);
        level = top_level;
      }
      int cta = blockIdx.x;
      uint32_t answers = 0;
      bool more = true;
      while (more) {
        ok = __all_sync(0xffffffffu, mbar_wait(&item_empty[item_pos.s], item_pos.ph ^ 1u, &abort_flag));
        if (!ok) break;
        if (cta < 0) {  // not the first item
          if (lane == 0) {
            fence_proxy_async_shared();
            mbar_arrive_expect_tx(&answer_full, 16);
            cancel_next(answer, &answer_full);
          }
          ok = __all_sync(0xffffffffu, mbar_wait(&answer_full, answers & 1u, &abort_flag));
          ++answers;
          if (!ok) {
            drain_wait(&answer_full, (answers - 1) & 1u);
            break;
          }
          cta = cancelled_cta(answer);
        }
        PromptItem it = {-1, 0, 0, 0, 0, 0, {0, 0}};
        if (cta == 0)
          for (int b = lane; b < a.B; b += 32) {
            int q, n, k, m;
            if (!prompt_borders(a, b, q, n, k, m) || n > a.max_q) raise_error(kErrBadIndex);
          }
        if (cta >= 0) {
          const int tile = cta / hx;
          it.hq = cta % hx;
          if (tile < base_tiles) base_b = base_tiles = 0, level = top_level;
          for (; by_level && level >= 0; --level) {
            const uint32_t there = __ballot_sync(0xffffffffu, level >= low_b && level < low_b + tiles_b);
            const int rank = tile - base_tiles;
            if (rank < __popc(there)) {
              const int src = __fns(there, 0, rank + 1);
              it.first = __shfl_sync(0xffffffffu, (level - low_b) * NT * per_tile, src);
              it.q0 = __shfl_sync(0xffffffffu, q_b, src);
              it.nq = __shfl_sync(0xffffffffu, n_b, src);
              it.k0 = __shfl_sync(0xffffffffu, k_b, src);
              it.nk = __shfl_sync(0xffffffffu, m_b, src);
              break;
            }
            base_tiles += __popc(there);
          }
          while (!by_level && base_b < a.B) {
            const int b = base_b + lane;
            int q, n = 0, k = 0, m = 0, tiles = 0;
            if (b < a.B && prompt_borders(a, b, q, n, k, m))
              tiles = ((n < a.max_q ? n : a.max_q) + NT * per_tile - 1) / (NT * per_tile);
            int upto = tiles;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const int v = __shfl_up_sync(0xffffffffu, upto, o);
              if (lane >= o) upto += v;
            }
            const int rank = tile - base_tiles;
            const uint32_t here = __ballot_sync(0xffffffffu, rank < upto);
            if (here != 0u) {  // the first sequence that reaches the rank; its last tokens see most keys
              const int src = __ffs(here) - 1;
              it.first = __shfl_sync(0xffffffffu, (upto - 1 - rank) * NT * per_tile, src);
              it.q0 = __shfl_sync(0xffffffffu, q, src);
              it.nq = __shfl_sync(0xffffffffu, n, src);
              it.k0 = __shfl_sync(0xffffffffu, k, src);
              it.nk = __shfl_sync(0xffffffffu, m, src);
              break;
            }
            base_tiles += __shfl_sync(0xffffffffu, upto, 31);
            base_b += 32;
          }
        }
        more = it.first >= 0;
        if (lane == 0) {
          items[item_pos.s] = it;
          mbar_arrive(&item_full[item_pos.s]);
        }
        item_pos.advance(1, 2);
        cta = -1;
      }
    } else if (warp == TMA_WARP) {
      RingPos pos;
      int issued = 0;
      LoneCopies raws, queries[NT];  // on v_raw and q_full
      while (next_item()) {
        auto load = [&](const CUtensorMap* map, int j, uint64_t* full) {
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[pos.s], pos.ph ^ 1u, &abort_flag));
          if (!ok) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(full, Cfg::kStageBytes);
            for (int c = 0; c < Cfg::kChunks; ++c)
              tma_load_3d(ring + pos.s * Cfg::kStageBytes + c * (BN * 128), map, full, 64 * c, hk, k0 + j * BN);
          }
          if (full == &v_raw) {  // the last block, with rows that are no keys of the sequence
            raws.start();
            ok = __all_sync(0xffffffffu, mbar_wait(&v_raw, raws.parity(), &abort_flag));
            if (!ok) return;
            for (int c = 0; c < Cfg::kChunks; ++c)
              for (int x = (nk - j * BN) * 8 + lane; x < BN * 8; x += 32)
                reinterpret_cast<uint4*>(ring + pos.s * Cfg::kStageBytes + c * (BN * 128))[x] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&kv_full[pos.s]);
          }
          pos.advance(1, ST);
          ++issued;
        };
        auto load_q = [&](int t) {
          if (blocks[t] == 0) return;
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[t], (queries[t].started & 1u) ^ 1u, &abort_flag));
          if (!ok) return;
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[t], Cfg::kQBytes);
            for (int c = 0; c < Cfg::kChunks; ++c)
              tma_load_3d(smem + t * Cfg::kQBytes + c * (128 * 128), &mapQ, &q_full[t], 64 * c, head0,
                          q0 + first + t * per_tile);
          }
          queries[t].start();
        };
        auto load_k = [&](int j) { load(&mapK, j, &kv_full[pos.s]); };
        auto load_v = [&](int j) { load(&mapV, j, (j + 1) * BN > nk ? &v_raw : &kv_full[pos.s]); };
        // in the order of the products below; the first K goes ahead, since its stage is free early
        if (most > 0) load_k(0);
#pragma unroll
        for (int t = 0; t < NT; ++t) load_q(t);
        for (int j = 0; j < most && ok; ++j) {
          if (OVER) load_v(j);
          if (j + 1 < most) load_k(j + 1);
          if (!OVER) load_v(j);
        }
        if (!ok) break;
      }
      if (abort_flag) {  // no copy may still be landing when the CTA exits
#pragma unroll
        for (int t = 0; t < NT; ++t) queries[t].drain([&](uint32_t parity) { drain_wait(&q_full[t], parity); });
        raws.drain([&](uint32_t parity) { drain_wait(&v_raw, parity); });
        for (int d = issued > ST ? issued - ST : 0; d < issued; ++d) drain_wait(&kv_full[d % ST], (uint32_t)(d / ST) & 1u);
      }
    } else {
      // An issuing warp per tile; where the weights take the scores' place (OVER) the first one serves both,
      // in turn: issued by two, the tiles' products mix, all end late, and both softmaxes run, then wait,
      // together (one 8192-token prompt 510 us against 480; two warps that take turns 580).
      const int t = warp - MMA_WARP;
      const uint32_t tm = (uint32_t)uniform((int)tmem);
      constexpr uint32_t id_s = prompt_idesc(BN, false), id_o = prompt_idesc(D, true);
      const uint64_t kd0 = smem_desc_sw128(smem_u32(ring));
      const uint64_t vd0 = smem_desc_sw128_mn(smem_u32(ring), BN * 128);
      RingPos pos;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar, parity, &abort_flag));
      };
      auto scores = [&](int u) {  // of tile u against the K block in the ring's current stage
        const uint64_t qd = smem_desc_sw128(smem_u32(smem + u * Cfg::kQBytes));
        const uint64_t kd = kd0 + (uint64_t)(pos.s * (Cfg::kStageBytes / 16));
        tc_fence_after();
        if (!ok || !elect_one()) return;
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_bf16_ss(tm + u * Cfg::kTileCols, qd + (uint64_t)(k / 4 * (128 * 128 / 16) + k % 4 * 2),
                      kd + (uint64_t)(k / 4 * (BN * 128 / 16) + k % 4 * 2), id_s, k > 0);
        mma_commit(&s_full[u]);
      };
      // block number x of tile u, its weights in buffer x & 1 of two, with the V block in ring stage vs
      auto weigh = [&](int u, uint32_t x, int vs, uint32_t acc) {
        const uint64_t vd = vd0 + (uint64_t)(vs * (Cfg::kStageBytes / 16));
        const uint32_t t_p = tm + u * Cfg::kTileCols + Cfg::kWeights + (Cfg::kBuffers == 2 ? (x & 1u) * 32 : 0);
        if (Cfg::kBuffers == 2) wait(&p_full[u][x & 1u], (x >> 1) & 1u);
        else wait(&p_full[u][0], x & 1u);
        tc_fence_after();
        if (!ok || !elect_one()) return;
#pragma unroll
        for (int k = 0; k < BN / 16; ++k)
          mma_bf16_ts(tm + Cfg::kAcc + u * D, t_p + k * 8, vd + (uint64_t)(k * (2048 / 16)), id_o, k > 0 ? 1u : acc);
        mma_commit(&o_done[u][x & 1u]);
      };
      auto commit = [&](uint64_t* bar) {  // arrives once the products so far are done
        if (ok && elect_one()) mma_commit(bar);
      };
      if constexpr (OVER) {
        uint32_t done[2] = {0, 0}, queries[2] = {0, 0};  // key blocks of the tiles so far, copies of their Q
        while (next_item()) {
          if (t != 0 || most == 0) continue;
          const int n[2] = {blocks[0], blocks[NT - 1]}, last = most;
          // K 0, then V j and K j + 1 in turn
          wait(&kv_full[pos.s], pos.ph);
#pragma unroll
          for (int u = 0; u < 2; ++u)
            if (n[u] > 0) {
              wait(&q_full[u], queries[u]++ & 1u);
              scores(u);
              if (n[u] == 1) commit(&q_empty[u]);
            }
          commit(&kv_empty[pos.s]);
          pos.advance(1, ST);
          for (int j = 0; j < last && ok; ++j) {
            wait(&kv_full[pos.s], pos.ph);
            const int vs = pos.s;
            pos.advance(1, ST);
            if (j + 1 < last) wait(&kv_full[pos.s], pos.ph);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              if (j < n[u]) weigh(u, done[u]++, vs, j > 0);
              if (j + 1 < n[u]) {
                scores(u);
                if (j + 2 == n[u]) commit(&q_empty[u]);
              }
            }
            commit(&kv_empty[vs]);
            if (j + 1 < last) {
              commit(&kv_empty[pos.s]);
              pos.advance(1, ST);
            }
          }
          if (!ok) break;
        }
      } else {
        uint32_t done = 0, queries = 0;
        auto skip = [&]() {  // a block that only the other tile sees
          wait(&kv_full[pos.s], pos.ph);
          if (ok && lane == 0) mbar_arrive(&kv_empty[pos.s]);
          pos.advance(1, ST);
        };
        while (next_item()) {
          const int n = t == 0 ? blocks[0] : blocks[NT - 1], last = most;
          // K 0, then K j + 1 and V j in turn: the next scores come as soon as block j's have been read. The
          // accumulator is free when the first weights are there, which come after the last output.
          if (n > 0) {
            wait(&q_full[t], queries++ & 1u);
            wait(&kv_full[pos.s], pos.ph);
            if (done > 0) wait(&s_free[t], (done - 1) & 1u);
            scores(t);
            if (n == 1) commit(&q_empty[t]);
            commit(&kv_empty[pos.s]);
            pos.advance(1, ST);
            for (int j = 0; j < n && ok; ++j, ++done) {
              if (j < n - 1) {
                wait(&kv_full[pos.s], pos.ph);
                wait(&s_free[t], done & 1u);
                scores(t);
                if (j == n - 2) commit(&q_empty[t]);
                commit(&kv_empty[pos.s]);
                pos.advance(1, ST);
              } else if (n < last) {
                skip();
              }
              wait(&kv_full[pos.s], pos.ph);
              weigh(t, done, pos.s, j > 0);
              commit(&kv_empty[pos.s]);
              pos.advance(1, ST);
            }
          }
          // what is left of the other tile's blocks
          for (int x = n == 0 ? 0 : n == last ? 2 * n : 2 * n + 1; x < 2 * last && ok; ++x) skip();
          if (!ok) break;
        }
      }
      // no product may still be running when the CTA exits; a commit counts those of the thread that gives it
      if (!ok && elect_one()) {
        mma_commit(&drain[t]);
        drain_wait(&drain[t], 0);
      }
    }
  } else {
    // ---- softmax: a thread per row
    if constexpr (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kMoreRegisters));
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_acc = tmem + lanes + Cfg::kAcc + t * D;
    const float sl2 = a.scale_log2;
    const float slack = 8.f / sl2;
    const bool wide = (reinterpret_cast<uintptr_t>(a.O) & 31u) == 0;
    uint32_t done = 0;  // key blocks of this tile so far
    while (next_item()) {
      const int token = first + t * per_tile + row / a.pack, head = head0 + row % a.pack;
      const int n = t == 0 ? blocks[0] : blocks[NT - 1];
      const int visible = seen(token);
      const int unmasked = seen(first + t * per_tile);  // keys that every row of the tile sees
      float m = -INFINITY, l = 0.f;
      float s[BN];
      const uint32_t t_s = tmem + lanes + t * Cfg::kTileCols;
      // Waits until block number x is in the accumulator. One barrier for even and one for odd blocks: when
      // x is asked for, block x - 2 has been waited for (or this tile's next scores, which come later), and
      // block x + 2 needs weights that this warp has not given yet, so that no phase is taken for another.
      auto weighed = [&](uint32_t x) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_done[t][x & 1u], (x >> 1) & 1u, &abort_flag));
        tc_fence_after();
        return ok;
      };
      // the scores of the block number x, once they are there; asynchronous: tmem_ld_wait
      auto fetch = [&](uint32_t x) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], x & 1u, &abort_flag));
        if (!ok) return;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < BN; c += 32) tmem_ld_nowait_x32(t_s + c, s + c);
      };
      if (n > 0) fetch(done);
      for (int j = 0; j < n && ok; ++j, ++done) {
        tmem_ld_wait(s);
        if (!OVER) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_free[t]);
        }
        if (a.sign != 1.f) {
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] *= a.sign;
        }
        if ((j + 1) * BN > unmasked) {
          const int lim = visible - j * BN;
#pragma unroll
          for (int c = 0; c < BN; ++c) s[c] = c < lim ? s[c] : -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < BN; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = c + 4 + i < BN ? fmaxf(fmaxf(mx[i], s[c + i]), s[c + 4 + i]) : fmaxf(mx[i], s[c + i]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool up = top > m + slack;
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, up)) {
          const float mn = up ? top : m;
          const float f = up ? ex2_fast((m - mn) * sl2) : 1.f;
          m = mn;
          l *= f;
          // the accumulator must hold the block before this one
          if (!OVER) {
            if (!weighed(done - 1)) break;
          }
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_ld_nowait_x32(t_acc + c, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f;
            tmem_st_32x32b_x32(t_acc + c, reinterpret_cast<const uint32_t(&)[32]>(o));
          }
        }
        const float shift = m == -INFINITY ? 0.f : -m * sl2;
        const F2 sl22(sl2, sl2), shift2(shift, shift);
        F2 sum[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
        if (!OVER && done >= Cfg::kBuffers) {  // the weights in this buffer have been used
          if (!weighed(done - Cfg::kBuffers)) break;
        }
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float p0, p1;
            fma2(F2(s[64 * h + 2 * i], s[64 * h + 2 * i + 1]), sl22, shift2).split(p0, p1);
            p0 = ex2_fast(p0);
            p1 = ex2_fast(p1);
            sum[i & 1] = add2(sum[i & 1], F2(p0, p1));
            p[i] = pack_bf16(p0, p1);
          }
          tmem_st_32x32b_x32(t_s + Cfg::kWeights + (Cfg::kBuffers == 2 ? (done & 1u) * 32 : h * 32), p);
          if (!OVER && h == PARTS - 1 && j + 1 < n) fetch(done + 1);  // under the store
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t][Cfg::kBuffers == 2 ? done & 1u : 0]);
        float l0, l1;
        add2(sum[0], sum[1]).split(l0, l1);
        l += l0 + l1;
        if (OVER && j + 1 < n) fetch(done + 1);
      }
      if (ok && n > 0) {
        weighed(done - 1);
      }
      const bool store = ok && token < nq;
      const bool some = l != 0.f;  // sees a key; a NaN among its scores is one in l, and stays one
      const float inv = some ? 1.f / l : 0.f;
      const size_t ih = (size_t)(q0 + token) * a.Hq + head;
      if (store && a.lse) a.lse[ih] = some ? (m * sl2 + log2f(l)) * 0.69314718055994530942f : -INFINITY;
      if (ok) {
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          if (n > 0) {
            tmem_ld_nowait_x32(t_acc + c, o);
            tmem_ld_wait(o);
          }
          if (store) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = some ? pack_bf16(o[2 * e] * inv, o[2 * e + 1] * inv) : 0u;
            uint16_t* dst = a.O + ih * D + c;
            if (wide) {  // whole sectors
              store_32(dst, w);
              store_32(dst + 16, w + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                reinterpret_cast<uint4*>(dst)[e] = make_uint4(w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]);
            }
          }
        }
      }
      if (!ok) break;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace hbl
