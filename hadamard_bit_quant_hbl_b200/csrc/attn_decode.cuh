// Attention of one new token per sequence over the paged low-bit cache (kv_cache.cuh):
//
//   s_t = scale q . k~_t,   p = softmax(s) over t < len,   o = sum_t p_t v~_t,
//   k~_t = gammaK_t (2 uK_t - L) / L,  v~_t = gammaV_t (2 uV_t - L) / L
//
// Per cached token and KV head there are D b / 2 bits to read and 4 G D operations to do (G query
// heads share a KV head), so the cache's bytes bound it as long as the codes reach the products
// cheaply: at three bits a fused multiply-add per code and head would already take longer than the
// copy. Both products therefore run on the tensor cores with the codes as fp16 operands straight
// from a mask (kv_cache.cuh), the cache on the 16-row side and the query heads on the 8-column side:
//
//   S^T[t][h] = sum_d uK[t][d] q[h][d]      rows: 16 tokens, contraction: features in the order in
//                                           which the masks deliver them, q arranged alike
//   O^T[d][h] = sum_t uV[t][d] w[t][h]      rows: features, contraction: the same 16 tokens
//
// q is scaled per head by a power of two to [2^14, 2^15) and rounded to fp16 (exact for bf16 values
// down to 2^-20 of the largest). scale gammaK (2 S - L sum q) / L gives the score; gammaV goes into
// the weights w = p gammaV, rounded to fp16, whose largest is kept between 2^6 and 2^15 by running the
// softmax's base over s + log2 of gammaV's binade: a weight below 2^-20 of the largest is rounded to steps of
// 2^-30 of it. (With a largest of 1 the steps were 2^-24, and 131072 tokens of 2^-25 each beside one of 1 vanished.)
// o = (2 O - L sum w) / (L sum p). Sums are fp32.
// Codes are positive, so O and L sum w grow with the number of tokens while their difference does not, and a
// tensor core's sum drops what lies below its last bits: summed over 131072 tokens and subtracted at the end, o
// was off by 1 to 6%. L sum w / 2 is therefore taken off O every 64 tokens (1 to 3% of the time).
// mma.sync does these products at the copy's pace (one 16x8x16 product per 256 codes) and takes A
// from registers, where the masks leave it; tcgen05 would take 128-row tiles of shared or tensor
// memory for at most 16 useful columns.
//
// gammaV's binade runs from -84 to 126 (a zero counts as -84): p is at most 2^13, so p / 2^binade stays
// in range, and a weight that leaves fp32's range below belongs to a token whose gamma is 2^96 times
// smaller than another's, or whose share is below 2^-30.
//
// Up to four query heads to a KV head fill less than half of the eight columns. There q is repeated in
// two or four groups of columns, and a lane keeps the scores of the chunk that its columns' group stands
// for: one softmax pass then serves two or four chunks of 16 tokens. The weights' other groups are
// zeroed for the product with a chunk's V, and the groups are joined like the pieces of the warps.
//
// Split: the (sequence, KV head, 64-token block) triples of the whole batch are laid end to end and
// divided evenly over the warps, whatever the lengths. A warp passes its blocks through a ring of its own
// and never waits for another one: a piece of a sequence that it does not hold alone goes to the workspace
// as (max, sum, o), and attn_decode_join_kernel adds the pieces in order. (Joining the four warps of a CTA
// at each piece's end instead took 84 us against 64 for a ragged batch of 64 sequences up to 8192 tokens.)
//
// No unit is full: the busiest is the integer pipe (a mask for every two codes) at 62% of its peak, with issue at
// 49% and DRAM at 47%. Masks and copies, each 120 to 150 us by themselves on the full batch below, overlap in part
// with the 12 warps that an SM holds. 64 sequences of 3500 to 4096 tokens, 32 heads, three bits 196 us = 4.1 TB/s;
// one of 131072, 8 KV heads of 4 queries, four bits 40 us. Three CTAs to an SM; a fourth, or deeper rings, gained
// nothing.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "drain.cuh"
#include "gemm_swap.cuh"
#include "kv_cache.cuh"

namespace hbl {

constexpr int kDecodeMaxB = 4096;   // sequences of one call
constexpr int kDecodeWarps = 4;
constexpr int kDecodeMaxUnits = 4 * 448;  // warps that share the work; bounds the workspace

// Where the pieces of a (sequence, column block) are.
struct DecodeChain {
  int unit, n;  // first warp's number, number of warps (1: the output is written already)
  int first;    // 0: it is that warp's first piece, 1: its last
  int pad;
};

struct DecodeAttnArgs {
  const uint16_t* Q;  // bf16; sequence b, head h at b * q_stride + h * D
  size_t q_stride;
  KvCacheView c;
  const int32_t* tables;  // [B][table_width] page numbers
  int table_width;
  int page_shift;       // log2(page_size / 16) when that is a power of two, else -1
  const int32_t* lens;  // [B]
  int B, Hq;
  int group, groups;  // query heads per block of columns; blocks per KV head
  float scale;        // scale * log2(e) / L
  uint16_t* O;        // bf16 [B][Hq][D]
  float* lse;         // [B][Hq] or nullptr
  DecodeChain* chains;  // [B][Hkv * groups]
  float* ws;            // [units][2][group][D + 4]: a warp's first piece, then its last
};

template <int D, int BITS, int NT>
struct DecodeCfg {
  using Rec = KvRec<D, BITS>;
  // records per block of the ring: the warps' two stages each within about 70 KB
  static constexpr int kChunks = Rec::kBytes <= 2304 ? 4 : Rec::kBytes <= 4608 ? 2 : 1;
  static constexpr int kBlock = 16 * kChunks;  // tokens
  static constexpr int kStageBytes = kChunks * Rec::kBytes;
  static constexpr int kStages = 2;
  static constexpr int kSmem = kDecodeWarps * kStages * kStageBytes;
};

__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements held as a fragment (row lane/4, columns 2(lane%4), +1).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// ---------------------------------------------------------------- codes as fp16 operands

template <int BITS>
struct HalfCodes {
  // codes of a 16-bit half-word, and the place p of each after the shift: its fp16 value is u 2^(p-24)
  static constexpr int kN = BITS == 3 ? 5 : 16 / BITS;
  static constexpr int kDirect = BITS == 8 ? 1 : BITS == 4 ? 2 : BITS == 3 ? 3 : 5;  // before the shift
  __host__ __device__ static constexpr int place(int s) { return BITS * (s < kDirect ? s : s - kDirect); }
};

// The codes of both halves of a word, one pair of fp16 operands per place.
template <int BITS>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t* out) {
  using H = HalfCodes<BITS>;
  constexpr uint32_t kMask = ((1u << BITS) - 1u) * 0x00010001u;
  const uint32_t hi = w >> (BITS * H::kDirect);
#pragma unroll
  for (int s = 0; s < H::kN; ++s) out[s] = (s < H::kDirect ? w : hi) & (kMask << H::place(s));
}

// Three bits: the pair of codes in the bits 15 of three words.
__device__ __forceinline__ uint32_t spare_pair(uint32_t w0, uint32_t w1, uint32_t w2) {
  return (((w0 >> 2) & 0x20002000u) | ((w1 >> 1) & 0x40004000u) | (w2 & 0x80008000u)) >> 13;
}

// Lane j (0..3) of a quad holds a quarter of a K row's features as D/8 pairs; pair i holds features
// lo and hi (of the quarter, or for 64 features of three bits of the group of 32 that two lanes share)
// at place p.
template <int D, int BITS>
struct KPairs {
  static constexpr int kN = D / 8;
  static constexpr bool kShared = BITS == 3 && D == 64;
  __host__ __device__ static constexpr int lo(int i, bool odd = false) {
    if (kShared) return i < 5 ? (odd ? 20 : 0) + i : odd ? (i == 7 ? 30 : 13 + i - 5) : 10 + i - 5;
    if (BITS == 3) return 32 * (i / 16) + (i % 16 == 15 ? 30 : 10 * (i % 16 / 5) + i % 16 % 5);
    using H = HalfCodes<BITS>;
    return 2 * H::kN * (i / H::kN) + i % H::kN;
  }
  __host__ __device__ static constexpr int hi(int i, bool odd = false) {
    if (BITS == 3) return lo(i, odd) + (lo(i, odd) % 32 == 30 ? 1 : 5);
    return lo(i) + HalfCodes<BITS>::kN;
  }
  __host__ __device__ static constexpr int place(int i) {
    if (kShared) return 3 * (i < 5 ? i % 3 : i - 5);
    if (BITS == 3) return i % 16 == 15 ? 0 : HalfCodes<3>::place(i % 16 % 5);
    return HalfCodes<BITS>::place(i % HalfCodes<BITS>::kN);
  }
};

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  }
}

// The D/8 pairs of lane j's quarter of a K row.
template <int D, int BITS>
__device__ __forceinline__ void k_pairs(const uint8_t* row, int j, uint32_t (&out)[D / 8]) {
  if constexpr (KPairs<D, BITS>::kShared) {
    uint32_t w[3];
    load_words<3>(row + (j >> 1) * 12, w);
    const bool odd = j & 1;
    uint32_t five[5];
    code_pairs<3>(odd ? w[2] : w[0], five);
    const uint32_t rest = odd ? ((w[1] >> 9) & 0x003f003fu) | (spare_pair(w[0], w[1], w[2]) << 6) : w[1];
#pragma unroll
    for (int s = 0; s < 5; ++s) out[s] = five[s];
#pragma unroll
    for (int s = 0; s < 3; ++s) out[5 + s] = rest & (0x00070007u << (3 * s));
  } else {
    constexpr int N = D * BITS / 128;
    uint32_t w[N];
    load_words<N>(row + j * (D * BITS / 32), w);
    if constexpr (BITS == 3) {
#pragma unroll
      for (int g = 0; g < N / 3; ++g) {
#pragma unroll
        for (int i = 0; i < 3; ++i) code_pairs<3>(w[3 * g + i], out + 16 * g + 5 * i);
        out[16 * g + 15] = spare_pair(w[3 * g], w[3 * g + 1], w[3 * g + 2]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) code_pairs<BITS>(w[i], out + i * HalfCodes<BITS>::kN);
    }
  }
}

// The lanes with lane/4 = g hold D/8 features of V; feature number c of them is feature(g, c) at place(c).
// The units (three bits: threes of units) go round the lane groups, so that a load touches every bank once.
template <int D, int BITS>
struct VCodes {
  static constexpr int kN = D / 8;
  static constexpr bool kShared = BITS == 3 && D == 64;
  __host__ __device__ static constexpr int place(int c) {
    if (kShared) return 3 * (c < 5 ? c % 3 : c - 5);
    if (BITS == 3) return c % 16 == 15 ? 0 : HalfCodes<3>::place(c % 16 % 5);
    return HalfCodes<BITS>::place(c % HalfCodes<BITS>::kN);
  }
  __host__ __device__ static constexpr int feature(int g, int c) {
    if (kShared) return 16 * (g >> 1) + ((g & 1) ? (c < 5 ? 10 + c : c == 7 ? 15 : 3 + c) : c);
    constexpr int kRun = BITS == 3 ? 16 : 16 / BITS;  // features of a unit, or of three
    return (c / kRun * 8 + g) * kRun + c % kRun;
  }
};

// Pairs of tokens (4j, 4j+1) -> a, (4j+2, 4j+3) -> b of the D/8 features of lane group g.
template <int D, int BITS>
__device__ __forceinline__ void v_codes(const uint8_t* v, int g, int j, uint32_t (&a)[D / 8], uint32_t (&b)[D / 8]) {
  if constexpr (VCodes<D, BITS>::kShared) {
    uint2 u[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) u[i] = *reinterpret_cast<const uint2*>(v + (3 * (g >> 1) + i) * 32 + j * 8);
    const bool odd = g & 1;
    uint32_t five[5];
    code_pairs<3>(odd ? u[2].x : u[0].x, five);
    uint32_t rest = odd ? ((u[1].x >> 9) & 0x003f003fu) | (spare_pair(u[0].x, u[1].x, u[2].x) << 6) : u[1].x;
#pragma unroll
    for (int s = 0; s < 5; ++s) a[s] = five[s];
#pragma unroll
    for (int s = 0; s < 3; ++s) a[5 + s] = rest & (0x00070007u << (3 * s));
    code_pairs<3>(odd ? u[2].y : u[0].y, five);
    rest = odd ? ((u[1].y >> 9) & 0x003f003fu) | (spare_pair(u[0].y, u[1].y, u[2].y) << 6) : u[1].y;
#pragma unroll
    for (int s = 0; s < 5; ++s) b[s] = five[s];
#pragma unroll
    for (int s = 0; s < 3; ++s) b[5 + s] = rest & (0x00070007u << (3 * s));
  } else {
    constexpr int N = D * BITS / 128;  // units of this lane group, in runs
    constexpr int kRun = BITS == 3 ? 3 : 1;
    uint2 u[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      u[i] = *reinterpret_cast<const uint2*>(v + (i / kRun * 8 * kRun + g * kRun + i % kRun) * 32 + j * 8);
    if constexpr (BITS == 3) {
#pragma unroll
      for (int k = 0; k < N / 3; ++k) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          code_pairs<3>(u[3 * k + i].x, a + 16 * k + 5 * i);
          code_pairs<3>(u[3 * k + i].y, b + 16 * k + 5 * i);
        }
        a[16 * k + 15] = spare_pair(u[3 * k].x, u[3 * k + 1].x, u[3 * k + 2].x);
        b[16 * k + 15] = spare_pair(u[3 * k].y, u[3 * k + 1].y, u[3 * k + 2].y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        code_pairs<BITS>(u[i].x, a + i * HalfCodes<BITS>::kN);
        code_pairs<BITS>(u[i].y, b + i * HalfCodes<BITS>::kN);
      }
    }
  }
}

// ---------------------------------------------------------------- the work's order

__device__ __forceinline__ int decode_len(const DecodeAttnArgs& a, int b) {
  const long long most = (long long)a.table_width * a.c.page_size;
  const int n = a.lens[b];
  return n < 0 ? 0 : n > most ? (int)most : n;
}

// First block of warp i of n, of `total` blocks.
__device__ __forceinline__ long long decode_first(long long total, int i, int n) { return total * i / n; }

// A piece: blocks j0 .. j1-1 of (sequence b, column block h); `rest` blocks of the warp follow it.
template <int BLOCK>
struct DecodePiece {
  int b, h, j0, j1, len;
  long long rest;
  __device__ __forceinline__ void cut() {
    const int nb = (len + BLOCK - 1) / BLOCK;
    const long long n = nb - j0;
    j1 = rest < n ? j0 + (int)rest : nb;
    rest -= j1 - j0;
  }
  // the next piece; false at the end of the warp's blocks
  __device__ __forceinline__ bool next(const DecodeAttnArgs& a) {
    if (rest <= 0) return false;
    if (++h == a.c.Hkv * a.groups) {
      h = 0;
      do {
        len = decode_len(a, ++b);
      } while (len == 0);
    }
    j0 = 0;
    cut();
    return true;
  }
};

// ---------------------------------------------------------------- the kernel

// R groups of 8 / R columns, each for another chunk (R = 1 where NT = 2).
template <int D, int BITS, int NT, int R>
__global__ void __launch_bounds__(32 * kDecodeWarps, D <= 128 && NT == 1 ? 3 : 2) attn_decode_kernel(const DecodeAttnArgs a) {
  using Cfg = DecodeCfg<D, BITS, NT>;
  using Rec = KvRec<D, BITS>;
  using KP = KPairs<D, BITS>;
  using VC = VCodes<D, BITS>;
  using Piece = DecodePiece<Cfg::kBlock>;
  constexpr int CH = Cfg::kChunks, ST = Cfg::kStages, TILES = D / 16;
  constexpr int GW = 8 / R;                        // columns of a group
  constexpr int SUB = R == 1 && CH > 1 ? 2 : 1;    // softmax passes between checks of the maximum
  constexpr int EVERY = 64 / Cfg::kBlock;          // blocks between two subtractions of the codes' middle
  static_assert(CH % (R * SUB) == 0 && (R == 1 || NT == 1), "");
  constexpr float kL = (float)((1 << BITS) - 1);
  extern __shared__ __align__(128) uint8_t dec_smem[];
  __shared__ __align__(8) uint64_t bars[kDecodeWarps][ST];
  __shared__ int valid[kDecodeWarps][ST][CH];  // tokens of each chunk that count
  __shared__ long long scan[kDecodeWarps];
  __shared__ int start_b[kDecodeWarps];
  __shared__ long long start_off[kDecodeWarps];
  __shared__ volatile int abort_flag;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, j = lane & 3;
  const int hcols = a.c.Hkv * a.groups;  // column blocks per sequence

  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int w = 0; w < kDecodeWarps; ++w)
      for (int s = 0; s < ST; ++s) mbar_init(&bars[w][s], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();

  // the batch's blocks, and where each warp's begin: a thread sums a run of consecutive sequences
  const int run = (a.B + 32 * kDecodeWarps - 1) / (32 * kDecodeWarps);
  const int b_lo = threadIdx.x * run, b_hi = b_lo + run < a.B ? b_lo + run : a.B;
  long long mine = 0;
  for (int b = b_lo; b < b_hi; ++b) {
    const int len = decode_len(a, b);
    if (blockIdx.x == 0 && len != a.lens[b]) raise_error(kErrBadIndex);
    mine += (len + Cfg::kBlock - 1) / Cfg::kBlock;
  }
  long long upto = mine;  // inclusive scan over the threads
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kDecodeWarps; ++w) {
    if (w < warp) upto += scan[w];
    total += scan[w];
  }
  total *= hcols;
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {  // empty sequences
    if (decode_len(a, b) > 0) continue;
    for (int x = threadIdx.x; x < a.Hq * D / 2; x += 32 * kDecodeWarps)
      reinterpret_cast<uint32_t*>(a.O + (size_t)b * a.Hq * D)[x] = 0;
    if (a.lse)
      for (int x = threadIdx.x; x < a.Hq; x += 32 * kDecodeWarps) a.lse[(size_t)b * a.Hq + x] = -INFINITY;
    for (int x = threadIdx.x; x < hcols; x += 32 * kDecodeWarps) a.chains[(size_t)b * hcols + x].n = 1;
  }
  const int units = total < (long long)gridDim.x * kDecodeWarps ? (int)total : gridDim.x * kDecodeWarps;
  // consecutive units in different CTAs: few units keep all SMs busy
#pragma unroll
  for (int w = 0; w < kDecodeWarps; ++w) {
    const int unit = w * gridDim.x + blockIdx.x;
    if (unit >= units) break;
    const long long first = decode_first(total, unit, units);
    long long at = (upto - mine) * hcols;
    if (first < at || first >= upto * hcols) continue;
    for (int b = b_lo; b < b_hi; ++b) {
      const long long n = (long long)((decode_len(a, b) + Cfg::kBlock - 1) / Cfg::kBlock) * hcols;
      if (first < at + n) {
        start_b[w] = b;
        start_off[w] = first - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  const int unit = warp * gridDim.x + blockIdx.x;
  if (unit >= units) return;
  const long long last = decode_first(total, unit + 1, units);
  Piece piece;
  piece.b = start_b[warp];
  piece.len = decode_len(a, piece.b);
  {
    const int nb = (piece.len + Cfg::kBlock - 1) / Cfg::kBlock;
    piece.h = (int)(start_off[warp] / nb);
    piece.j0 = (int)(start_off[warp] % nb);
    piece.rest = last - decode_first(total, unit, units);
    piece.cut();
  }

  // ---- this warp's ring of blocks, copied ahead of the products
  uint8_t* ring = dec_smem + warp * ST * Cfg::kStageBytes;
  Piece ahead = piece;
  int aj = ahead.j0;  // the next block of `ahead`
  bool more = true;
  RingCopies<ST> copies;
  const int per_page = a.c.page_size / kKvChunk;
  const bool whole_blocks = per_page % CH == 0;  // a block's records lie side by side
  int pages[CH];
  auto page_of = [&](int c) { return a.page_shift >= 0 ? c >> a.page_shift : c / per_page; };
  auto settle = [&]() {  // move `ahead` to the warp's next block and read its pages' numbers
    if (aj == ahead.j1) {
      more = more && ahead.next(a);
      aj = 0;
    }
    if (!more) return;
    const int32_t* table = a.tables + (size_t)ahead.b * a.table_width;
    pages[0] = table[page_of(aj * CH)];
    if (!whole_blocks) {
#pragma unroll
      for (int i = 1; i < CH; ++i)
        if ((aj * CH + i) * kKvChunk < ahead.len) pages[i] = table[page_of(aj * CH + i)];
    }
  };
  auto copy = [&](int stage) {
    if (!more) return;
    if (lane == 0) {
      const int hk = a.groups == 1 ? ahead.h : ahead.h / a.groups;
      uint64_t* bar = &bars[warp][stage];
      uint8_t* dst = ring + stage * Cfg::kStageBytes;
      auto source = [&](int page, int c) {
        const int in_page = a.page_shift >= 0 ? c & (per_page - 1) : c % per_page;
        return a.c.base + (((size_t)page * a.c.Hkv + hk) * per_page + in_page) * (size_t)Rec::kBytes;
      };
      const int c0 = aj * CH, tokens = ahead.len - c0 * kKvChunk;  // > 0
      if (whole_blocks) {
        const bool good = pages[0] >= 0 && pages[0] < a.c.num_pages;
        const int chunks = (tokens + kKvChunk - 1) / kKvChunk < CH ? (tokens + kKvChunk - 1) / kKvChunk : CH;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int n = tokens - i * kKvChunk;
          valid[warp][stage][i] = !good || n < 0 ? 0 : n < kKvChunk ? n : kKvChunk;
        }
        mbar_arrive_expect_tx(bar, good ? chunks * Rec::kBytes : 0);
        if (good) bulk_load_1d(dst, source(pages[0], c0), chunks * Rec::kBytes, bar);
        else raise_error(kErrBadIndex);
      } else {
        uint32_t bytes = 0;
        bool good[CH];
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int n = tokens - i * kKvChunk;
          good[i] = n > 0 && pages[i] >= 0 && pages[i] < a.c.num_pages;
          if (n > 0 && !good[i]) raise_error(kErrBadIndex);
          valid[warp][stage][i] = !good[i] ? 0 : n < kKvChunk ? n : kKvChunk;
          bytes += good[i] ? Rec::kBytes : 0;
        }
        mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
        for (int i = 0; i < CH; ++i)
          if (good[i]) bulk_load_1d(dst + i * Rec::kBytes, source(pages[i], c0 + i), Rec::kBytes, bar);
      }
    }
    copies.start();
    ++aj;
    settle();
  };
  settle();
#pragma unroll
  for (int s = 0; s < ST; ++s) copy(s);

  // fragment row r of a 16-token chunk is token 4(r/2) + r%2 for r < 8, two more for r >= 8, so that the
  // transposed weights' pairs of tokens are those of the words v_codes loads
  const int row0 = 4 * (g >> 1) + (g & 1);
  bool first_piece = true, ok = true;
  while (true) {
    // ---- q of this piece: fragment of the head in column g of each tile
    const int hk = piece.h / a.groups, hg = piece.h % a.groups;
    const int head0 = hk * (a.Hq / a.c.Hkv) + hg * a.group;
    const int left = a.Hq / a.c.Hkv - hg * a.group;
    const int nheads = left < a.group ? left : a.group;
    uint32_t qf[NT][KP::kN];
    float cA[NT][2], cB[NT][2];  // score = gammaK (cA S - cB), in powers of two, of columns 2j and 2j + 1
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      constexpr int QN = KP::kShared ? 32 : D / 4;
      uint32_t raw[QN / 2];
#pragma unroll
      for (int i = 0; i < QN / 2; ++i) raw[i] = 0;
      const int qh = R == 1 ? 8 * n + g : g % GW;  // the column's head
      if (qh < nheads) {
        const uint16_t* qp = a.Q + (size_t)piece.b * a.q_stride + (size_t)(head0 + qh) * D +
                             (KP::kShared ? (j >> 1) * 32 : j * (D / 4));
        load_words<QN / 2>(reinterpret_cast<const uint8_t*>(qp), raw);
      }
      auto qv = [&](int d) {
        const uint32_t w = raw[d >> 1];
        return __uint_as_float((d & 1) ? w & 0xffff0000u : w << 16);
      };
      float qmax = 0.f;
#pragma unroll
      for (int d = 0; d < QN; ++d) qmax = fmaxf(qmax, fabsf(qv(d)));
      qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 1));
      qmax = fmaxf(qmax, __shfl_xor_sync(0xffffffffu, qmax, 2));
      int e = (int)(__float_as_uint(qmax) >> 23) - 127;  // its binade
      e = e < -100 ? -100 : e > 126 ? 126 : e;
      // 2^(14 - e) may pass fp32's range, so it is applied in two steps
      const float up0 = __uint_as_float((uint32_t)(127 + (14 - e) / 2) << 23);
      const float up1 = __uint_as_float((uint32_t)(127 + (14 - e) - (14 - e) / 2) << 23);
      float qsum = 0.f;
#pragma unroll
      for (int i = 0; i < KP::kN; ++i) {
        float lo, hi;
        if constexpr (KP::kShared) {
          lo = (j & 1) ? qv(KP::lo(i, true)) : qv(KP::lo(i, false));
          hi = (j & 1) ? qv(KP::hi(i, true)) : qv(KP::hi(i, false));
        } else {
          lo = qv(KP::lo(i));
          hi = qv(KP::hi(i));
        }
        const __half2 r = __floats2half2_rn(lo * up0 * up1, hi * up0 * up1);
        const float2 f = __half22float2(r);
        qsum += f.x + f.y;
        constexpr float one = 1.f;
        const float down = one / (float)(1 << KP::place(i));
        const __half2 s = __floats2half2_rn(f.x * down, f.y * down);
        qf[n][i] = *reinterpret_cast<const uint32_t*>(&s);
      }
      qsum += __shfl_xor_sync(0xffffffffu, qsum, 1);
      qsum += __shfl_xor_sync(0xffffffffu, qsum, 2);
      // scale back: 2^(e - 14)
      const float back = a.scale * __uint_as_float((uint32_t)(127 + (e - 14) / 2) << 23) *
                         __uint_as_float((uint32_t)(127 + (e - 14) - (e - 14) / 2) << 23);
      const float ca = back * 33554432.f, cb = back * kL * qsum;  // 2 * 2^24: a code's value is u 2^-24
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        cA[n][i] = __shfl_sync(0xffffffffu, ca, 4 * (2 * j + i));
        cB[n][i] = __shfl_sync(0xffffffffu, cb, 4 * (2 * j + i));
      }
    }

    float acc[NT][TILES][4];
    float wsum[NT][4];  // sums of the rounded weights since the last subtraction: a product with ones, every row
                        // of it the same
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int t = 0; t < TILES; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[n][t][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) wsum[n][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) m[n][i] = -INFINITY, l[n][i] = 0.f;
    }

    for (int at = piece.j0; at < piece.j1; ++at) {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[warp][copies.stage], copies.parity, &abort_flag));
      if (!ok) break;  // flagged
      const int st = copies.stage;
      const uint8_t* stage = ring + st * Cfg::kStageBytes;
#pragma unroll
      for (int c0 = 0; c0 < CH; c0 += R * SUB) {
        float z[SUB][NT][4];  // score + binade of gammaV
        float down[SUB][2], ratio[SUB][2];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          float s[NT][4];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint8_t* rec = stage + (c0 + u * R + r) * Rec::kBytes;
            float sc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
            uint32_t k0[KP::kN], k1[KP::kN];
            k_pairs<D, BITS>(rec + row0 * Rec::kRow, j, k0);
            k_pairs<D, BITS>(rec + (row0 + 2) * Rec::kRow, j, k1);
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16_16816(sc[n], k0[2 * t], k1[2 * t], k0[2 * t + 1], k1[2 * t + 1], qf[n][2 * t], qf[n][2 * t + 1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[n][i] = r == 0 || 2 * j / GW == r ? sc[n][i] : s[n][i];
          }
          const int mine = c0 + u * R + 2 * j / GW;  // the chunk of this lane's columns
          const uint8_t* rec = stage + mine * Rec::kBytes;
          const int nv = valid[warp][st][mine];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = row0 + 2 * r;
            const bool in = row < nv;
            const float gk = reinterpret_cast<const float*>(rec + Rec::kGammaK)[row];
            const float gv = reinterpret_cast<const float*>(rec + Rec::kGammaV)[row];
            int e = (int)((__float_as_uint(gv) >> 23) & 0xffu);  // biased
            e = e < 43 ? 43 : e < 254 ? e : e == 255 ? 127 : 253;  // NaN in the weights alone, not in their base
            down[u][r] = __uint_as_float((uint32_t)(254 - e) << 23);
            ratio[u][r] = in ? gv * down[u][r] : 0.f;
            const float ef = __uint_as_float(0x4b000000u + (uint32_t)e) - (8388608.f + 127.f);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                z[u][n][2 * r + i] = in ? fmaf(gk, fmaf(cA[n][i], s[n][2 * r + i], -cB[n][i]), ef) : -INFINITY;
          }
        }
        // the base m lies 2^6 below the largest product when it moves, and moves only when one would pass 2^13:
        // with gammaV at up to four times its binade (in the last one) the weights stay below 2^15 (fp16: 2^16)
        bool grow = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = fmaxf(z[0][n][i], z[0][n][2 + i]);
            if constexpr (SUB == 2) top = fmaxf(top, fmaxf(z[1][n][i], z[1][n][2 + i]));
            grow |= top > m[n][i] + 13.f;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = -INFINITY;
#pragma unroll
              for (int u = 0; u < SUB; ++u) top = fmaxf(top, fmaxf(z[u][n][i], z[u][n][2 + i]));
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
              top = fmaxf(m[n][i], top - 6.f);
              const float f = top == -INFINITY ? 1.f : ex2_approx(m[n][i] - top);
              m[n][i] = top;
              l[n][i] *= f;
              wsum[n][i] *= f;
              wsum[n][2 + i] *= f;
#pragma unroll
              for (int t = 0; t < TILES; ++t) {
                acc[n][t][i] *= f;
                acc[n][t][2 + i] *= f;
              }
            }
        }
        float base[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) base[n][i] = m[n][i] == -INFINITY ? 0.f : m[n][i];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          uint32_t wb[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float w[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float p = ex2_approx(z[u][n][2 * r + i] - base[n][i]);
                l[n][i] = fmaf(p, down[u][r], l[n][i]);
                w[i] = p * ratio[u][r];
              }
              const __half2 h2 = __floats2half2_rn(w[0], w[1]);
              wb[n][r] = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h2));
            }
            constexpr uint32_t kOnes = 0x3c003c00u;
            mma_f16_16816(wsum[n], kOnes, kOnes, kOnes, kOnes, wb[n][0], wb[n][1]);
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            uint32_t va[VC::kN], vb[VC::kN];
            v_codes<D, BITS>(stage + (c0 + u * R + r) * Rec::kBytes + Rec::kV, g, j, va, vb);
            uint32_t wr[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) wr[n][i] = R == 1 || g / GW == r ? wb[n][i] : 0u;
#pragma unroll
            for (int t = 0; t < TILES; ++t)
#pragma unroll
              for (int n = 0; n < NT; ++n)
                mma_f16_16816(acc[n][t], va[2 * t], va[2 * t + 1], vb[2 * t], vb[2 * t + 1], wr[n][0], wr[n][1]);
          }
        }
      }
      if (EVERY == 1 || at % EVERY == EVERY - 1 || at + 1 == piece.j1) {  // less L/2 of the weights so far
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const F2 w(wsum[n][0], wsum[n][1]);
#pragma unroll
          for (int t = 0; t < TILES; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float half = kL * (float)(1 << VC::place(2 * t + i)) / 33554432.f;
              float* x = &acc[n][t][2 * i];
              fma2(w, F2(-half, -half), F2(x[0], x[1])).split(x[0], x[1]);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) wsum[n][i] = 0.f;
        }
      }
      __syncwarp();  // every lane is done with the stage
      copies.use();
      copy(st);
    }
    if (!ok) break;

    // ---- join the column groups, then the output or the piece's part of it
    const int nb = (piece.len + Cfg::kBlock - 1) / Cfg::kBlock;
    const bool whole = piece.j0 == 0 && piece.j1 == nb;
    float* slot = a.ws + (size_t)(2 * unit + (first_piece ? 0 : 1)) * a.group * (D + 4);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], o);
        if constexpr (R > 1) {  // the groups' columns of a head lie 8 / R apart: lanes j, j ^ 2 (, j ^ 1)
          float top = m[n][i];
#pragma unroll
          for (int o = GW / 2; o < 4; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float f = m[n][i] == -INFINITY ? 0.f : ex2_approx(m[n][i] - top);
          m[n][i] = top;
          auto sum = [&](float& x) {
            x *= f;
#pragma unroll
            for (int o = GW / 2; o < 4; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
          };
          sum(l[n][i]);
#pragma unroll
          for (int t = 0; t < TILES; ++t) {
            sum(acc[n][t][i]);
            sum(acc[n][t][2 + i]);
          }
        }
        const int col = 8 * n + 2 * j + i;
        if (2 * j >= GW || col >= nheads) continue;
        const size_t bh = (size_t)piece.b * a.Hq + head0 + col;
        const bool some = l[n][i] != 0.f;  // sees a token; a NaN among its scores is one in l, and stays one
        const float inv = !whole ? 1.f : some ? 1.f / l[n][i] : 0.f;
        auto value = [&](int c) {  // feature number c of this lane
          const float up = 33554432.f / (kL * (float)(1 << VC::place(c)));
          return acc[n][c >> 1][2 * (c & 1) + i] * up * inv;
        };
        constexpr int RUN = VC::kShared ? 1 : BITS == 8 ? 2 : 4;  // consecutive features
#pragma unroll
        for (int c = 0; c < VC::kN; c += RUN) {
          const int d = VC::feature(g, c);
          if (whole) {
            uint16_t* o = a.O + bh * D + d;
            if constexpr (RUN == 4) {
              *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(value(c), value(c + 1)), pack_bf16(value(c + 2), value(c + 3)));
            } else if constexpr (RUN == 2) {
              *reinterpret_cast<uint32_t*>(o) = pack_bf16(value(c), value(c + 1));
            } else {
              *o = (uint16_t)(pack_bf16(value(c), 0.f) & 0xffffu);
            }
          } else {
            float* o = slot + col * D + d;
            if constexpr (RUN == 4) {
              *reinterpret_cast<float4*>(o) = make_float4(value(c), value(c + 1), value(c + 2), value(c + 3));
            } else if constexpr (RUN == 2) {
              *reinterpret_cast<float2*>(o) = make_float2(value(c), value(c + 1));
            } else {
              *o = value(c);
            }
          }
        }
        if (g == 0) {
          if (!whole) {
            slot[a.group * D + col] = m[n][i];
            slot[a.group * D + a.group + col] = l[n][i];
          } else if (a.lse) {
            a.lse[bh] = some ? (m[n][i] + log2f(l[n][i])) * 0.69314718055994530942f : -INFINITY;
          }
        }
      }
    if (piece.j0 == 0 && lane == 0) {  // the pieces of the sequence that begins here
      DecodeChain ch = {unit, 1, first_piece ? 0 : 1, 0};
      if (!whole) {
        const long long end = last + nb - piece.j1;  // of its blocks: this piece is the warp's last
        int i1 = (int)((end - 1) * units / total);   // the last warp whose first block is below it
        while (i1 + 1 < units && decode_first(total, i1 + 1, units) < end) ++i1;
        while (decode_first(total, i1, units) >= end) --i1;
        ch.n = i1 - unit + 1;
      }
      a.chains[(size_t)piece.b * hcols + piece.h] = ch;
    }
    if (!piece.next(a)) break;
    first_piece = false;
  }
  if (!ok) {  // no copy may still be landing when the CTA exits, and the join has nothing of these pieces to add
    copies.drain([&](int s, uint32_t parity) { drain_wait(&bars[warp][s], parity); });
    do {
      if (piece.j0 == 0 && lane == 0) a.chains[(size_t)piece.b * hcols + piece.h] = DecodeChain{unit, 1, 0, 0};
    } while (piece.next(a));
  }
}

// The pieces of (sequence, column block) blockIdx.x, added in a fixed order. A CTA for each head of the
// column block; D / 4 threads take four features each, the groups of threads every so many-th piece, so
// that a long chain's reads are in flight together.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) attn_decode_join_kernel(const DecodeAttnArgs a) {
  constexpr int LANES = D / 4, GROUPS = THREADS / LANES;
  __shared__ float f[kDecodeMaxUnits], sums[kDecodeMaxUnits];
  __shared__ float red[THREADS / 32], parts[GROUPS][D];
  pdl_wait();
  pdl_launch_dependents();
  const DecodeChain ch = a.chains[blockIdx.x];
  if (ch.n <= 1) return;
  const int G = a.Hq / a.c.Hkv, hcols = a.c.Hkv * a.groups;
  const int b = blockIdx.x / hcols, h = blockIdx.x % hcols;
  const int col = blockIdx.y, in_kv = h % a.groups * a.group + col;
  if (in_kv >= G) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t slot = (size_t)a.group * (D + 4);
  const float* w0 = a.ws + 2 * (size_t)ch.unit * slot;
  auto place = [&](int i) { return w0 + (2 * i + (i == 0 ? ch.first : 0)) * slot; };
  // the first parts are on their way while the pieces' maxima are compared
  const int d0 = threadIdx.x % LANES * 4, group = threadIdx.x / LANES;
  auto part = [&](int i) { return *reinterpret_cast<const float4*>(place(i) + col * D + d0); };
  float4 v = group < ch.n ? part(group) : make_float4(0.f, 0.f, 0.f, 0.f);
  float top = -INFINITY;
  for (int i = threadIdx.x; i < ch.n; i += THREADS) {
    f[i] = place(i)[a.group * D + col];
    sums[i] = place(i)[a.group * D + a.group + col];
    top = fmaxf(top, f[i]);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) red[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, red[w]);
  __syncthreads();
  float sum = 0.f;
  for (int i = threadIdx.x; i < ch.n; i += THREADS) {
    f[i] = f[i] == -INFINITY ? 0.f : ex2_approx(f[i] - top);
    sum = fmaf(f[i], sums[i], sum);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) sum += red[w];
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int i = group; i < ch.n; i += GROUPS) {
    if (i != group) v = part(i);
    o[0] = fmaf(f[i], v.x, o[0]);
    o[1] = fmaf(f[i], v.y, o[1]);
    o[2] = fmaf(f[i], v.z, o[2]);
    o[3] = fmaf(f[i], v.w, o[3]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) parts[group][d0 + e] = o[e];
  __syncthreads();
  const size_t bh = (size_t)b * a.Hq + h / a.groups * G + in_kv;
  if (threadIdx.x < D) {
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) y += parts[i][threadIdx.x];
    a.O[bh * D + threadIdx.x] = (uint16_t)(pack_bf16(sum != 0.f ? y / sum : 0.f, 0.f) & 0xffffu);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[bh] = sum != 0.f ? (top + log2f(sum)) * 0.69314718055994530942f : -INFINITY;
}

}  // namespace hbl
