// The paged low-bit key-value cache: writing tokens (RoPE, per-head unsigned absmax quantisation)
// and reading them back.
//
// Method: the states are quantised as in qkv_quant.cuh (BitNet v2 walkthrough article, section
// "實驗結果": after RoPE, each head directly to unsigned integers through the absmax function):
//     gamma = max|x|,  u = RoundClip(L (x + gamma) / (2 gamma), 0, L),  x~ = (2u - L) gamma / L,
// L = 2^b - 1, ties to even, the middle code for a zero head.
//
// Layout: [page][KV head][chunk of 16 tokens] records of 4 D b + 128 bytes, so that the tokens of
// one head of one page are one contiguous range:
//   K codes    16 rows (one per token) of D b / 8 bytes
//   V codes    D b / 16 units of 16 bits, each unit for the 16 tokens in turn
//   gamma      fp32 [16] of K, then fp32 [16] of V
// The bits of a half-word are laid out for the products over the cache: u << p inside a 16-bit
// half is the fp16 number u 2^(p - 24) for every u << p below 2^11 (the subnormals and the first
// binade share one spacing), so a masked half-word is a tensor-core operand without a conversion.
// A product over K contracts pairs of codes of one token, so a token's codes are contiguous; a
// product over V contracts pairs of tokens of one feature, so V interleaves the tokens by half-word.
// Codes of 2, 4 and 8 bits are little-endian bit strings. Three-bit codes must not straddle a
// half-word: five go to each, at bits 0, 3, 6, 9, 12, and the codes left over sit in the bits 15.
// K: groups of 32 codes in 6 half-words, half-word h holding codes 5h .. 5h+4, bit i of code 30 + j
// in half-word 2i + j. V: groups of 16 codes in 3 units, bit j of code 15 in unit j.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace hbl {

constexpr int kKvChunk = 16;  // tokens per record

template <int D, int BITS>
struct KvRec {
  static constexpr int kRow = D * BITS / 8;          // bytes of a K row
  static constexpr int kUnits = D * BITS / 16;       // 16-bit units of a token's V codes
  static constexpr int kV = 16 * kRow;               // byte offset of the V codes
  static constexpr int kGammaK = 32 * kRow;          // byte offset of the scales
  static constexpr int kGammaV = kGammaK + 64;
  static constexpr int kBytes = kGammaK + 128;
};

__host__ __device__ constexpr size_t kv_record_bytes(int D, int bits) { return (size_t)4 * D * bits + 128; }

struct KvCacheView {
  uint8_t* base;
  int num_pages, page_size;  // page_size a multiple of 16
  int Hkv;
};

// Code d of the K row of token r in a record (any bit width, any place).
template <int D, int BITS>
__device__ __forceinline__ uint32_t kv_k_code(const uint8_t* rec, int r, int d) {
  const uint16_t* row = reinterpret_cast<const uint16_t*>(rec + r * KvRec<D, BITS>::kRow);
  if constexpr (BITS == 3) {
    const int g = d >> 5, c = d & 31;
    if (c < 30) return (row[6 * g + c / 5] >> (3 * (c % 5))) & 7u;
    const int j = c - 30;
    return (row[6 * g + j] >> 15) | ((row[6 * g + 2 + j] >> 15) << 1) | ((row[6 * g + 4 + j] >> 15) << 2);
  } else {
    return (row[d * BITS >> 4] >> (d * BITS & 15)) & ((1u << BITS) - 1u);
  }
}

// Code d of the V units of token r in a record.
template <int D, int BITS>
__device__ __forceinline__ uint32_t kv_v_code(const uint8_t* rec, int r, int d) {
  const uint16_t* v = reinterpret_cast<const uint16_t*>(rec + KvRec<D, BITS>::kV) + r;
  if constexpr (BITS == 3) {
    const int g = d >> 4, c = d & 15;
    if (c < 15) return (v[16 * (3 * g + c / 5)] >> (3 * (c % 5))) & 7u;
    return (v[16 * 3 * g] >> 15) | ((v[16 * (3 * g + 1)] >> 15) << 1) | ((v[16 * (3 * g + 2)] >> 15) << 2);
  } else {
    return (v[16 * (d * BITS >> 4)] >> (d * BITS & 15)) & ((1u << BITS) - 1u);
  }
}

// ---------------------------------------------------------------- append

struct KvAppendArgs {
  const uint16_t *Q, *K, *V;  // bf16 rows; head h of token t at t * stride + h * D
  size_t q_stride, k_stride, v_stride;
  const int32_t* pos;    // [T], or nullptr: no rotation
  const int32_t* slots;  // [T]: page * page_size + place in the page; negative: the token is not written
  float theta;
  int T, Hq;
  KvCacheView c;
  uint16_t* q_out;
  size_t qo_stride;
  int heads_per_cta;  // of Hq + 2 Hkv
};

constexpr int kAppendThreads = 256;
constexpr int kAppendTokens = 16;  // tokens per CTA: a chunk, when the slots follow one another

// The bits of four codes, staged between the quantising and the storing threads.
template <int BITS>
using KvPack = typename std::conditional<BITS == 8, uint32_t,
                                         typename std::conditional<BITS == 2, uint8_t, uint16_t>::type>::type;

// Heads staged at a time: 16 KB of packs, 16 heads at most.
template <int D, int BITS>
constexpr int kv_append_batch() {
  constexpr int n = 16384 / (kAppendTokens * (D / 4) * (int)sizeof(KvPack<BITS>));
  return n < 16 ? n : 16;
}

// Rounding to bf16 of two values, as one word.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// One CTA takes 16 tokens and a range of heads, counted through Q, K and V. D/8 lanes hold a head:
// lane s features 4s .. 4s+3 and D/2 + 4s .. D/2 + 4s + 3, which are each other's RoPE partners, so
// the rotation needs no exchange between lanes. Quantised codes are staged in shared memory as bit
// strings (four codes to a pack) and stored by threads that take consecutive tokens of one V unit,
// so that tokens which follow one another in the cache leave as whole sectors.
//
// A code is decided in fp32 unless the value lies within kNear of a .5 boundary, where L 2^-21 bounds
// the error of the fp32 rotation, of gamma and of the scaling (about L 2^-22); then the whole head is
// rotated, its gamma taken and its codes decided in fp64, so that the codes are those of a 64-bit
// evaluation.
template <int D, int BITS, bool ROPE>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const KvAppendArgs a) {
  using Rec = KvRec<D, BITS>;
  using Pack = KvPack<BITS>;
  constexpr int HALF = D / 2;
  constexpr int LPH = D / 8;        // lanes per head
  constexpr int HPW = 32 / LPH;     // heads per warp
  constexpr float kL = (float)((1 << BITS) - 1);
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
  constexpr float kNear = kL * 4.76837158203125e-7f;
  constexpr int PACKS = D / 4;
  constexpr int BATCH = kv_append_batch<D, BITS>();
  __shared__ float cs[ROPE ? kAppendTokens : 1][HALF], sn[ROPE ? kAppendTokens : 1][HALF];
  __shared__ __align__(16) Pack packs[BATCH][kAppendTokens][PACKS];
  __shared__ int tok_page[kAppendTokens], tok_row[kAppendTokens];

  const int t0 = blockIdx.x * kAppendTokens;
  const int nt = a.T - t0 < kAppendTokens ? a.T - t0 : kAppendTokens;
  const int Hkv = a.c.Hkv, Hall = a.Hq + 2 * Hkv;
  const int h_begin = blockIdx.y * a.heads_per_cta;
  const int h_end = h_begin + a.heads_per_cta < Hall ? h_begin + a.heads_per_cta : Hall;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nwarps = kAppendThreads / 32;
  const int sub = lane % LPH, hsub = lane / LPH;
  const int per_page = a.c.page_size / kKvChunk;

  pdl_wait();  // the states may come from the kernel before this one
  pdl_launch_dependents();
  if (threadIdx.x < kAppendTokens) {
    int page = -1, row = 0;
    if (threadIdx.x < nt) {
      const int s = a.slots[t0 + threadIdx.x];
      if (s >= 0) {
        if (s / a.c.page_size < a.c.num_pages) {
          page = s / a.c.page_size;
          row = s % a.c.page_size;
        } else {
          raise_error(kErrBadIndex);
        }
      }
    }
    tok_page[threadIdx.x] = page;
    tok_row[threadIdx.x] = row;
  }
  if constexpr (ROPE) {
    if (h_begin < a.Hq + Hkv) {
      const double two_pi = 6.283185307179586476925;
      const double lt = log((double)a.theta);
      for (int e = threadIdx.x; e < nt * HALF; e += kAppendThreads) {
        const int t = e / HALF, f = e % HALF;
        const double ang = (double)a.pos[t0 + t] * exp(-2.0 * (double)f / (double)D * lt);
        double s, c;
        sincos(ang - two_pi * rint(ang / two_pi), &s, &c);
        cs[t][f] = (float)c;
        sn[t][f] = (float)s;
      }
    }
  }
  __syncthreads();

  for (int hb = h_begin; hb < h_end; hb += BATCH) {
    const int nh = h_end - hb < BATCH ? h_end - hb : BATCH;
    const int hgroups = (nh + HPW - 1) / HPW;
    for (int it = warp; it < nt * hgroups; it += nwarps) {
      const int t = it / hgroups;
      const int hl = (it % hgroups) * HPW + hsub;  // head within the batch
      const bool live = hl < nh;
      const int h = hb + (live ? hl : 0);
      const int kind = h < a.Hq ? 0 : h < a.Hq + Hkv ? 1 : 2;
      const int hk = h - (kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + Hkv);
      const uint16_t* x = (kind == 0 ? a.Q + (size_t)(t0 + t) * a.q_stride
                                     : kind == 1 ? a.K + (size_t)(t0 + t) * a.k_stride
                                                 : a.V + (size_t)(t0 + t) * a.v_stride) + (size_t)hk * D + 4 * sub;
      const uint2 lo = *reinterpret_cast<const uint2*>(x);
      const uint2 hi = *reinterpret_cast<const uint2*>(x + HALF);
      float v[8];
      v[0] = __uint_as_float(lo.x << 16);
      v[1] = __uint_as_float(lo.x & 0xffff0000u);
      v[2] = __uint_as_float(lo.y << 16);
      v[3] = __uint_as_float(lo.y & 0xffff0000u);
      v[4] = __uint_as_float(hi.x << 16);
      v[5] = __uint_as_float(hi.x & 0xffff0000u);
      v[6] = __uint_as_float(hi.y << 16);
      v[7] = __uint_as_float(hi.y & 0xffff0000u);
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = v[e];
      if constexpr (ROPE) {
        if (kind < 2) {
          const float4 c4 = *reinterpret_cast<const float4*>(&cs[t][4 * sub]);
          const float4 s4 = *reinterpret_cast<const float4*>(&sn[t][4 * sub]);
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            w[e] = fmaf(-v[4 + e], s[e], v[e] * c[e]);
            w[4 + e] = fmaf(v[e], s[e], v[4 + e] * c[e]);
          }
        }
      }
      if (kind == 0 && live) {
        uint16_t* o = a.q_out + (size_t)(t0 + t) * a.qo_stride + (size_t)hk * D + 4 * sub;
        *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]));
        *reinterpret_cast<uint2*>(o + HALF) = make_uint2(pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7]));
      }
      if (!__any_sync(0xffffffffu, kind != 0 && live)) continue;
      float g = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) g = fmaxf(g, fabsf(w[e]));
#pragma unroll
      for (int o = LPH / 2; o >= 1; o >>= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
      const float mult = g > 0.f ? 0.5f * kL / g : 0.f;
      uint32_t q[8];
      bool near = !(g > 1e-30f && g < 1e30f);  // L / (2 gamma) or its products may leave fp32's range
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float tt = fmaf(w[e], mult, 0.5f * kL);
        const float y = tt + kMagic;
        q[e] = __float_as_uint(y) & 0xffu;
        near |= fabsf(tt - (y - kMagic)) > 0.5f - kNear;
      }
      // A zero is L/2 exactly, which the fp32 rounding above takes to the even code: no border case,
      // unless it comes from a rotation that cancelled.
      near = near && g > 0.f && kind != 0;
      if (near) {
        near = !(g > 1e-30f && g < 1e30f);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float tt = fmaf(w[e], mult, 0.5f * kL);
          const float y = tt + kMagic;
          const bool zero = v[e] == 0.f && (!ROPE || kind == 2 || v[e ^ 4] == 0.f);
          near |= !zero && fabsf(tt - (y - kMagic)) > 0.5f - kNear;
        }
      }
      if (__any_sync(0xffffffffu, near)) {
        // 64 bits: the heads of this warp once more (the other heads' codes come out the same)
        double xd[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) xd[e] = (double)v[e];
        if constexpr (ROPE) {
          if (kind < 2) {
            const double two_pi = 6.283185307179586476925;
            const double lt = log((double)a.theta);
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
              const double ang = (double)a.pos[t0 + t] * exp(-2.0 * (double)(4 * sub + e) / (double)D * lt);
              double s, c;
              sincos(ang - two_pi * rint(ang / two_pi), &s, &c);
              const double x0 = (double)v[e], x1 = (double)v[4 + e];
              xd[e] = x0 * c - x1 * s;
              xd[4 + e] = x0 * s + x1 * c;
            }
          }
        }
        double gd = 0.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) gd = fmax(gd, fabs(xd[e]));
#pragma unroll
        for (int o = LPH / 2; o >= 1; o >>= 1) gd = fmax(gd, __shfl_xor_sync(0xffffffffu, gd, o));
        g = (float)gd;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double L = (double)kL;
          // a zero is L/2 whatever the rounding of L gamma
          const double u = gd > 0.0 && xd[e] != 0.0 ? rint((L * xd[e] + L * gd) / (2.0 * gd)) : rint(0.5 * L);
          q[e] = (uint32_t)fmin(fmax(u, 0.0), L);
        }
      }
      if (kind != 0 && live) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t* c = q + 4 * half;
          packs[hl][t][half * (PACKS / 2) + sub] =
              (Pack)(c[0] | (c[1] << BITS) | (c[2] << (2 * BITS)) | (c[3] << (3 * BITS)));
        }
        if (sub == 0 && tok_page[t] >= 0) {
          const size_t rec = ((size_t)tok_page[t] * Hkv + hk) * per_page + tok_row[t] / kKvChunk;
          float* gp = reinterpret_cast<float*>(a.c.base + rec * Rec::kBytes + (kind == 1 ? Rec::kGammaK : Rec::kGammaV));
          gp[tok_row[t] % kKvChunk] = g;
        }
      }
    }
    __syncthreads();
    // store the batch: a thread takes 32 codes of a K row, or 16 codes of V
    constexpr int KG = D / 32, VG = D / 16;
    for (int i = threadIdx.x; i < nh * kAppendTokens * VG; i += kAppendThreads) {
      const int hl = i / (kAppendTokens * VG), r = i % (kAppendTokens * VG);
      const int h = hb + hl;
      if (h < a.Hq) continue;
      const bool is_k = h < a.Hq + Hkv;
      const int t = is_k ? r / KG : r % kAppendTokens;
      const int g = is_k ? r % KG : r / kAppendTokens;
      if (t >= nt || tok_page[t] < 0) continue;  // K uses the first half of the threads' items
      const int hk = h - a.Hq - (is_k ? 0 : Hkv);
      const int row = tok_row[t];
      uint8_t* rec = a.c.base +
                     (((size_t)tok_page[t] * Hkv + hk) * per_page + row / kKvChunk) * (size_t)Rec::kBytes;
      if (is_k) {
        const Pack* p = &packs[hl][t][g * 8];
        uint8_t* out = rec + (row % kKvChunk) * Rec::kRow + g * 4 * BITS;
        if constexpr (BITS == 2) {
          *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(p);
        } else if constexpr (BITS == 4) {
          *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(p);
        } else if constexpr (BITS == 8) {
          reinterpret_cast<uint4*>(out)[0] = reinterpret_cast<const uint4*>(p)[0];
          reinterpret_cast<uint4*>(out)[1] = reinterpret_cast<const uint4*>(p)[1];
        } else {
          const uint4 w4 = *reinterpret_cast<const uint4*>(p);  // eight packs of 12 bits
          const uint32_t pw[4] = {w4.x, w4.y, w4.z, w4.w};
          uint32_t s24[4];  // eight codes each
#pragma unroll
          for (int j = 0; j < 4; ++j) s24[j] = (pw[j] & 0xfffu) | ((pw[j] >> 16) << 12);
          const unsigned long long s0 = (unsigned long long)s24[0] | ((unsigned long long)s24[1] << 24);  // codes 0..15
          const unsigned long long s1 = (unsigned long long)s24[2] | ((unsigned long long)s24[3] << 24);  // 16..31
          uint32_t hw[6];
          hw[0] = (uint32_t)s0 & 0x7fffu;
          hw[1] = (uint32_t)(s0 >> 15) & 0x7fffu;
          hw[2] = (uint32_t)(s0 >> 30) & 0x7fffu;
          hw[3] = (uint32_t)(s0 >> 45) | (((uint32_t)s1 & 0xfffu) << 3);
          hw[4] = (uint32_t)(s1 >> 12) & 0x7fffu;
          hw[5] = (uint32_t)(s1 >> 27) & 0x7fffu;
          const uint32_t c30 = (uint32_t)(s1 >> 42) & 7u, c31 = (uint32_t)(s1 >> 45);
          uint32_t* o = reinterpret_cast<uint32_t*>(out);
#pragma unroll
          for (int j = 0; j < 3; ++j)
            o[j] = hw[2 * j] | (((c30 >> j) & 1u) << 15) | (hw[2 * j + 1] << 16) | (((c31 >> j) & 1u) << 31);
        }
      } else {
        const Pack* p = &packs[hl][t][g * 4];
        uint16_t* out = reinterpret_cast<uint16_t*>(rec + Rec::kV) + g * BITS * 16 + row % kKvChunk;
        if constexpr (BITS == 3) {
          const uint2 w2 = *reinterpret_cast<const uint2*>(p);
          const uint32_t a24 = (w2.x & 0xfffu) | ((w2.x >> 16) << 12), b24 = (w2.y & 0xfffu) | ((w2.y >> 16) << 12);
          const unsigned long long s = (unsigned long long)a24 | ((unsigned long long)b24 << 24);
          const uint32_t c15 = (uint32_t)(s >> 45);
#pragma unroll
          for (int j = 0; j < 3; ++j)
            out[16 * j] = (uint16_t)(((uint32_t)(s >> (15 * j)) & 0x7fffu) | (((c15 >> j) & 1u) << 15));
        } else {
          const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
          for (int j = 0; j < BITS; ++j) out[16 * j] = u[j];
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------- gather

struct KvGatherArgs {
  KvCacheView c;
  const int32_t* slots;  // [T]; negative: the token's rows are left as they are
  int T;
  uint16_t *K, *V;  // bf16 [T][Hkv][D]; either may be nullptr
};

constexpr int kGatherTokens = 16;

// x~ = (2u - L) gamma / L, rounded to bf16. One CTA takes 16 tokens of one head, a thread 16
// features of K or of V of one token.
template <int D, int BITS>
__global__ void __launch_bounds__(2 * kGatherTokens * D / 16) kv_gather_kernel(const KvGatherArgs a) {
  using Rec = KvRec<D, BITS>;
  constexpr int G = D / 16;
  constexpr float kL = (float)((1 << BITS) - 1);
  pdl_wait();
  pdl_launch_dependents();
  const int which = threadIdx.x / (kGatherTokens * G);
  const int r = threadIdx.x % (kGatherTokens * G);
  const int t = blockIdx.x * kGatherTokens + r / G, g = r % G, h = blockIdx.y;
  uint16_t* out = which == 0 ? a.K : a.V;
  if (t >= a.T || out == nullptr) return;
  const int s = a.slots[t];
  if (s < 0) return;
  const int page = s / a.c.page_size, row = s % a.c.page_size;
  if (page >= a.c.num_pages) {
    raise_error(kErrBadIndex);
    return;
  }
  const uint8_t* rec = a.c.base + (((size_t)page * a.c.Hkv + h) * (a.c.page_size / kKvChunk) + row / kKvChunk) *
                                      (size_t)Rec::kBytes;
  const int i = row % kKvChunk;
  const float step = reinterpret_cast<const float*>(rec + (which == 0 ? Rec::kGammaK : Rec::kGammaV))[i] / kL;
  uint32_t o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t u0 = which == 0 ? kv_k_code<D, BITS>(rec, i, 16 * g + 2 * e) : kv_v_code<D, BITS>(rec, i, 16 * g + 2 * e);
    const uint32_t u1 =
        which == 0 ? kv_k_code<D, BITS>(rec, i, 16 * g + 2 * e + 1) : kv_v_code<D, BITS>(rec, i, 16 * g + 2 * e + 1);
    o[e] = pack_bf16((2.f * (float)u0 - kL) * step, (2.f * (float)u1 - kL) * step);
  }
  uint4* dst = reinterpret_cast<uint4*>(out + ((size_t)t * a.c.Hkv + h) * D + 16 * g);
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace hbl
