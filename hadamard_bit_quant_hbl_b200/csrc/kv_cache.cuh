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

// Threads of a CTA: the warps' staged codes and the angles stay below 48 KB.
__host__ __device__ constexpr int kv_append_threads(int D, int bits) { return D * bits == 2048 ? 128 : 256; }

constexpr int kAppendTokens = 16;  // tokens per CTA: a chunk, when the slots follow one another

// The bits of four codes, staged between the quantising and the storing lanes.
template <int BITS>
using KvPack = typename std::conditional<BITS == 8, uint32_t,
                                         typename std::conditional<BITS == 2, uint8_t, uint16_t>::type>::type;

// Rounding to bf16 of two values, as one word.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The larger of two values, NaN if one of them is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Two floats in one register pair: Blackwell's fp32 multiply-adds take two at a time.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ void split(float& lo, float& hi) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The angle pos theta^(-2f / D), rounded to 64 bits, in turns less whole ones (|part| <= 1/2): the quotient by 2 pi
// with its low part, off by 2^-53 of a turn for any position, where one rounded product loses 2^-53 of all the turns.
__device__ __forceinline__ double rope_part(int pos, double inv_freq) {
  constexpr double hi = 0.15915494309189535, lo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double ang = (double)pos * inv_freq;
  const double turns = ang * hi;
  return (turns - rint(turns)) + fma(ang, lo, fma(ang, hi, -turns));
}

// Its cosine and sine in fp32: those of the leading 24 bits of the part (off by a step, 2^-24 below 1), turned on by
// the rest and rounded (half a step): off by 1.5 2^-24.
__device__ __forceinline__ void rope_cs(int pos, double inv_freq, float& c, float& s) {
  const double part = rope_part(pos, inv_freq);
  const float hi = (float)part;
  const float lo = (float)(part - (double)hi) * 6.2831853071795865f;
  float s0, c0;
  sincospif(2.f * hi, &s0, &c0);
  c = fmaf(-lo, s0, c0);
  s = fmaf(lo, c0, s0);
}

// The codes (plus the bits of kAppendMagic) and gamma of a lane's eight values of a head, all in 64 bits; codes 0 and
// gamma NaN for a head that is not finite.
// Out of line: inlined, it and its sincos push the common path out of the instruction cache (8192 tokens of
// 32 + 32 + 32 heads and their read-back 398 us against 236).
constexpr float kAppendMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
constexpr uint32_t kAppendMagicBits = 0x4b400000u;

static __device__ __noinline__ float append_exact(const float* v, uint32_t* y, int lanes, float kL, bool turn, int pos,
                                                  const double* inv_freq) {
  double xd[8];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) xd[e] = (double)v[e], bad |= !(fabsf(v[e]) < INFINITY);
  if (turn) {
#pragma unroll 1
    for (int e = 0; e < 4; ++e) {
      double s, c;
      sincospi(2.0 * rope_part(pos, inv_freq[e]), &s, &c);
      const double x0 = (double)v[e], x1 = (double)v[4 + e];
      xd[e] = x0 * c - x1 * s;
      xd[4 + e] = x0 * s + x1 * c;
    }
  }
  double gd = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) gd = fmax(gd, fabs(xd[e]));
  for (int o = lanes / 2; o >= 1; o >>= 1) {
    gd = fmax(gd, __shfl_xor_sync(0xffffffffu, gd, o));
    bad |= __shfl_xor_sync(0xffffffffu, (int)bad, o) != 0;
  }
  const double L = (double)kL;
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {
    // a zero is L/2 whatever the rounding of L gamma
    const double code = gd > 0.0 && xd[e] != 0.0 ? rint((L * xd[e] + L * gd) / (2.0 * gd)) : rint(0.5 * L);
    y[e] = kAppendMagicBits + (bad ? 0u : (uint32_t)fmin(fmax(code, 0.0), L));
  }
  return bad ? NAN : (float)gd;
}

// One CTA takes 16 tokens and a range of heads, counted through Q, K and V; a warp takes 256 / D heads
// of them at a time, through all the tokens. D / 8 lanes hold a head: lane s features 4s .. 4s+3 and
// D/2 + 4s .. D/2 + 4s + 3, which are each other's RoPE partners, so the rotation needs no exchange
// between lanes. Quantised codes are staged in the warp's shared memory as bit strings (four codes to a
// pack) and stored by lanes that take consecutive tokens of one V unit, so that tokens which follow one
// another in the cache leave as whole sectors.
//
// A code is decided in fp32 unless the value lies within kNear of a .5 boundary, where L 2^-21 bounds
// the error, in steps of 2^-23 L: 1.35 from the rotation and as much from gamma (cosine and sine off by
// 1.5 2^-24, two roundings, of states up to sqrt(2) gamma), 0.75 from the reciprocal (one step) and its product,
// 0.5 from the last sum, together 3.95 of 4. There the whole head is rotated, its gamma taken and its codes decided
// in fp64, from the same angle (rope_part), so that the codes are those of a 64-bit evaluation at any position. A
// lane's eight values go two at a time through the multiply-adds. No unit is full
// (issue 54%, DRAM 21%): it waits for its states (4.3 long-scoreboard stalls an issue, two tokens of 16 bytes a lane
// in flight). 8192 tokens of 32 + 32 + 32 heads of 128 at three bits 115 us for 322 MB, 2.8 TB/s.
template <int D, int BITS, bool ROPE>
__global__ void __launch_bounds__(kv_append_threads(D, BITS), 4) kv_append_kernel(const KvAppendArgs a) {
  using Rec = KvRec<D, BITS>;
  using Pack = KvPack<BITS>;
  constexpr int HALF = D / 2;
  constexpr int LPH = D / 8;        // lanes per head
  constexpr int HPW = 32 / LPH;     // heads per warp
  constexpr int THREADS = kv_append_threads(D, BITS), WARPS = THREADS / 32;
  constexpr int AHEAD = 2;          // tokens whose states are in flight behind the current one's
  constexpr uint32_t kCode = (1u << BITS) - 1u;
  constexpr float kL = (float)kCode;
  constexpr float kMagic = kAppendMagic;
  constexpr float kNear = kL * 4.76837158203125e-7f;
  constexpr int PACKS = D / 4;
  __shared__ float cs[ROPE ? kAppendTokens : 1][HALF], sn[ROPE ? kAppendTokens : 1][HALF];
  __shared__ double inv_freq[ROPE ? HALF : 1];
  __shared__ __align__(16) Pack packs[WARPS][HPW][kAppendTokens][PACKS];
  __shared__ float gammas[WARPS][HPW][kAppendTokens];
  __shared__ long long tok_base[kAppendTokens];  // byte offset of head 0's record; negative: not written
  __shared__ int tok_row[kAppendTokens];         // within it

  const int t0 = blockIdx.x * kAppendTokens;
  const int nt = a.T - t0 < kAppendTokens ? a.T - t0 : kAppendTokens;
  const int Hkv = a.c.Hkv, Hall = a.Hq + 2 * Hkv;
  const int h_begin = blockIdx.y * a.heads_per_cta;
  const int h_end = h_begin + a.heads_per_cta < Hall ? h_begin + a.heads_per_cta : Hall;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPH, hsub = lane / LPH;
  const int per_page = a.c.page_size / kKvChunk;
  const bool turn = ROPE && h_begin < a.Hq + Hkv;

  if (ROPE && turn) {
    // (exp(-2f / D log theta) would multiply the logarithm's rounding by up to its argument)
    for (int f = threadIdx.x; f < HALF; f += THREADS) inv_freq[f] = pow((double)a.theta, -2.0 * (double)f / (double)D);
  }
  pdl_wait();  // the states may come from the kernel before this one
  pdl_launch_dependents();
  if (threadIdx.x < kAppendTokens) {
    long long base = -1;
    int row = 0;
    if (threadIdx.x < nt) {
      const int s = a.slots[t0 + threadIdx.x];
      if (s >= 0) {
        const int page = s / a.c.page_size;
        row = s % a.c.page_size;
        if (page < a.c.num_pages) base = ((long long)page * Hkv * per_page + row / kKvChunk) * Rec::kBytes;
        else raise_error(kErrBadIndex);
      }
    }
    tok_base[threadIdx.x] = base;
    tok_row[threadIdx.x] = row % kKvChunk;
  }
  if constexpr (ROPE) {
    if (turn) {
      __syncthreads();
      for (int e = threadIdx.x; e < nt * HALF; e += THREADS) {
        const int t = e / HALF, f = e % HALF;
        rope_cs(a.pos[t0 + t], inv_freq[f], cs[t][f], sn[t][f]);
      }
    }
  }
  __syncthreads();

  for (int hb = h_begin + warp * HPW; hb < h_end; hb += WARPS * HPW) {
    const bool live = hb + hsub < h_end;
    const int h = live ? hb + hsub : hb;
    const int kind = h < a.Hq ? 0 : h < a.Hq + Hkv ? 1 : 2;
    const int hk = h - (kind == 0 ? 0 : kind == 1 ? a.Hq : a.Hq + Hkv);
    const size_t stride = kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride;
    const uint16_t* x = (kind == 0 ? a.Q : kind == 1 ? a.K : a.V) + (size_t)t0 * stride + (size_t)hk * D + 4 * sub;
    uint16_t* q_out = a.q_out + (size_t)t0 * a.qo_stride + (size_t)hk * D + 4 * sub;
    const bool any_kv = hb + HPW > a.Hq;  // of the warp's heads
    uint2 lo[AHEAD], hi[AHEAD];
    auto load = [&](int t, uint2& l, uint2& u) {
      t = t < nt ? t : nt - 1;
      l = __ldcs(reinterpret_cast<const uint2*>(x + (size_t)t * stride));  // read once
      u = __ldcs(reinterpret_cast<const uint2*>(x + (size_t)t * stride + HALF));
    };
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load(u, lo[u], hi[u]);
#pragma unroll 1
    for (int t = 0; t < nt; ++t) {
      const uint2 l0 = lo[0], h0 = hi[0];
#pragma unroll
      for (int u = 0; u + 1 < AHEAD; ++u) lo[u] = lo[u + 1], hi[u] = hi[u + 1];
      load(t + AHEAD, lo[AHEAD - 1], hi[AHEAD - 1]);
      {
        const float v[8] = {__uint_as_float(l0.x << 16), __uint_as_float(l0.x & 0xffff0000u),
                            __uint_as_float(l0.y << 16), __uint_as_float(l0.y & 0xffff0000u),
                            __uint_as_float(h0.x << 16), __uint_as_float(h0.x & 0xffff0000u),
                            __uint_as_float(h0.y << 16), __uint_as_float(h0.y & 0xffff0000u)};
        F2 w2[4] = {F2(v[0], v[1]), F2(v[2], v[3]), F2(v[4], v[5]), F2(v[6], v[7])};
        if constexpr (ROPE) {
          if (kind < 2) {
            const float4 c4 = *reinterpret_cast<const float4*>(&cs[t][4 * sub]);
            const float4 s4 = *reinterpret_cast<const float4*>(&sn[t][4 * sub]);
            const F2 c[2] = {F2(c4.x, c4.y), F2(c4.z, c4.w)}, s[2] = {F2(s4.x, s4.y), F2(s4.z, s4.w)};
            const F2 n[2] = {F2(-s4.x, -s4.y), F2(-s4.z, -s4.w)};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const F2 x0 = w2[e], x1 = w2[2 + e];
              w2[e] = fma2(x1, n[e], mul2(x0, c[e]));
              w2[2 + e] = fma2(x0, s[e], mul2(x1, c[e]));
            }
          }
        }
        float w[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) w2[e].split(w[2 * e], w[2 * e + 1]);
        if (kind == 0 && live) {
          uint16_t* o = q_out + (size_t)t * a.qo_stride;
          *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(w[0], w[1]), pack_bf16(w[2], w[3]));
          *reinterpret_cast<uint2*>(o + HALF) = make_uint2(pack_bf16(w[4], w[5]), pack_bf16(w[6], w[7]));
        }
        if (!any_kv) continue;
        float g = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) g = max_nan(g, fabsf(w[e]));
#pragma unroll
        for (int o = LPH / 2; o >= 1; o >>= 1) g = max_nan(g, __shfl_xor_sync(0xffffffffu, g, o));
        const float mult = g > 0.f ? 0.5f * kL * rcp_approx(g) : 0.f;
        uint32_t y[8];  // the code plus the magic bits
        float d[8], far = 0.f;
        const F2 mult2(mult, mult), half2(0.5f * kL, 0.5f * kL), magic2(kMagic, kMagic), minus2(-1.f, -1.f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const F2 tt = fma2(w2[e], mult2, half2), r = add2(tt, magic2);
          float r0, r1;
          r.split(r0, r1);
          y[2 * e] = __float_as_uint(r0);
          y[2 * e + 1] = __float_as_uint(r1);
          add2(tt, fma2(r, minus2, magic2)).split(d[2 * e], d[2 * e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) far = fmaxf(far, fabsf(d[e]));
        // in range, or the products may leave fp32's; a NaN or an infinity is not
        const bool range = g == 0.f || (g > 1e-30f && g < 1e30f);
        bool near = kind != 0 && !(range && far <= 0.5f - kNear);
        if (near) {
          // A zero is L/2 exactly, which the fp32 rounding takes to the even code: no border case,
          // unless it comes from a rotation that cancelled. A state that was not rotated lies on the border
          // above code k where L x = (2k + 1 - L) gamma, and bf16 values often do (for three bits whenever
          // gamma's significand divides by 7): both sides are exact in fp32. Left for 64 bits is the
          // border of code L/2 with a state so small that 64 bits may round it away.
          const bool turned = ROPE && kind < 2;
          near = !range;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool zero = v[e] == 0.f && (!turned || v[e ^ 4] == 0.f);
            if (zero || fabsf(d[e]) <= 0.5f - kNear) continue;
            const float tt = fmaf(w[e], mult, 0.5f * kL);
            const float k = rintf(tt - 0.5f), border = 2.f * k + 1.f - kL;
            if (turned || border == 0.f) {
              near = true;
            } else {
              const float at = kL * v[e] - border * g;
              const float odd = k - 2.f * floorf(0.5f * k);
              y[e] = __float_as_uint(k + (at > 0.f || (at == 0.f && odd != 0.f) ? 1.f : 0.f) + kMagic);
            }
          }
        }
        const uint32_t nears = __ballot_sync(0xffffffffu, near);
        if (nears != 0u) {
          // once more in fp64: the heads that need it, and no other (whose gamma could differ in its last bits, so
          // that a token's record depended on the heads that share its warp)
          constexpr uint32_t kHead = 0xffffffffu >> (32 - LPH);  // the lanes of the first head
          const bool again = (nears & (kHead << (hsub * LPH))) != 0u;
          float vs[8];
          uint32_t ys[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) vs[e] = v[e];
          const float ge = append_exact(vs, ys, LPH, kL, ROPE && kind < 2, ROPE ? a.pos[t0 + t] : 0,
                                        inv_freq + (ROPE ? 4 * sub : 0));
          if (again) {
            g = ge;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = ys[e];
          }
        }
        // four codes side by side: the sums of the magic bits wrap to a constant
        constexpr uint32_t kSum = kAppendMagicBits * (1u + (1u << BITS) + (1u << (2 * BITS)) + (1u << (3 * BITS)));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t* c = y + 4 * half;
          packs[warp][hsub][t][half * (PACKS / 2) + sub] =
              (Pack)(c[0] - kSum + (c[1] << BITS) + (c[2] << (2 * BITS)) + (c[3] << (3 * BITS)));
        }
        if (sub == 0) gammas[warp][hsub][t] = g;
      }
    }
    if (!any_kv) continue;
    __syncwarp();
    // store the heads: a lane takes 32 codes of a K row, or 16 codes of V, and first a scale
    constexpr int KG = D / 32, VG = D / 16;
    for (int hl = 0; hl < HPW && hb + hl < h_end; ++hl) {
      const int hh = hb + hl;
      if (hh < a.Hq) continue;
      const bool is_k = hh < a.Hq + Hkv;
      uint8_t* base = a.c.base + (size_t)(hh - a.Hq - (is_k ? 0 : Hkv)) * per_page * Rec::kBytes;
      if (lane < nt && tok_base[lane] >= 0)
        reinterpret_cast<float*>(base + tok_base[lane] + (is_k ? Rec::kGammaK : Rec::kGammaV))[tok_row[lane]] =
            gammas[warp][hl][lane];
      if (is_k) {
        for (int i = lane; i < nt * KG; i += 32) {
          const int t = i / KG, g = i % KG;
          if (tok_base[t] < 0) continue;
          const Pack* p = &packs[warp][hl][t][g * 8];
          uint8_t* out = base + tok_base[t] + tok_row[t] * Rec::kRow + g * 4 * BITS;
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
            for (int j = 0; j < 4; ++j) s24[j] = (pw[j] & 0xfffu) | ((pw[j] >> 4) & 0xfff000u);
            const uint32_t hw[6] = {s24[0] & 0x7fffu,  // codes 0-4, 5-9, ...
                                    (s24[0] >> 15) | ((s24[1] & 0x3fu) << 9),
                                    (s24[1] >> 6) & 0x7fffu,
                                    (s24[1] >> 21) | ((s24[2] & 0xfffu) << 3),
                                    (s24[2] >> 12) | ((s24[3] & 7u) << 12),
                                    (s24[3] >> 3) & 0x7fffu};
            const uint32_t c30 = (s24[3] >> 18) & 7u, c31 = s24[3] >> 21;
            uint32_t* o = reinterpret_cast<uint32_t*>(out);
#pragma unroll
            for (int j = 0; j < 3; ++j)
              o[j] = hw[2 * j] | (((c30 >> j) & 1u) << 15) | (hw[2 * j + 1] << 16) | (((c31 >> j) & 1u) << 31);
          }
        }
      } else {
        const int t = lane % kAppendTokens;
        if (t < nt && tok_base[t] >= 0) {
          uint16_t* out0 = reinterpret_cast<uint16_t*>(base + tok_base[t] + Rec::kV) + tok_row[t];
#pragma unroll
          for (int g0 = 0; g0 < VG; g0 += 2) {
            const int g = g0 + lane / kAppendTokens;
            const Pack* p = &packs[warp][hl][t][g * 4];
            uint16_t* out = out0 + g * BITS * 16;
            if constexpr (BITS == 3) {
              const uint2 w2 = *reinterpret_cast<const uint2*>(p);
              const uint32_t a24 = (w2.x & 0xfffu) | ((w2.x >> 4) & 0xfff000u), b24 = (w2.y & 0xfffu) | ((w2.y >> 4) & 0xfff000u);
              const uint32_t c15 = b24 >> 21;
              out[0] = (uint16_t)((a24 & 0x7fffu) | ((c15 & 1u) << 15));
              out[16] = (uint16_t)((a24 >> 15) | ((b24 & 0x3fu) << 9) | ((c15 & 2u) << 14));
              out[32] = (uint16_t)(((b24 >> 6) & 0x7fffu) | ((c15 & 4u) << 13));
            } else {
              const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
              for (int j = 0; j < BITS; ++j) out[16 * j] = u[j];
            }
          }
        }
      }
    }
    __syncwarp();
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
constexpr int kGatherHeads = 2;  // of a CTA at a time

// 32 codes of K in the words w (as they lie) or of V in w (its units paired to words), as bf16 pairs of
// (2u - L) step. A code at bit p >= 1 of a word, with the bits of 2^23 above it, is the float 2^23 + u 2^p;
// one multiply-add takes that to 2u - L exactly.
template <int BITS, bool IS_V>
__device__ __forceinline__ void kv_values(const uint32_t (&w)[BITS], float step, uint32_t (&out)[16]) {
  constexpr uint32_t kCode = (1u << BITS) - 1u;
  constexpr int PER = BITS == 3 ? 5 : 16 / BITS;  // codes of a half-word
  auto value = [&](uint32_t x, int p) {           // the code at bit p of x
    const float f = __uint_as_float((x & (kCode << p)) | 0x4b000000u);
    return fmaf(f, 2.f / (float)(1u << p), -(16777216.f / (float)(1u << p) + (float)kCode)) * step;
  };
  float v[32];
#pragma unroll
  for (int i = 0; i < BITS; ++i) {
    const uint32_t low = w[i] << 1, high = w[i] >> 15;
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int c = 0; c < PER; ++c) {
        const int hw = 2 * i + half;
        const int at = BITS != 3 ? hw * PER + c : IS_V ? hw / 3 * 16 + hw % 3 * 5 + c : hw * 5 + c;
        v[at] = value(half ? high : low, BITS * c + 1);
      }
  }
  if constexpr (BITS == 3) {
    // the codes left over, their bits in the bits 15 of K's even and odd half-words (of each three V units)
    uint32_t first, second;
    if (IS_V) {
      first = ((w[0] >> 14) & 2u) | ((w[0] >> 29) & 4u) | ((w[1] >> 12) & 8u);
      second = ((w[1] >> 30) & 2u) | ((w[2] >> 13) & 4u) | ((w[2] >> 28) & 8u);
    } else {
      first = ((w[0] >> 14) & 2u) | ((w[1] >> 13) & 4u) | ((w[2] >> 12) & 8u);
      second = ((w[0] >> 30) & 2u) | ((w[1] >> 29) & 4u) | ((w[2] >> 28) & 8u);
    }
    v[IS_V ? 15 : 30] = value(first, 1);
    v[31] = value(second, 1);
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) out[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
}

// 32 bytes in one store.
__device__ __forceinline__ void store_32(uint16_t* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// x~ = (2u - L) gamma / L, rounded to bf16. One CTA takes 16 tokens and passes their heads two at a time; a
// thread takes 32 features of K or of V of one token, the lanes consecutive tokens, so that V's interleaved
// units are read as whole sectors and every thread writes two. It writes 4 D bytes for D b / 4 + 8 read, and what
// it waits for are its reads (7.9 long-scoreboard stalls an issue, 1.9 of a full load-store queue; DRAM at 39% of
// its peak in a single cold call): 12.5 k tokens of 32 heads of 128 at three bits 57 us, 4.7 TB/s.
template <int D, int BITS>
__global__ void __launch_bounds__(kGatherHeads * 2 * kGatherTokens * D / 32) kv_gather_kernel(const KvGatherArgs a) {
  using Rec = KvRec<D, BITS>;
  constexpr int G = D / 32;
  constexpr float kL = (float)((1 << BITS) - 1);
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * kGatherTokens + threadIdx.x % kGatherTokens;
  const int g = threadIdx.x / kGatherTokens % G, which = threadIdx.x / (kGatherTokens * G) % 2;
  const int h0 = threadIdx.x / (kGatherTokens * G * 2) + blockIdx.y * kGatherHeads;
  uint16_t* out = which == 0 ? a.K : a.V;
  if (t >= a.T || out == nullptr) return;
  const int s = a.slots[t];
  if (s < 0) return;
  const int page = s / a.c.page_size, row = s % a.c.page_size;
  if (page >= a.c.num_pages) {
    raise_error(kErrBadIndex);
    return;
  }
  const int per_page = a.c.page_size / kKvChunk, i = row % kKvChunk;
  const uint8_t* rec0 = a.c.base + ((size_t)page * a.c.Hkv * per_page + row / kKvChunk) * (size_t)Rec::kBytes;
  // the next head's words are read before this one's values leave
  uint32_t next[BITS];
  float gamma = 0.f;
  auto read = [&](int h) {
    const uint8_t* rec = rec0 + (size_t)h * per_page * Rec::kBytes;
    gamma = reinterpret_cast<const float*>(rec + (which == 0 ? Rec::kGammaK : Rec::kGammaV))[i];
    if (which == 0) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(rec + i * Rec::kRow) + g * BITS;
#pragma unroll
      for (int e = 0; e < BITS; ++e) next[e] = p[e];
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(rec + Rec::kV) + 16 * (2 * g * BITS) + i;
#pragma unroll
      for (int e = 0; e < BITS; ++e) next[e] = (uint32_t)p[32 * e] | ((uint32_t)p[32 * e + 16] << 16);
    }
  };
  if (h0 < a.c.Hkv) read(h0);
  for (int h = h0; h < a.c.Hkv; h += kGatherHeads * gridDim.y) {
    uint32_t w[BITS], v[16];
    const float step = gamma / kL;
#pragma unroll
    for (int e = 0; e < BITS; ++e) w[e] = next[e];
    if (h + kGatherHeads * (int)gridDim.y < a.c.Hkv) read(h + kGatherHeads * gridDim.y);
    if (which == 0) kv_values<BITS, false>(w, step, v);
    else kv_values<BITS, true>(w, step, v);
    uint16_t* dst = out + ((size_t)t * a.c.Hkv + h) * D + 32 * g;
    if ((reinterpret_cast<uintptr_t>(out) & 31u) == 0) {
      store_32(dst, v);
      store_32(dst + 16, v + 8);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        reinterpret_cast<uint4*>(dst)[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
    }
  }
}

}  // namespace hbl
