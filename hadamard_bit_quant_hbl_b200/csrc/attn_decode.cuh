// Attention of one new token per sequence over the paged low-bit cache (kv_cache.cuh):
//
//   s_t = scale q . k~_t,   p = softmax(s) over t < len,   o = sum_t p_t v~_t
//
// with k~, v~ the values the cached codes stand for.
#pragma once

#include "common.cuh"
#include "kv_cache.cuh"

namespace hbl {

constexpr int kDecodeMaxB = 4096;  // sequences of one call

struct DecodeAttnArgs {
  const uint16_t* Q;  // bf16; sequence b, head h at b * q_stride + h * D
  size_t q_stride;
  KvCacheView c;
  const int32_t* tables;  // [B][table_width] page numbers
  int table_width;
  const int32_t* lens;  // [B]
  int B, Hq;
  float scale;
  uint16_t* O;  // bf16 [B][Hq][D]
  float* lse;   // [B][Hq] or nullptr
};

// One warp per (sequence, query head); lane l holds features l, l + 32, ...
template <int D, int BITS>
__global__ void __launch_bounds__(128) attn_decode_kernel(const DecodeAttnArgs a) {
  using Rec = KvRec<D, BITS>;
  constexpr int E = D / 32;
  constexpr float kL = (float)((1 << BITS) - 1);
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long bh = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (bh >= (long long)a.B * a.Hq) return;
  const int b = (int)(bh / a.Hq), h = (int)(bh % a.Hq), hk = h / (a.Hq / a.c.Hkv);
  const int per_page = a.c.page_size / kKvChunk;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)a.Q[(size_t)b * a.q_stride + (size_t)h * D + lane + 32 * e] << 16);
    o[e] = 0.f;
  }
  int len = a.lens[b];
  if (len < 0 || len > (long long)a.table_width * a.c.page_size) {
    raise_error(kErrBadIndex);
    len = len < 0 ? 0 : a.table_width * a.c.page_size;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < len; ++t) {
    const int page = a.tables[(size_t)b * a.table_width + t / a.c.page_size];
    if (page < 0 || page >= a.c.num_pages) {
      raise_error(kErrBadIndex);
      continue;
    }
    const int row = t % a.c.page_size, i = row % kKvChunk;
    const uint8_t* rec = a.c.base + (((size_t)page * a.c.Hkv + hk) * per_page + row / kKvChunk) * (size_t)Rec::kBytes;
    const float gk = reinterpret_cast<const float*>(rec + Rec::kGammaK)[i] / kL;
    const float gv = reinterpret_cast<const float*>(rec + Rec::kGammaV)[i] / kL;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], 2.f * (float)kv_k_code<D, BITS>(rec, i, lane + 32 * e) - kL, s);
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= gk * a.scale;
    const float mn = fmaxf(m, s);
    const float f = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e)
      o[e] = fmaf(p * gv, 2.f * (float)kv_v_code<D, BITS>(rec, i, lane + 32 * e) - kL, o[e] * f);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.O[(size_t)bh * D + lane + 32 * e] = (uint16_t)(pack_bf16(o[e] * inv, 0.f) & 0xffffu);
  if (a.lse && lane == 0) a.lse[bh] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace hbl
