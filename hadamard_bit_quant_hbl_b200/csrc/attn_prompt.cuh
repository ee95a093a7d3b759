// Attention over packed prompts with grouped heads:
//
//   query i of a sequence with nq queries and nk keys sees keys j <= i + nk - nq (causal) or all,
//   p = softmax(scale q . k),   o = sum_j p_j v_j
#pragma once

#include "common.cuh"
#include "kv_cache.cuh"

namespace hbl {

constexpr int kPromptMaxB = 4096;  // sequences of one call

struct PromptAttnArgs {
  const uint16_t *Q, *K, *V;  // bf16 rows; head h of token t at t * stride + h * D
  size_t q_stride, k_stride, v_stride;
  const int32_t *cu_q, *cu_k;  // [B + 1]
  int B, total_q, total_k, max_q, Hq, Hkv;
  float scale;
  int causal;
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

// One warp per (query, head); a lane holds a key's score, then lane l features l, l + 32, ... of V.
template <int D>
__global__ void __launch_bounds__(128) attn_prompt_kernel(const PromptAttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float qs[4][D];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int i = blockIdx.x * 4 + warp, h = blockIdx.y, hk = h / (a.Hq / a.Hkv);
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
      int nq, nk, q0, k0;
      if (!prompt_borders(a, b, q0, nq, k0, nk) || nq > a.max_q) raise_error(kErrBadIndex);
    }
  if (i >= a.total_q) return;
  int lo = 0, hi = a.B;  // the sequence: the last b with cu_q[b] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.cu_q[mid] <= i) lo = mid; else hi = mid;
  }
  int q0, nq, k0, nk;
  if (!prompt_borders(a, lo, q0, nq, k0, nk) || i < q0 || i >= q0 + nq || i - q0 >= a.max_q) return;
  int seen = a.causal ? i - q0 + 1 + nk - nq : nk;
  seen = seen < 0 ? 0 : seen > nk ? nk : seen;
  for (int d = lane; d < D; d += 32)
    qs[warp][d] = __uint_as_float((uint32_t)a.Q[(size_t)i * a.q_stride + (size_t)h * D + d] << 16);
  __syncwarp();
  float o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int j0 = 0; j0 < seen; j0 += 32) {
    const int j = j0 + lane;
    float s = -INFINITY;
    if (j < seen) {
      const uint4* k = reinterpret_cast<const uint4*>(a.K + (size_t)(k0 + j) * a.k_stride + (size_t)hk * D);
      s = 0.f;
      for (int d = 0; d < D; d += 8) {
        const uint4 u = k[d / 8];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s = fmaf(qs[warp][d + 2 * e], __uint_as_float(w[e] << 16), s);
          s = fmaf(qs[warp][d + 2 * e + 1], __uint_as_float(w[e] & 0xffff0000u), s);
        }
      }
      s *= a.scale;
    }
    float mx = s;
#pragma unroll
    for (int x = 16; x >= 1; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
    const float mn = fmaxf(m, mx);
    const float f = expf(m - mn), p = expf(s - mn);
    m = mn;
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
    const int n = seen - j0 < 32 ? seen - j0 : 32;
    for (int t = 0; t < n; ++t) {
      const float pt = __shfl_sync(0xffffffffu, p, t);
      const uint16_t* v = a.V + (size_t)(k0 + j0 + t) * a.v_stride + (size_t)hk * D;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(pt, __uint_as_float((uint32_t)v[lane + 32 * e] << 16), o[e]);
    }
  }
#pragma unroll
  for (int x = 16; x >= 1; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t ih = (size_t)i * a.Hq + h;
#pragma unroll
  for (int e = 0; e < E; ++e) a.O[ih * D + lane + 32 * e] = (uint16_t)(pack_bf16(o[e] * inv, 0.f) & 0xffffu);
  if (a.lse && lane == 0) a.lse[ih] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace hbl
