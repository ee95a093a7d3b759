// C ABI of the low-bit key-value cache and of the attention over it (declared in include/hbl.h):
// argument checks, kernel selection and launches, as in hbl.cu.
#include <math.h>

#include "hbl.h"

#include "attn_decode.cuh"
#include "attn_prompt.cuh"
#include "common.cuh"
#include "host.cuh"
#include "kv_cache.cuh"

using namespace hbl;

hbl_status hbl::attn_take_errors(cudaStream_t s, int* flags) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(flags, g_error_flags, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e != cudaSuccess) return cuda_fail(e);
  e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return cuda_fail(e);
  if (*flags) {
    const int zero = 0;
    e = cudaMemcpyToSymbolAsync(g_error_flags, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e);
  }
  return HBL_OK;
}

namespace {

bool head_ok(int D, int bits) {
  return (D == 64 || D == 128 || D == 256) && (bits == 2 || bits == 3 || bits == 4 || bits == 8);
}

// f(std::integral_constant<int, D>, std::integral_constant<int, bits>) for a supported pair
template <typename F>
hbl_status for_head(int D, int bits, F f) {
  auto at_d = [&](auto d) {
    switch (bits) {
      case 2: return f(d, std::integral_constant<int, 2>());
      case 3: return f(d, std::integral_constant<int, 3>());
      case 4: return f(d, std::integral_constant<int, 4>());
      default: return f(d, std::integral_constant<int, 8>());
    }
  };
  if (D == 64) return at_d(std::integral_constant<int, 64>());
  if (D == 128) return at_d(std::integral_constant<int, 128>());
  return at_d(std::integral_constant<int, 256>());
}

// Checks of the cache's shape and buffer shared by the three calls that take one.
hbl_status check_cache(const void* cache, size_t cache_bytes, int num_pages, int page_size, int Hkv, int D, int bits) {
  if (!cache || num_pages < 1 || page_size < 1 || Hkv < 1 || D < 1 || bits < 1) return HBL_EINVAL;
  if (!head_ok(D, bits) || page_size % kKvChunk != 0 || Hkv > 65535) return HBL_EUNSUPPORTED;
  if ((long long)num_pages * page_size > 0x7fffffffll) return HBL_EUNSUPPORTED;
  if (!aligned(cache, 16) || cache_bytes < hbl_kv_cache_bytes(num_pages, page_size, Hkv, D, bits)) return HBL_EINVAL;
  return HBL_OK;
}

bool rows_ok(const void* X, size_t stride, int H, int D) {
  return X && aligned(X, 16) && stride >= (size_t)H * D && stride % 8 == 0;
}

KvCacheView view(const void* cache, int num_pages, int page_size, int Hkv) {
  return KvCacheView{static_cast<uint8_t*>(const_cast<void*>(cache)), num_pages, page_size, Hkv};
}

// Query heads that one pass over a KV head takes: up to 16 columns, 8 for 256 features (whose
// accumulators take as many registers); more heads in equal passes.
int decode_group(int G, int D) {
  const int most = D == 256 ? 8 : 16;
  const int passes = (G + most - 1) / most;
  return (G + passes - 1) / passes;
}

template <int D, int BITS, int NT, int R>
hbl_status launch_decode_attn(DecodeAttnArgs a, cudaStream_t s) {
  using Cfg = DecodeCfg<D, BITS, NT>;
  static SmemLimit lim;
  auto* k = attn_decode_kernel<D, BITS, NT, R>;
  const cudaError_t e = allow_smem(k, Cfg::kSmem, lim);
  if (e != cudaSuccess) return cuda_fail(e);
  // every CTA resident at once, and no more than the tables have room for
  const long long blocks = ((long long)a.table_width * a.c.page_size + Cfg::kBlock - 1) / Cfg::kBlock;
  const long long want = blocks * a.B * a.c.Hkv * a.groups;
  int grid = resident_ctas(k, 32 * kDecodeWarps, Cfg::kSmem, lim);
  if (grid > kDecodeMaxUnits / kDecodeWarps) grid = kDecodeMaxUnits / kDecodeWarps;
  if (want < grid) grid = (int)want;
  const hbl_status st = launch_pdl(k, dim3(grid), dim3(32 * kDecodeWarps), Cfg::kSmem, s, a);
  if (st != HBL_OK) return st;
  // Few heads have long chains: up to one CTA per SM, more threads read a chain's pieces at once. Whole calls with
  // 1024 and with 256 threads, 32 heads on 8 of 128, us: one sequence of 131072 tokens (32 CTAs) 39.7, 41.5; one
  // of 16 heads on 1 30.8, 57.1; four of 32768 (128) 39.2, 39.6; eight of 16384 (256) 42.3, 38.5; 64 of 4096 105.8,
  // 67.9. (One of 500, short chains: 10.5, 9.4; the lengths are known to the device alone.)
  const dim3 joins((unsigned)(a.B * a.c.Hkv * a.groups), a.group);
  int dev = 0;
  cudaGetDevice(&dev);
  return (long long)joins.x * joins.y <= device_sms(dev)
             ? launch_pdl(attn_decode_join_kernel<D, 1024>, joins, dim3(1024), 0, s, a)
             : launch_pdl(attn_decode_join_kernel<D, 256>, joins, dim3(256), 0, s, a);
}

// bf16 states [T][H][D] with rows `stride` elements apart, in boxes of 64 features, `heads` heads and
// `tokens` tokens, laid out in 128-byte swizzled rows.
bool make_map_rows(CUtensorMap* map, const void* base, size_t stride, int T, int H, int D, int heads, int tokens) {
  auto enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)D * 2u, (cuuint64_t)stride * 2u};
  const cuuint32_t box[3] = {64u, (cuuint32_t)heads, (cuuint32_t)tokens};
  const cuuint32_t estr[3] = {1u, 1u, 1u};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int D>
hbl_status launch_prompt(const PromptAttnArgs& a, cudaStream_t s) {
  using Cfg = PromptCfg<D>;
  static SmemLimit lim;
  auto* k = attn_prompt_kernel<D>;
  const cudaError_t e = allow_smem(k, Cfg::kSmem, lim);
  if (e != cudaSuccess) return cuda_fail(e);
  if (Cfg::kTiles == 2) {
    // the kernel hands registers from some warps to others, which needs the launch to bring them all
    static const int regs = [k] {
      cudaFuncAttributes at;
      return cudaFuncGetAttributes(&at, k) == cudaSuccess ? at.numRegs : 0;
    }();
    if (regs != Cfg::kRegisters) return HBL_EUNSUPPORTED;
  }
  CUtensorMap mq, mk, mv;
  if (!make_map_rows(&mq, a.Q, a.q_stride, a.total_q, a.Hq, D, a.pack, 128 / a.pack)) return HBL_ECUDA;
  if (a.total_k > 0) {
    if (!make_map_rows(&mk, a.K, a.k_stride, a.total_k, a.Hkv, D, 1, Cfg::kKeys)) return HBL_ECUDA;
    if (!make_map_rows(&mv, a.V, a.v_stride, a.total_k, a.Hkv, D, 1, Cfg::kKeys)) return HBL_ECUDA;
  } else {
    mk = mv = mq;  // never read: there is no key block
  }
  // as many tile pairs as the borders could ask for, whatever they are
  const long long tokens = (long long)Cfg::kTiles * 128 / a.pack;
  long long tiles = a.total_q / tokens + a.B;
  const long long bound = (long long)a.B * ((a.max_q + tokens - 1) / tokens);
  if (bound < tiles) tiles = bound;
  long long grid = tiles * a.Hkv * a.groups;
  if (grid == 0) grid = 1;  // max_q = 0: the first CTA flags the sequences that have queries
  if (grid > 0x7fffffffll) return HBL_EUNSUPPORTED;
  return launch_pdl(k, dim3((unsigned)grid), dim3(Cfg::kThreads), Cfg::kSmem, s, mq, mk, mv, a);
}

}  // namespace

extern "C" {

size_t hbl_kv_cache_bytes(int num_pages, int page_size, int Hkv, int D, int bits) {
  if (num_pages <= 0 || page_size <= 0 || Hkv <= 0 || D <= 0 || bits <= 0) return 0;
  return (size_t)num_pages * Hkv * (page_size / kKvChunk) * kv_record_bytes(D, bits);
}

hbl_status hbl_kv_append(const void* Q, size_t q_stride, const void* K, size_t k_stride, const void* V, size_t v_stride,
                         const int32_t* pos, const int32_t* slots, float rope_theta, int T, int Hq, int Hkv, int D,
                         int bits, void* cache, size_t cache_bytes, int num_pages, int page_size, void* q_out,
                         size_t qo_stride, hbl_stream_t stream) {
  const hbl_status st = check_cache(cache, cache_bytes, num_pages, page_size, Hkv, D, bits);
  if (st != HBL_OK) return st;
  if (T < 0 || Hq < 0) return HBL_EINVAL;
  if (pos && !(rope_theta > 1.f && rope_theta < 3.0e38f)) return HBL_EINVAL;
  if (T == 0) return HBL_OK;
  if (!slots || !aligned(slots, 4) || (pos && !aligned(pos, 4))) return HBL_EINVAL;
  if (!rows_ok(K, k_stride, Hkv, D) || !rows_ok(V, v_stride, Hkv, D)) return HBL_EINVAL;
  if (Hq > 0 && (!rows_ok(Q, q_stride, Hq, D) || !rows_ok(q_out, qo_stride, Hq, D))) return HBL_EINVAL;
  if (Hq > 0 && Q == q_out && q_stride != qo_stride) return HBL_EINVAL;
  KvAppendArgs a;
  a.Q = static_cast<const uint16_t*>(Q);
  a.K = static_cast<const uint16_t*>(K);
  a.V = static_cast<const uint16_t*>(V);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.pos = pos;
  a.slots = slots;
  a.theta = rope_theta;
  a.T = T;
  a.Hq = Hq;
  a.c = view(cache, num_pages, page_size, Hkv);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.qo_stride = qo_stride;
  const int tiles = (T + kAppendTokens - 1) / kAppendTokens;
  const int heads = Hq + 2 * Hkv;
  // a CTA takes more heads (and builds the table of angles for more of them) as far as the tiles
  // alone fill the device several times over
  int dev = 0;
  cudaGetDevice(&dev);
  const int per_pass = kv_append_threads(D, bits) / 32 * (256 / D);  // heads that a CTA's warps take at once
  const int passes = (heads + per_pass - 1) / per_pass;
  const int want = 8 * device_sms(dev) / tiles;
  if (want <= passes) {
    a.heads_per_cta = (passes + want - 1) / (want < 1 ? 1 : want) * per_pass;
    if (want < 1) a.heads_per_cta = passes * per_pass;
  } else {  // few tokens: fewer heads than the warps could take, for the time of one pass
    a.heads_per_cta = (heads + want - 1) / want;
    if (a.heads_per_cta < 256 / D) a.heads_per_cta = 256 / D;
  }
  const int groups = (heads + a.heads_per_cta - 1) / a.heads_per_cta;
  const dim3 grid(tiles, groups);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return for_head(D, bits, [&](auto d, auto b) {
    return pos ? launch_pdl(kv_append_kernel<d(), b(), true>, grid, dim3(kv_append_threads(d(), b())), 0, s, a)
               : launch_pdl(kv_append_kernel<d(), b(), false>, grid, dim3(kv_append_threads(d(), b())), 0, s, a);
  });
}

hbl_status hbl_kv_gather(const void* cache, size_t cache_bytes, int num_pages, int page_size, const int32_t* slots,
                         int T, int Hkv, int D, int bits, void* K, void* V, hbl_stream_t stream) {
  const hbl_status st = check_cache(cache, cache_bytes, num_pages, page_size, Hkv, D, bits);
  if (st != HBL_OK) return st;
  if (T < 0) return HBL_EINVAL;
  if (T == 0) return HBL_OK;
  if (!slots || !aligned(slots, 4) || (!K && !V) || !aligned(K, 16) || !aligned(V, 16)) return HBL_EINVAL;
  KvGatherArgs a;
  a.c = view(cache, num_pages, page_size, Hkv);
  a.slots = slots;
  a.T = T;
  a.K = static_cast<uint16_t*>(K);
  a.V = static_cast<uint16_t*>(V);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return for_head(D, bits, [&](auto d, auto b) {
    // a CTA takes more heads (and finds its tokens' records for them) as far as the tokens alone fill
    // the device
    const int tiles = (T + kGatherTokens - 1) / kGatherTokens, pairs = (Hkv + kGatherHeads - 1) / kGatherHeads;
    int dev = 0;
    cudaGetDevice(&dev);
    const int want = 16 * device_sms(dev) / tiles;
    return launch_pdl(kv_gather_kernel<d(), b()>, dim3(tiles, want < 1 ? 1 : want < pairs ? want : pairs),
                      dim3(kGatherHeads * 2 * kGatherTokens * d() / 32), 0, s, a);
  });
}

size_t hbl_attn_decode_workspace(int B, int Hq, int Hkv, int D) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || Hq % Hkv != 0) return 0;
  const int G = Hq / Hkv, group = decode_group(G, D), groups = (G + group - 1) / group;
  return round_up((size_t)B * Hkv * groups * sizeof(DecodeChain) +
                      (size_t)kDecodeMaxUnits * 2 * group * (D + 4) * sizeof(float),
                  256);
}

hbl_status hbl_attn_decode(const void* Q, size_t q_stride, const void* cache, size_t cache_bytes, int num_pages,
                           int page_size, const int32_t* tables, int table_width, const int32_t* lens, int B, int Hq,
                           int Hkv, int D, int bits, float scale, void* workspace, size_t ws_bytes, void* O, float* lse,
                           hbl_stream_t stream) {
  const hbl_status st = check_cache(cache, cache_bytes, num_pages, page_size, Hkv, D, bits);
  if (st != HBL_OK) return st;
  if (B < 0 || Hq < 1 || Hq % Hkv != 0 || table_width < 1 || !isfinite(scale)) return HBL_EINVAL;
  if (B > kDecodeMaxB || Hq > 65535 || (long long)table_width * page_size > 0x7fffffffll) return HBL_EUNSUPPORTED;
  if (B == 0) return HBL_OK;
  if (!rows_ok(Q, q_stride, Hq, D) || !tables || !aligned(tables, 4) || !lens || !aligned(lens, 4)) return HBL_EINVAL;
  if (!O || !aligned(O, 16) || (lse && !aligned(lse, 4))) return HBL_EINVAL;
  if (!workspace || !aligned(workspace, 256) || ws_bytes < hbl_attn_decode_workspace(B, Hq, Hkv, D)) return HBL_EINVAL;
  DecodeAttnArgs a;
  a.Q = static_cast<const uint16_t*>(Q);
  a.q_stride = q_stride;
  a.c = view(cache, num_pages, page_size, Hkv);
  a.tables = tables;
  a.table_width = table_width;
  a.lens = lens;
  a.B = B;
  a.Hq = Hq;
  const int G = Hq / Hkv;
  a.group = decode_group(G, D);
  a.groups = (G + a.group - 1) / a.group;
  const int per_page = page_size / kKvChunk;
  a.page_shift = is_pow2(per_page) ? ilog2_c(per_page) : -1;
  a.scale = scale * 1.44269504088896340736f / (float)((1 << bits) - 1);
  a.O = static_cast<uint16_t*>(O);
  a.lse = lse;
  a.chains = static_cast<DecodeChain*>(workspace);
  a.ws = reinterpret_cast<float*>(a.chains + (size_t)B * Hkv * a.groups);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return for_head(D, bits, [&](auto d, auto b) {
    // groups of columns for as many chunks as the heads leave room for, and a block has
    constexpr int chunks = DecodeCfg<d(), b(), 1>::kChunks;
    if constexpr (d() <= 128) {
      if (a.group > 8) return launch_decode_attn<d(), b(), 2, 1>(a, s);
    }
    if constexpr (chunks >= 4) {
      if (a.group <= 2) return launch_decode_attn<d(), b(), 1, 4>(a, s);
    }
    if constexpr (chunks >= 2) {
      if (a.group <= 4) return launch_decode_attn<d(), b(), 1, 2>(a, s);
    }
    return launch_decode_attn<d(), b(), 1, 1>(a, s);
  });
}

hbl_status hbl_attn_prompt(const void* Q, size_t q_stride, const void* K, size_t k_stride, const void* V,
                           size_t v_stride, const int32_t* cu_q, const int32_t* cu_k, int B, int total_q, int total_k,
                           int max_q, int Hq, int Hkv, int D, float scale, int causal, void* O, float* lse,
                           hbl_stream_t stream) {
  if (B < 0 || total_q < 0 || total_k < 0 || max_q < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !isfinite(scale))
    return HBL_EINVAL;
  if (D < 1) return HBL_EINVAL;
  if ((D != 64 && D != 128 && D != 256) || B > kPromptMaxB || Hq > 65535) return HBL_EUNSUPPORTED;
  if (B == 0 || total_q == 0) return HBL_OK;
  if (!rows_ok(Q, q_stride, Hq, D) || !cu_q || !aligned(cu_q, 4) || !cu_k || !aligned(cu_k, 4)) return HBL_EINVAL;
  if (total_k > 0 && (!rows_ok(K, k_stride, Hkv, D) || !rows_ok(V, v_stride, Hkv, D))) return HBL_EINVAL;
  if (!O || !aligned(O, 16) || (lse && !aligned(lse, 4))) return HBL_EINVAL;
  PromptAttnArgs a;
  a.Q = static_cast<const uint16_t*>(Q);
  a.K = static_cast<const uint16_t*>(K);
  a.V = static_cast<const uint16_t*>(V);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.B = B;
  a.total_q = total_q;
  a.total_k = total_k;
  a.max_q = max_q;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.scale_log2 = scale == 0.f ? 1.f : fabsf(scale) * 1.44269504088896340736f;
  a.sign = scale > 0.f ? 1.f : scale < 0.f ? -1.f : 0.f;
  const int G = Hq / Hkv;
  a.pack = G & -G;  // the largest power of two that divides it
  if (a.pack > 128) a.pack = 128;
  a.groups = G / a.pack;
  a.causal = causal != 0;
  a.O = static_cast<uint16_t*>(O);
  a.lse = lse;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (D == 64) return launch_prompt<64>(a, s);
  if (D == 128) return launch_prompt<128>(a, s);
  return launch_prompt<256>(a, s);
}

}  // extern "C"
