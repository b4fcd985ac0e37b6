// Attention over the 8-bit paged key-value cache.
//
// Row i of sequence b stands at position p = kv_len - n + i and sees the cached tokens
// j in [max(0, p - window + 1), p] (causal) or [0, kv_len):
//   o = sum_j softmax_j(scale q . k_j) v_j,   k_j = (byte - 128) * k_scale[page], v_j alike,
// one pass with a running maximum m and sum l (fp32); no visible token gives o = 0 and lse = -inf.
//
// This is the plain kernel: one warp for a row and query head.
#include <cuda_runtime.h>

#include "internal.h"
#include "kv8.cuh"
#include "kv8.h"

namespace w8a8 {

struct AttnParams {
  Kv8Step step;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  long long q_stride, out_stride;
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  int pages, page_tokens, q_heads, kv_heads, window, causal;
  float scale;
  uint32_t* status;
};

template <bool kF16, int D>
__global__ void __launch_bounds__(32) kv8_attention_kernel(const __grid_constant__ AttnParams p) {
  pdl_trigger();
  pdl_wait();
  constexpr int E = D / 32;   // values a lane holds
  const int lane = threadIdx.x;
  const int i = blockIdx.x, b = blockIdx.y, qh = blockIdx.z;
  Seq s;
  if (!load_seq(p.step, b, p.page_tokens, false, p.status, s) || i >= s.n) return;
  const int h = qh / (p.q_heads / p.kv_heads);
  const int pos = s.len - s.n + i;
  const int end = p.causal ? pos + 1 : s.len;
  const int begin = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const uint16_t* q = p.q + (s.row0 + i) * p.q_stride + qh * D;
  float qv[E], o[E];
  for (int e = 0; e < E; ++e) {
    qv[e] = kF16 ? __half2float(__ushort_as_half(q[lane * E + e])) : __bfloat162float(__ushort_as_bfloat16(q[lane * E + e]));
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = begin; t < end; ++t) {
    const int page = __ldg(p.step.page_table + (size_t)b * p.step.table_width + t / p.page_tokens);
    if (page < 0 || page >= p.pages) {
      if (lane == 0) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
      continue;
    }
    const size_t at = (size_t)page * p.kv_heads + h;
    const size_t off = (at * p.page_tokens + t % p.page_tokens) * D + lane * E;
    float dot = 0.f;
    for (int e = 0; e < E; ++e) dot = fmaf(qv[e], (float)((int)p.kc[off + e] - 128), dot);
    for (int x = 16; x > 0; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
    const float sc = dot * p.ks[at] * p.scale;
    const float mn = fmaxf(m, sc);
    const float a = expf(m - mn), w = expf(sc - mn);
    l = l * a + w;
    const float wv = w * p.vs[at];
    for (int e = 0; e < E; ++e) o[e] = fmaf(wv, (float)((int)p.vc[off + e] - 128), o[e] * a);
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  uint16_t* out = p.out + (s.row0 + i) * p.out_stride + qh * D;
  for (int e = 0; e < E; ++e) out[lane * E + e] = (uint16_t)pack2<kF16>(o[e] * inv, 0.f);
  if (p.lse && lane == 0) p.lse[(size_t)(s.row0 + i) * p.q_heads + qh] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace w8a8

using namespace w8a8;

extern "C" size_t kv8_workspace_bytes(int q_heads, int kv_heads, int head_dim) {
  if (kv8_check_dims(kv_heads, head_dim) != W8A8_OK || q_heads < 0 || q_heads > 4096) return 0;
  return kWsHeaderBytes;
}

extern "C" int kv8_attention(const kv8_cache_t* cache, const kv8_step_t* step, const void* q, long long q_stride, int q_heads,
                             void* out, long long out_stride, float* lse, float scale, int window, unsigned flags, int dtype,
                             void* ws, size_t ws_bytes, void* stream) {
  int rc = kv8_check_cache(cache);
  if (rc == W8A8_OK) rc = kv8_check_step(step, cache);
  if (rc != W8A8_OK) return rc;
  if (flags & ~(unsigned)KV8_FLAG_NOT_CAUSAL) return W8A8_ERR_INVALID_ARG;
  if ((dtype != KV8_BF16 && dtype != KV8_F16) || q_heads < 1 || q_heads > 4096 || q_heads % cache->kv_heads != 0 || window < 0 ||
      ((flags & KV8_FLAG_NOT_CAUSAL) && window > 0))
    return W8A8_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale <= 3.0e38f)) return W8A8_ERR_INVALID_ARG;
  if (step->tokens == 0) return W8A8_OK;   // an empty tensor has no address
  const int D = cache->head_dim;
  if ((rc = kv8_check_rows(q, q_stride, q_heads, D)) != W8A8_OK) return rc;
  if ((rc = kv8_check_rows(out, out_stride, q_heads, D)) != W8A8_OK) return rc;
  if (!kv8_aligned(lse, 4)) return W8A8_ERR_MISALIGNED;
  if ((rc = kv8_check_ws(ws, ws_bytes, kv8_workspace_bytes(q_heads, cache->kv_heads, D))) != W8A8_OK) return rc;
  AttnParams p{};
  p.step = kv8_step_of(*step);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.q_stride = q_stride, p.out_stride = out_stride;
  p.kc = static_cast<const uint8_t*>(cache->k);
  p.vc = static_cast<const uint8_t*>(cache->v);
  p.ks = cache->k_scale;
  p.vs = cache->v_scale;
  p.pages = cache->pages, p.page_tokens = cache->page_tokens, p.q_heads = q_heads, p.kv_heads = cache->kv_heads;
  p.window = window, p.causal = (flags & KV8_FLAG_NOT_CAUSAL) ? 0 : 1;
  p.scale = scale;
  p.status = static_cast<uint32_t*>(ws);
  const dim3 grid((unsigned)step->max_tokens, (unsigned)step->seqs, (unsigned)q_heads);
  const bool f16 = dtype == KV8_F16;
  auto kern = D == 64 ? (f16 ? kv8_attention_kernel<true, 64> : kv8_attention_kernel<false, 64>)
            : D == 128 ? (f16 ? kv8_attention_kernel<true, 128> : kv8_attention_kernel<false, 128>)
                       : (f16 ? kv8_attention_kernel<true, 256> : kv8_attention_kernel<false, 256>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "kv8_attention");
}
