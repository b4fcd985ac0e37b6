// kv8_attention: the entry point, its workspace, and the instances of the kernel for few query rows.
#include "kv8_attention_few.cuh"

namespace w8a8 {
namespace attn {

// Two parts for each CTA of the variant that needs most.
template <int D, int NT>
static size_t parts_of(int sms) {
  return (size_t)sms * Layout<D, NT>::kCtas * 2 * Layout<D, NT>::kPart * sizeof(float);
}
static size_t parts_bytes(int head_dim, int sms) {
  const size_t few = head_dim == 64 ? parts_of<64, 4>(sms) : head_dim == 128 ? parts_of<128, 4>(sms) : parts_of<256, 2>(sms), many = many_parts_bytes(head_dim, sms);
  return few > many ? few : many;
}

constexpr size_t counters_bytes(int sms) { return ((size_t)sms * 12 * sizeof(uint32_t) + 255) / 256 * 256; }

int check_call(const kv8_cache_t* cache, const kv8_step_t* step, const void* q, long long q_stride, int q_heads, const void* out,
               long long out_stride, const float* lse, float scale, int dtype) {
  if ((dtype != KV8_BF16 && dtype != KV8_F16) || q_heads < 1 || q_heads > 4096 || q_heads % cache->kv_heads != 0)
    return W8A8_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale <= 3.0e38f)) return W8A8_ERR_INVALID_ARG;
  if (step->tokens == 0) return W8A8_OK;   // an empty tensor has no address
  int rc = kv8_check_rows(q, q_stride, q_heads, cache->head_dim);
  if (rc == W8A8_OK) rc = kv8_check_rows(out, out_stride, q_heads, cache->head_dim);
  if (rc != W8A8_OK) return rc;
  return kv8_aligned(lse, 4) ? W8A8_OK : W8A8_ERR_MISALIGNED;
}

cudaError_t fill_params(Params& p, const kv8_cache_t* cache, const kv8_step_t* step, const void* q, long long q_stride, int q_heads,
                        void* out, long long out_stride, float* lse, float scale, void* ws, int sms) {
  const int D = cache->head_dim;
  // The cache as rows of D bytes, one for each (page, kv head, token).
  const int P = cache->page_tokens;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)cache->pages * cache->kv_heads * P};
  const cuuint64_t strides[1] = {(cuuint64_t)D};
  const cuuint32_t box[2] = {(cuuint32_t)(D > 128 ? 128 : D), (cuuint32_t)kGranule};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapSwizzle swizzle = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  cudaError_t e = encode_tensor_map_2d(&p.kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->k, dims, strides, box, estr, swizzle);
  if (e == cudaSuccess)
    e = encode_tensor_map_2d(&p.vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->v, dims, strides, box, estr, swizzle);
  if (e != cudaSuccess) return e;
  p.step = kv8_step_of(*step);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.q_stride = q_stride, p.out_stride = out_stride;
  p.ks = cache->k_scale;
  p.vs = cache->v_scale;
  p.pages = cache->pages, p.q_heads = q_heads, p.kv_heads = cache->kv_heads;
  p.page_shift = P == 16 ? 4 : P == 32 ? 5 : P == 64 ? 6 : 7;
  p.group = q_heads / cache->kv_heads;
  p.window = 0, p.causal = 1;
  p.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* const w = static_cast<uint8_t*>(ws);
  p.status = reinterpret_cast<uint32_t*>(w);
  p.counters = reinterpret_cast<uint32_t*>(w + kWsHeaderBytes);
  p.group_counters = p.counters + (size_t)sms * 4;
  p.parts = reinterpret_cast<float*>(w + kWsHeaderBytes + counters_bytes(sms));
  p.seq0 = p.prefix = nullptr;
  p.groups = 0;
  p.rows32 = nullptr;
  p.items = nullptr;
  p.sms = sms, p.tile_rows = p.block = 0;
  p.prefix_fixed = p.prefix_unit = p.own_fixed = p.own_token = 0.f;
  return cudaSuccess;
}

cudaError_t launch_plain(const Params& p, int head_dim, bool f16, int sms, cudaStream_t s) {
  return f16 ? launch_rows<true, kPlain>(p, head_dim, sms, s) : launch_rows<false, kPlain>(p, head_dim, sms, s);
}

}  // namespace attn
}  // namespace w8a8

using namespace w8a8;

extern "C" size_t kv8_workspace_bytes(int q_heads, int kv_heads, int head_dim) {
  if (kv8_check_dims(kv_heads, head_dim) != W8A8_OK || q_heads < 0 || q_heads > 4096) return 0;
  const int sms = device_sm_count();
  return kWsHeaderBytes + attn::counters_bytes(sms) + attn::parts_bytes(head_dim, sms);
}

extern "C" int kv8_attention(const kv8_cache_t* cache, const kv8_step_t* step, const void* q, long long q_stride, int q_heads,
                             void* out, long long out_stride, float* lse, float scale, int window, unsigned flags, int dtype,
                             void* ws, size_t ws_bytes, void* stream) {
  int rc = kv8_check_cache(cache);
  if (rc == W8A8_OK) rc = kv8_check_step(step, cache);
  if (rc != W8A8_OK) return rc;
  if (flags & ~(unsigned)KV8_FLAG_NOT_CAUSAL) return W8A8_ERR_INVALID_ARG;
  if (window < 0 || ((flags & KV8_FLAG_NOT_CAUSAL) && window > 0)) return W8A8_ERR_INVALID_ARG;
  if ((rc = attn::check_call(cache, step, q, q_stride, q_heads, out, out_stride, lse, scale, dtype)) != W8A8_OK) return rc;
  if (step->tokens == 0) return W8A8_OK;
  const int D = cache->head_dim;
  if ((rc = kv8_check_ws(ws, ws_bytes, kv8_workspace_bytes(q_heads, cache->kv_heads, D))) != W8A8_OK) return rc;
  const int sms = device_sm_count();
  attn::Params p;
  cudaError_t e = attn::fill_params(p, cache, step, q, q_stride, q_heads, out, out_stride, lse, scale, ws, sms);
  if (e != cudaSuccess) return record_cuda_error(e, "kv8_attention");
  // No cache has more than 2^30 tokens: a longer window is none, and the kernels' first token stays inside 32 bits with
  // any number of rows.
  p.window = window < (1 << 30) ? window : 1 << 30, p.causal = (flags & KV8_FLAG_NOT_CAUSAL) ? 0 : 1;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  e = attn::launch_plain(p, D, dtype == KV8_F16, sms, s);
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "kv8_attention");
}
