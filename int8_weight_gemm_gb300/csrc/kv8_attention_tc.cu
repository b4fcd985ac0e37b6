// Instances of the kernel for many query rows that kv8_attention calls.
#include "kv8_attention_many.cuh"

namespace w8a8 {
namespace attn {

cudaError_t launch_many(const Params& p, int head_dim, bool f16, int sms, cudaStream_t s) {
  return launch_many_of<kPlain>(p, (long long)p.step.max_tokens * p.group, head_dim, f16, sms, s);
}

int many_tile_rows(int head_dim, long long rows) { return tile_rows_of(head_dim, rows); }

int many_block(int head_dim) { return head_dim == 256 ? TcLayout<256, 1>::kBlock : TcLayout<128, 1>::kBlock; }

size_t many_parts_bytes(int head_dim, int sms) {
  const int part = head_dim == 64 ? TcLayout<64, 2>::kPart : head_dim == 128 ? TcLayout<128, 2>::kPart : TcLayout<256, 1>::kPart;
  return (size_t)sms * 2 * part * sizeof(float);
}

}  // namespace attn
}  // namespace w8a8
