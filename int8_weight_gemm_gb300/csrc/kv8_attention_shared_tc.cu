// Instances of the kernel for many query rows that kv8_attention_shared calls.
#include "kv8_attention_many.cuh"

namespace w8a8 {
namespace attn {

cudaError_t launch_many_prefixes(const Params& p, int head_dim, bool f16, int sms, cudaStream_t s) {
  return launch_many_of<kPrefixes>(p, p.tile_rows, head_dim, f16, sms, s);
}

}  // namespace attn
}  // namespace w8a8
