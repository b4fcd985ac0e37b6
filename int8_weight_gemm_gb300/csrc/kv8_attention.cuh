// Pieces shared by the attention kernels over the 8-bit paged cache: their arguments, and the split of
// the work over the CTAs, which every CTA works out from the lengths on the device.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "kv8.cuh"
#include "kv8.h"

namespace w8a8 {
namespace attn {

constexpr int kGranule = 16;         // tokens of a warp's step
constexpr float kFloor = -3.0e38f;   // reference of a row that has seen nothing
constexpr float kSlack = 8.f;        // a reference moves when it is passed by this much (powers of two)
// Where the weights' reference r moves, the largest weight becomes 2^kHead: fp16 has that room above a weight of 1, and
// below it loses bits from 2^-14 and everything from 2^-25 on, which the sums of the probabilities, held in fp32, count in
// full.  So a weight keeps its 11 bits down to 2^-21 of the row's largest and is zero below 2^-32 of it.  (A strong token
// without values over tokens of 2^-21.5 of it: outputs off by 0.01 % instead of 6 %, with r at the largest weight.)
constexpr float kHead = 7.f;
constexpr float kRoom = kHead + kSlack;   // no weight passes 2^15
// How far r may lie from m: 2^(m - r) and its inverse stay normal numbers.  Where the upper limit holds r, by a score of
// 2^8 above m's and a value scale of nearly 2^128, a weight is at most 2^(8 + 128 - 125).
constexpr float kBelow = 120.f, kAbove = 125.f;
// A weight is p * (v_scale * 2^(m - r)).  Where that factor is above this, p may have left fp32's range
// while the weight has not, and the weight is taken from its own exponent.
constexpr float kFar = 1.2676506e30f;   // 2^100

struct Params {
  CUtensorMap kmap, vmap;   // the cache as rows of D bytes, boxes of 16 rows
  Kv8Step step;
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  long long q_stride, out_stride;
  const float* ks;
  const float* vs;
  int pages, page_shift, q_heads, kv_heads, group, window, causal;
  float scale_log2;        // scale * log2 e
  uint32_t* status;
  uint32_t* counters;      // [CTA] arrivals at the item that crosses the end of its run, zero between calls
  uint32_t* group_counters;   // [CTA][2] arrivals at a group of parts, by its first part's place, zero between calls
  float* parts;            // [CTA][2] parts of split items
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// a / b for a >= 0, b > 0: a 64-bit division is a long subroutine, and hardly ever needed.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// What the rows of a sequence cover: items of `tiles` row tiles and kv heads, each of `units` units
// from token `lo` (a granule's start) to `hi`; `span` = the lead and the units, its length in the split.
struct Span {
  Seq s;
  int tiles, units, span, lo, hi;
};

template <typename L>
__device__ __forceinline__ Span load_span(const Params& p, int b) {
  Span x;
  load_seq(p.step, b, 1 << p.page_shift, false, p.status, x.s);
  x.tiles = (int)quotient((long long)x.s.n * p.group + L::kRows - 1, L::kRows);
  x.hi = x.s.len;
  x.lo = p.window > 0 ? max(0, x.s.len - x.s.n - p.window + 1) & ~(kGranule - 1) : 0;
  x.units = max(1, (x.hi - x.lo + L::kUnit - 1) / L::kUnit);   // one that sees nothing still writes its rows
  x.span = L::kLead + x.units;
  return x;
}

// The equal runs: U units over `ctas`, the first U % ctas one longer.
struct Runs {
  long long a, r;
  __device__ Runs(long long U, int ctas) : a(quotient(U, ctas)), r(U - a * ctas) {}
  __device__ long long begin(int i) const { return i * a + (i < r ? i : r); }
  __device__ int owner(long long u) const {
    const long long head = r * (a + 1);
    return (int)(u < head ? quotient(u, a + 1) : r + quotient(u - head, a));
  }
};

// The kernel of many query rows (kv8_attention_tc.cu); its share of the workspace.
cudaError_t launch_many(const Params& p, int head_dim, bool f16, int sms, cudaStream_t s);
size_t many_parts_bytes(int head_dim, int sms);

}  // namespace attn
}  // namespace w8a8
