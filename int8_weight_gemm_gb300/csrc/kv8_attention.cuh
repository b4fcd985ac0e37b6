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
  // Sequences that share prefixes (kPrefixes, kOwn).
  const int* seq0;         // [groups + 1] first sequence of each group
  const int* prefix;       // [groups] tokens that its sequences have in common
  int groups;
  float* rows32;           // [tokens][q_heads] of D sums, (m, l, r, -): rows go here, unnormalised
  int4* items;             // kPrefixes: where an item's parts lie (item_of): first CTA, parts, place in the first one, -
  int sms;
  int tile_rows, block;    // rows of an item and tokens of a unit of kPrefixes' launch
  float prefix_fixed, prefix_unit, own_fixed, own_token;   // what the two launches cost an SM, in ns (prefix_sms)
};

// What a launch does: sequences over all they see (kv8_attention); groups of sequences over their shared prefixes, as if
// each group were one sequence that sees all of them; sequences over what is not shared.
enum Mode { kPlain, kPrefixes, kOwn };

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

// A sequence of a launch: also its first token that is not another launch's, and its row of the page table.
struct Rows : Seq {
  int lo, table;
};

// (The loads from here to prefix_sms are ordinary ones: kOwn makes them before it has waited, and so does the join.)

// The group of sequence b (-1: of none).
__device__ __forceinline__ int group_of(const Params& p, int b) {
  int lo = 0, n = p.groups;   // the last group that begins at or before b
  while (n > 1) {
    const int half = n >> 1;
    if (load<true>(p.seq0 + lo + half) <= b) lo += half;
    n -= half;
  }
  return load<true>(p.seq0 + lo) <= b && b < load<true>(p.seq0 + lo + 1) ? lo : -1;
}

// Group g as a sequence: the rows of all its sequences over their shared prefix, in whole pages; `table`: its first
// sequence.  No rows and no tokens where nothing is shared: a single sequence, or a first one that does not hold the
// prefix.  (Two rounds of loads: what depends on the first is asked for at once, at indices held in range.)
__device__ __forceinline__ void load_group(const Params& p, int g, Rows& s) {
  const int first = load<true>(p.seq0 + g), last = load<true>(p.seq0 + g + 1);
  const int whole = load<true>(p.prefix + g) & ~((1 << p.page_shift) - 1);
  const bool ok = first >= 0 && last >= first && last <= p.step.seqs;
  const int f = ok ? min(first, p.step.seqs - 1) : 0;
  const int len = load<true>(p.step.kv_len + f), r0 = load<true>(p.step.row0 + f), r1 = load<true>(p.step.row0 + (ok ? last : 0));
  if (!ok) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
  s.lo = 0;
  s.table = f;
  const bool shared = ok && last - first >= 2 && whole > 0 && len >= whole && (long long)whole <= (long long)p.step.table_width << p.page_shift &&
                      r0 >= 0 && r1 >= r0 && r1 <= p.step.tokens;
  s.len = shared ? whole : 0;
  s.row0 = shared ? r0 : 0;
  s.n = shared ? r1 - r0 : 0;
}

// Tokens of sequence b that its group's launch covers, and that group: all of the shared prefix where every row of the
// sequence sees all of it, else none.
__device__ __forceinline__ int shared_tokens(const Params& p, int b, const Seq& s, int& g, Rows& of) {
  if ((g = group_of(p, b)) < 0) return 0;
  load_group(p, g, of);
  return of.len > 0 && s.len - s.n >= of.len && s.row0 >= of.row0 && s.row0 + s.n <= of.row0 + of.n ? of.len : 0;
}

// Reads "sequence" b of the launch.
template <Mode kMode>
__device__ __forceinline__ void load_rows(const Params& p, int b, Rows& s) {
  if (kMode == kPrefixes) return load_group(p, b, s);
  s.lo = 0;
  s.table = b;
  load_seq<kMode == kOwn>(p.step, b, 1 << p.page_shift, false, p.status, s);
  if (kMode == kOwn) {
    int g;
    Rows of;
    s.lo = shared_tokens(p, b, s, g, of);
  }
}

// Sequences of the launch.
template <Mode kMode>
__device__ __forceinline__ int count_of(const Params& p) {
  return kMode == kPrefixes ? p.groups : p.step.seqs;
}

// The place of a row tile's entry in `items`: tiles of `rows` of the group's rows, which begin at row r0 of the step.
// (A group of x tiles' worth of rows has ceil(x) tiles; floor(a + x) - floor(a) + 1 places are never fewer.)
__device__ __forceinline__ size_t item_of(const Params& p, int g, int r0, int rows, int tile, int h) {
  return ((size_t)((long long)r0 * p.group / rows) + g + tile) * p.kv_heads + h;
}

// What the rows of a sequence cover: items of `tiles` row tiles and kv heads, each of `units` units
// from token `lo` (a granule's start) to `hi`; `span` = the lead and the units, its length in the split.
struct Span {
  Rows s;
  int tiles, units, span, lo, hi;
};

template <typename L, Mode kMode>
__device__ __forceinline__ Span load_span(const Params& p, int b) {
  Span x;
  load_rows<kMode>(p, b, x.s);
  x.tiles = (int)quotient((long long)x.s.n * p.group + L::kRows - 1, L::kRows);
  x.hi = x.s.len;
  x.lo = p.window > 0 ? max(0, x.s.len - x.s.n - p.window + 1) & ~(kGranule - 1) : kMode == kOwn ? x.s.lo : 0;
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

// The SMs that the groups' launch takes while the other takes the rest, worked out alike by every CTA of both (the whole
// block takes part): prefixes cost the matrix products' chain of waits, own tokens HBM's bandwidth, so side by side
// they finish sooner than one after the other.  The time of either falls with its SMs; the count is that of the
// smallest maximum, or all of them (the other launch then follows) where that is sooner.  0: nothing is shared.
// scratch: shared memory, 24 bytes a warp, free again behind the block's next barrier.
template <int kThreads>
__device__ __forceinline__ int prefix_sms(const Params& p, void* scratch) {
  long long (*const sums_sm)[kThreads / 32] = static_cast<long long (*)[kThreads / 32]>(scratch);
  uint32_t* const best_sm = reinterpret_cast<uint32_t*>(sums_sm + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long units = 0, own = 0;
  for (int b = threadIdx.x; b < p.step.seqs; b += kThreads) own += max(0, load<true>(p.step.kv_len + b));
  for (int g = kThreads - 1 - (int)threadIdx.x; g < p.groups; g += kThreads) {   // (by other warps: their loads go side by side)
    Rows s;
    load_group(p, g, s);
    if (s.n > 0) {
      units += ((long long)s.n * p.group + p.tile_rows - 1) / p.tile_rows * (3 + (s.len + p.block - 1) / p.block);
      own -= (long long)s.len * (load<true>(p.seq0 + g + 1) - s.table);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    units += __shfl_xor_sync(0xffffffffu, units, o);
    own += __shfl_xor_sync(0xffffffffu, own, o);
  }
  if (lane == 0) sums_sm[0][warp] = units, sums_sm[1][warp] = own;
  __syncthreads();
  units = own = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) units += sums_sm[0][w], own += sums_sm[1][w];
  if (units == 0) return 0;
  units *= p.kv_heads;
  const float a = p.prefix_unit * (float)units, b = p.own_token * (float)max(own, 0ll) * (float)p.kv_heads;
  uint32_t best = 0xffffffffu;
  const int sms = min(p.sms, 255);
  for (int n = threadIdx.x + 1; n <= sms; n += kThreads) {
    const float ta = p.prefix_fixed + fmaxf(a / n, p.prefix_unit), tb = p.own_fixed + b / (n < sms ? sms - n : sms);
    best = min(best, ((uint32_t)fminf(n < sms ? fmaxf(ta, tb) : ta + tb, 1.6e7f) << 8) | (uint32_t)n);
  }
  best = __reduce_min_sync(0xffffffffu, best);
  if (lane == 0) best_sm[warp] = best;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) best = min(best, best_sm[w]);
  return (int)(best & 255u) == sms ? p.sms : (int)(best & 255u);
}

// SMs of the launch of the sequences' own tokens beside `n` of the other.
__device__ __forceinline__ int own_sms(const Params& p, int n) { return n < p.sms ? p.sms - n : p.sms; }

// The kernel of many query rows (kv8_attention_many.cuh), kPlain and kPrefixes; its share of the workspace.
cudaError_t launch_many(const Params& p, int head_dim, bool f16, int sms, cudaStream_t s);
cudaError_t launch_many_prefixes(const Params& p, int head_dim, bool f16, int sms, cudaStream_t s);
size_t many_parts_bytes(int head_dim, int sms);
// Rows of one of its tiles for sequences of up to `rows` rows of a kv head; tokens of a unit.
int many_tile_rows(int head_dim, long long rows);
int many_block(int head_dim);

// kv8_attention.cu: arguments that both entry points check and fill in alike, and kv8_attention's launch.
int check_call(const kv8_cache_t* cache, const kv8_step_t* step, const void* q, long long q_stride, int q_heads, const void* out,
               long long out_stride, const float* lse, float scale, int dtype);
cudaError_t launch_plain(const Params& p, int head_dim, bool f16, int sms, cudaStream_t s);
cudaError_t fill_params(Params& p, const kv8_cache_t* cache, const kv8_step_t* step, const void* q, long long q_stride, int q_heads,
                        void* out, long long out_stride, float* lse, float scale, void* ws, int sms);

}  // namespace attn
}  // namespace w8a8
