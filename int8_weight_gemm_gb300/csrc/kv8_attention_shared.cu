// Attention over the 8-bit paged cache for sequences that share prefixes (kv8_attention_shared): the tokens that a
// group of sequences has in common are read once, for all of their rows.
//
// Mathematics.  The tokens that a row sees are the prefix, then its sequence's own.  Each side gives sums o relative to a
// reference r, and (m, l) of its softmax (kv8_attention_few.cuh); the two, and the parts of a side that was cut, join as
//   M = max m_i,  R = max r_i,  l = sum l_i 2^(m_i - M),  o = sum o_i 2^(r_i - R),  out = o 2^(R - M) / l.
//
// What bounds it: with the prefix read once its products do.  64 rows' heads of 4 a kv head are 256 rows over every
// prefix byte, work for the kernel of many rows (kv8_attention_many.cuh), which is bound by a chain of waits; the own
// tokens are a decode step's and stream at HBM speed (kv8_attention_few.cuh).  So a call is three launches: the groups
// over their prefixes as if each were one sequence, not causal; beside it, on the other SMs (prefix_sms), the sequences
// over their own tokens; and the join of the fp32 rows that the two leave.  A prefix of few items (a kv head's 256 rows
// each) is cut into several parts an item, which one CTA an item would read for longer than the products take: the join
// has a warp for each (row, head), on all SMs.
//
// Launches.  The groups' CTAs let the second launch begin when they have seen the work before them complete, so it may read
// what that work wrote; it waits for the groups' at its end, so that the join, which waits for it, sees both.
//
// Measured (32 query heads, 8 kv heads of 128; in brackets kv8_attention, whose re-reads hit L2): 64 sequences of 6101-8191
// tokens behind one prefix of 6016 61 us (141), some 35 us of it 148 MB of own tokens' stream and products beside it, 5 the
// start, 5 the join; behind 16000 with up to 400 own tokens 69 (299).  One launch after the other took 89, with the parts joined by
// rows (uncoalesced) 70, with eight warps a CTA of the second launch 66.
#include "kv8_attention_few.cuh"

namespace w8a8 {
namespace attn {

constexpr int kJoinThreads = 256;
constexpr int kFew = 4;   // parts
// Steps that kv8_attention's launch takes as they are (worth_sharing).
constexpr int kManyRows = 80;                                    // of a sequence and kv head
constexpr long long kFewTokens = 700000, kFewTokensWide = 400000;   // times kv heads, up to 16 rows and more

struct JoinParams {
  Params p;
  const float* own;      // [tokens][q_heads] of D sums, (m, l, r, -): over the sequences' own tokens
  const float* whole;    // the same over the prefixes, of items that were not cut
  const float* parts;    // of items that were
  int tile_shift;        // rows of an item: 2^tile_shift
};

// A CTA for a row and some of its query heads: a warp for each, in turns where there are many rows.
template <bool kF16, int D>
__global__ void __launch_bounds__(kJoinThreads) kv8_join_kernel(const __grid_constant__ JoinParams j) {
  const Params& p = j.p;
  pdl_trigger();
  __threadfence();   // (what is read before the wait is not older than the first launch's wait)
  const int lane = threadIdx.x & 31, row = blockIdx.x;
  // The row's sequence (the last that begins at or before it) and group.  None of this is written by the launches that
  // this one waits for.
  int b = 0;
  for (int n = p.step.seqs; n > 1;) {
    const int step = (n + 31) / 32;
    const bool in = lane * step < n && load<true>(p.step.row0 + b + lane * step) <= row;
    const uint32_t mask = __ballot_sync(0xffffffffu, in);
    const int k = mask ? 31 - __clz(mask) : 0;
    b += k * step;
    n = min(step, n - k * step);
  }
  Seq s;
  load_seq<true>(p.step, b, 1 << p.page_shift, false, p.status, s);
  auto holds_row = [&]() { return s.n > 0 && row >= s.row0 && row - s.row0 < s.n; };
  if (!holds_row()) {
    // Behind the last sequence, as a step's unused rows are (1000 sequences, 8000 rows: looked for all the same 235 us a call,
    // not 100); or the search met the offset of a sequence that is left out, and the row is another's.
    const int rows = load<true>(p.step.row0 + p.step.seqs);
    for (int b0 = row >= rows && rows >= 0 ? p.step.seqs : 0; b0 < p.step.seqs && !holds_row(); b0 += 32) {
      const int at = b0 + lane;
      const bool in = at < p.step.seqs && load<true>(p.step.row0 + at) <= row && row < load<true>(p.step.row0 + at + 1);
      for (uint32_t mask = __ballot_sync(0xffffffffu, in); mask && !holds_row(); mask &= mask - 1) {
        b = b0 + __ffs(mask) - 1;
        load_seq<true>(p.step, b, 1 << p.page_shift, false, p.status, s);
      }
    }
  }
  int g;
  Rows of;
  const bool shared = shared_tokens(p, b, s, g, of) > 0;
  pdl_wait();
  if (!holds_row()) return;   // of no sequence
  // Values of a head: four a lane (D = 64: by half a warp, the other half takes every other part; 256: two times four).
  constexpr int kV = D == 256 ? 2 : 1, kAt = D == 64 ? 2 : 1;
  const int d = 4 * (lane & (D == 64 ? 15 : 31));
  const size_t part_floats = (size_t)(D + 4) << j.tile_shift;
  // (item_of, by shifts.)
  const long long first_row = (long long)(row - of.row0) * p.group, first_item = ((long long)of.row0 * p.group >> j.tile_shift) + g;
  // What a head's own side left, and the place of its item: asked for one head ahead.
  struct Head {
    float4 t, acc[kV];
    int4 item;   // first CTA, parts, place in the first
    int within;
  };
  auto ask = [&](int head, Head& x) {
    const float* const own = j.own + ((size_t)row * p.q_heads + head) * (D + 4);
    x.item = make_int4(0, 0, 0, 0);
    x.within = 0;
    if (shared) {
      const int h = (int)((uint32_t)head / (uint32_t)p.group);
      const long long ri = first_row + (head - h * p.group);
      x.within = (int)ri & ((1 << j.tile_shift) - 1);
      x.item = p.items[(size_t)(first_item + (ri >> j.tile_shift)) * p.kv_heads + h];
    }
    x.t = *reinterpret_cast<const float4*>(own + D);
#pragma unroll
    for (int v = 0; v < kV; ++v) x.acc[v] = *reinterpret_cast<const float4*>(own + d + 128 * v);
  };
  const int step = gridDim.y * (kJoinThreads / 32);
  int head = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5);
  if (head >= p.q_heads) return;
  Head next;
  ask(head, next);
  for (; head < p.q_heads; head += step) {
    const Head x = next;
    if (head + step < p.q_heads) ask(head + step, next);
    const size_t at = (size_t)row * p.q_heads + head;
    const int4 item = x.item;
    const int within = x.within;
    int parts = item.y;
    if (item.x < 0 || parts < 0 || parts > p.sms - item.x || (uint32_t)item.z > 1u) {
      // No launch that ended well leaves this: nothing is read through it.
      if (lane == 0) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
      parts = 0;
    }
    float M = x.t.x, R = x.t.z, l = x.t.y;
    float4 acc[kV];
#pragma unroll
    for (int v = 0; v < kV; ++v) acc[v] = x.acc[v];
    // The row's columns from d on, and its statistics, in part i.  (An item that was not cut: its rows as they are; a part:
    // [D / 4][rows] of four columns, then the rows' statistics.  Neighbouring heads' columns share a line, so these loads
    // stay in the L1 cache.)
    const bool cut = parts != 1;
    const float* const part0 = cut ? j.parts + (size_t)item.x * 2 * part_floats + within * 4 : j.whole + at * (D + 4);
    const size_t col = cut ? (size_t)d << j.tile_shift : (size_t)d, cols128 = cut ? (size_t)128 << j.tile_shift : 128, stats = cut ? (size_t)D << j.tile_shift : D;
    auto part_of = [&](int i) { return part0 + (i > 0 ? (size_t)(2 * i) * part_floats : cut && item.z ? part_floats : 0); };
    auto sums_of = [&](int i, int v) { return *reinterpret_cast<const float4*>(part_of(i) + col + v * cols128); };
    auto stats_of = [&](int i) { return *reinterpret_cast<const float4*>(part_of(i) + stats); };
    auto add = [&](const float4 x, float f, int v) {
      acc[v].x = fmaf(x.x, f, acc[v].x), acc[v].y = fmaf(x.y, f, acc[v].y), acc[v].z = fmaf(x.z, f, acc[v].z), acc[v].w = fmaf(x.w, f, acc[v].w);
    };
    if (parts > 0 && parts <= kFew) {
      // Few parts: every lane does what a lane each would have to share (64 rows of 32 heads, 4 parts: the call 67.5 -> 66.4 us).
      float4 t[kFew], x[kFew][kV];
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        t[i] = make_float4(kFloor, 0.f, kFloor, 0.f);
        if (i < parts) {
          t[i] = stats_of(i);
#pragma unroll
          for (int v = 0; v < kV; ++v) x[i][v] = sums_of(i, v);
        }
      }
      float mn = M, rn = R;
#pragma unroll
      for (int i = 0; i < kFew; ++i) mn = fmaxf(mn, t[i].x), rn = fmaxf(rn, t[i].z);
      l *= ex2(M - mn);
      const float a0 = ex2(R - rn);
#pragma unroll
      for (int v = 0; v < kV; ++v) acc[v].x *= a0, acc[v].y *= a0, acc[v].z *= a0, acc[v].w *= a0;
      M = mn;
      R = rn;
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        if (i < parts) {
          l = fmaf(t[i].y, ex2(t[i].x - M), l);
          const float f = ex2(t[i].z - R);
#pragma unroll
          for (int v = 0; v < kV; ++v) add(x[i][v], f, v);
        }
      }
    } else if (parts > 0) {
      // References first: a lane for each part.
      float4 t = make_float4(kFloor, 0.f, kFloor, 0.f);
      if (lane < parts) t = stats_of(lane);
      float mm = t.x, rm = t.z, lt = t.y;
      for (int i = lane + 32; i < parts; i += 32) {
        const float4 x = stats_of(i);
        const float mn = fmaxf(mm, x.x);
        lt = lt * ex2(mm - mn) + x.y * ex2(x.x - mn);
        mm = mn;
        rm = fmaxf(rm, x.z);
      }
      float mn = fmaxf(M, mm), rn = fmaxf(R, rm);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        rn = fmaxf(rn, __shfl_xor_sync(0xffffffffu, rn, o));
      }
      lt *= ex2(mm - mn);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
      l = fmaf(l, ex2(M - mn), lt);
      const float a0 = D == 64 && lane >= 16 ? 0.f : ex2(R - rn);
#pragma unroll
      for (int v = 0; v < kV; ++v) acc[v].x *= a0, acc[v].y *= a0, acc[v].z *= a0, acc[v].w *= a0;
      M = mn;
      R = rn;
      const int odd = D == 64 ? lane >> 4 : 0;
      for (int i0 = 0; i0 < parts; i0 += 32) {
        float a = 0.f;
        if (i0 + lane < parts) a = ex2((i0 ? stats_of(i0 + lane).z : t.z) - R);
        const int n = min(32, parts - i0);
#pragma unroll 4
        for (int i = 0; i < n; i += kAt) {
          const float f = __shfl_sync(0xffffffffu, a, (i + odd) & 31);
          if (i + odd < n) {
#pragma unroll
            for (int v = 0; v < kV; ++v) add(sums_of(i0 + i + odd, v), f, v);
          }
        }
      }
      if (D == 64) {
        acc[0].x += __shfl_xor_sync(0xffffffffu, acc[0].x, 16), acc[0].y += __shfl_xor_sync(0xffffffffu, acc[0].y, 16);
        acc[0].z += __shfl_xor_sync(0xffffffffu, acc[0].z, 16), acc[0].w += __shfl_xor_sync(0xffffffffu, acc[0].w, 16);
      }
    }
    const float z = l == 0.f ? 0.f : __fdividef(1.f, l) * ex2(R - M);
    if (D > 64 || lane < 16) {
      uint16_t* const dst = p.out + row * p.out_stride + head * D + d;
#pragma unroll
      for (int v = 0; v < kV; ++v)
        *reinterpret_cast<uint2*>(dst + 128 * v) =
            make_uint2(pack2<kF16>(acc[v].x * z, acc[v].y * z), pack2<kF16>(acc[v].z * z, acc[v].w * z));
    }
    if (p.lse && lane == 0) p.lse[at] = l == 0.f ? -INFINITY : (M + lg2(l)) * 0.69314718056f;
  }
}

template <bool kF16, int D>
static cudaError_t launch_join(const JoinParams& j, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  // Enough CTAs for every SM's places; beyond that a row's lookups serve several heads.
  const int most = (j.p.q_heads + kJoinThreads / 32 - 1) / (kJoinThreads / 32), want = (4 * j.p.sms + j.p.step.tokens - 1) / j.p.step.tokens;
  cfg.gridDim = dim3((unsigned)j.p.step.tokens, (unsigned)(want < most ? want : most));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_join_kernel<kF16, D>, j);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool kF16>
static cudaError_t launch_join_of(const JoinParams& j, int head_dim, cudaStream_t s) {
  return head_dim == 64 ? launch_join<kF16, 64>(j, s) : head_dim == 128 ? launch_join<kF16, 128>(j, s) : launch_join<kF16, 256>(j, s);
}

// What the two launches cost an SM, in ns, for prefix_sms: measured.
static void set_costs(Params& p, int head_dim, long long rows) {
  p.prefix_fixed = 12000.f;
  p.prefix_unit = head_dim == 256 ? 1900.f : p.tile_rows == 256 ? 3000.f : 2200.f;
  p.own_fixed = 9000.f;
  p.own_token = (head_dim == 256 ? 2.f : 1.f) * (rows <= 8 ? 7.5f : rows <= 16 ? 9.f : rows <= 32 ? 25.f : 0.8f * (float)rows);
}

// Whether a step can gain by sharing, as far as the host can tell.  Sequences of many rows fill the products' tiles on their
// own, and those are the bound (us, as they are / shared): 32 windows of 16 tokens behind 4096, 32 query and 8 kv heads (64
// rows) 133 / 110; of 23 (92 rows) 137 / 145; 8 prompts of 256 (1024) 197 / 236.
// And the re-reads of a prefix hit L2, so a small cache, by what the page table has room for, is read in less time than the
// three launches take (128-wide heads): 16 sequences on 1200 tokens, 4 kv heads (20 MB) 11.7 / 24; 64 of
// 1700, 8 (213 MB) 46 / 42.5; 64 of 2700 (341 MB) 64 / 45; 64 of 7000 (897 MB) 141 / 62; 16 windows of 6 on 4300 (134 MB, 24
// rows) 48 / 45; heads of 64, 32 of 3000, 16 kv heads (196 MB) 50 / 41.  It is not always right: four groups of four windows of
// 6 behind 1001 to 4003 42.2 / 43.8; and a short step in a wide table, which the host cannot tell from a long one, 4 sequences on 700
// 8.4 / 18.1, 16 on 1400 11.7 / 24.2.
static bool worth_sharing(const kv8_cache_t* cache, const kv8_step_t* step, long long rows) {
  const long long tokens = (long long)step->seqs * step->table_width * cache->page_tokens * cache->kv_heads;
  return rows < kManyRows && tokens > (rows <= 16 ? kFewTokens : kFewTokensWide);
}

// The workspace behind that of kv8_attention: parts of cut prefixes, their places, and two buffers of fp32 rows.
struct SharedLayout {
  size_t parts, items, whole, own, bytes;
  SharedLayout(int tokens, int groups, int q_heads, int kv_heads, int head_dim, int sms) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    const size_t rows = up((size_t)tokens * q_heads * (head_dim + 4) * sizeof(float));
    parts = up(kv8_workspace_bytes(q_heads, kv_heads, head_dim));
    items = parts + up(many_parts_bytes(head_dim, sms));
    whole = items + up(((size_t)tokens * (q_heads / kv_heads) / many_tile_rows(head_dim, 1) + groups + 1) * kv_heads * sizeof(int4));
    own = whole + rows;
    bytes = own + rows;
  }
};

}  // namespace attn
}  // namespace w8a8

using namespace w8a8;

extern "C" size_t kv8_shared_workspace_bytes(int tokens, int groups, int q_heads, int kv_heads, int head_dim) {
  if (kv8_check_dims(kv_heads, head_dim) != W8A8_OK || q_heads < 1 || q_heads > 4096 || q_heads % kv_heads != 0 || tokens < 0 ||
      tokens > (1 << 22) || groups < 1 || groups > 65535)
    return 0;
  return attn::SharedLayout(tokens, groups, q_heads, kv_heads, head_dim, device_sm_count()).bytes;
}

extern "C" int kv8_attention_shared(const kv8_cache_t* cache, const kv8_step_t* step, const kv8_groups_t* groups, const void* q,
                                    long long q_stride, int q_heads, void* out, long long out_stride, float* lse, float scale,
                                    int dtype, void* ws, size_t ws_bytes, void* stream) {
  int rc = kv8_check_cache(cache);
  if (rc == W8A8_OK) rc = kv8_check_step(step, cache);
  if (rc != W8A8_OK) return rc;
  if (!groups || !groups->seq0 || !groups->prefix || groups->groups < 1 || groups->groups > 65535 || groups->max_rows < 1 ||
      groups->max_rows > (1 << 22))
    return W8A8_ERR_INVALID_ARG;
  if (!kv8_aligned(groups->seq0, 4) || !kv8_aligned(groups->prefix, 4)) return W8A8_ERR_MISALIGNED;
  if ((rc = attn::check_call(cache, step, q, q_stride, q_heads, out, out_stride, lse, scale, dtype)) != W8A8_OK) return rc;
  if (step->tokens == 0) return W8A8_OK;
  const int D = cache->head_dim, sms = device_sm_count();
  const attn::SharedLayout at(step->tokens, groups->groups, q_heads, cache->kv_heads, D, sms);
  if ((rc = kv8_check_ws(ws, ws_bytes, at.bytes)) != W8A8_OK) return rc;
  uint8_t* const w = static_cast<uint8_t*>(ws);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool f16 = dtype == KV8_F16;
  attn::JoinParams j;
  cudaError_t e = attn::fill_params(j.p, cache, step, q, q_stride, q_heads, out, out_stride, lse, scale, ws, sms);
  if (e != cudaSuccess) return record_cuda_error(e, "kv8_attention_shared");
  const long long rows = (long long)step->max_tokens * j.p.group;
  if (!attn::worth_sharing(cache, step, rows)) {
    e = attn::launch_plain(j.p, D, f16, sms, s);
    return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "kv8_attention_shared");
  }
  j.p.seq0 = groups->seq0;
  j.p.prefix = groups->prefix;
  j.p.groups = groups->groups;
  j.p.items = reinterpret_cast<int4*>(w + at.items);
  const long long group_rows = (long long)groups->max_rows * j.p.group;
  j.p.tile_rows = attn::many_tile_rows(D, group_rows);
  j.p.block = attn::many_block(D);
  attn::set_costs(j.p, D, rows);
  // The groups over their prefixes.
  attn::Params a = j.p;
  a.parts = reinterpret_cast<float*>(w + at.parts);
  a.rows32 = reinterpret_cast<float*>(w + at.whole);
  e = attn::launch_many_prefixes(a, D, f16, sms, s);
  if (e != cudaSuccess) return record_cuda_error(e, "kv8_attention_shared");
  // The sequences over their own tokens.
  attn::Params b = j.p;
  b.rows32 = reinterpret_cast<float*>(w + at.own);
  e = f16 ? attn::launch_rows<true, attn::kOwn>(b, D, sms, s) : attn::launch_rows<false, attn::kOwn>(b, D, sms, s);
  if (e != cudaSuccess) return record_cuda_error(e, "kv8_attention_shared");
  j.own = b.rows32;
  j.whole = a.rows32;
  j.parts = a.parts;
  j.tile_shift = j.p.tile_rows == 128 ? 7 : 8;
  e = f16 ? attn::launch_join_of<true>(j, D, s) : attn::launch_join_of<false>(j, D, s);
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "kv8_attention_shared");
}
