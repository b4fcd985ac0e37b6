// Attention over the 8-bit paged key-value cache: few query rows (single tokens, verify windows, small chunks).
//
// Row i of sequence b stands at position p = kv_len - n + i and sees the cached tokens
// j in [max(0, p - window + 1), p] (causal) or [0, kv_len):
//   o = sum_j softmax_j(scale q . k_j) v_j,   k_j = (byte - 128) * k_scale[page], v_j alike.
//
// What bounds it: every cached byte feeds 2 (rows / kv heads) multiply-adds, a handful for single
// tokens, so the cache has to stream at HBM speed and everything else has to hide behind it: at 6.8
// TB/s an SM has about 700 issue slots for a granule (16 tokens of a head, keys and values: 4 KiB at
// head_dim 128).
//
// Mathematics.  The n * G rows that share a kv head (n tokens, G query heads) are the columns of 8-wide
// tiles, the cached tokens the rows: S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16 (fp16 x fp16 ->
// fp32).  Rows as the narrow side make a tile of 8 where the other way round it would be 16: half the
// matrix instructions, exponentials and accumulators for up to 8 rows.
//  * Scores.  A cached byte b is used as the fp16 subnormal b * 2^-24 (one instruction makes two of
//    them, nothing is subtracted); 128 * sum_d q comes off each score in the multiply-add that applies
//    the scales.  A query row is scaled by a power of two (exact) that takes its largest value to
//    [2^13, 2^14), so bf16 queries lose nothing in fp16 down to 2^-27 of the row's largest.  The order
//    of d inside the product is free, and is chosen so that a lane's bytes are contiguous.
//  * One pass with running references.  p = 2^(s - m) sums to l in fp32.  The values' scale belongs to
//    the weights: w = 2^(s - m) * (v_scale * 2^(m - r)), rounded to fp16 (11 bits, against 8 for bf16:
//    with bf16 weights the error of a sum of independent values equals the output's own rounding), and
//    o = sum w (b - 128), the bytes converted exactly (the offset is not left to a subtraction at the
//    end: 128 sum w would be a thousand times the sum of a long cache's values).  r follows the largest
//    w as m follows the largest s, so neither a page of tiny values under the largest score nor the
//    reverse loses bits; it lies 2^7 below that w (kHead), so that a long tail of small weights is not
//    lost either.  Both references move only when a score or weight passes where they were put by 2^8:
//    w stays inside fp16's range, the sums are rescaled a few times per pass instead of at every
//    granule, and in between no lane needs another lane's maximum.
//  * Parts (warps of a CTA, CTAs of a split sequence) join as o 2^(r_i - r), l 2^(m_i - m), in a fixed
//    order whatever the order of arrival, so replays give the same bits.
//
// Layout and split.  A granule of one head is 16 rows of the cache: a 2-D tensor-map box per 128 bytes
// of head, whose hardware swizzle makes both operands' shared-memory reads conflict-free.  Every warp
// is its own pipeline (its ring of granules, its mbarriers, its running sums), so nothing in the loop
// waits for another warp; the page number and scales of its next 32 granules are one load a lane.
// The work is cut over all (sequence, row tile, kv head) items laid end to end, in units of one
// granule for each warp, into equal runs, one for each CTA: lengths live on the device, so each CTA
// finds its run from a scan of kv_len.  An item cut across CTAs is finished by the last of them to
// arrive.  Two to four CTAs share an SM, so that one's start, join and drain hide behind the others' streams.
//
// Measured (32 query heads, 8 kv heads of 128): 64 contexts of 6001-8191 148 us (6.3 TB/s, 93 % of a copy); one of
// 131071 49.8 (5.4 TB/s with its join); 16 of 257-4099 22.6, where starts and joins take half; windows of 6 tokens on
// 16 of 1001-5003 40.6, bound by issue slots and latency at 8 warps an SM.
#pragma once

#include "kv8_attention.cuh"

namespace w8a8 {
namespace attn {

// NT: 8-row tiles a warp holds.  A lane holds D NT / 4 sums, so the warps that an SM can hold follow
// from D NT: 16 of 128 registers, 12 of 168 or 8 of 255, in CTAs of four (eight for one tile of 128-wide heads: half
// the parts to join; but kOwn, whose many short items start and end behind each other's streams: 64 sequences of 85 to
// 2175 own tokens 66.5 us with eight, 62.1 with four).
template <int D, int NT, Mode kMode = kPlain>
struct Layout {
  static constexpr int kWarps = D * NT == 128 && NT == 1 && kMode == kPlain ? 8 : 4;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = (D * NT <= 128 ? 16 : D * NT <= 256 ? 12 : 8) / kWarps;   // CTAs on an SM
  static constexpr int kUnit = kGranule * kWarps;       // tokens of the split's unit
  static constexpr int kRows = 8 * NT;
  static constexpr int kBoxes = D > 128 ? D / 128 : 1;
  static constexpr int kBoxBytes = kGranule * (D > 128 ? 128 : D);
  static constexpr int kSide = kBoxes * kBoxBytes;      // keys (or values) of a granule
  static constexpr int kStage = 2 * kSide;
  static constexpr int kStages = 196608 / (kCtas * kWarps * kStage);   // a warp's ring
  static constexpr int kRing = kWarps * kStages * kStage;
  // The queries' fragments are the same for every warp: in shared memory where registers are short (D NT = 256, 32
  // contexts of 8000, 8 kv heads: 32 rows of 64 150 -> 122 us, 4 of 256 170.7 -> 168.6; 16 contexts of 3000, 16 rows of
  // 128 32.6 -> 31.6).
  static constexpr bool kQShared = D * NT >= 256;
  static constexpr int kQBytes = kQShared ? NT * (D / 16) * 32 * 8 : 0;
  static constexpr int kSmem = 1024 + kRing + kQBytes;
  // Whether the next granule's scores are worked out beside this one's weights and sums, two independent streams
  // of instructions: where there are registers for both.  (D = 128, one tile: 64 long contexts 148.4 -> 146.2 us, one
  // of 131071 tokens 51.3 -> 49.6; 24 rows 40.3 -> 46.8, D = 64 24.3 -> 25.8.)
  static constexpr bool kAhead = D == 128 && NT == 1;
  static constexpr int kRow = D + 4;                    // floats of a row in the join buffer
  // What an item costs beside its tokens (queries, first copies, join), in units: each item's place in
  // the split is that much longer, so a run that crosses into another item gets fewer tokens.
  static constexpr int kLead = 3;
  // Items of up to this many units are not cut where there is a CTA for each: a unit takes 0.9 us of a CTA alone, a
  // join 2.9 (200 tokens, 8 rows of 2 kv heads: 7.0 -> 5.8 us, 32 such sequences 8.9 -> 7.4, heads of 64 6.4 -> 5.7, 24
  // rows 11.0 -> 9.8; at five units 128-wide heads lose, 7.7 -> 8.2, at four those of 256, 7.9 -> 8.1).
  static constexpr int kWhole = D == 256 ? 3 : 4;
  // A part of a split item in the workspace: kRows x D sums, then (m, l, r, -) of each row.
  static constexpr int kPart = kRows * (D + 4);
  static_assert(kWarps * kRows * kRow * 4 <= kRing, "the join buffer lies over the rings");
  static_assert(kStages >= 2 && kStages <= 16, "ring depth");
  static_assert(kCtas * (kSmem + 5120) <= 232448, "shared memory of an SM");
};

// Transpose of an 8 x 8 matrix of 16-bit values held as two of row lane / 4 by each lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t t;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(t) : "r"(v));
  return t;
}

// Four output values at d of one joined query row, and with the first of them the row's lse.  (kOwn: in instances of its own,
// as it costs registers.)
template <bool kF16, Mode kMode>
__device__ __forceinline__ void store_row(const Params& p, int row0, int ri, int h, int d, int D, float4 acc, float M, float lt,
                                          float Rf) {
  const int orow = row0 + ri / p.group, head = h * p.group + ri % p.group;
  if (kMode == kOwn) {
    float* const dst = p.rows32 + ((size_t)orow * p.q_heads + head) * (D + 4);
    *reinterpret_cast<float4*>(dst + d) = acc;
    if (d == 0) *reinterpret_cast<float4*>(dst + D) = make_float4(M, lt, Rf, 0.f);
    return;
  }
  const float z = lt == 0.f ? 0.f : __fdividef(1.f, lt) * ex2(Rf - M);
  *reinterpret_cast<uint2*>(p.out + orow * p.out_stride + head * D + d) =
      make_uint2(pack2<kF16>(acc.x * z, acc.y * z), pack2<kF16>(acc.z * z, acc.w * z));
  if (p.lse && d == 0) p.lse[(size_t)orow * p.q_heads + head] = lt == 0.f ? -INFINITY : (M + lg2(lt)) * 0.69314718056f;
}

template <bool kF16, int D, int NT, Mode kMode>
__global__ void __launch_bounds__(Layout<D, NT, kMode>::kThreads, Layout<D, NT, kMode>::kCtas)
    kv8_attention_kernel(const __grid_constant__ Params p) {
  using L = Layout<D, NT, kMode>;
  constexpr int NS = L::kStages;
  constexpr int kWarps = L::kWarps, kThreads = L::kThreads;
  constexpr int kSteps = D / 16;    // k16 steps of a score; 16-row tiles of the output
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kWarps][NS];
  __shared__ long long scan_sm[kWarps];
  __shared__ int2 items_sm[kWarps];   // items, and the units of the longest
  __shared__ struct {
    Span x;
    int b;
    long long u;
  } start_sm;
  __shared__ float4 mlr_sm[kWarps][L::kRows];   // (m, l, r, -) of each warp's rows
  __shared__ float4 row_st[L::kRows];   // of each row: score multiplier, offset, first and one past the last token it sees
  __shared__ int2 range_sm[NT];
  __shared__ int last_sm, abort_flag, even_sm;
  uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint2* const qsm = reinterpret_cast<uint2*>(ring + L::kRing);   // [NT][kSteps][32] fragments

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  uint64_t* const bar = bars[warp];
  uint8_t* const stage0 = ring + warp * NS * L::kStage;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NS; ++i) mbar_init(&bar[i], 1);
    mbar_fence_init();
    if (warp == 0) {
      abort_flag = 0;
      tma_prefetch_desc(&p.kmap);
      tma_prefetch_desc(&p.vmap);
    }
  }
  pdl_trigger();
  // (kOwn starts beside the groups' launch, every CTA of which has seen the work before it complete when this one
  // begins; it waits for that launch at its end.  The fence, of acquire too, leaves nothing older in this SM's L1 cache for the
  // ordinary loads behind it.)
  if (kMode != kOwn) pdl_wait();
  else __threadfence();
  // CTAs that take part.
  const int room = kMode == kOwn ? min((int)gridDim.x, own_sms(p, prefix_sms<kThreads>(p, ring)) * L::kCtas) : (int)gridDim.x;

  if (kMode == kOwn) fence_async_shared();   // (the scratch of prefix_sms lies where copies will land)

  // ---------------------------------------------------------------- this CTA's run of units
  const int per = (p.step.seqs + kThreads - 1) / kThreads;   // sequences a thread scans
  const int s0 = min(p.step.seqs, (int)threadIdx.x * per), s1 = min(p.step.seqs, s0 + per);
  long long mine = 0;
  int items = 0, longest = 0;
  Span x;   // the last sequence that this thread looked at
  for (int b = s0; b < s1; ++b) {
    x = load_span<L, kMode>(p, b);
    mine += (long long)x.tiles * x.span;
    items = (int)min((long long)items + (long long)x.tiles * p.kv_heads, 1LL << 20);   // (more than any grid: all alike)
    if (x.tiles > 0) longest = max(longest, x.units);
  }
  mine *= p.kv_heads;
  long long incl = mine;
  int incl_items = items;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    const int ti = __shfl_up_sync(0xffffffffu, incl_items, o);
    if (lane >= o) incl += t, incl_items += ti;
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) scan_sm[warp] = incl, items_sm[warp] = make_int2(incl_items, longest);
  __syncthreads();
  long long before = incl - mine, U = 0;
  int before_items = incl_items - items, all_items = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan_sm[w], before_items += items_sm[w].x;
    U += scan_sm[w];
    all_items += items_sm[w].x;
    longest = max(longest, items_sm[w].y);
  }
  // Few short items: one to a CTA, at the length of the longest, and no parts to join.
  int even = 0;
  if (longest <= L::kWhole && all_items <= room) {
    even = L::kLead + longest;
    before = (long long)before_items * even, mine = (long long)items * even, U = (long long)all_items * even;
    x.span = even;
  }
  const int ctas = even ? all_items : (int)min((long long)room, U);
  if ((int)blockIdx.x >= ctas) {
    if (kMode == kOwn && blockIdx.x == 0) pdl_wait();
    return;
  }
  if (threadIdx.x == 0) even_sm = even;
  const Runs runs(U, ctas);
  const long long u0 = runs.begin(blockIdx.x), u1 = runs.begin(blockIdx.x + 1);
  if (u0 >= before && u0 < before + mine) {
    // The sequence of this thread's that holds u0.
    long long at = before;
    int b = s0;
    for (; per > 1; ++b) {
      x = load_span<L, kMode>(p, b);
      if (even) x.span = even;
      const long long n = (long long)x.tiles * x.span * p.kv_heads;
      if (u0 < at + n) break;
      at += n;
    }
    start_sm.x = x;
    start_sm.b = b;
    start_sm.u = at;
  }
  __syncthreads();
  x = start_sm.x;
  int b = start_sm.b;
  long long seq_u0 = start_sm.u;            // first unit of sequence b
  uint32_t count = 0;                       // granules this warp has taken (ring position and phase)
  bool dead = false;                        // a wait ran out: only the bookkeeping goes on

  for (long long u = u0; u < u1;) {
    // ---------------------------------------------------------------- the next segment: one item's part of the run
    while (u >= seq_u0 + (long long)x.tiles * x.span * p.kv_heads) {
      seq_u0 += (long long)x.tiles * x.span * p.kv_heads;
      x = load_span<L, kMode>(p, ++b);
      if (even_sm) x.span = even_sm;
    }
    const int item = (int)quotient(u - seq_u0, x.span);
    const long long item_u0 = seq_u0 + (long long)item * x.span;   // its lead, then its units
    const int ub = max((int)(u - item_u0) - L::kLead, 0), ue = (int)min((long long)x.span, u1 - item_u0) - L::kLead;
    u = item_u0 + L::kLead + ue;
    if (ue <= ub) continue;   // the run ends within the lead
    const int h = item % p.kv_heads, tile = item / p.kv_heads;
    const int T0 = x.lo + ub * L::kUnit, T1 = min(x.hi, x.lo + ue * L::kUnit);
    const int granules = (T1 - T0 + kGranule - 1) / kGranule;
    const int mine_n = granules > warp ? (granules - warp + kWarps - 1) / kWarps : 0;
    const int rows_left = x.s.n * p.group - tile * L::kRows;   // rows of the tile that exist
    const int* const table = p.step.page_table + (size_t)b * p.step.table_width;

    // The page, scales and cache row of this warp's granule j, held by lane j % 32 (batches of 32,
    // two in registers: the ring runs ahead of the use).
    float ks_r[2], vs_r[2];
    uint32_t bad_r[2] = {0u, 0u};
    int row_r = 0;
    auto fetch = [&](int base) {
      const int j = base + lane;
      const int t = T0 + (warp + j * kWarps) * kGranule;
      bool bad = false;
      float a = 0.f, v = 0.f;
      row_r = 0;
      if (j < mine_n) {
        const int page = load<kMode == kOwn>(table + (t >> p.page_shift));
        bad = page < 0 || page >= p.pages;
        if (!bad) {
          const size_t at = (size_t)page * p.kv_heads + h;
          row_r = (int)(at << p.page_shift) + (t & ((1 << p.page_shift) - 1));
          a = load<kMode == kOwn>(p.ks + at);
          v = load<kMode == kOwn>(p.vs + at);
        } else {
          atomicOr(p.status, W8A8_DEV_BAD_INDEX);
        }
      }
      const uint32_t mask = __ballot_sync(0xffffffffu, bad);
      if ((base >> 5) & 1) ks_r[1] = a, vs_r[1] = v, bad_r[1] = mask;
      else ks_r[0] = a, vs_r[0] = v, bad_r[0] = mask;
    };
    // Copy granule j into its slot: by the lane that holds its row.  (A bad page's granule copies row
    // 0 of the cache and is masked.)
    auto issue = [&](int j) {
      if (lane == (j & 31)) {
        const uint32_t slot = (count + (uint32_t)j) % NS;
        uint8_t* const dst = stage0 + slot * L::kStage;
        mbar_arrive_expect_tx(&bar[slot], L::kStage);
#pragma unroll
        for (int i = 0; i < L::kBoxes; ++i) {
          tma_load_2d(dst + i * L::kBoxBytes, &p.kmap, 128 * i, row_r, &bar[slot]);
          tma_load_2d(dst + L::kSide + i * L::kBoxBytes, &p.vmap, 128 * i, row_r, &bar[slot]);
        }
      }
    };
    // ---------------------------------------------------------------- this segment's queries
    // Fragment B of step s, column g: slots (2c, 2c + 1) hold d0, d0 + 2 and slots (2c + 8, 2c + 9) hold
    // d0 + 1, d0 + 3, d0 = the first of the lane's word s: the order in which a key's four bytes come
    // apart.  A lane's words: D / 4 contiguous values (D = 256: 32 of each half).
    uint32_t qb[L::kQShared ? 1 : NT][kSteps][2];
    float m[NT][2], l[NT][2], r[NT][2], hs[NT][2];
    int full_lo = 0, full_hi = 0x7fffffff;   // tokens that every row sees
    // The loads of the queries go out before the first copies of the cache, which would delay them by
    // everything that the rings hold.
    // (Shared fragments: warp w prepares tile w; every warp holds its own otherwise.)
    constexpr int kMine = L::kQShared ? 1 : NT;
    static_assert(!L::kQShared || NT <= kWarps, "a warp for each shared tile");
    uint4 rows_raw[kMine][D / 32];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int row = (L::kQShared ? warp : i) * 8 + g;
      const bool live = row < rows_left && row < L::kRows;
      const int ri = tile * L::kRows + (live ? row : 0);
      const uint16_t* const src = p.q + (x.s.row0 + ri / p.group) * p.q_stride + (h * p.group + ri % p.group) * D;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const int d = D == 256 ? 128 * (w >> 2) + 32 * c + 8 * (w & 3) : (D / 4) * c + 8 * w;
        rows_raw[i][w] = live ? load<kMode == kOwn>(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (!dead && mine_n > 0) {
      fetch(0);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        if (j < mine_n) issue(j);
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (L::kQShared && warp >= NT) break;
      const uint4 (&raw)[D / 32] = rows_raw[i];
      float amax = 0.f;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        float f[8];
        unpack8<kF16>(raw[w], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int ex = max((int)(__float_as_uint(amax) >> 23) - 127 - 13, -100);
      const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        float f[8];
        unpack8<kF16>(raw[w], f);
        __half hf[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          hf[k] = __float2half_rn(f[k] * down);
          sum += __half2float(hf[k]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const __half2 lo = __halves2half2(hf[4 * k], hf[4 * k + 2]), hi = __halves2half2(hf[4 * k + 1], hf[4 * k + 3]);
          const uint32_t b0 = *reinterpret_cast<const uint32_t*>(&lo), b1 = *reinterpret_cast<const uint32_t*>(&hi);
          if (L::kQShared) {
            qsm[(warp * kSteps + 2 * w + k) * 32 + lane] = make_uint2(b0, b1);
          } else {
            qb[L::kQShared ? 0 : i][2 * w + k][0] = b0;
            qb[L::kQShared ? 0 : i][2 * w + k][1] = b1;
          }
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      // score (in powers of two) = (acc - offs) * rowmul * k_scale
      // The row's own: by one lane of one warp (every warp works out the same where it holds all tiles).
      const int row = (L::kQShared ? warp : i) * 8 + g;
      const bool live = row < rows_left;
      const int pos = x.s.len - x.s.n + (tile * L::kRows + row) / p.group;
      const int end = !live ? 0x7fffffff : p.causal ? min(pos + 1, x.s.len) : x.s.len;
      const int beg = live && p.window > 0 ? max(0, pos - p.window + 1) : 0;
      if (c == 0 && (L::kQShared || warp == 0))
        row_st[row] = make_float4(p.scale_log2 * 16777216.f * __uint_as_float((uint32_t)(127 + ex) << 23), sum * (128.f / 16777216.f),
                                  __int_as_float(beg), __int_as_float(end));
      full_hi = min(full_hi, end);
      full_lo = max(full_lo, beg);
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[i][e] = kFloor;
        r[i][e] = kFloor;
        l[i][e] = 0.f;
        hs[i][e] = 0.f;
      }
    }
    full_hi = __reduce_min_sync(0xffffffffu, full_hi);
    full_lo = __reduce_max_sync(0xffffffffu, full_lo);
    if (L::kQShared) {
      // A warp has seen its own tile's rows alone.
      if (lane == 0 && warp < NT) range_sm[warp] = make_int2(full_lo, full_hi);
    }
    __syncthreads();
    if (L::kQShared) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        full_lo = max(full_lo, range_sm[i].x);
        full_hi = min(full_hi, range_sm[i].y);
      }
    }
    float o[NT][kSteps][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int n = 0; n < kSteps; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][n][k] = 0.f;

    // ---------------------------------------------------------------- the granules
    // Scores (before their scales) of granule j: tokens T + g and T + g + 8, rows 2c and 2c + 1 of each tile; two
    // chains of products where one tile alone would wait for each of its own.  False when the wait ran out.
    constexpr int kChains = NT == 1 ? 2 : 1;
    auto scores = [&](int j, float (&s)[NT][kChains][4]) {
      const uint32_t slot = (count + (uint32_t)j) % NS, phase = ((count + (uint32_t)j) / NS) & 1u;
      const uint8_t* const kst = stage0 + slot * L::kStage;
      const bool got = mbar_wait(&bar[slot], phase, &abort_flag, p.status);
      if (!__all_sync(0xffffffffu, got)) return false;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int t = 0; t < kChains; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][t][k] = 0.f;
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {    // 16 bytes of each of the two tokens
        uint4 kb[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int row = 8 * t + g;
          if (D == 64) kb[t] = *reinterpret_cast<const uint4*>(kst + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
          else kb[t] = *reinterpret_cast<const uint4*>(kst + (w >> 1) * L::kBoxBytes + row * 128 + (((2 * c + (w & 1)) ^ (row & 7)) << 4));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t w0 = k == 0 ? kb[0].x : k == 1 ? kb[0].y : k == 2 ? kb[0].z : kb[0].w;
          const uint32_t w1 = k == 0 ? kb[1].x : k == 1 ? kb[1].y : k == 2 ? kb[1].z : kb[1].w;
          const uint32_t a0 = w0 & 0x00FF00FFu, a1 = w1 & 0x00FF00FFu;
          const uint32_t a2 = __byte_perm(w0, 0u, 0x4341), a3 = __byte_perm(w1, 0u, 0x4341);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            uint2 q;
            if (L::kQShared) q = qsm[(i * kSteps + 4 * w + k) * 32 + lane];
            else q = make_uint2(qb[L::kQShared ? 0 : i][4 * w + k][0], qb[L::kQShared ? 0 : i][4 * w + k][1]);
            mma_f16_16816(s[i][k % kChains], a0, a1, a2, a3, q.x, q.y);
          }
        }
      }
      return true;
    };
    // A wait that runs out is recorded in the status word.  The copies in flight land before this CTA's shared
    // memory is given back; no more are issued.
    auto give_up = [&](int j) {
      dead = true;
      for (int i = j; i < min(j + NS, mine_n); ++i)
        mbar_wait_drain(&bar[(count + (uint32_t)i) % NS], ((count + (uint32_t)i) / NS) & 1u, p.status);
    };
    // Granule j takes the slot that this warp has read.  The copy's writes are of the asynchronous proxy: without
    // the fence they can overtake the lanes' reads, which a barrier of the warp alone does not hold up (seen as a
    // granule's values replaced by those of the one after it in the slot, in one of 10^5).  After the products the
    // reads have long returned and the fence costs nothing (before them 24 rows 40.2 -> 43.8 us, heads of 64 24.3 ->
    // 24.6).
    auto refill = [&](int j) {
      fence_async_shared();
      __syncwarp();
      if (j >= mine_n) return;
      if ((j & 31) == 0) fetch(j);
      issue(j);
    };
    float sn[NT][kChains][4];
    if (L::kAhead && mine_n > 0 && !dead && !scores(0, sn)) give_up(0);
    for (int j = 0; j < mine_n && !dead; ++j) {
      if (!L::kAhead && !scores(j, sn)) {
        give_up(j);
        break;
      }
      const uint8_t* const vst = stage0 + ((count + (uint32_t)j) % NS) * L::kStage + L::kSide;
      const int T = T0 + (warp + j * kWarps) * kGranule;
      const int par = (j >> 5) & 1;
      const float ks = __shfl_sync(0xffffffffu, par ? ks_r[1] : ks_r[0], j & 31);
      const float vs = __shfl_sync(0xffffffffu, par ? vs_r[1] : vs_r[0], j & 31);
      const bool bad = ((par ? bad_r[1] : bad_r[0]) >> (j & 31)) & 1u;
      float s[NT][4];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] = kChains == 2 ? sn[i][0][k] + sn[i][kChains - 1][k] : sn[i][0][k];
      if (L::kAhead && j + 1 < mine_n && !scores(j + 1, sn)) {
        give_up(j + 1);
        break;
      }
      const bool edge = T < full_lo || T + kGranule > full_hi || bad;
      const float lvs = lg2(fabsf(vs));   // (a weight has the sign of its page's scale)
      uint32_t pb[NT][2];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        float mx[2], f[2], z[4];   // z: scores in powers of two
        bool move = false, far = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float4 st = row_st[8 * i + 2 * c + e];
          const float c1 = ks * st.x;
          const float c0 = -st.y * c1;
#pragma unroll
          for (int t = 0; t < 2; ++t) z[2 * t + e] = fmaf(s[i][2 * t + e], c1, c0);
          if (edge) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int tok = T + 8 * t + g;
              if (bad || tok < __float_as_int(st.z) || tok >= __float_as_int(st.w)) z[2 * t + e] = -INFINITY;
            }
          }
          mx[e] = fmaxf(z[e], z[2 + e]);
          f[e] = hs[i][e] * vs;
          move = move || mx[e] > m[i][e] + kSlack || mx[e] + lvs > r[i][e] + kRoom || fabsf(f[e]) > kFar;
        }
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], w));
            if (mx[e] > m[i][e] + kSlack) {
              l[i][e] *= ex2(m[i][e] - mx[e]);
              m[i][e] = mx[e];
            }
            const float want = mx[e] + lvs;
            float rn = want > r[i][e] + kRoom ? want - kHead : r[i][e];
            rn = fminf(fmaxf(rn, m[i][e] - kBelow), m[i][e] + kAbove);
            const float a = ex2(r[i][e] - rn);
            r[i][e] = rn;
            hs[i][e] = ex2(m[i][e] - rn);
            f[e] = hs[i][e] * vs;
#pragma unroll
            for (int n = 0; n < kSteps; ++n) {
              o[i][n][e] *= a;
              o[i][n][2 + e] *= a;
            }
          }
          far = __any_sync(0xffffffffu, fabsf(f[0]) > kFar || fabsf(f[1]) > kFar);
        }
        float w[4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float pr = ex2(z[2 * t + e] - m[i][e]);
            l[i][e] += pr;
            w[2 * t + e] = pr * f[e];
            if (far && fabsf(f[e]) > kFar) w[2 * t + e] = copysignf(ex2(z[2 * t + e] + lvs - r[i][e]), vs);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const __half2 v = __floats2half2_rn(w[2 * t], w[2 * t + 1]);
          pb[i][t] = transpose8(*reinterpret_cast<const uint32_t*>(&v));   // tokens 2c, 2c + 1 (+ 8 t) of row g
        }
      }

      // Values: the lane takes 16 (8 for D = 64) contiguous d of tokens 2c, 2c + 1, 2c + 8, 2c + 9; a
      // matrix instruction's 16 rows are two of each lane's d, so its sums are contiguous too.
      constexpr int kWords = D == 64 ? 2 : 4;
#pragma unroll
      for (int bx = 0; bx < L::kBoxes; ++bx) {
        uint32_t vw[4][kWords];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int row = 2 * c + (t & 1) + 8 * (t >> 1);
          if (D == 64) {
            const uint2 v = *reinterpret_cast<const uint2*>(vst + row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
            vw[t][0] = v.x, vw[t][1] = v.y;
          } else {
            const uint4 v = *reinterpret_cast<const uint4*>(vst + bx * L::kBoxBytes + row * 128 + ((g ^ (row & 7)) << 4));
            vw[t][0] = v.x, vw[t][1] = v.y, vw[t][kWords - 2] = v.z, vw[t][kWords - 1] = v.w;
          }
        }
#pragma unroll
        for (int wd = 0; wd < kWords; ++wd) {
          uint32_t bf[2][4];   // [tokens 2c.. / 2c + 8..][d]
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t x01 = __byte_perm(vw[2 * t][wd], vw[2 * t + 1][wd], 0x5140);
            const uint32_t x23 = __byte_perm(vw[2 * t][wd], vw[2 * t + 1][wd], 0x7362);
            offset_bytes_to_half2_pairs(x01, bf[t][0], bf[t][1]);
            offset_bytes_to_half2_pairs(x23, bf[t][2], bf[t][3]);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < NT; ++i)
              mma_f16_16816(o[i][(bx * kWords + wd) * 2 + k], bf[0][2 * k], bf[0][2 * k + 1], bf[1][2 * k], bf[1][2 * k + 1], pb[i][0],
                            pb[i][1]);
        }
      }
      refill(j + NS);
    }
    count += (uint32_t)mine_n;

    // ---------------------------------------------------------------- join the warps, then the CTAs
    const bool whole = ub == 0 && ue >= x.units;
    const int slot = item_u0 <= u0 ? 0 : 1;   // the run's first segment, or its last
    float* const part = p.parts + ((size_t)blockIdx.x * 2 + slot) * L::kPart;
    float* const buf = reinterpret_cast<float*>(ring);
    const int rows = min(rows_left, L::kRows);
    __syncthreads();   // the rings hold no copy in flight: every granule issued has been waited for
#pragma unroll
    for (int i = 0; i < NT; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = l[i][e];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) t += __shfl_xor_sync(0xffffffffu, t, w);
        const int row = 8 * i + 2 * c + e;
        if (g == 0) mlr_sm[warp][row] = make_float4(m[i][e], t, r[i][e], 0.f);
        if (row < rows) {
          // A lane's sums of a row: D / 8 contiguous ones (D = 256: 16 of each half).
          float* const dst = buf + (warp * L::kRows + row) * L::kRow;
          constexpr int kTiles = D == 64 ? 4 : 8;   // output tiles of a box
#pragma unroll
          for (int n = 0; n < kSteps; n += 2)
            *reinterpret_cast<float4*>(dst + (n / kTiles) * 128 + 2 * kTiles * g + 2 * (n % kTiles)) =
                make_float4(o[i][n][e], o[i][n][2 + e], o[i][n + 1][e], o[i][n + 1][2 + e]);
        }
      }
    }
    __syncthreads();
    constexpr int kVec = D / 4;   // threads of a row, four values each
    for (int i = threadIdx.x; i < rows * kVec; i += kThreads) {
      const int row = i / kVec, d = 4 * (i % kVec);
      float M = kFloor, Rf = kFloor;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        M = fmaxf(M, mlr_sm[w][row].x);
        Rf = fmaxf(Rf, mlr_sm[w][row].z);
      }
      float lt = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        lt += mlr_sm[w][row].y * ex2(mlr_sm[w][row].x - M);
        const float a = ex2(mlr_sm[w][row].z - Rf);
        const float4 v = *reinterpret_cast<const float4*>(buf + (w * L::kRows + row) * L::kRow + d);
        acc.x = fmaf(v.x, a, acc.x), acc.y = fmaf(v.y, a, acc.y), acc.z = fmaf(v.z, a, acc.z), acc.w = fmaf(v.w, a, acc.w);
      }
      if (whole) {
        store_row<kF16, kMode>(p, x.s.row0, tile * L::kRows + row, h, d, D, acc, M, lt, Rf);
      } else {
        *reinterpret_cast<float4*>(part + row * D + d) = acc;
        if (d == 0) *reinterpret_cast<float4*>(part + L::kRows * D + row * 4) = make_float4(M, lt, Rf, 0.f);
      }
    }
    if (!whole) {
      // The part is written.  The item's parts (one of each of n consecutive CTAs) join in the CTAs' order: up to
      // kGroup of them by the last CTA to arrive; more of them first in groups of about sqrt(n), each by the last
      // of its CTAs, so that no CTA reads more than a few (131071 tokens, 57 parts of 16 rows: 81.5 us without
      // groups, 63.4 with them).
      constexpr int kGroup = 8;
      const int first = runs.owner(item_u0 + L::kLead), n = runs.owner(item_u0 + x.span - 1) - first + 1;
      const int first_slot = item_u0 <= runs.begin(first) ? 0 : 1;
      int group = n;
      if (n > kGroup) {
        group = kGroup;
        while (group * group < n) ++group;
      }
      const int groups = (n + group - 1) / group;
      // Part i: of CTA first + i, in its first place (the first CTA's: in the place of its last segment unless the
      // item begins its run).
      auto part_of = [&](int i) { return p.parts + ((size_t)(first + i) * 2 + (i == 0 ? first_slot : 0)) * L::kPart; };
      const int mine = (int)blockIdx.x - first, lead = mine / group * group;
      int base = lead, step = 1, count_n = min(group, n - lead);
      uint32_t* counter = groups > 1 ? p.group_counters + 2 * (first + lead) + (lead == 0 ? first_slot : 0) : p.counters + first;
      for (bool top = groups == 1;; top = true) {
        // (The barrier orders the CTA's stores before thread 0's release, and its acquire before the reads.)
        __syncthreads();
        if (threadIdx.x == 0) {
          const uint32_t old = atom_add_acq_rel_u32(counter, 1u);
          if (old >= (uint32_t)count_n) atomicOr(p.status, W8A8_DEV_COUNTER_CORRUPT);
          if (old == (uint32_t)count_n - 1) *counter = 0u;   // ready for the next call
          last_sm = old == (uint32_t)count_n - 1;
        }
        __syncthreads();
        if (!last_sm) break;
        // Threads take four values of a row at kB places at once, kP parts of each in flight.
        constexpr int kVec = D / 4, kPlaces = (L::kRows * kVec + kThreads - 1) / kThreads;
        constexpr int kB = kPlaces < 2 ? 1 : 2, kP = kB == 1 && D * NT == 128 ? 8 : 4;
        for (int at0 = threadIdx.x; at0 < rows * kVec; at0 += kB * kThreads) {
          float M[kB], Rf[kB], lt[kB];
          float4 acc[kB];
#pragma unroll
          for (int y = 0; y < kB; ++y) M[y] = kFloor, Rf[y] = kFloor, lt[y] = 0.f, acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int i = 0; i < count_n; i += kP) {
            float4 t[kP][kB], v[kP][kB];
#pragma unroll
            for (int z = 0; z < kP; ++z) {
              const float* const src = part_of(base + step * min(i + z, count_n - 1));
#pragma unroll
              for (int y = 0; y < kB; ++y) {
                const int at = at0 + y * kThreads;
                t[z][y] = make_float4(kFloor, 0.f, kFloor, 0.f);
                v[z][y] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i + z < count_n && at < rows * kVec) {
                  t[z][y] = __ldcg(reinterpret_cast<const float4*>(src + L::kRows * D) + at / kVec);
                  v[z][y] = __ldcg(reinterpret_cast<const float4*>(src) + at);
                }
              }
            }
#pragma unroll
            for (int y = 0; y < kB; ++y) {
              float mn = M[y], rn = Rf[y];
#pragma unroll
              for (int z = 0; z < kP; ++z) mn = fmaxf(mn, t[z][y].x), rn = fmaxf(rn, t[z][y].z);
              const float a0 = ex2(Rf[y] - rn);
              lt[y] *= ex2(M[y] - mn);
              acc[y].x *= a0, acc[y].y *= a0, acc[y].z *= a0, acc[y].w *= a0;
              M[y] = mn;
              Rf[y] = rn;
#pragma unroll
              for (int z = 0; z < kP; ++z) {
                lt[y] = fmaf(t[z][y].y, ex2(t[z][y].x - mn), lt[y]);
                const float a = ex2(t[z][y].z - rn);
                acc[y].x = fmaf(v[z][y].x, a, acc[y].x), acc[y].y = fmaf(v[z][y].y, a, acc[y].y);
                acc[y].z = fmaf(v[z][y].z, a, acc[y].z), acc[y].w = fmaf(v[z][y].w, a, acc[y].w);
              }
            }
          }
#pragma unroll
          for (int y = 0; y < kB; ++y) {
            const int at = at0 + y * kThreads;
            if (at >= rows * kVec) continue;
            const int row = at / kVec, d = 4 * (at % kVec);
            if (top) {
              store_row<kF16, kMode>(p, x.s.row0, tile * L::kRows + row, h, d, D, acc[y], M[y], lt[y], Rf[y]);
            } else {
              // The group's sums take the place of its first part's; its statistics once every thread has read them.
              *(reinterpret_cast<float4*>(part_of(base)) + at) = acc[y];
              if (d == 0) mlr_sm[0][row] = make_float4(M[y], lt[y], Rf[y], 0.f);
            }
          }
        }
        if (top) break;
        __syncthreads();
        for (int row = threadIdx.x; row < rows; row += kThreads)
          *(reinterpret_cast<float4*>(part_of(base) + L::kRows * D) + row) = mlr_sm[0][row];
        base = 0, step = group, count_n = groups;
        counter = p.counters + first;
      }
      __syncthreads();
    }
    if (u < u1) {
      // The join buffer lies over the rings: plain accesses to it come before the next copies.
      fence_async_shared();
      __syncthreads();
    }
  }
  if (kMode == kOwn && blockIdx.x == 0) pdl_wait();   // (the grid is not complete before it)
}

template <bool kF16, int D, int NT, Mode kMode>
static cudaError_t launch_few(const Params& p, int sms, cudaStream_t stream) {
  using L = Layout<D, NT, kMode>;
  auto kern = kv8_attention_kernel<kF16, D, NT, kMode>;
  cudaError_t e = ensure_smem_attribute((const void*)kern, L::kSmem);
  if (e != cudaSuccess) return e;
  // No more CTAs than units there can be (lengths are known to the device alone).
  const long long tiles = ((long long)p.step.max_tokens * p.group + L::kRows - 1) / L::kRows;
  const long long units = (((long long)p.step.table_width << p.page_shift) + L::kUnit - 1) / L::kUnit;
  const long long most = tiles * units >= sms * L::kCtas ? sms * L::kCtas : tiles * units * p.step.seqs * p.kv_heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(most < sms * L::kCtas ? most : sms * L::kCtas));
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = (size_t)L::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Whether the other kernel takes a step of `rows` rows of a sequence and kv head: enough rows for its tiles of 128, and
// enough tiles, as the parts of a tile cut over many CTAs cost it more to join than its products save.  Measured (us,
// here / there): heads of 128, 16 contexts of 2000, 8 kv heads (128 tiles) 40 rows 62 / 51, 128 rows 111 / 62; 8 of 500 (64
// tiles) 40 rows 21.6 / 22.2, 128 rows 30.1 / 29.6; 2 of 6000, 2 kv heads (4) 40 rows 25 / 29, 192 rows (8) 32 / 54; one of
// 16000, 4 kv heads, 192 rows 52 / 59.  Heads of 256 (16 rows a tile here): 8 of 3000, 4 kv heads 128 rows (32) 78 / 88, 192
// (64) 110 / 92; 2 of 6000, 2 kv heads 512 rows 74 / 96, 768 rows 103 / 101.
static bool takes_many(const Params& p, int head_dim, long long rows) {
  const long long fewest = head_dim == 256 ? 112 : 32, sure = head_dim == 256 ? 768 : 256;
  return rows > sure || (rows > fewest && (rows + 127) / 128 * p.step.seqs * p.kv_heads >= 64);
}

// The narrowest variant that holds a sequence's rows in one tile, else the widest.
template <bool kF16, Mode kMode>
static cudaError_t launch_rows(const Params& p, int head_dim, int sms, cudaStream_t s) {
  const long long rows = (long long)p.step.max_tokens * p.group;
  if (kMode == kPlain && takes_many(p, head_dim, rows)) return launch_many(p, head_dim, kF16, sms, s);
  if (head_dim == 64)
    return rows <= 8    ? launch_few<kF16, 64, 1, kMode>(p, sms, s)
           : rows <= 16 ? launch_few<kF16, 64, 2, kMode>(p, sms, s)
           : rows <= 24 ? launch_few<kF16, 64, 3, kMode>(p, sms, s)
                        : launch_few<kF16, 64, 4, kMode>(p, sms, s);
  if (head_dim == 128)
    return rows <= 8    ? launch_few<kF16, 128, 1, kMode>(p, sms, s)
           : rows <= 16 ? launch_few<kF16, 128, 2, kMode>(p, sms, s)
           : rows <= 24 ? launch_few<kF16, 128, 3, kMode>(p, sms, s)
                        : launch_few<kF16, 128, 4, kMode>(p, sms, s);
  return rows <= 8 ? launch_few<kF16, 256, 1, kMode>(p, sms, s) : launch_few<kF16, 256, 2, kMode>(p, sms, s);
}

}  // namespace attn
}  // namespace w8a8
