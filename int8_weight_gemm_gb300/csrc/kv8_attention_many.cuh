// Attention over the 8-bit paged key-value cache: many query rows (prompts, long verify windows), on the
// fifth-generation tensor cores (tcgen05, sm_103a).  The operator is that of kv8_attention_few.cuh.
//
// What bounds it: a cached byte feeds 2 (rows that share its head) multiply-adds, so from some 300 rows
// on the products do: a block of 128 tokens against 128 rows is 2 x 128 x 128 x D multiply-adds, 1024
// tensor cycles at D = 128, beside 16384 exponentials.
//
// Mathematics.  A tile is 128 of the n * G rows that share a kv head, a block 128 cached tokens.
//  S = Q K^T: both operands fp16 in shared memory (128-byte swizzle, K-major), fp32 accumulators in
//  tensor memory.  A query row is scaled by a power of two into [2^13, 2^14) (exact); keys and values are
//  the integers b - 128 (exact), their signs turned where a page's scale is negative.
//  Weights: p = 2^(s - m) sums to l in fp32, w = p * (v_scale * 2^(m - r)), rounded to fp16, goes back into
//  tensor memory over the scores it came from and is the first operand of O += W V.  The references m and r
//  of a row are those of the other kernel, for the same reasons: they move when a score or weight passes
//  where they were put by 2^8, and only then is O (and the weights already written of that block) rescaled, once the
//  products that add to O have completed.
//
// Layout and split.  One CTA an SM, all of its tensor memory: two streams of scores and outputs, each with
// four softmax warps (a thread is a row).  With more than 128 rows the streams are two row tiles over the
// same blocks; with up to 128 they are the even and the odd blocks of one tile, joined at the end, so that
// one stream's exponentials always run under the other's products.  Further warps:
//  - producer: page numbers and scales of four blocks in one load a lane, then a tensor-map box a granule
//    into a ring of 8-bit blocks (keys and values in turn);
//  - four converter warps: 8 bits -> fp16 operands, two blocks of each ahead of the products;
//  - one thread issues the products: W V of a block, then, when those have completed (the other stream's
//    are in the pipe meanwhile), the next scores into the same tensor memory.
// Heads of 256: the sums take half of tensor memory, so there is one stream, of one tile, with two places for the
// scores of a block of 64 tokens: the next block's scores are there when a block's weights are done.  Four warps do the
// exponentials and eight convert.  (Two prompts of 2048 on contexts of 6000, 16 query heads, 4 kv heads: 504 us, 663
// TFLOP/s; two streams of half the columns each, scoring twice, 886; 16 rows a warp 1923.)
// The work is cut like that of the other kernel: items (row tile, kv head) laid end to end in units of a
// block and cut into equal runs; an item cut across CTAs is finished by the last to arrive, parts joined
// in the CTAs' order, so replays give the same bits.
//
// Measured (32 query heads, 8 kv heads of 128): two prompts of 1900-2048 tokens on contexts of 5800-6144 422 us, 791
// TFLOP/s, 41 % of a large matrix product's rate.  What bounds it is a stream's chain (scores, weights, sums: four waits
// that wake a role, 250 cycles each, beside 2600 cycles of exponentials a block); the tensor pipe is busy 34 % of the
// time.
#pragma once

#include "kv8_attention.cuh"

namespace w8a8 {
namespace attn {

constexpr int kTileRows = 128;    // rows of a tile
constexpr int kProducerWarp = 12;   // after the softmax warps and the converters
constexpr int kMmaWarp = kProducerWarp + 1;
constexpr int kTcThreads = 32 * (kMmaWarp + 1);
constexpr int kScales = 8;        // blocks whose scales are held

template <int D, int kTiles>
struct TcLayout {
  static constexpr int kRows = kTiles * kTileRows;
  // Heads of 256: one stream with two places for scores, blocks of 64 tokens.
  static constexpr bool kWide = D > 128;
  static constexpr int kSoftWarps = kWide ? 4 : 8;    // four for each stream
  static constexpr int kConvWarps = 12 - kSoftWarps;
  static constexpr int kBox = D < 128 ? D : 128;      // columns of a copy
  static constexpr int kBoxes = D / kBox;
  static constexpr int kBlock = kWide ? 64 : 128;     // tokens of a block
  static constexpr int kGrans = kBlock / kGranule;    // granules of a block
  static constexpr int kUnit = kBlock;
  static constexpr int kLead = 3;
  static constexpr int kQBytes = kTileRows * D * 2;
  static constexpr int kHalf = kBlock * 128;          // 64 fp16 of each of a block's tokens
  static constexpr int kBlk16 = kBlock * D * 2;   // an fp16 block
  static constexpr int kSlot = kBlock * D;            // an 8-bit block
  // 8-bit blocks in flight: with one tile the cache comes from HBM at the pace of the products.
  static constexpr int kSlots = kTiles == 2 || kWide ? 2 : 4;
  static constexpr int kBytes = 1024 + kTiles * kQBytes + 4 * kBlk16 + kSlots * kSlot;
  static constexpr int kSCol = 0, kOCol = kWide ? 256 : kBlock, kStreamCols = 256;   // tensor-memory columns of a stream
  static constexpr int kPart = kRows * (D + 4);       // floats: sums, then (m, l, r, -) of each row
  static_assert(kBytes + 2048 <= 232448, "shared memory");
};

// One tile's tokens.
struct TileSpan {
  int lo, hi, units;
};

template <typename L, Mode kMode>
__device__ __forceinline__ TileSpan tile_span(const Params& p, const Rows& s, int tile) {
  TileSpan t;
  if (kMode == kPrefixes) {
    t.lo = 0;
    t.hi = s.len;
    t.units = max(1, (s.len + L::kBlock - 1) / L::kBlock);
    return t;
  }
  const int first = (int)quotient((long long)tile * L::kRows, p.group);
  const int last = min(s.n - 1, (int)quotient((long long)tile * L::kRows + L::kRows - 1, p.group));
  t.hi = p.causal ? max(0, s.len - s.n + last + 1) : s.len;
  t.lo = p.window > 0 ? max(0, s.len - s.n + first - p.window + 1) & ~(kGranule - 1) : s.lo;
  t.units = max(1, (t.hi - t.lo + L::kBlock - 1) / L::kBlock);
  return t;
}

template <typename L>
__device__ __forceinline__ int tiles_of(const Params& p, const Seq& s) {
  return (int)quotient((long long)s.n * p.group + L::kRows - 1, L::kRows);
}

// One segment, as the producer hands it to the other roles (nb = 0: the run is over).
struct Segment {
  int nb;                    // blocks
  int T0;                    // first token
  int row0, pos0, len;       // of the sequence: first row, position of its first row, cached tokens
  int h, tile, rows;         // kv head, row tile, rows of the tile that exist
  int whole;                 // the item's only part
  int slot;                  // else: its place among this CTA's parts,
  int first, parts, slot0;   //   and the item's first CTA, number of CTAs, and place in the first one
};
constexpr int kSegments = 4;   // segments under way

// A run's segments, one item's part each.  Items are ordered by sequence, kv head, row tile.
template <typename L, Mode kMode>
struct Walk {
  long long u, u1, item_u0;
  Rows s;
  TileSpan t;
  int b, h, tile, tiles, ub, ue;
  // Set on the item (b, h, tile) that begins at item_u0 at or before u.
  __device__ bool next(const Params& p) {
    while (u < u1) {
      while (u >= item_u0 + L::kLead + t.units) {
        item_u0 += L::kLead + t.units;
        if (++tile == tiles) {
          tile = 0;
          if (++h == p.kv_heads) {
            h = 0;
            do {
              load_rows<kMode>(p, ++b, s);
              tiles = tiles_of<L>(p, s);
            } while (tiles == 0);
          }
        }
        t = tile_span<L, kMode>(p, s, tile);
      }
      const int span = L::kLead + t.units;
      ub = max((int)(u - item_u0) - L::kLead, 0);
      ue = (int)min((long long)span, u1 - item_u0) - L::kLead;
      u = item_u0 + L::kLead + ue;
      if (ue > ub) return true;   // else the run ends within the lead
    }
    return false;
  }
  __device__ bool whole() const { return ub == 0 && ue == t.units; }
};

// 32 consecutive tensor-memory columns of this thread's lane (warp-wide); no wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,"
      "%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
        "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
// Wait for this thread's loads; the registers of one of them are operands, so that nothing that uses them
// is moved before it.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                 "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                 "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
// D[tmem_d] (+)= A[desc_a] * B[desc_b]^T, both operands in shared memory.  Issued by one thread.
__device__ __forceinline__ void umma_f16_ss(uint32_t tmem_d, uint64_t desc_a, uint64_t desc_b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(tmem_d),
      "l"(desc_a), "l"(desc_b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// One lane of the converged warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(on));
  return on != 0;
}

// Shared-memory descriptors with the 128-byte swizzle (rows of 128 bytes, atoms of 8 rows, 1024-byte
// aligned; version 1 in bits 46..47, layout 2 in bits 61..63).  K-major: the rows are the operand's rows,
// 64 of k each; atoms of rows 1024 bytes apart (stride field).
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}
// MN-major: the rows are k, 64 of n each; atoms of 8 k are 1024 bytes apart (stride field), the next 64 of
// n `lead` bytes (leading-dimension field).
__device__ __forceinline__ uint64_t desc_mnmajor(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)2 << 61);
}

__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  const bool ok = mbar_wait(bar, parity, abort, status);
  return __all_sync(0xffffffffu, ok) != 0;
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The rare step of a softmax warp when some row's reference r has moved: the sums O (`cols` columns; 0 for a
// first block) and the `chunks` x 16 columns of weights already written of this block, times the row's factor.
static __device__ __noinline__ void rescale(uint32_t t_o, int cols, uint32_t t_w, int chunks, float down) {
  tc_fence_after();
#pragma unroll 1
  for (int c = 0; c < cols; c += 16) {
    uint32_t o[16];
    tmem_ld16(t_o + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * down);
    tmem_st16(t_o + c, o);
  }
  tmem_wait_st();
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    uint32_t o[16];
    tmem_ld16(t_w + 16 * c, o);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 w = __half22float2(*reinterpret_cast<const __half2*>(&o[k]));
      o[k] = pack2<true>(w.x * down, w.y * down);
    }
    tmem_st16(t_w + 16 * c, o);
  }
  tmem_wait_st();
}

// Granule scales of a block, as the softmax and converter warps use them.
struct alignas(16) GranScale {
  float ks, vs;   // magnitudes
  float lvs;      // log2 vs
  float bias;     // of the scores: 0, or -inf where the granule is left out
};

template <bool kF16, int D, int kTiles, Mode kMode>
__global__ void __launch_bounds__(kTcThreads, 1) kv8_attention_tc_kernel(const __grid_constant__ Params p) {
  using L = TcLayout<D, kTiles>;
  constexpr int kSlots = L::kSlots, kBlock = L::kBlock, kGrans = L::kGrans, kSoftWarps = L::kSoftWarps, kConvWarps = L::kConvWarps;
  constexpr bool kWide = L::kWide, kAlternate = kTiles == 1 && !kWide;   // (the streams are one tile's even and odd blocks)
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t slot_full[kSlots], slot_empty[kSlots];   // 8-bit blocks
  __shared__ __align__(8) uint64_t sc_full[kScales];                        // scales of a block
  __shared__ __align__(8) uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];   // fp16 blocks
  __shared__ __align__(8) uint64_t q_full[2], s_full[2], p_ready[2], pv_done[2];   // of each stream
  __shared__ __align__(8) uint64_t seg_full[kSegments], seg_empty[kSegments];
  __shared__ __align__(8) uint64_t join_bar, final_bar;
  __shared__ Segment segs[kSegments];
  __shared__ GranScale scales[kScales][kGrans];
  __shared__ uint32_t turns[kScales][kGrans];   // fp16 factors of a granule's keys (low half) and values: 1 or -1
  __shared__ long long scan_sm[kTcThreads / 32];
  __shared__ struct {
    Rows s;
    int b;
    long long u;
  } start_sm;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, last_sm;

  uint8_t* const qtile = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const k16 = qtile + kTiles * L::kQBytes;   // [2]
  uint8_t* const v16 = k16 + 2 * L::kBlk16;           // [2]
  uint8_t* const ring = v16 + 2 * L::kBlk16;          // [kSlots] 8-bit blocks

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) mbar_init(&slot_full[i], 1), mbar_init(&slot_empty[i], kConvWarps);
#pragma unroll
    for (int i = 0; i < kScales; ++i) mbar_init(&sc_full[i], 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], kConvWarps), mbar_init(&v_full[i], kConvWarps);
      mbar_init(&k_empty[i], 1), mbar_init(&v_empty[i], 1);
      mbar_init(&q_full[i], 4), mbar_init(&s_full[i], 1), mbar_init(&p_ready[i], 4), mbar_init(&pv_done[i], 1);
    }
#pragma unroll
    for (int i = 0; i < kSegments; ++i) mbar_init(&seg_full[i], 1), mbar_init(&seg_empty[i], kConvWarps + 1 + kSoftWarps);
    mbar_init(&join_bar, kSoftWarps);
    mbar_init(&final_bar, 1);
    abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_desc(&p.kmap);
    tma_prefetch_desc(&p.vmap);
  }
  if (warp == kMmaWarp) tmem_alloc(&tmem_base, 512);
  tc_fence_before();
  // (kPrefixes: the launch of the sequences' own tokens starts when every CTA of this one has seen the work before it
  // complete.)
  if (kMode == kPlain) pdl_trigger();
  pdl_wait();
  if (kMode == kPrefixes) pdl_trigger();
  // CTAs that take part.
  const int room = kMode == kPrefixes ? min((int)gridDim.x, prefix_sms<kTcThreads>(p, qtile)) : (int)gridDim.x;

  // ---------------------------------------------------------------- this CTA's run of units
  const int seqs = count_of<kMode>(p), per = (seqs + kTcThreads - 1) / kTcThreads;   // sequences a thread scans
  const int s0 = min(seqs, (int)threadIdx.x * per), s1 = min(seqs, s0 + per);
  long long mine = 0;
  auto seq_units = [&](int b, Rows& s) {
    load_rows<kMode>(p, b, s);
    const int tiles = tiles_of<L>(p, s);
    if (kMode == kPrefixes) return (long long)tiles * (L::kLead + tile_span<L, kMode>(p, s, 0).units) * p.kv_heads;
    long long n = 0;
    for (int t = 0; t < tiles; ++t) n += L::kLead + tile_span<L, kMode>(p, s, t).units;
    return n * p.kv_heads;
  };
  for (int b = s0; b < s1; ++b) {
    Rows s;
    mine += seq_units(b, s);
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) scan_sm[warp] = incl;
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = 0;   // all 512 columns are this CTA's: they begin at the first
  long long before = incl - mine, U = 0;
#pragma unroll
  for (int w = 0; w < kTcThreads / 32; ++w) {
    if (w < warp) before += scan_sm[w];
    U += scan_sm[w];
  }
  const int ctas = (int)min((long long)room, U);
  const bool active = (int)blockIdx.x < ctas;
  const Runs runs(U, max(ctas, 1));
  const long long u0 = active ? runs.begin(blockIdx.x) : 0, u1 = active ? runs.begin(blockIdx.x + 1) : 0;
  if (active && u0 >= before && u0 < before + mine) {
    long long at = before;
    for (int b = s0; b < s1; ++b) {
      Rows s;
      const long long n = seq_units(b, s);
      if (u0 < at + n) {
        start_sm.s = s;
        start_sm.b = b;
        start_sm.u = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();

  // The next segment's place (of a role other than the producer), or null at the end of the run.
  uint32_t seg = 0;
  auto next_segment = [&]() -> const Segment* {
    if (!wait_all(&seg_full[seg % kSegments], (seg / kSegments) & 1u, &abort_flag, p.status)) return nullptr;
    const Segment* g = &segs[seg % kSegments];
    return g->nb > 0 ? g : nullptr;
  };
  auto end_segment = [&]() {
    arrive_warp(&seg_empty[seg % kSegments]);
    ++seg;
  };

  if (warp == kProducerWarp) {
    // ---------------------------------------------------------------- producer
    Walk<L, kMode> wk;
    wk.u = u0;
    wk.u1 = u1;
    if (active) {
      wk.s = start_sm.s;
      wk.b = start_sm.b;
      wk.tiles = tiles_of<L>(p, wk.s);
      long long head = 0;
      if (kMode == kPrefixes) head = (long long)wk.tiles * (L::kLead + tile_span<L, kMode>(p, wk.s, 0).units);
      else for (int t = 0; t < wk.tiles; ++t) head += L::kLead + tile_span<L, kMode>(p, wk.s, t).units;
      wk.h = (int)quotient(u0 - start_sm.u, head);
      wk.item_u0 = start_sm.u + wk.h * head;
      wk.tile = 0;
      wk.t = tile_span<L, kMode>(p, wk.s, 0);
      if (kMode == kPrefixes) {
        wk.tile = (int)quotient(u0 - wk.item_u0, L::kLead + wk.t.units);   // (all tiles of a group are alike)
        wk.item_u0 += (long long)wk.tile * (L::kLead + wk.t.units);
      }
    }
    uint32_t blk = 0;   // blocks of the CTA before this segment
    bool ok = true;
    uint32_t copies = 0;   // slots filled
    for (uint32_t seg = 0; ok; ++seg) {
      const bool more = wk.next(p);
      if (seg >= kSegments && !wait_all(&seg_empty[seg % kSegments], (seg / kSegments - 1) & 1u, &abort_flag, p.status)) break;
      const int nb = more ? wk.ue - wk.ub : 0;
      if (lane == 0) {
        Segment g{};
        if (more) {
          g.nb = nb;
          g.T0 = wk.t.lo + wk.ub * kBlock;
          g.row0 = wk.s.row0, g.pos0 = wk.s.len - wk.s.n, g.len = wk.s.len;
          g.h = wk.h, g.tile = wk.tile, g.rows = (int)min((long long)L::kRows, (long long)wk.s.n * p.group - (long long)wk.tile * L::kRows);
          g.whole = wk.whole();
          g.slot = wk.item_u0 <= u0 ? 0 : 1;
          g.first = runs.owner(wk.item_u0 + L::kLead);
          g.parts = runs.owner(wk.item_u0 + L::kLead + wk.t.units - 1) - g.first + 1;
          g.slot0 = wk.item_u0 <= runs.begin(g.first) ? 0 : 1;
          if (kMode == kPrefixes && wk.ub == 0) p.items[item_of(p, wk.b, wk.s.row0, L::kRows, wk.tile, wk.h)] = make_int4(g.first, g.parts, g.slot0, 0);
        }
        segs[seg % kSegments] = g;
      }
      arrive_warp(&seg_full[seg % kSegments]);
      if (!more) break;
      const int T0 = wk.t.lo + wk.ub * kBlock, T1 = min(wk.t.hi, wk.t.lo + wk.ue * kBlock);
      const int* const table = p.step.page_table + (size_t)(kMode == kPlain ? wk.b : wk.s.table) * p.step.table_width;
      constexpr int kFetch = 32 / kGrans;   // blocks
      for (int base = 0; ok && base < nb; base += kFetch) {
        // Lane: granule lane % kGrans of block base + lane / kGrans.
        const int t = T0 + base * kBlock + lane * kGranule;
        GranScale sc{0.f, 0.f, -INFINITY, -INFINITY};
        uint32_t turn = 0x3C003C00u;
        int row = 0;
        bool live = t < T1;
        if (live) {
          const int page = __ldg(table + (t >> p.page_shift));
          if (page < 0 || page >= p.pages) {
            atomicOr(p.status, W8A8_DEV_BAD_INDEX);
            live = false;
          } else {
            const size_t at = (size_t)page * p.kv_heads + wk.h;
            row = (int)(at << p.page_shift) + (t & ((1 << p.page_shift) - 1));
            const float ks = __ldg(p.ks + at), vs = __ldg(p.vs + at);
            sc.ks = fabsf(ks);
            sc.vs = fabsf(vs);
            sc.lvs = lg2(sc.vs);
            sc.bias = 0.f;
            turn = (ks < 0.f ? 0xBC00u : 0x3C00u) | ((vs < 0.f ? 0xBC00u : 0x3C00u) << 16);
          }
        }
        const uint32_t lives = __ballot_sync(0xffffffffu, live);
#pragma unroll
        for (int i = 0; i < kFetch; ++i) {
          if (base + i >= nb) break;
          const uint32_t n = blk + base + i;
          const bool own = lane / kGrans == i;
          if (own) scales[n % kScales][lane % kGrans] = sc, turns[n % kScales][lane % kGrans] = turn;
          arrive_warp(&sc_full[n % kScales]);
          const uint32_t bytes = (uint32_t)__popc((lives >> (kGrans * i)) & ((1u << kGrans) - 1u)) * kGranule * D;
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint32_t slot = (2 * n + side) % kSlots, use = (2 * n + side) / kSlots;
            if (use > 0 && !wait_all(&slot_empty[slot], (use - 1) & 1u, &abort_flag, p.status)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&slot_full[slot], bytes);
            ++copies;
            __syncwarp();
            if (own && live) {
              // (A box is 128 columns at most; those of a block's granules lie together.)
              uint8_t* const dst = ring + slot * L::kSlot + lane % kGrans * kGranule * L::kBox;
#pragma unroll
              for (int x = 0; x < L::kBoxes; ++x)
                tma_load_2d(dst + x * kBlock * L::kBox, side ? &p.vmap : &p.kmap, x * L::kBox, row, &slot_full[slot]);
            }
          }
          if (!ok) break;
        }
      }
      blk += nb;
    }
    // Every copy issued must land before the CTA may exit.
    if (lane == 0) {
      for (uint32_t s = 0; s < kSlots && s < copies; ++s) mbar_wait_drain(&slot_full[s], ((copies - 1 - s) / kSlots) & 1u, p.status);
    }
  } else if (warp >= kSoftWarps && warp < kProducerWarp) {
    // ---------------------------------------------------------------- converters
    const int cw = warp - kSoftWarps;
    uint32_t n = 0;   // block of the CTA
    bool ok = true;
    while (const Segment* g = ok ? next_segment() : nullptr) {
      const int nb = g->nb;
      end_segment();
      for (int j = 0; ok && j < nb; ++j, ++n) {
        if (!wait_all(&sc_full[n % kScales], (n / kScales) & 1u, &abort_flag, p.status)) {
          ok = false;
          break;
        }
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
          const uint32_t slot = (2 * n + side) % kSlots, use = (2 * n + side) / kSlots;
          const uint8_t* const src = ring + slot * L::kSlot;
          uint8_t* const dst = (side ? v16 : k16) + (n & 1) * L::kBlk16;
          if (!wait_all(&slot_full[slot], use & 1u, &abort_flag, p.status) ||
              (n >= 2 && !wait_all(side ? &v_empty[n & 1] : &k_empty[n & 1], ((n >> 1) - 1) & 1u, &abort_flag, p.status))) {
            ok = false;
            break;
          }
          // A warp takes its share of the tokens eight rows by four 16-byte pieces at a time, so that neither the reads
          // (swizzled by the copy) nor the writes (swizzled for the products) meet in a bank.  All reads go out first.
          constexpr int kEights = kBlock / 8 / kConvWarps, kY = D / 64;
          uint4 w[kEights][kY];
#pragma unroll
          for (int i = 0; i < kEights; ++i) {
            const int t = (kEights * cw + i) * 8 + (lane & 7);
#pragma unroll
            for (int y = 0; y < kY; ++y) {
              const int piece = (lane >> 3) + 4 * y;
              w[i][y] = D == 64 ? *reinterpret_cast<const uint4*>(src + t * 64 + ((piece ^ ((t >> 1) & 3)) << 4))
                                : *reinterpret_cast<const uint4*>(src + (piece >> 3) * kBlock * L::kBox + t * 128 + (((piece & 7) ^ (t & 7)) << 4));
            }
          }
#pragma unroll
          for (int i = 0; i < kEights; ++i) {
            const uint32_t turn = turns[n % kScales][(kEights * cw + i) >> 1];
            const uint32_t f = side ? turn >> 16 : turn & 0xFFFFu;
            const __half2 sg = __half2half2(__ushort_as_half((uint16_t)f));
            const __half2 of = __hmul2(sg, __half2half2(__ushort_as_half(0xE480)));   // -1152
            const int t = (kEights * cw + i) * 8 + (lane & 7);
#pragma unroll
            for (int y = 0; y < kY; ++y) {
              const int piece = (lane >> 3) + 4 * y;
              const uint32_t in[4] = {w[i][y].x, w[i][y].y, w[i][y].z, w[i][y].w};
              uint32_t out[8];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // fp16 0x6400 | b = 1024 + b, so (1024 + b) sg - 1152 sg = sg (b - 128), exactly.
                const uint32_t a = __byte_perm(in[k], 0x64646464u, 0x4140), c = __byte_perm(in[k], 0x64646464u, 0x4342);
                const __half2 ha = __hfma2(*reinterpret_cast<const __half2*>(&a), sg, of);
                const __half2 hc = __hfma2(*reinterpret_cast<const __half2*>(&c), sg, of);
                out[2 * k] = *reinterpret_cast<const uint32_t*>(&ha);
                out[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&hc);
              }
              uint8_t* const row = dst + (piece >> 2) * L::kHalf + t * 128;
              const int ch = 2 * (piece & 3);
              *reinterpret_cast<uint4*>(row + ((ch ^ (t & 7)) << 4)) = make_uint4(out[0], out[1], out[2], out[3]);
              *reinterpret_cast<uint4*>(row + (((ch + 1) ^ (t & 7)) << 4)) = make_uint4(out[4], out[5], out[6], out[7]);
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&slot_empty[slot]);
            mbar_arrive(side ? &v_full[n & 1] : &k_full[n & 1]);
          }
        }
      }
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- issuer
    // The whole warp walks the blocks and one elected lane issues.  A descriptor's low word is its start
    // address in 16 bytes and moves by constants.  (One warp for both streams: with one each, the products of
    // two accumulators mix in the pipe and each takes longer; prompt chunk 441 -> 521 us.)
    constexpr uint32_t idesc_s = idesc_f16_f32(kTileRows, kBlock);
    constexpr uint32_t idesc_o = idesc_f16_f32(kTileRows, D) | (1u << 16);   // B is MN-major
    const uint64_t dq = desc_kmajor(smem_addr(qtile)), dk = desc_kmajor(smem_addr(k16)), dv = desc_mnmajor(smem_addr(v16), L::kHalf);
    const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, k_hi = (uint32_t)(dk >> 32), v_lo = (uint32_t)dv, v_hi = (uint32_t)(dv >> 32);
    auto desc = [](uint32_t lo, uint32_t hi) { return (uint64_t)lo | ((uint64_t)hi << 32); };
    uint32_t blk = 0, cnt = 0;   // blocks of the CTA before this segment; steps of the first stream
    uint32_t cnt1 = 0;           // of the second
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_all(bar, parity, &abort_flag, p.status); };
    while (const Segment* g = ok ? next_segment() : nullptr) {
      const int nb = g->nb;
      const uint32_t q_use = seg & 1u;
      end_segment();
      if constexpr (kWide) {
        // Scores of a block go out before the products of the weights of the one before it, into the place of the
        // weights before those.
        ok = wait(&q_full[0], q_use);
#pragma unroll 1
        for (int i = -1; ok && i < nb; ++i) {
          const uint32_t n = blk + (uint32_t)i, nn = n + 1, u = n & 1u, uu = nn & 1u;
          if (i + 1 < nb) {
            ok = wait(&k_full[uu], (nn >> 1) & 1u) && (i < 1 || wait(&pv_done[uu], ((n - 1) >> 1) & 1u));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t kl = k_lo + uu * (uint32_t)(L::kBlk16 >> 4);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t qo = (uint32_t)(((k >> 2) * kTileRows * 128 + (k & 3) * 32) >> 4), ko = (uint32_t)(((k >> 2) * L::kHalf + (k & 3) * 32) >> 4);
                umma_f16_ss(uu * kBlock, desc(q_lo + qo, k_hi), desc(kl + ko, k_hi), idesc_s, k > 0);
              }
              umma_commit(&s_full[uu]);
              umma_commit(&k_empty[uu]);
            }
            __syncwarp();
          }
          if (i < 0) continue;
          ok = wait(&v_full[u], (n >> 1) & 1u) && wait(&p_ready[u], (n >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t lo = v_lo + u * (uint32_t)(L::kBlk16 >> 4);
#pragma unroll
            for (int k = 0; k < kBlock / 16; ++k)
              umma_f16_tmem_a(L::kOCol, u * kBlock + 8 * k, desc(lo + (uint32_t)(k * 16 * 128 >> 4), v_hi), idesc_o, i > 0 || k > 0);
            umma_commit(&pv_done[u]);
            umma_commit(&v_empty[u]);
          }
          __syncwarp();
        }
        blk += nb;
        continue;
      }
      const int n0 = kTiles == 2 ? nb : (nb + 1) / 2, n1 = kTiles == 2 ? nb : nb / 2;
      // Steps in order: (stream, turn) = (0, -1), (1, -1), (0, 0), (1, 0), ...: the products of a turn's weights
      // with its values, then, where there is one, the next turn's scores.
      ok = wait(&q_full[0], q_use) && (kTiles == 1 || wait(&q_full[1], q_use));
#pragma unroll 1
      for (int x = -2; ok && x < 2 * n0; ++x) {
        const int s = x & 1, i = (x + 2) / 2 - 1;
        if (i >= (s ? n1 : n0)) continue;
        const uint32_t t = (uint32_t)(s * L::kStreamCols);
        const bool more = i + 1 < (s ? n1 : n0);
        const uint32_t nn = blk + (uint32_t)(kTiles == 2 ? i + 1 : 2 * (i + 1) + s), ub = nn & 1u;   // the next turn's block
        if (i >= 0) {
          const uint32_t n = nn - (kTiles == 2 ? 1u : 2u), u = n & 1u, c = s ? cnt1 : cnt;
          ok = wait(&v_full[u], (n >> 1) & 1u) && wait(&p_ready[s], c & 1u);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t lo = v_lo + u * (uint32_t)(L::kBlk16 >> 4);
#pragma unroll
            for (int k = 0; k < kBlock / 16; ++k)
              umma_f16_tmem_a(t + L::kOCol, t + (uint32_t)(L::kSCol + 8 * k), desc(lo + (uint32_t)(k * 16 * 128 >> 4), v_hi), idesc_o, i > 0 || k > 0);
            umma_commit(&pv_done[s]);
            if (kTiles == 1 || s == 1) umma_commit(&v_empty[u]);
          }
          __syncwarp();
          if (s) ++cnt1;
          else ++cnt;
          // The next scores take the tensor memory of the weights that these products read.
          if (more) ok = wait(&k_full[ub], (nn >> 1) & 1u) && wait(&pv_done[s], c & 1u);
        } else if (more) {
          ok = wait(&k_full[ub], (nn >> 1) & 1u);
        }
        if (!ok || !more) continue;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t ql = q_lo + (kTiles == 2 ? s : 0) * (uint32_t)(L::kQBytes >> 4), kl = k_lo + ub * (uint32_t)(L::kBlk16 >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t qo = (uint32_t)(((k >> 2) * kTileRows * 128 + (k & 3) * 32) >> 4), ko = (uint32_t)(((k >> 2) * L::kHalf + (k & 3) * 32) >> 4);
            umma_f16_ss(t + L::kSCol, desc(ql + qo, k_hi), desc(kl + ko, k_hi), idesc_s, k > 0);
          }
          umma_commit(&s_full[s]);
          if (kTiles == 1 || s == 1) umma_commit(&k_empty[ub]);
        }
        __syncwarp();
      }
      blk += nb;
    }
    // Every product issued completes before tensor memory is freed.
    if (elect_one()) {
      umma_commit(&final_bar);
      mbar_wait_drain(&final_bar, 0, p.status);
    }
    __syncwarp();
  } else if (warp < kSoftWarps) {
    // ---------------------------------------------------------------- softmax warps
    const int st = warp >> 2, quad = warp & 3;
    const int row = 32 * quad + lane;                              // of the tile
    const int irow = kTiles == 2 ? st * kTileRows + row : row;     // of the item
    const uint32_t t_lane = tmem + ((uint32_t)(32 * quad) << 16) + (uint32_t)(st * L::kStreamCols);
    const uint32_t t_o = t_lane + L::kOCol;
    uint32_t blk = 0, cnt = 0, join_phase = 0;
    auto meet = [&]() {   // bounded meeting of the softmax warps
      arrive_warp(&join_bar);
      const bool ok = wait_all(&join_bar, join_phase, &abort_flag, p.status);
      join_phase ^= 1u;
      return ok;
    };
    // The products of a stream's block c with its values are done.  (A wide head's scores run a block ahead of them: one
    // barrier could be two phases behind, which its parity does not tell from done.)
    auto wait_sums = [&](uint32_t c) {
      return wait_all(&pv_done[kWide ? c & 1u : (uint32_t)st], (kWide ? c >> 1 : c) & 1u, &abort_flag, p.status);
    };
    bool ok = true;
    while (const Segment* g = ok ? next_segment() : nullptr) {
      const int nb = g->nb;
      const int ns = !kAlternate ? nb : st == 0 ? (nb + 1) / 2 : nb / 2;
      const int T0 = g->T0;
      const bool live = irow < g->rows;
      const int ri = g->tile * L::kRows + (live ? irow : 0);
      const int tok = ri / p.group, head = g->h * p.group + ri % p.group;
      const bool warp_live = (kTiles == 2 ? st * kTileRows : 0) + 32 * quad < g->rows;

      // ------------------------------------------------ queries: fp16, scaled by a power of two
      float rowmul;
      {
        const uint4* const src = reinterpret_cast<const uint4*>(p.q + (g->row0 + tok) * p.q_stride + head * D);
        float amax = 0.f;
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          float f[8];
          unpack8<kF16>(live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
          for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(f[k]));
        }
        const int ex = max((int)(__float_as_uint(amax) >> 23) - 127 - 13, -100);
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        rowmul = p.scale_log2 * __uint_as_float((uint32_t)(127 + ex) << 23);
        if (kTiles == 2 || st == 0) {
          uint8_t* const dst = qtile + (kTiles == 2 ? st : 0) * L::kQBytes + row * 128;
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {   // (out of the L1 cache now)
            float f[8];
            unpack8<kF16>(live ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] *= down;
            *reinterpret_cast<uint4*>(dst + (i >> 3) * kTileRows * 128 + (((i & 7) ^ (row & 7)) << 4)) = pack8<true>(f);
          }
          fence_async_shared();
          arrive_warp(&q_full[kTiles == 2 ? st : 0]);
        }
      }
      const int pos = g->pos0 + tok;
      const int end = !live ? 0x7fffffff : kMode == kPlain && p.causal ? min(pos + 1, g->len) : g->len;
      const int beg = kMode == kPlain && live && p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const int full_hi = __reduce_min_sync(0xffffffffu, end), full_lo = __reduce_max_sync(0xffffffffu, beg);

      // ------------------------------------------------ blocks
      float m = kFloor, r = kFloor, hs = 0.f, l = 0.f;
      for (int i = 0; ok && i < ns; ++i, ++cnt) {
        const int j = kAlternate ? 2 * i + st : i;
        const uint32_t n = blk + (uint32_t)j;
        // The place of the scores: a stream's own; the block's of a wide head.
        const uint32_t at = kWide ? n & 1u : (uint32_t)st, t_s = t_lane + L::kSCol + (kWide ? at * kBlock : 0u);
        const int T = T0 + j * kBlock;
        if (!wait_all(&sc_full[n % kScales], (n / kScales) & 1u, &abort_flag, p.status) ||
            !wait_all(&s_full[at], (kWide ? n >> 1 : cnt) & 1u, &abort_flag, p.status)) {
          ok = false;
          break;
        }
        if (warp_live) {
          tc_fence_after();
          const bool edge = T < full_lo || T + kBlock > full_hi;
          const GranScale* const sc = scales[n % kScales];
          // 32 tokens a turn.  (Not unrolled, and no load ahead: the warps of all roles together have to
          // stay inside the instruction cache, and a spilled register's home is far behind a shared memory
          // that leaves the L1 cache next to nothing.)  The weights are worked out beside the maxima, as if
          // no reference moved, and once more where one does.
#pragma unroll 1
          for (int ch = 0; ch < kBlock / 32; ++ch) {
            {
              uint32_t a[32];
              tmem_ld32(t_s + 32 * ch, a);
              const float4 g0 = *reinterpret_cast<const float4*>(&sc[2 * ch]), g1 = *reinterpret_cast<const float4*>(&sc[2 * ch + 1]);
              tmem_wait_ld32(a);
              if (edge) {
                // Scores that the row does not see.
                const int t0 = T + 32 * ch;
#pragma unroll
                for (int k = 0; k < 32; ++k)
                  if (t0 + k < beg || t0 + k >= end) a[k] = 0xFF800000u;
              }
              // Score a of a granule in powers of two: a * c1 + bias.  (A factor of zero would make a
              // hidden score's -inf a NaN.)
              const float c1[2] = {fmaxf(g0.x * rowmul, 1e-37f), fmaxf(g1.x * rowmul, 1e-37f)};
              const float vs[2] = {g0.y, g1.y}, lvs[2] = {g0.z, g1.z}, bias[2] = {g0.w, g1.w};
              float mx, mw;
              {
                float t[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t* const v = a + 16 * y;
                  float q[4];
#pragma unroll
                  for (int k = 0; k < 4; ++k) q[k] = max3(__uint_as_float(v[k]), __uint_as_float(v[4 + k]), __uint_as_float(v[8 + k]));
                  const float e = max3(__uint_as_float(v[12]), __uint_as_float(v[13]), __uint_as_float(v[14]));
                  t[y] = fmaf(max3(max3(q[0], q[1], q[2]), max3(q[3], e, __uint_as_float(v[15])), -INFINITY), c1[y], bias[y]);
                }
                mx = fmaxf(t[0], t[1]);
                mw = fmaxf(t[0] + lvs[0], t[1] + lvs[1]);
              }
              uint32_t w16[16];
              uint64_t sum;
              bool far = false, moved;
#pragma unroll 1
              do {
                sum = 0;   // (0, 0)
                const float f[2] = {hs * vs[0], hs * vs[1]};
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const float c0 = bias[y] - m;
                  const uint64_t c1p = pair(c1[y], c1[y]), c0p = pair(c0, c0), fp = pair(f[y], f[y]);
#pragma unroll
                  for (int k = 0; k < 16; k += 2) {
                    float e0, e1;
                    unpair(fma2(pair(__uint_as_float(a[16 * y + k]), __uint_as_float(a[16 * y + k + 1])), c1p, c0p), e0, e1);
                    const uint64_t pr = pair(ex2(e0), ex2(e1));
                    sum = add2(sum, pr);
                    float w0, w1;
                    unpair(mul2(pr, fp), w0, w1);
                    w16[8 * y + k / 2] = pack2<true>(w0, w1);
                  }
                }
                if (far) {
#pragma unroll
                  for (int y = 0; y < 2; ++y) {
                    if (f[y] > kFar) {
                      const float d0 = bias[y] + lvs[y] - r;
#pragma unroll
                      for (int k = 0; k < 16; k += 2)
                        w16[8 * y + k / 2] = pack2<true>(ex2(fmaf(__uint_as_float(a[16 * y + k]), c1[y], d0)),
                                                         ex2(fmaf(__uint_as_float(a[16 * y + k + 1]), c1[y], d0)));
                    }
                  }
                  break;
                }
                moved = __any_sync(0xffffffffu, mx > m + kSlack || mw > r + kRoom || fmaxf(f[0], f[1]) > kFar);
                if (moved) {
                  // Some row's reference moves: its sums so far are rescaled, and with them the weights of
                  // this block that are already written.
                  if (mx > m + kSlack) {
                    l *= ex2(m - mx);
                    m = mx;
                  }
                  float rn = mw > r + kRoom ? mw - kHead : r;
                  rn = fminf(fmaxf(rn, m - kBelow), m + kAbove);
                  const float down = ex2(r - rn);
                  r = rn;
                  hs = ex2(m - rn);
                  // What is worked out with the moved references stands, whether or not a limit keeps r below the
                  // largest weight: with no maxima left to compare, and `far` the third condition itself, the second
                  // turn is the last.
                  far = __any_sync(0xffffffffu, fmaxf(hs * vs[0], hs * vs[1]) > kFar);
                  mx = mw = -INFINITY;
                  if (i > 0 && !wait_sums(cnt - 1)) ok = false;
                  if (__any_sync(0xffffffffu, down != 1.f) && (i > 0 || ch > 0)) rescale(t_o, i > 0 ? D : 0, t_s, ch, down);
                }
              } while (moved);
              float l0, l1;
              unpair(sum, l0, l1);
              l += l0 + l1;
              tmem_st16(t_s + 16 * ch, w16);
            }
          }
          tmem_wait_st();
          tc_fence_before();
        }
        arrive_warp(&p_ready[at]);
      }
      blk += nb;
      if (!ok) break;

      // ------------------------------------------------ the segment's end
      if (ns > 0 && !wait_sums(cnt - 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float scale_own = 1.f, scale_other = 0.f;   // of the two streams' sums (one tile: they join here)
      // The second stream's (m, l, r), then kX columns of its sums at a time ([kX][128]), go over through the
      // queries' shared memory (every score has been computed).
      constexpr int kX = L::kQBytes / (kTileRows * 4);
      float* const xch = reinterpret_cast<float*>(qtile);
      if (kAlternate) {
        bool met = meet();   // the other stream's scores too
        if (st == 1) xch[row] = m, xch[kTileRows + row] = l, xch[2 * kTileRows + row] = r;
        met = met && meet();
        if (st == 0) {
          const float om = xch[row], ol = xch[kTileRows + row], orr = xch[2 * kTileRows + row];
          const float mn = fmaxf(m, om), rn = fmaxf(r, orr);
          l = l * ex2(m - mn) + ol * ex2(om - mn);
          scale_own = ex2(r - rn);
          scale_other = ex2(orr - rn);
          m = mn;
          r = rn;
        }
        if (!met) {
          ok = false;
          break;
        }
      }
      const bool whole = g->whole;
      float* const part = p.parts + ((size_t)blockIdx.x * 2 + g->slot) * L::kPart;
      float* const row32 = p.rows32 + ((size_t)(g->row0 + tok) * p.q_heads + head) * (D + 4);   // (rows32 given)
      const float z = l == 0.f ? 0.f : __fdividef(1.f, l) * ex2(r - m);
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        if (kAlternate && c0 % kX == 0) {
          if (!meet()) ok = false;
          if (st == 1) {
#pragma unroll 1
            for (int c = 0; c < kX; c += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + c0 + c, o);
              tmem_wait_ld32(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) xch[(c + k) * kTileRows + row] = ns > 0 ? __uint_as_float(o[k]) : 0.f;
            }
          }
          if (!meet()) ok = false;
          if (!ok) break;
        }
        if (kAlternate && st == 1) continue;
        uint32_t o[32];
        tmem_ld32(t_o + c0, o);
        tmem_wait_ld32(o);
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          v[k] = __uint_as_float(o[k]);
          if (kAlternate) v[k] = fmaf(v[k], scale_own, scale_other == 0.f ? 0.f : xch[(c0 % kX + k) * kTileRows + row] * scale_other);
        }
        if (live && (!whole || kMode != kPlain)) {
          // (A prefix's part: four columns of a row beside those of the next, as neighbouring threads store them.)
          constexpr int kStep = kMode == kPrefixes ? L::kRows : 1;
          float4* const dst = whole ? reinterpret_cast<float4*>(row32 + c0)
                                    : reinterpret_cast<float4*>(part) + (kMode == kPrefixes ? c0 / 4 * L::kRows + irow : (irow * D + c0) / 4);
#pragma unroll
          for (int k = 0; k < 32; k += 4) dst[k / 4 * (whole ? 1 : kStep)] = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        } else if (live) {
          uint4* const dst = reinterpret_cast<uint4*>(p.out + (g->row0 + tok) * p.out_stride + head * D + c0);
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = v[k + e] * z;
            if (l == 0.f) {
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] = 0.f;
            }
            dst[k / 8] = pack8<kF16>(y);
          }
        }
      }
      if (!ok) break;
      if (live && (kTiles == 2 || st == 0)) {
        if (!whole || kMode != kPlain) *reinterpret_cast<float4*>(whole ? row32 + D : part + L::kRows * D + irow * 4) = make_float4(m, l, r, 0.f);
        else if (p.lse) p.lse[(size_t)(g->row0 + tok) * p.q_heads + head] = l == 0.f ? -INFINITY : (m + lg2(l)) * 0.69314718056f;
      }
      tc_fence_before();
      if (!whole && kMode != kPrefixes) {   // (the parts of shared prefixes are joined by another kernel)
        // The part is written; the last CTA to arrive joins all of the item's, in the CTAs' order.  (The
        // meeting orders the warps' stores before thread 0's release, and its acquire before their reads.)
        // Many parts join first in groups of about sqrt(n), each by the last of its CTAs, so that no CTA reads more than
        // a few: one SM reads some 50 KB/us (256 rows on 16000 tokens, 4 kv heads,
        // 38 parts: 131 us without groups, 71 with them).
        constexpr int kGroup = 8;
        const int first = g->first, slot0 = g->slot0, np = g->parts, rows = g->rows;
        const float* const part0 = p.parts + ((size_t)first * 2 + slot0) * L::kPart;
        const float* const part1 = p.parts + (size_t)first * 2 * L::kPart;   // part i > 0: 2 i places on
        auto part_of = [&](int i) { return i == 0 ? part0 : part1 + (size_t)i * 2 * L::kPart; };
        int group = np;
        if (np > kGroup) {
          group = 3;
          while (group * group < np) ++group;
        }
        const int groups = (np + group - 1) / group, lead = ((int)blockIdx.x - first) / group * group;
        int base = lead, step = 1, count = min(group, np - lead);
        uint32_t* counter = groups > 1 ? p.group_counters + 2 * (first + lead) + (lead == 0 ? slot0 : 0) : p.counters + first;
        for (bool top = groups == 1;; top = true) {
          if (!meet()) {
            ok = false;
            break;
          }
          if (threadIdx.x == 0) {
            const uint32_t old = atom_add_acq_rel_u32(counter, 1u);
            if (old >= (uint32_t)count) atomicOr(p.status, W8A8_DEV_COUNTER_CORRUPT);
            if (old == (uint32_t)count - 1) *counter = 0u;   // ready for the next call
            last_sm = old == (uint32_t)count - 1;
          }
          if (!meet()) {
            ok = false;
            break;
          }
          if (!last_sm) break;
          // A thread for each row's statistics, then a warp for a row's sums, kAt rows at a time.
          float4* const row_sm = reinterpret_cast<float4*>(qtile);   // (m, l, r, -)
          if (irow < rows && (kTiles == 2 || st == 0)) {
            float mm = kFloor, rm = kFloor, lt = 0.f;
#pragma unroll 4
            for (int i = 0; i < count; ++i) {
              const float4 t = __ldcg(reinterpret_cast<const float4*>(part_of(base + step * i) + L::kRows * D) + irow);
              const float mn = fmaxf(mm, t.x);
              lt = lt * ex2(mm - mn) + t.y * ex2(t.x - mn);
              mm = mn;
              rm = fmaxf(rm, t.z);
            }
            row_sm[irow] = make_float4(mm, lt, rm, 0.f);
          }
          if (!meet()) ok = false;
          constexpr int kVec = D / 4, kAt = 4, kSoftThreads = 32 * kSoftWarps;   // kVec: threads of a row, four values each
          for (int at0 = threadIdx.x; at0 < rows * kVec; at0 += kAt * kSoftThreads) {
            float4 acc[kAt];
#pragma unroll
            for (int y = 0; y < kAt; ++y) acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int i = 0; i < count; ++i) {
              const float* const src = part_of(base + step * i);
              float4 v[kAt];
              float rr[kAt];
#pragma unroll
              for (int y = 0; y < kAt; ++y) {
                const int at = at0 + y * kSoftThreads;
                v[y] = make_float4(0.f, 0.f, 0.f, 0.f);
                rr[y] = 0.f;
                if (at < rows * kVec) {
                  v[y] = __ldcg(reinterpret_cast<const float4*>(src) + at);
                  rr[y] = __ldcg(src + L::kRows * D + (at / kVec) * 4 + 2);
                }
              }
#pragma unroll
              for (int y = 0; y < kAt; ++y) {
                const int at = at0 + y * kSoftThreads;
                if (at < rows * kVec) {
                  const float f = ex2(rr[y] - row_sm[at / kVec].z);
                  acc[y].x = fmaf(v[y].x, f, acc[y].x), acc[y].y = fmaf(v[y].y, f, acc[y].y);
                  acc[y].z = fmaf(v[y].z, f, acc[y].z), acc[y].w = fmaf(v[y].w, f, acc[y].w);
                }
              }
            }
#pragma unroll
            for (int y = 0; y < kAt; ++y) {
              const int at = at0 + y * kSoftThreads;
              if (at >= rows * kVec) continue;
              if (!top) {
                // The group's sums take the place of its first part's; its statistics once every thread has read them.
                *(reinterpret_cast<float4*>(const_cast<float*>(part_of(base))) + at) = acc[y];
                continue;
              }
              const int rw = at / kVec, d = 4 * (at % kVec);
              const float4 t = row_sm[rw];
              const int oi = g->tile * L::kRows + rw;
              const int orow = g->row0 + oi / p.group, oh = g->h * p.group + oi % p.group;
              const float zz = t.y == 0.f ? 0.f : __fdividef(1.f, t.y) * ex2(t.z - t.x);
              *reinterpret_cast<uint2*>(p.out + orow * p.out_stride + oh * D + d) =
                  make_uint2(pack2<kF16>(acc[y].x * zz, acc[y].y * zz), pack2<kF16>(acc[y].z * zz, acc[y].w * zz));
              if (p.lse && d == 0)
                p.lse[(size_t)orow * p.q_heads + oh] = t.y == 0.f ? -INFINITY : (t.x + lg2(t.y)) * 0.69314718056f;
            }
          }
          if (!meet()) ok = false;   // the statistics' place is the next queries', or the next join's
          if (top || !ok) break;
          if (irow < rows && (kTiles == 2 || st == 0))
            *(reinterpret_cast<float4*>(const_cast<float*>(part_of(base)) + L::kRows * D) + irow) = row_sm[irow];
          base = 0, step = group, count = groups;
          counter = p.counters + first;
        }
        if (!ok) break;
      }
      if (kAlternate && !meet()) ok = false;   // the exchange is over: the next queries may take its place
      end_segment();
    }
  }

  // Every role ends here; then the allocating warp returns the tensor memory.
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem_base, 512);
}

template <bool kF16, int D, int kTiles, Mode kMode>
static cudaError_t launch_tc(const Params& p, int sms, cudaStream_t stream) {
  using L = TcLayout<D, kTiles>;
  auto kern = kv8_attention_tc_kernel<kF16, D, kTiles, kMode>;
  cudaError_t e = ensure_smem_attribute((const void*)kern, L::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = (size_t)L::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

inline int tile_rows_of(int head_dim, long long rows) { return head_dim == 256 || rows <= kTileRows ? kTileRows : 2 * kTileRows; }

// `rows`: of a sequence (or group) and kv head, at most.
template <Mode kMode>
static cudaError_t launch_many_of(const Params& p, long long rows, int head_dim, bool f16, int sms, cudaStream_t s) {
  const bool one = tile_rows_of(head_dim, rows) == kTileRows;
  if (head_dim == 256) return f16 ? launch_tc<true, 256, 1, kMode>(p, sms, s) : launch_tc<false, 256, 1, kMode>(p, sms, s);
  if (head_dim == 64)
    return f16 ? (one ? launch_tc<true, 64, 1, kMode>(p, sms, s) : launch_tc<true, 64, 2, kMode>(p, sms, s))
               : (one ? launch_tc<false, 64, 1, kMode>(p, sms, s) : launch_tc<false, 64, 2, kMode>(p, sms, s));
  return f16 ? (one ? launch_tc<true, 128, 1, kMode>(p, sms, s) : launch_tc<true, 128, 2, kMode>(p, sms, s))
             : (one ? launch_tc<false, 128, 1, kMode>(p, sms, s) : launch_tc<false, 128, 2, kMode>(p, sms, s));
}

}  // namespace attn
}  // namespace w8a8
