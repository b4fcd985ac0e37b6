// Attention over the 8-bit paged key-value cache: few query rows (single tokens, verify windows).
//
// Row i of sequence b stands at position p = kv_len - n + i and sees the cached tokens
// j in [max(0, p - window + 1), p] (causal) or [0, kv_len):
//   o = sum_j softmax_j(scale q . k_j) v_j,   k_j = (byte - 128) * k_scale[page], v_j alike.
//
// What bounds it: every cached byte feeds 2 (rows / kv heads) multiply-adds, a handful for single
// tokens, so the cache has to stream at HBM speed and everything else has to hide behind it.
//
// Mathematics.  The n * G rows that share a kv head (n tokens, G query heads) are the rows of 16-row
// tiles; 16 cached tokens are a granule.
//  * Scores on mma.sync m16n8k16, fp16 x fp16 -> fp32.  A cached byte b is used as the fp16 subnormal
//    b * 2^-24 (one byte permute makes two of them, nothing is subtracted); 128 * sum_d q comes off
//    each score once.  A query row is scaled by a power of two (exact) that takes its largest value to
//    [2^13, 2^14), so bf16 queries lose nothing in fp16 down to 2^-27 of the row's largest.  The order
//    of d inside the matrix product is free, and is chosen so that a lane's bytes are 16 contiguous ones.
//  * One pass with running references.  p = 2^(s - m) sums to l in fp32.  The values' scale belongs to
//    the weights: w = 2^(s - m) * (v_scale * 2^(m - r)), rounded to fp16 (11 bits, against 8 for bf16:
//    with bf16 weights the error of a sum of independent values equals the output's own rounding), and
//    o = sum w (b - 128), the bytes converted exactly.  r follows the largest w as m follows the largest
//    s, so neither a page of tiny values under the largest score nor the reverse loses bits.  Both
//    references move only when a row's largest score or weight passes them by 2^8: w stays inside
//    fp16's range, and the sums are rescaled a few times per pass instead of at every granule.
//  * Parts (warps of a CTA, CTAs of a split sequence) join as o 2^(r_i - r), l 2^(m_i - m), in a fixed
//    order whatever the order of arrival, so replays give the same bits.
//
// Layout and split.  A granule of one head is 16 rows of the cache: a 2-D tensor-map box per 128 bytes
// of head, whose hardware swizzle makes both operands' shared-memory reads conflict-free.  Every warp
// is its own pipeline (its ring of granules, its mbarriers, its running sums), so nothing in the loop
// waits for another warp; the page number and scales of its next 32 granules are one load a lane.
// The work is cut over all (sequence, row tile, kv head) items laid end to end, in units of 64 tokens,
// into equal runs, one for each CTA: lengths live on the device, so each CTA finds its run from a scan
// of kv_len.  An item cut across CTAs is finished by the last of them to arrive.  Three CTAs of four
// warps share an SM (two where the accumulators are larger), so that one CTA's start, join and drain
// hide behind the others' streams.
#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "kv8.cuh"
#include "kv8.h"

namespace w8a8 {
namespace attn {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kGranule = 16;         // tokens of a warp's step
constexpr int kUnit = 64;            // tokens of the split's unit: a granule for each warp
constexpr float kFloor = -3.0e38f;   // reference of a row that has seen nothing
constexpr float kSlack = 8.f;        // a reference moves when it is passed by this much (powers of two)
constexpr float kSpan = 120.f;       // largest distance of the two references

// R: 16-row tiles a warp holds.
template <int D, int R>
struct Layout {
  static constexpr int kBoxes = D > 128 ? D / 128 : 1;
  static constexpr int kBoxBytes = kGranule * (D > 128 ? 128 : D);
  static constexpr int kSide = kBoxes * kBoxBytes;      // keys (or values) of a granule
  static constexpr int kStage = 2 * kSide;
  static constexpr int kCtas = D * R > 128 ? 2 : 3;      // CTAs on an SM
  static constexpr int kStages = (kCtas == 3 ? 16384 : 24576) / kStage;   // a warp's ring
  static constexpr int kRow = D + 4;                    // floats of a row in the join buffer
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSmem = 1024 + kRing;
  static constexpr int kRows = 16 * R;
  // A part of a split item in the workspace: kRows x D sums, then m, l, r of each row.
  static constexpr int kPart = kRows * (D + 4);
  static_assert(kWarps * 16 * kRow * 4 <= kRing, "the join buffer lies over the rings");
  static_assert(kStages >= 2 && kStages <= 16, "ring depth");
};

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

// What the rows of a sequence cover: items of `tiles` row tiles and kv heads, each of `units` units
// from token `lo` (a granule's start) to `hi`.
struct Span {
  Seq s;
  int tiles, units, lo, hi;
};

template <int kRows>
__device__ __forceinline__ Span load_span(const Params& p, int b) {
  Span x;
  load_seq(p.step, b, 1 << p.page_shift, false, p.status, x.s);
  x.tiles = (int)(((long long)x.s.n * p.group + kRows - 1) / kRows);
  x.hi = x.s.len;
  x.lo = p.window > 0 ? max(0, x.s.len - x.s.n - p.window + 1) & ~(kGranule - 1) : 0;
  x.units = max(1, (x.hi - x.lo + kUnit - 1) / kUnit);   // one that sees nothing still writes its rows
  return x;
}

// The equal runs: U units over `ctas`, the first U % ctas one longer.
struct Runs {
  long long a, r;
  __device__ Runs(long long U, int ctas) : a(U / ctas), r(U % ctas) {}
  __device__ long long begin(int i) const { return i * a + (i < r ? i : r); }
  __device__ int owner(long long u) const {
    const long long head = r * (a + 1);
    return (int)(u < head ? u / (a + 1) : r + (u - head) / a);
  }
};

template <bool kF16, int D, int R>
__global__ void __launch_bounds__(kThreads, Layout<D, R>::kCtas) kv8_attention_kernel(const __grid_constant__ Params p) {
  using L = Layout<D, R>;
  constexpr int NS = L::kStages;
  constexpr int kSteps = D / 16;    // k16 steps of a score
  constexpr int kCols = D / 8;      // n8 tiles of the output
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[kWarps][NS];
  __shared__ long long scan_sm[kWarps + 3];
  __shared__ float mlr_sm[kWarps][16][3];
  __shared__ int last_sm, abort_flag;
  uint8_t* const ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));

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
  pdl_wait();

  // ---------------------------------------------------------------- this CTA's run of units
  const int per = (p.step.seqs + kThreads - 1) / kThreads;   // sequences a thread scans
  const int s0 = min(p.step.seqs, (int)threadIdx.x * per), s1 = min(p.step.seqs, s0 + per);
  long long mine = 0;
  for (int b = s0; b < s1; ++b) {
    const Span x = load_span<L::kRows>(p, b);
    mine += (long long)x.tiles * x.units;
  }
  mine *= p.kv_heads;
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 31) scan_sm[warp] = incl;
  __syncthreads();
  long long before = incl - mine, U = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += scan_sm[w];
    U += scan_sm[w];
  }
  const int ctas = (int)min((long long)gridDim.x, U);
  if ((int)blockIdx.x >= ctas) return;
  const Runs runs(U, ctas);
  const long long u0 = runs.begin(blockIdx.x), u1 = runs.begin(blockIdx.x + 1);
  if (u0 >= before && u0 < before + mine) {
    // The sequence of this thread's that holds u0.
    long long at = before;
    for (int b = s0; b < s1; ++b) {
      const Span x = load_span<L::kRows>(p, b);
      const long long n = (long long)x.tiles * x.units * p.kv_heads;
      if (u0 < at + n) {
        scan_sm[kWarps] = b;
        scan_sm[kWarps + 1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int b = (int)scan_sm[kWarps];
  long long seq_u0 = scan_sm[kWarps + 1];   // first unit of sequence b
  Span x = load_span<L::kRows>(p, b);
  uint32_t count = 0;                       // granules this warp has taken (ring position and phase)
  bool dead = false;                        // a wait ran out: only the bookkeeping goes on

  for (long long u = u0; u < u1;) {
    // ---------------------------------------------------------------- the next segment: one item's part of the run
    while (u >= seq_u0 + (long long)x.tiles * x.units * p.kv_heads) {
      seq_u0 += (long long)x.tiles * x.units * p.kv_heads;
      x = load_span<L::kRows>(p, ++b);
    }
    const int item = (int)((u - seq_u0) / x.units);
    const long long item_u0 = seq_u0 + (long long)item * x.units;
    const int ub = (int)(u - item_u0), ue = (int)min((long long)x.units, u1 - item_u0);
    const int h = item % p.kv_heads, tile = item / p.kv_heads;
    const int T0 = x.lo + ub * kUnit, T1 = min(x.hi, x.lo + ue * kUnit);
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
        const int page = __ldg(table + (t >> p.page_shift));
        bad = page < 0 || page >= p.pages;
        if (!bad) {
          const size_t at = (size_t)page * p.kv_heads + h;
          row_r = (int)(at << p.page_shift) + (t & ((1 << p.page_shift) - 1));
          a = __ldg(p.ks + at);
          v = __ldg(p.vs + at);
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
    if (!dead && mine_n > 0) {
      fetch(0);
#pragma unroll
      for (int j = 0; j < NS; ++j)
        if (j < mine_n) issue(j);
    }

    // ---------------------------------------------------------------- this segment's queries
    // Fragment A of step s: slots (2c, 2c + 1) hold d0, d0 + 2 and slots (2c + 8, 2c + 9) hold d0 + 1,
    // d0 + 3, where d0 = dq(s): the order in which a key's four bytes come apart.
    uint32_t qa[R][kSteps][4];
    float rowmul[R][2], offs[R][2], m[R][2], l[R][2], r[R][2], hs[R][2];
    int beg[R][2], end[R][2];
    int full_lo = 0, full_hi = 0x7fffffff;   // tokens that every row sees
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = i * 16 + e * 8 + g;
        const bool live = row < rows_left;
        const int ri = tile * L::kRows + (live ? row : 0);
        const int tok = ri / p.group, head = h * p.group + ri % p.group;
        const uint16_t* const src = p.q + (x.s.row0 + tok) * p.q_stride + head * D;
        uint4 raw[D / 32];
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          // D <= 128: D / 4 contiguous values a lane; D = 256: 32 of each half.
          const int d = D == 256 ? 128 * (w >> 2) + 32 * c + 8 * (w & 3) : (D / 4) * c + 8 * w;
          raw[w] = live ? __ldg(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0u, 0u, 0u, 0u);
        }
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
            qa[i][2 * w + k][e] = *reinterpret_cast<const uint32_t*>(&lo);
            qa[i][2 * w + k][2 + e] = *reinterpret_cast<const uint32_t*>(&hi);
          }
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        offs[i][e] = sum * (128.f / 16777216.f);
        // score (in powers of two) = (acc - offs) * 2^24 * k_scale * scale * log2 e * 2^ex
        rowmul[i][e] = p.scale_log2 * 16777216.f * __uint_as_float((uint32_t)(127 + ex) << 23);
        m[i][e] = kFloor;
        r[i][e] = kFloor;
        l[i][e] = 0.f;
        hs[i][e] = 0.f;
        const int pos = x.s.len - x.s.n + tok;
        end[i][e] = !live ? 0x7fffffff : p.causal ? pos + 1 : x.s.len;
        beg[i][e] = live && p.window > 0 ? max(0, pos - p.window + 1) : 0;
        full_hi = min(full_hi, live ? min(end[i][e], x.s.len) : 0x7fffffff);
        full_lo = max(full_lo, beg[i][e]);
      }
    }
    full_hi = __reduce_min_sync(0xffffffffu, full_hi);
    full_lo = __reduce_max_sync(0xffffffffu, full_lo);
    float o[R][kCols][4];
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int n = 0; n < kCols; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][n][k] = 0.f;

    // ---------------------------------------------------------------- the granules
    for (int j = 0; j < mine_n && !dead; ++j) {
      const uint32_t slot = (count + (uint32_t)j) % NS, phase = ((count + (uint32_t)j) / NS) & 1u;
      const uint8_t* const kst = stage0 + slot * L::kStage;
      const uint8_t* const vst = kst + L::kSide;
      const bool got = mbar_wait(&bar[slot], phase, &abort_flag, p.status);
      if (!__all_sync(0xffffffffu, got)) {
        // A wait ran out (recorded in the status word).  The copies in flight land before this CTA's
        // shared memory is given back; no more are issued.
        dead = true;
        for (int i = j; i < min(j + NS, mine_n); ++i)
          mbar_wait_drain(&bar[(count + (uint32_t)i) % NS], ((count + (uint32_t)i) / NS) & 1u, p.status);
        break;
      }
      const int T = T0 + (warp + j * kWarps) * kGranule;
      const int par = (j >> 5) & 1;
      const float ks = __shfl_sync(0xffffffffu, par ? ks_r[1] : ks_r[0], j & 31);
      const float vs = __shfl_sync(0xffffffffu, par ? vs_r[1] : vs_r[0], j & 31);
      const bool bad = ((par ? bad_r[1] : bad_r[0]) >> (j & 31)) & 1u;

      // Scores of tokens T + 8 t + 2 c (+ 1), rows g and g + 8.
      float s[R][2][4];
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
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
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const uint32_t word = k == 0 ? kb[t].x : k == 1 ? kb[t].y : k == 2 ? kb[t].z : kb[t].w;
            const uint32_t b0 = word & 0x00FF00FFu, b1 = __byte_perm(word, 0u, 0x4341);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const uint32_t* a = qa[i][4 * w + k];
              mma_f16_16816(s[i][t], a[0], a[1], a[2], a[3], b0, b1);
            }
          }
        }
      }
      const bool edge = T < full_lo || T + kGranule > full_hi || bad;
      const float lvs = lg2(vs);
      uint32_t pa[R][4];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float c1 = ks * rowmul[i][e];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) s[i][t][2 * e + k] = (s[i][t][2 * e + k] - offs[i][e]) * c1;
          if (edge) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int tok = T + 8 * t + 2 * c + k;
                if (bad || tok < beg[i][e] || tok >= end[i][e] || tok >= x.s.len) s[i][t][2 * e + k] = -INFINITY;
              }
          }
          mx[e] = fmaxf(fmaxf(s[i][0][2 * e], s[i][0][2 * e + 1]), fmaxf(s[i][1][2 * e], s[i][1][2 * e + 1]));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        }
        const bool move = mx[0] > m[i][0] + kSlack || mx[1] > m[i][1] + kSlack || mx[0] + lvs > r[i][0] + kSlack ||
                          mx[1] + lvs > r[i][1] + kSlack;
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (mx[e] > m[i][e] + kSlack) {
              l[i][e] *= ex2(m[i][e] - mx[e]);
              m[i][e] = mx[e];
            }
            const float want = mx[e] + lvs;
            float rn = want > r[i][e] + kSlack ? want : r[i][e];
            rn = fminf(fmaxf(rn, m[i][e] - kSpan), m[i][e] + kSpan);
            const float a = ex2(r[i][e] - rn);
            r[i][e] = rn;
            hs[i][e] = ex2(m[i][e] - rn);
#pragma unroll
            for (int n = 0; n < kCols; ++n) {
              o[i][n][2 * e] *= a;
              o[i][n][2 * e + 1] *= a;
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = hs[i][e] * vs;
          float w[2][2];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float pr = ex2(s[i][t][2 * e + k] - m[i][e]);
              l[i][e] += pr;
              w[t][k] = pr * f;
            }
          const __half2 lo = __floats2half2_rn(w[0][0], w[0][1]), hi = __floats2half2_rn(w[1][0], w[1][1]);
          pa[i][e] = *reinterpret_cast<const uint32_t*>(&lo);
          pa[i][2 + e] = *reinterpret_cast<const uint32_t*>(&hi);
        }
      }

      // Values: the lane takes 16 (8 for D = 64) contiguous d of tokens 2c, 2c + 1, 2c + 8, 2c + 9, so
      // column n of tile q is d = 16 n + q (8 n + q): a lane's outputs are contiguous too.
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
        if (bx == L::kBoxes - 1) {
          // Every byte of the granule is in registers: its slot takes a later one.
          __syncwarp();
          const int jn = j + NS;
          if (jn < mine_n) {
            if ((jn & 31) == 0) fetch(jn);
            issue(jn);
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
          for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int i = 0; i < R; ++i)
              mma_f16_16816(o[i][bx * 4 * kWords + wd * 4 + d], pa[i][0], pa[i][1], pa[i][2], pa[i][3], bf[0][d], bf[1][d]);
        }
      }
    }
    count += (uint32_t)mine_n;

    // ---------------------------------------------------------------- join the warps, then the CTAs
    const bool whole = ub == 0 && ue == x.units;
    const int slot = u == u0 ? 0 : 1;
    float* const part = p.parts + ((size_t)blockIdx.x * 2 + slot) * L::kPart;
    float* const buf = reinterpret_cast<float*>(ring);
    // The rings hold no copy in flight: every granule issued has been waited for.
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i * 16 >= rows_left) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = l[i][e];
        t += __shfl_xor_sync(0xffffffffu, t, 1);
        t += __shfl_xor_sync(0xffffffffu, t, 2);
        if (c == 0) {
          mlr_sm[warp][8 * e + g][0] = m[i][e];
          mlr_sm[warp][8 * e + g][1] = t;
          mlr_sm[warp][8 * e + g][2] = r[i][e];
        }
        // A lane's sums of a row: D / 4 contiguous ones (D = 256: 32 of each half).
        if (i * 16 + 8 * e + g < rows_left) {
          float* const dst = buf + (warp * 16 + 8 * e + g) * L::kRow;
          constexpr int kHalf = D == 64 ? 8 : 16;
#pragma unroll
          for (int n = 0; n < kCols; n += 4) {
            const int base = (n / kHalf) * 128 + 2 * kHalf * c + (n % kHalf);
#pragma unroll
            for (int y = 0; y < 2; ++y)
              *reinterpret_cast<float4*>(dst + base + y * kHalf) =
                  make_float4(o[i][n][2 * e + y], o[i][n + 1][2 * e + y], o[i][n + 2][2 * e + y], o[i][n + 3][2 * e + y]);
          }
        }
      }
      __syncthreads();
      constexpr int kVec = D / 8;   // threads of a row, eight values each
      for (int row = threadIdx.x / kVec; row < 16 && i * 16 + row < rows_left; row += kThreads / kVec) {
        const int d = 8 * (threadIdx.x % kVec);
        float M = kFloor, Rf = kFloor;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          M = fmaxf(M, mlr_sm[w][row][0]);
          Rf = fmaxf(Rf, mlr_sm[w][row][2]);
        }
        float lt = 0.f, acc[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          lt += mlr_sm[w][row][1] * ex2(mlr_sm[w][row][0] - M);
          const float a = ex2(mlr_sm[w][row][2] - Rf);
          const float4 v0 = *reinterpret_cast<const float4*>(buf + (w * 16 + row) * L::kRow + d);
          const float4 v1 = *reinterpret_cast<const float4*>(buf + (w * 16 + row) * L::kRow + d + 4);
          const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = fmaf(v[k], a, acc[k]);
        }
        if (whole) {
          const int ri = tile * L::kRows + i * 16 + row;
          const int orow = x.s.row0 + ri / p.group, head = h * p.group + ri % p.group;
          const float z = lt == 0.f ? 0.f : __fdividef(1.f, lt) * ex2(Rf - M);
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] *= z;
          *reinterpret_cast<uint4*>(p.out + orow * p.out_stride + head * D + d) = pack8<kF16>(acc);
          if (p.lse && d == 0)
            p.lse[(size_t)orow * p.q_heads + head] = lt == 0.f ? -INFINITY : (M + lg2(lt)) * 0.69314718056f;
        } else {
          float4* const dst = reinterpret_cast<float4*>(part + (i * 16 + row) * D + d);
          dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
          dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
          if (d == 0) *reinterpret_cast<float4*>(part + L::kRows * D + (i * 16 + row) * 4) = make_float4(M, lt, Rf, 0.f);
        }
      }
      if (i + 1 < R) __syncthreads();
    }
    if (!whole) {
      // The part is written; the last CTA to arrive joins all of the item's, in the CTAs' order.
      const int first = runs.owner(item_u0), last = runs.owner(item_u0 + x.units - 1);
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const uint32_t n = (uint32_t)(last - first + 1);
        const uint32_t old = atom_add_acq_rel_u32(p.counters + first, 1u);
        if (old >= n) atomicOr(p.status, W8A8_DEV_COUNTER_CORRUPT);
        if (old == n - 1) p.counters[first] = 0u;   // ready for the next call
        last_sm = old == n - 1;
      }
      __syncthreads();
      if (last_sm) {
        __threadfence();
        constexpr int kVec = D / 8;
        const int rows = min(rows_left, L::kRows);
        // The first CTA's part is its last segment unless the item begins its run.
        const int first_slot = runs.begin(first) == item_u0 ? 0 : 1;
        for (int row = threadIdx.x / kVec; row < rows; row += kThreads / kVec) {
          const int d = 8 * (threadIdx.x % kVec);
          float M = kFloor, Rf = kFloor;
          for (int i = first; i <= last; ++i) {
            const float* src = p.parts + ((size_t)i * 2 + (i == first ? first_slot : 0)) * L::kPart;
            const float4 t = __ldcg(reinterpret_cast<const float4*>(src + L::kRows * D + row * 4));
            M = fmaxf(M, t.x);
            Rf = fmaxf(Rf, t.z);
          }
          float lt = 0.f, acc[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] = 0.f;
#pragma unroll 4
          for (int i = first; i <= last; ++i) {
            const float* src = p.parts + ((size_t)i * 2 + (i == first ? first_slot : 0)) * L::kPart;
            const float4 t = __ldcg(reinterpret_cast<const float4*>(src + L::kRows * D + row * 4));
            const float4 v0 = __ldcg(reinterpret_cast<const float4*>(src + row * D + d));
            const float4 v1 = __ldcg(reinterpret_cast<const float4*>(src + row * D + d + 4));
            lt += t.y * ex2(t.x - M);
            const float a = ex2(t.z - Rf);
            const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = fmaf(v[k], a, acc[k]);
          }
          const int ri = tile * L::kRows + row;
          const int orow = x.s.row0 + ri / p.group, head = h * p.group + ri % p.group;
          const float z = lt == 0.f ? 0.f : __fdividef(1.f, lt) * ex2(Rf - M);
#pragma unroll
          for (int k = 0; k < 8; ++k) acc[k] *= z;
          *reinterpret_cast<uint4*>(p.out + orow * p.out_stride + head * D + d) = pack8<kF16>(acc);
          if (p.lse && d == 0)
            p.lse[(size_t)orow * p.q_heads + head] = lt == 0.f ? -INFINITY : (M + lg2(lt)) * 0.69314718056f;
        }
      }
    }
    u = item_u0 + ue;
    if (u < u1) {
      // The join buffer lies over the rings: plain accesses to it come before the next copies.
      fence_async_shared();
      __syncthreads();
    }
  }
}

template <bool kF16, int D, int R>
static cudaError_t launch_few(const Params& p, int sms, cudaStream_t stream) {
  // No more CTAs than units there can be (lengths are known to the device alone).
  using L = Layout<D, R>;
  auto kern = kv8_attention_kernel<kF16, D, R>;
  cudaError_t e = ensure_smem_attribute((const void*)kern, L::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const long long tiles = ((long long)p.step.max_tokens * p.group + L::kRows - 1) / L::kRows;
  const long long units = (((long long)p.step.table_width << p.page_shift) + kUnit - 1) / kUnit;
  const long long most = tiles * units >= sms * L::kCtas ? sms * L::kCtas : tiles * units * p.step.seqs * p.kv_heads;
  cfg.gridDim = dim3((unsigned)(most < sms * L::kCtas ? most : sms * L::kCtas));
  cfg.blockDim = dim3(kThreads);
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

// Bytes of the parts of every variant of a head size.
template <int D, int R>
static size_t parts_bytes(int sms) {
  using L = Layout<D, R>;
  return (size_t)sms * L::kCtas * 2 * L::kPart * sizeof(float);
}

constexpr size_t counters_bytes(int sms) { return ((size_t)sms * 3 * sizeof(uint32_t) + 255) / 256 * 256; }

}  // namespace attn
}  // namespace w8a8

using namespace w8a8;

extern "C" size_t kv8_workspace_bytes(int q_heads, int kv_heads, int head_dim) {
  if (kv8_check_dims(kv_heads, head_dim) != W8A8_OK || q_heads < 0 || q_heads > 4096) return 0;
  const int sms = device_sm_count();
  size_t parts = 0;
  auto add = [&](size_t n) { parts = n > parts ? n : parts; };
  if (head_dim == 64) add(attn::parts_bytes<64, 1>(sms)), add(attn::parts_bytes<64, 2>(sms));
  else if (head_dim == 128) add(attn::parts_bytes<128, 1>(sms)), add(attn::parts_bytes<128, 2>(sms));
  else add(attn::parts_bytes<256, 1>(sms));
  return kWsHeaderBytes + attn::counters_bytes(sms) + parts;
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
  const int sms = device_sm_count();
  attn::Params p;
  // The cache as rows of D bytes, one for each (page, kv head, token).
  const int P = cache->page_tokens;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)cache->pages * cache->kv_heads * P};
  const cuuint64_t strides[1] = {(cuuint64_t)D};
  const cuuint32_t box[2] = {(cuuint32_t)(D > 128 ? 128 : D), (cuuint32_t)attn::kGranule};
  const cuuint32_t estr[2] = {1u, 1u};
  const CUtensorMapSwizzle swizzle = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  cudaError_t e = encode_tensor_map_2d(&p.kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->k, dims, strides, box, estr, swizzle);
  if (e == cudaSuccess)
    e = encode_tensor_map_2d(&p.vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache->v, dims, strides, box, estr, swizzle);
  if (e != cudaSuccess) return record_cuda_error(e, "kv8_attention");
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
  p.window = window, p.causal = (flags & KV8_FLAG_NOT_CAUSAL) ? 0 : 1;
  p.scale_log2 = scale * 1.4426950408889634f;
  uint8_t* const w = static_cast<uint8_t*>(ws);
  p.status = reinterpret_cast<uint32_t*>(w);
  p.counters = reinterpret_cast<uint32_t*>(w + kWsHeaderBytes);
  p.parts = reinterpret_cast<float*>(w + kWsHeaderBytes + attn::counters_bytes(sms));
  const bool f16 = dtype == KV8_F16;
  const bool few = (long long)step->max_tokens * p.group <= 16;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
#define KV8_FEW(D, R) (f16 ? attn::launch_few<true, D, R>(p, sms, s) : attn::launch_few<false, D, R>(p, sms, s))
  if (D == 64) e = few ? KV8_FEW(64, 1) : KV8_FEW(64, 2);
  else if (D == 128) e = few ? KV8_FEW(128, 1) : KV8_FEW(128, 2);
  else e = KV8_FEW(256, 1);
#undef KV8_FEW
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "kv8_attention");
}
