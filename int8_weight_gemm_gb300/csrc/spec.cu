// Ends of a speculative decoding step: the probabilities of a vocabulary from its logits (spec_probs), and the
// verification of drafted tokens against them from given random numbers (spec_verify).
#include <mutex>

#include "internal.h"
#include "kv8.cuh"

namespace w8a8 {
namespace spec {

// A 16-bit value as a float (exact).
template <bool kF16>
__device__ __forceinline__ float value16(uint16_t h) {
  return kF16 ? __half2float(__ushort_as_half(h)) : __uint_as_float((uint32_t)h << 16);
}

template <int kType>
struct Type {   // KV8_BF16, KV8_F16
  using T = uint16_t;
  static __device__ __forceinline__ void load4(const T* x, float (&f)[4]) {
    const uint2 v = *reinterpret_cast<const uint2*>(x);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = value16<kType == KV8_F16>((uint16_t)((i < 2 ? v.x : v.y) >> (16 * (i & 1))));
  }
  static __device__ __forceinline__ float load(const T* x) { return value16<kType == KV8_F16>(*x); }
};
template <>
struct Type<SPEC_F32> {
  using T = float;
  static __device__ __forceinline__ void load4(const T* x, float (&f)[4]) {
    const float4 v = *reinterpret_cast<const float4*>(x);
    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
  }
  static __device__ __forceinline__ float load(const T* x) { return *x; }
};

// ------------------------------------------------------------------------------------------------ probabilities
//   p_i = exp((x_i - m) / T) / sum_j exp((x_j - m) / T),   m = max x
//
// What bounds it: HBM, two bytes in and four out for each of a row's values (bf16), eight instructions beside them.
// A row is held in the registers of a cluster of up to eight CTAs, so it is read once and its exponentials are taken
// once: relative to the warp's own maximum, then times one factor that follows from all warps' maxima and sums, which go
// to every CTA through distributed shared memory, as stores that count towards its barrier: a barrier of the cluster
// would first wait for the previous row's stores to HBM.  A warp waits for the others once a row.  Clusters stay for
// several rows: a warp copies its part of the next row into shared memory as soon as it has this one's in registers, and
// the row after that is fetched into L2, so that loads hide behind a whole row's work (320 rows of 131072: loads into
// registers behind the stores 58 us, without the fetch into L2 94).
//
// Measured (bf16): 320 rows of 131072 48 us, 5.2 TB/s, 77 % of a copy's rate; 16 rows of 32000 3.7 us.  Beyond 131072 a thread
// holds 64 values and an SM one CTA: 320 rows of 151936 74 us (58 %), 201088 83 (69 %), 262144 95 (78 %).  Rows not in whole 16
// bytes, one value a load: 50257 in a stride of 50304 27.8 us (51 %; 50304 21.7), 131071 67.7.
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct ProbsParams {
  const void* x;
  long long x_stride;
  const float* inv_temp;
  float* out;
  long long out_stride;
  int rows, vocab, share, ctas;   // a CTA's values (a multiple of four), a row's CTAs
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Two floats into a CTA's shared memory, eight bytes towards the phase of its barrier.
__device__ __forceinline__ void st_async_v2f(uint32_t addr, float a, float b, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(a), "f"(b),
               "r"(bar)
               : "memory");
}
// Wait for a phase of this CTA's barrier, about a second at most (every warp of the row sends to it, so it does complete).
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
  if (mbar_test_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait_suspend(bar, parity))
    if (clock64() - t0 > kWaitTimeoutCycles) return false;
  return true;
}

// kE: values a thread holds, of its warp's 32 kE consecutive ones.  kVec: four neighbours at a time, by way of shared memory
// (rows, strides and the vocabulary in whole 16 bytes); else one, into the register.
template <int kType, int kE, bool kVec>
__global__ void __launch_bounds__(kThreads, kE <= 32 ? 2 : 1) spec_probs_kernel(const __grid_constant__ ProbsParams p) {
  using Ty = Type<kType>;
  using T = typename Ty::T;
  // Of each warp of the row, for two rows in turn: its maximum, and the sum of its exponentials (temperature 0: the place
  // of its first largest value).
  __shared__ __align__(8) float2 peers_sm[2][kMaxCluster * kWarps];
  __shared__ __align__(8) uint64_t full[2];
  __shared__ __align__(8) uint64_t loaded[kWarps];
  extern __shared__ __align__(16) uint8_t smem_raw[];   // kVec: a warp's part of the next row
  const int rank = (int)cluster_ctarank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int stride = gridDim.x / p.ctas;   // clusters
  if (threadIdx.x == 0) {
    mbar_init(&full[0], 1), mbar_init(&full[1], 1);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mbar_init(&loaded[w], 1);
    mbar_fence_init();
  }
  __syncwarp();
  // Behind this barrier every CTA has begun, and its barriers may be used: by its own warps too.
  cluster_arrive();
  pdl_trigger();
  pdl_wait();
  __syncwarp();
  cluster_wait();
  const int begin = rank * p.share, end = min(p.vocab, begin + p.share);
  // A thread's values: i-th of v at place first + (i / kN) * 32 * kN + i % kN of the row.
  constexpr int kN = kVec ? 4 : 1;
  const int warp_first = begin + warp * 32 * kE;
  const size_t first = (size_t)warp_first + kN * lane;
  const int left = end - (int)first;   // values from the thread's first on
  auto place = [](int i) { return (i / kN) * 32 * kN + i % kN; };
  float v[kE];
  T* const part = reinterpret_cast<T*>(smem_raw) + warp * 32 * kE;
  const uint32_t part_bytes = (uint32_t)(max(0, min(32 * kE, end - warp_first)) * (int)sizeof(T));
  auto fetch = [&](int row) {   // this warp's part of a row, by one lane
    if (kVec && lane == 0 && row < p.rows && part_bytes > 0) {
      mbar_arrive_expect_tx(&loaded[warp], part_bytes);
      bulk_g2s(part, static_cast<const T*>(p.x) + row * p.x_stride + warp_first, part_bytes, &loaded[warp]);
    }
  };
  auto ahead = [&](int row) {
    if (threadIdx.x == 0 && row < p.rows && end > begin) {
      // Whole 16-byte pieces of the CTA's share.
      const uintptr_t a = (reinterpret_cast<uintptr_t>(static_cast<const T*>(p.x) + row * p.x_stride + begin) + 15) & ~uintptr_t(15);
      const uintptr_t b = reinterpret_cast<uintptr_t>(static_cast<const T*>(p.x) + row * p.x_stride + end) & ~uintptr_t(15);
      if (b > a) bulk_prefetch_l2(reinterpret_cast<const void*>(a), (uint32_t)(b - a));
    }
  };
  int row = blockIdx.x / p.ctas;
  auto factor_of = [&](int row) { return p.inv_temp && row < p.rows ? fmaxf(p.inv_temp[row], 0.f) : 1.f; };   // (a NaN: 0)
  float next_inv = factor_of(row);
  fetch(row);
  ahead(row + stride);
  for (uint32_t n = 0; row < p.rows; row += stride, ++n) {
    // (The place of row n is written again for row n + 2 by warps that have every warp's numbers of row n + 1, which
    // each sends when it has read those of row n.)
    const uint32_t turn = n & 1u;
    bool got = true;
    if (kVec && part_bytes > 0) got = wait_phase(&loaded[warp], n & 1u);
    const T* const src = static_cast<const T*>(p.x) + row * p.x_stride + first;
#pragma unroll
    for (int i = 0; i < kE; i += kN) {
      float f[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (place(i) < left) {
        if (kVec) Ty::load4(part + kN * lane + place(i), f);
        else f[0] = Ty::load(src + place(i));
      }
#pragma unroll
      for (int k = 0; k < kN; ++k) v[i + k] = f[k];
    }
    if (kVec) {
      // (The copy's writes are the asynchronous proxy's: they come after the lanes' reads.)
      fence_async_shared();
      __syncwarp();
      fetch(row + stride);
    }
    ahead(row + 2 * stride);
    const float inv = next_inv;
    next_inv = factor_of(row + stride);
    const bool greedy = inv == INFINITY, steep = inv > 0x1p126f;
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kE; ++i) m = fmaxf(m, v[i]);   // (a NaN is passed over)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float second;
    if (greedy) {
      int at = p.vocab;
#pragma unroll
      for (int i = kE - 1; i >= 0; --i)
        if (v[i] == m) at = min(at, (int)first + place(i));
      second = __int_as_float(m == -INFINITY ? p.vocab : __reduce_min_sync(0xffffffffu, at));
    } else {
      if (m == INFINITY) {
        // Values of +inf share the row.
#pragma unroll
        for (int i = 0; i < kE; ++i) v[i] = v[i] == INFINITY ? 0.f : -INFINITY;
      }
      const float ref = fabsf(m) == INFINITY ? 0.f : m;
      uint64_t sum2[2] = {0, 0};   // (0, 0)
      auto weights = [&](float times, float k2) {
        const uint64_t ref2 = pair(-ref, -ref), k22 = pair(k2, k2), times2 = pair(times, times);
#pragma unroll
        for (int i = 0; i < kE; i += 2) {
          float a, b;
          const uint64_t d = add2(pair(v[i], v[i + 1]), ref2);
          unpair(mul2(times == 1.f ? d : mul2(d, times2), k22), a, b);
          v[i] = ex2(a);
          v[i + 1] = ex2(b);
          sum2[(i >> 1) & 1] = add2(sum2[(i >> 1) & 1], pair(v[i], v[i + 1]));
        }
      };
      // The product with log2 e is one factor with 1 / T; where it would pass the largest float, the differences take four of
      // it.  (A copy of its own: chosen inside one, 320 rows of 131072 49.3 us, not 47.4.)
      if (!steep) weights(1.f, inv * 1.44269504f);
      else weights(4.f, 0.25f * inv * 1.44269504f);
      auto total = [&]() {
        float a, b;
        unpair(add2(sum2[0], sum2[1]), a, b);
        a += b;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        return a;
      };
      second = total();
      if (second != second) {
        // Of logits that are NaN, or masked ones times 0: no weight.
        sum2[0] = sum2[1] = 0;
#pragma unroll
        for (int i = 0; i < kE; i += 2) {
          v[i] = v[i] != v[i] ? 0.f : v[i];
          v[i + 1] = v[i + 1] != v[i + 1] ? 0.f : v[i + 1];
          sum2[0] = add2(sum2[0], pair(v[i], v[i + 1]));
        }
        second = total();
      }
    }
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&full[turn], (uint32_t)(p.ctas * kWarps * sizeof(float2)));
    if (lane < p.ctas)
      st_async_v2f(cluster_map(smem_addr(&peers_sm[turn][rank * kWarps + warp]), lane), m, second, cluster_map(smem_addr(&full[turn]), lane));
    got = wait_phase(&full[turn], (n >> 1) & 1u) && got;
    constexpr int kPeers = kMaxCluster * kWarps / 32;   // a lane's
    float2 peers[kPeers];
    float M = -INFINITY;
#pragma unroll
    for (int c = 0; c < kPeers; ++c) {
      peers[c] = make_float2(-INFINITY, greedy ? __int_as_float(p.vocab) : 0.f);
      if (32 * c + lane < p.ctas * kWarps) peers[c] = peers_sm[turn][32 * c + lane];
      M = fmaxf(M, peers[c].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float factor = 1.f;
    int best = p.vocab;
    if (greedy) {
#pragma unroll
      for (int c = 0; c < kPeers; ++c)
        if (peers[c].x == M) best = min(best, __float_as_int(peers[c].y));
      best = __reduce_min_sync(0xffffffffu, best);
#pragma unroll
      for (int i = 0; i < kE; ++i) v[i] = (int)first + place(i) == best ? 1.f : 0.f;
    } else {
      const float k2 = inv * 1.44269504f;
      auto weight = [&](float x) {
        if (__builtin_expect(steep, 0)) return x == M ? 1.f : ex2(fmaxf(4.f * (x - M) * (0.25f * inv * 1.44269504f), -200.f));
        return x == M ? 1.f : ex2(fmaxf((x - M) * k2, -200.f));
      };
      float S = 0.f;
#pragma unroll
      for (int c = 0; c < kPeers; ++c) S = fmaf(peers[c].y, weight(peers[c].x), S);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
      factor = S > 0.f ? __fdiv_rn(weight(m), S) : 0.f;
    }
    if (!got) factor = NAN;
    float* const dst = p.out + row * p.out_stride;
#pragma unroll
    for (int i = 0; i < kE; i += kN) {
      if (place(i) < left) {
        float* const to = dst + first + place(i);
        if (kVec) *reinterpret_cast<float4*>(to) = make_float4(v[i] * factor, v[i + 1] * factor, v[i + 2] * factor, v[i + 3] * factor);
        else *to = v[i] * factor;
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------ verification
// A window's row r holds the target's probabilities p after its token, and the draft's q that the next row's token d was
// drawn from.  d is accepted where  accept * q(d) < p(d)  (a product of two fp32 numbers is exact in 64 bits).  The first
// row whose successor is not accepted draws the token after it from max(p - q, 0), the last row from p:
//   token = the first k with  sum_{i <= k} w_i > u * sum_i w_i.
// Whole numbers come out, which one rounding in a sum of 10^5 terms could change.  So the weights are taken in units of
// 2^-44 (rounded once, exact from 2^-20 on) as 64-bit integers: their sums do not depend on an order, and 2^18 of them
// of at most 1 stay below 2^62.
//
// What bounds it: HBM, p and q of one row a sequence, read once.  A sequence's row is cut into segments, one a warp;
// the last CTA to arrive finds the segment in which the draw lies from their sums and reads it again (out of L2).
//
// Measured: 64 windows of 2 to 8 over 131072 (fp32, with the draft's) 19.3 us, half of it 67 MB at HBM's rate, the rest a chain of
// loads before (offsets, token, its probabilities) and after (arrival, sums, segment); one window of 6 over 32000 6.0 us.
constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMinSegment = 512;
constexpr int kCtasPerSm = 4;

struct VerifyParams {
  const void *p, *q;
  long long p_stride, q_stride;
  const int *tokens, *row0;
  const float *accept, *sample;
  int *next, *take;
  int rows, vocab, ctas, segment;   // a sequence's CTAs, a warp's values
  uint32_t* status;
  uint32_t* counters;   // [seqs] arrivals, zero between calls
  long long* sums;      // [seqs][ctas * kVWarps]
};

// x, taken inside [0, 1] (a NaN: 0), in units of 2^-44 as two whole numbers, hi 2^23 + lo: the last bits of sums with
// constants whose own last bit is 2^-21 and 2^-44.  (Two of the conversions to 64 bits a value set the pace before: 64 rows of
// 131072 42 us.)  The constants' bits are still in, and leave in the difference of two values.
struct Units {
  int hi, lo;
};
constexpr float kHiStep = 6.f, kLoStep = 7.152557373046875e-07f;   // 1.5 * 2^2, 1.5 * 2^-21
__device__ __forceinline__ Units units(float x) {
  x = __saturatef(x);
  const float hi = __fadd_rn(x, kHiStep);
  const float lo = __fadd_rn(__fsub_rn(x, __fsub_rn(hi, kHiStep)), kLoStep);   // (the differences are exact)
  return {__float_as_int(hi), __float_as_int(lo)};
}
__device__ __forceinline__ long long weight_of(Units a, Units b) {
  return max((long long)(a.hi - b.hi) * (1 << 23) + (a.lo - b.lo), 0ll);
}

// What a row draws from.
struct Draw {
  int row, last;   // its place among the rows; 1: the window's last row draws from p
  int token;       // the rejected token (without q its weight is 0)
};

template <int kType, bool kVec>
__global__ void __launch_bounds__(kVThreads, kCtasPerSm) spec_verify_kernel(const __grid_constant__ VerifyParams p) {
  using Ty = Type<kType>;
  using T = typename Ty::T;
  __shared__ Draw draw_sm;
  __shared__ int window_sm[2];    // first row, rows
  __shared__ long long scan_sm[kVWarps];
  __shared__ int found_sm[2];     // segment, token
  __shared__ long long at_sm;     // weight still to pass inside the segment
  __shared__ int last_sm;
  pdl_trigger();
  pdl_wait();
  const int seq = blockIdx.x / p.ctas, cta = blockIdx.x % p.ctas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---------------------------------------------------------------- the window's tokens
  if (warp == 0) {
    const int r0 = p.row0[seq], r1 = p.row0[seq + 1];
    const bool ok = r0 >= 0 && r1 >= r0 && r1 <= p.rows;
    const int n = ok ? r1 - r0 : 0;
    if (!ok && lane == 0 && cta == 0) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
    int stop = n - 1, token = -1;
    for (int i0 = 0; i0 < n - 1; i0 += 32) {
      const int i = i0 + lane;
      bool in = true;
      int d = 0;
      if (i < n - 1) {
        const size_t r = (size_t)r0 + i;
        d = p.tokens[r + 1];
        in = d >= 0 && d < p.vocab;
        if (!in) {
          if (cta == 0) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
        } else {
          const float pd = __saturatef(Ty::load(static_cast<const T*>(p.p) + r * p.p_stride + d));
          const float qd = p.q ? __saturatef(Ty::load(static_cast<const T*>(p.q) + r * p.q_stride + d)) : 1.f;
          in = (double)__saturatef(p.accept[r]) * (double)qd < (double)pd;
        }
      }
      const uint32_t out = __ballot_sync(0xffffffffu, !in);
      if (out) {
        const int src = __ffs(out) - 1;
        stop = i0 + src;
        token = __shfl_sync(0xffffffffu, d, src);
        break;
      }
    }
    if (lane == 0) {
      found_sm[0] = found_sm[1] = 0, at_sm = 0;
      draw_sm = Draw{r0 + stop, stop == n - 1, token};
      window_sm[0] = r0, window_sm[1] = n;
    }
  }
  __syncthreads();
  const int r0 = window_sm[0], n = window_sm[1];
  if (n == 0) {
    if (cta == 0 && threadIdx.x == 0) p.take[seq] = 0;
    return;
  }
  const Draw draw = draw_sm;
  const T* const prow = static_cast<const T*>(p.p) + draw.row * p.p_stride;
  const T* const qrow = p.q && !draw.last ? static_cast<const T*>(p.q) + draw.row * p.q_stride : nullptr;
  const int none = draw.last || qrow ? -1 : draw.token;   // the token without weight

  // The sum of the weights of [a, b), a lane's share each (`target`: of p alone).  A token without weight is taken off by
  // the lane that has it.
  const Units zero = units(0.f);
  auto weight_at = [&](int i, bool target) {
    const bool diff = qrow && !target;
    return !target && i == none ? 0 : weight_of(units(Ty::load(prow + i)), diff ? units(Ty::load(qrow + i)) : zero);
  };
  auto weigh = [&](int a, int b, bool target) {
    long long s = 0;
    if (kVec) {
      int i = a + 4 * lane;
      if (qrow && !target) {
#pragma unroll 4
        for (; i + 4 <= b; i += 128) {
          float f[4], g[4];
          Ty::load4(prow + i, f);
          Ty::load4(qrow + i, g);
#pragma unroll
          for (int k = 0; k < 4; ++k) s += weight_of(units(f[k]), units(g[k]));
        }
      } else {
#pragma unroll 8
        for (; i + 4 <= b; i += 128) {
          float f[4];
          Ty::load4(prow + i, f);
#pragma unroll
          for (int k = 0; k < 4; ++k) s += weight_of(units(f[k]), zero);
        }
        if (!target && none >= a && none < i && ((none - a) >> 2) % 32 == lane) s -= weight_of(units(Ty::load(prow + none)), zero);
      }
      for (int k = i; k < min(b, i + 4); ++k) s += weight_at(k, target);
    } else {
#pragma unroll 8
      for (int i = a + lane; i < b; i += 32) s += weight_at(i, target);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  };
  const int segments = p.ctas * kVWarps;
  long long* const sums = p.sums + (size_t)seq * segments;
  auto segment_of = [&](int s, int& a, int& b) {
    a = (int)min((long long)p.vocab, (long long)s * p.segment), b = min(p.vocab, a + p.segment);
  };
  {
    int a, b;
    segment_of(cta * kVWarps + warp, a, b);
    const long long s = weigh(a, b, false);
    if (lane == 0) sums[cta * kVWarps + warp] = s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    // (The barrier orders the CTA's stores before this thread's release, and its acquire before the reads.)
    const uint32_t old = atom_add_acq_rel_u32(p.counters + seq, 1u);
    if (old >= (uint32_t)p.ctas) atomicOr(p.status, W8A8_DEV_COUNTER_CORRUPT);
    last_sm = old == (uint32_t)p.ctas - 1;
    if (last_sm) p.counters[seq] = 0u;   // ready for the next call
  }
  __syncthreads();
  if (!last_sm) return;

  // ---------------------------------------------------------------- the draw
  // Sum before this thread's share and of all, of one number a thread.
  auto scan = [&](long long mine, long long& all) {
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    __syncthreads();
    if (lane == 31) scan_sm[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    all = 0;
#pragma unroll
    for (int w = 0; w < kVWarps; ++w) {
      if (w < warp) before += scan_sm[w];
      all += scan_sm[w];
    }
    return before;
  };
  const float u = p.sample[draw.row];
  bool target = draw.last;
  int token = -1;
  for (;;) {
    const int per = (segments + kVThreads - 1) / kVThreads;
    const int s0 = min(segments, (int)threadIdx.x * per), s1 = min(segments, s0 + per);
    long long mine = 0, all;
    for (int s = s0; s < s1; ++s) mine += __ldcg(sums + s);
    const long long before = scan(mine, all);
    if (all > 0) {
      // floor(u * all): a whole number is above the product where it is above its floor.
      const uint32_t bits = __float_as_uint(__saturatef(u));
      const int ex = (int)(bits >> 23);
      const unsigned __int128 product = (unsigned __int128)(uint64_t)all * ((bits & 0x7FFFFFu) | (ex ? 0x800000u : 0u));
      const int down = 150 - max(ex, 1);   // u = fraction * 2^-down
      long long at = down < 100 ? (long long)(product >> down) : 0;
      at = min(at, all - 1);
      if (at >= before && at < before + mine) {
        at -= before;
        int s = s0;
        for (long long x; s + 1 < s1 && at >= (x = __ldcg(sums + s)); ++s) at -= x;
        found_sm[0] = s;
        at_sm = at;
      }
      __syncthreads();
      int a, b;
      segment_of(found_sm[0], a, b);
      const int share = (b - a + kVThreads - 1) / kVThreads;
      const int i0 = min(b, a + (int)threadIdx.x * share), i1 = min(b, i0 + share);
      mine = 0;
#pragma unroll 8
      for (int i = i0; i < i1; ++i) mine += weight_at(i, target);
      const long long ahead = scan(mine, all);
      at = at_sm;
      if (at >= ahead && at < ahead + mine) {
        at -= ahead;
        int i = i0;
        for (long long x; i + 1 < i1 && at >= (x = weight_at(i, target)); ++i) at -= x;
        found_sm[1] = i;
      }
      __syncthreads();
      token = found_sm[1];
      break;
    }
    // Nothing to draw from: p has nowhere more than q, or is zero but for the rejected token.  Then from p itself.
    if (target) {
      if (threadIdx.x == 0) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
      break;
    }
    target = true;
    __syncthreads();
    for (int s = warp; s < segments; s += kVWarps) {
      int a, b;
      segment_of(s, a, b);
      const long long x = weigh(a, b, true);
      if (lane == 0) __stcg(sums + s, x);
    }
    __syncthreads();
  }
  const int stop = draw.row - r0;
  for (int i = threadIdx.x; i < n; i += kVThreads) p.next[r0 + i] = i < stop ? p.tokens[r0 + i + 1] : i == stop ? token : -1;
  if (threadIdx.x == 0) p.take[seq] = stop + 1;
}

// ------------------------------------------------------------------------------------------------ host
static int size_of(int dtype) { return dtype == SPEC_F32 ? 4 : 2; }

// Rows of `size`-byte values: four at a time where every row begins on a boundary of four.
static bool vectors(const void* x, long long stride, int size) { return kv8_aligned(x, 4 * size) && stride % 4 == 0; }

static int check_rows(const void* x, long long stride, int rows, int vocab, int size) {
  if (!x || (rows > 1 && stride < vocab) || stride < 0 || stride > (1ll << 31)) return W8A8_ERR_INVALID_ARG;
  return kv8_aligned(x, size) ? W8A8_OK : W8A8_ERR_MISALIGNED;
}

template <typename P>
static cudaError_t launch(void (*kernel)(const P), long long grid, int threads, int cluster, int smem, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename P>
using Kernel = void (*)(const P);

template <int kE, bool kVec>
static Kernel<ProbsParams> probs_kernel(int dtype) {
  return dtype == SPEC_F32 ? spec_probs_kernel<SPEC_F32, kE, kVec>
         : dtype == KV8_F16 ? spec_probs_kernel<KV8_F16, kE, kVec>
                            : spec_probs_kernel<KV8_BF16, kE, kVec>;
}
template <bool kVec>
static Kernel<VerifyParams> verify_kernel(int dtype) {
  return dtype == SPEC_F32 ? spec_verify_kernel<SPEC_F32, kVec>
         : dtype == KV8_F16 ? spec_verify_kernel<KV8_F16, kVec>
                            : spec_verify_kernel<KV8_BF16, kVec>;
}

// Clusters of `ctas` CTAs that the current device holds at once.  (A cluster lies within one of its groups of SMs, so this is
// less than the SMs' places over the size; asked once for each kernel, size and device.)
static cudaError_t resident_clusters(Kernel<ProbsParams> kernel, int ctas, int smem, int* clusters) {
  struct Entry {
    const void* kernel;
    int ctas, device, clusters;
  };
  static Entry table[512];
  static int used = 0;
  static std::mutex mu;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < used; ++i)
    if (table[i].kernel == (const void*)kernel && table[i].ctas == ctas && table[i].device == device) {
      *clusters = table[i].clusters;
      return cudaSuccess;
    }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  if (smem > 0 && (e = ensure_smem_attribute((const void*)kernel, smem)) != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(clusters, (const void*)kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (*clusters < 1) *clusters = 1;
  if (used < 512) table[used++] = Entry{(const void*)kernel, ctas, device, *clusters};
  return cudaSuccess;
}

constexpr int kMaxVocab = 1 << 18;
constexpr int kMaxSeqs = 65535;
// (For any number of sequences: a workspace may serve calls of different ones, whose counters are zero between calls.)
constexpr size_t kCounterBytes = ((size_t)kMaxSeqs * sizeof(uint32_t) + 255) / 256 * 256;

// A sequence's CTAs: as many as the SMs hold for all sequences together, of segments that are worth a warp.
static int most_ctas(int vocab) { return (vocab + kMinSegment * kVWarps - 1) / (kMinSegment * kVWarps); }
static int verify_ctas(int seqs, int vocab, int sms) {
  const int most = most_ctas(vocab), want = sms * kCtasPerSm / seqs;
  return want < 1 ? 1 : want < most ? want : most;
}
// All sequences' CTAs at most, of any call with up to as many sequences and tokens (the quotient above rounds down, so the
// product itself may be larger for fewer sequences).
static size_t most_places(int seqs, int vocab, int sms) {
  const long long all = (long long)seqs * most_ctas(vocab), held = (long long)sms * kCtasPerSm, places = all < held ? all : held;
  return (size_t)(places > seqs ? places : seqs);
}

}  // namespace spec
}  // namespace w8a8

using namespace w8a8;

extern "C" int spec_probs(const void* logits, long long logits_stride, const float* inv_temp, float* out, long long out_stride, int rows,
                          int vocab, int dtype, void* stream) {
  if (rows < 0 || rows > (1 << 22) || vocab < 1 || vocab > spec::kMaxVocab || (dtype != KV8_BF16 && dtype != KV8_F16 && dtype != SPEC_F32))
    return W8A8_ERR_INVALID_ARG;
  if (rows == 0) return W8A8_OK;   // an empty tensor has no address
  const int size = spec::size_of(dtype);
  int rc = spec::check_rows(logits, logits_stride, rows, vocab, size);
  if (rc == W8A8_OK) rc = spec::check_rows(out, out_stride, rows, vocab, 4);
  if (rc != W8A8_OK) return rc;
  if (!kv8_aligned(inv_temp, 4)) return W8A8_ERR_MISALIGNED;
  // A row's CTAs (1, 2, 4 or 8: other clusters leave more of the SMs' places empty): as few as hold it at 32 values a
  // thread (64 for a vocabulary that eight would not hold), more while rows are few, so that every SM has some.
  const int sms = device_sm_count(), most = (vocab > 8 * 32 * spec::kThreads ? 64 : 32) * spec::kThreads;
  int ctas = 1;
  while (ctas < spec::kMaxCluster && ((long long)ctas * most < vocab || (long long)rows * ctas < sms)) ctas *= 2;
  spec::ProbsParams p{logits, logits_stride, inv_temp, out, out_stride, rows, vocab, ((vocab + ctas - 1) / ctas + 7) / 8 * 8, ctas};
  const int each = (p.share + spec::kThreads - 1) / spec::kThreads, held = each <= 8 ? 8 : each <= 16 ? 16 : each <= 32 ? 32 : 64;
  auto whole = [](const void* x, long long stride, int vocab, int size) {
    return kv8_aligned(x, 16) && stride * size % 16 == 0 && vocab * size % 16 == 0;
  };
  const bool vec = whole(logits, logits_stride, vocab, size) && whole(out, out_stride, vocab, 4);
  spec::Kernel<spec::ProbsParams> k =
      vec ? (held == 8 ? spec::probs_kernel<8, true>(dtype) : held == 16 ? spec::probs_kernel<16, true>(dtype)
             : held == 32 ? spec::probs_kernel<32, true>(dtype) : spec::probs_kernel<64, true>(dtype))
          : (held == 8 ? spec::probs_kernel<8, false>(dtype) : held == 16 ? spec::probs_kernel<16, false>(dtype)
             : held == 32 ? spec::probs_kernel<32, false>(dtype) : spec::probs_kernel<64, false>(dtype));
  const int smem = vec ? spec::kThreads * held * size : 0;
  int clusters = 0;
  cudaError_t e = spec::resident_clusters(k, ctas, smem, &clusters);
  if (e != cudaSuccess) return record_cuda_error(e, "spec_probs");
  const int grid = rows < clusters ? rows : clusters;
  e = spec::launch<spec::ProbsParams>(k, (long long)grid * ctas, spec::kThreads, ctas, smem, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "spec_probs");
}

extern "C" size_t spec_workspace_bytes(int seqs, int vocab) {
  if (seqs < 1 || seqs > spec::kMaxSeqs || vocab < 1 || vocab > spec::kMaxVocab) return 0;
  return kWsHeaderBytes + spec::kCounterBytes + spec::most_places(seqs, vocab, device_sm_count()) * spec::kVWarps * sizeof(long long);
}

extern "C" int spec_verify(const void* p, long long p_stride, const void* q, long long q_stride, const int32_t* tokens, const int32_t* row0,
                           int seqs, int rows, int vocab, const float* accept, const float* sample, int32_t* next, int32_t* take, int dtype,
                           void* ws, size_t ws_bytes, void* stream) {
  if (seqs < 1 || seqs > spec::kMaxSeqs || rows < 0 || rows > (1 << 22) || vocab < 1 || vocab > spec::kMaxVocab ||
      (dtype != KV8_BF16 && dtype != KV8_F16 && dtype != SPEC_F32) || !row0 || !take)
    return W8A8_ERR_INVALID_ARG;
  const int size = spec::size_of(dtype);
  int rc;
  if (rows > 0) {   // (without rows every sequence's take is 0: an empty tensor has no address)
    if ((rc = spec::check_rows(p, p_stride, rows, vocab, size)) != W8A8_OK) return rc;
    if (q && (rc = spec::check_rows(q, q_stride, rows, vocab, size)) != W8A8_OK) return rc;
    if (!tokens || !accept || !sample || !next) return W8A8_ERR_INVALID_ARG;
  }
  const void* const words[] = {tokens, row0, accept, sample, next, take};
  for (const void* w : words)
    if (!kv8_aligned(w, 4)) return W8A8_ERR_MISALIGNED;
  if ((rc = kv8_check_ws(ws, ws_bytes, spec_workspace_bytes(seqs, vocab))) != W8A8_OK) return rc;
  const int ctas = spec::verify_ctas(seqs, vocab, device_sm_count());
  const int segments = ctas * spec::kVWarps;
  uint8_t* const w = static_cast<uint8_t*>(ws);
  spec::VerifyParams a{};
  a.p = p, a.q = q, a.p_stride = p_stride, a.q_stride = q_stride;
  a.tokens = tokens, a.row0 = row0, a.accept = accept, a.sample = sample, a.next = next, a.take = take;
  a.rows = rows, a.vocab = vocab, a.ctas = ctas;
  a.segment = ((vocab + segments - 1) / segments + 127) / 128 * 128;
  a.status = reinterpret_cast<uint32_t*>(w);
  a.counters = reinterpret_cast<uint32_t*>(w + kWsHeaderBytes);
  a.sums = reinterpret_cast<long long*>(w + kWsHeaderBytes + spec::kCounterBytes);
  const bool vec = spec::vectors(p, p_stride, size) && (!q || spec::vectors(q, q_stride, size));
  const cudaError_t e = spec::launch<spec::VerifyParams>(vec ? spec::verify_kernel<true>(dtype) : spec::verify_kernel<false>(dtype),
                                                         (long long)seqs * ctas, spec::kVThreads, 0, 0, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "spec_verify");
}
