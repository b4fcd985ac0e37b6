// Ends of a speculative decoding step: the probabilities of a vocabulary from its logits (spec_probs), and the
// verification of drafted tokens against them from given random numbers (spec_verify).
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
// What bounds it: HBM, two bytes in and four out for each of a row's values (bf16), some ten instructions beside them.
// A row is held in the registers of a cluster of up to eight CTAs, so it is read once and its exponentials are taken
// once: relative to the CTA's own maximum, then times one factor that follows from all CTAs' maxima and sums, which go
// through distributed shared memory.
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

struct ProbsParams {
  const void* x;
  long long x_stride;
  const float* inv_temp;
  float* out;
  long long out_stride;
  int vocab, share, ctas;   // a CTA's values (a multiple of four), a row's CTAs
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// exp(t) for t <= 0 (a NaN: 0): the product with log2 e in two parts, as its rounding alone would be a relative error of
// 2^-18 at t = -64.
__device__ __forceinline__ float exp_of(float t) {
  t = fmaxf(t, -200.f);
  const float hi = t * 1.44269504f;
  const float lo = fmaf(t, 1.92596299e-8f, fmaf(t, 1.44269504f, -hi));   // 1.92596299e-8 = log2 e - 1.44269504f
  const float y = ex2(hi);
  return fmaf(y, lo * 0.69314718f, y);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_v2f(uint32_t addr, float a, float b) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

// kE: values a thread holds.  kVec: four neighbours at a time (rows and strides aligned for it), else one.
template <int kType, int kE, bool kVec>
__global__ void __launch_bounds__(kThreads, kE <= 32 ? 2 : 1) spec_probs_kernel(const __grid_constant__ ProbsParams p) {
  using Ty = Type<kType>;
  __shared__ float red_sm[2][kWarps];
  __shared__ int best_sm[kWarps];
  __shared__ __align__(8) float2 peers_sm[8];   // (maximum, sum) of each CTA of the row
  __shared__ __align__(8) float2 first_sm[8];   // greedy: index of each CTA's first largest value (as bits)
  const int rank = (int)cluster_ctarank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / p.ctas;
  cluster_arrive();   // the other CTAs' shared memory may be written once they have begun
  pdl_trigger();
  pdl_wait();
  const int begin = rank * p.share, end = min(p.vocab, begin + p.share);
  const typename Ty::T* const src = static_cast<const typename Ty::T*>(p.x) + row * p.x_stride;
  float* const dst = p.out + row * p.out_stride;
  // A thread's values: i-th of v at place begin + first + (i / kN) * kThreads * kN + i % kN.
  constexpr int kN = kVec ? 4 : 1;
  const int left = end - begin - kN * (int)threadIdx.x;   // values from the thread's first on
  const size_t first = (size_t)begin + kN * threadIdx.x;
  auto place = [](int i) { return (i / kN) * kThreads * kN + i % kN; };

  float v[kE];
#pragma unroll
  for (int i = 0; i < kE; i += kN) {
    float f[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    if (kVec && place(i) + kN <= left) {
      Ty::load4(src + first + place(i), f);
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k)
        if (place(i) + k < left) f[k] = Ty::load(src + first + place(i) + k);
    }
#pragma unroll
    for (int k = 0; k < kN; ++k) v[i + k] = f[k];
  }
  const float inv = p.inv_temp ? fmaxf(p.inv_temp[row], 0.f) : 1.f;   // (a NaN: 0)
  const bool greedy = inv == INFINITY;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kE; ++i) m = fmaxf(m, v[i]);   // (a NaN is passed over)
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red_sm[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, red_sm[0][w]);
  float sum = 0.f;
  if (!greedy) {
    // Values of +inf share the row; a CTA without a value above -inf has none.
    const bool top = m == INFINITY;
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < kE; ++i) {
      v[i] = exp_of(top ? (v[i] == INFINITY ? 0.f : -INFINITY) : (v[i] - ref) * inv);
      sum += v[i];
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red_sm[1][warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) sum += red_sm[1][w];
  cluster_wait();
  if ((int)threadIdx.x < p.ctas) st_cluster_v2f(cluster_map(smem_addr(&peers_sm[rank]), threadIdx.x), m, sum);
  cluster_arrive();
  cluster_wait();
  float M = -INFINITY;
  for (int c = 0; c < p.ctas; ++c) M = fmaxf(M, peers_sm[c].x);
  float factor = 0.f;
  int best = p.vocab;
  if (!greedy) {
    auto weight = [&](float x) { return x == M ? 1.f : exp_of((x - M) * inv); };
    float S = 0.f;
    for (int c = 0; c < p.ctas; ++c) S = fmaf(peers_sm[c].y, weight(peers_sm[c].x), S);
    factor = S > 0.f ? __fdiv_rn(weight(m), S) : 0.f;
  } else {
    // The first of the largest values, in the order of the row.
    int at = p.vocab;
    if (M > -INFINITY) {
#pragma unroll
      for (int i = kE - 1; i >= 0; --i)
        if (v[i] == M) at = (int)first + place(i);
    }
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) best_sm[warp] = at;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) best = min(best, best_sm[w]);
    if ((int)threadIdx.x < p.ctas) st_cluster_v2f(cluster_map(smem_addr(&first_sm[rank]), threadIdx.x), __int_as_float(best), 0.f);
    cluster_arrive();
    cluster_wait();
    for (int c = 0; c < p.ctas; ++c) best = min(best, __float_as_int(first_sm[c].x));
  }
#pragma unroll
  for (int i = 0; i < kE; i += kN) {
    const int at = (int)first + place(i);
    float f[4];
#pragma unroll
    for (int k = 0; k < kN; ++k) f[k] = greedy ? (at + k == best ? 1.f : 0.f) : v[i + k] * factor;
    if (kVec && place(i) + kN <= left) {
      *reinterpret_cast<float4*>(dst + first + place(i)) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k)
        if (place(i) + k < left) dst[first + place(i) + k] = f[k];
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
constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kMinSegment = 512;
constexpr int kCtasPerSm = 4;
constexpr float kUnits = 17592186044416.f;   // 2^44

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

__device__ __forceinline__ long long units(float x) { return __float2ll_rn(__saturatef(x) * kUnits); }   // (a NaN: 0)

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

  // The sum of the weights of [a, b) that this lane takes (`target`: of p alone).
  auto weigh = [&](int a, int b, bool target) {
    long long s = 0;
    const bool diff = qrow && !target;
    const int skip = target ? -1 : none;
    if (kVec) {
      int i = a + 4 * lane;
#pragma unroll 4
      for (; i + 4 <= b; i += 128) {
        float f[4], g[4] = {0.f, 0.f, 0.f, 0.f};
        Ty::load4(prow + i, f);
        if (diff) Ty::load4(qrow + i, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const long long w = units(f[k]) - (diff ? units(g[k]) : 0);
          s += i + k == skip ? 0 : max(w, 0ll);
        }
      }
      for (int k = i; k < min(b, i + 4); ++k) {
        const long long w = units(Ty::load(prow + k)) - (diff ? units(Ty::load(qrow + k)) : 0);
        s += k == skip ? 0 : max(w, 0ll);
      }
    } else {
#pragma unroll 8
      for (int i = a + lane; i < b; i += 32) {
        const long long w = units(Ty::load(prow + i)) - (diff ? units(Ty::load(qrow + i)) : 0);
        s += i == skip ? 0 : max(w, 0ll);
      }
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
      const bool diff = qrow && !target;
      const int skip = target ? -1 : none;
      auto weight = [&](int i) {
        const long long w = units(Ty::load(prow + i)) - (diff ? units(Ty::load(qrow + i)) : 0);
        return i == skip ? 0 : max(w, 0ll);
      };
      mine = 0;
      for (int i = i0; i < i1; ++i) mine += weight(i);
      const long long ahead = scan(mine, all);
      at = at_sm;
      if (at >= ahead && at < ahead + mine) {
        at -= ahead;
        int i = i0;
        for (long long x; i + 1 < i1 && at >= (x = weight(i)); ++i) at -= x;
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
static cudaError_t launch(void (*kernel)(const P), long long grid, int threads, int cluster, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
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

constexpr int kMaxVocab = 1 << 18;
constexpr int kMaxSeqs = 65535;
// (For any number of sequences: a workspace may serve calls of different ones, whose counters are zero between calls.)
constexpr size_t kCounterBytes = ((size_t)kMaxSeqs * sizeof(uint32_t) + 255) / 256 * 256;

// A sequence's CTAs: as many as the SMs hold for all sequences together, of segments that are worth a warp.
static int verify_ctas(int seqs, int vocab, int sms) {
  const int most = (vocab + kMinSegment * kVWarps - 1) / (kMinSegment * kVWarps), want = sms * kCtasPerSm / seqs;
  return want < 1 ? 1 : want < most ? want : most;
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
  // A row's CTAs: eight for few rows, so that every SM has some; else as few as hold it at 32 values a thread (64 for a
  // vocabulary that eight would not hold).
  const int sms = device_sm_count();
  const bool wide = vocab > 8 * 32 * spec::kThreads;
  int ctas = (vocab + (wide ? 64 : 32) * spec::kThreads - 1) / ((wide ? 64 : 32) * spec::kThreads);
  while (ctas < 8 && (long long)rows * ctas < 2 * sms) ++ctas;
  spec::ProbsParams p{logits, logits_stride, inv_temp, out, out_stride, vocab, ((vocab + ctas - 1) / ctas + 3) / 4 * 4, ctas};
  const int each = (p.share + spec::kThreads - 1) / spec::kThreads;
  const bool vec = spec::vectors(logits, logits_stride, size) && spec::vectors(out, out_stride, 4);
  spec::Kernel<spec::ProbsParams> k =
      vec ? (each <= 8 ? spec::probs_kernel<8, true>(dtype) : each <= 16 ? spec::probs_kernel<16, true>(dtype)
             : each <= 32 ? spec::probs_kernel<32, true>(dtype) : spec::probs_kernel<64, true>(dtype))
          : (each <= 8 ? spec::probs_kernel<8, false>(dtype) : each <= 16 ? spec::probs_kernel<16, false>(dtype)
             : each <= 32 ? spec::probs_kernel<32, false>(dtype) : spec::probs_kernel<64, false>(dtype));
  const cudaError_t e = spec::launch<spec::ProbsParams>(k, (long long)rows * ctas, spec::kThreads, ctas, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "spec_probs");
}

extern "C" size_t spec_workspace_bytes(int seqs, int vocab) {
  if (seqs < 1 || seqs > spec::kMaxSeqs || vocab < 1 || vocab > spec::kMaxVocab) return 0;
  return kWsHeaderBytes + spec::kCounterBytes + (size_t)seqs * spec::verify_ctas(seqs, vocab, device_sm_count()) * spec::kVWarps * sizeof(long long);
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
                                                         (long long)seqs * ctas, spec::kVThreads, 0, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "spec_verify");
}
