// Rotation of queries and keys with their norms, and the 8-bit paged key-value cache's append and
// read-back.
//
// Mathematics.
//  * Norm (optional), over one head's D values x: x * gamma / sqrt(mean x^2 + eps), in fp32.
//  * Rotation of the pair (a, b) by the position's angle: (a c - b s, b c + a s), each product and
//    sum rounded to fp32, for the first rot values of a head; pairs (i, i + rot / 2) or (2 i, 2 i + 1).
//  * Cache: one fp32 scale s for each (page, kv head), a byte standing for (byte - 128) * s.  A
//    page's scale is the largest magnitude it has been given over 127: with r tokens already in the
//    page, s = max(|s_old|, amax / 127) for r > 0 and amax / 127 for r = 0; x is held as
//    128 + clamp(round(x / s)).  When s changes, the r earlier tokens are held again at the new scale:
//    128 + round((byte - 128) * s_old / s).  Values are quantised from fp32: nothing is rounded to 16
//    bits on the way.  round = halves away from zero, division IEEE; s = 0 gives bytes 128; a NaN is
//    held as 0 and an infinity as the largest finite value, so no byte or scale of the cache is ever
//    not finite.
//
// What bounds them: single tokens and verify windows move a few hundred KB and are bound by launch
// and memory latency, prompts by HBM (values in, queries and bytes out).  So every kernel is one
// pass: a head is held by D / 8 lanes, 16 bytes a lane and load; the append's CTA holds its page's
// new values of one head in registers between the amax and the quantisation (four tokens a thread),
// so they are read once and the scale is known before the first byte is written.
//
// Measured (GPU time in a captured graph; a call from Python takes 4-5 us more): norms and rotation of 16383 rows of 40
// heads of 128 57.4 us (5.9 TB/s), of 16 rows 2.7; four prompts of 3501-4096 tokens (32 / 8 heads of 128) appended 78.4 us
// (4.4 TB/s), read back 20.5 (4.6), one after the other 97.6; 16 single tokens appended 5.0, their pages read back
// 3.4, one after the other 7.9.
#include <cuda_runtime.h>

#include "internal.h"
#include "kv8.cuh"
#include "kv8.h"

namespace w8a8 {

constexpr float kMaxFinite = 3.4028234e38f;

struct QkParams {
  const uint16_t* q;
  const uint16_t* k;
  uint16_t* q_out;
  uint16_t* k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;
  const uint16_t* gamma_q;
  const uint16_t* gamma_k;
  const float* cos_sin;
  const int* positions;
  float eps;
  int rot, max_pos, interleaved;
  int q_heads, kv_heads, tokens;
  int batches;   // kQkHeads heads a lane group takes one after the other
  uint32_t* status;
};

constexpr int kQkThreads = 256;
constexpr int kQkHeads = 4;   // heads of one row whose loads a lane group has in flight together

// Batches of kQkHeads heads a lane group takes: one where there are few groups (a second one would only add its
// latency), two where there are many, so that a position's rotation is read half as often (16383 rows of 40
// heads: 57.2 us with two, 59.3 with one, 60.3 with four; 16 rows: 2.7 with one, 3.8 with two).
static int batches_of(int heads, int rows) {
  const int chunks = (heads + kQkHeads - 1) / kQkHeads;
  return (long long)chunks * rows > 16384 && chunks > 1 ? 2 : 1;
}

// Whether the table has a row for the position; one that it does not have is recorded.
__device__ __forceinline__ bool in_table(const QkParams& p, int pos) {
  if (pos >= 0 && pos < p.max_pos) return true;
  atomicOr(p.status, W8A8_DEV_BAD_INDEX);
  return false;
}

// Heads h0 ... of one row (of q_heads queries, then kv_heads keys) through norm and rotation; `keep`: the row is written.
// (Its loads do not wait for what decides that, the position.)
template <bool kF16, int kLanes, bool kPaired>
__device__ __forceinline__ void turn_heads(const QkParams& p, int row, bool live, bool keep, int h0, int l, const Turn<kPaired>& t) {
  constexpr int D = 8 * kLanes;
  const int heads = p.q_heads + p.kv_heads;
  for (int b = 0; b < p.batches; ++b, h0 += kQkHeads) {
    uint4 raw[kQkHeads];
#pragma unroll
    for (int i = 0; i < kQkHeads; ++i) {
      const int h = h0 + i;
      raw[i] = make_uint4(0u, 0u, 0u, 0u);
      if (live && h < heads)
        raw[i] = load_head<kLanes, kPaired>(h < p.q_heads ? p.q + row * p.q_stride + h * D : p.k + row * p.k_stride + (h - p.q_heads) * D, l);
    }
    float x[kQkHeads][8], rs[kQkHeads];
#pragma unroll
    for (int i = 0; i < kQkHeads; ++i) unpack8<kF16>(raw[i], x[i]);
    if (p.gamma_q || p.gamma_k) norms_of<kLanes>(x, p.eps, rs);
#pragma unroll
    for (int i = 0; i < kQkHeads; ++i) {
      const int h = h0 + i;
      const bool is_q = h < p.q_heads;
      const uint16_t* gamma = is_q ? p.gamma_q : p.gamma_k;
      float g[8];
      if (gamma) unpack8<kF16>(load_head<kLanes, kPaired>(gamma, l), g);
      norm_turn<kPaired>(x[i], gamma != nullptr, rs[i], g, t, l, p.rot, p.interleaved != 0);
      if (keep && h < heads)
        store_head<kLanes, kPaired>(is_q ? p.q_out + row * p.q_out_stride + h * D : p.k_out + row * p.k_out_stride + (h - p.q_heads) * D,
                                    l, pack8<kF16>(x[i]));
    }
  }
}

template <bool kF16, int kLanes, bool kPaired>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const __grid_constant__ QkParams p) {
  pdl_trigger();
  pdl_wait();
  constexpr int kGroups = kQkThreads / kLanes;
  const int l = threadIdx.x % kLanes;
  const int row = blockIdx.x * kGroups + threadIdx.x / kLanes;
  const bool live = row < p.tokens;
  bool keep = live;
  Turn<kPaired> t;
  if (p.rot > 0) {
    const int pos = live ? __ldg(p.positions + row) : 0;
    const bool in = in_table(p, pos);
    keep = live && in;
    load_turn<kPaired>(p.cos_sin + (size_t)(in ? pos : 0) * p.rot, l, p.rot, p.interleaved != 0, t);
  }
  turn_heads<kF16, kLanes, kPaired>(p, row, live, keep, blockIdx.y * kQkHeads * p.batches, l, t);
}

// ------------------------------------------------------------------------------------------------
struct AppendParams {
  Kv8Step step;
  QkParams qk;           // q, q_out and the rotation; k = the new keys
  const uint16_t* v;
  long long v_stride;
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  int pages, page_tokens;
  int seq_pages;         // pages a sequence can touch
  int page_blocks;       // CTAs of the pages (seqs * seq_pages * kv_heads * 2), those of the queries after them
  int q_chunks;          // CTAs of one group of query rows
};

constexpr int kHeld = 4;   // tokens a thread holds
static_assert(kHeld == 4 && kQkHeads == 4, "norms_of takes four at a time");

// The byte that holds x at scale s.
__device__ __forceinline__ uint32_t hold(float x, float s) {
  if (s == 0.f) return 128u;
  const float q = fminf(fmaxf(roundf(__fdiv_rn(x, s)), -127.f), 127.f);
  return (uint32_t)((int)(x != x ? 0.f : q) + 128);
}

// hold() of eight values.  A division takes a dozen instructions, and its last bit matters only next to a half:
// x * (1 / s) is within 127 (2^-23 + 2^-24) < 3e-5 of the rounded quotient, so where it is further than 1e-4 from
// every half, the nearest whole number is hold()'s (adding 1.5 * 2^23 leaves it in the low bits).  The others
// (about 2 in 10^4), infinities, NaN, and scales whose reciprocal leaves fp32 go the long way.  inv = 1 / s.
__device__ __forceinline__ uint2 hold8(const float (&x)[8], float s, float inv) {
  uint32_t b[8];
  bool sure = s > 1e-37f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float q = __fmul_rn(x[i], inv);
    const float n = __fadd_rn(q, 12582912.f);
    sure = sure && fabsf(__fsub_rn(q, __fsub_rn(n, 12582912.f))) < 0.4999f;
    b[i] = __float_as_uint(n);
  }
  uint32_t w[2];
#pragma unroll
  for (int y = 0; y < 2; ++y)
    w[y] = __byte_perm(__byte_perm(b[4 * y], b[4 * y + 1], 0x0040), __byte_perm(b[4 * y + 2], b[4 * y + 3], 0x0040), 0x5410) ^ 0x80808080u;
  if (!sure) {
    w[0] = w[1] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= hold(x[i], s) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// CTAs of page_tokens * D / 32 threads (at most 32 kLanes).  A page's CTA: the new tokens of one page, one
// kv head, keys or values; thread (group g, lane l) takes a lane's values of the page's slots g + i * groups.  A
// query CTA: one row a lane group.  (Two CTAs of the widest page on an SM, four of half of it: 64 registers.)
template <bool kF16, int kLanes, bool kPaired>
__global__ void __launch_bounds__(32 * kLanes, kLanes == 32 ? 1 : 2) kv8_append_kernel(const __grid_constant__ AppendParams p) {
  pdl_trigger();
  pdl_wait();
  constexpr int D = 8 * kLanes;
  const int groups = blockDim.x / kLanes;
  const int l = threadIdx.x % kLanes, g = threadIdx.x / kLanes;
  const QkParams& c = p.qk;
  __shared__ float red[32];

  if ((int)blockIdx.x >= p.page_blocks) {
    // Queries: norm and rotation at the slots' positions.
    const int qb = blockIdx.x - p.page_blocks;
    const int row = (qb / p.q_chunks) * groups + g;
    const bool live = row < p.step.tokens;
    bool keep = live;
    Turn<kPaired> t;
    if (c.rot > 0) {
      int pos = 0;
      if (live) {
        if (c.positions) {
          pos = __ldg(c.positions + row);
        } else {
          // The row's sequence: the last one that begins at or before it (an empty one owns no row).
          int lo = 0, hi = p.step.seqs;
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(p.step.row0 + mid) <= row) lo = mid;
            else hi = mid;
          }
          pos = __ldg(p.step.kv_len + lo) - (__ldg(p.step.row0 + lo + 1) - row);
        }
      }
      const bool in = in_table(c, pos);
      keep = live && in;
      load_turn<kPaired>(c.cos_sin + (size_t)(in ? pos : 0) * c.rot, l, c.rot, c.interleaved != 0, t);
    }
    QkParams q = c;
    q.kv_heads = 0;   // the keys go into the cache
    turn_heads<kF16, kLanes, kPaired>(q, row, live, keep, (qb % p.q_chunks) * kQkHeads * c.batches, l, t);
    return;
  }

  int id = blockIdx.x;
  const bool is_v = id & 1;
  id >>= 1;
  const int h = id % c.kv_heads;
  id /= c.kv_heads;
  const int b = id / p.seq_pages;
  Seq s;
  if (!load_seq(p.step, b, p.page_tokens, true, c.status, s)) return;
  const int P = p.page_tokens;
  const int first_slot = s.len - s.n;
  const int pg = first_slot / P + id % p.seq_pages;   // page of the sequence
  if (s.n == 0 || pg * P >= s.len) return;
  const int page = __ldg(p.step.page_table + (size_t)b * p.step.table_width + pg);
  if (page < 0 || page >= p.pages) {
    if (threadIdx.x == 0) atomicOr(c.status, W8A8_DEV_BAD_INDEX);
    return;
  }
  const int lo = max(first_slot - pg * P, 0), hi = min(s.len - pg * P, P);   // the page's new slots: [lo, hi)
  const size_t at = (size_t)page * c.kv_heads + h;
  uint8_t* const bytes = (is_v ? p.vc : p.kc) + at * P * D;
  float* const scale = (is_v ? p.vs : p.ks) + at;
  const float old = lo > 0 ? *scale : 0.f;

  const uint16_t* const src = is_v ? p.v : c.k;
  const long long stride = is_v ? p.v_stride : c.k_stride;
  const bool norm = !is_v && c.gamma_k != nullptr;
  const int rot = is_v ? 0 : c.rot;
  float gk[8];
  if (norm) unpack8<kF16>(load_head<kLanes, kPaired>(c.gamma_k, l), gk);
  uint4 raw[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int t = g + i * groups;
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t >= lo && t < hi) raw[i] = load_head<kLanes, kPaired>(src + (s.row0 + pg * P + t - first_slot) * stride + h * D, l);
  }
  float x[kHeld][8], rs[kHeld];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) unpack8<kF16>(raw[i], x[i]);
  if (norm) norms_of<kLanes>(x, c.eps, rs);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int t = g + i * groups;
    const bool mine = t >= lo && t < hi;
    Turn<kPaired> turn;
    bool in = true;
    if (rot > 0) {
      const int pos = !mine ? 0 : c.positions ? __ldg(c.positions + s.row0 + pg * P + t - first_slot) : pg * P + t;
      in = in_table(c, pos);
      load_turn<kPaired>(c.cos_sin + (size_t)(in ? pos : 0) * rot, l, rot, c.interleaved != 0, turn);
    }
    norm_turn<kPaired>(x[i], norm, rs[i], gk, turn, l, rot, c.interleaved != 0);
    if (__builtin_expect(!in, 0)) {   // a key without a rotation is held as zeros: its slot will be read
      asm volatile("" ::: "memory");  // (a branch, not a selection of every value)
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[i][j]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) amax = fmaxf(amax, red[w]);
  const float fresh = __fdiv_rn(fminf(amax, kMaxFinite), 127.0f);
  const float now = fmaxf(fabsf(old), fresh);
  const bool again = lo > 0 && now != old;   // the earlier tokens are held at a new scale (of the other sign: byte 0 as 255)
  if (threadIdx.x == 0) *scale = now;
  const float inv = __fdiv_rn(1.0f, now);
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int t = g + i * groups;
    uint8_t* const dst = bytes + (size_t)t * D;
    if (t >= lo && t < hi) {
      store_bytes<kLanes, kPaired>(dst, l, hold8(x[i], now, inv));
    } else if (again && t < lo) {
      const uint2 was = load_bytes<kLanes, kPaired>(dst, l);
      const uint32_t u[2] = {was.x, was.y};
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = fminf(__fmul_rn((float)((int)((u[j >> 2] >> (8 * (j & 3))) & 0xFFu) - 128), old), __fmul_rn(127.f, now));
      store_bytes<kLanes, kPaired>(dst, l, hold8(v, now, inv));
    }
  }
}

// ------------------------------------------------------------------------------------------------
struct ReadParams {
  Kv8Step step;
  const uint8_t* kc;
  const uint8_t* vc;
  const float* ks;
  const float* vs;
  uint16_t* k_out;
  uint16_t* v_out;
  long long k_stride, v_stride;
  int pages, page_tokens, kv_heads, seq_pages;
  uint32_t* status;
};

// One CTA of page_tokens * D / 32 threads for a page's tokens of one kv head, keys or values.
template <bool kF16, int kLanes>
__global__ void __launch_bounds__(32 * kLanes) kv8_read_kernel(const __grid_constant__ ReadParams p) {
  pdl_trigger();
  pdl_wait();
  constexpr int D = 8 * kLanes;
  const int groups = blockDim.x / kLanes;
  const int l = threadIdx.x % kLanes, g = threadIdx.x / kLanes;
  int id = blockIdx.x;
  const bool is_v = id & 1;
  id >>= 1;
  const int h = id % p.kv_heads;
  id /= p.kv_heads;
  const int b = id / p.seq_pages;
  Seq s;
  if (!load_seq(p.step, b, p.page_tokens, true, p.status, s)) return;
  const int P = p.page_tokens;
  const int first_slot = s.len - s.n;
  const int pg = first_slot / P + id % p.seq_pages;
  if (s.n == 0 || pg * P >= s.len) return;
  const int page = __ldg(p.step.page_table + (size_t)b * p.step.table_width + pg);
  if (page < 0 || page >= p.pages) {
    if (threadIdx.x == 0) atomicOr(p.status, W8A8_DEV_BAD_INDEX);
    return;
  }
  const int lo = max(first_slot - pg * P, 0), hi = min(s.len - pg * P, P);
  const size_t at = (size_t)page * p.kv_heads + h;
  const uint8_t* const bytes = (is_v ? p.vc : p.kc) + at * P * D;
  const float scale = (is_v ? p.vs : p.ks)[at];
  uint16_t* const out = is_v ? p.v_out : p.k_out;
  const long long stride = is_v ? p.v_stride : p.k_stride;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int t = g + i * groups;
    if (t < lo || t >= hi) continue;
    const uint2 u = *reinterpret_cast<const uint2*>(bytes + (size_t)t * D + 8 * l);
    const uint32_t w[2] = {u.x, u.y};
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = (float)((int)((w[j >> 2] >> (8 * (j & 3))) & 0xFFu) - 128) * scale;
    const long long row = s.row0 + pg * P + t - first_slot;
    *reinterpret_cast<uint4*>(out + row * stride + h * D + 8 * l) = pack8<kF16>(f);
  }
}

// ------------------------------------------------------------------------------------------------ host
int kv8_check_dims(int kv_heads, int head_dim) {
  if (kv_heads < 1 || kv_heads > 1024) return W8A8_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return W8A8_ERR_UNSUPPORTED_SHAPE;
  return W8A8_OK;
}

int kv8_check_cache(const kv8_cache_t* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || c->pages < 1) return W8A8_ERR_INVALID_ARG;
  const int rc = kv8_check_dims(c->kv_heads, c->head_dim);
  if (rc != W8A8_OK) return rc;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return W8A8_ERR_UNSUPPORTED_SHAPE;
  // The cache's rows (page, head, token) are numbered in 31 bits; bytes and pages are not.
  if ((long long)c->pages * c->kv_heads * c->page_tokens > 0x7fffffffll) return W8A8_ERR_INVALID_ARG;
  if (!kv8_aligned(c->k, 16) || !kv8_aligned(c->v, 16) || !kv8_aligned(c->k_scale, 4) || !kv8_aligned(c->v_scale, 4))
    return W8A8_ERR_MISALIGNED;
  return W8A8_OK;
}

int kv8_check_step(const kv8_step_t* s, const kv8_cache_t* c) {
  if (!s || !s->row0 || !s->kv_len || !s->page_table) return W8A8_ERR_INVALID_ARG;
  if (s->seqs < 1 || s->seqs > 65535 || s->tokens < 0 || s->tokens > (1 << 22) || s->max_tokens < 1 ||
      s->max_tokens > (1 << 22) || s->table_width < 1)
    return W8A8_ERR_INVALID_ARG;
  if ((long long)s->table_width * c->page_tokens > (1ll << 30)) return W8A8_ERR_INVALID_ARG;
  if (!kv8_aligned(s->row0, 4) || !kv8_aligned(s->kv_len, 4) || !kv8_aligned(s->page_table, 4)) return W8A8_ERR_MISALIGNED;
  return W8A8_OK;
}

int kv8_check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return W8A8_ERR_INVALID_ARG;
  if (!kv8_aligned(ws, 256)) return W8A8_ERR_MISALIGNED;
  return ws_bytes < need ? W8A8_ERR_WORKSPACE_TOO_SMALL : W8A8_OK;
}

int kv8_check_prep(const qk_prep_t* p, int head_dim) {
  if (!p) return W8A8_OK;
  if ((p->gamma_q || p->gamma_k) && (!(p->eps >= 0.f) || !(p->eps <= 3.0e38f))) return W8A8_ERR_INVALID_ARG;
  if (p->rot_dim < 0 || p->rot_dim > head_dim) return W8A8_ERR_INVALID_ARG;
  if (p->rot_dim % 16 != 0) return W8A8_ERR_UNSUPPORTED_SHAPE;
  if (p->rot_dim > 0 && (!p->cos_sin || p->max_pos < 1)) return W8A8_ERR_INVALID_ARG;
  if (!kv8_aligned(p->gamma_q, 16) || !kv8_aligned(p->gamma_k, 16) || !kv8_aligned(p->cos_sin, 16))
    return W8A8_ERR_MISALIGNED;
  return W8A8_OK;
}

static void set_prep(QkParams& c, const qk_prep_t* p, const int32_t* positions) {
  if (!p) return;
  c.gamma_q = static_cast<const uint16_t*>(p->gamma_q);
  c.gamma_k = static_cast<const uint16_t*>(p->gamma_k);
  c.cos_sin = p->cos_sin;
  c.positions = positions;
  c.eps = p->eps;
  c.rot = p->rot_dim;
  c.max_pos = p->max_pos;
  c.interleaved = p->interleaved;
}

// Launch as a programmatic dependent of the work before it on the stream (each kernel here waits
// for that work before it touches memory).
template <typename P>
static cudaError_t launch(void (*kernel)(const P), dim3 grid, int threads, const P& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename P>
using Kernel = void (*)(const P);

// The instance for a type and a head size; ...: further template arguments.
#define KV8_PICK(name, P, f16, dim, ...)                                                                                  \
  ((dim) == 64 ? ((f16) ? (Kernel<P>)name<true, 8, ##__VA_ARGS__> : (Kernel<P>)name<false, 8, ##__VA_ARGS__>)              \
   : (dim) == 128 ? ((f16) ? (Kernel<P>)name<true, 16, ##__VA_ARGS__> : (Kernel<P>)name<false, 16, ##__VA_ARGS__>)         \
                  : ((f16) ? (Kernel<P>)name<true, 32, ##__VA_ARGS__> : (Kernel<P>)name<false, 32, ##__VA_ARGS__>))

// Whether a lane can hold whole pairs (load_head).
static bool paired(const QkParams& c, int head_dim) { return c.rot == head_dim && !c.interleaved; }

}  // namespace w8a8

using namespace w8a8;

extern "C" int qk_norm_rope(const qk_prep_t* prep, const void* q, long long q_stride, int q_heads, const void* k,
                            long long k_stride, int kv_heads, int head_dim, const int32_t* positions, int tokens,
                            void* q_out, long long q_out_stride, void* k_out, long long k_out_stride, int dtype, void* ws,
                            size_t ws_bytes, void* stream) {
  if (!prep || q_heads < 0 || q_heads > 4096 || kv_heads < 0 || kv_heads > 1024 || q_heads + kv_heads < 1 ||
      tokens < 0 || tokens > (1 << 22) || (dtype != KV8_BF16 && dtype != KV8_F16))
    return W8A8_ERR_INVALID_ARG;
  int rc = kv8_check_dims(kv_heads > 0 ? kv_heads : 1, head_dim);
  if (rc == W8A8_OK) rc = kv8_check_prep(prep, head_dim);
  if (rc != W8A8_OK) return rc;
  if (tokens == 0) return W8A8_OK;   // an empty tensor has no address
  if (prep->rot_dim > 0 && !positions) return W8A8_ERR_INVALID_ARG;
  if (!kv8_aligned(positions, 4)) return W8A8_ERR_MISALIGNED;
  if (q_heads > 0 && (rc = kv8_check_rows(q, q_stride, q_heads, head_dim)) != W8A8_OK) return rc;
  if (q_heads > 0 && (rc = kv8_check_rows(q_out, q_out_stride, q_heads, head_dim)) != W8A8_OK) return rc;
  if (kv_heads > 0 && (rc = kv8_check_rows(k, k_stride, kv_heads, head_dim)) != W8A8_OK) return rc;
  if (kv_heads > 0 && (rc = kv8_check_rows(k_out, k_out_stride, kv_heads, head_dim)) != W8A8_OK) return rc;
  if ((rc = kv8_check_ws(ws, ws_bytes, kWsHeaderBytes)) != W8A8_OK) return rc;
  QkParams c{};
  set_prep(c, prep, positions);
  c.q = static_cast<const uint16_t*>(q);
  c.k = static_cast<const uint16_t*>(k);
  c.q_out = static_cast<uint16_t*>(q_out);
  c.k_out = static_cast<uint16_t*>(k_out);
  c.q_stride = q_stride, c.k_stride = k_stride, c.q_out_stride = q_out_stride, c.k_out_stride = k_out_stride;
  c.q_heads = q_heads, c.kv_heads = kv_heads, c.tokens = tokens;
  c.status = static_cast<uint32_t*>(ws);
  const int groups = kQkThreads / (head_dim / 8);
  c.batches = batches_of(q_heads + kv_heads, tokens);
  const int chunk = kQkHeads * c.batches;
  const dim3 grid((unsigned)((tokens + groups - 1) / groups), (unsigned)((q_heads + kv_heads + chunk - 1) / chunk));
  const bool f16 = dtype == KV8_F16;
  const cudaError_t e = launch<QkParams>(paired(c, head_dim) ? KV8_PICK(qk_norm_rope_kernel, QkParams, f16, head_dim, true)
                                                             : KV8_PICK(qk_norm_rope_kernel, QkParams, f16, head_dim, false),
                                         grid, kQkThreads, c, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "qk_norm_rope");
}

extern "C" int kv8_append(const kv8_cache_t* cache, const kv8_step_t* step, const qk_prep_t* prep, const void* k,
                          long long k_stride, const void* v, long long v_stride, const void* q, long long q_stride, int q_heads,
                          void* q_out, long long q_out_stride, const int32_t* positions, int dtype, void* ws, size_t ws_bytes,
                          void* stream) {
  int rc = kv8_check_cache(cache);
  if (rc == W8A8_OK) rc = kv8_check_step(step, cache);
  if (rc == W8A8_OK) rc = kv8_check_prep(prep, cache->head_dim);
  if (rc != W8A8_OK) return rc;
  if ((dtype != KV8_BF16 && dtype != KV8_F16) || q_heads < 0 || q_heads > 4096) return W8A8_ERR_INVALID_ARG;
  if (step->tokens == 0) return W8A8_OK;   // an empty tensor has no address
  const int D = cache->head_dim;
  if ((rc = kv8_check_rows(k, k_stride, cache->kv_heads, D)) != W8A8_OK) return rc;
  if ((rc = kv8_check_rows(v, v_stride, cache->kv_heads, D)) != W8A8_OK) return rc;
  if (q_heads > 0 && (rc = kv8_check_rows(q, q_stride, q_heads, D)) != W8A8_OK) return rc;
  if (q_heads > 0 && (rc = kv8_check_rows(q_out, q_out_stride, q_heads, D)) != W8A8_OK) return rc;
  if (!kv8_aligned(positions, 4)) return W8A8_ERR_MISALIGNED;
  if ((rc = kv8_check_ws(ws, ws_bytes, kWsHeaderBytes)) != W8A8_OK) return rc;
  AppendParams p{};
  p.step = kv8_step_of(*step);
  set_prep(p.qk, prep, positions);
  p.qk.k = static_cast<const uint16_t*>(k);
  p.qk.k_stride = k_stride;
  p.qk.q = static_cast<const uint16_t*>(q);
  p.qk.q_stride = q_stride;
  p.qk.q_out = static_cast<uint16_t*>(q_out);
  p.qk.q_out_stride = q_out_stride;
  p.qk.q_heads = q_heads, p.qk.kv_heads = cache->kv_heads, p.qk.tokens = step->tokens;
  p.qk.status = static_cast<uint32_t*>(ws);
  p.v = static_cast<const uint16_t*>(v);
  p.v_stride = v_stride;
  p.kc = static_cast<uint8_t*>(cache->k);
  p.vc = static_cast<uint8_t*>(cache->v);
  p.ks = cache->k_scale;
  p.vs = cache->v_scale;
  p.pages = cache->pages;
  p.page_tokens = cache->page_tokens;
  p.seq_pages = kv8_pages_of(step->max_tokens, cache->page_tokens);
  const long long page_blocks = 2ll * step->seqs * p.seq_pages * cache->kv_heads;
  const int threads = cache->page_tokens * D / 32, groups = threads / (D / 8);
  p.qk.batches = batches_of(q_heads, step->tokens);
  p.q_chunks = (q_heads + kQkHeads * p.qk.batches - 1) / (kQkHeads * p.qk.batches);
  const long long blocks = page_blocks + (long long)p.q_chunks * ((step->tokens + groups - 1) / groups);
  if (blocks > 0x7fffffffll) return W8A8_ERR_INVALID_ARG;
  p.page_blocks = (int)page_blocks;
  const bool f16 = dtype == KV8_F16;
  const cudaError_t e = launch<AppendParams>(paired(p.qk, D) ? KV8_PICK(kv8_append_kernel, AppendParams, f16, D, true)
                                                             : KV8_PICK(kv8_append_kernel, AppendParams, f16, D, false),
                                             dim3((unsigned)blocks), threads, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "kv8_append");
}

extern "C" int kv8_read(const kv8_cache_t* cache, const kv8_step_t* step, void* k_out, long long k_stride, void* v_out,
                        long long v_stride, int dtype, void* ws, size_t ws_bytes, void* stream) {
  int rc = kv8_check_cache(cache);
  if (rc == W8A8_OK) rc = kv8_check_step(step, cache);
  if (rc != W8A8_OK) return rc;
  if (dtype != KV8_BF16 && dtype != KV8_F16) return W8A8_ERR_INVALID_ARG;
  if (step->tokens == 0) return W8A8_OK;
  const int D = cache->head_dim;
  if ((rc = kv8_check_rows(k_out, k_stride, cache->kv_heads, D)) != W8A8_OK) return rc;
  if ((rc = kv8_check_rows(v_out, v_stride, cache->kv_heads, D)) != W8A8_OK) return rc;
  if ((rc = kv8_check_ws(ws, ws_bytes, kWsHeaderBytes)) != W8A8_OK) return rc;
  ReadParams p{};
  p.step = kv8_step_of(*step);
  p.kc = static_cast<const uint8_t*>(cache->k);
  p.vc = static_cast<const uint8_t*>(cache->v);
  p.ks = cache->k_scale;
  p.vs = cache->v_scale;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.k_stride = k_stride, p.v_stride = v_stride;
  p.pages = cache->pages, p.page_tokens = cache->page_tokens, p.kv_heads = cache->kv_heads;
  p.seq_pages = kv8_pages_of(step->max_tokens, cache->page_tokens);
  p.status = static_cast<uint32_t*>(ws);
  const long long blocks = 2ll * step->seqs * p.seq_pages * cache->kv_heads;
  if (blocks > 0x7fffffffll) return W8A8_ERR_INVALID_ARG;
  const cudaError_t e = launch<ReadParams>(KV8_PICK(kv8_read_kernel, ReadParams, dtype == KV8_F16, D), dim3((unsigned)blocks),
                                           cache->page_tokens * D / 32, p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? W8A8_OK : record_cuda_error(e, "kv8_read");
}
