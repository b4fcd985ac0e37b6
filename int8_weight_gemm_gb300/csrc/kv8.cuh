// Device pieces shared by the 8-bit key-value cache kernels: 16-bit vectors, the rotation of one
// head's values, and the checks of a step's device-side indices.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "../../include/w8a8.h"
#include "common.cuh"
#include "kv8.h"

namespace w8a8 {

// Eight 16-bit values of a 16-byte vector as floats (exact), and back (round to nearest even).
template <bool kF16>
__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kF16) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (kF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kF16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<kF16>(f[0], f[1]), pack2<kF16>(f[2], f[3]), pack2<kF16>(f[4], f[5]), pack2<kF16>(f[6], f[7]));
}

// Two fp32 operations in one instruction (each rounded as the scalar one).
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// A head is held by a group of kLanes = head_dim / 8 lanes, eight values a lane.  kPaired (the whole head
// rotates, pairs half a head apart): lane l holds values 4 l ... 4 l + 3 of either half, so that both values
// of a pair are its own and no lane needs another's, and a position's cosines and sines are read once.
// Otherwise it holds values 8 l ... 8 l + 7.
template <int kLanes, bool kPaired>
__device__ __forceinline__ uint4 load_head(const uint16_t* head, int l) {
  if (!kPaired) return *reinterpret_cast<const uint4*>(head + 8 * l);
  const uint2 a = *reinterpret_cast<const uint2*>(head + 4 * l), b = *reinterpret_cast<const uint2*>(head + 4 * (kLanes + l));
  return make_uint4(a.x, a.y, b.x, b.y);
}
template <int kLanes, bool kPaired>
__device__ __forceinline__ void store_head(uint16_t* head, int l, const uint4 v) {
  if (!kPaired) {
    *reinterpret_cast<uint4*>(head + 8 * l) = v;
  } else {
    *reinterpret_cast<uint2*>(head + 4 * l) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(head + 4 * (kLanes + l)) = make_uint2(v.z, v.w);
  }
}
// The same of a head's bytes in the cache.
template <int kLanes, bool kPaired>
__device__ __forceinline__ uint2 load_bytes(const uint8_t* head, int l) {
  if (!kPaired) return *reinterpret_cast<const uint2*>(head + 8 * l);
  return make_uint2(*reinterpret_cast<const uint32_t*>(head + 4 * l), *reinterpret_cast<const uint32_t*>(head + 4 * (kLanes + l)));
}
template <int kLanes, bool kPaired>
__device__ __forceinline__ void store_bytes(uint8_t* head, int l, const uint2 v) {
  if (!kPaired) {
    *reinterpret_cast<uint2*>(head + 8 * l) = v;
  } else {
    *reinterpret_cast<uint32_t*>(head + 4 * l) = v.x;
    *reinterpret_cast<uint32_t*>(head + 4 * (kLanes + l)) = v.y;
  }
}

// The cosines and sines of a lane's values at one position (a row of the table: rot / 2 cosines, then rot / 2
// sines): one for each value, or (kPaired) for each pair.  Values at or beyond rot keep c = 1, s = 0.
template <bool kPaired>
struct Turn {
  float c[kPaired ? 4 : 8], s[kPaired ? 4 : 8];
};

template <bool kPaired>
__device__ __forceinline__ void load_turn(const float* row, int l, int rot, bool interleaved, Turn<kPaired>& t) {
  const int half = rot >> 1;
  if (kPaired) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + 4 * l)), s = __ldg(reinterpret_cast<const float4*>(row + half + 4 * l));
    t.c[0] = c.x, t.c[1] = c.y, t.c[2] = c.z, t.c[3] = c.w;
    t.s[0] = s.x, t.s[1] = s.y, t.s[2] = s.z, t.s[3] = s.w;
    return;
  }
  constexpr int N = kPaired ? 4 : 8;
  const int e = 8 * l;
  if (e >= rot) {
#pragma unroll
    for (int i = 0; i < N; ++i) t.c[i] = 1.f, t.s[i] = 0.f;
    return;
  }
  if (interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4*>(row + (e >> 1)));
    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + (e >> 1)));
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int i = 0; i < N; ++i) t.c[i] = cc[i >> 1], t.s[i] = ss[i >> 1];
  } else {
    const float* p = row + (e < half ? e : e - half);
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(p + i));
      const float4 s = __ldg(reinterpret_cast<const float4*>(p + half + i));
      t.c[i] = c.x, t.c[i + 1] = c.y, t.c[i + 2] = c.z, t.c[i + 3] = c.w;
      t.s[i] = s.x, t.s[i + 1] = s.y, t.s[i + 2] = s.z, t.s[i + 3] = s.w;
    }
  }
}

// rs[i] = 1 / sqrt(mean of the i-th of four heads' squares + eps).  Each lane brings its share of all four; the first
// two exchanges leave a lane with one head's sum, so the four cost little more than one, root included.  Every lane
// of the warp takes part.
template <int kLanes>
__device__ __forceinline__ void norms_of(const float (&x)[4][8], float eps, float (&rs)[4]) {
  float ss[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint64_t t = mul2(pair(x[h][0], x[h][1]), pair(x[h][0], x[h][1]));
#pragma unroll
    for (int i = 2; i < 8; i += 2) t = fma2(pair(x[h][i], x[h][i + 1]), pair(x[h][i], x[h][i + 1]), t);
    float lo, hi;
    unpair(t, lo, hi);
    ss[h] = lo + hi;
  }
  const int lane = threadIdx.x & 31;
  const bool b0 = lane & (kLanes / 2), b1 = lane & (kLanes / 4);
  float u = b0 ? ss[2] : ss[0], v = b0 ? ss[3] : ss[1];
  u += __shfl_xor_sync(0xffffffffu, b0 ? ss[0] : ss[2], kLanes / 2);
  v += __shfl_xor_sync(0xffffffffu, b0 ? ss[1] : ss[3], kLanes / 2);
  float s = b1 ? v : u;
  s += __shfl_xor_sync(0xffffffffu, b1 ? u : v, kLanes / 4);
#pragma unroll
  for (int o = kLanes / 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const float r = __frsqrt_rn(s * (1.0f / (8 * kLanes)) + eps);   // of head 2 b0 + b1
  const int base = lane & ~(kLanes - 1);
#pragma unroll
  for (int h = 0; h < 4; ++h) rs[h] = __shfl_sync(0xffffffffu, r, base + (h >> 1) * (kLanes / 2) + (h & 1) * (kLanes / 4));
}

// The norm's factors, then the rotation, of one head.  Every lane of the warp takes part (the shuffles are
// warp-wide).  The products and sums of the rotation are rounded one by one, in the order of its formula
// (a c - b s, b c + a s), so a value does not depend on how the compiler contracts them.
template <bool kPaired>
__device__ __forceinline__ void norm_turn(float (&x)[8], bool norm, float rs, const float (&gamma8)[8], const Turn<kPaired>& t, int l,
                                          int rot, bool interleaved) {
  if (norm) {
    const uint64_t r2 = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      unpair(mul2(mul2(pair(x[i], x[i + 1]), r2), pair(gamma8[i], gamma8[i + 1])), x[i], x[i + 1]);
  }
  if (rot == 0) return;
  if (kPaired) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t a = pair(x[i], x[i + 1]), b = pair(x[i + 4], x[i + 5]);
      const uint64_t c = pair(t.c[i], t.c[i + 1]), s = pair(t.s[i], t.s[i + 1]), n = pair(-t.s[i], -t.s[i + 1]);
      unpair(add2(mul2(a, c), mul2(b, n)), x[i], x[i + 1]);
      unpair(add2(mul2(b, c), mul2(a, s)), x[i + 4], x[i + 5]);
    }
    return;
  }
  constexpr int kMask = kPaired ? 3 : 7;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float a = x[i], b = x[i + 1];
      const float y = __fsub_rn(__fmul_rn(a, t.c[i & kMask]), __fmul_rn(b, t.s[i & kMask]));
      const float z = __fadd_rn(__fmul_rn(b, t.c[i & kMask]), __fmul_rn(a, t.s[i & kMask]));
      if (8 * l < rot) x[i] = y, x[i + 1] = z;
    }
  } else {
    // The other value of a pair is rot / 2 values, rot / 16 lanes, away.
    const int step = rot >> 4;
    const bool first = l < step, in = 8 * l < rot;
    const int src = (threadIdx.x & 31) + (in ? (first ? step : -step) : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, x[i], src);
      const float xc = __fmul_rn(x[i], t.c[i & kMask]), os = __fmul_rn(other, t.s[i & kMask]);
      if (in) x[i] = first ? __fsub_rn(xc, os) : __fadd_rn(xc, os);
    }
  }
}

// One sequence of a step, after the checks that keep every later index in bounds.
struct Seq {
  int row0, n, len;   // first row, rows, cached tokens after the step
};

// Reads sequence b.  `max_new`: the step's bound on a sequence's rows.  Returns false (and records
// W8A8_DEV_BAD_INDEX) where the indices make no sense: such a sequence is left out.  `within`: its
// rows have to fit its cached tokens.
__device__ __forceinline__ bool load_seq(const Kv8Step& st, int b, int page_tokens, bool within, uint32_t* status, Seq& s) {
  const int r0 = __ldg(st.row0 + b), r1 = __ldg(st.row0 + b + 1);
  s.row0 = r0;
  s.n = r1 - r0;
  s.len = __ldg(st.kv_len + b);
  const bool ok = r0 >= 0 && r1 >= r0 && r1 <= st.tokens && s.n <= st.max_tokens && s.len >= 0 &&
                  (long long)s.len <= (long long)st.table_width * page_tokens && (!within || s.n <= s.len);
  if (!ok) {
    atomicOr(status, W8A8_DEV_BAD_INDEX);
    s.n = 0;
    s.len = 0;
  }
  return ok;
}

}  // namespace w8a8
