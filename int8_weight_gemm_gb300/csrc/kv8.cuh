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

// Norm and rotation of one head.  Every lane of the warp takes part (the shuffles are warp-wide, xor or within
// a group).  The products and sums of the rotation are rounded one by one, in the order of its formula
// (a c - b s, b c + a s), so a value does not depend on how the compiler contracts them.
template <int kLanes, bool kPaired>
__device__ __forceinline__ void norm_turn(float (&x)[8], const float* gamma8, float eps, const Turn<kPaired>& t, int l, int rot,
                                          bool interleaved) {
  if (gamma8) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float rs = __fdiv_rn(1.0f, __fsqrt_rn(ss * (1.0f / (8 * kLanes)) + eps));
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * gamma8[i];
  }
  if (rot == 0) return;
  if (kPaired) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[i], b = x[i + 4];
      x[i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
      x[i + 4] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
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
