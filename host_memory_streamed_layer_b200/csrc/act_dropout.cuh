// Device helpers shared by the layer-norm, dropout and fused linear kernels:
// eight-element row pieces of fp32 or bf16 rows, the activations and their
// derivatives, and the counter-based dropout mask.
#pragma once

#include <math.h>

#include "mt_common.cuh"
#include "mt_internal.h"
#include "mt_kernels.h"

namespace mt {

typedef __nv_bfloat16 bf16;

constexpr int kMaxDevices = 64;  // of what a launcher keeps per device

// ---------------------------------------------------------------------------
// Eight consecutive elements of a row, as fp32. The row pieces start on
// 16-byte boundaries (row bases and pitches do); a piece cut short by the
// row's end is read and written element by element, so that nothing behind
// the last column is touched.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y), c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
  v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  v[4] = c.x, v[5] = c.y, v[6] = d.x, v[7] = d.y;
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8]) { unpack8(*reinterpret_cast<const uint4*>(p), v); }
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float (&v)[8]) { *reinterpret_cast<uint4*>(p) = pack8(v); }
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(bf16* p, float x) { *p = __float2bfloat16_rn(x); }

// The first n elements at p (all W where n >= W); zeros behind them.
template <int W, typename T>
__device__ __forceinline__ void load_n(const T* p, int n, float (&v)[W]) {
  static_assert(W == 8 || (W == 4 && (sizeof(T) == 4 || sizeof(T) == 2)), "whole vectors");
  if (n >= W) {
    if constexpr (W == 8) {
      load8(p, v);
    } else if constexpr (sizeof(T) == 4) {
      const float4 a = *reinterpret_cast<const float4*>(p);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
      v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e) v[e] = e < n ? to_float(p[e]) : 0.f;
  }
}
template <int W, typename T>
__device__ __forceinline__ void store_n(T* p, int n, const float (&v)[W]) {
  if (n >= W) {
    if constexpr (W == 8) {
      store8(p, v);
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (e < n) put(p + e, v[e]);
  }
}

// ---------------------------------------------------------------------------
// Activations, in fp32. With Phi the logistic function or the normal
// distribution function, each is z Phi and its slope Phi + z Phi'.
// GELU's tanh form is written through the logistic function,
// (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), which keeps its lower tail exact.
// ReLU passes NaN on; its slope at 0 is 0.
// ---------------------------------------------------------------------------
// 2^x and 1/x to about one unit in the last place, subnormal results flushed
// (one instruction each; the denormal handling around them costs three more).
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float logistic(float z) { return rcp_fast(1.f + exp2_fast(z * -1.44269504f)); }

// The normal distribution function and exp(-z^2 / 2), which its density and
// its own approximation share. The lower tail is Phi(-a) = exp(-a^2 / 2) R(a), and
// R, which falls like 1 / (a sqrt(2 pi)), is a polynomial in t = 1 / (1 + 0.27 a)
// without a constant term, fitted over 0 <= a <= 15 for the least relative error,
// 3.5e-8. So the tail keeps its digits (a polynomial fitted for the least absolute
// error loses them: 2e-3 at z = -5); what is left is the rounding of the
// exponent, (16 + 1.1 z^2) 2^-24 of Phi at most, until exp(-a^2 / 2) leaves the
// normal numbers at a = 13.2. Two numbers at a time, each step of their polynomials
// in one instruction: singly, its nine steps made the backward step of 16384 x
// 5504 x 2048 6 % slower (330 us instead of 312; 309 in pairs).
__device__ __forceinline__ float2 normal_cdf(float2 z, float2& gauss) {
  const float2 den = fma2(both(0.27f), make_float2(fabsf(z.x), fabsf(z.y)), both(1.f));
  const float2 t = make_float2(rcp_fast(den.x), rcp_fast(den.y)), e = mul2(mul2(z, z), both(-0.72134752f));
  gauss = make_float2(exp2_fast(e.x), exp2_fast(e.y));
  float2 poly = both(2.899530903e-02f);
  poly = fma2(t, poly, both(-1.266577542e-01f));
  poly = fma2(t, poly, both(1.701543480e-01f));
  poly = fma2(t, poly, both(-6.964881718e-02f));
  poly = fma2(t, poly, both(1.081413925e-01f));
  poly = fma2(t, poly, both(7.190877199e-02f));
  poly = fma2(t, poly, both(1.018484607e-01f));
  poly = fma2(t, poly, both(1.075372919e-01f));
  poly = fma2(t, poly, both(1.077210084e-01f));
  const float2 q = mul2(mul2(t, gauss), poly);
  return make_float2(z.x < 0.f ? q.x : 1.f - q.x, z.y < 0.f ? q.y : 1.f - q.y);
}

// Value and slope together (they share the transcendentals; what a caller does
// not use is not computed).
template <int ACT>
__device__ __forceinline__ void act_both(float z, float& value, float& slope) {
  static_assert(ACT != MT_ACT_GELU, "two at a time");
  if (ACT == MT_ACT_RELU) {
    value = z < 0.f ? 0.f : z;
    slope = z > 0.f ? 1.f : 0.f;
  } else if (ACT == MT_ACT_GELU_TANH) {
    const float s = logistic(z * (1.59576912f + 0.07135482f * z * z));
    const float w = s * (1.f - s);  // 0 where s has saturated; the polynomial beside it may then be infinite
    value = z * s;
    slope = s + (w > 0.f ? z * w * (1.59576912f + 0.21406446f * z * z) : 0.f);
  } else if (ACT == MT_ACT_SILU) {
    const float s = logistic(z);
    value = z * s;
    slope = s * (1.f + z * (1.f - s));
  } else {
    value = z;
    slope = 1.f;
  }
}
template <int ACT>
__device__ __forceinline__ void act_both(float2 z, float2& value, float2& slope) {
  if constexpr (ACT == MT_ACT_GELU) {
    float2 gauss;
    const float2 c = normal_cdf(z, gauss);
    value = mul2(z, c);
    slope = fma2(mul2(z, gauss), both(0.39894228f), c);
  } else {
    act_both<ACT>(z.x, value.x, slope.x);
    act_both<ACT>(z.y, value.y, slope.y);
  }
}
template <int ACT>
__device__ __forceinline__ float2 act_value(float2 z) {
  float2 v, s;
  act_both<ACT>(z, v, s);
  return v;
}
template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 z) {
  float2 v, s;
  act_both<ACT>(z, v, s);
  return s;
}

// Calls f with the activation as a compile-time constant.
#define MT_WITH_ACT(act, ...)                                   \
  switch (act) {                                                \
    case MT_ACT_RELU: { constexpr int ACT = MT_ACT_RELU; __VA_ARGS__; break; }           \
    case MT_ACT_GELU: { constexpr int ACT = MT_ACT_GELU; __VA_ARGS__; break; }           \
    case MT_ACT_GELU_TANH: { constexpr int ACT = MT_ACT_GELU_TANH; __VA_ARGS__; break; } \
    case MT_ACT_SILU: { constexpr int ACT = MT_ACT_SILU; __VA_ARGS__; break; }           \
    default: { constexpr int ACT = MT_ACT_NONE; __VA_ARGS__; break; }                    \
  }

// ---------------------------------------------------------------------------
// Dropout's mask: Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011). Element (t, j) of a
// matrix takes word j % 4 of the block with counter
// (j / 4, row0 + t, offset low, offset high) and key seed, and is dropped
// where that word is below p * 2^32. The mask depends on nothing but these
// numbers, so every kernel draws it again instead of storing it.
// ---------------------------------------------------------------------------
struct DropDesc {
  uint32_t on;         // 0: no dropout
  uint32_t threshold;  // an element is kept when its word is >= this
  float scale;         // 1 / (1 - p)
  uint32_t row0;
  uint64_t offset;
  const int64_t* offset_dev;  // added to offset when the kernel runs; may be NULL
  // The ten rounds' keys, which depend on the seed alone: as kernel parameters
  // they are constant operands of the rounds, not 20 additions beside them.
  uint32_t key0[10], key1[10];
};

// The offset's halves, which a kernel's threads share.
struct DropKey {
  uint32_t c2, c3;
};
__device__ __forceinline__ DropKey drop_key(const DropDesc& d) {
  const uint64_t off = d.offset + (d.on && d.offset_dev ? (uint64_t)*d.offset_dev : 0ull);
  return DropKey{(uint32_t)off, (uint32_t)(off >> 32)};
}
__device__ __forceinline__ uint4 philox4x32(uint32_t c0, uint32_t c1, const DropDesc& d, const DropKey& k) {
  uint32_t x0 = c0, x1 = c1, x2 = k.c2, x3 = k.c3;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)x0 * 0xD2511F53u, b = (uint64_t)x2 * 0xCD9E8D57u;
    x0 = (uint32_t)(b >> 32) ^ x1 ^ d.key0[i];
    x1 = (uint32_t)b;
    x2 = (uint32_t)(a >> 32) ^ x3 ^ d.key1[i];
    x3 = (uint32_t)a;
  }
  return make_uint4(x0, x1, x2, x3);
}
// v[0..3], columns 4 q .. 4 q + 3 of a row: a dropped element becomes 0
// whatever it held (NaN and infinities too), a kept one is scaled.
__device__ __forceinline__ void drop4(float* v, uint32_t q, uint32_t row, const DropDesc& d, const DropKey& k) {
  const uint4 w = philox4x32(q, row, d, k);
  v[0] = w.x >= d.threshold ? v[0] * d.scale : 0.f;
  v[1] = w.y >= d.threshold ? v[1] * d.scale : 0.f;
  v[2] = w.z >= d.threshold ? v[2] * d.scale : 0.f;
  v[3] = w.w >= d.threshold ? v[3] * d.scale : 0.f;
}

// Host: the kernels' description of a caller's dropout for `rows` rows, or
// MT_ERR_ARG: p outside [0, 1) or NaN, rows outside the counter's 32 bits.
inline int make_drop(const mt_dropout* u, int64_t rows, DropDesc* out) {
  *out = DropDesc{0, 0, 1.f, 0, 0, nullptr, {}, {}};
  if (!u) return MT_OK;
  if (!(u->p >= 0.f) || !(u->p < 1.f)) return MT_ERR_ARG;
  if (u->row0 < 0 || u->row0 > (int64_t(1) << 32) - rows) return MT_ERR_ARG;  // rows <= 2^30: nothing overflows
  if (u->p == 0.f) return MT_OK;
  out->on = 1;
  out->threshold = (uint32_t)llrint((double)u->p * 4294967296.0);
  out->scale = (float)(1.0 / (1.0 - (double)u->p));
  out->row0 = (uint32_t)u->row0;
  out->offset = (uint64_t)u->offset;
  out->offset_dev = u->offset_dev;
  for (uint32_t i = 0; i < 10; ++i) {
    out->key0[i] = (uint32_t)u->seed + i * 0x9E3779B9u;
    out->key1[i] = (uint32_t)((uint64_t)u->seed >> 32) + i * 0xBB67AE85u;
  }
  return MT_OK;
}

// Column sums of partials: out[j] = sum over rows r of part[r * pitch + j] for
// the n columns, in a fixed order; columns from n1 on go to out2. Launched
// behind the kernel that wrote `part` on the same stream.
int launch_column_sums(const float* part, int rows, int64_t pitch, int n, float* out, int n1, float* out2,
                       cudaStream_t st);

}  // namespace mt
