// Device-side reading of X_t for the gradient kernels, from the bf16 stream
// or from its 8-bit checkpoint, and the checkpoint's number format.
//
// A checkpoint holds, for each block of 32 channels of a stream, E4M3 codes q
// and one scale byte s; the value is q * 2^(s - 127).  s is the least one
// >= 1 with |x| <= 448 * 2^(s - 127) for every finite x of the block, so no
// finite value saturates and E4M3's rounding (at most 2^-4 of the value, or
// 2^-10 * 2^(s - 127) where E4M3 is subnormal) is the only one.  The scale is
// a power of two, so the value is exact in bf16 (4 significant bits) and
// feeds the matrix core without another rounding.  Values that are not finite
// become the NaN code and do not move the scale.  Under the largest scale
// byte, 247, codes stop at 240: the next one, 256 * 2^120 = 2^128, is past
// bf16's and fp32's range.
#pragma once

#include "mhc_device.h"

namespace mhc {

constexpr int kCkptMaxScale = 247;

// Bits of |x| for a pair of bf16, with 0 in the place of Inf and NaN: what a
// block's scale is chosen from (bf16 magnitudes order like their bits).
__device__ __forceinline__ uint32_t finite_magnitude(uint32_t w) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  const uint32_t a = lo >= 0x7f80u ? 0u : lo, b = hi >= 0x7f80u ? 0u : hi;
  return a > b ? a : b;
}
// Scale byte from the largest finite magnitude's bits: the exponent field is
// E, 448 = 1.75 * 2^8, and 0x60 are the mantissa bits of 1.75.
__device__ __forceinline__ int ckpt_scale(uint32_t amax) {
  const int s = (int)(amax >> 7) - 8 + ((amax & 0x7fu) > 0x60u ? 1 : 0);
  return s < 1 ? 1 : s;
}
// The same from the largest finite fp32 magnitude's bits.
__device__ __forceinline__ int ckpt_scale32(uint32_t amax) {
  const int s = (int)(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return s < 1 ? 1 : s;
}
// The largest of the four lanes that share a block.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0xB1, 0xF, 0xF, false);  // lane ^ 1
  x = x > y ? x : y;
  y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, 0x4E, 0xF, 0xF, false);  // lane ^ 2
  return x > y ? x : y;
}
__device__ __forceinline__ float ckpt_value(int s) { return __uint_as_float((uint32_t)s << 23); }          // 2^(s-127)
__device__ __forceinline__ float ckpt_inverse(int s) { return __uint_as_float((uint32_t)(254 - s) << 23); }  // 2^(127-s)

// Codes of eight channels under the scale byte s of their block (y is scaled in place).
__device__ __forceinline__ u32x2 held_codes(float (&y)[8], int s) {
  const float f = ckpt_inverse(s);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] *= f;
  if (s == kCkptMaxScale) {
    // 255 * 2^120 would round to 256 * 2^120 = 2^128, Inf in bf16 and fp32.
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (fabsf(y[e]) < 256.0f) y[e] = fminf(fmaxf(y[e], -240.0f), 240.0f);
  }
  u32x2 q;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    // |x| * 2^(127-s) <= 448 by the choice of s: no saturation is needed,
    // and Inf and NaN convert to the NaN code.
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * w], y[4 * w + 1], 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * w + 2], y[4 * w + 3], c, true);
    q[w] = (uint32_t)c;
  }
  return q;
}

// Eight channels of X_t as fp32.  CK: from codes (8 bytes) and a scale byte.
template <bool CK>
struct Held8;

template <>
struct Held8<false> {
  u32x4 v;
  __device__ __forceinline__ void load(const void *x, const uint8_t *, size_t vec, size_t) {
    v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(x) + vec);
  }
  __device__ __forceinline__ void widen(float (&o)[8]) const {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      o[2 * w] = bf16_lo(v[w]);
      o[2 * w + 1] = bf16_hi(v[w]);
    }
  }
};

template <>
struct Held8<true> {
  u32x2 v;
  int s;
  __device__ __forceinline__ void load(const void *x, const uint8_t *scales, size_t vec, size_t block) {
    v = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(x) + vec);
    s = scales[block];
  }
  __device__ __forceinline__ void widen(float (&o)[8]) const {
    const float f = ckpt_value(s);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const f32x2 a = fp8_lo2(v[w]), b = fp8_hi2(v[w]);
      o[4 * w] = a[0] * f;
      o[4 * w + 1] = a[1] * f;
      o[4 * w + 2] = b[0] * f;
      o[4 * w + 3] = b[1] * f;
    }
  }
};

// Eight codes and their scale byte as bf16 (exact, one conversion a pair).
__device__ __forceinline__ u32x4 held_bf16(u32x2 codes, int s) {
  const float f = ckpt_value(s);
  u32x4 o;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    o[2 * w] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)codes[w], f, false));
    o[2 * w + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)codes[w], f, true));
  }
  return o;
}

__device__ __forceinline__ void widen8(u32x4 v, float (&o)[8]) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    o[2 * w] = bf16_lo(v[w]);
    o[2 * w + 1] = bf16_hi(v[w]);
  }
}

}  // namespace mhc
