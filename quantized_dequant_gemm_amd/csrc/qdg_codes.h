// Encoders of activation rows: the rules of qdg_quantize_act and
// qdg_quantize_act_zp for the values that one lane holds, shared by the
// quantizers and by the row operators that end in codes (whose codes are
// therefore those of the quantizer over the same bf16 values, bit for bit);
// and the bf16 pairs, unaligned loads and lane exchanges that the row operators
// and the adapters share.
#pragma once
#include "qdg_device.h"

namespace qdg {

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __builtin_bit_cast(float, h << 16); }

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;
// A pair of binary32 values as bf16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t to_bf16_pair(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Sixteen bytes at any bf16 or binary32 element.
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_2_t;
typedef __attribute__((ext_vector_type(4), aligned(4))) uint32_t u32x4_4_t;

// Lane exchanges of DPP within 16 lanes: lanes differing in bit 0, bit 1, a
// mirror of 8 (bit 2, once bits 0 and 1 agree) and of 16 lanes (bit 3).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kMirror8 = 0x141, kMirror16 = 0x140;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32 | dpp<CTRL>((uint32_t)u));
}

// The least of three magnitudes; a NaN among them comes through.
__device__ __forceinline__ float least3(float a, float b, float c) {
  float r;
  asm("v_minimum3_f32 %0, |%1|, |%2|, |%3|" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}

// Value j of a run of bf16 pairs.
__device__ __forceinline__ float bf16_pair(uint32_t pair, int j) {
  return __builtin_bit_cast(float, j & 1 ? pair & 0xFFFF0000u : pair << 16);
}

// ------------------------------------------------------------------ symmetric int8
__device__ __forceinline__ u32x2_t encode_int8x8(const float (&f)[8], float inv) {
  u32x2_t out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float f0 = fminf(fmaxf(rintf(f[2 * i] * inv), -127.f), 127.f);
    const float f1 = fminf(fmaxf(rintf(f[2 * i + 1] * inv), -127.f), 127.f);
    const uint32_t b = ((uint32_t)(int)f0 & 0xFFu) | (((uint32_t)(int)f1 & 0xFFu) << 8);
    if (i & 1) out[i >> 1] |= b << 16;
    else out[i >> 1] = b;
  }
  return out;
}

// ------------------------------------------------------------------ fp8 E4M3
// gfx950's v_cvt_pk_fp8_f32 encodes two binary32 values as OCP E4M3 with
// round to nearest even (subnormal codes included, the sign kept for values
// that round to zero); inputs are clamped to the largest finite magnitude
// first, so no code is NaN.
__device__ __forceinline__ u32x2_t encode_fp8x8(const float (&f)[8], float inv) {
  u32x2_t out;
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = fminf(fmaxf(f[i] * inv, -448.f), 448.f);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * j], t[4 * j + 1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * j + 2], t[4 * j + 3], w, true);
    out[j] = (uint32_t)w;
  }
  return out;
}

// ------------------------------------------------------------------ MXFP4
// The biased exponent of a block whose largest magnitude is amax > 0:
// X + 127 with X = floor(log2(amax)) - 2, read from amax's exponent field (a
// subnormal amax, below 2^-126, gives the clamped X = -127).
__device__ __forceinline__ uint32_t fp4_block_exponent(float amax) {
  const int ef = (int)((__builtin_bit_cast(uint32_t, amax) >> 23) & 0xFFu);
  int X = ef == 0 ? -127 : ef - 127 - 2;
  X = X < -127 ? -127 : X;
  return (uint32_t)(X + 127);
}

// Eight values as E2M1 codes of x / 2^X, a product with the power of two
// 2^-X (X in [-127, 125]): exact for every value whose code is not 0.
// gfx950's v_cvt_scalef32_pk_fp4_f32 encodes two binary32 values with round
// to nearest even and saturation at +-6 (sign kept for values that round to
// zero); element 2j goes into the low nibble of byte j.
__device__ __forceinline__ uint32_t encode_fp4x8(const float (&f)[8], uint32_t e8) {
  const float inv = __builtin_bit_cast(float, (254u - e8) << 23);
  uint32_t out = 0;
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[0] * inv, f[1] * inv, 1.0f, 0);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[2] * inv, f[3] * inv, 1.0f, 1);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[4] * inv, f[5] * inv, 1.0f, 2);
  out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[6] * inv, f[7] * inv, 1.0f, 3);
  return out;
}

// ------------------------------------------------------------------ int8 with a zero point
// Range: a bf16 word as int16 orders the values from 0 up, as uint16 the
// negative ones by magnitude above all others, so hi and lo are packed
// 16-bit maxima; an infinity or a NaN shows as a maximum past the largest
// finite word, and only then the row's values are checked one by one.
// Encoding: y = fma(x, inv32, 1.5 * 2^23) carries rne(x * inv32) in its low
// bits. inv32 is off by 2^-24 of itself and |x * inv| <= 256, so the code is the
// binary64 one unless x * inv32 is within 2^-16 of the middle between two
// integers (kDoubt = 2^-15 is used); a chunk with such a value (or NaN) is encoded again
// in binary64: one chunk of 64 lanes in 16.
constexpr float kDoubt = 0.5f - 0x1p-15f;

__device__ __forceinline__ uint32_t pk_max_i16(uint32_t a, uint32_t b) {
  typedef __attribute__((ext_vector_type(2))) short i16x2_t;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(i16x2_t, a), __builtin_bit_cast(i16x2_t, b)));
}
__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  typedef __attribute__((ext_vector_type(2))) unsigned short u16x2_t;
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}

// The largest finite words of a run of bf16 pairs.
template <int ND>
__device__ __forceinline__ void zp_finite_max(const uint32_t (&w)[ND], uint32_t& hw, uint32_t& lw) {
#pragma unroll
  for (int j = 0; j < 2 * ND; ++j) {
    const uint32_t h = j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
    if ((h & 0x7FFFu) < 0x7F80u) {
      if (h < 0x8000u) hw = max(hw, h);
      lw = max(lw, h);
    }
  }
}

struct ZpRow {
  float scale, inv32;
  double inv, zero;
};

__device__ __forceinline__ ZpRow zp_row(float lo, float hi) {
  const bool any = hi > lo;
  ZpRow z;
  z.scale = any ? fmaxf((float)(((double)hi - (double)lo) / 255.0), 0x1p-126f) : 1.0f;
  z.inv = 1.0 / (double)z.scale;
  z.inv32 = (float)z.inv;
  z.zero = any ? fmin(fmax(rint(-128.0 - (double)lo * z.inv), -128.0), 127.0) : 0.0;
  return z;
}

// The codes of ND bf16 pairs. BRANCH: binary64 behind a branch, one value at a
// time, which takes fewer registers and instructions; else for all values side
// by side and chosen afterwards, which is shorter for a row by itself.
template <int ND, bool BRANCH>
__device__ __forceinline__ void encode_zp(const uint32_t (&v)[ND], const ZpRow& z, uint32_t (&out)[ND / 2]) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  const int shift = (int)z.zero - 0x4B400000;
  bool doubt = false;
  int c[2 * ND];
#pragma unroll
  for (int j = 0; j < 2 * ND; ++j) {
    const float f = bf16_pair(v[j >> 1], j);
    const float y = __builtin_fmaf(f, z.inv32, kMagic);
    doubt |= !(fabsf(__builtin_fmaf(f, z.inv32, kMagic - y)) < kDoubt);
    c[j] = min(max(__builtin_bit_cast(int, y) + shift, -128), 127);
  }
  if (doubt) {
#pragma unroll
    for (int j = 0; j < 2 * ND; ++j) {
      const float f = bf16_pair(v[j >> 1], j);
      const double d = f == f ? rint((double)f * z.inv) : 0.0;
      c[j] = (int)fmin(fmax(d + z.zero, -128.0), 127.0);
      if constexpr (BRANCH) __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int d = 0; d < ND / 2; ++d)
    out[d] = ((uint32_t)c[4 * d] & 0xFFu) | ((uint32_t)c[4 * d + 1] & 0xFFu) << 8 |
             ((uint32_t)c[4 * d + 2] & 0xFFu) << 16 | (uint32_t)c[4 * d + 3] << 24;
}

}  // namespace qdg
