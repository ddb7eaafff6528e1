// Activation quantization for the integer and fp8 paths (bf16 in).
//
// The pages name W8A8 and W4A8 as common configurations (kinachrichten,
// "Warum quantisierte Kernel wichtig sind"; jetabc, section on what
// quantization is) without the activation scheme. Implemented schemes:
//   int8, one fp32 scale per token:   inv = f32(127/amax), q = rne(clamp(x*inv))
//   fp8 E4M3 (OCP), one fp32 scale per token and 128-wide K group:
//                                     inv = f32(448/amax), q = e4m3_rne(clamp(x*inv))
//   MXFP4 (OCP MX), one E8M0 scale per token and 32-wide K block:
//                                     X = floor(log2(amax)) - 2, q = e2m1_rne_sat(x / 2^X)
// Scale = f32(amax/Q); amax = 0 gives scale 1 and zero codes. Every step is
// binary32 with RNE and correctly rounded division, so the codes are
// reproducible bit for bit by any implementation doing the same steps. The
// E4M3 and E2M1 encodes run on gfx950's conversion instructions
// (v_cvt_pk_fp8_f32, v_cvt_scalef32_pk_fp4_f32: round to nearest even, the
// sign kept on zero); the tests compare them with the oracle's encoders over
// every bf16 input magnitude the encodes can see.
#include "qdg_device.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

__device__ __forceinline__ float bf16_to_f32(uint32_t h) { return __builtin_bit_cast(float, h << 16); }


// MXFP4 per (token, 32-block): four lanes per block, 8 values (16 bytes) each;
// the block's amax comes from a 4-lane reduction. X is read from the
// exponent field of amax (a subnormal amax, below 2^-126, gives the clamped
// X = -127), and x / 2^X is a product with the power of two 2^-X, exact for
// every value whose code is not 0.
__global__ __launch_bounds__(256) void act_fp4_kernel(const uint16_t* __restrict__ a, uint8_t* __restrict__ q,
                                                      uint8_t* __restrict__ scales, int64_t blocks) {
  const int64_t gl = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t b = gl >> 2;  // block index: row * (K/32) + j
  const int sub = threadIdx.x & 3;
  if (b >= blocks) return;    // whole 4-lane segments exit together
  const u32x4_t v = *(const u32x4_t*)(a + b * 32 + sub * 8);
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_to_f32(v[j] & 0xFFFFu);
    f[2 * j + 1] = bf16_to_f32(v[j] >> 16);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
  amax = fmaxf(amax, __shfl_xor(amax, 1, 4));
  amax = fmaxf(amax, __shfl_xor(amax, 2, 4));
  uint32_t out = 0, e8 = 0;
  if (amax > 0.f) {
    const int ef = (int)((__builtin_bit_cast(uint32_t, amax) >> 23) & 0xFFu);
    int X = ef == 0 ? -127 : ef - 127 - 2;  // floor(log2(amax)) - 2
    X = X < -127 ? -127 : X;
    e8 = (uint32_t)(X + 127);
    const float inv = __builtin_bit_cast(float, (uint32_t)(127 - X) << 23);  // 2^-X, X in [-127, 125]
    // gfx950's v_cvt_scalef32_pk_fp4_f32 encodes two binary32 values as
    // E2M1 with round to nearest even and saturation at +-6 (sign kept for
    // values that round to zero); with scale 1 it encodes x / 2^X itself,
    // element 2j in the low nibble of byte j
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[0] * inv, f[1] * inv, 1.0f, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[2] * inv, f[3] * inv, 1.0f, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[4] * inv, f[5] * inv, 1.0f, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, f[6] * inv, f[7] * inv, 1.0f, 3);
  }
  *(uint32_t*)(q + b * 16 + sub * 4) = out;
  if (sub == 0) scales[b] = (uint8_t)e8;
}

// int8 per token: one workgroup per row.
__global__ __launch_bounds__(256) void act_int8_kernel(const uint16_t* __restrict__ a, int8_t* __restrict__ q,
                                                       float* __restrict__ scales, int64_t K) {
  const int64_t row = blockIdx.x;
  const uint16_t* x = a + row * K;
  float amax = 0.f;
  for (int64_t k = threadIdx.x * 8; k < K; k += 256 * 8) {
    const u32x4_t v = *(const u32x4_t*)(x + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      amax = fmaxf(amax, fabsf(bf16_to_f32(v[i] & 0xFFFFu)));
      amax = fmaxf(amax, fabsf(bf16_to_f32(v[i] >> 16)));
    }
  }
  for (int off = 32; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off));
  __shared__ float wmax[4];
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = amax;
  __syncthreads();
  amax = fmaxf(fmaxf(wmax[0], wmax[1]), fmaxf(wmax[2], wmax[3]));
  const bool nz = amax > 0.f;
  const float inv = nz ? __fdiv_rn(127.0f, amax) : 0.f;
  if (threadIdx.x == 0) scales[row] = nz ? __fdiv_rn(amax, 127.0f) : 1.0f;
  int8_t* y = q + row * K;
  for (int64_t k = threadIdx.x * 8; k < K; k += 256 * 8) {
    const u32x4_t v = *(const u32x4_t*)(x + k);
    u32x2_t out;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f0 = fminf(fmaxf(rintf(bf16_to_f32(v[i] & 0xFFFFu) * inv), -127.f), 127.f);
      const float f1 = fminf(fmaxf(rintf(bf16_to_f32(v[i] >> 16) * inv), -127.f), 127.f);
      const uint32_t b = ((uint32_t)(int)f0 & 0xFFu) | (((uint32_t)(int)f1 & 0xFFu) << 8);
      if (i & 1) out[i >> 1] |= b << 16;
      else out[i >> 1] = b;
    }
    *(u32x2_t*)(y + k) = out;
  }
}

// fp8 per (token, 128-group): 16 lanes per group, 8 values per lane.
__global__ __launch_bounds__(256) void act_fp8_kernel(const uint16_t* __restrict__ a, uint8_t* __restrict__ q,
                                                      float* __restrict__ scales, int64_t M, int64_t K) {
  const int64_t gid = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> 4;  // (row, group) index
  const int sub = threadIdx.x & 15;
  const int64_t groups = K / 128;
  if (gid >= M * groups) return;  // whole 16-lane segments exit together
  const int64_t row = gid / groups, g = gid % groups;
  const uint16_t* x = a + row * K + g * 128 + sub * 8;
  const u32x4_t v = *(const u32x4_t*)x;
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(v[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(v[i] >> 16);
  }
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
  for (int off = 8; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 16));
  const bool nz = amax > 0.f;
  const float inv = nz ? __fdiv_rn(448.0f, amax) : 0.f;
  if (sub == 0) scales[row * groups + g] = nz ? __fdiv_rn(amax, 448.0f) : 1.0f;
  // gfx950's v_cvt_pk_fp8_f32 encodes two binary32 values as OCP E4M3 with
  // round to nearest even (subnormal codes included, the sign kept for
  // values that round to zero); inputs are clamped to the largest finite
  // magnitude first, so no code is NaN
  u32x2_t out = {0, 0};
  if (nz) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = fminf(fmaxf(f[i] * inv, -448.f), 448.f);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * j], t[4 * j + 1], 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * j + 2], t[4 * j + 3], w, true);
      out[j] = (uint32_t)w;
    }
  }
  *(u32x2_t*)(q + row * K + g * 128 + sub * 8) = out;
}

}  // namespace

namespace {

// int8 activation codes -> two E4M3 planes, q = 16 * hi + lo with
// hi = q >> 4 in [-8, 7] and lo = q & 15 in [0, 15]: one thread per 16 codes.
// Both halves are integers that E4M3 holds exactly (at most 4 significant
// bits), so gfx950's v_cvt_pk_fp8_f32 (OCP E4M3, two values per
// instruction) encodes them without rounding.
__global__ __launch_bounds__(256) void act_i8_planes_kernel(const int8_t* __restrict__ qa, int64_t rows, int64_t K,
                                                          uint8_t* __restrict__ planes) {
  const int64_t q = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;  // 16-code chunk
  const int64_t per_row = K / 16;
  if (q >= rows * per_row) return;
  const int64_t r = q / per_row, k0 = (q % per_row) * 16;
  const u32x4_t v = *(const u32x4_t*)(qa + r * K + k0);
  u32x4_t hi, lo;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    float h[4], l[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int code = (int)(int8_t)(v[d] >> (8 * b));
      h[b] = (float)(code >> 4);
      l[b] = (float)(code & 15);
    }
    int wh = __builtin_amdgcn_cvt_pk_fp8_f32(h[0], h[1], 0, false);
    wh = __builtin_amdgcn_cvt_pk_fp8_f32(h[2], h[3], wh, true);
    int wl = __builtin_amdgcn_cvt_pk_fp8_f32(l[0], l[1], 0, false);
    wl = __builtin_amdgcn_cvt_pk_fp8_f32(l[2], l[3], wl, true);
    hi[d] = (uint32_t)wh;
    lo[d] = (uint32_t)wl;
  }
  uint8_t* row = planes + r * 2 * K + (k0 / 128) * 256 + (k0 % 128);
  *(u32x4_t*)row = hi;
  *(u32x4_t*)(row + 128) = lo;
}

}  // namespace

hipError_t launch_act_i8_planes(const int8_t* qa, int64_t rows, int64_t K, uint8_t* planes, hipStream_t s) {
  const int64_t threads = rows * (K / 16);
  if (threads == 0) return hipSuccess;
  hipLaunchKernelGGL(act_i8_planes_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, qa, rows, K,
                     planes);
  return hipGetLastError();
}

namespace {

// Asymmetric int8 per token (qdg_quantize_act_zp). The range [lo, hi] of the
// row's finite values and 0 maps onto the 256 codes; scale, zero point and
// codes are decided in binary64 from the binary32 scale. Bound by its bytes,
// 2 k read and k written a row: TPR threads hold a row in registers (CH
// chunks of 16 values each) between the range and the encoding, so it is read once.
// M = 4096, k = 14336: 40.6 us (4.3 TB/s); 53.7 us with a second read and binary64
// throughout.
//
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

// 16 values of a row from i on (dword d holds values 2 d and 2 d + 1), 0
// behind its end. The 16 bytes at i and at i + 8 are read only where they
// start inside the row.
__device__ __forceinline__ void load16(const uint16_t* x, int64_t i, int64_t k, uint32_t (&v)[8]) {
  const u32x4_t z = {0, 0, 0, 0};
  const u32x4_t a = i < k ? *(const u32x4_t*)(x + i) : z, b = i + 8 < k ? *(const u32x4_t*)(x + i + 8) : z;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    v[d] = a[d];
    v[4 + d] = b[d];
  }
  if (i + 16 > k) {
#pragma unroll
    for (int d = 0; d < 8; ++d) v[d] &= i + 2 * d + 1 < k ? ~0u : i + 2 * d < k ? 0xFFFFu : 0u;
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

// The codes of 16 values into q + i.
__device__ __forceinline__ void encode16(const uint32_t (&v)[8], const ZpRow& z, int8_t* q, int64_t i, int64_t k) {
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23
  const int shift = (int)z.zero - 0x4B400000;
  uint32_t out[4];
  bool doubt = false;
  int c[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float f = __builtin_bit_cast(float, j & 1 ? v[j >> 1] & 0xFFFF0000u : v[j >> 1] << 16);
    const float y = __builtin_fmaf(f, z.inv32, kMagic);
    doubt |= !(fabsf(__builtin_fmaf(f, z.inv32, kMagic - y)) < kDoubt);
    c[j] = min(max(__builtin_bit_cast(int, y) + shift, -128), 127);
  }
  if (doubt) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float f = __builtin_bit_cast(float, j & 1 ? v[j >> 1] & 0xFFFF0000u : v[j >> 1] << 16);
      const double d = f == f ? rint((double)f * z.inv) : 0.0;
      c[j] = (int)fmin(fmax(d + z.zero, -128.0), 127.0);
    }
  }
#pragma unroll
  for (int d = 0; d < 4; ++d)
    out[d] = ((uint32_t)c[4 * d] & 0xFFu) | ((uint32_t)c[4 * d + 1] & 0xFFu) << 8 |
             ((uint32_t)c[4 * d + 2] & 0xFFu) << 16 | (uint32_t)c[4 * d + 3] << 24;
  if (i + 16 <= k) {
    *(u32x4_t*)(q + i) = u32x4_t{out[0], out[1], out[2], out[3]};
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (i + j < k) q[i + j] = (int8_t)(out[j >> 2] >> (8 * (j & 3)));
  }
}

// The largest of both over the TPR threads of a row.
template <int TPR>
__device__ __forceinline__ void row_max2(uint32_t& a, uint32_t& b, uint32_t (&buf)[2][4]) {
  for (int m = 32; m > 0; m >>= 1) {
    a = max(a, (uint32_t)__shfl_xor((int)a, m));
    b = max(b, (uint32_t)__shfl_xor((int)b, m));
  }
  if constexpr (TPR == 256) {
    __syncthreads();  // a row before has read the buffer
    if ((threadIdx.x & 63) == 0) {
      buf[0][threadIdx.x >> 6] = a;
      buf[1][threadIdx.x >> 6] = b;
    }
    __syncthreads();
    a = max(max(buf[0][0], buf[0][1]), max(buf[0][2], buf[0][3]));
    b = max(max(buf[1][0], buf[1][1]), max(buf[1][2], buf[1][3]));
  }
}

// CH > 0: a row of at most 16 TPR CH values in registers; CH = 0: any length,
// read twice.
template <int TPR, int CH>
__global__ __launch_bounds__(256) void act_int8_zp_kernel(const uint16_t* __restrict__ a, int64_t lda, int64_t M,
                                                          int64_t k, int8_t* __restrict__ q, int64_t ldq,
                                                          float* __restrict__ scales, int32_t* __restrict__ zeros) {
  __shared__ uint32_t buf[2][4];
  constexpr int RPB = 256 / TPR;
  const int t = threadIdx.x % TPR;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < M; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + threadIdx.x / TPR;
    if (TPR < 256 && row >= M) break;  // whole waves: no barrier below
    const uint16_t* x = a + row * lda;
    uint32_t v[CH ? CH : 1][8];
    const int chunks = CH ? CH : (int)((k + 16 * TPR - 1) / (16 * TPR));
    uint32_t pos = 0, neg = 0;  // packed maxima
    auto chunk_max = [&](const uint32_t(&w)[8]) {
#pragma unroll
      for (int d = 0; d < 8; ++d) {
        pos = pk_max_i16(pos, w[d]);
        neg = pk_max_u16(neg, w[d]);
      }
    };
    if constexpr (CH > 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c) load16(x, (int64_t)(c * TPR + t) * 16, k, v[c]);
#pragma unroll
      for (int c = 0; c < CH; ++c) chunk_max(v[c]);
    } else {
      for (int c = 0; c < chunks; ++c) {
        load16(x, ((int64_t)c * TPR + t) * 16, k, v[0]);
        chunk_max(v[0]);
      }
    }
    uint32_t hw = max(pos & 0xFFFFu, pos >> 16), lw = max(neg & 0xFFFFu, neg >> 16);
    row_max2<TPR>(hw, lw, buf);
    if (hw >= 0x7F80u || lw >= 0xFF80u) {  // an infinity or a NaN: they do not count
      hw = lw = 0;
      auto finite_max = [&](const uint32_t(&w)[8]) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const uint32_t h = j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
          if ((h & 0x7FFFu) < 0x7F80u) {
            if (h < 0x8000u) hw = max(hw, h);
            lw = max(lw, h);
          }
        }
      };
      if constexpr (CH > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) finite_max(v[c]);
      } else {
        for (int c = 0; c < chunks; ++c) {
          load16(x, ((int64_t)c * TPR + t) * 16, k, v[0]);
          finite_max(v[0]);
        }
      }
      row_max2<TPR>(hw, lw, buf);
    }
    const ZpRow z = zp_row(lw >= 0x8000u ? bf16_to_f32(lw) : 0.f, bf16_to_f32(hw));
    if (t == 0) {
      scales[row] = z.scale;
      zeros[row] = (int32_t)z.zero;
    }
    int8_t* y = q + row * ldq;
    if constexpr (CH > 0) {
#pragma unroll
      for (int c = 0; c < CH; ++c)
        if ((int64_t)(c * TPR + t) * 16 < k) encode16(v[c], z, y, (int64_t)(c * TPR + t) * 16, k);
    } else {
      for (int c = 0; c < chunks; ++c) {
        const int64_t i = ((int64_t)c * TPR + t) * 16;
        if (i >= k) break;
        load16(x, i, k, v[0]);
        encode16(v[0], z, y, i, k);
      }
    }
  }
}

}  // namespace

hipError_t launch_quantize_act_zp(const void* a, int64_t lda, int64_t M, int64_t k, int8_t* qa, int64_t ldq,
                                  float* scales, int32_t* zeros, hipStream_t s) {
  auto go = [&](auto kernel, int64_t rows_per_block) {
    const int64_t blocks = (M + rows_per_block - 1) / rows_per_block;
    hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < (1 << 20) ? blocks : 1 << 20)), dim3(256), 0, s,
                       (const uint16_t*)a, lda, M, k, qa, ldq, scales, zeros);
    return hipGetLastError();
  };
  if (k <= 1024) return go(act_int8_zp_kernel<64, 1>, 4);
  if (k <= 4096) return go(act_int8_zp_kernel<256, 1>, 1);
  if (k <= 8192) return go(act_int8_zp_kernel<256, 2>, 1);
  if (k <= 16384) return go(act_int8_zp_kernel<256, 4>, 1);
  return go(act_int8_zp_kernel<256, 0>, 1);
}

hipError_t launch_quantize_act(int atype, const void* a, int64_t M, int64_t K, void* qa, float* scales,
                               hipStream_t s) {
  if (atype == QDG_A_INT8) {
    hipLaunchKernelGGL(act_int8_kernel, dim3((unsigned)M), dim3(256), 0, s, (const uint16_t*)a, (int8_t*)qa,
                       scales, K);
  } else if (atype == QDG_A_MXFP4) {
    const int64_t blocks = M * (K / 32);
    hipLaunchKernelGGL(act_fp4_kernel, dim3((unsigned)((blocks * 4 + 255) / 256)), dim3(256), 0, s,
                       (const uint16_t*)a, (uint8_t*)qa, (uint8_t*)scales, blocks);
  } else {
    const int64_t threads = M * (K / 128) * 16;
    hipLaunchKernelGGL(act_fp8_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s,
                       (const uint16_t*)a, (uint8_t*)qa, scales, M, K);
  }
  return hipGetLastError();
}

}  // namespace qdg
