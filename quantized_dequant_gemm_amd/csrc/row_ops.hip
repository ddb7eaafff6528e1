// Operators over whole rows that end in bf16 rows and / or in the codes of the
// quantized products: qdg_norm (a block's output joins the residual stream,
// the stream is normed for the next block) and qdg_gated_act (act(gate) * up).
//
// Every value is decided in binary64 and rounded once to binary32, from there
// to bf16, so rows and codes are reproducible bit for bit. Both operators are
// bound by their bytes: TPR threads hold a row in registers, CH chunks of eight
// neighbouring values each, so that it is read once whatever statistics the
// norms and the codes need. Rows may start at any element: the 16-byte loads
// and stores are unaligned ones, and only a chunk that the row's end cuts is
// moved by elements.
#include "qdg_codes.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_2_t;
typedef __attribute__((ext_vector_type(4), aligned(4))) uint32_t u32x4_4_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;

// Eight values of one type as they are stored: bf16 pairs or binary32.
template <bool F32>
struct Raw8 {
  uint32_t d[F32 ? 8 : 4];
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (F32) return __builtin_bit_cast(float, d[j]);
    else return bf16_pair(d[j >> 1], j);
  }
};

// Values i .. i + 7 of a row of n, 0 behind its end.
template <bool F32>
__device__ __forceinline__ Raw8<F32> load8(const void* row, int i, int n) {
  Raw8<F32> r;
  if (i + 8 <= n) {
    if constexpr (F32) {
      const u32x4_4_t a = *(const u32x4_4_t*)((const uint32_t*)row + i), b = *(const u32x4_4_t*)((const uint32_t*)row + i + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        r.d[j] = a[j];
        r.d[4 + j] = b[j];
      }
    } else {
      const u32x4_2_t a = *(const u32x4_2_t*)((const uint16_t*)row + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) r.d[j] = a[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < (F32 ? 8 : 4); ++j) {
      if constexpr (F32) {
        r.d[j] = i + j < n ? ((const uint32_t*)row)[i + j] : 0u;
      } else {
        r.d[j] = i + 2 * j < n ? ((const uint16_t*)row)[i + 2 * j] : 0u;
        if (i + 2 * j + 1 < n) r.d[j] |= (uint32_t)((const uint16_t*)row)[i + 2 * j + 1] << 16;
      }
    }
  }
  return r;
}

template <bool F32>
__device__ __forceinline__ void store8(void* row, int i, int n, const Raw8<F32>& r) {
  if (i + 8 <= n) {
    if constexpr (F32) {
      *(u32x4_4_t*)((uint32_t*)row + i) = u32x4_4_t{r.d[0], r.d[1], r.d[2], r.d[3]};
      *(u32x4_4_t*)((uint32_t*)row + i + 4) = u32x4_4_t{r.d[4], r.d[5], r.d[6], r.d[7]};
    } else {
      *(u32x4_2_t*)((uint16_t*)row + i) = u32x4_2_t{r.d[0], r.d[1], r.d[2], r.d[3]};
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) {
        if constexpr (F32) ((uint32_t*)row)[i + j] = r.d[j];
        else ((uint16_t*)row)[i + j] = (uint16_t)(r.d[j >> 1] >> (16 * (j & 1)));
      }
  }
}

// A pair of binary32 values as bf16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t to_bf16_pair(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Weights, biases and gates: bf16 or binary32 as the call says.
__device__ __forceinline__ void load_vec8(const void* p, bool f32, int i, int n, float (&w)[8]) {
  if (f32) {
    const Raw8<true> r = load8<true>(p, i, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = r[j];
  } else {
    const Raw8<false> r = load8<false>(p, i, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = r[j];
  }
}

// ------------------------------------------------------------------ reductions over the TPR threads of a row
template <int TPR, class T, class Op>
__device__ __forceinline__ T row_reduce(T v, Op op, T (&buf)[16]) {
  for (int m = 32; m > 0; m >>= 1) v = op(v, __shfl_xor(v, m));
  if constexpr (TPR > 64) {
    __syncthreads();  // a reduction before has read the buffer
    if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v = op(v, buf[w]);
  }
  return v;
}

struct Buffers {
  double sum[16];
  float amax[16];
  uint32_t hw[16], lw[16];
};

template <int TPR>
__device__ __forceinline__ double row_sum(double v, Buffers& b) {
  return row_reduce<TPR>(v, [](double x, double y) { return x + y; }, b.sum);
}

// ------------------------------------------------------------------ the end of a row
// The bf16 values o of a row (chunk c of thread t: values 8 (c TPR + t) and on;
// 0 behind the end) as rows and codes.
template <int TPR, int CH>
__device__ __forceinline__ void finish_row(const Raw8<false> (&o)[CH], int n, int64_t row, int t, const RowOut& out,
                                           Buffers& buf) {
  if (out.rows) {
    uint16_t* p = out.rows + row * out.ld;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if ((c * TPR + t) * 8 < n) store8<false>(p, (c * TPR + t) * 8, n, o[c]);
  }
  if (out.quant == QDG_Q_NONE) return;
  uint8_t* q = out.qa + row * out.ldq;
  auto store_codes = [&](int i, u32x2_t v) {
    if (i + 8 <= n) {
      *(u32x2_t*)(q + i) = v;  // qa and its stride are multiples of 16 bytes
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < n) q[i + j] = (uint8_t)((j < 4 ? v.x : v.y) >> (8 * (j & 3)));
    }
  };
  if (out.quant == QDG_Q_INT8_ZP) {
    uint32_t pos = 0, neg = 0;  // packed maxima
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        pos = pk_max_i16(pos, o[c].d[d]);
        neg = pk_max_u16(neg, o[c].d[d]);
      }
    uint32_t hw = max(pos & 0xFFFFu, pos >> 16), lw = max(neg & 0xFFFFu, neg >> 16);
    auto most = [](uint32_t x, uint32_t y) { return max(x, y); };
    hw = row_reduce<TPR>(hw, most, buf.hw);
    lw = row_reduce<TPR>(lw, most, buf.lw);
    if (hw >= 0x7F80u || lw >= 0xFF80u) {  // an infinity or a NaN: they do not count
      hw = lw = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c) zp_finite_max<4>(o[c].d, hw, lw);
      hw = row_reduce<TPR>(hw, most, buf.hw);
      lw = row_reduce<TPR>(lw, most, buf.lw);
    }
    const ZpRow z = zp_row(lw >= 0x8000u ? bf16_to_f32(lw) : 0.f, bf16_to_f32(hw));
    if (t == 0) {
      ((float*)out.scales)[row] = z.scale;
      out.zeros[row] = (int32_t)z.zero;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if ((c * TPR + t) * 8 < n) {
        uint32_t code[2];
        encode_zp<4>(o[c].d, z, code);
        store_codes((c * TPR + t) * 8, u32x2_t{code[0], code[1]});
      }
    return;
  }
  float amax[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    amax[c] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax[c] = fmaxf(amax[c], fabsf(o[c][j]));
  }
  if (out.quant == QDG_Q_INT8) {
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < CH; ++c) m = fmaxf(m, amax[c]);
    m = row_reduce<TPR>(m, [](float x, float y) { return fmaxf(x, y); }, buf.amax);
    const bool nz = m > 0.f;
    const float inv = nz ? __fdiv_rn(127.0f, m) : 0.f;
    if (t == 0) ((float*)out.scales)[row] = nz ? __fdiv_rn(m, 127.0f) : 1.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if ((c * TPR + t) * 8 < n) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = o[c][j];
        store_codes((c * TPR + t) * 8, encode_int8x8(f, inv));
      }
    return;
  }
  // groups of 128 (16 lanes) or blocks of 32 (4 lanes): n is a multiple, so
  // that the lanes of a group are all inside the row or all behind it
  const bool fp8 = out.quant == QDG_Q_FP8E4M3;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    float m = amax[c];
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    if (fp8) {
      m = fmaxf(m, __shfl_xor(m, 4));
      m = fmaxf(m, __shfl_xor(m, 8));
    }
    const int i = (c * TPR + t) * 8;
    if (i >= n) continue;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = o[c][j];
    const bool nz = m > 0.f;
    if (fp8) {
      *(u32x2_t*)(q + i) = nz ? encode_fp8x8(f, __fdiv_rn(448.0f, m)) : u32x2_t{0, 0};
      if ((t & 15) == 0) ((float*)out.scales)[row * (n / 128) + i / 128] = nz ? __fdiv_rn(m, 448.0f) : 1.0f;
    } else {
      const uint32_t e8 = nz ? fp4_block_exponent(m) : 0u;
      *(uint32_t*)(q + i / 2) = nz ? encode_fp4x8(f, e8) : 0u;
      if ((t & 3) == 0) ((uint8_t*)out.scales)[row * (n / 32) + i / 32] = (uint8_t)e8;
    }
  }
}

// ------------------------------------------------------------------ norms
// 1 / sqrt(mean of squares + eps) of the row v, and with LAYER its mean.
template <int TPR, int CH>
__device__ __forceinline__ void row_stats(const float (&v)[CH][8], int n, int t, bool layer, float eps, double& mean,
                                          double& rs, Buffers& buf) {
  mean = 0.0;
  if (layer) {
    double s = 0.0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) s += (double)v[c][j];
    mean = row_sum<TPR>(s, buf) / (double)n;
  }
  double s = 0.0;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double d = (double)v[c][j] - mean;
      if ((c * TPR + t) * 8 + j < n) s += d * d;
    }
  rs = 1.0 / sqrt(row_sum<TPR>(s, buf) / (double)n + (double)eps);
}

template <int TPR, int CH, bool XF, bool RF>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_kernel(NormArgs a) {
  __shared__ Buffers buf;
  constexpr int kThreads = TPR < 256 ? 256 : TPR, RPB = kThreads / TPR;
  const int t = threadIdx.x % TPR, n = a.n;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.M; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + threadIdx.x / TPR;
    if (TPR < 256 && row >= a.M) break;  // whole waves: no barrier below
    const void* x = (const char*)a.x + row * a.ldx * (XF ? 4 : 2);
    const void* r = a.residual ? (const char*)a.residual + row * a.ldr * (RF ? 4 : 2) : nullptr;
    const void* g = a.gate ? (const char*)a.gate + row * a.ldg * (a.wf32 ? 4 : 2) : nullptr;
    float v[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const Raw8<XF> w = load8<XF>(x, (c * TPR + t) * 8, n);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[c][j] = w[j];
    }
    double mean = 0.0, rs = 1.0;
    if (a.post_norm) row_stats<TPR, CH>(v, n, t, a.layer, a.eps, mean, rs, buf);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * TPR + t) * 8;
      Raw8<RF> w = {}, s;
      if (r) w = load8<RF>(r, i, n);
      float pw[8], pb[8], gw[8];
      if (a.post_weight) load_vec8(a.post_weight, a.wf32, i, n, pw);
      if (a.post_bias) load_vec8(a.post_bias, a.wf32, i, n, pb);
      if (g) load_vec8(g, a.wf32, i, n, gw);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        double d = (double)v[c][j];
        if (a.post_norm) {
          d = (d - mean) * rs;
          if (a.post_weight) d *= (double)pw[j] + (double)a.weight_offset;
          if (a.post_bias) d += (double)pb[j];
        }
        if (g) d *= (double)gw[j];
        if (r) d += (double)a.residual_scale * (double)w[j];
        v[c][j] = i + j < n ? (float)d : 0.f;
      }
      if constexpr (RF) {
#pragma unroll
        for (int j = 0; j < 8; ++j) s.d[j] = __builtin_bit_cast(uint32_t, v[c][j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s.d[j] = to_bf16_pair(v[c][2 * j], v[c][2 * j + 1]);
          v[c][2 * j] = s[2 * j];
          v[c][2 * j + 1] = s[2 * j + 1];
        }
      }
      if (a.residual_out && i < n) store8<RF>((char*)a.residual_out + row * a.lds * (RF ? 4 : 2), i, n, s);
    }
    if (!a.out.rows && a.out.quant == QDG_Q_NONE) continue;
    row_stats<TPR, CH>(v, n, t, a.layer, a.eps, mean, rs, buf);
    Raw8<false> o[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * TPR + t) * 8;
      float wt[8], bs[8];
      if (a.weight) load_vec8(a.weight, a.wf32, i, n, wt);
      if (a.bias) load_vec8(a.bias, a.wf32, i, n, bs);
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        double d = ((double)v[c][j] - mean) * rs;
        if (a.weight) d *= (double)wt[j] + (double)a.weight_offset;
        if (a.bias) d += (double)bs[j];
        y[j] = i + j < n ? (float)d : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) o[c].d[j] = to_bf16_pair(y[2 * j], y[2 * j + 1]);
    }
    finish_row<TPR, CH>(o, n, row, t, a.out, buf);
  }
}

// ------------------------------------------------------------------ gated activation
// SiLU: g / (1 + exp(-g)); GELU in its tanh form: g / (1 + exp(-2 z)),
// z = sqrt(2 / pi) (g + 0.044715 g^3), as 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)).
// Where the exponential overflows the quotient is 0 with the sign of g.
__device__ __forceinline__ double act64(double g, int act) {
  const double z = act == QDG_ACT_SILU ? g : 1.5957691216057308 * (g + 0.044715 * g * g * g);
  return g / (1.0 + exp(-z));
}

template <int TPR, int CH, bool YF>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void gated_kernel(GatedArgs a) {
  __shared__ Buffers buf;
  constexpr int kThreads = TPR < 256 ? 256 : TPR, RPB = kThreads / TPR;
  const int t = threadIdx.x % TPR, n = a.n;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.M; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + threadIdx.x / TPR;
    if (TPR < 256 && row >= a.M) break;  // whole waves: no barrier below
    const char* y = (const char*)a.y + row * a.ldy * (YF ? 4 : 2);
    Raw8<false> o[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * TPR + t) * 8;
      const Raw8<YF> g = load8<YF>(y, i, n), u = load8<YF>(y + (int64_t)n * (YF ? 4 : 2), i, n);
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (float)(act64((double)g[j], a.act) * (double)u[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[c].d[j] = to_bf16_pair(f[2 * j], f[2 * j + 1]);
    }
    finish_row<TPR, CH>(o, n, row, t, a.out, buf);
  }
}

// Rows a launch walks at once (a launch holds fewer than 2^32 threads).
constexpr int64_t kMaxBlocks = (int64_t)1 << 20;

template <class K, class A>
hipError_t go(K kernel, int threads, int rows_per_block, const A& a, hipStream_t s) {
  const int64_t blocks = (a.M + rows_per_block - 1) / rows_per_block;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(threads), 0, s, a);
  return hipGetLastError();
}

template <bool XF, bool RF>
hipError_t norm_shape(const NormArgs& a, hipStream_t s) {
  if (a.n <= 512) return go(norm_kernel<64, 1, XF, RF>, 256, 4, a, s);
  if (a.n <= 2048) return go(norm_kernel<256, 1, XF, RF>, 256, 1, a, s);
  if (a.n <= 4096) return go(norm_kernel<256, 2, XF, RF>, 256, 1, a, s);
  if (a.n <= 8192) return go(norm_kernel<256, 4, XF, RF>, 256, 1, a, s);
  if (a.n <= 16384) return go(norm_kernel<512, 4, XF, RF>, 512, 1, a, s);
  return go(norm_kernel<1024, 4, XF, RF>, 1024, 1, a, s);
}

template <bool YF>
hipError_t gated_shape(const GatedArgs& a, hipStream_t s) {
  if (a.n <= 512) return go(gated_kernel<64, 1, YF>, 256, 4, a, s);
  if (a.n <= 2048) return go(gated_kernel<256, 1, YF>, 256, 1, a, s);
  if (a.n <= 4096) return go(gated_kernel<256, 2, YF>, 256, 1, a, s);
  if (a.n <= 8192) return go(gated_kernel<256, 4, YF>, 256, 1, a, s);
  if (a.n <= 16384) return go(gated_kernel<512, 4, YF>, 512, 1, a, s);
  if (a.n <= 32768) return go(gated_kernel<1024, 4, YF>, 1024, 1, a, s);
  return go(gated_kernel<1024, 8, YF>, 1024, 1, a, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool xf32, bool rf32, hipStream_t s) {
  if (xf32) return rf32 ? norm_shape<true, true>(a, s) : norm_shape<true, false>(a, s);
  return rf32 ? norm_shape<false, true>(a, s) : norm_shape<false, false>(a, s);
}

hipError_t launch_gated_act(const GatedArgs& a, bool yf32, hipStream_t s) {
  return yf32 ? gated_shape<true>(a, s) : gated_shape<false>(a, s);
}

}  // namespace qdg
