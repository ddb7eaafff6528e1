// Operators over whole rows that end in bf16 rows and / or in the codes of the
// quantized products: qdg_norm (a block's output joins the residual stream,
// the stream is normed for the next block) and qdg_gated_act (act(gate) * up).
//
// Every value is decided in binary64 and rounded once to binary32, from there
// to bf16, so rows and codes are reproducible bit for bit. Sums are binary64;
// the values themselves are computed in binary32 beside a bound of their error,
// and only where that leaves the bf16 number open (one value in 3000 to 5000)
// they are computed again in binary64. Both operators are bound by their bytes:
// TPR threads hold a row in registers, CH chunks of eight neighbouring values
// each, so that it is read once whatever statistics the norms and the codes
// need. Rows may start at any element: the 16-byte loads and stores are
// unaligned ones; a chunk that the row's end cuts is read as the row's last
// eight values and shifted.
#include "qdg_codes.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

typedef __attribute__((ext_vector_type(2), aligned(2))) uint32_t u32x2_2_t;
typedef __attribute__((ext_vector_type(2), aligned(4))) uint32_t u32x2_4_t;
typedef __attribute__((aligned(2))) uint32_t u32_2_t;

// Eight values of one type as they are stored: bf16 pairs or binary32.
template <bool F32>
struct Raw8 {
  uint32_t d[F32 ? 8 : 4];
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (F32) return __builtin_bit_cast(float, d[j]);
    else return bf16_pair(d[j >> 1], j);
  }
  // Keeps the compiler from holding what it has converted from the values
  // (eight binary64 numbers are 16 registers) until they are needed again.
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int j = 0; j < (F32 ? 8 : 4); ++j) asm volatile("" : "+v"(d[j]));
  }
};

// Values i .. i + 7 of a row of n (i < n); settle8 then leaves 0 behind its end.
// Apart, so that the branch of cut chunks comes when all of a row's loads are on
// their way (4096 x 8190 77 -> 65 us). EVEN: n is a multiple of 8.
template <bool F32, bool EVEN>
__device__ __forceinline__ Raw8<F32> load8(const void* row, int i, int n) {
  Raw8<F32> r;
  if (!EVEN && n < 8) {  // the same for all lanes: a row that is no chunk
#pragma unroll
    for (int j = 0; j < (F32 ? 8 : 4); ++j) {
      if constexpr (F32) {
        r.d[j] = j < n ? ((const uint32_t*)row)[j] : 0u;
      } else {
        r.d[j] = 2 * j < n ? ((const uint16_t*)row)[2 * j] : 0u;
        if (2 * j + 1 < n) r.d[j] |= (uint32_t)((const uint16_t*)row)[2 * j + 1] << 16;
      }
    }
    return r;
  }
  const int at = EVEN ? i : min(i, n - 8);
  if constexpr (F32) {
    const u32x4_4_t a = *(const u32x4_4_t*)((const uint32_t*)row + at), b = *(const u32x4_4_t*)((const uint32_t*)row + at + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.d[j] = a[j];
      r.d[4 + j] = b[j];
    }
  } else {
    const u32x4_2_t a = *(const u32x4_2_t*)((const uint16_t*)row + at);
#pragma unroll
    for (int j = 0; j < 4; ++j) r.d[j] = a[j];
  }
  return r;
}
template <bool EVEN, bool F32>
__device__ __forceinline__ void settle8(Raw8<F32>& r, int i, int n) {
  const int skip = EVEN || n < 8 ? 0 : max(i - (n - 8), 0);  // values that a chunk before has
  if (skip) {
    constexpr int kPer = F32 ? 1 : 2, kD = F32 ? 8 : 4;  // values a dword, dwords
#pragma unroll
    for (int b = 4; b >= kPer; b >>= 1)
      if (skip & b)
#pragma unroll
        for (int j = 0; j < kD; ++j) r.d[j] = j + b / kPer < kD ? r.d[j + b / kPer] : 0u;
    if constexpr (!F32) {
      if (skip & 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) r.d[j] = r.d[j] >> 16 | (j < 3 ? r.d[j + 1] << 16 : 0u);
    }
  }
}

// The first values of r into values i .. of a row of n (i < n).
template <bool F32, bool EVEN>
__device__ __forceinline__ void store8(void* row, int i, int n, Raw8<F32> r) {
  if constexpr (F32) {
    uint32_t* p = (uint32_t*)row + i;
    if (EVEN || i + 8 <= n) {
      *(u32x4_4_t*)p = u32x4_4_t{r.d[0], r.d[1], r.d[2], r.d[3]};
      *(u32x4_4_t*)(p + 4) = u32x4_4_t{r.d[4], r.d[5], r.d[6], r.d[7]};
      return;
    }
    const int rest = n - i;
    if (rest & 4) {
      *(u32x4_4_t*)p = u32x4_4_t{r.d[0], r.d[1], r.d[2], r.d[3]};
      p += 4;
#pragma unroll
      for (int j = 0; j < 3; ++j) r.d[j] = r.d[4 + j];
    }
    if (rest & 2) {
      *(u32x2_4_t*)p = u32x2_4_t{r.d[0], r.d[1]};
      p += 2;
      r.d[0] = r.d[2];
    }
    if (rest & 1) *p = r.d[0];
  } else {
    uint16_t* p = (uint16_t*)row + i;
    if (EVEN || i + 8 <= n) {
      *(u32x4_2_t*)p = u32x4_2_t{r.d[0], r.d[1], r.d[2], r.d[3]};
      return;
    }
    const int rest = n - i;
    if (rest & 4) {
      *(u32x2_2_t*)p = u32x2_2_t{r.d[0], r.d[1]};
      p += 4;
      r.d[0] = r.d[2];
      r.d[1] = r.d[3];
    }
    if (rest & 2) {
      *(u32_2_t*)p = r.d[0];
      p += 2;
      r.d[0] = r.d[1];
    }
    if (rest & 1) *p = (uint16_t)r.d[0];
  }
}

// Eight codes into bytes i .. of a row of n (rows of codes start at a multiple of 16).
template <bool EVEN>
__device__ __forceinline__ void store_codes(uint8_t* row, int i, int n, u32x2_t v) {
  uint8_t* p = row + i;
  if (EVEN || i + 8 <= n) {
    *(u32x2_t*)p = v;
    return;
  }
  const int rest = n - i;
  uint32_t w = v.x;
  if (rest & 4) {
    *(uint32_t*)p = w;
    p += 4;
    w = v.y;
  }
  if (rest & 2) {
    *(uint16_t*)p = (uint16_t)w;
    p += 2;
    w >>= 16;
  }
  if (rest & 1) *p = (uint8_t)w;
}

// Between binary64 values: their chains side by side would take the registers
// that let another wave in.
__device__ __forceinline__ void one_at_a_time() { __builtin_amdgcn_sched_barrier(0); }

// Weights, biases and gates; where there is none, `absent` for each.
template <bool F32, bool EVEN>
__device__ __forceinline__ Raw8<F32> load_vec8(const void* p, float absent, int i, int n) {
  if (p) return load8<F32, EVEN>(p, i, n);
  const uint32_t bits = __builtin_bit_cast(uint32_t, absent), word = F32 ? bits : bits >> 16 | (bits & 0xFFFF0000u);
  Raw8<F32> r;
#pragma unroll
  for (int j = 0; j < (F32 ? 8 : 4); ++j) r.d[j] = word;
  return r;
}

// ------------------------------------------------------------------ reductions over the TPR threads of a row
// Rows of 16 lanes, then halves of 32, against each other: of two copies of v
// the swap leaves both rows (halves) in every lane.
template <bool HALVES>
__device__ __forceinline__ void swap_rows(uint32_t v, uint32_t& x, uint32_t& y) {
  const auto r = HALVES ? __builtin_amdgcn_permlane32_swap(v, v, false, false) : __builtin_amdgcn_permlane16_swap(v, v, false, false);
  x = r[0];
  y = r[1];
}
template <bool HALVES, class Op>
__device__ __forceinline__ uint32_t across(uint32_t v, Op op) {
  uint32_t x, y;
  swap_rows<HALVES>(v, x, y);
  return op(x, y);
}
template <bool HALVES, class Op>
__device__ __forceinline__ float across(float v, Op op) {
  uint32_t x, y;
  swap_rows<HALVES>(__builtin_bit_cast(uint32_t, v), x, y);
  return op(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}
template <bool HALVES, class Op>
__device__ __forceinline__ double across(double v, Op op) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  uint32_t x0, y0, x1, y1;
  swap_rows<HALVES>((uint32_t)u, x0, y0);
  swap_rows<HALVES>((uint32_t)(u >> 32), x1, y1);
  return op(__builtin_bit_cast(double, (uint64_t)x1 << 32 | x0), __builtin_bit_cast(double, (uint64_t)y1 << 32 | y0));
}

template <class T, class Op>
__device__ __forceinline__ T wave_reduce(T v, Op op) {
  v = op(v, dpp<kXor1>(v));
  v = op(v, dpp<kXor2>(v));
  v = op(v, dpp<kMirror8>(v));
  v = op(v, dpp<kMirror16>(v));
  v = across<false>(v, op);
  return across<true>(v, op);
}

// Two sets of one value for each wave, used in turn: whoever writes a set has
// passed the barrier of the reduction between, which every wave reaches after
// reading that set. So one barrier a reduction is enough.
struct Buffers {
  double v[2][16];
};

template <int TPR, class T, class Op>
__device__ __forceinline__ T row_reduce(T v, Op op, Buffers& b, int& turn) {
  v = wave_reduce(v, op);
  if constexpr (TPR > 64) {
    constexpr int kWaves = TPR / 64;  // 4, 8 or 16: a lane reads one, DPP joins them
    T* set = (T*)b.v[turn];
    turn ^= 1;
    if ((threadIdx.x & 63) == 0) set[threadIdx.x >> 6] = v;
    __syncthreads();
    v = set[threadIdx.x & (kWaves - 1)];
    v = op(v, dpp<kXor1>(v));
    v = op(v, dpp<kXor2>(v));
    if constexpr (kWaves > 4) v = op(v, dpp<kMirror8>(v));
    if constexpr (kWaves > 8) v = op(v, dpp<kMirror16>(v));
  }
  return v;
}

template <int TPR>
__device__ __forceinline__ double row_sum(double v, Buffers& b, int& turn) {
  return row_reduce<TPR>(v, [](double x, double y) { return x + y; }, b, turn);
}

__device__ __forceinline__ float max_f32(float a, float b) { return fmaxf(a, b); }

// ------------------------------------------------------------------ the end of a row
// The larger of both halves of a pair's magnitudes.
__device__ __forceinline__ uint32_t halves_max(uint32_t v) { return max(v & 0xFFFFu, v >> 16); }

// The largest magnitude of eight values that is no NaN.
__device__ __forceinline__ float amax8(const Raw8<false>& o) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(o[j]));
  return m;
}

__device__ __forceinline__ uint32_t abs_max8(const Raw8<false>& o) {
  uint32_t m = o.d[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int d = 1; d < 4; ++d) m = pk_max_u16(m, o.d[d] & 0x7FFF7FFFu);
  return m;
}

// The codes of qdg_quantize_act's int8 rule for a finite row: rne(f * inv) of
// the rounded product is the low byte of product + 1.5 * 2^23, and no product
// is above 127 (1 + 2^-23).
__device__ __forceinline__ u32x2_t encode_int8x8_finite(const Raw8<false>& o, float inv) {
  uint32_t c[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float p = o[j] * inv;
    asm volatile("" : "+v"(p));  // two roundings: not one fused product and sum
    c[j] = __builtin_bit_cast(uint32_t, p + 12582912.f);
  }
  u32x2_t out;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t lo = __builtin_amdgcn_perm(c[4 * h + 1], c[4 * h], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(c[4 * h + 3], c[4 * h + 2], 0x04000C0Cu);
    out[h] = lo | hi;
  }
  return out;
}

// The codes of the fp8 rule for a finite group: no product is above
// 448 (1 + 2^-23), which rounds to 448 (the next code would begin at 464).
__device__ __forceinline__ u32x2_t encode_fp8x8_finite(const float (&f)[8], float inv) {
  u32x2_t out;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j] * inv, f[4 * j + 1] * inv, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * j + 2] * inv, f[4 * j + 3] * inv, w, true);
    out[j] = (uint32_t)w;
  }
  return out;
}

// The bf16 values o of a row (chunk c of thread t: values 8 (c TPR + t) and on,
// with t counted from the row's or its piece's start; 0 behind the end) as rows
// and codes. int8 codes need the whole row, groups and blocks only theirs.
template <int TPR, int CH, bool EVEN>
__device__ __forceinline__ void finish_row(const Raw8<false> (&o)[CH], int n, int64_t row, int t, const RowOut& out,
                                           Buffers& buf, int& turn) {
  if (out.rows) {
    uint16_t* p = out.rows + row * out.ld;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if ((c * TPR + t) * 8 < n) store8<false, EVEN>(p, (c * TPR + t) * 8, n, o[c]);
  }
  if (out.quant == QDG_Q_NONE) return;
  uint8_t* q = out.qa + row * out.ldq;
  if (out.quant == QDG_Q_INT8_ZP) {
    uint32_t pos = 0, neg = 0;  // packed maxima
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        pos = pk_max_i16(pos, o[c].d[d]);
        neg = pk_max_u16(neg, o[c].d[d]);
      }
    uint32_t hw = halves_max(pos), lw = halves_max(neg);
    uint32_t both = row_reduce<TPR>(hw | lw << 16, pk_max_u16, buf, turn);
    hw = both & 0xFFFFu;
    lw = both >> 16;
    if (hw >= 0x7F80u || lw >= 0xFF80u) {  // an infinity or a NaN: they do not count
      hw = lw = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c) zp_finite_max<4>(o[c].d, hw, lw);
      both = row_reduce<TPR>(hw | lw << 16, pk_max_u16, buf, turn);
      hw = both & 0xFFFFu;
      lw = both >> 16;
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
        encode_zp<4, true>(o[c].d, z, code);
        store_codes<EVEN>(q, (c * TPR + t) * 8, n, u32x2_t{code[0], code[1]});
      }
    return;
  }
  if (out.quant == QDG_Q_INT8) {
    uint32_t word = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c) word = pk_max_u16(word, abs_max8(o[c]));
    word = row_reduce<TPR>(halves_max(word), [](uint32_t x, uint32_t y) { return max(x, y); }, buf, turn);
    const bool finite = word < 0x7F80u;
    float m = bf16_to_f32(word);
    if (!finite) {  // a NaN does not count
      m = 0.f;
#pragma unroll
      for (int c = 0; c < CH; ++c) m = fmaxf(m, amax8(o[c]));
      m = row_reduce<TPR>(m, max_f32, buf, turn);
    }
    const bool nz = m > 0.f;
    const float inv = nz ? __fdiv_rn(127.0f, m) : 0.f;
    if (t == 0) ((float*)out.scales)[row] = nz ? __fdiv_rn(m, 127.0f) : 1.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if ((c * TPR + t) * 8 < n) {
        u32x2_t code;
        // a row that is smaller than the quotient's range (inv infinite) takes the general way too
        if (finite && inv < 0x1p127f) {
          code = encode_int8x8_finite(o[c], inv);
        } else {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = o[c][j];
          code = encode_int8x8(f, inv);
        }
        store_codes<EVEN>(q, (c * TPR + t) * 8, n, code);
      }
    return;
  }
  // groups of 128 (16 lanes) or blocks of 32 (4 lanes): n is a multiple, so
  // that the lanes of a group are all inside the row or all behind it
  const bool fp8 = out.quant == QDG_Q_FP8E4M3;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    uint32_t word = abs_max8(o[c]);
    word = pk_max_u16(word, dpp<kXor1>(word));
    word = pk_max_u16(word, dpp<kXor2>(word));
    if (fp8) {
      word = pk_max_u16(word, dpp<kMirror8>(word));
      word = pk_max_u16(word, dpp<kMirror16>(word));
    }
    word = halves_max(word);
    float m = bf16_to_f32(word);
    const bool finite = !__any(word >= 0x7F80u);
    if (!finite) {  // a NaN does not count
      m = amax8(o[c]);
      m = fmaxf(m, dpp<kXor1>(m));
      m = fmaxf(m, dpp<kXor2>(m));
      if (fp8) {
        m = fmaxf(m, dpp<kMirror8>(m));
        m = fmaxf(m, dpp<kMirror16>(m));
      }
    }
    const int i = (c * TPR + t) * 8;
    if (i >= n) continue;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = o[c][j];
    const bool nz = m > 0.f;
    if (fp8) {
      const float inv = nz ? __fdiv_rn(448.0f, m) : 0.f;
      *(u32x2_t*)(q + i) = !nz ? u32x2_t{0, 0} : finite && inv < 0x1p120f ? encode_fp8x8_finite(f, inv) : encode_fp8x8(f, inv);
      if ((t & 15) == 0) ((float*)out.scales)[row * (n / 128) + i / 128] = nz ? __fdiv_rn(m, 448.0f) : 1.0f;
    } else {
      const uint32_t e8 = nz ? fp4_block_exponent(m) : 0u;
      *(uint32_t*)(q + i / 2) = nz ? encode_fp4x8(f, e8) : 0u;
      if ((t & 3) == 0) ((uint8_t*)out.scales)[row * (n / 32) + i / 32] = (uint8_t)e8;
    }
  }
}

// ------------------------------------------------------------------ doubt
// y is a binary32 value with an error of at most ULPS units in its last place:
// near enough to the middle of two bf16 numbers (low half 0x8000) it leaves the
// rounding open. 0 to 2 ULPS (in the high half) there, more elsewhere.
template <int ULPS>
__device__ __forceinline__ uint32_t to_middle(float y) {
  return (__builtin_bit_cast(uint32_t, y) << 16) + ((0x8000u + ULPS) << 16);
}
template <int ULPS>
constexpr uint32_t kMiddle = (uint32_t)(2 * ULPS) << 16 | 0xFFFFu;

// ------------------------------------------------------------------ norms
// kPlain: an RMS norm of the stream with bf16 weights, no bias, a join that one
// rounding of binary32 settles, no gate, and rows of whole chunks. kPlainGate:
// such a norm with a gate, whose check of the product's range takes registers
// (without an instance of its own 4096 x 4096 with fp8 codes alone takes 29.9 us
// instead of 26.8). kEven: anything else
// with bf16 weights in rows of whole chunks. kGeneral: bf16 weights, a cut last
// chunk. kF32Weights: any row (4096 x 4096 42.0 us, 33.1 with bf16 weights; with a
// bias 46.2; one more instance for whole chunks with a bias brought 4096 x 4096
// from 48.8 to 47.3 us and 4096 x 8192 layer from 109 to 114).
enum { kPlain, kPlainGate, kEven, kGeneral, kF32Weights };

// 1 / sqrt(x): v_rsq_f64 (2^-14 or better) and three steps of Newton's
// iteration, each of which squares the error; 0 and infinity stay as they are.
__device__ __forceinline__ double inverse_root(double x) {
  double y = __builtin_amdgcn_rsq(x);
  if (!(x > 0.0) || !(x < __builtin_inf())) return y;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const double e = __builtin_fma(-x * y, y, 1.0);  // 1 - x y^2
    y = __builtin_fma(0.5 * y, e, y);
  }
  return y;
}

// 1 / sqrt(mean of squares + eps) of the row v, and with LAYER its mean: s / n as
// s inv_n and a step of Newton's iteration, which is exact where the quotient
// is, so that a constant row (its sum is exact) has its value as mean. The
// variance is the mean of squares less the mean's square, which keeps 46 bits
// unless the mean is more than four deviations off 0; a row that lies further
// off is summed again around its mean.
template <int TPR, int CH, bool F32>
__device__ __forceinline__ void row_stats(Raw8<F32> (&v)[CH], int n, int t, bool layer, float eps, double inv_n, double& mean,
                                          double& rs, Buffers& buf, int& turn) {
  mean = 0.0;
  double s = 0.0, sq = 0.0;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (layer) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = (double)v[c][j];
        s += d;
        sq = __builtin_fma(d, d, sq);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double d = (double)v[c][j];
        sq = __builtin_fma(d, d, sq);
      }
    }
    v[c].renew();
  }
  if (layer) {
    s = row_sum<TPR>(s, buf, turn);
    mean = s * inv_n;
    mean = __builtin_fma(__builtin_fma(-mean, (double)n, s), inv_n, mean);
  }
  double var = row_sum<TPR>(sq, buf, turn) * inv_n;
  if (layer) {
    var -= mean * mean;
    if (!(var * 16.0 > mean * mean)) {  // the same for all threads of the row
      sq = 0.0;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int rest = n - (c * TPR + t) * 8;  // the zeros behind the end do not count
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double d = j < rest ? (double)v[c][j] - mean : 0.0;
          sq = __builtin_fma(d, d, sq);
          one_at_a_time();
        }
        v[c].renew();
      }
      var = row_sum<TPR>(sq, buf, turn) * inv_n;
    }
  }
  rs = inverse_root(var + (double)eps);
}

// What is absent is neutral: a factor 1, a term -0 (which leaves a sum its sign).
// The new stream of eight values: residual_scale * r + gate * t. Without a norm
// of x and with a product of at most 16 significant bits (short; a gate beside
// bf16 x and weights only), that is one rounding of binary32, where no product
// of the eight leaves binary32's normal range (or is 0).
template <bool PLAIN, bool GATE, bool XF, bool RF, bool WF, bool EVEN>
__device__ __forceinline__ Raw8<RF> join8(const NormArgs& a, const Raw8<XF>& x, const Raw8<RF>& r, const Raw8<WF>& g, int i,
                                          double mean, double rs) {
  const int n = a.n;
  const float scale = a.residual ? a.residual_scale : -1.0f;  // of zeros
  Raw8<RF> s;
  auto put = [&](int j, float lo, float hi) {  // values 2 j and 2 j + 1
    if constexpr (RF) {
      s.d[2 * j] = __builtin_bit_cast(uint32_t, lo);
      s.d[2 * j + 1] = __builtin_bit_cast(uint32_t, hi);
    } else {
      s.d[j] = to_bf16_pair(lo, hi);
    }
  };
  bool open = !(PLAIN || a.short_join);
  if (!open) {
    if (GATE && !XF && !WF && a.gate) {
      float least = __builtin_inff(), most = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = x[2 * j] * g[2 * j], p1 = x[2 * j + 1] * g[2 * j + 1];
        least = least3(least, p, p1);
        most = fmaxf(fmaxf(most, fabsf(p)), fabsf(p1));
        put(j, __builtin_fmaf(scale, r[2 * j], p), __builtin_fmaf(scale, r[2 * j + 1], p1));
      }
      open = !(least >= 0x1p-126f && most < __builtin_inff());
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) put(j, __builtin_fmaf(scale, r[2 * j], x[2 * j]), __builtin_fmaf(scale, r[2 * j + 1], x[2 * j + 1]));
    }
  }
  if (open) {
    Raw8<WF> w, b;
    if (!PLAIN) {
      w = load_vec8<WF, EVEN>(a.post_weight, 1.0f, i, n);
      b = load_vec8<WF, EVEN>(a.post_bias, -0.0f, i, n);
      settle8<EVEN>(w, i, n);
      settle8<EVEN>(b, i, n);
    }
    const double offset = a.post_weight ? (double)a.weight_offset : 0.0;
    const int rest = n - i;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      double d = (double)x[j];
      if (!PLAIN) d = (d - mean) * rs * ((double)w[j] + offset) + (double)b[j];
      d = __builtin_fma((double)scale, (double)r[j], d * (double)g[j]);
      v[j] = (float)d;
      if (j & 1) one_at_a_time();
    }
    if (!EVEN && rest < 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = j < rest ? v[j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) put(j, v[2 * j], v[2 * j + 1]);
  }
  return s;
}

// Eight normed values. y = (s rs) w carries four roundings of 2^-24 (rs,
// w + offset, both products): 4 units in the last place of y, 6 are allowed for.
// Not PLAIN (a bias or a mean): m = ((s - mean) rs) w, the mean in two binary32
// parts, y = m + b; m's error, with two more roundings, and the sum's are within
// 2^-21 |m| + 2^-23 |b| + 2^-44 |mean rs w|, and the roundings of both ends of
// that interval are compared. Where (s - mean) rs or y is below 2^-100, rs
// leaves the middle of binary32's range or w + offset may leave it, binary64 decides.
template <bool PLAIN, bool RF, bool WF, bool EVEN>
__device__ __forceinline__ Raw8<false> norm8(const NormArgs& a, const Raw8<RF>& s, const Raw8<WF>& w, const Raw8<WF>& b, int i,
                                             double mean, double rs, bool in_range) {
  Raw8<false> o;
  const float rs32 = (float)rs, offset = a.weight ? a.weight_offset : 0.f;
  float least = __builtin_inff();
  bool doubt = !in_range;
  const int rest = a.n - i;
  if constexpr (PLAIN) {
    uint32_t near = ~0u;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float p = s[j] * rs32;
      y[j] = p * (w[j] + offset);
      near = min(near, to_middle<6>(y[j]));
      least = least3(least, p, y[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) o.d[j] = to_bf16_pair(y[2 * j], y[2 * j + 1]);
    doubt |= near <= kMiddle<6>;
  } else {
    uint32_t differ = 0;
    const float mean_hi = (float)mean, mean_lo = (float)(mean - (double)mean_hi), off = fabsf(mean_hi) * rs32 * 0x1p-44f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo[2], hi[2], p[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float wj = w[2 * j + h] + offset, bj = b[2 * j + h];
        p[h] = ((s[2 * j + h] - mean_hi) - mean_lo) * rs32;
        const float m = p[h] * wj, sum = m + bj;
        const float e = __builtin_fmaf(fabsf(m), 0x1p-21f, __builtin_fmaf(fabsf(bj), 0x1p-23f, __builtin_fmaf(off, fabsf(wj), 0x1p-110f)));
        lo[h] = sum - e;
        hi[h] = sum + e;
      }
      least = least3(least, p[0], p[1]);
      o.d[j] = to_bf16_pair(lo[0], lo[1]);
      differ |= o.d[j] ^ to_bf16_pair(hi[0], hi[1]);
    }
    doubt |= differ != 0;
    if (!EVEN && rest < 8) {  // the zeros behind the end leave nothing open
      least = __builtin_inff();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < rest) least = least3(least, least, ((s[j] - mean_hi) - mean_lo) * rs32);
    }
  }
  doubt |= !(least > 0x1p-100f);
  if (doubt) {
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      double d = (PLAIN ? (double)s[j] : (double)s[j] - mean) * rs * ((double)w[j] + (double)offset);
      if (!PLAIN) d += (double)b[j];
      z[j] = (float)d;
      one_at_a_time();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) o.d[j] = to_bf16_pair(z[2 * j], z[2 * j + 1]);
  }
  if (!EVEN && rest < 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o.d[j] &= 2 * j + 1 < rest ? ~0u : 2 * j < rest ? 0xFFFFu : 0u;
  }
  return o;
}

// One pass over a row in registers: the join, its sum of squares (and sum), the
// normed values, the codes' statistics, rows and codes. 4096 x 4096 bf16 with
// rows and int8 zp codes 33 us (4.6 TB/s), 8192 x 8192 layer in binary32 with
// 4-bit codes 146 us (4.8), where HBM is what bounds it; 333 x 7168 norms on both sides 13.2 us (2.7 TB/s): one workgroup or two a
// CU, each a chain of load, two sums with a barrier, stores; 1 x 4096 3.8 us in a
// graph. Four waves a SIMD are 128 registers; kPlain in 256 threads has five in
// 96 (4096 x 4096 with fp8 codes alone 26.8 against 28.1 us, with a binary32
// stream 37.5 against 38.7), in 512 not (4096 x 8192 62.4 against 61.0: two
// workgroups a CU either way, and some spilled).
template <int TPR, int CH, bool XF, bool RF, int MODE>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, MODE == kPlain && TPR <= 256 ? 5 : 4) void norm_kernel(NormArgs a) {
  constexpr bool PLAIN = MODE == kPlain || MODE == kPlainGate, GATE = MODE != kPlain, WF = MODE == kF32Weights, EVEN = PLAIN || MODE == kEven;
  __shared__ Buffers buf;
  int turn = 0;
  constexpr int kThreads = TPR < 256 ? 256 : TPR, RPB = kThreads / TPR;
  const int t = threadIdx.x % TPR, n = a.n;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.M; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + threadIdx.x / TPR;
    if (TPR < 256 && row >= a.M) break;  // whole waves: no barrier below
    const char* x = (const char*)a.x + row * a.ldx * (XF ? 4 : 2);
    const char* r = (const char*)a.residual + row * a.ldr * (RF ? 4 : 2);
    const char* g = GATE && a.gate ? (const char*)a.gate + row * a.ldg * (WF ? 4 : 2) : nullptr;
    Raw8<XF> v[CH];
    Raw8<RF> s[CH];
    Raw8<WF> gate[CH], weight[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      v[c] = {};
      s[c] = {};
      const int i = (c * TPR + t) * 8;
      if (i < n) {
        v[c] = load8<XF, EVEN>(x, i, n);
        if (a.residual) s[c] = load8<RF, EVEN>(r, i, n);
        if (GATE) gate[c] = load_vec8<WF, EVEN>(g, 1.0f, i, n);
        weight[c] = load_vec8<WF, EVEN>(a.weight, 1.0f, i, n);
      }
    }
    if constexpr (!EVEN) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * TPR + t) * 8;
        settle8<EVEN>(v[c], i, n);
        settle8<EVEN>(s[c], i, n);
        settle8<EVEN>(gate[c], i, n);
        settle8<EVEN>(weight[c], i, n);
      }
    }
    double mean = 0.0, rs = 1.0;
    if (!PLAIN && a.post_norm) row_stats<TPR, CH, XF>(v, n, t, a.layer, a.eps, a.inv_n, mean, rs, buf, turn);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * TPR + t) * 8;
      if (i < n) {
        s[c] = join8<PLAIN, GATE, XF, RF, WF, EVEN>(a, v[c], s[c], gate[c], i, mean, rs);
        if (a.residual_out) store8<RF, EVEN>((char*)a.residual_out + row * a.lds * (RF ? 4 : 2), i, n, s[c]);
      }
      s[c].renew();
    }
    if (!a.out.rows && a.out.quant == QDG_Q_NONE) continue;
    row_stats<TPR, CH, RF>(s, n, t, !PLAIN && a.layer, a.eps, a.inv_n, mean, rs, buf, turn);
    // an offset below 2^100 keeps any weight inside binary32's range
    const bool in_range = rs > 0x1p-60 && rs < 0x1p60 && fabsf(a.weight_offset) < 0x1p100f;
    Raw8<false> o[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * TPR + t) * 8;
      o[c] = {};
      if (i < n) {
        Raw8<WF> b = load_vec8<WF, EVEN>(PLAIN ? nullptr : a.bias, -0.0f, i, n);
        settle8<EVEN>(b, i, n);
        o[c] = norm8<PLAIN, RF, WF, EVEN>(a, s[c], weight[c], b, i, mean, rs, in_range);
      }
      o[c].renew();
    }
    finish_row<TPR, CH, EVEN>(o, n, row, t, a.out, buf, turn);
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

// act(g) * u of eight values. In binary32: e = 2^t (1 + r ln 2), t = -g log2(e)
// rounded and r what that left out (within 2^-24 |t| 2^-24 and a rounding), so
// that e is within 2 units in its last place (v_exp_f32 has one) and a rounding;
// 1 + e, its reciprocal (one unit) and two products follow: at most 9 units in
// the last place, 11 are allowed for. GELU's t = -g (c1 + c3 g^2) is itself off
// by up to 2.5 roundings and those of its constants, 4 2^-24 |t|, which the
// exponential turns into as much times ln 2 of its value: within 2^-24 (22 + 4 |t|)
// all told, and both ends of that interval are compared. Where the value or the
// reciprocal is below 2^-100 (or a NaN), binary64 decides: above, u times the
// reciprocal keeps its digits (a product below binary32's normal range needs a
// gate above 2^26, whose reciprocal is 1, to come back above 2^-100).
template <bool YF>
__device__ __forceinline__ Raw8<false> gated8(const Raw8<YF>& g, const Raw8<YF>& u, int act) {
  Raw8<false> o;
  float y[8], off[8], least = __builtin_inff();
  bool doubt;
  if (act == QDG_ACT_SILU) {
    uint32_t near = ~0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      constexpr float kL = 1.44269504f, kLo = 1.92596303e-8f, kLn2 = 0.69314718f;  // log2(e) = kL + kLo
      const float h = __builtin_amdgcn_fmed3f(g[j], -256.f, 256.f);
      const float t = -h * kL, r = __builtin_fmaf(-h, kLo, __builtin_fmaf(-h, kL, -t));
      const float e = __builtin_amdgcn_exp2f(t) * __builtin_fmaf(r, kLn2, 1.0f);  // infinite from t = 128 on
      const float rc = __builtin_amdgcn_rcpf(1.0f + e);
      y[j] = (u[j] * rc) * g[j];
      near = min(near, to_middle<11>(y[j]));
      least = least3(least, y[j], rc);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) o.d[j] = to_bf16_pair(y[2 * j], y[2 * j + 1]);
    doubt = near <= kMiddle<11>;
  } else {
    uint32_t differ = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      constexpr float kC1 = -2.3022082f, kC3 = -0.10294324f;  // -2 sqrt(2 / pi) log2(e), and 0.044715 of it
      const float h = __builtin_amdgcn_fmed3f(g[j], -32.f, 32.f);
      const float t = h * __builtin_fmaf(h * h, kC3, kC1);
      const float rc = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
      y[j] = (u[j] * rc) * g[j];
      off[j] = __builtin_fmaf(fabsf(t), 0x1p-22f, 22 * 0x1p-24f) * y[j];
      least = least3(least, y[j], rc);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o.d[j] = to_bf16_pair(y[2 * j] - off[2 * j], y[2 * j + 1] - off[2 * j + 1]);
      differ |= o.d[j] ^ to_bf16_pair(y[2 * j] + off[2 * j], y[2 * j + 1] + off[2 * j + 1]);
    }
    doubt = differ != 0;
  }
  if (doubt || !(least > 0x1p-100f)) {  // which values' numbers are open? A lane's are computed one after the other.
    uint32_t open = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.d[j] = to_bf16_pair(y[2 * j], y[2 * j + 1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // the reciprocal is above 2^-100 with these gates
      bool is = !(fabsf(y[j]) > 0x1p-100f) || !(g[j] > (act == QDG_ACT_SILU ? -69.f : -8.5f));
      if (act == QDG_ACT_SILU) {
        is |= to_middle<11>(y[j]) <= kMiddle<11>;
      } else {
        const uint32_t both = to_bf16_pair(y[j] - off[j], y[j] + off[j]);
        is |= (both & 0xFFFFu) != both >> 16;
      }
      if (y[j] == 0.f && (g[j] == 0.f || u[j] == 0.f)) is = false;  // exactly 0
      open |= is ? 1u << j : 0u;
    }
    while (open) {
      const uint32_t bit = open & -open;
      open ^= bit;
      float gj = 0.f, uj = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        gj = bit >> j & 1 ? g[j] : gj;
        uj = bit >> j & 1 ? u[j] : uj;
      }
      const uint32_t b = to_bf16_pair((float)(act64((double)gj, act) * (double)uj), 0.f);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (bit >> j & 1) o.d[j >> 1] = j & 1 ? (o.d[j >> 1] & 0xFFFFu) | b << 16 : (o.d[j >> 1] & 0xFFFF0000u) | (b & 0xFFFFu);
    }
  }
  return o;
}

// A piece of TPR * CH * 8 columns of a row for each blockIdx.y: one for int8
// codes, which need the row's largest value. 4096 x 14336 with fp8 codes 70.5 us
// (4.2 TB/s): HBM, and some 40 vector instructions for each 64 values beside it,
// two of them transcendental; with int8 codes 68 us (28 bytes a lane spilled).
// Without the bound of four waves a SIMD the int8 instances take more registers
// and one row a CU (103 us). GELU 78 and 75 us, binary32 Y 106.
template <int TPR, int CH, bool YF, bool EVEN>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR, 4) void gated_kernel(GatedArgs a) {
  __shared__ Buffers buf;
  int turn = 0;
  constexpr int kThreads = TPR < 256 ? 256 : TPR, RPB = kThreads / TPR;
  const int t = threadIdx.x % TPR + blockIdx.y * (TPR * CH), n = a.n;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.M; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = r0 + threadIdx.x / TPR;
    if (TPR < 256 && row >= a.M) break;  // whole waves: no barrier below
    const char* y = (const char*)a.y + row * a.ldy * (YF ? 4 : 2);
    Raw8<YF> g[CH], u[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int i = (c * TPR + t) * 8;
      g[c] = u[c] = {};
      if (i < n) {
        g[c] = load8<YF, EVEN>(y, i, n);
        u[c] = load8<YF, EVEN>(y + (int64_t)n * (YF ? 4 : 2), i, n);
      }
    }
    if constexpr (!EVEN) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int i = (c * TPR + t) * 8;
        settle8<EVEN>(g[c], i, n);
        settle8<EVEN>(u[c], i, n);
      }
    }
    Raw8<false> o[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      o[c] = {};
      if ((c * TPR + t) * 8 < n) o[c] = gated8<YF>(g[c], u[c], a.act);
      o[c].renew();
    }
    finish_row<TPR, CH, EVEN>(o, n, row, t, a.out, buf, turn);
  }
}

// Rows a launch walks at once (a launch holds fewer than 2^32 threads).
constexpr int64_t kMaxBlocks = (int64_t)1 << 20;

template <class K, class A>
hipError_t go(K kernel, int threads, int rows_per_block, const A& a, hipStream_t s, int pieces = 1) {
  const int64_t blocks = (a.M + rows_per_block - 1) / rows_per_block, most = kMaxBlocks / pieces;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < most ? blocks : most), (unsigned)pieces), dim3(threads), 0, s, a);
  return hipGetLastError();
}

template <bool XF, bool RF, int MODE>
hipError_t norm_shape(const NormArgs& a, hipStream_t s) {
  // Up to 8192 values two workgroups or more of rows a CU, each thread two chunks:
  // one row's loads run beside another's sums (one chunk: 4096 x 4096 37 against
  // 34 us, 8192 x 8192 layer 196 against 144, 4096 x 3001 layer 49 against 38).
  // Short rows are a wave's, without barriers (16384 x 512 32 against 15 us).
  if (a.n <= 512) return go(norm_kernel<64, 1, XF, RF, MODE>, 256, 4, a, s);
  if (a.n <= 2048) return go(norm_kernel<256, 1, XF, RF, MODE>, 256, 1, a, s);
  if (a.n <= 4096) return go(norm_kernel<256, 2, XF, RF, MODE>, 256, 1, a, s);
  if (a.n <= 8192) return go(norm_kernel<512, 2, XF, RF, MODE>, 512, 1, a, s);
  if (a.n <= 16384) return go(norm_kernel<1024, 2, XF, RF, MODE>, 1024, 1, a, s);
  return go(norm_kernel<1024, 4, XF, RF, MODE>, 1024, 1, a, s);
}

template <bool XF, bool RF>
hipError_t norm_kind(const NormArgs& a, hipStream_t s) {
  if (a.wf32) return norm_shape<XF, RF, kF32Weights>(a, s);
  if (a.n % 8) return norm_shape<XF, RF, kGeneral>(a, s);
  const bool plain = !a.layer && !a.bias && a.short_join;
  if (!plain) return norm_shape<XF, RF, kEven>(a, s);
  if constexpr (!XF) {
    if (a.gate) return norm_shape<XF, RF, kPlainGate>(a, s);
  }
  return norm_shape<XF, RF, kPlain>(a, s);
}

template <bool YF, bool EVEN>
hipError_t gated_shape(const GatedArgs& a, hipStream_t s) {
  if (a.n <= 512) return go(gated_kernel<64, 1, YF, EVEN>, 256, 4, a, s);
  if (a.n <= 2048) return go(gated_kernel<256, 1, YF, EVEN>, 256, 1, a, s);
  if (a.n <= 4096) return go(gated_kernel<256, 2, YF, EVEN>, 256, 1, a, s);
  // in pieces, which fill the chip at fewer rows (16 x 14336 fp8 6.6 against 5.3 us, 4096 x 14336 74 against 71)
  if (a.out.quant != QDG_Q_INT8 && a.out.quant != QDG_Q_INT8_ZP)
    return go(gated_kernel<256, 2, YF, EVEN>, 256, 1, a, s, (a.n + 4095) / 4096);
  if (a.n <= 8192) return go(gated_kernel<512, 2, YF, EVEN>, 512, 1, a, s);
  // 1024 threads: one row a CU, its registers' most in flight; 512 hold two rows,
  // which binary32 Y has no registers for (16 x 14336 6.4 against 7.2 us, 4096 x 14336 90 against 66)
  if constexpr (!YF) {
    if (a.n <= 16384 && a.M > 256) return go(gated_kernel<512, 4, YF, EVEN>, 512, 1, a, s);
  }
  if (a.n <= 16384) return go(gated_kernel<1024, 2, YF, EVEN>, 1024, 1, a, s);
  if (a.n <= 32768) return go(gated_kernel<1024, 4, YF, EVEN>, 1024, 1, a, s);
  return go(gated_kernel<1024, 8, YF, EVEN>, 1024, 1, a, s);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, bool xf32, bool rf32, hipStream_t s) {
  if (xf32) return rf32 ? norm_kind<true, true>(a, s) : norm_kind<true, false>(a, s);
  return rf32 ? norm_kind<false, true>(a, s) : norm_kind<false, false>(a, s);
}

hipError_t launch_gated_act(const GatedArgs& a, bool yf32, hipStream_t s) {
  if (a.n % 8) return yf32 ? gated_shape<true, false>(a, s) : gated_shape<false, false>(a, s);
  return yf32 ? gated_shape<true, true>(a, s) : gated_shape<false, true>(a, s);
}

}  // namespace qdg
