// int8 x int8 products over row-major operands (qdg_gemm_i8, qdg_moe_gemm_i8):
//
//   Y[m][j] = sa[m] * sb[j] * (sum_k A[m][k] B[j][k] - za[m] * sum_k B[j][k]) + bias[j]
//
// with both sums exact in int32 on int8 MFMAs (16 x 16 x 64 in the rows kernel,
// 32 x 32 x 32 in the tiles) and dot products.
// The weights are the MFMA's row operand, so a lane of the result holds four
// consecutive columns of one row of Y. With the SiLU*mul epilogue the 16-column tiles
// of B alternate between gate and up rows, so that a lane holds both halves.

#include <algorithm>
#include <iterator>

#include "qdg_device.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

// The first row of B behind 16-column tile vt, and the rows that tile has.
template <bool SILU>
__device__ __forceinline__ void i8_tile(const I8Args& p, int vt, int& first, int& rows) {
  const int j = (SILU ? vt >> 1 : vt) * 16;
  first = (SILU && (vt & 1) ? p.cols : 0) + j;
  rows = p.cols - j;
}

// One form in every kernel, so that a row does not depend on which one ran.
// In binary32, as the outputs are at most: three roundings of half a step
// (2^-24) behind the exact sum, far below bf16's 2^-8.
__device__ __forceinline__ float i8_scale(int acc, float sa, float sb, float bias) {
  return __builtin_fmaf((float)acc * sa, sb, bias);
}

// As in the other families. exp(-x) passes binary32's range below -88.7, where
// the result counts as 0 (exactly: at most 2^-121).
__device__ __forceinline__ float i8_silu(float x) { return x / (1.0f + expf(-x)); }

// Four values to bf16 (v_cvt_pk_bf16_f32: nearest even).
__device__ __forceinline__ u32x2_t i8_bf16x4(f32x4_t v) {
  typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4_t;
  return __builtin_bit_cast(u32x2_t, __builtin_convertvector(v, bf16x4_t));
}

// Stores of vectors at any element (gfx950 takes them unaligned).
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(2)));

// Four consecutive outputs of one row: the integer sums (gate and up with
// SILU) of columns j0 .. j0 + 3 through scales, bias, epilogue and rounding.
template <bool SILU>
__device__ __forceinline__ void i8_finish(const I8Args& p, i32x4_t g, i32x4_t u, int yrow, int arow, int j0) {
  if (j0 >= p.cols) return;
  const int cnt = min(4, p.cols - j0);
  uint32_t out[4];
  if (p.otype == QDG_O_I32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = (uint32_t)g[i];
  } else {
    const float sa = p.a_scales[arow];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = j0 + min(i, cnt - 1);
      float y = i8_scale(g[i], sa, p.b_scales[c], p.bias ? p.bias[c] : 0.f);
      if constexpr (SILU) {
        y = i8_silu(y) * i8_scale(u[i], sa, p.b_scales[c + p.cols], p.bias ? p.bias[c + p.cols] : 0.f);
      }
      out[i] = __builtin_bit_cast(uint32_t, y);
    }
  }
  if (p.otype == QDG_O_BF16) {
    uint16_t* dst = (uint16_t*)p.Y + (int64_t)yrow * p.ldy + j0;
    const u32x2_t h = i8_bf16x4(__builtin_bit_cast(f32x4_t, u32x4_t{out[0], out[1], out[2], out[3]}));
    if (cnt == 4) {
      *(u32x2_any_t*)dst = h;
    } else {
      for (int i = 0; i < 4; ++i)
        if (i < cnt) dst[i] = (uint16_t)(h[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    uint32_t* dst = (uint32_t*)p.Y + (int64_t)yrow * p.ldy + j0;
    if (cnt == 4) {
      *(u32x4_any_t*)dst = u32x4_t{out[0], out[1], out[2], out[3]};
    } else {
      for (int i = 0; i < 4; ++i)
        if (i < cnt) dst[i] = out[i];
    }
  }
}

// The 16 bytes at row + k0, with the bytes from k on as zeros. A 16-byte
// chunk that starts behind the row's end is not read.
__device__ __forceinline__ u32x4_t i8_load_tail(const int8_t* row, int k0, int k) {
  const int left = k - k0;
  if (left <= 0) return u32x4_t{0, 0, 0, 0};
  u32x4_t v = *(const u32x4_t*)(row + k0);
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int b = left - 4 * d;
    v[d] &= b >= 4 ? ~0u : b <= 0 ? 0u : (1u << (8 * b)) - 1;
  }
  return v;
}

__device__ __forceinline__ int i8_sum16(u32x4_t v, int acc) {
#pragma unroll
  for (int d = 0; d < 4; ++d) acc = __builtin_amdgcn_sdot4((int)v[d], 0x01010101, acc, false);
  return acc;
}

constexpr int kRowWaves = 8;

// Up to 16 rows and few columns: fragments straight from memory, the K range
// split over the eight waves of a workgroup that owns 16 columns of Y. Bound by
// the weights' bytes: 16 KiB of loads in flight per CU at once and no barrier
// in the loop (1 x 4096 x 4096, weights in the last-level cache: 5.5 us, 3.3 us
// of it loop = 5 TB/s, from memory 7.2 us; cached also two column tiles per
// workgroup 7.5 us, the 64 x 64 LDS tiles 9.9 us; from 8192 columns on those are
// as fast, at 14336 faster: 12.2 against 17 us). K stays in one workgroup, so
// that few columns leave CUs idle (1 x 576 x 7168, 36 workgroups: 7.0 us).
template <bool SILU, bool ZP>
__global__ __launch_bounds__(64 * kRowWaves) void gemm_i8_rows_kernel(const I8Args p) {
  constexpr int KW = kRowWaves, NT = SILU ? 2 : 1;  // gate and up tile
  __shared__ i32x4_t red[KW][NT][64];
  __shared__ int zred[KW][NT][16];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nb = blockIdx.x;
  const int row = min(r, p.M - 1);
  const int8_t* ap = p.A + (int64_t)row * p.lda;
  const int8_t* bp[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    int first, rows;
    i8_tile<SILU>(p, nb * NT + nt, first, rows);
    bp[nt] = p.B + (int64_t)(first + min(r, rows - 1)) * p.ldb;
  }
  i32x4_t acc[NT];
  int zs[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    zs[nt] = 0;
    acc[nt] = i32x4_t{0, 0, 0, 0};
  }
  const int steps = (p.k + 63) / 64, full = p.k / 64;
  const int s0 = steps * wave / KW, s1 = steps * (wave + 1) / KW;
  for (int s = s0; s < min(s1, full); ++s) {
    const int k0 = s * 64 + 16 * c;
    u32x4_t b[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) b[nt] = *(const u32x4_t*)(bp[nt] + k0);
    const u32x4_t a = *(const u32x4_t*)(ap + k0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (ZP) zs[nt] = i8_sum16(b[nt], zs[nt]);
      acc[nt] = mfma_i8(b[nt], a, acc[nt]);
    }
  }
  if (s1 > full) {  // the step that the row's end cuts
    const int k0 = full * 64 + 16 * c;
    const u32x4_t a = i8_load_tail(ap, k0, p.k);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const u32x4_t b = i8_load_tail(bp[nt], k0, p.k);
      if constexpr (ZP) zs[nt] = i8_sum16(b, zs[nt]);
      acc[nt] = mfma_i8(b, a, acc[nt]);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    red[wave][nt][lane] = acc[nt];
    if constexpr (ZP) {
      int z = zs[nt];
      z += __shfl_xor(z, 16);
      z += __shfl_xor(z, 32);
      if (c == 0) zred[wave][nt][r] = z;
    }
  }
  __syncthreads();
  if (wave != 0 || r >= p.M) return;
  i32x4_t v[2] = {};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int w = 0; w < KW; ++w) v[nt] += red[w][nt][lane];
    if constexpr (ZP) {
      const int za = p.a_zeros[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int z = 0;
#pragma unroll
        for (int w = 0; w < KW; ++w) z += zred[w][nt][4 * c + i];
        v[nt][i] -= za * z;
      }
    }
  }
  i8_finish<SILU>(p, v[0], v[1], r, r, nb * 16 + 4 * c);
}

// The partials of a split product (columns in the order of B's tiles), added
// and finished: one thread per row and four columns of Y.
template <bool SILU>
__global__ __launch_bounds__(256) void gemm_i8_reduce_kernel(const I8Args p, int split) {
  const int64_t quads = (p.cols + 3) / 4;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= quads * p.M) return;
  const int row = (int)(t / quads), j0 = (int)(t % quads) * 4;
  const int c = SILU ? j0 / 16 * 32 + j0 % 16 : j0;
  i32x4_t v[2] = {};
  for (int s = 0; s < split; ++s) {
    const int32_t* src = p.partial + ((int64_t)s * p.M + row) * p.vcols + c;
    v[0] += *(const i32x4_t*)src;
    if constexpr (SILU) v[1] += *(const i32x4_t*)(src + 16);
  }
  i8_finish<SILU>(p, v[0], v[1], row, row, j0);
}

// ------------------------------------------------------------- LDS tiles
// Many rows: a BM x BN tile of Y per workgroup, 32 x 32 MFMA tiles, K in
// groups of 128 bytes through NS stages of LDS. A stage holds the rows of A
// and B as they are stored (128 bytes a row), copied by direct global -> LDS
// loads of 16 bytes a lane; the chunk of 16 bytes at slot j of row r is chunk
// j ^ f(r), so that the 16-byte fragment reads of 8 (or 16) neighbouring rows fall on
// different banks without padding.
//
// What bounds them: the 256 x 256 tile the card's power (8192^3: 2.3-2.4 POP/s
// with random codes, 3.1 with A all zero; 4096 x 14336 x 4096 240-265 us = 1.8-2.0
// POP/s); the small tiles the copies into LDS (16-20 TB/s
// over the card, so a 64 x 64 tile takes 0.19 us a group where its MFMAs take 0.06);
// with up to 64 rows the weights' way in (16 x 14336 x 4096 16.6 us = 3.6 TB/s from
// memory, 11.8 us = 5.0 TB/s out of the last-level cache). Row strides
// that are no multiple of 128 bytes split every copied piece over two lines:
// up to 1.6 times slower in the small tiles. Measured without gain: eight
// stages instead of four, eight waves sharing the steps of a group, copies of
// two groups at a time (8 % slower), four waves of 128 x 128 (spills, 13 % slower).
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((ext_vector_type(16))) int i32x16_t;

__device__ __forceinline__ i32x16_t mfma_i8_32(u32x4_t a, u32x4_t b, i32x16_t c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0,
                                               0);
}

__device__ __forceinline__ int i8_swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Where a wave's copies read: copy q takes 8 rows of A or B through a buffer
// resource that starts at the first of them and ends with the operand, so
// that rows and bytes behind the operand's end read as 0 without a branch
// (bytes between a row's end and its stride are masked before use). off: the
// lane's row and chunk.
template <int LOADS>
struct I8Src {
  __amdgpu_buffer_rsrc_t rsrc[LOADS];
  uint32_t off[LOADS];
};

// The resource for rows from `row` on of an operand of `rows` rows, its last
// row `len` bytes long. All of it is the same in every lane, and said to be: the
// 64-bit comparisons run on the vector unit, and a resource left in vector
// registers costs a loop around every copy.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t i8_rows_rsrc(const int8_t* base, int64_t row, int64_t rows,
                                                              int64_t ld, int64_t len) {
  int64_t left = (rows - 1 - row) * ld + len;
  left = left < 0 ? 0 : left > 0xFFFFFFFFll ? 0xFFFFFFFFll : left;
  const uint64_t at = (uint64_t)(base + (left > 0 ? row * ld : 0));
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(at >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void*)(hi << 32 | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane((int)(uint32_t)left), 0x00020000);
}

// Copies FROM .. TO - 1 of group g into one stage (every wave issues the same
// number). TAG, here and below, is not used: it gives every calling function
// its own specialization (hipcc's host pass rejects a second function that
// calls the same specialization of a device function using target builtins).
// Buffer loads, because the compiler tracks them apart from LDS reads; a
// global load to LDS in flight makes it wait for every LDS read where one
// would do.
template <int FROM, int TO, int LOADS, int NW, int TAG>
__device__ __forceinline__ void i8_load_stage(char* st, const I8Src<LOADS>& src, int wave, int g) {
#pragma unroll
  for (int q = FROM; q < TO; ++q)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(src.rsrc[q], (lds_void*)(st + (q * NW + wave) * 1024), 16,
                                             src.off[q] + (uint32_t)g * 128u, 0, 0, 0);
}

// Zeroes the bytes from k on of the 16 at byte kk of a row.
__device__ __forceinline__ u32x4_t i8_mask(u32x4_t v, int kk, int k) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int b = k - kk - 4 * d;
    v[d] &= b >= 4 ? ~0u : b <= 0 ? 0u : (1u << (8 * b)) - 1;
  }
  return v;
}

// The fragments of one 32-byte step of a wave's (32 TM) x (32 TN) tile.
template <int TM, int TN>
struct I8Frag {
  u32x4_t a[TM], b[TN];
};

template <int TM, int TN>
__device__ __forceinline__ void i8_frag_load(I8Frag<TM, TN>& f, const char* st, int a_lane, int b_lane, int at) {
#pragma unroll
  for (int t = 0; t < TN; ++t) f.b[t] = *(const u32x4_t*)(st + b_lane + t * 4096 + at);
#pragma unroll
  for (int t = 0; t < TM; ++t) f.a[t] = *(const u32x4_t*)(st + a_lane + t * 4096 + at);
}

// kk: the row byte that the lane's chunk holds (bytes from k on count 0).
template <int TM, int TN>
__device__ __forceinline__ void i8_frag_mask(I8Frag<TM, TN>& f, int kk, int k) {
#pragma unroll
  for (int t = 0; t < TN; ++t) f.b[t] = i8_mask(f.b[t], kk, k);
#pragma unroll
  for (int t = 0; t < TM; ++t) f.a[t] = i8_mask(f.a[t], kk, k);
}

// MFMAs FROM .. TO - 1 of the step's TM * TN.
template <int FROM, int TO, int TM, int TN, bool ZP, int TAG>
__device__ __forceinline__ void i8_frag_mma(const I8Frag<TM, TN>& f, i32x16_t (&acc)[TM][TN], int (&zs)[TN]) {
#pragma unroll
  for (int i = FROM; i < TO; ++i) {
    const int t = i / TM, m = i % TM;
    acc[m][t] = mfma_i8_32(f.b[t], f.a[m], acc[m][t]);
    if constexpr (ZP) {  // the column sums' dot products, spread over the tile's MFMAs
#pragma unroll
      for (int d = 4 * m / TM; d < 4 * (m + 1) / TM; ++d)
        zs[t] = __builtin_amdgcn_sdot4((int)f.b[t][d], 0x01010101, zs[t], false);
    }
  }
}

// The first half of a step's MFMAs with the copies of a group between them.
template <int I, int H, int LOADS, int NW, int TM, int TN, bool ZP, int TAG>
__device__ __forceinline__ void i8_mma_and_load(const I8Frag<TM, TN>& f, i32x16_t (&acc)[TM][TN], int (&zs)[TN],
                                                char* st, const I8Src<LOADS>& src, int wave, int g) {
  if constexpr (I < H) {
    i8_frag_mma<I, I + 1, TM, TN, ZP, TAG + I>(f, acc, zs);
    i8_load_stage<LOADS * I / H, LOADS*(I + 1) / H, LOADS, NW, TAG>(st, src, wave, g);
    __builtin_amdgcn_sched_barrier(0);
    i8_mma_and_load<I + 1, H, LOADS, NW, TM, TN, ZP, TAG>(f, acc, zs, st, src, wave, g);
  }
}

// Group g of the K loop. Its first fragments are in f0 already. Each step's
// fragment reads go out before the MFMAs of the step before; the barrier sits
// in front of the last step's MFMAs, where every wave has its last fragments
// of this group in registers: then the next group's first reads and the
// copies of group g + NS into this group's stage run under those MFMAs.
// LEFT: copies that may stay in flight while the next group's have landed.
template <int LOADS, int NW, int TM, int TN, int LEFT, bool ZP, bool MASK, int TAG>
__device__ __forceinline__ void i8_group(char* st, const char* next, const I8Src<LOADS>& src, int wave, int g,
                                         int load_g, int a_lane, int b_lane, const int (&at)[4], int half, int k,
                                         I8Frag<TM, TN>& f0, I8Frag<TM, TN>& f1, i32x16_t (&acc)[TM][TN],
                                         int (&zs)[TN]) {
  constexpr int MF = TM * TN, H = MF > 1 ? MF / 2 : 1;
  const int kk = g * 128 + half * 16;
  i8_frag_load(f1, st, a_lane, b_lane, at[1]);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (MASK) i8_frag_mask(f0, kk, k);
  i8_frag_mma<0, MF, TM, TN, ZP, TAG>(f0, acc, zs);
  __builtin_amdgcn_sched_barrier(0);
  i8_frag_load(f0, st, a_lane, b_lane, at[2]);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (MASK) i8_frag_mask(f1, kk + 32, k);
  i8_frag_mma<0, MF, TM, TN, ZP, TAG>(f1, acc, zs);
  __builtin_amdgcn_sched_barrier(0);
  i8_frag_load(f1, st, a_lane, b_lane, at[3]);
  __builtin_amdgcn_sched_barrier(0);
  if constexpr (MASK) i8_frag_mask(f0, kk + 64, k);
  i8_frag_mma<0, MF, TM, TN, ZP, TAG>(f0, acc, zs);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | (7 << 4) | (15 << 8) | ((LEFT >> 4) << 14));
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
  if constexpr (MASK) i8_frag_mask(f1, kk + 96, k);
  i8_mma_and_load<0, H, LOADS, NW, TM, TN, ZP, TAG>(f1, acc, zs, st, src, wave, load_g);
  i8_frag_load(f0, next, a_lane, b_lane, at[0]);
  __builtin_amdgcn_sched_barrier(0);
  i8_frag_mma<H, MF, TM, TN, ZP, TAG + 64>(f1, acc, zs);
  __builtin_amdgcn_sched_barrier(0);
}

// The same for small wave tiles (at most 4 MFMAs a step): the fragments of
// the whole next group are read under this group's MFMAs, where a read a step
// ahead would wait out the LDS latency at every step.
template <int LOADS, int NW, int TM, int TN, int LEFT, bool ZP, bool MASK, int TAG>
__device__ __forceinline__ void i8_group_whole(char* st, const char* next, const I8Src<LOADS>& src, int wave, int g,
                                               int load_g, int a_lane, int b_lane, const int (&at)[4], int half, int k,
                                               I8Frag<TM, TN> (&f)[4], I8Frag<TM, TN> (&fn)[4],
                                               i32x16_t (&acc)[TM][TN], int (&zs)[TN]) {
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | (7 << 4) | (15 << 8) | ((LEFT >> 4) << 14));
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): f is here, the stage is free
  asm volatile("s_barrier" ::: "memory");
#pragma unroll
  for (int s = 0; s < 4; ++s) i8_frag_load(fn[s], next, a_lane, b_lane, at[s]);
  __builtin_amdgcn_sched_barrier(0);
  i8_load_stage<0, LOADS, LOADS, NW, TAG>(st, src, wave, load_g);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if constexpr (MASK) i8_frag_mask(f[s], g * 128 + (2 * s + half) * 16, k);
    i8_frag_mma<0, TM * TN, TM, TN, ZP, TAG>(f[s], acc, zs);
  }
  __builtin_amdgcn_sched_barrier(0);
}

template <int WM, int WN, int TM, int TN, int NS, bool SILU, bool ZP, bool MOE>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_tile_kernel(const I8Args p, int m_blocks, int n_blocks,
                                                                     int m_run) {
  constexpr int NW = WM * WN, BM = 32 * TM * WM, BN = 32 * TN * WN, BYTES = (BM + BN) * 128;
  constexpr int LOADS = (BM + BN) / 8 / NW, TAG = ((WM * 8 + WN) * 8 + TM) * 512 + (TN * 8 + NS) * 8 + SILU * 4 + ZP * 2 + MOE;
  static_assert(BM / 8 % NW == 0 && BN / 8 % NW == 0, "every wave issues the same copies of A and of B");
  constexpr int A_LOADS = BM / 8 / NW;
  static_assert(NS >= 2 && NS <= 4 && NS * BYTES <= 160 * 1024, "two to four stages within LDS");
  static_assert(LOADS * (NS - 1) < 64, "vmcnt holds the copies in flight");
  // separate objects, so that the compiler can tell a copy into one stage
  // from a read of another
  __shared__ __attribute__((aligned(1024))) char st0[BYTES];
  __shared__ __attribute__((aligned(1024))) char st1[BYTES];
  __shared__ __attribute__((aligned(1024))) char st2[NS > 2 ? BYTES : 16];
  __shared__ __attribute__((aligned(1024))) char st3[NS > 3 ? BYTES : 16];
  char* const stage[4] = {st0, st1, st2, st3};
  const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  int mb, nb;
  if constexpr (MOE) {
    // an XCD takes runs of m_run blocks and walks them together, column block
    // by column block: the blocks of one expert share its weights in that
    // XCD's L2
    const int x = blockIdx.x % 8, j = blockIdx.x / 8;
    const int run = j / (m_run * n_blocks), at = j % (m_run * n_blocks);
    mb = (run * 8 + x) * m_run + at % m_run;
    nb = at / m_run;
    if (mb >= m_blocks) return;  // the grid covers whole rounds of runs
  } else {
    // XCD x takes the x-th eighth of the tile order, which walks 4 x 8 blocks
    // of tiles (as in the 8-bit tiles over packed weights)
    const int total = m_blocks * n_blocks;
    int lin = blockIdx.x;
    if (total % 8 == 0) lin = (lin % 8) * (total / 8) + lin / 8;
    if (m_blocks % 4 == 0 && n_blocks % 8 == 0) {
      const int sb = lin / 32, w = lin % 32;
      mb = (sb / (n_blocks / 8)) * 4 + w / 8;
      nb = (sb % (n_blocks / 8)) * 8 + w % 8;
    } else {
      mb = lin / n_blocks;
      nb = lin % n_blocks;
    }
  }
  // the pair behind a row of the tile, -1 for none (a 16-row block fills half
  // of a 32-row tile)
  auto pair_of = [&](int row) {
    if (row >= p.block_m) return -1;
    const int id = p.sorted_ids[mb * p.block_m + row];
    return (unsigned)id < (unsigned)p.num_pairs ? id : -1;
  };
  auto a_row_of = [&](int pair) { return p.a_per_pair ? pair : pair / p.top_k; };
  // What the epilogue needs of the rows and columns, and the rows of A, are
  // asked for here at once: one after the other, and at the end, they cost a memory
  // latency each.
  constexpr int TC = SILU ? 16 : 32;  // columns of Y from a 32-column tile
  const bool raw = p.otype == QDG_O_I32;
  int expert = 0, a_pair[A_LOADS], yr[TM], za[TM];  // yr < 0: no row
  float sa[TM];
  if constexpr (MOE) {
    const int used = __builtin_amdgcn_readfirstlane(*p.num_padded);
    expert = __builtin_amdgcn_readfirstlane(p.block_expert[mb]);
#pragma unroll
    for (int q = 0; q < A_LOADS; ++q) a_pair[q] = pair_of((q * NW + wave) * 8 + (lane >> 3));
#pragma unroll
    for (int m = 0; m < TM; ++m) yr[m] = pair_of((wm * TM + m) * 32 + r);
    if (mb * p.block_m >= used || (unsigned)expert >= (unsigned)p.num_experts) return;
  } else {
#pragma unroll
    for (int m = 0; m < TM; ++m) {
      yr[m] = mb * BM + (wm * TM + m) * 32 + r;
      if (yr[m] >= p.M) yr[m] = -1;
    }
  }
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int ar = yr[m] < 0 ? 0 : MOE ? a_row_of(yr[m]) : yr[m];
    sa[m] = raw ? 1.f : p.a_scales[ar];
    za[m] = ZP ? p.a_zeros[ar] : 0;
  }
  // 16-column tiles of B in the order the epilogue wants (gate and up tiles
  // alternate with SILU)
  const int vt0 = p.vt_first + nb * (BN / 16);
  static_assert(BN <= 64 * NW, "a thread for every column");
  float my_scale = 0.f, my_bias = 0.f;
  if (!raw && threadIdx.x < BN) {
    int first, rows;
    i8_tile<SILU>(p, vt0 + threadIdx.x / 16, first, rows);
    const int64_t at = (int64_t)expert * p.n + (rows > 0 ? first + min((int)threadIdx.x % 16, rows - 1) : 0);
    my_scale = p.b_scales[at];
    my_bias = p.bias ? p.bias[at] : 0.f;
  }
  I8Src<LOADS> src;
  const int64_t k16 = (p.k + 15) / 16 * 16;
#pragma unroll
  for (int q = 0; q < LOADS; ++q) {
    const int i = q * NW + wave;  // rows 8 i .. 8 i + 7 of the stage: A, then B
    const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 3) ^ (i & 1)) * 16u;
    if (q < A_LOADS) {
      if constexpr (MOE) {
        // A ends below kI8FarRow (checked by the host): rows that are not
        // there read zeros behind it
        src.rsrc[q] = i8_rows_rsrc(p.A, 0, p.M, p.lda, k16);
        src.off[q] = a_pair[q] < 0 ? kI8FarRow : (uint32_t)a_row_of(a_pair[q]) * (uint32_t)p.lda + chunk;
      } else {
        src.rsrc[q] = i8_rows_rsrc(p.A, mb * BM + i * 8, p.M, p.lda, k16);
        src.off[q] = (uint32_t)(lane >> 3) * (uint32_t)p.lda + chunk;
      }
    } else {
      const int row = i * 8 - BM;
      int first, rows;
      i8_tile<SILU>(p, vt0 + row / 16, first, rows);
      // rows behind a tile's last column are other rows of B or zeros, their
      // results are never stored
      src.rsrc[q] = i8_rows_rsrc(p.B + (int64_t)expert * p.n * p.ldb, rows > 0 ? first + row % 16 : p.n, p.n, p.ldb,
                                 k16);
      src.off[q] = (uint32_t)(lane >> 3) * (uint32_t)p.ldb + chunk;
    }
  }
  // this workgroup's groups of K: [g0, groups)
  const int all = (p.k + 127) / 128;
  const int g0 = (int)((int64_t)all * blockIdx.y / gridDim.y), groups = (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y);
  const int a_lane = (wm * TM * 32 + r) * 128, b_lane = (BM + wn * TN * 32 + r) * 128, sw = i8_swizzle(r);
  i32x16_t acc[TM][TN];
  int zs[TN];
#pragma unroll
  for (int t = 0; t < TN; ++t) {
    zs[t] = 0;
#pragma unroll
    for (int m = 0; m < TM; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][t][i] = 0;
  }
  int at[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) at[q] = ((2 * q + half) ^ sw) * 16;
#pragma unroll
  for (int q = 0; q < NS; ++q)
    i8_load_stage<0, LOADS, LOADS, NW, TAG>(stage[q], src, wave, min(g0 + q, groups - 1));
  constexpr int LEFT = LOADS * (NS - 1);
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | (7 << 4) | (15 << 8) | ((LEFT >> 4) << 14));
  asm volatile("s_barrier" ::: "memory");
  const int full = min(p.k / 128, groups);  // groups that need no mask
  int g = g0;
  // full rounds of NS groups with constant stages, then the rest, the last
  // group cut at k
  if constexpr (TM * TN <= 4 && NS % 2 == 0) {  // the two fragment sets alternate with the stages
    I8Frag<TM, TN> f[2][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) i8_frag_load(f[0][q], st0, a_lane, b_lane, at[q]);
    for (; g + NS <= full; g += NS) {
#pragma unroll
      for (int cur = 0; cur < NS; ++cur)
        i8_group_whole<LOADS, NW, TM, TN, LOADS*(NS - 2), ZP, false, TAG + (1 << 20)>(
            stage[cur], stage[(cur + 1) % NS], src, wave, g + cur, min(g + cur + NS, groups - 1), a_lane, b_lane, at,
            half, p.k, f[cur % 2], f[(cur + 1) % 2], acc, zs);
    }
    // at most NS groups are left: all copied
#pragma unroll
    for (int cur = 0; cur < NS; ++cur)
      if (g + cur < groups)
        i8_group_whole<LOADS, NW, TM, TN, 0, ZP, true, TAG + (1 << 21)>(
            stage[cur], stage[(cur + 1) % NS], src, wave, g + cur, groups - 1, a_lane, b_lane, at, half, p.k,
            f[cur % 2], f[(cur + 1) % 2], acc, zs);
  } else {
    I8Frag<TM, TN> f0, f1;
    i8_frag_load(f0, st0, a_lane, b_lane, at[0]);
    for (; g + NS <= full; g += NS) {
#pragma unroll
      for (int cur = 0; cur < NS; ++cur)
        i8_group<LOADS, NW, TM, TN, LOADS*(NS - 2), ZP, false, TAG + (1 << 20)>(
            stage[cur], stage[(cur + 1) % NS], src, wave, g + cur, min(g + cur + NS, groups - 1), a_lane, b_lane, at,
            half, p.k, f0, f1, acc, zs);
    }
#pragma unroll
    for (int cur = 0; cur < NS; ++cur)
      if (g + cur < groups)
        i8_group<LOADS, NW, TM, TN, 0, ZP, true, TAG + (1 << 21)>(
            stage[cur], stage[(cur + 1) % NS], src, wave, g + cur, groups - 1, a_lane, b_lane, at, half, p.k, f0, f1,
            acc, zs);
  }
  __builtin_amdgcn_s_waitcnt(0);  // the trailing copies have landed
  __syncthreads();

  // ---- epilogue. A lane holds row r of each 32-row tile and, of each
  // 32-column tile, the columns 8 q + 4 half .. + 3. Column scales and biases
  // (in the order of the tile's columns) and the column sums of B go through
  // LDS; so does each strip of 32 rows, so that stores are whole row segments.
  constexpr int PITCH = 128 + 16, STRIP = 32 * PITCH;  // a strip row: at most 128 bytes
  static_assert(NW / 2 * STRIP + BN * 8 + NW * TN * 128 <= BYTES, "the epilogue's buffers fit a stage");
  float* cscale = (float*)(st1 + NW / 2 * STRIP);
  float* cbias = cscale + BN;
  int* zbuf = (int*)(cbias + BN) + wave * TN * 32;
  char* strip = (wave < NW / 2 ? st0 : st1) + wave % (NW / 2) * STRIP;
  if (threadIdx.x < BN) {
    cscale[threadIdx.x] = my_scale;
    cbias[threadIdx.x] = my_bias;
  }
  if constexpr (ZP) {
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const int z = zs[t] + __shfl_xor(zs[t], 32);
      if (half == 0) zbuf[t * 32 + r] = z;
    }
  }
  __syncthreads();
  const int wave_col = (vt0 * 16 + wn * TN * 32) / (SILU ? 2 : 1);
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    auto sums = [&](int t, int q) {
      i32x4_t v;
      i32x4_t z = {0, 0, 0, 0};
      if constexpr (ZP) z = *(const i32x4_t*)(zbuf + t * 32 + q * 8 + half * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = acc[m][t][q * 4 + i] - za[m] * z[i];
      return v;
    };
    auto scaled = [&](int t, int q) {
      const int c = (wn * TN + t) * 32 + q * 8 + half * 4;
      const f32x4_t cs = *(const f32x4_t*)(cscale + c), cb = *(const f32x4_t*)(cbias + c);
      const i32x4_t v = sums(t, q);
      f32x4_t y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = i8_scale(v[i], sa[m], cs[i], cb[i]);
      return y;
    };
    auto out4 = [&](int t, int q) {  // columns 8 q + 4 half .. + 3 of tile t's TC
      if (raw) return __builtin_bit_cast(f32x4_t, sums(t, q));
      f32x4_t y = scaled(t, q);
      if constexpr (SILU) {
        const f32x4_t u = scaled(t, q + 2);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = i8_silu(y[i]) * u[i];
      }
      return y;
    };
    // the strip's rows of `cols` columns of es bytes out, from column c0 on
    auto flush = [&](void* base, int64_t ld, int limit, int c0, int cols, int es) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int per = cols * es / 16;  // 16-byte pieces of a row
#pragma unroll
      for (int i = lane; i < 32 * per; i += 64) {
        const int row = i / per, piece = i % per;
        const int y = __shfl(yr[m], row), j = c0 + piece * (16 / es);
        const u32x4_t v = *(const u32x4_t*)(strip + row * PITCH + piece * 16);
        if (y < 0 || j >= limit) continue;
        char* dst = (char*)base + ((int64_t)y * ld + j) * es;
        if (j + 16 / es <= limit) {
          *(u32x4_any_t*)dst = v;
        } else if (es == 4) {
          for (int e = 0; e < 4 && j + e < limit; ++e) ((uint32_t*)dst)[e] = v[e];
        } else {
          for (int e = 0; e < 8 && j + e < limit; ++e) ((uint16_t*)dst)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    if (gridDim.y > 1) {  // dense: int32 partials, columns in the order of B's tiles
#pragma unroll
      for (int t = 0; t < TN; ++t) {
#pragma unroll
        for (int q = 0; q < 4; ++q) *(i32x4_t*)(strip + r * PITCH + (q * 8 + half * 4) * 4) = sums(t, q);
        flush(p.partial + (int64_t)blockIdx.y * p.M * p.vcols, p.vcols, p.vcols, vt0 * 16 + (wn * TN + t) * 32, 32,
              4);
      }
    } else if (p.otype == QDG_O_BF16) {
#pragma unroll
      for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int q = 0; q < TC / 8; ++q)
          *(u32x2_t*)(strip + r * PITCH + (t * TC + q * 8 + half * 4) * 2) = i8_bf16x4(out4(t, q));
      flush(p.Y, p.ldy, p.cols, wave_col, TN * TC, 2);
    } else {
#pragma unroll
      for (int t = 0; t < TN; ++t) {
#pragma unroll
        for (int q = 0; q < TC / 8; ++q) *(f32x4_t*)(strip + r * PITCH + (q * 8 + half * 4) * 4) = out4(t, q);
        flush(p.Y, p.ldy, p.cols, wave_col + t * TC, TC, 4);
      }
    }
  }
}

template <int WM, int WN, int TM, int TN, int NS, bool MOE>
hipError_t launch_tile(const I8Args& a, bool silu, int m_blocks, int split, hipStream_t s, int n_limit = 0) {
  constexpr int BN = 32 * TN * WN, THREADS = 64 * WM * WN;
  const int n_blocks = n_limit ? n_limit : (a.vcols - a.vt_first * 16 + BN - 1) / BN;
  int64_t blocks = (int64_t)m_blocks * n_blocks;
  int m_run = 1;
  if (MOE) {
    // runs of up to 8 blocks while every XCD still gets two (the blocks in
    // use are at least num_pairs / block_m). T = 4096, 64-row blocks, gate+up:
    // runs of 1 2.64 ms, 2 2.11, 4 2.08, 8 2.06, 16 2.05, 32 2.33
    while (m_run < 8 && a.num_pairs / a.block_m >= 32 * m_run) m_run *= 2;
    blocks = (int64_t)(m_blocks + 8 * m_run - 1) / (8 * m_run) * (8 * m_run) * n_blocks;
  }
  if (blocks * THREADS >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks, split), dim3(THREADS), 0, s, a, m_blocks, n_blocks, m_run);
    return hipGetLastError();
  };
  if (silu)
    return a.a_zeros ? go(gemm_i8_tile_kernel<WM, WN, TM, TN, NS, true, true, MOE>)
                     : go(gemm_i8_tile_kernel<WM, WN, TM, TN, NS, true, false, MOE>);
  return a.a_zeros ? go(gemm_i8_tile_kernel<WM, WN, TM, TN, NS, false, true, MOE>)
                   : go(gemm_i8_tile_kernel<WM, WN, TM, TN, NS, false, false, MOE>);
}

// ------------------------------------------------------------- dense choice
// A dense product runs the rows kernel or one of five tiles, its K perhaps
// split over workgroups, by a time model: R rounds of tiles over G groups
// take R (G group + round) + 3 us. group: measured microseconds for a
// 128-byte group of K with the tiles filling the card once, and (many) where
// several rounds of tiles no longer find their operands in L2; round: a
// round's prologue and epilogue. Measured in microseconds, bf16 output, no
// zero points, operands from memory (the model's rates are of cached ones):
//                        64x64  128x64  128x128  128x256  256x256
//    256 x  4096 x 4096   13.4    17.3     22.0     32.6     53.6
//    256 x 14336 x 4096   36.9    35.1     26.9     35.9     55.3
//   1024 x  4096 x 4096   37.2    32.3     24.2     33.5     54.1
//   2048 x  4096 x 4096   70.7    63.5     47.1     38.1     55.5
//   4096 x  4096 x 4096  124.4   122.9     89.8     74.9     63.5
// A split adds a second kernel and the partials' traffic (64 x 512 x 16384,
// 64 x 64: 25.4 us whole, 7.6 + 4.2 us in eight).
enum I8Kernel { I8_ROWS, I8_64X64, I8_128X64, I8_128X128, I8_128X256, I8_256X256 };
struct I8Tile {
  I8Kernel kernel;
  int bm, bn;
  float group, many, round;
};
constexpr I8Tile kI8Tiles[] = {{I8_64X64, 64, 64, 0.19f, 0.27f, 1.f},
                               {I8_128X64, 128, 64, 0.33f, 0.36f, 1.5f},
                               {I8_128X128, 128, 128, 0.53f, 0.56f, 3.f},
                               {I8_128X256, 128, 256, 1.07f, 1.07f, 4.f},
                               {I8_256X256, 256, 256, 1.67f, 1.67f, 4.f}};
constexpr int kCus = 256;

int64_t i8_rounds(int64_t tiles) { return (tiles + kCus - 1) / kCus; }

float i8_rounds_us(const I8Tile& t, int64_t tiles, int64_t groups) {
  const int64_t rounds = i8_rounds(tiles);
  return (float)rounds * ((float)groups * (rounds > 1 ? t.many : t.group) + t.round);
}

// The tiles (kernel, its K in split parts) of the columns up to n_main column
// blocks, and with n_main > 0 another tile (rest, whole K) behind them.
struct I8Choice {
  I8Kernel kernel, rest;
  int split, n_main;
};

I8Choice choose_dense(int64_t M, int64_t vcols, int64_t k) {
  if (M <= 16 && vcols < 8192) return {I8_ROWS, I8_ROWS, 1, 0};
  const int64_t groups = (k + 127) / 128;
  I8Choice best = {I8_64X64, I8_64X64, 1, 0};
  float best_us = 0.f;
  for (const I8Tile& t : kI8Tiles) {
    const int64_t m_blocks = (M + t.bm - 1) / t.bm, n_blocks = (vcols + t.bn - 1) / t.bn, tiles = m_blocks * n_blocks;
    for (int s = 1; s <= 8; s *= 2) {
      if (s > 1 && (tiles * s > kCus || groups < 8 * s)) break;
      float us = i8_rounds_us(t, tiles * s, (groups + s - 1) / s) + 3.f;
      if (s > 1) us += 5.f + (float)(M * vcols * s) * 8e-6f / 4.f;  // written and read at about 4 TB/s
      if (best_us == 0.f || us < best_us) {
        best_us = us;
        best = {t.kernel, t.kernel, s, 0};
      }
    }
    // Whole rounds of this tile, and what the last round would hold of it in
    // smaller ones: 4096 x 4608 x 4096 is 1.1 rounds of 256 x 256 tiles (118 us
    // in two, 91 with the rest in 128 x 64, zero points); 4096 x 14336 x 4096
    // 3.5 (266, 265 us)
    const int64_t full = tiles / kCus, n_main = m_blocks > 0 ? full * kCus / m_blocks : 0;
    if (tiles % kCus == 0 || n_main < 1 || n_main >= n_blocks) continue;
    for (const I8Tile& r : kI8Tiles) {
      const int64_t rest = (M + r.bm - 1) / r.bm * ((vcols - n_main * t.bn + r.bn - 1) / r.bn);
      const float us = i8_rounds_us(t, m_blocks * n_main, groups) + i8_rounds_us(r, rest, groups) + 5.f;
      if (us < best_us) {
        best_us = us;
        best = {t.kernel, r.kernel, 1, (int)n_main};
      }
    }
  }
  return best;
}

hipError_t launch_dense_tile(I8Kernel kernel, const I8Args& a, bool silu, int split, hipStream_t s, int n_limit) {
  switch (kernel) {
    case I8_64X64: return launch_tile<2, 2, 1, 1, 4, false>(a, silu, (a.M + 63) / 64, split, s, n_limit);
    case I8_128X64: return launch_tile<4, 2, 1, 1, 4, false>(a, silu, (a.M + 127) / 128, split, s, n_limit);
    case I8_128X128: return launch_tile<2, 4, 2, 1, 4, false>(a, silu, (a.M + 127) / 128, split, s, n_limit);
    case I8_128X256: return launch_tile<2, 4, 2, 2, 3, false>(a, silu, (a.M + 127) / 128, split, s, n_limit);
    default: return launch_tile<2, 4, 4, 2, 2, false>(a, silu, (a.M + 255) / 256, split, s, n_limit);
  }
}

}  // namespace

int64_t gemm_i8_vcols(int64_t cols, bool silu) { return (cols + 15) / 16 * 16 * (silu ? 2 : 1); }

int gemm_i8_split(int64_t M, int64_t vcols, int64_t k) { return choose_dense(M, vcols, k).split; }

// Within 64 rows every tile's counts stay as they are, and a choice's time
// grows with its split times the rows: the split taken never grows there, so
// that equal splits at both ends are the split of all rows between.
int64_t gemm_i8_max_partial_rows(int64_t M, int64_t vcols, int64_t k) {
  // two parts of eight groups at least, and of the largest tiles, must fit one round
  const I8Tile& large = kI8Tiles[std::size(kI8Tiles) - 1];
  const int64_t limit = k > 15 * 128 ? kCus / 2 / ((vcols + large.bn - 1) / large.bn) * large.bm : 0;
  auto rows_of = [&](int64_t m) {
    const int64_t split = gemm_i8_split(m, vcols, k);
    return split > 1 ? split * m : 0;
  };
  int64_t most = 0;
  for (int64_t lo = 1, hi; lo <= std::min(M, limit); lo = hi + 1) {
    hi = std::min({(lo + 63) / 64 * 64, M, limit});
    if (lo <= 16 && hi > 16) hi = 16;  // up to here perhaps the rows kernel
    most = std::max(most, rows_of(hi));
    const int at_end = gemm_i8_split(hi, vcols, k);
    if (gemm_i8_split(lo, vcols, k) == at_end) continue;
    for (int64_t m = lo; m < hi && gemm_i8_split(m, vcols, k) != at_end; ++m) most = std::max(most, rows_of(m));
  }
  return most;
}

I8Instance gemm_i8_instance(int64_t M, int64_t vcols, int64_t k) {
  const I8Choice c = choose_dense(M, vcols, k);
  I8Instance r = {16, 16, c.split, vcols, 0, 0};  // the rows kernel: 16 columns a workgroup
  for (const I8Tile& t : kI8Tiles) {
    if (t.kernel == c.kernel) {
      r.block_m = t.bm;
      r.block_n = t.bn;
      if (c.n_main > 0) r.columns = (int64_t)c.n_main * t.bn;
    }
    if (c.n_main > 0 && t.kernel == c.rest) {
      r.rest_m = t.bm;
      r.rest_n = t.bn;
    }
  }
  return r;
}

hipError_t launch_gemm_i8(const I8Args& a, bool silu, hipStream_t s) {
  const I8Choice c = choose_dense(a.M, a.vcols, a.k);
  if (c.kernel == I8_ROWS) {
    const dim3 grid((unsigned)((a.cols + 15) / 16));
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(64 * kRowWaves), 0, s, a);
      return hipGetLastError();
    };
    if (silu) return a.a_zeros ? go(gemm_i8_rows_kernel<true, true>) : go(gemm_i8_rows_kernel<true, false>);
    return a.a_zeros ? go(gemm_i8_rows_kernel<false, true>) : go(gemm_i8_rows_kernel<false, false>);
  }
  hipError_t e = launch_dense_tile(c.kernel, a, silu, c.split, s, c.n_main);
  if (e != hipSuccess) return e;
  if (c.n_main > 0) {
    I8Args rest = a;
    for (const I8Tile& t : kI8Tiles)
      if (t.kernel == c.kernel) rest.vt_first = c.n_main * (t.bn / 16);
    return launch_dense_tile(c.rest, rest, silu, 1, s, 0);
  }
  if (c.split <= 1) return e;
  const int64_t threads = (int64_t)a.M * ((a.cols + 3) / 4);
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (silu)
    hipLaunchKernelGGL(gemm_i8_reduce_kernel<true>, grid, dim3(256), 0, s, a, c.split);
  else
    hipLaunchKernelGGL(gemm_i8_reduce_kernel<false>, grid, dim3(256), 0, s, a, c.split);
  return hipGetLastError();
}

// Expert blocks: the tile holds the block's rows. Two to four workgroups of
// four waves share a CU, so that one's prologue and epilogue run under the others'
// loops. Measured (E = 256, top-8; gate+up 4096 x 7168, down 7168 x 2048):
//   16 rows  32 x 128 tiles half filled (fragments straight from memory: T = 64 down 640 us against 535)
//   32 rows  32 x 256: T = 512 down 646 us, 32 x 128 720, 32 x 64 759
//   64 rows  64 x 256, four waves and two stages: T = 4096 gate+up 2.06 ms; eight waves and
//            four stages (one workgroup a CU) 2.28, 64 x 128 2.35
//   128 rows 128 x 128: T = 4096 gate+up 2.29 ms, 128 x 256 2.43
hipError_t launch_moe_gemm_i8(const I8Args& a, bool silu, int m_blocks, hipStream_t s) {
  switch (a.block_m) {
    case 16: return launch_tile<1, 4, 1, 1, 4, true>(a, silu, m_blocks, 1, s);
    case 32: return launch_tile<1, 4, 1, 2, 2, true>(a, silu, m_blocks, 1, s);
    case 64: return launch_tile<1, 4, 2, 2, 2, true>(a, silu, m_blocks, 1, s);
    case 128: return launch_tile<2, 2, 2, 2, 2, true>(a, silu, m_blocks, 1, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qdg
