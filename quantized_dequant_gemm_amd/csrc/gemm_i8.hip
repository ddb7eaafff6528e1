// int8 x int8 products over row-major operands (qdg_gemm_i8, qdg_moe_gemm_i8):
//
//   Y[m][j] = sa[m] * sb[j] * (sum_k A[m][k] B[j][k] - za[m] * sum_k B[j][k]) + bias[j]
//
// with both sums exact in int32 on v_mfma_i32_16x16x64_i8 and dot products.
// The weights are the MFMA's row operand, so a lane of the result holds four
// consecutive columns of one row of Y. With the SiLU*mul epilogue the 16-column tiles
// of B alternate between gate and up rows, so that a lane holds both halves.
#include <algorithm>

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
__device__ __forceinline__ float i8_scale(int acc, float sa, float sb, float bias) {
  return __builtin_fmaf((float)acc * sa, sb, bias);
}

__device__ __forceinline__ float i8_silu(float x) { return x / (1.0f + expf(-x)); }

// Four values to bf16 (v_cvt_pk_bf16_f32: nearest even).
__device__ __forceinline__ u32x2_t i8_bf16x4(f32x4_t v) {
  typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4_t;
  return __builtin_bit_cast(u32x2_t, __builtin_convertvector(v, bf16x4_t));
}

// Four consecutive outputs of one row: the integer sums (gate and up with
// SILU) of columns j0 .. j0 + 3 through scales, bias, epilogue and rounding.
template <bool SILU>
__device__ __forceinline__ void i8_finish(const I8Args& p, i32x4_t g, i32x4_t u, int64_t yrow, int arow, int expert,
                                          int j0) {
  if (j0 >= p.cols) return;
  const int cnt = min(4, p.cols - j0);
  uint32_t out[4];
  if (p.otype == QDG_O_I32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = (uint32_t)g[i];
  } else {
    const float sa = p.a_scales[arow];
    const int64_t col = (int64_t)expert * p.n + j0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = col + min(i, cnt - 1);
      float y = i8_scale(g[i], sa, p.b_scales[c], p.bias ? p.bias[c] : 0.f);
      if constexpr (SILU) {
        y = i8_silu(y) * i8_scale(u[i], sa, p.b_scales[c + p.cols], p.bias ? p.bias[c + p.cols] : 0.f);
      }
      out[i] = __builtin_bit_cast(uint32_t, y);
    }
  }
  if (p.otype == QDG_O_BF16) {
    uint16_t* dst = (uint16_t*)p.Y + yrow * p.ldy + j0;
    const u32x2_t h = i8_bf16x4(__builtin_bit_cast(f32x4_t, u32x4_t{out[0], out[1], out[2], out[3]}));
    if (cnt == 4 && p.y_vec) {
      *(u32x2_t*)dst = h;
    } else {
      for (int i = 0; i < 4; ++i)
        if (i < cnt) dst[i] = (uint16_t)(h[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    uint32_t* dst = (uint32_t*)p.Y + yrow * p.ldy + j0;
    if (cnt == 4 && p.y_vec) {
      *(u32x4_t*)dst = u32x4_t{out[0], out[1], out[2], out[3]};
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

// Few rows: fragments straight from memory, the K range split over the KW
// waves of a workgroup (and over gridDim.y workgroups through int32
// partials). MT 16-row tiles, NT 16-column tiles.
template <int MT, int NT, int KW, bool SILU, bool ZP, bool MOE>
__global__ __launch_bounds__(64 * KW) void gemm_i8_rows_kernel(const I8Args p, int n_blocks) {
  constexpr int TILES = MT * NT;
  __shared__ i32x4_t red[KW * TILES * 64];
  __shared__ int zred[KW][NT][16];
  const int lane = threadIdx.x & 63, r = lane & 15, c = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mb = blockIdx.x / n_blocks, nb = blockIdx.x % n_blocks;
  int expert = 0;
  if constexpr (MOE) {
    if (mb * MT * 16 >= *p.num_padded) return;
    expert = p.block_expert[mb];
    if ((unsigned)expert >= (unsigned)p.num_experts) return;
  }
  const int8_t* ap[MT];
  const int8_t* bp[NT];
  int yrow[MT], arow[MT];  // yrow < 0: no row
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int row = mb * MT * 16 + mt * 16 + r;
    if constexpr (MOE) {
      const int id = p.sorted_ids[row];
      const bool real = (unsigned)id < (unsigned)p.num_pairs;
      yrow[mt] = real ? id : -1;
      arow[mt] = real ? (p.a_per_pair ? id : id / p.top_k) : 0;
    } else {
      yrow[mt] = row < p.M ? row : -1;
      arow[mt] = min(row, p.M - 1);
    }
    ap[mt] = p.A + (int64_t)arow[mt] * p.lda + 16 * c;
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    int first, rows;
    i8_tile<SILU>(p, nb * NT + nt, first, rows);
    bp[nt] = p.B + ((int64_t)expert * p.n + (rows > 0 ? first + min(r, rows - 1) : 0)) * p.ldb + 16 * c;
  }
  i32x4_t acc[MT][NT];
  int zs[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    zs[nt] = 0;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) acc[mt][nt] = i32x4_t{0, 0, 0, 0};
  }
  const int steps = (p.k + 63) / 64, full = p.k / 64;
  const int parts = gridDim.y * KW, part = blockIdx.y * KW + wave;
  const int s0 = (int)((int64_t)steps * part / parts), s1 = (int)((int64_t)steps * (part + 1) / parts);
#pragma unroll 1
  for (int s = s0; s < min(s1, full); ++s) {
    u32x4_t a[MT], b[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) b[nt] = *(const u32x4_t*)(bp[nt] + s * 64);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) a[mt] = *(const u32x4_t*)(ap[mt] + s * 64);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (ZP) zs[nt] = i8_sum16(b[nt], zs[nt]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[mt][nt] = mfma_i8(b[nt], a[mt], acc[mt][nt]);
    }
  }
  if (s1 > full && s0 < s1) {  // the step that the row's end cuts
    u32x4_t a[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) a[mt] = i8_load_tail(ap[mt] - 16 * c, full * 64 + 16 * c, p.k);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const u32x4_t b = i8_load_tail(bp[nt] - 16 * c, full * 64 + 16 * c, p.k);
      if constexpr (ZP) zs[nt] = i8_sum16(b, zs[nt]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[mt][nt] = mfma_i8(b, a[mt], acc[mt][nt]);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) red[(wave * TILES + mt * NT + nt) * 64 + lane] = acc[mt][nt];
    if constexpr (ZP) {
      int z = zs[nt];
      z += __shfl_xor(z, 16);
      z += __shfl_xor(z, 32);
      if (c == 0) zred[wave][nt][r] = z;
    }
  }
  __syncthreads();
  constexpr int PER = SILU ? 2 : 1, UNITS = TILES / PER;
  for (int un = wave; un < UNITS; un += KW) {
    const int mt = un / (NT / PER), nt = un % (NT / PER) * PER;
    i32x4_t v[2] = {};
    int yr = -1, ar = 0;
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (m == mt) {
        yr = yrow[m];
        ar = arow[m];
      }
#pragma unroll
    for (int h = 0; h < PER; ++h) {
#pragma unroll
      for (int w = 0; w < KW; ++w) v[h] += red[(w * TILES + mt * NT + nt + h) * 64 + lane];
      if constexpr (ZP) {
        const int za = p.a_zeros[ar];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int z = 0;
#pragma unroll
          for (int w = 0; w < KW; ++w) z += zred[w][nt + h][4 * c + i];
          v[h][i] -= za * z;
        }
      }
    }
    if (yr < 0) continue;
    const int j0 = (nb * NT + nt) / PER * 16 + 4 * c;
    if (gridDim.y > 1) {
#pragma unroll
      for (int h = 0; h < PER; ++h) {
        int32_t* dst = p.partial + ((int64_t)blockIdx.y * p.M + yr) * p.n + h * p.cols + j0;
        for (int i = 0; i < 4; ++i)
          if (j0 + i < p.cols) dst[i] = v[h][i];
      }
    } else {
      i8_finish<SILU>(p, v[0], v[1], yr, ar, expert, j0);
    }
  }
}

// The partials of a split product, added and finished: one thread per row and
// four columns of Y.
template <bool SILU>
__global__ __launch_bounds__(256) void gemm_i8_reduce_kernel(const I8Args p, int split) {
  const int64_t quads = (p.cols + 3) / 4;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= quads * p.M) return;
  const int row = (int)(t / quads), j0 = (int)(t % quads) * 4;
  i32x4_t v[2] = {};
  for (int s = 0; s < split; ++s)
#pragma unroll
    for (int h = 0; h < (SILU ? 2 : 1); ++h) {
      const int32_t* src = p.partial + ((int64_t)s * p.M + row) * p.n + h * p.cols + j0;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[h][i] += j0 + i < p.cols ? src[i] : 0;
    }
  i8_finish<SILU>(p, v[0], v[1], row, row, 0, j0);
}

template <int MT, int NT, int KW, bool MOE>
hipError_t launch_rows(const I8Args& a, bool silu, int m_blocks, int split, hipStream_t s) {
  const int tiles = (a.cols + 15) / 16 * (silu ? 2 : 1);
  const int n_blocks = (tiles + NT - 1) / NT;
  const int64_t blocks = (int64_t)m_blocks * n_blocks;
  if (blocks * 64 * KW >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, split);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(64 * KW), 0, s, a, n_blocks);
    return hipGetLastError();
  };
  if (silu)
    return a.a_zeros ? go(gemm_i8_rows_kernel<MT, NT, KW, true, true, MOE>)
                     : go(gemm_i8_rows_kernel<MT, NT, KW, true, false, MOE>);
  return a.a_zeros ? go(gemm_i8_rows_kernel<MT, NT, KW, false, true, MOE>)
                   : go(gemm_i8_rows_kernel<MT, NT, KW, false, false, MOE>);
}

// ------------------------------------------------------------- LDS tiles
// Many rows: a BM x BN tile of Y per workgroup, 32 x 32 MFMA tiles, K in
// groups of 128 bytes through NS stages of LDS. A stage holds the rows of A
// and B as they are stored (128 bytes a row), copied by direct global -> LDS
// loads of 16 bytes a lane; the chunk of 16 bytes at slot j of row r is chunk
// j ^ f(r), so that the 16-byte fragment reads of 8 (or 16) neighbouring rows fall on
// different banks without padding.
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
// row `len` bytes long.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t i8_rows_rsrc(const int8_t* base, int64_t row, int64_t rows,
                                                              int64_t ld, int64_t len) {
  int64_t left = (rows - 1 - row) * ld + len;
  left = left < 0 ? 0 : left > 0xFFFFFFFFll ? 0xFFFFFFFFll : left;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(base + (left > 0 ? row * ld : 0)), (short)0,
                                           (int)(uint32_t)left, 0x00020000);
}

// Copies FROM .. TO - 1 of group g into one stage (every wave issues the same
// number). Buffer loads, because the compiler tracks them apart from LDS
// reads; a global load to LDS in flight makes it wait for every LDS read
// where one would do.
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
    if (ZP && m == 0) zs[t] = i8_sum16(f.b[t], zs[t]);
    acc[m][t] = mfma_i8_32(f.b[t], f.a[m], acc[m][t]);
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
  constexpr int MF = TM * TN, H = MF / 2;
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

template <int WM, int WN, int TM, int TN, int NS, bool SILU, bool ZP, bool MOE>
__global__ __launch_bounds__(64 * WM * WN) void gemm_i8_tile_kernel(const I8Args p, int m_blocks, int n_blocks) {
  constexpr int NW = WM * WN, BM = 32 * TM * WM, BN = 32 * TN * WN, BYTES = (BM + BN) * 128;
  constexpr int LOADS = (BM + BN) / 8 / NW, TAG = ((WM * 8 + WN) * 8 + TM) * 64 + TN * 8 + SILU * 4 + ZP * 2 + MOE;
  static_assert((BM + BN) / 8 % NW == 0, "every wave issues the same number of copies");
  static_assert(NS == 2 || NS == 3, "two or three stages");
  static_assert(NS * BYTES <= 160 * 1024, "stages exceed LDS");
  __shared__ __attribute__((aligned(1024))) char st0[BYTES];
  __shared__ __attribute__((aligned(1024))) char st1[BYTES];
  __shared__ __attribute__((aligned(1024))) char st2[NS == 3 ? BYTES : 16];
  char* const stage[3] = {st0, st1, st2};
  const int lane = threadIdx.x & 63, r = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;

  int mb, nb;
  if constexpr (MOE) {
    moe_tile_order(n_blocks, mb, nb);
    if (mb >= m_blocks) return;  // the grid covers whole groups of 8 blocks
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
  int expert = 0;
  if constexpr (MOE) {
    if (mb * BM >= *p.num_padded) return;
    expert = p.block_expert[mb];
    if ((unsigned)expert >= (unsigned)p.num_experts) return;
  }
  // 16-column tiles of B in the order the epilogue wants (gate and up tiles
  // alternate with SILU)
  const int vt0 = nb * (BN / 16);
  I8Src<LOADS> src;
  const int64_t k16 = (p.k + 15) / 16 * 16;
#pragma unroll
  for (int q = 0; q < LOADS; ++q) {
    const int i = q * NW + wave;  // rows 8 i .. 8 i + 7 of the stage: A, then B
    const uint32_t chunk = (uint32_t)((lane & 7) ^ (lane >> 3) ^ (i & 1)) * 16u;
    if (i < BM / 8) {
      if constexpr (MOE) {
        const int id = p.sorted_ids[mb * BM + i * 8 + (lane >> 3)];
        const int ar = (unsigned)id < (unsigned)p.num_pairs ? (p.a_per_pair ? id : id / p.top_k) : 0;
        src.rsrc[q] = i8_rows_rsrc(p.A, 0, p.M, p.lda, k16);  // at most 4 GiB (checked by the host)
        src.off[q] = (uint32_t)ar * (uint32_t)p.lda + chunk;
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
  const int groups = (p.k + 127) / 128;
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
    i8_load_stage<0, LOADS, LOADS, NW, TAG>(stage[q], src, wave, min(q, groups - 1));
  constexpr int LEFT = LOADS * (NS - 1);
  __builtin_amdgcn_s_waitcnt((LEFT & 15) | (7 << 4) | (15 << 8) | ((LEFT >> 4) << 14));
  asm volatile("s_barrier" ::: "memory");
  I8Frag<TM, TN> f0, f1;
  i8_frag_load(f0, st0, a_lane, b_lane, at[0]);
  const int full = p.k / 128;  // groups that need no mask
  int g = 0;
  for (; g + NS <= full; g += NS) {
#pragma unroll
    for (int cur = 0; cur < NS; ++cur)
      i8_group<LOADS, NW, TM, TN, LOADS*(NS - 2), ZP, false, TAG + (1 << 16)>(
          stage[cur], stage[(cur + 1) % NS], src, wave, g + cur, min(g + cur + NS, groups - 1), a_lane, b_lane, at,
          half, p.k, f0, f1, acc, zs);
  }
  // the remaining groups, the last one cut at k
#pragma unroll
  for (int cur = 0; cur < NS; ++cur)
    if (g + cur < groups)
      i8_group<LOADS, NW, TM, TN, 0, ZP, true, TAG + (1 << 17)>(
          stage[cur], stage[(cur + 1) % NS], src, wave, g + cur, groups - 1, a_lane, b_lane, at, half, p.k, f0, f1,
          acc, zs);
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
  const bool raw = p.otype == QDG_O_I32;
  if (!raw)
    for (int c = threadIdx.x; c < BN; c += 64 * NW) {
      int first, rows;
      i8_tile<SILU>(p, vt0 + c / 16, first, rows);
      const int64_t at = (int64_t)expert * p.n + (rows > 0 ? first + min(c % 16, rows - 1) : 0);
      cscale[c] = p.b_scales[at];
      cbias[c] = p.bias ? p.bias[at] : 0.f;
    }
  if constexpr (ZP) {
#pragma unroll
    for (int t = 0; t < TN; ++t) {
      const int z = zs[t] + __shfl_xor(zs[t], 32);
      if (half == 0) zbuf[t * 32 + r] = z;
    }
  }
  __syncthreads();
  constexpr int TC = SILU ? 16 : 32;  // columns of Y from a 32-column tile
  const int wave_col = (vt0 * 16 + wn * TN * 32) / (SILU ? 2 : 1);
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int grow = mb * BM + (wm * TM + m) * 32 + r;
    int yr = grow, ar = min(grow, p.M - 1);
    bool real = grow < p.M;
    if constexpr (MOE) {
      yr = p.sorted_ids[grow];
      real = (unsigned)yr < (unsigned)p.num_pairs;
      ar = !real ? 0 : p.a_per_pair ? yr : yr / p.top_k;
    }
    yr = real ? yr : -1;
    const int za = ZP ? p.a_zeros[ar] : 0;
    const float sa = raw ? 1.f : p.a_scales[ar];
    auto sums = [&](int t, int q) {
      i32x4_t v;
      i32x4_t z = {0, 0, 0, 0};
      if constexpr (ZP) z = *(const i32x4_t*)(zbuf + t * 32 + q * 8 + half * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = acc[m][t][q * 4 + i] - za * z[i];
      return v;
    };
    auto scaled = [&](int t, int q) {
      const int c = (wn * TN + t) * 32 + q * 8 + half * 4;
      const f32x4_t cs = *(const f32x4_t*)(cscale + c), cb = *(const f32x4_t*)(cbias + c);
      const i32x4_t v = sums(t, q);
      f32x4_t y;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = i8_scale(v[i], sa, cs[i], cb[i]);
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
    auto flush = [&](int c0, int cols, int es) {
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int per = cols * es / 16;  // 16-byte pieces of a row
#pragma unroll
      for (int i = lane; i < 32 * per; i += 64) {
        const int row = i / per, piece = i % per;
        const int y = __shfl(yr, row), j = c0 + piece * (16 / es);
        const u32x4_t v = *(const u32x4_t*)(strip + row * PITCH + piece * 16);
        if (y < 0 || j >= p.cols) continue;
        char* dst = (char*)p.Y + ((int64_t)y * p.ldy + j) * es;
        if (p.y_vec && j + 16 / es <= p.cols) {
          *(u32x4_t*)dst = v;
        } else if (es == 4) {
          for (int e = 0; e < 4 && j + e < p.cols; ++e) ((uint32_t*)dst)[e] = v[e];
        } else {
          for (int e = 0; e < 8 && j + e < p.cols; ++e) ((uint16_t*)dst)[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };
    if (p.otype == QDG_O_BF16) {
#pragma unroll
      for (int t = 0; t < TN; ++t)
#pragma unroll
        for (int q = 0; q < TC / 8; ++q)
          *(u32x2_t*)(strip + r * PITCH + (t * TC + q * 8 + half * 4) * 2) = i8_bf16x4(out4(t, q));
      flush(wave_col, TN * TC, 2);
    } else {
#pragma unroll
      for (int t = 0; t < TN; ++t) {
#pragma unroll
        for (int q = 0; q < TC / 8; ++q) *(f32x4_t*)(strip + r * PITCH + (q * 8 + half * 4) * 4) = out4(t, q);
        flush(wave_col + t * TC, TC, 4);
      }
    }
  }
}

template <int WM, int WN, int TM, int TN, int NS, bool MOE>
hipError_t launch_tile(const I8Args& a, bool silu, int m_blocks, hipStream_t s) {
  constexpr int BN = 32 * TN * WN, THREADS = 64 * WM * WN;
  const int tiles = (a.cols + 15) / 16 * (silu ? 2 : 1);
  const int n_blocks = (tiles + BN / 16 - 1) / (BN / 16);
  const int64_t blocks = (int64_t)(MOE ? moe_grid_blocks(m_blocks) : m_blocks) * n_blocks;
  if (blocks * THREADS >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(THREADS), 0, s, a, m_blocks, n_blocks);
    return hipGetLastError();
  };
  if (silu)
    return a.a_zeros ? go(gemm_i8_tile_kernel<WM, WN, TM, TN, NS, true, true, MOE>)
                     : go(gemm_i8_tile_kernel<WM, WN, TM, TN, NS, true, false, MOE>);
  return a.a_zeros ? go(gemm_i8_tile_kernel<WM, WN, TM, TN, NS, false, true, MOE>)
                   : go(gemm_i8_tile_kernel<WM, WN, TM, TN, NS, false, false, MOE>);
}

}  // namespace

int gemm_i8_split(int64_t M, int64_t n, int64_t k, bool silu) { return 1; }

hipError_t launch_gemm_i8(const I8Args& a, bool silu, int split, hipStream_t s) {
  hipError_t e;
  if (a.M <= 16)
    e = launch_rows<1, 2, 8, false>(a, silu, 1, split, s);
  else if (a.M <= 32)
    e = launch_rows<2, 2, 8, false>(a, silu, 1, split, s);
  else if (a.M <= 64)
    e = launch_rows<4, 2, 8, false>(a, silu, 1, split, s);
  else if (a.M <= 1024)
    return launch_tile<2, 4, 2, 1, 3, false>(a, silu, (a.M + 127) / 128, s);
  else
    return launch_tile<2, 4, 4, 2, 2, false>(a, silu, (a.M + 255) / 256, s);
  if (e != hipSuccess || split <= 1) return e;
  const int64_t threads = (int64_t)a.M * ((a.cols + 3) / 4);
  const dim3 grid((unsigned)((threads + 255) / 256));
  if (silu)
    hipLaunchKernelGGL(gemm_i8_reduce_kernel<true>, grid, dim3(256), 0, s, a, split);
  else
    hipLaunchKernelGGL(gemm_i8_reduce_kernel<false>, grid, dim3(256), 0, s, a, split);
  return hipGetLastError();
}

hipError_t launch_moe_gemm_i8(const I8Args& a, bool silu, int block_m, int m_blocks, hipStream_t s) {
  // the tiles address A with 32 bits
  const bool far = (int64_t)a.M * a.lda > (int64_t)0xFFFF0000;
  if (far && block_m == 64) return launch_rows<4, 2, 8, true>(a, silu, m_blocks, 1, s);
  if (far && block_m == 128) return launch_rows<8, 2, 4, true>(a, silu, m_blocks, 1, s);
  switch (block_m) {
    case 16: return launch_rows<1, 2, 8, true>(a, silu, m_blocks, 1, s);
    case 32: return launch_rows<2, 2, 8, true>(a, silu, m_blocks, 1, s);
    case 64: return launch_tile<2, 4, 1, 2, 3, true>(a, silu, m_blocks, s);
    case 128: return launch_tile<2, 4, 2, 2, 3, true>(a, silu, m_blocks, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qdg
