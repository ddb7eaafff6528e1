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
      float y = (float)g[i] * sa * p.b_scales[c];
      if (p.bias) y += p.bias[c];
      if constexpr (SILU) {
        float v = (float)u[i] * sa * p.b_scales[c + p.cols];
        if (p.bias) v += p.bias[c + p.cols];
        y = y / (1.0f + expf(-y)) * v;
      }
      out[i] = __builtin_bit_cast(uint32_t, y);
    }
  }
  if (p.otype == QDG_O_BF16) {
    uint16_t* dst = (uint16_t*)p.Y + yrow * p.ldy + j0;
#pragma unroll
    for (int i = 0; i < 4; ++i) out[i] = f32_to_bf16_rne(__builtin_bit_cast(float, out[i]));
    if (cnt == 4 && p.y_vec) {
      *(u32x2_t*)dst = u32x2_t{out[0] | out[1] << 16, out[2] | out[3] << 16};
    } else {
      for (int i = 0; i < 4; ++i)
        if (i < cnt) dst[i] = (uint16_t)out[i];
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

}  // namespace

int gemm_i8_split(int64_t M, int64_t n, int64_t k, bool silu) { return 1; }

hipError_t launch_gemm_i8(const I8Args& a, bool silu, int split, hipStream_t s) {
  hipError_t e;
  if (a.M <= 16)
    e = launch_rows<1, 2, 8, false>(a, silu, 1, split, s);
  else if (a.M <= 32)
    e = launch_rows<2, 2, 8, false>(a, silu, 1, split, s);
  else
    e = launch_rows<4, 2, 8, false>(a, silu, (a.M + 63) / 64, split, s);
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
  switch (block_m) {
    case 16: return launch_rows<1, 2, 8, true>(a, silu, m_blocks, 1, s);
    case 32: return launch_rows<2, 2, 8, true>(a, silu, m_blocks, 1, s);
    case 64: return launch_rows<4, 2, 8, true>(a, silu, m_blocks, 1, s);
    case 128: return launch_rows<8, 2, 4, true>(a, silu, m_blocks, 1, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace qdg
