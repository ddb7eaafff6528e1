// Low-rank adapters beside a shared projection (qdg_lora): for the rows m of
// adapter a, Y[m][j] += scale_a * sum_r T[m][r] B_a[j][r],
// T[m][r] = sum_k X[m][k] A_a[slice(j)][r][k].
//
// Two kernels over tiles of MT x 16 rows grouped by adapter: `down` leaves T as
// binary32 partials (K split over workgroups, and over the waves of each),
// `up` adds them in order and meets B. Few rows: bound by A and B; many: by Y's
// way there and back. T enters the second product as bf16 terms, T = hi + lo
// with an error of 2^-18 of T (binary32 Y: a third term, 2^-27): 16 ranks are
// one 16 x 16 x 32 MFMA, hi in its first 16 K values, lo in the others, the same
// B beside both.
#include "qdg_codes.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_2_t;
typedef __attribute__((ext_vector_type(4), aligned(4))) uint32_t u32x4_4_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;

__device__ __forceinline__ uint32_t to_bf16_pair(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Eight neighbouring bf16 values at any element.
__device__ __forceinline__ u32x4_t load_x8(const uint16_t* p) {
  const u32x4_2_t v = *(const u32x4_2_t*)p;
  return u32x4_t{v.x, v.y, v.z, v.w};
}

// Values i .. i + 7 of a row, 0 from value `end` on, by elements.
__device__ __forceinline__ u32x4_t load_x8_cut(const uint16_t* p, int i, int end) {
  uint32_t d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    d[j] = i + 2 * j < end ? p[i + 2 * j] : 0u;
    if (i + 2 * j + 1 < end) d[j] |= (uint32_t)p[i + 2 * j + 1] << 16;
  }
  return u32x4_t{d[0], d[1], d[2], d[3]};
}

// The adapter of a 16-row tile and its rank (0: nothing to add).
struct Adapter {
  int id, rank;
};
__device__ __forceinline__ Adapter adapter_of(const LoraArgs& a, int tile) {
  if (tile * 16 >= *a.num_padded) return {0, 0};
  const int e = a.block_adapter[tile * 16 / a.block_m];
  if (e < 0 || e >= a.num_adapters) return {0, 0};
  return {e, a.ranks ? min(max(a.ranks[e], 0), a.rank) : a.rank};
}
// Row l % 16 of a tile, -1: padding.
__device__ __forceinline__ int row_of(const LoraArgs& a, int tile) {
  const int r = a.sorted_ids[tile * 16 + (threadIdx.x & 15)];
  return r >= 0 && r < a.M ? r : -1;
}

// T of MT x 16 rows and NT x 16 columns (ranks of one or several slices):
// workgroup = (rows, columns, K part), its four waves share the K part. Padding
// rows read a row that is there and ranks behind the adapter's last one its
// last: what comes of them is not used.
template <int MT, int NT>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a, int row_tiles, int col_tiles) {
  __shared__ f32x4_t sum[4][MT * NT][64];
  const int groups = a.num_slices * a.rank_pad / 16;
  const int tile0 = (int)(blockIdx.x % row_tiles) * MT, g0 = (int)(blockIdx.x / row_tiles % col_tiles) * NT;
  const int part = blockIdx.x / row_tiles / col_tiles;
  const Adapter ad = adapter_of(a, tile0);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane >> 4, q = lane & 15;
  const int per = a.rank_pad / 16;
  const uint16_t* w[NT];
  bool any = false;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int g = min(g0 + u, groups - 1), slice = g / per, r0 = g % per * 16;
    any |= g0 + u < groups && r0 < ad.rank;
    w[u] = a.A + (((int64_t)ad.id * a.num_slices + slice) * a.rank + max(min(r0 + q, ad.rank - 1), 0)) * a.k;
  }
  if (!any) return;  // the whole workgroup
  const uint16_t* x[MT];
  int first = 0;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    int r = row_of(a, tile0 + m);
    const uint64_t there = __ballot(r >= 0);
    if (there) first = __builtin_amdgcn_readlane(r, __builtin_ctzll(there));
    x[m] = a.X + (int64_t)(r >= 0 ? r : first) * a.ldx;
  }
  // K in steps of 32; this wave takes steps [s0, s1) of the whole ones
  const int steps = a.k / 32, waves = 4 * a.split, me = part * 4 + wave;
  const int s0 = (int)((int64_t)steps * me / waves), s1 = (int)((int64_t)steps * (me + 1) / waves);
  f32x4_t acc[MT][NT] = {};
  u32x4_t xf[2][MT], wf[2][NT];
  auto fetch = [&](int s, u32x4_t(&xv)[MT], u32x4_t(&wv)[NT]) {
    const int k = s * 32 + c * 8;
#pragma unroll
    for (int u = 0; u < NT; ++u) wv[u] = load_x8(w[u] + k);
#pragma unroll
    for (int m = 0; m < MT; ++m) xv[m] = load_x8(x[m] + k);
  };
  auto multiply = [&](const u32x4_t(&xv)[MT], const u32x4_t(&wv)[NT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int u = 0; u < NT; ++u) acc[m][u] = mfma_bf16(wv[u], xv[m], acc[m][u]);
  };
  if (s0 < s1) {
    fetch(s0, xf[0], wf[0]);
    int s = s0;
    for (; s + 2 <= s1; s += 2) {
      fetch(s + 1, xf[1], wf[1]);
      multiply(xf[0], wf[0]);
      fetch(min(s + 2, s1 - 1), xf[0], wf[0]);
      multiply(xf[1], wf[1]);
    }
    if (s < s1) multiply(xf[0], wf[0]);
  }
  if (a.k % 32 && me == waves - 1) {  // the last step is cut
#pragma unroll
    for (int u = 0; u < NT; ++u) wf[0][u] = load_x8_cut(w[u], steps * 32 + c * 8, a.k);
#pragma unroll
    for (int m = 0; m < MT; ++m) xf[0][m] = load_x8_cut(x[m], steps * 32 + c * 8, a.k);
    multiply(xf[0], wf[0]);
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int u = 0; u < NT; ++u) sum[wave][m * NT + u][lane] = acc[m][u];
  __syncthreads();
  // a lane's value: row l % 16, ranks 4 (l / 16) .. + 3 of its group
  for (int f = wave; f < MT * NT; f += 4) {
    const int m = f / NT, g = g0 + f % NT;
    if (g >= groups) continue;
    const f32x4_t v = (sum[0][f][lane] + sum[1][f][lane]) + (sum[2][f][lane] + sum[3][f][lane]);
    f32x4_t* p = (f32x4_t*)a.partial + (((int64_t)part * row_tiles * MT + tile0 + m) * groups + g) * 64 + lane;
    *p = v;
  }
}

// What its bf16 rounding leaves of t; 0 where that is an infinity or NaN, which stands for itself.
__device__ __forceinline__ float rest(float t, float rounded) {
  return fabsf(rounded) < __builtin_inff() ? t - rounded : 0.f;
}
__device__ __forceinline__ u32x4_t bf16x8(const float (&v)[8]) {
  return u32x4_t{to_bf16_pair(v[0], v[1]), to_bf16_pair(v[2], v[3]), to_bf16_pair(v[4], v[5]), to_bf16_pair(v[6], v[7])};
}
__device__ __forceinline__ void subtract(float (&v)[8], const u32x4_t& r) {
  const uint32_t d[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = rest(v[j], bf16_pair(d[j >> 1], j));
}

// Y: workgroup = (MT x 16 rows, `span` units of 64 columns of one slice), a
// wave takes every fourth unit. The MFMA's rows are columns of Y: row q of its
// tile u stands for column 16 (q / 4) + 4 u + q % 4 of the unit, so that a lane
// of the result holds 16 neighbouring columns of one row.
constexpr int kUnit = 64;
template <int MT, bool YF>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a, int row_tiles, int chunks, int span) {
  extern __shared__ u32x4_t terms[];  // [MT][rank step][hi, lo and, with YF, the third][64]
  constexpr int kTerms = YF ? 2 : 1;
  const int tile0 = (int)(blockIdx.x / chunks) * MT;
  int chunk = blockIdx.x % chunks;
  const Adapter ad = adapter_of(a, tile0);
  if (ad.rank == 0) return;
  int slice = 0, j0 = 0;
  for (;; ++slice) {
    const int len = (a.slice_end[slice] - j0 + kUnit * span - 1) / (kUnit * span);
    if (chunk < len) break;
    chunk -= len;
    j0 = a.slice_end[slice];
  }
  const int j1 = a.slice_end[slice];
  j0 += chunk * span * kUnit;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane >> 4, q = lane & 15;
  const int per = a.rank_pad / 16, groups = a.num_slices * per, steps = (ad.rank + 15) / 16;
  int row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) row[m] = row_of(a, tile0 + m);
  // T of this slice: a thread adds eight ranks of one row over the K parts
  const float scale = a.scales ? a.scales[ad.id] : 1.0f;
  for (int i = threadIdx.x; i < MT * steps * 32; i += 256) {
    const int l = i & 31, f = i >> 5, m = f / steps, s = f % steps, h = l >> 4;
    const f32x4_t* p = (const f32x4_t*)a.partial + (((int64_t)tile0 + m) * groups + slice * per + s) * 64 + 32 * h + (l & 15);
    const int64_t stride = (int64_t)row_tiles * MT * groups * 64;
    f32x4_t v0 = {}, v1 = {};
    for (int k = 0; k < a.split; ++k) {
      v0 += p[k * stride];
      v1 += p[k * stride + 16];
    }
    float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s * 16 + h * 8 + j < ad.rank ? v[j] * scale : 0.f;
    u32x4_t* t = terms + (m * steps + s) * kTerms * 64 + l;
    t[0] = bf16x8(v);
    subtract(v, t[0]);
    t[32] = bf16x8(v);
    if constexpr (YF) {
      subtract(v, t[32]);
      t[64] = bf16x8(v);
      t[96] = u32x4_t{0, 0, 0, 0};
    }
  }
  __syncthreads();
  const uint16_t* b = a.B + (int64_t)ad.id * a.n * a.rank;
  const bool whole = a.rank % 8 == 0;
  for (int unit = wave; unit < span; unit += 4) {
    const int col0 = j0 + unit * kUnit, col = col0 + 16 * c;
    if (col0 >= j1) break;
    f32x4_t acc[MT][4] = {};
    for (int s = 0; s < steps; ++s) {
      const int r = s * 16 + 8 * (c & 1);
      u32x4_t bf[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint16_t* p = b + (int64_t)min(col0 + 16 * (q >> 2) + 4 * u + (q & 3), j1 - 1) * a.rank;
        if (whole) {
          bf[u] = load_x8(p + min(r, a.rank - 8));
#pragma unroll
          for (int j = 0; j < 4; ++j) bf[u][j] &= r + 2 * j + 1 < ad.rank ? ~0u : r + 2 * j < ad.rank ? 0xFFFFu : 0u;
        } else {
          bf[u] = load_x8_cut(p, r, ad.rank);
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int k = 0; k < kTerms; ++k) {
          const u32x4_t tf = terms[((m * steps + s) * kTerms + k) * 64 + lane];
#pragma unroll
          for (int u = 0; u < 4; ++u) acc[m][u] = mfma_bf16(bf[u], tf, acc[m][u]);
        }
    }
    if (col >= j1) continue;
    const int rest = j1 - col;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (row[m] < 0) continue;
      if constexpr (YF) {
        float* y = (float*)a.Y + (int64_t)row[m] * a.ldy + col;
        if (rest >= 16) {
          u32x4_4_t v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = ((const u32x4_4_t*)y)[u];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[u][i] = bits_as<uint32_t>(bits_as<float>((uint32_t)v[u][i]) + acc[m][u][i]);
            ((u32x4_4_t*)y)[u] = v[u];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < rest) y[j] += acc[m][j >> 2][j & 3];
        }
      } else {
        uint16_t* y = (uint16_t*)a.Y + (int64_t)row[m] * a.ldy + col;
        if (rest >= 16) {
          u32x4_2_t v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) v[h] = ((const u32x4_2_t*)y)[h];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t d = v[h][j];
              const f32x4_t& s = acc[m][2 * h + (j >> 1)];
              v[h][j] = to_bf16_pair(bf16_pair(d, 0) + s[2 * (j & 1)], bf16_pair(d, 1) + s[2 * (j & 1) + 1]);
            }
            ((u32x4_2_t*)y)[h] = v[h];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (j < rest) y[j] = (uint16_t)to_bf16_pair(bf16_to_f32(y[j]) + acc[m][j >> 2][j & 3], 0.f);
        }
      }
    }
  }
}

int tiles_per_group(int block_m) { return block_m >= 64 ? 4 : block_m / 16; }

}  // namespace

int64_t lora_blocks(int64_t M, int64_t E, int block_m) {
  const int64_t d = M < E ? M : E;  // adapters that rows may have, a cut block each
  return d + (M - d) / block_m;
}

int lora_rank_pad(int rank) { return (rank + 15) / 16 * 16; }

// Parts of K: enough workgroups for 256 CUs twice, each wave with four steps of 32 at least.
int lora_split(int64_t tiles, int block_m, int columns, int64_t k) {
  const int64_t groups = tiles / tiles_per_group(block_m) * ((columns / 16 + 3) / 4), most = (k + 511) / 512;
  int64_t split = groups > 0 ? 512 / groups : 1;
  if (split > most) split = most;
  return (int)(split < 1 ? 1 : split);
}

namespace {

template <int MT, int NT>
hipError_t down(const LoraArgs& a, int64_t row_tiles, int64_t col_tiles, hipStream_t s) {
  hipLaunchKernelGGL((lora_down_kernel<MT, NT>), dim3((unsigned)(row_tiles * col_tiles * a.split)), dim3(256), 0, s, a,
                     (int)row_tiles, (int)col_tiles);
  return hipGetLastError();
}

template <int MT>
hipError_t both(const LoraArgs& a, hipStream_t s) {
  const int64_t row_tiles = (int64_t)a.blocks * (a.block_m / 16) / MT;
  const int groups = a.num_slices * a.rank_pad / 16, nt = groups < 4 ? groups : 4;
  const int64_t col_tiles = (groups + nt - 1) / nt;
  int64_t units = 0;
  for (int i = 0; i < a.num_slices; ++i) units += (a.slice_end[i] - (i ? a.slice_end[i - 1] : 0) + kUnit - 1) / kUnit;
  // units a workgroup: four waves of one, more while 2048 workgroups are left
  int64_t span = row_tiles * units / 2048 / 4 * 4;
  span = span < 4 ? 4 : span > 32 ? 32 : span;
  int64_t chunks = 0;
  for (int i = 0; i < a.num_slices; ++i)
    chunks += (a.slice_end[i] - (i ? a.slice_end[i - 1] : 0) + kUnit * span - 1) / (kUnit * span);
  if (row_tiles * col_tiles * a.split >= (1 << 24) || row_tiles * chunks >= (1 << 24)) return hipErrorInvalidConfiguration;
  hipError_t e;
  switch (nt) {
    case 1: e = down<MT, 1>(a, row_tiles, col_tiles, s); break;
    case 2: e = down<MT, 2>(a, row_tiles, col_tiles, s); break;
    case 3: e = down<MT, 3>(a, row_tiles, col_tiles, s); break;
    default: e = down<MT, 4>(a, row_tiles, col_tiles, s); break;
  }
  if (e != hipSuccess) return e;
  const size_t lds = (size_t)MT * (a.rank_pad / 16) * (a.yf32 ? 2 : 1) * 64 * sizeof(u32x4_t);
  auto up = a.yf32 ? lora_up_kernel<MT, true> : lora_up_kernel<MT, false>;
  hipLaunchKernelGGL(up, dim3((unsigned)(row_tiles * chunks)), dim3(256), lds, s, a, (int)row_tiles, (int)chunks, (int)span);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  switch (tiles_per_group(a.block_m)) {
    case 1: return both<1>(a, s);
    case 2: return both<2>(a, s);
    default: return both<4>(a, s);
  }
}

}  // namespace qdg
