// Low-rank adapters beside a shared projection (qdg_lora): for the rows m of
// adapter a, Y[m][j] += scale_a * sum_r T[m][r] B_a[j][r],
// T[m][r] = sum_k X[m][k] A_a[slice(j)][r][k].
//
// Two kernels over 16-row tiles of the rows grouped by adapter: `down` leaves
// T as binary32 partials (K split over workgroups and waves), `up` adds them
// in order and meets B. Few rows: bound by A and B; many: by Y's way there and
// back. T enters the second product as two bf16 terms, T = hi + lo with an
// error of 2^-18 of T: 16 ranks are one 16 x 16 x 32 MFMA, hi in its first 16
// K values, lo in the others, the same B beside both.
#include "qdg_codes.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t u32x4_2_t;
typedef __attribute__((ext_vector_type(4), aligned(4))) float f32x4_4_t;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2_t;

__device__ __forceinline__ uint32_t to_bf16_pair(float lo, float hi) {
  const f32x2_t v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2_t));
}

// Eight neighbouring bf16 values from p + i on, 0 from value `end` of the row on.
__device__ __forceinline__ u32x4_t load_bf16x8(const uint16_t* p, int i, int end) {
  if (i + 8 <= end) {
    const u32x4_2_t v = *(const u32x4_2_t*)(p + i);
    return u32x4_t{v.x, v.y, v.z, v.w};
  }
  uint32_t d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    d[j] = i + 2 * j < end ? p[i + 2 * j] : 0u;
    if (i + 2 * j + 1 < end) d[j] |= (uint32_t)p[i + 2 * j + 1] << 16;
  }
  return u32x4_t{d[0], d[1], d[2], d[3]};
}

// What a tile of 16 rows is: its adapter, that adapter's rank (0: nothing to
// add), and the row of lane l % 16 (-1: padding).
struct Tile {
  int adapter, rank, row;
};
__device__ __forceinline__ Tile tile_of(const LoraArgs& a, int tile) {
  Tile t = {0, 0, -1};
  if (tile * 16 >= *a.num_padded) return t;
  const int e = a.block_adapter[tile * 16 / a.block_m];
  if (e < 0 || e >= a.num_adapters) return t;
  t.adapter = e;
  t.rank = a.ranks ? min(max(a.ranks[e], 0), a.rank) : a.rank;
  const int r = a.sorted_ids[tile * 16 + (threadIdx.x & 15)];
  t.row = r >= 0 && r < a.M ? r : -1;
  return t;
}

// T: workgroup = (tile, 16 ranks of a slice, K part), its four waves share the K part.
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a) {
  __shared__ float sum[4][64][4];
  const int cols = a.num_slices * a.rank_pad, groups = cols / 16, tiles = a.blocks * (a.block_m / 16);
  const int tile = blockIdx.x % tiles, group = blockIdx.x / tiles % groups, part = blockIdx.x / tiles / groups;
  const Tile t = tile_of(a, tile);
  const int slice = group * 16 / a.rank_pad, r0 = group * 16 % a.rank_pad;
  if (r0 >= t.rank) return;  // the whole workgroup
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane >> 4, r = r0 + (lane & 15);
  const uint16_t* x = a.X + (int64_t)max(t.row, 0) * a.ldx;
  const uint16_t* w = a.A + ((int64_t)t.adapter * a.num_slices + slice) * a.rank * a.k + (int64_t)min(r, a.rank - 1) * a.k;
  const int x_end = t.row >= 0 ? a.k : 0, w_end = r < t.rank ? a.k : 0;
  // K in steps of 32; this wave takes steps [s0, s1)
  const int steps = (a.k + 31) / 32, waves = 4 * a.split, me = part * 4 + wave;
  const int s0 = (int)((int64_t)steps * me / waves), s1 = (int)((int64_t)steps * (me + 1) / waves);
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int s = s0; s < s1; ++s)
    acc = mfma_bf16(load_bf16x8(w, s * 32 + c * 8, w_end), load_bf16x8(x, s * 32 + c * 8, x_end), acc);
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[wave][lane][i] = acc[i];
  __syncthreads();
  if (wave == 0) {  // lane: row l % 16, ranks r0 + 4 c + i
    float* p = a.partial + ((int64_t)part * tiles * 16 + tile * 16 + (lane & 15)) * cols + group * 16 + c * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = sum[0][lane][i] + sum[1][lane][i] + sum[2][lane][i] + sum[3][lane][i];
  }
}

// What its bf16 rounding leaves of t; 0 where that is an infinity or NaN, which stands for itself.
__device__ __forceinline__ float rest(float t, float rounded) {
  return fabsf(rounded) < __builtin_inff() ? t - rounded : 0.f;
}

// Y: wave = (tile, 64 columns of a slice). The MFMA's rows are columns of Y:
// row q of its tile u stands for column 16 (q / 4) + 4 u + q % 4, so that a
// lane of the result holds 16 neighbouring columns of one row.
constexpr int kUnit = 64;
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a, int units, int chunks) {
  const int tile = blockIdx.x / chunks;
  const Tile t = tile_of(a, tile);
  int unit = (blockIdx.x % chunks) * 4 + (threadIdx.x >> 6);
  if (t.rank == 0 || unit >= units) return;
  int slice = 0, j0 = 0;
  for (;; ++slice) {
    const int len = (a.slice_end[slice] - j0 + kUnit - 1) / kUnit;
    if (unit < len) break;
    unit -= len;
    j0 = a.slice_end[slice];
  }
  j0 += unit * kUnit;
  const int j1 = min(j0 + kUnit, a.slice_end[slice]);
  const int lane = threadIdx.x & 63, c = lane >> 4, q = lane & 15;
  const int cols = a.num_slices * a.rank_pad;
  const int64_t rows = (int64_t)a.blocks * a.block_m;
  const float scale = a.scales ? a.scales[t.adapter] : 1.0f;
  const float* p = a.partial + ((int64_t)tile * 16 + q) * cols + slice * a.rank_pad;
  const uint16_t* b = a.B + (int64_t)t.adapter * a.n * a.rank;
  f32x4_t acc[4] = {};
  for (int r0 = 0; r0 < t.rank; r0 += 16) {
    const int r = r0 + 8 * (c & 1);
    float v[8] = {};
    for (int s = 0; s < a.split; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += p[s * rows * cols + r + j];
    uint32_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lo = r + 2 * j < t.rank ? v[2 * j] * scale : 0.f, hi = r + 2 * j + 1 < t.rank ? v[2 * j + 1] * scale : 0.f;
      d[j] = to_bf16_pair(lo, hi);
      if (c >= 2) d[j] = to_bf16_pair(rest(lo, bf16_pair(d[j], 0)), rest(hi, bf16_pair(d[j], 1)));
    }
    const u32x4_t tf = {d[0], d[1], d[2], d[3]};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int col = j0 + 16 * (q >> 2) + 4 * u + (q & 3);
      const u32x4_t bf = load_bf16x8(b + (int64_t)min(col, a.n - 1) * a.rank, r, col < j1 ? t.rank : 0);
      acc[u] = mfma_bf16(bf, tf, acc[u]);
    }
  }
  const int col = j0 + 16 * c;
  if (t.row < 0 || col >= j1) return;
  if (a.yf32) {
    float* y = (float*)a.Y + (int64_t)t.row * a.ldy + col;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + 4 * u + i < j1) y[4 * u + i] += acc[u][i];
  } else {
    uint16_t* y = (uint16_t*)a.Y + (int64_t)t.row * a.ldy + col;
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (col + 4 * u + i < j1) y[4 * u + i] = (uint16_t)f32_to_bf16_rne(bf16_to_f32(y[4 * u + i]) + acc[u][i]);
  }
}

}  // namespace

int64_t lora_blocks(int64_t M, int64_t E, int block_m) {
  const int64_t d = M < E ? M : E;  // adapters that rows may have, a cut block each
  return d + (M - d) / block_m;
}

int lora_rank_pad(int rank) { return (rank + 15) / 16 * 16; }

// Parts of K: enough workgroups for 256 CUs twice, each with 8 steps of 32 a wave.
int lora_split(int64_t tiles, int columns, int64_t k) {
  const int64_t groups = tiles * (columns / 16), most = (k + 1023) / 1024;
  int64_t split = groups > 0 ? 512 / groups : 1;
  if (split > most) split = most;
  return (int)(split < 1 ? 1 : split);
}

int64_t lora_expand_units(const LoraArgs& a) {
  int64_t units = 0;
  for (int s = 0; s < a.num_slices; ++s) units += (a.slice_end[s] - (s ? a.slice_end[s - 1] : 0) + kUnit - 1) / kUnit;
  return units;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  const int64_t tiles = (int64_t)a.blocks * (a.block_m / 16);
  const int64_t groups = a.num_slices * a.rank_pad / 16;
  const int64_t units = lora_expand_units(a), chunks = (units + 3) / 4;
  if (tiles * groups * a.split >= (1 << 24) || tiles * chunks >= (1 << 24)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(lora_down_kernel, dim3((unsigned)(tiles * groups * a.split)), dim3(256), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(lora_up_kernel, dim3((unsigned)(tiles * chunks)), dim3(256), 0, s, a, (int)units, (int)chunks);
  return hipGetLastError();
}

}  // namespace qdg
