// Low-rank adapters beside a shared projection (qdg_lora): for the rows m of
// adapter a, Y[m][j] += scale_a * sum_r T[m][r] B_a[j][r],
// T[m][r] = sum_k X[m][k] A_a[slice(j)][r][k].
//
// Two kernels over 16-row tiles of the rows grouped by adapter: `down` leaves T
// as binary32 partials (K split over workgroups, and over the waves of each),
// `up` (few rows) or `wide` (many) adds them in order and meets B. For the
// fewest rows `fused` does both. Few rows: bound by A, B and the chain of
// dependent loads; many: by Y's way there and back. T enters the second product
// with all its 24 bits, as three bf16 terms: 16 ranks are two 16 x 16 x 32 MFMAs,
// one with the first term in 16 of its K values and the second in the others,
// one with the third in 16, the same B beside all.
//
// ODD instances serve a rank that is no multiple of 8 or a k that is none of 64:
// their loads may end behind a row, or a tensor.
#include "qdg_codes.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

// A value that is the same for all lanes, in a scalar register: what follows
// from it is then computed once for the wave.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// Read-only here, so by a scalar load.
template <class T>
__device__ __forceinline__ T scalar_load(const T* p) {
  return *(const __attribute__((address_space(4))) T*)p;
}

// Eight neighbouring bf16 values at any element.
__device__ __forceinline__ u32x4_t load_x8(const uint16_t* p) {
  const u32x4_2_t v = *(const u32x4_2_t*)p;
  return u32x4_t{v.x, v.y, v.z, v.w};
}

// The first `count` of eight values, 0 behind them.
__device__ __forceinline__ u32x4_t keep(u32x4_t v, int count) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] &= 2 * j + 1 < count ? ~0u : 2 * j < count ? 0xFFFFu : 0u;
  return v;
}

// Loads of eight values of which only the first ones may be there: `last` is the
// last place in the tensor that has eight. A place behind it is read from there;
// `fix` then shifts it and leaves the first `count` values, 0 behind them. Apart,
// so that several loads are on their way before the first is looked at.
__device__ __forceinline__ u32x4_t load_cut(const uint16_t* p, const uint16_t* last, const uint16_t* base, int count) {
  if (last < base) {  // the same for all: a tensor of fewer than eight values
    uint32_t d[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      d[j] = 2 * j < count ? p[2 * j] : 0u;
      if (2 * j + 1 < count) d[j] |= (uint32_t)p[2 * j + 1] << 16;
    }
    return u32x4_t{d[0], d[1], d[2], d[3]};
  }
  return load_x8(p < last ? p : last);
}
__device__ __forceinline__ u32x4_t fix(u32x4_t v, const uint16_t* p, const uint16_t* last, const uint16_t* base, int count) {
  const int skip = count > 0 && last >= base && p > last ? (int)(p - last) : 0;  // below 8 where a value is wanted
  if (skip) {
    if (skip & 4) v = u32x4_t{v.z, v.w, 0, 0};
    if (skip & 2) v = u32x4_t{v.y, v.z, v.w, 0};
    if (skip & 1) v = u32x4_t{v.x >> 16 | v.y << 16, v.y >> 16 | v.z << 16, v.z >> 16 | v.w << 16, v.w >> 16};
  }
  return keep(v, count);
}

// The adapter of a tile's rows and its rank (0: nothing to add), in scalar registers.
struct Adapter {
  int id, rank;
};
__device__ __forceinline__ Adapter adapter_of(const LoraArgs& a, int tile0) {
  const int padded = scalar_load(a.num_padded), e = scalar_load(a.block_adapter + (tile0 >> a.block_shift));
  Adapter r;
  r.id = max(min(e, a.num_adapters - 1), 0);
  r.rank = a.rank;
  if (a.ranks) r.rank = min(max(scalar_load(a.ranks + r.id), 0), a.rank);
  if (tile0 * 16 >= padded || e != r.id) r.rank = 0;
  return r;
}
// Workgroups go to the 8 XCDs in turn. In a grid that is a multiple of 8 wide
// each XCD takes a run of the groups of `mt` tiles that hold rows, with all their
// columns and K parts, so that an adapter's A and B come into one L2 or two, not
// into all, and T's partials stay in theirs (one row, k = 14336, rank 16: 8.6
// against 11.6 us with its workgroups on all XCDs). A narrower grid is that of
// fewer than 8 groups with more workgroups each than an XCD has CUs: they are
// spread (one row of rank 64, 28672 columns 11.7 against 18 us). -1: nothing for
// this one.
__device__ __forceinline__ int tile_group(const LoraArgs& a, int mt) {
  const int groups = (scalar_load(a.num_padded) / 16 + mt - 1) / mt;
  if (gridDim.x % 8) return (int)blockIdx.x < groups ? (int)blockIdx.x : -1;
  const int each = (groups + 7) / 8, g = (int)(blockIdx.x % 8) * each + (int)(blockIdx.x / 8);
  return (int)(blockIdx.x / 8) < each && g < groups ? g : -1;
}

// Row i of the grouped order, -1: padding.
__device__ __forceinline__ int row_at(const LoraArgs& a, int i) {
  const int r = a.sorted_ids[i];
  return r >= 0 && r < a.M ? r : -1;
}

// ------------------------------------------------------------------ T
// Operand tiles of 16 rows come in by whole 128-byte lines: of a step of 64
// values lane l reads eight of row 8 j + l / 8 (j = 0, 1) from 8 (l % 8) on, so
// that eight neighbouring lanes have a line. (Straight into the MFMA's layout,
// neighbouring lanes would be in 16 different rows, a lane a clock on the way
// in: 2048 rows, k = 14336 took 51 us so, 41 by lines.) A wave turns them in LDS of its own, chunk x of row q at
// place x ^ (q % 8), so that eight neighbouring lanes meet eight places on both
// sides (x ^ (q / 2), sixteen places, is as fast: 2048 rows of rank 64, k = 14336
// 39.5 us both, 512 rows of rank 16 11.4 against 11.3 to 11.5).
constexpr int kTileBytes = 2048;

// The rows of X that a lane reads. Padding comes last in a tile, so a tile with
// any row has its first one, which padding reads; a tile of padding reads row 0.
__device__ __forceinline__ void x_rows(const LoraArgs& a, int tile, const uint16_t* (&p)[2]) {
  const int l = threadIdx.x & 63;
  int row[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) row[j] = a.sorted_ids[tile * 16 + 8 * j + (l >> 3)];
  const int first = uniform(row[0]), there = first >= 0 && first < a.M ? first : 0;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    p[j] = a.X + (int64_t)(row[j] >= 0 && row[j] < a.M ? row[j] : there) * a.ldx + 8 * (l & 7);
}

// A group of 16 ranks from r0 on of a slice: where it starts, and the places of
// the lane's rows there (k <= 2^20: 32 bits hold them); ranks behind the
// adapter's last one read that.
struct ARows {
  const uint16_t* base;
  uint32_t at[2];
};
__device__ __forceinline__ ARows a_rows(const LoraArgs& a, const Adapter& ad, int slice, int r0) {
  const int l = threadIdx.x & 63;
  ARows w;
  w.base = a.A + ((int64_t)ad.id * a.num_slices + slice) * a.rank * a.k;
#pragma unroll
  for (int j = 0; j < 2; ++j)
    w.at[j] = (uint32_t)max(min(r0 + 8 * j + (l >> 3), ad.rank - 1), 0) * (uint32_t)a.k + 8 * (l & 7);
  return w;
}

// Sums over K of MT x NT products of 16 x 16, K in steps of 64 from s0 to s1
// (ODD: and the cut one behind the last where `tail`), ST steps on their way.
// lds: (MT + NT) tiles of this wave.
template <int MT, int NT, int ST, bool ODD>
__device__ __forceinline__ void inner_sums(const LoraArgs& a, const uint16_t* const (&x)[MT][2], const ARows (&w)[NT],
                                           char* lds, int s0, int s1, bool tail, f32x4_t (&acc)[MT][NT]) {
  const int l = threadIdx.x & 63, c = l >> 4, q = l & 15;
  char* put = lds + (l >> 3) * 128 + ((l & 7) ^ (l >> 3)) * 16;
  const char* get = lds + q * 128 + ((2 * c) ^ (q & 7)) * 16;
  const char* get1 = lds + q * 128 + ((2 * c + 1) ^ (q & 7)) * 16;
  struct Step {
    u32x4_t x[MT][2], w[NT][2];
  } in[ST];
  auto fetch = [&](int s, Step& f) {
    const int k = min(s, s1 - 1) * 64;  // the same loads on every path: the waits count them
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int u = 0; u < NT; ++u) f.w[u][j] = load_x8(w[u].base + k + w[u].at[j]);
#pragma unroll
      for (int m = 0; m < MT; ++m) f.x[m][j] = load_x8(x[m][j] + k);
    }
  };
  auto turn = [&](const Step& f) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int u = 0; u < NT; ++u) *(u32x4_t*)(put + (MT + u) * kTileBytes + j * 1024) = f.w[u][j];
#pragma unroll
      for (int m = 0; m < MT; ++m) *(u32x4_t*)(put + m * kTileBytes + j * 1024) = f.x[m][j];
    }
  };
  auto multiply = [&]() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_t wf[NT];
#pragma unroll
      for (int u = 0; u < NT; ++u) wf[u] = *(const u32x4_t*)((h ? get1 : get) + (MT + u) * kTileBytes);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const u32x4_t xf = *(const u32x4_t*)((h ? get1 : get) + m * kTileBytes);
#pragma unroll
        for (int u = 0; u < NT; ++u) acc[m][u] = mfma_bf16(wf[u], xf, acc[m][u]);
      }
    }
  };
  if (s0 < s1) {
#pragma unroll
    for (int i = 0; i < ST; ++i) fetch(s0 + i, in[i]);
    for (int s = s0; s < s1; s += ST) {
#pragma unroll
      for (int i = 0; i < ST; ++i) {
        if (i > 0 && s + i >= s1) break;
        turn(in[i]);
        fetch(s + i + ST, in[i]);
        multiply();
      }
    }
  }
  if (ODD && tail) {
    const int k = a.k / 64 * 64, count = a.k - k - 8 * (l & 7);
    Step f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int u = 0; u < NT; ++u) f.w[u][j] = load_cut(w[u].base + k + w[u].at[j], a.A_last, a.A, count);
#pragma unroll
      for (int m = 0; m < MT; ++m) f.x[m][j] = load_cut(x[m][j] + k, a.X_last, a.X, count);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int u = 0; u < NT; ++u) f.w[u][j] = fix(f.w[u][j], w[u].base + k + w[u].at[j], a.A_last, a.A, count);
#pragma unroll
      for (int m = 0; m < MT; ++m) f.x[m][j] = fix(f.x[m][j], x[m][j] + k, a.X_last, a.X, count);
    }
    turn(f);
    multiply();
  }
}

// T of MT x 16 rows and NT x 16 columns (ranks of one or several slices):
// workgroup = (rows, columns, K part), its four waves share the K part. What
// padding rows read is not used. Two operand tiles of loads a step for each MFMA
// pair: the way in bounds it, not the matrix cores. In a kernel trace 4096 rows,
// k = 4096, two slices of 16 ranks take 16 us at least, 19 at the median (33 MB of
// X once: 1.7 to 2.1 TB/s), 2048 rows, k = 14336, 64 ranks 22 and 29 (63 MB from
// memory, 2.2 to 2.9 TB/s; each adapter's A again for each 32 rows, from L2).
template <int MT, int NT, bool ODD>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs a, int tiles, int wave_steps) {
  __shared__ u32x4_t lds[4 * (MT + NT) * kTileBytes / 16 > 4 * MT * NT * 64 ? 4 * (MT + NT) * kTileBytes / 16 : 4 * MT * NT * 64];
  const int groups = a.num_slices * a.rank_pad / 16;
  const int group = tile_group(a, MT);
  if (group < 0 || group * MT >= tiles) return;
  const int tile0 = group * MT, g0 = blockIdx.y * NT, part = blockIdx.z;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const uint16_t* x[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) x_rows(a, tile0 + m, x[m]);
  const Adapter ad = adapter_of(a, tile0);
  ARows w[NT];
  bool any = false;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    // the slice of column group g0 + u, and its first rank there
    int r0 = min(g0 + u, groups - 1) * 16, slice = 0;
    while (r0 >= a.rank_pad) {
      r0 -= a.rank_pad;
      ++slice;
    }
    any |= g0 + u < groups && r0 < ad.rank;
    w[u] = a_rows(a, ad, slice, r0);
  }
  if (!any) return;  // the whole workgroup
  const int steps = a.k / 64, me = part * 4 + wave;
  const int s0 = min(me * wave_steps, steps), s1 = min(s0 + wave_steps, steps);
  f32x4_t acc[MT][NT] = {};
  inner_sums<MT, NT, (MT + NT > 4 ? 2 : MT + NT > 2 ? 3 : 4), ODD>(
      a, x, w, (char*)lds + wave * (MT + NT) * kTileBytes, s0, s1, a.k % 64 && me == 4 * a.split - 1, acc);
  __syncthreads();
  f32x4_t* sum = (f32x4_t*)lds;  // [4][MT * NT][64]
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int u = 0; u < NT; ++u) sum[(wave * MT * NT + m * NT + u) * 64 + lane] = acc[m][u];
  __syncthreads();
  // a lane's value: row l % 16, ranks 4 (l / 16) .. + 3 of its group
  for (int f = wave; f < MT * NT; f += 4) {
    const int m = f / NT, g = g0 + f % NT;
    if (g >= groups) continue;
    const f32x4_t* v = sum + f * 64 + lane;
    const f32x4_t t = (v[0] + v[MT * NT * 64]) + (v[2 * MT * NT * 64] + v[3 * MT * NT * 64]);
    *((f32x4_t*)a.partial + (((int64_t)part * tiles + tile0 + m) * groups + g) * 64 + lane) = t;
  }
}

// ------------------------------------------------------------------ the terms of T
// The bf16 numbers that binary32 values begin with; what is left of them is exact.
__device__ __forceinline__ uint32_t head_pair(float lo, float hi) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}
__device__ __forceinline__ u32x4_t heads(const float (&v)[8]) {
  return u32x4_t{head_pair(v[0], v[1]), head_pair(v[2], v[3]), head_pair(v[4], v[5]), head_pair(v[6], v[7])};
}
__device__ __forceinline__ float tail(float t) {
  return t - __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, t) & 0xFFFF0000u);
}

// Eight ranks of a row of T as terms, in the places of the MFMAs' operands: the
// first for lane groups 0 and 1, the second for 2 and 3; the third for 0 and 1,
// one place of zeros for 2 and 3. Each term is cut off, not rounded: none is
// larger than T, so that no term or product of one overflows where T's does
// not. An infinity or NaN (quiet, as a product's result) is its own first term,
// with nothing left.
constexpr int kTerms = 97;
__device__ __forceinline__ void store_terms(u32x4_t* t, int l, float (&v)[8]) {
  t[l] = heads(v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fabsf(v[j]) < __builtin_inff() ? tail(v[j]) : 0.f;
  t[32 + l] = heads(v);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = tail(v[j]);
  t[64 + l] = heads(v);
  if (l == 0) t[96] = u32x4_t{0, 0, 0, 0};
}
__device__ __forceinline__ int third_place() {
  const int lane = threadIdx.x & 63;
  return lane < 32 ? 64 + lane : 96;
}

// The terms of MT tiles' T for one slice, from the partials: terms
// [MT][steps][kTerms]. A thread adds eight ranks of one row over the parts.
template <int MT>
__device__ __forceinline__ void terms_of(const LoraArgs& a, const Adapter& ad, int tile0, int tiles, int slice, int steps,
                                         u32x4_t* terms) {
  const int per = a.rank_pad / 16, groups = a.num_slices * per;
  const float scale = a.scales ? scalar_load(a.scales + ad.id) : 1.0f;
  const int64_t stride = (int64_t)tiles * groups * 64;
  for (int i = threadIdx.x; i < MT * steps * 32; i += 256) {
    const int l = i & 31, f = i >> 5, h = l >> 4;
    int m = 0, s = f;
    while (s >= steps) {
      s -= steps;
      ++m;
    }
    const f32x4_t* p = (const f32x4_t*)a.partial + (((int64_t)tile0 + m) * groups + slice * per + s) * 64 + 32 * h + (l & 15);
    f32x4_t v0 = {}, v1 = {};
    for (int k = 0; k < a.split; k += 8) {  // eight parts' loads in flight
      f32x4_t w0[8], w1[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const f32x4_t* pk = p + min(k + j, a.split - 1) * stride;
        w0[j] = pk[0];
        w1[j] = pk[16];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + j < a.split) {
          v0 += w0[j];
          v1 += w1[j];
        }
    }
    float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s * 16 + h * 8 + j < ad.rank ? v[j] * scale : 0.f;
    store_terms(terms + (m * steps + s) * kTerms, l, v);
  }
}

// ------------------------------------------------------------------ Y, few rows
constexpr int kUnit = 64;

// Sixteen bytes of Y, `piece` of them behind element `at`.
template <bool YF>
__device__ __forceinline__ u32x4_t load_piece(const void* y, int64_t at, int piece) {
  if constexpr (YF) {
    const u32x4_4_t v = ((const u32x4_4_t*)((const float*)y + at))[piece];
    return u32x4_t{v.x, v.y, v.z, v.w};
  } else {
    const u32x4_2_t v = ((const u32x4_2_t*)((const uint16_t*)y + at))[piece];
    return u32x4_t{v.x, v.y, v.z, v.w};
  }
}
template <bool YF>
__device__ __forceinline__ void store_piece(void* y, int64_t at, int piece, const u32x4_t& v) {
  if constexpr (YF) ((u32x4_4_t*)((float*)y + at))[piece] = v;
  else ((u32x4_2_t*)((uint16_t*)y + at))[piece] = v;
}
// `cut` elements of a piece by themselves.
template <bool YF>
__device__ __forceinline__ u32x4_t load_elements(const void* y, int64_t at, int cut) {
  uint32_t d[8];
#pragma unroll
  for (int j = 0; j < (YF ? 4 : 8); ++j) {
    d[j] = 0;
    if (j < cut) {
      if constexpr (YF) d[j] = ((const uint32_t*)y)[at + j];
      else d[j] = ((const uint16_t*)y)[at + j];
    }
  }
  if constexpr (YF) return u32x4_t{d[0], d[1], d[2], d[3]};
  else return u32x4_t{d[0] | d[1] << 16, d[2] | d[3] << 16, d[4] | d[5] << 16, d[6] | d[7] << 16};
}
template <bool YF>
__device__ __forceinline__ void store_elements(void* y, int64_t at, int cut, const u32x4_t& v) {
#pragma unroll
  for (int j = 0; j < (YF ? 4 : 8); ++j)
    if (j < cut) {
      if constexpr (YF) ((uint32_t*)y)[at + j] = v[j];
      else ((uint16_t*)y)[at + j] = (uint16_t)(v[j >> 1] >> (16 * (j & 1)));
    }
}
// A piece plus as many sums.
__device__ __forceinline__ u32x4_t add_f32(const u32x4_t& y, const f32x4_t& s) {
  return __builtin_bit_cast(u32x4_t, __builtin_bit_cast(f32x4_t, y) + s);
}
__device__ __forceinline__ u32x4_t add_bf16(const u32x4_t& y, const f32x4_t& s0, const f32x4_t& s1) {
  const uint32_t d[4] = {y.x, y.y, y.z, y.w};
  return u32x4_t{to_bf16_pair(bf16_pair(d[0], 0) + s0.x, bf16_pair(d[0], 1) + s0.y),
                 to_bf16_pair(bf16_pair(d[1], 0) + s0.z, bf16_pair(d[1], 1) + s0.w),
                 to_bf16_pair(bf16_pair(d[2], 0) + s1.x, bf16_pair(d[2], 1) + s1.y),
                 to_bf16_pair(bf16_pair(d[3], 0) + s1.z, bf16_pair(d[3], 1) + s1.w)};
}

// Sixteen columns of MT rows of Y as they were: whole pieces, or by elements
// where the slice ends.
template <int MT, bool YF>
struct OldY {
  static constexpr int kP = YF ? 4 : 2, kE = YF ? 4 : 8;  // pieces, elements a piece
  u32x4_t piece[MT][kP];
  __device__ __forceinline__ void load(const LoraArgs& a, const int (&row)[MT], int col, int cut) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (row[m] < 0) continue;
      const int64_t at = (int64_t)row[m] * a.ldy + col;
      if (cut >= 16) {
#pragma unroll
        for (int h = 0; h < kP; ++h) piece[m][h] = load_piece<YF>(a.Y, at, h);
      } else {
#pragma unroll
        for (int h = 0; h < kP; ++h) piece[m][h] = load_elements<YF>(a.Y, at + h * kE, cut - h * kE);
      }
    }
  }
  __device__ __forceinline__ void add_and_store(const LoraArgs& a, const int (&row)[MT], int col, int cut,
                                                const f32x4_t (&acc)[MT][4]) {
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (row[m] < 0) continue;
      const int64_t at = (int64_t)row[m] * a.ldy + col;
#pragma unroll
      for (int h = 0; h < kP; ++h) {
        u32x4_t v;
        if constexpr (YF) v = add_f32(piece[m][h], acc[m][h]);
        else v = add_bf16(piece[m][h], acc[m][2 * h], acc[m][2 * h + 1]);
        if (cut >= 16) store_piece<YF>(a.Y, at, h, v);
        else store_elements<YF>(a.Y, at + h * kE, cut - h * kE, v);
      }
    }
  }
};

// B of one step of 16 ranks for the four column tiles of a unit of 64 columns.
// The MFMA's rows are columns of Y: row q of its tile u stands for column
// 16 (q / 4) + 4 u + q % 4 of the unit, so that a lane of the result holds 16
// neighbouring columns of one row. Where 32 bits hold its places (64 columns of
// 256 ranks), from a base that is the wave's.
template <bool ODD>
struct BTile {
  const uint16_t* base;
  uint32_t at[4];
  int left;  // ranks from the lane's first one on
  u32x4_t v[4];
  __device__ __forceinline__ void place(const LoraArgs& a, const Adapter& ad, int col0, int j1, int s) {
    const int lane = threadIdx.x & 63, q = lane & 15, r = s * 16 + 8 * (lane >> 4 & 1);
    base = a.B + ((int64_t)ad.id * a.n + col0) * a.rank;
    left = ad.rank - r;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      at[u] = (uint32_t)min(16 * (q >> 2) + 4 * u + (q & 3), j1 - 1 - col0) * (uint32_t)a.rank +
              (uint32_t)(ODD ? r : min(r, a.rank - 8));
  }
  __device__ __forceinline__ void load(const LoraArgs& a) {
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = ODD ? load_cut(base + at[u], a.B_last, a.B, left) : load_x8(base + at[u]);
  }
  __device__ __forceinline__ void settle(const LoraArgs& a) {
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = ODD ? fix(v[u], base + at[u], a.B_last, a.B, left) : keep(v[u], left);
  }
};

// An infinite or NaN entry of B is to meet an inner sum's first term only: 0, a
// rest of 0 or one of the other sign beside it would make its product a NaN. So
// where a wave's sums hold a NaN it computes them again with finite_part(B)
// beside the other terms: CAREFUL.
__device__ __forceinline__ u32x4_t finite_part(u32x4_t v) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] &= ((v[j] & 0x7F80u) == 0x7F80u ? 0u : 0xFFFFu) | ((v[j] & 0x7F800000u) == 0x7F800000u ? 0u : 0xFFFF0000u);
  return v;
}
// Does any of a wave's sums hold a NaN? (The least magnitude of all does then.)
template <int N>
__device__ __forceinline__ bool any_nan(const f32x4_t (&acc)[N]) {
  float m = 0.f;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    m = least3(m, acc[u].x, acc[u].y);
    m = least3(m, acc[u].z, acc[u].w);
  }
  return __any(m != m);
}

template <int MT, bool CAREFUL>
__device__ __forceinline__ void multiply_b(const u32x4_t (&bf)[4], const u32x4_t* terms, int steps, int s,
                                           f32x4_t (&acc)[MT][4]) {
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const u32x4_t* t = terms + (m * steps + s) * kTerms;
    const u32x4_t tf = t[threadIdx.x & 63], third = t[third_place()];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const u32x4_t b = CAREFUL && (threadIdx.x & 32) ? finite_part(bf[u]) : bf[u];
      acc[m][u] = mfma_bf16(b, tf, acc[m][u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) acc[m][u] = mfma_bf16(CAREFUL ? finite_part(bf[u]) : bf[u], third, acc[m][u]);
  }
}

// A workgroup's columns: `width` of them (or fewer) in one slice.
struct Columns {
  int slice, j0, j1;  // from j0 on; the slice ends at j1
};
__device__ __forceinline__ Columns columns_of(const LoraArgs& a, int chunk, int width) {
  Columns c = {0, 0, a.slice_end[0]};
  while (c.j0 + (int64_t)chunk * width >= c.j1) {
    chunk -= (c.j1 - c.j0 + width - 1) / width;
    c.j0 = c.j1;
    c.j1 = a.slice_end[++c.slice];
  }
  c.j0 += chunk * width;
  return c;
}

// Y: workgroup = (MT x 16 rows, `span` units of 64 columns of one slice), a
// wave takes every fourth unit. 250 rows of 12 adapters, rank 64, 4100 columns of
// binary32 10 to 11 us in a kernel trace (14 MB): a workgroup or two a CU, each the
// chain of grouping, partials, terms, products, so latency bounds it.
template <int MT, bool YF, bool ODD>
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs a, int tiles) {
  const int span = a.span;
  extern __shared__ u32x4_t terms[];  // [MT][rank step][kTerms]
  const int group = tile_group(a, MT);
  if (group < 0 || group * MT >= tiles) return;
  const int tile0 = group * MT;
  const Adapter ad = adapter_of(a, tile0);
  if (ad.rank == 0) return;
  const Columns cs = columns_of(a, blockIdx.y, span * kUnit);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane >> 4, steps = (ad.rank + 15) / 16;
  int row[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) row[m] = row_at(a, (tile0 + m) * 16 + (lane & 15));
  // Y and the first step's B are asked for before T is added up, each next
  // step's B before a product (more ahead costs a wave a SIMD: 250 rows of rank
  // 64, binary32, 10 -> 16 us)
  OldY<MT, YF> old;
  BTile<ODD> b;
  int col0 = cs.j0 + wave * kUnit;
  auto ask = [&]() {
    b.place(a, ad, col0, cs.j1, 0);
    b.load(a);
    old.load(a, row, col0 + 16 * c, cs.j1 - col0 - 16 * c);
  };
  if (col0 < cs.j1) ask();
  terms_of<MT>(a, ad, tile0, tiles, cs.slice, steps, terms);
  __syncthreads();
  for (int unit = wave; unit < span && col0 < cs.j1; unit += 4) {
    if (unit != wave) ask();
    f32x4_t acc[MT][4] = {};
    for (int s = 0; s < steps; ++s) {
      BTile<ODD> now = b;
      if (s + 1 < steps) {
        b.place(a, ad, col0, cs.j1, s + 1);
        b.load(a);
      }
      now.settle(a);
      multiply_b<MT, false>(now.v, terms, steps, s, acc);
    }
    bool nan = false;
#pragma unroll
    for (int m = 0; m < MT; ++m) nan |= any_nan(acc[m]);
    if (nan) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[m][u] = f32x4_t{};
      for (int s = 0; s < steps; ++s) {
        b.place(a, ad, col0, cs.j1, s);
        b.load(a);
        b.settle(a);
        multiply_b<MT, true>(b.v, terms, steps, s, acc);
      }
    }
    old.add_and_store(a, row, col0 + 16 * c, cs.j1 - col0 - 16 * c, acc);
    col0 += 4 * kUnit;
  }
}

// Both products in one launch, for few rows: workgroup = (16 rows, 8 units of
// 64 columns of one slice). Its eight waves share K, then take a unit each.
// Every workgroup of a slice computes T anew: (16 NT + 16) k values of A and X,
// most of them from the caches, in place of a second launch and the partials'
// way through memory. The unit's B and Y are asked for before T is ready. One
// row, k = n = 4096, rank 16 6.8 us: the chain of the grouping's loads, a wave's
// 512 values of k and three joins; 64 rows of 48 adapters, 6144 columns 11.4 us
// (22 MB of A and B).
constexpr int kFusedWaves = 8;
template <int NT, bool YF, bool ODD>
__global__ __launch_bounds__(64 * kFusedWaves) void lora_fused_kernel(LoraArgs a, int tiles) {
  // a wave's row of sums is 16 bytes longer, so that eight threads that add one value find it in eight places
  constexpr int kSumRow = NT * 64 + 1, kIn = kFusedWaves * (1 + NT) * kTileBytes / 16;
  __shared__ u32x4_t lds[kIn > kFusedWaves * kSumRow ? kIn : kFusedWaves * kSumRow];
  __shared__ u32x4_t terms[NT * kTerms];
  // a tile's workgroups are on one XCD, whose L2 holds the adapter for all, while that has the CUs (grid_x)
  const int tile = blockIdx.x;
  if (tile >= tiles) return;
  const uint16_t* x[1][2];
  x_rows(a, tile, x[0]);
  const Adapter ad = adapter_of(a, tile);
  if (ad.rank == 0) return;
  const Columns cs = columns_of(a, blockIdx.y, kFusedWaves * kUnit);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane >> 4, steps = (ad.rank + 15) / 16;
  const int row[1] = {row_at(a, tile * 16 + (lane & 15))};
  const float scale = a.scales ? scalar_load(a.scales + ad.id) : 1.0f;
  ARows w[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) w[u] = a_rows(a, ad, cs.slice, u * 16);
  const int col0 = cs.j0 + wave * kUnit, col = col0 + 16 * c;
  const bool mine = col0 < cs.j1;
  OldY<1, YF> old;
  BTile<ODD> b[NT];
  if (mine) {
#pragma unroll
    for (int s = 0; s < NT; ++s) {
      b[s].place(a, ad, col0, cs.j1, s);
      b[s].load(a);
    }
    old.load(a, row, col, cs.j1 - col);
  }
  const int all = a.k / 64, each = (all + kFusedWaves - 1) / kFusedWaves, s0 = min(wave * each, all), s1 = min(s0 + each, all);
  f32x4_t t[1][NT] = {};
  inner_sums<1, NT, (NT == 1 ? 4 : 3), ODD>(a, x, w, (char*)lds + wave * (1 + NT) * kTileBytes, s0, s1,
                                            a.k % 64 && wave == kFusedWaves - 1, t);
  __syncthreads();
  f32x4_t* sum = (f32x4_t*)lds;  // [waves][kSumRow]
#pragma unroll
  for (int u = 0; u < NT; ++u) sum[wave * kSumRow + u * 64 + lane] = t[0][u];
  __syncthreads();
  // eight threads add the waves' sums of four ranks of a row; a value and the
  // one of 16 places on, eight ranks, meet in lanes 8 apart
  for (int i = threadIdx.x; i < steps * 64 * kFusedWaves; i += 64 * kFusedWaves) {
    const int k = i & 7, half = i >> 3 & 1, item = i >> 4, l = item & 31, s = item >> 5, h = l >> 4;
    f32x4_t v = sum[k * kSumRow + s * 64 + 32 * h + 16 * half + (l & 15)];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] += dpp<kXor1>(v[j]);     // lanes that differ in bit 0
      v[j] += dpp<kXor2>(v[j]);     // bit 1
      v[j] += dpp<kMirror8>(v[j]);  // a mirror of eight: bit 2
    }
    f32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = dpp<kMirror16>(v[j]);  // a mirror of sixteen: the other half
    if ((i & 15) == 0) {
      float r[8] = {v.x, v.y, v.z, v.w, o.x, o.y, o.z, o.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = s * 16 + h * 8 + j < ad.rank ? r[j] * scale : 0.f;
      store_terms(terms + s * kTerms, l, r);
    }
  }
  __syncthreads();
  if (!mine) return;
  f32x4_t acc[1][4] = {};
#pragma unroll
  for (int s = 0; s < NT; ++s) {
    if (s >= steps) break;
    b[s].settle(a);
    multiply_b<1, false>(b[s].v, terms, steps, s, acc);
  }
  if (any_nan(acc[0])) {
#pragma unroll
    for (int u = 0; u < 4; ++u) acc[0][u] = f32x4_t{};
#pragma unroll
    for (int s = 0; s < NT; ++s)
      if (s < steps) multiply_b<1, true>(b[s].v, terms, steps, s, acc);
  }
  old.add_and_store(a, row, col, cs.j1 - col, acc);
}

// ------------------------------------------------------------------ Y, many rows
// Workgroup = (64 rows, `span` units of 128 columns of one slice), a wave has 16
// of the rows. The MFMA's columns are columns of Y: column q of its tile u
// stands for 8 q + u of the unit (binary32 Y: 64 (u / 4) + 4 q + u % 4), so that
// a lane of the result holds 16 bytes of a row and 16 neighbouring lanes 256
// bytes in a line: Y comes and goes by whole lines. B's unit goes through LDS
// for the four waves, [rank step][column][16 ranks], 16 bytes more every eight
// columns (a third of the LDS cycles still conflict); the next unit's B and Y are
// on their way meanwhile. In a kernel trace 4096 rows, 28672 columns of bf16, rank
// 16 take 85 us at least, 100 at the median (433 MB of Y there and back and B: 4.3
// to 5.1 TB/s, HBM), 2048 rows, rank 64, 4096 columns 15 and 17 (39 MB, 2.4 to 2.7
// TB/s: two rounds of workgroups). Four waves a SIMD where 128 registers hold a
// step (gate-up 104 -> 97 us), three with four steps of B on their way, two and no
// more beside binary32 Y (gate-up of rank 16 195 against 204 us with three).
constexpr int kWide = 128, kBStep = kWide * 32 + kWide / 8 * 16;
template <int STEPS, bool YF>
constexpr int kWideWaves = YF ? 2 : STEPS == 4 ? 3 : 4;
template <int STEPS, bool YF, bool ODD>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(kWideWaves<STEPS, YF>, YF ? 2 : 8)))
void lora_wide_kernel(LoraArgs a, int tiles) {
  const int span = a.span;
  // one side with four steps: 42 KB let a third workgroup in (4096 rows, rank 64 35.6 against 36.7 us)
  constexpr int kSides = STEPS == 4 ? 1 : 2;
  __shared__ u32x4_t terms[4 * STEPS * kTerms];
  __shared__ u32x4_t lds[kSides][STEPS * kBStep / 16];
  constexpr int kP = YF ? 2 : 1, kE = YF ? 4 : 8;  // pieces of a lane's row, elements a piece
  constexpr int kB = YF ? 8 : STEPS <= 2 ? 2 : 4;  // column tiles at a time, as many as registers hold
  const int group = tile_group(a, 4);
  if (group < 0 || group * 4 >= tiles) return;
  const int tile0 = group * 4;
  const Adapter ad = adapter_of(a, tile0);
  if (ad.rank == 0) return;
  const Columns cs = columns_of(a, blockIdx.y, span * kWide);
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), c = lane >> 4, q = lane & 15;
  const int steps = (ad.rank + 15) / 16, units = min(span, (cs.j1 - cs.j0 + kWide - 1) / kWide);
  int row[4];  // of 4 c + i; -1: padding
#pragma unroll
  for (int i = 0; i < 4; ++i) row[i] = row_at(a, (tile0 + wave) * 16 + 4 * c + i);
  // a row's place in Y; worked out anew each time where 64 bits of each row would
  // be registers that spill (rank 32 26.3 against 26.7 us; rank 16 114 against 112.5)
  auto place = [&](int i) {
    if constexpr (STEPS > 1 && !YF) asm volatile("" : "+v"(row[i]));
    return (int64_t)row[i] * a.ldy + (YF ? 4 : 8) * q;
  };
  // B: a thread has eight ranks of a column in each step
  const int bc = threadIdx.x >> 1, bh = threadIdx.x & 1;
  u32x4_t bin[STEPS];
  const uint16_t* bp = nullptr;
  auto load_b = [&](int unit) {
    const int col = min(cs.j0 + unit * kWide + bc, cs.j1 - 1);
    bp = a.B + ((int64_t)ad.id * a.n + col) * a.rank;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * 16 + 8 * bh;
      bin[s] = ODD ? load_cut(bp + r, a.B_last, a.B, ad.rank - r) : load_x8(bp + min(r, a.rank - 8));
    }
  };
  auto put_b = [&](int side) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      const int r = s * 16 + 8 * bh;
      bin[s] = ODD ? fix(bin[s], bp + r, a.B_last, a.B, ad.rank - r) : keep(bin[s], ad.rank - r);
      *(u32x4_t*)((char*)lds[side] + s * kBStep + bc * 32 + (bc >> 3) * 16 + bh * 16) = bin[s];
    }
  };
  u32x4_t y[4][kP];
  auto load_y = [&](int unit) {
    const int col0 = cs.j0 + unit * kWide;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (row[i] < 0) continue;
      const int64_t at = place(i) + col0;
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        const int cut = cs.j1 - col0 - 64 * p - kE * q;
        if (cut >= kE) y[i][p] = load_piece<YF>(a.Y, at + 64 * p, 0);
        else y[i][p] = load_elements<YF>(a.Y, at + 64 * p, cut);
      }
    }
  };
  load_b(0);
  load_y(0);
  terms_of<4>(a, ad, tile0, tiles, cs.slice, steps, terms);
  put_b(0);
  __syncthreads();
  for (int unit = 0; unit < units; ++unit) {
    u32x4_t was[4][kP];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int p = 0; p < kP; ++p) was[i][p] = y[i][p];
    const bool more = unit + 1 < units;
    if (more) {
      load_b(unit + 1);
      load_y(unit + 1);
    }
    f32x4_t acc[8] = {};
    const char* bl = (const char*)lds[unit & (kSides - 1)] + (YF ? q * 128 + (q >> 1) * 16 : q * 272) + (c & 1) * 16;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      if (s >= steps) break;
      const u32x4_t* tt = terms + (wave * steps + s) * kTerms;
      const u32x4_t tf = tt[lane], third = tt[third_place()];
#pragma unroll
      for (int g = 0; g < 8; g += kB) {
        u32x4_t bf[kB];
#pragma unroll
        for (int u = 0; u < kB; ++u)
          bf[u] = *(const u32x4_t*)(bl + s * kBStep + (YF ? (g + u) / 4 * 8 * 272 + (g + u) % 4 * 32 : (g + u) * 32));
#pragma unroll
        for (int u = 0; u < kB; ++u) acc[g + u] = mfma_bf16(tf, bf[u], acc[g + u]);
#pragma unroll
        for (int u = 0; u < kB; ++u) acc[g + u] = mfma_bf16(third, bf[u], acc[g + u]);
      }
    }
    if (any_nan(acc)) {
#pragma unroll
      for (int u = 0; u < 8; ++u) acc[u] = f32x4_t{};
      for (int s = 0; s < steps; ++s) {
        const u32x4_t* tt = terms + (wave * steps + s) * kTerms;
        const u32x4_t tf = tt[lane], third = tt[third_place()];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const u32x4_t bf = *(const u32x4_t*)(bl + s * kBStep + (YF ? u / 4 * 8 * 272 + u % 4 * 32 : u * 32));
          const u32x4_t fin = finite_part(bf);
          acc[u] = mfma_bf16(tf, lane & 32 ? fin : bf, acc[u]);
          acc[u] = mfma_bf16(third, fin, acc[u]);
          __builtin_amdgcn_sched_barrier(0);  // one tile at a time: registers
        }
      }
    }
    const int col0 = cs.j0 + unit * kWide;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (row[i] < 0) continue;
      const int64_t at = place(i) + col0;
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        const int cut = cs.j1 - col0 - 64 * p - kE * q;
        const f32x4_t s0 = {acc[4 * p][i], acc[4 * p + 1][i], acc[4 * p + 2][i], acc[4 * p + 3][i]};
        u32x4_t v;
        if constexpr (YF) v = add_f32(was[i][p], s0);
        else v = add_bf16(was[i][p], s0, f32x4_t{acc[4][i], acc[5][i], acc[6][i], acc[7][i]});
        if (cut >= kE) store_piece<YF>(a.Y, at + 64 * p, 0, v);
        else store_elements<YF>(a.Y, at + 64 * p, cut, v);
      }
    }
    if (kSides == 1) __syncthreads();
    if (more) put_b((unit + 1) & (kSides - 1));
    __syncthreads();
  }
}

int tiles_per_group(int block_m) { return block_m >= 64 ? 4 : block_m / 16; }

}  // namespace

int64_t lora_blocks(int64_t M, int64_t E, int block_m) {
  const int64_t d = M < E ? M : E;  // adapters that rows may have, a cut block each
  return d + (M - d) / block_m;
}

namespace {

int64_t chunks_of(const LoraArgs& a, int64_t width) {
  int64_t chunks = 0;
  for (int i = 0; i < a.num_slices; ++i) chunks += (a.slice_end[i] - (i ? a.slice_end[i - 1] : 0) + width - 1) / width;
  return chunks;
}

int clamp(int64_t v, int64_t lo, int64_t hi) { return (int)(v < lo ? lo : v > hi ? hi : v); }

}  // namespace

void lora_choose(LoraArgs* a) {
  const int64_t tiles = (int64_t)a->blocks * (a->block_m / 16);
  a->rank_pad = (a->rank + 15) / 16 * 16;
  const int nt = a->rank_pad / 16, groups = a->num_slices * nt;
  // One launch where T, anew for every 512 columns, costs less than the second
  // launch and the partials, while all workgroups run at once. n = 4096, 1 row of
  // rank 8: k = 1024 5.2 against 6.8 us, k = 4096 6.8 against 7.0, k = 14336 12.5
  // against 8.5; rank 32: k = 1024 6.8 against 7.4, k = 2560 7.9 against 7.5, k =
  // 4096 9.1 against 7.6. Larger blocks gain up to a workgroup a CU (200 rows of 2
  // adapters, 2048 columns 7.5 against 9.3 us; 512 rows of 4, 4096 columns, which
  // need 352, 13.6 against 10.8). Of blocks of one tile, each its own adapter's, two
  // fit a CU up to 16 ranks and bf16 Y (64 rows of 48 adapters, 6144 columns 11.4
  // against 12.2 us, 608 workgroups of k = 4096 12.6 against 14.1); of binary32 Y or
  // more ranks one fits. Some blocks have no rows and leave at once: 344 at most are
  // 256 with rows (k = 4096, binary32 9.1 against 10.3 us, 376 of them 14.7 against
  // 11.1; rank 32, k = 2048 9.8 against 10.8, 13.5 against 11.5; from 450 on the two
  // differ by up to 12 % either way, one launch ahead at a short k).
  const int workgroups = a->block_m > 16 ? 256 : nt == 1 && !a->yf32 ? 640 : 352;
  a->fused = (nt + 1) * (int64_t)a->k <= 8192 && nt <= 2 &&
             tiles * chunks_of(*a, kFusedWaves * kUnit) <= workgroups;
  // Parts of K: 512 workgroups (two a CU) where there is that much, each wave
  // with two steps of 64 at least.
  const int mt = groups > 2 && tiles_per_group(a->block_m) > 2 ? 2 : tiles_per_group(a->block_m);
  a->split = clamp(512 / (tiles / mt * ((groups + 3) / 4)), 1, (a->k + 511) / 512);
  // Units of columns a workgroup: each adds up T anew, split * rank_pad * 256
  // bytes for 64 rows, beside 32 KB of a unit's Y there and back; so more units
  // the more there is to add up, while 256 workgroups are left, and more while
  // 1024 are (4096 rows, rank 32, k = n = 4096: 29.0 us with one unit, 26.3 so). Few
  // rows: a unit for each of four waves, more while 768 workgroups are left (16
  // rows of as many adapters, 28672 columns: 10.6 us with one unit, 9.1 so).
  // 64 rows at once, Y by whole lines, from 64-row blocks on: 4096 rows of rank
  // 16, k = 4096, n = 28672 147 against 113 us, rank 64, n = 4096 41 against 36
  // (more than 64 ranks are more registers than hold the next unit's B and Y).
  a->wide = tiles_per_group(a->block_m) == 4 && a->rank_pad <= 64;
  if (a->wide) {
    const int64_t all = tiles / 4 * chunks_of(*a, kWide), t = (a->split * a->rank_pad + 127) / 128;
    const int64_t most = all / 256, by_count = all / 1024;
    a->span = clamp(t > by_count ? (t < most ? t : most) : by_count, 1, 16);
  } else {
    a->span = clamp(tiles / (mt < 2 ? mt : 2) * chunks_of(*a, kUnit) / 768 / 4 * 4, 4, 32);
  }
}

namespace {

// The grid's width for groups of `each` workgroups (see tile_group).
int64_t grid_x(int64_t groups, int64_t each) { return groups < 8 && each > 32 ? groups : (groups + 7) / 8 * 8; }

// A launch holds fewer than 2^32 threads, and 65535 workgroups in y and z.
bool too_many(int64_t x, int64_t y, int64_t z, int threads) {
  return y > 65535 || z > 65535 || x * y * z >= ((int64_t)1 << 32) / threads;
}

template <bool ODD, int NT>
hipError_t fused_nt(const LoraArgs& a, hipStream_t s) {
  const int64_t tiles = (int64_t)a.blocks * (a.block_m / 16), y = chunks_of(a, kFusedWaves * kUnit), x = grid_x(tiles, y);
  if (too_many(x, y, 1, 64 * kFusedWaves)) return hipErrorInvalidConfiguration;
  auto kernel = a.yf32 ? lora_fused_kernel<NT, true, ODD> : lora_fused_kernel<NT, false, ODD>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)x, (unsigned)y), dim3(64 * kFusedWaves), 0, s, a, (int)tiles);
  return hipGetLastError();
}

template <bool ODD, int MT, int NT>
hipError_t down(const LoraArgs& a, int64_t tiles, int64_t col_tiles, hipStream_t s) {
  const int waves = 4 * a.split;
  const dim3 grid((unsigned)grid_x(tiles / MT, col_tiles * a.split), (unsigned)col_tiles, (unsigned)a.split);
  hipLaunchKernelGGL((lora_down_kernel<MT, NT, ODD>), grid, dim3(256), 0, s, a, (int)tiles, (a.k / 64 + waves - 1) / waves);
  return hipGetLastError();
}

template <bool ODD, int STEPS>
hipError_t wide(const LoraArgs& a, dim3 grid, int64_t tiles, hipStream_t s) {
  auto kernel = a.yf32 ? lora_wide_kernel<STEPS, true, ODD> : lora_wide_kernel<STEPS, false, ODD>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, (int)tiles);
  return hipGetLastError();
}

template <bool ODD, int MT>
hipError_t two(const LoraArgs& a, hipStream_t s) {
  const int64_t tiles = (int64_t)a.blocks * (a.block_m / 16);
  const int groups = a.num_slices * a.rank_pad / 16, nt = groups < 4 ? groups : 4;
  const int64_t col_tiles = (groups + nt - 1) / nt;
  constexpr int LT = MT < 2 ? MT : 2;  // row tiles where there are many columns: registers
  const int64_t y = chunks_of(a, (int64_t)a.span * (a.wide ? kWide : kUnit)), x = grid_x(tiles / (a.wide ? 4 : LT), y);
  if (too_many(tiles + 7, col_tiles, a.split, 256) || too_many(x, y, 1, 256)) return hipErrorInvalidConfiguration;
  hipError_t e;
  switch (nt) {
    case 1: e = down<ODD, MT, 1>(a, tiles, col_tiles, s); break;
    case 2: e = down<ODD, MT, 2>(a, tiles, col_tiles, s); break;
    case 3: e = down<ODD, LT, 3>(a, tiles, col_tiles, s); break;
    default: e = down<ODD, LT, 4>(a, tiles, col_tiles, s); break;
  }
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)x, (unsigned)y);
  if (a.wide) {
    if (a.rank_pad == 16) return wide<ODD, 1>(a, grid, tiles, s);
    return a.rank_pad == 32 ? wide<ODD, 2>(a, grid, tiles, s) : wide<ODD, 4>(a, grid, tiles, s);
  }
  const size_t lds = (size_t)LT * (a.rank_pad / 16) * kTerms * sizeof(u32x4_t);
  auto kernel = a.yf32 ? lora_up_kernel<LT, true, ODD> : lora_up_kernel<LT, false, ODD>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), lds, s, a, (int)tiles);
  return hipGetLastError();
}

template <bool ODD>
hipError_t launch(const LoraArgs& a, hipStream_t s) {
  if (a.fused) return a.rank_pad == 16 ? fused_nt<ODD, 1>(a, s) : fused_nt<ODD, 2>(a, s);
  switch (tiles_per_group(a.block_m)) {
    case 1: return two<ODD, 1>(a, s);
    case 2: return two<ODD, 2>(a, s);
    default: return two<ODD, 4>(a, s);
  }
}

}  // namespace

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
  return a.k % 64 || a.rank % 8 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace qdg
