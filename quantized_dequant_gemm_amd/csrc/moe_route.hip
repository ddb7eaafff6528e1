// Expert routing: scores, grouped top-k and weights of each token.
//
//   s = softmax(l) or sigmoid(l);  c = s + bias (or the order of l);
//   value of a group = largest c or sum of its two largest; the best groups
//   stay; top_k of what stays by c; w = s, renormalised, scaled.
//
// One wave per token, EPL consecutive experts per lane (one vector load).
// Each round takes the wave-wide largest key with six DPP maxima and finds
// its owner with ballots.
//
// A choice must not hang on binary32 rounding, yet binary64 scores for every
// expert and 64-bit reductions cost three times the whole of the rest
// (8192 x 256 grouped: 31 us). So a key is an interval [lo, up] around
// its binary32 value that holds the exact one: the largest lower bound m of a
// round leaves the experts with up >= m as candidates, nearly always one. Where
// there are more, and where the intervals of group values overlap at the border
// of what stays, the wave computes those keys in binary64. Without a bias the
// keys are the logits themselves, exact (lo = up).
//
// Bounds of the binary32 scores (with a factor of two or more to spare):
// exp by v_exp_f32 of x * log2(e) is off by at most 2^-23 + 1.5 |x| 2^-24
// relative; 1 / (1 + t) adds 2^-24 + 2^-23 and does not widen what t brings:
// sigmoid 2^-20 + |x| 2^-22. Softmax subtracts first (|d| 2^-24 more) and
// divides by a sum whose terms with mass have |d| below about ln(1024):
// 2^-19 + |d| 2^-22. Adding the bias rounds by 2^-24 of the key: 2^-23.
// The weights of the top_k are computed in binary64, one lane each.
#include <algorithm>

#include "qdg_device.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

constexpr double kNegInf64 = -__builtin_inf();
constexpr float kInf = __builtin_inff();
constexpr int kWavesPerBlock = 4;

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_f32(float v) {
  const int i = __builtin_bit_cast(int, v);
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(i, i, CTRL, ROW_MASK, 0xF, false));
}

// Largest value of the wave (NaN ignored), in every lane.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_f32<0x111, 0xF>(v));  // row_shr:1, 2, 4, 8: lane 15 of each row of 16
  v = fmaxf(v, dpp_f32<0x112, 0xF>(v));
  v = fmaxf(v, dpp_f32<0x114, 0xF>(v));
  v = fmaxf(v, dpp_f32<0x118, 0xF>(v));
  v = fmaxf(v, dpp_f32<0x142, 0xA>(v));  // row_bcast:15 into rows 1 and 3
  v = fmaxf(v, dpp_f32<0x143, 0xC>(v));  // row_bcast:31 into rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}

__device__ __forceinline__ double wave_sum(double v) {
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ float readlane_f32(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

__device__ __forceinline__ float logit_f32(uint16_t h, int ltype) {
  if (ltype == QDG_L_F16) return (float)__builtin_bit_cast(_Float16, h);
  return __builtin_bit_cast(float, (uint32_t)h << 16);
}

// The EPL values of one lane: one wide load where the row allows it (vec)
// and the lane's experts all exist; absent experts read as fill.
template <int EPL>
__device__ __forceinline__ void load_row(const void* row, int ltype, bool vec, int e0, int E, float fill,
                                         float (&x)[EPL]) {
  if (ltype == QDG_L_F32) {
    const float* p = (const float*)row + e0;
    if (vec && e0 + EPL <= E) {
      typedef __attribute__((ext_vector_type(EPL < 4 ? EPL : 4))) float V;
#pragma unroll
      for (int q = 0; q < EPL; q += 4) {
        if constexpr (EPL == 1) {
          x[0] = p[0];
        } else {
          const V v = *(const V*)(p + q);
#pragma unroll
          for (int i = 0; i < (EPL < 4 ? EPL : 4); ++i) x[q + i] = v[i];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) x[j] = e0 + j < E ? p[j] : fill;
    }
  } else {
    const uint16_t* p = (const uint16_t*)row + e0;
    if (vec && e0 + EPL <= E) {
      if constexpr (EPL == 1) {
        x[0] = logit_f32(p[0], ltype);
      } else {
        constexpr int W = EPL < 8 ? EPL / 2 : 4;
        typedef __attribute__((ext_vector_type(W))) uint32_t V;
#pragma unroll
        for (int q = 0; q < EPL; q += 2 * W) {
          const V v = *(const V*)(p + q);
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const uint32_t u = v[i];
            x[q + 2 * i] = logit_f32((uint16_t)u, ltype);
            x[q + 2 * i + 1] = logit_f32((uint16_t)(u >> 16), ltype);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) x[j] = e0 + j < E ? logit_f32(p[j], ltype) : fill;
    }
  }
}

__device__ __forceinline__ double sigmoid64(double x) { return 1.0 / (1.0 + exp(-x)); }

// The two largest of a pair of ordered pairs.
__device__ __forceinline__ void top2_merge(float& m1, float& m2, float o1, float o2) {
  const float lo = fminf(m1, o1);
  m1 = fmaxf(m1, o1);
  m2 = fmaxf(lo, fmaxf(m2, o2));
}

// What the rare binary64 decisions read again: one token's row (cached by
// then), so that they keep no registers of the common path alive.
struct Row {
  const void* logits;
  const float* bias;
  int ltype, score, E;
  float top;     // softmax: the largest logit
  double sum64;  // softmax: sum of exp(l - top)

  __device__ __forceinline__ float logit(int e) const {
    const float x = ltype == QDG_L_F32 ? ((const float*)logits)[e] : logit_f32(((const uint16_t*)logits)[e], ltype);
    return x != x ? -kInf : fminf(x, 3.402823466e+38f);
  }
  __device__ __forceinline__ double key64(int e) const {
    const float x = logit(e), b = bias ? bias[e] : 0.f;
    if (x == -kInf || !(b > -kInf)) return kNegInf64;
    return (score == QDG_SCORE_SIGMOID ? sigmoid64((double)x) : exp((double)x - (double)top) / sum64) + (double)b;
  }
  __device__ __forceinline__ void set_sum(int lane) {
    double s = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 64) {
      const float x = logit(e);
      s += x == -kInf ? 0.0 : exp((double)x - (double)top);
    }
    sum64 = wave_sum(s);
  }
};

// Which groups stay, decided on binary64 values (two groups' intervals
// overlap at the border): a bit for each group.
__device__ __forceinline__ uint64_t groups64(Row& row, const qdg_route_config& c, int lane) {
  const int G = c.num_groups, per = c.num_experts / G;
  if (row.score == QDG_SCORE_SOFTMAX) row.set_sum(lane);
  double mine = kNegInf64;  // lane g: the value of group g
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    double m1 = kNegInf64, m2 = kNegInf64;
#pragma unroll 1
    for (int i = lane; i < per; i += 64) {
      const double k = row.key64(g * per + i);
      m2 = fmax(m2, fmin(m1, k));
      m1 = fmax(m1, k);
    }
#pragma unroll 1
    for (int m = 32; m > 0; m >>= 1) {
      const double o1 = __shfl_xor(m1, m), o2 = __shfl_xor(m2, m);
      m2 = fmax(fmin(m1, o1), fmax(m2, o2));
      m1 = fmax(m1, o1);
    }
    if (lane == g) mine = c.group_score == QDG_GROUP_MAX || m2 == kNegInf64 ? m1 : m1 + m2;
  }
  int rank = 0;
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    const double o = __shfl(mine, g);
    rank += o > mine || (o == mine && g < lane);
  }
  return __ballot(lane < G && rank < c.topk_groups);
}

// The expert with the largest binary64 key among the candidates (bit j of
// cand: the lane's expert e0 + j), equal ones the lowest.
__device__ __forceinline__ int best64(Row& row, uint32_t cand, int e0, int lane) {
  if (row.score == QDG_SCORE_SOFTMAX) row.set_sum(lane);
  double best = kNegInf64;
  int at = 1 << 30;
  for (; cand; cand &= cand - 1) {
    const int e = e0 + __builtin_ctz(cand);
    const double k = row.key64(e);
    if (at == 1 << 30 || k > best) {
      best = k;
      at = e;
    }
  }
#pragma unroll 1
  for (int d = 32; d > 0; d >>= 1) {
    const double ob = __shfl_xor(best, d);
    const int oa = __shfl_xor(at, d);
    if (oa != 1 << 30 && (at == 1 << 30 || ob > best || (ob == best && oa < at))) {
      best = ob;
      at = oa;
    }
  }
  return __builtin_amdgcn_readfirstlane(at);
}

template <int EPL>
__global__ __launch_bounds__(64 * kWavesPerBlock) void moe_route_kernel(
    const qdg_route_config c, const void* __restrict__ logits, int64_t ld, const float* __restrict__ bias, int64_t T,
    bool vec, int group_shift, int32_t* __restrict__ ids, float* __restrict__ weights,
    uint32_t* __restrict__ status) {
  __shared__ float2 keybuf[kWavesPerBlock][EPL * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = c.num_experts, G = c.num_groups, per = E / G, e0 = lane * EPL;
  const float nan = __builtin_nanf("");
  float b[EPL];
  bool bad_bias = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    b[j] = bias && e0 + j < E ? bias[e0 + j] : 0.f;
    bad_bias |= b[j] != b[j];
  }
  for (int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + wave; t < T; t += (int64_t)gridDim.x * kWavesPerBlock) {
    Row row{(const char*)logits + t * ld * (c.ltype == QDG_L_F32 ? 4 : 2), bias, c.ltype, c.score, E, 0.f, 1.0};
    float x[EPL];  // logits, -inf where masked by the logit
    load_row<EPL>(row.logits, c.ltype, vec, e0, E, -kInf, x);
    bool bad = bad_bias;
    float top = -kInf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      bad |= x[j] != x[j] || x[j] == kInf;
      x[j] = x[j] != x[j] ? -kInf : fminf(x[j], 3.402823466e+38f);
      top = fmaxf(top, x[j]);
    }
    if (status && bad) atomicOr(status, (uint32_t)QDG_FLAG_BAD_LOGIT);

    // intervals of the keys; without a bias of the scores, for the groups
    const bool score_keys = bias || G > 1;
    float lo[EPL], up[EPL];
    if (c.score == QDG_SCORE_SOFTMAX) row.top = top = wave_max(top);
    if (score_keys) {
      float inv = 1.f;
      if (c.score == QDG_SCORE_SOFTMAX) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          lo[j] = x[j] == -kInf ? 0.f : __expf(x[j] - top);
          sum += lo[j];
        }
        for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
        inv = sum > 0.f ? 1.0f / sum : 0.f;
      }
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        float s, ds;
        if (c.score == QDG_SCORE_SOFTMAX) {
          s = lo[j] * inv;
          ds = s * (0x1p-19f + (top - x[j]) * 0x1p-22f);
        } else {
          s = __builtin_amdgcn_rcpf(1.0f + __expf(-x[j]));
          ds = s * (0x1p-20f + fabsf(x[j]) * 0x1p-22f);
        }
        // a score below 2^-126 (flushed, or with a lost mantissa) is off by less than that
        ds += 0x1p-125f;
        if (!(ds < kInf)) ds = 0x1p-125f;  // |x| so large that s is 0 or 1 to the last bit
        const float k = s + b[j];
        const float d = ds + fabsf(k) * 0x1p-23f;
        const bool masked = x[j] == -kInf || !(b[j] > -kInf), fin = fabsf(k) < kInf;
        lo[j] = masked ? -kInf : fin ? fmaxf(k - d, -3.402823466e+38f) : k;
        up[j] = masked ? -kInf : fin ? k + d : k;
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) lo[j] = up[j] = x[j];
    }

    uint64_t stay = ~0ull;
    if (G > 1) {
      // lane g of the result: the interval of group g's value
      float l1 = -kInf, l2 = -kInf, u1 = -kInf, u2 = -kInf;
      int owner = lane;  // the lane that holds group g = lane's interval
      if (group_shift >= 0) {
        // a group is 2^group_shift whole lanes
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
          top2_merge(l1, l2, e0 + j < E ? lo[j] : -kInf, -kInf);
          top2_merge(u1, u2, e0 + j < E ? up[j] : -kInf, -kInf);
        }
        for (int m = 1; m < 1 << group_shift; m <<= 1) {
          top2_merge(l1, l2, __shfl_xor(l1, m), __shfl_xor(l2, m));
          top2_merge(u1, u2, __shfl_xor(u1, m), __shfl_xor(u2, m));
        }
        owner = lane << group_shift;
      } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) keybuf[wave][e0 + j] = make_float2(lo[j], up[j]);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (lane < G)
          for (int i = 0; i < per; ++i) {
            const float2 k = keybuf[wave][lane * per + i];
            top2_merge(l1, l2, k.x, -kInf);
            top2_merge(u1, u2, k.y, -kInf);
          }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      const bool one = c.group_score == QDG_GROUP_MAX;
      float vl = one || l2 == -kInf ? l1 : l1 + l2, vu = one || u2 == -kInf ? u1 : u1 + u2;
      if (!one) {  // the two sums' own rounding
        if (fabsf(vl) < kInf) vl -= fabsf(vl) * 0x1p-23f;
        if (fabsf(vu) < kInf) vu += fabsf(vu) * 0x1p-23f;
      }
      vl = __shfl(vl, owner & 63);
      vu = __shfl(vu, owner & 63);
      int maybe = 0, sure = 0;  // groups that may be ahead of this lane's, and that are
      for (int g = 0; g < G; ++g) {
        const float ol = readlane_f32(vl, g), ou = readlane_f32(vu, g);
        const bool tie = ou == -kInf && vu == -kInf;  // all masked, both: the index decides
        maybe += g != lane && (tie ? g < lane : ou >= vl);
        sure += g != lane && (tie ? g < lane : ol > vu);
      }
      const bool in = lane < G && maybe < c.topk_groups, out = sure >= c.topk_groups;
      stay = __ballot(in);
      if (__ballot(lane < G && !in && !out)) stay = groups64(row, c, lane);
    }
    const bool exact = !bias;  // the keys are the logits
    const bool lane_stays = group_shift < 0 || (stay >> (lane >> group_shift)) & 1;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if (exact) lo[j] = up[j] = x[j];
      const int e = e0 + j;
      const bool stays = group_shift < 0 && G > 1 ? e < E && (stay >> (e / per)) & 1 : lane_stays;
      if (e >= E || !stays) lo[j] = up[j] = nan;  // not to be taken
    }

    int my_id = 0;
    float my_x = -kInf;  // -inf: masked, weight 0
    for (int r = 0; r < c.top_k; ++r) {
      float m = lo[0];
#pragma unroll
      for (int j = 1; j < EPL; ++j) m = fmaxf(m, lo[j]);
      m = wave_max(m);
      uint32_t cand = 0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) cand |= (uint32_t)(up[j] >= m) << j;
      const uint64_t has = __ballot(cand != 0), more = __ballot((cand & (cand - 1)) != 0);
      int wl, ws;
      if (exact || m == -kInf || ((has & (has - 1)) == 0 && more == 0)) {
        wl = __builtin_ctzll(has);
        ws = __builtin_ctz(__builtin_amdgcn_readlane(cand, wl));
      } else {
        const int e = best64(row, cand, e0, lane);
        wl = e / EPL;
        ws = e % EPL;
      }
      float won = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (j == ws) {
          won = x[j];
          if (lane == wl) lo[j] = up[j] = nan;
        }
      won = readlane_f32(won, wl);
      if (lane == r) {
        my_id = wl * EPL + ws;
        my_x = m == -kInf ? -kInf : won;  // only masked experts are left
      }
    }

    // the weights, one lane each
    double w = 0.0;
    if (c.score == QDG_SCORE_SIGMOID) {
      if (my_x != -kInf) w = sigmoid64((double)my_x);
      if (c.renormalize) {
        const double sum = wave_sum(w);
        w = sum > 0.0 ? w / sum : 0.0;
      }
    } else {
      // renormalised weights need no more than the chosen experts' ratios
      const float ref = c.renormalize ? wave_max(my_x) : top;
      if (my_x != -kInf) w = exp((double)my_x - (double)ref);
      if (c.renormalize)
        row.sum64 = wave_sum(w);
      else
        row.set_sum(lane);
      w = row.sum64 > 0.0 ? w / row.sum64 : 0.0;
    }
    if (lane < c.top_k) {
      ids[t * c.top_k + lane] = my_id;
      weights[t * c.top_k + lane] = (float)(w * (double)c.scale);
    }
  }
}

}  // namespace

hipError_t launch_moe_route(const qdg_route_config& c, const void* logits, int64_t ld, const float* bias, int64_t T,
                            int32_t* ids, float* weights, uint32_t* status, hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>((T + kWavesPerBlock - 1) / kWavesPerBlock, 1 << 14));
  int epl = 1;
  while (epl * 64 < c.num_experts) epl *= 2;
  const size_t esz = c.ltype == QDG_L_F32 ? 4 : 2, load = std::min<size_t>(16, epl * esz);
  const bool vec = (uintptr_t)logits % load == 0 && (size_t)ld * esz % load == 0;
  const int per = c.num_experts / c.num_groups;
  const int lanes = per / epl;  // whole lanes of a group, where it is that
  const int group_shift =
      c.num_groups > 1 && per % epl == 0 && (lanes & (lanes - 1)) == 0 ? __builtin_ctz(lanes) : -1;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kWavesPerBlock), 0, s, c, logits, ld, bias, T, vec, group_shift, ids,
                       weights, status);
    return hipGetLastError();
  };
  switch (epl) {
    case 1: return go(moe_route_kernel<1>);
    case 2: return go(moe_route_kernel<2>);
    case 4: return go(moe_route_kernel<4>);
    case 8: return go(moe_route_kernel<8>);
    default: return go(moe_route_kernel<16>);
  }
}

}  // namespace qdg
