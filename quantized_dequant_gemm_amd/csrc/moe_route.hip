// Expert routing: scores, grouped top-k and weights of each token.
//
//   s = softmax(l) or sigmoid(l);  c = s + bias (or the order of l);
//   value of a group = largest c or sum of its two largest; the best groups
//   stay; top_k of what stays by c; w = s, renormalised, scaled.
//
// One wave per token, EPL consecutive experts per lane (one vector load). A
// key becomes one unsigned number: its binary32 bits in increasing order,
// the lowest bits replaced by the expert's index counted from the top, so
// that a round of the top_k is one wave-wide unsigned maximum (six DPP
// steps): it names the expert, and equal keys give the lowest index.
//
// A choice must not hang on binary32 rounding, yet binary64 scores and 64-bit
// reductions for all experts take two and a half times as long (8192 tokens x
// 256 experts in groups: 31.4 against 11.9 us, bound by some 470 vector
// instructions a token and the last tokens in doubt). So the top_k + 1 largest
// are taken in binary32 and the gaps between neighbours are compared with what
// the keys can be off by. Where a gap does not decide (some 4 % of the tokens
// of normal logits and biases), four more candidates are taken and ranked by
// binary64 keys, one lane each; if not even these hold the top_k for sure, the
// whole token is routed in binary64. Without a bias the keys are the logits:
// exact for 16-bit types, cut by the index bits for binary32 ones.
//
// Error bounds: exp as v_exp_f32 of x * log2(e) is off by 2^-23 + 1.5 |x| 2^-24
// relative. Sigmoid: 1 / (1 + t) adds 2^-24 + 2^-23 and passes on s (1 - s) of
// t's error, and s (1 - s) |x| < 0.3: off by less than 2^-21 absolute, half of
// score_err. Softmax, in units of 2^-24 and with d = x - top: the numerator
// (2 + 2.5 |d|) s, where s |d| < 0.4; the sum of 1024 terms 21 s for 15
// additions a lane and 6 across, and (2 + 2.5 D) s for its terms, D the mean of
// |d| under s; reciprocal and product 3 s. For 1024 experts 28 s + 1 + 2.5 D s
// stays below 30, score_err is 32. The bias added rounds by 2^-24 of the key,
// which key_low and key_high count.
//
// The weights of the top_k, one lane each: exp in binary32 (one unit in the
// last place, 2^-23) of the argument's upper part, times 1 + its lower part;
// sums and quotients in binary64, so a weight is off by 2^-22 + 2^-24.
#include <algorithm>
#include <type_traits>

#include "qdg_device.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

constexpr double kNegInf64 = -__builtin_inf();
constexpr float kInf = __builtin_inff();
constexpr float kMax = 3.402823466e+38f;  // largest finite
constexpr int kWavesPerBlock = 4;
constexpr int kMore = 4;  // candidates beyond top_k where the order is in doubt

// One step of a maximum over the wave: lanes without a source, and rows
// outside ROW_MASK, see 0.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROW_MASK, 0xF, false));
}

// Largest value of the wave, in every lane.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = dpp_max<0x111, 0xF>(v);  // row_shr:1, 2, 4, 8: lane 15 of each row of 16
  v = dpp_max<0x112, 0xF>(v);
  v = dpp_max<0x114, 0xF>(v);
  v = dpp_max<0x118, 0xF>(v);
  v = dpp_max<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  v = dpp_max<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Binary32 <-> unsigned in the same order.
__device__ __forceinline__ uint32_t order_of(float f) {
  const uint32_t u = __builtin_bit_cast(uint32_t, f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_order(uint32_t o) {
  return __builtin_bit_cast(float, o ^ (~(uint32_t)((int32_t)o >> 31) | 0x80000000u));
}

__device__ __forceinline__ double wave_sum(double v) {
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ float readlane_f32(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

__device__ __forceinline__ double readlane_f64(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, lane), hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ void top2_add(float& m1, float& m2, float v) {
  m2 = __builtin_amdgcn_fmed3f(m1, m2, v);
  m1 = fmaxf(m1, v);
}

__device__ __forceinline__ void sort2(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
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

// exp of the argument's negative only: exp(-x) passes binary64's range at x <
// -709.8, where the score is still a number down to 2^-1074.
__device__ __forceinline__ double sigmoid64(double x) {
  const double e = exp(-fabs(x));
  return (x >= 0.0 ? 1.0 : e) / (1.0 + e);
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
    return x != x ? -kInf : fminf(x, kMax);
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
// overlap at the border): a bit for each group. A group is 2^group_shift lanes
// of epl experts, or (group_shift < 0) any run, which the whole wave walks.
__device__ __forceinline__ uint64_t groups64(Row& row, const qdg_route_config& c, int epl, int group_shift, int lane) {
  const int G = c.num_groups, per = c.num_experts / G;
  if (row.score == QDG_SCORE_SOFTMAX) row.set_sum(lane);
  auto add = [](double& m1, double& m2, double k) {
    m2 = fmax(m2, fmin(m1, k));
    m1 = fmax(m1, k);
  };
  auto merge = [](double& m1, double& m2, int m) {
    const double o1 = __shfl_xor(m1, m), o2 = __shfl_xor(m2, m);
    m2 = fmax(fmin(m1, o1), fmax(m2, o2));
    m1 = fmax(m1, o1);
  };
  auto value = [&](double m1, double m2) {
    return c.group_score == QDG_GROUP_MAX || m2 == kNegInf64 ? m1 : m1 + m2;
  };
  double mine = kNegInf64;  // lane g: the value of group g
  if (group_shift >= 0) {
    double m1 = kNegInf64, m2 = kNegInf64;
#pragma unroll 1
    for (int e = lane * epl; e < min((lane + 1) * epl, c.num_experts); ++e) add(m1, m2, row.key64(e));
#pragma unroll 1
    for (int m = 1; m < 1 << group_shift; m <<= 1) merge(m1, m2, m);
    mine = __shfl(value(m1, m2), (lane << group_shift) & 63);
  } else {
#pragma unroll 1
    for (int g = 0; g < G; ++g) {
      double m1 = kNegInf64, m2 = kNegInf64;
#pragma unroll 1
      for (int i = lane; i < per; i += 64) add(m1, m2, row.key64(g * per + i));
#pragma unroll 1
      for (int m = 32; m > 0; m >>= 1) merge(m1, m2, m);
      if (lane == g) mine = value(m1, m2);
    }
  }
  int rank = 0;
#pragma unroll 1
  for (int g = 0; g < G; ++g) {
    const double o = __shfl(mine, g);
    rank += o > mine || (o == mine && g < lane);
  }
  return __ballot(lane < G && rank < c.topk_groups);
}

// A token routed in binary64: the id that lane r < top_k takes.
__device__ __forceinline__ int route64(Row& row, const qdg_route_config& c, uint64_t stay, int lane) {
  const int E = c.num_experts, per = E / c.num_groups;
  if (row.score == QDG_SCORE_SOFTMAX && row.bias) row.set_sum(lane);
  uint32_t taken = 0;  // bit i: expert lane + 64 i
  int id = 0;
#pragma unroll 1
  for (int r = 0; r < c.top_k; ++r) {
    double best = kNegInf64;
    int at = 1 << 30;
#pragma unroll 1
    for (int e = lane, i = 0; e < E; e += 64, ++i) {
      if ((taken >> i & 1) || !(stay >> (e / per) & 1)) continue;
      const double k = row.bias ? row.key64(e) : (double)row.logit(e);
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
    if ((at & 63) == lane) taken |= 1u << (at >> 6);
    if (r == lane) id = at;
  }
  return id;
}

// The largest of the wave's ordered keys, taken out (0: none is left). Up to
// four per lane are sorted, so that the first is the lane's largest.
template <int EPL>
__device__ __forceinline__ uint32_t take_largest(uint32_t (&o)[EPL]) {
  uint32_t m = o[0];
  if constexpr (EPL > 4) {
#pragma unroll
    for (int j = 1; j < EPL; ++j) m = max(m, o[j]);
  }
  m = wave_max(m);
  if constexpr (EPL > 4) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) o[j] = o[j] == m ? 0u : o[j];
  } else {
    const bool pop = o[0] == m;
#pragma unroll
    for (int j = 0; j < EPL; ++j) o[j] = pop ? (j + 1 < EPL ? o[j + 1] : 0u) : o[j];
  }
  return m;
}

// What a binary32 score is off by at most.
__device__ __forceinline__ constexpr float score_err(bool sigmoid) { return sigmoid ? 0x1p-20f : 0x1p-19f; }

// Bounds of the exact key behind an ordered one whose low bits are cut.
__device__ __forceinline__ float key_low(uint32_t o, uint32_t index_mask, float err) {
  const float k = of_order(o & ~index_mask);
  return k - err - fabsf(k) * 0x1p-23f;
}
__device__ __forceinline__ float key_high(uint32_t o, uint32_t index_mask, float err) {
  const float k = of_order(o | index_mask);
  return k + err + fabsf(k) * 0x1p-23f;
}

// exp(a - b) for a <= b in binary64 with binary32's relative error 2^-23,
// 0 below 2^-126 (where the difference may pass binary32's largest value).
__device__ __forceinline__ double exp_diff(float a, float b) {
  const double d = fmax((double)a - (double)b, -256.0);
  const float hi = (float)d, lo = (float)(d - (double)hi);
  const float e = expf(hi);
  return (double)__builtin_fmaf(e, lo, e);
}

// 1 / v, off by less than 2^-40.
__device__ __forceinline__ double rcp64(double v) {
  const double r = __builtin_amdgcn_rcp(v);
  return __builtin_fma(__builtin_fma(-v, r, 1.0), r, r);
}

template <int EPL, bool SIGMOID, bool BIAS, bool GROUPS>
__global__ __launch_bounds__(64 * kWavesPerBlock) void moe_route_kernel(
    const qdg_route_config c, const void* __restrict__ logits, int64_t ld, const float* __restrict__ bias, int64_t T,
    bool vec, int group_shift, uint32_t index_mask, int32_t* __restrict__ ids, float* __restrict__ weights,
    uint32_t* __restrict__ status) {
  __shared__ float keybuf[kWavesPerBlock][EPL * 64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int E = c.num_experts, G = GROUPS ? c.num_groups : 1, per = E / G, e0 = lane * EPL;
  float b[EPL];
  bool bad_bias = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    b[j] = BIAS && e0 + j < E ? bias[e0 + j] : 0.f;
    bad_bias |= b[j] != b[j];
  }
  // one token a wave: in a loop over tokens the constants of the rare binary64
  // paths would be kept in registers for all of it
  const int64_t t = (int64_t)blockIdx.x * kWavesPerBlock + wave;
  if (t >= T) return;  // whole waves; no barrier below
  Row row{(const char*)logits + t * ld * (c.ltype == QDG_L_F32 ? 4 : 2), bias, c.ltype, c.score, E, 0.f, 1.0};
  float x[EPL];  // logits, -inf where masked by the logit
  load_row<EPL>(row.logits, c.ltype, vec, e0, E, -kInf, x);
  bool bad = bad_bias;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    bad |= x[j] != x[j] || x[j] == kInf;
    x[j] = x[j] != x[j] ? -kInf : fminf(x[j], kMax);
  }
  if (status && bad) atomicOr(status, (uint32_t)QDG_FLAG_BAD_LOGIT);
  if constexpr (!SIGMOID) {
    float top = x[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) top = fmaxf(top, x[j]);
    row.top = of_order(wave_max(order_of(top)));
  }

  float key[EPL];  // s + bias; -inf where masked
  if constexpr (BIAS || GROUPS) {
    float inv = 1.f;
    if constexpr (!SIGMOID) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        key[j] = x[j] == -kInf ? 0.f : __expf(x[j] - row.top);
        sum += key[j];
      }
      for (int m = 32; m > 0; m >>= 1) sum += __shfl_xor(sum, m);
      inv = __builtin_amdgcn_rcpf(sum);
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const float s = !SIGMOID ? key[j] * inv : __builtin_amdgcn_rcpf(1.0f + __expf(-x[j]));
      key[j] = x[j] == -kInf || !(b[j] > -kInf) ? -kInf : s + b[j];
    }
  }

  uint64_t stay = ~0ull;
  if constexpr (GROUPS) {
    float m1 = -kInf, m2 = -kInf;  // lane of group g: its two largest keys
    int owner = lane;              // the lane that holds group g = lane's
    if (group_shift >= 0) {
      // a group is 2^group_shift whole lanes
#pragma unroll
      for (int j = 0; j < EPL; ++j) top2_add(m1, m2, e0 + j < E ? key[j] : -kInf);
      for (int m = 1; m < 1 << group_shift; m <<= 1) {
        const float o1 = __shfl_xor(m1, m), o2 = __shfl_xor(m2, m);
        m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
        m1 = fmaxf(m1, o1);
      }
      owner = lane << group_shift;
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) keybuf[wave][e0 + j] = key[j];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lane < G)
        for (int i = 0; i < per; ++i) top2_add(m1, m2, keybuf[wave][lane * per + i]);
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    const float v = c.group_score == QDG_GROUP_MAX || m2 == -kInf ? m1 : m1 + m2;
    // two keys' errors and the roundings of keys and sum
    const float err = fabsf(v) < kInf ? 2.f * score_err(SIGMOID) + (fabsf(m1) + (m2 == -kInf ? 0.f : fabsf(m2))) * 0x1p-22f : 0.f;
    // a sum below binary32's range is no mask: anywhere under its largest magnitude
    const float vl = __shfl(v - err, owner & 63);
    const float vu = __shfl(v == -kInf && m1 > -kInf ? -kMax : v + err, owner & 63);
    int maybe = 0;  // groups that may be ahead of this lane's
    for (int g = 0; g < G; ++g) {
      const float ou = readlane_f32(vu, g);
      const bool tie = ou == -kInf && vu == -kInf;  // all masked, both: the index decides
      maybe += g != lane && (tie ? g < lane : ou >= vl);
    }
    const bool in = lane < G && maybe < c.topk_groups;
    stay = __ballot(in);
    if (__popcll(stay) != c.topk_groups) stay = groups64(row, c, EPL, group_shift, lane);
  }

  // the ordered keys
  const bool lane_stays = group_shift < 0 || (stay >> (lane >> group_shift)) & 1;
  uint32_t o[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = e0 + j;
    const bool stays = GROUPS && group_shift < 0 ? e < E && (stay >> (e / per)) & 1 : lane_stays;
    // -0 and 0 are one key
    o[j] = e < E && stays ? (order_of((BIAS ? key[j] : x[j]) + 0.f) & ~index_mask) | (index_mask - (uint32_t)e) : 0u;
  }
  if constexpr (EPL == 2) sort2(o[0], o[1]);
  if constexpr (EPL == 4) {
    sort2(o[0], o[1]);
    sort2(o[2], o[3]);
    sort2(o[0], o[2]);
    sort2(o[1], o[3]);
    sort2(o[1], o[2]);
  }
  // rounds 0 .. top_k: lane r keeps the r-th largest
  uint32_t mine = 0;
  for (int r = 0; r <= c.top_k; ++r) {
    const uint32_t m = take_largest<EPL>(o);
    mine = lane == r ? m : mine;
  }
  if (BIAS || c.ltype == QDG_L_F32) {
    // does each gap to the next decide?
    const uint32_t next = (uint32_t)__shfl_down((int)mine, 1);
    const bool checked = lane < c.top_k && next != 0 && (mine & ~index_mask) != (order_of(-kInf) & ~index_mask);
    const bool sure = BIAS ? key_low(mine, index_mask, score_err(SIGMOID)) > key_high(next, index_mask, score_err(SIGMOID))
                           : (mine ^ next) > index_mask;  // exact but for the cut bits
    if (__ballot(checked && !sure)) {
      // kMore candidates more, ranked by binary64 keys, one lane each
      uint32_t last = 0;
      for (int r = c.top_k + 1; r < c.top_k + kMore; ++r) {
        last = take_largest<EPL>(o);
        mine = lane == r ? last : mine;
      }
      if (!SIGMOID && BIAS) row.set_sum(lane);
      int cand = (int)(index_mask - (mine & index_mask));
      double k = kNegInf64;
      if (mine != 0) k = BIAS ? row.key64(cand) : (double)row.logit(cand);
      else cand = 1 << 30;
      int rank = 0;
      for (int i = 0; i < c.top_k + kMore; ++i) {
        const double ok = readlane_f64(k, i);
        const int oc = __builtin_amdgcn_readlane(cand, i);
        rank += ok > k || (ok == k && oc < cand);
      }
      // what was not taken is at most `last`; masked experts follow the index
      const uint64_t kth = __ballot(lane < c.top_k + kMore && rank == c.top_k - 1);
      const double kth_key = readlane_f64(k, __builtin_ctzll(kth));
      const double rest = BIAS ? (double)key_high(last, index_mask, score_err(SIGMOID)) : (double)of_order(last | index_mask);
      const bool whole = last == 0 || (last & ~index_mask) == (order_of(-kInf) & ~index_mask);
      int id = 0;
      if (whole || kth_key > rest) {
        for (int i = 0; i < c.top_k + kMore; ++i) {
          const int to = __builtin_amdgcn_readlane(rank, i), oc = __builtin_amdgcn_readlane(cand, i);
          if (lane == to) id = oc;
        }
      } else {
        id = route64(row, c, stay, lane);
      }
      mine = index_mask - (uint32_t)id;
    }
  }
  const int id = (int)(index_mask - (mine & index_mask));

  // the weights
  float my_x = -kInf;
  if (lane < c.top_k) {
    my_x = row.logit(id);
    if (BIAS && !(bias[id] > -kInf)) my_x = -kInf;  // masked: weight 0
  }
  double w = 0.0;
  const float ref = SIGMOID ? 0.f : row.top;
  // scores near or past the end of binary32
  const bool far = __ballot(my_x != -kInf && my_x - ref < -80.f) != 0;
  if (far) {
    if (my_x != -kInf) w = SIGMOID ? sigmoid64((double)my_x) : exp((double)my_x - (double)ref);
  } else if (my_x != -kInf) {
    w = SIGMOID ? rcp64(1.0 + (double)expf(-my_x)) : exp_diff(my_x, ref);
  }
  if (c.renormalize) {
    row.sum64 = w;
    for (int m = 1; m < c.top_k; m <<= 1) row.sum64 += __shfl_xor(row.sum64, m);
  } else if (!SIGMOID) {
    double sum = 0.0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) sum += x[j] == -kInf ? 0.0 : exp_diff(x[j], row.top);
    row.sum64 = wave_sum(sum);
  }
  if (c.renormalize || !SIGMOID) w = !(row.sum64 > 0.0) ? 0.0 : far ? w / row.sum64 : w * rcp64(row.sum64);
  if (lane < c.top_k) {
    ids[t * c.top_k + lane] = id;
    weights[t * c.top_k + lane] = (float)(w * (double)c.scale);
  }
}

}  // namespace

hipError_t launch_moe_route(const qdg_route_config& c, const void* logits, int64_t ld, const float* bias, int64_t T,
                            int32_t* ids, float* weights, uint32_t* status, hipStream_t s) {
  const dim3 grid((unsigned)((T + kWavesPerBlock - 1) / kWavesPerBlock));
  int epl = 1;
  while (epl * 64 < c.num_experts) epl *= 2;
  const size_t esz = c.ltype == QDG_L_F32 ? 4 : 2, load = std::min<size_t>(16, epl * esz);
  const bool vec = (uintptr_t)logits % load == 0 && (size_t)ld * esz % load == 0;
  const int per = c.num_experts / c.num_groups;
  const int lanes = per / epl;  // whole lanes of a group, where it is that
  const int group_shift =
      c.num_groups > 1 && per % epl == 0 && (lanes & (lanes - 1)) == 0 ? __builtin_ctz(lanes) : -1;
  uint32_t index_mask = 0;
  while ((int)index_mask + 1 < c.num_experts) index_mask = index_mask * 2 + 1;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(64 * kWavesPerBlock), 0, s, c, logits, ld, bias, T, vec, group_shift,
                       index_mask, ids, weights, status);
    return hipGetLastError();
  };
  // one instance for each score, with and without bias and groups: a single
  // one for all spilled scalar registers at 256 experts (8192 x 256 grouped
  // 18.0 us). Of these only softmax with a bias at more than 512 experts does,
  // 20 of them, 32 with groups, into vector registers.
  auto pick = [&](auto experts_per_lane) {
    constexpr int N = decltype(experts_per_lane)::value;
    const bool sg = c.score == QDG_SCORE_SIGMOID, gr = c.num_groups > 1;
    if (sg && bias) return gr ? go(moe_route_kernel<N, true, true, true>) : go(moe_route_kernel<N, true, true, false>);
    if (sg) return gr ? go(moe_route_kernel<N, true, false, true>) : go(moe_route_kernel<N, true, false, false>);
    if (bias) return gr ? go(moe_route_kernel<N, false, true, true>) : go(moe_route_kernel<N, false, true, false>);
    return gr ? go(moe_route_kernel<N, false, false, true>) : go(moe_route_kernel<N, false, false, false>);
  };
  switch (epl) {
    case 1: return pick(std::integral_constant<int, 1>());
    case 2: return pick(std::integral_constant<int, 2>());
    case 4: return pick(std::integral_constant<int, 4>());
    case 8: return pick(std::integral_constant<int, 8>());
    default: return pick(std::integral_constant<int, 16>());
  }
}

}  // namespace qdg
