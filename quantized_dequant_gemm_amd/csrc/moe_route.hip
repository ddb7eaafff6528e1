// Expert routing: scores, grouped top-k and weights of each token.
//
//   s = softmax(l) or sigmoid(l);  c = s + bias (or the order of l);
//   value of a group = largest c or sum of its two largest; the best groups
//   stay; top_k of what stays by c; w = s, renormalised, scaled.
#include <algorithm>

#include "qdg_device.h"
#include "qdg_internal.h"

namespace qdg {
namespace {

constexpr double kNegInf = -__builtin_inf();

__device__ __forceinline__ double shfl_xor_f64(double v, int m) { return __shfl_xor(v, m); }

__device__ __forceinline__ float load_logit(const void* p, int64_t i, int ltype) {
  if (ltype == QDG_L_F32) return ((const float*)p)[i];
  const uint16_t h = ((const uint16_t*)p)[i];
  if (ltype == QDG_L_F16) return (float)__builtin_bit_cast(_Float16, h);
  return __builtin_bit_cast(float, (uint32_t)h << 16);
}

// One wave per token; lane l holds experts l, l + 64, ... (EPL of them).
template <int EPL>
__global__ __launch_bounds__(256) void moe_route_kernel(const qdg_route_config c, const void* __restrict__ logits,
                                                        int64_t ld, const float* __restrict__ bias, int64_t T,
                                                        int32_t* __restrict__ ids, float* __restrict__ weights,
                                                        uint32_t* __restrict__ status) {
  __shared__ double keybuf[4][EPL * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int E = c.num_experts, G = c.num_groups, per = E / G;
  for (int64_t t0 = (int64_t)blockIdx.x * 4; t0 < T; t0 += (int64_t)gridDim.x * 4) {
    const int64_t t = t0 + wave;
    const bool live = t < T;  // waves without a token still reach the barriers
    double l[EPL], s[EPL], key[EPL];
    bool masked[EPL], gone[EPL];
    bool bad = false;
    double mx = kNegInf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = j * 64 + lane;
      float x = -__builtin_inff();
      if (live && e < E) x = load_logit(logits, t * ld + e, c.ltype);
      if (x != x) {
        bad = true;
        x = -__builtin_inff();
      }
      if (x == __builtin_inff()) {
        bad = true;
        x = 3.402823466e+38f;
      }
      const float b = bias && e < E ? bias[e] : 0.f;
      if (b != b) bad = true;
      masked[j] = x == -__builtin_inff() || b != b || b == -__builtin_inff();
      gone[j] = e >= E;
      l[j] = (double)x;
      if (x != -__builtin_inff()) mx = fmax(mx, l[j]);
      key[j] = (double)b;
    }
    if (status && bad && live) atomicOr(status, (uint32_t)QDG_FLAG_BAD_LOGIT);
    if (c.score == QDG_SCORE_SOFTMAX) {
      for (int m = 32; m > 0; m >>= 1) mx = fmax(mx, shfl_xor_f64(mx, m));
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        s[j] = l[j] == kNegInf ? 0.0 : exp(l[j] - mx);
        sum += s[j];
      }
      for (int m = 32; m > 0; m >>= 1) sum += shfl_xor_f64(sum, m);
#pragma unroll
      for (int j = 0; j < EPL; ++j) s[j] = sum > 0.0 ? s[j] / sum : 0.0;
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) s[j] = l[j] == kNegInf ? 0.0 : 1.0 / (1.0 + exp(-l[j]));
    }
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      key[j] = masked[j] ? kNegInf : s[j] + key[j];
      if (masked[j]) s[j] = 0.0;
      keybuf[wave][j * 64 + lane] = key[j];  // a group's value is taken over s (+ bias)
      if (!bias && !masked[j]) key[j] = l[j];
    }
    if (G > 1) {
      __syncthreads();
      double value = kNegInf;
      if (lane < G) {
        double m1 = kNegInf, m2 = kNegInf;
        for (int i = 0; i < per; ++i) {
          const double v = keybuf[wave][lane * per + i];
          m2 = fmax(m2, fmin(m1, v));
          m1 = fmax(m1, v);
        }
        value = c.group_score == QDG_GROUP_MAX || m2 == kNegInf ? m1 : m1 + m2;
      }
      int rank = 0;
      for (int g = 0; g < G; ++g) {
        const double v = __shfl(value, g);
        rank += v > value || (v == value && g < lane);
      }
      const uint64_t stay = __ballot(lane < G && rank < c.topk_groups);
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (!gone[j]) gone[j] = !((stay >> ((j * 64 + lane) / per)) & 1);
      __syncthreads();
    }
    // top_k rounds of a wave-wide largest (key, lowest index)
    int my_id = 0;
    double my_s = 0.0, total = 0.0;
    for (int r = 0; r < c.top_k; ++r) {
      double best = kNegInf;
      int at = 1 << 30;
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = j * 64 + lane;
        if (!gone[j] && (key[j] > best || (key[j] == best && e < at))) {
          best = key[j];
          at = e;
        }
      }
      for (int m = 32; m > 0; m >>= 1) {
        const double ob = shfl_xor_f64(best, m);
        const int oa = __shfl_xor(at, m);
        if (ob > best || (ob == best && oa < at)) {
          best = ob;
          at = oa;
        }
      }
      double sc = 0.0;
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (j * 64 + lane == at) {
          gone[j] = true;
          sc = s[j];
        }
      sc = __shfl(sc, at & 63);
      total += sc;
      if (lane == r) {
        my_id = at;
        my_s = sc;
      }
    }
    if (live && lane < c.top_k) {
      double w = my_s;
      if (c.renormalize) w = total > 0.0 ? w / total : 0.0;
      ids[t * c.top_k + lane] = my_id;
      weights[t * c.top_k + lane] = (float)(w * (double)c.scale);
    }
  }
}

}  // namespace

hipError_t launch_moe_route(const qdg_route_config& c, const void* logits, int64_t ld, const float* bias, int64_t T,
                            int32_t* ids, float* weights, uint32_t* status, hipStream_t s) {
  const dim3 grid((unsigned)std::min<int64_t>((T + 3) / 4, 1 << 20));
  const int epl = (c.num_experts + 63) / 64;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, c, logits, ld, bias, T, ids, weights, status);
    return hipGetLastError();
  };
  if (epl <= 1) return go(moe_route_kernel<1>);
  if (epl <= 2) return go(moe_route_kernel<2>);
  if (epl <= 4) return go(moe_route_kernel<4>);
  if (epl <= 8) return go(moe_route_kernel<8>);
  return go(moe_route_kernel<16>);
}

}  // namespace qdg
