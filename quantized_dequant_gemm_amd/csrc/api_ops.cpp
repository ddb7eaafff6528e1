// C ABI of the operators that need no plan: expert routing, the asymmetric
// activation quantizer and the int8 products over row-major operands.
// Validation here, kernels in moe_route.hip, actquant.hip and gemm_i8.hip.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "qdg_internal.h"

using namespace qdg;

namespace {

qdg_status fail(qdg_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return report_error(st, buf);
}

qdg_status hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return QDG_OK;
  return fail(QDG_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// hipErrorInvalidConfiguration: the launcher found more tiles than a launch holds.
qdg_status i8_launch_status(hipError_t e, const char* what) {
  if (e == hipErrorInvalidConfiguration)
    return fail(QDG_ERR_UNSUPPORTED, "%s: the output has more tiles than one launch holds (2^32 threads)", what);
  return hip_status(e, what);
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 28;  // eight rows within 32-bit offsets
constexpr int64_t kMaxSide = (int64_t)1 << 26;  // rows and columns of the int8 products
constexpr int64_t kMaxTokens = ((int64_t)1 << 26) - 4;  // routed: one wave each, a launch holds fewer than 2^32 threads

// The checks that the dense and the grouped product share.
qdg_status check_i8(const qdg_i8_config* c) {
  if (!c) return fail(QDG_ERR_INVALID_ARG, "config is NULL");
  if (c->n < 1 || c->k < 1) return fail(QDG_ERR_INVALID_ARG, "n and k must be positive");
  if (c->n > kMaxSide) return fail(QDG_ERR_UNSUPPORTED, "n must be at most 2^26");
  if (c->k > 65536) return fail(QDG_ERR_UNSUPPORTED, "k must be at most 65536 (int32 sums)");
  if (c->num_experts < 1) return fail(QDG_ERR_INVALID_ARG, "num_experts must be positive");
  if (c->num_experts > 1024) return fail(QDG_ERR_UNSUPPORTED, "at most 1024 experts");
  if (c->otype != QDG_O_BF16 && c->otype != QDG_O_F32 && c->otype != QDG_O_I32)
    return fail(QDG_ERR_INVALID_ARG, "otype must be BF16, F32 or I32");
  if (c->epilogue != QDG_EPI_NONE && c->epilogue != QDG_EPI_SILU_MUL)
    return fail(QDG_ERR_INVALID_ARG, "bad epilogue");
  if (c->reserved != 0) return fail(QDG_ERR_INVALID_ARG, "reserved must be 0");
  if (c->epilogue == QDG_EPI_SILU_MUL) {
    if (c->otype == QDG_O_I32) return fail(QDG_ERR_UNSUPPORTED, "the SiLU*mul epilogue has no int32 output");
    if (c->n % 2) return fail(QDG_ERR_INVALID_ARG, "the SiLU*mul epilogue needs an even n");
  }
  const int64_t cols = c->epilogue == QDG_EPI_SILU_MUL ? c->n / 2 : c->n;
  if (c->lda < c->k || c->ldb < c->k || c->ldy < cols)
    return fail(QDG_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (c->lda > kMaxStride || c->ldb > kMaxStride) return fail(QDG_ERR_UNSUPPORTED, "lda and ldb must be at most 2^28");
  if (c->lda % 16 || c->ldb % 16) return fail(QDG_ERR_MISALIGNED, "lda and ldb must be multiples of 16 bytes");
  return QDG_OK;
}

// Checks of the operands and the kernel arguments they give.
qdg_status i8_args(const qdg_i8_config* c, const int8_t* A, const float* a_scales, const int32_t* a_zeros,
                   const int8_t* B, const float* b_scales, const float* bias, void* Y, I8Args* out) {
  if (!A || !B || !Y) return fail(QDG_ERR_INVALID_ARG, "NULL pointer");
  if (c->otype != QDG_O_I32 && (!a_scales || !b_scales)) return fail(QDG_ERR_INVALID_ARG, "scales are NULL");
  if (!aligned(A, 16) || !aligned(B, 16)) return fail(QDG_ERR_MISALIGNED, "A and B must be 16-byte aligned");
  if (!aligned(a_scales, 4) || !aligned(a_zeros, 4) || !aligned(b_scales, 4) || !aligned(bias, 4))
    return fail(QDG_ERR_MISALIGNED, "scales, zero points and bias must be 4-byte aligned");
  const size_t esz = c->otype == QDG_O_BF16 ? 2 : 4;
  if (!aligned(Y, esz)) return fail(QDG_ERR_MISALIGNED, "Y must be aligned to its element size");
  I8Args a = {};
  a.A = A;
  a.a_scales = a_scales;
  a.a_zeros = a_zeros;
  a.B = B;
  a.b_scales = b_scales;
  a.bias = c->otype == QDG_O_I32 ? nullptr : bias;
  a.Y = Y;
  a.lda = c->lda;
  a.ldb = c->ldb;
  a.ldy = c->ldy;
  a.n = (int)c->n;
  a.k = (int)c->k;
  a.cols = (int)(c->epilogue == QDG_EPI_SILU_MUL ? c->n / 2 : c->n);
  a.vcols = (int)gemm_i8_vcols(a.cols, c->epilogue == QDG_EPI_SILU_MUL);
  a.otype = c->otype;
  a.num_experts = c->num_experts;
  *out = a;
  return QDG_OK;
}

int64_t i8_vcols(const qdg_i8_config* c) {
  const bool silu = c->epilogue == QDG_EPI_SILU_MUL;
  return gemm_i8_vcols(silu ? c->n / 2 : c->n, silu);
}

// Bytes of the partials of a product of M rows.
size_t i8_workspace(const qdg_i8_config* c, int64_t M) {
  const int64_t vcols = i8_vcols(c);
  const int split = M > 0 ? gemm_i8_split(M, vcols, c->k) : 1;
  return split > 1 ? (size_t)split * (size_t)M * (size_t)vcols * sizeof(int32_t) : 0;
}

}  // namespace

extern "C" {

qdg_status qdg_moe_route(const qdg_route_config* cfg, const void* logits, int64_t ld, const float* bias, int64_t T,
                         int32_t* topk_ids, float* topk_weights, uint32_t* status, void* stream) {
  if (!cfg) return fail(QDG_ERR_INVALID_ARG, "config is NULL");
  qdg_route_config c = *cfg;
  if (c.num_groups == 0) c.num_groups = 1;
  if (c.num_groups == 1) c.topk_groups = 1;
  if (T < 0 || c.num_experts < 1 || c.top_k < 1 || c.num_groups < 1)
    return fail(QDG_ERR_INVALID_ARG, "bad T, num_experts, top_k or num_groups");
  if (c.num_experts > 1024) return fail(QDG_ERR_UNSUPPORTED, "at most 1024 experts");
  if (c.top_k > 32) return fail(QDG_ERR_UNSUPPORTED, "top_k must be at most 32");
  if (c.num_groups > 64) return fail(QDG_ERR_UNSUPPORTED, "at most 64 groups");
  if (T > kMaxTokens) return fail(QDG_ERR_UNSUPPORTED, "T must be at most 2^26 - 4");
  if (c.ltype != QDG_L_BF16 && c.ltype != QDG_L_F16 && c.ltype != QDG_L_F32)
    return fail(QDG_ERR_INVALID_ARG, "ltype must be BF16, F16 or F32");
  if (c.score != QDG_SCORE_SOFTMAX && c.score != QDG_SCORE_SIGMOID) return fail(QDG_ERR_INVALID_ARG, "bad score");
  if (c.group_score != QDG_GROUP_MAX && c.group_score != QDG_GROUP_TOP2)
    return fail(QDG_ERR_INVALID_ARG, "bad group_score");
  if (c.num_experts % c.num_groups) return fail(QDG_ERR_INVALID_ARG, "num_groups must divide num_experts");
  if (c.topk_groups < 1 || c.topk_groups > c.num_groups)
    return fail(QDG_ERR_INVALID_ARG, "topk_groups must be in [1, num_groups]");
  if (c.top_k > c.topk_groups * (c.num_experts / c.num_groups))
    return fail(QDG_ERR_INVALID_ARG, "top_k exceeds the experts of the groups that stay");
  if (!std::isfinite(c.scale)) return fail(QDG_ERR_INVALID_ARG, "scale must be finite");
  if (ld < c.num_experts) return fail(QDG_ERR_INVALID_ARG, "ld is shorter than a row");
  if (T == 0) return QDG_OK;
  if (!logits || !topk_ids || !topk_weights) return fail(QDG_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(logits, c.ltype == QDG_L_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(topk_weights, 4) || !aligned(status, 4))
    return fail(QDG_ERR_MISALIGNED, "pointers must be aligned to their elements");
  return hip_status(launch_moe_route(c, logits, ld, bias, T, topk_ids, topk_weights, status, (hipStream_t)stream),
                    "moe_route launch");
}

qdg_status qdg_quantize_act_zp(const void* a_bf16, int64_t lda, int64_t M, int64_t k, int8_t* qa, int64_t ldq,
                               float* a_scales, int32_t* a_zeros, void* stream) {
  if (M < 0 || k < 1) return fail(QDG_ERR_INVALID_ARG, "bad M or k");
  if (lda < k || ldq < k) return fail(QDG_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (M >= kMaxRows) return fail(QDG_ERR_UNSUPPORTED, "M must be below 2^31");
  if (k > ((int64_t)1 << 30)) return fail(QDG_ERR_UNSUPPORTED, "k must be at most 2^30");
  if (lda % 8 || ldq % 16) return fail(QDG_ERR_MISALIGNED, "lda must be a multiple of 8, ldq of 16");
  if (M == 0) return QDG_OK;
  if (!a_bf16 || !qa || !a_scales || !a_zeros) return fail(QDG_ERR_INVALID_ARG, "NULL pointer");
  if (!aligned(a_bf16, 16) || !aligned(qa, 16))
    return fail(QDG_ERR_MISALIGNED, "a_bf16 and qa must be 16-byte aligned");
  if (!aligned(a_scales, 4) || !aligned(a_zeros, 4))
    return fail(QDG_ERR_MISALIGNED, "a_scales and a_zeros must be 4-byte aligned");
  return hip_status(launch_quantize_act_zp(a_bf16, lda, M, k, qa, ldq, a_scales, a_zeros, (hipStream_t)stream),
                    "quantize_act_zp launch");
}

qdg_status qdg_gemm_i8_workspace(const qdg_i8_config* cfg, int64_t M, size_t* bytes) {
  const qdg_status st = check_i8(cfg);
  if (st != QDG_OK) return st;
  if (!bytes) return fail(QDG_ERR_INVALID_ARG, "bytes is NULL");
  if (cfg->num_experts != 1) return fail(QDG_ERR_INVALID_ARG, "the dense product has one expert");
  if (M < 0) return fail(QDG_ERR_INVALID_ARG, "M < 0");
  if (M > kMaxSide) return fail(QDG_ERR_UNSUPPORTED, "M must be at most 2^26");
  *bytes = (size_t)gemm_i8_max_partial_rows(M, i8_vcols(cfg), cfg->k) * (size_t)i8_vcols(cfg) * sizeof(int32_t);
  return QDG_OK;
}

int qdg_gemm_i8_describe(const qdg_i8_config* cfg, int64_t M, char* buf, size_t len) {
  if (check_i8(cfg) != QDG_OK || cfg->num_experts != 1 || M < 0 || M > kMaxSide) return -1;
  const I8Instance i = gemm_i8_instance(M > 0 ? M : 1, i8_vcols(cfg), cfg->k);
  char rest[48] = "none";
  if (i.rest_m) snprintf(rest, sizeof rest, "%dx%d", i.rest_m, i.rest_n);
  return snprintf(buf, buf ? len : 0,
                  "gemm-i8 dense n=%lld k=%lld M=%lld: family=%s block_m=%d block_n=%d split_k=%d columns=%lld rest=%s "
                  "epilogue=%s arch=gfx950",
                  (long long)cfg->n, (long long)cfg->k, (long long)M, i.block_m == 16 ? "rows" : "tile", i.block_m,
                  i.block_n, i.split, (long long)i.columns, rest,
                  cfg->epilogue == QDG_EPI_SILU_MUL ? "silu_mul" : "none");
}

qdg_status qdg_gemm_i8(const qdg_i8_config* cfg, const int8_t* A, const float* a_scales, const int32_t* a_zeros,
                       const int8_t* B, const float* b_scales, const float* bias, void* Y, int64_t M,
                       void* workspace, size_t ws_bytes, void* stream) {
  qdg_status st = check_i8(cfg);
  if (st != QDG_OK) return st;
  if (cfg->num_experts != 1) return fail(QDG_ERR_INVALID_ARG, "the dense product has one expert");
  if (M < 0) return fail(QDG_ERR_INVALID_ARG, "M < 0");
  if (M > kMaxSide) return fail(QDG_ERR_UNSUPPORTED, "M must be at most 2^26");
  if (M == 0) return QDG_OK;
  I8Args a;
  st = i8_args(cfg, A, a_scales, a_zeros, B, b_scales, bias, Y, &a);
  if (st != QDG_OK) return st;
  a.M = (int)M;
  const size_t need = i8_workspace(cfg, M);
  if (need > 0) {
    if (!workspace || ws_bytes < need)
      return fail(QDG_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace ? ws_bytes : 0, need);
    if (!aligned(workspace, 16)) return fail(QDG_ERR_MISALIGNED, "workspace must be 16-byte aligned");
    a.partial = (int32_t*)workspace;
  }
  return i8_launch_status(launch_gemm_i8(a, cfg->epilogue == QDG_EPI_SILU_MUL, (hipStream_t)stream),
                    "gemm_i8 launch");
}

qdg_status qdg_moe_gemm_i8(const qdg_i8_config* cfg, const int8_t* A, const float* a_scales, const int32_t* a_zeros,
                           const int8_t* B, const float* b_scales, const float* bias, const int32_t* sorted_ids,
                           const int32_t* block_expert, const int32_t* num_padded, int64_t T, int32_t top_k,
                           int32_t block_m, int32_t a_per_pair, void* Y, void* stream) {
  qdg_status st = check_i8(cfg);
  if (st != QDG_OK) return st;
  int64_t capacity = 0;  // also checks T, top_k, num_experts and block_m
  st = qdg_moe_align_capacity(T, top_k, cfg->num_experts, block_m, &capacity);
  if (st != QDG_OK) return st;
  if (T == 0) return QDG_OK;
  if (!sorted_ids || !block_expert || !num_padded) return fail(QDG_ERR_INVALID_ARG, "NULL routing array");
  if (!aligned(sorted_ids, 4) || !aligned(block_expert, 4) || !aligned(num_padded, 4))
    return fail(QDG_ERR_MISALIGNED, "routing arrays must be 4-byte aligned");
  I8Args a;
  st = i8_args(cfg, A, a_scales, a_zeros, B, b_scales, bias, Y, &a);
  if (st != QDG_OK) return st;
  a.M = (int)(a_per_pair ? T * top_k : T);
  a.sorted_ids = sorted_ids;
  a.block_expert = block_expert;
  a.num_padded = num_padded;
  a.num_pairs = (int)(T * top_k);
  a.top_k = top_k;
  a.a_per_pair = a_per_pair ? 1 : 0;
  a.block_m = block_m;
  if ((int64_t)a.M * a.lda > (int64_t)kI8FarRow)
    return fail(QDG_ERR_UNSUPPORTED, "A is longer than 3.75 GiB: route fewer tokens at a time");
  return i8_launch_status(launch_moe_gemm_i8(a, cfg->epilogue == QDG_EPI_SILU_MUL, (int)(capacity / block_m),
                                       (hipStream_t)stream),
                    "moe_gemm_i8 launch");
}

}  // extern "C"
