// C ABI of the operators around the products: norms with gate, residual and
// codes, the gated activation, and low-rank adapters. Validation here, kernels
// in row_ops.hip and lora.hip.
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

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool is_float(int32_t type) { return type == QDG_O_BF16 || type == QDG_O_F32; }
size_t size_of(int32_t type) { return type == QDG_O_F32 ? 4 : 2; }

constexpr int64_t kMaxRows = (int64_t)1 << 31;
constexpr int64_t kMaxStride = (int64_t)1 << 31;
constexpr int64_t kMaxNorm = 32768, kMaxGated = 65536;
constexpr int64_t kMaxSide = (int64_t)1 << 20;
constexpr int64_t kMaxLoraRows = (int64_t)1 << 20;

bool bad_stride(int64_t ld, int64_t n) { return ld < n || ld > kMaxStride; }

// Where rows and codes go; `any`: whether there are any.
qdg_status check_out(int64_t n, int32_t quant, int64_t ldo, int64_t ldq, void* out, void* qa, void* a_scales,
                     int32_t* a_zeros, bool pointers, RowOut* o) {
  if (quant < QDG_Q_NONE || quant > QDG_Q_MXFP4) return fail(QDG_ERR_INVALID_ARG, "bad quant");
  if (out && bad_stride(ldo, n)) return fail(QDG_ERR_INVALID_ARG, "ldo must be in [n, 2^31]");
  if (!aligned(out, 2)) return fail(QDG_ERR_MISALIGNED, "out must be aligned to its element");
  *o = {};
  o->rows = (uint16_t*)out;
  o->ld = ldo;
  o->quant = quant;
  if (quant == QDG_Q_NONE) return QDG_OK;
  if (quant == QDG_Q_FP8E4M3 && n % 128) return fail(QDG_ERR_UNSUPPORTED, "fp8 codes need n a multiple of 128");
  if (quant == QDG_Q_MXFP4 && n % 32) return fail(QDG_ERR_UNSUPPORTED, "MXFP4 codes need n a multiple of 32");
  const int64_t bytes = quant == QDG_Q_MXFP4 ? n / 2 : n;
  if (bad_stride(ldq, bytes)) return fail(QDG_ERR_INVALID_ARG, "ldq must be in [the bytes of a row, 2^31]");
  if (ldq % 16) return fail(QDG_ERR_MISALIGNED, "ldq must be a multiple of 16 bytes");
  if (pointers) {
    if (!qa || !a_scales) return fail(QDG_ERR_INVALID_ARG, "qa or a_scales is NULL");
    if (quant == QDG_Q_INT8_ZP && !a_zeros) return fail(QDG_ERR_INVALID_ARG, "a_zeros is NULL");
  }
  if (!aligned(qa, 16)) return fail(QDG_ERR_MISALIGNED, "qa must be 16-byte aligned");
  if (quant != QDG_Q_MXFP4 && !aligned(a_scales, 4)) return fail(QDG_ERR_MISALIGNED, "a_scales must be 4-byte aligned");
  if (!aligned(a_zeros, 4)) return fail(QDG_ERR_MISALIGNED, "a_zeros must be 4-byte aligned");
  o->qa = (uint8_t*)qa;
  o->ldq = ldq;
  o->scales = a_scales;
  o->zeros = a_zeros;
  return QDG_OK;
}

qdg_status check_block_m(int32_t block_m) {
  if (block_m != 16 && block_m != 32 && block_m != 64 && block_m != 128)
    return fail(QDG_ERR_UNSUPPORTED, "block_m must be 16, 32, 64 or 128");
  return QDG_OK;
}

qdg_status check_lora(const qdg_lora_config* c, int64_t M, int32_t block_m) {
  if (!c) return fail(QDG_ERR_INVALID_ARG, "config is NULL");
  if (c->n < 1 || c->k < 1 || c->rank < 1 || c->num_adapters < 1 || c->num_slices < 1)
    return fail(QDG_ERR_INVALID_ARG, "n, k, rank, num_adapters and num_slices must be positive");
  if (c->n > kMaxSide || c->k > kMaxSide) return fail(QDG_ERR_UNSUPPORTED, "n and k must be at most 2^20");
  if (c->rank > 256) return fail(QDG_ERR_UNSUPPORTED, "rank must be at most 256");
  if (c->num_adapters > 1024) return fail(QDG_ERR_UNSUPPORTED, "at most 1024 adapters");
  if (c->num_slices > 4) return fail(QDG_ERR_UNSUPPORTED, "at most 4 slices");
  for (int i = 0; i < c->num_slices; ++i)
    if (c->slice_end[i] <= (i ? c->slice_end[i - 1] : 0))
      return fail(QDG_ERR_INVALID_ARG, "slice_end must ascend from above 0");
  if (c->slice_end[c->num_slices - 1] != c->n) return fail(QDG_ERR_INVALID_ARG, "the last slice must end at n");
  if (!is_float(c->otype)) return fail(QDG_ERR_INVALID_ARG, "otype must be BF16 or F32");
  if (bad_stride(c->ldx, c->k) || bad_stride(c->ldy, c->n))
    return fail(QDG_ERR_INVALID_ARG, "a row stride is shorter than its row or above 2^31");
  if (M < 0) return fail(QDG_ERR_INVALID_ARG, "M < 0");
  if (M > kMaxLoraRows) return fail(QDG_ERR_UNSUPPORTED, "M must be at most 2^20");
  return check_block_m(block_m);
}

// The geometry of a call whose rows make up to `blocks` blocks, and what runs it.
LoraArgs lora_geometry(const qdg_lora_config* c, int64_t blocks, int32_t block_m) {
  LoraArgs a = {};
  a.ldx = c->ldx;
  a.ldy = c->ldy;
  a.n = (int)c->n;
  a.k = (int)c->k;
  a.num_adapters = c->num_adapters;
  a.num_slices = c->num_slices;
  a.rank = c->rank;
  for (int i = 0; i < c->num_slices; ++i) a.slice_end[i] = (int)c->slice_end[i];
  a.block_m = block_m;
  a.block_shift = block_m == 16 ? 0 : block_m == 32 ? 1 : block_m == 64 ? 2 : 3;
  a.blocks = (int)blocks;
  a.yf32 = c->otype == QDG_O_F32;
  lora_choose(&a);
  return a;
}

// Bytes of the inner sums.
int64_t lora_bytes(const LoraArgs& a) {
  return a.fused ? 0 : (int64_t)a.split * a.blocks * a.block_m * a.num_slices * a.rank_pad * (int64_t)sizeof(float);
}

}  // namespace

extern "C" {

qdg_status qdg_norm(const qdg_norm_config* cfg, const void* x, const void* residual, const void* gate,
                    const void* post_weight, const void* post_bias, const void* weight, const void* bias, int64_t M,
                    void* residual_out, void* out, void* qa, void* a_scales, int32_t* a_zeros, void* stream) {
  if (!cfg) return fail(QDG_ERR_INVALID_ARG, "config is NULL");
  const qdg_norm_config& c = *cfg;
  if (c.n < 1 || M < 0) return fail(QDG_ERR_INVALID_ARG, "bad n or M");
  if (c.n > kMaxNorm) return fail(QDG_ERR_UNSUPPORTED, "n must be at most 32768");
  if (M >= kMaxRows) return fail(QDG_ERR_UNSUPPORTED, "M must be below 2^31");
  if (c.kind != QDG_NORM_RMS && c.kind != QDG_NORM_LAYER) return fail(QDG_ERR_INVALID_ARG, "bad kind");
  if (c.post_norm != 0 && c.post_norm != 1) return fail(QDG_ERR_INVALID_ARG, "post_norm must be 0 or 1");
  if (!is_float(c.xtype) || !is_float(c.rtype) || !is_float(c.wtype))
    return fail(QDG_ERR_INVALID_ARG, "xtype, rtype and wtype must be BF16 or F32");
  if (c.reserved != 0) return fail(QDG_ERR_INVALID_ARG, "reserved must be 0");
  if (!(c.eps >= 0.0f) || !std::isfinite(c.eps) || !std::isfinite(c.residual_scale) || !std::isfinite(c.weight_offset))
    return fail(QDG_ERR_INVALID_ARG, "eps must not be negative; eps, residual_scale and weight_offset must be finite");
  RowOut o;
  const qdg_status st = check_out(c.n, c.quant, c.ldo, c.ldq, out, qa, a_scales, a_zeros, M > 0, &o);
  if (st != QDG_OK) return st;
  if (bad_stride(c.ldx, c.n) || (residual && bad_stride(c.ldr, c.n)) || (residual_out && bad_stride(c.lds, c.n)) ||
      (gate && c.ldg != 0 && bad_stride(c.ldg, c.n)))
    return fail(QDG_ERR_INVALID_ARG, "a row stride is shorter than its row or above 2^31");
  if (!c.post_norm && (post_weight || post_bias))
    return fail(QDG_ERR_INVALID_ARG, "post_weight and post_bias need post_norm");
  if (M == 0) return QDG_OK;
  if (!x) return fail(QDG_ERR_INVALID_ARG, "x is NULL");
  if (!residual_out && !out && c.quant == QDG_Q_NONE)
    return fail(QDG_ERR_INVALID_ARG, "no output: residual_out, out or codes");
  if (!aligned(x, size_of(c.xtype)) || !aligned(residual, size_of(c.rtype)) || !aligned(residual_out, size_of(c.rtype)) ||
      !aligned(gate, size_of(c.wtype)) || !aligned(post_weight, size_of(c.wtype)) ||
      !aligned(post_bias, size_of(c.wtype)) || !aligned(weight, size_of(c.wtype)) || !aligned(bias, size_of(c.wtype)))
    return fail(QDG_ERR_MISALIGNED, "pointers must be aligned to their elements");
  if (residual_out && residual_out == residual && c.lds != c.ldr)
    return fail(QDG_ERR_INVALID_ARG, "a residual updated in place has one stride: lds must be ldr");
  if (out && out == x && (c.xtype != QDG_O_BF16 || c.ldo != c.ldx))
    return fail(QDG_ERR_INVALID_ARG, "rows written over x need bf16 x and ldo = ldx");
  NormArgs a = {};
  a.x = x;
  a.residual = residual;
  a.gate = gate;
  a.post_weight = post_weight;
  a.post_bias = post_bias;
  a.weight = weight;
  a.bias = bias;
  a.residual_out = residual_out;
  a.ldx = c.ldx;
  a.ldr = c.ldr;
  a.ldg = c.ldg;
  a.lds = c.lds;
  a.M = M;
  a.n = (int)c.n;
  a.layer = c.kind == QDG_NORM_LAYER;
  a.post_norm = c.post_norm != 0;
  a.wf32 = c.wtype == QDG_O_F32;
  a.short_join = !a.post_norm && (!gate || (c.xtype == QDG_O_BF16 && !a.wf32));
  a.eps = c.eps;
  a.inv_n = 1.0 / (double)c.n;
  a.residual_scale = c.residual_scale;
  a.weight_offset = c.weight_offset;
  a.out = o;
  return hip_status(launch_norm(a, c.xtype == QDG_O_F32, c.rtype == QDG_O_F32, (hipStream_t)stream), "norm launch");
}

qdg_status qdg_gated_act(const qdg_gated_config* cfg, const void* Y, int64_t M, void* out, void* qa, void* a_scales,
                         int32_t* a_zeros, void* stream) {
  if (!cfg) return fail(QDG_ERR_INVALID_ARG, "config is NULL");
  const qdg_gated_config& c = *cfg;
  if (c.n < 1 || M < 0) return fail(QDG_ERR_INVALID_ARG, "bad n or M");
  if (c.n > kMaxGated) return fail(QDG_ERR_UNSUPPORTED, "n must be at most 65536");
  if (M >= kMaxRows) return fail(QDG_ERR_UNSUPPORTED, "M must be below 2^31");
  if (c.act != QDG_ACT_SILU && c.act != QDG_ACT_GELU_TANH) return fail(QDG_ERR_INVALID_ARG, "bad act");
  if (!is_float(c.ytype)) return fail(QDG_ERR_INVALID_ARG, "ytype must be BF16 or F32");
  if (c.reserved != 0) return fail(QDG_ERR_INVALID_ARG, "reserved must be 0");
  RowOut o;
  const qdg_status st = check_out(c.n, c.quant, c.ldo, c.ldq, out, qa, a_scales, a_zeros, M > 0, &o);
  if (st != QDG_OK) return st;
  if (bad_stride(c.ldy, 2 * c.n)) return fail(QDG_ERR_INVALID_ARG, "ldy must be in [2 n, 2^31]");
  if (M == 0) return QDG_OK;
  if (!Y) return fail(QDG_ERR_INVALID_ARG, "Y is NULL");
  if (!out && c.quant == QDG_Q_NONE) return fail(QDG_ERR_INVALID_ARG, "no output: out or codes");
  if (!aligned(Y, size_of(c.ytype))) return fail(QDG_ERR_MISALIGNED, "Y must be aligned to its element");
  GatedArgs a = {};
  a.y = Y;
  a.ldy = c.ldy;
  a.M = M;
  a.n = (int)c.n;
  a.act = c.act;
  a.out = o;
  return hip_status(launch_gated_act(a, c.ytype == QDG_O_F32, (hipStream_t)stream), "gated_act launch");
}

qdg_status qdg_lora_workspace(const qdg_lora_config* cfg, int64_t M, int32_t block_m, size_t* bytes) {
  const qdg_status st = check_lora(cfg, M, block_m);
  if (st != QDG_OK) return st;
  if (!bytes) return fail(QDG_ERR_INVALID_ARG, "bytes is NULL");
  // fewer blocks may be split where many are not; from 512 blocks on none is
  int64_t most = 0;
  const int64_t blocks = M > 0 ? lora_blocks(M, cfg->num_adapters, block_m) : 0;
  for (int64_t b = 1; b <= blocks; ++b) {
    if (b == 513) b = blocks;
    const int64_t need = lora_bytes(lora_geometry(cfg, b, block_m));
    most = need > most ? need : most;
  }
  *bytes = (size_t)most;
  return QDG_OK;
}

qdg_status qdg_lora(const qdg_lora_config* cfg, const void* X, const void* A, const void* B, const int32_t* ranks,
                    const float* scales, const int32_t* sorted_ids, const int32_t* block_adapter,
                    const int32_t* num_padded, int64_t M, int32_t block_m, void* Y, void* workspace, size_t ws_bytes,
                    void* stream) {
  const qdg_status st = check_lora(cfg, M, block_m);
  if (st != QDG_OK) return st;
  if (M == 0) return QDG_OK;
  if (!X || !A || !B || !Y) return fail(QDG_ERR_INVALID_ARG, "NULL pointer");
  if (!sorted_ids || !block_adapter || !num_padded) return fail(QDG_ERR_INVALID_ARG, "NULL grouping array");
  if (!aligned(X, 2) || !aligned(A, 2) || !aligned(B, 2) || !aligned(Y, size_of(cfg->otype)) || !aligned(ranks, 4) ||
      !aligned(scales, 4) || !aligned(sorted_ids, 4) || !aligned(block_adapter, 4) || !aligned(num_padded, 4))
    return fail(QDG_ERR_MISALIGNED, "pointers must be aligned to their elements");
  LoraArgs a = lora_geometry(cfg, lora_blocks(M, cfg->num_adapters, block_m), block_m);
  const size_t need = (size_t)lora_bytes(a);
  if (need > 0 && (!workspace || ws_bytes < need))
    return fail(QDG_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", workspace ? ws_bytes : 0, need);
  if (!aligned(workspace, 16)) return fail(QDG_ERR_MISALIGNED, "workspace must be 16-byte aligned");
  a.X = (const uint16_t*)X;
  a.A = (const uint16_t*)A;
  a.B = (const uint16_t*)B;
  a.X_last = a.X + (M - 1) * cfg->ldx + cfg->k - 8;
  a.A_last = a.A + (int64_t)cfg->num_adapters * cfg->num_slices * cfg->rank * cfg->k - 8;
  a.B_last = a.B + (int64_t)cfg->num_adapters * cfg->n * cfg->rank - 8;
  a.ranks = ranks;
  a.scales = scales;
  a.sorted_ids = sorted_ids;
  a.block_adapter = block_adapter;
  a.num_padded = num_padded;
  a.Y = Y;
  a.partial = (float*)workspace;
  a.M = M;
  const hipError_t e = launch_lora(a, (hipStream_t)stream);
  if (e == hipErrorInvalidConfiguration)
    return fail(QDG_ERR_UNSUPPORTED, "lora: the output has more tiles than one launch holds (2^32 threads)");
  return hip_status(e, "lora launch");
}

}  // extern "C"
