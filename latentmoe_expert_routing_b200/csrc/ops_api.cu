// C ABI of the stand-alone operators: argument checks, then one launch each.
#include <cuda_runtime.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "latentmoe.h"

using namespace lmoe;

namespace {

bool multiple16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool known(moe_dtype d) { return d == MOE_FP32 || d == MOE_BF16; }
int64_t bytes_of(moe_dtype d) { return d == MOE_BF16 ? 2 : 4; }
moe_status done(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

moe_status check_route(const void* logits, moe_dtype dtype, int64_t ld, int T, int E, int k,
                       moe_score score, float scale) {
  if (T < 0 || E <= 0 || k <= 0 || k > E || ld < E || !known(dtype) || !(scale - scale == 0.f) ||
      (score != MOE_SCORE_SIGMOID && score != MOE_SCORE_SOFTMAX))
    return MOE_ERR_INVALID_ARG;
  if (E > 1024 || k > 64) return MOE_ERR_UNSUPPORTED;
  if (T > 0 && (!logits || !aligned(logits, bytes_of(dtype)))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// rows of D elements at p, ld apart
bool rows_ok(const void* p, int64_t ld, int D, moe_dtype dt) {
  return p && multiple16(p) && ld >= D && (ld * bytes_of(dt)) % 16 == 0;
}

moe_status check_norm(const moe_norm_args* a) {
  if (!a || a->T < 0 || a->D <= 0 || a->D % 8 || !known(a->dtype)) return MOE_ERR_INVALID_ARG;
  if (!(a->eps > 0.f) || !(a->eps < INFINITY) || !(a->residual_scale - a->residual_scale == 0.f))
    return MOE_ERR_INVALID_ARG;
  if (a->gate_kind < MOE_GATE_NONE || a->gate_kind > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
  if (a->D > 16384) return MOE_ERR_UNSUPPORTED;
  if (a->post_weight && !multiple16(a->post_weight)) return MOE_ERR_INVALID_ARG;
  if (a->pre_weight && !multiple16(a->pre_weight)) return MOE_ERR_INVALID_ARG;
  if (a->T == 0) return MOE_OK;
  switch (a->gate_kind) {
    case MOE_GATE_CHANNEL:
      if (!a->gate || !multiple16(a->gate)) return MOE_ERR_INVALID_ARG;
      break;
    case MOE_GATE_TOKEN:
      if (!a->gate || !aligned(a->gate, bytes_of(a->dtype)) || a->ldg < 1) return MOE_ERR_INVALID_ARG;
      break;
    case MOE_GATE_FULL:
      if (!rows_ok(a->gate, a->ldg, a->D, a->dtype)) return MOE_ERR_INVALID_ARG;
      break;
    default:
      break;
  }
  if (!rows_ok(a->y, a->ldy, a->D, a->dtype) || !rows_ok(a->r, a->ldr, a->D, a->dtype))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

bool codes_ok(const void* p, int64_t ld, int64_t K) { return p && multiple16(p) && ld >= K && ld % 16 == 0; }

}  // namespace

extern "C" {

moe_status moe_route_topk(const void* logits, moe_dtype dtype, int64_t ld, const float* bias,
                          int T, int n_experts, int top_k, moe_score score, int n_group,
                          int topk_group, int renorm, float scale, int32_t* topk_idx,
                          float* topk_w, void* stream) {
  if (n_group < 1 || topk_group < 1 || topk_group > n_group) return MOE_ERR_INVALID_ARG;
  if (n_group > 1 && n_experts > 0 &&
      (n_experts % n_group || n_experts / n_group < 2 ||
       top_k > (int64_t)topk_group * (n_experts / n_group)))
    return MOE_ERR_INVALID_ARG;
  const moe_status st = check_route(logits, dtype, ld, T, n_experts, top_k, score, scale);
  if (st != MOE_OK) return st;
  if (n_group > 64) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!topk_idx || !topk_w || !aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(bias, 4))
    return MOE_ERR_INVALID_ARG;
  return done(launch_route_topk(logits, dtype, ld, bias, T, n_experts, top_k, score, n_group,
                                topk_group, renorm != 0, scale, topk_idx, topk_w,
                                (cudaStream_t)stream));
}

moe_status moe_route_topk_backward(const void* logits, moe_dtype dtype, int64_t ld,
                                   const int32_t* topk_idx, const float* topk_w, const float* dw,
                                   int T, int n_experts, int top_k, moe_score score, int renorm,
                                   float scale, void* dlogits, int64_t ldd, void* stream) {
  const moe_status st = check_route(logits, dtype, ld, T, n_experts, top_k, score, scale);
  if (st != MOE_OK) return st;
  if (ldd < n_experts) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!topk_idx || !topk_w || !dw || !dlogits || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
      !aligned(dw, 4) || !aligned(dlogits, bytes_of(dtype)))
    return MOE_ERR_INVALID_ARG;
  return done(launch_route_topk_bwd(logits, dtype, ld, topk_idx, topk_w, dw, T, n_experts, top_k,
                                    score, renorm != 0, scale, dlogits, ldd,
                                    (cudaStream_t)stream));
}

size_t moe_route_group_workspace(int T, int top_k, int n_experts) {
  if (T < 0 || top_k <= 0 || n_experts <= 0) return 0;
  return route_group_workspace((long)T * top_k, n_experts);
}

moe_status moe_route_group(const int32_t* topk_idx, int T, int top_k, int n_experts,
                           int32_t* counts, int32_t* offsets, int32_t* perm, int32_t* pos,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const int64_t P = (int64_t)T * top_k;
  if (T < 0 || top_k <= 0 || n_experts <= 0 || P > 0x7fffffff || !counts || !offsets ||
      !aligned(counts, 4) || !aligned(offsets, 4))
    return MOE_ERR_INVALID_ARG;
  if (n_experts > 1024) return MOE_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  if (P == 0) {
    cudaError_t e = cudaMemsetAsync(counts, 0, (size_t)n_experts * 4, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(offsets, 0, (size_t)(n_experts + 1) * 4, s);
    return done(e);
  }
  if (!topk_idx || !perm || !pos || !workspace || !aligned(topk_idx, 4) || !aligned(perm, 4) ||
      !aligned(pos, 4) || !multiple16(workspace) ||
      workspace_bytes < route_group_workspace(P, n_experts))
    return MOE_ERR_INVALID_ARG;
  return done(launch_route_group(topk_idx, P, n_experts, counts, offsets, perm, pos, workspace, s));
}

moe_status moe_norm_residual(const moe_norm_args* a, void* stream) {
  const moe_status st = check_norm(a);
  if (st != MOE_OK) return st;
  if (a->T == 0) return MOE_OK;
  if (!rows_ok(a->x, a->ldx, a->D, a->dtype)) return MOE_ERR_INVALID_ARG;
  if (a->pre_weight && !rows_ok(a->h, a->ldh, a->D, a->dtype)) return MOE_ERR_INVALID_ARG;
  if (!aligned(a->rstd_y, 4) || !aligned(a->rstd_r, 4)) return MOE_ERR_INVALID_ARG;
  return done(launch_norm_fwd(*a, (cudaStream_t)stream));
}

size_t moe_norm_residual_workspace(int T, int D) {
  // nothing for what the gradient refuses (below 8 columns there is no shape at all)
  return T <= 0 || D <= 0 || D % 8 || D > 16384 ? 0 : norm_bwd_workspace(T, D);
}

moe_status moe_norm_residual_backward(const moe_norm_args* a, void* workspace,
                                      size_t workspace_bytes, void* stream) {
  const moe_status st = check_norm(a);
  if (st != MOE_OK) return st;
  if ((a->post_weight && (!a->dpost_weight || !multiple16(a->dpost_weight))) ||
      (a->pre_weight && (!a->dpre_weight || !multiple16(a->dpre_weight))))
    return MOE_ERR_INVALID_ARG;
  cudaStream_t s = (cudaStream_t)stream;
  const bool gate_sum = a->gate_kind == MOE_GATE_CHANNEL;
  if (gate_sum && (!a->dgate || !multiple16(a->dgate))) return MOE_ERR_INVALID_ARG;
  if (a->T == 0) {
    cudaError_t e = cudaSuccess;
    const size_t n = (size_t)a->D * 4;
    if (a->post_weight) e = cudaMemsetAsync(a->dpost_weight, 0, n, s);
    if (e == cudaSuccess && a->pre_weight) e = cudaMemsetAsync(a->dpre_weight, 0, n, s);
    if (e == cudaSuccess && gate_sum) e = cudaMemsetAsync(a->dgate, 0, n, s);
    return done(e);
  }
  if (!rows_ok(a->dx, a->lddx, a->D, a->dtype) || !rows_ok(a->dy, a->lddy, a->D, a->dtype))
    return MOE_ERR_INVALID_ARG;
  if (a->dr && !rows_ok(a->dr, a->lddr, a->D, a->dtype)) return MOE_ERR_INVALID_ARG;
  if (a->pre_weight && (!rows_ok(a->dh, a->lddh, a->D, a->dtype) || !a->rstd_r || !aligned(a->rstd_r, 4)))
    return MOE_ERR_INVALID_ARG;
  if (a->post_weight && (!a->rstd_y || !aligned(a->rstd_y, 4))) return MOE_ERR_INVALID_ARG;
  if (a->gate_kind == MOE_GATE_TOKEN && (!a->dgate || !aligned(a->dgate, 4))) return MOE_ERR_INVALID_ARG;
  if (a->gate_kind == MOE_GATE_FULL && !rows_ok(a->dgate, a->lddg, a->D, a->dtype))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || !multiple16(workspace) || workspace_bytes < norm_bwd_workspace(a->T, a->D))
    return MOE_ERR_INVALID_ARG;
  return done(launch_norm_bwd(*a, workspace, s));
}

moe_status moe_quantize_fp8(const void* x, moe_dtype dtype, int x_rows, int K, int64_t ldx,
                            const int32_t* perm, int rows, int k, int relu2, uint8_t* codes,
                            int64_t ldc, float* scales, int64_t lds, void* stream) {
  if (x_rows < 0 || rows < 0 || K <= 0 || ldx < K || !known(dtype) || lds < rows || ldc < K ||
      ldc % 16 || (perm ? k <= 0 : rows != x_rows))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if ((!x && x_rows > 0) || !aligned(x, bytes_of(dtype)) || !aligned(perm, 4) || !scales ||
      !aligned(scales, 4) || !codes_ok(codes, ldc, K))
    return MOE_ERR_INVALID_ARG;
  if (K > 0x7fffffff - 1024) return MOE_ERR_UNSUPPORTED;      // a CTA's columns end within 32 bits
  return done(launch_quantize_fp8_rows(x, dtype, rows, K, ldx, perm, k, x_rows, relu2 != 0, codes,
                                       ldc, scales, lds, (cudaStream_t)stream));
}

moe_status moe_quantize_fp8_t(const void* x, moe_dtype dtype, int rows, int K, int64_t ldx,
                              uint8_t* codes, int64_t ldc, float* scales, int64_t lds,
                              void* stream) {
  if (rows < 0 || K <= 0 || ldx < K || !known(dtype) || lds < K || ldc < rows || ldc % 16)
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!x || !aligned(x, bytes_of(dtype)) || !scales || !aligned(scales, 4) ||
      !codes_ok(codes, ldc, rows))
    return MOE_ERR_INVALID_ARG;
  if (ceil_div(rows, 128) > 65535) return MOE_ERR_UNSUPPORTED;
  return done(launch_quantize_fp8_cols(x, dtype, rows, K, ldx, codes, ldc, scales, lds,
                                       (cudaStream_t)stream));
}

moe_status moe_quantize_fp8_weight(const void* w, moe_dtype dtype, int n_mat, int N, int K,
                                   int64_t ldw, uint8_t* codes, int64_t ldc, float* scales,
                                   uint8_t* codes_t, int64_t ldct, float* scales_t, void* stream) {
  if (n_mat <= 0 || N <= 0 || K <= 0 || ldw < K || !known(dtype) || !w ||
      !aligned(w, bytes_of(dtype)) || !scales || !aligned(scales, 4) || !codes_ok(codes, ldc, K))
    return MOE_ERR_INVALID_ARG;
  if ((codes_t != nullptr) != (scales_t != nullptr)) return MOE_ERR_INVALID_ARG;
  if (codes_t && (!codes_ok(codes_t, ldct, N) || !aligned(scales_t, 4))) return MOE_ERR_INVALID_ARG;
  if (n_mat > 65535 || ceil_div(K, 128) > 65535) return MOE_ERR_UNSUPPORTED;
  return done(launch_quantize_fp8_weight(w, dtype, n_mat, N, K, ldw, codes, ldc, scales, codes_t,
                                         ldct, scales_t, (cudaStream_t)stream));
}

moe_status moe_gemm_fp8(const moe_fp8_gemm* g, void* stream) {
  if (!g || g->M < 0 || g->N <= 0 || g->K <= 0 || !known(g->out_dtype) || g->ldo < g->N ||
      g->lda_scales < g->M || g->ldb_scales < 0 || (g->ldb_scales > 0 && g->ldb_scales < g->N))
    return MOE_ERR_INVALID_ARG;
  if (g->offsets) {
    if (g->n_groups <= 0 || g->ldb_scales > 0 || !aligned(g->offsets, 4)) return MOE_ERR_INVALID_ARG;
    if (g->n_groups > 1024) return MOE_ERR_UNSUPPORTED;
  }
  if (g->M == 0) return MOE_OK;
  if (!codes_ok(g->a, g->lda, g->K) || !codes_ok(g->b, g->ldb, g->K) || !g->a_scales ||
      !g->b_scales || !aligned(g->a_scales, 4) || !aligned(g->b_scales, 4) || !g->out ||
      !aligned(g->out, bytes_of(g->out_dtype)))
    return MOE_ERR_INVALID_ARG;
  // row coordinates of a TMA box and tile counts are 32-bit
  const int64_t rows_b = (int64_t)(g->offsets ? g->n_groups : 1) * g->N;
  if (rows_b > 0x7fffffff - 256 || g->M > 0x7fffffff - 256 || g->K > 0x7fffffff - 256 ||
      ((int64_t)g->M / 16 + (g->offsets ? g->n_groups : 1)) * ((int64_t)g->N / 128 + 1) > 0x3fffffff)
    return MOE_ERR_UNSUPPORTED;
  return done(launch_fp8_gemm(*g, (cudaStream_t)stream));
}

}  // extern "C"
