// C ABI of the operators at the ends of a model: token embedding and layer norm.
// Validation runs on the host before any HIP call.
#include <math.h>

#include "flce_embed.h"
#include "flce_norm.h"

namespace flce {

static bool ends_dtype_ok(int d) { return d == FLCE_F32 || d == FLCE_BF16 || d == FLCE_F16; }
static bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
static size_t size_of(int dtype) { return dtype == FLCE_F32 ? 4 : 2; }

static constexpr int64_t kMaxNormRows = int64_t(1) << 31;
static constexpr int64_t kMaxNormCols = int64_t(1) << 20;
static constexpr int64_t kMaxElements = int64_t(1) << 40;

static int norm_args(const flce_norm_params* p, NormArgs* a) {
  if (!p || p->rows < 0 || p->cols < 1 || p->ld_x < 0 || p->ld_grad < 0) return FLCE_ERR_INVALID_ARG;
  if (!ends_dtype_ok(p->dtype) || (p->param_dtype != p->dtype && p->param_dtype != FLCE_F32) || p->reserved != 0)
    return FLCE_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f) || !isfinite(p->eps)) return FLCE_ERR_INVALID_ARG;
  *a = NormArgs{};
  a->rows = p->rows;
  a->ld_x = p->ld_x ? p->ld_x : p->cols;
  a->ld_dy = p->ld_grad ? p->ld_grad : p->cols;
  if (a->ld_x < p->cols || a->ld_dy < p->cols) return FLCE_ERR_INVALID_ARG;
  if (p->rows > kMaxNormRows || p->cols > kMaxNormCols) return FLCE_ERR_UNSUPPORTED;
  if (p->rows > 0 && (a->ld_x > kMaxElements / p->rows || a->ld_dy > kMaxElements / p->rows)) return FLCE_ERR_UNSUPPORTED;
  a->cols = (int)p->cols;
  a->eps = p->eps;
  a->dtype = p->dtype;
  a->param_dtype = p->param_dtype;
  a->parts = norm_parts(p->rows, p->cols);
  return FLCE_OK;
}

// Token numbers and rows are held in 32 bits by the gradient's sort.
static constexpr int64_t kMaxEmbedRows = (int64_t(1) << 31) - 1;

static int embedding_plan(const flce_embedding_params* p, EmbedPlan* pl) {
  if (!p || p->n_tokens < 0 || p->hidden < 1 || p->vocab < 1) return FLCE_ERR_INVALID_ARG;
  if (!ends_dtype_ok(p->dtype) || !ends_dtype_ok(p->grad_weight_dtype)) return FLCE_ERR_INVALID_ARG;
  if ((p->flags & ~(FLCE_ACCUMULATE_GRAD_WEIGHT | FLCE_TARGETS_INT32)) != 0 || !isfinite(p->scale))
    return FLCE_ERR_INVALID_ARG;
  if (p->n_tokens > kMaxEmbedRows || p->vocab > kMaxEmbedRows || p->hidden > (int64_t(1) << 20))
    return FLCE_ERR_UNSUPPORTED;
  if (p->n_tokens > kMaxElements / p->hidden || p->vocab > kMaxElements / p->hidden) return FLCE_ERR_UNSUPPORTED;
  *pl = EmbedPlan{};
  pl->n = p->n_tokens;
  pl->v = p->vocab;
  pl->h = (int)p->hidden;
  pl->dtype = p->dtype;
  pl->grad_dtype = p->grad_weight_dtype;
  pl->ids_i32 = (p->flags & FLCE_TARGETS_INT32) != 0;
  pl->accumulate = (p->flags & FLCE_ACCUMULATE_GRAD_WEIGHT) != 0;
  pl->scale = p->scale;
  pl->ignore_index = p->ignore_index;
  plan_embedding_backward(pl);
  return FLCE_OK;
}

}  // namespace flce

using namespace flce;

extern "C" {

int flce_embedding_workspace_size(const flce_embedding_params* p, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  EmbedPlan pl;
  const int rc = embedding_plan(p, &pl);
  if (rc != FLCE_OK) return rc;
  *bytes = pl.w_bytes;
  return FLCE_OK;
}

int flce_embedding_forward(const flce_embedding_params* p, const void* ids, const void* weight, void* out,
                           void* stream) {
  EmbedPlan pl;
  const int rc = embedding_plan(p, &pl);
  if (rc != FLCE_OK) return rc;
  if (pl.n > 0 && (!ids || !weight || !out)) return FLCE_ERR_INVALID_ARG;
  const size_t e = size_of(pl.dtype);
  if (!aligned_to(ids, pl.ids_i32 ? 4 : 8) || !aligned_to(weight, e) || !aligned_to(out, e)) return FLCE_ERR_UNSUPPORTED;
  return launch_embedding_forward(pl, ids, weight, out, static_cast<hipStream_t>(stream)) == hipSuccess ? FLCE_OK
                                                                                                      : FLCE_ERR_HIP;
}

int flce_embedding_backward(const flce_embedding_params* p, const void* ids, const void* grad_out, void* grad_weight,
                            void* workspace, size_t workspace_bytes, void* stream) {
  EmbedPlan pl;
  const int rc = embedding_plan(p, &pl);
  if (rc != FLCE_OK) return rc;
  if (!grad_weight || !workspace || (pl.n > 0 && (!ids || !grad_out))) return FLCE_ERR_INVALID_ARG;
  if (!aligned_to(ids, pl.ids_i32 ? 4 : 8) || !aligned_to(grad_out, size_of(pl.dtype)) ||
      !aligned_to(grad_weight, size_of(pl.grad_dtype)) || !aligned_to(workspace, 16))
    return FLCE_ERR_UNSUPPORTED;
  if (workspace_bytes < pl.w_bytes) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  const hipError_t e = launch_embedding_backward(pl, ids, grad_out, grad_weight, static_cast<char*>(workspace),
                                                 static_cast<hipStream_t>(stream));
  return e == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

int flce_layer_norm_workspace_size(const flce_norm_params* p, size_t* bytes) {
  if (!bytes) return FLCE_ERR_INVALID_ARG;
  NormArgs a;
  const int rc = norm_args(p, &a);
  if (rc != FLCE_OK) return rc;
  *bytes = (size_t(a.parts) * 2 * size_t(a.cols) * 4 + 255) / 256 * 256;
  return FLCE_OK;
}

int flce_layer_norm_forward(const flce_norm_params* p, const void* x, const void* weight, const void* bias, void* y,
                            float* mean, float* rstd, void* stream) {
  NormArgs a;
  const int rc = norm_args(p, &a);
  if (rc != FLCE_OK) return rc;
  if ((a.rows > 0 && (!x || !y)) || (mean == nullptr) != (rstd == nullptr)) return FLCE_ERR_INVALID_ARG;
  const size_t e = size_of(a.dtype), pe = size_of(a.param_dtype);
  if (!aligned_to(x, e) || !aligned_to(y, e) || !aligned_to(weight, pe) || !aligned_to(bias, pe) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return FLCE_ERR_UNSUPPORTED;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  return launch_norm_forward(a, static_cast<hipStream_t>(stream)) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

int flce_layer_norm_backward(const flce_norm_params* p, const void* x, const void* weight, const float* mean,
                             const float* rstd, const void* grad_y, void* grad_x, void* grad_weight, void* grad_bias,
                             void* workspace, size_t workspace_bytes, void* stream) {
  NormArgs a;
  const int rc = norm_args(p, &a);
  if (rc != FLCE_OK) return rc;
  if (a.rows > 0 && (!x || !mean || !rstd || !grad_y)) return FLCE_ERR_INVALID_ARG;
  const bool columns = grad_weight || grad_bias;
  if (columns && !workspace) return FLCE_ERR_INVALID_ARG;
  const size_t e = size_of(a.dtype), pe = size_of(a.param_dtype);
  if (!aligned_to(x, e) || !aligned_to(weight, pe) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
      !aligned_to(grad_y, e) || !aligned_to(grad_x, e) || !aligned_to(grad_weight, pe) || !aligned_to(grad_bias, pe) ||
      !aligned_to(workspace, 16))
    return FLCE_ERR_UNSUPPORTED;
  size_t need = 0;
  (void)flce_layer_norm_workspace_size(p, &need);
  if (columns && workspace_bytes < need) return FLCE_ERR_WORKSPACE_TOO_SMALL;
  a.x = x;
  a.weight = weight;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = grad_y;
  a.dx = grad_x;
  a.dw = grad_weight;
  a.db = grad_bias;
  a.part = static_cast<float*>(workspace);
  return launch_norm_backward(a, static_cast<hipStream_t>(stream)) == hipSuccess ? FLCE_OK : FLCE_ERR_HIP;
}

}  // extern "C"
