// The C ABI of the dense operators: argument checks, scratch and launches.
#include <cuda_runtime.h>

#include <math.h>

#include <algorithm>

#include "dense.cuh"

namespace {

inline cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

enum : int { F32 = 1, HALVES = 2, F8 = 4 };  // types an argument may have

const char *type_name(int32_t t) {
  return t == SS_VALUES_F32 ? "float32" : t == SS_VALUES_BF16 ? "bfloat16" : t == SS_VALUES_F16 ? "float16"
         : t == SS_VALUES_F8 ? "8-bit" : "unknown";
}

// Checks one matrix: its size, leading dimension, type, pointer and the
// pointer's alignment to its type.
ss_status check(ss_handle *h, const ss_dense *m, int64_t rows, int64_t cols, int types, const char *call,
                const char *name) {
  if (!m) return report(h, SS_ERR_INVALID_ARG, "%s: null %s", call, name);
  const int kind = m->type == SS_VALUES_F32                                    ? F32
                   : m->type == SS_VALUES_BF16 || m->type == SS_VALUES_F16     ? HALVES
                   : m->type == SS_VALUES_F8                                   ? F8
                                                                               : 0;
  if (!(kind & types))
    return report(h, SS_ERR_INVALID_ARG, "%s: %s has type %s (%d)", call, name, type_name(m->type), m->type);
  if (m->n_rows != rows || m->n_cols != cols)
    return report(h, SS_ERR_INVALID_ARG, "%s: %s is %lld x %lld, expected %lld x %lld", call, name,
                  (long long)m->n_rows, (long long)m->n_cols, (long long)rows, (long long)cols);
  if (rows < 0 || cols < 0) return report(h, SS_ERR_INVALID_ARG, "%s: %s has a negative size", call, name);
  if (rows >= SS_DENSE_MAX || cols >= SS_DENSE_MAX)
    return report(h, SS_ERR_LIMIT, "%s: %s is beyond %lld rows or columns", call, name, (long long)SS_DENSE_MAX);
  if (m->ld < cols) return report(h, SS_ERR_INVALID_ARG, "%s: %s: ld %lld < %lld columns", call, name, (long long)m->ld, (long long)cols);
  if (rows > 0 && cols > 0 && !m->data) return report(h, SS_ERR_INVALID_ARG, "%s: %s: null data", call, name);
  if (reinterpret_cast<uintptr_t>(m->data) % (uintptr_t)dense::size_of(m->type) != 0)
    return report(h, SS_ERR_INVALID_ARG, "%s: %s is not aligned to its type", call, name);
  return SS_OK;
}

ss_status same_type(ss_handle *h, const ss_dense *m, int32_t type, const char *call, const char *name) {
  if (m->type == type) return SS_OK;
  return report(h, SS_ERR_INVALID_ARG, "%s: %s has type %s, expected %s", call, name, type_name(m->type), type_name(type));
}

ss_status check_kept(ss_handle *h, const ss_kept *m, int64_t rows, int64_t cols, const char *call, const char *name) {
  if (!m) return report(h, SS_ERR_INVALID_ARG, "%s: null %s", call, name);
  if (m->n_rows != rows || m->n_cols != cols)
    return report(h, SS_ERR_INVALID_ARG, "%s: %s is %lld x %lld, expected %lld x %lld", call, name, (long long)m->n_rows,
                  (long long)m->n_cols, (long long)rows, (long long)cols);
  const int64_t groups = (cols + SS_KEPT_GROUP - 1) / SS_KEPT_GROUP;
  if (m->ld < cols || m->ld_scale < groups)
    return report(h, SS_ERR_INVALID_ARG, "%s: %s: ld %lld < %lld columns or ld_scale %lld < %lld groups", call, name,
                  (long long)m->ld, (long long)cols, (long long)m->ld_scale, (long long)groups);
  if (rows > 0 && cols > 0 && (!m->codes || !m->scale)) return report(h, SS_ERR_INVALID_ARG, "%s: %s: null data", call, name);
  return SS_OK;
}

ss_dense or_none(const ss_dense *m) { return m ? *m : ss_dense{nullptr, 0, 0, 0, 0}; }

#define SS_TRY(expr)                        \
  do {                                      \
    const ss_status st_ = (expr);           \
    if (st_ != SS_OK) return st_;           \
  } while (0)
#define SS_RUN(h, call)                                            \
  do {                                                             \
    const cudaError_t e_ = (call);                                 \
    if (e_ != cudaSuccess) return report_cuda((h), e_, #call);     \
  } while (0)

ss_status check_scratch(ss_handle *h, const void *scratch, int64_t bytes, int64_t need, const char *call) {
  if (bytes >= need && (need == 0 || scratch) && reinterpret_cast<uintptr_t>(scratch) % SS_SCRATCH_ALIGN == 0) return SS_OK;
  return report(h, SS_ERR_INVALID_ARG, "%s: %lld bytes of scratch aligned to %d are needed, %lld given at %p", call,
                (long long)need, SS_SCRATCH_ALIGN, (long long)bytes, scratch);
}

ss_status check_distill(ss_handle *h, const ss_dense *logits, const float *scores, const int64_t *items, int32_t k,
                        float temperature, float teacher_temperature, const char *call) {
  if (!logits) return report(h, SS_ERR_INVALID_ARG, "%s: null logits", call);
  SS_TRY(check(h, logits, logits->n_rows, logits->n_cols, F32 | HALVES, call, "logits"));
  if (k < 1 || k > SS_DISTILL_LIST_MAX)
    return report(h, SS_ERR_LIMIT, "%s: k = %d outside [1, %d]", call, k, SS_DISTILL_LIST_MAX);
  if (logits->n_rows > 0 && (!scores || !items)) return report(h, SS_ERR_INVALID_ARG, "%s: null list", call);
  for (float t : {temperature, teacher_temperature})
    if (!(t >= SS_DISTILL_TEMPERATURE_MIN) || !(t <= 1.0f / SS_DISTILL_TEMPERATURE_MIN))
      return report(h, SS_ERR_INVALID_ARG, "%s: temperature %g outside [%g, %g]", call, (double)t,
                    (double)SS_DISTILL_TEMPERATURE_MIN, 1.0 / (double)SS_DISTILL_TEMPERATURE_MIN);
  return SS_OK;
}

distill_args distill_of(const ss_dense *logits, const float *scores, const int64_t *items, int32_t k,
                        float temperature, float teacher_temperature, const float *weight) {
  distill_args a = {};
  a.logits = *logits;
  a.scores = scores;
  a.items = items;
  a.k = k;
  a.temperature = temperature;
  a.teacher_temperature = teacher_temperature;
  a.weight = weight;
  return a;
}

ss_status run_distill(ss_handle *h, const distill_args &a, int32_t mode, void *stream) {
  if (a.logits.n_rows == 0) return SS_OK;
  SS_RUN(h, cudaSetDevice(h->device));
  int queued = 0;
  SS_RUN(h, launch_distill(h, a, mode, as_stream(stream), &queued));
  h->launches += queued;
  return SS_OK;
}

}  // namespace

extern "C" {

ss_status ss_rms_norm(ss_handle *h, const ss_dense *x, const ss_dense *residual, const ss_dense *weight, float eps,
                      const ss_dense *total, const ss_dense *y, float *scale, float *rstd, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_rms_norm";
  if (!x) return report(h, SS_ERR_INVALID_ARG, "%s: null x", call);
  const int64_t R = x->n_rows, D = x->n_cols;
  SS_TRY(check(h, x, R, D, F32 | HALVES, call, "x"));
  if (D < 1) return report(h, SS_ERR_INVALID_ARG, "%s: rows of no columns", call);
  SS_TRY(check(h, weight, 1, D, F32 | HALVES, call, "weight"));
  if (weight->type != SS_VALUES_F32) SS_TRY(same_type(h, weight, x->type, call, "weight"));
  if (residual) {
    SS_TRY(check(h, residual, R, D, F32 | HALVES, call, "residual"));
    SS_TRY(same_type(h, residual, x->type, call, "residual"));
  }
  if (total) {
    if (!residual) return report(h, SS_ERR_INVALID_ARG, "%s: total without a residual (it would be x)", call);
    SS_TRY(check(h, total, R, D, F32 | HALVES, call, "total"));
    SS_TRY(same_type(h, total, x->type, call, "total"));
  }
  SS_TRY(check(h, y, R, D, F32 | HALVES | F8, call, "y"));
  if (y->type != SS_VALUES_F8) SS_TRY(same_type(h, y, x->type, call, "y"));
  if ((y->type == SS_VALUES_F8) != (scale != nullptr) && R > 0)
    return report(h, SS_ERR_INVALID_ARG, "%s: scale goes with an 8-bit y, and only with one", call);
  if (!(eps >= 0.0f) || isinf(eps)) return report(h, SS_ERR_INVALID_ARG, "%s: eps %g", call, (double)eps);
  if (R == 0) return SS_OK;
  SS_RUN(h, cudaSetDevice(h->device));
  rms_args a = {*x, or_none(residual), *weight, or_none(total), *y, scale, rstd, eps};
  int queued = 0;
  SS_RUN(h, launch_rms_norm(h, a, as_stream(stream), &queued));
  h->launches += queued;
  return SS_OK;
}

int64_t ss_rms_norm_backward_scratch(const ss_handle *h, int64_t n_rows, int64_t n_cols) {
  return h && n_rows > 0 && n_cols > 0 && n_rows < SS_DENSE_MAX && n_cols < SS_DENSE_MAX
             ? rms_grad_scratch(h, n_rows, n_cols)
             : 0;
}

static ss_status rms_norm_backward(ss_handle *h, const ss_dense *grad_y, const ss_dense *total, const ss_kept *kept,
                                   const ss_dense *weight, const float *rstd, const ss_dense *grad_total, const ss_dense *grad_x,
                                   const ss_dense *grad_weight, void *scratch, int64_t scratch_bytes, void *stream, const char *call) {
  const int64_t R = total->n_rows, D = total->n_cols;
  if (D < 1) return report(h, SS_ERR_INVALID_ARG, "%s: rows of no columns", call);
  SS_TRY(check(h, grad_y, R, D, F32 | HALVES, call, "grad_y"));
  SS_TRY(same_type(h, grad_y, total->type, call, "grad_y"));
  SS_TRY(check(h, weight, 1, D, F32 | HALVES, call, "weight"));
  if (weight->type != SS_VALUES_F32) SS_TRY(same_type(h, weight, total->type, call, "weight"));
  if (grad_total) {
    SS_TRY(check(h, grad_total, R, D, F32 | HALVES, call, "grad_total"));
    SS_TRY(same_type(h, grad_total, total->type, call, "grad_total"));
  }
  SS_TRY(check(h, grad_x, R, D, F32 | HALVES, call, "grad_x"));
  SS_TRY(same_type(h, grad_x, total->type, call, "grad_x"));
  SS_TRY(check(h, grad_weight, 1, D, F32 | HALVES, call, "grad_weight"));
  SS_TRY(same_type(h, grad_weight, weight->type, call, "grad_weight"));
  if (R > 0 && !rstd) return report(h, SS_ERR_INVALID_ARG, "%s: null rstd", call);
  SS_TRY(check_scratch(h, scratch, scratch_bytes, kept ? rms_kept_grad_scratch(h, R, D, total->type) : rms_grad_scratch(h, R, D), call));
  SS_RUN(h, cudaSetDevice(h->device));
  rms_grad_args a = {*grad_y, *total, *weight, or_none(grad_total), *grad_x, *grad_weight, rstd,
                     static_cast<float *>(scratch), kept ? *kept : ss_kept{}};
  int queued = 0;
  SS_RUN(h, launch_rms_norm_grad(h, a, as_stream(stream), &queued));
  h->launches += queued;
  return SS_OK;
}

ss_status ss_rms_norm_backward(ss_handle *h, const ss_dense *grad_y, const ss_dense *total, const ss_dense *weight,
                               const float *rstd, const ss_dense *grad_total, const ss_dense *grad_x,
                               const ss_dense *grad_weight, void *scratch, int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_rms_norm_backward";
  if (!total) return report(h, SS_ERR_INVALID_ARG, "%s: null total", call);
  SS_TRY(check(h, total, total->n_rows, total->n_cols, F32 | HALVES, call, "total"));
  return rms_norm_backward(h, grad_y, total, nullptr, weight, rstd, grad_total, grad_x, grad_weight, scratch, scratch_bytes, stream, call);
}

int64_t ss_rms_norm_kept_backward_scratch(const ss_handle *h, int64_t n_rows, int64_t n_cols, int32_t type) {
  return h && n_rows > 0 && n_cols > 0 && n_rows < SS_DENSE_MAX && n_cols < SS_DENSE_MAX
             ? rms_kept_grad_scratch(h, n_rows, n_cols, type)
             : 0;
}

ss_status ss_rms_norm_kept_backward(ss_handle *h, const ss_dense *grad_y, const ss_kept *total, const ss_dense *weight,
                                    const float *rstd, const ss_dense *grad_total, const ss_dense *grad_x,
                                    const ss_dense *grad_weight, void *scratch, int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_rms_norm_kept_backward";
  if (!grad_y) return report(h, SS_ERR_INVALID_ARG, "%s: null grad_y", call);
  const int64_t R = grad_y->n_rows, D = grad_y->n_cols;
  SS_TRY(check(h, grad_y, R, D, F32 | HALVES, call, "grad_y"));
  SS_TRY(check_kept(h, total, R, D, call, "total"));
  const ss_dense like = {nullptr, R, D, D, grad_y->type};
  return rms_norm_backward(h, grad_y, &like, total, weight, rstd, grad_total, grad_x, grad_weight, scratch, scratch_bytes, stream, call);
}

static ss_status check_activation(ss_handle *h, int32_t activation, const char *call) {
  if (activation >= SS_ACT_NONE && activation <= SS_ACT_LOG1P_RELU) return SS_OK;
  return report(h, SS_ERR_INVALID_ARG, "%s: unknown activation %d", call, activation);
}

static ss_status check_linear(ss_handle *h, const ss_dense *x, const ss_dense *w, int types, int32_t activation,
                              const char *call) {
  if (!x || !w) return report(h, SS_ERR_INVALID_ARG, "%s: null %s", call, x ? "w" : "x");
  SS_TRY(check(h, x, x->n_rows, x->n_cols, types, call, "x"));
  SS_TRY(check(h, w, w->n_rows, x->n_cols, types, call, "w"));
  SS_TRY(same_type(h, w, x->type, call, "w"));
  return check_activation(h, activation, call);
}

int64_t ss_linear_scratch(const ss_handle *h, const ss_dense *x, const ss_dense *w) {
  return h && x && w ? linear_scratch(h, *x, *w, false) : 0;
}
int64_t ss_linear_keep_scratch(const ss_handle *h, const ss_dense *x, const ss_dense *w) {
  return h && x && w ? linear_scratch(h, *x, *w, true) : 0;
}

static ss_status linear(ss_handle *h, const ss_dense *x, const float *x_scale, const ss_dense *w, const float *w_scale,
                        const float *bias, int32_t activation, const ss_dense *residual, const ss_dense *pre, const ss_kept *keep,
                        const ss_dense *y, void *scratch, int64_t scratch_bytes, void *stream, const char *call) {
  SS_TRY(check_linear(h, x, w, HALVES | F8, activation, call));
  const int64_t M = x->n_rows, N = w->n_rows;
  const bool f8 = x->type == SS_VALUES_F8;
  if (f8 != (x_scale != nullptr) || f8 != (w_scale != nullptr)) {
    if (!(f8 && (M == 0 || N == 0)))
      return report(h, SS_ERR_INVALID_ARG, "%s: x_scale and w_scale go with 8-bit inputs, and only with them", call);
  }
  SS_TRY(check(h, y, M, N, F32 | HALVES, call, "y"));
  if (!f8 && y->type != SS_VALUES_F32) SS_TRY(same_type(h, y, x->type, call, "y"));
  if (residual) {
    SS_TRY(check(h, residual, M, N, F32 | HALVES, call, "residual"));
    SS_TRY(same_type(h, residual, y->type, call, "residual"));
  }
  if (pre) {
    SS_TRY(check(h, pre, M, N, F32 | HALVES, call, "pre"));
    SS_TRY(same_type(h, pre, y->type, call, "pre"));
  }
  if (keep) {
    SS_TRY(check_kept(h, keep, M, N, call, "pre"));
    if (x->n_cols < 1) return report(h, SS_ERR_INVALID_ARG, "%s: rows of no columns", call);
  }
  SS_TRY(check_scratch(h, scratch, scratch_bytes, linear_scratch(h, *x, *w, keep != nullptr), call));
  SS_RUN(h, cudaSetDevice(h->device));
  linear_args a = {*x, *w, or_none(residual), or_none(pre), *y, x_scale, w_scale, bias, activation,
                   static_cast<unsigned char *>(scratch), keep ? *keep : ss_kept{}};
  int queued = 0;
  SS_RUN(h, launch_linear(h, a, as_stream(stream), &queued));
  h->launches += queued;
  return SS_OK;
}

ss_status ss_linear(ss_handle *h, const ss_dense *x, const float *x_scale, const ss_dense *w, const float *w_scale,
                    const float *bias, int32_t activation, const ss_dense *residual, const ss_dense *pre,
                    const ss_dense *y, void *scratch, int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  return linear(h, x, x_scale, w, w_scale, bias, activation, residual, pre, nullptr, y, scratch, scratch_bytes, stream, "ss_linear");
}

ss_status ss_linear_keep(ss_handle *h, const ss_dense *x, const float *x_scale, const ss_dense *w, const float *w_scale,
                         const float *bias, int32_t activation, const ss_dense *residual, const ss_kept *pre,
                         const ss_dense *y, void *scratch, int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  if (!pre) return report(h, SS_ERR_INVALID_ARG, "ss_linear_keep: null pre");
  return linear(h, x, x_scale, w, w_scale, bias, activation, residual, nullptr, pre, y, scratch, scratch_bytes, stream, "ss_linear_keep");
}

int64_t ss_linear_backward_scratch(const ss_handle *h, const ss_dense *grad_y, const ss_dense *x, const ss_dense *w,
                                   int32_t activation) {
  return h && grad_y && x && w ? linear_grad_scratch(h, *grad_y, *x, *w, activation, false) : 0;
}

int64_t ss_linear_kept_backward_scratch(const ss_handle *h, const ss_dense *grad_y, const ss_dense *w, int32_t activation) {
  if (!h || !grad_y || !w) return 0;
  const ss_dense x = {nullptr, grad_y->n_rows, w->n_cols, w->n_cols, w->type};
  return linear_grad_scratch(h, *grad_y, x, *w, activation, true);
}

static ss_status linear_backward(ss_handle *h, const ss_dense *grad_y, const ss_dense *x, const ss_kept *x_kept, const ss_dense *w,
                                 const ss_dense *pre, const ss_kept *pre_kept, int32_t activation, const ss_dense *grad_x,
                                 const ss_dense *grad_w, float *grad_bias, void *scratch, int64_t scratch_bytes, int64_t need,
                                 void *stream, const char *call) {
  const int64_t M = x->n_rows, N = w->n_rows, K = x->n_cols;
  SS_TRY(check(h, grad_y, M, N, HALVES, call, "grad_y"));
  SS_TRY(same_type(h, grad_y, x->type, call, "grad_y"));
  if (activation != SS_ACT_NONE && pre_kept) {
    SS_TRY(check_kept(h, pre_kept, M, N, call, "pre"));
  } else if (activation != SS_ACT_NONE) {
    SS_TRY(check(h, pre, M, N, HALVES, call, "pre"));
    SS_TRY(same_type(h, pre, x->type, call, "pre"));
  }
  for (const ss_dense *g : {grad_x, grad_w}) {
    if (!g) continue;
    const char *name = g == grad_x ? "grad_x" : "grad_w";
    SS_TRY(check(h, g, g == grad_x ? M : N, K, F32 | HALVES, call, name));
    if (g->type != SS_VALUES_F32) SS_TRY(same_type(h, g, x->type, call, name));
  }
  SS_TRY(check_scratch(h, scratch, scratch_bytes, need, call));
  SS_RUN(h, cudaSetDevice(h->device));
  const bool act = activation != SS_ACT_NONE;
  linear_grad_args a = {*grad_y,          *x, *w, act && !pre_kept ? *pre : or_none(nullptr), or_none(grad_x), or_none(grad_w), grad_bias, activation,
                        static_cast<unsigned char *>(scratch), x_kept ? *x_kept : ss_kept{}, act && pre_kept ? *pre_kept : ss_kept{}};
  int queued = 0;
  SS_RUN(h, launch_linear_grad(h, a, as_stream(stream), &queued));
  h->launches += queued;
  return SS_OK;
}

ss_status ss_linear_backward(ss_handle *h, const ss_dense *grad_y, const ss_dense *x, const ss_dense *w,
                             const ss_dense *pre, int32_t activation, const ss_dense *grad_x, const ss_dense *grad_w,
                             float *grad_bias, void *scratch, int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_linear_backward";
  SS_TRY(check_linear(h, x, w, HALVES, activation, call));
  const int64_t need = grad_y ? linear_grad_scratch(h, *grad_y, *x, *w, activation, false) : 0;
  return linear_backward(h, grad_y, x, nullptr, w, pre, nullptr, activation, grad_x, grad_w, grad_bias, scratch, scratch_bytes, need, stream, call);
}

ss_status ss_linear_kept_backward(ss_handle *h, const ss_dense *grad_y, const ss_dense *x, const ss_kept *x_kept,
                                  const ss_dense *w, const ss_dense *pre, const ss_kept *pre_kept, int32_t activation,
                                  const ss_dense *grad_x, const ss_dense *grad_w, float *grad_bias, void *scratch,
                                  int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_linear_kept_backward";
  if (!grad_y || !w) return report(h, SS_ERR_INVALID_ARG, "%s: null %s", call, grad_y ? "w" : "grad_y");
  if ((x != nullptr) == (x_kept != nullptr) || (activation != SS_ACT_NONE && (pre != nullptr) == (pre_kept != nullptr)))
    return report(h, SS_ERR_INVALID_ARG, "%s: x or x_kept, and pre or pre_kept", call);
  const ss_dense like = {nullptr, grad_y->n_rows, w->n_cols, w->n_cols, w->type};
  if (x) {
    SS_TRY(check_linear(h, x, w, HALVES, activation, call));
  } else {
    SS_TRY(check_kept(h, x_kept, like.n_rows, like.n_cols, call, "x"));
    SS_TRY(check(h, w, w->n_rows, w->n_cols, HALVES, call, "w"));
    SS_TRY(check_activation(h, activation, call));
  }
  const int64_t need = linear_grad_scratch(h, *grad_y, like, *w, activation, true);
  return linear_backward(h, grad_y, x ? x : &like, x_kept, w, pre, pre_kept, activation, grad_x, grad_w, grad_bias, scratch, scratch_bytes, need, stream, call);
}

ss_status ss_compress(ss_handle *h, const ss_dense *x, const ss_kept *out, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_compress";
  if (!x) return report(h, SS_ERR_INVALID_ARG, "%s: null x", call);
  SS_TRY(check(h, x, x->n_rows, x->n_cols, F32 | HALVES, call, "x"));
  SS_TRY(check_kept(h, out, x->n_rows, x->n_cols, call, "out"));
  SS_RUN(h, cudaSetDevice(h->device));
  int queued = 0;
  SS_RUN(h, launch_compress(*x, *out, as_stream(stream), &queued));
  h->launches += queued;
  return SS_OK;
}

ss_status ss_expand(ss_handle *h, const ss_kept *x, const ss_dense *y, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_expand";
  if (!y) return report(h, SS_ERR_INVALID_ARG, "%s: null y", call);
  SS_TRY(check(h, y, y->n_rows, y->n_cols, F32 | HALVES, call, "y"));
  SS_TRY(check_kept(h, x, y->n_rows, y->n_cols, call, "x"));
  SS_RUN(h, cudaSetDevice(h->device));
  int queued = 0;
  SS_RUN(h, launch_expand(*x, *y, as_stream(stream), &queued));
  h->launches += queued;
  return SS_OK;
}

ss_status ss_distill(ss_handle *h, const ss_dense *logits, const float *scores, const int64_t *items, int32_t k,
                     float temperature, float teacher_temperature, const float *weight, float *loss, float *stats,
                     void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  SS_TRY(check_distill(h, logits, scores, items, k, temperature, teacher_temperature, "ss_distill"));
  if (logits->n_rows > 0 && (!loss || !stats)) return report(h, SS_ERR_INVALID_ARG, "ss_distill: null output");
  distill_args a = distill_of(logits, scores, items, k, temperature, teacher_temperature, weight);
  a.loss = loss;
  a.stats = stats;
  return run_distill(h, a, DISTILL_FORWARD, stream);
}

ss_status ss_distill_backward(ss_handle *h, const float *grad_loss, const ss_dense *logits, const float *scores,
                              const int64_t *items, int32_t k, float temperature, float teacher_temperature,
                              const float *weight, const float *stats, const ss_dense *grad_logits, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_distill_backward";
  SS_TRY(check_distill(h, logits, scores, items, k, temperature, teacher_temperature, call));
  SS_TRY(check(h, grad_logits, logits->n_rows, logits->n_cols, F32 | HALVES, call, "grad_logits"));
  SS_TRY(same_type(h, grad_logits, logits->type, call, "grad_logits"));
  if (logits->n_rows > 0 && !stats) return report(h, SS_ERR_INVALID_ARG, "%s: null stats", call);
  if (logits->n_rows > 0 && logits->n_cols > 0 && grad_logits->data == logits->data)
    return report(h, SS_ERR_INVALID_ARG, "%s: grad_logits must not be the logits (ss_distill_step takes that)", call);
  distill_args a = distill_of(logits, scores, items, k, temperature, teacher_temperature, weight);
  a.grad_loss = grad_loss;
  a.stats = const_cast<float *>(stats);
  a.grad_logits = *grad_logits;
  return run_distill(h, a, DISTILL_BACKWARD, stream);
}

ss_status ss_distill_step(ss_handle *h, const float *grad_loss, const ss_dense *logits, const float *scores,
                          const int64_t *items, int32_t k, float temperature, float teacher_temperature,
                          const float *weight, float *loss, const ss_dense *grad_logits, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_distill_step";
  SS_TRY(check_distill(h, logits, scores, items, k, temperature, teacher_temperature, call));
  SS_TRY(check(h, grad_logits, logits->n_rows, logits->n_cols, F32 | HALVES, call, "grad_logits"));
  SS_TRY(same_type(h, grad_logits, logits->type, call, "grad_logits"));
  if (logits->n_rows > 0 && !loss) return report(h, SS_ERR_INVALID_ARG, "%s: null loss", call);
  if (grad_logits->data == logits->data && grad_logits->ld != logits->ld && logits->n_rows > 1 && logits->n_cols > 0)
    return report(h, SS_ERR_INVALID_ARG, "%s: grad_logits in the logits' place with another ld", call);
  distill_args a = distill_of(logits, scores, items, k, temperature, teacher_temperature, weight);
  a.grad_loss = grad_loss;
  a.loss = loss;
  a.grad_logits = *grad_logits;
  return run_distill(h, a, DISTILL_STEP, stream);
}

static ss_status check_xent(ss_handle *h, const ss_dense *x, const ss_dense *w, const int64_t *targets, float temperature,
                            const char *call) {
  if (!x || !w) return report(h, SS_ERR_INVALID_ARG, "%s: null %s", call, x ? "w" : "x");
  SS_TRY(check(h, x, x->n_rows, x->n_cols, HALVES, call, "x"));
  SS_TRY(check(h, w, w->n_rows, x->n_cols, HALVES, call, "w"));
  SS_TRY(same_type(h, w, x->type, call, "w"));
  if (x->n_cols < 1) return report(h, SS_ERR_INVALID_ARG, "%s: rows of no columns", call);
  if (w->n_rows < 1) return report(h, SS_ERR_INVALID_ARG, "%s: no items", call);
  if (x->n_rows > 0 && !targets) return report(h, SS_ERR_INVALID_ARG, "%s: null targets", call);
  if (!(temperature >= SS_DISTILL_TEMPERATURE_MIN) || !(temperature <= 1.0f / SS_DISTILL_TEMPERATURE_MIN))
    return report(h, SS_ERR_INVALID_ARG, "%s: temperature %g outside [%g, %g]", call, (double)temperature,
                  (double)SS_DISTILL_TEMPERATURE_MIN, 1.0 / (double)SS_DISTILL_TEMPERATURE_MIN);
  return SS_OK;
}

static ss_status run_xent(ss_handle *h, xent_args &a, int32_t mode, void *scratch, int64_t scratch_bytes, void *stream, const char *call) {
  for (const ss_dense *g : {&a.grad_x, &a.grad_w}) {
    if (!g->data && g->type == 0 && g->n_rows == 0) continue;
    const char *name = g == &a.grad_x ? "grad_x" : "grad_w";
    SS_TRY(check(h, g, g == &a.grad_x ? a.x.n_rows : a.w.n_rows, a.x.n_cols, F32 | HALVES, call, name));
    if (g->type != SS_VALUES_F32) SS_TRY(same_type(h, g, a.x.type, call, name));
  }
  SS_TRY(check_scratch(h, scratch, scratch_bytes, xent_scratch(h, a.x, a.w, mode), call));
  a.scratch = static_cast<unsigned char *>(scratch);
  SS_RUN(h, cudaSetDevice(h->device));
  int queued = 0;
  SS_RUN(h, launch_xent(h, a, mode, as_stream(stream), &queued));
  h->launches += queued;
  return SS_OK;
}

static int64_t scratch_of_xent(const ss_handle *h, const ss_dense *x, const ss_dense *w, int32_t mode) {
  const bool ok = h && x && w && x->n_rows >= 0 && x->n_rows < SS_DENSE_MAX && x->n_cols > 0 && x->n_cols < SS_DENSE_MAX &&
                  w->n_rows > 0 && w->n_rows < SS_DENSE_MAX;
  return ok ? xent_scratch(h, *x, *w, mode) : 0;
}
int64_t ss_cross_entropy_scratch(const ss_handle *h, const ss_dense *x, const ss_dense *w) {
  return scratch_of_xent(h, x, w, XENT_LOSS);
}
int64_t ss_cross_entropy_backward_scratch(const ss_handle *h, const ss_dense *x, const ss_dense *w) {
  return scratch_of_xent(h, x, w, XENT_BACKWARD);
}
int64_t ss_cross_entropy_step_scratch(const ss_handle *h, const ss_dense *x, const ss_dense *w) {
  return scratch_of_xent(h, x, w, XENT_STEP);
}

ss_status ss_cross_entropy(ss_handle *h, const ss_dense *x, const ss_dense *w, const float *bias, const int64_t *targets,
                           float temperature, const float *weight, float *loss, float *stats, void *scratch,
                           int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_cross_entropy";
  SS_TRY(check_xent(h, x, w, targets, temperature, call));
  if (x->n_rows > 0 && (!loss || !stats)) return report(h, SS_ERR_INVALID_ARG, "%s: null output", call);
  if (reinterpret_cast<uintptr_t>(stats) % 8) return report(h, SS_ERR_INVALID_ARG, "%s: stats are not aligned to 8 bytes", call);
  xent_args a = {*x, *w, {}, {}, bias, targets, weight, nullptr, loss, stats, nullptr, temperature, nullptr};
  return run_xent(h, a, XENT_LOSS, scratch, scratch_bytes, stream, call);
}

ss_status ss_cross_entropy_backward(ss_handle *h, const float *grad_loss, const ss_dense *x, const ss_dense *w,
                                    const float *bias, const int64_t *targets, float temperature, const float *weight,
                                    const float *stats, const ss_dense *grad_x, const ss_dense *grad_w, float *grad_bias,
                                    void *scratch, int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_cross_entropy_backward";
  SS_TRY(check_xent(h, x, w, targets, temperature, call));
  if (x->n_rows > 0 && !stats) return report(h, SS_ERR_INVALID_ARG, "%s: null stats", call);
  if (reinterpret_cast<uintptr_t>(stats) % 8) return report(h, SS_ERR_INVALID_ARG, "%s: stats are not aligned to 8 bytes", call);
  xent_args a = {*x,        *w,      or_none(grad_x),             or_none(grad_w), bias,        targets, weight,
                 grad_loss, nullptr, const_cast<float *>(stats), grad_bias,       temperature, nullptr};
  return run_xent(h, a, XENT_BACKWARD, scratch, scratch_bytes, stream, call);
}

ss_status ss_cross_entropy_step(ss_handle *h, const float *grad_loss, const ss_dense *x, const ss_dense *w, const float *bias,
                                const int64_t *targets, float temperature, const float *weight, float *loss,
                                const ss_dense *grad_x, const ss_dense *grad_w, float *grad_bias, void *scratch,
                                int64_t scratch_bytes, void *stream) {
  if (!h) return SS_ERR_INVALID_ARG;
  const char *call = "ss_cross_entropy_step";
  SS_TRY(check_xent(h, x, w, targets, temperature, call));
  if (x->n_rows > 0 && !loss) return report(h, SS_ERR_INVALID_ARG, "%s: null loss", call);
  xent_args a = {*x,        *w,   or_none(grad_x), or_none(grad_w), bias,        targets, weight,
                 grad_loss, loss, nullptr,         grad_bias,       temperature, nullptr};
  return run_xent(h, a, XENT_STEP, scratch, scratch_bytes, stream, call);
}

}  // extern "C"
