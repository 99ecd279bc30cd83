// C ABI of the operators in front of the FFN (declared in include/moe_mxfp4.h): the
// residual add with its norm, the dense product, the router's gate and its balance
// loss. Argument checks and workspace sizes; nothing here allocates, synchronizes or
// reads device memory.
#include "host_internal.h"

using namespace moe;

namespace {

inline int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }
inline bool aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
template <typename... P>
bool all_aligned(P... p) {
  return (aligned(p) && ...);
}
inline bool is_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }
inline bool finite(float f) { return f - f == 0.f; }

int check_norm(int32_t T, int32_t H, float eps, int32_t weight_type) {
  if (T < 0 || H <= 0 || !(eps >= 0.f) || !finite(eps) || !is_type(weight_type)) return MOE_EINVAL;
  if (H % 128 || H > kMaxSmallDim || T > kMaxRows) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

int check_linear(const moe_linear_dims* d) {
  if (!d || d->M < 0 || d->N < 1 || d->K < 1 || d->act < MOE_ACT_NONE || d->act > MOE_ACT_SIGMOID || !is_type(d->type))
    return MOE_EINVAL;
  if (d->K % 128 || d->K > kMaxCols || d->N > kMaxCols || d->M > kMaxRows ||
      (int64_t)d->N * d->K >= (int64_t)1 << 31)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

int check_gate(const moe_gate_dims* d) {
  if (!d || d->T < 0 || d->E < 1 || d->E > kMaxExperts || d->K < 1 || d->K > kMaxTopK || d->K > d->E ||
      d->score < MOE_SCORE_SOFTMAX || d->score > MOE_SCORE_SQRTSOFTPLUS || (d->renorm != 0 && d->renorm != 1) ||
      !is_type(d->logits_type) || !finite(d->scale))
    return MOE_EINVAL;
  return d->T > kMaxRows ? MOE_EUNSUPPORTED : MOE_OK;
}

}  // namespace

extern "C" {

int moe_add_norm(int32_t T, int32_t H, float eps, const uint16_t* x, const uint16_t* residual, const void* weight,
                 int32_t weight_type, uint16_t* h, uint16_t* y, uint8_t* x_q, uint8_t* x_s, void* stream) {
  const int rc = check_norm(T, H, eps, weight_type);
  if (rc != MOE_OK || T == 0) return rc;
  if (!x || !weight || !x_q != !x_s || (!h && !y && !x_q)) return MOE_EINVAL;
  if (!all_aligned(x, residual, weight, h, y, x_q, x_s)) return MOE_EINVAL;
  return hip_status(launch_add_norm(x, residual, weight, weight_type == MOE_TYPE_F32, h, y, x_q, x_s, T, H, eps,
                                    (hipStream_t)stream));
}

size_t moe_add_norm_grad_workspace_bytes(int32_t T, int32_t H) {
  if (check_norm(T, H, 0.f, MOE_TYPE_F32) != MOE_OK) return 0;
  return sizeof(float) * (size_t)norm_grad_parts(T, H) * H;
}

int moe_add_norm_grad(int32_t T, int32_t H, float eps, const uint16_t* dy, const uint16_t* h, const void* weight,
                      int32_t weight_type, const uint16_t* dh, uint16_t* dx, float* dweight, void* ws, size_t ws_bytes,
                      void* stream) {
  const int rc = check_norm(T, H, eps, weight_type);
  if (rc != MOE_OK) return rc;
  if (!dweight || !weight || (T > 0 && (!dy || !h || !dx || !ws))) return MOE_EINVAL;
  if (!all_aligned(dy, h, weight, dh, dx, dweight, ws)) return MOE_EINVAL;
  if (ws_bytes < moe_add_norm_grad_workspace_bytes(T, H)) return MOE_EWORKSPACE;
  return hip_status(launch_add_norm_grad(dy, h, weight, weight_type == MOE_TYPE_F32, dh, dx, dweight,
                                         static_cast<float*>(ws), T, H, eps, (hipStream_t)stream));
}

size_t moe_linear_workspace_bytes(const moe_linear_dims* dims) {
  if (check_linear(dims) != MOE_OK || dims->M == 0) return 0;
  return linear_parts_bytes(dims->M, dims->N, dims->K);
}

int moe_linear(const moe_linear_dims* dims, const uint16_t* x, const uint16_t* w, const float* bias,
               const void* residual, void* y, float* z, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_linear(dims);
  if (rc != MOE_OK || dims->M == 0) return rc;
  if (!x || !w || !y || !all_aligned(x, w, bias, residual, y, z, ws)) return MOE_EINVAL;
  const size_t need = linear_parts_bytes(dims->M, dims->N, dims->K);
  if (need && !ws) return MOE_EINVAL;
  if (ws_bytes < need) return MOE_EWORKSPACE;
  return hip_status(launch_linear(*dims, x, w, bias, residual, y, z, static_cast<float*>(ws), (hipStream_t)stream));
}

size_t moe_linear_grad_workspace_bytes(const moe_linear_dims* dims) {
  if (check_linear(dims) != MOE_OK || dims->M == 0) return 0;
  return linear_grad_ws_bytes(*dims);
}

int moe_linear_grad(const moe_linear_dims* dims, const void* dy, const uint16_t* x, const uint16_t* w, const float* z,
                    uint16_t* dx, uint16_t* dw, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_linear(dims);
  if (rc != MOE_OK) return rc;
  if (!all_aligned(dy, x, w, z, dx, dw, dbias, ws)) return MOE_EINVAL;
  if (dims->M > 0) {
    if (!dy || (dw && !x) || (dx && !w) || (dims->act != MOE_ACT_NONE && !z) || !ws) return MOE_EINVAL;
    if (ws_bytes < linear_grad_ws_bytes(*dims)) return MOE_EWORKSPACE;
  }
  return hip_status(launch_linear_grad(*dims, dy, x, w, z, dx, dw, dbias, ws, (hipStream_t)stream));
}

int moe_gate(const moe_gate_dims* dims, const void* logits, const float* bias, const int32_t* n_valid,
             int32_t* topk_ids, float* topk_weights, void* stream) {
  const int rc = check_gate(dims);
  if (rc != MOE_OK || dims->T == 0) return rc;
  if (!logits || !topk_ids || !topk_weights || !all_aligned(logits, bias, n_valid, topk_ids, topk_weights))
    return MOE_EINVAL;
  return hip_status(launch_gate(*dims, logits, bias, n_valid, topk_ids, topk_weights, (hipStream_t)stream));
}

int moe_gate_grad(const moe_gate_dims* dims, const void* logits, const int32_t* topk_ids, const float* d_weights,
                  const float* add, float* d_logits, void* stream) {
  const int rc = check_gate(dims);
  if (rc != MOE_OK || dims->T == 0) return rc;
  if (!logits || !topk_ids || !d_weights || !d_logits ||
      !all_aligned(logits, topk_ids, d_weights, add, d_logits))
    return MOE_EINVAL;
  return hip_status(launch_gate_grad(*dims, logits, topk_ids, d_weights, add, d_logits, (hipStream_t)stream));
}

size_t moe_balance_loss_workspace_bytes(const moe_gate_dims* dims, int32_t B) {
  if (check_gate(dims) != MOE_OK || B < 1) return 0;
  return sizeof(double) * (size_t)balance_parts(*dims, B);
}

int moe_balance_loss(const moe_gate_dims* dims, int32_t B, float alpha, const void* logits, const int32_t* topk_ids,
                     const int32_t* seq_offsets, float* loss, int32_t* counts, float* d_logits, void* ws,
                     size_t ws_bytes, void* stream) {
  const int rc = check_gate(dims);
  if (rc != MOE_OK) return rc;
  if (B < 1 || !finite(alpha) || (!seq_offsets && B != 1)) return MOE_EINVAL;
  if ((int64_t)B * dims->E >= (int64_t)1 << 31) return MOE_EUNSUPPORTED;
  const size_t need = sizeof(double) * (size_t)balance_parts(*dims, B);
  if (!loss || !counts || (dims->T > 0 && (!logits || !topk_ids || !d_logits)) || (need && !ws)) return MOE_EINVAL;
  if (!all_aligned(logits, topk_ids, seq_offsets, loss, counts, d_logits, ws)) return MOE_EINVAL;
  if (ws_bytes < need) return MOE_EWORKSPACE;
  return hip_status(launch_balance(*dims, B, alpha, logits, topk_ids, seq_offsets, loss, counts, d_logits,
                                   static_cast<double*>(ws), (hipStream_t)stream));
}

}  // extern "C"
