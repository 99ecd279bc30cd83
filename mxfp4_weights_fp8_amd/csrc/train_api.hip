// C ABI of the operators that train the routed experts (declared in include/moe_mxfp4.h):
// rows by expert and back, the experts' products, the gated activation with its input in 8
// bits. Argument checks and workspace sizes; nothing here allocates, synchronizes or reads
// device memory.
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

int check_rows(int32_t T, int32_t H, int32_t K, int32_t multiple) {
  if (T < 0 || H < 1 || K < 1 || K > kMaxTopK) return MOE_EINVAL;
  if (H % multiple || H > kMaxSmallDim || T > kMaxRows || (int64_t)T * K > kMaxPairs) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

int check_experts(const moe_expert_dims* d) {
  if (!d || d->P < 0 || d->N < 1 || d->K < 1 || d->E < 1 || d->E > kMaxExperts || !is_type(d->type)) return MOE_EINVAL;
  if (d->N % 128 || d->K % 128 || d->N > kMaxCols || d->K > kMaxCols || (int64_t)d->N * d->K >= (int64_t)1 << 31 ||
      d->P > kMaxPairs)
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

int check_glu(const moe_glu_dims* d) {
  if (!d || d->R < 0 || d->I < 1 || d->E < 0 || d->E > kMaxExperts || d->act < MOE_ACT_NONE || d->act > MOE_ACT_SIGMOID)
    return MOE_EINVAL;
  return d->I % 128 || d->I > kMaxSmallDim || d->R > kMaxPairs ? MOE_EUNSUPPORTED : MOE_OK;
}
inline const int32_t* live_rows(const moe_glu_dims& d, const int32_t* offsets) { return d.E ? offsets + d.E : nullptr; }

}  // namespace

extern "C" {

int moe_sort_rows(int32_t T, int32_t H, int32_t K, const void* x, const uint8_t* x_s, const int32_t* pair_rows,
                  uint16_t* rows, void* stream) {
  const int rc = check_rows(T, H, K, x_s ? 128 : 8);
  if (rc != MOE_OK || T == 0) return rc;
  if (!x || !pair_rows || !rows || !all_aligned(x, x_s, pair_rows, rows)) return MOE_EINVAL;
  return hip_status(launch_sort_rows(T, H, K, x, x_s, pair_rows, rows, (hipStream_t)stream));
}

int moe_restore_act(int32_t T, int32_t H, const uint8_t* x_q, const uint8_t* x_s, uint16_t* x, void* stream) {
  const int rc = check_rows(T, H, 1, 128);
  if (rc != MOE_OK || T == 0) return rc;
  if (!x_q || !x_s || !x || !all_aligned(x_q, x_s, x)) return MOE_EINVAL;
  return hip_status(launch_sort_rows(T, H, 1, x_q, x_s, nullptr, x, (hipStream_t)stream));
}

int moe_return_rows(int32_t T, int32_t H, int32_t K, const uint16_t* rows, const int32_t* pair_rows,
                    const float* weights, const void* add, int32_t type, void* y, void* stream) {
  const int rc = check_rows(T, H, K, 8);
  if (rc != MOE_OK) return rc;
  if (!is_type(type)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!rows || !pair_rows || !y || !all_aligned(rows, pair_rows, weights, add, y)) return MOE_EINVAL;
  return hip_status(
      launch_return_rows(T, H, K, rows, pair_rows, weights, add, type == MOE_TYPE_F32, y, (hipStream_t)stream));
}

int moe_return_rows_grad(int32_t T, int32_t H, int32_t K, const void* dy, int32_t type, const uint16_t* rows,
                         const int32_t* pair_rows, const float* weights, uint16_t* d_rows, float* d_weights,
                         void* stream) {
  const int rc = check_rows(T, H, K, 8);
  if (rc != MOE_OK) return rc;
  if (!is_type(type)) return MOE_EINVAL;
  if (T == 0) return MOE_OK;
  if (!dy || !pair_rows || (d_weights && !rows) || (!d_rows && !d_weights)) return MOE_EINVAL;
  if (!all_aligned(dy, rows, pair_rows, weights, d_rows, d_weights)) return MOE_EINVAL;
  return hip_status(launch_return_rows_grad(T, H, K, dy, type == MOE_TYPE_F32, rows, pair_rows, weights, d_rows,
                                            d_weights, (hipStream_t)stream));
}

size_t moe_expert_linear_workspace_bytes(const moe_expert_dims* dims) {
  return check_experts(dims) != MOE_OK || dims->P == 0 ? 0 : expert_linear_ws_bytes(*dims);
}

int moe_expert_linear(const moe_expert_dims* dims, const uint16_t* x, const uint16_t* w, const int32_t* expert_offsets,
                      void* y, void* ws, size_t ws_bytes, void* stream) {
  const int rc = check_experts(dims);
  if (rc != MOE_OK || dims->P == 0) return rc;
  if (!x || !w || !expert_offsets || !y || !all_aligned(x, w, expert_offsets, y, ws)) return MOE_EINVAL;
  const size_t need = expert_linear_ws_bytes(*dims);
  if (need && !ws) return MOE_EINVAL;
  if (ws_bytes < need) return MOE_EWORKSPACE;
  return hip_status(launch_expert_linear(*dims, x, w, expert_offsets, y, ws, (hipStream_t)stream));
}

size_t moe_expert_linear_grad_workspace_bytes(const moe_expert_dims* dims) {
  return check_experts(dims) != MOE_OK ? 0 : expert_linear_grad_ws_bytes(*dims);
}

int moe_expert_linear_grad(const moe_expert_dims* dims, const uint16_t* dy, const uint16_t* x, const uint16_t* w,
                           const int32_t* expert_offsets, uint16_t* dx, void* dw, void* ws, size_t ws_bytes,
                           void* stream) {
  const int rc = check_experts(dims);
  if (rc != MOE_OK) return rc;
  if (dims->P > 0 && ((!dy && (dx || dw)) || (dx && !w) || (dw && !x))) return MOE_EINVAL;
  if (!expert_offsets || !ws || !all_aligned(dy, x, w, expert_offsets, dx, dw, ws)) return MOE_EINVAL;
  if (ws_bytes < expert_linear_grad_ws_bytes(*dims)) return MOE_EWORKSPACE;
  return hip_status(launch_expert_linear_grad(*dims, dy, x, w, expert_offsets, dx, dw, ws, (hipStream_t)stream));
}

int moe_glu(const moe_glu_dims* dims, const uint16_t* z, const int32_t* expert_offsets, uint16_t* h, uint8_t* z_q,
            uint8_t* z_s, void* stream) {
  const int rc = check_glu(dims);
  if (rc != MOE_OK || dims->R == 0) return rc;
  if (!z || !h || !z_q != !z_s || (dims->E && !expert_offsets)) return MOE_EINVAL;
  if (!all_aligned(z, expert_offsets, h, z_q, z_s)) return MOE_EINVAL;
  return hip_status(launch_glu(*dims, z, live_rows(*dims, expert_offsets), h, z_q, z_s, (hipStream_t)stream));
}

int moe_glu_grad(const moe_glu_dims* dims, const uint16_t* dh, const uint16_t* z, const uint8_t* z_q,
                 const uint8_t* z_s, const int32_t* expert_offsets, uint16_t* dz, uint16_t* h, void* stream) {
  const int rc = check_glu(dims);
  if (rc != MOE_OK || dims->R == 0) return rc;
  if (!dh || !dz || !z_q != !z_s || !z == !z_q || (dims->E && !expert_offsets)) return MOE_EINVAL;
  if (!all_aligned(dh, z, z_q, z_s, expert_offsets, dz, h)) return MOE_EINVAL;
  return hip_status(
      launch_glu_grad(*dims, dh, z, z_q, z_s, live_rows(*dims, expert_offsets), dz, h, (hipStream_t)stream));
}

}  // extern "C"
