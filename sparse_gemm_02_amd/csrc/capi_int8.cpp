// C ABI of the RMS norm and the int8 products: argument checks, then kernel
// launches.  As in capi.cpp every check comes before the first launch.
// Declarations and the meaning of every argument: include/slope_int8.h.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "../../include/slope.h"
#include "launch.h"

using slope::Dt;

namespace {

bool dt_ok(int d) { return d == SLOPE_F32 || d == SLOPE_BF16 || d == SLOPE_F16; }
bool in_range(int64_t v) { return v >= 0 && v <= SLOPE_MAX_DIM; }
slope_status from_hip(hipError_t e) { return e == hipSuccess ? SLOPE_OK : SLOPE_ERR_HIP; }

// A pointer that has to be there (required) and, if there, aligned to `align`.
slope_status ptr(const void* p, bool required, unsigned align = 16) {
  if (!p) return required ? SLOPE_ERR_INVALID_ARG : SLOPE_OK;
  return (reinterpret_cast<uintptr_t>(p) & (align - 1)) ? SLOPE_ERR_ALIGN : SLOPE_OK;
}

// Two arguments that share memory (empty ones may have one address).
bool same(const void* a, const void* b, int64_t elements) { return a && a == b && elements > 0; }

#define SLOPE_TRY(x)                       \
  do {                                     \
    slope_status _st = (x);                \
    if (_st != SLOPE_OK) return _st;       \
  } while (0)

slope_status check_gamma(slope_dtype dt, slope_dtype gamma_dt) {
  if (!dt_ok(dt) || !dt_ok(gamma_dt)) return SLOPE_ERR_INVALID_ARG;
  return gamma_dt == dt || gamma_dt == SLOPE_F32 ? SLOPE_OK : SLOPE_ERR_UNSUPPORTED;
}

slope_status check_spmm(slope_dtype out_dt, const int8_t* Xq, const float* x_scale, int64_t T, int64_t K,
                        const void* packed_w, int64_t packed_w_bytes, const float* w_scale, int64_t N, void* Y) {
  if (!dt_ok(out_dt) || T < 0 || K < 0 || N < 0 || packed_w_bytes < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(ptr(Xq, true));
  SLOPE_TRY(ptr(packed_w, true));
  SLOPE_TRY(ptr(Y, true));
  SLOPE_TRY(ptr(x_scale, true, 4));
  SLOPE_TRY(ptr(w_scale, true, 4));
  if (K % 16 || N % 4) return SLOPE_ERR_SHAPE;
  if (!in_range(T) || !in_range(N) || K > SLOPE_I8_MAX_COLS) return SLOPE_ERR_UNSUPPORTED;
  return packed_w_bytes < slope::packed_sparse_i8_bytes(N, K) ? SLOPE_ERR_WORKSPACE : SLOPE_OK;
}

}  // namespace

extern "C" {

slope_status slope_rmsnorm(slope_dtype dt, const void* X, const void* residual_or_null, slope_dtype gamma_dt,
                           const void* gamma_or_null, int64_t T, int64_t K, double eps, void* H_or_null,
                           void* Y_or_null, int8_t* q_or_null, float* q_scale_or_null, float* rstd_or_null,
                           void* stream) {
  if (T < 0 || K < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(check_gamma(dt, gamma_dt));
  SLOPE_TRY(ptr(X, true));
  SLOPE_TRY(ptr(residual_or_null, false));
  SLOPE_TRY(ptr(gamma_or_null, false));
  SLOPE_TRY(ptr(H_or_null, false));
  SLOPE_TRY(ptr(Y_or_null, false));
  SLOPE_TRY(ptr(q_scale_or_null, false, 4));
  SLOPE_TRY(ptr(rstd_or_null, false, 4));
  if (!H_or_null && !Y_or_null && !q_or_null && !rstd_or_null) return SLOPE_ERR_INVALID_ARG;
  if ((q_or_null == nullptr) != (q_scale_or_null == nullptr)) return SLOPE_ERR_INVALID_ARG;
  if (same(H_or_null, Y_or_null, T * K) || same(q_scale_or_null, rstd_or_null, T)) return SLOPE_ERR_INVALID_ARG;
  if (!(eps >= (double)FLT_MIN && eps <= (double)FLT_MAX)) return SLOPE_ERR_INVALID_ARG;
  if (q_or_null && dt == SLOPE_F32) return SLOPE_ERR_UNSUPPORTED;   // codes come from 16-bit values
  if (!in_range(T) || !in_range(K)) return SLOPE_ERR_UNSUPPORTED;
  return from_hip(slope::launch_rmsnorm((Dt)dt, X, residual_or_null, (Dt)gamma_dt, gamma_or_null, T, K, (float)eps,
                                        H_or_null, Y_or_null, q_or_null, q_scale_or_null, rstd_or_null,
                                        (hipStream_t)stream));
}

slope_status slope_rmsnorm_bwd_workspace_bytes(int64_t T, int64_t K, int64_t* bytes) {
  if (!bytes || T < 0 || K < 0) return SLOPE_ERR_INVALID_ARG;
  if (!in_range(T) || !in_range(K)) return SLOPE_ERR_UNSUPPORTED;
  *bytes = slope::rmsnorm_bwd_workspace_bytes(T, K);
  return SLOPE_OK;
}

slope_status slope_rmsnorm_bwd(slope_dtype dt, const void* dY, const void* H, const float* rstd, slope_dtype gamma_dt,
                               const void* gamma_or_null, const void* dH_or_null, int64_t T, int64_t K,
                               void* dX_or_null, void* dgamma_or_null, int accumulate, void* workspace_or_null,
                               int64_t workspace_bytes, void* stream) {
  if (T < 0 || K < 0 || workspace_bytes < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(check_gamma(dt, gamma_dt));
  SLOPE_TRY(ptr(dY, true));
  SLOPE_TRY(ptr(H, true));
  SLOPE_TRY(ptr(rstd, true, 4));
  SLOPE_TRY(ptr(gamma_or_null, false));
  SLOPE_TRY(ptr(dH_or_null, false));
  SLOPE_TRY(ptr(dX_or_null, false));
  SLOPE_TRY(ptr(dgamma_or_null, false));
  SLOPE_TRY(ptr(workspace_or_null, false));
  if (!dX_or_null && !dgamma_or_null) return SLOPE_ERR_INVALID_ARG;
  if (same(dX_or_null, H, T * K)) return SLOPE_ERR_INVALID_ARG;   // (dY or dH in place, H not)
  if (!in_range(T) || !in_range(K)) return SLOPE_ERR_UNSUPPORTED;
  const int64_t need = dgamma_or_null ? slope::rmsnorm_bwd_workspace_bytes(T, K) : 0;
  if (need > 0 && (!workspace_or_null || workspace_bytes < need)) return SLOPE_ERR_WORKSPACE;
  return from_hip(slope::launch_rmsnorm_bwd((Dt)dt, dY, H, rstd, (Dt)gamma_dt, gamma_or_null, dH_or_null, T, K,
                                            dX_or_null, dgamma_or_null, accumulate, workspace_or_null,
                                            (hipStream_t)stream));
}

slope_status slope_quantize_rows_i8(slope_dtype dt, const void* X, int64_t T, int64_t K, int8_t* q, float* scale,
                                    void* stream) {
  if (!dt_ok(dt) || T < 0 || K < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(ptr(X, true));
  SLOPE_TRY(ptr(q, true, 1));
  SLOPE_TRY(ptr(scale, true, 4));
  if (dt == SLOPE_F32) return SLOPE_ERR_UNSUPPORTED;   // codes come from 16-bit values
  if (!in_range(T) || !in_range(K)) return SLOPE_ERR_UNSUPPORTED;
  return from_hip(slope::launch_quantize_rows_i8((Dt)dt, X, T, K, q, scale, (hipStream_t)stream));
}

slope_status slope_packed_sparse_i8_bytes(int64_t rows, int64_t cols, int64_t* bytes) {
  if (!bytes || rows < 0 || cols < 0) return SLOPE_ERR_INVALID_ARG;
  if (cols % 16) return SLOPE_ERR_SHAPE;
  if (!in_range(rows) || cols > SLOPE_I8_MAX_COLS) return SLOPE_ERR_UNSUPPORTED;
  *bytes = slope::packed_sparse_i8_bytes(rows, cols);
  return SLOPE_OK;
}

slope_status slope_pack_sparse_i8(slope_dtype dt, const void* values, const uint32_t* meta, int64_t rows,
                                  int64_t cols, float* w_scale, void* packed, int64_t packed_bytes, void* stream) {
  if (!dt_ok(dt) || rows < 0 || cols < 0 || packed_bytes < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(ptr(values, true));
  SLOPE_TRY(ptr(meta, true));
  SLOPE_TRY(ptr(packed, true));
  SLOPE_TRY(ptr(w_scale, true, 4));
  if (dt == SLOPE_F32) return SLOPE_ERR_UNSUPPORTED;   // codes come from 16-bit values
  if (cols % 16) return SLOPE_ERR_SHAPE;
  if (!in_range(rows) || cols > SLOPE_I8_MAX_COLS) return SLOPE_ERR_UNSUPPORTED;
  if (packed_bytes < slope::packed_sparse_i8_bytes(rows, cols)) return SLOPE_ERR_WORKSPACE;
  return from_hip(slope::launch_pack_sparse_i8((Dt)dt, values, meta, rows, cols, w_scale, packed, (hipStream_t)stream));
}

slope_status slope_spmm_i8_packed(slope_dtype out_dt, const int8_t* Xq, const float* x_scale, int64_t T, int64_t K,
                                  const void* packed_w, int64_t packed_w_bytes, const float* w_scale, int64_t N,
                                  void* Y, void* stream) {
  SLOPE_TRY(check_spmm(out_dt, Xq, x_scale, T, K, packed_w, packed_w_bytes, w_scale, N, Y));
  return from_hip(slope::launch_spmm_i8((Dt)out_dt, Xq, x_scale, T, K, packed_w, w_scale, N, Y, (hipStream_t)stream));
}

slope_status slope_spmm_i8_decode(slope_dtype out_dt, const int8_t* Xq, const float* x_scale, int64_t T, int64_t K,
                                  const void* packed_w, int64_t packed_w_bytes, const float* w_scale, int64_t N,
                                  void* Y, void* stream) {
  SLOPE_TRY(check_spmm(out_dt, Xq, x_scale, T, K, packed_w, packed_w_bytes, w_scale, N, Y));
  if (T > SLOPE_I8_DECODE_MAX_TOKENS) return SLOPE_ERR_UNSUPPORTED;
  return from_hip(slope::launch_spmm_i8_decode((Dt)out_dt, Xq, x_scale, T, K, packed_w, w_scale, N, Y,
                                               (hipStream_t)stream));
}

}  // extern "C"
