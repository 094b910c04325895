// C ABI of the microscaled operators: argument checks, then kernel launches.  As in
// capi.cpp every check comes before the first launch.  Declarations and the meaning
// of every argument: include/slope_mx.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>
#include <new>
#include <utility>
#include <vector>

#include "../../include/slope.h"
#include "adamw_args.h"
#include "launch.h"
#include "mxfp4.h"

using slope::Dt;

namespace {

constexpr int64_t kPackedMaxCols = 1 << 21;   // of 16-bit tile chunks
bool in_range(int64_t v) { return v >= 0 && v <= SLOPE_MAX_DIM; }
bool dt_ok(int d) { return d == SLOPE_F32 || d == SLOPE_BF16 || d == SLOPE_F16; }
int64_t size_of(int d) { return d == SLOPE_F32 ? 4 : 2; }
slope_status from_hip(hipError_t e) { return e == hipSuccess ? SLOPE_OK : SLOPE_ERR_HIP; }

// A pointer that has to be there (required) and, if there, aligned to `align`.
slope_status ptr(const void* p, bool required, unsigned align = 16) {
  if (!p) return required ? SLOPE_ERR_INVALID_ARG : SLOPE_OK;
  return (reinterpret_cast<uintptr_t>(p) & (align - 1)) ? SLOPE_ERR_ALIGN : SLOPE_OK;
}

#define SLOPE_TRY(x)                       \
  do {                                     \
    slope_status _st = (x);                \
    if (_st != SLOPE_OK) return _st;       \
  } while (0)

// Whether two of the written byte ranges [first, second) overlap, or one of them and one that is read.
typedef std::pair<uintptr_t, uintptr_t> Range;
typedef std::vector<Range> Ranges;
Range range(const void* p, int64_t bytes) {
  return Range(reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes);
}
bool overlap(Ranges& written, const Ranges& read) {
  std::sort(written.begin(), written.end());
  for (size_t i = 1; i < written.size(); ++i)
    if (written[i].first < written[i - 1].second) return true;
  for (const auto& r : read) {                       // the last written range that begins before its end
    const auto w = std::lower_bound(written.begin(), written.end(), std::make_pair(r.second, uintptr_t(0)));
    if (w != written.begin() && std::prev(w)->second > r.first) return true;
  }
  return false;
}
// Refuses a call (of at least one value) whose written ranges overlap each other or one that is read.
slope_status apart(std::initializer_list<Range> written, std::initializer_list<Range> read) {
  try {
    Ranges w(written);
    return overlap(w, Ranges(read)) ? SLOPE_ERR_INVALID_ARG : SLOPE_OK;
  } catch (const std::bad_alloc&) {
    return SLOPE_ERR_HIP;
  }
}

}  // namespace

extern "C" {

slope_status slope_adamw_multi(int state_bits, int64_t count, const int32_t* param_dt, const int32_t* grad_dt,
                               void* const* params, const void* const* grads, void* const* m, void* const* v,
                               uint8_t* const* m_exp, uint8_t* const* v_exp, const int64_t* n,
                               const slope_adamw_params* hp, uint64_t seed, void* stream) {
  if ((state_bits != 8 && state_bits != 32) || count < 0) return SLOPE_ERR_INVALID_ARG;
  const bool eight = state_bits == 8;
  slope::AdamWStep c;
  SLOPE_TRY(slope::adamw_step(hp, &c));
  if (count == 0) return SLOPE_OK;
  if (!param_dt || !grad_dt || !params || !grads || !m || !v || !n || (eight && (!m_exp || !v_exp)))
    return SLOPE_ERR_INVALID_ARG;
  try {
    Ranges written, read;
    written.reserve((size_t)count * (eight ? 5 : 3));
    read.reserve((size_t)count);
    auto writes = [&](const void* p, int64_t bytes) { written.push_back(range(p, bytes)); };
    for (int64_t i = 0; i < count; ++i) {
      if (!dt_ok(param_dt[i]) || !dt_ok(grad_dt[i]) || n[i] < 0) return SLOPE_ERR_INVALID_ARG;
      if (n[i] > slope::kMultiMaxElems) return SLOPE_ERR_UNSUPPORTED;
      if (n[i] == 0) continue;
      const int64_t e = size_of(param_dt[i]);
      SLOPE_TRY(ptr(params[i], true, (unsigned)e));
      SLOPE_TRY(ptr(grads[i], true, (unsigned)size_of(grad_dt[i])));
      SLOPE_TRY(ptr(m[i], true, eight ? 1 : 4));
      SLOPE_TRY(ptr(v[i], true, eight ? 1 : 4));
      writes(params[i], n[i] * e);
      read.push_back(range(grads[i], n[i] * size_of(grad_dt[i])));
      writes(m[i], n[i] * (eight ? 1 : 4));
      writes(v[i], n[i] * (eight ? 1 : 4));
      if (eight) {
        const int64_t blocks = (n[i] + SLOPE_MX_BLOCK - 1) / SLOPE_MX_BLOCK;
        SLOPE_TRY(ptr(m_exp[i], true, 1));
        SLOPE_TRY(ptr(v_exp[i], true, 1));
        writes(m_exp[i], blocks);
        writes(v_exp[i], blocks);
      }
    }
    if (overlap(written, read)) return SLOPE_ERR_INVALID_ARG;
  } catch (const std::bad_alloc&) {
    return SLOPE_ERR_HIP;
  }
  const slope::AdamWTensors t{count, param_dt, grad_dt, params, grads, m, v, m_exp, v_exp, n};
  return from_hip(slope::launch_adamw_multi(eight, t, c, seed, (hipStream_t)stream));
}

slope_status slope_adamw8_double_prune_packed(slope_dtype dt, slope_dtype grad_dt, void* values_s, const uint32_t* meta_s,
                                              const void* dW_values, uint8_t* m, uint8_t* m_exp, uint8_t* v, uint8_t* v_exp,
                                              int64_t N, int64_t K, const slope_adamw_params* hp, uint64_t seed,
                                              void* packed_s, int64_t packed_s_bytes, void* packed_dpT,
                                              int64_t packed_dpT_bytes, void* stream) {
  if (!dt_ok(dt) || !dt_ok(grad_dt) || N < 0 || K < 0 || packed_s_bytes < 0 || packed_dpT_bytes < 0)
    return SLOPE_ERR_INVALID_ARG;
  for (const void* p : {(const void*)values_s, (const void*)meta_s, dW_values, (const void*)m, (const void*)v, (const void*)packed_s,
                        (const void*)packed_dpT})
    SLOPE_TRY(ptr(p, true));
  SLOPE_TRY(ptr(m_exp, true, 1));
  SLOPE_TRY(ptr(v_exp, true, 1));
  slope::AdamWStep c;
  SLOPE_TRY(slope::adamw_step(hp, &c));
  if (dt == SLOPE_F32) return SLOPE_ERR_UNSUPPORTED;   // 16-bit values only
  if (N % 16 || K % 64) return SLOPE_ERR_SHAPE;        // a block of moments lies in one row
  if (K > kPackedMaxCols || N > kPackedMaxCols) return SLOPE_ERR_UNSUPPORTED;
  const int64_t n = N * K / 2, chunks_s = slope::packed_sparse_bytes(N, K), chunks_dpT = slope::packed_sparse_bytes(K, N);
  if (packed_s_bytes < chunks_s || packed_dpT_bytes < chunks_dpT) return SLOPE_ERR_WORKSPACE;
  if (n == 0) return SLOPE_OK;
  SLOPE_TRY(apart({range(values_s, 2 * n), range(m, n), range(m_exp, n / SLOPE_MX_BLOCK), range(v, n),
                   range(v_exp, n / SLOPE_MX_BLOCK), range(packed_s, chunks_s), range(packed_dpT, chunks_dpT)},
                  {range(meta_s, N * (K / 32) * 4), range(dW_values, n * size_of(grad_dt))}));
  return from_hip(slope::launch_adamw8_double_prune_packed((Dt)dt, (Dt)grad_dt, values_s, meta_s, dW_values, m, m_exp, v, v_exp,
                                                           N, K, c, seed, packed_s, packed_dpT, (hipStream_t)stream));
}

slope_status slope_adamw_moments(slope_dtype out_dt, const uint8_t* m_or_null, const uint8_t* m_exp_or_null,
                                 const uint8_t* v_or_null, const uint8_t* v_exp_or_null, int64_t n,
                                 void* m_out_or_null, void* v_out_or_null, void* stream) {
  if (!dt_ok(out_dt) || n < 0) return SLOPE_ERR_INVALID_ARG;
  const int in_m = !!m_or_null + !!m_exp_or_null + !!m_out_or_null, in_v = !!v_or_null + !!v_exp_or_null + !!v_out_or_null;
  if (in_m % 3 || in_v % 3 || in_m + in_v == 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(ptr(m_out_or_null, false, (unsigned)size_of(out_dt)));
  SLOPE_TRY(ptr(v_out_or_null, false, (unsigned)size_of(out_dt)));
  if (out_dt == SLOPE_F16 || n > slope::kMultiMaxElems) return SLOPE_ERR_UNSUPPORTED;
  if (n == 0) return SLOPE_OK;
  const int64_t blocks = (n + SLOPE_MX_BLOCK - 1) / SLOPE_MX_BLOCK;
  const auto of = [](const void* p, int64_t bytes) { return range(p, p ? bytes : 0); };
  SLOPE_TRY(apart({of(m_out_or_null, n * size_of(out_dt)), of(v_out_or_null, n * size_of(out_dt))},
                  {of(m_or_null, n), of(m_exp_or_null, blocks), of(v_or_null, n), of(v_exp_or_null, blocks)}));
  return from_hip(slope::launch_adamw_moments((Dt)out_dt, m_or_null, m_exp_or_null, v_or_null, v_exp_or_null, n,
                                              m_out_or_null, v_out_or_null, (hipStream_t)stream));
}

slope_status slope_mxfp4_row_bytes(int64_t K, int64_t* code_bytes, int64_t* scale_bytes) {
  if (!code_bytes || !scale_bytes || K < 0) return SLOPE_ERR_INVALID_ARG;
  if (!in_range(K)) return SLOPE_ERR_UNSUPPORTED;
  *code_bytes = slope::mx_code_bytes(K);
  *scale_bytes = slope::mx_scale_bytes(K);
  return SLOPE_OK;
}

slope_status slope_quantize_mxfp4(slope_dtype dt, const void* X, int64_t T, int64_t K, uint8_t* codes, uint8_t* exps,
                                  void* stream) {
  if (!dt_ok(dt) || T < 0 || K < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(ptr(X, true, (unsigned)size_of(dt)));
  SLOPE_TRY(ptr(codes, true));
  SLOPE_TRY(ptr(exps, true));
  if (!in_range(T) || !in_range(K)) return SLOPE_ERR_UNSUPPORTED;
  return from_hip(slope::launch_quantize_mxfp4((Dt)dt, X, T, K, codes, exps, (hipStream_t)stream));
}

slope_status slope_mxfp4_values(slope_dtype out_dt, const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K,
                                void* out, void* stream) {
  if (!dt_ok(out_dt) || T < 0 || K < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(ptr(codes, true));
  SLOPE_TRY(ptr(exps, true));
  SLOPE_TRY(ptr(out, true, (unsigned)size_of(out_dt)));
  if (!in_range(T) || !in_range(K)) return SLOPE_ERR_UNSUPPORTED;
  return from_hip(slope::launch_mxfp4_values((Dt)out_dt, codes, exps, T, K, out, (hipStream_t)stream));
}

slope_status slope_packed_sparse_mxfp4_bytes(int64_t rows, int64_t cols, int64_t* bytes) {
  if (!bytes || rows < 0 || cols < 0) return SLOPE_ERR_INVALID_ARG;
  if (cols % 16) return SLOPE_ERR_SHAPE;
  if (!in_range(rows) || cols > SLOPE_MXFP4_MAX_COLS) return SLOPE_ERR_UNSUPPORTED;
  *bytes = slope::packed_sparse_mxfp4_bytes(rows, cols);
  return SLOPE_OK;
}

slope_status slope_pack_sparse_mxfp4(slope_dtype dt, const void* values, const uint32_t* meta, int64_t rows,
                                     int64_t cols, void* packed, int64_t packed_bytes, void* stream) {
  if (!dt_ok(dt) || rows < 0 || cols < 0 || packed_bytes < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(ptr(values, true));
  SLOPE_TRY(ptr(meta, true));
  SLOPE_TRY(ptr(packed, true));
  if (dt == SLOPE_F32) return SLOPE_ERR_UNSUPPORTED;   // a weight's values are in 16 bits
  if (cols % 16) return SLOPE_ERR_SHAPE;
  if (!in_range(rows) || cols > SLOPE_MXFP4_MAX_COLS) return SLOPE_ERR_UNSUPPORTED;
  if (packed_bytes < slope::packed_sparse_mxfp4_bytes(rows, cols)) return SLOPE_ERR_WORKSPACE;
  return from_hip(slope::launch_pack_sparse_mxfp4((Dt)dt, values, meta, rows, cols, packed, (hipStream_t)stream));
}

slope_status slope_spmm_mxfp4_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t* bytes) {
  if (!bytes || T < 0 || K < 0 || N < 0) return SLOPE_ERR_INVALID_ARG;
  if (K % 16 || N % 4) return SLOPE_ERR_SHAPE;
  if (!in_range(T) || !in_range(N) || K > SLOPE_MXFP4_MAX_COLS) return SLOPE_ERR_UNSUPPORTED;
  *bytes = slope::spmm_mxfp4_scratch_bytes(T, K, N);
  return SLOPE_OK;
}

slope_status slope_spmm_mxfp4_packed(slope_dtype out_dt, const uint8_t* codes, const uint8_t* exps, int64_t T,
                                     int64_t K, const void* packed_w, int64_t packed_w_bytes, int64_t N, void* Y,
                                     void* workspace_or_null, int64_t workspace_bytes, void* stream) {
  if (!dt_ok(out_dt) || T < 0 || K < 0 || N < 0 || packed_w_bytes < 0 || workspace_bytes < 0) return SLOPE_ERR_INVALID_ARG;
  SLOPE_TRY(ptr(codes, true));
  SLOPE_TRY(ptr(exps, true));
  SLOPE_TRY(ptr(packed_w, true));
  SLOPE_TRY(ptr(Y, true));
  SLOPE_TRY(ptr(workspace_or_null, false));
  if (K % 16 || N % 4) return SLOPE_ERR_SHAPE;
  if (!in_range(T) || !in_range(N) || K > SLOPE_MXFP4_MAX_COLS) return SLOPE_ERR_UNSUPPORTED;
  if (packed_w_bytes < slope::packed_sparse_mxfp4_bytes(N, K)) return SLOPE_ERR_WORKSPACE;
  return from_hip(slope::launch_spmm_mxfp4((Dt)out_dt, codes, exps, T, K, packed_w, N, Y, workspace_or_null, workspace_bytes,
                                           (hipStream_t)stream));
}

}  // extern "C"
