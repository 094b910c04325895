/*
 * slope_int8.h - RMS norm with residual addition and per-token 8-bit codes, its
 * gradient, and the 2:4 sparse products on 8-bit integer codes.  Part of the C
 * ABI of libslope.so (included by slope.h; its conventions on memory, streams,
 * alignment and errors hold here).
 *
 * Notation.  X [T, K] activations, one token per row; W_s [N, K] a 2:4 weight
 * in the compressed form of slope.h; Xq, q int8 codes; x_scale [T] and w_scale
 * [N] float32, one for each token and each channel.
 *
 * The 8-bit integer reading.  A row u (a token of X, or the kept values of one
 * row of W_s) becomes codes in [-127, 127] and one scale:
 *   amax  = max |u|        code = the integer nearest to 127 u / amax, ties to even
 *   scale = amax / 127     a code stands for the value code * scale
 * The quotient is decided exactly, not in rounded arithmetic, so the codes are
 * a function of the row's values alone (no order of a sum enters, also after
 * the norm below, where rstd is common to a whole row and cancels).  A row of
 * zeros has codes 0 and scale 0.  A row that holds an infinity, a NaN or a
 * product past float32's range has codes 0 and scale NaN, so everything computed
 * from it is NaN.  (The pages
 * that slope.h names give no 8-bit format; slope_quantize_e4m3's reading has
 * one scale for a whole tensor.)
 */
#ifndef SLOPE_INT8_H_
#define SLOPE_INT8_H_

#include "slope.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens slope_spmm_i8_decode takes at most. */
#define SLOPE_I8_DECODE_MAX_TOKENS 64

/* Largest reduction width of the int8 products: with it a sum of K/2 products
 * of two codes stays inside int32. */
#define SLOPE_I8_MAX_COLS (1 << 18)

/* Residual addition, root-mean-square norm and per-token codes, in one pass:
 *   h    = X + residual          (float32 sum rounded to dt; h = X without one)
 *   rstd = 1 / sqrt(mean_k h^2 + eps)
 *   y    = h * rstd * gamma      (float32, rounded to dt once)
 *   q, q_scale = the 8-bit integer reading of the row u = h * gamma, the
 *          products taken exactly, the scale amax / 127 * rstd
 * h is used as rounded, so a gradient or a later call that starts from H sees
 * the same numbers.  Sums are float32 (a row whose squares' sum passes float32's
 * range has rstd 0, and so y and q_scale 0).
 *   X, residual_or_null  [T, K] dt
 *   gamma_or_null        [K] gamma_dt (dt or F32), NULL = all ones
 *   eps                  positive, a normal number in float32
 *   H_or_null            [T, K] dt output: h
 *   Y_or_null            [T, K] dt output: y
 *   q_or_null            [T, K] int8 output with q_scale_or_null [T] float32
 *                        output; both or neither
 *   rstd_or_null         [T] float32 output
 * At least one output.  H and Y may be X or residual themselves (in place), but
 * not each other; other outputs overlap nothing.  q, q_scale and rstd need only
 * their element type's alignment.  Any K >= 1; K = 0 or T = 0 does nothing.
 * Errors: SLOPE_ERR_UNSUPPORTED for codes of an F32 X or another gamma_dt;
 * SLOPE_ERR_INVALID_ARG for a missing output, one of q and q_scale alone, an
 * eps outside its range, H and Y the same, or q_scale and rstd the same. */
slope_status slope_rmsnorm(slope_dtype dt, const void* X, const void* residual_or_null, slope_dtype gamma_dt,
                           const void* gamma_or_null, int64_t T, int64_t K, double eps, void* H_or_null,
                           void* Y_or_null, int8_t* q_or_null, float* q_scale_or_null, float* rstd_or_null,
                           void* stream);

/* Bytes of device workspace slope_rmsnorm_bwd needs for its gradient of gamma:
 * float32 partial sums, one row of K for each group of tokens.  Host-only. */
slope_status slope_rmsnorm_bwd_workspace_bytes(int64_t T, int64_t K, int64_t* bytes);

/* Gradient of slope_rmsnorm's y (and of h, when it is used further on):
 *   a = dY * gamma,  xh = H * rstd,  c = mean_k (a * xh)
 *   dX = rstd * (a - xh * c) + dH      (the gradient of X and of residual)
 *   dgamma = sum over tokens of dY * xh
 * For codes the same formula is the straight-through gradient.
 *   dY, H   [T, K] dt; H the forward's h (X where it had no residual)
 *   rstd    [T] float32 as the forward wrote it
 *   gamma_or_null [K] gamma_dt (dt or F32), NULL = all ones
 *   dH_or_null    [T, K] dt: the gradient that reaches h by other ways
 *   dX_or_null    [T, K] dt output; may be dY or dH themselves, not H
 *   dgamma_or_null [K] gamma_dt output; accumulate != 0 adds to its contents
 *   workspace     of slope_rmsnorm_bwd_workspace_bytes(T, K) bytes, scratch;
 *                 only used (and only checked) with dgamma
 * At least one output.  float32 arithmetic, sums over tokens in a fixed order,
 * one rounding of each output.  T = 0 gives dgamma = 0 (or leaves it, with
 * accumulate).  Errors: SLOPE_ERR_UNSUPPORTED for another gamma_dt,
 * SLOPE_ERR_WORKSPACE for a short or missing workspace, SLOPE_ERR_INVALID_ARG
 * for a missing output or dX and H the same. */
slope_status slope_rmsnorm_bwd(slope_dtype dt, const void* dY, const void* H, const float* rstd, slope_dtype gamma_dt,
                               const void* gamma_or_null, const void* dH_or_null, int64_t T, int64_t K,
                               void* dX_or_null, void* dgamma_or_null, int accumulate, void* workspace_or_null,
                               int64_t workspace_bytes, void* stream);

/* The 8-bit integer reading of each row of X [T, K] (BF16 or F16), for
 * activations that no norm precedes and for dY: q [T, K] int8, scale [T]
 * float32, both overwritten.  Any K (K = 0: scales 0).  Errors:
 * SLOPE_ERR_UNSUPPORTED for F32. */
slope_status slope_quantize_rows_i8(slope_dtype dt, const void* X, int64_t T, int64_t K, int8_t* q, float* scale,
                                    void* stream);

/* Bytes of the int8 tile-chunk form of a compressed [rows, cols] matrix (see
 * slope_pack_sparse_i8).  Host-only; SLOPE_ERR_SHAPE if cols % 16 != 0,
 * SLOPE_ERR_UNSUPPORTED if cols > SLOPE_I8_MAX_COLS. */
slope_status slope_packed_sparse_i8_bytes(int64_t rows, int64_t cols, int64_t* bytes);

/* int8 tile chunks of a compressed 16-bit 2:4 matrix (values [rows, cols/2],
 * meta [rows, ceil(cols/32)] as slope_compress24 or slope_double_prune write
 * them): every row by the 8-bit integer reading over its kept values, w_scale
 * [rows] float32 <- the rows' scales.  Chunk (t, s) holds rows 256t .. 256t+255
 * and dense columns 128s .. 128s+127, 20480 bytes at offset (t *
 * ceil(cols/128) + s) * 20480, laid out as slope_pack_sparse_e4m3's chunks with
 * int8 codes in place of E4M3's: each row's 64 codes (64 bytes at row*64;
 * 16-byte granule c at c ^ ((row / 4) % 4)), then each row's four metadata
 * words (16 bytes at 16384 + row*16); rows past `rows` and columns past `cols`
 * are 0.  packed: caller-owned, at least slope_packed_sparse_i8_bytes(rows,
 * cols) bytes, overwritten.  Errors: SLOPE_ERR_UNSUPPORTED for F32 or cols >
 * SLOPE_I8_MAX_COLS, SLOPE_ERR_SHAPE if cols % 16 != 0, SLOPE_ERR_WORKSPACE if
 * packed is short. */
slope_status slope_pack_sparse_i8(slope_dtype dt, const void* values, const uint32_t* meta, int64_t rows,
                                  int64_t cols, float* w_scale, void* packed, int64_t packed_bytes, void* stream);

/* The 2:4 sparse product on int8 codes:
 *   Y [T, N] = (Xq [T, K] . W_q^T) * (x_scale[t] * w_scale[n])
 * Xq, x_scale from slope_rmsnorm or slope_quantize_rows_i8; packed_w, w_scale
 * from slope_pack_sparse_i8 of W_s (rows N, cols K), or of W_dp^T (rows K,
 * cols N) with dY's codes, for dX.  The sum of products is exact (int32); it is
 * converted to float32, multiplied by the float32 product of the two scales and
 * rounded to out_dt (BF16, F16 or F32).  Y is overwritten.  No adapter term
 * (slope_lowrank_add adds it).  Codes may be any int8 values.  Errors:
 * SLOPE_ERR_SHAPE unless K % 16 == 0 and N % 4 == 0; SLOPE_ERR_UNSUPPORTED for
 * K > SLOPE_I8_MAX_COLS; SLOPE_ERR_WORKSPACE if packed_w is short. */
slope_status slope_spmm_i8_packed(slope_dtype out_dt, const int8_t* Xq, const float* x_scale, int64_t T, int64_t K,
                                  const void* packed_w, int64_t packed_w_bytes, const float* w_scale, int64_t N,
                                  void* Y, void* stream);

/* slope_spmm_i8_packed for T <= SLOPE_I8_DECODE_MAX_TOKENS tokens, where the
 * cost is the weight's stream from memory: the same arguments and the same
 * results, bit for bit, without a workspace (slope_spmm_i8_packed takes the same
 * path for that many tokens; this entry refuses more).  Errors: those of
 * slope_spmm_i8_packed, SLOPE_ERR_UNSUPPORTED for more tokens. */
slope_status slope_spmm_i8_decode(slope_dtype out_dt, const int8_t* Xq, const float* x_scale, int64_t T, int64_t K,
                                  const void* packed_w, int64_t packed_w_bytes, const float* w_scale, int64_t N,
                                  void* Y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SLOPE_INT8_H_ */
