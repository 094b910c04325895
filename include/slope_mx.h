/*
 * slope_mx.h - microscaled formats: small floating-point codes with one power-of-two
 * scale for each block of 32 values.  The AdamW step over many tensors at once with
 * moments held so, in 8 bits; and the 2:4 sparse product on 4-bit codes.  Part of the
 * C ABI of libslope.so (included by slope.h; its conventions on memory, streams and
 * errors hold here).
 *
 * A scale is one byte b standing for 2^(b - 127); 255 marks a block without values:
 * everything in it is NaN.
 */
#ifndef SLOPE_MX_H_
#define SLOPE_MX_H_

#include "slope.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values with one scale. */
#define SLOPE_MX_BLOCK 32

/* One AdamW step (slope_adamw's formula and its float32 arithmetic) on `count`
 * tensors, in one launch for up to 56 tensors of one pair of types.
 *
 * state_bits = 32: m[i], v[i] are float32 [n[i]]; results are slope_adamw's on each
 * tensor, bit for bit; m_exp and v_exp are not looked at.
 *
 * state_bits = 8: m[i], v[i] are codes, uint8 [n[i]], and m_exp[i], v_exp[i] the
 * scales, uint8 [ceil(n[i] / 32)], one for 32 consecutive values (the last block may be
 * short).  m is in E4M3 (sign, 4 exponent bits with bias 7, 3 mantissa bits), v in
 * E5M3 without a sign (5 exponent bits with bias 15, 3 mantissa bits; no infinities,
 * no NaN).  All bytes zero are moments of zero.  Of a block's new moments x in float32
 *   scale  2^E, E = max(-127, floor(log2 max |x|) - top), top = 7 for m, 15 for v
 *   code   |x| 2^-E as a place on the format's grid, to 2^-20 of a code, rounded down
 *          after 20 random bits are added below the last bit kept (stochastic
 *          rounding); a positive v never becomes zero
 * and with an infinity or a NaN in the block its scale is 255 and its codes are 0.
 * The weights' update uses the moments before they are rounded, with a square root and a
 * reciprocal within a unit in the last place each (and correctly rounded for eps near 0).
 * The random bits of value j of tensor i are those of a 32-bit word: m takes bits
 * 31..12, v bits 19..0.  With r = low 32 bits of j / 8 and z_i the low 32 bits of
 * SplitMix64 (Steele, Lea and Flood, 2014) at state seed + i * 0x9E3779B97F4A7C15,
 * s = r * 0x9E3779B1 ^ z_i, s = (s ^ s >> 16) * 0xBB67AE85, s ^= s >> 15, and the
 * words of values 8r .. 8r+7 are the next eight states of Marsaglia's xorshift (13,
 * 17, 5).  Give every step another seed.  Equal arguments give equal results.
 *
 *   state_bits           8 or 32
 *   count                tensors; the arrays below are host memory, read during the call
 *   param_dt, grad_dt    [count] slope_dtype values
 *   params               [count] the weights, updated in place
 *   grads                [count] their gradients
 *   m, v, m_exp, v_exp   [count] the moments, updated in place
 *   n                    [count] numbers of values (0: the tensor is left out)
 *   hp                   hyper-parameters; step counts from 1
 * Tensors need only their element type's alignment.  The step's number and the seed are
 * the call's own: a call recorded into a graph repeats them at each replay.
 * Errors: slope_adamw's, and SLOPE_ERR_INVALID_ARG for other state_bits, count < 0
 * or a written tensor that shares memory with another one or a gradient; SLOPE_ERR_ALIGN for a tensor not
 * aligned to its elements; SLOPE_ERR_UNSUPPORTED for n[i] > 2^34. */
slope_status slope_adamw_multi(int state_bits, int64_t count, const int32_t* param_dt, const int32_t* grad_dt,
                               void* const* params, const void* const* grads, void* const* m, void* const* v,
                               uint8_t* const* m_exp, uint8_t* const* v_exp, const int64_t* n,
                               const slope_adamw_params* hp, uint64_t seed, void* stream);

/* slope_adamw_double_prune_packed with 8-bit moments: one step on the compressed values of
 * W_s, whose new values are written in place and into W_s's tile chunks, and the double
 * prune of the updated W_s into W_dp^T's.  Values, codes and scales are bitwise those of
 * slope_adamw_multi on a list of this one tensor (m, v [N, K/2] codes, m_exp, v_exp [N * K / 64]
 * scales, the same seed), the chunks those of slope_pack_sparse and
 * slope_double_prune_packed of the new values.  dt BF16 or F16; grad_dt BF16, F16 or F32.
 * m_exp and v_exp may have any address.  Errors: those of slope_adamw_double_prune_packed,
 * SLOPE_ERR_SHAPE unless K % 64 == 0 (the blocks of moments lie in one row), and
 * SLOPE_ERR_INVALID_ARG for a written tensor (chunks included) that shares memory with another one. */
slope_status slope_adamw8_double_prune_packed(slope_dtype dt, slope_dtype grad_dt, void* values_s, const uint32_t* meta_s,
                                              const void* dW_values, uint8_t* m, uint8_t* m_exp, uint8_t* v, uint8_t* v_exp,
                                              int64_t N, int64_t K, const slope_adamw_params* hp, uint64_t seed,
                                              void* packed_s, int64_t packed_s_bytes, void* packed_dpT,
                                              int64_t packed_dpT_bytes, void* stream);

/* The values of 8-bit moments (code * 2^E; NaN where the scale is 255): m, v codes
 * [n], m_exp, v_exp scales [ceil(n / 32)], outputs [n] in out_dt: BF16 or F32, both
 * hold every value exactly (bfloat16 has four significant bits to spare).  Either
 * moment may be left out: its three arguments are NULL.  Any alignment of the codes;
 * outputs need their element's.  Errors: SLOPE_ERR_INVALID_ARG for an incomplete
 * moment or none, or an output that shares memory with another argument;
 * SLOPE_ERR_UNSUPPORTED for F16 or n > 2^34. */
slope_status slope_adamw_moments(slope_dtype out_dt, const uint8_t* m_or_null, const uint8_t* m_exp_or_null,
                                 const uint8_t* v_or_null, const uint8_t* v_exp_or_null, int64_t n,
                                 void* m_out_or_null, void* v_out_or_null, void* stream);

/* Largest reduction width of the 4-bit product. */
#define SLOPE_MXFP4_MAX_COLS (1 << 21)

/* In the calls below outputs and workspaces share memory with no other argument (not checked).
 *
 * 4-bit floating point with a scale for 32 values.  Of each 32 consecutive values x of
 * a row (the last block filled up with zeros):
 *   scale  2^E, E = max(-127, e - 2), e the exponent of the largest magnitude rounded to
 *          two significant bits (ties away from zero)
 *   code   the E2M1 number (sign, 2 exponent bits with bias 1, 1 mantissa bit:
 *          magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6) nearest to x 2^-E, ties to the even
 *          code, beyond 6 the code of 6
 * and with an infinity or a NaN in the block its scale is 255 and its codes are 0.
 *
 * Rows of codes: a row of K values takes 64 ceil(K / 128) bytes of codes, 16 for each
 * block, and 16 ceil(K / 512) bytes of scales, one for each block; those of blocks past
 * K are 0.  Within a block value 4g + p is nibble g of the p-th 32-bit word (g = 0..7,
 * p = 0..3). */

/* Bytes of codes and of scales of one row of K values.  Host-only. */
slope_status slope_mxfp4_row_bytes(int64_t K, int64_t* code_bytes, int64_t* scale_bytes);

/* Codes and scales of the rows of X [T, K] (BF16, F16 or F32; any K): codes
 * [T, code_bytes], exps [T, scale_bytes], both overwritten whole.  X needs its element's
 * alignment, codes and exps 16 bytes.  K = 0 or T = 0 does nothing. */
slope_status slope_quantize_mxfp4(slope_dtype dt, const void* X, int64_t T, int64_t K, uint8_t* codes, uint8_t* exps,
                                  void* stream);

/* out [T, K] out_dt <- the values that rows of codes stand for (NaN where the scale is
 * 255).  BF16 and F32 hold them exactly, down to the least, 2^-128; but from 2^128 on they are
 * infinities, and a finite value of at least 1.75 * 2^127 is coded as 2^128 (in a product it
 * counts as that).  F16 rounds to its own range.  out needs its element's alignment. */
slope_status slope_mxfp4_values(slope_dtype out_dt, const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K,
                                void* out, void* stream);

/* Bytes of the 4-bit tile-chunk form of a compressed [rows, cols] matrix (see
 * slope_pack_sparse_mxfp4).  Host-only; SLOPE_ERR_SHAPE if cols % 16 != 0,
 * SLOPE_ERR_UNSUPPORTED if cols > SLOPE_MXFP4_MAX_COLS. */
slope_status slope_packed_sparse_mxfp4_bytes(int64_t rows, int64_t cols, int64_t* bytes);

/* 4-bit tile chunks of a compressed 16-bit 2:4 matrix (values [rows, cols/2], meta
 * [rows, ceil(cols/32)] as slope_compress24 or slope_double_prune write them): 3.25 bits
 * for a dense value.  A block is 32 dense columns, its 16 kept values coded as above.
 * Chunk (t, s) holds rows 64t .. 64t+63 and dense columns 128s .. 128s+127 (four blocks a
 * row), 3328 bytes at offset (t * ceil(cols/128) + s) * 3328:
 *   codes      block b of row r at ((b / 2) * 64 + r) * 16 + (b % 2) * 8: two words, the
 *              first and the second kept code of its groups of four, nibble g for group g
 *   positions  at 2048 + ((b / 2) * 64 + r) * 8 + (b % 2) * 4: a word whose nibble g has
 *              the bits of group g's kept positions
 *   scales     at 3 * 1024 + r * 4 + b: one byte
 * Rows past `rows` and columns past `cols` have codes and scales 0.  packed: caller-owned,
 * at least slope_packed_sparse_mxfp4_bytes(rows, cols) bytes, overwritten.  Errors:
 * SLOPE_ERR_UNSUPPORTED for F32 or cols > SLOPE_MXFP4_MAX_COLS, SLOPE_ERR_SHAPE if cols %
 * 16 != 0, SLOPE_ERR_WORKSPACE if packed is short. */
slope_status slope_pack_sparse_mxfp4(slope_dtype dt, const void* values, const uint32_t* meta, int64_t rows,
                                     int64_t cols, void* packed, int64_t packed_bytes, void* stream);

/* Bytes of device workspace that make slope_spmm_mxfp4_packed fastest: partial sums of up
 * to eight parts of K where T <= 64 tokens of a long K meet few outputs (20480 -> 5120 at 64),
 * 0 elsewhere.  Of the current device.  Host-only; errors as the product's. */
slope_status slope_spmm_mxfp4_workspace_bytes(int64_t T, int64_t K, int64_t N, int64_t* bytes);

/* The 2:4 sparse product on 4-bit floating point:
 *   Y [T, N] = Xq [T, K] . W_q^T
 * of the values that the codes stand for; codes, exps from slope_quantize_mxfp4, packed_w
 * from slope_pack_sparse_mxfp4 of W_s (rows N, cols K), or of W_dp^T (rows K, cols N)
 * with dY's codes, for dX.  float32 sums (the matrix instruction's; which order depends on the
 * sizes and the workspace), rounded once to out_dt (BF16, F16 or F32).  Any T; Y is
 * overwritten, K = 0 gives 0.  No adapter term (slope_lowrank_add adds it).  Y needs 16-byte
 * alignment.  workspace: NULL, or device memory (16-byte aligned, scratch) of any size: of
 * less than slope_spmm_mxfp4_workspace_bytes(T, K, N) bytes the call uses what helps it.
 * Errors: SLOPE_ERR_SHAPE unless K % 16 == 0 and N % 4 == 0; SLOPE_ERR_UNSUPPORTED for K >
 * SLOPE_MXFP4_MAX_COLS; SLOPE_ERR_WORKSPACE if packed_w is short. */
slope_status slope_spmm_mxfp4_packed(slope_dtype out_dt, const uint8_t* codes, const uint8_t* exps, int64_t T,
                                     int64_t K, const void* packed_w, int64_t packed_w_bytes, int64_t N, void* Y,
                                     void* workspace_or_null, int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SLOPE_MX_H_ */
