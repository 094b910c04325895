// Rows of 16-bit (or fp32) values: vector access at element alignment, and the
// 8-bit integer codes of a row (shared by the RMS norm, the row quantizer and
// the int8 weight packing).
#pragma once
#include "common.h"

namespace slope {

// E consecutive elements, loaded and stored in one access.  Only the element's
// own alignment is assumed (a row of odd width starts anywhere): gfx950 takes
// 16-byte global accesses at any address.
template <typename V, int E>
struct __attribute__((packed, aligned(sizeof(V)))) Pack {
  V v[E];
};
template <typename V, int E>
__device__ __forceinline__ Pack<V, E> load_pack(const V* p) {
  return *reinterpret_cast<const Pack<V, E>*>(p);
}
template <typename V, int E>
__device__ __forceinline__ void store_pack(V* p, const Pack<V, E>& x) {
  *reinterpret_cast<Pack<V, E>*>(p) = x;
}

__device__ __forceinline__ float elem_f32(uint16_t v) { return bf16_bits_to_f32(v); }
__device__ __forceinline__ float elem_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float elem_f32(float v) { return v; }
template <typename V> __device__ __forceinline__ V elem_of(float f);
template <> __device__ __forceinline__ uint16_t elem_of<uint16_t>(float f) { return f32_to_bf16_bits(f); }
template <> __device__ __forceinline__ _Float16 elem_of<_Float16>(float f) { return (_Float16)f; }
template <> __device__ __forceinline__ float elem_of<float>(float f) { return f; }

// |u| for a row's maximum, with NaN taken as infinity (fmax would drop it).
__device__ __forceinline__ float finite_or_inf(float u) {
  const float a = __builtin_fabsf(u);
  return a < __builtin_inff() ? a : __builtin_inff();
}
__device__ __forceinline__ double finite_or_inf(double u) {
  const double a = __builtin_fabs(u);
  return a < __builtin_inf() ? a : __builtin_inf();
}
__device__ __forceinline__ float max_of(float a, float b) { return a > b ? a : b; }
__device__ __forceinline__ double max_of(double a, double b) { return a > b ? a : b; }

// Codes of a row whose largest |u| is `amax` (U = float where every u is exact
// in fp32, double where a 16-bit value meets an fp32 gamma).
//
// code = the integer nearest to 127 u / amax, ties to even.  The quotient comes
// from one fp32 reciprocal and is within 2^-16 of the true one (|q| <= 127: two
// roundings of 2^-24 each), so its rounding is decided unless it lies within
// 1e-4 of a border k + 1/2; there the sign of 254 u - (2k + 1) amax decides,
// which is exact in double (at most 43 significant bits in either product).
// About one value in 5000 takes that branch.
template <typename U> struct RowCodes;

__device__ __forceinline__ float border_code(double u, double amax, float q, float k) {
  const double twice = 2.0 * (double)k + (q > k ? 1.0 : -1.0);   // twice the border next to q
  const double d = 254.0 * u - twice * amax;
  const int lo = (int)(0.5 * (twice - 1.0));                     // the codes on its two sides: lo, lo + 1
  return (float)(d > 0.0 ? lo + 1 : d < 0.0 ? lo : lo + (lo & 1));
}

template <> struct RowCodes<float> {
  float amax, lift, inv;
  bool bad;
  __device__ __forceinline__ explicit RowCodes(float a) : amax(a) {
    bad = !(a < __builtin_inff());
    // a power of two that keeps the reciprocal of a tiny amax finite
    lift = a < 0x1p-60f ? 0x1p60f : 1.0f;
    inv = (a > 0.0f && !bad) ? 127.0f / (a * lift) : 0.0f;
  }
  __device__ __forceinline__ float scale() const { return bad ? __builtin_nanf("") : amax / 127.0f; }
  __device__ __forceinline__ int code(float u) const {
    const float q = (u * lift) * inv;
    float k = __builtin_rintf(q);
    if (__builtin_fabsf(q - k) > 0.4999f) k = border_code((double)u, (double)amax, q, k);
    return bad ? 0 : (int)k;
  }
};

template <> struct RowCodes<double> {
  double amax, inv;
  bool bad;
  __device__ __forceinline__ explicit RowCodes(double a) : amax(a) {
    bad = !(a < __builtin_inf());
    inv = (a > 0.0 && !bad) ? 127.0 / a : 0.0;
  }
  __device__ __forceinline__ float scale() const { return bad ? __builtin_nanf("") : (float)amax / 127.0f; }
  __device__ __forceinline__ int code(double u) const {
    const float q = (float)(u * inv);
    float k = __builtin_rintf(q);
    if (__builtin_fabsf(q - k) > 0.4999f) k = border_code(u, amax, q, k);
    return bad ? 0 : (int)k;
  }
};

}  // namespace slope
