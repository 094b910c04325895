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

// ---------------------------------------------------------------- codes of a row
// code = the integer nearest to 127 u / amax, ties to even; amax = max |u| of the
// row, u = h g the exact product of two stored values.  u is seen as p = fp32(h g)
// and what the rounding left, h g - p (zero where g has 16 bits too: the product
// then fits).

// The larger of a and |p|; a NaN stays (one instruction takes two values of p).
__device__ __forceinline__ float max_mag(float a, float p) {
  return __builtin_elementwise_maximum(a, __builtin_fabsf(p));
}
// Bits of |p|: they order like magnitudes, with infinity and NaN on top, so a row
// without a finite maximum shows in the largest.
__device__ __forceinline__ uint32_t mag_bits(float p) { return __float_as_uint(p) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }
// |f w| - |p| for p = fp32(f w), exact
__device__ __forceinline__ float left_over(float f, float w, float p) {
  return __builtin_copysignf(1.0f, p) * __builtin_fmaf(f, w, -p);
}

constexpr float kUnsure = 0.49995f;                    // from an integer: the rounding may go either way
constexpr float kCodeMagic = 12582912.0f;             // 1.5 * 2^23: adding it rounds to an integer, ties to even

// Below it a row's products leave fp32's normal range, and p may have lost bits that
// no left-over shows.
constexpr uint32_t kTinyBits = 0x0D800000u;           // 2^-100
__device__ __forceinline__ bool tiny_bits(uint32_t hi) { return hi < kTinyBits; }

// Codes of a row whose largest |p| has the bits `hi` and whose largest |u| is amax:
// hi and the largest left-over of the values with that p, or, in a row of tiny_bits,
// the largest of the products themselves.
//
// The quotient from one fp32 reciprocal, q = p * (127 / hi), is within 4e-5 of
// the true one (|q| <= 127; p, hi, the division and the product each round by
// 2^-24 of it at most: 3.1e-5), so its rounding is decided unless it lies within
// 5e-5 of a border k + 1/2.  There the sign of 254 u - (2k + 1) amax decides, which is
// exact in double (products of at most 43 bits).  About one value in 10000 takes
// that branch.  Rows of tiny_bits go by double throughout.
struct RowCodes {
  double amax;
  uint32_t hi;
  float inv;
  bool bad, tiny;
  __device__ __forceinline__ RowCodes(uint32_t hi_, double amax_) : amax(amax_), hi(hi_) {
    bad = hi >= 0x7F800000u;
    tiny = tiny_bits(hi);
    inv = bad || tiny ? 0.f : 127.0f / __uint_as_float(hi);
  }
  // (a tiny row's own scale may be far below fp32's normal range where the product
  // with the norm's factor is not: one rounding of both)
  __device__ __forceinline__ float scale(float rstd) const {
    if (bad) return __builtin_nanf("");
    return tiny ? (float)(amax / 127.0 * (double)rstd) : __uint_as_float(hi) / 127.0f * rstd;
  }
  // the code beside the border next to q (k = q rounded)
  __device__ __forceinline__ float at_border(double u, float q, float k) const {
    const double twice = 2.0 * (double)k + (q > k ? 1.0 : -1.0), d = 254.0 * u - twice * amax;
    const int below = (int)(0.5 * (twice - 1.0));     // the codes on its two sides: below, below + 1
    return (float)(d > 0.0 ? below + 1 : d < 0.0 ? below : below + (below & 1));
  }
  // one value, any row
  __device__ __forceinline__ int code(double u) const {
    if (bad || amax == 0.0) return 0;
    const double q = 127.0 * u / amax;
    const float k = (float)__builtin_rint(q);
    return (int)(__builtin_fabs(q - k) > 0.4999 ? at_border(u, (float)q, k) : k);
  }
  // The four codes of p[0..3], one a byte (an ordinary row).  u(i) gives the exact
  // product of value i.
  template <typename F>
  __device__ __forceinline__ uint32_t four(const float (&p)[4], F&& u) const {
    float t[4], far = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float q = p[i] * inv;
      t[i] = q + kCodeMagic;
      far = __builtin_fmaxf(far, __builtin_fabsf(q - (t[i] - kCodeMagic)));
    }
    if (far > kUnsure) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float q = p[i] * inv, k = t[i] - kCodeMagic;
        if (__builtin_fabsf(q - k) > kUnsure) t[i] = at_border(u(i), q, k) + kCodeMagic;
      }
    }
    // the low bytes of t are the codes in two's complement
    return __builtin_amdgcn_perm(__float_as_uint(t[1]), __float_as_uint(t[0]), 0x0C0C0400u) |
           __builtin_amdgcn_perm(__float_as_uint(t[3]), __float_as_uint(t[2]), 0x04000C0Cu);
  }
};

}  // namespace slope
