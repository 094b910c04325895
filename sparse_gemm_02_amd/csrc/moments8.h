// AdamW with 8-bit moments (blocks of 32 consecutive values with a power-of-two scale each):
// what the kernels that update them share (device side).
//
// A moment x of a block is held as a code of three bits after the
// leading one: E4M3 for m, E5M3 without a sign for v.  A power of two scales the
// block, so scaling rounds nothing and a code is decided by the bits of the fp32
// moment alone.  Scaled so that the format's smallest normal number is float's
// (2^-126), a value's float bits are 8 times its place on the format's grid, in
// units of 2^-23 of a code, subnormal codes included: adding 20 random bits below
// the last bit kept and cutting there rounds it up with the probability of the
// part cut off.  Rounding to nearest would not do: beta2 = 0.999 moves v by a
// thousandth of itself a step, and codes lie an eighth apart, so v would stand
// still; rounded this way its expectation follows the exact average.
#pragma once
#include "adamw.h"
#include "rows8.h"

namespace slope {

// The eight values rounded to their format.
template <typename T>
__device__ __forceinline__ Pack<T, 8> rounded8(const float (&in)[8]) {
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(Pack<T, 8>, in);
  } else {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      b[i] = out16_bits<T>(in[i]);
      // In slope_adamw the compiler rounds the step's last fused multiply-add straight to
      // fp16.  It has to do the same here, and does where each conversion is a value of its
      // own and no branch lies between.
      if constexpr (__is_same(T, _Float16)) asm("" : "+v"(b[i]));
    }
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = b[2 * i] | (b[2 * i + 1] << 16);
    return __builtin_bit_cast(Pack<T, 8>, w);
  }
}

constexpr int kBadExp = 255;                         // a block with an infinity or a NaN
constexpr int kTopM = 7, kDownM = 120;               // largest magnitude in [2^7, 2^8); 2^-6 * 2^-120 = 2^-126
constexpr int kTopV = 15, kDownV = 112;              // in [2^15, 2^16); 2^-14 * 2^-112 = 2^-126

__device__ __forceinline__ float nan_f32() { return __uint_as_float(0x7FC00000u); }
// 2^(b - 127), NaN for 255
__device__ __forceinline__ float exp_value(uint32_t b) {
  return b == (uint32_t)kBadExp ? nan_f32() : b == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}

// Eight m's from their codes and the block's scale.
__device__ __forceinline__ void decode_m(u32x2 w, uint32_t e, float (&m)[8]) {
  const float s = exp_value(e);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
    m[4 * i] = lo[0] * s;
    m[4 * i + 1] = lo[1] * s;
    m[4 * i + 2] = hi[0] * s;
    m[4 * i + 3] = hi[1] * s;
  }
}
// Eight v's; those of a bad block are whatever 2^128 makes of them (the caller's part).
__device__ __forceinline__ void decode_v(u32x2 w, uint32_t e, float (&v)[8]) {
  const int up = (int)e - 127 + kDownV;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = __builtin_ldexpf(__uint_as_float(((w[i / 4] >> (8 * (i % 4))) & 0xFFu) << 20), up);
}

// Largest magnitude of the 32 values that four neighbouring lanes hold (a NaN stays).
__device__ __forceinline__ float block_max(const float (&x)[8]) {
  float a = max_mag(__builtin_fabsf(x[0]), x[1]);
#pragma unroll
  for (int i = 2; i < 8; ++i) a = max_mag(a, x[i]);
  a = max_mag(a, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(a), 0xB1, 0xF, 0xF, false)));
  return max_mag(a, __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(a), 0x4E, 0xF, 0xF, false)));
}
// The scale's byte of a block whose largest magnitude has the bits hi.
__device__ __forceinline__ uint32_t scale_byte(uint32_t hi, int top) {
  if (hi >= 0x7F800000u) return kBadExp;
  const int b = (int)(hi >> 23) - top;               // 127 + floor(log2) - top
  return b < 0 ? 0u : (uint32_t)b;
}
// Top bytes of eight words.
__device__ __forceinline__ u32x2 top_bytes(const uint32_t (&t)[8]) {
  u32x2 w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __builtin_amdgcn_perm(t[4 * i + 1], t[4 * i], 0x0C0C0703u);
    const uint32_t hi = __builtin_amdgcn_perm(t[4 * i + 3], t[4 * i + 2], 0x07030C0Cu);
    w[i] = lo | hi;
  }
  return w;
}

// Random bits of a run of eight values: a hashed start from the run's number
// within its tensor and the tensor's seed, then Marsaglia's xorshift (13, 17, 5).
struct Noise {
  uint32_t s;
  __device__ __forceinline__ Noise(uint32_t run, uint32_t seed) {
    s = run * 0x9E3779B1u ^ seed;
    s = (s ^ (s >> 16)) * 0xBB67AE85u;
    s ^= s >> 15;
  }
  __device__ __forceinline__ uint32_t next() {
    s ^= s << 13;
    s ^= s >> 17;
    s ^= s << 5;
    return s;
  }
};

// New codes of eight m's and v's of a block with the scale bytes em, ev.  With the
// scaled value's bits (28 of them) moved up by four, the code is the top byte of
// their sum with 24 random bits (the lowest four never carry).
__device__ __forceinline__ void encode(const float (&m)[8], const float (&v)[8], uint32_t em, uint32_t ev, Noise noise,
                                       u32x2& cm, u32x2& cv) {
  const int dm = 127 - (int)em - kDownM, dv = 127 - (int)ev - kDownV;
  uint32_t tm[8], tv[8], least = ~0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t r = noise.next();
    const uint32_t ym = __float_as_uint(__builtin_ldexpf(__builtin_fabsf(m[i]), dm));
    const uint32_t yv = __float_as_uint(__builtin_ldexpf(v[i], dv));
    tm[i] = (((ym << 4) + (r >> 8)) & 0x7FFFFFFFu) | (__float_as_uint(m[i]) & 0x80000000u);
    tv[i] = (yv + (r & 0xFFFFFu)) << 4;
    least = tv[i] < least ? tv[i] : least;
  }
  if (least < (1u << 24)) {                          // a positive v never becomes zero: m would be divided by eps
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (v[i] > 0.0f && tv[i] < (1u << 24)) tv[i] = 1u << 24;
  }
  const u32x2 zero = {0u, 0u};
  cm = em == (uint32_t)kBadExp ? zero : top_bytes(tm);
  cv = ev == (uint32_t)kBadExp ? zero : top_bytes(tv);
}

// adamw_apply with the hardware's square root and reciprocal, each within a unit in the
// last place (the moments, whose bits decide codes, are computed the same way).  With the
// correctly rounded ones the 8-bit step of 16-bit weights is bound by the vector units:
// 160 million bf16 values 328 us, so 308; of fp32 ones 480 either way.
__device__ __forceinline__ float adamw_apply_fast(float p, float g, float& m, float& v, const AdamWStep& c) {
#pragma clang fp contract(off)
  m = __builtin_fmaf(c.beta1, m, c.omb1 * g);
  v = __builtin_fmaf(c.beta2, v, c.omb2 * (g * g));
  const float den = __builtin_fmaf(__builtin_amdgcn_sqrtf(v), c.inv_sqrt_bc2, c.eps);
  return __builtin_fmaf(-c.step_size, m * __builtin_amdgcn_rcpf(den), p * c.decay);
}

template <typename PT, bool FAST>
__device__ __forceinline__ Pack<PT, 8> step8(float (&p)[8], const float (&g)[8], float (&m)[8], float (&v)[8],
                                             const AdamWStep& c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) p[i] = FAST ? adamw_apply_fast(p[i], g[i], m[i], v[i], c) : adamw_apply(p[i], g[i], m[i], v[i], c);
  return rounded8<PT>(p);
}


// Eight moments of each kind, a run of a block, and their block's scales.
struct Run8 {
  u32x2 m, v;
  uint32_t em, ev;
};
// One step on a run's weights p and gradients g; four neighbouring lanes hold a block.  `left` values
// of the run are there: the others' codes are zeros, and they are no part of the block's largest.
template <typename PT, bool FAST>
__device__ __forceinline__ Pack<PT, 8> update8(float (&p)[8], const float (&g)[8], Run8& r, int64_t left, AdamWStep c,
                                               Noise noise) {
  float m[8], v[8];
  decode_m(r.m, r.em, m);
  decode_v(r.v, r.ev, v);
  if (r.ev == (uint32_t)kBadExp) c.beta2 = nan_f32();   // every v of the block is a NaN
  const Pack<PT, 8> np = step8<PT, FAST>(p, g, m, v, c);
  if (left < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= left) m[i] = v[i] = 0.0f;
  }
  r.em = scale_byte(__float_as_uint(block_max(m)), kTopM);
  r.ev = scale_byte(__float_as_uint(block_max(v)), kTopV);
  encode(m, v, r.em, r.ev, noise, r.m, r.v);
  return np;
}

// Whether a step takes the hardware's root and reciprocal.  The root of a v below 2^-126 is
// zero there: eps has to be so large that it does not show.
inline bool fast_step(const AdamWStep& c) { return c.eps >= 0x1p-39f * c.inv_sqrt_bc2; }

// 32 bits for tensor i of a call (SplitMix64 of Steele, Lea and Flood, 2014).
inline uint32_t tensor_seed(uint64_t seed, int64_t i) {
  uint64_t z = seed + (uint64_t)(i + 1) * 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return (uint32_t)(z ^ (z >> 31));
}

}  // namespace slope
