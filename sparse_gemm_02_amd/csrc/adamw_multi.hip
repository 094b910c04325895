// One AdamW step over many tensors in one launch, with moments in fp32 or in 8
// bits (blocks of 32 consecutive values with a power-of-two scale each), and the
// 8-bit moments as values.
//
// 8-bit moments.  A moment x of a block is held as a code of three bits after the
// leading one: E4M3 for m, E5M3 without a sign for v.  A power of two scales the
// block, so scaling rounds nothing and a code is decided by the bits of the fp32
// moment alone.  Scaled so that the format's smallest normal number is float's
// (2^-126), a value's float bits are 8 times its place on the format's grid, in
// units of 2^-23 of a code, subnormal codes included: adding 20 random bits below
// the last bit kept and cutting there rounds it up with the probability of the
// part cut off.  Rounding to nearest would not do: beta2 = 0.999 moves v by a
// thousandth of itself a step, and codes lie an eighth apart, so v would stand
// still; rounded this way its expectation follows the exact average.
#include <algorithm>
#include <type_traits>

#include "adamw.h"
#include "adamw_args.h"
#include "rows8.h"

namespace slope {

namespace {

constexpr int kThreads = 256, kPerThread = 8, kSlice = kThreads * kPerThread;
constexpr int kTensors = 56;                          // of one launch: its arguments stay below 4 KB

struct MultiArgs {
  void* p[kTensors];
  const void* g[kTensors];
  void* m[kTensors];
  void* v[kTensors];
  uint8_t* me[kTensors];
  uint8_t* ve[kTensors];
  int64_t n[kTensors];
  uint32_t first[kTensors];                          // first block of the tensor
  uint32_t seed[kTensors];
  int32_t count;
};
static_assert(sizeof(MultiArgs) + sizeof(AdamWStep) <= 4096, "kernel arguments");

// Eight elements of one or two bytes past the caches' usual order (NT): what they hold is
// not used again before it would be displaced.  A wave's access covers whole lines; fp32 ones,
// two accesses a lane with every second 16 bytes, lose by it (2^27 fp32 values 674 -> 740 us).
template <typename V>
__device__ __forceinline__ Pack<V, 8> load_nt(const V* p) {
  typedef uint32_t Words __attribute__((ext_vector_type(2 * sizeof(V)), aligned(1)));
  const Words w = __builtin_nontemporal_load(reinterpret_cast<const Words*>(p));
  return __builtin_bit_cast(Pack<V, 8>, w);
}
template <typename V>
__device__ __forceinline__ void store_nt(V* p, const Pack<V, 8>& x) {
  typedef uint32_t Words __attribute__((ext_vector_type(2 * sizeof(V)), aligned(1)));
  __builtin_nontemporal_store(__builtin_bit_cast(Words, x), reinterpret_cast<Words*>(p));
}

// Eight values e .. e + 7 of the n at p (those that are not there read as zero, and e may
// be negative).
template <bool NT, typename T>
__device__ __forceinline__ void load8(const T* p, int64_t e, int64_t n, float (&out)[8]) {
  if (e >= 0 && e + 8 <= n) {
    Pack<T, 8> x;
    if constexpr (NT && sizeof(T) < 4) x = load_nt(p + e);
    else x = load_pack<T, 8>(p + e);
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = elem_f32(x.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) out[i] = (uint64_t)(e + i) < (uint64_t)n ? elem_f32(p[e + i]) : 0.0f;
  }
}
template <bool NT, typename T>
__device__ __forceinline__ void store8(T* p, int64_t e, int64_t n, const Pack<T, 8>& x) {
  if (e >= 0 && e + 8 <= n) {
    if constexpr (NT && sizeof(T) < 4) store_nt(p + e, x);
    else store_pack<T, 8>(p + e, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((uint64_t)(e + i) < (uint64_t)n) p[e + i] = x.v[i];
  }
}
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
template <bool NT>
__device__ __forceinline__ u32x2 load_codes(const uint8_t* p, int64_t left) {
  if (left >= 8) {
    Pack<uint8_t, 8> x;
    if constexpr (NT) x = load_nt(p);
    else x = load_pack<uint8_t, 8>(p);
    return __builtin_bit_cast(u32x2, x);
  }
  u32x2 w = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < left) w[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  return w;
}
template <bool NT>
__device__ __forceinline__ void store_codes(uint8_t* p, int64_t left, u32x2 w) {
  if (left >= 8) {
    const auto x = __builtin_bit_cast(Pack<uint8_t, 8>, w);
    if constexpr (NT) store_nt(p, x);
    else store_pack<uint8_t, 8>(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

// ---------------------------------------------------------------- 8-bit moments
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

// ---------------------------------------------------------------- the step
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

// Values by which m's start is past a 32-byte border: with fp32 moments a thread's eight
// values begin there, since tensors that follow each other in one buffer begin anywhere
// (6 million fp32 values at an odd place 34 us, from the tensor's first value on 40).
__host__ __device__ __forceinline__ int lead32(const void* m) { return (int)(reinterpret_cast<uintptr_t>(m) / 4 % 8); }

// A block of threads takes 2048 values of one tensor, a thread eight of them; four lanes
// hold a block of 32.  Bound by memory: 160 million bf16 weights and gradients with 8-bit
// moments 278 us (10.1 bytes a value read and written, 5.9 TB/s; a copy reaches 5.1), with
// fp32 moments 609 (22 bytes, 5.8).  Two or four such parts a block of
// threads take 3 to 4 % longer from 2^24 values on and nothing less below.
template <typename PT, typename GT, bool EIGHT, bool FAST, bool NT>
__global__ __launch_bounds__(kThreads) void adamw_multi_kernel(const MultiArgs a, const AdamWStep c0) {
  int lo = 0, hi = a.count;                          // the last tensor whose first block is not behind this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.first[mid] <= blockIdx.x) lo = mid; else hi = mid;
  }
  const int64_t n = a.n[lo];
  PT* p = (PT*)a.p[lo];
  const GT* g = (const GT*)a.g[lo];
  int64_t e = (int64_t)(blockIdx.x - a.first[lo]) * kSlice + threadIdx.x * kPerThread;
  float pf[8], gf[8], mf[8], vf[8];
  AdamWStep c = c0;
  if constexpr (EIGHT) {
    load8<NT>(p, e, n, pf);
    load8<NT>(g, e, n, gf);
    const int64_t left = n - e, at = left > 0 ? e : 0, block = at / 32;   // lanes past the end: no access, zeros
    uint8_t* m = (uint8_t*)a.m[lo];
    uint8_t* v = (uint8_t*)a.v[lo];
    const uint32_t em = left > 0 ? a.me[lo][block] : 0u, ev = left > 0 ? a.ve[lo][block] : 0u;
    decode_m(load_codes<NT>(m + at, left), em, mf);
    decode_v(load_codes<NT>(v + at, left), ev, vf);
    if (ev == (uint32_t)kBadExp) c.beta2 = nan_f32();   // every v of the block is a NaN
    const Pack<PT, 8> np = step8<PT, FAST>(pf, gf, mf, vf, c);
    if (left < 8) {                                  // nothing is there: no part of the block's largest
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= left) mf[i] = vf[i] = 0.0f;
    }
    const uint32_t nm = scale_byte(__float_as_uint(block_max(mf)), kTopM);
    const uint32_t nv = scale_byte(__float_as_uint(block_max(vf)), kTopV);
    u32x2 cm, cv;
    encode(mf, vf, nm, nv, Noise((uint32_t)(e / 8), a.seed[lo]), cm, cv);
    if (left > 0) {
      store_codes<NT>(m + at, left, cm);
      store_codes<NT>(v + at, left, cv);
      if (threadIdx.x % 4 == 0) {
        a.me[lo][block] = (uint8_t)nm;
        a.ve[lo][block] = (uint8_t)nv;
      }
    }
    store8<NT>(p, e, n, np);
  } else {
    float* m = (float*)a.m[lo];
    float* v = (float*)a.v[lo];
    e -= lead32(m);
    load8<NT>(p, e, n, pf);
    load8<NT>(g, e, n, gf);
    load8<NT>(m, e, n, mf);
    load8<NT>(v, e, n, vf);
    const Pack<PT, 8> np = step8<PT, FAST>(pf, gf, mf, vf, c);
    store8<NT>(m, e, n, rounded8<float>(mf));
    store8<NT>(v, e, n, rounded8<float>(vf));
    store8<NT>(p, e, n, np);
  }
}

// The values that 8-bit codes stand for.  n values, each thread eight of one moment:
// 160 million of both as bf16 156 us, 6.2 TB/s (178 with blocks that loop, 163 without NT).
template <typename O, bool V, bool NT>
__device__ __forceinline__ void values8(const uint8_t* codes, const uint8_t* exps, int64_t n, O* out) {
  const int64_t e = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kPerThread, left = n - e;
  if (left <= 0) return;
  const uint32_t b = exps[e / 32];
  const u32x2 w = load_codes<NT>(codes + e, left);
  float f[8];
  if constexpr (V) {
    decode_v(w, b, f);
    if (b == (uint32_t)kBadExp) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = nan_f32();
    }
  } else {
    decode_m(w, b, f);
  }
  store8<NT>(out, e, n, rounded8<O>(f));
}
template <typename O, bool NT>
__global__ __launch_bounds__(kThreads) void moments_kernel(const uint8_t* __restrict__ m, const uint8_t* __restrict__ me,
                                                           const uint8_t* __restrict__ v, const uint8_t* __restrict__ ve,
                                                           int64_t n, O* __restrict__ mo, O* __restrict__ vo) {
  if (blockIdx.y == 0 && mo) values8<O, false, NT>(m, me, n, mo);
  if (blockIdx.y == 1 && vo) values8<O, true, NT>(v, ve, n, vo);
}

// From these many values on a call's tensors pass the last-level cache (256 MB) before anything reads
// them again.  8-bit moments, bf16, 2^25 values 68.5 us, so 64.7; 2^27: 247 and 235 (fp32 weights 393
// and 370); 7 million fp16 values that stay there, and their moments read out next: 28.7, so 29.8.  fp32
// moments, bf16 weights, 2^24: 71.4 and 67.1; 2^27: 533 and 506.
constexpr int64_t streams_from(bool eight) { return int64_t(1) << (eight ? 25 : 24); }

struct Form {
  bool eight, fast, nt;
};
template <typename PT, typename GT>
hipError_t go(const Form& f, const MultiArgs& a, unsigned blocks, const AdamWStep& c, hipStream_t s) {
  if (!f.eight && !f.nt) adamw_multi_kernel<PT, GT, false, false, false><<<blocks, kThreads, 0, s>>>(a, c);
  else if (!f.eight) adamw_multi_kernel<PT, GT, false, false, true><<<blocks, kThreads, 0, s>>>(a, c);
  else if (!f.fast) adamw_multi_kernel<PT, GT, true, false, false><<<blocks, kThreads, 0, s>>>(a, c);
  else if (!f.nt) adamw_multi_kernel<PT, GT, true, true, false><<<blocks, kThreads, 0, s>>>(a, c);
  else adamw_multi_kernel<PT, GT, true, true, true><<<blocks, kThreads, 0, s>>>(a, c);
  return hipGetLastError();
}
template <typename PT>
hipError_t go_grad(Dt g, const Form& f, const MultiArgs& a, unsigned blocks, const AdamWStep& c, hipStream_t s) {
  if (g == Dt::BF16) return go<PT, uint16_t>(f, a, blocks, c, s);
  if (g == Dt::F16) return go<PT, _Float16>(f, a, blocks, c, s);
  return go<PT, float>(f, a, blocks, c, s);
}
hipError_t launch_one(Dt p, Dt g, const Form& f, const MultiArgs& a, unsigned blocks, const AdamWStep& c, hipStream_t s) {
  if (p == Dt::BF16) return go_grad<uint16_t>(g, f, a, blocks, c, s);
  if (p == Dt::F16) return go_grad<_Float16>(g, f, a, blocks, c, s);
  return go_grad<float>(g, f, a, blocks, c, s);
}

// 32 bits for tensor i of a call (SplitMix64 of Steele, Lea and Flood, 2014).
uint32_t tensor_seed(uint64_t seed, int64_t i) {
  uint64_t z = seed + (uint64_t)(i + 1) * 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return (uint32_t)(z ^ (z >> 31));
}

}  // namespace

// A launch takes tensors of one pair of types; most lists have one or two pairs.
hipError_t launch_adamw_multi(bool eight, const AdamWTensors& t, const AdamWStep& c, uint64_t seed, hipStream_t s) {
  // The hardware's root of a v below 2^-126 is zero: eps has to be so large that it does not show.
  const bool fast = eight && c.eps >= 0x1p-39f * c.inv_sqrt_bc2;
  for (int pair = 0; pair < 9; ++pair) {
    const int pd = pair / 3, gd = pair % 3;
    int64_t total = 0;
    for (int64_t i = 0; i < t.count; ++i)
      if (t.param_dt[i] == pd && t.grad_dt[i] == gd) total += t.n[i];
    if (total == 0) continue;
    const Form form{eight, fast, total >= streams_from(eight)};
    MultiArgs a;
    int64_t blocks = 0;
    a.count = 0;
    auto flush = [&]() {
      if (a.count == 0) return hipSuccess;
      const hipError_t e = launch_one((Dt)pd, (Dt)gd, form, a, (unsigned)blocks, c, s);
      a.count = 0;
      blocks = 0;
      return e;
    };
    constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;   // below 2^32 threads
    static_assert(kMultiMaxElems / kSlice + 1 <= kMaxBlocks, "a tensor's blocks");
    for (int64_t i = 0; i < t.count; ++i) {
      if (t.param_dt[i] != pd || t.grad_dt[i] != gd || t.n[i] == 0) continue;
      const int64_t need = cdiv(t.n[i] + (eight ? 0 : lead32(t.m[i])), kSlice);
      if (a.count == kTensors || blocks + need > kMaxBlocks) {
        const hipError_t e = flush();
        if (e != hipSuccess) return e;
      }
      const int k = a.count++;
      a.p[k] = t.p[i];
      a.g[k] = t.g[i];
      a.m[k] = t.m[i];
      a.v[k] = t.v[i];
      a.me[k] = eight ? t.me[i] : nullptr;
      a.ve[k] = eight ? t.ve[i] : nullptr;
      a.n[k] = t.n[i];
      a.first[k] = (uint32_t)blocks;
      a.seed[k] = tensor_seed(seed, i);
      blocks += need;
    }
    const hipError_t e = flush();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw_moments(Dt out, const uint8_t* m, const uint8_t* me, const uint8_t* v, const uint8_t* ve,
                                int64_t n, void* mo, void* vo, hipStream_t s) {
  if (n == 0) return hipSuccess;
  const dim3 grid((unsigned)cdiv(n, kSlice), 2);
  auto put = [&](auto* m_to, auto* v_to) {
    using O = std::remove_pointer_t<decltype(m_to)>;
    if (n >= streams_from(true)) moments_kernel<O, true><<<grid, kThreads, 0, s>>>(m, me, v, ve, n, m_to, v_to);
    else moments_kernel<O, false><<<grid, kThreads, 0, s>>>(m, me, v, ve, n, m_to, v_to);
  };
  if (out == Dt::BF16) put((uint16_t*)mo, (uint16_t*)vo);
  else put((float*)mo, (float*)vo);
  return hipGetLastError();
}

}  // namespace slope
