// 4-bit floating point with a power-of-two scale for 32 values: the codes of rows, the
// values they stand for, and the tile chunks of a 2:4 weight.
//
// E2M1 has two significant bits, so the scale of a block, a power of two, rounds
// nothing: a code is the E2M1 number nearest to x / 2^E (ties to the even code, beyond
// 6 the code of 6), by gfx950's scaled conversion (checked against a host model over
// all 16-bit patterns).  E is the exponent of the largest magnitude rounded to E2M1's
// two bits, less two: magnitudes up to 7 * 2^E, the middle between 6 and the next
// E2M1 number 8, become 6, larger ones raise E.
//
// The order of a block's 32 values: word p (of four) holds in nibble g value 4g + p.
// A 2:4 weight's kept codes are held as two words, the first and the second kept one of
// eight groups, with eight nibbles of kept positions.  Word p of the dense block is
// then one of the two words under a mask that the nibbles' bit p makes, for eight
// groups at a time.
#include <algorithm>

#include "common.h"
#include "launch.h"
#include "mxfp4.h"
#include "rows8.h"

namespace slope {

namespace {

constexpr int kThreads = 256;

// The scale's byte of a block whose largest magnitude has the bits hi (infinities and
// NaN: kMxBad).
__device__ __forceinline__ uint32_t scale_byte(uint32_t hi) {
  if (hi >= 0x7F800000u) return kMxBad;
  const int b = (int)((hi + 0x200000u) >> 23) - 2;
  return b < 0 ? 0u : (uint32_t)b;
}
__device__ __forceinline__ float scale_value(uint32_t b) { return b ? __uint_as_float(b << 23) : __uint_as_float(0x00400000u); }

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// The codes of a and b in byte I of `old`.
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t old, uint16_t a, uint16_t b, float scale) {
  const bf16x2 x = {__builtin_bit_cast(__bf16, a), __builtin_bit_cast(__bf16, b)};
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, x, scale, I);
}
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t old, _Float16 a, _Float16 b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, f16x2{a, b}, scale, I);
}
template <int I>
__device__ __forceinline__ uint32_t codes2(uint32_t old, float a, float b, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, I);
}
// The codes of eight values x[0], x[step], .. as the nibbles of a word.
template <int STEP, typename In>
__device__ __forceinline__ uint32_t codes8(const In* x, float scale) {
  uint32_t w = codes2<0>(0u, x[0], x[STEP], scale);
  w = codes2<1>(w, x[2 * STEP], x[3 * STEP], scale);
  w = codes2<2>(w, x[4 * STEP], x[5 * STEP], scale);
  return codes2<3>(w, x[6 * STEP], x[7 * STEP], scale);
}

// Up to N values from p on into x; the others are zero.
template <int N, typename In>
__device__ __forceinline__ void load_some(const In* p, int64_t left, In (&x)[N]) {
  constexpr int E = 16 / sizeof(In);
  if (left >= N) {
#pragma unroll
    for (int j = 0; j < N / E; ++j) {
      const Pack<In, E> v = load_pack<In, E>(p + j * E);
#pragma unroll
      for (int i = 0; i < E; ++i) x[j * E + i] = v.v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < left ? p[i] : In(0);
  }
}
template <int N, typename In>
__device__ __forceinline__ uint32_t largest(const In (&x)[N]) {
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) a = max_mag(a, elem_f32(x[i]));
  return __float_as_uint(a);
}

// ---------------------------------------------------------------- rows
// Items of a launch (fewer than 2^31 threads' parts), per_row of them a row: item / per_row
// is a product's high half with ceil(2^(31 + shift) / per_row), 2^shift >= per_row
// (Granlund and Montgomery, 1994).  64-bit divisions took longer than the memory.
struct Items {
  uint32_t count, per_row, factor, shift;
  Items(int64_t rows, int64_t per_row_) : count((uint32_t)(rows * per_row_)), per_row((uint32_t)per_row_), shift(2) {
    while ((int64_t(1) << shift) < per_row_) ++shift;
    factor = (uint32_t)((((uint64_t)1 << (31 + shift)) + (uint64_t)per_row_ - 1) / (uint64_t)per_row_);
  }
  __device__ __forceinline__ uint32_t row(uint32_t i) const { return __umulhi(i, factor) >> (shift - 1); }
};

template <int CTRL>
__device__ __forceinline__ uint32_t of_quad(uint32_t w) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)w, CTRL, 0xF, 0xF, false);
}
// Byte p of lane q becomes byte q of lane p, in four neighbouring lanes: neighbours
// exchange bytes, pairs of them halves.
struct QuadBytes {
  uint32_t bytes, halves;
  __device__ __forceinline__ explicit QuadBytes(int lane)
      : bytes(lane & 1 ? 0x03070105u : 0x06020400u), halves(lane & 2 ? 0x03020706u : 0x05040100u) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const {
    w = __builtin_amdgcn_perm(of_quad<0xB1>(w), w, bytes);
    return __builtin_amdgcn_perm(of_quad<0x4E>(w), w, halves);
  }
};

// A thread makes a block of 32 values; what lies past K is zero.  Bound by memory: 8192 x
// 9216 bf16 34.7 us, 5.5 TB/s of what it reads and writes (a copy reaches 5.1).  With eight
// values a thread, as below, 34.2 to 36.5, and short rows longer.
template <typename In>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const In* __restrict__ X, Items items, uint32_t K,
                                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= items.count) return;
  const uint32_t coded = (uint32_t)mx_code_bytes(K);
  const uint32_t t = items.row(i), block = i - t * items.per_row, k = block * 32;
  In x[32];
  load_some<32>(X + ((uint64_t)t * K + (k < K ? k : 0)), (int64_t)K - k, x);
  const uint32_t b = scale_byte(largest(x));
  const float s = scale_value(b);
  u32x4 w = {codes8<4>(x, s), codes8<4>(x + 1, s), codes8<4>(x + 2, s), codes8<4>(x + 3, s)};
  if (b == kMxBad) w = u32x4{0u, 0u, 0u, 0u};
  if (block * 16 < coded) *reinterpret_cast<u32x4*>(codes + ((uint64_t)t * coded + block * 16)) = w;
  exps[i] = (uint8_t)b;
}

// The values of one byte's two codes, times s.  (Exact where they are float32 numbers;
// the conversion's own scaling is not used, since s may be a NaN or below 2^-126.)
template <int BYTE>
__device__ __forceinline__ void values2(uint32_t w, float s, float& low, float& high) {
  const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, BYTE);
  low = v[0] * s;
  high = v[1] * s;
}
constexpr int kPer = 2;

// Four neighbouring lanes hold a block, in memory a word each, in registers byte q of all
// four.  An item of 16-bit output is a lane's eight values, of fp32 output four (16 bytes both):
// eight lanes hold a block then, and lane r has the group r.
// Two items a thread, loaded first.  8192 x 9216 bf16 34.8 us, 5.5 TB/s (a thread with a
// whole block's 64-byte store 74 us, one item a thread 40.8, four 36.9); fp32 4096 x 9216 34.1.
template <typename O>
__global__ __launch_bounds__(kThreads) void values_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ exps, Items items, uint32_t K,
                                                          O* __restrict__ out) {
  constexpr int E = 16 / sizeof(O), LANES = 32 / E;
  const uint32_t i0 = blockIdx.x * (kPer * kThreads) + threadIdx.x;
  const uint32_t coded = (uint32_t)mx_code_bytes(K), scales = (uint32_t)mx_scale_bytes(K);
  const QuadBytes turn(threadIdx.x);
  uint32_t w[kPer], b[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const uint32_t i = i0 + u * kThreads, t = items.row(i), block = (i - t * items.per_row) / LANES;
    w[u] = b[u] = 0u;
    if (i < items.count) {
      w[u] = *reinterpret_cast<const uint32_t*>(codes + ((uint64_t)t * coded + block * 16 + threadIdx.x % 4 * 4));
      b[u] = exps[(uint64_t)t * scales + block];
    }
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const uint32_t i = i0 + u * kThreads, t = items.row(i), k = (i - t * items.per_row) * E;
    uint32_t own = turn(w[u]);                       // byte p: the values p of the groups 2q and 2q + 1
    const float s = b[u] == kMxBad ? __builtin_nanf("") : scale_value(b[u]);
    float f[E];
    if constexpr (E == 8) {
      values2<0>(own, s, f[0], f[4]);
      values2<1>(own, s, f[1], f[5]);
      values2<2>(own, s, f[2], f[6]);
      values2<3>(own, s, f[3], f[7]);
    } else {                                         // lane r of eight: the groups of lane r / 2 of either four
      own = threadIdx.x & 4 ? of_quad<0xFA>(own) : of_quad<0x50>(own);
      own >>= threadIdx.x % 2 * 4;
      f[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(own, 1.0f, 0)[0] * s;
      f[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(own, 1.0f, 1)[0] * s;
      f[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(own, 1.0f, 2)[0] * s;
      f[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(own, 1.0f, 3)[0] * s;
    }
    u32x4 h;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (E == 4)
        h[j] = __float_as_uint(f[j]);
      else if constexpr (__is_same(O, uint16_t))     // every value is a bf16 number: its upper half
        h[j] = __builtin_amdgcn_perm(__float_as_uint(f[2 * j + 1]), __float_as_uint(f[2 * j]), 0x07060302u);
      else
        h[j] = out16_bits<O>(f[2 * j]) | ((uint32_t)out16_bits<O>(f[2 * j + 1]) << 16);
    }
    const auto y = __builtin_bit_cast(Pack<O, E>, h);
    if (i >= items.count) continue;
    O* o = out + ((uint64_t)t * K + k);
    if (k + E <= K) {
      store_pack<O, E>(o, y);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (k + e < K) o[e] = y.v[e];
    }
  }
}

// ---------------------------------------------------------------- tile chunks
// A thread makes one row's block of 32 dense columns: 16 kept values, one metadata word.
// 27648 x 9216 91.6 us, 4.3 TB/s of what it reads and writes (once for a weight that is served).
template <typename In>
__global__ __launch_bounds__(kThreads) void pack_kernel(const In* __restrict__ vals, const uint32_t* __restrict__ meta,
                                                        int64_t M, int64_t K, int64_t stages, int64_t tile0,
                                                        uint8_t* __restrict__ out) {
  const int64_t tile = tile0 + blockIdx.x / (uint32_t)stages, stage = blockIdx.x % (uint32_t)stages;
  const int r = threadIdx.x >> 2, b = threadIdx.x & 3;   // row and block within the chunk
  const int64_t row = tile * kMxRows + r, k = stage * kMxCols + b * 32, half = K / 2, wpr = (K / 4 + 7) / 8;
  const bool live = row < M && k < K;
  In x[16];
  load_some<16>(vals + (live ? row * half + k / 2 : 0), live ? half - k / 2 : 0, x);
  const uint32_t word = live ? meta[row * wpr + k / 32] : 0u;
  const uint32_t e = live ? scale_byte(largest(x)) : 0u;
  const float s = scale_value(e);
  uint32_t first = codes8<2>(x, s), second = codes8<2>(x + 1, s), kept = 0u;
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const uint32_t n = (word >> (4 * g)) & 15u;
    kept |= ((1u << (n & 3u)) | (1u << (n >> 2))) << (4 * g);
  }
  if (e == kMxBad) first = second = 0u;
  if (!live) kept = 0u;                                // (a short block's last groups have codes 0)
  uint8_t* c = out + (tile * stages + stage) * kMxChunkBytes;
  *reinterpret_cast<u32x2*>(c + ((b >> 1) * kMxRows + r) * 16 + (b & 1) * 8) = u32x2{first, second};
  *reinterpret_cast<uint32_t*>(c + kMxMaskAt + ((b >> 1) * kMxRows + r) * 8 + (b & 1) * 4) = kept;
  c[kMxScaleAt + r * 4 + b] = (uint8_t)e;
}

// go(first row, items) for groups of rows of fewer than 2^30 items.
template <typename Go>
hipError_t over_rows(int64_t T, int64_t K, int64_t per_row, const Go& go) {
  if (T == 0 || K == 0) return hipSuccess;
  const int64_t most = std::max<int64_t>(1, (int64_t(1) << 30) / per_row);
  for (int64_t t = 0; t < T; t += most) {
    go(t, Items(std::min(most, T - t), per_row));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}
template <typename In>
hipError_t quantize(const In* X, int64_t T, int64_t K, uint8_t* codes, uint8_t* exps, hipStream_t s) {
  return over_rows(T, K, mx_scale_bytes(K), [&](int64_t t, const Items& items) {
    const In* x = X + t * K;
    uint8_t *c = codes + t * mx_code_bytes(K), *e = exps + t * mx_scale_bytes(K);
    quantize_kernel<<<(unsigned)cdiv(items.count, kThreads), kThreads, 0, s>>>(x, items, (uint32_t)K, c, e);
  });
}
template <typename O>
hipError_t values(const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K, O* Y, hipStream_t s) {
  return over_rows(T, K, cdiv(K, 32) * (2 * sizeof(O)), [&](int64_t t, const Items& items) {
    const uint8_t *c = codes + t * mx_code_bytes(K), *e = exps + t * mx_scale_bytes(K);
    O* y = Y + t * K;
    values_kernel<<<(unsigned)cdiv(items.count, kPer * kThreads), kThreads, 0, s>>>(c, e, items, (uint32_t)K, y);
  });
}

}  // namespace

int64_t packed_sparse_mxfp4_bytes(int64_t rows, int64_t cols) {
  return cdiv(rows, kMxRows) * cdiv(cols, kMxCols) * kMxChunkBytes;
}

hipError_t launch_quantize_mxfp4(Dt dt, const void* X, int64_t T, int64_t K, uint8_t* codes, uint8_t* exps,
                                 hipStream_t s) {
  if (dt == Dt::BF16) return quantize((const uint16_t*)X, T, K, codes, exps, s);
  if (dt == Dt::F16) return quantize((const _Float16*)X, T, K, codes, exps, s);
  return quantize((const float*)X, T, K, codes, exps, s);
}

hipError_t launch_mxfp4_values(Dt out, const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K, void* Y,
                               hipStream_t s) {
  if (out == Dt::BF16) return values(codes, exps, T, K, (uint16_t*)Y, s);
  if (out == Dt::F16) return values(codes, exps, T, K, (_Float16*)Y, s);
  return values(codes, exps, T, K, (float*)Y, s);
}

hipError_t launch_pack_sparse_mxfp4(Dt dt, const void* values, const uint32_t* meta, int64_t M, int64_t K, void* packed,
                                    hipStream_t s) {
  if (M == 0 || K == 0) return hipSuccess;
  const int64_t stages = cdiv(K, kMxCols);
  const int64_t tiles = cdiv(M, kMxRows), most = (int64_t(1) << 23) / stages;   // of a launch: below 2^32 threads
  for (int64_t t = 0; t < tiles; t += most) {
    const unsigned blocks = (unsigned)(std::min(most, tiles - t) * stages);
    if (dt == Dt::F16)
      pack_kernel<<<blocks, kThreads, 0, s>>>((const _Float16*)values, meta, M, K, stages, t, (uint8_t*)packed);
    else
      pack_kernel<<<blocks, kThreads, 0, s>>>((const uint16_t*)values, meta, M, K, stages, t, (uint8_t*)packed);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace slope
