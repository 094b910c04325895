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

// A thread makes a block of 32 values; what lies past K is zero.
template <typename In>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const In* __restrict__ X, int64_t T, int64_t K,
                                                            uint8_t* __restrict__ codes, uint8_t* __restrict__ exps) {
  const int64_t per_row = mx_scale_bytes(K), coded = mx_code_bytes(K) / 16;
  const int64_t all = T * per_row, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += stride) {
    const int64_t t = i / per_row, block = i - t * per_row, k = block * 32;
    In x[32];
    load_some<32>(X + t * K + (k < K ? k : 0), K - k, x);
    const uint32_t b = scale_byte(largest(x));
    const float s = scale_value(b);
    u32x4 w = {codes8<4>(x, s), codes8<4>(x + 1, s), codes8<4>(x + 2, s), codes8<4>(x + 3, s)};
    if (b == kMxBad) w = u32x4{0u, 0u, 0u, 0u};
    if (block < coded) *reinterpret_cast<u32x4*>(codes + (t * coded + block) * 16) = w;
    exps[i] = (uint8_t)b;
  }
}

// ---------------------------------------------------------------- values
// A thread makes eight values, a quarter of a block: byte q of each of its four words.
template <typename O>
__global__ __launch_bounds__(kThreads) void values_kernel(const uint8_t* __restrict__ codes,
                                                          const uint8_t* __restrict__ exps, int64_t T, int64_t K,
                                                          O* __restrict__ out) {
  const int64_t per_row = (K + 7) / 8, all = T * per_row, stride = (int64_t)gridDim.x * kThreads;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < all; i += stride) {
    const int64_t t = i / per_row, k = (i - t * per_row) * 8;
    const u32x4 w = *reinterpret_cast<const u32x4*>(codes + t * mx_code_bytes(K) + k / 32 * 16);
    const int shift = (int)(k & 24);                 // byte k / 8 % 4
    const uint32_t b = exps[t * mx_scale_bytes(K) + k / 32];
    const float s = b == kMxBad ? __builtin_nanf("") : scale_value(b);
    Pack<O, 8> y;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t two = w[p] >> shift;
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        // magnitudes 0, 1/2, 1, 3/2, 2, 3, 4, 6: the three bits are an exponent of bias 1 and one more bit
        const uint32_t c = two >> (4 * g);
        const float v = __uint_as_float(((c & 7u) << 22) | ((c & 8u) << 28)) * 0x1p126f;
        y.v[4 * g + p] = elem_of<O>(v * s);
      }
    }
    O* o = out + t * K + k;
    if (K - k >= 8) {
      store_pack<O, 8>(o, y);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < K) o[e] = y.v[e];
    }
  }
}

// ---------------------------------------------------------------- tile chunks
// A thread makes one row's block of 32 dense columns: 16 kept values, one metadata word.
template <typename In>
__global__ __launch_bounds__(kThreads) void pack_kernel(const In* __restrict__ vals, const uint32_t* __restrict__ meta,
                                                        int64_t M, int64_t K, int64_t stages, uint8_t* __restrict__ out) {
  const int64_t tile = blockIdx.x / stages, stage = blockIdx.x % stages;
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

unsigned grid_for(int64_t threads) { return (unsigned)std::min<int64_t>(cdiv(threads, kThreads), 256 * 64); }

}  // namespace

int64_t packed_sparse_mxfp4_bytes(int64_t rows, int64_t cols) {
  return cdiv(rows, kMxRows) * cdiv(cols, kMxCols) * kMxChunkBytes;
}

hipError_t launch_quantize_mxfp4(Dt dt, const void* X, int64_t T, int64_t K, uint8_t* codes, uint8_t* exps,
                                 hipStream_t s) {
  if (T == 0 || K == 0) return hipSuccess;
  const unsigned grid = grid_for(T * mx_scale_bytes(K));
  if (dt == Dt::BF16) quantize_kernel<<<grid, kThreads, 0, s>>>((const uint16_t*)X, T, K, codes, exps);
  else if (dt == Dt::F16) quantize_kernel<<<grid, kThreads, 0, s>>>((const _Float16*)X, T, K, codes, exps);
  else quantize_kernel<<<grid, kThreads, 0, s>>>((const float*)X, T, K, codes, exps);
  return hipGetLastError();
}

hipError_t launch_mxfp4_values(Dt out, const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K, void* Y,
                               hipStream_t s) {
  if (T == 0 || K == 0) return hipSuccess;
  const unsigned grid = grid_for(T * cdiv(K, 8));
  if (out == Dt::BF16) values_kernel<<<grid, kThreads, 0, s>>>(codes, exps, T, K, (uint16_t*)Y);
  else if (out == Dt::F16) values_kernel<<<grid, kThreads, 0, s>>>(codes, exps, T, K, (_Float16*)Y);
  else values_kernel<<<grid, kThreads, 0, s>>>(codes, exps, T, K, (float*)Y);
  return hipGetLastError();
}

hipError_t launch_pack_sparse_mxfp4(Dt dt, const void* values, const uint32_t* meta, int64_t M, int64_t K, void* packed,
                                    hipStream_t s) {
  if (M == 0 || K == 0) return hipSuccess;
  const int64_t stages = cdiv(K, kMxCols);
  const unsigned blocks = (unsigned)(cdiv(M, kMxRows) * stages);
  if (dt == Dt::F16)
    pack_kernel<<<blocks, kThreads, 0, s>>>((const _Float16*)values, meta, M, K, stages, (uint8_t*)packed);
  else
    pack_kernel<<<blocks, kThreads, 0, s>>>((const uint16_t*)values, meta, M, K, stages, (uint8_t*)packed);
  return hipGetLastError();
}

}  // namespace slope
