// The 2:4 sparse product on 4-bit floating point codes, Y[t][n] = sum over blocks of
// 2^(Ex + Ew) sum x w, on gfx950's v_mfma_scale_f32_32x32x64_f8f6f4.
//
// Lane layout of the instruction (checked against a host model): lane l's A operand is
// one block of 32 codes of row l%32, k 32*(l/32) .. +31, in four registers, and a
// scale byte; B likewise of column l%32; D as every 32x32 MFMA.  The sums of 144 and
// 576 steps were within 2e-7 of the exact ones (two-norm).  There is no sparse form of
// it: the weight travels as kept codes and positions (3.25 bits for a dense value) as
// far as a wave's registers, and is expanded there (17 operations for 32 values a
// lane, which the matrix instructions of other waves cover).
//
// A stage is 128 k, four blocks; MFMA step s of a stage takes blocks s (lanes 0..31)
// and 2 + s (lanes 32..63), so that a lane's two blocks are neighbours.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.h"
#include "dma.h"
#include "launch.h"
#include "mxfp4.h"
#include "mxfp4_plan.h"
#include "rows8.h"
#include "tile_map.h"

namespace slope {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

template <int S>
__device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 xa = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 xb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(xa, xb, c, 4, 4, S, (int)sa, S, (int)sb);
}

template <typename O>
__device__ __forceinline__ void store4(O* p, const float (&y)[4]) {
  if constexpr (sizeof(O) == 2) {
    u32x2 w;
    w[0] = out16_bits<O>(y[0]) | ((uint32_t)out16_bits<O>(y[1]) << 16);
    w[1] = out16_bits<O>(y[2]) | ((uint32_t)out16_bits<O>(y[3]) << 16);
    *reinterpret_cast<u32x2*>(p) = w;
  } else {
    *reinterpret_cast<f32x4*>(p) = f32x4{y[0], y[1], y[2], y[3]};
  }
}

template <typename O>
struct Args {
  const uint8_t *codes, *exps;
  const char* packed;
  int M, T, stages;
  O* Y;
  float* scratch;                                    // of the parts of a split call
  hipStream_t s;
};

// ---------------------------------------------------------------- few tokens
// T <= 64: the weight's stream from HBM is the cost.  A block owns 32 FM rows and all
// of K; its W waves take pairs of stages in turn, and their sums are added through LDS in
// a fixed order, so one launch makes the output and nothing is scratch, unless the call is
// split (below).  The weight
// goes straight from memory into registers.  X, which every block reads (from L2), comes
// as whole 128-byte lines, eight lanes a token, and passes through the wave's own piece
// of LDS.  Its scales come to LDS at the start, all of them: loaded pair by pair they
// would take a line for each token's 8 bytes, as many as the codes do (64 tokens, 20480 ->
// 5120: 26.7 us that way, 22.3 so; 36864 -> 9216: 54.8 and 48.2).
//
// A last odd stage's partner is past K: the weight's codes and scales are zero there
// (beyond the chunks), X's scales too (a row's are padded), and its codes are some codes
// or zero: their products are zero.
template <int FM>
struct DecodeA {
  u32x4 a[FM];
  u32x2 kept[FM];
  uint32_t s[FM];
};

// R loads of eight tokens bring a pair's X rows; D pairs are in flight.  No barrier in
// the loop, since no wave reads another's piece of LDS.  Lanes of columns t >= T read a
// row that is there (their sums are not stored).
//
// NT: a large weight's loads do not displace what the caches hold (decode_launch).
//
// SPLIT: blocks z take a part of K each, whole groups of four stages, and write their sums
// to Y + z T M.
template <int R, int FM, int D, int W, int WPS, bool SPLIT, bool NT, typename O>
__global__ __launch_bounds__(64 * W, WPS) void decode_mxfp4_kernel(const uint8_t* __restrict__ codes,
                                                                        const uint8_t* __restrict__ exps,
                                                                        const char* __restrict__ packed, int M, int T,
                                                                        int stages, O* __restrict__ Y) {
  constexpr int FT = R > 4 ? 2 : 1, XB = R * 1024;   // LDS bytes of a pair's X rows
  constexpr int AUX = NT ? 2 : 0;                    // the loads' cache policy: non-temporal
  constexpr int PER = kMxRows / (32 * FM);           // blocks a chunk
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, h = lane >> 5;
  const int64_t t0 = (int64_t)blockIdx.y * (8 * R);  // the block's tokens (all of them up to 64)
  const int groups = (stages + 3) / 4, z = SPLIT ? blockIdx.z : 0, parts = SPLIT ? gridDim.z : 1;
  const int g0 = SPLIT ? groups * z / parts : 0, span = SPLIT ? groups * (z + 1) / parts - g0 : groups;
  if constexpr (SPLIT) Y += (int64_t)z * T * M;
  const int row_c = stages * 64, row_s = (stages + 3) / 4 * 16;
  codes += t0 * row_c;
  exps += t0 * row_s;
  T = T - t0 < 8 * R ? (int)(T - t0) : 8 * R;
  const int64_t line = (int64_t)stages * kMxChunkBytes;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(packed + (blockIdx.x / PER) * line, line);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(codes, (int64_t)T * row_c);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(exps, (int64_t)T * row_s);
  uint32_t row[FM], x_src[R], t_at[FT];
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) row[fm] = (blockIdx.x % PER) * (32 * FM) + fm * 32 + (lane & 31);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int t = j * 8 + (lane >> 3);
    x_src[j] = (uint32_t)(t < T ? t : T - 1) * row_c + (lane & 7) * 16;
  }
#pragma unroll
  for (int ft = 0; ft < FT; ++ft) {
    const int t = ft * 32 + (lane & 31);
    t_at[ft] = t < T ? t : T - 1;
  }
  char* own = lds + wave * XB;
  const u32x2* scales = reinterpret_cast<const u32x2*>(lds + W * XB);
  struct Set {
    DecodeA<FM> a[2];
    u32x4 x[R];
  };
  const int p0 = 2 * g0, p1 = z + 1 < parts ? p0 + 2 * span : (stages + 1) / 2;   // the block's pairs
  const int last = 2 * p1 < stages ? 2 * p1 : stages;
  auto load_x = [&](Set& f, int pair) {
#pragma unroll
    for (int j = 0; j < R; ++j) f.x[j] = load16(rx, pair < p1 ? x_src[j] + pair * 128 : kOutOfRange);
  };
  auto load_a = [&](Set& f, int pair) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = 2 * pair + u;
      const uint32_t c = at < last ? (uint32_t)at * kMxChunkBytes : kOutOfRange;   // beyond: zero codes
#pragma unroll
      for (int fm = 0; fm < FM; ++fm) {
        f.a[u].a[fm] = __builtin_amdgcn_raw_buffer_load_b128(ra, c + (h * kMxRows + row[fm]) * 16, 0, AUX);
        f.a[u].kept[fm] = __builtin_bit_cast(
            u32x2, __builtin_amdgcn_raw_buffer_load_b64(ra, c + kMxMaskAt + (h * kMxRows + row[fm]) * 8, 0, AUX));
        f.a[u].s[fm] = __builtin_amdgcn_raw_buffer_load_b32(ra, c + kMxScaleAt + row[fm] * 4, 0, AUX);
      }
    }
  };
  f32x16 acc[FM][FT];
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int ft = 0; ft < FT; ++ft) acc[fm][ft] = f32x16{};
  auto step = [&](Set& f, int pair) {
    u32x2 sb[FT];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int t = j * 8 + (lane >> 3);
      *reinterpret_cast<u32x4*>(own + t * 128 + (((lane & 7) ^ ((t ^ (t >> 3)) & 7)) << 4)) = f.x[j];
    }
#pragma unroll
    for (int ft = 0; ft < FT; ++ft) {
      const u32x2 w = scales[(pair - p0) * (8 * R) + t_at[ft]];
      sb[ft] = u32x2{w[0] >> (16 * h), w[1] >> (16 * h)};
    }
    compiler_fence();                                // the wave's LDS operations run in order: no wait, no barrier
    load_x(f, pair + D * W);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      u32x4 b[FT][2];
#pragma unroll
      for (int ft = 0; ft < FT; ++ft)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tc = ft * 32 + (lane & 31), t = tc < 8 * R ? tc : 8 * R - 1;
          b[ft][i] = *reinterpret_cast<const u32x4*>(own + t * 128 + (((4 * u + 2 * h + i) ^ ((t ^ (t >> 3)) & 7)) << 4));
        }
#pragma unroll
      for (int fm = 0; fm < FM; ++fm) {
        const DecodeA<FM>& a = f.a[u];
        const uint32_t sa = a.s[fm] >> (16 * h);
        const u32x4 a0 = expand24(a.a[fm][0], a.a[fm][1], a.kept[fm][0]);
        const u32x4 a1 = expand24(a.a[fm][2], a.a[fm][3], a.kept[fm][1]);
#pragma unroll
        for (int ft = 0; ft < FT; ++ft) {
          acc[fm][ft] = mfma<0>(a0, b[ft][0], acc[fm][ft], sa, sb[ft][u]);
          acc[fm][ft] = mfma<1>(a1, b[ft][1], acc[fm][ft], sa, sb[ft][u]);
        }
      }
    }
    load_a(f, pair + D * W);
    compiler_fence();                                // the next step's writes stay behind these reads
  };
  Set f[D];
  // pair p0 + p's 8 bytes of token t at (p * 8R + t) * 8: reads without bank conflicts (rows of
  // a multiple of 256 bytes, as they come, would all lie in the same banks)
  const int all = T * span;
  for (int i0 = threadIdx.x; i0 < all; i0 += 4 * 64 * W) {
    u32x4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * 64 * W;
      v[j] = load16(rs, SPLIT ? i / span * row_s + (g0 + i % span) * 16 : i * 16);   // past the last row: zeros
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * 64 * W, t = i / span, c = i - t * span;
      u32x2* to = reinterpret_cast<u32x2*>(lds + W * XB) + 2 * c * (8 * R) + t;
      if (i < all) {
        to[0] = u32x2{v[j][0], v[j][1]};
        to[8 * R] = u32x2{v[j][2], v[j][3]};
      }
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load_x(f[d], p0 + wave + d * W);
    load_a(f[d], p0 + wave + d * W);
  }
  __syncthreads();                                   // (the first pairs are waited for next anyway)
  for (int p = p0 + wave; p < p1; p += D * W) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (p + d * W < p1) step(f[d], p + d * W);
  }
  // the waves' sums: the upper half of them hands its own to the lower half first
  constexpr int HALF = W / 2, ALL = FM * FT * 256;
  f32x4* sums = reinterpret_cast<f32x4*>(lds);
  __syncthreads();                                   // every wave is done with its X rows
  f32x4* mine = sums + (wave % HALF) * ALL + lane;
  auto part = [&](int f, int q) {
    const f32x16& v = acc[f / FT][f % FT];
    return f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
  };
  if (wave >= HALF) {
#pragma unroll
    for (int i = 0; i < FM * FT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) mine[(i * 4 + q) * 64] = part(i, q);
  }
  __syncthreads();
  if (wave < HALF) {
#pragma unroll
    for (int i = 0; i < FM * FT; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) mine[(i * 4 + q) * 64] += part(i, q);
  }
  __syncthreads();
  // group g = (fm, ft, q, lane): token ft*32 + lane%32, rows fm*32 + 8q + 4*(lane/32) .. +3
  for (int g = threadIdx.x; g < ALL; g += 64 * W) {
    const int i = g >> 8, fm = i / FT, ft = i % FT, q = (g >> 6) & 3, l = g & 63;
    const int t = ft * 32 + (l & 31);
    const int64_t m = ((int64_t)blockIdx.x * FM + fm) * 32 + 8 * q + 4 * (l >> 5);
    if (t >= T || m >= M) continue;
    f32x4 v = sums[g];
#pragma unroll
    for (int w = 1; w < HALF; ++w) v += sums[w * ALL + g];
    const float y[4] = {v[0], v[1], v[2], v[3]};
    store4<O>(Y + (t0 + t) * M + m, y);
  }
}

// A weight of at least 64 MB, read once by a call, is not expected in the 256 MB
// last-level cache at the next call, and its lines leave X's where they are.  us, from HBM and (a
// single weight, called again and again) from the cache, without NT / with it:
//   9216 -> 27648, 105 MB   1 token 20.5 / 18.8 and 17.2 / 17.5   64: 29.5 / 27.5 and 21.9 / 26.8
//   9216 -> 9216, 35 MB              9.9 /  9.1 and  7.3 /  7.7       16.1 / 14.9 and 12.2 / 13.5
constexpr int64_t kStreamBytes = int64_t(64) << 20;

template <int R, int FM, int D, int W, int WPS, bool SPLIT, typename O>
hipError_t decode_launch(const Args<O>& a, int parts) {
  constexpr int FT = R > 4 ? 2 : 1, SUMS = W * FM * FT * 2048;
  static_assert(W <= 8, "decode_lds");
  const int lds = std::max(W * R * 1024 + (int)cdiv(cdiv(a.stages, 4), parts) * 128 * R, SUMS);   // X rows and scales; sums
  auto go = [&](auto kern, LdsLimit& limit) {
    const hipError_t e = limit.set((const void*)kern, kLdsBytes);
    if (e != hipSuccess) return e;
    kern<<<dim3((unsigned)cdiv(a.M, 32 * FM), (unsigned)cdiv(a.T, 8 * R), parts), 64 * W, lds, a.s>>>(
        a.codes, a.exps, a.packed, a.M, a.T, a.stages, a.Y);
    return hipGetLastError();
  };
  static LdsLimit once, streams;
  if (a.T <= 8 * R && cdiv(a.M, kMxRows) * a.stages * kMxChunkBytes >= kStreamBytes)
    return go(decode_mxfp4_kernel<R, FM, D, W, WPS, SPLIT, true, O>, streams);
  return go(decode_mxfp4_kernel<R, FM, D, W, WPS, SPLIT, false, O>, once);
}
template <int R, int FM, int D, int W, int WPS, typename O>
hipError_t decode_go(const Args<O>& a) {
  return decode_launch<R, FM, D, W, WPS, false>(a, 1);
}

// The parts' sums added in order and rounded: n4 groups of four outputs.  All parts are
// loaded before the first sum.
template <typename O>
__global__ __launch_bounds__(256) void join_kernel(const f32x4* __restrict__ sums, int64_t n4, int parts,
                                                   O* __restrict__ Y) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  f32x4 part[kMostParts];
#pragma unroll
  for (int z = 0; z < kMostParts; ++z) part[z] = z < parts ? sums[z * n4 + i] : f32x4{};
  f32x4 v = part[0];
#pragma unroll
  for (int z = 1; z < kMostParts; ++z) v += part[z];
  const float y[4] = {v[0], v[1], v[2], v[3]};
  store4<O>(Y + 4 * i, y);
}
template <int R, int FM, int D, int W, int WPS, typename O>
hipError_t split_go(const Args<O>& a, int parts) {
  const Args<float> p{a.codes, a.exps, a.packed, a.M, a.T, a.stages, a.scratch, nullptr, a.s};
  const hipError_t e = decode_launch<R, FM, D, W, WPS, true>(p, parts);
  if (e != hipSuccess) return e;
  const int64_t n4 = (int64_t)a.T * a.M / 4;
  join_kernel<O><<<(unsigned)cdiv(n4, 256), 256, 0, a.s>>>((const f32x4*)a.scratch, n4, parts, a.Y);
  return hipGetLastError();
}

// ---------------------------------------------------------------- tiles
// Transposed output tiles Out^T = W . X^T of BM x BT, stages in a ring of LDS slots
// filled by buffer-to-LDS loads: the weight's chunks as they are (a fragment's reads
// are contiguous), X's rows of 64 bytes with granule c of row r at c ^ ((r>>2)&3).  X's
// scales come for four stages at a time, 16 bytes a row, into a ring of two.

// What a tile's block reads: the chunks of its rows, the rows of its tokens.
template <class G>
struct Sources {
  __amdgpu_buffer_rsrc_t a, b, s;
  int64_t m0, t0, line;
  int row_c, row_s;
  __device__ __forceinline__ Sources(const uint8_t* codes, const uint8_t* exps, const char* packed, int M, int T,
                                     int stages, int tm, int tt)
      : m0((int64_t)tm * G::BM), t0((int64_t)tt * G::BT), line((int64_t)stages * kMxChunkBytes) {
    row_c = stages * 64;
    row_s = (stages + 3) / 4 * 16;
    const int rows = (int)((T - t0) < G::BT ? (T - t0) : G::BT);
    const int64_t left = (M - m0 + kMxRows - 1) / kMxRows, chunks = left < G::BM / kMxRows ? left : G::BM / kMxRows;
    a = make_rsrc(packed + m0 / kMxRows * line, chunks * line);
    b = make_rsrc(codes + t0 * row_c, (int64_t)rows * row_c);
    s = make_rsrc(exps + t0 * row_s, (int64_t)rows * row_s);
  }
};

// The sums rounded and stored to Y[t][m].  A lane holds four rows m of one token; each
// wave turns 32 tokens at a time through its own piece of LDS (`lds` is free in all of the
// block by now) and stores whole lines.  M % 4 == 0.
template <class G, typename O>
__device__ __forceinline__ void store_tile(char* lds, const f32x16 (&acc)[G::FM][G::FT], O* __restrict__ Y, int M, int T,
                                           int64_t m0, int64_t t0, int lane, int wave) {
  constexpr int ROW = G::WM * (int)sizeof(O) + 16;   // a token's rows, padded against bank conflicts
  constexpr int PER = 16 / (int)sizeof(O), LANES = G::WM / PER, TOKENS = 64 / LANES;   // 16-byte pieces
  static_assert(G::WAVES * 32 * ROW <= G::LDS_BYTES, "the ring holds every wave's piece");
  char* own = lds + wave * (32 * ROW);
  const int64_t tw = t0 + wave / G::WGM * G::WT, mw = m0 + wave % G::WGM * G::WM;
  const int h4 = 4 * (lane >> 5);
  const int64_t m = mw + (lane % LANES) * PER;
#pragma unroll
  for (int ft = 0; ft < G::FT; ++ft) {
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float y[4] = {acc[fm][ft][4 * q], acc[fm][ft][4 * q + 1], acc[fm][ft][4 * q + 2], acc[fm][ft][4 * q + 3]};
        store4<O>(reinterpret_cast<O*>(own + (lane & 31) * ROW) + fm * 32 + 8 * q + h4, y);
      }
    compiler_fence();                                // (a wave's LDS operations run in order)
#pragma unroll
    for (int j = 0; j < 32; j += TOKENS) {
      const int row = j + lane / LANES;
      const int64_t t = tw + ft * 32 + row;
      const Pack<O, PER> y = *reinterpret_cast<const Pack<O, PER>*>(
          __builtin_assume_aligned(own + row * ROW + (lane % LANES) * 16, 16));
      if (t < T) {
        O* p = Y + t * M + m;
        if (m + PER <= M) {
          store_pack<O, PER>(p, y);
        } else if (m < M) {                          // 16-bit outputs, M % 8 == 4: the last four
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = y.v[i];
        }
      }
    }
    compiler_fence();
  }
}

template <class G>
__device__ __forceinline__ void clear_acc(f32x16 (&acc)[G::FM][G::FT]) {
#pragma unroll
  for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) acc[fm][ft] = f32x16{};
}

// ---------------------------------------------------------------- 128 x 64 tiles
// Several blocks a compute unit: while one waits for its stage, another multiplies.
// Four waves of 32 rows; one barrier a stage.
template <int BM_, int BT_, int WGM_, int WGT_, int NST_>
struct GeoS {
  static constexpr int BM = BM_, BT = BT_, WGM = WGM_, WGT = WGT_, WAVES = WGM * WGT, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WGM, WT = BT / WGT, FM = WM / 32, FT = WT / 32, NST = NST_;
  static constexpr int A_BYTES = BM / kMxRows * kMxChunkBytes, B_BYTES = BT * 64, S_BYTES = BT * 16;
  static constexpr int SLOT = A_BYTES + B_BYTES, LDS_BYTES = NST * SLOT + 2 * S_BYTES;
  // loads of a wave and stage: the weight's (four a chunk: 1, 1 and 1 KB, 256 bytes), X's (1
  // KB); with every fourth stage one of 64 rows' scales by the first S_WAVES waves
  static constexpr int A_DMA = BM / kMxRows * 4 / WAVES, B_DMA = B_BYTES / 1024 / WAVES, S_WAVES = BT / 64;
  static_assert(BM % kMxRows == 0 && A_DMA * WAVES == BM / kMxRows * 4 && B_DMA * WAVES * 1024 == B_BYTES &&
                S_WAVES <= WAVES && BT % 64 == 0, "tile and wave split");
  static_assert(NST <= 5, "a slot of scales is read before it is filled again (and one load of scales at most waited for)");
  static_assert(LDS_BYTES <= kLdsBytes, "LDS budget");
};

template <class G, typename O>
__global__ __launch_bounds__(G::THREADS, 1) void tiles_mxfp4_kernel(const uint8_t* __restrict__ codes,
                                                                    const uint8_t* __restrict__ exps,
                                                                    const char* __restrict__ packed, int M, int T,
                                                                    int stages, O* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % G::WGM, wt = wave / G::WGM, h = lane >> 5;
  int tm, tt;
  tile_of_block(blockIdx.x, gridDim.x, (M + G::BM - 1) / G::BM, (T + G::BT - 1) / G::BT, 8, tm, tt);
  const Sources<G> src(codes, exps, packed, M, T, stages, tm, tt);
  // The next stage's source offsets.  Past the last stage they lie in another chunk or
  // row, or beyond the resource; what they bring is not multiplied.
  uint32_t a_src[G::A_DMA], b_src[G::B_DMA], s_src = (uint32_t)(wave * 64 + lane) * src.row_s;
#pragma unroll
  for (int j = 0; j < G::A_DMA; ++j) {
    const int i = wave * G::A_DMA + j;               // load i % 4 of chunk i / 4
    a_src[j] = (uint32_t)((i / 4) * src.line) + (i % 4) * 1024 + lane * (i % 4 == 3 ? 4 : 16);
  }
#pragma unroll
  for (int j = 0; j < G::B_DMA; ++j) {
    const int row = (wave * G::B_DMA + j) * 16 + (lane >> 2);
    b_src[j] = (uint32_t)row * src.row_c + (((lane & 3) ^ ((row >> 2) & 3)) << 4);
  }
  int next = 0;                                      // the stage to load next
  auto issue = [&](int slot) {                       // this wave's share of it, into the slot at `slot`
#pragma unroll
    for (int j = 0; j < G::A_DMA; ++j) {
      const int i = wave * G::A_DMA + j;
      char* to = lds + slot + (i / 4) * kMxChunkBytes + (i % 4) * 1024;
      if (i % 4 == 3) dma4(src.a, to, a_src[j]);
      else dma16(src.a, to, a_src[j]);
      a_src[j] += kMxChunkBytes;
    }
    char* b = lds + slot + G::A_BYTES + wave * (G::B_DMA * 1024);
#pragma unroll
    for (int j = 0; j < G::B_DMA; ++j) {
      dma16(src.b, b + j * 1024, b_src[j]);
      b_src[j] += 64;
    }
    if (next % 4 == 0) {
      if (wave < G::S_WAVES) dma16(src.s, lds + G::NST * G::SLOT + (next / 4 % 2) * G::S_BYTES + wave * 1024, s_src);
      s_src += 16;
    }
    ++next;
  };
  // until this wave's share of all but its newest NST - 2 stages is in LDS
  auto wait_older = [&]() {
    constexpr int KEEP = G::NST - 2, N = KEEP * (G::A_DMA + G::B_DMA);
    if (wave < G::S_WAVES && ((next - 1) >> 2) != ((next - 1 - KEEP) >> 2)) wait_vmcnt<N + 1>();   // a load of scales among them
    else wait_vmcnt<N>();
  };
  f32x16 acc[G::FM][G::FT];
  clear_acc<G>(acc);
#pragma unroll
  for (int i = 0; i < G::NST - 1; ++i) issue(i * G::SLOT);
  int cur = 0, refill = (G::NST - 1) * G::SLOT;
  auto after = [](int slot) { return slot == (G::NST - 1) * G::SLOT ? 0 : slot + G::SLOT; };
  for (int s = 0; s < stages; ++s) {
    wait_older();
    barrier();                                       // the stage is there; every wave has read the one before
    compiler_fence();
    issue(refill);
    const char* base = lds + cur;
    const char* scales = lds + G::NST * G::SLOT + (s / 4 % 2) * G::S_BYTES + s % 4 * 4;
    u32x4 b[G::FT][2];
    uint32_t sb[G::FT];
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) {
      const int row = wt * G::WT + ft * 32 + (lane & 31);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        b[ft][i] = *reinterpret_cast<const u32x4*>(base + G::A_BYTES + row * 64 + (((2 * h + i) ^ ((row >> 2) & 3)) << 4));
      sb[ft] = *reinterpret_cast<const uint32_t*>(scales + row * 16) >> (16 * h);   // a lane's two bytes to the low half
    }
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
      const int row = wm * G::WM + fm * 32 + (lane & 31), at = h * kMxRows + row % kMxRows;
      const char* c = base + (row / kMxRows) * kMxChunkBytes;
      const u32x4 a = *reinterpret_cast<const u32x4*>(c + at * 16);
      const u32x2 kept = *reinterpret_cast<const u32x2*>(c + kMxMaskAt + at * 8);
      const uint32_t sa = *reinterpret_cast<const uint32_t*>(c + kMxScaleAt + (row % kMxRows) * 4) >> (16 * h);
      const u32x4 a0 = expand24(a[0], a[1], kept[0]), a1 = expand24(a[2], a[3], kept[1]);
#pragma unroll
      for (int ft = 0; ft < G::FT; ++ft) {
        acc[fm][ft] = mfma<0>(a0, b[ft][0], acc[fm][ft], sa, sb[ft]);
        acc[fm][ft] = mfma<1>(a1, b[ft][1], acc[fm][ft], sa, sb[ft]);
      }
    }
    wait_lgkmcnt0();
    cur = after(cur);
    refill = after(refill);
  }
  wait_vmcnt<0>();                                   // no load into the ring is left
  barrier();
  compiler_fence();
  store_tile<G>(lds, acc, Y, M, T, src.m0, src.t0, lane, wave);
}

// ---------------------------------------------------------------- woven tiles
// The large tiles.  A wave's stream of matrix instructions is woven with everything else:
// after each of them come an LDS read of what is multiplied one step later, a load into
// LDS, and a part of an expansion (17 operations for 32 values a lane).  In a block's order
// instead (read, expand, multiply) a stage of 256 x 256 took 2200 cycles of one block
// alone, 1024 of them products: every wave stood in the reads at once.  Woven it takes
// 1600.  One barrier a stage; a stage's reads of the weight run one stage ahead of its
// products and the loads three.
//
// Measured, 8192 x 9216 x 9216 bf16: 360 to 426 us a call with random kept positions, 350 to 392 with
// equal ones (the operands' bits are part of the power); by counters the matrix cores are busy
// 50 % of the time at 1.72 GHz, LDS 35 %.  Timing copies on one card, equal positions, where the whole
// took 335 to 347: products and barriers alone 250 to 270, without the loads 344 of 386, without the
// reads 331, without the products 248, without the expansion 338.  Two groups of four waves half a
// stage apart, one reading while the other multiplies: 336 to 358; four waves of 128 x 128: 373.
template <int BM_, int BT_, int WGM_, int WGT_, int NST_>
struct GeoW {
  static constexpr int BM = BM_, BT = BT_, WGM = WGM_, WGT = WGT_, WAVES = WGM * WGT, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WGM, WT = BT / WGT, FM = WM / 32, FT = WT / 32, NST = NST_;
  static constexpr int CHUNK = 4096;                 // of LDS: a chunk's 3328 bytes, and what the scales' load writes behind them
  static constexpr int A_BYTES = BM / kMxRows * CHUNK, B_BYTES = BT * 64, S_BYTES = BT * 16;
  static constexpr int SLOT = A_BYTES + B_BYTES, LDS_BYTES = NST * SLOT + 2 * S_BYTES;
  // 1 KB loads of a wave and stage, and with every fourth stage one of 64 rows' scales by
  // every wave (some rows by several)
  static constexpr int A_DMA = A_BYTES / 1024 / WAVES, B_DMA = B_BYTES / 1024 / WAVES, S_PARTS = BT / 64;
  static_assert(A_DMA * WAVES * 1024 == A_BYTES && B_DMA * WAVES * 1024 == B_BYTES && WAVES % S_PARTS == 0,
                "tile and wave split");
  static_assert(WM == kMxRows, "a wave has one chunk's rows");
  static_assert(NST >= 4 && NST <= 5, "a slot of scales is read before it is filled again (and one load of scales at most waited for)");
  static_assert(LDS_BYTES <= kLdsBytes, "LDS budget");
};

template <class G>
struct WovenA {                                      // a stage's weight operands, not expanded, and both sides' scales
  u32x4 a[G::FM];
  u32x2 kept[G::FM];
  uint32_t sa[G::FM], sb[G::FT];
};

// An anchor: the value is computed before the next side effect of the code (a load into LDS,
// a barrier), where it stands, not later where it is used.  In vector registers, or in
// accumulation registers for the accumulators of a block of four waves.
template <bool ACC = false, typename V>
__device__ __forceinline__ void anchor(V& v) {
  if constexpr (ACC) asm volatile("" : "+a"(v));
  else asm volatile("" : "+v"(v));
}

// 16 bytes from resource offset `off` + the wave's `base` to LDS.
__device__ __forceinline__ void dma16_at(__amdgpu_buffer_rsrc_t r, char* to, uint32_t off, int base) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)to, 16, off, base, 0, 0);
}

template <class G, typename O>
__device__ __forceinline__ void woven_tile(char* lds, const uint8_t* codes, const uint8_t* exps, const char* packed, int M,
                                           int T, int stages, int tm, int tt, O* __restrict__ Y) {
  constexpr int LOADS = G::A_DMA + G::B_DMA, NM = G::FM * G::FT;   // of a stage; products of a step
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave % G::WGM, wt = wave / G::WGM, h = lane >> 5, r = lane & 31;
  const Sources<G> src(codes, exps, packed, M, T, stages, tm, tt);
  uint32_t a_src[G::A_DMA], b_src[G::B_DMA];
#pragma unroll
  for (int j = 0; j < G::A_DMA; ++j) {
    const int i = wave * G::A_DMA + j;               // KB i % 4 of chunk i / 4; the last one has 256 bytes
    a_src[j] = i % 4 < 3 || lane < 16 ? (uint32_t)((i / 4) * src.line) + (i % 4) * 1024 + lane * 16 : kOutOfRange;
  }
#pragma unroll
  for (int j = 0; j < G::B_DMA; ++j) {
    const int row = (wave * G::B_DMA + j) * 16 + (lane >> 2);
    b_src[j] = (uint32_t)row * src.row_c + (((lane & 3) ^ ((row >> 2) & 3)) << 4);
  }
  const int s_part = wave % G::S_PARTS;
  const uint32_t s_src = (uint32_t)(s_part * 64 + lane) * src.row_s;
  auto issue_one = [&](int q, int slot, int at) {    // load q of stage `at`
    if (q < G::A_DMA)
      dma16_at(src.a, lds + slot + (wave * G::A_DMA + q) * 1024, a_src[q], at * kMxChunkBytes);
    else
      dma16_at(src.b, lds + slot + G::A_BYTES + (wave * G::B_DMA + q - G::A_DMA) * 1024, b_src[q - G::A_DMA], at * 64);
  };
  auto issue_scales = [&](int stage, int at) {       // those of four stages, with the first of them
    if (stage % 4 == 0)
      dma16_at(src.s, lds + G::NST * G::SLOT + (stage / 4 % 2) * G::S_BYTES + s_part * 1024, s_src, at / 4 * 16);
  };
  // Until this wave's share of all but its newest NST - 3 stages is in LDS, `next` stages being issued.
  auto wait_older = [&](int next) {
    constexpr int KEEP = G::NST - 3, N = KEEP * LOADS;
    if (((next - 1) >> 2) != ((next - 1 - KEEP) >> 2)) wait_vmcnt<N + 1>();   // a load of scales among them
    else wait_vmcnt<N>();
  };
  // fragment addresses within a slot; rows 32 fm and tokens 32 ft further on by constants
  const int a_at = wm * G::CHUNK, code_at = a_at + (h * kMxRows + r) * 16, mask_at = a_at + kMxMaskAt + (h * kMxRows + r) * 8,
            scale_at = a_at + kMxScaleAt + r * 4 + h * 2;
  const int row = wt * G::WT + r, swizzle = (row >> 2) & 3;
  const int b0_at = G::A_BYTES + row * 64 + (((2 * h) ^ swizzle) << 4), b1_at = G::A_BYTES + row * 64 + (((2 * h + 1) ^ swizzle) << 4);
  const int s_at = G::NST * G::SLOT + row * 16 + h * 2;

  f32x16 acc[G::FM][G::FT];
  clear_acc<G>(acc);
#pragma unroll
  for (int i = 0; i < G::NST - 1; ++i) {
    const int at = i < stages ? i : stages - 1;
#pragma unroll
    for (int q = 0; q < LOADS; ++q) issue_one(q, i * G::SLOT, at);
    issue_scales(i, at);
  }
  wait_older(G::NST - 1);                            // stages 0 and 1 are there
  barrier();
  compiler_fence();
  WovenA<G> now, then;
  u32x4 w0[G::FM], w1[G::FM], b0[G::FT], b1[G::FT], k[G::FM];
#pragma unroll
  for (int fm = 0; fm < G::FM; ++fm) {
    now.a[fm] = *reinterpret_cast<const u32x4*>(lds + code_at + fm * 512);
    now.kept[fm] = *reinterpret_cast<const u32x2*>(lds + mask_at + fm * 256);
    now.sa[fm] = *reinterpret_cast<const uint16_t*>(lds + scale_at + fm * 128);
    w0[fm] = expand24(now.a[fm][0], now.a[fm][1], now.kept[fm][0]);
  }
#pragma unroll
  for (int ft = 0; ft < G::FT; ++ft) {
    b0[ft] = *reinterpret_cast<const u32x4*>(lds + b0_at + ft * 2048);
    now.sb[ft] = *reinterpret_cast<const uint16_t*>(lds + s_at + ft * 512);
  }
  // Part i of 3 FM of expand24 of step `st` of f's operands into w.
  auto expand_part = [&](u32x4 (&w)[G::FM], const WovenA<G>& f, int st, int i) {
    const int fm = i / 3;
    const uint32_t kept = f.kept[fm][st], first = f.a[fm][2 * st], second = f.a[fm][2 * st + 1];
    if (i % 3 == 0) {
      k[fm][0] = wide_nibbles(kept & 0x11111111u);
      k[fm][1] = wide_nibbles((kept >> 1) & 0x11111111u);
    } else if (i % 3 == 1) {
      k[fm][2] = wide_nibbles((kept >> 2) & 0x11111111u);
      k[fm][3] = wide_nibbles((kept >> 3) & 0x11111111u);
    } else {
      w[fm] = expanded(first, second, k[fm]);
    }
  };
  int cur = 0, refill = (G::NST - 1) * G::SLOT;
  for (int s = 0; s < stages; ++s) {
    const int next = cur == (G::NST - 1) * G::SLOT ? 0 : cur + G::SLOT;
    const char* x = lds + (s_at + ((s + 1) / 4 % 2) * G::S_BYTES + (s + 1) % 4 * 4);   // the next stage's scales
    const int load = s + G::NST - 1, at = load < stages ? load : stages - 1;   // past the last stage: that one again, not multiplied
    issue_scales(load, at);
    // Step 0's products.  Between them: step 1's X and the next stage's weight are read, a stage to
    // come is loaded, step 1's weight is expanded.  (Past the last stage the reads bring an earlier
    // stage's bytes, not multiplied.)
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const int fm = i / G::FT, ft = i % G::FT;
      acc[fm][ft] = mfma<0>(w0[fm], b0[ft], acc[fm][ft], now.sa[fm], now.sb[ft]);
      anchor<(G::WAVES < 8)>(acc[fm][ft]);
      constexpr int READS = G::FT + 2 * G::FM;
#pragma unroll
      for (int q = 0; q < READS; ++q) {
        if (q * NM / READS != i) continue;
        if (q < G::FT) b1[q] = *reinterpret_cast<const u32x4*>(lds + (cur + b1_at) + q * 2048);
        else if ((q - G::FT) % 2 == 0) then.a[(q - G::FT) / 2] = *reinterpret_cast<const u32x4*>(lds + (next + code_at) + (q - G::FT) / 2 * 512);
        else then.kept[(q - G::FT) / 2] = *reinterpret_cast<const u32x2*>(lds + (next + mask_at) + (q - G::FT) / 2 * 256);
      }
#pragma unroll
      for (int q = 0; q < LOADS; ++q)
        if (q * NM / LOADS == i) issue_one(q, refill, at);
#pragma unroll
      for (int q = 0; q < 3 * G::FM; ++q)
        if (q * NM / (3 * G::FM) == i) expand_part(w1, now, 1, q);
      __builtin_amdgcn_sched_barrier(0);
    }
    // Step 1's products.  Between them: the next stage's X and scales are read, its step 0's weight is
    // expanded.
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      const int fm = i / G::FT, ft = i % G::FT;
      acc[fm][ft] = mfma<1>(w1[fm], b1[ft], acc[fm][ft], now.sa[fm], now.sb[ft]);
      anchor<(G::WAVES < 8)>(acc[fm][ft]);
      constexpr int READS = 2 * G::FT + G::FM;
#pragma unroll
      for (int q = 0; q < READS; ++q) {
        if (q * (NM - 2) / READS != i) continue;     // (all under way two products before the barrier)
        if (q < G::FT) b0[q] = *reinterpret_cast<const u32x4*>(lds + (next + b0_at) + q * 2048);
        else if (q < G::FT + G::FM) then.sa[q - G::FT] = *reinterpret_cast<const uint16_t*>(lds + (next + scale_at) + (q - G::FT) * 128);
        else then.sb[q - G::FT - G::FM] = *reinterpret_cast<const uint16_t*>(x + (q - G::FT - G::FM) * 512);
      }
#pragma unroll
      for (int q = 0; q < 3 * G::FM; ++q)
        if (q * NM / (3 * G::FM) == i) expand_part(w0, then, 0, q);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) anchor(w0[fm]);
    now = then;
    // This wave's reads of the stage's slot, which is filled next, are complete without a wait: their
    // values were operands of the products above, each of which is anchored before this.  What is still
    // under way comes from the next slot.
    compiler_fence();
    wait_older(load + 1);                            // the wave's share of stage s + 2 is there
    barrier();
    compiler_fence();
    refill = cur;
    cur = next;
  }
  wait_vmcnt<0>();                                   // no load into the ring is left
  barrier();
  compiler_fence();
  store_tile<G>(lds, acc, Y, M, T, src.m0, src.t0, lane, wave);
}

typedef GeoS<128, 64, 4, 1, 4> Mid;
typedef GeoW<256, 128, 4, 1, 5> Wide;                // four waves of 64 x 128
typedef GeoW<256, 256, 4, 2, 4> Full;                // eight waves of 64 x 128
typedef GeoW<256, 128, 4, 2, 4> Half;                // eight waves of 64 x 64
static_assert(Mid::BM == kMidRows && Mid::BT == kMidTokens, "many_plan");

template <typename O>
__global__ __launch_bounds__(Wide::THREADS, 1) void wide_mxfp4_kernel(const uint8_t* __restrict__ codes,
                                                                      const uint8_t* __restrict__ exps,
                                                                      const char* __restrict__ packed, int M, int T,
                                                                      int stages, O* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int tm, tt;
  tile_of_block(blockIdx.x, gridDim.x, (M + Wide::BM - 1) / Wide::BM, (T + Wide::BT - 1) / Wide::BT, 8, tm, tt);
  woven_tile<Wide, O>(lds, codes, exps, packed, M, T, stages, tm, tt, Y);
}

// The first rows_full row tiles in 256 x 256 tiles, the others in 256 x 128
// (full_width_rows: a grid that would end in a partly filled round of blocks
// ends sooner so; 8192 x 9216 x 9216 has 4.5 rounds of full tiles).
template <typename O>
__global__ __launch_bounds__(Full::THREADS, 2) void large_mxfp4_kernel(const uint8_t* __restrict__ codes,
                                                                       const uint8_t* __restrict__ exps,
                                                                       const char* __restrict__ packed, int M, int T,
                                                                       int stages, int rows_full, O* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int rows = (M + 255) / 256, full = (T + 255) / 256 * rows_full;
  int tm, tt;
  if ((int)blockIdx.x < full) {
    tile_of_block(blockIdx.x, full, rows_full, (T + 255) / 256, 8, tm, tt);
    woven_tile<Full, O>(lds, codes, exps, packed, M, T, stages, tm, tt, Y);
  } else {
    tile_of_block(blockIdx.x - full, gridDim.x - full, rows - rows_full, (T + 127) / 128, 8, tm, tt);
    woven_tile<Half, O>(lds, codes, exps, packed, M, T, stages, rows_full + tm, tt, Y);
  }
}

// device_compute_units, asked once for each device (1 us of a 5 us call).
int64_t compute_units() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kDevices) return device_compute_units();
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) known[dev].store(n = (int)device_compute_units(), std::memory_order_relaxed);
  return n;
}

template <typename O>
hipError_t mid_go(const Args<O>& a) {
  tiles_mxfp4_kernel<Mid, O><<<(unsigned)(cdiv(a.M, Mid::BM) * cdiv(a.T, Mid::BT)), Mid::THREADS, Mid::LDS_BYTES, a.s>>>(
      a.codes, a.exps, a.packed, a.M, a.T, a.stages, a.Y);
  return hipGetLastError();
}
static_assert(Mid::LDS_BYTES <= 64 * 1024, "no attribute needed");

template <typename O>
hipError_t wide_go(const Args<O>& a) {
  static LdsLimit limit;
  const hipError_t e = limit.set((const void*)wide_mxfp4_kernel<O>, Wide::LDS_BYTES);
  if (e != hipSuccess) return e;
  wide_mxfp4_kernel<O><<<(unsigned)(cdiv(a.M, Wide::BM) * cdiv(a.T, Wide::BT)), Wide::THREADS, Wide::LDS_BYTES, a.s>>>(
      a.codes, a.exps, a.packed, a.M, a.T, a.stages, a.Y);
  return hipGetLastError();
}

template <typename O>
hipError_t large_go(const Args<O>& a, int64_t rows_full) {
  static LdsLimit limit;
  const hipError_t e = limit.set((const void*)large_mxfp4_kernel<O>, Full::LDS_BYTES);
  if (e != hipSuccess) return e;
  const int64_t all = rows_full * cdiv(a.T, 256) + (cdiv(a.M, 256) - rows_full) * cdiv(a.T, 128);
  large_mxfp4_kernel<O><<<(unsigned)all, Full::THREADS, Full::LDS_BYTES, a.s>>>(a.codes, a.exps, a.packed, a.M, a.T,
                                                                                a.stages, (int)rows_full, a.Y);
  return hipGetLastError();
}

template <typename O>
hipError_t few_go(const Args<O>& a, const FewPlan& f) {
  if (f.parts > 1) {
    if (f.tokens == 8) return split_go<1, 2, 1, 8, 4, O>(a, f.parts);
    if (f.tokens == 16) return f.one ? split_go<2, 2, 1, 8, 4, O>(a, f.parts) : split_go<2, 2, 1, 4, 4, O>(a, f.parts);
    if (f.tokens == 32) return f.one ? split_go<4, 2, 1, 8, 4, O>(a, f.parts) : split_go<4, 2, 1, 4, 4, O>(a, f.parts);
    return f.one ? split_go<8, 2, 1, 8, 2, O>(a, f.parts) : split_go<8, 2, 1, 4, 2, O>(a, f.parts);
  }
  if (f.tokens == 8) {
    if (f.wide) return decode_go<1, 2, 1, 8, 4, O>(a);
    return f.one ? decode_go<1, 1, 2, 8, 4, O>(a) : decode_go<1, 1, 1, 8, 4, O>(a);
  }
  if (f.tokens == 16) {
    if (!f.wide) return decode_go<2, 1, 1, 8, 4, O>(a);
    return f.one ? decode_go<2, 2, 1, 8, 4, O>(a) : decode_go<2, 2, 1, 4, 4, O>(a);
  }
  if (f.tokens == 32) {
    if (!f.wide) return decode_go<4, 1, 1, 8, 4, O>(a);
    return f.one ? decode_go<4, 2, 1, 8, 4, O>(a) : decode_go<4, 2, 1, 4, 4, O>(a);
  }
  if (!f.wide) return decode_go<8, 1, 1, 8, 2, O>(a);
  return f.one ? decode_go<8, 2, 1, 8, 2, O>(a) : decode_go<8, 2, 1, 4, 2, O>(a);
}

// Any number of tokens.
template <typename O>
hipError_t spmm_launch(const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K, const void* packed, int64_t M,
                       void* Y, void* scratch, int64_t scratch_bytes, hipStream_t s) {
  const Args<O> a{codes, exps, (const char*)packed, (int)M, (int)T, (int)cdiv(K, kMxCols), (O*)Y, (float*)scratch, s};
  if (T <= 64) {
    const FewPlan plan = few_plan(T, M, a.stages, scratch ? most_parts(T, M, a.stages, scratch_bytes) : 1, compute_units());
    return plan.tokens ? few_go<O>(a, plan) : mid_go<O>(a);
  }
  const ManyPlan plan = many_plan(T, M, a.stages, compute_units());
  switch (plan.kernel) {
    case Many::Direct32: return decode_go<8, 1, 1, 8, 2, O>(a);
    case Many::Direct64: return decode_go<8, 2, 1, 4, 2, O>(a);
    case Many::Mid: return mid_go<O>(a);
    case Many::Wide: return wide_go<O>(a);
    default: return large_go<O>(a, plan.rows_full);
  }
}

}  // namespace

int64_t spmm_mxfp4_scratch_bytes(int64_t T, int64_t K, int64_t M) {
  if (T == 0 || T > 64 || K == 0 || M == 0) return 0;
  const int64_t stages = cdiv(K, kMxCols);
  const int parts = few_plan(T, M, stages, most_parts(T, M, stages, INT64_MAX), compute_units()).parts;
  return parts > 1 ? parts * 4 * T * M : 0;
}

hipError_t launch_spmm_mxfp4(Dt out, const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K, const void* packed,
                             int64_t M, void* Y, void* scratch, int64_t scratch_bytes, hipStream_t s) {
  if (T == 0 || M == 0) return hipSuccess;
  if (K == 0) return launch_fill_zero(out, Y, T * M, s);
  if (out == Dt::BF16) return spmm_launch<uint16_t>(codes, exps, T, K, packed, M, Y, scratch, scratch_bytes, s);
  if (out == Dt::F16) return spmm_launch<_Float16>(codes, exps, T, K, packed, M, Y, scratch, scratch_bytes, s);
  return spmm_launch<float>(codes, exps, T, K, packed, M, Y, scratch, scratch_bytes, s);
}

}  // namespace slope
