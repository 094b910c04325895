// 2:4 sparse products on 8-bit integer codes, Y[t][n] = (Xq . W_q^T) x_scale[t]
// w_scale[n], on gfx950's v_smfmac_i32_32x32x64_i8, and the packing of the
// weight's codes.
//
// Lane layout of the instruction (that of the E4M3 form, checked against a host
// model): lane l's A operand is the 16 kept codes of row l%32, dense k
// 32*(l/32) .. 32*(l/32)+31 of the 64-wide step, its index one stored metadata
// word; its B operand column l%32, k = 16*(l/32) + e and 32 + 16*(l/32) + e;
// D as every 32x32 MFMA.  Sums are exact in int32 for K <= 2^18.
#include "common.h"
#include "dma.h"
#include "gemm_tile.h"
#include "launch.h"
#include "rows8.h"
#include "tile_map.h"

namespace slope {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------- tile chunks
// int8 tile chunk (t, s): rows 256t .., dense columns 128s .., as the E4M3
// chunks: each row's 64 codes (granule c at c ^ ((row/4) % 4)), then each row's
// four metadata words.
constexpr int kChunkRows = 256, kChunkCols = 128;
constexpr int kChunkValueBytes = kChunkRows * 64, kChunkBytes = kChunkValueBytes + kChunkRows * 16;

// One block takes 32 rows of one row tile, eight lanes a row: a first walk over
// the rows' kept values for their largest magnitudes, a second (served by the
// caches) for the codes, written as chunk pieces.  Lane k of a row takes its
// compressed values 8k .. 8k+7 of each chunk and metadata word k.
template <typename In>
__global__ __launch_bounds__(256) void pack_i8_kernel(const In* __restrict__ vals, const uint32_t* __restrict__ meta,
                                                      int64_t M, int64_t K, int64_t stages, float* __restrict__ scale,
                                                      char* __restrict__ out) {
  const int k = threadIdx.x & 7, r = (int)(blockIdx.x & 7) * 32 + (threadIdx.x >> 3);
  const int64_t tile = blockIdx.x >> 3, row = tile * kChunkRows + r;
  const bool live = row < M;
  const int64_t half = K / 2, wpr = (K / 4 + 7) / 8;
  const In* v = vals + (live ? row : 0) * half;
  const uint32_t* m = meta + (live ? row : 0) * wpr;
  float am = 0.f;
  for (int64_t c = 8 * k; c < half; c += 64) {
    const Pack<In, 8> p = load_pack<In, 8>(v + c);
#pragma unroll
    for (int e = 0; e < 8; ++e) am = max_of(am, finite_or_inf(elem_f32(p.v[e])));
  }
#pragma unroll
  for (int x = 4; x >= 1; x >>= 1) am = max_of(am, __shfl_xor(am, x));
  const RowCodes<float> codes(am);
  if (live && k == 0) scale[row] = codes.scale();
  for (int64_t s = 0; s < stages; ++s) {
    char* chunk = out + (tile * stages + s) * kChunkBytes;
    const int64_t c0 = s * 64 + 8 * k, word = 4 * s + (k & 3);
    const Pack<In, 8> p = load_pack<In, 8>(v + (c0 < half ? c0 : 0));
    const uint32_t mw = m[word < wpr ? word : 0];
    u32x2 o = {0u, 0u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      o[e >> 2] |= ((uint32_t)codes.code(elem_f32(p.v[e])) & 0xFFu) << (8 * (e & 3));
    const bool ok = live && c0 < half;               // K % 16 == 0: all eight inside or outside
    if (!ok) o = u32x2{0u, 0u};
    *reinterpret_cast<u32x2*>(chunk + r * 64 + (((k >> 1) ^ ((r >> 2) & 3)) << 4) + 8 * (k & 1)) = o;
    if (k < 4)
      *reinterpret_cast<uint32_t*>(chunk + kChunkValueBytes + r * 16 + 4 * k) = (live && word < wpr) ? mw : 0u;
  }
}

// float of the exact sum times the product of the two scales, rounded to fp32
// (and then once more to the output format).  The compiler would fuse the
// product with a conversion to fp16 (one rounding where the definition has two);
// the empty asm keeps it a value of its own, so every kernel gives the same bits.
__device__ __forceinline__ float scaled(int acc, float st, float sn) {
  float y = (float)acc * (st * sn);
  asm("" : "+v"(y));
  return y;
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

// ---------------------------------------------------------------- the GEMM
// 256 x 256 transposed output tile Out^T = W_q . Xq^T, eight waves of 128 x 64,
// stages of 128 dense k in a ring of three LDS slots filled by buffer-to-LDS
// loads; one barrier a stage, the slot refilled among the second k step's
// MFMAs.  LDS granules: A row r c ^ ((r>>2)&3), B row r c ^ ((r^(r>>3))&7), so
// that fragment reads are free of bank conflicts.
struct GeoI8 {
  static constexpr int BM = 256, BT = 256, WGM = 2, WGT = 4, WAVES = 8, THREADS = 512;
  static constexpr int WM = BM / WGM, WT = BT / WGT, FM = WM / 32, FT = WT / 32;
  static constexpr int KS = 128, NST = 3;
  static constexpr int A_BYTES = BM * 64, B_BYTES = BT * 128, META_STAGE = BM * 16;
  static constexpr int CHUNK_BYTES = A_BYTES + META_STAGE;
  static constexpr int SLOT = A_BYTES + B_BYTES + META_STAGE, LDS_BYTES = NST * SLOT;
  static constexpr int A_DMA = A_BYTES / 1024 / WAVES, B_DMA = B_BYTES / 1024 / WAVES, M_DMA = META_STAGE / 256 / WAVES;
  static constexpr int DMA_PER_STAGE = A_DMA + B_DMA + M_DMA;
  static_assert(CHUNK_BYTES == kChunkBytes && A_BYTES == kChunkValueBytes, "chunks are the stage slices");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS budget");
};

template <typename O>
__global__ __launch_bounds__(GeoI8::THREADS, 1) void spmm_i8_kernel(const int8_t* __restrict__ Xq,
                                                                  const char* __restrict__ packed, int M, int T,
                                                                  int Kred, const float* __restrict__ x_scale,
                                                                  const float* __restrict__ w_scale,
                                                                  O* __restrict__ Y) {
  typedef GeoI8 G;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave % G::WGM, wt = wave / G::WGM;
  const int tiles_m = (M + G::BM - 1) / G::BM, tiles_t = (T + G::BT - 1) / G::BT;
  int tm, tt;
  tile_of_block(blockIdx.x, gridDim.x, tiles_m, tiles_t, 8, tm, tt);
  const int64_t m0 = (int64_t)tm * G::BM, t0 = (int64_t)tt * G::BT;
  const int stages = (Kred + G::KS - 1) / G::KS;
  const int rows_t = (int)((T - t0) < G::BT ? (T - t0) : G::BT);
  const __amdgpu_buffer_rsrc_t ra =
      make_rsrc(packed + (int64_t)tm * stages * G::CHUNK_BYTES, (int64_t)stages * G::CHUNK_BYTES);
  const __amdgpu_buffer_rsrc_t rb = make_rsrc(Xq + t0 * Kred, (int64_t)rows_t * Kred);

  uint32_t b_src[G::B_DMA];
  int b_k[G::B_DMA];
#pragma unroll
  for (int j = 0; j < G::B_DMA; ++j) {
    const int row = wave * (G::BT / G::WAVES) + j * 8 + (lane >> 3);
    const int c = (lane & 7) ^ ((row ^ (row >> 3)) & 7);
    b_src[j] = (uint32_t)row * Kred + c * 16;
    b_k[j] = c * 16;                                 // first k of the granule within the stage
  }
  auto issue = [&](int s) {
    char* base = lds + (s % G::NST) * G::SLOT;
    const uint32_t chunk = (uint32_t)s * G::CHUNK_BYTES;
    const bool live = s < stages;
#pragma unroll
    for (int j = 0; j < G::A_DMA; ++j) {
      const uint32_t part = wave * (G::A_BYTES / G::WAVES) + j * 1024;
      dma16(ra, base + part, live ? chunk + part + lane * 16 : kOutOfRange);
    }
#pragma unroll
    for (int j = 0; j < G::B_DMA; ++j) {
      const bool ok = live && s * G::KS + b_k[j] < Kred;
      dma16(rb, base + G::A_BYTES + wave * (G::B_BYTES / G::WAVES) + j * 1024, ok ? b_src[j] + s * G::KS : kOutOfRange);
    }
#pragma unroll
    for (int j = 0; j < G::M_DMA; ++j) {
      const uint32_t part = wave * (G::META_STAGE / G::WAVES) + j * 256;
      dma4(ra, base + G::A_BYTES + G::B_BYTES + part, live ? chunk + G::A_BYTES + part + lane * 4 : kOutOfRange);
    }
  };

  int a_off[2][G::FM], m_off[2][G::FM], b_off[2][G::FT][2];
#pragma unroll
  for (int fm = 0; fm < G::FM; ++fm) {
    const int row = wm * G::WM + fm * 32 + (lane & 31);
    const int sw = (row >> 2) & 3;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      a_off[ks][fm] = row * 64 + (((2 * ks + (lane >> 5)) ^ sw) * 16);
      m_off[ks][fm] = G::A_BYTES + G::B_BYTES + row * 16 + (2 * ks + (lane >> 5)) * 4;
    }
  }
#pragma unroll
  for (int ft = 0; ft < G::FT; ++ft) {
    const int row = wt * G::WT + ft * 32 + (lane & 31);
    const int sw = (row ^ (row >> 3)) & 7;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      b_off[ks][ft][0] = G::A_BYTES + row * 128 + (((4 * ks + (lane >> 5)) ^ sw) * 16);
      b_off[ks][ft][1] = G::A_BYTES + row * 128 + (((4 * ks + 2 + (lane >> 5)) ^ sw) * 16);
    }
  }
  struct Frags {
    i32x4 a[G::FM];
    int ix[G::FM];
    i32x8 b[G::FT];
  };
  auto read_frags = [&](Frags& f, int s, int ks) {
    const char* base = lds + (s % G::NST) * G::SLOT;
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
      f.a[fm] = *reinterpret_cast<const i32x4*>(base + a_off[ks][fm]);
      f.ix[fm] = *reinterpret_cast<const int*>(base + m_off[ks][fm]);
    }
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(base + b_off[ks][ft][0]);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(base + b_off[ks][ft][1]);
      f.b[ft] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  };
  i32x16 acc[G::FM][G::FT];
#pragma unroll
  for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) acc[fm][ft] = i32x16{};
  auto mma_col = [&](const Frags& f, int ft) {
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm)
      acc[fm][ft] = __builtin_amdgcn_smfmac_i32_32x32x64_i8(f.a[fm], f.b[ft], acc[fm][ft], f.ix[fm], 0, 0);
  };
  auto mma = [&](const Frags& f) {
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) mma_col(f, ft);
  };

#pragma unroll
  for (int p = 0; p < G::NST; ++p) issue(p);
  wait_vmcnt<G::DMA_PER_STAGE * (G::NST - 1)>();
  barrier();
  compiler_fence();
  Frags f0, f1;
  read_frags(f0, 0, 0);
  for (int s = 0; s < stages; ++s) {
    read_frags(f1, s, 1);
    mma(f0);
    __builtin_amdgcn_sched_barrier(0);
    wait_lgkmcnt0();
    wait_vmcnt<G::DMA_PER_STAGE * (G::NST - 2)>();
    barrier();
    if (s + 1 < stages) read_frags(f0, s + 1, 0);
    mma_col(f1, 0);
    __builtin_amdgcn_sched_barrier(0);
    issue(s + G::NST);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ft = 1; ft < G::FT; ++ft) mma_col(f1, ft);
  }
  wait_vmcnt<0>();
#pragma unroll
  for (int ft = 0; ft < G::FT; ++ft) {
    const int64_t t = t0 + wt * G::WT + ft * 32 + (lane & 31);
    if (t >= T) continue;
    const float st = x_scale[t];
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t m = m0 + wm * G::WM + fm * 32 + 8 * q + 4 * (lane >> 5);
        if (m >= M) continue;                        // M % 4 == 0: all four inside or outside
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = scaled(acc[fm][ft][4 * q + i], st, w_scale[m + i]);
        store4<O>(Y + t * M + m, y);
      }
    }
  }
}

template <typename O>
hipError_t spmm_launch(const int8_t* Xq, const float* xs, int64_t T, int64_t K, const void* packed, const float* ws,
                       int64_t M, void* Y, hipStream_t s) {
  typedef GeoI8 G;
  const int64_t nb = cdiv(M, G::BM) * cdiv(T, G::BT);
  auto kern = spmm_i8_kernel<O>;
  static LdsLimit limit;
  const hipError_t e = limit.set((const void*)kern, G::LDS_BYTES);
  if (e != hipSuccess) return e;
  kern<<<(unsigned)nb, G::THREADS, G::LDS_BYTES, s>>>(Xq, (const char*)packed, (int)M, (int)T, (int)K, xs, ws, (O*)Y);
  return hipGetLastError();
}

// ---------------------------------------------------------------- few tokens
// T <= 64: the weight's stream from HBM is the cost (0.625 bytes per dense
// weight).  A block owns 32 FM rows and all of K; its W waves take the stages
// in turn, and their int32 sums are added through LDS (exact in any order), so
// one launch makes the output and nothing is scratch.  The weight goes straight
// from memory into registers; X (which every block reads, from L2) comes as
// whole 128-byte lines, eight lanes a token, and passes through the wave's own
// piece of LDS, for a wave that loads its fragments from memory touches 32
// lines with every load (64 tokens, 20480 -> 5120: 46 us that way, 23 so).
//
// Within a stage of 128 k the MFMA steps are not the stage's halves: step s
// takes metadata words s (lanes 0..31) and 2 + s (lanes 32..63), so that a lane
// needs two neighbouring words (one 8-byte load) and two neighbouring granules.
// Its B operand is then k 32s + 16h .. and 64 + 32s + 16h .. (h = lane / 32).
//
// Measured (bf16 out; floor: the weight at a copy's 5.13 TB/s): 9216 -> 27648 at
// 1 / 16 / 64 tokens 31.2 / 34.1 / 44.9 us (floor 31.0), 9216 -> 9216 11.1 /
// 11.8 / 16.4 (10.3), 5120 -> 15360 10.4 / 10.7 / 12.6 (9.6), 20480 -> 5120 12.6
// / 14.4 / 23.2 (12.8), 36864 -> 9216 42.3 / 50.8 / 74.4 (41.4).  At one token
// HBM bounds it; at 64 the L1s, through which every block draws all of X.
template <int FM>
struct DecodeA {
  i32x4 a[FM][2];
  u32x2 ix[FM];
};

// The weight of the block's 32 FM rows, stage by stage.
template <int FM>
struct DecodeIn {
  __amdgpu_buffer_rsrc_t ra;
  uint32_t a_off[FM][2], m_off[FM];
  int stages;
  __device__ __forceinline__ DecodeIn(const char* packed, int Kred, int lane) {
    constexpr int PER = kChunkRows / (32 * FM);      // blocks a row tile
    stages = (Kred + kChunkCols - 1) / kChunkCols;
    const int tile = blockIdx.x / PER, h = lane >> 5;
    ra = make_rsrc(packed + (int64_t)tile * stages * kChunkBytes, (int64_t)stages * kChunkBytes);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int r = (int)(blockIdx.x % PER) * 32 * FM + fm * 32 + (lane & 31);
#pragma unroll
      for (int s = 0; s < 2; ++s) a_off[fm][s] = r * 64 + (((2 * h + s) ^ ((r >> 2) & 3)) << 4);
      m_off[fm] = kChunkValueBytes + r * 16 + h * 8;
    }
  }
  __device__ __forceinline__ void load(DecodeA<FM>& d, int s) const {
    const uint32_t c = s < stages ? (uint32_t)s * kChunkBytes : kOutOfRange;   // beyond: zero codes
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
#pragma unroll
      for (int i = 0; i < 2; ++i) d.a[fm][i] = __builtin_bit_cast(i32x4, load16(ra, c + a_off[fm][i]));
      d.ix[fm] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(ra, c + m_off[fm], 0, 0));
    }
  }
};

// The block's sums over its W waves (through `lds`, W / 2 * FM * FT * 4 KB: the
// upper half of the waves hands its sums to the lower half first), scaled and
// stored.  Columns t >= T are not.
template <int W, int FM, int FT, typename O>
__device__ __forceinline__ void decode_store(char* lds, const i32x16 (&acc)[FM][FT], int M, int T,
                                             const float* __restrict__ x_scale, const float* __restrict__ w_scale,
                                             O* __restrict__ Y) {
  constexpr int HALF = W / 2, ALL = FM * FT * 256;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  i32x4* sums = reinterpret_cast<i32x4*>(lds);
  __syncthreads();                                   // every wave is done with its X rows
  i32x4* mine = sums + (wave % HALF) * ALL + lane;
  if (wave >= HALF) {
#pragma unroll
    for (int f = 0; f < FM * FT; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x16& v = acc[f / FT][f % FT];
        mine[(f * 4 + q) * 64] = i32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
  }
  __syncthreads();
  if (wave < HALF) {
#pragma unroll
    for (int f = 0; f < FM * FT; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const i32x16& v = acc[f / FT][f % FT];
        mine[(f * 4 + q) * 64] += i32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
  }
  __syncthreads();
  // group g = (fm, ft, q, lane): token ft*32 + lane%32, rows fm*32 + 8q + 4*(lane/32) .. +3
  for (int g = threadIdx.x; g < ALL; g += 64 * W) {
    const int f = g >> 8, fm = f / FT, ft = f % FT, q = (g >> 6) & 3, l = g & 63;
    const int t = ft * 32 + (l & 31);
    const int64_t m = ((int64_t)blockIdx.x * FM + fm) * 32 + 8 * q + 4 * (l >> 5);
    if (t >= T || m >= M) continue;
    i32x4 v = sums[g];
#pragma unroll
    for (int w = 1; w < HALF; ++w) v += sums[w * ALL + g];
    const float st = x_scale[t];
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = scaled(v[i], st, w_scale[m + i]);
    store4<O>(Y + (int64_t)t * M + m, y);
  }
}

// R loads of eight tokens bring a stage's X rows; D sets of G stages are in
// flight.  No barrier in the loop, since no wave reads another's piece of LDS.
// Lanes of columns t >= T read a row that is there (their sums are not stored).
template <int R, int FM, int G, int D, int W, int WPS, typename O>
__global__ __launch_bounds__(64 * W, WPS) void decode_i8_kernel(const int8_t* __restrict__ Xq,
                                                                     const char* __restrict__ packed, int M, int T,
                                                                     int Kred, const float* __restrict__ x_scale,
                                                                     const float* __restrict__ w_scale,
                                                                     O* __restrict__ Y) {
  constexpr int FT = R > 4 ? 2 : 1, XB = R * 1024;   // LDS bytes of a stage's X rows
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const DecodeIn<FM> in(packed, Kred, lane);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(Xq, (int64_t)T * Kred);
  char* own = lds + wave * (G * XB);
  uint32_t x_src[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int t = j * 8 + (lane >> 3);
    x_src[j] = (uint32_t)(t < T ? t : T - 1) * Kred;
  }
  const int c16 = (lane & 7) * 16;                   // this lane's granule of a row's 128 bytes
  struct Set {
    DecodeA<FM> a[G];
    u32x4 x[G][R];
  };
  auto load_x = [&](Set& f, int s) {
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const int k = (s + u * W) * kChunkCols + c16;  // K % 16 == 0: a granule is inside or outside a row
#pragma unroll
      for (int j = 0; j < R; ++j) f.x[u][j] = load16(rx, k < Kred ? x_src[j] + k : kOutOfRange);
    }
  };
  auto load_a = [&](Set& f, int s) {
#pragma unroll
    for (int u = 0; u < G; ++u) in.load(f.a[u], s + u * W);
  };
  i32x16 acc[FM][FT];
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int ft = 0; ft < FT; ++ft) acc[fm][ft] = i32x16{};
  auto step = [&](Set& f, int s) {
#pragma unroll
    for (int u = 0; u < G; ++u)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int t = j * 8 + (lane >> 3);
        *reinterpret_cast<u32x4*>(own + u * XB + t * 128 + (((lane & 7) ^ ((t ^ (t >> 3)) & 7)) << 4)) = f.x[u][j];
      }
    compiler_fence();                                // the wave's LDS operations run in order: no wait, no barrier
    load_x(f, s + D * G * W);
#pragma unroll
    for (int u = 0; u < G; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int ft = 0; ft < FT; ++ft) {
          const int t0 = ft * 32 + (lane & 31), t = t0 < 8 * R ? t0 : 8 * R - 1;
          const int sw = (t ^ (t >> 3)) & 7, c = 2 * i + (lane >> 5);
          const char* row = own + u * XB + t * 128;
          const i32x4 lo = *reinterpret_cast<const i32x4*>(row + ((c ^ sw) << 4));
          const i32x4 hi = *reinterpret_cast<const i32x4*>(row + (((c + 4) ^ sw) << 4));
          const i32x8 b = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int fm = 0; fm < FM; ++fm)
            acc[fm][ft] = __builtin_amdgcn_smfmac_i32_32x32x64_i8(f.a[u].a[fm][i], b, acc[fm][ft],
                                                                  (int)f.a[u].ix[fm][i], 0, 0);
        }
    load_a(f, s + D * G * W);
    compiler_fence();                                // the next step's writes stay behind these reads
  };
  Set f[D];
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load_x(f[d], wave + d * G * W);
    load_a(f[d], wave + d * G * W);
  }
  for (int s = wave; s < in.stages; s += D * G * W) {
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (s + d * G * W < in.stages) step(f[d], s + d * G * W);
  }
  decode_store<W, FM, FT, O>(lds, acc, M, T, x_scale, w_scale, Y);
}

template <typename O>
struct DecodeArgs {
  const int8_t* Xq;
  const char* packed;
  int M, T, K;
  const float *xs, *ws;
  O* Y;
  hipStream_t s;
};
template <int R, int FM, int G, int D, int W, int WPS, typename O>
hipError_t decode_go(const DecodeArgs<O>& a) {
  constexpr int FT = R > 4 ? 2 : 1;
  constexpr int LDS = W * (G * R * 1024 > FM * FT * 2048 ? G * R * 1024 : FM * FT * 2048);   // X rows; sums
  static LdsLimit limit;
  auto kern = decode_i8_kernel<R, FM, G, D, W, WPS, O>;
  const hipError_t e = limit.set((const void*)kern, LDS);
  if (e != hipSuccess) return e;
  kern<<<(unsigned)cdiv(a.M, 32 * FM), 64 * W, LDS, a.s>>>(a.Xq, a.packed, a.M, a.T, a.K, a.xs, a.ws, a.Y);
  return hipGetLastError();
}

// 64 rows a block where that leaves 128 blocks or more (9216 outputs, 9216 wide,
// 32 tokens: 11.9 us against 16.4 with 32 rows): every block draws all of X, so
// wider ones draw it less often.  Below, 64 rows would leave too many compute
// units idle (5120 outputs, 20480 wide, 32 tokens: 20.4 us against 16.6).
// Waves, stages and sets as measured best over the five shapes above: the
// registers are kept to 128 (two blocks a compute unit) up to 32 tokens; at 64
// the 64-row block needs more, and four waves beat eight (44.9 against 46.8 us).
template <typename O>
hipError_t decode_launch(const int8_t* Xq, const float* xs, int64_t T, int64_t K, const void* packed, const float* ws,
                         int64_t M, void* Y, hipStream_t s) {
  const DecodeArgs<O> a{Xq, (const char*)packed, (int)M, (int)T, (int)K, xs, ws, (O*)Y, s};
  const bool wide = M > 127 * 64;
  if (T <= 8) return wide ? decode_go<1, 2, 1, 2, 8, 4, O>(a) : decode_go<1, 1, 2, 2, 8, 4, O>(a);
  if (T <= 16) return wide ? decode_go<2, 2, 1, 2, 8, 4, O>(a) : decode_go<2, 1, 1, 2, 16, 4, O>(a);
  if (T <= 32) return wide ? decode_go<4, 2, 1, 1, 8, 4, O>(a) : decode_go<4, 1, 1, 2, 8, 4, O>(a);
  return wide ? decode_go<8, 2, 1, 1, 4, 2, O>(a) : decode_go<8, 1, 1, 1, 8, 4, O>(a);
}

}  // namespace

int64_t packed_sparse_i8_bytes(int64_t rows, int64_t cols) {
  return cdiv(rows, kChunkRows) * cdiv(cols, kChunkCols) * kChunkBytes;
}

hipError_t launch_pack_sparse_i8(Dt dt, const void* values, const uint32_t* meta, int64_t M, int64_t K, float* scale,
                                 void* packed, hipStream_t s) {
  if (M == 0) return hipSuccess;
  const int64_t stages = cdiv(K, kChunkCols);
  const unsigned blocks = (unsigned)(cdiv(M, kChunkRows) * (kChunkRows / 32));
  if (dt == Dt::F16)
    pack_i8_kernel<_Float16><<<blocks, 256, 0, s>>>((const _Float16*)values, meta, M, K, stages, scale, (char*)packed);
  else
    pack_i8_kernel<uint16_t><<<blocks, 256, 0, s>>>((const uint16_t*)values, meta, M, K, stages, scale, (char*)packed);
  return hipGetLastError();
}

hipError_t launch_spmm_i8(Dt out, const int8_t* Xq, const float* x_scale, int64_t T, int64_t K, const void* packed,
                          const float* w_scale, int64_t M, void* Y, hipStream_t s) {
  if (T == 0 || M == 0) return hipSuccess;
  if (out == Dt::BF16) return spmm_launch<uint16_t>(Xq, x_scale, T, K, packed, w_scale, M, Y, s);
  if (out == Dt::F16) return spmm_launch<_Float16>(Xq, x_scale, T, K, packed, w_scale, M, Y, s);
  return spmm_launch<float>(Xq, x_scale, T, K, packed, w_scale, M, Y, s);
}

hipError_t launch_spmm_i8_decode(Dt out, const int8_t* Xq, const float* x_scale, int64_t T, int64_t K,
                                 const void* packed, const float* w_scale, int64_t M, void* Y, hipStream_t s) {
  if (T == 0 || M == 0) return hipSuccess;
  if (out == Dt::BF16) return decode_launch<uint16_t>(Xq, x_scale, T, K, packed, w_scale, M, Y, s);
  if (out == Dt::F16) return decode_launch<_Float16>(Xq, x_scale, T, K, packed, w_scale, M, Y, s);
  return decode_launch<float>(Xq, x_scale, T, K, packed, w_scale, M, Y, s);
}

}  // namespace slope
