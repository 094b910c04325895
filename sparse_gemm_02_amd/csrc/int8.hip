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
// weight).  A block owns 32 rows and all of K; its waves take the stages in
// turn and read their operands straight from memory into registers, U stages'
// loads together.  The waves' int32 sums are added through LDS (exact in any
// order), so one launch makes the output and nothing is scratch.
constexpr int kDecodeWaves = 8, kDecodeStages = 4;

template <int FT, typename O>
__global__ __launch_bounds__(64 * kDecodeWaves) void decode_i8_kernel(const int8_t* __restrict__ Xq,
                                                                     const char* __restrict__ packed, int M, int T,
                                                                     int Kred, const float* __restrict__ x_scale,
                                                                     const float* __restrict__ w_scale,
                                                                     O* __restrict__ Y) {
  constexpr int W = kDecodeWaves, U = kDecodeStages;
  __shared__ i32x4 sums[W][FT][4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int stages = (Kred + kChunkCols - 1) / kChunkCols;
  const int tile = blockIdx.x >> 3, r = (int)(blockIdx.x & 7) * 32 + (lane & 31);
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(packed + (int64_t)tile * stages * kChunkBytes, (int64_t)stages * kChunkBytes);
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(Xq, (int64_t)T * Kred);
  uint32_t a_off[2], m_off[2], x_off[FT];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    a_off[ks] = r * 64 + (((2 * ks + (lane >> 5)) ^ ((r >> 2) & 3)) << 4);
    m_off[ks] = kChunkValueBytes + r * 16 + (2 * ks + (lane >> 5)) * 4;
  }
#pragma unroll
  for (int ft = 0; ft < FT; ++ft) {
    const int t = ft * 32 + (lane & 31);
    x_off[ft] = t < T ? (uint32_t)t * Kred + 16 * (lane >> 5) : kOutOfRange;
  }
  i32x16 acc[FT];
#pragma unroll
  for (int ft = 0; ft < FT; ++ft) acc[ft] = i32x16{};
  for (int sb = wave; sb < stages; sb += W * U) {
    i32x4 a[U][2], lo[U][2][FT], hi[U][2][FT];
    int ix[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = sb + u * W;
      const bool live = s < stages;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const uint32_t c = (uint32_t)s * kChunkBytes;
        a[u][ks] = __builtin_bit_cast(i32x4, load16(ra, live ? c + a_off[ks] : kOutOfRange));
        ix[u][ks] = (int)__builtin_amdgcn_raw_buffer_load_b32(ra, live ? c + m_off[ks] : kOutOfRange, 0, 0);
        const int k0 = s * kChunkCols + 64 * ks;     // K % 16 == 0: 16 codes inside or outside a row
        const bool in_lo = live && k0 + 16 * (lane >> 5) < Kred, in_hi = live && k0 + 32 + 16 * (lane >> 5) < Kred;
#pragma unroll
        for (int ft = 0; ft < FT; ++ft) {
          const bool ok = x_off[ft] != kOutOfRange;
          lo[u][ks][ft] = __builtin_bit_cast(i32x4, load16(rx, ok && in_lo ? x_off[ft] + k0 : kOutOfRange));
          hi[u][ks][ft] = __builtin_bit_cast(i32x4, load16(rx, ok && in_hi ? x_off[ft] + k0 + 32 : kOutOfRange));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int ft = 0; ft < FT; ++ft) {
          const i32x8 b = __builtin_shufflevector(lo[u][ks][ft], hi[u][ks][ft], 0, 1, 2, 3, 4, 5, 6, 7);
          acc[ft] = __builtin_amdgcn_smfmac_i32_32x32x64_i8(a[u][ks], b, acc[ft], ix[u][ks], 0, 0);
        }
  }
#pragma unroll
  for (int ft = 0; ft < FT; ++ft)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      sums[wave][ft][q][lane] = i32x4{acc[ft][4 * q], acc[ft][4 * q + 1], acc[ft][4 * q + 2], acc[ft][4 * q + 3]};
  __syncthreads();
  // group g = (ft, q, lane): token ft*32 + lane%32, rows 8q + 4*(lane/32) .. +3
  for (int g = threadIdx.x; g < FT * 4 * 64; g += 64 * W) {
    const int ft = g >> 8, q = (g >> 6) & 3, l = g & 63;
    const int t = ft * 32 + (l & 31);
    const int64_t m = (int64_t)tile * kChunkRows + (blockIdx.x & 7) * 32 + 8 * q + 4 * (l >> 5);
    if (t >= T || m >= M) continue;
    i32x4 v = sums[0][ft][q][l];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[w][ft][q][l];
    const float st = x_scale[t];
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = scaled(v[i], st, w_scale[m + i]);
    store4<O>(Y + (int64_t)t * M + m, y);
  }
}

template <typename O>
hipError_t decode_launch(const int8_t* Xq, const float* xs, int64_t T, int64_t K, const void* packed, const float* ws,
                         int64_t M, void* Y, hipStream_t s) {
  const unsigned blocks = (unsigned)cdiv(M, 32);
  if (T <= 32)
    decode_i8_kernel<1, O><<<blocks, 64 * kDecodeWaves, 0, s>>>(Xq, (const char*)packed, (int)M, (int)T, (int)K, xs,
                                                               ws, (O*)Y);
  else
    decode_i8_kernel<2, O><<<blocks, 64 * kDecodeWaves, 0, s>>>(Xq, (const char*)packed, (int)M, (int)T, (int)K, xs,
                                                               ws, (O*)Y);
  return hipGetLastError();
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
