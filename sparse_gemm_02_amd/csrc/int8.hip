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
// compressed values 8k .. 8k+7 of each chunk and metadata word k.  Made once for a
// weight: 27648 x 9216 165 to 182 us (2.5 to 2.7 TB/s of 1.125 bytes in and 0.625
// out, the first walk's latency and the second walk's).
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
  uint32_t am = 0u;
  for (int64_t c = 8 * k; c < half; c += 64) {
    const Pack<In, 8> p = load_pack<In, 8>(v + c);
#pragma unroll
    for (int e = 0; e < 8; ++e) am = max_bits(am, mag_bits(elem_f32(p.v[e])));
  }
#pragma unroll
  for (int x = 4; x >= 1; x >>= 1) am = max_bits(am, (uint32_t)__shfl_xor((int)am, x));
  const RowCodes codes(am, (double)__uint_as_float(am));
  if (live && k == 0) scale[row] = codes.scale(1.0f);
  for (int64_t s = 0; s < stages; ++s) {
    char* chunk = out + (tile * stages + s) * kChunkBytes;
    const int64_t c0 = s * 64 + 8 * k, word = 4 * s + (k & 3);
    const Pack<In, 8> p = load_pack<In, 8>(v + (c0 < half ? c0 : 0));
    const uint32_t mw = m[word < wpr ? word : 0];
    u32x2 o = {0u, 0u};
    if (codes.tiny) {                                // (and rows of zeros)
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e >> 2] |= ((uint32_t)codes.code(elem_f32(p.v[e])) & 0xFFu) << (8 * (e & 3));
    } else if (!codes.bad) {
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const float f[4] = {elem_f32(p.v[4 * w]), elem_f32(p.v[4 * w + 1]), elem_f32(p.v[4 * w + 2]), elem_f32(p.v[4 * w + 3])};
        o[w] = codes.four(f, [&](int i) { return (double)f[i]; });
      }
    }
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
// Transposed output tiles Out^T = W_q . Xq^T of BM x BT, stages of 128 dense k in
// a ring of LDS slots (three or four) filled by buffer-to-LDS loads of 16 bytes a lane.
// LDS granules: A row r c ^ ((r>>2)&3), B row r c ^ ((r^(r>>3))&7), so that
// fragment reads are free of bank conflicts (the metadata's reads use half of the
// banks; laid out over all of them they changed no time).  MFMA step s of a stage takes
// granules 2h + s of A, words 2h + s of its metadata, and granules 2s + h and 4 +
// 2s + h of B (h = lane / 32; the few-token kernel below says why).
//
// Every source and LDS address is kept and stepped (one add a load and stage):
// with offsets, ring slots and bounds computed anew each stage the same schedule
// took 436 us for 8192 x 9216 x 9216, against 389 (and less since tiles are stored
// by whole lines: below).
template <int BM_, int BT_, int WGM_, int WGT_, int BLOCKS_, int NST_ = 3>
struct GeoI8 {
  static constexpr int BM = BM_, BT = BT_, WGM = WGM_, WGT = WGT_, WAVES = WGM * WGT, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WGM, WT = BT / WGT, FM = WM / 32, FT = WT / 32;
  static constexpr int KS = kChunkCols, NST = NST_;   // slots of the ring
  static constexpr int BLOCKS = BLOCKS_;             // blocks a compute unit holds
  static constexpr int A_BYTES = BM * 64, B_BYTES = BT * 128, META_BYTES = BM * 16;
  static constexpr int SLOT = A_BYTES + B_BYTES + META_BYTES, LDS_BYTES = NST * SLOT;
  // 1 KB loads of a wave and stage; the metadata's go to the first META_WAVES waves
  static constexpr int A_DMA = A_BYTES / 1024 / WAVES, B_DMA = B_BYTES / 1024 / WAVES, META_WAVES = META_BYTES / 1024;
  static constexpr int PER_CHUNK = kChunkRows / BM;  // tiles in a chunk's rows
  static_assert(kChunkRows % BM == 0 && A_BYTES % (1024 * WAVES) == 0 && B_BYTES % (1024 * WAVES) == 0 &&
                META_BYTES % 1024 == 0 && META_WAVES <= WAVES, "tile and wave split");
  static_assert(BLOCKS * LDS_BYTES <= 160 * 1024, "LDS budget");
};

template <class G>
struct FragsI8 {                                     // one step's operands
  i32x4 a[G::FM];
  i32x8 b[G::FT];
};

// What a wave of a tile loads, reads and stores.
template <class G>
struct TileI8 {
  __amdgpu_buffer_rsrc_t ra, rb;
  char* lds;
  int lane, wave, wm, wt, stages, M, T;
  int64_t m0, t0;
  // Next stage's source offsets.  Past the last stage A's lie beyond its resource
  // (zeros), B's in the next row or beyond; neither is multiplied.  A stage that
  // ends past K brings the next row's first codes too: the weight's codes there
  // are zero.
  uint32_t a_src, m_src, b_src[G::B_DMA];
  int a_off[2], m_off, b_off[2][G::FT][2];           // fragment addresses within a slot

  // tile (tm, tt) of BM rows and BT tokens
  __device__ __forceinline__ TileI8(char* lds_, const int8_t* Xq, const char* packed, int M_, int T_, int Kred, int tm,
                                    int tt)
      : lds(lds_), M(M_), T(T_) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave % G::WGM;
    wt = wave / G::WGM;
    m0 = (int64_t)tm * G::BM;
    t0 = (int64_t)tt * G::BT;
    stages = (Kred + G::KS - 1) / G::KS;
    const int rows_t = (int)((T - t0) < G::BT ? (T - t0) : G::BT);
    ra = make_rsrc(packed + (int64_t)(tm / G::PER_CHUNK) * stages * kChunkBytes, (int64_t)stages * kChunkBytes);
    rb = make_rsrc(Xq + t0 * Kred, (int64_t)rows_t * Kred);
    const uint32_t row0 = (uint32_t)(tm % G::PER_CHUNK) * G::BM;    // the tile's first row within the chunk
    a_src = row0 * 64 + wave * (G::A_BYTES / G::WAVES) + lane * 16;
    m_src = kChunkValueBytes + row0 * 16 + wave * 1024 + lane * 16;
#pragma unroll
    for (int j = 0; j < G::B_DMA; ++j) {
      const int row = wave * (G::BT / G::WAVES) + j * 8 + (lane >> 3);
      b_src[j] = (uint32_t)row * Kred + (((lane & 7) ^ ((row ^ (row >> 3)) & 7)) << 4);
    }
    const int h = lane >> 5, arow = wm * G::WM + (lane & 31);
    m_off = G::A_BYTES + G::B_BYTES + arow * 16 + h * 8;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      a_off[s] = arow * 64 + (((2 * h + s) ^ ((arow >> 2) & 3)) << 4);
#pragma unroll
      for (int ft = 0; ft < G::FT; ++ft) {
        const int row = wt * G::WT + ft * 32 + (lane & 31), sw = (row ^ (row >> 3)) & 7;
        b_off[s][ft][0] = G::A_BYTES + row * 128 + (((2 * s + h) ^ sw) << 4);
        b_off[s][ft][1] = G::A_BYTES + row * 128 + (((4 + 2 * s + h) ^ sw) << 4);
      }
    }
  }
  static __device__ __forceinline__ int after(int slot) { return slot == (G::NST - 1) * G::SLOT ? 0 : slot + G::SLOT; }
  // this wave's share of the next stage, into the slot at `slot`
  __device__ __forceinline__ void issue(int slot) {
    char* a = lds + slot + wave * (G::A_BYTES / G::WAVES);
#pragma unroll
    for (int j = 0; j < G::A_DMA; ++j) dma16(ra, a + j * 1024, a_src + j * 1024);
    char* b = lds + slot + G::A_BYTES + wave * (G::B_BYTES / G::WAVES);
#pragma unroll
    for (int j = 0; j < G::B_DMA; ++j) dma16(rb, b + j * 1024, b_src[j]);
    if (wave < G::META_WAVES) dma16(ra, lds + slot + G::A_BYTES + G::B_BYTES + wave * 1024, m_src);
    a_src += kChunkBytes;
    m_src += kChunkBytes;
#pragma unroll
    for (int j = 0; j < G::B_DMA; ++j) b_src[j] += G::KS;
  }
  // until this wave's share of all but its newest NST - 2 stages is in LDS
  __device__ __forceinline__ void wait_older() const {
    if (wave < G::META_WAVES) wait_vmcnt<(G::NST - 2) * (G::A_DMA + G::B_DMA + 1)>();
    else wait_vmcnt<(G::NST - 2) * (G::A_DMA + G::B_DMA)>();
  }
  __device__ __forceinline__ void read_meta(u32x2 (&x)[G::FM], int slot) const {
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) x[fm] = *reinterpret_cast<const u32x2*>(lds + slot + m_off + fm * 512);
  }
  __device__ __forceinline__ void read(FragsI8<G>& f, int slot, int s) const {
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) {
      const i32x4 lo = *reinterpret_cast<const i32x4*>(lds + slot + b_off[s][ft][0]);
      const i32x4 hi = *reinterpret_cast<const i32x4*>(lds + slot + b_off[s][ft][1]);
      f.b[ft] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) f.a[fm] = *reinterpret_cast<const i32x4*>(lds + slot + a_off[s] + fm * 2048);
  }
  static __device__ __forceinline__ void multiply(i32x16 (&acc)[G::FM][G::FT], const FragsI8<G>& f,
                                                  const u32x2 (&x)[G::FM], int s, int ft) {
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm)
      acc[fm][ft] = __builtin_amdgcn_smfmac_i32_32x32x64_i8(f.a[fm], f.b[ft], acc[fm][ft], (int)x[fm][s], 0, 0);
  }
  // The sums scaled and stored to Y[t][m].  A lane holds four rows m of one token;
  // stored as they are, every store would touch 32 lines with 16 bytes each (7 us
  // a 256 x 256 tile).  So each wave turns 32 tokens at a time through its own
  // piece of the ring (free by now), and stores whole lines.  The lane's scales
  // are all loaded first, from clamped, valid places (a load behind a bounds test
  // would be waited for by itself); M % 4 == 0.
  template <typename O>
  __device__ __forceinline__ void store(const i32x16 (&acc)[G::FM][G::FT], const float* __restrict__ x_scale,
                                        const float* __restrict__ w_scale, O* __restrict__ Y) const {
    constexpr int ROW = G::WM * (int)sizeof(O) + 16;  // a token's rows, padded against bank conflicts
    constexpr int PER = 16 / (int)sizeof(O), LANES = G::WM / PER, TOKENS = 64 / LANES;   // 16-byte pieces
    static_assert(G::WAVES * 32 * ROW <= G::LDS_BYTES, "the ring holds every wave's piece");
    wait_vmcnt<0>();                                 // no load into the ring is left
    wait_lgkmcnt0();
    barrier();
    compiler_fence();
    char* own = lds + wave * (32 * ROW);
    float st[G::FT];
    Pack<float, 4> sn[G::FM][4];
    const int64_t tw = t0 + wt * G::WT, mw = m0 + wm * G::WM;
    const int h4 = 4 * (lane >> 5);
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) {
      const int64_t t = tw + ft * 32 + (lane & 31);
      st[ft] = x_scale[t < T ? t : T - 1];
    }
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t m = mw + fm * 32 + 8 * q + h4;
        sn[fm][q] = load_pack<float, 4>(w_scale + (m < M ? m : M - 4));
      }
    const int64_t m = mw + (lane % LANES) * PER;
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) {
#pragma unroll
      for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = scaled(acc[fm][ft][4 * q + i], st[ft], sn[fm][q].v[i]);
          store4<O>(reinterpret_cast<O*>(own + (lane & 31) * ROW) + fm * 32 + 8 * q + h4, y);
        }
      compiler_fence();                              // (a wave's LDS operations run in order)
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
          } else if (m < M) {                        // 16-bit outputs, M % 8 == 4: the last four
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = y.v[i];
          }
        }
      }
      compiler_fence();
    }
  }
};

template <class G>
__device__ __forceinline__ void clear_acc(i32x16 (&acc)[G::FM][G::FT]) {
#pragma unroll
  for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) acc[fm][ft] = i32x16{};
}

// Small tiles, one or several blocks a compute unit: each step's fragments are read
// ahead of the step before, one barrier a stage, the slot refilled among the
// second step's MFMAs; while one block waits, another multiplies.
template <class G, typename O>
__global__ __launch_bounds__(G::THREADS, G::BLOCKS* G::WAVES / 4) void spmm_i8_kernel(
    const int8_t* __restrict__ Xq, const char* __restrict__ packed, int M, int T, int Kred,
    const float* __restrict__ x_scale, const float* __restrict__ w_scale, O* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int tm, tt;
  tile_of_block(blockIdx.x, gridDim.x, (M + G::BM - 1) / G::BM, (T + G::BT - 1) / G::BT, 8, tm, tt);
  TileI8<G> t(lds, Xq, packed, M, T, Kred, tm, tt);
  i32x16 acc[G::FM][G::FT];
  clear_acc<G>(acc);
#pragma unroll
  for (int i = 0; i < G::NST - 1; ++i) t.issue(i * G::SLOT);
  t.wait_older();
  barrier();
  compiler_fence();
  FragsI8<G> f0, f1;
  u32x2 x0[G::FM], x1[G::FM];
  int cur = 0, next = G::SLOT;
  t.issue((G::NST - 1) * G::SLOT);
  t.read_meta(x0, cur);
  t.read(f0, cur, 0);
  for (int s = 0; s < t.stages; ++s) {
    t.read(f1, cur, 1);
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) t.multiply(acc, f0, x0, 0, ft);
    __builtin_amdgcn_sched_barrier(0);
    wait_lgkmcnt0();                                 // this wave's reads of the stage are complete
    t.wait_older();
    barrier();
    compiler_fence();
    t.read_meta(x1, next);                           // (past the last stage: a slot of earlier codes, not multiplied)
    t.read(f0, next, 0);
    t.multiply(acc, f1, x0, 1, 0);
    __builtin_amdgcn_sched_barrier(0);
    t.issue(cur);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int ft = 1; ft < G::FT; ++ft) t.multiply(acc, f1, x0, 1, ft);
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) x0[fm] = x1[fm];
    cur = next;
    next = t.after(next);
  }
  t.store(acc, x_scale, w_scale, Y);
}

// The large tiles, eight waves in two groups half a stage apart (waves 0..3 and
// 4..7, one of each on every SIMD).  While one group multiplies a stage, the
// other reads its fragments of it from LDS and issues its share of the stage
// after next, then they change places; a barrier ends each phase.  A wave's LDS
// reads are complete before the barrier that ends its memory phase, so a slot is
// free (both groups have read it) in the phase its refill is issued.
//
// 8192 x 9216 x 9216, bf16 out: 360 to 400 us with the clock that the card holds
// (1.8 GHz at 376), 3.7e15 dense-equivalent operations a second, half of what the
// instruction alone reaches in a tight loop.  Counted, a stage of a full tile takes
// about 2030 cycles, 1024 of them products (the matrix cores are busy 49% of the
// time): a phase lasts some 1015 cycles where its products take 512, so the memory
// phase, twice as long as the products beside it, is what bounds the loop.
// Timing copies of it (of 388 us then): without the loads into LDS
// 310, without the reads from it 306, without the products 327, products alone
// 275.  Slower were: one schedule for all waves (5 to 8%), 128 x 128 a wave in
// four waves, a raised priority for the multiplying waves, the refill issued
// before the reads; groups of 2, 4, 6 and 16 row tiles in the tile order.
template <class G, typename O>
__device__ __forceinline__ void ping_pong_tile(char* lds, const int8_t* Xq, const char* packed, int M, int T, int Kred,
                                               int tm, int tt, const float* __restrict__ x_scale,
                                               const float* __restrict__ w_scale, O* __restrict__ Y) {
  static_assert(G::WAVES == 8 && G::NST == 3, "two groups of four waves, three slots");
  TileI8<G> t(lds, Xq, packed, M, T, Kred, tm, tt);
  FragsI8<G> f[2];
  u32x2 x[G::FM];
  i32x16 acc[G::FM][G::FT];
  clear_acc<G>(acc);
  auto phase_end = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    compiler_fence();
    __builtin_amdgcn_sched_barrier(0);
  };
  int cur = 0, refill = 2 * G::SLOT;
  auto memory_phase = [&]() {
    t.read_meta(x, cur);
    t.read(f[0], cur, 0);
    t.read(f[1], cur, 1);
    t.issue(refill);
    cur = t.after(cur);
    refill = t.after(refill);
    wait_lgkmcnt0();
  };
  auto multiply_phase = [&]() {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int ft = 0; ft < G::FT; ++ft) t.multiply(acc, f[s], x, s, ft);
    __builtin_amdgcn_sched_barrier(0);
  };
  t.issue(0);
  t.issue(G::SLOT);
  t.wait_older();
  phase_end();
  if (t.wave < 4) {
    for (int s = 0; s < t.stages; ++s) {
      memory_phase();
      phase_end();
      multiply_phase();
      t.wait_older();                                // this wave's share of stage s + 1 is there
      phase_end();
    }
    phase_end();
  } else {
    phase_end();
    for (int s = 0; s < t.stages; ++s) {
      memory_phase();
      t.wait_older();
      phase_end();
      multiply_phase();
      phase_end();
    }
  }
  t.store(acc, x_scale, w_scale, Y);
}

typedef GeoI8<256, 256, 2, 4, 1> FullI8;
typedef GeoI8<256, 128, 4, 2, 1> HalfI8;
typedef GeoI8<128, 128, 2, 2, 2> SmallI8;
typedef GeoI8<128, 128, 4, 2, 1, 4> SingleI8;
typedef GeoI8<128, 64, 4, 1, 1, 4> NarrowI8;
typedef GeoI8<64, 64, 2, 2, 1, 4> LeastI8;

// The first rows_full row tiles in 256 x 256 tiles, the others in 256 x 128
// (full_width_rows: a grid that would end in a partly filled round of blocks
// ends sooner so; 8192 x 9216 x 9216 has 4.5 rounds of full tiles).
template <typename O>
__global__ __launch_bounds__(FullI8::THREADS, 2) void spmm_i8_large_kernel(
    const int8_t* __restrict__ Xq, const char* __restrict__ packed, int M, int T, int Kred, int rows_full,
    const float* __restrict__ x_scale, const float* __restrict__ w_scale, O* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int rows = (M + 255) / 256, full = (T + 255) / 256 * rows_full;
  int tm, tt;
  if ((int)blockIdx.x < full) {
    tile_of_block(blockIdx.x, full, rows_full, (T + 255) / 256, 8, tm, tt);
    ping_pong_tile<FullI8, O>(lds, Xq, packed, M, T, Kred, tm, tt, x_scale, w_scale, Y);
  } else {
    tile_of_block(blockIdx.x - full, gridDim.x - full, rows - rows_full, (T + 127) / 128, 8, tm, tt);
    ping_pong_tile<HalfI8, O>(lds, Xq, packed, M, T, Kred, rows_full + tm, tt, x_scale, w_scale, Y);
  }
}

template <typename O>
struct SpmmArgs {
  const int8_t* Xq;
  const char* packed;
  int M, T, K;
  const float *xs, *ws;
  O* Y;
  hipStream_t s;
};

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
// Measured (us, bf16 out, with the better of 64 and 32 rows; floor: the weight at the
// 6.04 TB/s of a large read): 9216 -> 27648 at 1 / 16 / 64 tokens 30.3 / 33.9 / 44.6
// (floor 26.4), 9216 -> 9216 10.9 / 11.8 / 18.3 (8.8), 5120 -> 15360 10.2 / 10.8 /
// 13.2 (8.1), 20480 -> 5120 12.7 / 14.4 / 23.2 (10.9), 36864 -> 9216 42.2 / 50.5 /
// 77.2 (35.2); decode_launch below gives some of them to the GEMM's tiles.  At one
// token HBM bounds it.  At 64 a block takes in all of X beside its weight, at about
// 75 GB/s a compute unit whatever its queue (two and three sets in flight, 12 and 16
// waves: the same or slower; what sets that rate is not established), and a long
// reduction leaves units without a block (20480 -> 5120: 160 blocks).
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
  const int64_t t0 = (int64_t)blockIdx.y * (8 * R);  // the block's tokens (all of them up to 64)
  Xq += t0 * Kred;
  T = T - t0 < 8 * R ? (int)(T - t0) : 8 * R;
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
  decode_store<W, FM, FT, O>(lds, acc, M, T, x_scale + t0, w_scale, Y + t0 * M);
}

template <int R, int FM, int G, int D, int W, int WPS, typename O>
hipError_t decode_go(const SpmmArgs<O>& a) {
  constexpr int FT = R > 4 ? 2 : 1;
  constexpr int LDS = W * (G * R * 1024 > FM * FT * 2048 ? G * R * 1024 : FM * FT * 2048);   // X rows; sums
  auto kern = decode_i8_kernel<R, FM, G, D, W, WPS, O>;
  if constexpr (LDS > 64 * 1024) {
    static LdsLimit limit;
    const hipError_t e = limit.set((const void*)kern, LDS);
    if (e != hipSuccess) return e;
  }
  kern<<<dim3((unsigned)cdiv(a.M, 32 * FM), (unsigned)cdiv(a.T, 8 * R)), 64 * W, LDS, a.s>>>(a.Xq, a.packed, a.M, a.T, a.K, a.xs, a.ws, a.Y);
  return hipGetLastError();
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

template <class G, typename O>
hipError_t tiles_go(const SpmmArgs<O>& a) {
  static LdsLimit limit;
  auto kern = spmm_i8_kernel<G, O>;
  const hipError_t e = limit.set((const void*)kern, G::LDS_BYTES);
  if (e != hipSuccess) return e;
  kern<<<(unsigned)(cdiv(a.M, G::BM) * cdiv(a.T, G::BT)), G::THREADS, G::LDS_BYTES, a.s>>>(a.Xq, a.packed, a.M, a.T, a.K,
                                                                                        a.xs, a.ws, a.Y);
  return hipGetLastError();
}

// Tiles of the GEMM's kind in one round: where BM rows a tile leave more than half
// of the compute units one tile each, and none two, its deeper queue of weight
// streams faster than the kernel above (us, tiles against the better of its two forms):
//   9216 -> 27648 (216 tiles of 128): 1 token 29.8 / 30.3, 32: 30.3 / 36.4, 64: 33.5 / 44.6
//   9216 -> 36864 (144 of 256):       1 token 39.3 / 40.3, 32: 43.0 / 49.9, 64: 48.1 / 63.9
//   5120 -> 20480 (160 of 128):       1 token 11.5 / 14.3, 32: 12.4 / 15.9, 64: 13.2 / 19.2
//   5120 -> 15360 (240 of 64):                             32: 11.0 / 11.1, 64: 11.3 / 13.2
//   9216 -> 9216 (144 of 64):                              32: 16.9 / 12.0, 64: 16.9 / 18.3
// (so 64 rows only from 33 tokens on).  With fewer tiles a compute unit's share
// takes longer (20480 -> 5120, 80 tiles of 64, 64 tokens: 32.8 / 23.2).
//
// Otherwise 64 rows a block where that leaves 128 blocks or more (9216 outputs, 9216 wide,
// 32 tokens: 12.0 us against 16.6 with 32 rows): every block draws all of X, so
// wider ones draw it less often.  Below, 64 rows would leave too many compute
// units idle (5120 outputs, 20480 wide, 32 tokens: 20.7 us against 16.7).
// Waves, stages and sets as measured best over the five shapes above: the
// registers are kept to 128 (two blocks a compute unit) up to 32 tokens; at 64
// the 64-row block needs more, and four waves beat eight (44.9 against 46.8 us).
template <typename O>
hipError_t decode_launch(const int8_t* Xq, const float* xs, int64_t T, int64_t K, const void* packed, const float* ws,
                         int64_t M, void* Y, hipStream_t s) {
  const SpmmArgs<O> a{Xq, (const char*)packed, (int)M, (int)T, (int)K, xs, ws, (O*)Y, s};
  const int64_t cus = compute_units();
  auto one_round = [&](int bm) { return 2 * cdiv(M, bm) > cus && cdiv(M, bm) <= cus; };
  if (T > 32 && one_round(64)) return tiles_go<LeastI8, O>(a);
  if (one_round(128)) return T <= 32 ? tiles_go<GeoI8<128, 32, 4, 1, 1, 4>, O>(a) : tiles_go<NarrowI8, O>(a);
  if (one_round(256))
    return T <= 32 ? tiles_go<GeoI8<256, 32, 4, 1, 1, 4>, O>(a) : tiles_go<GeoI8<256, 64, 4, 1, 1, 4>, O>(a);
  const bool wide = M > 127 * 64;
  if (T <= 8) return wide ? decode_go<1, 2, 1, 2, 8, 4, O>(a) : decode_go<1, 1, 2, 2, 8, 4, O>(a);
  if (T <= 16) return wide ? decode_go<2, 2, 1, 2, 8, 4, O>(a) : decode_go<2, 1, 1, 2, 16, 4, O>(a);
  if (T <= 32) return wide ? decode_go<4, 2, 1, 1, 8, 4, O>(a) : decode_go<4, 1, 1, 2, 8, 4, O>(a);
  return wide ? decode_go<8, 2, 1, 1, 4, 2, O>(a) : decode_go<8, 1, 1, 1, 8, 4, O>(a);
}

// Any number of tokens.  Five kernels, chosen by their estimated time in units
// of a stage (us for 128 k), fitted to sweeps of 65 .. 8192 tokens over 9216 ->
// 9216 / 27648, 20480 -> 5120, 5120 -> 5120 / 15360, 4096 -> 1024 and 768 -> 2304:
//   large   0.010 a unit of full_width_rows' cost (100 a round of full tiles, 65
//           of half tiles)
//   small   128 x 128 tiles: 0.42 up to one a compute unit (eight waves, four
//           slots: 5120 -> 20480 at 128 tokens 17.6 us, as below 18.8), then 0.35 +
//           0.0014 a tile (two a unit, four waves and three slots each)
//   narrow  128 x 64 tiles, at most one a compute unit: 0.25, or 64 x 64: 0.215.
//           A compute unit takes in some 70 GB/s by LDS-DMA however deep the ring
//           (four slots here; three 43 us, six 40, eight 41 for 20480 -> 5120 at
//           256 tokens) and however many waves (eight: 40), so where one round of
//           smaller tiles is enough, less to load is faster.
//   direct  the few-token kernel over groups of 64 tokens, 64 rows a block: 0.13 +
//           0.0006 a block; up to 128 such blocks 32 rows (4096 -> 1024 at 512
//           tokens 7.3 us against 9.2; 5120 -> 5120 at 65, 160 blocks, 12.8
//           against 11.5)
// Measured, us (large / small, up to one tile a compute unit in its eight-wave form /
// 128 x 64 / 64 x 64 / direct with 64 rows), the rule's choice starred:
//   9216 -> 9216    128 tokens  37.7 /  26.3 /  20.3* /  22.8  /  24.1
//                   256         37.7 /  26.7*/  31.3  /  33.7  /  36.3
//                   512         38.7*/  45.7 /  49.6  /  54.4  /  61.4
//                  1000         58.3*/  73.1 /  80.9  /  99.4  / 109
//                  8192        359 * / 465   /        /        / 882
//   20480 -> 5120    65         75.9 /  52.4 /  38.6  /  33.1* /  31.4
//                   256         76.8 /  52.8 /  39.4* /  47.5  /  50.7
//                   512         77.2 /  53.5*/  68.9  /  73.1  /  77.3
//                  1000         78.8*/  99.3 / 104    / 125    / 129
//   5120 -> 5120     65         22.4 /  16.4 /  12.8  /  10.9* /  11.5
//                   256         23.3 /  17.1 /  13.2* /  15.5  /  15.9
//   9216 -> 27648   128         54.3 /  41.6*/  50.8  /  65.0  /  76.1
//                   512         80.8*/ 118   / 147    / 181    / 207
//   4096 -> 1024    512         19.3 /  14.1 /  11.1  /   9.6  /   9.2 (32 rows 7.3*)
template <typename O>
hipError_t spmm_launch(const int8_t* Xq, const float* xs, int64_t T, int64_t K, const void* packed, const float* ws,
                       int64_t M, void* Y, hipStream_t s) {
  if (T <= 64) return decode_launch<O>(Xq, xs, T, K, packed, ws, M, Y, s);
  const SpmmArgs<O> a{Xq, (const char*)packed, (int)M, (int)T, (int)K, xs, ws, (O*)Y, s};
  const int64_t cus = compute_units(), rows = cdiv(M, 256), cols = cdiv(T, 256), halves = cdiv(T, 128);
  const int64_t rows_full = full_width_rows(rows, cols, halves, cus);
  const double large = 0.010 * (100 * cdiv(rows_full * cols, cus) + 65 * cdiv((rows - rows_full) * halves, cus));
  const int64_t tiles = cdiv(M, 128) * halves;
  const double small = tiles <= cus ? 0.42 : 0.35 + 0.0014 * (256.0 / cus) * tiles;
  const int64_t blocks = cdiv(M, 64) * cdiv(T, 64);
  const double narrow = blocks <= cus ? 0.215 : cdiv(M, 128) * cdiv(T, 64) <= cus ? 0.25 : small;
  const double direct = 0.13 + 0.0006 * (256.0 / cus) * blocks;
  // (a grid's second dimension ends at 65535)
  if (direct <= narrow && direct <= small && direct <= large && cdiv(T, 64) <= 65535)
    return blocks <= 128 ? decode_go<8, 1, 1, 1, 8, 4, O>(a) : decode_go<8, 2, 1, 1, 4, 2, O>(a);
  if (narrow < small && narrow <= large)
    return blocks <= cus ? tiles_go<LeastI8, O>(a) : tiles_go<NarrowI8, O>(a);
  if (small <= large) return tiles <= cus ? tiles_go<SingleI8, O>(a) : tiles_go<SmallI8, O>(a);
  static LdsLimit limit;
  auto kern = spmm_i8_large_kernel<O>;
  const hipError_t e = limit.set((const void*)kern, FullI8::LDS_BYTES);
  if (e != hipSuccess) return e;
  const int64_t all = rows_full * cols + (rows - rows_full) * halves;
  kern<<<(unsigned)all, FullI8::THREADS, FullI8::LDS_BYTES, s>>>(a.Xq, a.packed, a.M, a.T, a.K, (int)rows_full, xs, ws,
                                                                 a.Y);
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
