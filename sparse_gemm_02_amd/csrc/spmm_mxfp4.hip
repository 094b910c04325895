// The 2:4 sparse product on 4-bit floating point codes, Y[t][n] = sum over blocks of
// 2^(Ex + Ew) sum x w, on gfx950's v_mfma_scale_f32_32x32x64_f8f6f4.
//
// Lane layout of the instruction (checked against a host model): lane l's A operand is
// one block of 32 codes of row l%32, k 32*(l/32) .. +31, in four registers, and a
// scale byte; B likewise of column l%32; D as every 32x32 MFMA.  The sums of 144 and
// 576 steps were within 2e-7 of the exact ones (two-norm).  There is no sparse form of
// it: the weight travels as kept codes and positions (3.25 bits for a dense value) as
// far as a wave's registers, and is expanded there (21 operations for 32 values a
// lane, which the matrix instructions of other waves cover).
//
// A stage is 128 k, four blocks; MFMA step s of a stage takes blocks s (lanes 0..31)
// and 2 + s (lanes 32..63), so that a lane's two blocks are neighbours.
#include "common.h"
#include "dma.h"
#include "launch.h"
#include "mxfp4.h"
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

// ---------------------------------------------------------------- the GEMM
// Transposed output tiles Out^T = W . X^T of BM x BT, stages in a ring of LDS slots
// filled by buffer-to-LDS loads: the weight's chunks as they are (a fragment's reads
// are contiguous), X's rows of 64 bytes with granule c of row r at c ^ ((r>>2)&3), X's
// scales as one word a row.
template <int BM_, int BT_, int WGM_, int WGT_, int BLOCKS_, int NST_>
struct Geo {
  static constexpr int BM = BM_, BT = BT_, WGM = WGM_, WGT = WGT_, WAVES = WGM * WGT, THREADS = 64 * WAVES;
  static constexpr int WM = BM / WGM, WT = BT / WGT, FM = WM / 32, FT = WT / 32;
  static constexpr int NST = NST_, BLOCKS = BLOCKS_;
  static constexpr int A_BYTES = BM / kMxRows * kMxChunkBytes, B_BYTES = BT * 64, S_BYTES = BT * 4;
  static constexpr int SLOT = A_BYTES + B_BYTES + S_BYTES, LDS_BYTES = NST * SLOT;
  // loads of a wave and stage: the weight's (four a chunk: 1, 1 and 1 KB, 256 bytes), X's (1
  // KB), and one of 64 rows' scales by the first S_WAVES waves
  static constexpr int A_DMA = BM / kMxRows * 4 / WAVES, B_DMA = B_BYTES / 1024 / WAVES, S_WAVES = BT / 64;
  static_assert(BM % kMxRows == 0 && A_DMA * WAVES == BM / kMxRows * 4 && B_DMA * WAVES * 1024 == B_BYTES &&
                S_WAVES <= WAVES && BT % 64 == 0, "tile and wave split");
  static_assert(BLOCKS * LDS_BYTES <= 160 * 1024, "LDS budget");
};

template <class G>
struct Frags {                                       // one stage's operands, the weight's not expanded
  u32x4 a[G::FM], b[G::FT][2];
  u32x2 kept[G::FM];
  uint32_t sa[G::FM], sb[G::FT];
};

template <class G>
struct Tile {
  __amdgpu_buffer_rsrc_t ra, rb, rs;
  char* lds;
  int lane, wave, wm, wt, stages, M, T;
  int64_t m0, t0;
  // Next stage's source offsets.  Past the last stage they lie in another chunk or row,
  // or beyond the resource; what they bring is not multiplied.
  uint32_t a_src[G::A_DMA], b_src[G::B_DMA], s_src;
  int b_off[G::FT][2], s_off;                        // fragment addresses within a slot

  __device__ __forceinline__ Tile(char* lds_, const uint8_t* codes, const uint8_t* exps, const char* packed, int M_,
                                  int T_, int stages_, int tm, int tt)
      : lds(lds_), stages(stages_), M(M_), T(T_) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave % G::WGM;
    wt = wave / G::WGM;
    m0 = (int64_t)tm * G::BM;
    t0 = (int64_t)tt * G::BT;
    const int rows_t = (int)((T - t0) < G::BT ? (T - t0) : G::BT);
    const int chunks = (int)((M - m0 + kMxRows - 1) / kMxRows);
    const int64_t line = (int64_t)stages * kMxChunkBytes;
    ra = make_rsrc(packed + m0 / kMxRows * line, (chunks < G::BM / kMxRows ? chunks : G::BM / kMxRows) * line);
    rb = make_rsrc(codes + t0 * (stages * 64), (int64_t)rows_t * (stages * 64));
    rs = make_rsrc(exps + t0 * (stages * 4), (int64_t)rows_t * (stages * 4));
#pragma unroll
    for (int j = 0; j < G::A_DMA; ++j) {
      const int i = wave * G::A_DMA + j;             // load i % 4 of chunk i / 4
      a_src[j] = (uint32_t)((i / 4) * line) + (i % 4) * 1024 + lane * (i % 4 == 3 ? 4 : 16);
    }
#pragma unroll
    for (int j = 0; j < G::B_DMA; ++j) {
      const int row = (wave * G::B_DMA + j) * 16 + (lane >> 2);
      b_src[j] = (uint32_t)row * (stages * 64) + (((lane & 3) ^ ((row >> 2) & 3)) << 4);
    }
    s_src = (uint32_t)(wave * 64 + lane) * (stages * 4);
    const int h = lane >> 5;
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) {
      const int row = wt * G::WT + ft * 32 + (lane & 31);
#pragma unroll
      for (int s = 0; s < 2; ++s) b_off[ft][s] = G::A_BYTES + row * 64 + (((2 * h + s) ^ ((row >> 2) & 3)) << 4);
    }
    s_off = G::A_BYTES + G::B_BYTES + (wt * G::WT + (lane & 31)) * 4;
  }
  static __device__ __forceinline__ int after(int slot) { return slot == (G::NST - 1) * G::SLOT ? 0 : slot + G::SLOT; }
  // this wave's share of the next stage, into the slot at `slot`
  __device__ __forceinline__ void issue(int slot) {
#pragma unroll
    for (int j = 0; j < G::A_DMA; ++j) {
      const int i = wave * G::A_DMA + j;
      char* to = lds + slot + (i / 4) * kMxChunkBytes + (i % 4) * 1024;
      if (i % 4 == 3) dma4(ra, to, a_src[j]);
      else dma16(ra, to, a_src[j]);
      a_src[j] += kMxChunkBytes;
    }
    char* b = lds + slot + G::A_BYTES + wave * (G::B_DMA * 1024);
#pragma unroll
    for (int j = 0; j < G::B_DMA; ++j) {
      dma16(rb, b + j * 1024, b_src[j]);
      b_src[j] += 64;
    }
    if (wave < G::S_WAVES) dma4(rs, lds + slot + G::A_BYTES + G::B_BYTES + wave * 256, s_src);
    s_src += 4;
  }
  // until this wave's share of all but its newest NST - 2 stages is in LDS
  __device__ __forceinline__ void wait_older() const {
    if (wave < G::S_WAVES) wait_vmcnt<(G::NST - 2) * (G::A_DMA + G::B_DMA + 1)>();
    else wait_vmcnt<(G::NST - 2) * (G::A_DMA + G::B_DMA)>();
  }
  __device__ __forceinline__ void read(Frags<G>& f, int slot) const {
    const int h = lane >> 5;
    const char* base = lds + slot;
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
      const int row = wm * G::WM + fm * 32 + (lane & 31);
      const char* c = base + (row / kMxRows) * kMxChunkBytes;
      f.a[fm] = *reinterpret_cast<const u32x4*>(c + (h * kMxRows + row % kMxRows) * 16);
      f.kept[fm] = *reinterpret_cast<const u32x2*>(c + kMxMaskAt + (h * kMxRows + row % kMxRows) * 8);
      f.sa[fm] = *reinterpret_cast<const uint32_t*>(c + kMxScaleAt + (row % kMxRows) * 4);
    }
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) {
      f.b[ft][0] = *reinterpret_cast<const u32x4*>(base + b_off[ft][0]);
      f.b[ft][1] = *reinterpret_cast<const u32x4*>(base + b_off[ft][1]);
      f.sb[ft] = *reinterpret_cast<const uint32_t*>(base + s_off + ft * 128);
    }
  }
  __device__ __forceinline__ void multiply(f32x16 (&acc)[G::FM][G::FT], const Frags<G>& f) const {
    const int shift = (lane >> 5) * 16;              // a lane's two scale bytes to the low half
    uint32_t sb[G::FT];
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) sb[ft] = f.sb[ft] >> shift;
#pragma unroll
    for (int fm = 0; fm < G::FM; ++fm) {
      const uint32_t sa = f.sa[fm] >> shift;
      const u32x4 a0 = expand24(f.a[fm][0], f.a[fm][1], f.kept[fm][0]);
      const u32x4 a1 = expand24(f.a[fm][2], f.a[fm][3], f.kept[fm][1]);
#pragma unroll
      for (int ft = 0; ft < G::FT; ++ft) acc[fm][ft] = mfma<0>(a0, f.b[ft][0], acc[fm][ft], sa, sb[ft]);
#pragma unroll
      for (int ft = 0; ft < G::FT; ++ft) acc[fm][ft] = mfma<1>(a1, f.b[ft][1], acc[fm][ft], sa, sb[ft]);
    }
  }
  // The sums rounded and stored to Y[t][m].  A lane holds four rows m of one token; each
  // wave turns 32 tokens at a time through its own piece of the ring (free by now) and
  // stores whole lines.  M % 4 == 0.
  template <typename O>
  __device__ __forceinline__ void store(const f32x16 (&acc)[G::FM][G::FT], O* __restrict__ Y) const {
    constexpr int ROW = G::WM * (int)sizeof(O) + 16;  // a token's rows, padded against bank conflicts
    constexpr int PER = 16 / (int)sizeof(O), LANES = G::WM / PER, TOKENS = 64 / LANES;   // 16-byte pieces
    static_assert(G::WAVES * 32 * ROW <= G::LDS_BYTES, "the ring holds every wave's piece");
    wait_vmcnt<0>();                                 // no load into the ring is left
    wait_lgkmcnt0();
    barrier();
    compiler_fence();
    char* own = lds + wave * (32 * ROW);
    const int64_t tw = t0 + wt * G::WT, mw = m0 + wm * G::WM;
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

template <class G, typename O>
__global__ __launch_bounds__(G::THREADS, G::BLOCKS* G::WAVES / 4) void spmm_mxfp4_kernel(
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ exps, const char* __restrict__ packed, int M, int T,
    int stages, O* __restrict__ Y) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int tm, tt;
  tile_of_block(blockIdx.x, gridDim.x, (M + G::BM - 1) / G::BM, (T + G::BT - 1) / G::BT, 8, tm, tt);
  Tile<G> t(lds, codes, exps, packed, M, T, stages, tm, tt);
  f32x16 acc[G::FM][G::FT];
#pragma unroll
  for (int fm = 0; fm < G::FM; ++fm)
#pragma unroll
    for (int ft = 0; ft < G::FT; ++ft) acc[fm][ft] = f32x16{};
#pragma unroll
  for (int i = 0; i < G::NST - 1; ++i) t.issue(i * G::SLOT);
  int cur = 0, refill = (G::NST - 1) * G::SLOT;
  Frags<G> f;
  for (int s = 0; s < stages; ++s) {
    t.wait_older();
    barrier();                                       // the stage is there; every wave has read the one before
    compiler_fence();
    t.issue(refill);
    t.read(f, cur);
    t.multiply(acc, f);
    wait_lgkmcnt0();
    cur = t.after(cur);
    refill = t.after(refill);
  }
  t.store(acc, Y);
}

template <typename O>
struct Args {
  const uint8_t *codes, *exps;
  const char* packed;
  int M, T, stages;
  O* Y;
  hipStream_t s;
};

template <class G, typename O>
hipError_t tiles_go(const Args<O>& a) {
  static LdsLimit limit;
  auto kern = spmm_mxfp4_kernel<G, O>;
  const hipError_t e = limit.set((const void*)kern, G::LDS_BYTES);
  if (e != hipSuccess) return e;
  kern<<<(unsigned)(cdiv(a.M, G::BM) * cdiv(a.T, G::BT)), G::THREADS, G::LDS_BYTES, a.s>>>(a.codes, a.exps, a.packed,
                                                                                        a.M, a.T, a.stages, a.Y);
  return hipGetLastError();
}

template <typename O>
hipError_t spmm_launch(const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K, const void* packed, int64_t M,
                       void* Y, hipStream_t s) {
  const Args<O> a{codes, exps, (const char*)packed, (int)M, (int)T, (int)cdiv(K, kMxCols), (O*)Y, s};
  if (cdiv(M, 256) * cdiv(T, 256) >= 256) return tiles_go<Geo<256, 256, 4, 2, 1, 4>, O>(a);
  return tiles_go<Geo<64, 64, 2, 2, 1, 4>, O>(a);
}

}  // namespace

hipError_t launch_spmm_mxfp4(Dt out, const uint8_t* codes, const uint8_t* exps, int64_t T, int64_t K, const void* packed,
                             int64_t M, void* Y, hipStream_t s) {
  if (T == 0 || M == 0) return hipSuccess;
  if (K == 0) return launch_fill_zero(out, Y, T * M, s);
  if (out == Dt::BF16) return spmm_launch<uint16_t>(codes, exps, T, K, packed, M, Y, s);
  if (out == Dt::F16) return spmm_launch<_Float16>(codes, exps, T, K, packed, M, Y, s);
  return spmm_launch<float>(codes, exps, T, K, packed, M, Y, s);
}

}  // namespace slope
