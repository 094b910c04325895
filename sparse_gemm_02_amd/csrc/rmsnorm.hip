// Residual addition, root-mean-square norm and per-token int8 codes in one pass
// over the rows, and the norm's gradient.
//
//   h = x + res (rounded to the format),  rstd = 1 / sqrt(mean h^2 + eps)
//   y = h rstd g,   u = h g,  code = nearest(127 u / max|u|),  scale = max|u| / 127 rstd
//
// Bound by HBM: per element x, res (2 + 2 bytes) in, h (2) and y (2) or the
// code (1) out.  A row is read once into registers, its sum of squares and its
// largest |h g| are reduced together (the codes do not need rstd: it is common
// to the row and cancels), and the outputs are made from the registers.
// Measured (kernel times, medians): 8192 x 9216 bf16 with residual and codes 99 us
// (5.3 TB/s; a plain copy reaches 5.1), with y in place of the codes 106; 16384 x
// 1024 21 us; 1021 x 5120 fp16 with an fp32 gamma 9.4 us and 2047 x 771 fp32 6.6 us,
// of which one row alone takes 4.2.  Codes without a residual (8192 x 9216, 44 us at
// a copy's rate): bf16 without a gamma 44 us, fp16 50, with an fp16 gamma 52 (the
// vector units issue 80% of the cycles: the arithmetic bounds it), with an fp32 gamma
// 72 (63%: the search for the left-over, with its reduction, comes on top).
//
// Gradient:  a = dy g,  xh = h rstd,  c = mean(a xh)
//   dx = rstd (a - xh c) + dh,   dg = sum over tokens of dy xh
// The same row layout; a block keeps its columns over many rows, so dg's
// partial sums stay in registers, and a second kernel adds the blocks' rows in
// order.  Measured, with both kernels: 8192 x 9216 bf16 with dh 120 us (5.1 TB/s),
// 16384 x 1024 30, 4096 x 5120 38, 8192 x 768 fp16 15.1 us (11.2 and 3.9: launches
// and the first loads, not bandwidth).  Above 1536 vectors a row (12288 elements of
// 16 bits) a thread has four vectors, and 1024 threads leave it 128 registers: with
// 16-bit rows and a gamma these forms spill (7 to 59 of them, 135 in the odd-width
// form of fp16 rows and an fp32 gamma).  8192 x 16384 with dh (209 us at a copy's rate):
// bf16 298, fp16 with an fp32 gamma 442; 8192 x 16387: 450 and 903.  Few long rows
// (512 x 20480, 31 us against 12) pay for the partial rows too.
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "rows8.h"

namespace slope {

namespace {

// Elements per 16-byte access of a format.
template <typename In> constexpr int vec_elems() { return 16 / (int)sizeof(In); }

// Sums and maxima over lanes: the same in every lane, in a fixed order.  Lanes
// change values by cross-lane moves in the vector unit (a shuffle through LDS takes
// some 100 cycles for each of its six steps; one row of 9216: 4.9 us with them,
// 4.2 so).
template <int CTRL, typename V>
__device__ __forceinline__ V lane_move(V v) {
  return __builtin_bit_cast(V, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false));
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return __builtin_fmaxf(a, b); }
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max_bits(a, b); }
};
// over each sixteen lanes
template <class Op, typename V>
__device__ __forceinline__ V fold16(V v) {
  v = Op()(v, lane_move<0xB1>(v));                   // neighbours
  v = Op()(v, lane_move<0x4E>(v));                   // pairs of four
  v = Op()(v, lane_move<0x141>(v));                  // eight lanes mirrored
  return Op()(v, lane_move<0x140>(v));               // sixteen lanes mirrored
}
// over the wave
template <class Op, typename V>
__device__ __forceinline__ V fold(V v) {
  v = fold16<Op>(v);
  const uint32_t a = __builtin_bit_cast(uint32_t, v);
  const auto x = __builtin_amdgcn_permlane16_swap(a, a, false, false);
  v = Op()(__builtin_bit_cast(V, (uint32_t)x[0]), __builtin_bit_cast(V, (uint32_t)x[1]));
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto y = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  return Op()(__builtin_bit_cast(V, (uint32_t)y[0]), __builtin_bit_cast(V, (uint32_t)y[1]));
}
// over the values that a block's waves (at most 16) have put into `part`
template <class Op, typename V>
__device__ __forceinline__ V fold_waves(const V* part, int waves, V none) {
  const int w = threadIdx.x & 15;
  return fold16<Op>(w < waves ? part[w] : none);
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = __builtin_fmax(v, __shfl_xor(v, m));
  return v;
}

// A value that all lanes share, in scalar registers.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }
__device__ __forceinline__ float uniform(float v) { return __uint_as_float(uniform(__float_as_uint(v))); }
__device__ __forceinline__ double uniform(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  return __builtin_bit_cast(double, u32x2{uniform(w[0]), uniform(w[1])});
}

// The vectors of a row of K >= E elements: vector i holds elements E i .. E i +
// E - 1; the last one, when K is not a multiple of E (RAGGED), is moved back to
// end at K, and its first `skip` elements belong to the vector before it.  A
// vector past the row (skip == E) is read at element 0.
template <int E, bool RAGGED>
struct RowVec {
  int at, skip;
  __device__ __forceinline__ RowVec(int i, int K) {
    const int full = E * i;
    const bool live = full < K;
    if constexpr (RAGGED) {
      const int last = K - E;
      at = live ? (full < last ? full : last) : 0;
      skip = live ? full - at : E;
    } else {
      at = live ? full : 0;
      skip = live ? 0 : E;
    }
  }
  __device__ __forceinline__ bool mine(int e) const { return RAGGED ? e >= skip : skip == 0; }
};

template <typename V, int E, bool RAGGED>
__device__ __forceinline__ void store_vec(V* row, const RowVec<E, RAGGED>& r, const Pack<V, E>& x) {
  if (r.skip == 0) {
    store_pack<V, E>(row + r.at, x);
  } else if (RAGGED && r.skip < E) {
#pragma unroll
    for (int e = 1; e < E; ++e)
      if (e >= r.skip) row[r.at + e] = x.v[e];
  }
}

template <typename V, int E, bool RAGGED, bool TWICE>
__device__ __forceinline__ void put_vec(V* row, const RowVec<E, RAGGED>& r, const Pack<V, E>& x) {
  if constexpr (!TWICE) store_vec<V, E, RAGGED>(row, r, x);
  else if (r.skip < E) store_pack<V, E>(row + r.at, x);
}

// Zeros in place of a vector's elements that are not its own, so that no sum or
// maximum sees them.
template <typename V, int E, bool RAGGED>
__device__ __forceinline__ void drop_foreign(Pack<V, E>& x, const RowVec<E, RAGGED>& r) {
  if (r.skip != 0) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (!r.mine(e)) x.v[e] = elem_of<V>(0.f);
  }
}

// The compiler takes x for a new value here: what was computed from it before is
// not kept in registers for later but computed again.
template <typename V, int E>
__device__ __forceinline__ void forget(Pack<V, E>& x) {
  struct Words {
    uint32_t w[E * sizeof(V) / 4 > 0 ? E * sizeof(V) / 4 : 1];
  };
  if constexpr (E * sizeof(V) % 4 == 0) {
    Words y = __builtin_bit_cast(Words, x);
#pragma unroll
    for (uint32_t& w : y.w) asm("" : "+v"(w));
    x = __builtin_bit_cast(Pack<V, E>, y);
  }
}

// gamma's type, or none (all ones)
struct Ones {};
template <typename GT> constexpr bool kHasGamma = !std::is_same<GT, Ones>::value;
template <typename GT, int E>
struct Gamma {
  Pack<GT, E> g;
  __device__ __forceinline__ void load(const GT* p) { g = load_pack<GT, E>(p); }
  __device__ __forceinline__ float operator()(int e) const { return elem_f32(g.v[e]); }
  template <bool RAGGED>
  __device__ __forceinline__ void drop(const RowVec<E, RAGGED>& r) { drop_foreign<GT, E, RAGGED>(g, r); }
};
template <int E>
struct Gamma<Ones, E> {
  __device__ __forceinline__ void load(const Ones*) {}
  __device__ __forceinline__ float operator()(int) const { return 1.f; }
  template <bool RAGGED>
  __device__ __forceinline__ void drop(const RowVec<E, RAGGED>&) {}
};

// An fp32 gamma against 16-bit rows: products that fp32 does not hold exactly.
// (fp32 rows have no codes.)
template <typename In, typename GT>
constexpr bool kWide = std::is_same<GT, float>::value && !std::is_same<In, float>::value;
// Products that may leave fp32's range below (fp16 values times fp16 ones do not).
template <typename In, typename GT>
constexpr bool kMayVanish = kWide<In, GT> || (std::is_same<In, uint16_t>::value && kHasGamma<GT>);

struct NormOut {
  void *H, *Y;
  int8_t* q;
  float *qs, *rstd;
  bool norm;                                       // false: codes of x itself
};

// One row per block (WAVE: per wave, four rows a block), N vectors a thread.  All
// of the row's loads are issued before the first use: written as the formula
// reads, with loads under `if (residual)`, the compiler waited for each vector
// before it asked for the next (one row of 9216: 6.4 us against 4.9).
template <typename In, typename GT, int E, int N, bool WAVE, bool RAGGED>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void rms_row_kernel(const In* X, const In* res, const GT* gamma,
                                                                    int64_t T, int K, float eps, NormOut o) {
  typedef RowVec<E, RAGGED> Vec;
  constexpr bool WIDE = kWide<In, GT>;
  // gamma stays in registers between its two uses unless they would spill
  constexpr bool KEEP = N < 8;
  constexpr bool CODES = !std::is_same<In, float>::value;
  // The foreign elements of a row's last vector are the row's own too, loaded
  // twice.  TWICE: they are worked on and stored twice, with the same values, and
  // only the sum leaves them out (16384 x 1001 fp32 43.5 us; with zeros in their
  // place and the others stored one by one 59).  With more values a thread the registers
  // it takes cost more (2000 x 12301 bf16 55 us against 52).
  constexpr bool TWICE = RAGGED && N * E <= 16;
  // An h in place of an input is stored when every load of the row is complete:
  // another thread may have yet to load an element that this one stores.
  const bool late = TWICE && o.H && (o.H == (const void*)X || o.H == (const void*)res);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;
  if (WAVE && row >= T) return;
  const int tid = WAVE ? lane : (int)threadIdx.x, tpr = WAVE ? 64 : (int)blockDim.x;
  const In* x = X + row * K;
  const In* xr = res ? res + row * K : x;            // no residual: the row's first vector, and not used
  Pack<In, E> h[N], r[N];
  Gamma<GT, E> g[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int at = Vec(j * tpr + tid, K).at;
    h[j] = load_pack<In, E>(x + at);
    r[j] = load_pack<In, E>(xr + (res ? at : 0));
    if (KEEP) g[j].load(gamma + at);
  }
  __builtin_amdgcn_sched_barrier(0);
  float ss = 0.f;
  float top[N];                                      // largest |h g| (as fp32) of each vector
  uint32_t mine = 0u;                                // bits of the thread's largest
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const Vec rv(j * tpr + tid, K);
    top[j] = 0.f;
    if (res) {
#pragma unroll
      for (int e = 0; e < E; ++e) h[j].v[e] = elem_of<In>(elem_f32(h[j].v[e]) + elem_f32(r[j].v[e]));
    }
    if constexpr (TWICE) {
      if (o.H && !late && rv.skip < E) store_pack<In, E>((In*)o.H + row * K + rv.at, h[j]);
    } else {
      drop_foreign<In, E, RAGGED>(h[j], rv);
      if (o.H) store_vec<In, E, RAGGED>((In*)o.H + row * K, rv, h[j]);
    }
    if (!KEEP) g[j].load(gamma + rv.at);
    if (!TWICE && CODES) g[j].drop(rv);              // its foreign elements need not be finite
    const float before = ss;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float f = elem_f32(h[j].v[e]);
      ss = __builtin_fmaf(f, f, ss);
      // (with the second form for eight vectors the compiler spills a hundred
      // registers: 2048 x 32768 214 us against 107)
      if (o.q && !KEEP) mine = max_bits(mine, mag_bits(f * g[j](e)));
      else if (CODES && KEEP) top[j] = max_mag(top[j], f * g[j](e));
    }
    if (KEEP) mine = max_bits(mine, mag_bits(top[j]));
    if (TWICE && rv.skip != 0) {
      ss = before;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float f = rv.mine(e) ? elem_f32(h[j].v[e]) : 0.f;
        ss = __builtin_fmaf(f, f, ss);
      }
    }
  }
  ss = fold<Add>(ss);
  uint32_t hi = o.q ? fold<Max>(mine) : 0u;
  if constexpr (!WAVE) {
    __shared__ float sums[16];
    __shared__ uint32_t maxs[16];
    if (lane == 0) {
      sums[wave] = ss;
      maxs[wave] = hi;
    }
    __syncthreads();
    ss = fold_waves<Add>(sums, tpr / 64, 0.f);
    hi = fold_waves<Max>(maxs, tpr / 64, 0u);
  }
  hi = uniform(hi);
  float lo = 0.f;
  if constexpr (WIDE) {
    // of the values that share the row's largest p (one, as a rule), the largest
    // left-over: looked for where a vector has such a value (16384 x 1792 fp16 23.0
    // us; in all of a thread's vectors 28.1; carried along with every maximum more).
    if (o.q) {
      float r = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < N; ++j) forget<In, E>(h[j]);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if ((KEEP ? mag_bits(top[j]) : mine) != hi) continue;
        if (!KEEP) g[j].load(gamma + Vec(j * tpr + tid, K).at);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float f = elem_f32(h[j].v[e]), w = g[j](e), p = f * w;
          if (mag_bits(p) == hi) r = __builtin_fmaxf(r, left_over(f, w, p));
        }
      }
      lo = fold<Max>(r);
      if constexpr (!WAVE) {
        __shared__ float rests[16];
        if (lane == 0) rests[wave] = lo;
        __syncthreads();
        lo = fold_waves<Max>(rests, tpr / 64, -__builtin_inff());
      }
    }
  }
  double amax = (double)__uint_as_float(hi) + (double)lo;
  if constexpr (kMayVanish<In, GT>) {
    if (o.q && tiny_bits(hi)) {                      // the same for the whole row
      double m = 0.0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        forget<In, E>(h[j]);
        if (!KEEP) g[j].load(gamma + Vec(j * tpr + tid, K).at);
#pragma unroll
        for (int e = 0; e < E; ++e)
          m = __builtin_fmax(m, __builtin_fabs((double)elem_f32(h[j].v[e]) * (double)g[j](e)));
      }
      amax = wave_max(m);
      if constexpr (!WAVE) {
        __shared__ double tops[16];
        if (lane == 0) tops[wave] = amax;
        __syncthreads();
        amax = tops[0];
        for (int w = 1; w < tpr / 64; ++w) amax = __builtin_fmax(amax, tops[w]);
      }
    }
  }
  const float rstd = uniform(o.norm ? 1.0f / sqrtf(ss / (float)K + eps) : 1.0f);
  const RowCodes codes(hi, uniform(amax));
  if (tid == 0) {
    if (o.rstd) o.rstd[row] = rstd;
    if (o.q) o.qs[row] = codes.scale(rstd);
  }
  if (late) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const Vec rv(j * tpr + tid, K);
      if (rv.skip < E) store_pack<In, E>((In*)o.H + row * K + rv.at, h[j]);
    }
  }
  if (!o.Y && !o.q) return;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const Vec rv(j * tpr + tid, K);
    forget<In, E>(h[j]);
    if (!KEEP) g[j].load(gamma + rv.at);
    if (o.Y) {
      Pack<In, E> y;
#pragma unroll
      for (int e = 0; e < E; ++e) y.v[e] = elem_of<In>(elem_f32(h[j].v[e]) * rstd * g[j](e));
      put_vec<In, E, RAGGED, TWICE>((In*)o.Y + row * K, rv, y);
    }
    if constexpr (!std::is_same<In, float>::value) {
      if (!o.q) continue;
      Pack<int8_t, E> c;
      auto exact = [&](int e) { return (double)elem_f32(h[j].v[e]) * (double)g[j](e); };
      bool slow = true;
      if constexpr (E % 4 == 0) {
        slow = codes.bad || codes.tiny;
        if (!slow) {
#pragma unroll
          for (int w = 0; w < E / 4; ++w) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = elem_f32(h[j].v[4 * w + i]) * g[j](4 * w + i);
            const uint32_t b = codes.four(p, [&](int i) { return exact(4 * w + i); });
#pragma unroll
            for (int i = 0; i < 4; ++i) c.v[4 * w + i] = (int8_t)(b >> (8 * i));
          }
        }
      }
      if (slow) {
#pragma unroll 1
        for (int e = 0; e < E; ++e) {
          // (an indexed element would put the vectors in memory: pick it by compares)
          double u = 0.0;
#pragma unroll
          for (int i = 0; i < E; ++i) u = i == e ? exact(i) : u;
          const int8_t k = (int8_t)codes.code(u);
#pragma unroll
          for (int i = 0; i < E; ++i) c.v[i] = i == e ? k : c.v[i];
        }
      }
      put_vec<int8_t, E, RAGGED, TWICE>(o.q + row * K, rv, c);
    }
  }
}

template <typename GT>
__device__ __forceinline__ float gamma_at(const GT* gamma, int64_t k) {
  if constexpr (kHasGamma<GT>) return elem_f32(gamma[k]);
  return 1.f;
}

// Rows too long for registers: two walks over the row.  The second reads h back
// from H where it was written (X or the residual may be H itself).
template <typename In, typename GT>
__global__ __launch_bounds__(1024) void rms_long_kernel(const In* X, const In* res, const GT* gamma, int64_t K,
                                                        float eps, NormOut o) {
  __shared__ float sums[16], rests[16];
  __shared__ uint32_t maxs[16];
  __shared__ double tops[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x, base = row * K;
  In* H = (In*)o.H;
  auto sum_at = [&](int64_t k) -> In {
    return res ? elem_of<In>(elem_f32(X[base + k]) + elem_f32(res[base + k])) : X[base + k];
  };
  float ss = 0.f;
  uint32_t mine = 0u;
  for (int64_t k = threadIdx.x; k < K; k += 1024) {
    const In h = sum_at(k);
    const float f = elem_f32(h);
    ss = __builtin_fmaf(f, f, ss);
    mine = max_bits(mine, mag_bits(f * gamma_at(gamma, k)));
    if (H) H[base + k] = h;
  }
  ss = fold<Add>(ss);
  uint32_t hi = fold<Max>(mine);
  if (lane == 0) {
    sums[wave] = ss;
    maxs[wave] = hi;
  }
  __syncthreads();
  ss = fold_waves<Add>(sums, 16, 0.f);
  hi = fold_waves<Max>(maxs, 16, 0u);
  float lo = 0.f;
  if constexpr (kWide<In, GT>) {
    float r = -__builtin_inff();
    if (mine == hi) {
      for (int64_t k = threadIdx.x; k < K; k += 1024) {
        const float f = elem_f32(H ? H[base + k] : sum_at(k)), w = gamma_at(gamma, k), p = f * w;
        if (mag_bits(p) == hi) r = __builtin_fmaxf(r, left_over(f, w, p));
      }
    }
    r = fold<Max>(r);
    if (lane == 0) rests[wave] = r;
    __syncthreads();
    lo = fold_waves<Max>(rests, 16, -__builtin_inff());
  }
  double amax = (double)__uint_as_float(hi) + (double)lo;
  if constexpr (kMayVanish<In, GT>) {
    if (o.q && tiny_bits(hi)) {                      // the same for the whole row
      double m = 0.0;
      for (int64_t k = threadIdx.x; k < K; k += 1024)
        m = __builtin_fmax(m, __builtin_fabs((double)elem_f32(H ? H[base + k] : sum_at(k)) * (double)gamma_at(gamma, k)));
      m = wave_max(m);
      if (lane == 0) tops[wave] = m;
      __syncthreads();
      amax = tops[0];
      for (int w = 1; w < 16; ++w) amax = __builtin_fmax(amax, tops[w]);
    }
  }
  const float rstd = o.norm ? 1.0f / sqrtf(ss / (float)K + eps) : 1.0f;
  const RowCodes codes(hi, amax);
  if (threadIdx.x == 0) {
    if (o.rstd) o.rstd[row] = rstd;
    if (o.q) o.qs[row] = codes.scale(rstd);
  }
  if (!o.Y && !o.q) return;
  for (int64_t k = threadIdx.x; k < K; k += 1024) {   // each element by the thread that made it
    const float f = elem_f32(H ? H[base + k] : sum_at(k));
    const float g = gamma_at(gamma, k);
    if (o.q) o.q[base + k] = (int8_t)codes.code((double)f * (double)g);
    if (o.Y) ((In*)o.Y)[base + k] = elem_of<In>(f * rstd * g);
  }
}

template <typename In, typename GT, int E, int N, bool WAVE>
void rms_rows(const In* X, const In* res, const GT* gamma, int64_t T, int64_t K, float eps, const NormOut& o,
              hipStream_t s) {
  const int threads = WAVE ? 256 : (int)(cdiv(cdiv(cdiv(K, E), N), 64) * 64);
  const unsigned blocks = (unsigned)(WAVE ? cdiv(T, 4) : T);
  if (K % E == 0) rms_row_kernel<In, GT, E, N, WAVE, false><<<blocks, threads, 0, s>>>(X, res, gamma, T, (int)K, eps, o);
  else rms_row_kernel<In, GT, E, N, WAVE, true><<<blocks, threads, 0, s>>>(X, res, gamma, T, (int)K, eps, o);
}

template <typename In, typename GT>
hipError_t rms_launch(const void* X_, const void* res_, const void* gamma_, int64_t T, int64_t K, float eps,
                      const NormOut& o, hipStream_t s) {
  constexpr int E = vec_elems<In>();
  const In *X = (const In*)X_, *res = (const In*)res_;
  const GT* gamma = (const GT*)gamma_;
  const int64_t v = cdiv(K, E);
  if (K < E) rms_row_kernel<In, GT, 1, 1, true, false><<<(unsigned)cdiv(T, 4), 256, 0, s>>>(X, res, gamma, T, (int)K, eps, o);
  else if (v <= 64) rms_rows<In, GT, E, 1, true>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 128) rms_rows<In, GT, E, 2, true>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 256) rms_rows<In, GT, E, 4, true>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 1024) rms_rows<In, GT, E, 2, false>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 3 * 1024) rms_rows<In, GT, E, 3, false>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 8192) rms_rows<In, GT, E, 8, false>(X, res, gamma, T, K, eps, o, s);
  else rms_long_kernel<In, GT><<<(unsigned)T, 1024, 0, s>>>(X, res, gamma, K, eps, o);
  return hipGetLastError();
}

// ---------------------------------------------------------------- gradient

constexpr int kBwdWaves = 8;                            // waves of a block whose waves take a row each
constexpr int kBwdBlocks = 512;                         // partial rows of dgamma, at most
constexpr int64_t kBwdMaxVecs = 4096;                   // vectors of a row kept in registers (1024 threads x 4)

// Groups of tokens with a partial row of dgamma each, a function of the sizes
// alone (the workspace's size); fewer for rows past 2^25 / kBwdBlocks columns,
// so that the workspace stays below 128 MiB up to a million columns.
int64_t bwd_groups(int64_t T, int64_t K) {
  int64_t most = (int64_t(1) << 25) / (K < 1 ? 1 : K);
  most = most < 8 ? 8 : most > kBwdBlocks ? kBwdBlocks : most;
  return T < most ? T : most;
}

// A block (WAVE: each of its eight waves) takes every gridDim-th row and keeps its
// columns, so dgamma's partial sums stay in registers.  The next row's loads are
// issued before this row's sum is taken.
template <typename In, typename GT, int E, int N, bool WAVE, bool RAGGED>
__global__ __launch_bounds__(N == 4 ? 1024 : 512, N == 4 ? 4 : 2) void rms_bwd_kernel(const In* dY, const In* __restrict__ H,
                                                                   const float* __restrict__ rstd, const GT* gamma,
                                                                   const In* dH, int64_t T, int K, In* dX,
                                                                   float* __restrict__ part) {
  typedef RowVec<E, RAGGED> Vec;
  constexpr bool AHEAD = N < 4;                       // four vectors a thread: the registers hold one row, no gamma
  // As in the forward: elements of two vectors worked on and stored twice (one by
  // one where dX is dH, which another thread may not have loaded yet); 4096 x 3333
  // bf16 32.1 us, once only 34.7.
  constexpr bool TWICE = RAGGED && AHEAD && N * E <= 16;
  const bool once = !TWICE || dX == dH;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tid = WAVE ? lane : (int)threadIdx.x, tpr = WAVE ? 64 : (int)blockDim.x;
  const int64_t first = WAVE ? (int64_t)blockIdx.x * kBwdWaves + wave : (int64_t)blockIdx.x;
  const int64_t step = WAVE ? (int64_t)gridDim.x * kBwdWaves : (int64_t)gridDim.x;
  const float inv_k = 1.0f / (float)K;
  const In* dHr = dH ? dH : dY;                       // no dH: dY's first vector, and not used
  float dg[N][E];
  Gamma<GT, E> g[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    if (AHEAD) g[j].load(gamma + Vec(j * tpr + tid, K).at);
#pragma unroll
    for (int e = 0; e < E; ++e) dg[j][e] = 0.f;
  }
  struct Row {
    Pack<In, E> dy[N], h[N], r[N];
    float rs;
  };
  auto load = [&](Row& w, int64_t row) {
    const int64_t base = row * K;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int at = Vec(j * tpr + tid, K).at;
      w.dy[j] = load_pack<In, E>(dY + base + at);
      w.h[j] = load_pack<In, E>(H + base + at);
      if (AHEAD) w.r[j] = load_pack<In, E>(dHr + (dH ? base + at : 0));
    }
    w.rs = rstd[row];
  };
  __shared__ float sums[2][16];
  int slot = 0;
  Row now, next;
  if (first < T) load(now, first);
  for (int64_t row = first; row < T; row += step) {
    const int64_t base = row * K;
    if (AHEAD) load(next, row + step < T ? row + step : row);
    __builtin_amdgcn_sched_barrier(0);
    const float rs = now.rs;
    float c = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const Vec rv(j * tpr + tid, K);
      if (!AHEAD) g[j].load(gamma + rv.at);
      if constexpr (!TWICE) {
        drop_foreign<In, E, RAGGED>(now.dy[j], rv);
        drop_foreign<In, E, RAGGED>(now.h[j], rv);
      }
      const float before = c;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float p = elem_f32(now.dy[j].v[e]) * (elem_f32(now.h[j].v[e]) * rs);
        dg[j][e] += p;                               // (a foreign element's sum is not stored)
        // (a foreign element's gamma need not be finite)
        c = __builtin_fmaf(p, TWICE || rv.mine(e) ? g[j](e) : 0.f, c);
      }
      if (TWICE && rv.skip != 0) {
        c = before;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float p = elem_f32(now.dy[j].v[e]) * (elem_f32(now.h[j].v[e]) * rs);
          c = __builtin_fmaf(rv.mine(e) ? p : 0.f, rv.mine(e) ? g[j](e) : 0.f, c);
        }
      }
    }
    if (dX) {
      c = fold<Add>(c);
      if constexpr (!WAVE) {
        // two slots in turn: a row's sums are read before the slot is written again
        if (lane == 0) sums[slot][wave] = c;
        __syncthreads();
        if constexpr (AHEAD) {
          c = fold_waves<Add>(sums[slot], tpr / 64, 0.f);
        } else {                                     // (fewer registers spilled: 512 x 20480 36 us against 43)
          c = sums[slot][0];
          for (int w = 1; w < tpr / 64; ++w) c += sums[slot][w];
        }
        slot ^= 1;
      }
      c *= inv_k;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const Vec rv(j * tpr + tid, K);
        if (!AHEAD) {
          now.r[j] = load_pack<In, E>(dHr + (dH ? base + rv.at : 0));
          g[j].load(gamma + rv.at);
        }
        forget<In, E>(now.dy[j]);
        forget<In, E>(now.h[j]);
        Pack<In, E> out;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float a = elem_f32(now.dy[j].v[e]) * g[j](e), xh = elem_f32(now.h[j].v[e]) * rs;
          const float d = rs * (a - xh * c);
          out.v[e] = elem_of<In>(dH ? d + elem_f32(now.r[j].v[e]) : d);
        }
        if (once) store_vec<In, E, RAGGED>(dX + base, rv, out);
        else if (rv.skip < E) store_pack<In, E>(dX + base + rv.at, out);
      }
    }
    if (AHEAD) now = next;
    else if (row + step < T) load(now, row + step);
  }
  if (!part) return;
  float* dst = part + (int64_t)blockIdx.x * K;
  if constexpr (WAVE) {
    // the waves' sums side by side in LDS, added in wave order
    __shared__ float all[kBwdWaves][N * E * 64];
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) all[wave][(j * E + e) * 64 + lane] = dg[j][e];
    __syncthreads();
    for (int at = threadIdx.x; at < N * E * 64; at += 64 * kBwdWaves) {
      const Vec rv((at / (64 * E)) * 64 + at % 64, K);
      const int e = at / 64 % E;
      if (!rv.mine(e)) continue;
      float s = all[0][at];
#pragma unroll
      for (int w = 1; w < kBwdWaves; ++w) s += all[w][at];
      dst[rv.at + e] = s;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const Vec rv(j * tpr + tid, K);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (rv.mine(e)) dst[rv.at + e] = dg[j][e];
    }
  }
}

// Rows too long for registers: dgamma's partial rows column by column (run
// before dX is written, which may be dY), then dX in two walks of each row.
template <typename In>
__global__ __launch_bounds__(256) void rms_dgamma_long_kernel(const In* __restrict__ dY, const In* __restrict__ H,
                                                              const float* __restrict__ rstd, int64_t T, int64_t K,
                                                              float* __restrict__ part) {
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (k >= K) return;
  float s = 0.f;
  for (int64_t row = blockIdx.y; row < T; row += gridDim.y)
    s += elem_f32(dY[row * K + k]) * (elem_f32(H[row * K + k]) * rstd[row]);
  part[(int64_t)blockIdx.y * K + k] = s;
}

template <typename In, typename GT>
__global__ __launch_bounds__(1024) void rms_dx_long_kernel(const In* dY, const In* __restrict__ H,
                                                           const float* __restrict__ rstd, const GT* gamma,
                                                           const In* dH, int64_t K, In* dX) {
  __shared__ float sums[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x, base = row * K;
  const float rs = rstd[row];
  float c = 0.f;
  for (int64_t k = threadIdx.x; k < K; k += 1024)
    c += elem_f32(dY[base + k]) * gamma_at(gamma, k) * (elem_f32(H[base + k]) * rs);
  c = fold<Add>(c);
  if (lane == 0) sums[wave] = c;
  __syncthreads();
  c = fold_waves<Add>(sums, 16, 0.f);
  c /= (float)K;
  for (int64_t k = threadIdx.x; k < K; k += 1024) {
    const float a = elem_f32(dY[base + k]) * gamma_at(gamma, k);
    float d = rs * (a - elem_f32(H[base + k]) * rs * c);
    if (dH) d += elem_f32(dH[base + k]);
    dX[base + k] = elem_of<In>(d);
  }
}

// dgamma[k] = sum over the groups, in a fixed order: 32 columns a block, 32 threads
// a column with a thirty-second of the rows each (sixteen loads in flight), their
// sums added in order.
template <typename GT>
__global__ __launch_bounds__(1024) void rms_dgamma_reduce_kernel(const float* __restrict__ part, int groups,
                                                                 int64_t K, int accumulate, GT* __restrict__ out) {
  __shared__ float sums[32][33];
  const int c = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t k = (int64_t)blockIdx.x * 32 + c, kc = k < K ? k : K - 1;
  const int per = (groups + 31) / 32, g0 = y * per, g1 = g0 + per < groups ? g0 + per : groups;
  float s = 0.f;
  for (int g = g0; g < g1; g += 16) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = part[(int64_t)(g + i < g1 ? g + i : g) * K + kc];
#pragma unroll
    for (int i = 0; i < 16; ++i) s += g + i < g1 ? v[i] : 0.f;
  }
  sums[y][c] = s;
  __syncthreads();
  if (y == 0 && k < K) {
    float d = accumulate ? elem_f32(out[k]) : 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) d += sums[w][c];
    out[k] = elem_of<GT>(d);
  }
}

template <typename In, typename GT, int E, int N, bool WAVE>
int64_t bwd_rows(const In* dY, const In* H, const float* rstd, const GT* gamma, const In* dH, int64_t T, int64_t K,
                 In* dX, float* part, hipStream_t s) {
  const int threads = WAVE ? 64 * kBwdWaves : (int)(cdiv(cdiv(cdiv(K, E), N), 64) * 64);
  // a block of three or four vectors a thread leaves no room for a second one on
  // its compute unit: one round of 256 blocks (8192 x 9216: 119 us against 128
  // with 512).  Narrower rows take 512 (4096 x 2304: 20.4 us against 25.5).
  // Rows of one wave: 256 blocks of eight waves.
  int64_t groups = bwd_groups(WAVE ? cdiv(T, kBwdWaves) : T, K);
  if ((WAVE || N >= 3) && groups > 256) groups = 256;
  if (K % E == 0)
    rms_bwd_kernel<In, GT, E, N, WAVE, false><<<(unsigned)groups, threads, 0, s>>>(dY, H, rstd, gamma, dH, T, (int)K,
                                                                                   dX, part);
  else
    rms_bwd_kernel<In, GT, E, N, WAVE, true><<<(unsigned)groups, threads, 0, s>>>(dY, H, rstd, gamma, dH, T, (int)K,
                                                                                  dX, part);
  return groups;
}

// DG: dgamma's type (gamma's, which may not be there)
template <typename In, typename GT, typename DG>
hipError_t bwd_launch(const void* dY_, const void* H_, const float* rstd, const void* gamma_, const void* dH_,
                      int64_t T, int64_t K, void* dX_, void* dgamma, int accumulate, float* part, hipStream_t s) {
  constexpr int E = vec_elems<In>();
  const In *dY = (const In*)dY_, *H = (const In*)H_, *dH = (const In*)dH_;
  const GT* gamma = (const GT*)gamma_;
  In* dX = (In*)dX_;
  if (!dgamma) part = nullptr;
  int64_t groups = 0;
  const int64_t v = cdiv(K, E);
  if (T == 0) {
  } else if (K < E) {
    groups = bwd_groups(cdiv(T, kBwdWaves), K);
    rms_bwd_kernel<In, GT, 1, 1, true, false><<<(unsigned)groups, 64 * kBwdWaves, 0, s>>>(dY, H, rstd, gamma, dH, T, (int)K,
                                                                                     dX, part);
  } else if (v <= 64) groups = bwd_rows<In, GT, E, 1, true>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 128) groups = bwd_rows<In, GT, E, 2, true>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 512) groups = bwd_rows<In, GT, E, 1, false>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 1536) groups = bwd_rows<In, GT, E, 3, false>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= kBwdMaxVecs) groups = bwd_rows<In, GT, E, 4, false>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else {
    groups = bwd_groups(T, K);
    if (dgamma)
      rms_dgamma_long_kernel<In><<<dim3((unsigned)cdiv(K, 256), (unsigned)groups), 256, 0, s>>>(dY, H, rstd, T, K,
                                                                                              part);
    if (dX) rms_dx_long_kernel<In, GT><<<(unsigned)T, 1024, 0, s>>>(dY, H, rstd, gamma, dH, K, dX);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dgamma) return e;
  rms_dgamma_reduce_kernel<DG><<<(unsigned)cdiv(K, 32), 1024, 0, s>>>(part, (int)groups, K, accumulate, (DG*)dgamma);
  return hipGetLastError();
}

// Rows of one launch: a grid ends below 2^32 threads, a row takes 1024 at most.
constexpr int64_t kLaunchRows = int64_t(1) << 21;

template <typename In>
hipError_t rms_any(const void* X_, const void* res_, bool wide, const void* gamma, int64_t T, int64_t K, float eps,
                   const NormOut& all, hipStream_t s) {
  for (int64_t t = 0; t < T; t += kLaunchRows) {
    const int64_t n = T - t < kLaunchRows ? T - t : kLaunchRows, at = t * K;
    const In *X = (const In*)X_ + at, *res = res_ ? (const In*)res_ + at : nullptr;
    const NormOut o{all.H ? (In*)all.H + at : nullptr, all.Y ? (In*)all.Y + at : nullptr, all.q ? all.q + at : nullptr,
                    all.q ? all.qs + t : nullptr, all.rstd ? all.rstd + t : nullptr, all.norm};
    const hipError_t e = !gamma ? rms_launch<In, Ones>(X, res, gamma, n, K, eps, o, s)
                         : wide ? rms_launch<In, float>(X, res, gamma, n, K, eps, o, s)
                                : rms_launch<In, In>(X, res, gamma, n, K, eps, o, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename In>
hipError_t bwd_any(const void* dY, const void* H, const float* rstd, bool wide, const void* gamma, const void* dH,
                   int64_t T, int64_t K, void* dX, void* dgamma, int accumulate, float* part, hipStream_t s) {
  if (!gamma)
    return wide ? bwd_launch<In, Ones, float>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s)
                : bwd_launch<In, Ones, In>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s);
  return wide ? bwd_launch<In, float, float>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s)
              : bwd_launch<In, In, In>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s);
}

}  // namespace

hipError_t launch_rmsnorm(Dt dt, const void* X, const void* res, Dt gamma_dt, const void* gamma, int64_t T, int64_t K,
                          float eps, void* H, void* Y, int8_t* q, float* qs, float* rstd, hipStream_t s) {
  if (T == 0 || K == 0) return hipSuccess;
  const NormOut o{H, Y, q, qs, rstd, true};
  const bool wide = gamma_dt == Dt::F32;
  if (dt == Dt::F32) return rms_any<float>(X, res, wide, gamma, T, K, eps, o, s);
  if (dt == Dt::F16) return rms_any<_Float16>(X, res, wide, gamma, T, K, eps, o, s);
  return rms_any<uint16_t>(X, res, wide, gamma, T, K, eps, o, s);
}

hipError_t launch_quantize_rows_i8(Dt dt, const void* X, int64_t T, int64_t K, int8_t* q, float* scale,
                                   hipStream_t s) {
  if (K == 0) return launch_fill_zero(Dt::F32, scale, T, s);   // rows of no values: the scale of zeros
  if (T == 0) return hipSuccess;
  const NormOut o{nullptr, nullptr, q, scale, nullptr, false};
  return dt == Dt::F16 ? rms_any<_Float16>(X, nullptr, false, nullptr, T, K, 0.f, o, s)
                       : rms_any<uint16_t>(X, nullptr, false, nullptr, T, K, 0.f, o, s);
}

int64_t rmsnorm_bwd_workspace_bytes(int64_t T, int64_t K) { return bwd_groups(T, K) * K * 4; }

hipError_t launch_rmsnorm_bwd(Dt dt, const void* dY, const void* H, const float* rstd, Dt gamma_dt, const void* gamma,
                              const void* dH, int64_t T, int64_t K, void* dX, void* dgamma, int accumulate,
                              void* workspace, hipStream_t s) {
  if (K == 0) return hipSuccess;
  float* part = (float*)workspace;
  const bool wide = gamma_dt == Dt::F32;          // dgamma's type too, so also without a gamma
  if (dt == Dt::F32) return bwd_any<float>(dY, H, rstd, wide, gamma, dH, T, K, dX, dgamma, accumulate, part, s);
  if (dt == Dt::F16) return bwd_any<_Float16>(dY, H, rstd, wide, gamma, dH, T, K, dX, dgamma, accumulate, part, s);
  return bwd_any<uint16_t>(dY, H, rstd, wide, gamma, dH, T, K, dX, dgamma, accumulate, part, s);
}

}  // namespace slope
