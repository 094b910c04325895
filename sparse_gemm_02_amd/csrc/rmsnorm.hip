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
//
// Gradient:  a = dy g,  xh = h rstd,  c = mean(a xh)
//   dx = rstd (a - xh c) + dh,   dg = sum over tokens of dy xh
// The same row layout; a block keeps its columns over many rows, so dg's
// partial sums stay in registers, and a second kernel adds the blocks' rows in
// order.
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "rows8.h"

namespace slope {

namespace {

// Elements per 16-byte access of a format.
template <typename In> constexpr int vec_elems() { return 16 / (int)sizeof(In); }

// Sum of v over the 64 lanes, the same in every lane (fixed order).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
  return v;
}
template <typename U>
__device__ __forceinline__ U wave_max(U v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = max_of(v, __shfl_xor(v, m));
  return v;
}

// The vectors of a row of K >= E elements: vector i holds elements E i .. E i +
// E - 1; the last one, when K is not a multiple of E, is moved back to end at
// K, and its first `skip` elements belong to the vector before it.
template <int E>
struct RowVec {
  int at, skip;
  bool live;
  __device__ __forceinline__ RowVec(int i, int K) {
    const int full = E * i;
    live = full < K;
    const int last = K - E;
    at = live ? (full < last ? full : last) : 0;
    skip = live ? full - at : E;
  }
};

template <typename V, int E>
__device__ __forceinline__ void store_vec(V* row, const RowVec<E>& r, const Pack<V, E>& x) {
  if (!r.live) return;
  if (r.skip == 0) {
    store_pack<V, E>(row + r.at, x);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e >= r.skip) row[r.at + e] = x.v[e];
  }
}

// Products h g whose size sets the codes: exact in fp32 for a 16-bit g, in
// double for an fp32 one.  (fp32 rows have no codes.)
template <typename In, typename GT>
using Prod = typename std::conditional<std::is_same<GT, float>::value && !std::is_same<In, float>::value, double,
                                       float>::type;

struct NormOut {
  void *H, *Y;
  int8_t* q;
  float *qs, *rstd;
  bool norm;                                       // false: codes of x itself
};

// One row per block (WAVE: per wave, four rows a block), N vectors a thread.
template <typename In, typename GT, int E, int N, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void rms_row_kernel(const In* X, const In* res,
                                                                    const GT* __restrict__ gamma, int64_t T, int K,
                                                                    float eps, NormOut o) {
  typedef Prod<In, GT> U;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = WAVE ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;
  if (WAVE && row >= T) return;
  const int tid = WAVE ? lane : (int)threadIdx.x, tpr = WAVE ? 64 : (int)blockDim.x;
  const In* x = X + row * K;
  Pack<In, E> h[N];
#pragma unroll
  for (int j = 0; j < N; ++j) h[j] = load_pack<In, E>(x + RowVec<E>(j * tpr + tid, K).at);
  if (res) {
    const In* rr = res + row * K;
    Pack<In, E> r[N];
#pragma unroll
    for (int j = 0; j < N; ++j) r[j] = load_pack<In, E>(rr + RowVec<E>(j * tpr + tid, K).at);
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) h[j].v[e] = elem_of<In>(elem_f32(h[j].v[e]) + elem_f32(r[j].v[e]));
  }
  float ss = 0.f;
  U am = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const RowVec<E> rv(j * tpr + tid, K);
    Pack<GT, E> g;
    if (gamma) g = load_pack<GT, E>(gamma + rv.at);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float f = e >= rv.skip ? elem_f32(h[j].v[e]) : 0.f;
      ss = __builtin_fmaf(f, f, ss);
      if (o.q) {
        const U u = gamma ? (U)f * (U)elem_f32(g.v[e]) : (U)f;
        am = max_of(am, e >= rv.skip ? finite_or_inf(u) : (U)0);
      }
    }
    if (o.H) store_vec<In, E>((In*)o.H + row * K, rv, h[j]);
  }
  ss = wave_sum(ss);
  if (o.q) am = wave_max(am);
  if constexpr (!WAVE) {
    __shared__ float sums[16];
    __shared__ U maxs[16];
    if (lane == 0) {
      sums[wave] = ss;
      maxs[wave] = am;
    }
    __syncthreads();
    ss = sums[0];
    am = maxs[0];
    for (int w = 1; w < tpr / 64; ++w) {
      ss += sums[w];
      am = max_of(am, maxs[w]);
    }
  }
  const float rstd = o.norm ? 1.0f / sqrtf(ss / (float)K + eps) : 1.0f;
  const RowCodes<U> codes(am);
  if (tid == 0) {
    if (o.rstd) o.rstd[row] = rstd;
    if (o.q) o.qs[row] = codes.scale() * rstd;
  }
  if (!o.Y && !o.q) return;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const RowVec<E> rv(j * tpr + tid, K);
    Pack<GT, E> g;
    if (gamma) g = load_pack<GT, E>(gamma + rv.at);
    if (o.Y) {
      Pack<In, E> y;
#pragma unroll
      for (int e = 0; e < E; ++e)
        y.v[e] = elem_of<In>(elem_f32(h[j].v[e]) * rstd * (gamma ? elem_f32(g.v[e]) : 1.f));
      store_vec<In, E>((In*)o.Y + row * K, rv, y);
    }
    if (o.q) {
      Pack<int8_t, E> c;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const U f = (U)elem_f32(h[j].v[e]);
        c.v[e] = (int8_t)codes.code(gamma ? f * (U)elem_f32(g.v[e]) : f);
      }
      store_vec<int8_t, E>(o.q + row * K, rv, c);
    }
  }
}

// Rows too long for registers: two walks over the row.  The second reads h back
// from H where it was written (X or the residual may be H itself).
template <typename In, typename GT>
__global__ __launch_bounds__(1024) void rms_long_kernel(const In* X, const In* res, const GT* __restrict__ gamma,
                                                        int64_t K, float eps, NormOut o) {
  typedef Prod<In, GT> U;
  __shared__ float sums[16];
  __shared__ U maxs[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x, base = row * K;
  In* H = (In*)o.H;
  auto sum_at = [&](int64_t k) -> In {
    return res ? elem_of<In>(elem_f32(X[base + k]) + elem_f32(res[base + k])) : X[base + k];
  };
  float ss = 0.f;
  U am = 0;
  for (int64_t k = threadIdx.x; k < K; k += 1024) {
    const In h = sum_at(k);
    const float f = elem_f32(h);
    ss = __builtin_fmaf(f, f, ss);
    if (o.q) am = max_of(am, finite_or_inf(gamma ? (U)f * (U)elem_f32(gamma[k]) : (U)f));
    if (H) H[base + k] = h;
  }
  ss = wave_sum(ss);
  am = wave_max(am);
  if (lane == 0) {
    sums[wave] = ss;
    maxs[wave] = am;
  }
  __syncthreads();
  ss = sums[0];
  am = maxs[0];
  for (int w = 1; w < 16; ++w) {
    ss += sums[w];
    am = max_of(am, maxs[w]);
  }
  const float rstd = o.norm ? 1.0f / sqrtf(ss / (float)K + eps) : 1.0f;
  const RowCodes<U> codes(am);
  if (threadIdx.x == 0) {
    if (o.rstd) o.rstd[row] = rstd;
    if (o.q) o.qs[row] = codes.scale() * rstd;
  }
  if (!o.Y && !o.q) return;
  for (int64_t k = threadIdx.x; k < K; k += 1024) {   // each element by the thread that made it
    const float f = elem_f32(H ? H[base + k] : sum_at(k));
    const float g = gamma ? elem_f32(gamma[k]) : 1.f;
    if (o.q) o.q[base + k] = (int8_t)codes.code((U)f * (U)g);
    if (o.Y) ((In*)o.Y)[base + k] = elem_of<In>(f * rstd * g);
  }
}

template <typename In, typename GT, int E, int N>
void rms_block(const In* X, const In* res, const GT* gamma, int64_t T, int64_t K, float eps, const NormOut& o,
               hipStream_t s) {
  const int threads = (int)(cdiv(cdiv(cdiv(K, E), N), 64) * 64);
  rms_row_kernel<In, GT, E, N, false><<<(unsigned)T, threads, 0, s>>>(X, res, gamma, T, (int)K, eps, o);
}
template <typename In, typename GT, int E, int N>
void rms_wave(const In* X, const In* res, const GT* gamma, int64_t T, int64_t K, float eps, const NormOut& o,
              hipStream_t s) {
  rms_row_kernel<In, GT, E, N, true><<<(unsigned)cdiv(T, 4), 256, 0, s>>>(X, res, gamma, T, (int)K, eps, o);
}

template <typename In, typename GT>
hipError_t rms_launch(const void* X_, const void* res_, const void* gamma_, int64_t T, int64_t K, float eps,
                      const NormOut& o, hipStream_t s) {
  constexpr int E = vec_elems<In>();
  const In *X = (const In*)X_, *res = (const In*)res_;
  const GT* gamma = (const GT*)gamma_;
  const int64_t v = cdiv(K, E);
  if (K < E) rms_wave<In, GT, 1, 1>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 64) rms_wave<In, GT, E, 1>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 128) rms_wave<In, GT, E, 2>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 256) rms_wave<In, GT, E, 4>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 512) rms_block<In, GT, E, 1>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 1024) rms_block<In, GT, E, 2>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 1536) rms_block<In, GT, E, 3>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 2048) rms_block<In, GT, E, 4>(X, res, gamma, T, K, eps, o, s);
  else if (v <= 8192) rms_block<In, GT, E, 8>(X, res, gamma, T, K, eps, o, s);
  else rms_long_kernel<In, GT><<<(unsigned)T, 1024, 0, s>>>(X, res, gamma, K, eps, o);
  return hipGetLastError();
}

// ---------------------------------------------------------------- gradient

constexpr int kBwdWaveBlocks = 512, kBwdBlocks = 768;   // partial rows of dgamma, at most
constexpr int64_t kBwdMaxVecs = 4096;                   // vectors of a row kept in registers (512 threads x 8)

// Groups of tokens with a partial row of dgamma each, a function of the sizes
// alone (the workspace's size); fewer for rows past 2^25 / kBwdBlocks columns,
// so that the workspace stays below 128 MiB up to a million columns.
int64_t bwd_groups(int64_t T, int64_t K) {
  int64_t most = (int64_t(1) << 25) / (K < 1 ? 1 : K);
  most = most < 8 ? 8 : most > kBwdBlocks ? kBwdBlocks : most;
  return T < most ? T : most;
}

template <typename In, typename GT, int E, int N, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 512) void rms_bwd_kernel(const In* dY, const In* __restrict__ H,
                                                                   const float* __restrict__ rstd,
                                                                   const GT* __restrict__ gamma, const In* dH,
                                                                   int64_t T, int K, In* dX, float* __restrict__ part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int tid = WAVE ? lane : (int)threadIdx.x, tpr = WAVE ? 64 : (int)blockDim.x;
  const int64_t first = WAVE ? (int64_t)blockIdx.x * 4 + wave : (int64_t)blockIdx.x;
  const int64_t step = WAVE ? (int64_t)gridDim.x * 4 : (int64_t)gridDim.x;
  const float inv_k = 1.0f / (float)K;
  float dg[N][E];
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) dg[j][e] = 0.f;
  __shared__ float sums[2][8];
  int slot = 0;
  for (int64_t row = first; row < T; row += step) {
    const int64_t base = row * K;
    Pack<In, E> dy[N], h[N], r[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const RowVec<E> rv(j * tpr + tid, K);
      dy[j] = load_pack<In, E>(dY + base + rv.at);
      h[j] = load_pack<In, E>(H + base + rv.at);
      if (dH) r[j] = load_pack<In, E>(dH + base + rv.at);
    }
    const float rs = rstd[row];
    float c = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const RowVec<E> rv(j * tpr + tid, K);
      Pack<GT, E> g;
      if (gamma) g = load_pack<GT, E>(gamma + rv.at);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = e >= rv.skip ? elem_f32(dy[j].v[e]) : 0.f;
        const float xh = e >= rv.skip ? elem_f32(h[j].v[e]) * rs : 0.f;
        const float p = d * xh;
        dg[j][e] += p;
        c = __builtin_fmaf(p, gamma ? elem_f32(g.v[e]) : 1.f, c);
      }
    }
    if (!dX) continue;
    c = wave_sum(c);
    if constexpr (!WAVE) {
      // two slots in turn: a row's sums are read before the slot is written again
      if (lane == 0) sums[slot][wave] = c;
      __syncthreads();
      c = sums[slot][0];
      for (int w = 1; w < tpr / 64; ++w) c += sums[slot][w];
      slot ^= 1;
    }
    c *= inv_k;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const RowVec<E> rv(j * tpr + tid, K);
      Pack<GT, E> g;
      if (gamma) g = load_pack<GT, E>(gamma + rv.at);
      Pack<In, E> out;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float a = elem_f32(dy[j].v[e]) * (gamma ? elem_f32(g.v[e]) : 1.f);
        const float xh = elem_f32(h[j].v[e]) * rs;
        float d = rs * (a - xh * c);
        if (dH) d += elem_f32(r[j].v[e]);
        out.v[e] = elem_of<In>(d);
      }
      store_vec<In, E>(dX + base, rv, out);
    }
  }
  if (!part) return;
  float* dst = part + (int64_t)blockIdx.x * K;
  if constexpr (!WAVE) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const RowVec<E> rv(j * tpr + tid, K);
      if (!rv.live) continue;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e >= rv.skip) dst[rv.at + e] = dg[j][e];
    }
  } else {
    // the four waves' sums, added in wave order
    __shared__ float all[N * E * 64];
    for (int w = 0; w < 4; ++w) {
      if (wave == w) {
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int at = (j * E + e) * 64 + lane;
            all[at] = w == 0 ? dg[j][e] : all[at] + dg[j][e];
          }
      }
      __syncthreads();
    }
    if (wave == 0) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const RowVec<E> rv(j * 64 + lane, K);
        if (!rv.live) continue;
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (e >= rv.skip) dst[rv.at + e] = all[(j * E + e) * 64 + lane];
      }
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
                                                           const float* __restrict__ rstd,
                                                           const GT* __restrict__ gamma, const In* dH, int64_t K,
                                                           In* dX) {
  __shared__ float sums[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x, base = row * K;
  const float rs = rstd[row];
  float c = 0.f;
  for (int64_t k = threadIdx.x; k < K; k += 1024)
    c += elem_f32(dY[base + k]) * (gamma ? elem_f32(gamma[k]) : 1.f) * (elem_f32(H[base + k]) * rs);
  c = wave_sum(c);
  if (lane == 0) sums[wave] = c;
  __syncthreads();
  c = sums[0];
  for (int w = 1; w < 16; ++w) c += sums[w];
  c /= (float)K;
  for (int64_t k = threadIdx.x; k < K; k += 1024) {
    const float a = elem_f32(dY[base + k]) * (gamma ? elem_f32(gamma[k]) : 1.f);
    float d = rs * (a - elem_f32(H[base + k]) * rs * c);
    if (dH) d += elem_f32(dH[base + k]);
    dX[base + k] = elem_of<In>(d);
  }
}

// dgamma[k] = sum over the groups, in a fixed order: 16 waves take a sixteenth
// of the rows each for the block's 64 columns, and the 16 sums are added in
// wave order.
template <typename GT>
__global__ __launch_bounds__(1024) void rms_dgamma_reduce_kernel(const float* __restrict__ part, int groups,
                                                                 int64_t K, int accumulate, GT* __restrict__ out) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + lane, kc = k < K ? k : K - 1;
  const int per = (groups + 15) / 16, g0 = wave * per, g1 = g0 + per < groups ? g0 + per : groups;
  float s = 0.f;
  for (int g = g0; g < g1; g += 8) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[(int64_t)(g + i < g1 ? g + i : g) * K + kc];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += g + i < g1 ? v[i] : 0.f;
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && k < K) {
    float d = accumulate ? elem_f32(out[k]) : 0.f;
    for (int w = 0; w < 16; ++w) d += sums[w][lane];
    out[k] = elem_of<GT>(d);
  }
}

template <typename In, typename GT, int E, int N>
int64_t bwd_block(const In* dY, const In* H, const float* rstd, const GT* gamma, const In* dH, int64_t T, int64_t K,
                  In* dX, float* part, hipStream_t s) {
  const int threads = (int)(cdiv(cdiv(cdiv(K, E), N), 64) * 64);
  const int64_t groups = bwd_groups(T, K);
  rms_bwd_kernel<In, GT, E, N, false><<<(unsigned)groups, threads, 0, s>>>(dY, H, rstd, gamma, dH, T, (int)K, dX,
                                                                            part);
  return groups;
}
template <typename In, typename GT, int E, int N>
int64_t bwd_wave(const In* dY, const In* H, const float* rstd, const GT* gamma, const In* dH, int64_t T, int64_t K,
                 In* dX, float* part, hipStream_t s) {
  const int64_t need = cdiv(T, 4), groups = need < kBwdWaveBlocks ? need : kBwdWaveBlocks;
  rms_bwd_kernel<In, GT, E, N, true><<<(unsigned)groups, 256, 0, s>>>(dY, H, rstd, gamma, dH, T, (int)K, dX, part);
  return groups;
}

template <typename In, typename GT>
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
  } else if (K < E) groups = bwd_wave<In, GT, 1, 1>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 64) groups = bwd_wave<In, GT, E, 1>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 128) groups = bwd_wave<In, GT, E, 2>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 256) groups = bwd_block<In, GT, E, 1>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 768) groups = bwd_block<In, GT, E, 2>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 1536) groups = bwd_block<In, GT, E, 3>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= 2048) groups = bwd_block<In, GT, E, 4>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else if (v <= kBwdMaxVecs) groups = bwd_block<In, GT, E, 8>(dY, H, rstd, gamma, dH, T, K, dX, part, s);
  else {
    groups = bwd_groups(T, K);
    if (dgamma)
      rms_dgamma_long_kernel<In><<<dim3((unsigned)cdiv(K, 256), (unsigned)groups), 256, 0, s>>>(dY, H, rstd, T, K,
                                                                                              part);
    if (dX) rms_dx_long_kernel<In, GT><<<(unsigned)T, 1024, 0, s>>>(dY, H, rstd, gamma, dH, K, dX);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !dgamma) return e;
  rms_dgamma_reduce_kernel<GT><<<(unsigned)cdiv(K, 64), 1024, 0, s>>>(part, (int)groups, K, accumulate, (GT*)dgamma);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(Dt dt, const void* X, const void* res, Dt gamma_dt, const void* gamma, int64_t T, int64_t K,
                          float eps, void* H, void* Y, int8_t* q, float* qs, float* rstd, hipStream_t s) {
  if (T == 0 || K == 0) return hipSuccess;
  const NormOut o{H, Y, q, qs, rstd, true};
  const bool wide = gamma && gamma_dt == Dt::F32;
  if (dt == Dt::F32) return rms_launch<float, float>(X, res, gamma, T, K, eps, o, s);
  if (dt == Dt::F16)
    return wide ? rms_launch<_Float16, float>(X, res, gamma, T, K, eps, o, s)
                : rms_launch<_Float16, _Float16>(X, res, gamma, T, K, eps, o, s);
  return wide ? rms_launch<uint16_t, float>(X, res, gamma, T, K, eps, o, s)
              : rms_launch<uint16_t, uint16_t>(X, res, gamma, T, K, eps, o, s);
}

hipError_t launch_quantize_rows_i8(Dt dt, const void* X, int64_t T, int64_t K, int8_t* q, float* scale,
                                   hipStream_t s) {
  if (T == 0 || K == 0) return hipSuccess;
  const NormOut o{nullptr, nullptr, q, scale, nullptr, false};
  return dt == Dt::F16 ? rms_launch<_Float16, _Float16>(X, nullptr, nullptr, T, K, 0.f, o, s)
                       : rms_launch<uint16_t, uint16_t>(X, nullptr, nullptr, T, K, 0.f, o, s);
}

int64_t rmsnorm_bwd_workspace_bytes(int64_t T, int64_t K) { return bwd_groups(T, K) * K * 4; }

hipError_t launch_rmsnorm_bwd(Dt dt, const void* dY, const void* H, const float* rstd, Dt gamma_dt, const void* gamma,
                              const void* dH, int64_t T, int64_t K, void* dX, void* dgamma, int accumulate,
                              void* workspace, hipStream_t s) {
  if (K == 0) return hipSuccess;
  float* part = (float*)workspace;
  const bool wide = gamma_dt == Dt::F32;          // dgamma's type too, so also without a gamma
  if (dt == Dt::F32) return bwd_launch<float, float>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s);
  if (dt == Dt::F16)
    return wide ? bwd_launch<_Float16, float>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s)
                : bwd_launch<_Float16, _Float16>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s);
  return wide ? bwd_launch<uint16_t, float>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s)
              : bwd_launch<uint16_t, uint16_t>(dY, H, rstd, gamma, dH, T, K, dX, dgamma, accumulate, part, s);
}

}  // namespace slope
