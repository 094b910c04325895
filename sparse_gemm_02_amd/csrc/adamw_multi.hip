// One AdamW step over many tensors in one launch, with moments in fp32 or in 8
// bits (blocks of 32 consecutive values with a power-of-two scale each: moments8.h), and
// the 8-bit moments as values.
#include <algorithm>
#include <type_traits>

#include "adamw_args.h"
#include "moments8.h"

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
  float pf[8], gf[8];
  if constexpr (EIGHT) {
    load8<NT>(p, e, n, pf);
    load8<NT>(g, e, n, gf);
    const int64_t left = n - e, at = left > 0 ? e : 0, block = at / 32;   // lanes past the end: no access, zeros
    uint8_t* m = (uint8_t*)a.m[lo];
    uint8_t* v = (uint8_t*)a.v[lo];
    Run8 r{load_codes<NT>(m + at, left), load_codes<NT>(v + at, left), left > 0 ? a.me[lo][block] : 0u,
           left > 0 ? a.ve[lo][block] : 0u};
    const Pack<PT, 8> np = update8<PT, FAST>(pf, gf, r, left, c0, Noise((uint32_t)(e / 8), a.seed[lo]));
    if (left > 0) {
      store_codes<NT>(m + at, left, r.m);
      store_codes<NT>(v + at, left, r.v);
      if (threadIdx.x % 4 == 0) {
        a.me[lo][block] = (uint8_t)r.em;
        a.ve[lo][block] = (uint8_t)r.ev;
      }
    }
    store8<NT>(p, e, n, np);
  } else {
    float* m = (float*)a.m[lo];
    float* v = (float*)a.v[lo];
    float mf[8], vf[8];
    e -= lead32(m);
    load8<NT>(p, e, n, pf);
    load8<NT>(g, e, n, gf);
    load8<NT>(m, e, n, mf);
    load8<NT>(v, e, n, vf);
    const Pack<PT, 8> np = step8<PT, FAST>(pf, gf, mf, vf, c0);
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

}  // namespace

// A launch takes tensors of one pair of types; most lists have one or two pairs.
hipError_t launch_adamw_multi(bool eight, const AdamWTensors& t, const AdamWStep& c, uint64_t seed, hipStream_t s) {
  const bool fast = eight && fast_step(c);
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
