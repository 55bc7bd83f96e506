// Rows of logits: log probabilities of given tokens with the entropy and the
// most likely alternatives, and the acceptance of drafted tokens.
//
// One pass over a row keeps, per thread, an anchor m near the running maximum
// and, with t = c (x - m) and c = log2(e) / T,
//   s = sum 2^t,   a = sum 2^t t,
// from which lse = m / T + ln s and entropy = ln s - ln 2 a / s.
//
// A row is read once, by a cluster of up to 4 CTAs where there are few rows;
// the parts' sums meet in the shared memory of the cluster's first CTA.
//
// Bound by memory, the special function unit (one 2^x a logit: 30 us for the
// 1.3e8 logits below) and latency.  1024 rows of 131072 bf16: 50.5 us, 5.3 TB/s, 81% of
// a copy's rate, and 58.5 with the 8 most likely tokens; the loads and maxima alone take
// 47.  4 rows: 5.4 and 8.7 us, of which launch, joins and the search are most.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <stdint.h>

#include <type_traits>

#include "f32x2.cuh"
#include "status.cuh"

namespace wmtp {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowUnroll = 4;                      // 16-byte loads of a thread's batch; two batches are in flight
constexpr int kBatch = kRowUnroll * kRowThreads;  // vecs of a CTA's batch
constexpr int kRowCluster = 4;                     // most CTAs that share a row
constexpr int kCells = 16;                         // of a thread, in the search for the largest logits
constexpr int kMaxCells = 512;
constexpr int kMaxCandidates = 1024;
constexpr int kFinalCluster = 16;
constexpr int kFinalThreads = 256;
constexpr int kFinalWarps = kFinalThreads / 32;
constexpr int kMaxTop = 64;

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// ex2.approx: relative error 2^-22, its flush of denormal results far below
// what a sum that starts at 1 can hold.
__device__ __forceinline__ float exp2_fast(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}

// The larger of x and lo; NaN stays NaN.
__device__ __forceinline__ float at_least(float x, float lo) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(lo));
  return r;
}

// f(x - m) for a product or quotient f: by halves where the difference of two
// finite logits passes fp32, whatever T makes of it.
template <typename F>
__device__ __forceinline__ float of_difference(float x, float m, F f) {
  const float d = x - m;
  return d > -INFINITY ? f(d) : 2.f * f(0.5f * x - 0.5f * m);
}
__device__ __forceinline__ float times_difference(float x, float m, float c) {
  return of_difference(x, m, [c](float d) { return d * c; });
}

// Stands for lower logits and -inf in exponents, so that none is infinite.
constexpr float kLowest = -9.9530379158544574e29f;  // bf16 0xf149

// 16 bytes of a row.  unpack: as floats.  Top, top_of: the largest value of
// several vecs (NaN aside).  exponents: x c - A with x no lower than kLowest,
// in pairs; NaN stays.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  using Top = float;
  static __device__ __forceinline__ Top top_empty() { return -INFINITY; }
  static __device__ __forceinline__ void top_add(Top& t, uint4 u) {
    t = fmaxf(fmaxf(t, fmaxf(__uint_as_float(u.x), __uint_as_float(u.y))),
              fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
  }
  static __device__ __forceinline__ float top_of(Top t) { return t; }
  static __device__ __forceinline__ void unpack(uint4 u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ void exponents(uint4 u, uint64_t c, uint64_t minus_a, uint64_t (&t)[2]) {
    float x[4];
    unpack(u, x);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      t[i] = fma2(pack2(at_least(x[2 * i], kLowest), at_least(x[2 * i + 1], kLowest)), c, minus_a);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  using Top = uint32_t;
  static __device__ __forceinline__ Top top_empty() { return 0xff80ff80u; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ void top_add(Top& t, uint4 u) {
    t = larger(larger(t, larger(u.x, u.y)), larger(u.z, u.w));
  }
  static __device__ __forceinline__ float top_of(Top t) {
    return fmaxf(__uint_as_float(t << 16), __uint_as_float(t & 0xffff0000u));
  }
  static __device__ __forceinline__ void unpack(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void exponents(uint4 u, uint64_t c, uint64_t minus_a, uint64_t (&t)[4]) {
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(w[i]), "r"(0xf149f149u));
      t[i] = fma2(pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)), c, minus_a);
    }
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  using Top = uint32_t;
  static __device__ __forceinline__ Top top_empty() { return 0xfc00fc00u; }
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ void top_add(Top& t, uint4 u) {
    t = larger(larger(t, larger(u.x, u.y)), larger(u.z, u.w));
  }
  static __device__ __forceinline__ float2 both(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ float top_of(Top t) { return fmaxf(both(t).x, both(t).y); }
  static __device__ __forceinline__ void unpack(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = both(w[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ void exponents(uint4 u, uint64_t c, uint64_t minus_a, uint64_t (&t)[4]) {
    float x[8];
    unpack(u, x);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      t[i] = fma2(pack2(at_least(x[2 * i], kLowest), at_least(x[2 * i + 1], kLowest)), c, minus_a);
  }
};

// A row in aligned groups of 16 bytes ("vecs"), of which this CTA takes
// [v0, v1), a run of columns.  The first and the last vec of a row may reach
// beyond it: their other columns are not read and count as masked (-inf).
template <typename T>
struct Part {
  static constexpr int N = Vec<T>::N;
  const T* p;
  int V, off, v0, v1;
  __device__ __forceinline__ Part(const T* row, int vocab, int rank, int parts) : p(row), V(vocab) {
    off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    const int n = (off + V + N - 1) / N, per = (n + parts - 1) / parts;
    v0 = min(rank * per, n);
    v1 = min(v0 + per, n);
  }
  __device__ __forceinline__ int col(int i) const { return i * N - off; }
  // Nothing but masked columns.
  static __device__ __forceinline__ uint4 none() {
    const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
    return make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ uint4 load(int i) const {
    const int c = col(i);
    if (c >= 0 && c + N <= V) return *reinterpret_cast<const uint4*>(p + c);
    uint32_t w[4];
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = c + j >= 0 && c + j < V ? __float_as_uint(as_float(p[c + j])) : 0xff800000u;
    } else {
      const uint32_t none = std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
      const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int a = c + 2 * j, b = a + 1;
        w[j] = (a >= 0 && a < V ? h[a] : none) | ((b >= 0 && b < V ? h[b] : none) << 16);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Running sums of a part of a row, relative to m.
struct RowSum {
  float m, s, a;
};

// Moves the sums to a larger m.  Where the factor is 0 the exponent may be
// infinite; NaN in s stays.
__device__ __forceinline__ void row_sum_raise(RowSum& r, float m, float c) {
  const float t = times_difference(r.m, m, c);
  const float f = exp2_fast(t);
  r.a = f * (r.a + t * r.s);
  r.s *= f;
  if (f == 0.f) r.a = r.s;
  r.m = m;
}

// Both are raised, the larger one by a factor of 1: they overlap, and no lanes part
// (4 rows of 131072 bf16, top 5: 8.5 us; raising only the smaller one 9.3).
__device__ __forceinline__ void row_sum_merge(RowSum& r, RowSum o, float c) {
  const float m = fmaxf(r.m, o.m);
  row_sum_raise(r, m, c);
  row_sum_raise(o, m, c);
  r.s += o.s;
  r.a += o.a;
}

// A thread's sums, and its largest logit with the place where it is first met:
// one of the kRowUnroll vecs from `vec` on, as many threads apart as there are.
struct ThreadSum {
  RowSum r;
  float best;
  int vec;
};

// A thread's sums where x c may not be finite or loses the digits of x - m:
// very large logits, lowest values of the type alone, extreme temperatures.
template <typename T>
__device__ __noinline__ RowSum part_sums_extreme(const Part<T>& part, float c, float best) {
  RowSum r = {best, 0.f, 0.f};
  for (int i = part.v0 + threadIdx.x; i < part.v1; i += kRowThreads) {
    float x[Vec<T>::N];
    Vec<T>::unpack(part.load(i), x);
    for (int j = 0; j < Vec<T>::N; ++j) {
      const float t = times_difference(x[j], best, c), e = exp2_fast(t);
      r.s += e;
      r.a += e == 0.f ? 0.f : e * t;
    }
  }
  return r;
}

// Sums of this thread's share of a part, relative to A = m c rounded: the
// exponent x c - A takes one fused instruction and one rounding, and 2^(m c - A),
// the same for all of them, is put right at the end.  The anchor is raised only
// once a logit passes it by 2^8 in weight, not at each new maximum, which some lane
// of a warp meets nearly always.
// cells (NULL: none): `used` cells of the thread, kRowThreads apart, the largest
// logit of each run of 2^shift batches.
template <typename T>
__device__ __forceinline__ ThreadSum part_sums(const Part<T>& part, float c, float* cells, int used, int shift) {
  using V = Vec<T>;
  ThreadSum z = {{0.f, 0.f, 0.f}, -INFINITY, part.v0};
  const float slack = 8.f / c;
  const uint64_t c2 = pack2(c, c);
  uint64_t s2 = 0, a2 = 0, minus_a2 = 0;
  float raise_at = kLowest;  // what lies below counts as masked here
  auto sums = [&]() {
    float s0, s1, a0, a1;
    unpack2(s2, s0, s1);
    unpack2(a2, a0, a1);
    return make_float2(s0 + s1, a0 + a1);
  };
  auto step = [&](const uint4 (&u)[kRowUnroll], int i) {
    typename V::Top t = V::top_empty();
#pragma unroll
    for (const uint4& v : u) V::top_add(t, v);
    const float top = V::top_of(t);
    if (cells != nullptr) {
      float* cell = cells + ((i - part.v0) / kBatch >> shift) * kRowThreads;
      *cell = fmaxf(*cell, top);
    }
    if (top > z.best) z.best = top, z.vec = i;
    if (top > raise_at) {
      const float2 o = sums();
      const float by = __fmul_rn(z.r.m, c) - __fmul_rn(top, c), f = exp2_fast(by);
      z.r.m = top;
      raise_at = top + slack;
      // a run of -1e10, say, has lost all digits against its anchor, and may have overflowed
      const bool gone = o.x == 0.f || (f == 0.f && o.x == o.x);
      s2 = pack2(gone ? 0.f : f * o.x, 0.f);
      a2 = pack2(gone ? 0.f : f * (o.y + by * o.x), 0.f);
      minus_a2 = pack2(__fmul_rn(-top, c), __fmul_rn(-top, c));
    }
#pragma unroll
    for (const uint4& v : u) {
      uint64_t t2[V::N / 2];
      V::exponents(v, c2, minus_a2, t2);
#pragma unroll
      for (int j = 0; j < V::N / 2; ++j) {
        float t0, t1;
        unpack2(t2[j], t0, t1);
        const uint64_t e = pack2(exp2_fast(t0), exp2_fast(t1));
        s2 = add2(s2, e);
        a2 = fma2(e, t2[j], a2);
      }
    }
  };
  if (cells != nullptr) {
    cells += threadIdx.x;
    for (int k = 0; k < used; ++k) cells[k * kRowThreads] = -INFINITY;
  }
  int i = part.v0 + threadIdx.x;
  uint4 u0[kRowUnroll], u1[kRowUnroll];
  auto cut = [&]() {  // a batch that the row or the part cuts
#pragma unroll
    for (int k = 0; k < kRowUnroll; ++k)
      u0[k] = i + k * kRowThreads < part.v1 ? part.load(i + k * kRowThreads) : part.none();
    step(u0, i);
    i += kBatch;
  };
  if (part.col(i) < 0) cut();
  // whole batches, the next one's loads in flight while one is summed
  const int whole = part.v1 - (part.col(part.v1) > part.V ? 1 : 0) - (kRowUnroll - 1) * kRowThreads;
  if (i < whole) {
    const uint4* v = reinterpret_cast<const uint4*>(part.p + part.col(i));
    auto fetch = [&](uint4 (&u)[kRowUnroll]) {
#pragma unroll
      for (int k = 0; k < kRowUnroll; ++k) u[k] = v[k * kRowThreads];
      v += kBatch;
    };
    fetch(u0);
    while (true) {
      const bool one = i + kBatch < whole, two = i + 2 * kBatch < whole;
      if (one) fetch(u1);
      step(u0, i);
      i += kBatch;
      if (!one) break;
      if (two) fetch(u0);
      step(u1, i);
      i += kBatch;
      if (!two) break;
    }
  }
  if (i < part.v1) cut();
  const float2 o = sums();
  z.r.s = o.x, z.r.a = o.y;
  if (z.best == -INFINITY) {  // masked: no weight (kLowest has some from T = 1e28 on), but NaN stays
    z.r.m = -FLT_MAX;
    if (o.x == o.x) z.r.s = z.r.a = 0.f;
  } else if (z.best > -1e29f && fabsf(z.r.m) < 1e29f && fabsf(z.r.m * c) < 1e6f && c > 1e-20f && c < 1e7f) {
    const float low = fmaf(z.r.m, c, -__fmul_rn(z.r.m, c)), f = exp2f(-low);
    z.r.s = f * o.x;
    z.r.a = f * (o.y - low * o.x);
  } else {
    z.r = part_sums_extreme<T>(part, c, z.best);
  }
  return z;
}

// Whole numbers in the order of the logits: larger first, then lower columns.
// 0 is below every logit.
__device__ __forceinline__ uint64_t logit_key(float x, int col) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 is 0
  const uint32_t o = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return (static_cast<uint64_t>(o) << 32) | (0xffffffffu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ float key_logit(uint64_t k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ int key_col(uint64_t k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }
__device__ __forceinline__ uint64_t max_key(uint64_t a, uint64_t b) { return a > b ? a : b; }

// The sums of the block's threads, on warp 0.
__device__ __forceinline__ RowSum block_sums(RowSum r, float c, RowSum* s_part) {
  auto halve = [&](int from) {
#pragma unroll
    for (int o = from; o > 0; o >>= 1) {
      const RowSum u = {__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                        __shfl_xor_sync(0xffffffffu, r.a, o)};
      row_sum_merge(r, u, c);
    }
  };
  halve(16);
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = r;
  __syncthreads();
  if (threadIdx.x < 32) {
    r = s_part[threadIdx.x & (kRowThreads / 32 - 1)];
    halve(kRowThreads / 64);
  }
  return r;
}

// The largest key of the part below `bound`, on every thread.  0: none above -inf.
template <typename T>
__device__ __noinline__ uint64_t part_best(const Part<T>& part, uint64_t bound, uint64_t* s_best) {
  uint64_t best = 0;
  for (int i = part.v0 + threadIdx.x; i < part.v1; i += kRowThreads) {
    float x[Vec<T>::N];
    Vec<T>::unpack(part.load(i), x);
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) {
      const uint64_t k = logit_key(x[j], part.col(i) + j);
      if (x[j] > -INFINITY && k < bound) best = max_key(best, k);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max_key(best, __shfl_xor_sync(0xffffffffu, best, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_best[threadIdx.x >> 5] = best;
  __syncthreads();
  best = s_best[0];
  for (int w = 1; w < kRowThreads / 32; ++w) best = max_key(best, s_best[w]);
  return best;
}

struct TopShared {
  float cells[kCells * kRowThreads];
  uint64_t keys[kRowThreads / 2];
  uint64_t cand[kMaxCandidates];
  uint64_t warp_best[kRowWarps];
  uint64_t bound;
  int cell[kMaxCells];
  int listed, count;
};

// The keys of part_top where very many logits stand at its bound, `lowest`: those
// above it, then the first columns at it, chunk by chunk until there are enough
// (a row masked with -1e4 that leaves fewer than top_k tokens has its first masked
// columns behind them).  Returns -1 if too many are above.
template <typename T>
__device__ __noinline__ int part_top_ties(const Part<T>& part, float lowest, int top_k, TopShared& sh, uint64_t* out) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();
  if (tid == 0) sh.count = 0;
  __syncthreads();
  for (int i = part.v0 + tid; i < part.v1; i += kRowThreads) {
    float x[N];
    Vec<T>::unpack(part.load(i), x);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!(x[j] > lowest)) continue;
      const int at = atomicAdd(&sh.count, 1);
      if (at < kMaxCandidates) sh.cand[at] = logit_key(x[j], part.col(i) + j);
    }
  }
  __syncthreads();
  const int above = sh.count;
  if (above > kMaxCandidates) return -1;
  for (int i = tid; i < above; i += kRowThreads) {
    const uint64_t k = sh.cand[i];
    int r = 0;
    for (int j = 0; j < above; ++j) r += sh.cand[j] > k;
    if (r < top_k) out[r] = k;
  }
  int n = above;
  for (int base = part.v0; base < part.v1 && n < top_k; base += kRowThreads) {
    float x[N];
    int mine = 0;
    Vec<T>::unpack(base + tid < part.v1 ? part.load(base + tid) : part.none(), x);
#pragma unroll
    for (int j = 0; j < N; ++j) mine += x[j] == lowest;
    int scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += u;
    }
    __syncthreads();
    if (lane == 31) sh.cell[warp] = scan;
    __syncthreads();
    int at = n + scan - mine, total = 0;
    for (int w = 0; w < kRowWarps; ++w) {
      if (w < warp) at += sh.cell[w];
      total += sh.cell[w];
    }
    for (int j = 0; j < N; ++j)
      if (x[j] == lowest && at < top_k) out[at++] = logit_key(x[j], part.col(base + tid) + j);
    n += total;
  }
  return min(n, top_k);
}

// The part's `top_k` largest keys, in order, to out[0 .. top_k), 0 behind the
// last one.  Returns how many there are.
//
// The pass over the row leaves each thread its best logit and the best of each of its
// cells; the keys lie between those of the first and the last column that they may
// stand in.  The top_k-th largest of the lower bounds of groups of threads
// bounds the part's top_k-th key from below, and what lies above it is in the cells
// whose upper bound reaches it, about top_k of them: only these are read again
// (from L2), and the few keys above the bound sorted by counting.  Should a list
// overflow, logits equal to the bound are taken in order; the keys are taken one
// pass each where even those above it are too many (one thread holds hundreds
// of the largest logits).
template <typename T>
__device__ __forceinline__ int part_top(const Part<T>& part, const ThreadSum& z, int used, int shift, int top_k,
                                        TopShared& sh, uint64_t* out) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x;
  uint64_t least = 0;
  if (z.best > -INFINITY) least = logit_key(z.best, part.col(z.vec + (kRowUnroll - 1) * kRowThreads) + N - 1);
  const int lanes = top_k <= 16 ? 8 : top_k <= 32 ? 4 : 2;  // of a group: twice top_k groups bound well
  for (int o = lanes / 2; o > 0; o >>= 1) least = max_key(least, __shfl_xor_sync(0xffffffffu, least, o));
  if (tid % lanes == 0) sh.keys[tid / lanes] = least;
  if (tid == 0) sh.listed = sh.count = 0, sh.bound = 0;
  for (int i = tid; i < top_k; i += kRowThreads) out[i] = 0;
  __syncthreads();
  // each thread ranks its group's key among its share of the keys
  int rank = 0;
#pragma unroll 4
  for (int i = tid % lanes; i < kRowThreads / lanes; i += lanes) rank += sh.keys[i] > least;
  for (int o = lanes / 2; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
  if (rank == top_k - 1 && tid % lanes == 0) sh.bound = least;  // 0 where there are fewer: every cell
  __syncthreads();
  const uint64_t bound = sh.bound;
  const float lowest = bound != 0 ? key_logit(bound) : -FLT_MAX;
  auto first_vec = [&](int cell) { return part.v0 + (cell / kRowThreads << shift) * kBatch + cell % kRowThreads; };
  if (z.best >= lowest)
    for (int i = tid; i < used * kRowThreads; i += kRowThreads) {
      const float x = sh.cells[i];
      if (!(x >= lowest) || logit_key(x, max(part.col(first_vec(i)), 0)) < bound) continue;
      const int at = atomicAdd(&sh.listed, 1);
      if (at < kMaxCells) sh.cell[at] = i;
    }
  __syncthreads();
  const int listed = sh.listed, vecs = kRowUnroll << shift;
  for (int i = tid; i < min(listed, kMaxCells) << (shift + 2); i += kRowThreads) {
    const int v = first_vec(sh.cell[i >> (shift + 2)]) + (i & (vecs - 1)) * kRowThreads;
    if (v >= part.v1) continue;
    float x[N];
    Vec<T>::unpack(part.load(v), x);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!(x[j] >= lowest)) continue;
      const uint64_t k = logit_key(x[j], part.col(v) + j);
      if (k < bound) continue;
      const int at = atomicAdd(&sh.count, 1);
      if (at < kMaxCandidates) sh.cand[at] = k;
    }
  }
  __syncthreads();
  int n = sh.count;
  if (listed <= kMaxCells && n <= kMaxCandidates) {
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t k = sh.cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += sh.cand[j] > k;
      if (r < top_k) out[r] = k;
    }
    n = min(n, top_k);
  } else {
    n = part_top_ties(part, lowest, top_k, sh, out);
    if (n < 0) {
      uint64_t below = ~0ull;
      for (n = 0; n < top_k; ++n) {
        below = part_best<T>(part, below, sh.warp_best);
        if (below == 0) break;
        if (tid == 0) out[n] = below;
      }
    }
  }
  __syncthreads();
  return n;
}

// 1 / T, or NaN for a T that is no temperature, or so low that log2(e) / T, which
// the exponents are multiplied with, passes fp32 (below 4.25e-39).
__device__ __forceinline__ float inverse_temperature(float t) {
  const float inv_t = 1.f / t;
  return t > 0.f && t < INFINITY && inv_t * kLog2e < INFINITY ? inv_t : NAN;
}

// NaN or +inf somewhere in the row, or no temperature.
__device__ __forceinline__ bool row_bad(const RowSum& r, float inv_t) {
  return !(r.s < INFINITY) || !(r.m < INFINITY) || !(inv_t == inv_t);
}

struct LogprobArgs {
  const void* logits;
  long long row_stride;
  const float* temperature;
  const int32_t* tokens;
  float *logprobs, *entropy, *lse, *top_logprobs;
  int32_t *top_ids, *status;
  int V, num_tokens, top_k;
};

// What a CTA knows of its part of a row.
struct PartSum {
  RowSum r;
  int n;          // keys in its list
  uint64_t best;  // the largest key
};

// One cluster per row; its first CTA joins the parts and writes the results.
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 1024 / kRowThreads) logprob_kernel(LogprobArgs a) {
  __shared__ RowSum s_part[kRowThreads / 32];
  __shared__ PartSum s_sums[kRowCluster];
  __shared__ uint64_t s_top[kRowCluster * kMaxTop];
  __shared__ uint64_t s_mine[kMaxTop];
  __shared__ TopShared s_sel;
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), rank = cluster.block_rank();
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int r = blockIdx.x / parts, tid = threadIdx.x;
  const T* p = static_cast<const T*>(a.logits) + r * a.row_stride;
  const float inv_t = inverse_temperature(a.temperature != nullptr ? a.temperature[r] : 1.f), c = inv_t * kLog2e;
  // the given tokens' logits, while the row is read
  const int32_t* ids = a.tokens + static_cast<size_t>(r) * a.num_tokens;
  int id = -1;
  float x_id = 0.f;
  if (rank == 0 && tid < a.num_tokens) {
    id = ids[tid];
    if (id >= 0 && id < a.V) x_id = as_float(p[id]);
  }
  const Part<T> part(p, a.V, rank, parts);
  const int batches = (part.v1 - part.v0 + kBatch - 1) / kBatch;
  int shift = 0;
  while ((batches - 1) >> shift >= kCells) ++shift;
  const int used = (batches + (1 << shift) - 1) >> shift;
  const ThreadSum z = part_sums<T>(part, c, a.top_k > 0 ? s_sel.cells : nullptr, used, shift);
  RowSum sum = block_sums(z.r, c, s_part);
  const int mine = a.top_k > 0 ? part_top<T>(part, z, used, shift, a.top_k, s_sel, parts > 1 ? s_mine : s_top) : 0;
  if (parts > 1) {
    // the first CTA has started by now, so its shared memory may be written
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (tid == 0) cluster.map_shared_rank(s_sums, 0)[rank] = {sum, mine, 0};
    uint64_t* top = cluster.map_shared_rank(s_top, 0) + rank * kMaxTop;
    for (int i = tid; i < a.top_k; i += kRowThreads) top[i] = s_mine[i];
    cluster.sync();
    if (rank != 0) return;
  } else {
    if (tid == 0) s_sums[0] = {sum, mine, 0};
    __syncthreads();
  }
  sum = s_sums[0].r;
  int have = s_sums[0].n;
  for (int i = 1; i < parts; ++i) {
    row_sum_merge(sum, s_sums[i].r, c);
    have += s_sums[i].n;
  }
  const bool bad = row_bad(sum, inv_t), none = sum.s == 0.f;
  const float ln_s = bad ? NAN : logf(sum.s);
  if (bad && tid == 0) set_status(a.status, kDevLogits);
  for (int j = tid; j < a.num_tokens; j += kRowThreads) {
    if (j != tid) id = ids[j];
    const bool in = id >= 0 && id < a.V;
    if (j != tid && in) x_id = as_float(p[id]);
    if (!in && id != -1) set_status(a.status, kDevTokenOob);
    a.logprobs[static_cast<size_t>(r) * a.num_tokens + j] =
        bad ? NAN : (none || !in) ? -INFINITY : times_difference(x_id, sum.m, inv_t) - ln_s;
  }
  if (tid == 0) {
    if (a.lse != nullptr) a.lse[r] = bad ? NAN : none ? -INFINITY : sum.m * inv_t + ln_s;
    if (a.entropy != nullptr) a.entropy[r] = bad ? NAN : none ? 0.f : ln_s - kLn2 * sum.a / sum.s;
  }
  // every part's list is in order: a key's place is its own in its list plus,
  // in each other list, the number of keys above it
  const size_t o = static_cast<size_t>(r) * a.top_k;
  for (int i = tid; i < kMaxTop * parts && !bad; i += kRowThreads) {
    const int l = i / kMaxTop, at = i % kMaxTop;
    if (at >= s_sums[l].n) continue;
    const uint64_t key = s_top[i];
    int place = at;
#pragma unroll
    for (int other = 0; other < kRowCluster; ++other) {
      if (other >= parts || other == l) continue;
      int above = 0;
#pragma unroll
      for (int step = kMaxTop; step > 0; step >>= 1)
        if (above + step <= s_sums[other].n && s_top[other * kMaxTop + above + step - 1] > key) above += step;
      place += above;
    }
    if (place >= a.top_k) continue;
    a.top_ids[o + place] = key_col(key);
    a.top_logprobs[o + place] = times_difference(key_logit(key), sum.m, inv_t) - ln_s;
  }
  for (int i = (bad ? 0 : have) + tid; i < a.top_k; i += kRowThreads) {  // places without a token
    a.top_ids[o + i] = -1;
    a.top_logprobs[o + i] = bad ? NAN : -INFINITY;
  }
}

// ---------------------------------------------------------------- acceptance
// What the decision needs of one row.
struct alignas(16) RowStat {
  float m, s;
  int32_t best;  // lowest column with the largest logit
  int32_t bad;   // defines no distribution
};

// What is left to do for a sequence: the draw of its token `k`.
struct Draw {
  int32_t k;  // -1: nothing
  int32_t drafted, minus;
  float pm, ps, qm, qs, u;
};

struct AcceptArgs {
  const void *target, *draft;
  long long target_batch, target_row, draft_batch, draft_row;
  const int32_t *draft_tokens, *num_draft;
  const float *uniforms, *temperature;
  int32_t *tokens, *count, *status;
  float* logprobs;
  RowStat* stats;  // [B][num_q] of the target, then [B][num_q - 1] of the draft
  int B, num_q, V;
};

__device__ __forceinline__ float accept_temperature(const AcceptArgs& a, int b) {
  return a.temperature != nullptr ? a.temperature[b] : 1.f;
}

// One cluster per row of the target and of the draft.
template <typename T>
__global__ void __launch_bounds__(kRowThreads, 1024 / kRowThreads) accept_rows_kernel(AcceptArgs a) {
  __shared__ RowSum s_part[kRowThreads / 32];
  __shared__ PartSum s_sums[kRowCluster];
  __shared__ uint64_t s_warp[kRowThreads / 32];
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), rank = cluster.block_rank(), tid = threadIdx.x;
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int at = blockIdx.x / parts, rows_t = a.B * a.num_q;
  const bool target = at < rows_t;
  const int r = target ? at : at - rows_t;
  const int per = target ? a.num_q : a.num_q - 1;
  const int b = r / per, i = r % per;
  const float temp = accept_temperature(a, b);
  const bool greedy = temp == 0.f;
  const int nd = a.num_draft != nullptr ? a.num_draft[b] : a.num_q - 1;
  const bool idle = target ? i > nd : (i >= nd || greedy);  // never looked at
  if (!idle) {
    const T* p = target ? static_cast<const T*>(a.target) + b * a.target_batch + i * a.target_row
                        : static_cast<const T*>(a.draft) + b * a.draft_batch + i * a.draft_row;
    const Part<T> part(p, a.V, rank, parts);
    const float inv_t = greedy ? 1.f : inverse_temperature(temp);
    const float c = inv_t * kLog2e;
    const ThreadSum z = part_sums<T>(part, c, nullptr, 0, 0);
    RowSum sum = block_sums(z.r, c, s_part);
    uint64_t best = 0;
    if (greedy) {  // the lowest column with the largest logit
      if (z.best > -INFINITY) {
#pragma unroll
        for (int k = kRowUnroll - 1; k >= 0; --k) {
          const int v = z.vec + k * kRowThreads;
          if (v >= part.v1) continue;
          float x[Vec<T>::N];
          Vec<T>::unpack(part.load(v), x);
#pragma unroll
          for (int j = Vec<T>::N - 1; j >= 0; --j)
            if (x[j] == z.best) best = logit_key(x[j], part.col(v) + j);
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) best = max_key(best, __shfl_xor_sync(0xffffffffu, best, o));
      if ((tid & 31) == 0) s_warp[tid >> 5] = best;
      __syncthreads();
      for (int w = 0; w < kRowThreads / 32; ++w) best = max_key(best, s_warp[w]);
    }
    if (parts > 1) {
      asm volatile("barrier.cluster.wait;" ::: "memory");
      if (tid == 0) cluster.map_shared_rank(s_sums, 0)[rank] = {sum, 0, best};
      cluster.sync();
    } else if (tid == 0) {
      s_sums[0] = {sum, 0, best};
    }
    if (rank == 0 && tid == 0) {
      sum = s_sums[0].r;
      for (int k = 1; k < parts; ++k) {
        row_sum_merge(sum, s_sums[k].r, c);
        best = max_key(best, s_sums[k].best);
      }
      a.stats[at] = {sum.m, sum.s, best != 0 ? key_col(best) : -1, row_bad(sum, inv_t) || sum.s == 0.f};
    }
  } else if (parts > 1) {
    asm volatile("barrier.cluster.wait;" ::: "memory");
  }
}

// exp in 64 bits, for weights: 2^(u / 32) with u = k + r, |r| <= 1/2, is
// 2^(k div 32) * 2^((k mod 32) / 32) * (1 + z + z^2/2 + z^3/6 + z^4/24),
// z = r ln2 / 32; the Taylor series' next term is below 1.3e-12.  The 32
// factors 2^(j / 32) are held by a warp's lanes.  All lanes take part.  u is
// raised to -32000 (the comparison of the upper words as unsigned numbers
// orders negative ones by size): 2^-1000 stands for 0, and sums below
// kNoWeight are taken for it.
constexpr unsigned kLeast = 0xc0df4000u;  // upper word of -32000.0
constexpr double kNoWeight = 1e-250;
__device__ __forceinline__ double lane_factor() { return exp2((threadIdx.x & 31) / 32.0); }
template <int K>
__device__ __forceinline__ void exp_weights(double (&u)[K], double factor) {  // step by step for all K: they overlap
  constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: rounds to whole numbers
  constexpr double c1 = 0.69314718055994530942 / 32, c2 = c1 * c1 / 2, c3 = c1 * c1 * c1 / 6, c4 = c1 * c1 * c1 * c1 / 24;
  int k[K];
  double z[K];
#pragma unroll
  for (int i = 0; i < K; ++i)
    u[i] = __hiloint2double(min(static_cast<unsigned>(__double2hiint(u[i])), kLeast), __double2loint(u[i]));
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const double kd = u[i] + kMagic;
    k[i] = __double2loint(kd);
    u[i] -= kd - kMagic;
  }
#pragma unroll
  for (int i = 0; i < K; ++i) z[i] = fma(u[i], c4, c3);
#pragma unroll
  for (int i = 0; i < K; ++i) z[i] = fma(u[i], z[i], c2);
#pragma unroll
  for (int i = 0; i < K; ++i) z[i] = fma(u[i], z[i], c1);
#pragma unroll
  for (int i = 0; i < K; ++i) z[i] *= u[i];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const double f = __shfl_sync(0xffffffffu, factor, k[i] & 31);
    u[i] = fma(f, z[i], f);
  }
#pragma unroll
  for (int i = 0; i < K; ++i)
    u[i] = __hiloint2double(__double2hiint(u[i]) + (k[i] >> 5) * (1 << 20), __double2loint(u[i]));
}

// The weights of the token that follows: p, or what p has above q (both not
// normalised: p_i - r q_i with r = sum p / sum q).  In 64 bits: a draw takes the
// token in which the cumulated weight passes u, and with V tokens a relative
// error e of that sum moves the border over a token with probability V e (1e-2 at
// V = 131072 and the 1e-7 of fp32).
template <typename T>
struct FinalWeights {
  const T *p, *q;  // q NULL: nothing to take away, or all of it on `drafted`
  double pm, qm, scale;  // 32 log2(e) / T
  double r, factor;
  int drafted;  // -1: no draft to take away
  // e: of p's logits; f: of q's.
  template <int K>
  __device__ __forceinline__ void pe(const float (&x)[K], double (&e)[K]) const {
#pragma unroll
    for (int i = 0; i < K; ++i) e[i] = (x[i] - pm) * scale;
    exp_weights(e, factor);
  }
  template <int K>
  __device__ __forceinline__ void qe(const float (&x)[K], double (&f)[K]) const {
#pragma unroll
    for (int i = 0; i < K; ++i) f[i] = (x[i] - qm) * scale;
    exp_weights(f, factor);
  }
  // Of the columns col, col + step, ...
  template <int K>
  __device__ __forceinline__ void weights(const float (&xp)[K], const float (&xq)[K], int col, int step, double (&v)[K]) const {
    pe(xp, v);
    if (q != nullptr) {
      double f[K];
      qe(xq, f);
#pragma unroll
      for (int i = 0; i < K; ++i) v[i] = fmax(fma(-r, f[i], v[i]), 0.0);
    } else {
#pragma unroll
      for (int i = 0; i < K; ++i) v[i] = col + i * step == drafted ? 0.0 : v[i];
    }
  }
};

__device__ __forceinline__ double warp_total(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kFinalUnroll = 8;
constexpr int kOverlap = 4;  // columns of a lane worked on at once
constexpr int kLast = 4;  // columns of a lane in the last step of a draw

// f(logits of p, logits of q, first column) for the columns [c0, c1), a warp's,
// kOverlap at a time, 32 apart; columns behind c1 are masked.  kFinalUnroll
// loads in flight.
template <typename T, typename F>
__device__ __forceinline__ void warp_columns(const T* p, const T* q, int c0, int c1, F f) {
  const int lane = threadIdx.x & 31;
  for (int base = c0; base < c1; base += 32 * kFinalUnroll) {
    float xp[kFinalUnroll / kOverlap][kOverlap], xq[kFinalUnroll / kOverlap][kOverlap];
    if (base + 32 * kFinalUnroll <= c1) {
#pragma unroll
      for (int k = 0; k < kFinalUnroll; ++k) {
        const int c = base + lane + 32 * k;
        xp[k / kOverlap][k % kOverlap] = as_float(p[c]);
        xq[k / kOverlap][k % kOverlap] = q != nullptr ? as_float(q[c]) : 0.f;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kFinalUnroll; ++k) {
        const int c = base + lane + 32 * k;
        xp[k / kOverlap][k % kOverlap] = c < c1 ? as_float(p[c]) : -INFINITY;
        xq[k / kOverlap][k % kOverlap] = q != nullptr && c < c1 ? as_float(q[c]) : -INFINITY;
      }
    }
#pragma unroll
    for (int k = 0; k < kFinalUnroll; k += kOverlap)
      if (base + 32 * k < c1) f(xp[k / kOverlap], xq[k / kOverlap], base + lane + 32 * k);
  }
}

template <typename T>
__device__ __forceinline__ double warp_weight(const FinalWeights<T>& w, int c0, int c1) {
  double sum = 0.0;
  warp_columns(w.p, w.q, c0, c1, [&](const float (&xp)[kOverlap], const float (&xq)[kOverlap], int col) {
    double v[kOverlap];
    w.weights(xp, xq, col, 32, v);
#pragma unroll
    for (int i = 0; i < kOverlap; ++i) sum += v[i];
  });
  return warp_total(sum);
}

// A warp's running total over v, lane by lane; *all: the total.
template <int K>
struct Running {
  double v[K], before, all;  // before this lane's first
  __device__ __forceinline__ void scan() {
    double mine = 0.0;
#pragma unroll
    for (int i = 0; i < K; ++i) mine += v[i];
    double s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double u = __shfl_up_sync(0xffffffffu, s, o);
      if ((threadIdx.x & 31) >= o) s += u;
    }
    all = __shfl_sync(0xffffffffu, s, 31);
    before = s - mine;
  }
  // The first entry with a weight at which the running total passes `want`, and the
  // total before it; where rounding lets none pass, the last one with a weight.
  __device__ __forceinline__ int pick(double want, double* skipped) const {
    int at = -1, last = -1;
    double b = before, at_before = 0.0, last_before = 0.0;
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if (v[i] > kNoWeight) {
        last = i, last_before = b;
        if (at < 0 && b + v[i] > want) at = i, at_before = b;
      }
      b += v[i];
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at >= 0), any = __ballot_sync(0xffffffffu, last >= 0);
    const int from = hit != 0 ? __ffs(hit) - 1 : any != 0 ? 31 - __clz(any) : 0;
    *skipped = __shfl_sync(0xffffffffu, hit != 0 ? at_before : last_before, from);
    return from * K + max(__shfl_sync(0xffffffffu, hit != 0 ? at : last, from), 0);
  }
};

// One cluster per sequence.  Bound by the 64-bit units and, for few sequences, by
// the latency of its steps: 32 sequences of 5 drafts and 129281 tokens take 19 us here
// after 17 in the rows' pass (3 to decide, 11 for the weights, 5 to pick), 1 of 3
// drafts and 131072 tokens 8 after 4, 64 of one row each 35 in all.  64 registers spill
// 64 bytes a thread.
//
// The weights' sums take one pass: p_i - r q_i is above 0 for the same i whether
// r is exact or from the rows' fp32 sums, but for those within 1e-7 of 0; so the sums
// of p, of q, and of both over the i with a weight give the exact r and with it
// each run's sum.
template <typename T>
__global__ void __launch_bounds__(kFinalThreads, 4) accept_kernel(AcceptArgs a) {
  constexpr int kMost = kFinalCluster * kFinalWarps, kPer = kMost / 32;
  __shared__ double s_sum[4][kMost];  // of each warp's run: p, q, p and q where there is a weight
  __shared__ double s_sub[kFinalWarps];
  __shared__ Draw s_draw;
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), rank = cluster.block_rank();
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const double factor = lane_factor();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x / parts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.num_q;
  const float temp = accept_temperature(a, b);
  const T* target = static_cast<const T*>(a.target) + b * a.target_batch;
  const T* draft = a.draft != nullptr ? static_cast<const T*>(a.draft) + b * a.draft_batch : nullptr;
  if (warp == 0) {
    const int nd = a.num_draft != nullptr ? a.num_draft[b] : n - 1;
    // a lane for each row; those behind num_draft hold nothing, and are not looked at
    RowStat ts = RowStat(), ds = RowStat();
    float u = 0.f;
    int id = -1;
    if (lane < n) {
      ts = a.stats[static_cast<size_t>(b) * n + lane];
      u = a.uniforms[static_cast<size_t>(b) * n + lane];
    }
    if (lane < n - 1) {
      if (draft != nullptr) ds = a.stats[static_cast<size_t>(a.B) * n + static_cast<size_t>(b) * (n - 1) + lane];
      id = a.draft_tokens[static_cast<size_t>(b) * (n - 1) + lane];
    }
    int32_t* tokens = a.tokens + static_cast<size_t>(b) * n;
    float* lps = a.logprobs != nullptr ? a.logprobs + static_cast<size_t>(b) * n : nullptr;
    if (nd < 0 || nd > n - 1) {
      if (rank == 0 && lane < n) {
        tokens[lane] = -1;
        if (lps != nullptr) lps[lane] = 0.f;
      }
      if (lane == 0) s_draw.k = -1;
      if (rank == 0 && lane == 0) {
        set_status(a.status, kDevLenOob);
        a.count[b] = 0;
      }
    } else {
      const bool greedy = temp == 0.f, with_q = !greedy && draft != nullptr;
      const float inv_t = greedy ? 1.f : 1.f / temp;
      const bool in = lane >= nd || (id >= 0 && id < a.V);
      const bool row_is_bad = lane <= nd && (ts.bad || (lane < nd && with_q && ds.bad));
      float lp = 0.f;
      bool ok = false;
      if (lane < nd && in && !row_is_bad) {
        const float y = times_difference(as_float(target[lane * a.target_row + id]), ts.m, inv_t);
        const float qd = with_q ? expf(times_difference(as_float(draft[lane * a.draft_row + id]), ds.m, inv_t)) / ds.s : 1.f;
        lp = y - logf(ts.s);
        ok = greedy ? id == ts.best : u * qd < expf(y) / ts.s;
      }
      const unsigned stops = __ballot_sync(0xffffffffu, lane < nd && !ok);
      const int k = stops != 0 ? __ffs(stops) - 1 : nd;
      const bool bad = __shfl_sync(0xffffffffu, row_is_bad, k);
      const bool draws = !bad && !greedy;
      const float last_u = __shfl_sync(0xffffffffu, u, n - 1);
      if (lane == k) {
        const bool rejected = stops != 0;
        s_draw = {draws ? k : -1, rejected ? id : -1, rejected && with_q, ts.m, ts.s, ds.m, ds.s, last_u};
        if (rank == 0) {
          a.count[b] = bad ? k : k + 1;
          if (bad || !in) set_status(a.status, bad ? kDevLogits : kDevTokenOob);
        }
        if (greedy && !bad) {
          id = ts.best;
          lp = times_difference(as_float(target[k * a.target_row + id]), ts.m, inv_t) - logf(ts.s);
        }
      }
      if (rank == 0 && lane < n && (lane != k || !draws)) {  // a drawn token is written where it is found
        const bool there = lane < k || (lane == k && !bad);
        tokens[lane] = there ? id : -1;
        if (lps != nullptr) lps[lane] = there ? lp : 0.f;
      }
    }
  }
  asm volatile("barrier.cluster.wait;" ::: "memory");  // every CTA has started
  __syncthreads();
  const Draw d = s_draw;
  if (d.k < 0) return;
  const bool minus = d.minus != 0;
  FinalWeights<T> w = {target + d.k * a.target_row, minus ? draft + d.k * a.draft_row : nullptr, d.pm, d.qm,
                       32.0 * 1.4426950408889634074 / static_cast<double>(temp),
                       minus ? static_cast<double>(d.ps) / d.qs : 0.0, factor, d.drafted};
  // warps take runs of columns, in order
  const int runs = parts * kFinalWarps, run = rank * kFinalWarps + warp;
  const int len = (a.V + 32 * runs - 1) / (32 * runs) * 32;
  const long long first = static_cast<long long>(run) * len;
  const int c0 = static_cast<int>(min(first, static_cast<long long>(a.V)));
  const int c1 = static_cast<int>(min(first + len, static_cast<long long>(a.V)));
  double all_p = 0.0, all_q = 0.0, over_p = 0.0, over_q = 0.0;
  if (minus) {
    warp_columns(w.p, w.q, c0, c1, [&](const float (&xp)[kOverlap], const float (&xq)[kOverlap], int) {
      double e[kOverlap], f[kOverlap];
      w.pe(xp, e);
      w.qe(xq, f);
#pragma unroll
      for (int i = 0; i < kOverlap; ++i) {
        all_p += e[i];
        all_q += f[i];
        const bool over = e[i] > w.r * f[i];
        over_p += over ? e[i] : 0.0;
        over_q += over ? f[i] : 0.0;
      }
    });
    all_q = warp_total(all_q), over_q = warp_total(over_q);
  } else {
    warp_columns<T>(w.p, nullptr, c0, c1, [&](const float (&xp)[kOverlap], const float (&)[kOverlap], int col) {
      double e[kOverlap];
      w.pe(xp, e);
#pragma unroll
      for (int i = 0; i < kOverlap; ++i) {
        all_p += e[i];
        over_p += col + 32 * i == w.drafted ? 0.0 : e[i];
      }
    });
  }
  all_p = warp_total(all_p), over_p = warp_total(over_p);
  if (lane < parts) {  // to every CTA
    double* to = cluster.map_shared_rank(&s_sum[0][0], lane) + run;
    to[0] = all_p, to[kMost] = all_q, to[2 * kMost] = over_p, to[3 * kMost] = over_q;
  }
  cluster.sync();
  // every warp picks the run; with r exact now
  Running<kPer> sums;
  auto entry = [&](int which, int i) { return i < runs ? s_sum[which][i] : 0.0; };
  if (minus) {
    double sp = 0.0, sq = 0.0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sp += entry(0, kPer * lane + i), sq += entry(1, kPer * lane + i);
    w.r = warp_total(sp) / warp_total(sq);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    sums.v[i] = fmax(entry(2, kPer * lane + i) - w.r * entry(3, kPer * lane + i), 0.0);
  sums.scan();
  if (!(sums.all > kNoWeight)) {  // q takes all of p away: draw from p
    w.q = nullptr, w.drafted = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sums.v[i] = entry(0, kPer * lane + i);
    sums.scan();
  }
  const double want = static_cast<double>(d.u) * sums.all;
  double before;
  const int mine = sums.pick(want, &before);
  if (mine / kFinalWarps != rank) return;
  // the run's CTA: an equal share of what is left to each warp, until kLast columns to a lane are
  const long long lo = static_cast<long long>(mine) * len;
  int hi = static_cast<int>(min(lo + len, static_cast<long long>(a.V))), from = static_cast<int>(lo);
  Running<1> part;
  while (hi - from > kFinalThreads * kLast) {
    const int sub = (hi - from + 32 * kFinalWarps - 1) / (32 * kFinalWarps) * 32;
    const int s0 = min(from + warp * sub, hi), s1 = min(s0 + sub, hi);
    const double v = warp_weight(w, s0, s1);
    if (lane == 0) s_sub[warp] = v;
    __syncthreads();
    part.v[0] = lane < kFinalWarps ? s_sub[lane] : 0.0;
    __syncthreads();
    part.scan();
    double skipped;
    from += part.pick(want - before, &skipped) * sub;
    before += skipped;
    hi = min(from + sub, hi);
  }
  const int c = from + tid * kLast;
  Running<kLast> last;
  float xp[kLast], xq[kLast];
#pragma unroll
  for (int i = 0; i < kLast; ++i) {
    xp[i] = c + i < hi ? as_float(w.p[c + i]) : -INFINITY;
    xq[i] = c + i < hi && w.q != nullptr ? as_float(w.q[c + i]) : -INFINITY;
  }
  w.weights(xp, xq, c, 1, last.v);
  last.scan();
  if (lane == 0) s_sub[warp] = last.all;
  __syncthreads();
  part.v[0] = lane < kFinalWarps ? s_sub[lane] : 0.0;
  part.scan();
  double skipped;
  const int at = part.pick(want - before, &skipped);
  if (warp != at) return;
  const int pick = min(from + warp * 32 * kLast + last.pick(want - before - skipped, &before), a.V - 1);
  if (lane == 0) {
    const size_t o = static_cast<size_t>(b) * n + d.k;
    a.tokens[o] = pick;
    if (a.logprobs != nullptr)
      a.logprobs[o] =
          of_difference(as_float(w.p[pick]), d.pm, [temp](float y) { return y / temp; }) - logf(d.ps);
  }
}

}  // namespace wmtp
