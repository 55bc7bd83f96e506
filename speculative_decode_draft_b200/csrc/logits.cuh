// Rows of logits: log probabilities of given tokens with the entropy and the
// most likely alternatives, and the acceptance of drafted tokens.
//
// One pass over a row keeps, per thread, the running maximum m and, with
// t = (x - m) c and c = log2(e) / T,
//   s = sum 2^t,   a = sum 2^t t,
// from which lse = m / T + ln s and entropy = ln s - ln 2 * a / s.  x - m is
// taken before the scale: that keeps the digits of large logits, and a row
// of the type's lowest value has differences of 0.
//
// A row is read once, by a cluster of up to 8 CTAs where there are few rows;
// the parts' sums meet in the shared memory of the cluster's first CTA.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <stdint.h>

#include <type_traits>

#include "status.cuh"

namespace wmtp {

namespace cg = cooperative_groups;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowUnroll = 4;      // 16-byte loads in flight per thread
constexpr int kMaxCluster = 8;     // CTAs that share a row
constexpr int kGroups = kRowThreads / 4;
constexpr int kMaxCandidates = 1024;
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

// 16 bytes of a row as floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y), x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
};

// Two fp32 values in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// The larger of x and lo; NaN stays NaN.
__device__ __forceinline__ float at_least(float x, float lo) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(lo));
  return r;
}

// The largest value of 16 bytes (NaN aside).
__device__ __forceinline__ float vec_max(const float (&x)[4]) { return fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])); }
__device__ __forceinline__ float vec_max(const float (&x)[8]) {
  return fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
}

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
  __device__ __forceinline__ uint4 load(int i) const {
    const int c = col(i);
    if (c >= 0 && c + N <= V) return __ldg(reinterpret_cast<const uint4*>(p + c));
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

// Running sums of a part of a row.  m starts at the lowest finite value, so
// that x - m of a masked -inf is -inf and never NaN; NaN and +inf reach s.
struct RowSum {
  float m, s, a;
};

// Moves the sums to a larger maximum.  The clamp keeps 0 * inf out: below
// -1000 the factor is 0 in any case.
__device__ __forceinline__ void row_sum_raise(RowSum& r, float m, float c) {
  const float d = fmaxf((r.m - m) * c, -1000.f);
  const float f = exp2_fast(d);
  r.a = f * (r.a + d * r.s);
  r.s *= f;
  r.m = m;
}

__device__ __forceinline__ void row_sum_merge(RowSum& r, RowSum o, float c) {
  if (o.m > r.m) row_sum_raise(r, o.m, c);
  if (r.m > o.m) row_sum_raise(o, r.m, c);
  r.s += o.s;
  r.a += o.a;
}

// A thread's sums, and its largest logit with the first vec that holds it.
struct ThreadSum {
  RowSum r;
  float best;
  int vec;
};

// Sums of this thread's share of a part.  Per logit: the widening of its 16
// bits, a maximum, and 2^x on the special function unit; the difference, the
// scale and the two sums take half an instruction each.
template <typename T>
__device__ __forceinline__ ThreadSum part_sums(const Part<T>& part, float c) {
  constexpr int N = Vec<T>::N;
  ThreadSum z = {{-FLT_MAX, 0.f, 0.f}, -INFINITY, part.v0};
  const uint64_t c2 = pack2(c, c);
  auto step = [&](const uint4 (&u)[kRowUnroll], int i, int n) {
    float x[kRowUnroll][N], top[kRowUnroll], most = -INFINITY;
#pragma unroll
    for (int k = 0; k < kRowUnroll; ++k) {
      if (k >= n) break;
      Vec<T>::unpack(u[k], x[k]);
      top[k] = vec_max(x[k]);
      most = fmaxf(most, top[k]);
    }
    if (most > z.best) {
#pragma unroll
      for (int k = kRowUnroll - 1; k >= 0; --k)
        if (k < n && top[k] == most) z.vec = i + k * kRowThreads;
      z.best = most;
      if (most > z.r.m) row_sum_raise(z.r, most, c);
    }
    const uint64_t m2 = pack2(-z.r.m, -z.r.m);
    uint64_t s2 = pack2(z.r.s, 0.f), a2 = pack2(z.r.a, 0.f);
#pragma unroll
    for (int k = 0; k < kRowUnroll; ++k) {
      if (k >= n) break;
#pragma unroll
      for (int j = 0; j < N; j += 2) {
        float t0, t1;
        unpack2(mul2(add2(pack2(x[k][j], x[k][j + 1]), m2), c2), t0, t1);
        t0 = at_least(t0, -1000.f), t1 = at_least(t1, -1000.f);  // 0 * -inf
        const uint64_t e2 = pack2(exp2_fast(t0), exp2_fast(t1));
        s2 = add2(s2, e2);
        a2 = fma2(e2, pack2(t0, t1), a2);
      }
    }
    float lo, hi;
    unpack2(s2, lo, hi);
    z.r.s = lo + hi;
    unpack2(a2, lo, hi);
    z.r.a = lo + hi;
  };
  int i = part.v0 + threadIdx.x;
  for (; i + (kRowUnroll - 1) * kRowThreads < part.v1; i += kRowUnroll * kRowThreads) {
    uint4 u[kRowUnroll];
#pragma unroll
    for (int k = 0; k < kRowUnroll; ++k) u[k] = part.load(i + k * kRowThreads);
    step(u, i, kRowUnroll);
  }
  for (; i < part.v1; i += kRowThreads) {
    uint4 u[kRowUnroll];
    u[0] = part.load(i);
    step(u, i, 1);
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
    r = s_part[threadIdx.x & (kRowWarps - 1)];
    halve(kRowWarps / 2);
  }
  return r;
}

// The largest key of the part below `bound`, on every thread.  0: none above -inf.
template <typename T>
__device__ uint64_t part_best(const Part<T>& part, uint64_t bound, uint64_t* s_best) {
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
  for (int w = 1; w < kRowWarps; ++w) best = max_key(best, s_best[w]);
  return best;
}

struct TopShared {
  uint64_t keys[kGroups];
  uint64_t cand[kMaxCandidates];
  uint64_t warp_best[kRowWarps];
  uint64_t bound;
  int group[kMaxTop];
  int count;
};

// The part's `top_k` largest keys, in order, to out[0 .. top_k).
//
// Four threads are a group, and a key at or below its best logit's is known
// from the pass over the row.  The top_k-th largest of the groups' keys bounds
// the part's top_k-th logit from below, and what lies above it is in the
// top_k groups that reach it: only their vecs are read again (from L2), and
// the few logits above the bound sorted by counting.  Should one group hold so
// many of them that the list overflows, the keys are taken one pass each.
template <typename T>
__device__ void part_top(const Part<T>& part, const ThreadSum& z, int top_k, TopShared& sh, uint64_t* out) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x;
  // the vec's last column: at or below the best logit's own key
  uint64_t key = z.best > -INFINITY ? logit_key(z.best, part.col(z.vec) + N - 1) : 0;
#pragma unroll
  for (int o = 2; o > 0; o >>= 1) key = max_key(key, __shfl_xor_sync(0xffffffffu, key, o));
  if ((tid & 3) == 0) sh.keys[tid >> 2] = key;
  if (tid == 0) sh.count = 0, sh.bound = 0;
  for (int i = tid; i < top_k; i += kRowThreads) sh.group[i] = -1, out[i] = 0;
  __syncthreads();
  // each thread ranks its group's key among a quarter of the keys
  int rank = 0;
#pragma unroll 8
  for (int i = tid & 3; i < kGroups; i += 4) rank += sh.keys[i] > key;
  rank += __shfl_xor_sync(0xffffffffu, rank, 1);
  rank += __shfl_xor_sync(0xffffffffu, rank, 2);
  if ((tid & 3) == 0 && key != 0 && rank < top_k) {
    sh.group[rank] = tid >> 2;
    if (rank == top_k - 1) sh.bound = key;
  }
  __syncthreads();
  const uint64_t bound = sh.bound;
  const float least = bound != 0 ? key_logit(bound) : -FLT_MAX;
  const int rounds = (part.v1 - part.v0 + kRowThreads - 1) / kRowThreads;
  for (int i = tid; i < top_k * rounds * 4; i += kRowThreads) {
    const int g = sh.group[i / (rounds * 4)];
    const int v = part.v0 + (i / 4 % rounds) * kRowThreads + g * 4 + (i & 3);
    if (g < 0 || v >= part.v1) continue;
    float x[N];
    Vec<T>::unpack(part.load(v), x);
    if (!(vec_max(x) >= least)) continue;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!(x[j] >= least)) continue;
      const uint64_t k = logit_key(x[j], part.col(v) + j);
      if (k < bound) continue;
      const int at = atomicAdd(&sh.count, 1);
      if (at < kMaxCandidates) sh.cand[at] = k;
    }
  }
  __syncthreads();
  const int n = sh.count;
  if (n <= kMaxCandidates) {
    for (int i = tid; i < n; i += kRowThreads) {
      const uint64_t k = sh.cand[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += sh.cand[j] > k;
      if (r < top_k) out[r] = k;
    }
  } else {
    uint64_t below = ~0ull;
    for (int i = 0; i < top_k && below != 0; ++i) {
      below = part_best(part, below, sh.warp_best);
      if (tid == 0) out[i] = below;
    }
  }
  __syncthreads();
}

// A row's temperature: 1 / T, or NaN for one that is no temperature.
__device__ __forceinline__ float inverse_temperature(const float* temperature, int row) {
  const float t = temperature != nullptr ? temperature[row] : 1.f;
  return (t > 0.f && t < INFINITY) ? 1.f / t : NAN;
}

// NaN or +inf somewhere in the row, or no temperature.
__device__ __forceinline__ bool row_bad(const RowSum& r, float inv_t) {
  return !(r.s < INFINITY) || !(r.m < INFINITY) || !(inv_t > 0.f && inv_t < INFINITY);
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

// One cluster per row; its first CTA joins the parts and writes the results.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) logprob_kernel(LogprobArgs a) {
  __shared__ RowSum s_part[kRowWarps];
  __shared__ RowSum s_sums[kMaxCluster];
  __shared__ uint64_t s_top[kMaxCluster * kMaxTop];
  __shared__ uint64_t s_mine[kMaxTop];
  __shared__ TopShared s_sel;
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), rank = cluster.block_rank();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const int r = blockIdx.x / parts, tid = threadIdx.x;
  const T* p = static_cast<const T*>(a.logits) + r * a.row_stride;
  const Part<T> part(p, a.V, rank, parts);
  const float inv_t = inverse_temperature(a.temperature, r), c = inv_t * kLog2e;
  const ThreadSum z = part_sums(part, c);
  RowSum sum = block_sums(z.r, c, s_part);
  if (a.top_k > 0) part_top(part, z, a.top_k, s_sel, parts > 1 ? s_mine : s_top);
  // the first CTA has started by now, so its shared memory may be written
  if (parts > 1) {
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (tid == 0) cluster.map_shared_rank(s_sums, 0)[rank] = sum;
    uint64_t* top = cluster.map_shared_rank(s_top, 0) + rank * kMaxTop;
    for (int i = tid; i < a.top_k; i += kRowThreads) top[i] = s_mine[i];
    cluster.sync();
    if (rank != 0) return;
  } else {
    if (tid == 0) s_sums[0] = sum;
    __syncthreads();
  }
  sum = s_sums[0];
  for (int i = 1; i < parts; ++i) row_sum_merge(sum, s_sums[i], c);
  const bool bad = row_bad(sum, inv_t), none = sum.s == 0.f;
  const float ln_s = bad ? NAN : logf(sum.s);
  if (bad && tid == 0) set_status(a.status, kDevLogits);
  for (int j = tid; j < a.num_tokens; j += kRowThreads) {
    const int id = a.tokens[static_cast<size_t>(r) * a.num_tokens + j];
    const bool in = id >= 0 && id < a.V;
    if (!in && id != -1) set_status(a.status, kDevTokenOob);
    a.logprobs[static_cast<size_t>(r) * a.num_tokens + j] =
        bad ? NAN : (none || !in) ? -INFINITY : (as_float(p[id]) - sum.m) * inv_t - ln_s;
  }
  if (tid == 0) {
    if (a.lse != nullptr) a.lse[r] = bad ? NAN : none ? -INFINITY : sum.m * inv_t + ln_s;
    if (a.entropy != nullptr) a.entropy[r] = bad ? NAN : none ? 0.f : ln_s - kLn2 * sum.a / sum.s;
  }
  // every part's list is in order: a key's place is its own in its list plus,
  // in each other list, the number of keys above it
  const size_t o = static_cast<size_t>(r) * a.top_k;
  for (int i = tid; i < parts * a.top_k; i += kRowThreads) {
    const int l = i / a.top_k, at = i % a.top_k;
    const uint64_t key = s_top[l * kMaxTop + at];
    int place = at;
    if (key == 0 || bad) continue;
    for (int other = 0; other < parts; ++other) {
      if (other == l) continue;
      int lo = 0, hi = a.top_k;  // the first key below this one
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (s_top[other * kMaxTop + mid] > key)
          lo = mid + 1;
        else
          hi = mid;
      }
      place += lo;
    }
    if (place >= a.top_k) continue;
    a.top_ids[o + place] = key_col(key);
    a.top_logprobs[o + place] = (key_logit(key) - sum.m) * inv_t - ln_s;
  }
  if (a.top_k == 0) return;
  int have = 0;  // places without a token
  for (int l = 0; l < parts; ++l) {
    int lo = 0, hi = a.top_k;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (s_top[l * kMaxTop + mid] != 0)
        lo = mid + 1;
      else
        hi = mid;
    }
    have += lo;
  }
  for (int i = (bad ? 0 : have) + tid; i < a.top_k; i += kRowThreads) {
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
__global__ void __launch_bounds__(kRowThreads) accept_rows_kernel(AcceptArgs a) {
  __shared__ RowSum s_part[kRowWarps];
  __shared__ RowSum s_sums[kMaxCluster];
  __shared__ uint64_t s_best[kMaxCluster];
  __shared__ uint64_t s_warp[kRowWarps];
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), rank = cluster.block_rank(), tid = threadIdx.x;
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
  if (target ? i > nd : (i >= nd || greedy)) return;  // never looked at
  if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  const T* p = target ? static_cast<const T*>(a.target) + b * a.target_batch + i * a.target_row
                      : static_cast<const T*>(a.draft) + b * a.draft_batch + i * a.draft_row;
  const Part<T> part(p, a.V, rank, parts);
  const float inv_t = greedy ? 1.f : (temp > 0.f && temp < INFINITY) ? 1.f / temp : NAN;
  const float c = inv_t * kLog2e;
  const ThreadSum z = part_sums(part, c);
  RowSum sum = block_sums(z.r, c, s_part);
  uint64_t best = 0;
  if (greedy) {  // the lowest column with the largest logit
    if (z.best > -INFINITY) {
      float x[Vec<T>::N];
      Vec<T>::unpack(part.load(z.vec), x);
#pragma unroll
      for (int j = Vec<T>::N - 1; j >= 0; --j)
        if (x[j] == z.best) best = logit_key(x[j], part.col(z.vec) + j);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = max_key(best, __shfl_xor_sync(0xffffffffu, best, o));
    if ((tid & 31) == 0) s_warp[tid >> 5] = best;
    __syncthreads();
    for (int w = 0; w < kRowWarps; ++w) best = max_key(best, s_warp[w]);
  }
  if (parts > 1) {
    asm volatile("barrier.cluster.wait;" ::: "memory");
    if (tid == 0) {
      cluster.map_shared_rank(s_sums, 0)[rank] = sum;
      cluster.map_shared_rank(s_best, 0)[rank] = best;
    }
    cluster.sync();
  } else if (tid == 0) {
    s_sums[0] = sum, s_best[0] = best;
  }
  if (rank != 0 || tid != 0) return;
  sum = s_sums[0];
  for (int k = 1; k < parts; ++k) {
    row_sum_merge(sum, s_sums[k], c);
    best = max_key(best, s_best[k]);
  }
  a.stats[at] = {sum.m, sum.s, best != 0 ? key_col(best) : -1, row_bad(sum, inv_t) || sum.s == 0.f};
}

// exp in 64 bits, for weights: 2^(u / 32) with u = k + r, |r| <= 1/2, is
// 2^(k div 32) * 2^((k mod 32) / 32) * (1 + z + z^2/2 + z^3/6 + z^4/24),
// z = r ln2 / 32; the Taylor series' next term is below 1.3e-12.  The 32
// factors 2^(j / 32) are held by a warp's lanes.  All lanes take part.
__device__ __forceinline__ double lane_factor() { return exp2((threadIdx.x & 31) / 32.0); }
__device__ __forceinline__ double exp_weight(double u, double factor) {
  constexpr double kMagic = 6755399441055744.0;  // 1.5 * 2^52: rounds to whole numbers
  constexpr double c1 = 0.69314718055994530942 / 32, c2 = c1 * c1 / 2, c3 = c1 * c1 * c1 / 6, c4 = c1 * c1 * c1 * c1 / 24;
  const bool none = !(u > -32000.0);  // below 2^-1000: 0
  u = none ? 0.0 : u;
  const double kd = u + kMagic;
  const int k = __double2loint(kd);
  const double r = u - (kd - kMagic);
  const double z = r * fma(r, fma(r, fma(r, c4, c3), c2), c1);
  const double f = __shfl_sync(0xffffffffu, factor, k & 31);
  const double e = fma(f, z, f);
  return none ? 0.0 : __hiloint2double(__double2hiint(e) + (k >> 5) * (1 << 20), __double2loint(e));
}

// The weights of the token that follows: p, or what p has above q.  In 64
// bits: a draw takes the token in which the cumulated weight passes u, and with
// V tokens a relative error e of that sum moves the border over a token with
// probability V e (1e-2 at V = 131072 and the 1e-7 of fp32).
template <typename T>
struct FinalWeights {
  const T *p, *q;  // q NULL: none, or all of it on `drafted`
  double pm, qm, scale;     // 32 log2(e) / T
  double p_part, q_part;    // 1 / sum
  double factor;
  int drafted;  // -1: no draft to take away
  bool residual;
  __device__ __forceinline__ double pe(float x) const { return exp_weight((x - pm) * scale, factor); }
  __device__ __forceinline__ double qe(float x) const { return exp_weight((x - qm) * scale, factor); }
  __device__ __forceinline__ double operator()(float xp, float xq, int col) const {
    const double e = pe(xp);
    if (!residual) return e;
    if (q == nullptr) return col == drafted ? 0.0 : e;
    return fmax(e * p_part - qe(xq) * q_part, 0.0);
  }
};

__device__ __forceinline__ double warp_total(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

constexpr int kFinalUnroll = 8;

// f(logit of p, logit of q, column) of the columns [c0, c1), a warp's; columns
// behind c1 are masked.  32 columns at a time, kFinalUnroll loads in flight.
template <typename T, typename F>
__device__ __forceinline__ void warp_columns(const FinalWeights<T>& w, bool with_q, int c0, int c1, F f) {
  const int lane = threadIdx.x & 31;
  for (int base = c0; base < c1; base += 32 * kFinalUnroll) {
    float xp[kFinalUnroll], xq[kFinalUnroll];
#pragma unroll
    for (int k = 0; k < kFinalUnroll; ++k) {
      const int c = base + 32 * k + lane;
      xp[k] = c < c1 ? as_float(w.p[c]) : -INFINITY;
      xq[k] = with_q && c < c1 ? as_float(w.q[c]) : -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < kFinalUnroll; ++k)
      if (base + 32 * k < c1) f(xp[k], xq[k], base + 32 * k + lane);
  }
}

template <typename T>
__device__ __forceinline__ double warp_weight(const FinalWeights<T>& w, int c0, int c1) {
  double sum = 0.0;
  warp_columns(w, w.residual && w.q != nullptr, c0, c1, [&](float xp, float xq, int col) { sum += w(xp, xq, col); });
  return warp_total(sum);
}

// The first of n sums (at most 128, in shared memory) above 0 at which the
// running total passes `want`, and the total before it; where rounding lets none
// pass, the last one above 0.  *all: the total.  The same on every lane.
__device__ __forceinline__ int warp_pick(const double* sums, int n, double want, double* before, double* all) {
  const int lane = threadIdx.x & 31;
  double v[4], mine = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = 4 * lane + i < n ? sums[4 * lane + i] : 0.0;
    mine += v[i];
  }
  double scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += u;
  }
  *all = __shfl_sync(0xffffffffu, scan, 31);
  double b = __shfl_up_sync(0xffffffffu, scan, 1);
  if (lane == 0) b = 0.0;
  int at = -1, last = -1;
  double at_before = 0.0, last_before = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (at < 0 && v[i] > 0.0 && b + v[i] > want) at = 4 * lane + i, at_before = b;
    if (v[i] > 0.0) last = 4 * lane + i, last_before = b;
    b += v[i];
  }
  const unsigned hit = __ballot_sync(0xffffffffu, at >= 0), any = __ballot_sync(0xffffffffu, last >= 0);
  if (hit != 0) {
    *before = __shfl_sync(0xffffffffu, at_before, __ffs(hit) - 1);
    return __shfl_sync(0xffffffffu, at, __ffs(hit) - 1);
  }
  const int from = any != 0 ? 31 - __clz(any) : 0;
  *before = __shfl_sync(0xffffffffu, last_before, from);
  return __shfl_sync(0xffffffffu, last, from);
}

// One cluster per sequence.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) accept_kernel(AcceptArgs a) {
  constexpr int kMost = kMaxCluster * kRowWarps;
  __shared__ double s_p[kMost], s_q[kMost], s_w[2][kMost], s_sub[kRowWarps];
  const cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), rank = cluster.block_rank();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x / parts, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.num_q;
  const float temp = accept_temperature(a, b);
  const bool greedy = temp == 0.f;
  const float inv_t = greedy ? 1.f : 1.f / temp;
  const int nd = a.num_draft != nullptr ? a.num_draft[b] : n - 1;
  const T* target = static_cast<const T*>(a.target) + b * a.target_batch;
  const T* draft = a.draft != nullptr ? static_cast<const T*>(a.draft) + b * a.draft_batch : nullptr;
  const RowStat* ts = a.stats + static_cast<size_t>(b) * n;
  const RowStat* ds = a.stats + static_cast<size_t>(a.B) * n + static_cast<size_t>(b) * (n - 1);
  const int32_t* d = a.draft_tokens + static_cast<size_t>(b) * (n - 1);
  int32_t* tokens = a.tokens + static_cast<size_t>(b) * n;
  float* lps = a.logprobs != nullptr ? a.logprobs + static_cast<size_t>(b) * n : nullptr;
  const bool writes = rank == 0 && warp == 0;
  if (nd < 0 || nd > n - 1) {
    if (writes && lane < n) {
      tokens[lane] = -1;
      if (lps != nullptr) lps[lane] = 0.f;
    }
    if (writes && lane == 0) {
      set_status(a.status, kDevLenOob);
      a.count[b] = 0;
    }
    return;
  }
  // every warp takes the same decisions, a lane for each drafted token
  int id = -1;
  float lp = 0.f;
  bool ok = false, row_is_bad = false, in = true;
  if (lane <= nd) {
    const RowStat t = ts[lane];
    row_is_bad = t.bad;
    if (lane < nd) {
      id = d[lane];
      in = id >= 0 && id < a.V;
      const bool with_q = !greedy && draft != nullptr;
      const RowStat q = with_q ? ds[lane] : RowStat();
      if (with_q && q.bad) row_is_bad = true;
      if (in && !row_is_bad) {
        const float y = (as_float(target[lane * a.target_row + id]) - t.m) * inv_t;
        lp = y - logf(t.s);
        const float qd = with_q ? expf((as_float(draft[lane * a.draft_row + id]) - q.m) * inv_t) / q.s : 1.f;
        ok = greedy ? id == t.best : a.uniforms[static_cast<size_t>(b) * n + lane] * qd < expf(y) / t.s;
      }
    }
  }
  const unsigned stops = __ballot_sync(0xffffffffu, lane < nd && !ok);
  const int k = stops != 0 ? __ffs(stops) - 1 : nd;
  const bool bad = __shfl_sync(0xffffffffu, row_is_bad, k);
  const bool stray = __shfl_sync(0xffffffffu, !in, k);
  if (writes) {
    if (lane < n && (lane != k || bad)) {  // the token that follows is written where it is found
      tokens[lane] = lane < k ? id : -1;
      if (lps != nullptr) lps[lane] = lane < k ? lp : 0.f;
    }
    if (lane == 0) {
      a.count[b] = bad ? k : k + 1;
      if (bad || stray) set_status(a.status, bad ? kDevLogits : kDevTokenOob);
    }
  }
  if (bad) return;
  const RowStat pk = ts[k];
  auto emit = [&](int pick) {
    tokens[k] = pick;
    if (lps != nullptr) lps[k] = (as_float(target[k * a.target_row + pick]) - pk.m) * inv_t - logf(pk.s);
  };
  if (greedy) {
    if (writes && lane == 0) emit(pk.best);
    return;
  }
  const bool rejected = stops != 0, minus = rejected && draft != nullptr;
  FinalWeights<T> w = {target + k * a.target_row, minus ? draft + k * a.draft_row : nullptr, pk.m,
                       minus ? ds[k].m : 0.0, 32.0 * 1.4426950408889634074 / static_cast<double>(temp), 1.0, 1.0,
                       lane_factor(), rejected ? d[k] : -1, rejected};
  // warps take runs of columns, in order
  const int runs = parts * kRowWarps, run = rank * kRowWarps + warp;
  const int len = (a.V + 32 * runs - 1) / (32 * runs) * 32;
  const long long first = static_cast<long long>(run) * len;
  const int c0 = static_cast<int>(min(first, static_cast<long long>(a.V)));
  const int c1 = static_cast<int>(min(first + len, static_cast<long long>(a.V)));
  auto share = [&](double* sums, double v) {  // to every CTA of the cluster
    if (lane < parts) cluster.map_shared_rank(sums, lane)[run] = v;
  };
  double before = 0.0, total = 0.0;
  cluster.sync();  // every CTA has started
  if (minus) {
    double ps = 0.0, qs = 0.0;
    warp_columns(w, true, c0, c1, [&](float xp, float xq, int) {
      ps += w.pe(xp);
      qs += w.qe(xq);
    });
    share(s_p, warp_total(ps));
    share(s_q, warp_total(qs));
    cluster.sync();
    warp_pick(s_p, runs, 0.0, &before, &total);
    w.p_part = 1.0 / total;
    warp_pick(s_q, runs, 0.0, &before, &total);
    w.q_part = 1.0 / total;
  }
  const double u = a.uniforms[static_cast<size_t>(b) * n + n - 1];
  const double* sums = s_w[0];
  share(s_w[0], warp_weight(w, c0, c1));
  cluster.sync();
  warp_pick(sums, runs, 0.0, &before, &total);
  if (!(total > 0.0)) {  // q takes all of p away: draw from p
    w.residual = false;
    sums = s_w[1];
    share(s_w[1], warp_weight(w, c0, c1));
    cluster.sync();
    warp_pick(sums, runs, 0.0, &before, &total);
  }
  const double want = u * total;
  const int mine = warp_pick(sums, runs, want, &before, &total);
  if (mine / kRowWarps != rank) return;
  // the run's CTA: a sixteenth of what is left to each warp, until two steps of 32 columns are left
  long long lo = static_cast<long long>(mine) * len;
  int hi = static_cast<int>(min(lo + len, static_cast<long long>(a.V))), from = static_cast<int>(lo);
  while (hi - from > 64) {
    const int sub = (hi - from + 32 * kRowWarps - 1) / (32 * kRowWarps) * 32;
    const int s0 = min(from + warp * sub, hi), s1 = min(s0 + sub, hi);
    const double v = warp_weight(w, s0, s1);
    if (lane == 0) s_sub[warp] = v;
    __syncthreads();
    double skipped, all;
    const int at = warp_pick(s_sub, kRowWarps, want - before, &skipped, &all);
    __syncthreads();
    before += skipped;
    from = from + max(at, 0) * sub;
    hi = min(from + sub, hi);
  }
  if (warp != 0) return;
  int pick = -1, last = -1;
  warp_columns(w, w.residual && w.q != nullptr, from, hi, [&](float xp, float xq, int col) {
    const double v = w(xp, xq, col);
    double scan = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double up = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += up;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, v > 0.0 && before + scan > want);
    const unsigned any = __ballot_sync(0xffffffffu, v > 0.0);
    if (pick < 0 && hit != 0) pick = col - lane + __ffs(hit) - 1;
    if (any != 0) last = col - lane + 31 - __clz(any);
    before += __shfl_sync(0xffffffffu, scan, 31);
  });
  if (lane == 0) emit(pick >= 0 ? pick : last);
}

}  // namespace wmtp
