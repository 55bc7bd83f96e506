// Rows of logits: log probabilities of given tokens with the entropy and the
// most likely alternatives, and the acceptance of drafted tokens.
//
// One pass over a row keeps, per thread, the running maximum m and, with
// t = (x - m) c and c = log2(e) / T,
//   s = sum 2^t,   a = sum 2^t t,
// from which lse = m / T + ln s and entropy = ln s - ln 2 * a / s.  x - m is
// taken before the scale: that keeps the digits of large logits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>
#include <stdint.h>

#include "status.cuh"

namespace wmtp {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRowThreads = 512;
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

// A row, cut where 16-byte loads may begin and end: `head` columns, `vecs`
// groups of Vec<T>::N, the rest.
template <typename T>
struct Row {
  const T* p;
  int V, head, vecs;
  __device__ __forceinline__ Row(const T* row, int vocab) : p(row), V(vocab) {
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
    head = min(off == 0 ? 0 : Vec<T>::N - off, V);
    vecs = (V - head) / Vec<T>::N;
  }
  // f(x, column) for every column of this thread's share.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int i = threadIdx.x; i < head; i += kRowThreads) f(as_float(p[i]), i);
    const uint4* v = reinterpret_cast<const uint4*>(p + head);
    for (int i = threadIdx.x; i < vecs; i += kRowThreads) {
      float x[Vec<T>::N];
      Vec<T>::unpack(__ldg(v + i), x);
#pragma unroll
      for (int j = 0; j < Vec<T>::N; ++j) f(x[j], head + i * Vec<T>::N + j);
    }
    for (int i = head + vecs * Vec<T>::N + threadIdx.x; i < V; i += kRowThreads) f(as_float(p[i]), i);
  }
};

// Running sums of a part of a row.  m starts at the lowest finite value, so
// that x - m of a masked -inf is -inf and never NaN; NaN and +inf reach s.
struct RowSum {
  float m, s, a;
};

__device__ __forceinline__ RowSum row_sum_empty() { return {-FLT_MAX, 0.f, 0.f}; }

// Moves the sums to a larger maximum.  The clamp keeps 0 * inf out: below
// -1000 the factor is 0 in any case.
__device__ __forceinline__ void row_sum_raise(RowSum& r, float m, float c) {
  const float d = fmaxf((r.m - m) * c, -1000.f);
  const float f = exp2_fast(d);
  r.a = f * (r.a + d * r.s);
  r.s *= f;
  r.m = m;
}

__device__ __forceinline__ void row_sum_add(RowSum& r, float x, float c) {
  const float t = (x - r.m) * c;
  const float e = exp2_fast(t);
  r.s += e;
  r.a += e * fmaxf(t, -1000.f);  // 0 * -inf
}

__device__ __forceinline__ void row_sum_merge(RowSum& r, RowSum o, float c) {
  if (o.m > r.m) row_sum_raise(r, o.m, c);
  if (r.m > o.m) row_sum_raise(o, r.m, c);
  r.s += o.s;
  r.a += o.a;
}

// Whole numbers in the order of the logits: larger first, then lower columns.
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

// The sums of a whole row, on every thread.
template <typename T>
__device__ RowSum row_sums(const Row<T>& row, float c, RowSum* s_part) {
  RowSum r = row_sum_empty();
  row.each([&](float x, int) {
    if (x > r.m) row_sum_raise(r, x, c);
    row_sum_add(r, x, c);
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    RowSum u = {__shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o),
                __shfl_xor_sync(0xffffffffu, r.a, o)};
    row_sum_merge(r, u, c);
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = r;
  __syncthreads();
  r = s_part[0];
  for (int w = 1; w < kRowThreads / 32; ++w) row_sum_merge(r, s_part[w], c);
  return r;
}

// The largest key below `bound`, on every thread.  0: none above -inf.
template <typename T>
__device__ uint64_t row_best(const Row<T>& row, uint64_t bound, uint64_t* s_best) {
  uint64_t best = 0;
  row.each([&](float x, int col) {
    const uint64_t k = logit_key(x, col);
    if (x > -INFINITY && k < bound && k > best) best = k;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t u = __shfl_xor_sync(0xffffffffu, best, o);
    best = u > best ? u : best;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_best[threadIdx.x >> 5] = best;
  __syncthreads();
  best = s_best[0];
  for (int w = 1; w < kRowThreads / 32; ++w) best = s_best[w] > best ? s_best[w] : best;
  return best;
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

// One CTA per row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) logprob_kernel(LogprobArgs a) {
  __shared__ RowSum s_part[kRowThreads / 32];
  __shared__ uint64_t s_best[kRowThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int r = blockIdx.x, tid = threadIdx.x;
  const T* p = static_cast<const T*>(a.logits) + r * a.row_stride;
  const Row<T> row(p, a.V);
  const float inv_t = inverse_temperature(a.temperature, r);
  const RowSum sum = row_sums(row, inv_t * kLog2e, s_part);
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
  uint64_t bound = ~0ull;
  for (int k = 0; k < a.top_k; ++k) {
    if (!bad && bound != 0) bound = row_best(row, bound, s_best);
    if (tid == 0) {
      const size_t o = static_cast<size_t>(r) * a.top_k + k;
      const bool there = !bad && bound != 0;
      a.top_ids[o] = there ? key_col(bound) : -1;
      a.top_logprobs[o] = there ? (key_logit(bound) - sum.m) * inv_t - ln_s : bad ? NAN : -INFINITY;
    }
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

// One CTA per row of the target and of the draft.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) accept_rows_kernel(AcceptArgs a) {
  __shared__ RowSum s_part[kRowThreads / 32];
  __shared__ uint64_t s_best[kRowThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rows_t = a.B * a.num_q;
  const bool target = static_cast<int>(blockIdx.x) < rows_t;
  const int r = target ? blockIdx.x : blockIdx.x - rows_t;
  const int per = target ? a.num_q : a.num_q - 1;
  const int b = r / per, i = r % per;
  const float temp = accept_temperature(a, b);
  const bool greedy = temp == 0.f;
  const int nd = a.num_draft != nullptr ? a.num_draft[b] : a.num_q - 1;
  if (target ? i > nd : (i >= nd || greedy)) return;  // never looked at
  const T* p = target ? static_cast<const T*>(a.target) + b * a.target_batch + i * a.target_row
                      : static_cast<const T*>(a.draft) + b * a.draft_batch + i * a.draft_row;
  const Row<T> row(p, a.V);
  const float inv_t = greedy ? 1.f : (temp > 0.f && temp < INFINITY) ? 1.f / temp : NAN;
  const RowSum sum = row_sums(row, inv_t * kLog2e, s_part);
  RowStat st = {sum.m, sum.s, -1, row_bad(sum, inv_t) || sum.s == 0.f};
  if (greedy && !st.bad) st.best = key_col(row_best(row, ~0ull, s_best));
  if (threadIdx.x == 0) a.stats[blockIdx.x] = st;
}

// The weights of the token that follows: p, or what p has above q.  In 64
// bits: a draw takes the token in which the cumulated weight passes u, and with
// V tokens a relative error e of that sum moves the border over a token with
// probability V e (1e-2 at V = 131072 and the 1e-7 of fp32).
template <typename T>
struct FinalWeights {
  const T *p, *q;  // q NULL: none, or all of it on `drafted`
  double pm, qm, inv_t;
  double p_scale, q_scale;  // 1 / sum
  int drafted;              // -1: no draft to take away
  bool residual;
  __device__ __forceinline__ double pe(int col) const { return exp((as_float(p[col]) - pm) * inv_t); }
  __device__ __forceinline__ double qe(int col) const { return exp((as_float(q[col]) - qm) * inv_t); }
  __device__ __forceinline__ double operator()(int col) const {
    if (!residual) return pe(col);
    if (q == nullptr) return col == drafted ? 0.0 : pe(col);
    return fmax(pe(col) * p_scale - qe(col) * q_scale, 0.0);
  }
};

// One CTA per sequence.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) accept_kernel(AcceptArgs a) {
  __shared__ double s_sum[kRowThreads];
  __shared__ int s_pick;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int b = blockIdx.x, tid = threadIdx.x, n = a.num_q;
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
  for (int i = tid; i < n; i += kRowThreads) {
    tokens[i] = -1;
    if (lps != nullptr) lps[i] = 0.f;
  }
  __syncthreads();
  if (nd < 0 || nd > n - 1) {
    if (tid == 0) {
      set_status(a.status, kDevLenOob);
      a.count[b] = 0;
    }
    return;
  }
  auto logprob = [&](int i, int id) {
    return (as_float(target[i * a.target_row + id]) - ts[i].m) * inv_t - logf(ts[i].s);
  };
  // every thread takes the same decisions; thread 0 writes them down
  int k = 0;
  bool bad = false, rejected = false;
  for (; k < nd; ++k) {
    const int id = d[k];
    const bool in = id >= 0 && id < a.V;
    if (ts[k].bad || (!greedy && draft != nullptr && ds[k].bad)) {
      bad = true;
      break;
    }
    if (!in && tid == 0) set_status(a.status, kDevTokenOob);
    bool ok = false;
    if (greedy) {
      ok = in && id == ts[k].best;
    } else if (in) {
      const float p = expf((as_float(target[k * a.target_row + id]) - ts[k].m) * inv_t) / ts[k].s;
      const float q =
          draft == nullptr ? 1.f : expf((as_float(draft[k * a.draft_row + id]) - ds[k].m) * inv_t) / ds[k].s;
      ok = a.uniforms[static_cast<size_t>(b) * n + k] * q < p;
    }
    if (!ok) {
      rejected = true;
      break;
    }
    if (tid == 0) {
      tokens[k] = id;
      if (lps != nullptr) lps[k] = logprob(k, id);
    }
  }
  bad = bad || ts[k].bad;
  if (bad) {
    if (tid == 0) {
      set_status(a.status, kDevLogits);
      a.count[b] = k;
    }
    return;
  }
  int pick;
  if (greedy) {
    pick = ts[k].best;
  } else {
    const bool minus = rejected && draft != nullptr;
    FinalWeights<T> w = {target + k * a.target_row, minus ? draft + k * a.draft_row : nullptr, ts[k].m,
                         minus ? ds[k].m : 0.0, 1.0 / static_cast<double>(temp), 1.0, 1.0, rejected ? d[k] : -1,
                         rejected};
    // thread shares are runs of columns, in order
    const int share = (a.V + kRowThreads - 1) / kRowThreads;
    const int c0 = min(tid * share, a.V), c1 = min(c0 + share, a.V);
    auto total_of = [&](auto f) {
      double mine = 0.0, all = 0.0;
      for (int c = c0; c < c1; ++c) mine += f(c);
      __syncthreads();
      s_sum[tid] = mine;
      __syncthreads();
      for (int i = 0; i < kRowThreads; ++i) all += s_sum[i];
      return all;
    };
    if (minus) {
      w.p_scale = 1.0 / total_of([&](int c) { return w.pe(c); });
      w.q_scale = 1.0 / total_of([&](int c) { return w.qe(c); });
    }
    double total = total_of(w);
    if (!(total > 0.0)) {  // q takes all of p away: draw from p
      w.residual = false;
      total = total_of(w);
    }
    const double want = static_cast<double>(a.uniforms[static_cast<size_t>(b) * n + n - 1]) * total;
    if (tid == 0) {
      double before = 0.0;
      int i = 0, last = -1;
      for (; i < kRowThreads; ++i) {
        if (s_sum[i] > 0.0) last = i;
        if (before + s_sum[i] > want) break;
        before += s_sum[i];
      }
      if (i == kRowThreads) {  // u * total came out as total: the last token with a weight
        i = last;
        before -= s_sum[i];
      }
      int c = min(i * share, a.V), end = min(c + share, a.V), found = -1;
      for (; c < end; ++c) {
        const double v = w(c);
        if (v > 0.0) found = c;
        before += v;
        if (before > want) break;
      }
      s_pick = found;
    }
    __syncthreads();
    pick = s_pick;
  }
  if (tid == 0) {
    tokens[k] = pick;
    if (lps != nullptr) lps[k] = logprob(k, pick);
    a.count[b] = k + 1;
  }
}

}  // namespace wmtp
