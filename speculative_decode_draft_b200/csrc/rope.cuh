// Queries and keys encoded for the attention: the RMS norm of each head, the
// position rotation, and the write of K and V into the paged cache.
//
//   y = x * rsqrt(mean(x^2) + eps) * (weight + offset)
//   (a, b) -> factor * (a cos - b sin, b cos + a sin),  angle = 2 pi t turn / 2^64
//
// All in fp32, rounded to bf16 once, at the store.  The angle: t * turn is
// taken modulo 2^64, which drops whole turns exactly, and its upper 32 bits
// are the fraction of a turn to 2^-32; far positions are as exact as near ones
// (t * f in fp32 would be off by 0.06 rad at a million tokens).
//
// Bound by memory: each head row is read and written once, (in + 2) D bytes.
// The instructions come close, so they are few: the cosines of a lane's four
// pairs are worked out once for all rows of its slice, products go in packed pairs, and
// heads of 64, 128 and 256 have kernels of their own without tests for the head's
// end.  32768 tokens of 20 heads of 256 in bf16: 133 us, 5.0 TB/s, 77% of a
// copy's rate (a warp per head row, angles worked out for each: 513 us), interleaved
// 138, in fp32 170, 90%; 4 blocks of 64 registers per SM (3 of 80: 152 us), 2 rows in
// flight (1: 155, 4: 130 but 7.9 instead of 7.5 us for 1537 tokens).  64 registers
// spill 36 to 108 bytes a thread, 248 for fp32 in chunks of 1.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>
#include <string.h>

#include "f32x2.cuh"
#include "status.cuh"

namespace wmtp {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = 32 * kRopeWarps;
constexpr int kRopeMaxDim = 256;
constexpr int kRopeRows = 2;  // loaded before the first is used

struct RopeArgs {
  const void *q, *k, *v;  // NULL: absent
  long long q_token, q_head, k_token, k_head, v_token, v_head;  // strides, elements
  const int32_t* positions;
  const int64_t* slots;  // NULL: no cache
  __nv_bfloat16 *k_pool, *v_pool;
  long long num_slots;  // num_pages * page_size
  int page_size;
  const void *qw, *kw;  // NULL: no norm
  int weight_f32;
  float offset, eps;
  const uint64_t* turn;
  int rotary_dim, interleaved;
  float factor;
  __nv_bfloat16 *q_out, *k_out;
  int tokens, Hq, Hkv, D;
  int lanes, slices, per_slice;
  float inv_dim;
  int32_t* status;
};

// P elements, read and written at once.
template <int Bytes>
struct Raw;
template <>
struct Raw<2> {
  using Type = uint16_t;
};
template <>
struct Raw<4> {
  using Type = uint32_t;
};
template <>
struct Raw<8> {
  using Type = uint2;
};
template <>
struct Raw<16> {
  using Type = uint4;
};

template <typename In, int P>
struct Chunk {
  using Type = typename Raw<P * sizeof(In)>::Type;
  static __device__ __forceinline__ Type load(const In* p) { return *reinterpret_cast<const Type*>(p); }
  static __device__ __forceinline__ void widen(Type raw, float (&x)[P]) {
    if constexpr (sizeof(In) == 4) {
      memcpy(x, &raw, sizeof(raw));
    } else if constexpr (P == 1) {
      x[0] = __uint_as_float(static_cast<uint32_t>(raw) << 16);
    } else {
      uint32_t w[P / 2];
      memcpy(w, &raw, sizeof(raw));
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  }
  static __device__ __forceinline__ void store(In* p, const float (&x)[P]) {  // In is bf16
    if constexpr (P == 1) {
      *p = __float2bfloat16_rn(x[0]);
    } else {
      uint32_t w[P / 2];
#pragma unroll
      for (int i = 0; i < P / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        memcpy(&w[i], &h, 4);
      }
      Type raw;
      memcpy(&raw, w, sizeof(raw));
      *reinterpret_cast<Type*>(p) = raw;
    }
  }
};

// cos and sin of pair i at position t.
__device__ __forceinline__ float2 rope_turn(const RopeArgs& a, int t, int i) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<uint32_t>(t)) * a.turn[i];
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * a.factor, s * a.factor);
}

// A group of `lanes` (D / 8, rounded up to a power of two) takes a slice of a
// token's head rows.  A lane holds four pairs of a row, a[i] and b[i], so that
// the pairs' cosines serve all its rows.  They are read and written as chunks
// of P elements: for the half layout the a's at c and the b's at
// c + rotary_dim / 2 (P = 4 where that is a multiple of 4, else 2 or 1), for
// the interleaved layout as they stand.  Elements behind rotary_dim go as pairs
// that are not turned.  kLanes: the group's lanes where they hold exactly a
// head (D = 8, 16, 32 lanes' 8), else 0.
template <typename In, int P, bool kInterleaved, int kLanes>
struct RopeLane {
  static constexpr int kChunks = 8 / P;
  int at[kChunks];     // element of each chunk
  bool live[kChunks];  // inside the head
  bool turned[4];
  uint64_t cos2[2], sin2[2], minus_sin2[2];

  // Which of the lane's eight values chunk c holds at i: a[j] or b[j].
  static __device__ __forceinline__ constexpr int pair(int c, int i) {
    return kInterleaved ? (c * P + i) / 2 : c / 2 * P + i;
  }
  static __device__ __forceinline__ constexpr bool is_b(int c, int i) { return kInterleaved ? i % 2 : c % 2; }

  __device__ __forceinline__ void place(const RopeArgs& a, int lane) {
    const int half = a.rotary_dim / 2;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (kInterleaved) {
        at[c] = lane * 8 + c * P;
        live[c] = kLanes != 0 || at[c] < a.D;
      } else {
        const int first = (lane + c / 2 * a.lanes) * P;  // of the pair of chunks
        live[c] = kLanes != 0 || 2 * first < a.D;
        at[c] = first >= half ? 2 * first + c % 2 * P : first + c % 2 * half;
      }
    }
  }
  __device__ __forceinline__ void turn(const RopeArgs& a, int lane, int pos) {
    const int half = a.rotary_dim / 2;
    float2 cs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int j = kInterleaved ? lane * 4 + i : (lane + i / P * a.lanes) * P + i % P;
      turned[i] = j < half;
      cs[i] = turned[i] ? rope_turn(a, pos, j) : make_float2(1.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      cos2[i] = pack2(cs[2 * i].x, cs[2 * i + 1].x);
      sin2[i] = pack2(cs[2 * i].y, cs[2 * i + 1].y);
      minus_sin2[i] = pack2(-cs[2 * i].y, -cs[2 * i + 1].y);
    }
  }
  template <typename T>
  __device__ __forceinline__ void load(const T* row, typename Chunk<T, P>::Type (&raw)[kChunks]) const {
#pragma unroll
    for (int c = 0; c < kChunks; ++c)
      if (kLanes != 0 || live[c]) raw[c] = Chunk<T, P>::load(row + at[c]);
  }
  template <typename T>
  __device__ __forceinline__ void widen(const typename Chunk<T, P>::Type (&raw)[kChunks], float (&a)[4], float (&b)[4]) const {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float x[P];
      Chunk<T, P>::widen(raw[c], x);
#pragma unroll
      for (int i = 0; i < P; ++i) (is_b(c, i) ? b : a)[pair(c, i)] = kLanes != 0 || live[c] ? x[i] : 0.f;
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* row, const float (&a)[4], const float (&b)[4]) const {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      float x[P];
#pragma unroll
      for (int i = 0; i < P; ++i) x[i] = (is_b(c, i) ? b : a)[pair(c, i)];
      if (kLanes != 0 || live[c]) Chunk<__nv_bfloat16, P>::store(row + at[c], x);
    }
  }
};

__device__ __forceinline__ void pack4(const float (&x)[4], uint64_t (&p)[2]) {
  p[0] = pack2(x[0], x[1]), p[1] = pack2(x[2], x[3]);
}
__device__ __forceinline__ void unpack4(const uint64_t (&p)[2], float (&x)[4]) {
  unpack2(p[0], x[0], x[1]), unpack2(p[1], x[2], x[3]);
}

// Rows [r0, r1) of queries or of keys: norm, turn, store.  `src`, `out`,
// `cache`: of row 0 (out, cache may be NULL).
template <typename In, int P, bool kInterleaved, int kLanes>
__device__ __forceinline__ void rope_rows(const RopeArgs& args, const RopeLane<In, P, kInterleaved, kLanes>& l, unsigned mask, int r0,
                                          int r1, const In* src, long long src_step, const void* weight, __nv_bfloat16* out,
                                          __nv_bfloat16* cache, long long cache_step) {
  using L = RopeLane<In, P, kInterleaved, kLanes>;
  float a[4], b[4];
  uint64_t ga[2], gb[2];
  if (weight != nullptr) {
    const uint64_t offset = pack2(args.offset, args.offset);
    if (args.weight_f32) {
      if constexpr (P * sizeof(float) <= 16) {
        typename Chunk<float, P>::Type raw[L::kChunks];
        l.load(static_cast<const float*>(weight), raw);
        l.template widen<float>(raw, a, b);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 w = l.live[0] ? reinterpret_cast<const float2*>(static_cast<const float*>(weight) + l.at[0])[i]
                                     : make_float2(0.f, 0.f);
          a[i] = w.x, b[i] = w.y;
        }
      }
    } else {
      typename Chunk<__nv_bfloat16, P>::Type raw[L::kChunks];
      l.load(static_cast<const __nv_bfloat16*>(weight), raw);
      l.template widen<__nv_bfloat16>(raw, a, b);
    }
    pack4(a, ga), pack4(b, gb);
#pragma unroll
    for (int i = 0; i < 2; ++i) ga[i] = add2(ga[i], offset), gb[i] = add2(gb[i], offset);
  }
  const bool partly = args.rotary_dim < args.D;
  src += r0 * src_step;
  if (out != nullptr) out += static_cast<long long>(r0) * args.D;
  if (cache != nullptr) cache += r0 * cache_step;
  auto row = [&](const typename Chunk<In, P>::Type (&raw)[L::kChunks]) {
    uint64_t a2[2], b2[2];
    l.template widen<In>(raw, a, b);
    pack4(a, a2), pack4(b, b2);
    if (weight != nullptr) {
      uint64_t s2 = mul2(a2[0], a2[0]);
      s2 = fma2(a2[1], a2[1], s2);
      s2 = fma2(b2[0], b2[0], s2);
      s2 = fma2(b2[1], b2[1], s2);
      float s, t;
      unpack2(s2, s, t);
      s += t;
      if constexpr (kLanes != 0) {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(mask, s, o);
      } else {
        for (int o = args.lanes / 2; o > 0; o >>= 1) s += __shfl_xor_sync(mask, s, o);
      }
      const float scale = rsqrtf(fmaf(s, args.inv_dim, args.eps));
      const uint64_t scale2 = pack2(scale, scale);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a2[i] = mul2(mul2(a2[i], scale2), ga[i]);
        b2[i] = mul2(mul2(b2[i], scale2), gb[i]);
      }
    }
    uint64_t c2[2], d2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c2[i] = fma2(a2[i], l.cos2[i], mul2(b2[i], l.minus_sin2[i]));
      d2[i] = fma2(b2[i], l.cos2[i], mul2(a2[i], l.sin2[i]));
    }
    float c[4], d[4];
    unpack4(c2, c), unpack4(d2, d);
    if (partly) {  // not by cos 1 and sin 0: an infinity beside would leave NaN
      unpack4(a2, a), unpack4(b2, b);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!l.turned[i]) c[i] = a[i], d[i] = b[i];
    }
    if (out != nullptr) {
      l.store(out, c, d);
      out += args.D;
    }
    if (cache != nullptr) {
      l.store(cache, c, d);
      cache += cache_step;
    }
  };
  int r = r0;
  for (; r + kRopeRows <= r1; r += kRopeRows) {
    typename Chunk<In, P>::Type raw[kRopeRows][L::kChunks];
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u, src += src_step) l.load(src, raw[u]);
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) row(raw[u]);
  }
  for (; r < r1; ++r, src += src_step) {
    typename Chunk<In, P>::Type raw[L::kChunks];
    l.load(src, raw);
    row(raw);
  }
}

// Blocks that an SM holds at once of the kernel for chunks of `chunk` elements.
__host__ __device__ constexpr int rope_blocks(int in_bytes, int chunk) { return chunk >= 4 || in_bytes == 4 ? 4 : 3; }

template <typename In, int P, bool kInterleaved, int kLanes>
__global__ void __launch_bounds__(kRopeThreads, rope_blocks(sizeof(In), P)) rope_kernel(RopeArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lanes = kLanes != 0 ? kLanes : a.lanes, lane = threadIdx.x & (lanes - 1), sub = (threadIdx.x & 31) & ~(lanes - 1);
  const unsigned mask = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1) << sub;
  const long long group = (static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x) / lanes;
  const int t = static_cast<int>(group / a.slices), slice = static_cast<int>(group - static_cast<long long>(t) * a.slices);
  if (t >= a.tokens) return;
  const int pos = a.positions[t];
  if (pos < 0) return;
  const int nq = a.q != nullptr ? a.Hq : 0, nk = a.k != nullptr ? a.Hkv : 0, nv = a.v != nullptr ? a.Hkv : 0;
  const int rows = nq + nk + nv, r0 = slice * a.per_slice, r1 = min(r0 + a.per_slice, rows);
  RopeLane<In, P, kInterleaved, kLanes> l;
  l.place(a, lane);
  if (r0 < nq + nk) l.turn(a, lane, pos);
  if (r0 < nq)
    rope_rows(a, l, mask, r0, min(r1, nq), static_cast<const In*>(a.q) + t * a.q_token, a.q_head, a.qw,
              a.q_out + static_cast<long long>(t) * a.Hq * a.D, nullptr, 0);
  if (r1 <= nq) return;
  const long long slot = a.slots != nullptr ? a.slots[t] : -1;
  const bool cached = slot >= 0 && slot < a.num_slots;
  if (!cached && slot != -1 && lane == 0) set_status(a.status, kDevPageOob);
  const long long page = cached ? slot / a.page_size : 0, in_page = cached ? slot - page * a.page_size : 0;
  const long long cell = (page * a.Hkv * a.page_size + in_page) * a.D, step = static_cast<long long>(a.page_size) * a.D;
  const int k0 = max(r0 - nq, 0), k1 = min(r1 - nq, nk);
  if (k0 < k1)
    rope_rows(a, l, mask, k0, k1, static_cast<const In*>(a.k) + t * a.k_token, a.k_head, a.kw,
              a.k_out != nullptr ? a.k_out + static_cast<long long>(t) * a.Hkv * a.D : nullptr,
              cached ? a.k_pool + cell : nullptr, step);
  if (!cached) return;
  for (int h = max(r0 - nq - nk, 0); h < r1 - nq - nk; ++h) {
    typename Chunk<In, P>::Type raw[8 / P];
    float x[4], y[4];
    l.load(static_cast<const In*>(a.v) + t * a.v_token + h * a.v_head, raw);
    l.template widen<In>(raw, x, y);
    l.store(a.v_pool + cell + h * step, x, y);
  }
}

}  // namespace wmtp
