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
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "status.cuh"

namespace wmtp {

constexpr int kRopeWarps = 8;
constexpr int kRopeThreads = 32 * kRopeWarps;
constexpr int kRopeMaxDim = 256;

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
  int32_t* status;
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// cos and sin of pair i at position t.
__device__ __forceinline__ float2 rope_turn(const RopeArgs& a, int t, int i) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<uint32_t>(t)) * a.turn[i];
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * a.factor, s * a.factor);
}

// One warp per head row (of q, k or v) of a token; a lane holds 8 elements.
template <typename In>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  __shared__ float s_row[kRopeWarps][kRopeMaxDim];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nq = a.q != nullptr ? a.Hq : 0, nk = a.k != nullptr ? a.Hkv : 0, nv = a.v != nullptr ? a.Hkv : 0;
  const long long row = static_cast<long long>(blockIdx.x) * kRopeWarps + warp;
  const int per = nq + nk + nv;
  if (row >= static_cast<long long>(a.tokens) * per) return;
  const int t = static_cast<int>(row / per);
  int h = static_cast<int>(row % per);
  const int pos = a.positions[t];
  if (pos < 0) return;
  const int e = lane * 8;
  const bool live = e < a.D;
  const int kind = h < nq ? 0 : h < nq + nk ? 1 : 2;
  h -= kind == 0 ? 0 : kind == 1 ? nq : nq + nk;
  const In* src = static_cast<const In*>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                  t * (kind == 0 ? a.q_token : kind == 1 ? a.k_token : a.v_token) +
                  h * (kind == 0 ? a.q_head : kind == 1 ? a.k_head : a.v_head);
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live) load8(src + e, x);
  const void* w = kind == 0 ? a.qw : kind == 1 ? a.kw : nullptr;
  if (w != nullptr) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = rsqrtf(ss / a.D + a.eps);
    if (live) {
      float g[8];
      if (a.weight_f32)
        load8(static_cast<const float*>(w) + e, g);
      else
        load8(static_cast<const __nv_bfloat16*>(w) + e, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * r * (g[i] + a.offset);
    }
  }
  if (kind != 2 && a.rotary_dim > 0) {
    if (live)
#pragma unroll
      for (int i = 0; i < 8; ++i) s_row[warp][e + i] = x[i];
    __syncwarp();
    const int half = a.rotary_dim / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = e + i;
      if (c >= a.rotary_dim) continue;
      const bool second = a.interleaved ? (c & 1) != 0 : c >= half;
      const int pair = a.interleaved ? c >> 1 : second ? c - half : c;
      const int other = a.interleaved ? c ^ 1 : second ? c - half : c + half;
      const float2 cs = rope_turn(a, pos, pair);
      const float o = s_row[warp][other];
      x[i] = second ? x[i] * cs.x + o * cs.y : x[i] * cs.x - o * cs.y;
    }
  }
  if (!live) return;
  if (kind == 0) {
    store8(a.q_out + (static_cast<long long>(t) * a.Hq + h) * a.D + e, x);
    return;
  }
  if (kind == 1 && a.k_out != nullptr) store8(a.k_out + (static_cast<long long>(t) * a.Hkv + h) * a.D + e, x);
  if (a.slots != nullptr) {
    const long long slot = a.slots[t];
    if (slot >= 0 && slot < a.num_slots) {
      const long long page = slot / a.page_size, r = slot % a.page_size;
      store8((kind == 1 ? a.k_pool : a.v_pool) + ((page * a.Hkv + h) * a.page_size + r) * a.D + e, x);
    } else if (slot != -1) {
      set_status(a.status, kDevPageOob);
    }
  }
}

}  // namespace wmtp
