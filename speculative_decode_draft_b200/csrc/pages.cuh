// Page tables and slot maps from sequence lengths.
//
// A sequence of n tokens holds ceil(n / P) pages.  The free list is a stack:
// with c free pages, R returned and A taken by one call, the returned page of
// rank r (counted in order of sequence and page) goes to entry c + R - 1 - r,
// and the taken page of rank a comes from entry c + R - 1 - a.  Both are known
// from two prefix sums over the sequences, so every page moves on its own.
#pragma once

#include <stdint.h>

#include "status.cuh"

namespace wmtp {

constexpr int kPagesThreads = 1024;
constexpr int kSlotThreads = 256;

struct PagesArgs {
  int32_t* page_table;  // [B][max_pages]
  int32_t* kv_len;      // [B]
  const int32_t* new_len;
  int32_t* free_pages;  // [num_pages]
  int32_t* free_count;  // [1]
  int32_t* cu;          // [B + 1] or NULL
  int32_t* positions;
  int64_t* slots;
  int32_t* status;
  int B, max_pages, P, num_pages, max_tokens;
};

// Inclusive prefix sum over the block's threads; *total: the sum of them all.
__device__ __forceinline__ long long block_scan(long long v, long long* s_warp, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // s_warp free again
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return v + (warp > 0 ? s_warp[warp - 1] : 0);
}

struct SeqChange {
  int old_len, new_len, hold, want;
  bool valid;
};

__device__ __forceinline__ SeqChange seq_change(const PagesArgs& a, int b) {
  SeqChange c;
  c.old_len = b < a.B ? a.kv_len[b] : 0;
  c.new_len = b < a.B ? a.new_len[b] : 0;
  const int cap = a.max_pages * a.P;
  c.valid = b < a.B && c.old_len >= 0 && c.old_len <= cap && c.new_len >= 0 && c.new_len <= cap;
  c.hold = c.valid ? (c.old_len + a.P - 1) / a.P : 0;
  c.want = c.valid ? (c.new_len + a.P - 1) / a.P : 0;
  return c;
}

// One CTA: lengths, page moves, cu.
__global__ void __launch_bounds__(kPagesThreads) pages_kernel(PagesArgs a) {
  __shared__ long long s_warp[32];
  long long total;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int count = *a.free_count;
  // 1. pages returned, in order of sequence and page
  long long released = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPagesThreads) {
    const SeqChange c = seq_change(a, b0 + tid);
    if (b0 + tid < a.B && !c.valid) set_status(a.status, kDevLenOob);
    released += max(c.hold - c.want, 0);
  }
  block_scan(released, s_warp, &total);
  released = total;
  if (count < 0 || count + released > a.num_pages) {
    if (tid == 0) set_status(a.status, kDevPool);
    if (a.cu != nullptr)
      for (int b = tid; b <= a.B; b += kPagesThreads) a.cu[b] = 0;
    return;
  }
  const long long top = count + released;
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPagesThreads) {
    const SeqChange c = seq_change(a, b0 + tid);
    const int n = max(c.hold - c.want, 0);
    const long long first = before + block_scan(n, s_warp, &total) - n;
    before += total;
    int32_t* row = a.page_table + static_cast<size_t>(b0 + tid) * a.max_pages;
    for (int j = 0; j < n; ++j) {
      const int32_t page = row[c.want + j];
      if (page < 0 || page >= a.num_pages) set_status(a.status, kDevPageOob);
      a.free_pages[top - 1 - (first + j)] = page;
      row[c.want + j] = -1;
    }
  }
  __syncthreads();
  // 2. pages taken, while they and the rows of the slot map last.  The sums
  // count the refused sequences too, so whatever grows behind the first one
  // that does not fit is refused with it
  long long taken = 0, grown = 0, used_pages = 0, used_rows = 0;
  if (tid == 0 && a.cu != nullptr) a.cu[0] = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPagesThreads) {
    const int b = b0 + tid;
    const SeqChange c = seq_change(a, b);
    const int grow = c.valid ? max(c.new_len - c.old_len, 0) : 0;
    const int need = max(c.want - c.hold, 0);
    const long long need_end = taken + block_scan(need, s_warp, &total);
    taken += total;
    const long long grow_end = grown + block_scan(grow, s_warp, &total);
    grown += total;
    const bool served = c.valid && (grow == 0 || (need_end <= top && (a.cu == nullptr || grow_end <= a.max_tokens)));
    if (c.valid && !served) set_status(a.status, kDevPool);
    if (served) {
      int32_t* row = a.page_table + static_cast<size_t>(b) * a.max_pages;
      for (int j = 0; j < need; ++j) row[c.hold + j] = a.free_pages[top - 1 - (need_end - need + j)];
      a.kv_len[b] = c.new_len;
    }
    block_scan(served ? need : 0, s_warp, &total);
    used_pages += total;
    const long long rows_end = used_rows + block_scan(served ? grow : 0, s_warp, &total);
    used_rows += total;
    if (a.cu != nullptr && b < a.B) a.cu[b + 1] = static_cast<int32_t>(rows_end);
  }
  if (tid == 0) *a.free_count = static_cast<int32_t>(top - used_pages);
}

// The slot map, a thread per row: the sequence of row t is the last one with
// cu[b] <= t; its length now is its old one plus its rows.
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(PagesArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long t = static_cast<long long>(blockIdx.x) * kSlotThreads + threadIdx.x;
  if (t >= a.max_tokens) return;
  int pos = -1;
  int64_t slot = -1;
  if (t < a.cu[a.B]) {
    int lo = 0, hi = a.B - 1;  // the first b with cu[b + 1] > t
    while (lo < hi) {
      const int mid = lo + (hi - lo) / 2;
      if (a.cu[mid + 1] > t)
        hi = mid;
      else
        lo = mid + 1;
    }
    pos = a.kv_len[lo] - (a.cu[lo + 1] - static_cast<int>(t));
    const int page = a.page_table[static_cast<size_t>(lo) * a.max_pages + pos / a.P];
    if (page >= 0 && page < a.num_pages)
      slot = static_cast<int64_t>(page) * a.P + pos % a.P;
    else
      set_status(a.status, kDevPageOob);
  }
  a.positions[t] = pos;
  a.slots[t] = slot;
}

}  // namespace wmtp
