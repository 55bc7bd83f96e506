// Page tables and slot maps from sequence lengths.
//
// A sequence of n tokens holds ceil(n / P) pages.  The free list is a stack:
// with c free pages, R returned and A taken by one call, the returned page of
// rank r (counted in order of sequence and page) goes to entry c + R - 1 - r,
// and the taken page of rank a comes from entry c + R - 1 - a.  So the page
// returned with rank r is the one taken with rank r, and pages of rank R on come from
// the old entries: with the two prefix sums known every page moves on its own, to
// the stack and to its new sequence at once, and nothing is read that the call writes.
//
// What is moved is small (8 bytes a page, 12 a token); the time is latency.  Up
// to kFewSeqs sequences with kFewTokens rows of map take one block and one launch,
// with a warp's lanes as the sequences.  More take two launches over all SMs: every
// block works the prefix sums out for itself and moves its share of the pages, and the
// slot map follows, which also writes what the first kernel's blocks still read,
// lengths and count.  Device time in us of a call by itself in one block and over all
// SMs: 4 or 32 sequences of 4 tokens 8.4 and 10.6, 32 of 128 with 4096 rows of map 12.1
// and 11.8; 2048 pages moved 10.4 and 9.7, 65536 70 and 9.  How many pages move is known on
// the device only and few do in a step, so the rule does not go by it; what that
// costs is an end of many long requests in one call, at the worst (32 of 2^20
// tokens on pages of 16) 2.6 ms against 30 us.
// Among others a call takes 2.6 us for 4 sequences and 4 tokens each, 12.6 us for 512 sequences, 17,000
// pages and a map of 1,048,579 rows (12.6 MB, 2 us of a copy's rate).
#pragma once

#include <stdint.h>

#include "status.cuh"

namespace wmtp {

constexpr int kFewSeqs = 32;
constexpr int kFewTokens = 4096;
constexpr int kFewThreads = 512;
constexpr int kMoveThreads = 512;
constexpr int kManyBlocks = 8;  // where the sums do not fit shared memory; else one per SM
constexpr int kSlotThreads = 256;
constexpr int kSlotRows = 4;
constexpr int kStaged = 2048;  // sequences whose sums are searched in shared memory

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
  bool wide;  // positions and slots may be written 16 bytes at a time
  int32_t* after;  // the new free count, then the new lengths: for the second kernel
  int32_t* sums;   // [kManyBlocks][2][B + 1], above kStaged sequences
};

struct SeqChange {
  int old_len, new_len, give, need, grow;
  bool valid;
};

__device__ __forceinline__ SeqChange seq_change(const PagesArgs& a, int b) {
  SeqChange c = {0, 0, 0, 0, 0, false};
  if (b >= a.B) return c;
  c.old_len = a.kv_len[b];
  c.new_len = a.new_len[b];
  const int cap = a.max_pages * a.P;
  c.valid = c.old_len >= 0 && c.old_len <= cap && c.new_len >= 0 && c.new_len <= cap;
  if (!c.valid) {
    if (blockIdx.x == 0) set_status(a.status, kDevLenOob);
    return c;
  }
  const int hold = (c.old_len + a.P - 1) / a.P, want = (c.new_len + a.P - 1) / a.P;
  c.give = max(hold - want, 0);
  c.need = max(want - hold, 0);
  c.grow = max(c.new_len - c.old_len, 0);
  return c;
}

// The first b of [0, n) with end[b] > i.
__device__ __forceinline__ int first_above(const int32_t* end, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (end[mid] > i)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Moves the page of rank i: returned, taken, or both.  given, taken: pages
// before each sequence, [B + 1].
__device__ __forceinline__ void move_page(const PagesArgs& a, const int32_t* given, const int32_t* taken, int top, int i) {
  int32_t page;
  if (i < given[a.B]) {
    const int b = first_above(given + 1, a.B, i);
    const int want = (a.new_len[b] + a.P - 1) / a.P;
    int32_t* entry = a.page_table + static_cast<size_t>(b) * a.max_pages + want + (i - given[b]);
    page = *entry;
    *entry = -1;
    if (page < 0 || page >= a.num_pages) set_status(a.status, kDevPageOob);
    a.free_pages[top - 1 - i] = page;
  } else {
    page = a.free_pages[top - 1 - i];
  }
  if (i < taken[a.B]) {
    const int b = first_above(taken + 1, a.B, i);
    const int hold = (a.kv_len[b] + a.P - 1) / a.P;  // the old length
    a.page_table[static_cast<size_t>(b) * a.max_pages + hold + (i - taken[b])] = page;
  }
}

// Row t of the slot map, of sequence b (the first whose tokens end behind it).
__device__ __forceinline__ void map_slot(const PagesArgs& a, const int32_t* cu, int b, int t, int32_t* pos, int64_t* slot) {
  *pos = a.new_len[b] - (cu[b + 1] - t);
  const int page = a.page_table[static_cast<size_t>(b) * a.max_pages + *pos / a.P];
  *slot = static_cast<int64_t>(page) * a.P + *pos % a.P;
  if (page < 0 || page >= a.num_pages) {
    *slot = -1;
    set_status(a.status, kDevPageOob);
  }
}

// Inclusive prefix sum over a warp's lanes.
__device__ __forceinline__ long long warp_scan(long long v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// One block: all of it, for up to 32 sequences.
__global__ void __launch_bounds__(kFewThreads) pages_few_kernel(PagesArgs a) {
  __shared__ int32_t s_given[kFewSeqs + 1], s_taken[kFewSeqs + 1], s_cu[kFewSeqs + 1], s_top;
  __shared__ bool s_served[kFewSeqs];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  if (tid < 32) {
    const int count = *a.free_count;
    SeqChange c = seq_change(a, tid);
    const long long given = warp_scan(c.give);
    const long long top = count + __shfl_sync(0xffffffffu, given, 31);
    const bool sound = count >= 0 && top <= a.num_pages;
    if (!sound) {
      if (tid == 0) set_status(a.status, kDevPool);
      c = {0, 0, 0, 0, 0, false};
    }
    // served in order while pages and rows last: the sums count the refused
    // sequences too, so whatever grows behind the first one that does not fit is
    // refused with it
    const long long need_end = warp_scan(c.need), grow_end = warp_scan(c.grow);
    const bool served =
        c.valid && (c.grow == 0 || (need_end <= top && (a.cu == nullptr || grow_end <= a.max_tokens)));
    if (c.valid && !served) set_status(a.status, kDevPool);
    const long long taken = warp_scan(served ? c.need : 0), rows = warp_scan(served ? c.grow : 0);
    s_served[tid] = served;
    s_given[tid + 1] = sound ? static_cast<int32_t>(given) : 0;
    s_taken[tid + 1] = static_cast<int32_t>(taken);
    s_cu[tid + 1] = a.cu != nullptr ? static_cast<int32_t>(rows) : 0;
    if (a.cu != nullptr && tid < a.B) a.cu[tid + 1] = static_cast<int32_t>(rows);
    if (tid == 31) {
      if (sound) *a.free_count = static_cast<int32_t>(top - taken);
      s_top = static_cast<int32_t>(top);
    }
    if (tid == 0) {
      s_given[0] = s_taken[0] = s_cu[0] = 0;
      if (a.cu != nullptr) a.cu[0] = 0;
    }
  }
  __syncthreads();
  const int moves = max(s_given[a.B], s_taken[a.B]);
  for (int i = tid; i < moves; i += kFewThreads) move_page(a, s_given, s_taken, s_top, i);
  __syncthreads();
  for (int t = tid; t < a.max_tokens; t += kFewThreads) {
    int32_t pos = -1;
    int64_t slot = -1;
    if (t < s_cu[a.B]) map_slot(a, s_cu, first_above(s_cu + 1, a.B, t), t, &pos, &slot);
    a.positions[t] = pos;
    a.slots[t] = slot;
  }
  if (tid < a.B && s_served[tid]) a.kv_len[tid] = a.new_len[tid];  // read as the old one by the moves
}

// Inclusive prefix sums of N values over the block's threads (N warps at least),
// on top of *carry; *carry: with the block's totals added.
template <int N>
__device__ __forceinline__ void block_scan(long long (&v)[N], long long (&carry)[N], long long (*s_warp)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = warp_scan(v[n]);
  __syncthreads();  // s_warp free again
  if (lane == 31)
    for (int n = 0; n < N; ++n) s_warp[n][warp] = v[n];
  __syncthreads();
  // lanes without a warp of their own carry the total on
  if (warp < N) s_warp[warp][lane] = warp_scan(lane < static_cast<int>(blockDim.x >> 5) ? s_warp[warp][lane] : 0);
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] += carry[n] + (warp > 0 ? s_warp[n][warp - 1] : 0);
    carry[n] += s_warp[n][31];
  }
}

// Many sequences, 1: prefix sums, by every block for itself, and the pages.
__global__ void __launch_bounds__(kMoveThreads) pages_kernel(PagesArgs a) {
  __shared__ long long s_warp[3][32];
  __shared__ int32_t s_given[kStaged + 1], s_taken[kStaged + 1];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const bool writes = blockIdx.x == 0;
  int32_t* given = a.B <= kStaged ? s_given : a.sums + static_cast<size_t>(blockIdx.x) * 2 * (a.B + 1);
  int32_t* taken = a.B <= kStaged ? s_taken : given + a.B + 1;
  const int count = *a.free_count;
  long long ends[3] = {0, 0, 0}, v[3];  // given, needed, grown
  SeqChange c;
  for (int b0 = 0; b0 < a.B; b0 += kMoveThreads) {
    c = seq_change(a, b0 + tid);
    v[0] = c.give, v[1] = c.need, v[2] = c.grow;
    block_scan(v, ends, s_warp);
    if (b0 + tid < a.B) given[b0 + tid + 1] = static_cast<int32_t>(min(v[0], 0x7fffffffLL));
  }
  const long long top = count + ends[0];
  const bool sound = count >= 0 && top <= a.num_pages;
  // served in order while pages and rows last: the sums count the refused
  // sequences too, so whatever grows behind the first one that does not fit is
  // refused with it
  long long again[3] = {0, 0, 0}, used[2] = {0, 0};  // pages, rows
  for (int b0 = 0; b0 < a.B; b0 += kMoveThreads) {
    const int b = b0 + tid;
    if (a.B > kMoveThreads) {  // else the only round's sums are still there
      c = seq_change(a, b);
      v[0] = c.give, v[1] = c.need, v[2] = c.grow;
      block_scan(v, again, s_warp);
    }
    const bool served =
        sound && c.valid && (c.grow == 0 || (v[1] <= top && (a.cu == nullptr || v[2] <= a.max_tokens)));
    long long w[2] = {served ? c.need : 0, served ? c.grow : 0};
    block_scan(w, used, s_warp);
    if (b < a.B) {
      taken[b + 1] = static_cast<int32_t>(w[0]);
      if (writes) {
        if (sound && c.valid && !served) set_status(a.status, kDevPool);
        a.after[1 + b] = served ? c.new_len : c.old_len;
        if (a.cu != nullptr) a.cu[b + 1] = static_cast<int32_t>(w[1]);
      }
    }
  }
  if (tid == 0) {
    given[0] = taken[0] = 0;
    if (writes) {
      a.after[0] = sound ? static_cast<int32_t>(top - used[0]) : count;
      if (a.cu != nullptr) a.cu[0] = 0;
      if (!sound) set_status(a.status, kDevPool);
    }
  }
  if (!sound) return;
  __syncthreads();
  const long long moves = max(ends[0], used[0]);
  for (long long i = static_cast<long long>(blockIdx.x) * kMoveThreads + tid; i < moves; i += kMoveThreads * gridDim.x)
    move_page(a, given, taken, static_cast<int>(top), static_cast<int>(i));
}

// 2: lengths and count, and the slot map, kSlotRows rows to a thread.
__global__ void __launch_bounds__(kSlotThreads) slots_kernel(PagesArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long first = (static_cast<long long>(blockIdx.x) * kSlotThreads + threadIdx.x) * kSlotRows;
  __shared__ int32_t s_cu[kStaged + 1];
  for (int b = blockIdx.x * kSlotThreads + threadIdx.x; b < a.B; b += kSlotThreads * gridDim.x) a.kv_len[b] = a.after[1 + b];
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.free_count = a.after[0];
  if (a.max_tokens == 0) return;
  const int rows = a.cu[a.B];
  const bool staged = a.B <= kStaged && first - threadIdx.x * kSlotRows < rows;
  if (staged) {
    for (int b = threadIdx.x; b <= a.B; b += kSlotThreads) s_cu[b] = a.cu[b];
    __syncthreads();
  }
  if (first >= a.max_tokens) return;
  const int32_t* cu = staged ? s_cu : a.cu;
  const int t0 = static_cast<int>(first), n = min(kSlotRows, a.max_tokens - t0);
  int32_t pos[kSlotRows];
  int64_t slot[kSlotRows];
  int b = t0 < rows ? first_above(cu + 1, a.B, t0) : 0;
#pragma unroll
  for (int i = 0; i < kSlotRows; ++i) {
    pos[i] = -1, slot[i] = -1;
    if (i >= n || t0 + i >= rows) continue;
    while (cu[b + 1] <= t0 + i) ++b;
    map_slot(a, cu, b, t0 + i, &pos[i], &slot[i]);
  }
  if (n == kSlotRows && a.wide) {
    *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    longlong2* to = reinterpret_cast<longlong2*>(a.slots + t0);
    to[0] = make_longlong2(slot[0], slot[1]);
    to[1] = make_longlong2(slot[2], slot[3]);
  } else {
    for (int i = 0; i < n; ++i) a.positions[t0 + i] = pos[i], a.slots[t0 + i] = slot[i];
  }
}

}  // namespace wmtp
