// libwmtp: the C ABI declared in include/wmtp_step.h.
//
// Host side only: argument validation, workspace sizing and kernel launches.
// The work runs in the kernels of rope.cuh, pages.cuh and logits.cuh.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "host.cuh"
#include "logits.cuh"
#include "pages.cuh"
#include "rope.cuh"
#include "wmtp_step.h"

namespace wmtp {
namespace {

constexpr int kMaxVocab = 1 << 30;
constexpr int kMaxAcceptQ = 32;
constexpr long long kMaxGridX = 0x7fffffffLL;

bool dtype_bytes(int32_t dtype, int* bytes) {
  *bytes = dtype == WMTP_FP32 ? 4 : 2;
  return dtype == WMTP_BF16 || dtype == WMTP_FP16 || dtype == WMTP_FP32;
}

bool words_ok(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!aligned(p, 4)) return false;
  return true;
}

// A [tokens][heads][D] view that 16-byte loads can read.
bool heads_ok(const void* p, int64_t token_stride, int64_t head_stride, int bytes) {
  return aligned(p, 16) && token_stride >= 0 && head_stride >= 0 && token_stride * bytes % 16 == 0 &&
         head_stride * bytes % 16 == 0;
}

// Bytes next to one another, or rows of them in a [tokens][heads] view.
struct Block {
  __int128 at, bytes;  // at 0: absent
  Block(const void* p, __int128 n) : at(reinterpret_cast<uintptr_t>(p)), bytes(n) {}
  bool meets(const Block& o) const { return at != 0 && o.at != 0 && at < o.at + o.bytes && o.at < at + bytes; }
};
struct HeadRows {
  Block row;  // the first one
  __int128 tokens, heads, token_step, head_step;
  bool meets(const Block& o) const {
    const Block span(reinterpret_cast<const void*>(static_cast<uintptr_t>(row.at)),
                     (tokens - 1) * token_step + (heads - 1) * head_step + row.bytes);
    if (!span.meets(o)) return false;
    for (__int128 h = 0; h < heads; ++h) {
      const __int128 first = row.at + h * head_step;
      // the first token whose row ends behind the block's start
      const __int128 before = o.at - first - row.bytes;
      const __int128 t = token_step == 0 || before < 0 ? 0 : before / token_step + 1;
      const __int128 start = first + t * token_step;
      if (t < tokens && start + row.bytes > o.at && start < o.at + o.bytes) return true;
    }
    return false;
  }
};

template <typename F>
F by_dtype(int32_t dtype, F fp32, F fp16, F bf16) {
  return dtype == WMTP_FP32 ? fp32 : dtype == WMTP_FP16 ? fp16 : bf16;
}

// Slices of a token's head rows, one for each group of lanes: as many as fit the
// warps that the SMs hold at once; one where the tokens alone fill them, since each
// slice works its angles out again.  Device time in us of 20 rows of 256 with 1, 3, 10
// slices: 16 tokens 8.5, 4.5, 3.1; 1537 10.2, 7.5, 12.0; 4096 17.6, 19.9, 29.1.
int rope_slices(long long tokens, int rows, int lanes, long long warps) {
  const long long n = warps * 32 / lanes / tokens;
  return n < 1 ? 1 : n < rows ? static_cast<int>(n) : rows;
}

// CTAs that share each of `rows` rows: more while they are no more than five for
// each SM (four are resident) and each keeps a whole batch.  Device time in us with
// 1, 2, 4 CTAs a row of 131072 bf16, top 8: 4 rows 14.6, 10.6, 8.7; 300 rows 32.4,
// 30.8, 34.2; 1024 rows 58.4, 69.7, 92.8.  More than 4 were not tried.
int row_cluster(long long rows, int vocab, int bytes, int sms) {
  int c = 1;
  const long long vecs = static_cast<long long>(vocab) * bytes / 16;
  while (c < kRowCluster && rows * c * 2 <= 5LL * sms && vecs / (2 * c) >= kBatch) c *= 2;
  return c;
}

// CTAs per sequence for the token that follows: few of them of each sequence meet on
// one SM.  Device time in us of the whole call with at most 8 and 16: 1 sequence of 3
// drafts 15.4 and 12.2; 32 of 5 48.4 and 36.4; 16 of 8 33.2 and 28.7.
int final_cluster(long long batch, int vocab, int sms, int most) {
  int c = 1;
  while (c < most && batch * c < 4LL * sms && vocab / (2 * c) >= 4 * kFinalThreads) c *= 2;
  return c;
}

// Clusters of a kernel without dynamic shared memory that fit the device at once; -1:
// the runtime does not say.
template <typename Kern>
int clusters_that_fit(Kern kern, int threads, int cluster) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = -1;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();
    return -1;
  }
  return n;
}

}  // namespace
}  // namespace wmtp

using namespace wmtp;

extern "C" {

wmtp_status wmtp_qk_norm_rope(const wmtp_params* params, const wmtp_rope* rope, int32_t tokens, int32_t in_dtype,
                              const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* k,
                              int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride,
                              int64_t v_head_stride, const int32_t* positions, const int64_t* slots,
                              const wmtp_paged_kv* kv, const void* q_weight, const void* k_weight,
                              int32_t weight_dtype, float weight_offset, float eps, void* q_out, void* k_out,
                              int32_t* status_word, void* stream) {
  if (params == nullptr || tokens < 0) return WMTP_ERR_INVALID_ARG;
  const int D = params->head_dim;
  if (params->num_heads_q <= 0 || params->num_heads_kv <= 0) return WMTP_ERR_INVALID_ARG;
  if (params->num_heads_q > kMaxGridYZ || params->num_heads_kv > kMaxGridYZ) return WMTP_ERR_UNSUPPORTED;
  if (D <= 0 || D % 8 != 0 || D > kRopeMaxDim) return WMTP_ERR_UNSUPPORTED;
  if (in_dtype != WMTP_BF16 && in_dtype != WMTP_FP32) return WMTP_ERR_UNSUPPORTED;
  if (weight_dtype != WMTP_BF16 && weight_dtype != WMTP_FP32) return WMTP_ERR_UNSUPPORTED;
  if (!std::isfinite(weight_offset) || !std::isfinite(eps) || eps < 0.f) return WMTP_ERR_INVALID_ARG;
  if (rope != nullptr) {
    if (rope->rotary_dim < 0 || rope->rotary_dim > D || rope->rotary_dim % 2 != 0) return WMTP_ERR_INVALID_ARG;
    if (rope->rotary_dim > 0 && rope->turn == nullptr) return WMTP_ERR_INVALID_ARG;
    if (!std::isfinite(rope->factor) || !aligned(rope->turn, 8)) return WMTP_ERR_INVALID_ARG;
  }
  // queries have a place to go, keys one at least, values the cache
  if ((q == nullptr) != (q_out == nullptr) || (q == nullptr && k == nullptr)) return WMTP_ERR_INVALID_ARG;
  if (k == nullptr ? (k_out != nullptr || slots != nullptr) : (k_out == nullptr && slots == nullptr))
    return WMTP_ERR_INVALID_ARG;
  if ((slots == nullptr) != (v == nullptr)) return WMTP_ERR_INVALID_ARG;
  if (slots != nullptr) {
    if (!supported_page(params->page_size)) return WMTP_ERR_UNSUPPORTED;
    if (kv == nullptr || kv->k_pool == nullptr || kv->v_pool == nullptr || kv->num_pages <= 0 ||
        !aligned(kv->k_pool, 16) || !aligned(kv->v_pool, 16) || !aligned(slots, 8))
      return WMTP_ERR_INVALID_ARG;
  }
  if (tokens == 0) return WMTP_OK;
  if (positions == nullptr || !aligned(positions, 4)) return WMTP_ERR_INVALID_ARG;
  const int bytes = in_dtype == WMTP_FP32 ? 4 : 2;
  if (!heads_ok(q, q_token_stride, q_head_stride, bytes) || !heads_ok(k, k_token_stride, k_head_stride, bytes) ||
      !heads_ok(v, v_token_stride, v_head_stride, bytes))
    return WMTP_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(q_out, 16) || !aligned(k_out, 16))
    return WMTP_ERR_INVALID_ARG;
  {
    // Tokens are encoded in any order: no output may lie over what another token
    // still reads or writes.  Rows that replace themselves may.
    const __int128 T = tokens, row = 2LL * D;
    const int Hq = params->num_heads_q, Hkv = params->num_heads_kv;
    const HeadRows rq = {{q, D * bytes}, T, Hq, q_token_stride * bytes, q_head_stride * bytes};
    const HeadRows rk = {{k, D * bytes}, T, Hkv, k_token_stride * bytes, k_head_stride * bytes};
    const HeadRows rv = {{v, D * bytes}, T, Hkv, v_token_stride * bytes, v_head_stride * bytes};
    const Block qo(q_out, T * Hq * row), ko(k_out, T * Hkv * row);
    const __int128 pool = slots != nullptr ? static_cast<__int128>(kv->num_pages) * params->page_size * Hkv * row : 0;
    const Block kp(slots != nullptr ? kv->k_pool : nullptr, pool), vp(slots != nullptr ? kv->v_pool : nullptr, pool);
    auto same = [&](const void* x, const void* out, int heads, int64_t token, int64_t head) {
      return x == out && bytes == 2 && (tokens == 1 || token == static_cast<int64_t>(heads) * D) && (heads == 1 || head == D);
    };
    if ((rq.meets(qo) && !same(q, q_out, Hq, q_token_stride, q_head_stride)) || rk.meets(qo) || rv.meets(qo) ||
        (rk.meets(ko) && !same(k, k_out, Hkv, k_token_stride, k_head_stride)) || rq.meets(ko) || rv.meets(ko) ||
        qo.meets(ko) || qo.meets(kp) || qo.meets(vp) || ko.meets(kp) || ko.meets(vp) || kp.meets(vp))
      return WMTP_ERR_INVALID_ARG;
  }
  RopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = q, a.k = k, a.v = v;
  a.q_token = q_token_stride, a.q_head = q_head_stride;
  a.k_token = k_token_stride, a.k_head = k_head_stride;
  a.v_token = v_token_stride, a.v_head = v_head_stride;
  a.positions = positions;
  a.slots = slots;
  if (slots != nullptr) {
    a.k_pool = static_cast<__nv_bfloat16*>(kv->k_pool);
    a.v_pool = static_cast<__nv_bfloat16*>(kv->v_pool);
    a.num_slots = static_cast<long long>(kv->num_pages) * params->page_size;
    a.page_size = params->page_size;
  }
  a.qw = q_weight, a.kw = k_weight;
  a.weight_f32 = weight_dtype == WMTP_FP32;
  a.offset = weight_offset, a.eps = eps;
  if (rope != nullptr) {
    a.turn = rope->turn;
    a.rotary_dim = rope->rotary_dim;
    a.interleaved = rope->interleaved != 0;
    a.factor = rope->factor;
  }
  a.q_out = static_cast<__nv_bfloat16*>(q_out);
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.tokens = tokens, a.Hq = params->num_heads_q, a.Hkv = params->num_heads_kv, a.D = D;
  a.status = status_word;
  const int rows = (q != nullptr ? a.Hq : 0) + (k != nullptr ? a.Hkv : 0) + (v != nullptr ? a.Hkv : 0);
  a.inv_dim = 1.f / D;
  a.lanes = 1;
  while (a.lanes * 8 < D) a.lanes *= 2;
  const int half = a.rotary_dim / 2;
  const int chunk = a.interleaved ? 16 / bytes : half % 4 == 0 ? 4 : half % 2 == 0 ? 2 : 1;
  int dev = 0;
  DeviceInfo info;
  const wmtp_status s = current_device(&dev, &info);
  if (s != WMTP_OK) return s;
  a.slices = rope_slices(tokens, rows, a.lanes, static_cast<long long>(info.sms) * rope_blocks(bytes, chunk) * kRopeWarps);
  a.per_slice = (rows + a.slices - 1) / a.slices;
  a.slices = (rows + a.per_slice - 1) / a.per_slice;
  const int groups = kRopeThreads / a.lanes;
  const long long grid = (static_cast<long long>(tokens) * a.slices + groups - 1) / groups;
  if (grid > kMaxGridX) return WMTP_ERR_UNSUPPORTED;
  const int full = a.lanes * 8 == D ? a.lanes : 0;
  auto pick = [&](auto in) {
    using In = decltype(in);
    constexpr int kRun = 16 / sizeof(In);
    if (a.interleaved)
      return full == 32   ? rope_kernel<In, kRun, true, 32>
             : full == 16 ? rope_kernel<In, kRun, true, 16>
             : full == 8  ? rope_kernel<In, kRun, true, 8>
                          : rope_kernel<In, kRun, true, 0>;
    if (chunk == 4)
      return full == 32   ? rope_kernel<In, 4, false, 32>
             : full == 16 ? rope_kernel<In, 4, false, 16>
             : full == 8  ? rope_kernel<In, 4, false, 8>
                          : rope_kernel<In, 4, false, 0>;
    return chunk == 2 ? rope_kernel<In, 2, false, 0> : rope_kernel<In, 1, false, 0>;
  };
  auto kern = in_dtype == WMTP_FP32 ? pick(float()) : pick(__nv_bfloat16());
  return launch_plain(true, kern, dim3(static_cast<unsigned>(grid)), dim3(kRopeThreads),
                      static_cast<cudaStream_t>(stream), a);
}

wmtp_status wmtp_pages_resize(const wmtp_params* params, int32_t batch, int32_t* page_table, int32_t max_pages,
                              int32_t* kv_len, const int32_t* new_len, int32_t* free_pages, int32_t* free_count,
                              int32_t num_pages, int32_t* cu_tokens, int32_t* positions, int64_t* slots,
                              int32_t max_tokens, void* workspace, size_t* workspace_bytes, int32_t* status_word,
                              void* stream) {
  if (params == nullptr || batch < 0 || max_tokens < 0 || workspace_bytes == nullptr) return WMTP_ERR_INVALID_ARG;
  if (!supported_page(params->page_size) || batch > kMaxGridYZ) return WMTP_ERR_UNSUPPORTED;
  if (max_pages <= 0 || num_pages <= 0) return WMTP_ERR_INVALID_ARG;
  if (static_cast<long long>(max_pages) * params->page_size > (1LL << 30)) return WMTP_ERR_UNSUPPORTED;
  const bool map = max_tokens > 0, few = batch <= kFewSeqs && max_tokens <= kFewTokens;
  const bool staged = batch <= kStaged;
  const size_t seqs = static_cast<size_t>(batch) + 1;
  const size_t need = few ? 0 : align_up((staged ? seqs : (1 + 2 * kManyBlocks) * seqs) * sizeof(int32_t), kWsAlign);
  if (workspace == nullptr && free_pages == nullptr) {
    *workspace_bytes = need;
    return WMTP_OK;
  }
  if (*workspace_bytes < need || !aligned(workspace, kWsAlign) || (workspace == nullptr && need > 0))
    return WMTP_ERR_WORKSPACE;
  if (map != (cu_tokens != nullptr) || map != (positions != nullptr) || map != (slots != nullptr))
    return WMTP_ERR_INVALID_ARG;
  if (free_pages == nullptr || free_count == nullptr || (batch > 0 && (page_table == nullptr || kv_len == nullptr ||
                                                                       new_len == nullptr)))
    return WMTP_ERR_INVALID_ARG;
  if (!words_ok({page_table, kv_len, new_len, free_pages, free_count, cu_tokens, positions}) || !aligned(slots, 8))
    return WMTP_ERR_INVALID_ARG;
  if (batch == 0 && !map) return WMTP_OK;
  PagesArgs a;
  a.page_table = page_table, a.kv_len = kv_len, a.new_len = new_len;
  a.free_pages = free_pages, a.free_count = free_count;
  a.cu = cu_tokens, a.positions = positions, a.slots = slots;
  a.status = status_word;
  a.B = batch, a.max_pages = max_pages, a.P = params->page_size, a.num_pages = num_pages, a.max_tokens = max_tokens;
  a.wide = aligned(positions, 16) && aligned(slots, 16);
  a.after = static_cast<int32_t*>(workspace), a.sums = a.after + seqs;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (few) return launch_plain(true, pages_few_kernel, dim3(1), dim3(kFewThreads), st, a);
  int dev = 0;
  DeviceInfo info;
  wmtp_status s = current_device(&dev, &info);
  if (s != WMTP_OK) return s;
  s = launch_plain(true, pages_kernel, dim3(static_cast<unsigned>(staged ? info.sms : kManyBlocks)), dim3(kMoveThreads), st, a);
  if (s != WMTP_OK) return s;
  const long long blocks = (max_tokens + 1LL * kSlotThreads * kSlotRows - 1) / (kSlotThreads * kSlotRows);
  return launch_plain(true, slots_kernel, dim3(static_cast<unsigned>(blocks > 0 ? blocks : 1)), dim3(kSlotThreads), st, a);
}

wmtp_status wmtp_token_logprobs(int32_t rows, int32_t vocab, int32_t dtype, const void* logits, int64_t row_stride,
                                const float* temperature, const int32_t* tokens, int32_t num_tokens, int32_t top_k,
                                float* logprobs_out, float* entropy_out, float* lse_out, float* top_logprobs_out,
                                int32_t* top_ids_out, int32_t* status_word, void* stream) {
  int bytes = 0;
  if (rows < 0 || vocab <= 0 || num_tokens < 0 || top_k < 0) return WMTP_ERR_INVALID_ARG;
  if (!dtype_bytes(dtype, &bytes) || vocab > kMaxVocab || top_k > kMaxTop) return WMTP_ERR_UNSUPPORTED;
  if (row_stride < vocab && rows > 1) return WMTP_ERR_INVALID_ARG;
  if (num_tokens > 0 && rows > 0 && (tokens == nullptr || logprobs_out == nullptr)) return WMTP_ERR_INVALID_ARG;
  if (top_k > 0 && rows > 0 && (top_logprobs_out == nullptr || top_ids_out == nullptr)) return WMTP_ERR_INVALID_ARG;
  if (rows == 0) return WMTP_OK;
  if (logits == nullptr || !aligned(logits, bytes)) return WMTP_ERR_INVALID_ARG;
  if (!words_ok({temperature, tokens, logprobs_out, entropy_out, lse_out, top_logprobs_out, top_ids_out}))
    return WMTP_ERR_INVALID_ARG;
  LogprobArgs a;
  a.logits = logits, a.row_stride = row_stride, a.temperature = temperature, a.tokens = tokens;
  a.logprobs = logprobs_out, a.entropy = entropy_out, a.lse = lse_out, a.top_logprobs = top_logprobs_out;
  a.top_ids = top_ids_out, a.status = status_word;
  a.V = vocab, a.num_tokens = num_tokens, a.top_k = top_k;
  int dev = 0;
  DeviceInfo info;
  const wmtp_status s = current_device(&dev, &info);
  if (s != WMTP_OK) return s;
  const int c = row_cluster(rows, vocab, bytes, info.sms);
  auto kern = by_dtype(dtype, logprob_kernel<float>, logprob_kernel<__half>, logprob_kernel<__nv_bfloat16>);
  return launch_clusters(true, kern, dim3(static_cast<unsigned>(rows) * c), dim3(kRowThreads), c,
                         static_cast<cudaStream_t>(stream), a);
}

wmtp_status wmtp_accept_draft(int32_t batch, int32_t num_q, int32_t vocab, int32_t dtype, const void* target,
                              int64_t target_batch_stride, int64_t target_row_stride, const void* draft,
                              int64_t draft_batch_stride, int64_t draft_row_stride, const int32_t* draft_tokens,
                              const float* uniforms, const int32_t* num_draft, const float* temperature,
                              int32_t* tokens_out, int32_t* count_out, float* logprobs_out, void* workspace,
                              size_t* workspace_bytes, int32_t* status_word, void* stream) {
  int bytes = 0;
  if (batch < 0 || num_q <= 0 || vocab <= 0 || workspace_bytes == nullptr) return WMTP_ERR_INVALID_ARG;
  if (!dtype_bytes(dtype, &bytes) || vocab > kMaxVocab || num_q > kMaxAcceptQ || batch > kMaxGridYZ)
    return WMTP_ERR_UNSUPPORTED;
  const size_t need = align_up(static_cast<size_t>(batch) * (2 * num_q - 1) * sizeof(RowStat), kWsAlign);
  if (workspace == nullptr) {
    *workspace_bytes = need;
    return WMTP_OK;
  }
  if (*workspace_bytes < need || !aligned(workspace, kWsAlign)) return WMTP_ERR_WORKSPACE;
  if (batch == 0) return WMTP_OK;
  if (target == nullptr || uniforms == nullptr || tokens_out == nullptr || count_out == nullptr)
    return WMTP_ERR_INVALID_ARG;
  if (num_q > 1 && draft_tokens == nullptr) return WMTP_ERR_INVALID_ARG;
  if (!aligned(target, bytes) || !aligned(draft, bytes) ||
      !words_ok({draft_tokens, uniforms, num_draft, temperature, tokens_out, count_out, logprobs_out}))
    return WMTP_ERR_INVALID_ARG;
  if (target_batch_stride < 0 || target_row_stride < 0 || draft_batch_stride < 0 || draft_row_stride < 0)
    return WMTP_ERR_INVALID_ARG;
  AcceptArgs a;
  a.target = target, a.target_batch = target_batch_stride, a.target_row = target_row_stride;
  a.draft = num_q > 1 ? draft : nullptr, a.draft_batch = draft_batch_stride, a.draft_row = draft_row_stride;
  a.draft_tokens = draft_tokens, a.num_draft = num_draft, a.uniforms = uniforms, a.temperature = temperature;
  a.tokens = tokens_out, a.count = count_out, a.logprobs = logprobs_out, a.status = status_word;
  a.stats = static_cast<RowStat*>(workspace);
  a.B = batch, a.num_q = num_q, a.V = vocab;
  const unsigned rows = static_cast<unsigned>(batch) * (num_q + (a.draft != nullptr ? num_q - 1 : 0));
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  DeviceInfo info;
  wmtp_status s = current_device(&dev, &info);
  if (s != WMTP_OK) return s;
  int c = row_cluster(rows, vocab, bytes, info.sms);
  auto rows_kern =
      by_dtype(dtype, accept_rows_kernel<float>, accept_rows_kernel<__half>, accept_rows_kernel<__nv_bfloat16>);
  s = launch_clusters(true, rows_kern, dim3(rows * c), dim3(kRowThreads), c, st, a);
  if (s != WMTP_OK) return s;
  auto kern = by_dtype(dtype, accept_kernel<float>, accept_kernel<__half>, accept_kernel<__nv_bfloat16>);
  static WidestOnce once[3];
  c = final_cluster(batch, vocab, info.sms, widest_cluster(once[dtype], dev, kFinalCluster, [&] {
                      return clusters_that_fit(kern, kFinalThreads, kFinalCluster);
                    }));
  return launch_clusters(true, kern, dim3(static_cast<unsigned>(batch) * c), dim3(kFinalThreads), c, st, a);
}

}  // extern "C"
