// Argument checks, output allocation and marshalling of the wmtp_step.h calls for
// speculative_decode_draft_b200/step.py.  Compiled, because these calls are short: a
// verify block's kernels take 3 to 12 us, and host time with it is 4 to 10 us a call;
// the same in Python over ctypes was 14 to 19.
//
// The calls themselves are in libwmtp.so; init() gets their addresses from the ctypes
// handle, so the library is found in one place.  Everything runs on the tensors'
// device and its current stream; outputs and scratch come from PyTorch's allocator on
// that stream.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <limits>
#include <string>

#include "wmtp_step.h"

namespace {

decltype(&wmtp_qk_norm_rope) f_rope = nullptr;
decltype(&wmtp_pages_resize) f_pages = nullptr;
decltype(&wmtp_token_logprobs) f_logprobs = nullptr;
decltype(&wmtp_accept_draft) f_accept = nullptr;

// Python's TypeError and ValueError, with a printf-style message.
template <bool kType>
struct Refusal : public torch::PyTorchError {
  __attribute__((format(printf, 2, 3))) explicit Refusal(const char* format, ...) {
    char buf[512];
    va_list args;
    va_start(args, format);
    std::vsnprintf(buf, sizeof(buf), format, args);
    va_end(args);
    msg = buf;
  }
  PyObject* python_type() override { return kType ? PyExc_TypeError : PyExc_ValueError; }
};
using TypeError = Refusal<true>;
using ValueError = Refusal<false>;

using Sizes = std::initializer_list<int64_t>;
using c10::ScalarType;

std::string text(c10::IntArrayRef sizes) {
  std::string s = "[";
  for (size_t i = 0; i < sizes.size(); ++i) s += (i ? ", " : "") + std::to_string(sizes[i]);
  return s + "]";
}

const char* text(ScalarType t) {
  return t == ScalarType::Int ? "torch.int32" : t == ScalarType::Long ? "torch.int64" : t == ScalarType::Float ? "torch.float32"
         : t == ScalarType::BFloat16 ? "torch.bfloat16" : c10::toString(t);
}

// A tensor, or NULL for None where that is allowed.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw TypeError("%s must be a torch.Tensor", name);
  return &THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, const char* name, int device) {
  if (!t.is_cuda()) throw ValueError("%s must be a CUDA tensor", name);
  if (t.get_device() != device)
    throw ValueError("%s is on cuda:%d, expected cuda:%d", name, static_cast<int>(t.get_device()), device);
}

// dtype, device, contiguity; the address (NULL for NULL).
void* plain(const at::Tensor* t, const char* name, ScalarType type, int device) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != type)
    throw TypeError("%s must be %s, got %s", name, text(type), text(t->scalar_type()));
  on_device(*t, name, device);
  if (!t->is_contiguous()) throw ValueError("%s must be contiguous", name);
  return t->data_ptr();
}

void* shaped(const at::Tensor* t, const char* name, ScalarType type, int device, c10::IntArrayRef sizes) {
  void* p = plain(t, name, type, device);
  if (t != nullptr && t->sizes() != sizes)
    throw ValueError("%s must be %s, got %s", name, text(sizes).c_str(), text(t->sizes()).c_str());
  return p;
}

int32_t i32(int64_t v, const char* name) {
  if (v > std::numeric_limits<int32_t>::max()) throw ValueError("%s: too large", name);
  return static_cast<int32_t>(v);
}

int32_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  if (v < 0) throw ValueError("%s must not be negative", name);
  return i32(v, name);
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(v);
}

wmtp_params params(PyObject* o) {
  Py_buffer view;
  if (PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) != 0) throw python_error();
  wmtp_params p;
  const bool fits = view.len == sizeof(p);
  if (fits) std::memcpy(&p, view.buf, sizeof(p));
  PyBuffer_Release(&view);
  if (!fits) throw TypeError("p must be made by params()");
  return p;
}

int32_t logit_type(const at::Tensor& t, const char* name) {
  if (t.dim() > 0 && t.size(-1) > 1 && t.stride(-1) != 1)
    throw ValueError("%s: the logits of a row must be next to one another", name);
  switch (t.scalar_type()) {
    case ScalarType::BFloat16: return WMTP_BF16;
    case ScalarType::Half: return WMTP_FP16;
    case ScalarType::Float: return WMTP_FP32;
    default: throw TypeError("%s must be bf16, fp16 or fp32, got %s", name, text(t.scalar_type()));
  }
}

// Strides of axes with one entry say nothing.
int64_t row_stride(const at::Tensor& t, int axis) { return t.size(axis) > 1 ? t.stride(axis) : t.size(-1); }

at::Tensor make(c10::IntArrayRef sizes, ScalarType type, int device) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device))));
}

void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

void* status_of(PyObject* o, int device) { return plain(tensor(o, "status", true), "status", ScalarType::Int, device); }

void count_args(Py_ssize_t have, Py_ssize_t want) {
  if (have != want) throw TypeError("%d arguments, expected %d", static_cast<int>(have), static_cast<int>(want));
}

// (status code, tensors), None for those that are not there.
PyObject* answer(wmtp_status code, std::initializer_list<const at::Tensor*> out) {
  PyObject* tuple = PyTuple_New(1 + static_cast<Py_ssize_t>(out.size()));
  if (tuple == nullptr) throw python_error();
  PyTuple_SET_ITEM(tuple, 0, PyLong_FromLong(code));
  Py_ssize_t i = 1;
  for (const at::Tensor* t : out) {
    PyObject* o = t != nullptr && t->defined() ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    PyTuple_SET_ITEM(tuple, i++, o);
  }
  return tuple;
}

template <typename F>
wmtp_status without_gil(F f) {
  wmtp_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  return s;
}

// ---------------------------------------------------------------- calls
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 4);
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) throw ValueError("a call's address is missing");
  }
  f_rope = reinterpret_cast<decltype(f_rope)>(p[0]);
  f_pages = reinterpret_cast<decltype(f_pages)>(p[1]);
  f_logprobs = reinterpret_cast<decltype(f_logprobs)>(p[2]);
  f_accept = reinterpret_cast<decltype(f_accept)>(p[3]);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// A [..., heads, dim] view with one token stride.
struct Heads {
  const void* p = nullptr;
  int64_t token = 0, head = 0;
};

Heads heads(const at::Tensor* t, const char* name, ScalarType type, int device, c10::IntArrayRef lead, int64_t count,
            int64_t dim) {
  Heads h;
  if (t == nullptr) return h;
  on_device(*t, name, device);
  if (t->scalar_type() != type)
    throw TypeError("%s must be %s, got %s", name, text(type), text(t->scalar_type()));
  c10::SmallVector<int64_t, 4> want(lead.begin(), lead.end());
  want.push_back(count);
  want.push_back(dim);
  if (t->sizes() != c10::IntArrayRef(want))
    throw ValueError("%s must be %s, got %s", name, text(want).c_str(), text(t->sizes()).c_str());
  const auto st = t->strides();
  const size_t axes = lead.size();
  if (dim > 1 && st[axes + 1] != 1)
    throw ValueError("%s: the elements of a head must be next to one another", name);
  h.p = t->data_ptr();
  h.head = count > 1 ? st[axes] : 0;  // strides of axes with one entry say nothing
  if (axes == 2 && lead[1] > 1) {
    if (lead[0] > 1 && st[0] != lead[1] * st[1]) throw ValueError("%s: tokens must be evenly spaced", name);
    h.token = st[1];
  } else {
    h.token = lead[0] > 1 ? st[0] : 0;
  }
  return h;
}

// (p, turn | None, interleaved, factor, q, k, v, positions, slots, k_pool, v_pool, q_weight, k_weight, eps,
//  weight_offset, q_out, k_out, status) -> (code, q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 18);
  const wmtp_params p = params(a[0]);
  const at::Tensor* turn = tensor(a[1], "rope.turn", true);
  const at::Tensor *q = tensor(a[4], "q", true), *k = tensor(a[5], "k", true), *v = tensor(a[6], "v", true);
  const at::Tensor* first = q != nullptr ? q : k;
  if (first == nullptr) throw ValueError("q or k is needed");
  if (!first->is_cuda()) throw ValueError("%s must be a CUDA tensor", q != nullptr ? "q" : "k");
  const int device = static_cast<int>(first->get_device());
  const c10::cuda::OptionalCUDAGuard guard(first->device());
  const ScalarType type = first->scalar_type();
  if (type != ScalarType::BFloat16 && type != ScalarType::Float)
    throw TypeError("q, k and v must be bf16 or fp32, got %s", text(type));
  if (first->dim() != 3 && first->dim() != 4)
    throw ValueError("q and k must be [tokens, heads, dim] or [batch, tokens, heads, dim]");
  const c10::IntArrayRef lead = first->sizes().slice(0, first->dim() - 2);
  const int64_t D = p.head_dim;
  const Heads hq = heads(q, "q", type, device, lead, p.num_heads_q, D);
  const Heads hk = heads(k, "k", type, device, lead, p.num_heads_kv, D);
  const Heads hv = heads(v, "v", type, device, lead, p.num_heads_kv, D);
  const void* positions = shaped(tensor(a[7], "positions"), "positions", ScalarType::Int, device, lead);
  const at::Tensor* slots = tensor(a[8], "slots", true);
  wmtp_paged_kv kv;
  std::memset(&kv, 0, sizeof(kv));
  if (slots != nullptr) {
    shaped(slots, "slots", ScalarType::Long, device, lead);
    if (a[9] == Py_None || a[10] == Py_None) throw ValueError("slots need a cache");
    const at::Tensor *kp = tensor(a[9], "cache.k_pool"), *vp = tensor(a[10], "cache.v_pool");
    const int64_t pages = kp->dim() > 0 ? kp->size(0) : 0;
    const Sizes pool = {pages, p.num_heads_kv, p.page_size, D};
    kv.k_pool = shaped(kp, "cache.k_pool", ScalarType::BFloat16, device, pool);
    kv.v_pool = shaped(vp, "cache.v_pool", ScalarType::BFloat16, device, pool);
    kv.num_pages = i32(pages, "cache.k_pool");
  }
  const at::Tensor *qw = tensor(a[11], "q_weight", true), *kw = tensor(a[12], "k_weight", true);
  ScalarType wt = ScalarType::BFloat16;
  for (const at::Tensor* w : {qw, kw}) {
    const char* name = w == qw ? "q_weight" : "k_weight";
    if (w == nullptr) continue;
    wt = w->scalar_type();
    if (wt != ScalarType::BFloat16 && wt != ScalarType::Float) throw TypeError("%s must be bf16 or fp32", name);
    shaped(w, name, wt, device, {D});
  }
  if (qw != nullptr && kw != nullptr && qw->scalar_type() != kw->scalar_type())
    throw TypeError("q_weight and k_weight must have one dtype");
  wmtp_rope rope;
  std::memset(&rope, 0, sizeof(rope));
  if (turn != nullptr) {
    rope.turn = static_cast<const uint64_t*>(plain(turn, "rope.turn", ScalarType::Long, device));
    rope.rotary_dim = i32(2 * turn->numel(), "rope.turn");
    rope.interleaved = PyObject_IsTrue(a[2]);
    rope.factor = number(a[3]);
  }
  const float eps = number(a[13]), offset = number(a[14]);
  c10::SmallVector<int64_t, 4> sq(lead.begin(), lead.end()), sk(lead.begin(), lead.end());
  sq.append({p.num_heads_q, D});
  sk.append({p.num_heads_kv, D});
  at::Tensor qo, ko;
  if (a[15] != Py_None)
    qo = *tensor(a[15], "q_out"), shaped(&qo, "q_out", ScalarType::BFloat16, device, sq);
  else if (q != nullptr)
    qo = make(sq, ScalarType::BFloat16, device);
  if (a[16] != Py_None)
    ko = *tensor(a[16], "k_out"), shaped(&ko, "k_out", ScalarType::BFloat16, device, sk);
  else if (k != nullptr && slots == nullptr)
    ko = make(sk, ScalarType::BFloat16, device);
  int32_t* status = static_cast<int32_t*>(status_of(a[17], device));
  int64_t tokens = 1;
  for (const int64_t s : lead) tokens *= s;
  wmtp_status code = WMTP_OK;
  if (tokens > 0) {  // empty tensors have no address
    void* st = stream_of(device);
    const int32_t count = i32(tokens, "q");
    void *qp = qo.defined() ? qo.data_ptr() : nullptr, *kp = ko.defined() ? ko.data_ptr() : nullptr;
    code = without_gil([&] {
      return f_rope(&p, turn != nullptr ? &rope : nullptr, count, type == ScalarType::Float ? WMTP_FP32 : WMTP_BF16,
                    hq.p, hq.token, hq.head, hk.p, hk.token, hk.head, hv.p, hv.token, hv.head,
                    static_cast<const int32_t*>(positions),
                    slots != nullptr ? static_cast<const int64_t*>(slots->data_ptr()) : nullptr,
                    slots != nullptr ? &kv : nullptr, qw != nullptr ? qw->data_ptr() : nullptr,
                    kw != nullptr ? kw->data_ptr() : nullptr, wt == ScalarType::Float ? WMTP_FP32 : WMTP_BF16, offset, eps, qp,
                    kp, status, st);
    });
  }
  return answer(code, {&qo, &ko});
  END_HANDLE_TH_ERRORS
}

// (p, free, count, page_table, kv_len, new_len, max_tokens, status) -> (code, cu_tokens, positions, slots)
PyObject* pages_resize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 8);
  const wmtp_params p = params(a[0]);
  const at::Tensor* table = tensor(a[3], "page_table");
  if (!table->is_cuda()) throw ValueError("page_table must be a CUDA tensor");
  const int device = static_cast<int>(table->get_device());
  const c10::cuda::OptionalCUDAGuard guard(table->device());
  if (table->dim() != 2) throw ValueError("page_table must be [batch, max_pages]");
  const int64_t B = table->size(0), width = table->size(1);
  int32_t* tp = static_cast<int32_t*>(plain(table, "page_table", ScalarType::Int, device));
  int32_t* len = static_cast<int32_t*>(shaped(tensor(a[4], "kv_len"), "kv_len", ScalarType::Int, device, {B}));
  const int32_t* new_len = static_cast<int32_t*>(shaped(tensor(a[5], "new_len"), "new_len", ScalarType::Int, device, {B}));
  const at::Tensor* free = tensor(a[1], "pool.free");
  int32_t* fp = static_cast<int32_t*>(shaped(free, "pool.free", ScalarType::Int, device, {free->numel()}));
  int32_t* count = static_cast<int32_t*>(shaped(tensor(a[2], "pool.count"), "pool.count", ScalarType::Int, device, {1}));
  const int32_t most = integer(a[6], "max_tokens");
  int32_t* status = static_cast<int32_t*>(status_of(a[7], device));
  const int32_t batch = i32(B, "page_table"), pages = i32(width, "page_table"), total = i32(free->numel(), "pool.free");
  at::Tensor cu, positions, slots, ws;
  if (most > 0) {
    cu = make({B + 1}, ScalarType::Int, device);
    positions = make({most}, ScalarType::Int, device);
    slots = make({most}, ScalarType::Long, device);
  }
  int32_t *cp = most > 0 ? static_cast<int32_t*>(cu.data_ptr()) : nullptr,
          *pp = most > 0 ? static_cast<int32_t*>(positions.data_ptr()) : nullptr;
  int64_t* sp = most > 0 ? static_cast<int64_t*>(slots.data_ptr()) : nullptr;
  size_t size = 0;
  wmtp_status code = f_pages(&p, batch, tp, pages, len, new_len, nullptr, nullptr, total, cp, pp, sp, most, nullptr, &size,
                             nullptr, nullptr);
  if (code == WMTP_OK) {
    if (size > 0) ws = make({static_cast<int64_t>(size)}, ScalarType::Byte, device);
    void *wp = size > 0 ? ws.data_ptr() : nullptr, *st = stream_of(device);
    code = without_gil([&] {
      return f_pages(&p, batch, tp, pages, len, new_len, fp, count, total, cp, pp, sp, most, wp, &size, status, st);
    });
  }
  return answer(code, {&cu, &positions, &slots});
  END_HANDLE_TH_ERRORS
}

// (logits, tokens, top_k, temperature, status) -> (code, logprobs, entropy, lse, top_logprobs, top_ids)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 5);
  const at::Tensor *x = tensor(a[0], "logits"), *tokens = tensor(a[1], "tokens");
  if (!x->is_cuda()) throw ValueError("logits must be a CUDA tensor");
  const int device = static_cast<int>(x->get_device());
  const c10::cuda::OptionalCUDAGuard guard(x->device());
  const int32_t type = logit_type(*x, "logits");
  if (x->dim() != 2 || tokens->dim() != 2) throw ValueError("logits must be [rows, vocab] and tokens [rows, n]");
  const int64_t R = x->size(0), V = x->size(1), given = tokens->size(1);
  const int32_t* ids = static_cast<int32_t*>(shaped(tokens, "tokens", ScalarType::Int, device, {R, given}));
  const at::Tensor* temperature = tensor(a[3], "temperature", true);
  const float* tp = static_cast<float*>(shaped(temperature, "temperature", ScalarType::Float, device, {R}));
  const int32_t top_k = integer(a[2], "top_k");
  int32_t* status = static_cast<int32_t*>(status_of(a[4], device));
  const at::Tensor lp = make({R, given}, ScalarType::Float, device), entropy = make({R}, ScalarType::Float, device),
                   lse = make({R}, ScalarType::Float, device);
  at::Tensor top, top_ids;
  if (top_k > 0) {
    top = make({R, top_k}, ScalarType::Float, device);
    top_ids = make({R, top_k}, ScalarType::Int, device);
  }
  const int32_t rows = i32(R, "logits"), vocab = i32(V, "logits"), num = i32(given, "tokens");
  void* st = stream_of(device);
  const wmtp_status code = without_gil([&] {
    return f_logprobs(rows, vocab, type, x->data_ptr(), row_stride(*x, 0), tp, ids, num, top_k,
                      static_cast<float*>(lp.data_ptr()), static_cast<float*>(entropy.data_ptr()),
                      static_cast<float*>(lse.data_ptr()), top_k > 0 ? static_cast<float*>(top.data_ptr()) : nullptr,
                      top_k > 0 ? static_cast<int32_t*>(top_ids.data_ptr()) : nullptr, status, st);
  });
  return answer(code, {&lp, &entropy, &lse, &top, &top_ids});
  END_HANDLE_TH_ERRORS
}

// (target_logits, draft_tokens, uniforms, draft_logits, num_draft, temperature, status) -> (code, tokens, count, logprobs)
PyObject* accept_draft(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count_args(n, 7);
  const at::Tensor* x = tensor(a[0], "target_logits");
  if (!x->is_cuda()) throw ValueError("target_logits must be a CUDA tensor");
  const int device = static_cast<int>(x->get_device());
  const c10::cuda::OptionalCUDAGuard guard(x->device());
  const int32_t type = logit_type(*x, "target_logits");
  if (x->dim() != 3) throw ValueError("target_logits must be [batch, gamma + 1, vocab]");
  const int64_t B = x->size(0), rows = x->size(1), V = x->size(2);
  if (rows < 1) throw ValueError("target_logits needs a row for the token that follows");
  const int32_t* drafts =
      static_cast<int32_t*>(shaped(tensor(a[1], "draft_tokens"), "draft_tokens", ScalarType::Int, device, {B, rows - 1}));
  const float* u = static_cast<float*>(shaped(tensor(a[2], "uniforms"), "uniforms", ScalarType::Float, device, {B, rows}));
  const at::Tensor* draft = tensor(a[3], "draft_logits", true);
  int64_t draft_batch = 0, draft_row = 0;
  if (draft != nullptr) {
    logit_type(*draft, "draft_logits");
    if (!draft->is_cuda() || draft->get_device() != device || draft->scalar_type() != x->scalar_type())
      throw TypeError("draft_logits must have the device and dtype of target_logits");
    const Sizes want = {B, rows - 1, V};
    if (draft->sizes() != c10::IntArrayRef(want))
      throw ValueError("draft_logits must be %s, got %s", text(want).c_str(), text(draft->sizes()).c_str());
    draft_batch = row_stride(*draft, 0), draft_row = row_stride(*draft, 1);
  }
  const int32_t* num = static_cast<int32_t*>(shaped(tensor(a[4], "num_draft", true), "num_draft", ScalarType::Int, device, {B}));
  const float* temperature =
      static_cast<float*>(shaped(tensor(a[5], "temperature", true), "temperature", ScalarType::Float, device, {B}));
  int32_t* status = static_cast<int32_t*>(status_of(a[6], device));
  const int32_t batch = i32(B, "target_logits"), num_q = i32(rows, "target_logits"), vocab = i32(V, "target_logits");
  size_t size = 0;
  wmtp_status code = f_accept(batch, num_q, vocab, type, nullptr, 0, 0, nullptr, 0, 0, nullptr, nullptr, nullptr, nullptr,
                              nullptr, nullptr, nullptr, nullptr, &size, nullptr, nullptr);
  at::Tensor tokens, count, lp;
  if (code == WMTP_OK) {
    tokens = make({B, rows}, ScalarType::Int, device);
    count = make({B}, ScalarType::Int, device);
    lp = make({B, rows}, ScalarType::Float, device);
    if (size == 0) size = 256;  // an empty batch: a workspace that is not NULL all the same
    const at::Tensor ws = make({static_cast<int64_t>(size)}, ScalarType::Byte, device);
    void* st = stream_of(device);
    code = without_gil([&] {
      return f_accept(batch, num_q, vocab, type, x->data_ptr(), row_stride(*x, 0), row_stride(*x, 1),
                      draft != nullptr ? draft->data_ptr() : nullptr, draft_batch, draft_row, drafts, u, num, temperature,
                      static_cast<int32_t*>(tokens.data_ptr()), static_cast<int32_t*>(count.data_ptr()),
                      static_cast<float*>(lp.data_ptr()), ws.data_ptr(), &size, status, st);
    });
  }
  return answer(code, {&tokens, &count, &lp});
  END_HANDLE_TH_ERRORS
}

#define WMTP_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {WMTP_METHOD(init),           WMTP_METHOD(qk_norm_rope), WMTP_METHOD(pages_resize),
                         WMTP_METHOD(token_logprobs), WMTP_METHOD(accept_draft), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_step_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__step_binding() { return PyModule_Create(&module); }
