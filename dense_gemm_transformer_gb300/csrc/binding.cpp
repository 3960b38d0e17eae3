// binding.cpp -- the operators on a paged cache for torch tensors: a CPython
// module that checks a call's tensors, fills the C ABI's structs (gemm.h) and
// calls the library.
//
// Marshalling only.  It is native because a small call is shorter than the
// same checks in Python.  The library is not linked: the functions' addresses
// come from the one that the package has loaded (bind).
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <exception>
#include <optional>
#include <string>

#include "gemm.h"

namespace {

PyObject* g_error = nullptr;  // GemmError

// The library's functions, in the order that bind takes their addresses.
struct Library {
  decltype(&gemm_rotary) rotary;
  decltype(&gemm_paged_attention) paged_attention;
  decltype(&gemm_cache_grow) cache_grow;
  decltype(&gemm_cache_shrink) cache_shrink;
  decltype(&gemm_cache_fork) cache_fork;
  decltype(&gemm_cache_compact) cache_compact;
  decltype(&gemm_cache_copy) cache_copy;
} g_lib;
constexpr Py_ssize_t kFunctions = sizeof(Library) / sizeof(void*);

// What a check throws: a Python exception to be.
struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused{PyExc_ValueError, what}; }
[[noreturn]] void refuse_type(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
struct Raised {};  // a Python exception is set already

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Raised{};
  return p;
}
gemm_handle_t handle_of(PyObject* o) {  // None: a closed handle, which the library refuses
  return static_cast<gemm_handle_t>(o == Py_None ? nullptr : address(o));
}

// A stream as it is given: a torch stream or a raw handle.
void* stream_of(PyObject* given) {
  if (PyLong_Check(given)) return address(given);
  PyObject* raw = PyObject_GetAttrString(given, "cuda_stream");
  if (raw == nullptr) throw Raised{};
  void* s = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  if (PyErr_Occurred()) throw Raised{};
  return s;
}

// The current device, -1 where there is none.
c10::DeviceIndex current_device() {
  c10::DeviceIndex current = -1;
  return c10::cuda::GetDevice(&current) == cudaSuccess ? current : static_cast<c10::DeviceIndex>(-1);
}

// While it lives, new tensors come from the memory of the call's stream, as
// under torch.cuda.stream: a block of the current stream's could still be in
// use by work that the call's stream does not wait for.
class OutputsOn {
 public:
  OutputsOn(PyObject* given, const at::Tensor& like) {
    // (a tensor of another device is refused by Device::on)
    if (given == Py_None || !like.is_cuda() || like.get_device() != current_device()) return;
    const c10::DeviceIndex device = like.get_device();
    void* raw = stream_of(given);
    current_ = c10::cuda::getCurrentCUDAStream(device);
    if (raw == current_->stream()) return;
    guard_.emplace(raw == nullptr || raw == cudaStreamLegacy
                       ? c10::cuda::getDefaultCUDAStream(device)
                       : c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(raw), device));
  }
  // An output that the caller gets: it will most likely be read on the stream
  // that is current for the caller.
  at::Tensor give_back(at::Tensor t) const {
    if (guard_) t.record_stream(*current_);
    return t;
  }

 private:
  std::optional<c10::cuda::CUDAStream> current_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

// The tensors of a call are on the current device (as the library asks of its
// handle); its stream is the one given or the device's current one.
struct Device {
  int index = -1;
  void on(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    if (index < 0) {
      index = t.get_device();
      if (index != current_device()) refuse(std::string(name) + " must be on the current device");
    }
    if (t.get_device() != index) refuse("all tensors must be on one device");
  }
  void* stream(PyObject* given) const {
    if (given == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
    return stream_of(given);
  }
};

int type_code(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat: return GEMM_TYPE_FP32;
    case at::kBFloat16: return GEMM_TYPE_BF16;
    case at::kHalf: return GEMM_TYPE_FP16;
    default: refuse_type("float32, bfloat16 or float16 tensors are needed");
  }
}

// A dimension of one may have any stride.
int64_t stride(const at::Tensor& t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; }

// [tokens, heads, head_dim]
void heads(Device& dev, const at::Tensor& t, const char* name, int64_t dim, int64_t* token, int64_t* head) {
  dev.on(t, name);
  if (t.dim() != 3) refuse(std::string(name) + " must be a 3-D CUDA tensor [tokens, heads, head_dim]");
  if (t.stride(2) != 1 && t.size(2) > 1) refuse(std::string(name) + " needs unit stride along its last dimension");
  if (dim >= 0 && t.size(2) != dim)
    refuse(std::string(name) + " has head size " + std::to_string(t.size(2)) + ", not " + std::to_string(dim));
  *token = stride(t, 0);
  *head = stride(t, 1);
}

// [pages, page_size, kv_heads, head_dim]
void pages(Device& dev, const at::Tensor& t, const char* name, int64_t kv_heads, int64_t dim, int64_t* page,
           int64_t* slot, int64_t* head) {
  dev.on(t, name);
  if (t.dim() != 4 || t.size(2) != kv_heads || t.size(3) != dim)
    refuse(std::string(name) + " must be a CUDA tensor [pages, page_size, " + std::to_string(kv_heads) + ", " +
           std::to_string(dim) + "]");
  if (t.stride(3) != 1 && dim > 1) refuse(std::string(name) + " needs unit stride along its last dimension");
  *page = stride(t, 0);
  *slot = stride(t, 1);
  *head = stride(t, 2);
}

template <typename T>
const T* vector(Device& dev, const at::Tensor& t, const char* name, int64_t n, at::ScalarType type) {
  dev.on(t, name);
  if (t.dim() != 1 || t.scalar_type() != type || t.numel() != n || (n > 1 && t.stride(0) != 1))
    refuse(std::string(name) + " must be a contiguous CUDA vector of " + std::to_string(n) + " " + c10::toString(type));
  return static_cast<const T*>(t.data_ptr());
}

// A new tensor on the device of `like`, for the caller.
at::Tensor fresh(const OutputsOn& outputs, const at::Tensor& like, const char* name, at::IntArrayRef sizes,
                 at::ScalarType type) {
  if (!like.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return outputs.give_back(at::empty(sizes, like.options().dtype(type)));
}

PyObject* give(at::Tensor t) {
  PyObject* o = THPVariable_Wrap(std::move(t));
  if (o == nullptr) throw Raised{};
  return o;
}

// One call of the library, other threads running meanwhile (a launch waits
// while the stream's queue is full).
template <typename F, typename... A>
void call(const char* what, F fn, A... args) {
  PyThreadState* state = PyEval_SaveThread();
  const gemm_status_t status = fn(args...);
  PyEval_RestoreThread(state);
  if (status == GEMM_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(status), what);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised{};
}

int32_t size32(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse(std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(n);
}

template <PyObject* (*F)(PyObject* const*)>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments are needed, %zd given", want, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const Raised&) {
  } catch (...) {  // torch's own, as torch raises them (memory that could not be had among them)
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// ------------------------------------------------------------------ rotary

// k, v, slots and freqs may be None; k_out and v_out are pools with slots.
void run_rotary(PyObject* handle, const at::Tensor& q, PyObject* k_, PyObject* v_, PyObject* positions, PyObject* slots,
                PyObject* freqs, PyObject* amplitude, PyObject* interleaved, bool inverse, const at::Tensor& q_out,
                PyObject* k_out_, PyObject* v_out_, PyObject* stream) {
  Device dev;
  gemm_rotary_t a;
  std::memset(&a, 0, sizeof(a));
  heads(dev, q, "q", -1, &a.q_token, &a.q_head);
  const int64_t tokens = q.size(0), dim = q.size(2);
  a.in_type = type_code(q);
  a.out_type = type_code(q_out);
  if (q_out.sizes() != q.sizes()) refuse("q_out must have q's shape");
  heads(dev, q_out, "q_out", dim, &a.q_out_token, &a.q_out_head);
  a.heads = size32(q.size(1), "heads");
  a.head_dim = size32(dim, "head_dim");
  a.interleaved = truth(interleaved);
  a.inverse = inverse;
  a.amplitude = static_cast<float>(real(amplitude));
  a.tokens = tokens;
  a.q = q.data_ptr();
  a.q_out = q_out.data_ptr();
  a.position_bytes = 8;
  if (k_ != Py_None) {
    const at::Tensor &k = tensor(k_, "k"), &k_out = tensor(k_out_, slots == Py_None ? "k_out" : "k_pages");
    heads(dev, k, "k", dim, &a.k_token, &a.k_head);
    a.kv_heads = size32(k.size(1), "kv_heads");
    if (k.size(0) != tokens) refuse("k has another number of tokens than q");
    if (k.scalar_type() != q.scalar_type() || k_out.scalar_type() != q_out.scalar_type())
      refuse_type("k and its output must have the types of q and its output");
    a.k = k.data_ptr();
    a.k_out = k_out.data_ptr();
    if (slots == Py_None) {
      if (k_out.sizes() != k.sizes()) refuse("k_out must have k's shape");
      heads(dev, k_out, "k_out", dim, &a.k_out_token, &a.k_out_head);
    } else {
      const at::Tensor &v = tensor(v_, "v"), &v_out = tensor(v_out_, "v_pages");
      heads(dev, v, "v", dim, &a.v_token, &a.v_head);
      if (v.sizes() != k.sizes() || v.scalar_type() != k.scalar_type() || v_out.scalar_type() != k_out.scalar_type())
        refuse("v and its pool must have the shape and type of k and its pool");
      pages(dev, k_out, "k_pages", a.kv_heads, dim, &a.k_out_page, &a.k_out_token, &a.k_out_head);
      pages(dev, v_out, "v_pages", a.kv_heads, dim, &a.v_out_page, &a.v_out_token, &a.v_out_head);
      if (v_out.size(0) != k_out.size(0) || v_out.size(1) != k_out.size(1))
        refuse("k_pages and v_pages must have the same pages");
      a.num_pages = k_out.size(0);
      a.page_size = size32(k_out.size(1), "page_size");
      if (a.page_size < 1) refuse("page_size must be positive");
      a.v = v.data_ptr();
      a.v_out = v_out.data_ptr();
      a.slots = vector<int64_t>(dev, tensor(slots, "slots"), "slots", tokens, at::kLong);
    }
  }
  if (freqs != Py_None) {
    const at::Tensor &f = tensor(freqs, "freqs"), &p = tensor(positions, "positions");
    a.freqs = vector<double>(dev, f, "freqs", f.numel(), at::kDouble);
    if (2 * f.numel() > dim) refuse("freqs has more than head_dim / 2 frequencies");
    a.rotary_dim = static_cast<int32_t>(2 * f.numel());
    if (p.scalar_type() == at::kInt) {
      a.position_bytes = 4;
      a.positions = vector<int32_t>(dev, p, "positions", tokens, at::kInt);
    } else {
      a.positions = vector<int64_t>(dev, p, "positions", tokens, at::kLong);
    }
  }
  call("gemm_rotary", g_lib.rotary, handle_of(handle), &a, dev.stream(stream));
}

// handle, q, k, positions, freqs, amplitude, interleaved, inverse, q_out, k_out, stream
PyObject* rotary(PyObject* const* x) {
  const at::Tensor& q = tensor(x[1], "q");
  const OutputsOn outputs(x[10], q);
  const at::Tensor q_out = x[8] == Py_None ? fresh(outputs, q, "q", q.sizes(), q.scalar_type()) : tensor(x[8], "q_out");
  PyObject *qo = x[8] == Py_None ? give(q_out) : Py_NewRef(x[8]), *ko = nullptr;
  try {
    if (x[2] == Py_None) {
      ko = Py_NewRef(Py_None);
    } else if (x[9] == Py_None) {
      const at::Tensor& k = tensor(x[2], "k");
      ko = give(fresh(outputs, k, "k", k.sizes(), k.scalar_type()));
    } else {
      ko = Py_NewRef(x[9]);
    }
    run_rotary(x[0], q, x[2], Py_None, x[3], Py_None, x[4], x[5], x[6], truth(x[7]), q_out, ko, Py_None, x[10]);
    PyObject* both = PyTuple_Pack(2, qo, ko);
    Py_DECREF(qo);
    Py_DECREF(ko);
    return both;
  } catch (...) {
    Py_XDECREF(qo);
    Py_XDECREF(ko);
    throw;
  }
}

// handle, q, k, v, positions, slots, k_pages, v_pages, freqs, amplitude, interleaved, q_out, stream
PyObject* rotary_append(PyObject* const* x) {
  const at::Tensor& q = tensor(x[1], "q");
  const at::Tensor& pool = tensor(x[6], "k_pages");
  if (x[2] == Py_None || x[3] == Py_None || x[5] == Py_None) refuse_type("k, v and slots are needed");
  const OutputsOn outputs(x[12], q);
  const at::Tensor q_out =
      x[11] == Py_None ? fresh(outputs, q, "q", q.sizes(), pool.scalar_type()) : tensor(x[11], "q_out");
  run_rotary(x[0], q, x[2], x[3], x[4], x[5], x[8], x[9], x[10], false, q_out, x[6], x[7], x[12]);
  return x[11] == Py_None ? give(q_out) : Py_NewRef(x[11]);
}

// --------------------------------------------------------------- attention

void table_of(Device& dev, const at::Tensor& t, int32_t* sequences, int32_t* width, int64_t* row) {
  dev.on(t, "table");
  if (t.dim() != 2 || t.scalar_type() != at::kInt || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("table must be an int32 CUDA matrix with unit stride along its rows");
  *sequences = size32(t.size(0), "sequences");
  *width = size32(t.size(1), "table width");
  *row = stride(t, 0);
}

// handle, q, k_pages, v_pages, table, kv_lens, cu_q, max_q, max_kv, scale, softcap, window, out, return_lse, stream
PyObject* paged_attention(PyObject* const* x) {
  const at::Tensor &q = tensor(x[1], "q"), &k = tensor(x[2], "k_pages"), &v = tensor(x[3], "v_pages");
  const at::Tensor& table = tensor(x[4], "table");
  Device dev;
  gemm_paged_attention_t a;
  std::memset(&a, 0, sizeof(a));
  heads(dev, q, "q", -1, &a.q_token, &a.q_head);
  const int64_t tokens = q.size(0), dim = q.size(2);
  const int64_t kv_heads = k.dim() == 4 ? k.size(2) : 0;
  pages(dev, k, "k_pages", kv_heads, dim, &a.k_page, &a.k_slot, &a.k_head);
  pages(dev, v, "v_pages", kv_heads, dim, &a.v_page, &a.v_slot, &a.v_head);
  if (v.sizes() != k.sizes()) refuse("k_pages and v_pages must have the same shape");
  if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type() || type_code(q) == GEMM_TYPE_FP32)
    refuse_type("q and the pages must all be bfloat16 or all float16");
  table_of(dev, table, &a.sequences, &a.table_width, &a.table_row);
  a.kv_lens = vector<int32_t>(dev, tensor(x[5], "kv_lens"), "kv_lens", a.sequences, at::kInt);
  if (x[6] != Py_None) {
    a.cu_q = vector<int32_t>(dev, tensor(x[6], "cu_q"), "cu_q", static_cast<int64_t>(a.sequences) + 1, at::kInt);
    if (x[7] == Py_None) refuse("cu_q needs max_q, the most new tokens of a sequence");
    a.max_q = integer32(x[7], "max_q");
  } else {
    if (tokens != a.sequences) refuse("without cu_q, q has one token for each sequence");
    a.max_q = 1;
  }
  a.type = type_code(q);
  a.heads = size32(q.size(1), "heads");
  a.kv_heads = size32(kv_heads, "kv_heads");
  a.head_dim = size32(dim, "head_dim");
  a.page_size = size32(k.size(1), "page_size");
  a.window = integer32(x[11], "window");
  a.scale = x[9] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(dim)))
                          : static_cast<float>(real(x[9]));
  a.softcap = static_cast<float>(real(x[10]));
  a.tokens = tokens;
  a.num_pages = k.size(0);
  a.max_kv = integer(x[8]);
  const OutputsOn outputs(x[14], q);
  at::Tensor out;
  if (x[12] == Py_None) {
    out = fresh(outputs, q, "q", q.sizes(), q.scalar_type());
  } else {
    out = tensor(x[12], "out");
    if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type()) refuse("out must have q's shape and type");
  }
  heads(dev, out, "out", dim, &a.out_token, &a.out_head);
  at::Tensor lse;
  const bool with_lse = truth(x[13]);
  if (with_lse) {
    lse = fresh(outputs, q, "q", {tokens, q.size(1)}, at::kFloat);
    a.lse = static_cast<float*>(lse.data_ptr());
  }
  a.q = q.data_ptr();
  a.k_pages = k.data_ptr();
  a.v_pages = v.data_ptr();
  a.table = static_cast<const int32_t*>(table.data_ptr());
  a.out = out.data_ptr();
  call("gemm_paged_attention", g_lib.paged_attention, handle_of(x[0]), &a, dev.stream(x[14]));
  PyObject* o = x[12] == Py_None ? give(std::move(out)) : Py_NewRef(x[12]);
  if (!with_lse) return o;
  PyObject* l = give(std::move(lse));
  PyObject* both = PyTuple_Pack(2, o, l);
  Py_DECREF(o);
  Py_DECREF(l);
  return both;
}

// ------------------------------------------------------------------- pages

// A pool [..., pages, page_size, kv_heads, head_dim] or [..., pages,
// elements], its pages contiguous, its leading dimensions one strided one.
void pool_of(Device& dev, const at::Tensor& t, gemm_cache_t& c, int i, int64_t* count, int64_t* bytes) {
  dev.on(t, "a pool");
  const int64_t inner = t.dim() >= 4 ? 3 : 1, lead = t.dim() - inner - 1;
  if (lead < 0) refuse("a pool must have pages along dimension -4, or -2 of fewer than four dimensions");
  // the dimensions of a page by stride: contiguous in some order
  int64_t expected = 1;
  bool used[3] = {false, false, false};
  for (int64_t n = 0; n < inner; ++n) {
    int best = -1;
    for (int64_t d = 0; d < inner; ++d)
      if (!used[d] && (best < 0 || t.stride(lead + 1 + d) < t.stride(lead + 1 + best) ||
                       (t.stride(lead + 1 + d) == t.stride(lead + 1 + best) &&
                        t.size(lead + 1 + d) < t.size(lead + 1 + best))))
        best = static_cast<int>(d);
    used[best] = true;
    const int64_t size = t.size(lead + 1 + best);
    if (size > 1 && t.stride(lead + 1 + best) != expected) refuse("a pool's pages must be contiguous");
    expected *= size > 1 ? size : 1;
  }
  int64_t elements = 1, groups = 1, group_stride = 0;
  bool strided = false;
  for (int64_t d = lead + 1; d < t.dim(); ++d) elements *= t.size(d);
  for (int64_t d = lead - 1; d >= 0; --d) {
    if (t.size(d) > 1) {
      if (strided && t.stride(d) != group_stride * groups)
        refuse("a pool's leading dimensions must be one strided dimension");
      if (!strided) group_stride = t.stride(d);
      strided = true;
    }
    groups *= t.size(d);
  }
  const int64_t size = t.element_size();
  c.pools[i] = t.data_ptr();
  c.pool_groups[i] = groups;
  c.pool_group_stride[i] = group_stride * size;
  c.pool_page_stride[i] = stride(t, lead) * size;
  *count = t.size(lead);
  *bytes = elements * size;
}

// The state (table and refs, and lens unless it is None; or none of them) and
// the pools (a sequence of tensors, or None).
gemm_cache_t cache_of(Device& dev, PyObject* pools, PyObject* table, PyObject* lens, PyObject* refs,
                      PyObject* page_size) {
  gemm_cache_t c;
  std::memset(&c, 0, sizeof(c));
  c.page_size = page_size == nullptr ? 1 : integer32(page_size, "page_size");
  if (c.page_size < 1) refuse("page_size must be positive");
  if (table != nullptr) {
    const at::Tensor &t = tensor(table, "table"), &r = tensor(refs, "refs");
    table_of(dev, t, &c.sequences, &c.table_width, &c.table_row);
    c.table = static_cast<int32_t*>(t.data_ptr());
    c.num_pages = r.numel();
    c.refs = const_cast<int32_t*>(vector<int32_t>(dev, r, "refs", c.num_pages, at::kInt));
    if (lens != nullptr)
      c.lens = const_cast<int32_t*>(vector<int32_t>(dev, tensor(lens, "lens"), "lens", c.sequences, at::kInt));
  }
  if (pools == nullptr) return c;
  PyObject* fast = PySequence_Fast(pools, "pools must be a sequence of tensors");
  if (fast == nullptr) throw Raised{};
  try {
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(fast);
    if (n > 8) refuse("at most 8 pools");
    for (Py_ssize_t i = 0; i < n; ++i) {
      int64_t count, bytes;
      pool_of(dev, tensor(PySequence_Fast_GET_ITEM(fast, i), "a pool"), c, static_cast<int>(i), &count, &bytes);
      if (i == 0) {
        c.page_bytes = bytes;
        if (table == nullptr) c.num_pages = count;
      }
      if (count != c.num_pages)
        refuse("a pool has " + std::to_string(count) + " pages, not " + std::to_string(c.num_pages));
      if (bytes != c.page_bytes) refuse("the pools' pages must have the same size");
    }
    c.pool_count = static_cast<int32_t>(n);
  } catch (...) {
    Py_DECREF(fast);
    throw;
  }
  Py_DECREF(fast);
  return c;
}

PyObject* pack(std::initializer_list<at::Tensor> tensors) {
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(tensors.size()));
  if (t == nullptr) throw Raised{};
  Py_ssize_t i = 0;
  for (const at::Tensor& x : tensors) {
    PyObject* o = THPVariable_Wrap(x);
    if (o == nullptr) {
      Py_DECREF(t);
      throw Raised{};
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// handle, table, lens, refs, page_size, seqs, counts, tokens, stream, pools
PyObject* cache_grow(PyObject* const* x) {
  Device dev;
  const gemm_cache_t c = cache_of(dev, x[9] == Py_None ? nullptr : x[9], x[1], x[2], x[3], x[4]);
  const at::Tensor& seqs = tensor(x[5], "seqs");
  const int64_t n = seqs.numel(), tokens = integer(x[7]);
  if (tokens < 0) refuse("tokens must not be negative");
  const int32_t* s = vector<int32_t>(dev, seqs, "seqs", n, at::kInt);
  const int32_t* k = vector<int32_t>(dev, tensor(x[6], "counts"), "counts", n, at::kInt);
  const OutputsOn outputs(x[8], seqs);
  at::Tensor positions = fresh(outputs, seqs, "seqs", {tokens}, at::kLong);
  at::Tensor slots = fresh(outputs, seqs, "seqs", {tokens}, at::kLong);
  at::Tensor info = fresh(outputs, seqs, "seqs", {3}, at::kInt);
  call("gemm_cache_grow", g_lib.cache_grow, handle_of(x[0]), &c, n, s, k, tokens,
       static_cast<int64_t*>(positions.data_ptr()), static_cast<int64_t*>(slots.data_ptr()),
       static_cast<int32_t*>(info.data_ptr()), dev.stream(x[8]));
  return pack({positions, slots, info});
}

// handle, table, lens, refs, page_size, seqs, counts, stream
PyObject* cache_shrink(PyObject* const* x) {
  Device dev;
  const gemm_cache_t c = cache_of(dev, nullptr, x[1], x[2], x[3], x[4]);
  const at::Tensor& seqs = tensor(x[5], "seqs");
  const int64_t n = seqs.numel();
  const int32_t* s = vector<int32_t>(dev, seqs, "seqs", n, at::kInt);
  const int32_t* k = x[6] == Py_None ? nullptr : vector<int32_t>(dev, tensor(x[6], "counts"), "counts", n, at::kInt);
  call("gemm_cache_shrink", g_lib.cache_shrink, handle_of(x[0]), &c, n, s, k, dev.stream(x[7]));
  Py_RETURN_NONE;
}

// handle, pools, table, lens, refs, page_size, parents, children, stream
PyObject* cache_fork(PyObject* const* x) {
  Device dev;
  const gemm_cache_t c = cache_of(dev, x[1], x[2], x[3], x[4], x[5]);
  const at::Tensor& parents = tensor(x[6], "parents");
  const int64_t n = parents.numel();
  const int32_t* p = vector<int32_t>(dev, parents, "parents", n, at::kInt);
  const int32_t* k = vector<int32_t>(dev, tensor(x[7], "children"), "children", n, at::kInt);
  const OutputsOn outputs(x[8], parents);
  at::Tensor copied = fresh(outputs, parents, "parents", {n}, at::kInt);
  at::Tensor info = fresh(outputs, parents, "parents", {3}, at::kInt);
  call("gemm_cache_fork", g_lib.cache_fork, handle_of(x[0]), &c, n, p, k, static_cast<int32_t*>(copied.data_ptr()),
       static_cast<int32_t*>(info.data_ptr()), dev.stream(x[8]));
  return pack({copied, info});
}

// handle, pools, table, refs, stream
PyObject* cache_compact(PyObject* const* x) {
  Device dev;
  const gemm_cache_t c = cache_of(dev, x[1], x[2], nullptr, x[3], nullptr);
  const at::Tensor& table = tensor(x[2], "table");
  const OutputsOn outputs(x[4], table);
  at::Tensor info = fresh(outputs, table, "table", {2}, at::kInt);
  call("gemm_cache_compact", g_lib.cache_compact, handle_of(x[0]), &c, static_cast<int32_t*>(info.data_ptr()),
       dev.stream(x[4]));
  return give(std::move(info));
}

// handle, pools, src, dst, stream
PyObject* cache_copy(PyObject* const* x) {
  Device dev;
  const at::Tensor& src = tensor(x[2], "src");
  const int64_t n = src.numel();
  const int32_t* s = vector<int32_t>(dev, src, "src", n, at::kInt);
  const int32_t* d = vector<int32_t>(dev, tensor(x[3], "dst"), "dst", n, at::kInt);
  const gemm_cache_t c = cache_of(dev, x[1], nullptr, nullptr, nullptr, nullptr);
  call("gemm_cache_copy", g_lib.cache_copy, handle_of(x[0]), &c, n, s, d, dev.stream(x[4]));
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  return guarded<F>(self, args, n, N);
}
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<F, N>)), METH_FASTCALL, nullptr};
}

// bind(error, addresses): the exception that a status other than GEMM_OK
// raises, and the functions of Library.
PyObject* bind(PyObject* const* x) {
  if (!PyTuple_Check(x[1]) || PyTuple_GET_SIZE(x[1]) != kFunctions) refuse_type("a tuple of the functions is needed");
  void* fn[kFunctions];
  for (Py_ssize_t i = 0; i < kFunctions; ++i) {
    fn[i] = address(PyTuple_GET_ITEM(x[1], i));
    if (fn[i] == nullptr) refuse("a function of the library is missing");
  }
  std::memcpy(&g_lib, fn, sizeof(g_lib));
  Py_XSETREF(g_error, Py_NewRef(x[0]));
  Py_RETURN_NONE;
}

// The current device.
PyObject* device(PyObject* const*) { return PyLong_FromLong(c10::cuda::current_device()); }

PyMethodDef g_methods[] = {
    method<rotary, 11>("rotary"),
    method<rotary_append, 13>("rotary_append"),
    method<paged_attention, 15>("paged_attention"),
    method<cache_grow, 10>("cache_grow"),
    method<cache_shrink, 8>("cache_shrink"),
    method<cache_fork, 9>("cache_fork"),
    method<cache_compact, 5>("cache_compact"),
    method<cache_copy, 5>("cache_copy"),
    method<device, 0>("device"),
    method<bind, 2>("bind"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
