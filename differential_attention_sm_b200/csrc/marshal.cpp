// marshal.cpp — argument checks and marshalling of the serving operators for
// the Python binding (module _marshal, built by build.py with the host
// compiler).  Like the ctypes layer it only hands tensors' addresses and sizes
// to the library's C entry points; all arithmetic happens there.
//
// These calls take 3 to 10 us on the GPU.  Checked and passed from Python they
// took 13 to 20 us (the norm: 21 arguments 2, checks 2, two outputs 3),
// from here 6 to 11 with their launches.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <string>

#include "diffattn.h"

// The torch whose headers this was compiled against (build.py passes it).
#ifndef DA_TORCH_VERSION
#error "DA_TORCH_VERSION is not defined"
#endif

namespace {

#define DA_CALLS(X)                           \
  X(diffattn_page_plan_workspace_size)        \
  X(diffattn_page_plan)                       \
  X(diffattn_page_release)                    \
  X(diffattn_kv4_append)                      \
  X(diffattn_kv4_read)                        \
  X(diffattn_v2_decode_kv4_workspace_size)    \
  X(diffattn_v2_decode_kv4)                   \
  X(diffattn_v1_decode_kv4_workspace_size)    \
  X(diffattn_v1_decode_kv4)                   \
  X(diffattn_qk_norm_rope)                    \
  X(diffattn_qk_norm_rope_bwd_workspace_size) \
  X(diffattn_qk_norm_rope_bwd)

struct Library {
#define X(name) decltype(&::name) name = nullptr;
  DA_CALLS(X)
#undef X
};
Library lib;
PyObject* error_class = nullptr;

// ---- arguments ---------------------------------------------------------------
[[noreturn]] void refuse(PyObject* type, const char* format, ...) {
  va_list a;
  va_start(a, format);
  PyErr_FormatV(type, format, a);
  va_end(a);
  throw python_error();
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}
const at::Tensor* optional(PyObject* o, const char* name) {
  return o == Py_None ? nullptr : &tensor(o, name);
}
const at::Tensor* status_word(PyObject* o) {
  const at::Tensor* t = optional(o, "dev_status");
  if (t && (t->scalar_type() != at::kInt || t->numel() < 1))
    refuse(PyExc_TypeError, "dev_status must be an int32 word");
  return t;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int small(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v != (int)v) refuse(PyExc_ValueError, "%s is out of range", name);
  return (int)v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return (float)v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// A dense tensor of one type and shape (no shape: any).
void need(const char* name, const at::Tensor& t, at::ScalarType type) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s must be %s, not %s", name, c10::toString(type),
                           c10::toString(t.scalar_type()));
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "%s must be contiguous", name);
}
void need(const char* name, const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
  need(name, t, type);
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, "%s has shape %s, expected %s", name, shape_text(t.sizes()).c_str(),
                            shape_text(shape).c_str());
}
int as_int(const char* name, int64_t v) {
  if (v != (int)v) refuse(PyExc_ValueError, "%s is too large", name);
  return (int)v;
}

da_dtype code(const char* name, const at::Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return DA_BF16;
  if (t.scalar_type() == at::kFloat) return DA_FP32;
  refuse(PyExc_TypeError, "%s: unsupported dtype %s", name, c10::toString(t.scalar_type()));
}

// Token stride of t [T, H, d], whose heads of a token lie in a row.
int64_t token_stride(const char* name, const at::Tensor& t) {
  if (t.dim() != 3)
    refuse(PyExc_ValueError, "%s must be [tokens, heads, width], not %s", name,
                            shape_text(t.sizes()).c_str());
  const int64_t T = t.size(0), H = t.size(1), d = t.size(2);
  if ((d > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != d))
    refuse(PyExc_ValueError, "%s: the heads of a token must lie in a row", name);
  return T > 1 ? t.stride(0) : (H > 1 ? H : 1) * d;
}
int64_t token_stride(const char* name, const at::Tensor& t, int64_t tokens, at::ScalarType type) {
  if (t.dim() == 3 && t.size(0) != tokens)
    refuse(PyExc_ValueError, "%s must have %lld tokens, not %lld", name, (long long)tokens,
                            (long long)t.size(0));
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, "%s must be %s, not %s", name, c10::toString(type),
                           c10::toString(t.scalar_type()));
  return token_stride(name, t);
}

// A call's device and stream, made current for it: what it allocates (and fills)
// is ordered on that stream.
class On {
 public:
  template <typename... Ts>
  On(PyObject* stream, const at::Tensor& first, const Ts&... others)
      : index_(checked(first, others...)), guard_((c10::DeviceIndex)index_) {
    if (stream == Py_None) {
      stream_ = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index_).stream();
    } else {
      if (PyLong_Check(stream)) {
        stream_ = (cudaStream_t)(uintptr_t)integer(stream);
      } else {
        PyObject* raw = PyObject_GetAttrString(stream, "cuda_stream");
        if (!raw) throw python_error();
        stream_ = (cudaStream_t)(uintptr_t)PyLong_AsUnsignedLongLong(raw);
        Py_DECREF(raw);
        if (PyErr_Occurred()) throw python_error();
      }
      stream_guard_.reset_stream(
          c10::cuda::getStreamFromExternal(stream_, (c10::DeviceIndex)index_).unwrap());
    }
  }
  void* stream() const { return stream_; }
  // Scratch of a call that brings none.
  at::Tensor scratch(size_t bytes) const {
    return at::empty({(int64_t)(bytes ? bytes : 1)},
                     at::TensorOptions().dtype(at::kByte).device(at::kCUDA,
                                                                 (c10::DeviceIndex)index_));
  }

 private:
  static const at::Tensor* pointer(const at::Tensor& t) { return &t; }
  static const at::Tensor* pointer(const at::Tensor* t) { return t; }
  template <typename... Ts>
  static int checked(const at::Tensor& first, const Ts&... others) {
    if (!first.is_cuda()) refuse(PyExc_ValueError, "tensors must be CUDA tensors");
    const int at = first.get_device();
    for (const at::Tensor* t : {pointer(others)..., (const at::Tensor*)nullptr})
      if (t && t->defined() && (!t->is_cuda() || t->get_device() != at))
        refuse(PyExc_ValueError, "tensors lie on different devices (cuda:%d, %s)", at,
                                t->device().str().c_str());
    return at;
  }
  int index_;
  c10::cuda::CUDAGuard guard_;
  c10::cuda::OptionalCUDAStreamGuard stream_guard_;
  cudaStream_t stream_ = nullptr;
};

template <typename T = void>
T* address(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* address(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// Runs a call of the library without the interpreter's lock (a full launch
// queue blocks) and raises its error.
template <typename F>
void call(const char* name, F f) {
  PyThreadState* state = PyEval_SaveThread();
  const int status = f();
  PyEval_RestoreThread(state);
  if (status == DA_OK) return;
  PyObject* e = PyObject_CallFunction(error_class, "si", name, status);
  if (e) {
    PyErr_SetObject(error_class, e);
    Py_DECREF(e);
  }
  throw python_error();
}

void count(const char* name, Py_ssize_t have, Py_ssize_t want) {
  if (!error_class) refuse(PyExc_ValueError, "the library is not loaded");
  if (have != want) refuse(PyExc_TypeError, "%s takes %d arguments", name, (int)want);
}

// Scratch that the caller brought, or fresh scratch held by `own`.
struct Scratch {
  at::Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
  template <typename F>
  Scratch(const On& on, const at::Tensor* given, F size) {
    if (given) {
      if (!given->is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
      p = given->data_ptr();
      bytes = given->nbytes();
    } else if (const size_t n = size()) {
      own = on.scratch(n);
      p = own.data_ptr();
      bytes = n;
    }
  }
};

void put(PyObject* dict, const char* key, const at::Tensor& t) {
  PyObject* v = t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
  const int bad = !v || PyDict_SetItemString(dict, key, v);
  Py_XDECREF(v);
  if (bad) throw python_error();
}

// ---- page plan -----------------------------------------------------------------
struct Lists {
  int requests, max_pages, n_pages;
};
Lists page_lists(const char* first_name, const at::Tensor& first, const at::Tensor& lens,
                 const at::Tensor& table, const at::Tensor& pages, const at::Tensor& n_free) {
  const int64_t R = first.numel();
  need(first_name, first, at::kInt, {R});
  need("cache_lens", lens, at::kInt, {R});
  need("block_table", table, at::kInt);
  need("free_pages", pages, at::kInt, {pages.numel()});
  need("free_count", n_free, at::kInt, {1});
  if (table.dim() != 2 || table.size(0) != R)
    refuse(PyExc_ValueError, "block_table must be [%lld, max_pages], not %s", (long long)R,
                            shape_text(table.sizes()).c_str());
  return {as_int("the number of requests", R), as_int("max_pages", table.size(1)),
          as_int("the number of pages", pages.numel())};
}

// Elements [from, from + n) of a flat tensor that needs no gradient, without the
// dispatcher's view bookkeeping (six views cost 4 us through it).
at::Tensor piece(const at::Tensor& flat, int64_t from, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(
      c10::TensorImpl::VIEW, c10::Storage(flat.storage()), flat.key_set(), flat.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(flat.storage_offset() + from);
  t.unsafeGetTensorImpl()->set_sizes_and_strides(at::IntArrayRef{n}, at::IntArrayRef{1});
  return t;
}

// The lengths and the count outlive the step; with more slot rows than these they
// have an allocation of their own (0.4 us), so as not to keep the slot map alive.
constexpr int64_t kShareRows = 4096;

constexpr const char* kPlanNames[6] = {"slots",  "positions",  "offsets",
                                       "served", "cache_lens", "free_count"};

// (new_lens, cache_lens, block_table, free_pages, free_count, page_size, n_slots, out, workspace,
//  dev_status, stream)
PyObject* page_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count("page_plan", n, 11);
  const at::Tensor &new_lens = tensor(a[0], "new_lens"), &lens = tensor(a[1], "cache_lens"),
                   &table = tensor(a[2], "block_table"), &pages = tensor(a[3], "free_pages"),
                   &n_free = tensor(a[4], "free_count");
  const Lists s = page_lists("new_lens", new_lens, lens, table, pages, n_free);
  const int page_size = small(a[5], "page_size"), n_slots = small(a[6], "n_slots");
  if (n_slots < 0) refuse(PyExc_ValueError, "n_slots is negative");
  const at::Tensor *ws = optional(a[8], "workspace"), *status = status_word(a[9]);
  const int64_t R = s.requests;
  const int64_t sizes[6] = {n_slots, n_slots, R + 1, R, R, 1};
  at::Tensor out[6];
  const bool fresh = a[7] == Py_None;
  if (!fresh) {
    for (int i = 0; i < 6; ++i) {
      PyObject* key = PyUnicode_FromString(kPlanNames[i]);
      PyObject* v = key ? PyObject_GetItem(a[7], key) : nullptr;
      Py_XDECREF(key);
      if (!v) throw python_error();
      const bool is_tensor = THPVariable_Check(v);
      if (is_tensor) out[i] = THPVariable_Unpack(v);
      Py_DECREF(v);
      if (!is_tensor) refuse(PyExc_TypeError, "%s must be a tensor", kPlanNames[i]);
      need(kPlanNames[i], out[i], at::kInt, {sizes[i]});
    }
  }
  On on(a[10], new_lens, lens, table, pages, n_free, ws, status, out[0], out[1], out[2], out[3],
        out[4], out[5]);
  // New outputs, and the scratch if none was brought, are pieces of one allocation
  // (or two).
  void* scratch = ws ? ws->data_ptr() : nullptr;
  size_t scratch_bytes = ws ? ws->nbytes() : 0;
  if (ws && !ws->is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
  at::Tensor own;
  const size_t scratch_need = ws ? 0 : lib.diffattn_page_plan_workspace_size(s.requests, n_slots);
  if (fresh) {
    const int64_t pieces = 2 * (int64_t)n_slots + 3 * R + 2;
    own = at::empty({pieces + (int64_t)(scratch_need + 3) / 4}, new_lens.options());
    const bool apart = n_slots > kShareRows;
    at::Tensor kept;
    if (apart) kept = at::empty({R + 1}, new_lens.options());
    int64_t from = 0;
    for (int i = 0; i < 6; ++i) {
      if (i == 4 && apart) from = 0;
      out[i] = piece(i >= 4 && apart ? kept : own, from, sizes[i]);
      from += sizes[i];
    }
    scratch = scratch_need ? address<int>(own) + pieces : scratch;
  } else if (scratch_need) {
    own = on.scratch(scratch_need);
    scratch = own.data_ptr();
  }
  if (scratch_need) scratch_bytes = scratch_need;
  call("diffattn_page_plan", [&] {
    return lib.diffattn_page_plan(
        address<int>(new_lens), address<int>(lens), address<int>(table), address<int>(pages),
        address<int>(n_free), s.requests, s.max_pages, s.n_pages, page_size, n_slots,
        address<int>(out[0]), address<int>(out[1]), address<int>(out[2]), address<int>(out[3]),
        address<int>(out[4]), address<int>(out[5]), scratch, scratch_bytes,
        address<int>(status), on.stream());
  });
  if (!fresh) return Py_NewRef(a[7]);
  PyObject* result = PyDict_New();
  if (!result) throw python_error();
  for (int i = 0; i < 6; ++i) put(result, kPlanNames[i], out[i]);
  return result;
  END_HANDLE_TH_ERRORS
}

// (release, cache_lens, block_table, free_pages, free_count, page_size, dev_status, stream)
PyObject* page_release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count("page_release", n, 8);
  const at::Tensor &release = tensor(a[0], "release"), &lens = tensor(a[1], "cache_lens"),
                   &table = tensor(a[2], "block_table"), &pages = tensor(a[3], "free_pages"),
                   &n_free = tensor(a[4], "free_count");
  const Lists s = page_lists("release", release, lens, table, pages, n_free);
  const int page_size = small(a[5], "page_size");
  const at::Tensor* status = status_word(a[6]);
  On on(a[7], release, lens, table, pages, n_free, status);
  call("diffattn_page_release", [&] {
    return lib.diffattn_page_release(address<int>(release), address<int>(lens),
                                     address<int>(table), address<int>(pages),
                                     address<int>(n_free), s.requests, s.max_pages, s.n_pages,
                                     page_size, address<int>(status), on.stream());
  });
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// ---- 4-bit cache -----------------------------------------------------------------
struct Cache {
  int pages, heads, page_size;
};
Cache kv4_cache(const at::Tensor& cache) {
  need("cache", cache, at::kByte);
  if (cache.dim() != 3 || cache.size(2) % 144)
    refuse(PyExc_ValueError, "cache must be [n_pages, n_kv_heads, page_size * 144], not %s",
                            shape_text(cache.sizes()).c_str());
  return {as_int("the number of pages", cache.size(0)), as_int("the number of heads", cache.size(1)),
          as_int("the page size", cache.size(2) / 144)};
}

// (k, v, slots, cache, dev_status, stream)
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count("kv4_append", n, 6);
  const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &slots = tensor(a[2], "slots"),
                   &cache = tensor(a[3], "cache");
  if (v.sizes() != k.sizes()) refuse(PyExc_ValueError, "k and v differ in shape");
  const da_dtype dtype = code("k", k);
  const int64_t ks = token_stride("k", k), vs = token_stride("v", v, k.size(0), k.scalar_type());
  need("slots", slots, at::kInt, {k.size(0)});
  const Cache c = kv4_cache(cache);
  if (c.heads != k.size(1))
    refuse(PyExc_ValueError, "cache holds %d heads, k %lld", c.heads, (long long)k.size(1));
  const at::Tensor* status = status_word(a[4]);
  On on(a[5], k, v, slots, cache, status);
  const int tokens = as_int("the number of tokens", k.size(0)),
            width = as_int("the width", k.size(2));
  call("diffattn_kv4_append", [&] {
    return lib.diffattn_kv4_append(address(k), ks, address(v), vs, dtype, address<int>(slots),
                                   tokens, c.heads, width, address(cache), c.pages, c.page_size,
                                   address<int>(status), on.stream());
  });
  return Py_NewRef(a[3]);
  END_HANDLE_TH_ERRORS
}

// (cache, slots, k, v, dtype code, dev_status, stream); k and v None: new tensors of zeros
PyObject* kv4_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count("kv4_read", n, 7);
  const at::Tensor &cache = tensor(a[0], "cache"), &slots = tensor(a[1], "slots");
  const Cache c = kv4_cache(cache);
  need("slots", slots, at::kInt, {slots.numel()});
  const int64_t T = slots.numel();
  const at::Tensor* status = status_word(a[5]);
  const bool fresh = a[2] == Py_None;
  at::Tensor k, v;
  if (!fresh) {
    k = tensor(a[2], "k");
    v = tensor(a[3], "v");
    code("k", k);
    need("k", k, k.scalar_type(), {T, c.heads, 128});
    need("v", v, k.scalar_type(), {T, c.heads, 128});
  }
  On on(a[6], cache, slots, k, v, status);
  if (fresh) {
    const auto options =
        cache.options().dtype(small(a[4], "dtype") == DA_BF16 ? at::kBFloat16 : at::kFloat);
    k = at::zeros({T, c.heads, 128}, options);
    v = at::zeros({T, c.heads, 128}, options);
  }
  const int tokens = as_int("the number of tokens", T);
  const da_dtype dtype = code("k", k);
  call("diffattn_kv4_read", [&] {
    return lib.diffattn_kv4_read(address(cache), c.pages, c.page_size, address<int>(slots), tokens,
                                 c.heads, 128, address(k), address(v), dtype,
                                 address<int>(status), on.stream());
  });
  PyObject *pk = fresh ? THPVariable_Wrap(k) : Py_NewRef(a[2]),
           *pv = fresh ? THPVariable_Wrap(v) : Py_NewRef(a[3]);
  if (!pk || !pv) throw python_error();
  PyObject* r = PyTuple_New(2);
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, pk);
  PyTuple_SET_ITEM(r, 1, pv);
  return r;
  END_HANDLE_TH_ERRORS
}

// ---- decode -------------------------------------------------------------------------
// (form, q, cache, block_table, cache_lens, lam, window, apply_norm, norm_weight, norm_eps,
//  lambda_init, workspace, out, dev_status, stream)
PyObject* decode_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count("decode_kv4", n, 15);
  const bool v1 = small(a[0], "form") == 1;
  const at::Tensor &q = tensor(a[1], "q"), &cache = tensor(a[2], "cache"),
                   &table = tensor(a[3], "block_table"), &lens = tensor(a[4], "cache_lens"),
                   &lam = tensor(a[5], "lam");
  const da_dtype dtype = code("q", q);
  need("q", q, q.scalar_type());
  if (q.dim() != 3)
    refuse(PyExc_ValueError, "q must be [batch, heads, width], not %s",
                            shape_text(q.sizes()).c_str());
  const int64_t B = q.size(0), H = q.size(1), d = q.size(2);
  const Cache c = kv4_cache(cache);
  if (v1 && c.heads != H)
    refuse(PyExc_ValueError, "cache holds %d heads, q %lld", c.heads, (long long)H);
  if (v1 && d % 2)  // a head's width is passed as that of its two branches
    refuse(PyExc_ValueError, "q's width must be that of two branches, not %lld", (long long)d);
  need("block_table", table, at::kInt);
  if (table.dim() != 2 || table.size(0) != B)
    refuse(PyExc_ValueError, "block_table must be [%lld, max_pages], not %s", (long long)B,
                            shape_text(table.sizes()).c_str());
  need("cache_lens", lens, at::kInt, {B});
  const int64_t heads = v1 ? H : H / 2;
  need("lam", lam, at::kFloat, {heads});
  const int window = small(a[6], "window");
  const at::Tensor *gain = optional(a[8], "norm_weight"), *ws = optional(a[11], "workspace"),
                   *given = optional(a[12], "out"), *status = status_word(a[13]);
  if (gain) need("norm_weight", *gain, at::kFloat, {128});
  const int64_t width = v1 ? 128 : d;
  if (given) need("out", *given, q.scalar_type(), {B, heads, width});
  const int batch = as_int("the batch", B), qh = as_int("the number of heads", H),
            max_pages = as_int("max_pages", table.size(1)), dim = as_int("the width", d);
  On on(a[14], q, cache, table, lens, lam, gain, ws, given, status);
  const at::Tensor out = given ? *given : at::empty({B, heads, width}, q.options());
  if (v1) {
    Scratch s(on, ws, [&] { return lib.diffattn_v1_decode_kv4_workspace_size(batch, qh); });
    const bool norm = truth(a[7]);
    const float eps = real(a[9]), lambda_init = real(a[10]);
    call("diffattn_v1_decode_kv4", [&] {
      return lib.diffattn_v1_decode_kv4(
          address(q), address(cache), c.pages, c.page_size, address<int>(table), max_pages,
          address<int>(lens), window, address(out), dtype, batch, qh, dim / 2, 128,
          address<float>(lam), norm, address<float>(gain), eps, lambda_init, s.p, s.bytes,
          address<int>(status), on.stream());
    });
  } else {
    Scratch s(on, ws, [&] {
      return lib.diffattn_v2_decode_kv4_workspace_size(batch, qh, c.heads);
    });
    call("diffattn_v2_decode_kv4", [&] {
      return lib.diffattn_v2_decode_kv4(address(q), address(cache), c.pages, c.page_size,
                                        address<int>(table), max_pages, address<int>(lens), window,
                                        address(out), dtype, batch, qh, c.heads, dim,
                                        address<float>(lam), s.p, s.bytes, address<int>(status),
                                        on.stream());
    });
  }
  if (given) return Py_NewRef(a[12]);
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// ---- QK norm and rotation --------------------------------------------------------------
struct Heads {
  da_dtype dtype;
  int64_t T, Hq, Hk, d, qs, ks;
  int rot, tokens, n_q, n_k, dim;
};
Heads norm_heads(const at::Tensor& q, const at::Tensor* k, const at::Tensor* pos,
                 const at::Tensor* freq, const at::Tensor* wq, const at::Tensor* wk) {
  Heads h{};
  h.dtype = code("q", q);
  h.qs = token_stride("q", q);
  h.T = q.size(0), h.Hq = q.size(1), h.d = q.size(2);
  if (k) {
    h.ks = token_stride("k", *k, h.T, q.scalar_type());
    h.Hk = k->size(1);
    if (k->size(2) != h.d) refuse(PyExc_ValueError, "q and k differ in width");
  }
  if (wq) need("q_weight", *wq, at::kFloat, {h.d});
  if (wk) need("k_weight", *wk, at::kFloat, {h.d});
  if (freq) {
    need("inv_freq", *freq, at::kFloat, {freq->numel()});
    h.rot = as_int("inv_freq", 2 * freq->numel());
  }
  if (pos) need("positions", *pos, at::kInt, {h.T});
  h.tokens = as_int("the number of tokens", h.T);
  h.n_q = as_int("the number of heads", h.Hq);
  h.n_k = as_int("the number of heads", h.Hk);
  h.dim = as_int("the width", h.d);
  return h;
}

// (q, k, positions, inv_freq, q_weight, k_weight, norm_eps, interleaved, q_out, k_out, stream)
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count("qk_norm_rope", n, 11);
  const at::Tensor& q = tensor(a[0], "q");
  const at::Tensor *k = optional(a[1], "k"), *pos = optional(a[2], "positions"),
                   *freq = optional(a[3], "inv_freq"), *wq = optional(a[4], "q_weight"),
                   *wk = optional(a[5], "k_weight");
  const Heads h = norm_heads(q, k, pos, freq, wq, wk);
  const bool fresh = a[8] == Py_None;
  at::Tensor qo, ko;
  if (!fresh) {
    qo = tensor(a[8], "q out");
    if (k) ko = tensor(a[9], "k out");
    if (qo.sizes() != q.sizes() || (k && ko.sizes() != k->sizes()))
      refuse(PyExc_ValueError, "outputs must have the inputs' shapes");
  }
  On on(a[10], q, k, pos, freq, wq, wk, qo, ko);
  if (fresh) {
    qo = at::empty({h.T, h.Hq, h.d}, q.options());
    if (k) ko = at::empty({h.T, h.Hk, h.d}, q.options());
  }
  const int64_t qos = token_stride("q out", qo, h.T, q.scalar_type());
  const int64_t kos = k ? token_stride("k out", ko, h.T, q.scalar_type()) : 0;
  const float eps = real(a[6]);
  const bool interleaved = truth(a[7]);
  call("diffattn_qk_norm_rope", [&] {
    return lib.diffattn_qk_norm_rope(address(q), h.qs, address(k), h.ks, h.dtype, h.tokens, h.n_q,
                                     h.n_k, h.dim, address<float>(wq), address<float>(wk), eps,
                                     address<int>(pos), address<float>(freq), h.rot, interleaved,
                                     address(qo), qos, k ? address(ko) : nullptr, kos,
                                     on.stream());
  });
  PyObject *pq = fresh ? THPVariable_Wrap(qo) : Py_NewRef(a[8]),
           *pk = !fresh ? Py_NewRef(a[9]) : k ? THPVariable_Wrap(ko) : Py_NewRef(Py_None);
  PyObject* r = pq && pk ? PyTuple_New(2) : nullptr;
  if (!r) throw python_error();
  PyTuple_SET_ITEM(r, 0, pq);
  PyTuple_SET_ITEM(r, 1, pk);
  return r;
  END_HANDLE_TH_ERRORS
}

// (q, k, dq_out, dk_out, positions, inv_freq, q_weight, k_weight, norm_eps, interleaved,
//  workspace, stream)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  count("qk_norm_rope_bwd", n, 12);
  const at::Tensor &q = tensor(a[0], "q"), &gq = tensor(a[2], "dq_out");
  const at::Tensor *k = optional(a[1], "k"), *gk = optional(a[3], "dk_out"),
                   *pos = optional(a[4], "positions"), *freq = optional(a[5], "inv_freq"),
                   *wq = optional(a[6], "q_weight"), *wk = optional(a[7], "k_weight"),
                   *ws = optional(a[10], "workspace");
  const Heads h = norm_heads(q, k, pos, freq, wq, wk);
  if (gq.sizes() != q.sizes() || (k && (!gk || gk->sizes() != k->sizes())))
    refuse(PyExc_ValueError, "the gradients must have the inputs' shapes");
  const int64_t gqs = token_stride("dq_out", gq, h.T, at::kFloat);
  const int64_t gks = k ? token_stride("dk_out", *gk, h.T, at::kFloat) : 0;
  On on(a[11], q, k, gq, gk, pos, freq, wq, wk, ws);
  const auto options = gq.options();
  const at::Tensor dq = at::empty({h.T, h.Hq, h.d}, options);
  at::Tensor dk, dwq, dwk;
  if (k) dk = at::empty({h.T, h.Hk, h.d}, options);
  if (wq) dwq = at::empty({h.d}, options);
  if (k && wk) dwk = at::empty({h.d}, options);
  Scratch s(on, ws, [&] {
    return lib.diffattn_qk_norm_rope_bwd_workspace_size(h.tokens, h.n_q, h.n_k, h.dim);
  });
  const float eps = real(a[8]);
  const bool interleaved = truth(a[9]);
  call("diffattn_qk_norm_rope_bwd", [&] {
    return lib.diffattn_qk_norm_rope_bwd(
        address(q), h.qs, address(k), h.ks, h.dtype, address<float>(gq), gqs,
        k ? address<float>(gk) : nullptr, gks, h.tokens, h.n_q, h.n_k, h.dim, address<float>(wq),
        address<float>(wk), eps, address<int>(pos), address<float>(freq), h.rot, interleaved,
        address<float>(dq), k ? address<float>(dk) : nullptr,
        dwq.defined() ? address<float>(dwq) : nullptr,
        dwk.defined() ? address<float>(dwk) : nullptr, s.p, s.bytes, on.stream());
  });
  PyObject* r = PyDict_New();
  if (!r) throw python_error();
  put(r, "dq", dq);
  put(r, "dk", dk);
  put(r, "dq_weight", dwq);
  put(r, "dk_weight", dwk);
  return r;
  END_HANDLE_TH_ERRORS
}

// (handle of the loaded library, exception class of a failed call)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2) refuse(PyExc_TypeError, "bind takes 2 arguments");
  void* handle = PyLong_AsVoidPtr(a[0]);
  if (!handle && PyErr_Occurred()) throw python_error();
  Library found;
#define X(name)                                                              \
  found.name = reinterpret_cast<decltype(&::name)>(dlsym(handle, #name)); \
  if (!found.name) refuse(PyExc_ValueError, "the library lacks %s", #name);
  DA_CALLS(X)
#undef X
  lib = found;
  Py_XSETREF(error_class, Py_NewRef(a[1]));
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

#define DA_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&name)), METH_FASTCALL, nullptr }
PyMethodDef methods[] = {DA_METHOD(bind),       DA_METHOD(page_plan),
                         DA_METHOD(page_release), DA_METHOD(kv4_append),
                         DA_METHOD(kv4_read),   DA_METHOD(decode_kv4),
                         DA_METHOD(qk_norm_rope), DA_METHOD(qk_norm_rope_bwd),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT,
                      "_marshal",
                      "Argument marshalling of the serving operators (see binding.py).",
                      -1,
                      methods,
                      nullptr,
                      nullptr,
                      nullptr,
                      nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", DA_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
