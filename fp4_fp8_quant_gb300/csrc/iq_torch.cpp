// Marshalling of PyTorch tensors for the calls whose work on the GPU is as short
// as Python's part of them: checks of types, shapes, strides and devices in one
// place, allocation of the results, and the C entry (include/iq.h), whose address
// the Python binding hands over.  Nothing is computed here.  Python's lock is given
// up while memory is allocated and kernels are launched: either may wait for the
// GPU, and for a host callback that needs the lock.
//
// Every function ends with a raw stream or None (PyTorch's current one) and
// returns its result, or None where a tensor is not what the call takes (the
// Python binding then says which and why), or the status code of the C entry as an
// int.

#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/TensorImpl.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <limits>
#include <optional>

namespace {

using Stream = void*;

// The C entries, as include/iq.h declares them.
int (*quant_rows_entry)(const void*, int, const int32_t*, int, int, int, void*, int, int32_t*, Stream);
int (*route_entry)(const void*, int, long long, int, int, int, int, int, float, float*, int32_t*, int32_t*, int32_t*, int32_t*,
                   void*, size_t, Stream);
size_t (*route_workspace)(int, int);
int (*grouped_entry)(const void*, long long, const int32_t*, int, int, const void*, const uint8_t*, int, int, const int32_t*, int,
                     void*, long long, void*, size_t, Stream);
size_t (*grouped_workspace)(int, int);
int (*combine_entry)(const void*, long long, int, const int32_t*, const float*, int, int, int, const void*, long long, void*,
                     long long, Stream);
int (*adapters_entry)(const void*, long long, int, int, const void*, const void*, const float*, int, int, int, const int32_t*,
                      const int32_t*, int, const void*, long long, void*, long long, void*, size_t, Stream);
size_t (*adapters_workspace)(int, int);

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool codes(const at::Tensor& t) { return t.scalar_type() == at::kByte || t.scalar_type() == at::kFloat8_e4m3fn; }

bool fits(int64_t v) { return v <= std::numeric_limits<int>::max(); }

// A 2-D tensor on `device` whose rows are contiguous.
bool matrix(const at::Tensor& t, at::Device device) {
  return t.dim() == 2 && t.device() == device && (t.stride(1) == 1 || t.size(1) <= 1) && fits(t.size(0)) && fits(t.size(1));
}

long long row_stride(const at::Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1); }

// A contiguous tensor of a type and shape on `device`.
bool whole(const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape, at::Device device) {
  return t.scalar_type() == type && t.sizes() == at::IntArrayRef(shape) && t.device() == device && t.is_contiguous();
}

bool bf16_matrix(const at::Tensor& t, int64_t rows, int64_t cols, at::Device device) {
  return t.scalar_type() == at::kBFloat16 && matrix(t, device) && t.size(0) == rows && t.size(1) == cols;
}

at::Tensor make(std::initializer_list<int64_t> shape, at::ScalarType type, at::Device device) {
  return at::detail::empty_cuda(at::IntArrayRef(shape), type, device, std::nullopt);
}

// Several results in one allocation, 256 bytes apart or more: the caching allocator's
// part of a call is some 0.8 us per tensor (routing, five results: 8.9 -> 5.8 us of host
// time; memory asked for past the dispatcher, in make(): 5.0).  One of them keeps all
// of it alive and is saved with all of it, so larger results get memory of their own:
// past kShared, where the kernels' time hides the allocator's.
constexpr int64_t kShared = 1 << 20;
struct Part {
  std::initializer_list<int64_t> shape;
  at::ScalarType type;
};
template <size_t kParts>
void make_parts(const Part (&parts)[kParts], at::Device device, at::Tensor (&out)[kParts]) {
  int64_t at[kParts], total = 0;
  for (size_t i = 0; i < kParts; ++i) {
    int64_t size = static_cast<int64_t>(c10::elementSize(parts[i].type));
    for (int64_t n : parts[i].shape) size *= n;
    at[i] = total;
    total += (size + 255) / 256 * 256;
  }
  if (total > kShared) {
    for (size_t i = 0; i < kParts; ++i) out[i] = make(parts[i].shape, parts[i].type, device);
    return;
  }
  const at::Tensor all = make({total}, at::kByte, device);
  for (size_t i = 0; i < kParts; ++i) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), c10::scalarTypeToTypeMeta(parts[i].type));
    impl->set_storage_offset(at[i] / static_cast<int64_t>(c10::elementSize(parts[i].type)));
    impl->set_sizes_contiguous(at::IntArrayRef(parts[i].shape));
    out[i] = at::Tensor(std::move(impl));
  }
}

// The given workspace, if any; false for something else.
bool workspace_of(PyObject* given, at::Device device, at::Tensor& ws) {
  if (given == Py_None) return true;
  const at::Tensor* t = tensor(given);
  if (t == nullptr || t->scalar_type() != at::kByte || t->device() != device || !t->is_contiguous()) return false;
  ws = *t;
  return true;
}

// One of `need` bytes, where none was given.
void make_workspace(PyObject* given, size_t need, at::Device device, at::Tensor& ws) {
  if (given == Py_None && need > 0) ws = make({static_cast<int64_t>(need)}, at::kByte, device);
}

void* data(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes(const at::Tensor& t) { return t.defined() ? static_cast<size_t>(t.numel()) : 0; }

// Whether a tensor is on the current GPU, where the kernels run.
bool here(const at::Tensor& t) { return t.is_cuda() && t.device().index() == c10::cuda::current_device(); }

// The given raw stream, or PyTorch's current one for None.
Stream stream_of(PyObject* o) {
  return o == Py_None ? c10::cuda::getCurrentCUDAStream().stream() : reinterpret_cast<Stream>(PyLong_AsUnsignedLongLong(o));
}

// Without Python's lock as long as it lives.  Nothing of Python is touched meanwhile:
// the arguments' tensors belong to the caller.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

PyObject* status(int code) { return PyLong_FromLong(code); }

// Calls f and turns C++ exceptions into the Python ones that PyTorch's own calls raise
// (torch.OutOfMemoryError for an allocation that failed).
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const std::exception&) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

// x, rows, y | None, scales | None, stream -> (y, scales)
PyObject* quant_rows(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x = tensor(a[0]), *rows = tensor(a[1]);
    if (x == nullptr || rows == nullptr || !here(*x) || x->scalar_type() != at::kBFloat16) Py_RETURN_NONE;
    const at::Device device = x->device();
    if (!matrix(*x, device) || rows->dim() != 1 || !fits(rows->size(0))) Py_RETURN_NONE;
    const int64_t M = rows->size(0), K = x->size(1), groups = std::max<int64_t>(1, (K + 511) / 512), wide = (M + 3) / 4 * 4;
    if (!whole(*rows, at::kInt, {M}, device)) Py_RETURN_NONE;
    at::Tensor y, scales;
    if (a[2] != Py_None) {
      const at::Tensor* t = tensor(a[2]);
      if (t == nullptr || !codes(*t) || !matrix(*t, device) || t->size(0) != M || t->size(1) != K) Py_RETURN_NONE;
      y = *t;
    }
    if (a[3] != Py_None) {
      const at::Tensor* t = tensor(a[3]);
      if (t == nullptr || !whole(*t, at::kInt, {groups, wide}, device)) Py_RETURN_NONE;
      scales = *t;
    }
    const int64_t ldx = row_stride(*x), ldy = y.defined() ? row_stride(y) : K;
    if (!fits(ldx) || !fits(ldy)) Py_RETURN_NONE;
    const Stream stream = stream_of(a[4]);
    int code;
    {
      Unlocked unlocked;
      if (!y.defined() && !scales.defined()) {
        at::Tensor made[2];
        make_parts({{{M, K}, at::kByte}, {{groups, wide}, at::kInt}}, device, made);
        y = std::move(made[0]);
        scales = std::move(made[1]);
      } else if (!y.defined()) {
        y = make({M, K}, at::kByte, device);
      } else if (!scales.defined()) {
        scales = make({groups, wide}, at::kInt, device);
      }
      code = quant_rows_entry(data(*x), static_cast<int>(x->size(0)), static_cast<const int32_t*>(data(*rows)),
                              static_cast<int>(M), static_cast<int>(K), static_cast<int>(ldx), data(y),
                              static_cast<int>(ldy), static_cast<int32_t*>(data(scales)), stream);
    }
    if (code != 0) return status(code);
    return Py_BuildValue("NN", THPVariable_Wrap(y), THPVariable_Wrap(scales));
  });
}

// logits, k, score, normalize, scale, workspace | None, stream
//   -> (weights, experts, slots, rows, row_start)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* l = tensor(a[0]);
    const long k = PyLong_AsLong(a[1]), score = PyLong_AsLong(a[2]);
    const int normalize = PyObject_IsTrue(a[3]);
    const double scale = PyFloat_AsDouble(a[4]);
    if (PyErr_Occurred()) return nullptr;
    if (l == nullptr || !here(*l) || (l->scalar_type() != at::kFloat && l->scalar_type() != at::kBFloat16)) Py_RETURN_NONE;
    const at::Device device = l->device();
    if (!matrix(*l, device)) Py_RETURN_NONE;
    const int64_t T = l->size(0), E = l->size(1);
    if (k < 1 || k > E || k > 32 || !fits(T * k)) Py_RETURN_NONE;
    at::Tensor ws;
    if (!workspace_of(a[5], device, ws)) Py_RETURN_NONE;
    const Stream stream = stream_of(a[6]);
    at::Tensor made[5];
    const at::Tensor &w = made[0], &experts = made[1], &slots = made[2], &rows = made[3], &start = made[4];
    int code;
    {
      Unlocked unlocked;
      make_workspace(a[5], route_workspace(static_cast<int>(T), static_cast<int>(E)), device, ws);
      make_parts({{{T, k}, at::kFloat}, {{T, k}, at::kInt}, {{T, k}, at::kInt}, {{T * k}, at::kInt}, {{E + 1}, at::kInt}}, device, made);
      code = route_entry(data(*l), l->scalar_type() == at::kBFloat16, row_stride(*l), static_cast<int>(T),
                         static_cast<int>(E), static_cast<int>(k), static_cast<int>(score), normalize,
                         static_cast<float>(scale), static_cast<float*>(data(w)), static_cast<int32_t*>(data(experts)),
                         static_cast<int32_t*>(data(slots)), static_cast<int32_t*>(data(rows)),
                         static_cast<int32_t*>(data(start)), data(ws), bytes(ws), stream);
    }
    if (code != 0) return status(code);
    return Py_BuildValue("NNNNN", THPVariable_Wrap(w), THPVariable_Wrap(experts), THPVariable_Wrap(slots),
                         THPVariable_Wrap(rows), THPVariable_Wrap(start));
  });
}

// The given output rows, if any; false for something else.
bool output_of(PyObject* given, int64_t rows, int64_t cols, at::Device device, at::Tensor& out) {
  if (given == Py_None) return true;
  const at::Tensor* t = tensor(given);
  if (t == nullptr || !bf16_matrix(*t, rows, cols, device)) return false;
  out = *t;
  return true;
}

// x, x_scales, w, w_sf, row_start, gated, out | None, workspace | None, stream -> out
PyObject* grouped_gemm(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x = tensor(a[0]), *xs = tensor(a[1]), *w = tensor(a[2]), *ws_f = tensor(a[3]), *start = tensor(a[4]);
    if (!x || !xs || !w || !ws_f || !start || !here(*x) || !codes(*x) || !codes(*w) || w->dim() != 3) Py_RETURN_NONE;
    const at::Device device = x->device();
    if (!matrix(*x, device)) Py_RETURN_NONE;
    const int gated = PyObject_IsTrue(a[5]);
    if (gated < 0) return nullptr;
    const int64_t M = x->size(0), K = x->size(1), G = w->size(0), N = w->size(1);
    if (w->size(2) != K || w->device() != device || !w->is_contiguous() || !fits(G) || !fits(N) ||
        !whole(*xs, at::kInt, {(K + 511) / 512, (M + 3) / 4 * 4}, device) ||
        !whole(*ws_f, at::kByte, {G, (N + 127) / 128, K / 128}, device) || !whole(*start, at::kInt, {G + 1}, device)) {
      Py_RETURN_NONE;
    }
    at::Tensor out, ws;
    const int64_t n_out = gated ? N / 2 : N;
    if (!output_of(a[6], M, n_out, device, out) || !workspace_of(a[7], device, ws)) Py_RETURN_NONE;
    const Stream stream = stream_of(a[8]);
    int code;
    {
      Unlocked unlocked;
      if (!out.defined()) out = make({M, n_out}, at::kBFloat16, device);
      make_workspace(a[7], grouped_workspace(static_cast<int>(M), static_cast<int>(K)), device, ws);
      code = grouped_entry(data(*x), row_stride(*x), static_cast<const int32_t*>(data(*xs)), static_cast<int>(M),
                           static_cast<int>(K), data(*w), static_cast<const uint8_t*>(data(*ws_f)), static_cast<int>(G),
                           static_cast<int>(N), static_cast<const int32_t*>(data(*start)), gated, data(out),
                           row_stride(out), data(ws), bytes(ws), stream);
    }
    return code != 0 ? status(code) : THPVariable_Wrap(out);
  });
}

// y, slots, weights, add | None, out | None, stream -> out
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *y = tensor(a[0]), *slots = tensor(a[1]), *w = tensor(a[2]), *add = tensor(a[3]);
    if (!y || !slots || !w || (!add && a[3] != Py_None) || !here(*y) || y->scalar_type() != at::kBFloat16 || slots->dim() != 2) {
      Py_RETURN_NONE;
    }
    const at::Device device = y->device();
    if (!matrix(*y, device)) Py_RETURN_NONE;
    const int64_t S = y->size(0), N = y->size(1), T = slots->size(0), k = slots->size(1);
    if (!fits(T) || !fits(k) || !whole(*slots, at::kInt, {T, k}, device) || !whole(*w, at::kFloat, {T, k}, device) ||
        (add && !bf16_matrix(*add, T, N, device))) {
      Py_RETURN_NONE;
    }
    at::Tensor out;
    if (!output_of(a[4], T, N, device, out)) Py_RETURN_NONE;
    const Stream stream = stream_of(a[5]);
    int code;
    {
      Unlocked unlocked;
      if (!out.defined()) out = make({T, N}, at::kBFloat16, device);
      code = combine_entry(data(*y), row_stride(*y), static_cast<int>(S), static_cast<const int32_t*>(data(*slots)),
                           static_cast<const float*>(data(*w)), static_cast<int>(T), static_cast<int>(k),
                           static_cast<int>(N), add ? data(*add) : nullptr, add ? row_stride(*add) : 0, data(out),
                           row_stride(out), stream);
    }
    return code != 0 ? status(code) : THPVariable_Wrap(out);
  });
}

// x, base | None, a, b, scale, row_start, adapter, out | None, workspace | None, stream -> out
PyObject* adapters(PyObject*, PyObject* const* p, Py_ssize_t) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x = tensor(p[0]), *base = tensor(p[1]), *a = tensor(p[2]), *b = tensor(p[3]), *scale = tensor(p[4]),
                     *start = tensor(p[5]), *used = tensor(p[6]);
    if (!x || (!base && p[1] != Py_None) || !a || !b || !scale || !start || !used || !here(*x) ||
        x->scalar_type() != at::kBFloat16 || a->dim() != 3 || b->dim() != 3 || used->dim() != 1) {
      Py_RETURN_NONE;
    }
    const at::Device device = x->device();
    if (!matrix(*x, device)) Py_RETURN_NONE;
    const int64_t T = x->size(0), K = x->size(1), A = a->size(0), r = a->size(1), N = b->size(1), R = used->size(0);
    if (!fits(A) || !fits(r) || !fits(N) || !fits(R) || !whole(*a, at::kBFloat16, {A, r, K}, device) ||
        !whole(*b, at::kBFloat16, {A, N, r}, device) || !whole(*scale, at::kFloat, {A}, device) ||
        !whole(*start, at::kInt, {R + 1}, device) || !whole(*used, at::kInt, {R}, device) ||
        (base && !bf16_matrix(*base, T, N, device))) {
      Py_RETURN_NONE;
    }
    at::Tensor out, ws;
    if (!output_of(p[7], T, N, device, out) || !workspace_of(p[8], device, ws)) Py_RETURN_NONE;
    const Stream stream = stream_of(p[9]);
    int code;
    {
      Unlocked unlocked;
      if (!out.defined()) out = make({T, N}, at::kBFloat16, device);
      make_workspace(p[8], adapters_workspace(static_cast<int>(T), static_cast<int>(r)), device, ws);
      code = adapters_entry(data(*x), row_stride(*x), static_cast<int>(T), static_cast<int>(K), data(*a), data(*b),
                            static_cast<const float*>(data(*scale)), static_cast<int>(A), static_cast<int>(r),
                            static_cast<int>(N), static_cast<const int32_t*>(data(*start)),
                            static_cast<const int32_t*>(data(*used)), static_cast<int>(R), base ? data(*base) : nullptr,
                            base ? row_stride(*base) : 0, data(out), row_stride(out), data(ws), bytes(ws), stream);
    }
    return code != 0 ? status(code) : THPVariable_Wrap(out);
  });
}

// Takes the addresses of the C entries, in this order.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* p[8];
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "eight addresses");
    return nullptr;
  }
  for (int i = 0; i < 8; ++i) p[i] = PyLong_AsVoidPtr(a[i]);
  if (PyErr_Occurred()) return nullptr;
  quant_rows_entry = reinterpret_cast<decltype(quant_rows_entry)>(p[0]);
  route_entry = reinterpret_cast<decltype(route_entry)>(p[1]);
  route_workspace = reinterpret_cast<decltype(route_workspace)>(p[2]);
  grouped_entry = reinterpret_cast<decltype(grouped_entry)>(p[3]);
  grouped_workspace = reinterpret_cast<decltype(grouped_workspace)>(p[4]);
  combine_entry = reinterpret_cast<decltype(combine_entry)>(p[5]);
  adapters_entry = reinterpret_cast<decltype(adapters_entry)>(p[6]);
  adapters_workspace = reinterpret_cast<decltype(adapters_workspace)>(p[7]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {{"bind", fast(bind), METH_FASTCALL, nullptr},
                         {"quant_rows", fast(quant_rows), METH_FASTCALL, nullptr},
                         {"route", fast(route), METH_FASTCALL, nullptr},
                         {"grouped_gemm", fast(grouped_gemm), METH_FASTCALL, nullptr},
                         {"combine", fast(combine), METH_FASTCALL, nullptr},
                         {"adapters", fast(adapters), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_iq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__iq_torch() { return PyModule_Create(&module); }
