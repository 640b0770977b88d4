// Python module _tensors: checks torch tensors and hands their pointers, sizes and strides to the C ABI.
//
// For the operators of a decode step, whose kernels take 2 to 6 us: the same
// checks in Python and a ctypes call took 7 to 10 us per call, this takes 2.1 to 2.3. The module
// calls nothing of PyTorch but the tensors' accessors, the current stream and the current device; all arithmetic is the library's.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>

#include "../../include/tl.h"

namespace {

struct Refused {};      // a Python exception is set

// What PagedKVCache hands over the address of: its description, and the number of the GPU that it lies on.
struct Cache : tl_kv_cache {
  int device;
};

[[noreturn]] void refuse(const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(PyExc_ValueError, format, args);
  va_end(args);
  throw Refused{};
}

// A CUDA tensor, or nothing for None where `optional`.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse("%s must be a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse("%s must be a CUDA tensor", name);
  return &t;
}

// All of a call's tensors lie on one GPU, which is where it is launched.
void on_device(const at::Tensor* t, int device, const char* name) {
  if (t != nullptr && t->device().index() != device) refuse("%s is on GPU %d, not on GPU %d", name, static_cast<int>(t->device().index()), device);
}

// Makes it the current device meanwhile, where it is not.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(int device) {
    if (c10::cuda::current_device() != device) guard.set_index(static_cast<c10::DeviceIndex>(device));
  }
};

const char* type_name(at::ScalarType t) { return c10::toString(t); }

void want_type(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type) refuse("%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
}

int half_code(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return TL_BF16;
  if (t.scalar_type() == at::kHalf) return TL_F16;
  refuse("%s must be BFloat16 or Half, got %s", name, type_name(t.scalar_type()));
}

// [tokens, heads, dim], the heads of a token contiguous and the tokens any distance apart, which is returned
int64_t token_rows(const at::Tensor& t, int64_t heads, int64_t dim, at::ScalarType type, const char* name) {
  want_type(t, type, name);
  const auto size = t.sizes(), stride = t.strides();
  if (size.size() != 3 || size[1] != heads || size[2] != dim)
    refuse("%s must be [tokens, %lld, %lld]", name, static_cast<long long>(heads), static_cast<long long>(dim));
  if (stride[2] != 1 || (stride[1] != dim && heads > 1)) refuse("%s: the heads of a token must be contiguous", name);
  return stride[0];
}

// [rows, cols] with contiguous rows any distance apart, which is returned
int64_t matrix(const at::Tensor& t, int64_t rows, int64_t cols, const char* name) {
  const auto size = t.sizes(), stride = t.strides();
  if (size.size() != 2 || size[0] != rows || size[1] != cols || (stride[1] != 1 && cols > 1))
    refuse("%s must be [%lld, %lld] with contiguous rows", name, static_cast<long long>(rows), static_cast<long long>(cols));
  return stride[0];
}

// a contiguous vector of n
const void* vector(const at::Tensor& t, at::ScalarType type, int64_t n, const char* name) {
  want_type(t, type, name);
  if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) refuse("%s must be a contiguous vector [%lld]", name, static_cast<long long>(n));
  return t.data_ptr();
}

int fits(int64_t n, const char* name) {
  if (n > INT32_MAX) refuse("%s has too many rows", name);
  return static_cast<int>(n);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

// None: the current stream of the tensor's device; else a cudaStream_t's address
void* stream_of(PyObject* o, const at::Tensor& t) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
  return reinterpret_cast<void*>(static_cast<intptr_t>(integer(o)));
}

template <typename F>
PyObject* call(const char* name, Py_ssize_t got, Py_ssize_t want, F&& f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// kv_append(cache, k, v, positions, slots, cos_sin, interleaved, q, q_out, stream) -> tl_status
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("kv_append", n, 10, [&] {
    const auto* c = reinterpret_cast<const Cache*>(static_cast<intptr_t>(integer(a[0])));
    const at::Tensor &k = *tensor(a[1], "k"), &v = *tensor(a[2], "v"), &slots = *tensor(a[4], "slots");
    const at::Tensor *cos_sin = tensor(a[5], "cos_sin", true), *q = tensor(a[7], "q", true);
    on_device(&k, c->device, "k"), on_device(&v, c->device, "v"), on_device(&slots, c->device, "slots");
    on_device(cos_sin, c->device, "cos_sin"), on_device(q, c->device, "q");
    const at::Tensor* const at = cos_sin != nullptr ? tensor(a[3], "positions") : nullptr;
    on_device(at, c->device, "positions");
    const int code = half_code(k, "k");
    const auto type = k.scalar_type();
    const int64_t ldk = token_rows(k, c->kv_heads, c->head_dim, type, "k"), ldv = token_rows(v, c->kv_heads, c->head_dim, type, "v");
    const int64_t T = k.size(0);
    if (v.size(0) != T) refuse("k and v must have the same number of tokens");
    int64_t heads = 0, ldq = 0, ldo = 0;
    const void* pq = nullptr;
    void* po = nullptr;
    if (q != nullptr) {
      const at::Tensor& out = *tensor(a[8], "q_out");
      on_device(&out, c->device, "q_out");
      if (q->dim() != 3) refuse("q must be [tokens, heads, %d]", c->head_dim);
      heads = q->size(1);
      ldq = token_rows(*q, heads, c->head_dim, type, "q");
      ldo = token_rows(out, heads, c->head_dim, type, "q_out");
      if (q->size(0) != T || out.size(0) != T) refuse("q, q_out and k must have the same number of tokens");
      pq = q->data_ptr();
      po = out.data_ptr();
    }
    const float* table = nullptr;
    const int32_t* positions = nullptr;
    int64_t rows = 0, rot = 0;
    if (cos_sin != nullptr) {
      want_type(*cos_sin, at::kFloat, "cos_sin");
      if (cos_sin->dim() != 2 || !cos_sin->is_contiguous()) refuse("cos_sin must be a contiguous matrix [positions, channels]");
      rows = cos_sin->size(0);
      rot = cos_sin->size(1);
      table = static_cast<const float*>(cos_sin->data_ptr());
      positions = static_cast<const int32_t*>(vector(*at, at::kInt, T, "positions"));
    }
    const int interleaved = PyObject_IsTrue(a[6]);
    if (interleaved < 0) throw Refused{};
    const OnDevice guard(c->device);
    return tl_kv_append(c, pq, k.data_ptr(), v.data_ptr(), code, fits(T, "k"), fits(heads, "q"), ldq, ldk, ldv, po, ldo, table,
                        fits(rows, "cos_sin"), fits(rot, "cos_sin"), interleaved, positions,
                        static_cast<const int64_t*>(vector(slots, at::kLong, T, "slots")), stream_of(a[9], k));
  });
}

// paged_attention(cache, q, pages, lens, scale, window, out, lse, workspace, stream) -> tl_status
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("paged_attention", n, 10, [&] {
    const auto* c = reinterpret_cast<const Cache*>(static_cast<intptr_t>(integer(a[0])));
    const at::Tensor &q = *tensor(a[1], "q"), &pages = *tensor(a[2], "pages"), &lens = *tensor(a[3], "lens");
    const at::Tensor &out = *tensor(a[6], "out"), *lse = tensor(a[7], "lse", true), &ws = *tensor(a[8], "workspace");
    on_device(&q, c->device, "q"), on_device(&pages, c->device, "pages"), on_device(&lens, c->device, "lens");
    on_device(&out, c->device, "out"), on_device(lse, c->device, "lse"), on_device(&ws, c->device, "workspace");
    const int code = half_code(q, "q");
    if (q.dim() != 3) refuse("q must be [requests, heads, %d]", c->head_dim);
    const int64_t B = q.size(0), heads = q.size(1);
    const int64_t ldq = token_rows(q, heads, c->head_dim, q.scalar_type(), "q");
    const int64_t ldo = token_rows(out, heads, c->head_dim, q.scalar_type(), "out");
    if (out.size(0) != B) refuse("out and q must have the same number of requests");
    want_type(pages, at::kInt, "pages");
    if (pages.dim() != 2) refuse("pages must be a matrix [requests, max_pages]");
    const int64_t width = pages.size(1), ldp = matrix(pages, B, width, "pages");
    float* pl = nullptr;
    if (lse != nullptr) {
      want_type(*lse, at::kFloat, "lse");
      if (!lse->is_contiguous()) refuse("lse must be contiguous");
      matrix(*lse, B, heads, "lse");
      pl = static_cast<float*>(lse->data_ptr());
    }
    const double scale = PyFloat_AsDouble(a[4]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refused{};
    const int64_t window = integer(a[5]);
    const int tokens = window > INT32_MAX ? 0 : window < 0 ? -1 : static_cast<int>(window);      // wider than any length: all; negative: refused
    const OnDevice guard(c->device);
    return tl_paged_attention(c, q.data_ptr(), code, fits(B, "q"), fits(heads, "q"), ldq, static_cast<const int32_t*>(pages.data_ptr()),
                              fits(width, "pages"), ldp, static_cast<const int32_t*>(vector(lens, at::kInt, B, "lens")),
                              static_cast<float>(scale), tokens, out.data_ptr(), ldo, pl,
                              ws.data_ptr(), ws.nbytes(), stream_of(a[9], q));
  });
}

// lora_apply(A, B, scale, plan, plan_tokens, x, base, out, stream) -> tl_status
PyObject* lora_apply(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("lora_apply", n, 9, [&] {
    const at::Tensor &A = *tensor(a[0], "A"), &B = *tensor(a[1], "B"), &scale = *tensor(a[2], "scale"), &plan = *tensor(a[3], "plan");
    const at::Tensor &x = *tensor(a[5], "x"), &base = *tensor(a[6], "base"), &out = *tensor(a[7], "out");
    const int device = A.device().index();
    on_device(&B, device, "B"), on_device(&scale, device, "scale"), on_device(&plan, device, "plan");
    on_device(&x, device, "x"), on_device(&base, device, "base"), on_device(&out, device, "out");
    const int64_t adapters = A.size(0), rank = A.size(1), K = A.size(2), N = B.size(1), M = integer(a[4]);
    const int code = half_code(A, "A");
    want_type(x, A.scalar_type(), "x");
    int y_code = TL_F32;
    if (base.scalar_type() != at::kFloat) y_code = half_code(base, "base");
    want_type(out, base.scalar_type(), "out");
    const int64_t ldx = matrix(x, M, K, "x"), ldb = matrix(base, M, N, "base"), ldy = matrix(out, M, N, "out");
    const OnDevice guard(device);
    return tl_lora_apply(x.data_ptr(), ldx, A.data_ptr(), B.data_ptr(), static_cast<const float*>(scale.data_ptr()), code,
                         fits(adapters, "A"), fits(rank, "A"), plan.data_ptr(), fits(M, "x"), fits(N, "B"), fits(K, "A"), base.data_ptr(),
                         ldb, out.data_ptr(), ldy, y_code, stream_of(a[8], x));
  });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(kv_append), METHOD(paged_attention), METHOD(lora_apply), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
