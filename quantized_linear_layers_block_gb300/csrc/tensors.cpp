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

// [tokens, heads, dim], the heads of a token contiguous and the tokens any distance apart, which is returned. (Without tokens the strides
// say nothing: torch.tensor of an empty numpy array has zeros.)
int64_t token_rows(const at::Tensor& t, int64_t heads, int64_t dim, at::ScalarType type, const char* name) {
  want_type(t, type, name);
  const auto size = t.sizes(), stride = t.strides();
  if (size.size() != 3 || size[1] != heads || size[2] != dim)
    refuse("%s must be [tokens, %lld, %lld]", name, static_cast<long long>(heads), static_cast<long long>(dim));
  if (size[0] > 0 && (stride[2] != 1 || (stride[1] != dim && heads > 1))) refuse("%s: the heads of a token must be contiguous", name);
  return stride[0];
}

// [rows, cols] with contiguous rows any distance apart, which is returned
int64_t matrix(const at::Tensor& t, int64_t rows, int64_t cols, const char* name) {
  const auto size = t.sizes(), stride = t.strides();
  if (size.size() != 2 || size[0] != rows || size[1] != cols || (stride[1] != 1 && cols > 1 && rows > 0))
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

// a contiguous vector of n floats, or nothing for None
const float* weights(PyObject* o, int64_t n, int device, const char* name) {
  const at::Tensor* const t = tensor(o, name, true);
  if (t == nullptr) return nullptr;
  on_device(t, device, name);
  return static_cast<const float*>(vector(*t, at::kFloat, n, name));
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Refused{};
  return x;
}

// The arguments of kv_append but its stream, which `stream` is; `norms` are q_norm, k_norm, eps, or NULL for none.
int append(PyObject* const* a, PyObject* const* norms, PyObject* stream) {
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
  const float *q_norm = nullptr, *k_norm = nullptr;
  double eps = 1.0;
  if (norms != nullptr) {
    q_norm = weights(norms[0], c->head_dim, c->device, "q_norm");
    k_norm = weights(norms[1], c->head_dim, c->device, "k_norm");
    eps = number(norms[2]);
  }
  const OnDevice guard(c->device);
  return tl_kv_append_norm(c, pq, k.data_ptr(), v.data_ptr(), code, fits(T, "k"), fits(heads, "q"), ldq, ldk, ldv, po, ldo, q_norm, k_norm,
                           static_cast<float>(eps), table, fits(rows, "cos_sin"), fits(rot, "cos_sin"), interleaved, positions,
                           static_cast<const int64_t*>(vector(slots, at::kLong, T, "slots")), stream_of(stream, k));
}

// kv_append(cache, k, v, positions, slots, cos_sin, interleaved, q, q_out, stream) -> tl_status
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("kv_append", n, 10, [&] { return append(a, nullptr, a[9]); });
}

// kv_append_norm(cache, k, v, positions, slots, cos_sin, interleaved, q, q_out, q_norm, k_norm, eps, stream) -> tl_status
PyObject* kv_append_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("kv_append_norm", n, 13, [&] { return append(a, a + 9, a[12]); });
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
    const double scale = number(a[4]);
    const int64_t window = integer(a[5]);
    const int tokens = window > INT32_MAX ? 0 : window < 0 ? -1 : static_cast<int>(window);      // wider than any length: all; negative: refused
    const OnDevice guard(c->device);
    return tl_paged_attention(c, q.data_ptr(), code, fits(B, "q"), fits(heads, "q"), ldq, static_cast<const int32_t*>(pages.data_ptr()),
                              fits(width, "pages"), ldp, static_cast<const int32_t*>(vector(lens, at::kInt, B, "lens")),
                              static_cast<float>(scale), tokens, out.data_ptr(), ldo, pl,
                              ws.data_ptr(), ws.nbytes(), stream_of(a[9], q));
  });
}

// What the calls on drafted trees share: starts [B + 1], lens [B], pages [B, width], all on one GPU.
struct Trees {
  const int32_t *starts, *lens, *pages;
  int64_t ldp;
  int B, width;
  Trees(PyObject* s, PyObject* p, PyObject* l, int device) {
    const at::Tensor &st = *tensor(s, "starts"), &pg = *tensor(p, "pages"), &ln = *tensor(l, "lens");
    on_device(&st, device, "starts"), on_device(&pg, device, "pages"), on_device(&ln, device, "lens");
    B = requests(st);
    starts = static_cast<const int32_t*>(st.data_ptr());
    lens = static_cast<const int32_t*>(vector(ln, at::kInt, B, "lens"));
    want_type(pg, at::kInt, "pages");
    if (pg.dim() != 2) refuse("pages must be a matrix [requests, max_pages]");
    width = fits(pg.size(1), "pages");
    ldp = matrix(pg, B, width, "pages");
    pages = static_cast<const int32_t*>(pg.data_ptr());
  }
  static int requests(const at::Tensor& starts) {
    if (starts.dim() != 1 || starts.size(0) < 1) refuse("starts must be a vector [requests + 1]");
    vector(starts, at::kInt, starts.size(0), "starts");
    return fits(starts.size(0) - 1, "starts");
  }
};

// tree_plan(cache, parents, starts, lens, pages, masks, positions, slots, stream) -> tl_status
PyObject* tree_plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("tree_plan", n, 9, [&] {
    const auto* c = reinterpret_cast<const Cache*>(static_cast<intptr_t>(integer(a[0])));
    const at::Tensor &parents = *tensor(a[1], "parents"), &masks = *tensor(a[5], "masks"), &positions = *tensor(a[6], "positions"),
                     &slots = *tensor(a[7], "slots");
    on_device(&parents, c->device, "parents"), on_device(&masks, c->device, "masks"), on_device(&positions, c->device, "positions");
    on_device(&slots, c->device, "slots");
    const Trees trees(a[2], a[4], a[3], c->device);
    const int64_t T = parents.dim() == 1 ? parents.size(0) : 0;
    const auto* const up = static_cast<const int32_t*>(vector(parents, at::kInt, T, "parents"));
    auto* const pm = static_cast<int64_t*>(const_cast<void*>(vector(masks, at::kLong, T, "masks")));
    auto* const pp = static_cast<int32_t*>(const_cast<void*>(vector(positions, at::kInt, T, "positions")));
    auto* const ps = static_cast<int64_t*>(const_cast<void*>(vector(slots, at::kLong, T, "slots")));
    const OnDevice guard(c->device);
    return tl_tree_plan(up, trees.starts, trees.B, fits(T, "parents"), trees.lens, trees.pages, trees.width, trees.ldp, c->page_size,
                        c->num_pages, pm, pp, ps, stream_of(a[8], parents));
  });
}

// tree_attention(cache, q, masks, starts, pages, lens, scale, window, sinks, out, lse, workspace, stream) -> tl_status
PyObject* tree_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("tree_attention", n, 13, [&] {
    const auto* c = reinterpret_cast<const Cache*>(static_cast<intptr_t>(integer(a[0])));
    const at::Tensor &q = *tensor(a[1], "q"), &masks = *tensor(a[2], "masks"), &out = *tensor(a[9], "out");
    const at::Tensor *lse = tensor(a[10], "lse", true), &ws = *tensor(a[11], "workspace");
    on_device(&q, c->device, "q"), on_device(&masks, c->device, "masks"), on_device(&out, c->device, "out");
    on_device(lse, c->device, "lse"), on_device(&ws, c->device, "workspace");
    const Trees trees(a[3], a[4], a[5], c->device);
    const int code = half_code(q, "q");
    if (q.dim() != 3) refuse("q must be [tokens, heads, %d]", c->head_dim);
    const int64_t T = q.size(0), heads = q.size(1);
    const int64_t ldq = token_rows(q, heads, c->head_dim, q.scalar_type(), "q");
    const int64_t ldo = token_rows(out, heads, c->head_dim, q.scalar_type(), "out");
    if (out.size(0) != T) refuse("out and q must have the same number of tokens");
    float* pl = nullptr;
    if (lse != nullptr) {
      want_type(*lse, at::kFloat, "lse");
      if (!lse->is_contiguous()) refuse("lse must be contiguous");
      matrix(*lse, T, heads, "lse");
      pl = static_cast<float*>(lse->data_ptr());
    }
    const double scale = number(a[6]);
    const int64_t window = integer(a[7]), sinks = integer(a[8]);
    // wider than any length: all (and then no sinks, which lie in it); negative: refused
    const bool all = window > INT32_MAX;
    const int tokens = all ? 0 : window < 0 ? -1 : static_cast<int>(window);
    const int first = sinks < 0 ? -1 : all ? 0 : sinks > INT32_MAX ? INT32_MAX : static_cast<int>(sinks);
    const auto* const pm = static_cast<const int64_t*>(vector(masks, at::kLong, T, "masks"));
    const OnDevice guard(c->device);
    return tl_tree_attention(c, q.data_ptr(), code, trees.B, fits(T, "q"), fits(heads, "q"), ldq, pm, trees.starts, trees.pages, trees.width,
                             trees.ldp, trees.lens, static_cast<float>(scale), tokens, first, out.data_ptr(), ldo, pl, ws.data_ptr(),
                             ws.nbytes(), stream_of(a[12], q));
  });
}

// verify_tree(target, draft, tokens, parents, starts, uniform, path, counts, next, stream) -> tl_status
PyObject* verify_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("verify_tree", n, 10, [&] {
    const at::Tensor &target = *tensor(a[0], "target"), *draft = tensor(a[1], "draft", true), &tokens = *tensor(a[2], "tokens");
    const at::Tensor &parents = *tensor(a[3], "parents"), &starts = *tensor(a[4], "starts"), &uniform = *tensor(a[5], "uniform");
    const at::Tensor &path = *tensor(a[6], "path"), &counts = *tensor(a[7], "counts"), &next = *tensor(a[8], "next");
    const int device = target.device().index();
    on_device(draft, device, "draft"), on_device(&tokens, device, "tokens"), on_device(&parents, device, "parents");
    on_device(&starts, device, "starts"), on_device(&uniform, device, "uniform"), on_device(&path, device, "path");
    on_device(&counts, device, "counts"), on_device(&next, device, "next");
    if (target.dim() != 2) refuse("target must be a matrix [tokens, vocabulary]");
    const int64_t T = target.size(0), vocab = target.size(1);
    want_type(target, at::kFloat, "target");
    const int64_t ldt = matrix(target, T, vocab, "target");
    int64_t ldd = 0;
    const float* pd = nullptr;
    if (draft != nullptr) {
      want_type(*draft, at::kFloat, "draft");
      ldd = matrix(*draft, T, vocab, "draft");
      pd = static_cast<const float*>(draft->data_ptr());
    }
    const int B = Trees::requests(starts);
    auto ints = [&](const at::Tensor& t, int64_t size, const char* name) { return static_cast<int32_t*>(const_cast<void*>(vector(t, at::kInt, size, name))); };
    const int32_t *const pt = ints(tokens, T, "tokens"), *const pp = ints(parents, T, "parents");
    int32_t *const po = ints(path, T, "path"), *const pc = ints(counts, B, "counts"), *const pn = ints(next, B, "next");
    const auto* const pu = static_cast<const float*>(vector(uniform, at::kFloat, T, "uniform"));
    const OnDevice guard(device);
    return tl_verify_tree(static_cast<const float*>(target.data_ptr()), ldt, pd, ldd, fits(vocab, "the vocabulary"), pt, pp,
                          static_cast<const int32_t*>(starts.data_ptr()), B, fits(T, "target"), pu, po, pc, pn, stream_of(a[9], target));
  });
}

// kv_compact(cache, path, counts, starts, pages, lens, stream) -> tl_status
PyObject* kv_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("kv_compact", n, 7, [&] {
    const auto* c = reinterpret_cast<const Cache*>(static_cast<intptr_t>(integer(a[0])));
    const at::Tensor &path = *tensor(a[1], "path"), &counts = *tensor(a[2], "counts");
    on_device(&path, c->device, "path"), on_device(&counts, c->device, "counts");
    const Trees trees(a[3], a[4], a[5], c->device);
    const int64_t T = path.dim() == 1 ? path.size(0) : 0;
    const auto* const nodes = static_cast<const int32_t*>(vector(path, at::kInt, T, "path"));
    const auto* const pc = static_cast<const int32_t*>(vector(counts, at::kInt, trees.B, "counts"));
    const OnDevice guard(c->device);
    return tl_kv_compact(c, nodes, pc, trees.starts, trees.B, fits(T, "path"), trees.pages, trees.width, trees.ldp, trees.lens, stream_of(a[6], path));
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
PyMethodDef methods[] = {METHOD(kv_append),      METHOD(kv_append_norm), METHOD(paged_attention),
                         METHOD(lora_apply),     METHOD(tree_plan),      METHOD(tree_attention),
                         METHOD(verify_tree),    METHOD(kv_compact),     {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
