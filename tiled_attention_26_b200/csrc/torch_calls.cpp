// Direct calls of the KV cache and shared-prefix entry points for torch tensors.
//
// These calls sit in every step of a serving loop and their kernels take a few microseconds; checking
// a dozen tensors and marshalling twenty arguments in Python took ten to twenty.  Each function here
// takes the arguments of its Python counterpart, and either makes the call and returns its status
// (with the outputs), or returns None without side effects where anything is not the plain case (a
// wrong type, shape, device or layout, a tensor subclass, another current device).  The Python
// function then takes its own way, which names what is wrong.
//
// The C functions are those of the loaded libfa.so: init() receives their addresses.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/DimVector.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>

#include "../../include/fa.h"

namespace {

struct Library {
  decltype(&fa_kv_quantize_int8) quantize8;
  decltype(&fa_kv_quantize_int4) quantize4;
  decltype(&fa_kv_dequantize_int8) dequantize8;
  decltype(&fa_kv_dequantize_int4) dequantize4;
  decltype(&fa_kv_append_int8_paged) append8;
  decltype(&fa_kv_append_int4_paged) append4;
  decltype(&fa_kv_gather_int8_paged) gather8;
  decltype(&fa_kv_gather_int4_paged) gather4;
  decltype(&fa_decode_int8_shared) shared8;
  decltype(&fa_decode_int4_shared) shared4;
  decltype(&fa_decode_shared_workspace_bytes) shared_bytes;
} L;

using Shape = at::IntArrayRef;

// The argument as a plain torch.Tensor, or null.
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool is(const at::Tensor& t, at::ScalarType type, c10::Device dev, Shape shape) {
  return t.scalar_type() == type && t.device() == dev && t.sizes() == shape && t.is_contiguous();
}

// CUDA, the current device, strided.
bool here(const at::Tensor& t) {
  return t.is_cuda() && t.layout() == at::kStrided && t.device().index() == c10::cuda::current_device();
}

// An optional tensor argument: None -> true and null; otherwise it must match.
bool optional(PyObject* o, at::ScalarType type, c10::Device dev, Shape shape, const at::Tensor** out) {
  *out = nullptr;
  if (o == Py_None) return true;
  *out = tensor(o);
  return *out != nullptr && is(**out, type, dev, shape);
}

// Lets other Python threads run while a buffer is allocated and the kernels are launched: either may block (a
// full launch queue, an allocator that waits for memory), and what it waits for may need Python.  What is
// used meanwhile is held by the caller's frame; no Python object is touched.
class Unlocked {
 public:
  Unlocked() : state_(PyEval_SaveThread()) {}
  ~Unlocked() { PyEval_RestoreThread(state_); }
  Unlocked(const Unlocked&) = delete;
  Unlocked& operator=(const Unlocked&) = delete;

 private:
  PyThreadState* state_;
};

// A new tensor, without the dispatcher's way to it: a paged gather with its two outputs takes 5.3 us of
// host time so, 5.9 us through at::empty. Deterministic mode fills new tensors, which at::empty does.
at::Tensor empty(Shape shape, at::ScalarType type, c10::Device dev) {
  const at::Context& ctx = at::globalContext();
  if (ctx.deterministicAlgorithms() && ctx.deterministicFillUninitializedMemory())
    return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
  return at::detail::empty_cuda(shape, type, dev, c10::nullopt);
}

// An output argument: the caller's tensor, or None, for which make() allocates one (without the interpreter's
// lock, after every argument has been checked).
struct Output {
  at::Tensor t;
  at::ScalarType type;
  at::DimVector shape;

  void make(c10::Device dev) {
    if (!t.defined()) t = empty(shape, type, dev);
  }
};
bool output(PyObject* o, at::ScalarType type, c10::Device dev, Shape shape, Output* out) {
  out->type = type;
  out->shape = shape;
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o);
  if (t == nullptr || !is(*t, type, dev, shape)) return false;
  out->t = *t;
  return true;
}

void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
template <class T>
T* ptr_as(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <class T>
T* ptr_as(const at::Tensor* t) {
  return static_cast<T*>(ptr(t));
}

void* stream_of(c10::Device dev) { return c10::cuda::getCurrentCUDAStream(dev.index()).stream(); }

bool fits_int(int64_t x) { return x >= 0 && x <= 0x7fffffff; }

at::ScalarType code_type(long bits) { return bits == 8 ? at::kChar : at::kByte; }

// A page pool and a block table.
struct Pool {
  const at::Tensor *k, *v, *ks, *vs, *table;
  int pages, page, Hkv, D, B, max_pages;
};
// a: k_pages, v_pages, k_scale_pages, v_scale_pages
bool pool(PyObject* const* a, PyObject* table, long bits, Pool* p) {
  p->k = tensor(a[0]);
  p->v = tensor(a[1]);
  p->ks = tensor(a[2]);
  p->vs = tensor(a[3]);
  p->table = tensor(table);
  if (!p->k || !p->v || !p->ks || !p->vs || !p->table || !here(*p->k) || p->k->dim() != 4 ||
      p->table->dim() != 2)
    return false;
  const c10::Device dev = p->k->device();
  const int64_t n = p->k->size(0), P = p->k->size(1), H = p->k->size(2), row = p->k->size(3);
  if (!is(*p->k, code_type(bits), dev, {n, P, H, row}) || !is(*p->v, code_type(bits), dev, {n, P, H, row}) ||
      !is(*p->ks, at::kFloat, dev, {n, H, P}) || !is(*p->vs, at::kFloat, dev, {n, H, P}) ||
      !is(*p->table, at::kInt, dev, p->table->sizes()))
    return false;
  const int64_t D = bits == 8 ? row : 2 * row;
  if (!fits_int(n) || !fits_int(P) || !fits_int(H) || !fits_int(D) || !fits_int(p->table->size(0)) ||
      !fits_int(p->table->size(1)))
    return false;
  p->pages = static_cast<int>(n);
  p->page = static_cast<int>(P);
  p->Hkv = static_cast<int>(H);
  p->D = static_cast<int>(D);
  p->B = static_cast<int>(p->table->size(0));
  p->max_pages = static_cast<int>(p->table->size(1));
  return true;
}

// Token rows [N, Hkv, D] or [B, T, Hkv, D]: each row contiguous, rows evenly spaced.
bool token_rows(const at::Tensor& t, const Pool& p, int64_t* n, int64_t* step) {
  const int64_t d = t.dim();
  if (t.scalar_type() != at::kBFloat16 || t.device() != p.k->device() || (d != 3 && d != 4) ||
      t.size(d - 2) != p.Hkv || t.size(d - 1) != p.D || t.numel() == 0)
    return false;
  if ((t.stride(d - 1) != 1 && p.D > 1) || (t.stride(d - 2) != p.D && p.Hkv > 1)) return false;
  *n = t.size(0);
  *step = t.stride(0);
  if (d == 4) {
    *n = t.size(0) * t.size(1);
    if (t.size(1) > 1) {
      *step = t.stride(1);
      if (t.size(0) > 1 && t.stride(0) != t.size(1) * t.stride(1)) return false;
    }
  }
  if (*n <= 1) *step = std::max<int64_t>(*step, static_cast<int64_t>(p.Hkv) * p.D);
  return fits_int(*n);
}

PyObject* none() { Py_RETURN_NONE; }

// (bits, k, v, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, positions, cu_tokens)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 10) return none();
  const long bits = PyLong_AsLong(a[0]);
  const at::Tensor *k = tensor(a[1]), *v = tensor(a[2]), *pos, *cu;
  Pool p;
  int64_t n, nv, ks, vs;
  if (!k || !v || !pool(a + 3, a[7], bits, &p) || k->sizes() != v->sizes() ||
      !token_rows(*k, p, &n, &ks) || !token_rows(*v, p, &nv, &vs))
    return none();
  const c10::Device dev = k->device();
  if (!optional(a[8], at::kInt, dev, {p.B}, &pos) || !optional(a[9], at::kInt, dev, {p.B + 1}, &cu) ||
      (cu == nullptr && k->dim() == 4 && k->size(0) != p.B))
    return none();
  const int N = static_cast<int>(n);
  int rc;
  {
    Unlocked unlocked;
    rc = bits == 8
             ? L.append8(k->data_ptr(), v->data_ptr(), ks, vs, ptr_as<int8_t>(p.k), ptr_as<int8_t>(p.v),
                         ptr_as<float>(p.ks), ptr_as<float>(p.vs), ptr_as<int32_t>(p.table),
                         ptr_as<int32_t>(pos), ptr_as<int32_t>(cu), N, p.B, p.Hkv, p.page, p.max_pages,
                         p.pages, p.D, stream_of(dev))
             : L.append4(k->data_ptr(), v->data_ptr(), ks, vs, ptr_as<uint8_t>(p.k), ptr_as<uint8_t>(p.v),
                         ptr_as<float>(p.ks), ptr_as<float>(p.vs), ptr_as<int32_t>(p.table),
                         ptr_as<int32_t>(pos), ptr_as<int32_t>(cu), N, p.B, p.Hkv, p.page, p.max_pages,
                         p.pages, p.D, stream_of(dev));
  }
  return PyLong_FromLong(rc);
}

// (bits, k_pages, v_pages, k_scale_pages, v_scale_pages, block_table, num_tokens, positions,
//  cu_tokens, k, v) -> (status, k, v)
PyObject* kv_gather(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 11 || !PyLong_CheckExact(a[6])) return none();
  const long bits = PyLong_AsLong(a[0]);
  int overflow = 0;
  const long long n = PyLong_AsLongLongAndOverflow(a[6], &overflow);
  Pool p;
  const at::Tensor *pos, *cu;
  if (overflow || !fits_int(n) || !pool(a + 1, a[5], bits, &p)) return none();
  const c10::Device dev = p.k->device();
  Output k, v;
  if (!optional(a[7], at::kInt, dev, {p.B}, &pos) || !optional(a[8], at::kInt, dev, {p.B + 1}, &cu) ||
      !output(a[9], at::kBFloat16, dev, {n, p.Hkv, p.D}, &k) ||
      !output(a[10], at::kBFloat16, dev, {n, p.Hkv, p.D}, &v))
    return none();
  const int N = static_cast<int>(n);
  int rc;
  {
    Unlocked unlocked;
    k.make(dev);
    v.make(dev);
    rc = bits == 8
             ? L.gather8(ptr_as<int8_t>(p.k), ptr_as<int8_t>(p.v), ptr_as<float>(p.ks),
                         ptr_as<float>(p.vs), ptr_as<int32_t>(p.table), ptr_as<int32_t>(pos),
                         ptr_as<int32_t>(cu), k.t.data_ptr(), v.t.data_ptr(), N, p.B, p.Hkv, p.page,
                         p.max_pages, p.pages, p.D, stream_of(dev))
             : L.gather4(ptr_as<uint8_t>(p.k), ptr_as<uint8_t>(p.v), ptr_as<float>(p.ks),
                         ptr_as<float>(p.vs), ptr_as<int32_t>(p.table), ptr_as<int32_t>(pos),
                         ptr_as<int32_t>(cu), k.t.data_ptr(), v.t.data_ptr(), N, p.B, p.Hkv, p.page,
                         p.max_pages, p.pages, p.D, stream_of(dev));
  }
  return Py_BuildValue("(iNN)", rc, THPVariable_Wrap(k.t), THPVariable_Wrap(v.t));
}

// (bits, k, v, k_codes, v_codes, k_scale, v_scale) -> (status, k_codes, v_codes, k_scale, v_scale)
PyObject* kv_quantize(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 7) return none();
  const long bits = PyLong_AsLong(a[0]);
  const at::Tensor *k = tensor(a[1]), *v = tensor(a[2]);
  if (!k || !v || !here(*k) || k->dim() != 4) return none();
  const c10::Device dev = k->device();
  const int64_t B = k->size(0), S = k->size(1), H = k->size(2), D = k->size(3);
  const int64_t row = bits == 8 ? D : D / 2;
  Output kc, vc, ks, vs;
  if (!fits_int(B) || !fits_int(S) || !fits_int(H) || !fits_int(D) ||
      !is(*k, at::kBFloat16, dev, {B, S, H, D}) || !is(*v, at::kBFloat16, dev, {B, S, H, D}) ||
      !output(a[3], code_type(bits), dev, {B, S, H, row}, &kc) ||
      !output(a[4], code_type(bits), dev, {B, S, H, row}, &vc) ||
      !output(a[5], at::kFloat, dev, {B, H, S}, &ks) || !output(a[6], at::kFloat, dev, {B, H, S}, &vs))
    return none();
  const int b = static_cast<int>(B), s = static_cast<int>(S), h = static_cast<int>(H),
            d = static_cast<int>(D);
  int rc;
  {
    Unlocked unlocked;
    for (Output* x : {&kc, &vc, &ks, &vs}) x->make(dev);
    rc = bits == 8 ? L.quantize8(k->data_ptr(), v->data_ptr(), ptr_as<int8_t>(kc.t), ptr_as<int8_t>(vc.t),
                                 ptr_as<float>(ks.t), ptr_as<float>(vs.t), b, s, h, d, stream_of(dev))
                   : L.quantize4(k->data_ptr(), v->data_ptr(), ptr_as<uint8_t>(kc.t),
                                 ptr_as<uint8_t>(vc.t), ptr_as<float>(ks.t), ptr_as<float>(vs.t), b, s, h,
                                 d, stream_of(dev));
  }
  return Py_BuildValue("(iNNNN)", rc, THPVariable_Wrap(kc.t), THPVariable_Wrap(vc.t),
                       THPVariable_Wrap(ks.t), THPVariable_Wrap(vs.t));
}

// (bits, k_codes, v_codes, k_scale, v_scale, k, v) -> (status, k, v)
PyObject* kv_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 7) return none();
  const long bits = PyLong_AsLong(a[0]);
  const at::Tensor *kc = tensor(a[1]), *vc = tensor(a[2]), *ks = tensor(a[3]), *vs = tensor(a[4]);
  if (!kc || !vc || !ks || !vs || !here(*kc) || kc->dim() != 4) return none();
  const c10::Device dev = kc->device();
  const int64_t B = kc->size(0), S = kc->size(1), H = kc->size(2), row = kc->size(3);
  const int64_t D = bits == 8 ? row : 2 * row;
  Output k, v;
  if (!fits_int(B) || !fits_int(S) || !fits_int(H) || !fits_int(D) ||
      !is(*kc, code_type(bits), dev, {B, S, H, row}) || !is(*vc, code_type(bits), dev, {B, S, H, row}) ||
      !is(*ks, at::kFloat, dev, {B, H, S}) || !is(*vs, at::kFloat, dev, {B, H, S}) ||
      !output(a[5], at::kBFloat16, dev, {B, S, H, D}, &k) ||
      !output(a[6], at::kBFloat16, dev, {B, S, H, D}, &v))
    return none();
  const int b = static_cast<int>(B), s = static_cast<int>(S), h = static_cast<int>(H),
            d = static_cast<int>(D);
  int rc;
  {
    Unlocked unlocked;
    k.make(dev);
    v.make(dev);
    rc = bits == 8 ? L.dequantize8(ptr_as<int8_t>(*kc), ptr_as<int8_t>(*vc), ptr_as<float>(*ks),
                                   ptr_as<float>(*vs), k.t.data_ptr(), v.t.data_ptr(), b, s, h, d,
                                   stream_of(dev))
                   : L.dequantize4(ptr_as<uint8_t>(*kc), ptr_as<uint8_t>(*vc), ptr_as<float>(*ks),
                                   ptr_as<float>(*vs), k.t.data_ptr(), v.t.data_ptr(), b, s, h, d,
                                   stream_of(dev));
  }
  return Py_BuildValue("(iNN)", rc, THPVariable_Wrap(k.t), THPVariable_Wrap(v.t));
}

// (bits, q, k_pages, v_pages, k_scale_pages, v_scale_pages, prefix_table, prefix_len, block_table,
//  seqlens, num_splits, scale, o, lse, workspace, return_lse) -> (status, o, lse)
PyObject* decode_shared(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 16 || !PyLong_CheckExact(a[10])) return none();
  const long bits = PyLong_AsLong(a[0]);
  const at::Tensor *q = tensor(a[1]), *pt = tensor(a[6]), *pl = tensor(a[7]), *sl = tensor(a[9]), *lse_in;
  Pool p;
  if (!q || !pt || !pl || !sl || !pool(a + 2, a[8], bits, &p) || q->dim() != 4 || q->size(1) != 1)
    return none();
  const c10::Device dev = p.k->device();
  const int64_t B = q->size(0), Hq = q->size(2);
  if (!is(*q, at::kBFloat16, dev, {B, 1, Hq, p.D}) || p.B != B || !fits_int(Hq) || pt->dim() != 1 ||
      !fits_int(pt->size(0)) || !is(*pt, at::kInt, dev, pt->sizes()) || !is(*pl, at::kInt, dev, {1}) ||
      !is(*sl, at::kInt, dev, {B}) || !optional(a[13], at::kFloat, dev, {B, Hq}, &lse_in))
    return none();
  double scale = 0;
  if (a[11] == Py_None) {
    scale = 1.0 / std::sqrt(static_cast<double>(p.D));
  } else if (PyFloat_CheckExact(a[11])) {
    scale = PyFloat_AS_DOUBLE(a[11]);
  } else {
    return none();
  }
  int overflow = 0;
  const long splits = PyLong_AsLongAndOverflow(a[10], &overflow);
  const int max_prefix = static_cast<int>(pt->size(0));
  const int64_t prefix_keys = static_cast<int64_t>(max_prefix) * p.page;
  const int64_t own_keys = static_cast<int64_t>(p.max_pages) * p.page;
  if (overflow || !fits_int(splits) || !fits_int(prefix_keys) || !fits_int(own_keys)) return none();
  Output o;
  at::Tensor ws, lse;
  if (!output(a[12], at::kBFloat16, dev, {B, 1, Hq, p.D}, &o)) return none();
  if (a[14] != Py_None) {
    const at::Tensor* w = tensor(a[14]);
    if (w == nullptr || w->device() != dev || !w->is_contiguous()) return none();
    ws = *w;
  }
  const int return_lse = PyObject_IsTrue(a[15]);
  if (return_lse < 0) return none();
  if (lse_in != nullptr) lse = *lse_in;
  int rc;
  {
    Unlocked unlocked;
    o.make(dev);
    if (!ws.defined()) {
      const size_t need =
          L.shared_bytes(p.B, static_cast<int>(Hq), p.Hkv, p.D, static_cast<int>(prefix_keys),
                         static_cast<int>(own_keys), static_cast<int>(splits));
      ws = empty({static_cast<int64_t>(std::max<size_t>(need, 1))}, at::kByte, dev);
    }
    if (!lse.defined() && return_lse) lse = empty({B, Hq}, at::kFloat, dev);
    float* lse_ptr = lse.defined() ? ptr_as<float>(lse) : nullptr;
    rc = bits == 8
             ? L.shared8(q->data_ptr(), ptr_as<int8_t>(p.k), ptr_as<int8_t>(p.v), ptr_as<float>(p.ks),
                         ptr_as<float>(p.vs), ptr_as<int32_t>(pt), ptr_as<int32_t>(pl),
                         ptr_as<int32_t>(p.table), ptr_as<int32_t>(sl), o.t.data_ptr(), lse_ptr, p.B,
                         static_cast<int>(Hq), p.Hkv, p.page, max_prefix, p.max_pages, p.pages, p.D,
                         static_cast<float>(scale), static_cast<int>(splits), ws.data_ptr(), ws.nbytes(),
                         stream_of(dev))
             : L.shared4(q->data_ptr(), ptr_as<uint8_t>(p.k), ptr_as<uint8_t>(p.v), ptr_as<float>(p.ks),
                         ptr_as<float>(p.vs), ptr_as<int32_t>(pt), ptr_as<int32_t>(pl),
                         ptr_as<int32_t>(p.table), ptr_as<int32_t>(sl), o.t.data_ptr(), lse_ptr, p.B,
                         static_cast<int>(Hq), p.Hkv, p.page, max_prefix, p.max_pages, p.pages, p.D,
                         static_cast<float>(scale), static_cast<int>(splits), ws.data_ptr(), ws.nbytes(),
                         stream_of(dev));
  }
  PyObject* lse_obj;
  if (lse.defined()) {
    lse_obj = THPVariable_Wrap(lse);
  } else {
    Py_INCREF(Py_None);
    lse_obj = Py_None;
  }
  return Py_BuildValue("(iNN)", rc, THPVariable_Wrap(o.t), lse_obj);
}

// Nothing is launched when a C++ exception (an allocation that fails) ends F: the Python function then
// meets and reports the same.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  try {
    PyObject* r = F(self, args, n);
    if (PyErr_Occurred() && r != nullptr) {  // (an argument that is no number: not the plain case)
      Py_DECREF(r);
      PyErr_Clear();
      return none();
    }
    return r;
  } catch (const std::exception&) {
    PyErr_Clear();
    return none();
  }
}

// init(addresses of the C functions, in the order of Library)
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void** fields = reinterpret_cast<void**>(&L);
  if (n != static_cast<Py_ssize_t>(sizeof(Library) / sizeof(void*))) {
    PyErr_SetString(PyExc_TypeError, "wrong number of addresses");
    return nullptr;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    fields[i] = PyLong_AsVoidPtr(a[i]);
    if (fields[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  Py_RETURN_NONE;
}

#define FA_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {FA_METHOD(init),        FA_METHOD(kv_append),     FA_METHOD(kv_gather),
                         FA_METHOD(kv_quantize), FA_METHOD(kv_dequantize), FA_METHOD(decode_shared),
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls() { return PyModule_Create(&module); }
