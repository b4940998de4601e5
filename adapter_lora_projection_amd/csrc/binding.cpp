// Tensor marshalling of the decode-step operators for Python: checks the tensors, takes sizes and
// strides from them, allocates outputs and calls the C entry points on the current stream of their
// device. At decode sizes a call is shorter than the interpreter's share of such work (a call of 11
// tensors took 12 us through ctypes and tensor attributes, 4 us of it on the GPU), so it is native. No
// arithmetic and no state here: an operand's values never pass through this file.
//
// A function returns its result, or the status of the C entry point as an int if it is not LORA_OK.
#include <ATen/ATen.h>
#include <Python.h>
#include <c10/hip/HIPStream.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <string>

#include "../../include/lora_mi355x.h"

namespace {

struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse(const std::string& what) { throw Refused{PyExc_ValueError, what}; }
[[noreturn]] void refuse_type(const std::string& what) { throw Refused{PyExc_TypeError, what}; }

// A tensor argument; null for None.
const at::Tensor* opt(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse_type(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& req(PyObject* o, const char* name) {
  const at::Tensor* t = opt(o, name);
  if (t == nullptr) refuse_type(std::string(name) + " must be a tensor");
  return *t;
}

double as_double(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse_type("scale and eps must be numbers");
  }
  return v;
}

const void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

lora_dtype half_code(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return LORA_BF16;
  if (t.scalar_type() == at::kHalf) return LORA_F16;
  refuse_type(std::string(name) + " must be bf16 or fp16");
}

void same_dtype(const at::Tensor& t, const at::Tensor& ref, const char* name) {
  if (t.scalar_type() != ref.scalar_type())
    refuse_type(std::string(name) + " must have the dtype " + c10::toString(ref.scalar_type()));
}

// Row pitch of a matrix whose rows are contiguous (the pitch of a single row does not matter).
int64_t pitch(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(std::string(name) + " must be a 2-D tensor");
  if (t.size(1) > 1 && t.stride(1) != 1) refuse(std::string(name) + " must have a unit column stride");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

void vector_of(const at::Tensor& t, at::ScalarType type, int64_t n, const char* name) {
  if (t.scalar_type() != type || t.dim() != 1 || (n >= 0 && t.size(0) != n) || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " vector" +
           (n >= 0 ? " of " + std::to_string(n) : ""));
}

// The one GPU of all operands.
template <size_t N>
int device_of(const at::Tensor* const (&ts)[N]) {
  int dev = -2;
  for (const at::Tensor* t : ts) {
    if (t == nullptr) continue;
    if (!t->is_cuda()) refuse("all tensors must be on the GPU");
    const int d = t->get_device();
    if (dev == -2) dev = d;
    else if (d != dev) refuse("all tensors must be on one GPU");
  }
  return dev;
}

// Output [rows][cols]: a new tensor like `ref`, or the caller's, of that shape with contiguous rows.
at::Tensor output(const at::Tensor* given, int64_t rows, int64_t cols, const at::Tensor& ref, const char* name) {
  if (given == nullptr) return at::empty({rows, cols}, ref.options());
  if (given->scalar_type() != ref.scalar_type() || given->dim() != 2 || given->size(0) != rows || given->size(1) != cols)
    refuse(std::string(name) + " must be [" + std::to_string(rows) + "][" + std::to_string(cols) + "] of dtype " +
           c10::toString(ref.scalar_type()));
  pitch(*given, name);
  return *given;
}

// Refuses an output of which an element may be one of the matrix `in`. Column blocks of one buffer (equal
// pitches) are told apart; other interleavings are not.
void no_overlap(const at::Tensor& out, const at::Tensor& in, const char* oname, const char* iname) {
  if (out.numel() == 0 || in.numel() == 0) return;
  const int64_t lo = pitch(out, oname), li = pitch(in, iname);
  const int64_t eo = (out.size(0) - 1) * lo + out.size(1), ei = (in.size(0) - 1) * li + in.size(1);
  const int64_t size = int64_t(out.element_size());
  const int64_t d = reinterpret_cast<intptr_t>(out.data_ptr()) - reinterpret_cast<intptr_t>(in.data_ptr());
  if (d >= ei * size || -d >= eo * size) return;
  if (out.size(0) > 1 && in.size(0) > 1 && lo == li) {
    const int64_t c = ((d % (lo * size)) + lo * size) % (lo * size);  // where out's columns start in in's rows
    if (c >= in.size(1) * size && c + out.size(1) * size <= lo * size) return;
  }
  refuse(std::string(oname) + " must not overlap " + iname);
}

// The pair of caches [pages][page size][heads][D], of one shape and strides.
struct Cache {
  int64_t pages, page, heads, D, ps, ts, hs;
};
Cache cache_of(const at::Tensor& k, const at::Tensor& v, const at::Tensor& ref) {
  if (k.dim() != 4 || k.sizes() != v.sizes())
    refuse("k_cache and v_cache must be [pages][page size][heads][D], of one shape");
  same_dtype(k, ref, "k_cache");
  same_dtype(v, ref, "v_cache");
  if (k.strides() != v.strides()) refuse("k_cache and v_cache must have the same strides");
  if (k.size(3) < 1) refuse("the caches must have D >= 1");
  if (k.size(3) > 1 && k.stride(3) != 1) refuse("the caches must have a unit stride along D");
  // a stride of an extent of one place is never used
  return {k.size(0), k.size(1), k.size(2), k.size(3), k.size(0) > 1 ? k.stride(0) : 0,
          k.size(1) > 1 ? k.stride(1) : 0, k.size(2) > 1 ? k.stride(2) : 0};
}

int32_t narrow(int64_t v, const char* name) {
  if (v < 0 || v > INT32_MAX) refuse(std::string(name) + " is too large");
  return int32_t(v);
}

// Calls `f` with the current stream of `dev`, that device being current.
template <typename F>
lora_status launch(int dev, F f) {
  int was = -1;
  if (hipGetDevice(&was) != hipSuccess) return LORA_EHIP;
  if (was != dev && hipSetDevice(dev) != hipSuccess) return LORA_EHIP;
  const lora_status st = f(static_cast<void*>(c10::hip::getCurrentHIPStream(c10::DeviceIndex(dev)).stream()));
  if (was != dev && hipSetDevice(was) != hipSuccess) return LORA_EHIP;
  return st;
}

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* arity(const char* name) {
  PyErr_SetString(PyExc_TypeError, (std::string(name) + ": wrong number of arguments").c_str());
  return nullptr;
}

PyObject* status(lora_status s) { return PyLong_FromLong(long(s)); }

// linear_w4(x, data, dtype code, K, N, group, zero_points, out)
PyObject* linear_w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) return arity("linear_w4");
  return guarded([&]() -> PyObject* {
    const at::Tensor &x = req(a[0], "x"), &data = req(a[1], "data");
    const at::Tensor* given = opt(a[7], "out");
    const long code = PyLong_AsLong(a[2]);
    const int64_t K = PyLong_AsLongLong(a[3]), N = PyLong_AsLongLong(a[4]);
    const int32_t group = int32_t(PyLong_AsLong(a[5])), zp = a[6] == Py_True;
    const lora_dtype dt = half_code(x, "x");
    if (long(dt) != code) refuse_type("x must have the dtype of the weight's scales");
    const int64_t ldx = pitch(x, "x");
    if (x.size(1) != K) refuse("x must be [M][" + std::to_string(K) + "]");
    vector_of(data, at::kByte, -1, "data");
    if (size_t(data.numel()) < lora_linear_w4_prepared_size(dt, K, N, group, zp)) refuse("data is not a weight of these sizes");
    if (given != nullptr) output(given, x.size(0), N, x, "out");
    if (given != nullptr) no_overlap(*given, x, "out", "x");
    const int dev = device_of({&x, &data, given});
    const at::Tensor out = output(given, x.size(0), N, x, "out");
    const int64_t ldy = pitch(out, "out");
    const size_t bytes = lora_linear_w4_workspace_size(dt, x.size(0), K, N, group);
    at::Tensor ws;
    if (bytes > 0) ws = at::empty({int64_t(bytes)}, x.options().dtype(at::kByte));
    const lora_status st = launch(dev, [&](void* stream) {
      return lora_linear_w4(dt, x.size(0), K, N, group, zp, x.data_ptr(), ldx, data.data_ptr(), out.data_ptr(), ldy,
                            bytes > 0 ? ws.data_ptr() : nullptr, bytes, stream);
    });
    return st == LORA_OK ? THPVariable_Wrap(out) : status(st);
  });
}

// rope_append(q, k, v, table, positions, slots, k_cache, v_cache, q_norm, k_norm, eps, interleaved, q_out)
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return arity("rope_append");
  return guarded([&]() -> PyObject* {
    const at::Tensor &q = req(a[0], "q"), &k = req(a[1], "k"), &v = req(a[2], "v"), &table = req(a[3], "table");
    const at::Tensor &positions = req(a[4], "positions"), &slots = req(a[5], "slots");
    const at::Tensor &kc = req(a[6], "k_cache"), &vc = req(a[7], "v_cache");
    const at::Tensor *qn = opt(a[8], "q_norm"), *kn = opt(a[9], "k_norm"), *given = opt(a[12], "q_out");
    const float eps = float(as_double(a[10]));
    const int interleaved = PyObject_IsTrue(a[11]);
    if (interleaved < 0) return nullptr;
    lora_dtype dt;
    if (q.scalar_type() == at::kFloat) dt = LORA_F32;
    else dt = half_code(q, "q (if not float32)");
    const Cache c = cache_of(kc, vc, q);
    const int64_t ldq = pitch(q, "q"), ldk = pitch(k, "k"), ldv = pitch(v, "v");
    const int64_t T = q.size(0), nq = q.size(1);
    if (nq % c.D != 0) refuse("q must be [T][Hq * D]");
    for (const at::Tensor* t : {&k, &v})
      if (t->size(0) != T || t->size(1) != c.heads * c.D) refuse("k and v must be [T][" + std::to_string(c.heads * c.D) + "]");
    same_dtype(k, q, "k");
    same_dtype(v, q, "v");
    if (qn != nullptr) vector_of(*qn, q.scalar_type(), c.D, "q_norm");
    if (kn != nullptr) vector_of(*kn, q.scalar_type(), c.D, "k_norm");
    if (table.scalar_type() != at::kFloat || table.dim() != 2 || !table.is_contiguous())
      refuse("table must be a contiguous float32 [rows][rot]");
    vector_of(positions, at::kInt, T, "positions");
    vector_of(slots, at::kLong, T, "slots");
    if (given != nullptr) output(given, T, nq, q, "q_out");
    if (given != nullptr && (given->data_ptr() != q.data_ptr() || pitch(*given, "q_out") != ldq)) no_overlap(*given, q, "q_out", "q");
    const int dev = device_of({&q, &k, &v, &table, &positions, &slots, &kc, &vc, qn, kn, given});
    const at::Tensor out = output(given, T, nq, q, "q_out");
    const int64_t ldqo = pitch(out, "q_out");
    const int32_t Hq = narrow(nq / c.D, "q"), Hkv = narrow(c.heads, "k_cache"), D = narrow(c.D, "k_cache");
    const int32_t page = narrow(c.page, "k_cache"), rot = narrow(table.size(1), "table");
    const lora_status st = launch(dev, [&](void* stream) {
      return lora_rope_append(dt, T, Hq, Hkv, D, rot, interleaved, c.pages, page, table.size(0), q.data_ptr(), ldq,
                              k.data_ptr(), ldk, v.data_ptr(), ldv, static_cast<const float*>(table.data_ptr()),
                              static_cast<const int32_t*>(positions.data_ptr()),
                              static_cast<const int64_t*>(slots.data_ptr()), ptr(qn), ptr(kn), eps, out.data_ptr(),
                              ldqo, kc.data_ptr(), vc.data_ptr(), c.ps, c.ts, c.hs, stream);
    });
    return st == LORA_OK ? THPVariable_Wrap(out) : status(st);
  });
}

// The width of a page list [n][width] with its lengths [n]; 0 for None.
int64_t page_list(const at::Tensor* pages, const at::Tensor* lens, int64_t n, const char* pname, const char* lname) {
  if ((pages == nullptr) != (lens == nullptr)) refuse(std::string(pname) + " and " + lname + " must be given together");
  if (pages == nullptr) return 0;
  if (pages->scalar_type() != at::kInt || pages->dim() != 2 || pages->size(0) != n || !pages->is_contiguous())
    refuse(std::string(pname) + " must be a contiguous int32 [" + std::to_string(n) + "][width]");
  vector_of(*lens, at::kInt, n, lname);
  return pages->size(1);
}

// prefix_attention(q, k_cache, v_cache, seg_indptr, permutation, prefix_pages, prefix_lens, own_pages,
//                  own_lens, scale, out, return_lse, workspace) -> out or (out, lse)
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 13) return arity("prefix_attention");
  return guarded([&]() -> PyObject* {
    const at::Tensor &q = req(a[0], "q"), &kc = req(a[1], "k_cache"), &vc = req(a[2], "v_cache");
    const at::Tensor &indptr = req(a[3], "seg_indptr"), *perm = opt(a[4], "permutation");
    const at::Tensor *pp = opt(a[5], "prefix_pages"), *pl = opt(a[6], "prefix_lens");
    const at::Tensor *op = opt(a[7], "own_pages"), *ol = opt(a[8], "own_lens");
    const float scale = float(as_double(a[9]));
    const at::Tensor *given = opt(a[10], "out"), *ws = opt(a[12], "workspace");
    const int with_lse = PyObject_IsTrue(a[11]);
    if (with_lse < 0) return nullptr;
    const lora_dtype dt = half_code(q, "q");
    const Cache c = cache_of(kc, vc, q);
    const int64_t ldq = pitch(q, "q"), T = q.size(0), nq = q.size(1);
    if (nq % c.D != 0) refuse("q must be [T][Hq * D]");
    vector_of(indptr, at::kInt, -1, "seg_indptr");
    if (indptr.size(0) < 1) refuse("seg_indptr must have at least one entry");
    const int64_t G = indptr.size(0) - 1;
    if (perm != nullptr) vector_of(*perm, at::kInt, T, "permutation");
    const int64_t wp = page_list(pp, pl, G, "prefix_pages", "prefix_lens");
    const int64_t wo = page_list(op, ol, T, "own_pages", "own_lens");
    if (given != nullptr) output(given, T, nq, q, "out");
    if (ws != nullptr) vector_of(*ws, at::kByte, -1, "workspace");
    if (given != nullptr) no_overlap(*given, q, "out", "q");
    const int dev = device_of({&q, &kc, &vc, &indptr, perm, pp, pl, op, ol, given, ws});
    const int32_t Hq = narrow(nq / c.D, "q"), Hkv = narrow(c.heads, "k_cache"), D = narrow(c.D, "k_cache");
    const int32_t page = narrow(c.page, "k_cache"), g = narrow(G, "seg_indptr");
    const at::Tensor out = output(given, T, nq, q, "out");
    const int64_t ldo = pitch(out, "out");
    at::Tensor lse, own_ws;
    if (with_lse) lse = at::empty({T, Hq}, q.options().dtype(at::kFloat));
    if (ws == nullptr) {
      own_ws = at::empty({int64_t(lora_prefix_attention_workspace_size(dt, T, g, Hq, Hkv, D, page, wp, wo))},
                         q.options().dtype(at::kByte));
      ws = &own_ws;
    }
    auto i32 = [](const at::Tensor* t) { return static_cast<const int32_t*>(ptr(t)); };
    const lora_status st = launch(dev, [&](void* stream) {
      return lora_prefix_attention(dt, T, g, Hq, Hkv, D, c.pages, page, q.data_ptr(), ldq, kc.data_ptr(), vc.data_ptr(),
                                   c.ps, c.ts, c.hs, i32(&indptr), i32(perm), i32(pp), wp, i32(pl), i32(op), wo, i32(ol),
                                   scale, out.data_ptr(), ldo, with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                                   ws->data_ptr(), size_t(ws->numel()), stream);
    });
    if (st != LORA_OK) return status(st);
    if (!with_lse) return THPVariable_Wrap(out);
    return Py_BuildValue("(NN)", THPVariable_Wrap(out), THPVariable_Wrap(lse));
  });
}

PyMethodDef methods[] = {
    {"linear_w4", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear_w4)), METH_FASTCALL, nullptr},
    {"rope_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope_append)), METH_FASTCALL, nullptr},
    {"prefix_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prefix_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Tensor marshalling of the decode-step operators.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
