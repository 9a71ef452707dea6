// Argument marshalling of the decoder-layer calls for Python: checks of the
// tensors, output allocation and the C call, as one function of the CPython
// API for each operator.  These calls are made once or more for each layer and
// token, and one of a few tokens takes the GPU 2 to 8 us; the same checks
// written in Python over ctypes took 9 us of host time beside the launch's 3.5.
// No arithmetic and no launch is here: the C entry points of libfp8lin do that.
#include <Python.h>
#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/hip/EmptyTensor.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/fp8lin.h"

namespace {

using at::Tensor;
using Sizes = std::initializer_list<int64_t>;

PyObject *g_status_check = nullptr;  // _binding._check: raises Fp8LinError for a status other than FP8L_OK

// A Python error that is already set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const std::string &text) {
  PyErr_SetString(type, text.c_str());
  throw Raised{};
}

std::string text_of(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); i++) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

bool given(PyObject *o) { return o != Py_None; }

// The tensor in o: of this type (or of `bytes`, the float8 type that the bytes stand
// for), on the GPU, contiguous and (unless sizes is empty) of these sizes.
const Tensor &want(PyObject *o, const char *name, at::ScalarType type, Sizes sizes = {},
                   at::ScalarType bytes = at::ScalarType::Undefined) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + ": expected a torch.Tensor");
  const Tensor &t = THPVariable_Unpack(o);
  const at::ScalarType got = t.scalar_type();
  if (got != type && (bytes == at::ScalarType::Undefined || got != bytes))
    raise(PyExc_TypeError,
          std::string(name) + ": expected dtype " + c10::toString(type) + ", got " + c10::toString(got));
  if (!t.is_cuda()) raise(PyExc_ValueError, std::string(name) + ": expected a device tensor");
  if (!t.is_contiguous()) raise(PyExc_ValueError, std::string(name) + ": expected a contiguous tensor");
  if (sizes.size() && t.sizes() != at::IntArrayRef(sizes))
    raise(PyExc_ValueError, std::string(name) + ": expected shape " + text_of(sizes) + ", got " + text_of(t.sizes()));
  int current = -1;
  if (hipGetDevice(&current) != hipSuccess || t.get_device() != current)
    raise(PyExc_ValueError, std::string(name) + ": expected a tensor on the current device");
  return t;
}

// want() for a tensor of `dims` dimensions.
const Tensor &want_dims(PyObject *o, const char *name, at::ScalarType type, int64_t dims,
                        at::ScalarType bytes = at::ScalarType::Undefined) {
  const Tensor &t = want(o, name, type, {}, bytes);
  if (t.dim() != dims)
    raise(PyExc_ValueError,
          std::string(name) + ": expected " + std::to_string(dims) + " dimensions, got " + text_of(t.sizes()));
  return t;
}

// An output: the caller's tensor, or a new one beside `like` (the allocator's own
// call: 0.3 us less for each tensor than at::empty with its dispatch).
Tensor output(PyObject *o, const char *name, at::ScalarType type, Sizes sizes, const Tensor &like,
              at::ScalarType bytes = at::ScalarType::Undefined) {
  if (given(o)) return want(o, name, type, sizes, bytes);
  return at::detail::empty_cuda(sizes, type, like.device(), std::nullopt);
}

template <class T = void>
T *data(const Tensor &t) {
  return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr;
}

bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

int64_t whole(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

hipStream_t stream_of(PyObject *o) {
  void *p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised{};
  return static_cast<hipStream_t>(p);
}

void check(const char *fn, fp8l_status status) {
  if (status == FP8L_OK) return;
  PyObject *r = PyObject_CallFunction(g_status_check, "si", fn, (int)status);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, fn);
  throw Raised{};
}

// The C call, without the interpreter's lock.
template <class Call>
fp8l_status unlocked(Call call) {
  struct Released {
    PyThreadState *state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }  // also when a tensor without storage throws
  } released;
  return call();
}

PyObject *wrap_or_none(const Tensor &t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

// Runs f and turns C++ exceptions into Python's.
template <class F>
PyObject *guarded(Py_ssize_t got, Py_ssize_t expected, F f) {
  if (got != expected) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", expected, got);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised &) {
    return nullptr;
  } catch (const c10::Error &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    return nullptr;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// (ue8m0, x, w, res, eps, keep_y, quantize, h, y, q, s, stream) -> (h, y, q, s)
PyObject *add_rmsnorm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const bool ue8m0 = truth(a[0]), keep_y = truth(a[5]), quantize = truth(a[6]);
    const char *fn = ue8m0 ? "fp8_add_rmsnorm_ue8m0" : "fp8_add_rmsnorm";
    const Tensor &x = want_dims(a[1], "x", at::kBFloat16, 2);
    const int64_t M = x.size(0), K = x.size(1);
    const Tensor &w = want(a[2], "w", at::kBFloat16, {K});
    if (!keep_y && !quantize) raise(PyExc_ValueError, std::string(fn) + ": keep_y=False needs quantize=True");
    Tensor res, h, y, q, s;
    if (given(a[3])) {
      res = want(a[3], "res", at::kBFloat16, {M, K});
      h = output(a[7], "h", at::kBFloat16, {M, K}, x);
    } else if (given(a[7])) {
      raise(PyExc_ValueError, std::string(fn) + ": h is written only where res is given (without it h = x)");
    }
    if (keep_y) y = output(a[8], "y", at::kBFloat16, {M, K}, x);
    if (quantize) {
      q = output(a[9], "q", at::kByte, {M, K}, x, at::kFloat8_e4m3fn);
      s = ue8m0 ? output(a[10], "scales", at::kByte, {M, K / 128}, x, at::kFloat8_e8m0fnu)
                : output(a[10], "scales", at::kFloat, {M, K / 128}, x);
    }
    const float eps = (float)real(a[4]);
    hipStream_t stream = stream_of(a[11]);
    const auto *xp = data<uint16_t>(x), *rp = data<uint16_t>(res), *wp = data<uint16_t>(w);
    auto *hp = data<uint16_t>(h), *yp = data<uint16_t>(y);
    auto *qp = data<uint8_t>(q);
    void *sp = data(s);
    check(fn, unlocked([&] {
            return ue8m0 ? fp8_add_rmsnorm_ue8m0(xp, rp, wp, eps, M, K, hp, yp, qp, static_cast<uint8_t *>(sp), stream)
                         : fp8_add_rmsnorm(xp, rp, wp, eps, M, K, hp, yp, qp, static_cast<float *>(sp), stream);
          }));
    PyObject *out = PyTuple_New(4);
    if (!out) throw Raised{};
    PyTuple_SET_ITEM(out, 0, wrap_or_none(h));
    PyTuple_SET_ITEM(out, 1, wrap_or_none(y));
    PyTuple_SET_ITEM(out, 2, wrap_or_none(q));
    PyTuple_SET_ITEM(out, 3, wrap_or_none(s));
    return out;
  });
}

struct Cache {
  Tensor k, v, ks, vs;
  int64_t pages, heads, page, dim;
};

Cache want_cache(PyObject *const *a, bool fp8) {
  Cache c;
  const at::ScalarType type = fp8 ? at::kByte : at::kBFloat16;
  const at::ScalarType bytes = fp8 ? at::kFloat8_e4m3fn : at::ScalarType::Undefined;
  c.k = want_dims(a[0], "k_cache", type, 4, bytes);
  c.pages = c.k.size(0);
  c.heads = c.k.size(1);
  c.page = c.k.size(2);
  c.dim = c.k.size(3);
  c.v = want(a[1], "v_cache", type, {c.pages, c.heads, c.page, c.dim}, bytes);
  if (fp8) {
    c.ks = want(a[2], "k_scale", at::kFloat, {c.pages, c.heads, c.page});
    c.vs = want(a[3], "v_scale", at::kFloat, {c.pages, c.heads, c.page});
  }
  return c;
}

// (fp8, qkv, positions, slots, cos_sin, k_cache, v_cache, k_scale, v_scale, interleaved, q, stream) -> q
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 12, [&] {
    const bool fp8 = truth(a[0]);
    const Cache c = want_cache(a + 5, fp8);
    const Tensor &qkv = want_dims(a[1], "qkv", at::kBFloat16, 2);
    const int64_t T = qkv.size(0), width = qkv.size(1);
    const int64_t Hq = c.dim > 0 ? width / c.dim - 2 * c.heads : 0;
    if (Hq <= 0 || width % c.dim)
      raise(PyExc_ValueError, "qkv: " + std::to_string(width) + " columns do not hold query heads beside 2 x " +
                                  std::to_string(c.heads) + " heads of " + std::to_string(c.dim));
    const Tensor &positions = want(a[2], "positions", at::kInt, {T});
    const Tensor &slots = want(a[3], "slots", at::kLong, {T});
    const Tensor &table = want_dims(a[4], "cos_sin", at::kFloat, 2);
    const int interleaved = truth(a[9]);
    const Tensor q = output(a[10], "q", at::kBFloat16, {T, Hq, c.dim}, qkv);
    hipStream_t stream = stream_of(a[11]);
    const int64_t max_pos = table.size(0), rot = table.size(1);
    const auto *xp = data<uint16_t>(qkv);
    const auto *pp = data<int32_t>(positions);
    const auto *lp = data<int64_t>(slots);
    const auto *tp = data<float>(table);
    auto *qp = data<uint16_t>(q);
    check(fp8 ? "kv_rope_append_fp8" : "kv_rope_append", unlocked([&] {
            return fp8 ? kv_rope_append_fp8(xp, pp, lp, tp, T, Hq, c.heads, c.dim, rot, interleaved, max_pos, c.pages,
                                            c.page, qp, data<uint8_t>(c.k), data<uint8_t>(c.v), data<float>(c.ks),
                                            data<float>(c.vs), stream)
                       : kv_rope_append(xp, pp, lp, tp, T, Hq, c.heads, c.dim, rot, interleaved, max_pos, c.pages,
                                        c.page, qp, data<uint16_t>(c.k), data<uint16_t>(c.v), stream);
          }));
    return THPVariable_Wrap(q);
  });
}

// (fp8, q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, scale, softcap, window, max_len, return_lse, o,
// lse, stream) -> o or (o, lse); scale and max_len None: D^-0.5 and the table's width
PyObject *paged_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject * {
    const bool fp8 = truth(a[0]), return_lse = truth(a[12]);
    const Cache c = want_cache(a + 2, fp8);
    const Tensor &q = want_dims(a[1], "q", at::kBFloat16, 3);
    const int64_t B = q.size(0), Hq = q.size(1);
    if (q.size(2) != c.dim)
      raise(PyExc_ValueError, "q: expected heads of " + std::to_string(c.dim) + ", got " + text_of(q.sizes()));
    const Tensor &table = want_dims(a[6], "block_table", at::kInt, 2);
    if (table.size(0) != B)
      raise(PyExc_ValueError, "block_table: expected " + std::to_string(B) + " rows, got " + text_of(table.sizes()));
    const Tensor &lens = want(a[7], "seq_lens", at::kInt, {B});
    const int64_t max_pages = table.size(1);
    const float scale = given(a[8]) ? (float)real(a[8]) : (float)(1.0 / std::sqrt((double)c.dim));
    const float softcap = (float)real(a[9]);
    const int64_t window = whole(a[10]), max_len = given(a[11]) ? whole(a[11]) : max_pages * c.page;
    const Tensor o = output(a[13], "o", at::kBFloat16, {B, Hq, c.dim}, q);
    Tensor lse;
    if (return_lse || given(a[14])) lse = output(a[14], "lse", at::kFloat, {B, Hq}, q);
    hipStream_t stream = stream_of(a[15]);
    const auto *qp = data<uint16_t>(q);
    const auto *tp = data<int32_t>(table), *np = data<int32_t>(lens);
    auto *op = data<uint16_t>(o);
    auto *sp = data<float>(lse);
    check(fp8 ? "paged_decode_attention_fp8" : "paged_decode_attention", unlocked([&] {
            return fp8 ? paged_decode_attention_fp8(qp, data<uint8_t>(c.k), data<uint8_t>(c.v), data<float>(c.ks),
                                                    data<float>(c.vs), tp, np, B, Hq, c.heads, c.dim, c.pages, c.page,
                                                    max_pages, max_len, scale, softcap, window, op, sp, stream)
                       : paged_decode_attention(qp, data<uint16_t>(c.k), data<uint16_t>(c.v), tp, np, B, Hq, c.heads,
                                                c.dim, c.pages, c.page, max_pages, max_len, scale, softcap, window, op,
                                                sp, stream);
          }));
    if (!return_lse) return THPVariable_Wrap(o);
    PyObject *out = PyTuple_New(2);
    if (!out) throw Raised{};
    PyTuple_SET_ITEM(out, 0, THPVariable_Wrap(o));
    PyTuple_SET_ITEM(out, 1, THPVariable_Wrap(lse));
    return out;
  });
}

PyObject *set_status_check(PyObject *, PyObject *f) {
  Py_INCREF(f);
  Py_XSETREF(g_status_check, f);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"add_rmsnorm", (PyCFunction)(void (*)())add_rmsnorm, METH_FASTCALL, nullptr},
    {"rope_append", (PyCFunction)(void (*)())rope_append, METH_FASTCALL, nullptr},
    {"paged_decode", (PyCFunction)(void (*)())paged_decode, METH_FASTCALL, nullptr},
    {"set_status_check", set_status_check, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
