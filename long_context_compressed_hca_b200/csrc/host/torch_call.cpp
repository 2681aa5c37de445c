// torch_call.cpp -- the low-bit decode calls from tensors: checks of device,
// type, shape and layout, then the C ABI.
//
// A decode step makes these calls one by one, and at one token a kernel takes
// 2 to 10 us.  The checks in Python through ctypes take 7 to 13 us of host
// time per call (about 1 us per tensor and 2 for the foreign call), here well
// below 1 us beside the launch itself.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "hca.h"

namespace {

PyObject *g_error = nullptr;     // binding.HcaError

struct Bad {
  int code;
  std::string msg;
};
struct PyFailed {};              // a Python exception is set
[[noreturn]] void bad(const std::string &msg) { throw Bad{HCA_ERR_INVALID, msg}; }

std::string type_name(c10::ScalarType t) {
  switch (t) {
    case c10::kFloat: return "torch.float32";
    case c10::kBFloat16: return "torch.bfloat16";
    case c10::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
    case c10::kByte: return "torch.uint8";
    case c10::kInt: return "torch.int32";
    case c10::kLong: return "torch.int64";
    default: return c10::toString(t);
  }
}
std::string shape_name(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

// The element types an argument may have, the usual one first.
struct Types {
  c10::ScalarType a, b;
  int n;
};
constexpr Types kF32{c10::kFloat, c10::kFloat, 1}, kBF16{c10::kBFloat16, c10::kBFloat16, 1},
    kF32orBF16{c10::kFloat, c10::kBFloat16, 2}, kU8{c10::kByte, c10::kByte, 1}, kI32{c10::kInt, c10::kInt, 1},
    kI64{c10::kLong, c10::kLong, 1}, kE4M3{c10::kFloat8_e4m3fn, c10::kByte, 2}, kNone{c10::kFloat, c10::kFloat, 0};
Types types_of(hca_dtype d) {
  return d == HCA_F32 ? kF32 : d == HCA_BF16 ? kBF16 : d == HCA_FP8E4M3 ? kE4M3 : kNone;
}
hca_dtype code_of(const at::Tensor &t) { return t.scalar_type() == c10::kFloat ? HCA_F32 : HCA_BF16; }

const at::Tensor &tensor(const char *name, PyObject *o) {
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}
// The current device, which has to be the one of t.
int device_of(const at::Tensor &t) {
  if (!t.is_cuda()) bad("tensors must be on the current CUDA device (one is on the host)");
  return c10::cuda::current_device();
}
// Address of a tensor, which is on device dev, of one of the types and the
// shape; dense, or with rows ld elements apart.
const void *take(const char *name, const at::Tensor &t, c10::IntArrayRef shape, Types ty, int dev, int64_t ld = 0) {
  const std::string n(name);
  if (!t.is_cuda() || t.get_device() != dev) bad(n + " must be on the current CUDA device (it is on " + t.device().str() + ")");
  const c10::ScalarType st = t.scalar_type();
  if (!ty.n || (st != ty.a && st != ty.b))
    bad(n + " has dtype " + type_name(st) + ", expected " + (ty.n ? type_name(ty.a) : "another"));
  if (t.sizes() != shape) bad(n + " has shape " + shape_name(t.sizes()) + ", expected " + shape_name(shape));
  const bool ok = !ld ? t.is_contiguous()
                      : (shape[1] == 1 || t.stride(1) == 1) && (shape[0] <= 1 || t.stride(0) == ld);
  if (!ok) bad(n + (ld ? " must have contiguous rows " + std::to_string(ld) + " elements apart" : " must be contiguous"));
  return t.const_data_ptr();
}
const void *take(const char *name, PyObject *o, c10::IntArrayRef shape, Types ty, int dev, int64_t ld = 0) {
  return take(name, tensor(name, o), shape, ty, dev, ld);
}
// The same of an argument that may be None.
const void *take_or_null(const char *name, PyObject *o, c10::IntArrayRef shape, Types ty, int dev, int64_t ld = 0) {
  return o == Py_None ? nullptr : take(name, o, shape, ty, dev, ld);
}
// Address of a tensor that the call writes: a lazy clone gets memory of its own
// first.  Asked for before the inputs', one of which may be the same tensor.
void *take_out(const char *name, const at::Tensor &t, c10::IntArrayRef shape, Types ty, int dev, int64_t ld = 0) {
  take(name, t, shape, ty, dev, ld);
  return t.mutable_data_ptr();
}
void *take_out(const char *name, PyObject *o, c10::IntArrayRef shape, Types ty, int dev, int64_t ld = 0) {
  return take_out(name, tensor(name, o), shape, ty, dev, ld);
}
struct Scratch {
  void *p = nullptr;
  size_t n = 0;
};
Scratch scratch(PyObject *o, int dev) {
  Scratch s;
  if (o == Py_None) return s;
  const at::Tensor &t = tensor("ws", o);
  s.p = take_out("ws", t, t.sizes(), Types{t.scalar_type(), t.scalar_type(), 1}, dev);
  s.n = t.numel() * t.element_size();
  return s;
}

// A ctypes structure as the C ABI's.
template <typename T>
struct Desc {
  Py_buffer b{};
  Desc(const char *name, PyObject *o) {
    if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) throw PyFailed{};
    if (b.len != (Py_ssize_t)sizeof(T)) {
      PyBuffer_Release(&b);
      bad(std::string(name) + " is of another type");
    }
  }
  ~Desc() { PyBuffer_Release(&b); }
  Desc(const Desc &) = delete;
  const T *get() const { return static_cast<const T *>(b.buf); }
  const T *operator->() const { return get(); }
};
long long integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFailed{};
  return v;
}
int int32(const char *name, PyObject *o) {
  const long long v = integer(o);
  if (v != (int)v) bad(std::string(name) + " does not fit 32 bits");
  return (int)v;
}
void *stream_of(PyObject *o) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
  PyObject *h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw PyFailed{};
  void *s = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!s && PyErr_Occurred()) throw PyFailed{};
  return s;
}

// Runs f, which makes a C ABI call and returns its status; a status other than
// HCA_OK and a refusal become HcaError(code, message).
template <typename F>
PyObject *call(Py_ssize_t given, Py_ssize_t want, F f) {
  int code = HCA_OK;
  std::string msg;
  try {
    if (given != want) bad("expected " + std::to_string(want) + " arguments, got " + std::to_string(given));
    code = f();
    if (code == HCA_OK) return PyLong_FromLong(HCA_OK);
    msg = hca_last_error();
  } catch (const PyFailed &) {
    return nullptr;
  } catch (const Bad &b) {
    code = b.code;
    msg = b.msg;
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
  PyObject *args = Py_BuildValue("(is)", code, msg.c_str());
  if (args) PyErr_SetObject(g_error, args);
  Py_XDECREF(args);
  return nullptr;
}
template <typename F>
int unlocked(F f) {              // without the interpreter's lock
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return rc;
}

// (desc, x, res, gamma, res_out, out, out_scale, stream)
PyObject *add_rms_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 8, [&] {
    const Desc<hca_norm_desc> d("desc", a[0]);
    const at::Tensor &x = tensor("x", a[1]);
    const int dev = device_of(x);
    const int64_t shape[2] = {d->rows, d->d}, row[1] = {d->d};
    const Types rt = types_of(d->res_dtype);
    void *pro = a[4] == Py_None ? nullptr : take_out("res_out", a[4], shape, rt, dev, d->ldr);
    const void *px = take("x", x, shape, types_of(d->x_dtype), dev, d->ldx);
    const void *pr = take_or_null("res", a[2], shape, rt, dev, d->ldr);
    const void *pg = take_or_null("gamma", a[3], row, kF32, dev);
    void *po = take_out("out", a[5], shape, types_of(d->out_dtype), dev, d->ldo);
    void *ps = nullptr;
    if (d->out_dtype == HCA_FP8E4M3) {
      if (a[6] == Py_None) bad("an e4m3 output needs out_scale");
      const int64_t ss[2] = {d->rows, d->scale_group > 0 ? d->d / d->scale_group : 1};
      ps = take_out("out_scale", a[6], ss, kF32, dev);
    }
    void *s = stream_of(a[7]);
    return unlocked([&] {
      return hca_add_rms_norm(d.get(), px, pr, static_cast<const float *>(pg), pro, po, static_cast<float *>(ps), s);
    });
  });
}

// (desc, x, x_scale, codes, scales, row_scale, out, ws, stream)
PyObject *w4_linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 9, [&] {
    const Desc<hca_w4_desc> d("desc", a[0]);
    const at::Tensor &x = tensor("x", a[1]);
    const int dev = device_of(x);
    const int64_t T = d->T, N = d->N, K = d->K, g = d->groups, G = d->scale_group > 0 ? d->scale_group : 1;
    const int64_t sx[2] = {T, g * K}, st[1] = {T}, st1[2] = {T, 1}, sc[2] = {g * N, K / 2}, sr[1] = {g * N},
                  ss[3] = {g, K / G, (N + 15) / 16 * 16}, so[2] = {T, g * N};
    const void *px = take("x", x, sx, types_of(d->x_dtype), dev, d->ldx);
    const void *ps = nullptr;
    if (a[2] != Py_None) {       // [T], or [T, 1] as add_rms_norm writes them
      const at::Tensor &t = tensor("x_scale", a[2]);
      ps = t.dim() == 2 ? take("x_scale", t, st1, kF32, dev) : take("x_scale", t, st, kF32, dev);
    }
    const void *pc = take("codes", a[3], sc, kU8, dev);
    const void *pw = take("scales", a[4], ss, kE4M3, dev);
    const void *pr = take("row_scale", a[5], sr, kF32, dev);
    void *po = take_out("out", a[6], so, types_of(d->out_dtype), dev, d->ldo);
    const Scratch ws = scratch(a[7], dev);
    void *s = stream_of(a[8]);
    return unlocked([&] {
      return hca_w4_linear(d.get(), px, static_cast<const float *>(ps), pc, pw, static_cast<const float *>(pr), po, ws.p,
                           ws.n, s);
    });
  });
}

// Number of the records in t [.., record bytes].
int64_t records(const char *name, const at::Tensor &t, int c, int rd) {
  const int64_t rec = (int64_t)hca_kv_fp4_row_bytes(c, rd);
  if (rec == 0) bad("unsupported (c, rd) = (" + std::to_string(c) + ", " + std::to_string(rd) + ")");
  if (t.dim() == 0 || t.size(-1) != rec) {
    bad(std::string(name) + " has shape " + shape_name(t.sizes()) + ", expected records of " + std::to_string(rec) + " bytes");
  }
  return t.numel() / rec;
}

// (x, c, rd, records, slots, stream)
PyObject *kv_quant_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 6, [&] {
    const at::Tensor &x = tensor("x", a[0]), &r = tensor("records", a[3]);
    const int c = int32("c", a[1]), rd = int32("rd", a[2]), dev = device_of(x);
    const int64_t nrec = records("records", r, c, rd);
    void *po = take_out("records", r, r.sizes(), kU8, dev);
    const int64_t rows = x.dim() ? x.size(0) : 0, sx[2] = {rows, c}, sr[1] = {rows};
    const void *px = take("x", x, sx, kF32orBF16, dev);
    const void *ps = take_or_null("slots", a[4], sr, kI64, dev);
    void *s = stream_of(a[5]);
    return unlocked([&] {
      return hca_kv_quant_fp4(px, code_of(x), rows, c, rd, po, nrec, static_cast<const long long *>(ps), s);
    });
  });
}

// (records, c, rd, out, slots, stream)
PyObject *kv_dequant_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 6, [&] {
    const at::Tensor &r = tensor("records", a[0]), &out = tensor("out", a[3]);
    const int c = int32("c", a[1]), rd = int32("rd", a[2]), dev = device_of(out);
    const int64_t nrec = records("records", r, c, rd);
    const void *pi = take("records", r, r.sizes(), kU8, dev);
    const int64_t rows = out.dim() ? out.size(0) : 0, so[2] = {rows, c}, sr[1] = {rows};
    void *po = take_out("out", out, so, kBF16, dev);
    const void *ps = take_or_null("slots", a[4], sr, kI64, dev);
    void *s = stream_of(a[5]);
    return unlocked([&] {
      return hca_kv_dequant_fp4(pi, nrec, static_cast<const long long *>(ps), rows, c, rd, po, s);
    });
  });
}

// (desc, q, cache struct, cache rows, pages, idx, kv_win, sink, positions, max_pos, o, ws, stream)
PyObject *attend_fp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return call(n, 13, [&] {
    const Desc<hca_attn_desc> d("desc", a[0]);
    const Desc<hca_fp4_cache> cache("cache", a[2]);
    const at::Tensor &q = tensor("q", a[1]), &rows = tensor("cache rows", a[3]);
    const int dev = device_of(q);
    const int64_t B = d->B, c = d->c, sq[3] = {B, d->n_h, c}, si[2] = {B, d->k}, sw[3] = {B, d->w > 0 ? d->w : 1, c},
                  sh[1] = {d->n_h}, sb[1] = {B}, sp[2] = {B, cache->max_pages};
    const void *pq = take("q", q, sq, kBF16, dev);
    void *po = take_out("o", a[10], sq, kBF16, dev);
    const int64_t nrec = records("cache rows", rows, d->c, d->rd);
    const void *pr = take("cache rows", rows, rows.sizes(), kU8, dev);
    const void *pg = take_or_null("pages", a[4], sp, kI32, dev);
    if (pr != cache->rows || pg != static_cast<const void *>(cache->pages))
      bad("the cache's tensors have moved since fp4_cache made it");
    if (cache->cap > 0 && nrec != (int64_t)cache->n_pages * cache->cap)
      bad("the cache has " + std::to_string(nrec) + " records, " + std::to_string((int64_t)cache->n_pages * cache->cap) +
          " when fp4_cache made it");
    if (a[4] == Py_None && rows.size(0) != B)
      bad("the cache has " + std::to_string(rows.size(0)) + " sequences, expected " + std::to_string(B));
    const void *pi = take_or_null("idx", a[5], si, kI32, dev);
    const void *pk = take_or_null("kv_win", a[6], sw, kBF16, dev);
    const void *ps = take_or_null("sink", a[7], sh, kF32, dev);
    const void *pp = take("positions", a[8], sb, kI32, dev);
    const int max_pos = int32("max_pos", a[9]);
    const Scratch ws = scratch(a[11], dev);
    void *s = stream_of(a[12]);
    return unlocked([&] {
      return hca_attend_fp4(d.get(), pq, cache.get(), static_cast<const int32_t *>(pi), pk, static_cast<const float *>(ps),
                            static_cast<const int32_t *>(pp), max_pos, po, ws.p, ws.n, s);
    });
  });
}

// The class of the errors that the calls raise.
PyObject *set_error(PyObject *, PyObject *cls) {
  Py_INCREF(cls);
  Py_XDECREF(g_error);
  g_error = cls;
  Py_RETURN_NONE;
}

#define CALL(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {CALL(add_rms_norm), CALL(w4_linear), CALL(kv_quant_fp4), CALL(kv_dequant_fp4), CALL(attend_fp4),
                           {"set_error", set_error, METH_O, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_call", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_call() { return PyModule_Create(&g_module); }
