// Host path of quantize_grouped_gemm_amd.lm: checks, output allocation and
// the call of the C ABI (include/mxlm.h) for the ordinary case, in one C++
// function per operator. A small call's kernels take 3 to 10 us; the host's part of
// the call takes 4 to 6 us here with one launch and 10 with two, and 11 to 21 with
// the same steps in Python.
//
// Every function returns the dict of outputs, an int (the status of a call
// that the library refused), or None where the arguments are anything but
// ordinary; lm then goes through its own checks, which say what is wrong.

#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/mxlm.h"

namespace {

using at::Tensor;

constexpr auto kBF = at::kBFloat16;
constexpr auto kF32 = at::kFloat;
constexpr auto kU8 = at::kByte;

PyObject *kSum, *kRstd, *kQRow, *kSRow, *kQCol, *kSCol, *kQCk, *kSCk, *kDx, *kDw, *kLogp, *kEntropy, *kStats, *kTopLogp,
    *kTopIdx, *kRceil, *kFloor, *kK128, *kPlain;

// The current device if o is a device tensor, else -1 (without asking a
// runtime that may find no device).
int device_for(PyObject* o) {
  return THPVariable_CheckExact(o) && THPVariable_Unpack(o).is_cuda() ? c10::hip::current_device() : -1;
}

// A tensor argument, or nullptr if it is not a tensor on the current device.
const Tensor* tensor(PyObject* o, int dev) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.get_device() != dev) return nullptr;
  return &t;
}

bool whole(const Tensor* t, at::ScalarType ty, std::initializer_list<int64_t> shape) {
  return t && t->scalar_type() == ty && t->sizes() == at::IntArrayRef(shape) && t->is_contiguous();
}

// Row stride of a matrix of contiguous rows, or -1. Strides that no second row
// or column makes use of do not matter.
int64_t rows_ld(const Tensor* t, at::ScalarType ty, int64_t R, int64_t C) {
  if (!t || t->scalar_type() != ty || t->dim() != 2 || t->size(0) != R || t->size(1) != C ||
      (C > 1 && t->stride(1) != 1) || (R > 1 && t->stride(0) < C))
    return -1;
  return R > 1 ? t->stride(0) : C;
}

struct Format {
  mx_scale_mode mode;
  mx_scale_layout layout;
  int64_t step;
  bool ok;
};

bool same(PyObject* s, PyObject* interned) {
  return s == interned || (PyUnicode_Check(s) && PyUnicode_Compare(s, interned) == 0);
}

Format format(PyObject* mode, PyObject* layout) {
  Format f{MX_RCEIL, MX_SCALES_K128, 128, true};
  if (same(mode, kFloor)) f.mode = MX_FLOOR;
  else if (!same(mode, kRceil)) f.ok = false;
  if (same(layout, kPlain)) {
    f.layout = MX_SCALES_PLAIN;
    f.step = 32;
  } else if (!same(layout, kK128)) {
    f.ok = false;
  }
  return f;
}

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

// The dict of outputs under construction.
struct Out {
  PyObject* d;
  at::Device device;
  explicit Out(int dev) : d(PyDict_New()), device(at::kCUDA, (c10::DeviceIndex)dev) {}
  ~Out() { Py_XDECREF(d); }
  void* add(PyObject* key, at::IntArrayRef shape, at::ScalarType ty) {
    Tensor t(at::detail::empty_cuda(shape, ty, device, std::nullopt));
    void* p = t.data_ptr();
    PyObject* o = THPVariable_Wrap(std::move(t));
    PyDict_SetItem(d, key, o);
    Py_DECREF(o);
    return p;
  }
  struct Codes {
    uint8_t *q = nullptr, *s = nullptr;
  };
  // Codes and scales always go together, so they share one allocation: the
  // scales 256-byte aligned behind the codes.
  Codes codes(PyObject* q, PyObject* s, int64_t R, int64_t C, const Format& f) {
    const int64_t at = up(R * C, 256);
    const Tensor base(at::detail::empty_cuda({at + R * C / 32}, kU8, device, std::nullopt));
    uint8_t* p = static_cast<uint8_t*>(base.data_ptr());
    part(q, base, 0, {R, C});
    if (f.layout == MX_SCALES_K128) part(s, base, at, {C / 128, R, 4});
    else part(s, base, at, {R, C / 32});
    return Codes{p, p + at};
  }
  // Small outputs of one lifetime share one allocation as well, 16-byte aligned.
  struct Shared {
    Tensor base;
    int64_t at = 0;
  };
  Shared shared(int64_t bytes) { return Shared{Tensor(at::detail::empty_cuda({bytes}, kU8, device, std::nullopt))}; }
  void* add(Shared& s, PyObject* key, at::IntArrayRef shape, at::ScalarType ty) {   // 4-byte types
    void* p = static_cast<char*>(s.base.data_ptr()) + s.at;
    int64_t n = 1;
    for (int64_t d : shape) n *= d;
    part(key, s.base, s.at / 4, shape, c10::scalarTypeToTypeMeta(ty));
    s.at += up(4 * n, 16);
    return p;
  }
  void part(PyObject* key, const Tensor& base, int64_t offset, at::IntArrayRef shape,
            caffe2::TypeMeta ty = c10::scalarTypeToTypeMeta(kU8)) {
    Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(), ty);
    t.unsafeGetTensorImpl()->set_storage_offset(offset);
    t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
    PyObject* o = THPVariable_Wrap(std::move(t));
    PyDict_SetItem(d, key, o);
    Py_DECREF(o);
  }
  PyObject* done(mx_status st) {
    if (st != MX_OK) return PyLong_FromLong(st);
    PyObject* r = d;
    d = nullptr;
    return r;
  }
};

void* stream(int dev) { return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream(); }

#define NOT_ORDINARY(cond) \
  if (cond) Py_RETURN_NONE

// Runs f, turning C++ exceptions (an allocation that failed) into torch's
// Python ones.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// x, w, r, eps, mode, layout, colwise, checkpoint
PyObject* add_rmsnorm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    NOT_ORDINARY(n != 8);
    const int dev = device_for(a[0]);
    NOT_ORDINARY(dev < 0);
    const Tensor *x = tensor(a[0], dev), *w = tensor(a[1], dev), *r = a[2] == Py_None ? nullptr : tensor(a[2], dev);
    const Format f = format(a[4], a[5]);
    NOT_ORDINARY(!x || x->dim() != 2 || !f.ok || (a[2] != Py_None && !r) || !PyFloat_CheckExact(a[3]) ||
                 !PyBool_Check(a[6]) || !PyBool_Check(a[7]));
    const int64_t T = x->size(0), C = x->size(1);
    const int64_t ld = rows_ld(x, kBF, T, C), ld_r = r ? rows_ld(r, kBF, T, C) : 0;
    NOT_ORDINARY(ld < 0 || ld_r < 0 || !whole(w, kF32, {C}) || C <= 0 || C % f.step || C > 16384);
    Out out(dev);
    void* sum = r ? out.add(kSum, {T, C}, kBF) : nullptr;
    float* rstd = static_cast<float*>(out.add(kRstd, {T}, kF32));
    const Out::Codes row = out.codes(kQRow, kSRow, T, C, f);
    Out::Codes col, ck;
    if (a[6] == Py_True) col = out.codes(kQCol, kSCol, C, up(T, f.step), f);
    if (a[7] == Py_True) ck = out.codes(kQCk, kSCk, T, C, f);
    return out.done(mx_add_rmsnorm_quant(x->data_ptr(), ld, r ? r->data_ptr() : nullptr, ld_r,
                                         static_cast<const float*>(w->data_ptr()), T, C, (float)PyFloat_AS_DOUBLE(a[3]),
                                         f.mode, f.layout, sum, rstd, row.q, row.s, col.q, col.s, ck.q, ck.s, stream(dev)));
  });
}

// dy, w, rstd, x, q_ck, s_ck, dsum, mode, layout, rowwise, colwise
PyObject* add_rmsnorm_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    NOT_ORDINARY(n != 11);
    const int dev = device_for(a[0]);
    NOT_ORDINARY(dev < 0);
    const Tensor *dy = tensor(a[0], dev), *w = tensor(a[1], dev), *rstd = tensor(a[2], dev);
    const Tensor *x = nullptr, *q = nullptr, *s = nullptr, *ds = nullptr;
    const Format f = format(a[7], a[8]);
    NOT_ORDINARY(!dy || dy->dim() != 2 || !f.ok || !PyBool_Check(a[9]) || !PyBool_Check(a[10]));
    NOT_ORDINARY((a[3] == Py_None) == (a[4] == Py_None));
    const int64_t T = dy->size(0), C = dy->size(1);
    const int64_t ld = rows_ld(dy, kBF, T, C);
    int64_t ld_x = 0, ld_s = 0;
    if (a[3] != Py_None) {
      x = tensor(a[3], dev);
      ld_x = rows_ld(x, kBF, T, C);
    } else {
      q = tensor(a[4], dev);
      s = tensor(a[5], dev);
      NOT_ORDINARY(!whole(q, kU8, {T, C}));
      NOT_ORDINARY(f.layout == MX_SCALES_K128 ? !whole(s, kU8, {C / 128, T, 4}) : !whole(s, kU8, {T, C / 32}));
    }
    if (a[6] != Py_None) {
      ds = tensor(a[6], dev);
      ld_s = rows_ld(ds, kBF, T, C);
    }
    NOT_ORDINARY(ld < 0 || ld_x < 0 || ld_s < 0 || !whole(w, kF32, {C}) || !whole(rstd, kF32, {T}) || C <= 0 ||
                 C % f.step || C > 16384);
    Out out(dev);
    void* dx = out.add(kDx, {T, C}, kBF);
    float* dw = static_cast<float*>(out.add(kDw, {C}, kF32));
    Out::Codes row, col;
    if (a[9] == Py_True) row = out.codes(kQRow, kSRow, T, C, f);
    if (a[10] == Py_True) col = out.codes(kQCol, kSCol, C, up(T, f.step), f);
    const Tensor work(at::detail::empty_cuda({mx_add_rmsnorm_bwd_work(T, C)}, kF32, out.device, std::nullopt));
    return out.done(mx_add_rmsnorm_bwd(
        dy->data_ptr(), ld, static_cast<const float*>(w->data_ptr()), static_cast<const float*>(rstd->data_ptr()),
        x ? x->data_ptr() : nullptr, ld_x, q ? static_cast<const uint8_t*>(q->data_ptr()) : nullptr,
        s ? static_cast<const uint8_t*>(s->data_ptr()) : nullptr, ds ? ds->data_ptr() : nullptr, ld_s, T, C, f.mode,
        f.layout, dx, dw, row.q, row.s, col.q, col.s, static_cast<float*>(work.data_ptr()), stream(dev)));
  });
}

// a, b, mode, layout
PyObject* swiglu_ckpt_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    NOT_ORDINARY(n != 4);
    const int dev = device_for(a[0]);
    NOT_ORDINARY(dev < 0);
    const Tensor *p = tensor(a[0], dev), *b = tensor(a[1], dev);
    const Format f = format(a[2], a[3]);
    NOT_ORDINARY(!p || !b || p->dim() != 2 || !f.ok);
    const int64_t T = p->size(0), H = p->size(1);
    const int64_t ld = rows_ld(p, kBF, T, H);
    NOT_ORDINARY(ld < 0 || rows_ld(b, kBF, T, H) != ld || H <= 0 || H % f.step);
    Out out(dev);
    const Out::Codes row = out.codes(kQRow, kSRow, T, H, f), col = out.codes(kQCol, kSCol, H, up(T, f.step), f),
                     ck = out.codes(kQCk, kSCk, T, 2 * H, f);
    return out.done(mx_swiglu_ckpt_fwd(p->data_ptr(), b->data_ptr(), ld, T, H, f.mode, f.layout, row.q, row.s, col.q,
                                       col.s, ck.q, ck.s, stream(dev)));
  });
}

// dh, q_ck, s_ck, mode, layout
PyObject* swiglu_ckpt_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    NOT_ORDINARY(n != 5);
    const int dev = device_for(a[0]);
    NOT_ORDINARY(dev < 0);
    const Tensor *dh = tensor(a[0], dev), *q = tensor(a[1], dev), *s = tensor(a[2], dev);
    const Format f = format(a[3], a[4]);
    NOT_ORDINARY(!dh || dh->dim() != 2 || !f.ok);
    const int64_t T = dh->size(0), H = dh->size(1);
    const int64_t ld = rows_ld(dh, kBF, T, H);
    NOT_ORDINARY(ld < 0 || H <= 0 || H % f.step || !whole(q, kU8, {T, 2 * H}));
    NOT_ORDINARY(f.layout == MX_SCALES_K128 ? !whole(s, kU8, {2 * H / 128, T, 4}) : !whole(s, kU8, {T, 2 * H / 32}));
    Out out(dev);
    const Out::Codes row = out.codes(kQRow, kSRow, T, 2 * H, f), col = out.codes(kQCol, kSCol, 2 * H, up(T, f.step), f);
    return out.done(mx_swiglu_ckpt_bwd(dh->data_ptr(), ld, static_cast<const uint8_t*>(q->data_ptr()),
                                       static_cast<const uint8_t*>(s->data_ptr()), T, H, f.mode, f.layout, row.q, row.s,
                                       col.q, col.s, stream(dev)));
  });
}

// Logits: bf16 or float32 [T, V] with its targets; false if not ordinary.
struct Logits {
  const Tensor *x, *t;
  int64_t T, V, ld, ignore;
  float scale;
  mx_dtype dt;
};

bool logits(Logits& l, PyObject* x, PyObject* t, PyObject* scale, PyObject* ignore, int dev) {
  l.x = tensor(x, dev);
  l.t = tensor(t, dev);
  if (!l.x || !l.t || l.x->dim() != 2 || !PyFloat_CheckExact(scale) || !PyLong_CheckExact(ignore)) return false;
  const double s = PyFloat_AS_DOUBLE(scale);
  int overflow = 0;
  l.ignore = PyLong_AsLongLongAndOverflow(ignore, &overflow);
  if (overflow || !(s >= 1e-6 && s <= 1e6)) return false;
  l.scale = (float)s;
  l.T = l.x->size(0);
  l.V = l.x->size(1);
  const auto ty = l.x->scalar_type();
  if (ty != kBF && ty != kF32) return false;
  l.dt = ty == kF32 ? MX_F32 : MX_BF16;
  l.ld = rows_ld(l.x, ty, l.T, l.V);
  return l.ld >= 0 && l.V >= 1 && whole(l.t, at::kLong, {l.T});
}

// x, targets, scale, top, ignore_index
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    NOT_ORDINARY(n != 5);
    const int dev = device_for(a[0]);
    NOT_ORDINARY(dev < 0);
    Logits l;
    NOT_ORDINARY(!logits(l, a[0], a[1], a[2], a[4], dev) || !PyLong_CheckExact(a[3]));
    int overflow = 0;
    const int64_t top = PyLong_AsLongLongAndOverflow(a[3], &overflow);
    NOT_ORDINARY(overflow || top < 0 || top > 64 || top > l.V);
    Out out(dev);
    Out::Shared sh = out.shared(2 * up(4 * l.T, 16) + up(8 * l.T, 16) + 2 * up(4 * l.T * top, 16));
    float* logp = static_cast<float*>(out.add(sh, kLogp, {l.T}, kF32));
    float* ent = static_cast<float*>(out.add(sh, kEntropy, {l.T}, kF32));
    float* stats = static_cast<float*>(out.add(sh, kStats, {l.T, 2}, kF32));
    float* tl = top ? static_cast<float*>(out.add(sh, kTopLogp, {l.T, top}, kF32)) : nullptr;
    int32_t* ti = top ? static_cast<int32_t*>(out.add(sh, kTopIdx, {l.T, top}, at::kInt)) : nullptr;
    const int64_t bytes = mx_token_logprobs_work(l.T, l.V, (int32_t)top);
    Tensor work;
    if (bytes) work = Tensor(at::detail::empty_cuda({bytes}, kU8, out.device, std::nullopt));
    return out.done(mx_token_logprobs(l.x->data_ptr(), l.dt, l.ld, l.T, l.V, static_cast<const int64_t*>(l.t->data_ptr()),
                                      l.ignore, l.scale, (int32_t)top, logp, ent, stats, tl, ti,
                                      bytes ? work.data_ptr() : nullptr, nullptr, stream(dev)));
  });
}

// x, targets, stats, entropy, dlogp, dent, scale, mode, layout, ignore_index
PyObject* token_logprobs_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    NOT_ORDINARY(n != 10);
    const int dev = device_for(a[0]);
    NOT_ORDINARY(dev < 0);
    Logits l;
    const Format f = format(a[7], a[8]);
    NOT_ORDINARY(!f.ok || !logits(l, a[0], a[1], a[6], a[9], dev));
    const Tensor *stats = tensor(a[2], dev), *ent = tensor(a[3], dev), *dl = nullptr, *de = nullptr;
    NOT_ORDINARY(!whole(stats, kF32, {l.T, 2}) || !whole(ent, kF32, {l.T}));
    if (a[4] != Py_None) {
      dl = tensor(a[4], dev);
      NOT_ORDINARY(!whole(dl, kF32, {l.T}));
    }
    if (a[5] != Py_None) {
      de = tensor(a[5], dev);
      NOT_ORDINARY(!whole(de, kF32, {l.T}));
    }
    const int64_t Vp = up(l.V, f.step);
    Out out(dev);
    const Out::Codes row = out.codes(kQRow, kSRow, l.T, Vp, f), col = out.codes(kQCol, kSCol, Vp, up(l.T, f.step), f);
    auto fp = [](const Tensor* t) { return t ? static_cast<const float*>(t->data_ptr()) : nullptr; };
    return out.done(mx_token_logprobs_bwd(l.x->data_ptr(), l.dt, l.ld, l.T, l.V,
                                          static_cast<const int64_t*>(l.t->data_ptr()), l.ignore, fp(stats), fp(ent),
                                          fp(dl), fp(de), l.scale, f.mode, f.layout, row.q, row.s, col.q, col.s, nullptr,
                                          stream(dev)));
  });
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {METHOD(add_rmsnorm_quant),  METHOD(add_rmsnorm_bwd), METHOD(swiglu_ckpt_fwd),
                          METHOD(swiglu_ckpt_bwd),    METHOD(token_logprobs),  METHOD(token_logprobs_bwd),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_lmhost", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__lmhost() {
  auto key = [](PyObject*& slot, const char* s) { slot = PyUnicode_InternFromString(s); };
  key(kSum, "sum"); key(kRstd, "rstd");
  key(kQRow, "q_row"); key(kSRow, "s_row"); key(kQCol, "q_col"); key(kSCol, "s_col"); key(kQCk, "q_ck"); key(kSCk, "s_ck");
  key(kDx, "dx"); key(kDw, "dw");
  key(kLogp, "logp"); key(kEntropy, "entropy"); key(kStats, "stats"); key(kTopLogp, "top_logp"); key(kTopIdx, "top_idx");
  key(kRceil, "rceil"); key(kFloor, "floor"); key(kK128, "k128"); key(kPlain, "plain");
  return PyModule_Create(&kModule);
}
