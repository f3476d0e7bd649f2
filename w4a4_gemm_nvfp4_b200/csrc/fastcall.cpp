// fastcall.cpp -- the host path of the calls whose host time counts.
//
// A decode step's kernels take a few microseconds, and the checks and argument
// marshalling of a call cost as much in Python (gemv: 8.0 us a call there, 3.8
// here, of which the launch is 2.3; gemm_gated 11.4 and 5.4).  Each function
// below does in one step what the wrapper of the same name in _lib.py does for
// the common call (buffers on the current device, the current stream, nothing
// out of order) and returns None for every other call, which the wrapper then
// takes itself, with its detailed checks and errors.  Nothing is computed here:
// the work is the same entry point of libnvfp4.so.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include "nvfp4.h"

namespace {

PyObject *s_codes, *s_scales, *s_global_scale, *s_rows, *s_K;  // attribute names
PyObject *d_bf16, *d_f32;                                      // torch dtypes

// A plain torch.Tensor's at::Tensor, or null (another type, a subclass).
const at::Tensor* tensor(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}

bool integer(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// An owned attribute, released at the end of the scope.
struct Attr {
  PyObject* o;
  Attr(PyObject* of, PyObject* name) : o(PyObject_GetAttr(of, name)) {
    if (!o) PyErr_Clear();
  }
  ~Attr() { Py_XDECREF(o); }
  Attr(const Attr&) = delete;
  Attr& operator=(const Attr&) = delete;
};

// A [rows, cols] matrix of `type` on the current device with unit column stride
// and rows that do not overlap; its row pitch.
bool matrix(const at::Tensor& t, at::ScalarType type, int device, int64_t* pitch) {
  if (!t.is_cuda() || t.scalar_type() != type || t.dim() != 2 || t.get_device() != device ||
      t.layout() != at::kStrided)
    return false;
  const int64_t rows = t.size(0), cols = t.size(1);
  *pitch = rows == 1 ? cols : t.stride(0);
  return (t.stride(1) == 1 || cols <= 1) && *pitch >= cols;
}

bool buffer(PyObject* o, at::ScalarType type, int device, int64_t numel, void** p) {
  const at::Tensor* t = o ? tensor(o) : nullptr;
  if (!t || !t->is_cuda() || t->scalar_type() != type || t->get_device() != device || !t->is_contiguous() ||
      t->numel() < numel)
    return false;
  *p = t->data_ptr();
  return true;
}

struct Operand {
  int64_t rows, K;
  void *codes, *scales, *alpha;
};

// An NVFP4Tensor with buffers as large as its sizes ask for.
bool operand(PyObject* q, int device, Operand* w) {
  const Attr rows(q, s_rows), K(q, s_K);
  if (!rows.o || !K.o || !integer(rows.o, &w->rows) || !integer(K.o, &w->K) || w->rows < 1 || w->K < 1 ||
      w->rows > (1ll << 30) || w->K > (1ll << 30))
    return false;
  const Attr codes(q, s_codes), scales(q, s_scales), alpha(q, s_global_scale);
  return buffer(codes.o, at::kByte, device, w->rows * (w->K / 2), &w->codes) &&
         buffer(scales.o, at::kByte, device, (w->rows + 127) / 128 * 128 * (w->K / 16), &w->scales) &&
         buffer(alpha.o, at::kFloat, device, 1, &w->alpha);
}

// The output: `out` when it is given and fits, else a new [M, N] of the type.
bool output(PyObject* out, PyObject* type, int64_t M, int64_t N, const at::Tensor& like, int device, at::Tensor* t,
            int64_t* pitch, int* code) {
  if (out != Py_None) {
    const at::Tensor* o = tensor(out);
    if (!o) return false;
    const at::ScalarType st = o->scalar_type();
    if (type != Py_None && type != (st == at::kFloat ? d_f32 : d_bf16)) return false;
    if (st != at::kFloat && st != at::kBFloat16) return false;
    if (!matrix(*o, st, device, pitch) || o->size(0) != M || o->size(1) != N) return false;
    *code = st == at::kFloat ? NVFP4_OUT_FP32 : NVFP4_OUT_BF16;
    *t = *o;
    return true;
  }
  const bool fp32 = type == d_f32;
  if (!fp32 && type != Py_None && type != d_bf16) return false;
  *t = at::empty({M, N}, like.options().dtype(fp32 ? at::kFloat : at::kBFloat16));
  *pitch = N;
  *code = fp32 ? NVFP4_OUT_FP32 : NVFP4_OUT_BF16;
  return true;
}

// `out` itself when it was given, else the new tensor.
PyObject* give(PyObject* out, const at::Tensor& t) {
  if (out != Py_None) return Py_NewRef(out);
  return THPVariable_Wrap(t);
}

void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

// No C++ exception leaves a function: the wrapper meets the same error itself.
template <typename F>
PyObject* guarded(F f) {
  try {
    PyObject* r = f();
    if (r) return r;
  } catch (...) {
  }
  PyErr_Clear();
  Py_RETURN_NONE;
}

// gemv(x, w, out_dtype, out)
PyObject* gemv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 4) return nullptr;
    const at::Tensor* x = tensor(a[0]);
    const int device = c10::cuda::current_device();
    int64_t ldx, ldy;
    int code;
    Operand w;
    if (!x || !matrix(*x, at::kBFloat16, device, &ldx) || !operand(a[1], device, &w) || x->size(1) != w.K)
      return nullptr;
    at::Tensor y;
    if (!output(a[3], a[2], x->size(0), w.rows, *x, device, &y, &ldy, &code)) return nullptr;
    if (nvfp4_gemv(x->data_ptr(), x->size(0), w.K, ldx, w.codes, w.scales, static_cast<const float*>(w.alpha), w.rows,
                   y.data_ptr(), ldy, code, stream_of(device)) != NVFP4_OK)
      return nullptr;
    return give(a[3], y);
  });
}

// gemv_gated(x, w_gate, w_up, act code, out_dtype, out)
PyObject* gemv_gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t act;
    if (n != 6 || !integer(a[3], &act)) return nullptr;
    const at::Tensor* x = tensor(a[0]);
    const int device = c10::cuda::current_device();
    int64_t ldx, ldy;
    int code;
    Operand g, u;
    if (!x || !matrix(*x, at::kBFloat16, device, &ldx) || !operand(a[1], device, &g) || !operand(a[2], device, &u) ||
        x->size(1) != g.K || u.K != g.K || u.rows != g.rows)
      return nullptr;
    at::Tensor y;
    if (!output(a[5], a[4], x->size(0), g.rows, *x, device, &y, &ldy, &code)) return nullptr;
    if (nvfp4_gemv_gated(x->data_ptr(), x->size(0), g.K, ldx, g.codes, g.scales, static_cast<const float*>(g.alpha),
                         u.codes, u.scales, static_cast<const float*>(u.alpha), g.rows, static_cast<int>(act),
                         y.data_ptr(), ldy, code, stream_of(device)) != NVFP4_OK)
      return nullptr;
    return give(a[5], y);
  });
}

constexpr int64_t kBlock = 32;

// gemm_gated(a, w_gate, w_up, act code, out_dtype, out, keep): with `keep` true
// the result is (h, checkpoint codes, checkpoint scales), both new.
PyObject* gemm_gated(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t act;
    if (n != 7 || !integer(a[3], &act)) return nullptr;
    const int device = c10::cuda::current_device();
    Operand x, g, u;
    if (!operand(a[0], device, &x) || !operand(a[1], device, &g) || !operand(a[2], device, &u) || g.K != x.K ||
        u.K != x.K || u.rows != g.rows)
      return nullptr;
    const Attr alpha(a[0], s_global_scale);
    const at::Tensor* like = alpha.o ? tensor(alpha.o) : nullptr;
    at::Tensor h, codes, scales;
    int64_t ldh;
    int code;
    if (!like || !output(a[5], a[4], x.rows, g.rows, *like, device, &h, &ldh, &code)) return nullptr;
    if (a[6] == Py_True) {
      const int64_t blocks = (g.rows + kBlock - 1) / kBlock;
      codes = at::empty({2, x.rows, blocks * kBlock}, like->options().dtype(at::kChar));
      scales = at::empty({2, x.rows, blocks}, like->options().dtype(at::kBFloat16));
    }
    if (nvfp4_gemm_gated(x.codes, x.scales, static_cast<const float*>(x.alpha), g.codes, g.scales,
                         static_cast<const float*>(g.alpha), u.codes, u.scales, static_cast<const float*>(u.alpha),
                         x.rows, g.rows, x.K, static_cast<int>(act), h.data_ptr(), ldh, code,
                         codes.defined() ? codes.data_ptr() : nullptr, scales.defined() ? scales.data_ptr() : nullptr,
                         nullptr, 0, stream_of(device)) != NVFP4_OK)
      return nullptr;
    PyObject* out = give(a[5], h);
    if (!out || !codes.defined()) return out;
    PyObject *pc = THPVariable_Wrap(codes), *ps = THPVariable_Wrap(scales);
    PyObject* r = pc && ps ? PyTuple_Pack(3, out, pc, ps) : nullptr;
    Py_DECREF(out);
    Py_XDECREF(pc);
    Py_XDECREF(ps);
    return r;
  });
}

// gated_backward(dh, codes, scales, rows, cols, act code, recompute): dgu, or
// (dgu, h), all new.
PyObject* gated_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t rows, cols, act, ldd;
    if (n != 7 || !integer(a[3], &rows) || !integer(a[4], &cols) || !integer(a[5], &act)) return nullptr;
    const at::Tensor* dh = tensor(a[0]);
    const int device = c10::cuda::current_device();
    if (!dh || !matrix(*dh, at::kBFloat16, device, &ldd) || dh->size(0) != rows || dh->size(1) != cols || rows < 1 ||
        cols < 1 || rows > (1ll << 30) || cols > (1ll << 30))
      return nullptr;
    const int64_t blocks = (cols + kBlock - 1) / kBlock;
    void *codes, *scales;
    if (!buffer(a[1], at::kChar, device, 2 * rows * blocks * kBlock, &codes) ||
        !buffer(a[2], at::kBFloat16, device, 2 * rows * blocks, &scales))
      return nullptr;
    const at::Tensor dgu = at::empty({rows, 2 * cols}, dh->options());
    at::Tensor h;
    if (a[6] == Py_True) h = at::empty({rows, cols}, dh->options());
    if (nvfp4_gated_backward(dh->data_ptr(), ldd, codes, scales, rows, cols, static_cast<int>(act), dgu.data_ptr(),
                             2 * cols, h.defined() ? h.data_ptr() : nullptr, cols, stream_of(device)) != NVFP4_OK)
      return nullptr;
    PyObject* p = THPVariable_Wrap(dgu);
    if (!p || !h.defined()) return p;
    PyObject* q = THPVariable_Wrap(h);
    PyObject* r = q ? PyTuple_Pack(2, p, q) : nullptr;
    Py_DECREF(p);
    Py_XDECREF(q);
    return r;
  });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(gemv), METHOD(gemv_gated), METHOD(gemm_gated), METHOD(gated_backward),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__fastcall() {
  PyObject* torch = PyImport_ImportModule("torch");
  if (!torch) return nullptr;
  d_bf16 = PyObject_GetAttrString(torch, "bfloat16");
  d_f32 = PyObject_GetAttrString(torch, "float32");
  Py_DECREF(torch);
  s_codes = PyUnicode_InternFromString("codes");
  s_scales = PyUnicode_InternFromString("scales");
  s_global_scale = PyUnicode_InternFromString("global_scale");
  s_rows = PyUnicode_InternFromString("rows");
  s_K = PyUnicode_InternFromString("K");
  if (!d_bf16 || !d_f32 || !s_codes || !s_scales || !s_global_scale || !s_rows || !s_K) return nullptr;
  PyObject* m = PyModule_Create(&module);
  // the torch that this was compiled for: the package uses it with no other
  if (m && PyModule_AddStringConstant(m, "built_for", BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
