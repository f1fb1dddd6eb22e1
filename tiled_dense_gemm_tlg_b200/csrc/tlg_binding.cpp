// Native argument marshalling for the microscaled (MX) entry points and those around the linear layers: checks the tensors,
// allocates outputs that were not given with torch's allocator, and calls libtlg.  Nothing is
// computed here.  A small call is bound by its host side: from Python, with ctypes, the checks
// and allocations cost 9 to 17 us a call, several times the kernels' time.
//
// Every function takes its arguments by position (the Python wrappers fill in defaults) and
// returns the outputs, or the library's status as an int when it is not TLG_OK.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cstdint>
#include <exception>
#include <optional>

#include "tlg.h"

namespace {

// Raised inside a function whose Python exception is already set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const char *format, const char *name) {
  PyErr_Format(type, format, name);
  throw Raised();
}

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a tensor", name);
  return THPVariable_Unpack(o);
}

// An optional tensor: nullptr for None.
const at::Tensor *maybe(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }

int64_t integer(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

struct Mat {
  void *p;
  int64_t ld;
};

// A row-major 2-D tensor whose rows do not overlap.
Mat mat(const at::Tensor &t, const char *name) {
  if (t.dim() != 2) raise(PyExc_ValueError, "%s must be a 2-D tensor", name);
  const int64_t rows = t.size(0), cols = t.size(1), ld = t.stride(0);
  if (cols > 1 && t.stride(1) != 1)
    raise(PyExc_ValueError, "%s must be row-major (unit stride along its last dimension)", name);
  if (rows > 1 && ld < cols) raise(PyExc_ValueError, "%s has overlapping rows", name);
  return {t.data_ptr(), ld > cols ? ld : cols};
}

bool is_shape(const at::Tensor &t, int64_t rows, int64_t cols) {
  return t.dim() == 2 && t.size(0) == rows && t.size(1) == cols;
}

tlg_type type_of(const at::Tensor &t, const char *name) {
  switch (t.scalar_type()) {
    case at::kFloat: return TLG_TYPE_F32;
    case at::kHalf: return TLG_TYPE_F16;
    case at::kBFloat16: return TLG_TYPE_BF16;
    default: raise(PyExc_TypeError, "%s must be fp32, fp16 or bf16", name);
  }
}

at::ScalarType scalar_type(int64_t type) {
  return type == TLG_TYPE_F32 ? at::kFloat : type == TLG_TYPE_F16 ? at::kHalf : at::kBFloat16;
}

at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, const at::Device &device) {
  if (device.is_cuda()) return at::detail::empty_cuda(sizes, type, device, c10::nullopt);
  return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
}

void same_device(const at::Tensor &like, const at::Tensor *t) {
  if (t != nullptr && t->device() != like.device())
    raise(PyExc_ValueError, "all tensors must be on one device%s", "");
}

// The stream of a call on `like`'s device: the one given, else torch's current one.  A given
// stream is the current one while the call lasts, so that outputs and a workspace allocated
// here belong to it: the workspace goes back to the allocator on return, and only work behind
// the call on the same stream may get its memory.
class Stream {
 public:
  Stream(PyObject *o, const at::Tensor &like) {
    if (o != Py_None) {
      handle_ = reinterpret_cast<cudaStream_t>(integer(o));
      if (like.is_cuda()) {
        const auto device = static_cast<c10::DeviceIndex>(like.get_device());
        guard_.emplace(handle_ == nullptr ? c10::cuda::getDefaultCUDAStream(device)
                                          : c10::cuda::getStreamFromExternal(handle_, device));
      }
    } else if (like.is_cuda()) {
      handle_ = c10::cuda::getCurrentCUDAStream(like.get_device()).stream();
    }
  }
  operator void *() const { return handle_; }

 private:
  cudaStream_t handle_ = nullptr;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
};

int64_t blocks_of(int64_t cols) { return (cols + 31) / 32; }
int64_t block_bytes(int64_t format) { return format == TLG_MX_E2M1 ? 16 : 32; }
int64_t scale_bytes(int64_t rows, int64_t blocks) { return (rows + 127) / 128 * ((blocks + 3) / 4) * 512; }

struct Mx {
  at::Tensor q, s;
  Mat m;
};

// An MX matrix's two buffers.
Mx mx(const at::Tensor &q, const at::Tensor &s, int64_t rows, int64_t blocks, int64_t format) {
  Mx x{q, s, mat(q, "Q")};
  if (q.scalar_type() != at::kByte || !is_shape(q, rows, blocks * block_bytes(format))) {
    PyErr_Format(PyExc_ValueError, "Q must be a uint8 tensor of shape (%lld, %lld)", static_cast<long long>(rows),
                 static_cast<long long>(blocks * block_bytes(format)));
    throw Raised();
  }
  if (s.scalar_type() != at::kByte || !s.is_contiguous() || s.numel() < scale_bytes(rows, blocks)) {
    PyErr_Format(PyExc_ValueError, "S must be a contiguous uint8 tensor of at least %lld bytes",
                 static_cast<long long>(scale_bytes(rows, blocks)));
    throw Raised();
  }
  return x;
}

// The MX matrix an operator writes, allocated where not given.
Mx mx_out(PyObject *q, PyObject *s, int64_t rows, int64_t cols, int64_t format, const at::Tensor &like) {
  const int64_t blocks = blocks_of(cols);
  const at::Tensor *gq = maybe(q, "Q"), *gs = maybe(s, "S");
  same_device(like, gq);
  same_device(like, gs);
  return mx(gq != nullptr ? *gq : empty({rows, blocks * block_bytes(format)}, at::kByte, like.device()),
            gs != nullptr ? *gs : empty({scale_bytes(rows, blocks)}, at::kByte, like.device()), rows, blocks, format);
}

// The rows x cols matrix an operator writes, allocated where not given.
at::Tensor out_matrix(PyObject *o, const char *name, int64_t rows, int64_t cols, at::ScalarType type,
                      const at::Tensor &like) {
  const at::Tensor *given = maybe(o, name);
  if (given == nullptr) return empty({rows, cols}, type, like.device());
  same_device(like, given);
  if (given->scalar_type() != type || !is_shape(*given, rows, cols)) {
    PyErr_Format(PyExc_ValueError, "%s must be %s of shape (%lld, %lld)", name, c10::toString(type),
                 static_cast<long long>(rows), static_cast<long long>(cols));
    throw Raised();
  }
  return *given;
}

PyObject *wrap(const at::Tensor &t) { return THPVariable_Wrap(t); }

PyObject *tuple_of(PyObject *a, PyObject *b, PyObject *c = nullptr) {
  PyObject *t = PyTuple_New(c != nullptr ? 3 : 2);
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  if (c != nullptr) PyTuple_SET_ITEM(t, 2, c);
  return t;
}

// Runs f(args) with its C++ exceptions as Python ones.
template <typename F>
PyObject *guarded(Py_ssize_t nargs, Py_ssize_t want, F f) {
  if (nargs != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, nargs);
    return nullptr;
  }
  try {
    return f();
  } catch (const Raised &) {
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (X, format, transposed, Q, S, stream)
PyObject *mx_quantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject * {
    const at::Tensor &x = tensor(a[0], "X");
    const Stream stream(a[5], x);
    const Mat m = mat(x, "X");
    const tlg_type type = type_of(x, "X");
    const int64_t format = integer(a[1]);
    const bool t = integer(a[2]) != 0;
    const int64_t rows = x.size(t ? 1 : 0), cols = x.size(t ? 0 : 1);
    const Mx o = mx_out(a[3], a[4], rows, cols, format, x);
    const tlg_status st =
        tlg_mx_quantize(static_cast<tlg_mx_format>(format), rows, cols, t ? TLG_OP_T : TLG_OP_N, type, m.p, m.ld,
                        o.m.p, o.m.ld, o.s.data_ptr(), stream);
    return st != TLG_OK ? PyLong_FromLong(st) : tuple_of(wrap(o.q), wrap(o.s));
  });
}

// (Q, S, cols, format, type, X, stream)
PyObject *mx_dequantize(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject * {
    const at::Tensor &q = tensor(a[0], "Q"), &s = tensor(a[1], "S");
    const int64_t cols = integer(a[2]), format = integer(a[3]), type = integer(a[4]);
    const int64_t rows = q.dim() == 2 ? q.size(0) : 0;
    const Stream stream(a[6], q);
    const Mx in = mx(q, s, rows, blocks_of(cols), format);
    same_device(q, &s);
    const at::Tensor x = out_matrix(a[5], "X", rows, cols, scalar_type(type), q);
    const Mat m = mat(x, "X");
    const tlg_status st =
        tlg_mx_dequantize(static_cast<tlg_mx_format>(format), rows, cols, in.m.p, in.m.ld, s.data_ptr(),
                          static_cast<tlg_type>(type), m.p, m.ld, stream);
    return st != TLG_OK ? PyLong_FromLong(st) : wrap(x);
  });
}

// (A, SA, B, SB, bias, activation, residual, C, type, address of a tlg_config or 0, stream)
PyObject *gemm_mxfp4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    const at::Tensor &ta = tensor(a[0], "A"), &tsa = tensor(a[1], "SA"), &tb = tensor(a[2], "B"),
                     &tsb = tensor(a[3], "SB");
    if (ta.dim() != 2 || tb.dim() != 2 || ta.size(1) != tb.size(1) || ta.size(1) % 16 != 0)
      raise(PyExc_ValueError, "A and B must be 2-D and hold whole blocks of one K%s", "");
    const Stream stream(a[10], ta);
    const int64_t M = ta.size(0), N = tb.size(0), blocks = ta.size(1) / 16, type = integer(a[8]);
    const Mx A = mx(ta, tsa, M, blocks, TLG_MX_E2M1), B = mx(tb, tsb, N, blocks, TLG_MX_E2M1);
    for (const at::Tensor *t : {&tsa, &tb, &tsb}) same_device(ta, t);
    const at::ScalarType dtype = scalar_type(type);
    const at::Tensor c = out_matrix(a[7], "C", M, N, dtype, ta);
    const Mat m = mat(c, "C");
    tlg_fused_epilogue e = {nullptr, static_cast<int32_t>(integer(a[5])), nullptr, 0};
    if (const at::Tensor *bias = maybe(a[4], "bias")) {
      same_device(ta, bias);
      if (bias->scalar_type() != (type == TLG_TYPE_BF16 ? at::kBFloat16 : at::kHalf) || bias->dim() != 1 ||
          bias->size(0) != N || (N > 1 && bias->stride(0) != 1))
        raise(PyExc_ValueError, "bias must be a contiguous %s vector with an element for each column of C",
              type == TLG_TYPE_BF16 ? "bf16" : "fp16");
      e.bias = bias->data_ptr();
    }
    if (const at::Tensor *r = maybe(a[6], "residual")) {
      same_device(ta, r);
      if (r->scalar_type() != dtype || !is_shape(*r, M, N))
        raise(PyExc_ValueError, "residual must have C's type and shape%s", "");
      const Mat mr = mat(*r, "residual");
      e.residual = mr.p;
      e.ldr = mr.ld;
    }
    const tlg_status st = tlg_gemm_mxfp4(
        M, N, blocks * 32, A.m.p, A.m.ld, tsa.data_ptr(), B.m.p, B.m.ld, tsb.data_ptr(), &e, m.p, m.ld,
        static_cast<tlg_type>(type), reinterpret_cast<const tlg_config *>(integer(a[9])), stream);
    return st != TLG_OK ? PyLong_FromLong(st) : wrap(c);
  });
}

// (Z, activation, Y, Q, S, stream)
PyObject *act_forward_mx(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject * {
    const at::Tensor &z = tensor(a[0], "Z");
    const Stream stream(a[5], z);
    const Mat mz = mat(z, "Z");
    const tlg_type type = type_of(z, "Z");
    const int64_t rows = z.size(0), cols = z.size(1);
    const at::Tensor y = out_matrix(a[2], "Y", rows, cols, z.scalar_type(), z);
    const Mat my = mat(y, "Y");
    const Mx o = mx_out(a[3], a[4], rows, cols, TLG_MX_E4M3, z);
    const tlg_status st = tlg_act_forward_mx(rows, cols, static_cast<tlg_activation>(integer(a[1])), type, mz.p, mz.ld,
                                             my.p, my.ld, o.m.p, o.m.ld, o.s.data_ptr(), stream);
    return st != TLG_OK ? PyLong_FromLong(st) : tuple_of(wrap(y), wrap(o.q), wrap(o.s));
  });
}

// (dY, Q, S, activation, dZ, dbias, whether to sum, workspace, stream)
PyObject *act_backward_mx(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject * {
    const at::Tensor &dy = tensor(a[0], "dY"), &q = tensor(a[1], "Q"), &s = tensor(a[2], "S");
    const Mat my = mat(dy, "dY");
    const Stream stream(a[8], dy);
    const tlg_type type = type_of(dy, "dY");
    const int64_t rows = dy.size(0), cols = dy.size(1);
    const Mx in = mx(q, s, rows, blocks_of(cols), TLG_MX_E4M3);
    same_device(dy, &q);
    same_device(dy, &s);
    const at::Tensor dz = out_matrix(a[4], "dZ", rows, cols, dy.scalar_type(), dy);
    const Mat mz = mat(dz, "dZ");
    at::Tensor db, ws;
    size_t ws_bytes = 0;
    if (a[5] != Py_None || integer(a[6]) != 0) {
      if (const at::Tensor *given = maybe(a[5], "dbias")) {
        same_device(dy, given);
        if (given->scalar_type() != at::kFloat || given->dim() != 1 || given->size(0) != cols || !given->is_contiguous())
          raise(PyExc_ValueError, "dbias must be a contiguous fp32 vector with an element for each column%s", "");
        db = *given;
      } else {
        db = empty({cols}, at::kFloat, dy.device());
      }
      if (const at::Tensor *given = maybe(a[7], "workspace")) {
        same_device(dy, given);
        if (!given->is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", "workspace");
        ws = *given;
        ws_bytes = ws.nbytes();
      } else {
        const tlg_status st = tlg_act_backward_mx_workspace_size(rows, cols, type, &ws_bytes);
        if (st != TLG_OK) return PyLong_FromLong(st);
        if (ws_bytes != 0) ws = empty({static_cast<int64_t>(ws_bytes)}, at::kByte, dy.device());
      }
    }
    const tlg_status st = tlg_act_backward_mx(
        rows, cols, static_cast<tlg_activation>(integer(a[3])), type, my.p, my.ld, in.m.p, in.m.ld, s.data_ptr(), mz.p,
        mz.ld, db.defined() ? static_cast<float *>(db.data_ptr()) : nullptr, ws.defined() ? ws.data_ptr() : nullptr,
        ws_bytes, stream);
    if (st != TLG_OK) return PyLong_FromLong(st);
    PyObject *none = Py_None;
    if (!db.defined()) Py_INCREF(none);
    return tuple_of(wrap(dz), db.defined() ? wrap(db) : none);
  });
}

// A stack of row-major matrices, `stride` elements apart.
struct Stack {
  Mat m;
  int64_t stride;
};

Stack stack(const at::Tensor &t, const char *name) {
  if (t.dim() != 3) raise(PyExc_ValueError, "%s must be a 3-D tensor", name);
  const int64_t rows = t.size(1), cols = t.size(2), ld = t.stride(1);
  if (cols > 1 && t.stride(2) != 1)
    raise(PyExc_ValueError, "%s must be row-major (unit stride along its last dimension)", name);
  if (rows > 1 && ld < cols) raise(PyExc_ValueError, "%s has overlapping rows", name);
  return {{t.data_ptr(), ld > cols ? ld : cols}, t.size(0) > 1 ? t.stride(0) : 0};
}

// The groups' offsets and their number.
int32_t groups_of(const at::Tensor &o) {
  if (o.scalar_type() != at::kInt || o.dim() != 1 || o.size(0) < 1 || !o.is_contiguous())
    raise(PyExc_ValueError, "offsets must be a contiguous int32 vector with an element more than there are groups%s", "");
  return static_cast<int32_t>(std::min<int64_t>(o.size(0) - 1, INT32_MAX));
}

// (A, B, offsets, transposed, activation, C, type, stream); type -1: A's
PyObject *gemm_grouped(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject * {
    const at::Tensor &ta = tensor(a[0], "A"), &tb = tensor(a[1], "B"), &to = tensor(a[2], "offsets");
    const Stream stream(a[7], ta);
    const Mat ma = mat(ta, "A");
    const Stack b = stack(tb, "B");
    const tlg_type type = type_of(ta, "A");
    const int32_t groups = groups_of(to);
    const bool t = integer(a[3]) != 0;
    const int64_t rows = ta.size(0), K = ta.size(1), N = tb.size(t ? 1 : 2), out = integer(a[6]);
    if (tb.scalar_type() != ta.scalar_type()) raise(PyExc_TypeError, "A and B must have one type%s", "");
    if (tb.size(0) != groups || tb.size(t ? 2 : 1) != K)
      raise(PyExc_ValueError, "B must hold a matrix for each group, with A's columns as its inner dimension%s", "");
    same_device(ta, &tb);
    same_device(ta, &to);
    const at::Tensor c = out_matrix(a[5], "C", rows, N, scalar_type(out < 0 ? type : out), ta);
    const Mat mc = mat(c, "C");
    const tlg_status st = tlg_gemm_grouped(
        rows, N, K, groups, static_cast<const int32_t *>(to.data_ptr()), type, ma.p, ma.ld, t ? TLG_OP_T : TLG_OP_N,
        b.m.p, b.m.ld, b.stride, static_cast<tlg_activation>(integer(a[4])), mc.p, mc.ld,
        static_cast<tlg_type>(out < 0 ? type : out), stream);
    return st != TLG_OK ? PyLong_FromLong(st) : wrap(c);
  });
}

// (A, dC, offsets, transposed, dB, type, stream); type -1: A's
PyObject *gemm_grouped_dw(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject * {
    const at::Tensor &ta = tensor(a[0], "A"), &td = tensor(a[1], "dC"), &to = tensor(a[2], "offsets");
    const Stream stream(a[6], ta);
    const Mat ma = mat(ta, "A"), md = mat(td, "dC");
    const tlg_type type = type_of(ta, "A");
    const int32_t groups = groups_of(to);
    const bool t = integer(a[3]) != 0;
    const int64_t rows = ta.size(0), K = ta.size(1), N = td.size(1), out = integer(a[5]) < 0 ? type : integer(a[5]);
    if (td.scalar_type() != ta.scalar_type()) raise(PyExc_TypeError, "A and dC must have one type%s", "");
    if (td.size(0) != rows) raise(PyExc_ValueError, "A and dC must have the same rows%s", "");
    same_device(ta, &td);
    same_device(ta, &to);
    at::Tensor db;
    if (const at::Tensor *given = maybe(a[4], "dB")) {
      same_device(ta, given);
      if (given->scalar_type() != scalar_type(out) || given->dim() != 3 || given->size(0) != groups ||
          given->size(1) != (t ? N : K) || given->size(2) != (t ? K : N))
        raise(PyExc_ValueError, "dB must be of the output type and hold a matrix in B's layout for each group%s", "");
      db = *given;
    } else {
      db = empty({groups, t ? N : K, t ? K : N}, scalar_type(out), ta.device());
    }
    const Stack b = stack(db, "dB");
    const tlg_status st = tlg_gemm_grouped_dw(
        rows, N, K, groups, static_cast<const int32_t *>(to.data_ptr()), type, ma.p, ma.ld, md.p, md.ld,
        t ? TLG_OP_T : TLG_OP_N, b.m.p, b.m.ld, b.stride, static_cast<tlg_type>(out), stream);
    return st != TLG_OK ? PyLong_FromLong(st) : wrap(db);
  });
}

// A contiguous vector of n elements of a type.
void *vector(const at::Tensor &t, const char *name, int64_t n, at::ScalarType type) {
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || !t.is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s vector of %lld elements", name, c10::toString(type),
                 static_cast<long long>(n));
    throw Raised();
  }
  return t.data_ptr();
}

double real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}

// (X, weight, residual, eps, H, Y, format or -1, Q, S, rstd, stream) -> (Y, H, rstd) or (Q, S, H, rstd)
PyObject *rmsnorm_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    const at::Tensor &x = tensor(a[0], "X"), &w = tensor(a[1], "weight");
    const Stream stream(a[10], x);
    const Mat mx_ = mat(x, "X");
    const tlg_type type = type_of(x, "X");
    const int64_t rows = x.size(0), cols = x.size(1), format = integer(a[6]);
    const float eps = static_cast<float>(real(a[3]));
    same_device(x, &w);
    void *pw = vector(w, "weight", cols, x.scalar_type());
    const at::Tensor *r = maybe(a[2], "residual");
    Mat mr = {nullptr, 0}, mh = {nullptr, 0};
    at::Tensor h = x;
    if (r != nullptr || a[4] != Py_None) {
      h = out_matrix(a[4], "H", rows, cols, x.scalar_type(), x);
      mh = mat(h, "H");
    }
    if (r != nullptr) {
      same_device(x, r);
      if (r->scalar_type() != x.scalar_type() || !is_shape(*r, rows, cols))
        raise(PyExc_ValueError, "residual must have X's type and shape%s", "");
      mr = mat(*r, "residual");
    }
    at::Tensor rstd;
    if (const at::Tensor *given = maybe(a[9], "rstd")) {
      same_device(x, given);
      vector(*given, "rstd", rows, at::kFloat);
      rstd = *given;
    } else {
      rstd = empty({rows}, at::kFloat, x.device());
    }
    float *ps = static_cast<float *>(rstd.data_ptr());
    if (format < 0) {
      const at::Tensor y = out_matrix(a[5], "Y", rows, cols, x.scalar_type(), x);
      const Mat my = mat(y, "Y");
      const tlg_status st = tlg_rmsnorm_forward(rows, cols, type, mx_.p, mx_.ld, mr.p, mr.ld, pw, eps, mh.p, mh.ld, my.p,
                                                my.ld, ps, stream);
      return st != TLG_OK ? PyLong_FromLong(st) : tuple_of(wrap(y), wrap(h), wrap(rstd));
    }
    const Mx o = mx_out(a[7], a[8], rows, cols, format, x);
    const tlg_status st =
        tlg_rmsnorm_forward_mx(rows, cols, type, mx_.p, mx_.ld, mr.p, mr.ld, pw, eps, mh.p, mh.ld,
                               static_cast<tlg_mx_format>(format), o.m.p, o.m.ld, o.s.data_ptr(), ps, stream);
    if (st != TLG_OK) return PyLong_FromLong(st);
    PyObject *t = PyTuple_New(4);
    PyTuple_SET_ITEM(t, 0, wrap(o.q));
    PyTuple_SET_ITEM(t, 1, wrap(o.s));
    PyTuple_SET_ITEM(t, 2, wrap(h));
    PyTuple_SET_ITEM(t, 3, wrap(rstd));
    return t;
  });
}

// (dY, H, weight, rstd, dH, dX, dweight, whether to sum, workspace, stream)
PyObject *rmsnorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject * {
    const at::Tensor &dy = tensor(a[0], "dY"), &h = tensor(a[1], "H"), &w = tensor(a[2], "weight"),
                     &rstd = tensor(a[3], "rstd");
    const Stream stream(a[9], dy);
    const Mat my = mat(dy, "dY");
    const tlg_type type = type_of(dy, "dY");
    const int64_t rows = dy.size(0), cols = dy.size(1);
    for (const at::Tensor *t : {&h, &w, &rstd}) same_device(dy, t);
    if (h.scalar_type() != dy.scalar_type() || !is_shape(h, rows, cols))
      raise(PyExc_ValueError, "H must have dY's type and shape%s", "");
    const Mat mh = mat(h, "H");
    void *pw = vector(w, "weight", cols, dy.scalar_type());
    const float *ps = static_cast<const float *>(vector(rstd, "rstd", rows, at::kFloat));
    Mat md = {nullptr, 0};
    if (const at::Tensor *d = maybe(a[4], "dH")) {
      same_device(dy, d);
      if (d->scalar_type() != dy.scalar_type() || !is_shape(*d, rows, cols))
        raise(PyExc_ValueError, "dH must have dY's type and shape%s", "");
      md = mat(*d, "dH");
    }
    const at::Tensor dx = out_matrix(a[5], "dX", rows, cols, dy.scalar_type(), dy);
    const Mat mx_ = mat(dx, "dX");
    at::Tensor dw, ws;
    size_t ws_bytes = 0;
    if (a[6] != Py_None || integer(a[7]) != 0) {
      if (const at::Tensor *given = maybe(a[6], "dweight")) {
        same_device(dy, given);
        vector(*given, "dweight", cols, at::kFloat);
        dw = *given;
      } else {
        dw = empty({cols}, at::kFloat, dy.device());
      }
      if (const at::Tensor *given = maybe(a[8], "workspace")) {
        same_device(dy, given);
        if (!given->is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", "workspace");
        ws = *given;
        ws_bytes = ws.nbytes();
      } else {
        const tlg_status st = tlg_rmsnorm_backward_workspace_size(rows, cols, type, &ws_bytes);
        if (st != TLG_OK) return PyLong_FromLong(st);
        if (ws_bytes != 0) ws = empty({static_cast<int64_t>(ws_bytes)}, at::kByte, dy.device());
      }
    }
    const tlg_status st = tlg_rmsnorm_backward(
        rows, cols, type, my.p, my.ld, mh.p, mh.ld, pw, ps, md.p, md.ld, mx_.p, mx_.ld,
        dw.defined() ? static_cast<float *>(dw.data_ptr()) : nullptr, ws.defined() ? ws.data_ptr() : nullptr, ws_bytes,
        stream);
    if (st != TLG_OK) return PyLong_FromLong(st);
    PyObject *none = Py_None;
    if (!dw.defined()) Py_INCREF(none);
    return tuple_of(wrap(dx), dw.defined() ? wrap(dw) : none);
  });
}

// (X, Q, S, Z, group, bias, activation, residual, C, type, stream); type -1: X's
PyObject *gemv_q4(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject * {
    const at::Tensor &x = tensor(a[0], "X"), &q = tensor(a[1], "Q"), &s = tensor(a[2], "S");
    const Stream stream(a[10], x);
    const Mat mx_ = mat(x, "X"), mq = mat(q, "Q");
    const tlg_type type = type_of(x, "X");
    const int64_t M = x.size(0), K = x.size(1), N = q.size(0), group = integer(a[4]);
    const int64_t out = integer(a[9]) < 0 ? type : integer(a[9]);
    if (group < 1) raise(PyExc_ValueError, "group must be positive%s", "");
    const int64_t groups = K / group + (K % group != 0);
    if (q.scalar_type() != at::kByte || q.size(1) != blocks_of(K) * 16)
      raise(PyExc_ValueError, "Q must be a uint8 matrix of 16 bytes for every 32 columns of X%s", "");
    if (s.scalar_type() != x.scalar_type() || !is_shape(s, N, groups) || !s.is_contiguous())
      raise(PyExc_ValueError, "S must be contiguous, of X's type, with a scale for each row of Q and group%s", "");
    same_device(x, &q);
    same_device(x, &s);
    const uint8_t *pz = nullptr;
    if (const at::Tensor *z = maybe(a[3], "Z")) {
      same_device(x, z);
      if (z->scalar_type() != at::kByte || !is_shape(*z, N, groups) || !z->is_contiguous())
        raise(PyExc_ValueError, "Z must be contiguous, uint8, with S's shape%s", "");
      pz = static_cast<const uint8_t *>(z->data_ptr());
    }
    const at::Tensor c = out_matrix(a[8], "C", M, N, scalar_type(out), x);
    const Mat mc = mat(c, "C");
    tlg_fused_epilogue e = {nullptr, static_cast<int32_t>(integer(a[6])), nullptr, 0};
    if (const at::Tensor *bias = maybe(a[5], "bias")) {
      same_device(x, bias);
      e.bias = vector(*bias, "bias", N, x.scalar_type());
    }
    if (const at::Tensor *r = maybe(a[7], "residual")) {
      same_device(x, r);
      if (r->scalar_type() != scalar_type(out) || !is_shape(*r, M, N))
        raise(PyExc_ValueError, "residual must have C's type and shape%s", "");
      const Mat mr = mat(*r, "residual");
      e.residual = mr.p;
      e.ldr = mr.ld;
    }
    const tlg_status st = tlg_gemv_q4(M, N, K, type, mx_.p, mx_.ld, mq.p, mq.ld, s.data_ptr(), pz, group, &e, mc.p, mc.ld,
                                      static_cast<tlg_type>(out), stream);
    return st != TLG_OK ? PyLong_FromLong(st) : wrap(c);
  });
}

#define TLG_METHOD(NAME) {#NAME, reinterpret_cast<PyCFunction>(NAME), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {TLG_METHOD(mx_quantize),     TLG_METHOD(mx_dequantize),   TLG_METHOD(gemm_mxfp4),
                          TLG_METHOD(act_forward_mx), TLG_METHOD(act_backward_mx),
                          TLG_METHOD(gemm_grouped),    TLG_METHOD(gemm_grouped_dw),
                          TLG_METHOD(rmsnorm_forward), TLG_METHOD(rmsnorm_backward), TLG_METHOD(gemv_q4),
                          {nullptr, nullptr, 0, nullptr}};
// The docstring says which torch and Python this was compiled for; the build looks for it.
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", TLG_BUILT_FOR, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
