// The feed-forward operators on torch tensors, as the Python module
// _ff_native: checks of the tensors, new outputs, and the calls of
// libgb300gemm.so.  The calls for few tokens take less time on the GPU than
// their arguments take to check from Python (one token through a 4096 x 4096
// 4-bit matrix: 14 us a call through ctypes), so this part is native.
// roofline_gb300/feedforward.py is the interface.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <stdexcept>
#include <string>
#include <vector>

#include "gb300_gemm.h"

namespace {

using at::Tensor;

[[noreturn]] void refuse(const std::string &what) { throw std::invalid_argument(what); }

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a torch tensor");
  return THPVariable_Unpack(o);
}

int dtype_code(const Tensor &t, const char *name) {
  if (t.scalar_type() == at::kBFloat16) return GEMM_DT_BF16;
  if (t.scalar_type() == at::kFloat) return GEMM_DT_F32;
  refuse(std::string(name) + ": float32 or bfloat16 wanted");
}

std::string shape_of(int64_t r, int64_t c) { return std::to_string(r) + " x " + std::to_string(c); }

void check(const Tensor &t, const char *name, int64_t rows, int64_t cols, at::ScalarType type,
           int device) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
    refuse(std::string(name) + " must be " + shape_of(rows, cols));
  if (t.scalar_type() != type) refuse(std::string(name) + " must be " + c10::toString(type));
  if (!t.is_cuda() || t.get_device() != device)
    refuse(std::string(name) + " must be on CUDA device " + std::to_string(device));
}

// An integer argument from lo to hi; refused, not narrowed, beyond them: the
// library takes ints, and a matrix's width is checked for this very value.
int64_t integer(PyObject *o, const char *name, int64_t lo, int64_t hi) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer of 64 bits at most");
  }
  if (v < lo || v > hi)
    refuse(std::string(name) + " must be from " + std::to_string(lo) + " to " + std::to_string(hi));
  return v;
}
// Which activations and groups there are the library says itself.
int act_of(PyObject *o) { return (int)integer(o, "act", INT_MIN, INT_MAX); }
int64_t group_of(PyObject *o) { return integer(o, "group", 1, INT_MAX); }

// Leading dimension of the matrix that dimension `row` of a tensor counts the
// rows of.  The stride of a single row is never used; a stride of 0 between
// rows (an expanded tensor) is none that the library can be told: 0.
int64_t leading(const Tensor &t, int row) {
  const int64_t rows = t.size(row), cols = t.size(1 - row);
  if (rows > 1 && cols > 0) return t.stride(row);
  return cols > 0 ? cols : 1;
}
bool unit(const Tensor &t, int dim) { return t.size(dim) <= 1 || t.stride(dim) == 1; }

// The same of a row-major matrix, with the checks.
int64_t leading(const Tensor &t, const char *name) {
  if (!unit(t, 1)) refuse(std::string(name) + " must have unit column stride");
  const int64_t ld = leading(t, 0);
  if (ld < 1) refuse(std::string(name) + " must not be expanded along its rows");
  return ld;
}

// The matrix that sets a call's type and device.
struct First {
  const Tensor &t;
  int64_t rows, cols, ld;
  int dtype, device;
  at::ScalarType type;
  First(PyObject *o, const char *name) : t(tensor(o, name)) {
    if (!t.is_cuda() || t.dim() != 2) refuse(std::string(name) + " must be a 2-D CUDA tensor");
    rows = t.size(0);
    cols = t.size(1);
    ld = leading(t, name);
    dtype = dtype_code(t, name);
    device = t.get_device();
    type = t.scalar_type();
  }
  Tensor make(at::IntArrayRef sizes, at::IntArrayRef strides, at::ScalarType as) const {
    return at::empty_strided(sizes, strides, t.options().dtype(as));
  }
};

// The ways a D x F weight can be read: row-major is op N (ld[0] > 0), W.t() of
// a stored F x D matrix op T (ld[1] > 0); one row or column may be either.
struct Weight {
  int64_t ld[2] = {0, 0};
  Weight(const Tensor &t, const char *name) {
    if (unit(t, 1)) ld[GEMM_OP_N] = leading(t, 0);
    if (unit(t, 0)) ld[GEMM_OP_T] = leading(t, 1);
    if (!ld[0] && !ld[1])
      refuse(std::string(name) + " must have a unit row or column stride, and not be expanded");
  }
};

int common_op(const Weight &g, const Weight &u) {
  for (int op : {GEMM_OP_N, GEMM_OP_T})
    if (g.ld[op] && u.ld[op]) return op;
  refuse("Wg and Wu must be stored in the same order");
}

// What a call returned; raised as gemm.GemmError.
struct Failed {
  int code;
  const char *what;
};

template <typename F>
void call(const char *what, F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS if (rc != GEMM_OK) throw Failed{rc, what};
}

// The stream of a call: the one whose handle is given, or (None) torch's current
// one.  It is torch's current stream while this lives, so that new tensors are
// of its memory: whatever used that before is ahead of the call in the stream.
// (Of the caller's stream's memory, a kernel that is still to run there could
// use it at the same time.)
class OnStream {
  c10::cuda::CUDAStream before_, on_;
  c10::cuda::CUDAStreamGuard guard_;

  static c10::cuda::CUDAStream of(PyObject *o, const c10::cuda::CUDAStream &current, int device) {
    if (o == Py_None) return current;
    const unsigned long long v = PyLong_AsUnsignedLongLong(o);
    if (v == (unsigned long long)-1 && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("stream: a stream's handle wanted");
    }
    return c10::cuda::getStreamFromExternal(
        reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(v)), (c10::DeviceIndex)device);
  }

 public:
  OnStream(PyObject *o, int device)
      : before_(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device)),
        on_(of(o, before_, device)), guard_(on_) {}
  operator cudaStream_t() const { return on_.stream(); }
  // For the caching allocator, when they are freed: a new tensor is used on the
  // caller's stream too, one that the caller gave on this one.
  void made(const Tensor &t) const { note(t, before_); }
  void given(const Tensor &t) const { note(t, on_); }

 private:
  void note(const Tensor &t, const c10::cuda::CUDAStream &s) const {
    if (t.defined() && on_.stream() != before_.stream()) t.record_stream(s.unwrap());
  }
};
// A call's scratch: the caller's tensor, or torch's memory of the call's stream
// while this lives.  (Not the library's one buffer per device: calls on two
// streams would write it at once, and a graph would keep its address when a
// larger call has freed it.)
class Scratch {
  void *own_ = nullptr;

 public:
  void *p = nullptr;
  size_t bytes = 0;
  Scratch(PyObject *given, uint64_t need, const OnStream &s, int device) {
    if (given != Py_None) {
      const Tensor &t = tensor(given, "workspace");
      if (!t.is_cuda() || t.get_device() != device || !t.is_contiguous())
        refuse("workspace must be a contiguous tensor on CUDA device " + std::to_string(device));
      p = t.data_ptr();
      bytes = t.nbytes();
      s.given(t);
    }
    if (bytes == 0 && need > 0) {
      p = own_ = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(need, s);
      bytes = need;
    }
  }
  Scratch(const Scratch &) = delete;
  ~Scratch() {
    if (own_) c10::cuda::CUDACachingAllocator::raw_delete(own_);
  }
};

// Scratch bytes of the block: where BF16 matrices (data, leading dimension,
// rows) all lie on 16-byte boundaries, those of aligned ones.
struct Rows {
  const void *p;
  int64_t ld, rows;
};
uint64_t block_bytes(int backward, int dtype, int op, int64_t M, int64_t D, int64_t F,
                     std::initializer_list<Rows> read) {
  uint64_t need = 0;
  bool aligned = true;
  for (const Rows &r : read)
    aligned = aligned && reinterpret_cast<uintptr_t>(r.p) % 16 == 0 && (r.rows == 1 || r.ld % 8 == 0);
  // sizes that it refuses the call itself refuses too
  return gated_ff_workspace(backward, dtype, op, M, D, F, aligned, &need) == GEMM_OK ? need : 0;
}
// A tensor that a call has written: autograd is to know that what it may have
// kept of it is no longer there.
void written(const Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
void *address(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }
PyObject *wrap(const Tensor &t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
int64_t positive(int64_t x) { return x > 0 ? x : 1; }

PyObject *triple(const Tensor &a, const Tensor &b, const Tensor &c) {
  PyObject *r = PyTuple_New(3);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, wrap(a));
  PyTuple_SET_ITEM(r, 1, wrap(b));
  PyTuple_SET_ITEM(r, 2, wrap(c));
  return r;
}

// gated_ff(X, Wg, Wu, act, save, out, stream, workspace)
PyObject *gated_ff_(PyObject *const *a) {
  const First x(a[0], "X");
  const Tensor &wg = tensor(a[1], "Wg"), &wu = tensor(a[2], "Wu");
  const int64_t M = x.rows, D = x.cols, F = wg.dim() == 2 ? wg.size(1) : -1;
  check(wg, "Wg", D, F, x.type, x.device);
  check(wu, "Wu", D, F, x.type, x.device);
  const Weight g(wg, "Wg"), u(wu, "Wu");
  const int op = common_op(g, u), act = act_of(a[3]);
  const OnStream s(a[6], x.device);
  Tensor H, G, U;
  int64_t ldh = positive(F);
  if (a[5] == Py_None) {
    H = x.make({M, F}, {F, 1}, x.type);
    s.made(H);
  } else {
    H = tensor(a[5], "out");
    check(H, "out", M, F, x.type, x.device);
    ldh = leading(H, "out");
    s.given(H);
  }
  const int64_t lds = (positive(F) + 7) / 8 * 8;  // rows on 16-byte boundaries, for wide stores
  const bool save = a[4] == Py_True;
  if (save) {
    G = x.make({M, F}, {lds, 1}, at::kFloat);
    U = x.make({M, F}, {lds, 1}, at::kFloat);
    s.made(G);
    s.made(U);
  }
  const int64_t wr = op == GEMM_OP_N ? D : F;
  const Scratch ws(a[7],
                   block_bytes(0, x.dtype, op, M, D, F,
                               {{x.t.data_ptr(), x.ld, M}, {wg.data_ptr(), g.ld[op], wr},
                                {wu.data_ptr(), u.ld[op], wr}}),
                   s, x.device);
  call("gated_ff", [&] {
    return gated_ff(x.dtype, act, op, M, D, F, x.t.data_ptr(), x.ld, wg.data_ptr(), g.ld[op],
                    wu.data_ptr(), u.ld[op], H.data_ptr(), ldh, static_cast<float *>(address(G)),
                    lds, static_cast<float *>(address(U)), lds, ws.p, ws.bytes, s);
  });
  if (a[5] != Py_None) written(H);
  return save ? triple(H, G, U) : wrap(H);
}

// gated_ff_backward(dH, X, Wg, Wu, G, U, act, need_dx, need_dw, stream, workspace)
PyObject *gated_ff_backward_(PyObject *const *a) {
  const First x(a[1], "X");
  const Tensor &dh = tensor(a[0], "dH"), &wg = tensor(a[2], "Wg"), &wu = tensor(a[3], "Wu"),
               &G = tensor(a[4], "G"), &U = tensor(a[5], "U");
  const int64_t M = x.rows, D = x.cols, F = wg.dim() == 2 ? wg.size(1) : -1;
  check(wg, "Wg", D, F, x.type, x.device);
  check(wu, "Wu", D, F, x.type, x.device);
  check(dh, "dH", M, F, x.type, x.device);
  check(G, "G", M, F, at::kFloat, x.device);
  check(U, "U", M, F, at::kFloat, x.device);
  const Weight g(wg, "Wg"), u(wu, "Wu");
  const int op = common_op(g, u), act = act_of(a[6]);
  const int64_t ldh = leading(dh, "dH"), ldg = leading(G, "G"), ldu = leading(U, "U");
  const OnStream s(a[9], x.device);
  Tensor dX, dWg, dWu;
  if (a[7] == Py_True) dX = x.make({M, D}, {D, 1}, x.type);
  if (a[8] == Py_True) {
    const int64_t s0 = op == GEMM_OP_N ? F : 1, s1 = op == GEMM_OP_N ? 1 : D;
    dWg = x.make({D, F}, {s0, s1}, x.type);
    dWu = x.make({D, F}, {s0, s1}, x.type);
  }
  for (const Tensor *t : {&dX, &dWg, &dWu}) s.made(*t);
  const int64_t ldw = positive(op == GEMM_OP_N ? F : D);
  if (dX.defined() || dWg.defined()) {
    const int64_t wr = op == GEMM_OP_N ? D : F;
    const Scratch ws(a[10],
                     block_bytes(1, x.dtype, op, M, D, F,
                                 {{x.t.data_ptr(), x.ld, M}, {wg.data_ptr(), g.ld[op], wr},
                                  {wu.data_ptr(), u.ld[op], wr}}),
                     s, x.device);
    call("gated_ff_backward", [&] {
      return gated_ff_backward(
          x.dtype, act, op, M, D, F, dh.data_ptr(), ldh, x.t.data_ptr(), x.ld, wg.data_ptr(),
          g.ld[op], wu.data_ptr(), u.ld[op], static_cast<const float *>(G.data_ptr()), ldg,
          static_cast<const float *>(U.data_ptr()), ldu, address(dX), positive(D), address(dWg),
          ldw, address(dWu), ldw, ws.p, ws.bytes, s);
    });
  }
  return triple(dX, dWg, dWu);
}

// One quantised matrix: codes, scales and zero points (or None).
struct Quantised {
  const Tensor &q, &s;
  const void *z = nullptr;
  int64_t ldq;
  Quantised(PyObject *oq, PyObject *os, PyObject *oz, int64_t N, const First &x, int64_t group,
            const char *name)
      : q(tensor(oq, name)), s(tensor(os, "scales")) {
    const int64_t width = (x.cols + 1) / 2, groups = (x.cols + group - 1) / group;
    check(q, name, N, width, at::kByte, x.device);
    ldq = leading(q, name);
    scales(s, "scales", N, groups, x);
    if (oz != Py_None) {
      const Tensor &t = tensor(oz, "zeros");
      scales(t, "zeros", N, groups, x);
      z = t.data_ptr();
    }
  }
  static void scales(const Tensor &t, const char *name, int64_t N, int64_t groups, const First &x) {
    check(t, name, N, groups, x.type, x.device);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
  }
};

int64_t rows_of(PyObject *o, const char *name) {
  const Tensor &t = tensor(o, name);
  if (t.dim() != 2) refuse(std::string(name) + " must be a 2-D tensor");
  return t.size(0);
}

// q4_matmul(X, Wq, scales, zeros, group, out, stream)
PyObject *q4_matmul_(PyObject *const *a) {
  const First x(a[0], "X");
  const int64_t group = group_of(a[4]), N = rows_of(a[1], "Wq");
  const Quantised w(a[1], a[2], a[3], N, x, group, "Wq");
  const OnStream s(a[6], x.device);
  Tensor Y;
  int64_t ldy = positive(N);
  if (a[5] == Py_None) {
    Y = x.make({x.rows, N}, {N, 1}, x.type);
    s.made(Y);
  } else {
    Y = tensor(a[5], "out");
    check(Y, "out", x.rows, N, x.type, x.device);
    ldy = leading(Y, "out");
    s.given(Y);
  }
  call("q4_matmul", [&] {
    return q4_matmul(x.dtype, x.rows, N, x.cols, x.t.data_ptr(), x.ld, w.q.data_ptr(), w.ldq,
                     w.s.data_ptr(), w.z, (int)group, Y.data_ptr(), ldy, s);
  });
  if (a[5] != Py_None) written(Y);
  return wrap(Y);
}

// q4_gated(X, Wq_g, scales_g, zeros_g, Wq_u, scales_u, zeros_u, group, act, out, stream)
PyObject *q4_gated_(PyObject *const *a) {
  const First x(a[0], "X");
  const int64_t group = group_of(a[7]), N = rows_of(a[1], "Wq_g");
  const Quantised g(a[1], a[2], a[3], N, x, group, "Wq_g"), u(a[4], a[5], a[6], N, x, group, "Wq_u");
  const int act = act_of(a[8]);
  const OnStream s(a[10], x.device);
  Tensor H;
  int64_t ldh = positive(N);
  if (a[9] == Py_None) {
    H = x.make({x.rows, N}, {N, 1}, x.type);
    s.made(H);
  } else {
    H = tensor(a[9], "out");
    check(H, "out", x.rows, N, x.type, x.device);
    ldh = leading(H, "out");
    s.given(H);
  }
  call("q4_gated", [&] {
    return q4_gated(x.dtype, act, x.rows, N, x.cols, x.t.data_ptr(), x.ld, g.q.data_ptr(), g.ldq,
                    g.s.data_ptr(), g.z, u.q.data_ptr(), u.ldq, u.s.data_ptr(), u.z, (int)group,
                    H.data_ptr(), ldh, s);
  });
  if (a[9] != Py_None) written(H);
  return wrap(H);
}

// Whether a tensor's elements are all those from its first address on, in any
// order: the norm and the scaling take them as they lie (the gradient of a
// weight given as W.t() is F x D in storage).
bool dense(const Tensor &t) { return t.is_contiguous() || t.is_non_overlapping_and_dense(); }
// Whether the elements of two dense tensors correspond as they lie.
bool same_order(const Tensor &a, const Tensor &b) {
  if (a.is_contiguous() && b.is_contiguous()) return a.numel() == b.numel();
  if (a.sizes() != b.sizes()) return false;
  for (int64_t d = 0; d < a.dim(); ++d)
    if (a.size(d) > 1 && a.stride(d) != b.stride(d)) return false;
  return true;
}

// grad_norm_clip(grads, outs, max_norm, stream, workspace); lists, outs may be None
PyObject *grad_norm_clip_(PyObject *const *a) {
  if (!PyList_Check(a[0]) || (a[1] != Py_None && !PyList_Check(a[1])))
    refuse("grads and out must be lists");
  const Py_ssize_t n = PyList_GET_SIZE(a[0]);
  if (a[1] != Py_None && PyList_GET_SIZE(a[1]) != n) refuse("out must match grads in number");
  std::vector<int> dtypes(n);
  std::vector<const void *> in(n);
  std::vector<void *> out(a[1] != Py_None ? n : 0);
  std::vector<int64_t> sizes(n);
  int device = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const Tensor &t = tensor(PyList_GET_ITEM(a[0], i), "grads");
    if (!t.is_cuda() || !dense(t) || (device >= 0 && t.get_device() != device))
      refuse("grads must be CUDA tensors of one device, dense in any order of their dimensions");
    device = t.get_device();
    dtypes[i] = dtype_code(t, "grads");
    in[i] = t.data_ptr();
    sizes[i] = t.numel();
    if (a[1] == Py_None) continue;
    const Tensor &o = tensor(PyList_GET_ITEM(a[1], i), "out");
    if (!o.is_cuda() || o.get_device() != device || o.scalar_type() != t.scalar_type() ||
        !same_order(t, o))
      refuse("out must match grads in sizes, dtypes, device and order of storage");
    out[i] = o.data_ptr();
  }
  const double max_norm = PyFloat_AsDouble(a[2]);
  if (max_norm == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("max_norm must be a number");
  }
  if (device < 0) device = c10::cuda::current_device();
  const OnStream s(a[3], device);
  Tensor norm = at::empty({}, at::TensorOptions().dtype(at::kFloat).device(at::kCUDA, device));
  s.made(norm);
  const Scratch ws(a[4], grad_norm_clip_workspace(n), s, device);
  call("grad_norm_clip", [&] {
    return grad_norm_clip(n, dtypes.data(), in.data(), a[1] == Py_None ? nullptr : out.data(),
                          sizes.data(), (float)max_norm, static_cast<float *>(norm.data_ptr()),
                          ws.p, ws.bytes, s);
  });
  if (a[1] != Py_None)
    for (Py_ssize_t i = 0; i < n; ++i) written(THPVariable_Unpack(PyList_GET_ITEM(a[1], i)));
  return wrap(norm);
}

// A function of N positional arguments; C++ exceptions end here.
template <PyObject *(*F)(PyObject *const *), int N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments wanted, got %zd", N, n);
    return nullptr;
  }
  try {
    PyObject *r = F(args);
    if (r && PyErr_Occurred()) {  // an argument that was not the number it should be
      Py_DECREF(r);
      return nullptr;
    }
    return r;
  } catch (const Failed &e) {
    PyObject *m = PyImport_ImportModule("roofline_gb300.gemm");
    PyObject *cls = m ? PyObject_GetAttrString(m, "GemmError") : nullptr;
    PyObject *err = cls ? PyObject_CallFunction(cls, "is", e.code, e.what) : nullptr;
    if (err) PyErr_SetObject(cls, err);
    Py_XDECREF(err);
    Py_XDECREF(cls);
    Py_XDECREF(m);
  } catch (const std::invalid_argument &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception &e) {  // out of memory among them
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define FF_ENTRY(name, f, n) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FF_ENTRY("gated_ff", gated_ff_, 8),
                          FF_ENTRY("gated_ff_backward", gated_ff_backward_, 11),
                          FF_ENTRY("q4_matmul", q4_matmul_, 7), FF_ENTRY("q4_gated", q4_gated_, 11),
                          FF_ENTRY("grad_norm_clip", grad_norm_clip_, 5),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_ff_native", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ff_native(void) { return PyModule_Create(&kModule); }
