// The Python side of the operators around the product (ops.py), as a CPython extension: checks of
// torch tensors, allocation of outputs and workspaces, and the calls of the C ABI (gemm_ops.h).  In
// Python the same takes 7 us a call, twice what enqueuing a kernel does; here it is under 3.
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>
#include <vector>

#include "../../include/gemm_ops.h"

namespace {

struct Refused : std::exception {   // becomes a ValueError
  std::string text;
  explicit Refused(std::string s) : text(std::move(s)) {}
  const char *what() const noexcept override { return text.c_str(); }
};
struct PythonError {};              // already set
struct Status {                     // a gemm_status other than GEMM_OK
  int value;
  const char *where;
};

PyObject *raw_stream, *gemm_error, *out_of_memory, *str_row, *str_tile;

std::string list_of(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}
std::string type_name(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kDouble: return "torch.float64";
    case at::kHalf: return "torch.float16";
    default: return c10::toString(t);
  }
}
[[noreturn]] void refuse(const std::string &what, const at::Tensor &t, const std::string &want) {
  throw Refused(what + " must be " + want + "; got " + type_name(t.scalar_type()) + " " +
                list_of(t.sizes()) + " with strides " + list_of(t.strides()));
}

// what the kernels read is the memory at data_ptr(), by strides
bool plain(const at::Tensor &t) { return t.layout() == at::kStrided && !t.is_neg(); }
[[noreturn]] void refuse_layout(const std::string &what, const at::Tensor &t) {
  throw Refused(what + (t.layout() == at::kStrided
                            ? " is a lazily negated view; pass what resolve_neg() gives"
                            : " must be a strided tensor"));
}

const at::Tensor &tensor(const std::string &what, PyObject *o) {
  if (!THPVariable_Check(o)) throw Refused(what + " must be a torch tensor");
  const at::Tensor &t = THPVariable_Unpack(o);
  if (!plain(t)) refuse_layout(what, t);
  return t;
}
// None stands for an undefined tensor
const at::Tensor &maybe(const char *what, PyObject *o) {
  static const at::Tensor none;
  return o == Py_None ? none : tensor(what, o);
}

bool is_type(at::ScalarType t) { return t == at::kFloat || t == at::kBFloat16; }
int gemm_type(at::ScalarType t) { return t == at::kFloat ? GEMM_F32 : GEMM_BF16; }

struct On {   // the GPU that all operands are on
  int device = -1;
  void operator()(const std::string &what, const at::Tensor &t) {
    if (!t.defined()) return;
    if (!t.is_cuda())
      throw Refused(what + " is on " + t.device().str() + "; every operand must be on the GPU");
    const int at = t.get_device();
    if (device < 0) device = at;
    if (at != device)
      throw Refused(what + " is on GPU " + std::to_string(at) + ", other operands on GPU " +
                    std::to_string(device));
  }
};

struct Rows {
  int64_t rows, cols, stride;
};
Rows rows_of(const char *what, const at::Tensor &t) {
  if (t.dim() != 2 || !is_type(t.scalar_type())) refuse(what, t, "a float32 or bfloat16 matrix");
  Rows r{t.size(0), t.size(1), t.stride(0)};
  if (r.cols > 1 && t.stride(1) != 1)
    refuse(what, t, "a matrix of packed rows (columns next to each other)");
  if (r.rows <= 1)
    r.stride = r.cols;
  else if (0 < r.stride && r.stride < r.cols)
    refuse(what, t, "a matrix whose rows do not overlap");
  return r;
}
void vector_of(const char *what, const at::Tensor &t, int64_t n, at::ScalarType one,
               at::ScalarType other) {
  if ((t.scalar_type() != one && t.scalar_type() != other) || t.dim() != 1 || t.size(0) != n ||
      !t.is_contiguous())
    refuse(what, t, "a packed vector of " + std::to_string(n) + ", " + type_name(one) +
                        (one == other ? "" : " or " + type_name(other)));
}

// A tensor that a call wrote into: autograd then refuses to use what it saved of it before.
void written(const at::Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

at::Tensor make(const at::Tensor &like, at::IntArrayRef sizes, at::ScalarType t) {
  return at::empty(sizes, like.options().dtype(t).requires_grad(false));
}
struct Workspace {
  at::Tensor held;
  void *ptr = nullptr;
  size_t bytes;
  Workspace(const at::Tensor &like, size_t n) : bytes(n) {
    if (n) {
      held = make(like, {(int64_t)n}, at::kByte);
      ptr = held.data_ptr();
    }
  }
};

void ok(int status, const char *where) {
  if (status != GEMM_OK) throw Status{status, where};
}
// torch's current stream of a GPU, which is made the current one as long as this lives
struct Stream {
  c10::DeviceGuard guard;
  void *ptr;
  explicit Stream(int device)
      : guard(c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)device)) {
    PyObject *index = PyLong_FromLong(device);
    PyObject *s = index ? PyObject_CallOneArg(raw_stream, index) : nullptr;
    Py_XDECREF(index);
    if (!s) throw PythonError{};
    ptr = PyLong_AsVoidPtr(s);
    Py_DECREF(s);
    if (PyErr_Occurred()) throw PythonError{};
  }
};

void *data(const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

PyObject *tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject *out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) throw PythonError{};
  Py_ssize_t i = 0;
  for (const auto &t : ts) {
    PyObject *o = t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None);
    if (!o) {
      Py_DECREF(out);
      throw PythonError{};
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

int block_of(const std::string &what, PyObject *o) {
  for (int k = 0; k < 2; ++k) {
    const int same = PyObject_RichCompareBool(o, k ? str_tile : str_row, Py_EQ);
    if (same < 0) throw PythonError{};
    if (same) return k ? GEMM_BLOCK_TILE : GEMM_BLOCK_ROW;
  }
  PyObject *r = PyObject_Repr(o);
  const char *s = r ? PyUnicode_AsUTF8(r) : nullptr;
  const std::string got = s ? s : "?";
  Py_XDECREF(r);
  PyErr_Clear();
  throw Refused(what + " must be one of ['row', 'tile']; got " + got);
}
int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m; }

// Runs a function's body and turns what it throws into Python's exceptions.
template <class F>
PyObject *guarded(F &&body) {
  try {
    return body();
  } catch (const Refused &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const Status &e) {
    if (PyObject *err = PyObject_CallFunction(gemm_error, "is", e.value, e.where)) {
      PyErr_SetObject(gemm_error, err);
      Py_DECREF(err);
    }
  } catch (const PythonError &) {
  } catch (const c10::OutOfMemoryError &e) {
    PyErr_SetString(out_of_memory, e.what_without_backtrace());
  } catch (const c10::Error &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (x, block, rows side, columns side, pow2) -> (codes, scales, codes_t, scales_t), None where not
// asked for; scales as they are stored, one row a block column
PyObject *block_quantize(PyObject *, PyObject *const *arg, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor &x = tensor("x", arg[0]);
    const Rows r = rows_of("x", x);
    const int block = block_of("block", arg[1]);
    On on;
    on("x", x);
    at::Tensor out[4];
    for (int side = 0; side < 2; ++side) {
      if (arg[2 + side] != Py_True) continue;
      const int64_t rows = side ? r.cols : r.rows, cols = side ? r.rows : r.cols;
      out[2 * side] = make(x, {rows, up(cols, 16) * 16}, at::kByte);
      out[2 * side + 1] =
          make(x, {up(cols, 128), block == GEMM_BLOCK_ROW ? rows : up(rows, 128)}, at::kFloat);
    }
    if (r.rows && r.cols) {
      const Stream s(on.device);
      const auto pitch = [&](int i) { return out[i].defined() ? out[i].size(1) : 0; };
      ok(gemm_block_quantize(x.data_ptr(), gemm_type(x.scalar_type()), r.rows, r.cols, r.stride,
                             block, arg[4] == Py_True, data(out[0]), pitch(0),
                             (float *)data(out[1]), pitch(1), data(out[2]), pitch(2),
                             (float *)data(out[3]), pitch(3), s.ptr),
         "gemm_block_quantize");
    }
    for (int i : {1, 3})
      if (out[i].defined()) out[i] = out[i].t();
    return tuple_of({out[0], out[1], out[2], out[3]});
  });
}

struct Operand {
  at::Tensor data, scales;
  int64_t rows, pitch, spitch;
  int block;
};
Operand operand(const std::string &what, PyObject *const *arg, int64_t K) {
  Operand q;
  q.block = block_of(what + ".block", arg[2]);
  q.data = tensor(what + ".data", arg[0]);
  q.scales = tensor(what + ".scales", arg[1]);
  const at::Tensor &d = q.data, &s = q.scales;
  const int64_t width = up(K, 16) * 16;
  if (d.dim() != 2 || (d.scalar_type() != at::kByte && d.scalar_type() != at::kFloat8_e4m3fn) ||
      d.size(1) != width)
    refuse(what + ".data", d,
           "uint8 or float8_e4m3fn codes (rows, " + std::to_string(width) + ")");
  q.rows = d.size(0);
  q.pitch = q.rows > 1 && width ? d.stride(0) : width;
  if ((width > 1 && d.stride(1) != 1) || q.pitch < width || q.pitch % 16)
    refuse(what + ".data", d, "packed rows at multiples of 16 bytes");
  const int64_t kb = up(K, 128), sr = q.block == GEMM_BLOCK_ROW ? q.rows : up(q.rows, 128);
  if (s.scalar_type() != at::kFloat || s.dim() != 2 || s.size(0) != sr || s.size(1) != kb)
    refuse(what + ".scales", s,
           "float32 (" + std::to_string(sr) + ", " + std::to_string(kb) + ")");
  q.spitch = kb > 1 ? s.stride(1) : sr;
  if ((sr > 1 && s.stride(0) != 1) || q.spitch < sr)
    refuse(what + ".scales", s,
           "stored with the scales of one block column next to each other (the transpose of a "
           "packed matrix)");
  return q;
}
bool packed(const at::Tensor &t, int64_t M, int64_t N) {
  return is_type(t.scalar_type()) && t.dim() == 2 && t.size(0) == M && t.size(1) == N &&
         t.is_contiguous();
}

// (a.data, a.scales, a.block, b.data, b.scales, b.block, K, pow2, fp32 out, bias, source, out, exact)
// -> C
PyObject *block_gemm(PyObject *, PyObject *const *arg, Py_ssize_t) {
  return guarded([&] {
    const int64_t K = PyLong_AsLongLong(arg[6]);
    if (K < 0) {
      if (PyErr_Occurred()) throw PythonError{};
      throw Refused("K must not be negative");
    }
    const Operand a = operand("a", arg, K), b = operand("b", arg + 3, K);
    if (a.block != GEMM_BLOCK_ROW)
      throw Refused("a must have block \"row\": one scale per row and 128 columns");
    const int64_t M = a.rows, N = b.rows;
    const at::Tensor &bias = maybe("bias_col", arg[9]), &source = maybe("source", arg[10]);
    at::Tensor out = maybe("out", arg[11]);
    const std::string shape =
        "a packed float32 or bfloat16 matrix (" + std::to_string(M) + ", " + std::to_string(N) + ")";
    if (out.defined() && !packed(out, M, N)) refuse("out", out, shape);
    if (bias.defined()) vector_of("bias_col", bias, N, at::kFloat, at::kFloat);
    if (source.defined() && !packed(source, M, N)) refuse("source", source, shape);
    On on;
    on("a", a.data);
    on("a.scales", a.scales);
    on("b", b.data);
    on("b.scales", b.scales);
    on("bias_col", bias);
    on("source", source);
    on("out", out);
    const bool given = out.defined();
    if (!given) out = make(a.data, {M, N}, arg[8] == Py_True ? at::kFloat : at::kBFloat16);
    if (M && N) {
      gemm_block_desc d{};
      d.M = M;
      d.N = N;
      d.K = K;
      d.lda = a.pitch;
      d.ldb = b.pitch;
      d.scale_lda = a.spitch;
      d.scale_ldb = b.spitch;
      d.block_b = b.block;
      d.pow2 = arg[7] == Py_True;
      d.dtype_c = gemm_type(out.scalar_type());
      d.dtype_source = source.defined() ? gemm_type(source.scalar_type()) : GEMM_F32;
      d.exact = arg[12] == Py_True;
      size_t need = 0;
      ok(gemm_block_workspace(&d, &need), "gemm_block_workspace");
      const Stream s(on.device);
      const Workspace w(a.data, need);
      const int st = gemm_block_run(&d, a.data.data_ptr(), (const float *)a.scales.data_ptr(),
                                    b.data.data_ptr(), (const float *)b.scales.data_ptr(),
                                    out.data_ptr(), (const float *)data(bias), data(source), w.ptr,
                                    w.bytes, s.ptr);
      if (st == GEMM_ERR_INVALID_ARG)   // what else is invalid has been refused above
        throw Refused("out overlaps source, or bias_col, and is not the source itself");
      ok(st, "gemm_block_run");
    }
    if (given) written(out);
    PyObject *r = THPVariable_Wrap(out);
    if (!r) throw PythonError{};
    return r;
  });
}

// (x, rows side, columns side) -> (codes, scales, codes_t, scales_t), None where not asked for
PyObject *int8_quantize(PyObject *, PyObject *const *arg, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor &x = tensor("x", arg[0]);
    const Rows r = rows_of("x", x);
    On on;
    on("x", x);
    at::Tensor out[4];
    for (int side = 0; side < 2; ++side) {
      if (arg[1 + side] != Py_True) continue;
      const int64_t rows = side ? r.cols : r.rows, cols = side ? r.rows : r.cols;
      out[2 * side] = make(x, {rows, up(cols, 16) * 16}, at::kChar);
      out[2 * side + 1] = make(x, {rows}, at::kFloat);
      if (cols == 0) out[2 * side + 1].fill_(0x1p-120);   // rows of nothing: the smallest scale
    }
    if (r.rows && r.cols) {
      size_t need = 0;
      ok(gemm_int8_quantize_workspace(r.rows, r.cols, out[0].defined(), out[2].defined(), &need),
         "gemm_int8_quantize_workspace");
      const Stream s(on.device);
      const Workspace w(x, need);
      const auto pitch = [&](int i) { return out[i].defined() ? out[i].size(1) : 0; };
      ok(gemm_int8_quantize(x.data_ptr(), gemm_type(x.scalar_type()), r.rows, r.cols, r.stride,
                            data(out[0]), pitch(0), (float *)data(out[1]), data(out[2]), pitch(2),
                            (float *)data(out[3]), w.ptr, w.bytes, s.ptr),
         "gemm_int8_quantize");
    }
    return tuple_of({out[0], out[1], out[2], out[3]});
  });
}

// (a.data, a.scales, b.data, b.scales, K, fp32 out, bias, source, out) -> C
PyObject *int8_gemm(PyObject *, PyObject *const *arg, Py_ssize_t) {
  return guarded([&] {
    const int64_t K = PyLong_AsLongLong(arg[4]);
    if (K < 0) {
      if (PyErr_Occurred()) throw PythonError{};
      throw Refused("K must not be negative");
    }
    On on;
    at::Tensor codes[2], scales[2];
    int64_t pitch[2];
    const int64_t width = up(K, 16) * 16;
    for (int k = 0; k < 2; ++k) {
      const std::string what = k ? "b" : "a";
      codes[k] = tensor(what + ".data", arg[2 * k]);
      scales[k] = tensor(what + ".scales", arg[2 * k + 1]);
      const at::Tensor &d = codes[k], &sc = scales[k];
      if (d.dim() != 2 || d.scalar_type() != at::kChar || d.size(1) != width)
        refuse(what + ".data", d, "int8 codes (rows, " + std::to_string(width) + ")");
      pitch[k] = d.size(0) > 1 && width ? d.stride(0) : width;
      if ((width > 1 && d.stride(1) != 1) || pitch[k] < width || pitch[k] % 16)
        refuse(what + ".data", d, "packed rows at multiples of 16 bytes");
      vector_of((what + ".scales").c_str(), sc, d.size(0), at::kFloat, at::kFloat);
      on(what, d);
      on(what + ".scales", sc);
    }
    const int64_t M = codes[0].size(0), N = codes[1].size(0);
    const at::Tensor &bias = maybe("bias_col", arg[6]), &source = maybe("source", arg[7]);
    at::Tensor out = maybe("out", arg[8]);
    const std::string shape =
        "a packed float32 or bfloat16 matrix (" + std::to_string(M) + ", " + std::to_string(N) + ")";
    if (out.defined() && !packed(out, M, N)) refuse("out", out, shape);
    if (bias.defined()) vector_of("bias_col", bias, N, at::kFloat, at::kFloat);
    if (source.defined() && !packed(source, M, N)) refuse("source", source, shape);
    on("bias_col", bias);
    on("source", source);
    on("out", out);
    const bool given = out.defined();
    if (!given) out = make(codes[0], {M, N}, arg[5] == Py_True ? at::kFloat : at::kBFloat16);
    if (M && N) {
      gemm_int8_desc d{};
      d.M = M;
      d.N = N;
      d.K = K;
      d.lda = pitch[0];
      d.ldb = pitch[1];
      d.dtype_c = gemm_type(out.scalar_type());
      d.dtype_source = source.defined() ? gemm_type(source.scalar_type()) : GEMM_F32;
      size_t need = 0;
      ok(gemm_int8_workspace(&d, &need), "gemm_int8_workspace");
      const Stream s(on.device);
      const Workspace w(codes[0], need);
      const int st = gemm_int8_run(&d, codes[0].data_ptr(), (const float *)scales[0].data_ptr(),
                                   codes[1].data_ptr(), (const float *)scales[1].data_ptr(),
                                   out.data_ptr(), (const float *)data(bias), data(source), w.ptr,
                                   w.bytes, s.ptr);
      if (st == GEMM_ERR_INVALID_ARG)   // what else is invalid has been refused above
        throw Refused("out overlaps an operand, bias_col, or a source that is not out itself");
      ok(st, "gemm_int8_run");
    }
    if (given) written(out);
    PyObject *r = THPVariable_Wrap(out);
    if (!r) throw PythonError{};
    return r;
  });
}

// (x, weight, bias, eps) -> (y, mean, rstd)
PyObject *layer_norm(PyObject *, PyObject *const *arg, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor &x = tensor("x", arg[0]);
    const Rows r = rows_of("x", x);
    if (r.cols == 0) throw Refused("x has rows of no elements, which have no mean");
    const at::Tensor &w = tensor("weight", arg[1]), &b = maybe("bias", arg[2]);
    vector_of("weight", w, r.cols, at::kFloat, x.scalar_type());
    if (b.defined()) vector_of("bias", b, r.cols, w.scalar_type(), w.scalar_type());
    const double eps = PyFloat_AsDouble(arg[3]);
    if (eps == -1.0 && PyErr_Occurred()) throw PythonError{};
    On on;
    on("x", x);
    on("weight", w);
    on("bias", b);
    at::Tensor y = make(x, {r.rows, r.cols}, x.scalar_type());
    at::Tensor mean = make(x, {r.rows}, at::kFloat), rstd = make(x, {r.rows}, at::kFloat);
    if (r.rows) {
      const Stream s(on.device);
      ok(gemm_layer_norm(x.data_ptr(), gemm_type(x.scalar_type()), r.rows, r.cols, r.stride,
                         w.data_ptr(), data(b), gemm_type(w.scalar_type()), (float)eps,
                         y.data_ptr(), (float *)mean.data_ptr(), (float *)rstd.data_ptr(), s.ptr),
         "gemm_layer_norm");
    }
    return tuple_of({y, mean, rstd});
  });
}

// (dy, x, weight, mean, rstd) -> (dx, dweight, dbias)
PyObject *layer_norm_backward(PyObject *, PyObject *const *arg, Py_ssize_t) {
  return guarded([&] {
    const at::Tensor &dy = tensor("dy", arg[0]), &x = tensor("x", arg[1]);
    const Rows r = rows_of("x", x), dr = rows_of("dy", dy);
    if (r.cols == 0) throw Refused("x has rows of no elements, which have no mean");
    if (dr.rows != r.rows || dr.cols != r.cols || dy.scalar_type() != x.scalar_type())
      refuse("dy", dy, type_name(x.scalar_type()) + " " + list_of(x.sizes()) + " like x");
    const at::Tensor &w = tensor("weight", arg[2]), &mean = tensor("mean", arg[3]),
                     &rstd = tensor("rstd", arg[4]);
    vector_of("weight", w, r.cols, at::kFloat, x.scalar_type());
    vector_of("mean", mean, r.rows, at::kFloat, at::kFloat);
    vector_of("rstd", rstd, r.rows, at::kFloat, at::kFloat);
    On on;
    on("dy", dy);
    on("x", x);
    on("weight", w);
    on("mean", mean);
    on("rstd", rstd);
    at::Tensor dx = make(x, {r.rows, r.cols}, x.scalar_type());
    at::Tensor dw = make(w, {r.cols}, w.scalar_type()), db = make(w, {r.cols}, w.scalar_type());
    size_t need = 0;
    ok(gemm_layer_norm_backward_workspace(r.rows, r.cols, &need),
       "gemm_layer_norm_backward_workspace");
    const Stream s(on.device);
    const Workspace ws(x, need);
    ok(gemm_layer_norm_backward(dy.data_ptr(), dr.stride, x.data_ptr(), r.stride,
                                gemm_type(x.scalar_type()), r.rows, r.cols, w.data_ptr(),
                                gemm_type(w.scalar_type()), (const float *)mean.data_ptr(),
                                (const float *)rstd.data_ptr(), dx.data_ptr(), dw.data_ptr(),
                                db.data_ptr(), ws.ptr, ws.bytes, s.ptr),
       "gemm_layer_norm_backward");
    return tuple_of({dx, dw, db});
  });
}

struct Sequence {   // a list or tuple of Python objects, or what can be made one (which may be read once)
  PyObject *fast;
  explicit Sequence(PyObject *o) : fast(PySequence_Fast(o, "a sequence of tensors is wanted")) {
    if (!fast) throw PythonError{};
  }
  ~Sequence() { Py_DECREF(fast); }
  Sequence(const Sequence &) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  PyObject *operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// (gradients, out or None, max_norm or None) -> norm
PyObject *norm(PyObject *, PyObject *const *arg, Py_ssize_t) {
  return guarded([&] {
    const Sequence grads(arg[0]);
    double max_norm = 0.0;
    const bool clip = arg[2] != Py_None;
    if (clip) {
      max_norm = PyFloat_AsDouble(arg[2]);
      if (PyErr_Occurred()) throw PythonError{};
      if (!(max_norm >= 0.0)) throw Refused("max_norm must not be negative or NaN");
    }
    const bool into = arg[1] != Py_None;
    const Sequence outs(into ? arg[1] : grads.fast);
    if (outs.size() != grads.size())
      throw Refused("out has " + std::to_string(outs.size()) + " tensors for " +
                    std::to_string(grads.size()) + " gradients");
    if (grads.size() == 0) throw Refused("the list of gradients is empty");
    std::vector<gemm_tensor> list((size_t)grads.size());
    int device = -1;
    for (Py_ssize_t i = 0; i < grads.size(); ++i) {
      if (!THPVariable_Check(grads[i]))
        throw Refused("gradient " + std::to_string(i) + " must be a torch tensor");
      const at::Tensor &g = THPVariable_Unpack(grads[i]);
      const auto name = [&] { return "gradient " + std::to_string(i); };
      if (!plain(g)) refuse_layout(name(), g);
      if (!is_type(g.scalar_type()) || !g.is_contiguous())
        refuse(name(), g, "packed float32 or bfloat16");
      if (!g.is_cuda() || (device >= 0 && g.get_device() != device)) {
        On on;
        on.device = device;
        on(name(), g);
      }
      device = g.get_device();
      gemm_tensor &t = list[(size_t)i];
      t.data = t.out = g.data_ptr();
      t.numel = g.numel();
      t.dtype = gemm_type(g.scalar_type());
      if (into && outs[i] != grads[i]) {
        const at::Tensor &o = tensor("out " + std::to_string(i), outs[i]);
        if (o.scalar_type() != g.scalar_type() || o.numel() != t.numel || !o.is_contiguous())
          refuse("out " + std::to_string(i), o,
                 "packed " + type_name(g.scalar_type()) + " of " + std::to_string(t.numel) +
                     " elements");
        if (!o.is_cuda() || o.get_device() != device) {
          On on;
          on.device = device;
          on("out " + std::to_string(i), o);
        }
        t.out = o.data_ptr();
      }
    }
    const at::Tensor &first = THPVariable_Unpack(grads[0]);
    const int64_t count = grads.size();
    size_t need = 0;
    ok(gemm_grad_norm_workspace(list.data(), count, &need), "gemm_grad_norm_workspace");
    const Stream s(device);
    at::Tensor out = make(first, {}, at::kFloat);
    const Workspace w(first, need);
    if (clip) {
      const int st = gemm_clip_grad_norm(list.data(), count, (float)max_norm,
                                         (float *)out.data_ptr(), w.ptr, w.bytes, s.ptr);
      if (st == GEMM_ERR_INVALID_ARG)   // what else is invalid has been refused above
        throw Refused("what is written for one gradient overlaps another one, or its output");
      ok(st, "gemm_clip_grad_norm");
      for (Py_ssize_t i = 0; i < outs.size(); ++i) written(THPVariable_Unpack(outs[i]));
    } else {
      ok(gemm_grad_norm(list.data(), count, (float *)out.data_ptr(), w.ptr, w.bytes, s.ptr),
         "gemm_grad_norm");
    }
    PyObject *r = THPVariable_Wrap(out);
    if (!r) throw PythonError{};
    return r;
  });
}

double real(const char *what, PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  if (!(v - v == 0.0)) throw Refused(std::string(what) + " must be a finite number");
  return v;
}
// One element of a type in device memory, or an undefined tensor if o is no tensor.
const at::Tensor &held(const char *what, PyObject *o, at::ScalarType type, On &on) {
  static const at::Tensor none;
  if (!THPVariable_Check(o)) return none;
  const at::Tensor &t = tensor(what, o);
  if (t.scalar_type() != type || t.numel() != 1)
    refuse(what, t, std::string(type == at::kLong ? "an int64" : "a float32") +
                        " tensor of one element, or a number");
  on(what, t);
  return t;
}

// (params, grads, m, v, m_scales, v_scales, step, lr, beta1, beta2, eps, weight_decay, norm, max_norm,
// copies) -> None
PyObject *adamw_step(PyObject *, PyObject *const *arg, Py_ssize_t) {
  return guarded([&] {
    const Sequence params(arg[0]), grads(arg[1]);
    const bool copying = arg[14] != Py_None;
    const Sequence copies(copying ? arg[14] : params.fast);
    if (params.size() == 0) throw Refused("the list of parameters is empty");
    if (grads.size() != params.size() || copies.size() != params.size())
      throw Refused("there are " + std::to_string(grads.size()) + " gradients" +
                    (copying ? " and " + std::to_string(copies.size()) + " copies" : "") + " for " +
                    std::to_string(params.size()) + " parameters");
    On on;
    std::vector<gemm_adamw_tensor> list((size_t)params.size());
    int64_t blocks = 0;
    // (names are made only for what is refused: a list of 193 takes 4 us so)
    const auto elsewhere = [&](const at::Tensor &t) {
      if (!t.is_cuda() || (on.device >= 0 && t.get_device() != on.device)) return true;
      on.device = t.get_device();
      return false;
    };
    for (Py_ssize_t i = 0; i < params.size(); ++i) {
      const auto name = [&](const char *kind) { return kind + (" " + std::to_string(i)); };
      if (!THPVariable_Check(params[i])) throw Refused(name("parameter") + " must be a torch tensor");
      if (!THPVariable_Check(grads[i])) throw Refused(name("gradient") + " must be a torch tensor");
      const at::Tensor &p = THPVariable_Unpack(params[i]), &g = THPVariable_Unpack(grads[i]);
      if (!plain(p)) refuse_layout(name("parameter"), p);
      if (!plain(g)) refuse_layout(name("gradient"), g);
      if (!is_type(p.scalar_type()) || !p.is_contiguous())
        refuse(name("parameter"), p, "packed float32 or bfloat16");
      if (!is_type(g.scalar_type()) || !g.is_contiguous() || g.sizes() != p.sizes())
        refuse(name("gradient"), g, "packed float32 or bfloat16 " + list_of(p.sizes()) +
                                        " like its parameter");
      if (elsewhere(p)) on(name("parameter"), p);
      if (elsewhere(g)) on(name("gradient"), g);
      gemm_adamw_tensor &t = list[(size_t)i];
      t = gemm_adamw_tensor{p.data_ptr(), g.data_ptr(), nullptr, p.numel(),
                            gemm_type(p.scalar_type()), gemm_type(g.scalar_type())};
      blocks += up(t.numel, 128);
      if (copying && copies[i] != Py_None) {
        const at::Tensor &c = tensor("copy", copies[i]);
        if (c.scalar_type() != at::kBFloat16 || !c.is_contiguous() || c.sizes() != p.sizes())
          refuse(name("copy"), c, "packed bfloat16 " + list_of(p.sizes()) + " like its parameter");
        if (elsewhere(c)) on(name("copy"), c);
        t.copy = c.data_ptr();
      }
    }
    gemm_adamw_desc d{};
    at::Tensor state[4];
    const char *const names[4] = {"state.m", "state.v", "state.m_scales", "state.v_scales"};
    const bool e4m3 = arg[4] != Py_None || arg[5] != Py_None;
    d.dtype_state = e4m3 ? GEMM_FP8_E4M3 : GEMM_F32;
    for (int k = 0; k < (e4m3 ? 4 : 2); ++k) {
      const at::Tensor &t = state[k] = tensor(names[k], arg[2 + k]);
      const at::ScalarType type = t.scalar_type();
      const bool codes = type == at::kByte || type == at::kFloat8_e4m3fn;
      const int64_t n = k < 2 ? blocks * 128 : blocks;
      if (t.dim() != 1 || t.size(0) != n || !t.is_contiguous() ||
          (e4m3 && k < 2 ? !codes : type != at::kFloat))
        refuse(names[k], t, std::string("a packed vector of ") + std::to_string(n) +
                                (e4m3 && k < 2 ? ", float8_e4m3fn or uint8" : ", torch.float32") +
                                ", as adamw_state gives");
      if (elsewhere(t)) on(names[k], t);
    }
    d.m = state[0].data_ptr();
    d.v = state[1].data_ptr();
    d.m_scales = (float *)data(state[2]);
    d.v_scales = (float *)data(state[3]);
    const at::Tensor &step = held("step", arg[6], at::kLong, on);
    if (step.defined()) {
      d.step_at = (const int64_t *)step.data_ptr();
    } else {
      d.step = PyLong_AsLongLong(arg[6]);
      if (d.step == -1 && PyErr_Occurred()) throw PythonError{};
      if (d.step < 1) throw Refused("step counts from 1; got " + std::to_string(d.step));
    }
    const at::Tensor &lr = held("lr", arg[7], at::kFloat, on);
    if (lr.defined())
      d.lr_at = (const float *)lr.data_ptr();
    else
      d.lr = real("lr", arg[7]);
    d.beta1 = real("beta1", arg[8]);
    d.beta2 = real("beta2", arg[9]);
    for (double b : {d.beta1, d.beta2})
      if (!(b >= 0.0 && b < 1.0)) throw Refused("betas must lie in [0, 1)");
    d.eps = real("eps", arg[10]);
    if (d.eps < 0.0) throw Refused("eps must not be negative");
    d.weight_decay = real("weight_decay", arg[11]);
    if ((arg[12] == Py_None) != (arg[13] == Py_None))
      throw Refused("norm and max_norm go together");
    if (arg[12] != Py_None) {
      const at::Tensor &norm = held("norm", arg[12], at::kFloat, on);
      if (!norm.defined()) throw Refused("norm must be a torch tensor, as grad_norm gives");
      d.norm = (const float *)norm.data_ptr();
      d.max_norm = PyFloat_AsDouble(arg[13]);
      if (d.max_norm == -1.0 && PyErr_Occurred()) throw PythonError{};
      if (!(d.max_norm >= 0.0)) throw Refused("max_norm must not be negative or NaN");
    }
    {
      const Stream s(on.device);
      const int st = gemm_adamw_step(list.data(), params.size(), &d, s.ptr);
      if (st == GEMM_ERR_INVALID_ARG)   // what else is invalid has been refused above
        throw Refused("something that is written (a parameter, a copy, the state) overlaps something else");
      ok(st, "gemm_adamw_step");
    }
    for (Py_ssize_t i = 0; i < params.size(); ++i) {
      written(THPVariable_Unpack(params[i]));
      if (list[(size_t)i].copy) written(THPVariable_Unpack(copies[i]));
    }
    for (const at::Tensor &t : state)
      if (t.defined()) written(t);
    Py_RETURN_NONE;
  });
}

#define DG_CALL(name, count)                                                                   \
  PyObject *call_##name(PyObject *self, PyObject *const *arg, Py_ssize_t n) {                  \
    if (n != count) {                                                                          \
      PyErr_SetString(PyExc_TypeError, #name " takes " #count " arguments");                   \
      return nullptr;                                                                          \
    }                                                                                          \
    return name(self, arg, n);                                                                 \
  }
DG_CALL(block_quantize, 5)
DG_CALL(block_gemm, 13)
DG_CALL(layer_norm, 4)
DG_CALL(layer_norm_backward, 5)
DG_CALL(norm, 3)
DG_CALL(int8_quantize, 3)
DG_CALL(int8_gemm, 9)
DG_CALL(adamw_step, 15)
#undef DG_CALL

#define DG_METHOD(name) {#name, (PyCFunction)(void (*)(void))call_##name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {DG_METHOD(block_quantize), DG_METHOD(block_gemm), DG_METHOD(layer_norm),
                         DG_METHOD(layer_norm_backward), DG_METHOD(norm),
                         DG_METHOD(int8_quantize), DG_METHOD(int8_gemm), DG_METHOD(adamw_step),
                         {nullptr, nullptr, 0, nullptr}};
#undef DG_METHOD
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

PyObject *attribute(const char *from, const char *name) {
  PyObject *m = PyImport_ImportModule(from);
  PyObject *o = m ? PyObject_GetAttrString(m, name) : nullptr;
  Py_XDECREF(m);
  return o;
}

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  raw_stream = attribute("torch._C", "_cuda_getCurrentRawStream");
  gemm_error = raw_stream ? attribute("dense_gemm_design_amd._lib", "GemmError") : nullptr;
  out_of_memory = gemm_error ? attribute("torch", "OutOfMemoryError") : nullptr;
  str_row = PyUnicode_InternFromString("row");
  str_tile = PyUnicode_InternFromString("tile");
  if (!raw_stream || !gemm_error || !out_of_memory || !str_row || !str_tile) return nullptr;
  return PyModule_Create(&module);
}
