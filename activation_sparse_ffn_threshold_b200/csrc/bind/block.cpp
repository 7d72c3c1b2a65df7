// block.cpp -- the calls of block.py in native code: checks of tensors, allocations, and the C entry
// points of libsfnn.so.  One token's norm takes 4 us on the GPU and 13 in Python; here most of what is
// left is the launch.
//
// A function returns its results, or the entry point's status (an int) where that is not SFNN_OK.  A
// call that is refused here raises TypeError or ValueError.  Results lie on the tensors' device and
// belong to its current stream.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/DynamicTypes.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <string>
#include <vector>

#include "sfnn.h"

namespace {

struct Refused {
  PyObject *type;
  std::string what;
};
[[noreturn]] void refuse(PyObject *type, const char *format, ...) {
  char text[400];
  va_list a;
  va_start(a, format);
  vsnprintf(text, sizeof text, format, a);
  va_end(a);
  throw Refused{type, text};
}

// A tensor whose memory holds its values (the imaginary part of a conjugate is negated when it is read).
const at::Tensor &plain(PyObject *o) {
  const at::Tensor &t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided) refuse(PyExc_TypeError, "a strided tensor was expected");
  if (t.is_neg()) refuse(PyExc_TypeError, "a tensor is negated lazily: resolve_neg() gives one that is not");
  return t;
}
const at::Tensor *tensor(PyObject *o) {  // null for None
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, "a tensor was expected, not %s", Py_TYPE(o)->tp_name);
  return &plain(o);
}
const at::Tensor &cuda_tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return plain(o);
}
std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const char *name_of(at::ScalarType t) { return c10::toString(t); }
int code_of(at::ScalarType t) {  // -1: not one of ours
  return t == at::kHalf ? SFNN_F16 : t == at::kBFloat16 ? SFNN_BF16 : t == at::kFloat ? SFNN_F32 : -1;
}
int code16(at::ScalarType t) {
  if (t != at::kHalf && t != at::kBFloat16)
    refuse(PyExc_TypeError, "the dense operators take fp16 or bf16 tensors, got %s", name_of(t));
  return code_of(t);
}

// A tensor [..., cols] as rows that lie evenly apart.
struct Rows {
  void *p;
  int64_t rows, cols, ld;
};
Rows rows_of(const at::Tensor &t, const char *name, int64_t want = -1) {
  const int64_t n = t.dim();
  if (n < 1) refuse(PyExc_ValueError, "%s must have at least one dimension", name);
  const auto size = t.sizes(), stride = t.strides();
  Rows r;
  r.p = t.data_ptr();
  r.cols = size[n - 1];
  if (want >= 0 && r.cols != want)
    refuse(PyExc_ValueError, "%s must have %lld columns, got %lld", name, (long long)want, (long long)r.cols);
  r.rows = 1;
  r.ld = r.cols;
  for (int64_t i = 0; i < n - 1; ++i) r.rows *= size[i];
  if (r.rows > 0x7fffffffll || r.cols > 0x7fffffffll)
    refuse(PyExc_ValueError, "%s: %lld rows of %lld columns do not fit 32 bits", name, (long long)r.rows, (long long)r.cols);
  if (!t.numel() || t.is_contiguous()) return r;
  if (r.cols > 1 && stride[n - 1] != 1) refuse(PyExc_ValueError, "%s: the elements of a row must be contiguous", name);
  int64_t span = -1;  // the stride that the next dimension outwards must have
  for (int64_t i = n - 2; i >= 0; --i) {
    if (size[i] == 1) continue;
    if (span < 0)
      r.ld = stride[i];
    else if (stride[i] != span)
      refuse(PyExc_ValueError, "%s: its leading dimensions must be viewable as rows", name);
    span = stride[i] * size[i];
  }
  if (r.ld < r.cols && r.rows > 1) refuse(PyExc_ValueError, "%s: rows must not overlap", name);
  if (r.rows == 1) r.ld = r.cols;
  return r;
}
// An operand of the tensor cores: 16-byte aligned rows of one type.
Rows operand(const at::Tensor &t, const char *name, at::ScalarType dtype, int64_t cols = -1) {
  if (!t.is_cuda() || t.scalar_type() != dtype) refuse(PyExc_TypeError, "%s must be a CUDA tensor of %s", name, name_of(dtype));
  const Rows r = rows_of(t, name, cols);
  if (r.rows && (reinterpret_cast<uintptr_t>(r.p) % 16 || r.ld % 8))
    refuse(PyExc_ValueError, "%s: rows must start on 16-byte boundaries and not overlap", name);
  return r;
}
void *channels(const at::Tensor *t, const char *name, int64_t d, at::ScalarType dtype, c10::Device device) {
  if (!t) return nullptr;
  if (t->device() != device || t->scalar_type() != dtype || t->dim() != 1 || t->size(0) != d || !t->is_contiguous())
    refuse(PyExc_ValueError, "%s must be a contiguous %s tensor of %lld elements on the others' device", name, name_of(dtype),
           (long long)d);
  return t->data_ptr();
}
// Whether two sets of rows of `ea` and `eb` bytes a value share memory.  Rows equally far apart may lie
// between one another (columns of one buffer); others whose ranges meet count as sharing it.
bool share(const Rows &a, int64_t ea, const Rows &b, int64_t eb) {
  if (!a.rows || !a.cols || !b.rows || !b.cols) return false;
  const int64_t la = a.ld * ea, lb = b.ld * eb, ca = a.cols * ea, cb = b.cols * eb;
  const int64_t pa = reinterpret_cast<int64_t>(a.p), pb = reinterpret_cast<int64_t>(b.p);
  if (pa + (a.rows - 1) * la + ca <= pb || pb + (b.rows - 1) * lb + cb <= pa) return false;
  const int64_t ld = a.rows > 1 ? la : lb;
  if (a.rows > 1 && b.rows > 1 && la != lb) return true;
  const int64_t off = ((pb - pa) % ld + ld) % ld;  // b's columns, from a's on
  return off < ca || off + cb > ld;
}
void apart(const Rows &out, int64_t eo, const at::Tensor *t, const char *name) {
  if (!t) return;
  if (share(out, eo, rows_of(*t, name), t->element_size())) refuse(PyExc_ValueError, "out must not overlap %s", name);
}
void same_shape(const at::Tensor &t, const char *name, at::IntArrayRef shape) {
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, "%s must have the shape %s, got %s", name, shape_text(shape).c_str(), shape_text(t.sizes()).c_str());
}
void same_device(const at::Tensor &t, c10::Device device) {
  if (t.device() != device) refuse(PyExc_ValueError, "all tensors must be on one device");
}

// What a forward pass kept, as it may come back from saved-tensor hooks.
const at::Tensor &kept(PyObject *o, const char *name, at::ScalarType dtype, at::IntArrayRef shape, c10::Device device) {
  const at::Tensor *t = tensor(o);
  if (!t || t->device() != device || t->scalar_type() != dtype || t->sizes() != shape ||
      !t->is_contiguous())
    refuse(PyExc_ValueError, "%s must be as the forward pass saved them: a contiguous %s tensor of shape %s on x's device", name,
           name_of(dtype), shape_text(shape).c_str());
  return *t;
}

// What was written in place: autograd then refuses a backward pass that saved what was there before.
void written(const at::Tensor &t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType dtype, c10::Device device) {
  return at::Tensor(at::detail::empty_cuda(size, dtype, device, c10::nullopt));
}
sfnn_stream_t stream_of(c10::Device device) {
  return reinterpret_cast<sfnn_stream_t>(c10::cuda::getCurrentCUDAStream(device.index()).stream());
}

PyObject *wrap(const at::Tensor &t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
// A tuple of new references.
PyObject *tuple(std::initializer_list<PyObject *> items) {
  PyObject *t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  bool ok = t != nullptr;
  for (PyObject *o : items) {
    ok = ok && o;
    if (t && o)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_XDECREF(o);
  }
  if (!ok) Py_CLEAR(t);
  return t;
}
// The entry points run without the interpreter's lock, as a full queue may hold a launch up.
template <class Call>
sfnn_status unlocked(Call call) {
  PyThreadState *state = PyEval_SaveThread();
  const sfnn_status s = call();  // (does not throw)
  PyEval_RestoreThread(state);
  return s;
}
PyObject *status(sfnn_status s) { return PyLong_FromLong((long)s); }

int32_t *error_word(PyObject *o) { return static_cast<int32_t *>(PyLong_AsVoidPtr(o)); }
double number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
long whole(PyObject *o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v == 1;
}
at::ScalarType dtype_of(PyObject *o) {
  if (!THPDtype_Check(o)) refuse(PyExc_TypeError, "a dtype was expected, not %s", Py_TYPE(o)->tp_name);
  return reinterpret_cast<THPDtype *>(o)->scalar_type;
}
PyObject *dtype_object(at::ScalarType t) {
  PyObject *o = reinterpret_cast<PyObject *>(torch::getTHPDtype(t));
  Py_INCREF(o);
  return o;
}

#define NATIVE_BEGIN(count)                                                                     \
  HANDLE_TH_ERRORS try {                                                                        \
    if (n != (count)) refuse(PyExc_TypeError, "%d arguments expected, got %d", (count), (int)n); \
  using namespace at
#define NATIVE_END                                  \
  }                                                 \
  catch (const Refused &r) {                        \
    PyErr_SetString(r.type, r.what.c_str());        \
    return nullptr;                                 \
  }                                                 \
  END_HANDLE_TH_ERRORS

// ------------------------------------------------------------------ linear
// The descriptor of x [..., K], w [N, K] and b.
sfnn_linear_desc linear_desc(const at::Tensor &x, const at::Tensor &w, const at::Tensor *b, int act, at::ScalarType y_dtype) {
  const at::ScalarType dt = x.scalar_type();
  sfnn_linear_desc q{};
  q.dtype = code16(dt);
  const Rows rx = operand(x, "x", dt), rw = operand(w, "w", dt, rx.cols);
  if (w.dim() != 2 || !rx.cols || rx.cols % 8 || !rw.rows)
    refuse(PyExc_ValueError, "w must be [N, K] with K a positive multiple of 8, got %s", shape_text(w.sizes()).c_str());
  if (y_dtype != dt && y_dtype != at::kFloat)
    refuse(PyExc_TypeError, "the output is %s or fp32, not %s", name_of(dt), name_of(y_dtype));
  same_device(w, x.device());
  q.T = (int32_t)rx.rows, q.K = (int32_t)rx.cols, q.N = (int32_t)rw.rows;
  q.y_dtype = code_of(y_dtype);
  q.act = act;
  q.x = rx.p, q.ldx = rx.ld;
  q.w = rw.p, q.ldw = rw.ld;
  q.b = channels(b, "b", rw.rows, dt, x.device());
  return q;
}
// Values of the output's shape and type.
Rows output(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType dtype, c10::Device device) {
  if (t.scalar_type() != dtype || t.sizes() != shape || t.device() != device)
    refuse(PyExc_ValueError, "%s must be a %s tensor of shape %s on x's device", name, name_of(dtype), shape_text(shape).c_str());
  return rows_of(t, name);
}

// (x, w, b, act, residual, out_dtype, save, out, err) -> (y, slopes)
PyObject *linear_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  NATIVE_BEGIN(9);
  const at::Tensor &x = cuda_tensor(a[0], "x"), &w = cuda_tensor(a[1], "w");
  const at::Tensor *b = tensor(a[2]), *res = tensor(a[4]), *out = tensor(a[7]);
  const int act = (int)whole(a[3]);
  const at::ScalarType dt = a[5] != Py_None ? dtype_of(a[5]) : res ? res->scalar_type() : x.scalar_type();
  const sfnn_linear_desc q = linear_desc(x, w, b, act, dt);
  const c10::Device device = x.device();
  c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = q.N;
  Rows r{nullptr, 0, 0, q.N}, ry;
  if (res) r = output(*res, "residual", shape, dt, device);
  const c10::cuda::CUDAGuard guard(device);
  at::Tensor y, slopes, ws;
  if (out) {
    ry = output(*out, "out", shape, dt, device);
    const int64_t size = out->element_size();
    apart(ry, size, &x, "x");
    apart(ry, size, &w, "w");
    apart(ry, size, b, "b");
    if (!res || r.p != ry.p || r.ld != ry.ld) apart(ry, size, res, "the residual");  // (it may be the residual)
    y = *out;
  } else {
    y = empty(shape, dt, device);
    ry = Rows{y.data_ptr(), q.T, q.N, q.N};
  }
  if (truth(a[6]) && act != SFNN_LINEAR_NONE) slopes = empty({sfnn_linear_slope_bytes(q.T, q.N, act)}, at::kByte, device);
  if (q.T) {
    const int64_t bytes = sfnn_linear_workspace(q.T, q.K, q.N, 0);
    if (bytes > 0) ws = empty({bytes}, at::kByte, device);
    void *ps = slopes.defined() ? slopes.data_ptr() : nullptr, *pw = ws.defined() ? ws.data_ptr() : nullptr;
    int32_t *err = error_word(a[8]);
    sfnn_stream_t stream = stream_of(device);
    const sfnn_status st = unlocked([&] { return sfnn_linear_forward(&q, r.p, r.ld, ry.p, ry.ld, ps, pw, bytes, err, stream); });
    if (st != SFNN_OK) return status(st);
  }
  if (out) {
    written(*out);
    Py_INCREF(a[7]);
  }
  return tuple({out ? a[7] : wrap(y), wrap(slopes)});
  NATIVE_END
}

// (dy, x, slopes, act, N, y_dtype, has_b, w, need, err) -> (dx, dw, db)
PyObject *linear_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  NATIVE_BEGIN(10);
  const at::Tensor &dy = cuda_tensor(a[0], "dy"), &x = cuda_tensor(a[1], "x"), &w = cuda_tensor(a[7], "w");
  const at::ScalarType y_dtype = dtype_of(a[5]);
  const sfnn_linear_desc q = linear_desc(x, w, nullptr, (int)whole(a[3]), y_dtype);
  if (q.N != whole(a[4])) refuse(PyExc_ValueError, "w must have the forward pass's shape");
  if (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 3) refuse(PyExc_ValueError, "need must be three truth values");
  const c10::Device device = x.device();
  c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = q.N;
  const Rows r = output(dy, "dy", shape, y_dtype, device);
  const void *ps = nullptr;
  if (q.act != SFNN_LINEAR_NONE)
    ps = kept(a[2], "slopes", at::kByte, {sfnn_linear_slope_bytes(q.T, q.N, q.act)}, device).data_ptr();
  const c10::cuda::CUDAGuard guard(device);
  const at::ScalarType dt = x.scalar_type();
  at::Tensor dx, dw, db;
  if (truth(PyTuple_GET_ITEM(a[8], 0))) dx = empty(x.sizes(), dt, device);
  if (truth(PyTuple_GET_ITEM(a[8], 1))) dw = empty(w.sizes(), dt, device);
  if (truth(PyTuple_GET_ITEM(a[8], 2)) && truth(a[6])) db = empty({q.N}, dt, device);
  const int64_t bytes = std::max<int64_t>(16, sfnn_linear_workspace(q.T, q.K, q.N, 1));
  const at::Tensor ws = empty({bytes}, at::kByte, device);
  auto p = [](const at::Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; };
  int32_t *err = error_word(a[9]);
  sfnn_stream_t stream = stream_of(device);
  const sfnn_status st = unlocked(
      [&] { return sfnn_linear_backward(&q, ps, r.p, r.ld, p(dx), p(dw), p(db), ws.data_ptr(), bytes, err, stream); });
  if (st != SFNN_OK) return status(st);
  return tuple({wrap(dx), wrap(dw), wrap(db)});
  NATIVE_END
}

// ------------------------------------------------------------------ norms
struct NormInputs {
  const at::Tensor *x, *z, *gate, *w, *b, *post_w, *post_b;
};
NormInputs norm_inputs(PyObject *const *a) {
  NormInputs t;
  t.x = &cuda_tensor(a[0], "x");
  const at::Tensor **rest[6] = {&t.z, &t.gate, &t.w, &t.b, &t.post_w, &t.post_b};
  for (int i = 0; i < 6; ++i) *rest[i] = tensor(a[1 + i]);
  return t;
}
// Values [..., d] of the 16-bit type or fp32.
Rows values(const at::Tensor &t, const char *name, at::ScalarType dtype, const at::Tensor &like, int *code) {
  same_device(t, like.device());
  const at::ScalarType dt = t.scalar_type();
  if (dt != dtype && dt != at::kFloat)
    refuse(PyExc_TypeError, "%s must be a tensor of fp32 or %s, got %s", name, name_of(dtype), name_of(dt));
  if (&t != &like) same_shape(t, name, like.sizes());
  *code = code_of(dt);
  return rows_of(t, name);
}
// The descriptor; `dtype` is the 16-bit type, found where it is not given (kUndefined).
sfnn_norm_desc norm_desc(const NormInputs &t, PyObject *const *o, at::ScalarType &dtype) {
  sfnn_norm_desc q{};
  q.pre = (int32_t)whole(o[0]), q.post = (int32_t)whole(o[1]);
  q.residual_scale = (float)number(o[2]), q.branch_scale = (float)number(o[3]), q.eps = (float)number(o[4]);
  for (const at::Tensor *p : {t.w, t.x, t.z, t.gate, t.b, t.post_w, t.post_b})  // the first one's that has one
    if (dtype == at::ScalarType::Undefined && p && p->scalar_type() != at::kFloat) dtype = p->scalar_type();
  if (dtype == at::ScalarType::Undefined) {
    if (q.pre) refuse(PyExc_TypeError, "dtype (fp16 or bf16) must be given where x, z and the weights do not tell it");
    dtype = at::kHalf;
  }
  if (dtype != at::kHalf && dtype != at::kBFloat16) refuse(PyExc_TypeError, "the norms give fp16 or bf16, not %s", name_of(dtype));
  q.dtype = code_of(dtype);
  const c10::Device device = t.x->device();
  const Rows x = values(*t.x, "x", dtype, *t.x, &q.x_dtype);
  q.T = (int32_t)x.rows, q.d = (int32_t)x.cols;
  q.x = x.p, q.ldx = x.ld;
  q.z_dtype = q.x_dtype;
  if (t.z) {
    const Rows z = values(*t.z, "z", dtype, *t.x, &q.z_dtype);
    q.z = z.p, q.ldz = z.ld;
  } else if (q.post || t.gate || !q.pre || q.residual_scale != 1.f) {
    refuse(PyExc_ValueError, "without z there is neither a post norm, a gate nor a residual scale, and a pre norm must be given");
  }
  if (x.cols < 1 || x.cols > 32768) refuse(PyExc_ValueError, "the norms take rows of 1 to 32768 values, got %lld", (long long)x.cols);
  if (t.gate) {
    if (t.gate->dim() == 1) {
      q.gate = channels(t.gate, "gate", x.cols, dtype, device);
    } else {
      int code;
      const Rows g = values(*t.gate, "gate", dtype, *t.x, &code);
      if (code == SFNN_F32) refuse(PyExc_TypeError, "gate must be a CUDA tensor of %s", name_of(dtype));
      q.gate = g.p, q.ldg = g.ld;
    }
  }
  if ((!q.pre && (t.w || t.b)) || (!q.post && (t.post_w || t.post_b)))
    refuse(PyExc_ValueError, "weights are given for a norm that is not there");
  q.w = channels(t.w, "w", x.cols, dtype, device);
  q.b = channels(t.b, "b", x.cols, dtype, device);
  q.post_w = channels(t.post_w, "post_w", x.cols, dtype, device);
  q.post_b = channels(t.post_b, "post_b", x.cols, dtype, device);
  return q;
}

// (x, z, gate, w, b, post_w, post_b, pre, post, residual_scale, branch_scale, eps, dtype, save, out, err)
// -> (r, h, stats, dtype)
PyObject *norm_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  NATIVE_BEGIN(16);
  const NormInputs t = norm_inputs(a);
  at::ScalarType dtype = a[12] == Py_None ? at::ScalarType::Undefined : dtype_of(a[12]);
  const sfnn_norm_desc q = norm_desc(t, a + 7, dtype);
  const bool save = truth(a[13]);
  const at::Tensor *out = tensor(a[14]);
  const c10::Device device = t.x->device();
  Rows r{nullptr, 0, 0, q.d};
  if (out) {
    if (!t.z) refuse(PyExc_ValueError, "without z nothing is written to out: r is x");
    int code;
    r = values(*out, "out", dtype, *t.x, &code);
    if (code != q.x_dtype) refuse(PyExc_ValueError, "out must be a tensor of x's type on its device");
    if (save && r.p == q.x) refuse(PyExc_ValueError, "x is needed by the backward pass: out must not be x");
    const int64_t size = out->element_size();
    if (r.p != q.x || r.ld != q.ldx) apart(r, size, t.x, "x but for x itself");
    apart(r, size, t.z, "z");
    apart(r, size, t.gate, "gate");
    apart(r, size, t.w, "w");
    apart(r, size, t.b, "b");
    apart(r, size, t.post_w, "post_w");
    apart(r, size, t.post_b, "post_b");
  }
  const c10::cuda::CUDAGuard guard(device);
  at::Tensor made, h, stats;
  if (t.z && !out) {
    made = empty(t.x->sizes(), t.x->scalar_type(), device);
    r.p = made.data_ptr();
  }
  if (q.pre) h = empty(t.x->sizes(), dtype, device);
  if (save) stats = empty({q.T, 4}, at::kFloat, device);
  void *ph = h.defined() ? h.data_ptr() : nullptr;
  float *ps = save ? stats.data_ptr<float>() : nullptr;
  int32_t *err = error_word(a[15]);
  sfnn_stream_t stream = stream_of(device);
  const sfnn_status st = unlocked([&] { return sfnn_norm_forward(&q, r.p, r.ld, ph, q.d, ps, err, stream); });
  if (st != SFNN_OK) return status(st);
  if (out) written(*out);
  PyObject *given = out ? a[14] : t.z ? nullptr : a[0];  // r is out, or x itself
  Py_XINCREF(given);
  return tuple({given ? given : wrap(made), wrap(h), wrap(stats), dtype_object(dtype)});
  NATIVE_END
}

// (x, z, gate, w, b, post_w, post_b, pre, post, residual_scale, branch_scale, eps, dtype, stats, dr, dh,
// need, err) -> the seven gradients
PyObject *norm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  NATIVE_BEGIN(18);
  const NormInputs t = norm_inputs(a);
  at::ScalarType dtype = dtype_of(a[12]);
  const sfnn_norm_desc q = norm_desc(t, a + 7, dtype);
  const c10::Device device = t.x->device();
  const at::Tensor &stats = kept(a[13], "stats", at::kFloat, {q.T, 4}, device);
  const at::Tensor *dr = tensor(a[14]), *dh = tensor(a[15]);
  Rows r{nullptr, 0, 0, 0}, h{nullptr, 0, 0, 0};
  int code;
  if (dr) {
    r = values(*dr, "dr", dtype, *t.x, &code);
    if (code != q.x_dtype) refuse(PyExc_TypeError, "dr must be a tensor of %s", name_of(t.x->scalar_type()));
  }
  if (dh) {
    if (!q.pre) refuse(PyExc_ValueError, "the forward pass made no h");
    h = values(*dh, "dh", dtype, *t.x, &code);
    if (code != q.dtype) refuse(PyExc_TypeError, "dh must be a tensor of %s", name_of(dtype));
  }
  if (!PyTuple_Check(a[16]) || PyTuple_GET_SIZE(a[16]) != 7) refuse(PyExc_ValueError, "need must be seven truth values");
  const c10::cuda::CUDAGuard guard(device);
  const at::Tensor *of[7] = {t.x, t.z, t.gate, t.w, t.b, t.post_w, t.post_b};
  at::Tensor grad[7];
  void *p[7] = {};
  for (int i = 0; i < 7; ++i)
    if (of[i] && truth(PyTuple_GET_ITEM(a[16], i))) {
      grad[i] = empty(of[i]->sizes(), of[i]->scalar_type(), device);
      p[i] = grad[i].data_ptr();
    }
  const int64_t bytes = sfnn_norm_workspace(q.T, q.d);
  const at::Tensor ws = empty({bytes}, at::kByte, device);
  const float *ps = stats.data_ptr<float>();
  int32_t *err = error_word(a[17]);
  sfnn_stream_t stream = stream_of(device);
  const sfnn_status st = unlocked([&] {
    return sfnn_norm_backward(&q, ps, r.p, r.ld, h.p, h.ld, p[0], p[1], p[2], p[3], p[4], p[5], p[6], ws.data_ptr(), bytes, err,
                              stream);
  });
  if (st != SFNN_OK) return status(st);
  return tuple({wrap(grad[0]), wrap(grad[1]), wrap(grad[2]), wrap(grad[3]), wrap(grad[4]), wrap(grad[5]), wrap(grad[6])});
  NATIVE_END
}

// ------------------------------------------------------------------ clipping
// (grads, outs or None, max_norm, scale, eps) -> norm; grads and outs are lists
PyObject *clip_grad_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  NATIVE_BEGIN(5);
  if (!PyList_Check(a[0]) || (a[1] != Py_None && !PyList_Check(a[1]))) refuse(PyExc_TypeError, "lists of tensors were expected");
  const Py_ssize_t count = PyList_GET_SIZE(a[0]);
  const bool apart = a[1] != Py_None;
  if (!count) refuse(PyExc_ValueError, "there are no gradients");
  if (apart && PyList_GET_SIZE(a[1]) != count)
    refuse(PyExc_ValueError, "%d gradients, but %d outputs", (int)count, (int)PyList_GET_SIZE(a[1]));
  const double max_norm = number(a[2]), scale = number(a[3]), eps = number(a[4]);
  if (!(max_norm >= 0 && eps >= 0 && scale >= 0 && std::isfinite(scale)))
    refuse(PyExc_ValueError, "max_norm, scale and eps must not be negative, nor scale infinite");
  const c10::Device device = cuda_tensor(PyList_GET_ITEM(a[0], 0), "a gradient").device();
  std::vector<sfnn_grad> table((size_t)count);
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor &g = cuda_tensor(PyList_GET_ITEM(a[0], i), "a gradient");
    same_device(g, device);
    const int code = code_of(g.scalar_type());
    if (code < 0) refuse(PyExc_TypeError, "gradients are fp16, bf16 or fp32, got %s", name_of(g.scalar_type()));
    if (!g.is_contiguous() && !g.is_non_overlapping_and_dense())
      refuse(PyExc_ValueError, "a gradient's values must lie without gaps");
    void *to = g.data_ptr();
    if (apart) {
      const at::Tensor &o = cuda_tensor(PyList_GET_ITEM(a[1], i), "an output");
      same_device(o, device);
      const bool alike = o.numel() == g.numel() && o.scalar_type() == g.scalar_type() &&
                         ((o.is_contiguous() && g.is_contiguous()) || (o.sizes() == g.sizes() && o.strides() == g.strides()));
      if (!alike) refuse(PyExc_ValueError, "each output must have its gradient's type, size and order of values");
      to = o.data_ptr();
    }
    table[(size_t)i] = sfnn_grad{g.data_ptr(), to, g.numel(), code};
  }
  const c10::cuda::CUDAGuard guard(device);
  at::Tensor norm = empty({}, at::kFloat, device);
  const int64_t bytes = sfnn_clip_workspace((int32_t)count);
  const at::Tensor ws = empty({bytes}, at::kByte, device);
  float *pn = norm.data_ptr<float>();
  sfnn_stream_t stream = stream_of(device);
  const sfnn_status st = unlocked([&] {
    return sfnn_clip_grad_norm(table.data(), (int32_t)count, (float)max_norm, (float)scale, (float)eps, pn, ws.data_ptr(), bytes,
                               stream);
  });
  if (st != SFNN_OK) return status(st);
  for (Py_ssize_t i = 0; i < count; ++i) written(*tensor(PyList_GET_ITEM(apart ? a[1] : a[0], i)));
  return wrap(norm);
  NATIVE_END
}

PyMethodDef methods[] = {
    {"linear_forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(linear_forward)), METH_FASTCALL, nullptr},
    {"linear_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(linear_backward)), METH_FASTCALL, nullptr},
    {"norm_forward", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_forward)), METH_FASTCALL, nullptr},
    {"norm_backward", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(norm_backward)), METH_FASTCALL, nullptr},
    {"clip_grad_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(clip_grad_norm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block(void) { return PyModule_Create(&module); }
