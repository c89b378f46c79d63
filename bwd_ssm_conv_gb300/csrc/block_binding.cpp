// block_binding.cpp -- the Python module behind block.py: takes PyTorch tensors apart, checks what
// the C ABI (ssm_block.h) cannot see, makes the results and calls the entry point on the stream.
// No computation happens here.
//
// The host is all that bounds a call for a token or a small layer, so the marshalling is compiled:
// add_norm's forward and backward of a small fp32 layer take the host 14 us (three launches and seven
// allocations) where the same checks in Python took 38, a token's call 2.9 where it took 7.3.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <optional>

#include "ssm.h"
#include "ssm_block.h"

namespace {

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

constexpr int64_t kBlock = 32;  // columns per scale of a checkpoint
PyTypeObject* ckpt8_type = nullptr;  // block.Ckpt8

// ---- arguments ----------------------------------------------------------------------------------
const Tensor* tensor(PyObject* o, const char* name) {  // nullptr for None
  if (o == Py_None) return nullptr;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& needed(PyObject* o, const char* name) {
  const Tensor* t = tensor(o, name);
  TORCH_CHECK_TYPE(t, name, " must be a tensor");
  return *t;
}
int io_code(ScalarType s) {
  return s == at::kFloat ? SSM_F32 : (s == at::kBFloat16 ? SSM_BF16 : -1);
}
int io_of(const Tensor& t, const char* name) {
  const int io = io_code(t.scalar_type());
  TORCH_CHECK_TYPE(io >= 0, name, " must be float32 or bfloat16, got ", t.scalar_type());
  return io;
}
// Every tensor of a call lies on the GPU of its first.
struct Named {
  const Tensor* t;  // nullptr: not given
  const char* name;
};
Named some(const Tensor& t, const char* name) { return {t.defined() ? &t : nullptr, name}; }
void together(Named first, std::initializer_list<Named> others) {
  TORCH_CHECK_VALUE(first.t->is_cuda(), first.name, " must be a CUDA tensor");
  const at::Device home = first.t->device();
  for (const Named& o : others)
    TORCH_CHECK_VALUE(!o.t || o.t->device() == home, o.name, " must be a CUDA tensor on ", home,
                      ", as ", first.name, " is; got ", o.t->device());
}
int64_t columns(const Tensor& t, const char* name) {
  TORCH_CHECK_VALUE(t.dim() >= 1, name, " must have at least one dimension");
  return t.size(-1);
}
int64_t rows_in(const Tensor& t, int64_t cols) { return cols ? t.numel() / cols : 0; }

// The one stride between the rows of a tensor that is not contiguous.
int64_t row_stride(const Tensor& t, const char* name) {
  const int64_t cols = t.size(-1);
  TORCH_CHECK_VALUE(cols <= 1 || t.stride(-1) == 1, name, "'s last dimension must be dense");
  int64_t ld = -1, span = 0;  // outer dimensions step over whole inner ones
  for (int64_t d = t.dim() - 2; d >= 0; d--) {
    const int64_t size = t.size(d), stride = t.stride(d);
    if (size == 1) continue;
    if (ld < 0) {
      ld = stride, span = size * stride;
    } else {
      TORCH_CHECK_VALUE(stride == span, name, "'s rows must lie at one stride");
      span *= size;
    }
  }
  if (ld < 0) ld = cols;
  TORCH_CHECK_VALUE(ld >= cols, name, "'s rows must not overlap");
  return ld;
}

// An activation [..., cols]: its pointer and row stride (0: rows without gaps).
struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
  Rows() {}
  Rows(const Tensor* t, const char* name) {
    if (!t) return;
    TORCH_CHECK_VALUE(t->is_cuda(), name, " must be a CUDA tensor");
    p = t->data_ptr();
    if (!t->is_contiguous()) ld = row_stride(*t, name);
  }
  Rows(const Tensor* t, const char* name, IntArrayRef shape, ScalarType dtype) {
    if (!t) return;
    TORCH_CHECK_VALUE(t->is_cuda(), name, " must be a CUDA tensor");
    TORCH_CHECK_VALUE(t->sizes() == shape, name, " must have shape ", shape, ", got ", t->sizes());
    TORCH_CHECK_TYPE(t->scalar_type() == dtype, name, " must be ", dtype, ", got ",
                     t->scalar_type());
    *this = Rows(t, name);
  }
};

// A contiguous fp32 tensor of n elements.
float* f32(const Tensor* t, const char* name, int64_t n) {
  if (!t) return nullptr;
  TORCH_CHECK_VALUE(t->scalar_type() == at::kFloat && t->is_cuda() && t->numel() == n &&
                        t->is_contiguous(),
                    name, " must be a contiguous fp32 CUDA tensor of ", n, " elements");
  return (float*)t->data_ptr();
}

// ---- 8-bit checkpoints ------------------------------------------------------------------------
struct Kept {
  int8_t* q = nullptr;
  uint8_t* e = nullptr;
};
at::DimVector scale_shape(IntArrayRef shape) {
  at::DimVector s(shape.begin(), shape.end());
  s.back() = (s.back() + kBlock - 1) / kBlock;
  return s;
}
// The two tensors of a checkpoint (a pair); nullptr for anything that is not a tuple.
struct Pair {
  const Tensor* q = nullptr;
  const Tensor* e = nullptr;
  Pair(PyObject* o, const char* name) {
    if (!PyTuple_Check(o)) return;
    TORCH_CHECK_VALUE(PyTuple_GET_SIZE(o) == 2, name, " must be a pair of tensors (q, e)");
    q = &needed(PyTuple_GET_ITEM(o, 0), name);
    e = &needed(PyTuple_GET_ITEM(o, 1), name);
  }
};
Kept kept(const Pair& c, const char* name, IntArrayRef shape) {
  if (!c.q) return {};
  const Tensor &q = *c.q, &e = *c.e;
  TORCH_CHECK_VALUE(q.scalar_type() == at::kChar && e.scalar_type() == at::kByte && q.is_cuda() &&
                        e.is_cuda() && q.is_contiguous() && e.is_contiguous(),
                    name, " must hold contiguous int8 and uint8 CUDA tensors");
  TORCH_CHECK_VALUE(q.sizes() == shape && e.sizes() == scale_shape(shape), name,
                    " must hold an activation of shape ", shape, ", got ", q.sizes(),
                    " with scales ", e.sizes());
  return {(int8_t*)q.data_ptr(), (uint8_t*)e.data_ptr()};
}

// ---- results ------------------------------------------------------------------------------------
Tensor make(IntArrayRef shape, ScalarType dtype, const Tensor& like) {
  return at::Tensor(at::detail::empty_cuda(shape, dtype, like.device(), std::nullopt));
}
struct NewCkpt8 {
  Tensor q, e;
  NewCkpt8() {}
  NewCkpt8(bool want, const Tensor& like) {
    if (!want) return;
    q = make(like.sizes(), at::kChar, like);
    e = make(scale_shape(like.sizes()), at::kByte, like);
  }
  int8_t* pq() const { return q.defined() ? (int8_t*)q.data_ptr() : nullptr; }
  uint8_t* pe() const { return e.defined() ? (uint8_t*)e.data_ptr() : nullptr; }
};
template <typename T = void> T* ptr(const Tensor& t) {
  return t.defined() ? (T*)t.data_ptr() : nullptr;
}

// New references; nullptr with the exception set when there is no memory for them.
PyObject* give(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* pack(std::initializer_list<PyObject*> items) {  // takes the references
  PyObject* r = PyTuple_New((Py_ssize_t)items.size());
  bool ok = r != nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    ok = ok && o;
    if (r) PyTuple_SET_ITEM(r, i++, o);
    else Py_XDECREF(o);
  }
  if (!ok) Py_CLEAR(r);
  return r;
}
PyObject* give(const NewCkpt8& c) {
  if (!c.q.defined()) Py_RETURN_NONE;
  PyObject* pair = pack({give(c.q), give(c.e)});
  if (!pair) return nullptr;
  PyObject* args = PyTuple_Pack(1, pair);
  Py_DECREF(pair);
  if (!args) return nullptr;
  PyObject* r = PyTuple_Type.tp_new(ckpt8_type, args, nullptr);
  Py_DECREF(args);
  return r;
}

// ---- streams and workspaces -----------------------------------------------------------------------
int64_t int_attr(PyObject* o, const char* name) {
  PyObject* v = PyObject_GetAttrString(o, name);
  if (!v) throw python_error();
  const int64_t r = (int64_t)PyLong_AsUnsignedLongLongMask(v);
  Py_DECREF(v);
  if (r == -1 && PyErr_Occurred()) throw python_error();
  return r;
}
// The call's device, that of its first tensor t, and its stream: the current one there, or a
// torch.cuda.Stream of it.  Both are current while this object lives.  What the call allocates
// therefore comes from the memory of the stream that it runs on: a block that was freed with work
// pending on the caller's stream is never handed to another one.  Made before anything is allocated.
struct On {
  c10::cuda::OptionalCUDAGuard device;       // only where another device is current
  c10::cuda::OptionalCUDAStreamGuard guard;  // only for another stream
  const c10::cuda::CUDAStream now;
  void* raw;
  On(PyObject* stream, const Tensor& t)
      : now(c10::cuda::getCurrentCUDAStream(t.device().index())), raw(now.stream()) {
    const at::Device home = t.device();
    if (stream != Py_None) {
      const c10::Stream s = c10::Stream::unpack3(
          int_attr(stream, "stream_id"), (c10::DeviceIndex)int_attr(stream, "device_index"),
          (c10::DeviceType)int_attr(stream, "device_type"));
      TORCH_CHECK_VALUE(s.device() == home, "stream must be one of ", home,
                        ", where the tensors are; got one of ", s.device());
      raw = (void*)(uintptr_t)int_attr(stream, "cuda_stream");
      if (s != now.unwrap()) guard.reset_stream(s);
    }
    if (c10::cuda::current_device() != home.index()) device.set_index(home.index());
  }
  // Results made for another stream are marked as used on the caller's current one too, so that
  // freeing them with work pending there does not give their memory to the other stream's next call.
  void made(std::initializer_list<const Tensor*> ts) const {
    if (!guard.current_stream()) return;
    for (const Tensor* t : ts)
      if (t->defined()) t->record_stream(now.unwrap());
  }
};

struct Workspace {
  Tensor mine;
  void* p;
  size_t bytes;
  Workspace(size_t need, const Tensor* given, const Tensor& like) : bytes(need < 256 ? 256 : need) {
    if (given) {
      bytes = given->numel() * given->element_size();
      TORCH_CHECK_VALUE(given->is_cuda() && given->is_contiguous() && bytes >= need,
                        "workspace too small (or not a contiguous CUDA tensor)");
      p = given->data_ptr();
    } else {
      mine = make({(int64_t)bytes}, at::kByte, like);
      p = mine.data_ptr();
    }
  }
};

ssm_norm_desc norm_desc(int64_t rows, int64_t cols, int64_t group, int io, int res_io,
                        unsigned flags, double eps) {
  const auto in_int = [](int64_t v) { return v > 0x7fffffff || v < 0 ? -1 : (int)v; };
  ssm_norm_desc d{};
  d.rows = rows, d.cols = in_int(cols), d.group = in_int(group);
  d.io = io, d.res_io = res_io, d.flags = flags, d.eps = (float)eps;
  return d;
}

bool yes(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
void args_are(Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n);
}
// Preallocated results, a tuple of n.
void outs_are(PyObject* o, Py_ssize_t n, const char* what) {
  TORCH_CHECK_VALUE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == n, "out must be ", what);
}

// Runs an entry point without the interpreter's lock, as a launch may wait for the GPU's queue.
template <typename F> int call(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f();
  Py_END_ALLOW_THREADS
  return rc;
}

// Every function here returns its results as a tuple, or the entry point's status where that is not
// SSM_OK.
#define SSM_FUNCTION(name) PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t n)

// x, w, residual, scale, eps, res_dtype, save8, save_x8, save_out8, want_res, want_rstd, out, stream
SSM_FUNCTION(add_norm_fwd) {
  HANDLE_TH_ERRORS
  args_are(n, 13);
  const Tensor& x = needed(a[0], "x");
  const Tensor *w = tensor(a[1], "w"), *residual = tensor(a[2], "residual"),
               *scale = tensor(a[3], "scale");
  const int io = io_of(x, "x");
  const IntArrayRef shape = x.sizes();
  const int64_t cols = columns(x, "x");
  ScalarType rdt = x.scalar_type();
  if (residual) {
    rdt = residual->scalar_type();
  } else if (a[5] != Py_None) {
    TORCH_CHECK_TYPE(THPDtype_Check(a[5]), "res_dtype must be a torch.dtype");
    rdt = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
  }
  const bool given = a[11] != Py_None;
  const Tensor *go = nullptr, *gr = nullptr;
  if (given) {
    outs_are(a[11], 2, "(out, res_out)");
    go = tensor(PyTuple_GET_ITEM(a[11], 0), "out"), gr = tensor(PyTuple_GET_ITEM(a[11], 1), "res_out");
  }
  together({&x, "x"}, {{w, "w"}, {residual, "residual"}, {scale, "scale"}, {go, "out"},
                       {gr, "res_out"}});
  const Rows rx(&x, "x"), rr(residual, "residual", shape, rdt);
  const float *ps = f32(scale, "scale", cols), *pw = f32(w, "w", cols);
  const On on(a[12], x);
  Tensor o, res;
  Rows ro, rs;
  if (given) {
    ro = Rows(go, "out", shape, x.scalar_type()), rs = Rows(gr, "res_out", shape, rdt);
    if (go) o = *go;
    if (gr) res = *gr;
  } else {
    o = make(shape, x.scalar_type(), x);
    ro.p = o.data_ptr();
    if (yes(a[9])) {
      res = make(shape, rdt, x);
      rs.p = res.data_ptr();
    }
  }
  Tensor rstd;
  if (yes(a[10])) rstd = make(shape.slice(0, shape.size() - 1), at::kFloat, x);
  const NewCkpt8 res8(yes(a[6]), x), x8(yes(a[7]), x), out8(yes(a[8]), x);
  const ssm_norm_desc d =
      norm_desc(rows_in(x, cols), cols, 0, io, io_code(rdt), 0, number(a[4]));
  on.made({&rstd, &res8.q, &res8.e, &x8.q, &x8.e, &out8.q, &out8.e});
  if (!given) on.made({&o, &res});
  const int rc = call([&] {
    return ssm_add_norm_fwd(&d, rx.p, rx.ld, rr.p, rr.ld, ps, pw, ro.p, ro.ld, rs.p, rs.ld,
                            ptr<float>(rstd), res8.pq(), res8.pe(), x8.pq(), x8.pe(), out8.pq(),
                            out8.pe(), on.raw);
  });
  if (rc) return PyLong_FromLong(rc);
  return pack({give(o), give(res), give(rstd), give(res8), give(x8), give(out8)});
  END_HANDLE_TH_ERRORS
}

// d_out, res, rstd, w, d_res_out, scale, x, res_dtype, want_dres, want_dx, ws, out, stream
SSM_FUNCTION(add_norm_bwd) {
  HANDLE_TH_ERRORS
  args_are(n, 13);
  const Tensor& d_out = needed(a[0], "d_out");
  const Pair res8(a[1], "res"), x8(a[6], "x");
  const Tensor *res = res8.q ? nullptr : &needed(a[1], "res"),
               *x = x8.q ? nullptr : tensor(a[6], "x");
  const Tensor *rstd = tensor(a[2], "rstd"), *w = tensor(a[3], "w"),
               *up = tensor(a[4], "d_res_out"), *scale = tensor(a[5], "scale");
  const int io = io_of(d_out, "d_out");
  const IntArrayRef shape = d_out.sizes();
  const ScalarType dt = d_out.scalar_type();
  const int64_t cols = columns(d_out, "d_out"), rows = rows_in(d_out, cols);
  ScalarType rdt = dt;
  if (up) {
    rdt = up->scalar_type();
  } else if (res) {
    rdt = res->scalar_type();
  } else if (a[7] != Py_None) {
    TORCH_CHECK_TYPE(THPDtype_Check(a[7]), "res_dtype must be a torch.dtype");
    rdt = reinterpret_cast<THPDtype*>(a[7])->scalar_type;
  }
  Tensor g[4];  // d_res, d_x, d_w, d_scale
  const bool given = a[11] != Py_None;
  if (given) {
    outs_are(a[11], 4, "d_res, d_x, d_w and d_scale");
    for (int i = 0; i < 4; i++)
      if (const Tensor* t = tensor(PyTuple_GET_ITEM(a[11], i), "out")) g[i] = *t;
  }
  const Tensor* given_ws = tensor(a[10], "ws");
  together({&d_out, "d_out"},
           {{res, "res"}, {res8.q, "res"}, {res8.e, "res"}, {rstd, "rstd"}, {w, "w"},
            {up, "d_res_out"}, {scale, "scale"}, {x, "x"}, {x8.q, "x"}, {x8.e, "x"}, some(g[0], "d_res"),
            some(g[1], "d_x"), some(g[2], "d_w"), some(g[3], "d_scale"), {given_ws, "ws"}});
  const Rows rd(&d_out, "d_out"), ru(up, "d_res_out", shape, rdt), rr(res, "res", shape, rdt);
  const Kept kr = kept(res8, "res", shape);
  const Rows rx(x, "x", shape, dt);
  const Kept kx = kept(x8, "x", shape);
  const float *pr = f32(rstd, "rstd", rows), *ps = f32(scale, "scale", cols),
              *pw = f32(w, "w", cols);
  const On on(a[12], d_out);
  Rows go, gx;
  if (given) {
    if (g[0].defined()) go = Rows(&g[0], "d_res", shape, rdt);
    if (g[1].defined()) gx = Rows(&g[1], "d_x", shape, dt);
    if (g[2].defined()) f32(&g[2], "d_w", cols);
    if (g[3].defined()) f32(&g[3], "d_scale", cols);
  } else {
    if (yes(a[8])) g[0] = make(shape, rdt, d_out), go.p = g[0].data_ptr();
    if (yes(a[9])) g[1] = make(shape, dt, d_out), gx.p = g[1].data_ptr();
    if (w) g[2] = make(w->sizes(), at::kFloat, d_out);
    if (scale && (x || x8.q)) g[3] = make(scale->sizes(), at::kFloat, d_out);
  }
  const ssm_norm_desc d = norm_desc(rows, cols, 0, io, io_code(rdt), 0, 1.0);
  const int sums = g[2].defined() + g[3].defined();
  const Workspace ws(sums ? ssm_norm_bwd_workspace_size(&d, sums) : 0, given_ws, d_out);
  if (!given) on.made({&g[0], &g[1], &g[2], &g[3]});
  const int rc = call([&] {
    return ssm_add_norm_bwd(&d, rd.p, rd.ld, ru.p, ru.ld, rr.p, rr.ld, kr.q, kr.e, rx.p, rx.ld,
                            kx.q, kx.e, pr, ps, pw, go.p, go.ld, gx.p, gx.ld, ptr<float>(g[2]),
                            ptr<float>(g[3]), ws.p, ws.bytes, on.raw);
  });
  if (rc) return PyLong_FromLong(rc);
  return pack({give(g[0]), give(g[1]), give(g[2]), give(g[3])});
  END_HANDLE_TH_ERRORS
}

// y, z, w, group, eps, flags, save8, save_out8, want_rstd, out, stream
SSM_FUNCTION(gated_norm_fwd) {
  HANDLE_TH_ERRORS
  args_are(n, 11);
  const Tensor &y = needed(a[0], "y"), &z = needed(a[1], "z");
  const Tensor *w = tensor(a[2], "w"), *out = tensor(a[9], "out");
  const int io = io_of(y, "y");
  const IntArrayRef shape = y.sizes();
  const ScalarType dt = y.scalar_type();
  const int64_t cols = columns(y, "y"), group = integer(a[3]);
  together({&y, "y"}, {{&z, "z"}, {w, "w"}, {out, "out"}});
  const Rows ry(&y, "y"), rz(&z, "z", shape, dt);
  const float* pw = f32(w, "w", cols);
  const On on(a[10], y);
  Tensor o, rstd;
  Rows ro(out, "out", shape, dt);
  if (out) o = *out;
  else o = make(shape, dt, y), ro.p = o.data_ptr();
  if (yes(a[8])) {
    at::DimVector s(shape.begin(), shape.end());
    s.back() = group > 0 && cols > group ? cols / group : 1;
    rstd = make(s, at::kFloat, y);
  }
  const bool save8 = yes(a[6]);
  const NewCkpt8 y8(save8, y), z8(save8, y), out8(yes(a[7]), y);
  const ssm_norm_desc d = norm_desc(rows_in(y, cols), cols, group, io, io,
                                    (unsigned)integer(a[5]), number(a[4]));
  on.made({&rstd, &y8.q, &y8.e, &z8.q, &z8.e, &out8.q, &out8.e});
  if (!out) on.made({&o});
  const int rc = call([&] {
    return ssm_gated_norm_fwd(&d, ry.p, ry.ld, rz.p, rz.ld, pw, ro.p, ro.ld, ptr<float>(rstd),
                              y8.pq(), y8.pe(), z8.pq(), z8.pe(), out8.pq(), out8.pe(), on.raw);
  });
  if (rc) return PyLong_FromLong(rc);
  return pack({give(o), give(rstd), give(y8), give(z8), give(out8)});
  END_HANDLE_TH_ERRORS
}

// d_out, y, z, rstd, w, group, flags, ws, out, stream
SSM_FUNCTION(gated_norm_bwd) {
  HANDLE_TH_ERRORS
  args_are(n, 10);
  const Tensor& d_out = needed(a[0], "d_out");
  const Pair y8(a[1], "y"), z8(a[2], "z");
  const Tensor *y = y8.q ? nullptr : &needed(a[1], "y"), *z = z8.q ? nullptr : &needed(a[2], "z");
  const Tensor *rstd = tensor(a[3], "rstd"), *w = tensor(a[4], "w");
  const int io = io_of(d_out, "d_out");
  const IntArrayRef shape = d_out.sizes();
  const ScalarType dt = d_out.scalar_type();
  const int64_t cols = columns(d_out, "d_out"), rows = rows_in(d_out, cols), group = integer(a[5]);
  Tensor g[3];  // d_y, d_z, d_w
  const bool given = a[8] != Py_None;
  if (given) {
    outs_are(a[8], 3, "d_y, d_z and d_w");
    for (int i = 0; i < 3; i++)
      if (const Tensor* t = tensor(PyTuple_GET_ITEM(a[8], i), "out")) g[i] = *t;
  }
  const Tensor* given_ws = tensor(a[7], "ws");
  together({&d_out, "d_out"},
           {{y, "y"}, {y8.q, "y"}, {y8.e, "y"}, {z, "z"}, {z8.q, "z"}, {z8.e, "z"}, {rstd, "rstd"},
            {w, "w"}, some(g[0], "d_y"), some(g[1], "d_z"), some(g[2], "d_w"), {given_ws, "ws"}});
  const Rows rd(&d_out, "d_out"), ry(y, "y", shape, dt);
  const Kept ky = kept(y8, "y", shape);
  const Rows rz(z, "z", shape, dt);
  const Kept kz = kept(z8, "z", shape);
  const float *pr = f32(rstd, "rstd", rows * (group > 0 ? cols / group : 1)),
              *pw = f32(w, "w", cols);
  const On on(a[9], d_out);
  Rows gy, gz;
  if (given) {
    if (g[0].defined()) gy = Rows(&g[0], "d_y", shape, dt);
    if (g[1].defined()) gz = Rows(&g[1], "d_z", shape, dt);
    if (g[2].defined()) f32(&g[2], "d_w", cols);
  } else {
    g[0] = make(shape, dt, d_out), gy.p = g[0].data_ptr();
    g[1] = make(shape, dt, d_out), gz.p = g[1].data_ptr();
    if (w) g[2] = make(w->sizes(), at::kFloat, d_out);
  }
  const ssm_norm_desc d = norm_desc(rows, cols, group, io, io, (unsigned)integer(a[6]), 1.0);
  const Workspace ws(g[2].defined() ? ssm_norm_bwd_workspace_size(&d, 1) : 0, given_ws, d_out);
  if (!given) on.made({&g[0], &g[1], &g[2]});
  const int rc = call([&] {
    return ssm_gated_norm_bwd(&d, rd.p, rd.ld, ry.p, ry.ld, ky.q, ky.e, rz.p, rz.ld, kz.q, kz.e,
                              pr, pw, gy.p, gy.ld, gz.p, gz.ld, ptr<float>(g[2]), ws.p, ws.bytes,
                              on.raw);
  });
  if (rc) return PyLong_FromLong(rc);
  return pack({give(g[0]), give(g[1]), give(g[2])});
  END_HANDLE_TH_ERRORS
}

// x, out, stream
SSM_FUNCTION(ckpt8_save) {
  HANDLE_TH_ERRORS
  args_are(n, 3);
  const Tensor& x = needed(a[0], "x");
  const int io = io_of(x, "x");
  const int64_t cols = columns(x, "x");
  const Pair given(a[1], "out");
  TORCH_CHECK_TYPE(given.q || a[1] == Py_None, "out must be a pair of tensors (q, e)");
  together({&x, "x"}, {{given.q, "out"}, {given.e, "out"}});
  const Rows rx(&x, "x");
  const On on(a[2], x);
  NewCkpt8 made;
  Kept k;
  if (given.q) {
    k = kept(given, "out", x.sizes());
  } else {
    made = NewCkpt8(true, x);
    k = {made.pq(), made.pe()};
  }
  on.made({&made.q, &made.e});
  const int rc = call([&] {
    return ssm_ckpt8_save(rx.p, rx.ld, k.q, k.e, rows_in(x, cols),
                          cols > 0x7fffffff ? 0x7fffffff : (int)cols, io, on.raw);
  });
  if (rc) return PyLong_FromLong(rc);
  if (given.q) {
    Py_INCREF(a[1]);
    return a[1];
  }
  return give(made);
  END_HANDLE_TH_ERRORS
}

// c, dtype, out, stream
SSM_FUNCTION(ckpt8_load) {
  HANDLE_TH_ERRORS
  args_are(n, 4);
  const Pair c(a[0], "c");
  TORCH_CHECK_TYPE(c.q, "c must be a pair of tensors (q, e)");
  const Tensor* out = tensor(a[2], "out");
  together({c.q, "c"}, {{c.e, "c"}, {out, "out"}});
  const IntArrayRef shape = c.q->sizes();
  const int64_t cols = columns(*c.q, "c");
  const Kept k = kept(c, "c", shape);
  const On on(a[3], *c.q);
  Tensor o;
  if (out) {
    o = *out;
  } else {
    TORCH_CHECK_TYPE(THPDtype_Check(a[1]), "dtype must be a torch.dtype");
    o = make(shape, reinterpret_cast<THPDtype*>(a[1])->scalar_type, *c.q);
  }
  const int io = io_of(o, "out");
  const Rows ro(&o, "out", shape, o.scalar_type());
  if (!out) on.made({&o});
  const int rc = call([&] {
    return ssm_ckpt8_load(k.q, k.e, ro.p, ro.ld, rows_in(*c.q, cols),
                          cols > 0x7fffffff ? 0x7fffffff : (int)cols, io, on.raw);
  });
  if (rc) return PyLong_FromLong(rc);
  return give(o);
  END_HANDLE_TH_ERRORS
}

// g, x8, flags, ws, out, stream
SSM_FUNCTION(ckpt8_wgrad) {
  HANDLE_TH_ERRORS
  args_are(n, 6);
  const Tensor& g = needed(a[0], "g");
  const Pair x8(a[1], "x8");
  TORCH_CHECK_TYPE(x8.q, "x8 must be a pair of tensors (q, e)");
  const Tensor* out = tensor(a[4], "out");
  const unsigned flags = (unsigned)integer(a[2]);
  const bool accumulate = flags & SSM_WGRAD_ACCUMULATE;
  const int io = io_of(g, "g");
  const int64_t m = columns(g, "g"), k = columns(*x8.q, "x8"), tokens = rows_in(g, m);
  TORCH_CHECK_VALUE(!accumulate || out, "accumulate needs the tensor to add to (out)");
  const int64_t want[2] = {m, k};
  TORCH_CHECK_VALUE(!out || out->sizes() == IntArrayRef(want), "out must have shape ",
                    IntArrayRef(want), ", got ", out ? out->sizes() : IntArrayRef());
  const Tensor* given_ws = tensor(a[3], "ws");
  together({&g, "g"}, {{x8.q, "x8"}, {x8.e, "x8"}, {out, "out"}, {given_ws, "ws"}});
  const Rows rg(&g, "g");
  at::DimVector shape(g.sizes().begin(), g.sizes().end());
  shape.back() = k;
  const Kept x = kept(x8, "x8", shape);
  const On on(a[5], g);
  const Tensor o = out ? *out : make(want, at::kFloat, g);
  float* po = f32(&o, "out", m * k);
  TORCH_CHECK_VALUE(m <= 0x7fffffff && k <= 0x7fffffff, "g and x8 are too wide");
  const uintptr_t row = (uintptr_t)(rg.ld ? rg.ld : m) * g.element_size();  // fp32 g may lie anywhere
  const int aligned = !((uintptr_t)x.q & 15) && (io == SSM_F32 || !(((uintptr_t)rg.p | row) & 15));
  const Workspace ws(ssm_ckpt8_wgrad_workspace_size(tokens, (int)m, (int)k, io, aligned),
                     given_ws, g);
  if (!out) on.made({&o});
  const int rc = call([&] {
    return ssm_ckpt8_wgrad(rg.p, rg.ld, x.q, x.e, po, tokens, (int)m, (int)k, io, flags, ws.p,
                           ws.bytes, on.raw);
  });
  if (rc) return PyLong_FromLong(rc);
  return give(o);
  END_HANDLE_TH_ERRORS
}

// The type of the checkpoints that the functions return (a pair of tensors).
PyObject* use_ckpt8(PyObject*, PyObject* type) {
  if (!PyType_Check(type) || !PyType_IsSubtype((PyTypeObject*)type, &PyTuple_Type)) {
    PyErr_SetString(PyExc_TypeError, "expected a tuple type");
    return nullptr;
  }
  Py_INCREF(type);
  Py_XDECREF((PyObject*)ckpt8_type);
  ckpt8_type = (PyTypeObject*)type;
  Py_RETURN_NONE;
}

#define SSM_METHOD(name) \
  {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {SSM_METHOD(add_norm_fwd),
                         SSM_METHOD(add_norm_bwd),
                         SSM_METHOD(gated_norm_fwd),
                         SSM_METHOD(gated_norm_bwd),
                         SSM_METHOD(ckpt8_save),
                         SSM_METHOD(ckpt8_load),
                         SSM_METHOD(ckpt8_wgrad),
                         {"use_ckpt8", use_ckpt8, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module{PyModuleDef_HEAD_INIT, "_block", nullptr, -1, methods,
                   nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__block() { return PyModule_Create(&module); }
