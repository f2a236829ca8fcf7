// Python entry of the 8-bit serving calls: argument checks, output tensors and
// the current stream, around the C ABI of libpiq.so.  The other entries are
// bound through ctypes; these sit in a decoding loop, where a call's kernels take
// a few microseconds and ctypes with its checks took 10 to 20 of the host's.
//
// Every function takes its arguments by position (the package's functions of the
// same names fill in the defaults) and raises TypeError, ValueError, or through
// the package's check function PiqError.
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <optional>

#include "../../include/piq.h"

namespace {

PyObject* g_check = nullptr;  // check(status, where): raises for a negative status

// Leaves a function with the Python error that is set.
struct Raised {};

[[noreturn]] void fail(PyObject* type, const char* format, const char* name) {
  PyErr_Format(type, format, name);
  throw Raised();
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) fail(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return t;
}

// A tensor of rows: every dimension but the first contiguous.  The row stride.
int64_t row_stride(const at::Tensor& t, int64_t ndim, const char* name) {
  if (t.dim() != ndim) fail(PyExc_ValueError, "%s has the wrong number of dimensions", name);
  const auto shape = t.sizes();
  const auto stride = t.strides();
  int64_t want = 1;
  for (int64_t i = ndim - 1; i > 0; --i) {
    if (stride[i] != want && shape[i] > 1 && shape[0] > 0)
      fail(PyExc_ValueError, "the rows of %s must be contiguous", name);
    want *= shape[i];
  }
  return shape[0] > 1 ? stride[0] : std::max(stride[0], want);
}

void need_type(const at::Tensor& t, at::ScalarType type, const char* name) {
  if (t.scalar_type() != type) fail(PyExc_TypeError, "%s has the wrong dtype", name);
}

void need_device(const at::Tensor& t, const at::Device& dev, const char* name) {
  if (t.device() != dev) fail(PyExc_ValueError, "%s is on another device", name);
}

const at::Tensor& flat(PyObject* o, at::ScalarType type, at::IntArrayRef shape,
                       const at::Device& dev, const char* name) {
  const at::Tensor& t = cuda_tensor(o, name);
  need_type(t, type, name);
  if (t.sizes() != shape || !t.is_contiguous())
    fail(PyExc_ValueError, "%s must be contiguous and of the matching shape", name);
  need_device(t, dev, name);
  return t;
}

int dtype_code(at::ScalarType t, bool fp32, const char* name) {
  switch (t) {
    case at::kBFloat16: return PIQ_BF16;
    case at::kHalf: return PIQ_FP16;
    case at::kFloat:
      if (fp32) return PIQ_FP32;
      [[fallthrough]];
    default: fail(PyExc_TypeError, "%s has an unsupported dtype", name);
  }
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}

void check(int rc, const char* where) {
  if (rc == PIQ_OK) return;
  PyObject* r = g_check ? PyObject_CallFunction(g_check, "is", rc, where) : nullptr;
  if (r != nullptr) {
    Py_DECREF(r);
    PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, rc);
  } else if (!PyErr_Occurred()) {
    PyErr_Format(PyExc_RuntimeError, "%s: status %d", where, rc);
  }
  throw Raised();
}

// The tensors' device made current, and with a stream of its own (a handle, or
// None) that stream, so that what the call allocates comes from its memory.
class On {
 public:
  On(const at::Device& dev, PyObject* stream) : device_(dev) {
    if (stream != Py_None) {
      const auto handle = reinterpret_cast<cudaStream_t>(PyLong_AsVoidPtr(stream));
      if (PyErr_Occurred()) throw Raised();
      guard_.emplace(c10::cuda::getStreamFromExternal(handle, dev.index()));
      stream_ = handle;
    } else {
      stream_ = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    }
  }
  void* stream() const { return stream_; }

 private:
  c10::cuda::CUDAGuard device_;
  std::optional<c10::cuda::CUDAStreamGuard> guard_;
  cudaStream_t stream_ = nullptr;
};

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

int32_t* status_of(PyObject* o, const at::Device& dev) {
  if (o == Py_None) return nullptr;
  return flat(o, at::kInt, {2}, dev, "status").data_ptr<int32_t>();
}

// The caller's workspace if it is large enough, else a new one.
at::Tensor workspace_of(PyObject* o, size_t bytes, const at::Device& dev) {
  if (bytes == 0) return at::Tensor();
  if (o != Py_None) {
    const at::Tensor& t = cuda_tensor(o, "workspace");
    need_type(t, at::kByte, "workspace");
    need_device(t, dev, "workspace");
    if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", "workspace");
    if (static_cast<size_t>(t.numel()) >= bytes) return t;
  }
  return empty({static_cast<int64_t>(bytes)}, at::kByte, dev);
}

// The cache's tensors and its ragged batch.
struct Cache {
  int8_t *k, *v;
  float *ks, *vs;
  int64_t pages, heads, block, dim;
  const int32_t *cu, *lens, *table;
  int64_t batch, width, ldt;
  at::Device dev;
};

Cache cache_of(PyObject* const* a, PyObject* cu, PyObject* lens, PyObject* table) {
  const at::Tensor& k = cuda_tensor(a[0], "cache.k");
  const at::Device dev = k.device();
  if (k.dim() != 4) fail(PyExc_ValueError, "%s must be [pages, kv_heads, block, head_dim]", "cache.k");
  const auto shape = k.sizes();
  flat(a[0], at::kChar, shape, dev, "cache.k");
  const at::Tensor& v = flat(a[1], at::kChar, shape, dev, "cache.v");
  const at::Tensor& ks = flat(a[2], at::kFloat, shape.slice(0, 2), dev, "cache.k_scale");
  const at::Tensor& vs = flat(a[3], at::kFloat, shape.slice(0, 2), dev, "cache.v_scale");
  const at::Tensor& t = cuda_tensor(table, "block_table");
  need_type(t, at::kInt, "block_table");
  const int64_t ldt = row_stride(t, 2, "block_table");
  need_device(t, dev, "block_table");
  const int64_t batch = t.size(0);
  const at::Tensor& c = flat(cu, at::kInt, {batch + 1}, dev, "cu");
  const at::Tensor& l = flat(lens, at::kInt, {batch}, dev, "lengths");
  return Cache{k.data_ptr<int8_t>(), v.data_ptr<int8_t>(), ks.data_ptr<float>(),
               vs.data_ptr<float>(), shape[0], shape[1], shape[2], shape[3],
               c.data_ptr<int32_t>(), l.data_ptr<int32_t>(), t.data_ptr<int32_t>(), batch,
               t.size(1), ldt, dev};
}

// k or v, in or out: [rows, kv_heads, head_dim] of the cache.
int64_t head_rows(const at::Tensor& t, const Cache& c, const char* name) {
  const int64_t ld = row_stride(t, 3, name);
  if (t.size(1) != c.heads || t.size(2) != c.dim)
    fail(PyExc_ValueError, "%s must be [tokens, kv_heads, head_dim] of the cache", name);
  need_device(t, c.dev, name);
  return ld;
}

// int8_quantize_rows(X, stream) -> (codes, scales)
PyObject* quantize_rows(PyObject* const* a) {
  const at::Tensor& x = cuda_tensor(a[0], "X");
  const int dtype = dtype_code(x.scalar_type(), true, "X");
  const int64_t ldx = row_stride(x, 2, "X");
  const int64_t rows = x.size(0), cols = x.size(1), ldc = (cols + 15) / 16 * 16;
  const On on(x.device(), a[1]);
  at::Tensor codes = empty({rows, ldc}, at::kChar, x.device());
  at::Tensor scales = empty({rows}, at::kFloat, x.device());
  check(piq_int8_quantize_rows(x.data_ptr(), dtype, rows, cols, ldx, codes.data_ptr<int8_t>(), ldc,
                               scales.data_ptr<float>(), on.stream()),
        "piq_int8_quantize_rows");
  if (ldc != cols) codes = codes.narrow(1, 0, cols);
  return Py_BuildValue("NN", THPVariable_Wrap(codes), THPVariable_Wrap(scales));
}

// int8_linear(X, W, w_scale, bias, out, stream, workspace, status) -> out
PyObject* linear(PyObject* const* a) {
  const at::Tensor& x = cuda_tensor(a[0], "X");
  const int dtype = dtype_code(x.scalar_type(), true, "X");
  const int64_t ldx = row_stride(x, 2, "X");
  const at::Tensor& w = cuda_tensor(a[1], "W");
  need_type(w, at::kChar, "W");
  const int64_t ldw = row_stride(w, 2, "W");
  const at::Device dev = x.device();
  need_device(w, dev, "W");
  const int64_t tokens = x.size(0), in = x.size(1), out = w.size(0);
  if (w.size(1) != in) fail(PyExc_ValueError, "%s disagree on the input dimension", "W and X");
  const float* sw = flat(a[2], at::kFloat, {out}, dev, "w_scale").data_ptr<float>();
  const float* bias = nullptr;
  if (a[3] != Py_None) bias = flat(a[3], at::kFloat, {out}, dev, "bias").data_ptr<float>();
  const On on(dev, a[5]);
  at::Tensor y;
  int64_t ldy = out;
  if (a[4] == Py_None) {
    y = empty({tokens, out}, x.scalar_type(), dev);
  } else {
    y = cuda_tensor(a[4], "out");
    need_type(y, x.scalar_type(), "out");
    need_device(y, dev, "out");
    ldy = row_stride(y, 2, "out");
    if (y.size(0) != tokens || y.size(1) != out)
      fail(PyExc_ValueError, "%s must be [tokens, out]", "out");
  }
  int32_t* const status = status_of(a[7], dev);
  size_t bytes = 0;
  check(piq_int8_linear_workspace_bytes(tokens, out, in, &bytes),
        "piq_int8_linear_workspace_bytes");
  const at::Tensor ws = workspace_of(a[6], bytes, dev);
  check(piq_int8_linear(x.data_ptr(), dtype, tokens, in, ldx, w.data_ptr<int8_t>(), out, ldw, sw,
                        bias, y.data_ptr(), ldy, status, ws.defined() ? ws.data_ptr() : nullptr,
                        bytes, on.stream()),
        "piq_int8_linear");
  return THPVariable_Wrap(y);
}

// kv8_append(cache.k, .v, .k_scale, .v_scale, k, v, cu, lens_before, table, stream, status)
PyObject* append(PyObject* const* a) {
  const Cache c = cache_of(a, a[6], a[7], a[8]);
  const at::Tensor& k = cuda_tensor(a[4], "k");
  const at::Tensor& v = cuda_tensor(a[5], "v");
  const int dtype = dtype_code(k.scalar_type(), true, "k");
  need_type(v, k.scalar_type(), "v");
  const int64_t ldk = head_rows(k, c, "k"), ldv = head_rows(v, c, "v");
  if (k.size(0) != v.size(0)) fail(PyExc_ValueError, "%s disagree on the tokens", "k and v");
  const On on(c.dev, a[9]);
  check(piq_kv8_append(k.data_ptr(), v.data_ptr(), dtype, k.size(0), ldk, ldv, c.cu, c.lens,
                       c.batch, c.table, c.width, c.ldt, c.k, c.v, c.ks, c.vs, c.pages,
                       static_cast<int>(c.heads), static_cast<int>(c.dim),
                       static_cast<int>(c.block), status_of(a[10], c.dev), on.stream()),
        "piq_kv8_append");
  Py_RETURN_NONE;
}

// kv8_read(cache x 4, cu, start, table, rows, dtype, out_k, out_v, stream, status) -> (k, v)
PyObject* read(PyObject* const* a) {
  const Cache c = cache_of(a, a[4], a[5], a[6]);
  const int64_t rows = integer(a[7]);
  if (!THPDtype_Check(a[8])) fail(PyExc_TypeError, "%s must be a torch.dtype", "dtype");
  const at::ScalarType type = reinterpret_cast<THPDtype*>(a[8])->scalar_type;
  const int dtype = dtype_code(type, true, "dtype");
  const On on(c.dev, a[11]);
  at::Tensor k, v;
  if (a[9] == Py_None) {
    if (rows < 0) fail(PyExc_ValueError, "%s must not be negative", "rows");
    k = empty({rows, c.heads, c.dim}, type, c.dev);
    v = empty({rows, c.heads, c.dim}, type, c.dev);
  } else {
    k = cuda_tensor(a[9], "out");
    v = cuda_tensor(a[10], "out");
    need_type(k, type, "out");
    need_type(v, type, "out");
  }
  const int64_t ldk = head_rows(k, c, "out"), ldv = head_rows(v, c, "out");
  if (k.size(0) != rows || v.size(0) != rows)
    fail(PyExc_ValueError, "%s must be two tensors of `rows` rows", "out");
  check(piq_kv8_read(c.k, c.v, c.ks, c.vs, c.pages, static_cast<int>(c.heads),
                     static_cast<int>(c.dim), static_cast<int>(c.block), c.cu, c.lens, c.batch,
                     c.table, c.width, c.ldt, rows, k.data_ptr(), v.data_ptr(), dtype, ldk, ldv,
                     status_of(a[12], c.dev), on.stream()),
        "piq_kv8_read");
  return Py_BuildValue("NN", THPVariable_Wrap(k), THPVariable_Wrap(v));
}

// kv8_attention(cache x 4, q, cu, lens, table, max_new, max_len, scale, window, return_lse, out,
//               stream, workspace, status) -> out or (out, lse)
PyObject* attention(PyObject* const* a) {
  const Cache c = cache_of(a, a[5], a[6], a[7]);
  const at::Tensor& q = cuda_tensor(a[4], "q");
  const int dtype = dtype_code(q.scalar_type(), false, "q");
  const int64_t ldq = row_stride(q, 3, "q");
  need_device(q, c.dev, "q");
  if (q.size(2) != c.dim) fail(PyExc_ValueError, "%s disagree on head_dim", "q and the cache");
  const int64_t tokens = q.size(0), heads = q.size(1);
  const int64_t max_new = integer(a[8]), max_len = integer(a[9]), window = integer(a[11]);
  if (heads > INT32_MAX || window > INT32_MAX || window < INT32_MIN)
    fail(PyExc_ValueError, "%s out of range", "heads or window");
  const double scale =
      a[10] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.dim)) : PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) throw Raised();
  const int truth = PyObject_IsTrue(a[12]);
  if (truth < 0) throw Raised();
  const On on(c.dev, a[14]);
  at::Tensor out, lse;
  int64_t ldo = heads * c.dim;
  if (a[13] == Py_None) {
    out = empty(q.sizes(), q.scalar_type(), c.dev);
  } else {
    out = cuda_tensor(a[13], "out");
    need_type(out, q.scalar_type(), "out");
    need_device(out, c.dev, "out");
    if (out.sizes() != q.sizes()) fail(PyExc_ValueError, "%s must have q's shape", "out");
    ldo = row_stride(out, 3, "out");
  }
  if (truth) lse = empty({tokens, heads}, at::kFloat, c.dev);
  int32_t* const status = status_of(a[16], c.dev);
  size_t bytes = 0;
  check(piq_kv8_attention_workspace_bytes(tokens, static_cast<int>(heads),
                                          static_cast<int>(c.heads), static_cast<int>(c.dim),
                                          c.batch, max_new, max_len, static_cast<int>(window),
                                          &bytes),
        "piq_kv8_attention_workspace_bytes");
  const at::Tensor ws = workspace_of(a[15], bytes, c.dev);
  check(piq_kv8_attention(q.data_ptr(), dtype, tokens, ldq, static_cast<int>(heads), c.cu, c.lens,
                          c.batch, c.table, c.width, c.ldt, c.k, c.v, c.ks, c.vs, c.pages,
                          static_cast<int>(c.heads), static_cast<int>(c.dim),
                          static_cast<int>(c.block), static_cast<float>(scale),
                          static_cast<int>(window), max_new, max_len, out.data_ptr(), ldo,
                          truth ? lse.data_ptr<float>() : nullptr, status, ws.data_ptr(), bytes,
                          on.stream()),
        "piq_kv8_attention");
  if (!truth) return THPVariable_Wrap(out);
  return Py_BuildValue("NN", THPVariable_Wrap(out), THPVariable_Wrap(lse));
}

// One Python function: a fixed number of arguments, every C++ exception turned
// into a Python one.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_check(PyObject*, PyObject* f) {
  Py_INCREF(f);
  Py_XDECREF(g_check);
  g_check = f;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<F, N>)),
          METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    {"set_check", set_check, METH_O, nullptr},
    method<quantize_rows, 2>("int8_quantize_rows"),
    method<linear, 8>("int8_linear"),
    method<append, 11>("kv8_append"),
    method<read, 13>("kv8_read"),
    method<attention, 17>("kv8_attention"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "piq_serve",
                        "The 8-bit serving calls of libpiq on torch tensors.", -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit_piq_serve() { return PyModule_Create(&g_module); }
