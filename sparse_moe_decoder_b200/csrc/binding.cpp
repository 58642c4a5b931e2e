// The argument checks and calls of the decode-step operators for Python.
//
// A decode step makes these calls once a layer, and their kernels take a few microseconds at decode sizes; checking a
// dozen tensors and converting thirty arguments in Python took several times as long as the launch (10 to 15 us of
// host time a call against 4 to 7 here).  Each function checks its tensors (type, shape, device, layout), raises TypeError or
// ValueError, calls the C entry point on the tensors' device and on its current stream (or the one given), and
// returns the entry point's status.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "zmoe.h"

namespace {

struct Bad {
  PyObject* type;
  std::string what;
};

std::string text(const char* s) { return s; }
std::string text(const std::string& s) { return s; }
std::string text(int64_t v) { return std::to_string(v); }

template <typename... A>
[[noreturn]] void bad(PyObject* type, const A&... parts) {
  throw Bad{type, (text(parts) + ...)};
}

std::string dims(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + text(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) bad(PyExc_TypeError, name, " must be a CUDA tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) bad(PyExc_TypeError, name, " must be a CUDA tensor");
  return t;
}

void need_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type) bad(PyExc_TypeError, name, " must be ", c10::toString(type), ", got ", c10::toString(t.scalar_type()));
}

void need_device(const at::Tensor& t, const char* name, int dev) {
  if (t.get_device() != dev) bad(PyExc_ValueError, name, " is on ", t.device().str(), ", the call's tensors are on cuda:", dev);
}

const at::Tensor& contiguous(PyObject* o, const char* name, int64_t ndim) {
  const at::Tensor& t = cuda_tensor(o, name);
  if (!t.is_contiguous()) bad(PyExc_ValueError, name, " must be contiguous");
  if (ndim >= 0 && t.dim() != ndim) bad(PyExc_ValueError, name, " must have ", ndim, " dims, got shape ", dims(t.sizes()));
  return t;
}

void need_shape(const at::Tensor& t, const char* name, std::initializer_list<int64_t> shape) {
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) bad(PyExc_ValueError, name, " must have shape ", dims(want), ", got ", dims(t.sizes()));
}

// The address of an optional contiguous tensor of this shape, device and, unless `any`, type.
void* address(PyObject* o, const char* name, int dev, std::initializer_list<int64_t> shape, at::ScalarType type,
              bool any = false) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = contiguous(o, name, -1);
  if (!any) need_type(t, name, type);
  need_shape(t, name, shape);
  need_device(t, name, dev);
  return t.data_ptr();
}

zmoe_dtype code_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return ZMOE_F32;
  if (t.scalar_type() == at::kBFloat16) return ZMOE_BF16;
  bad(PyExc_TypeError, "libzmoe computes in float32 or bfloat16, got ", c10::toString(t.scalar_type()));
}

int integer(PyObject* o, const char* name) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(PyExc_TypeError, name, " must be an integer");
  }
  if (v < INT32_MIN || v > INT32_MAX) bad(PyExc_ValueError, name, " does not fit 32 bits");
  return static_cast<int>(v);
}

float real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(PyExc_TypeError, name, " must be a number");
  }
  return static_cast<float>(v);
}

bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    bad(PyExc_TypeError, name, " must be true or false");
  }
  return v == 1;
}

int size32(int64_t v, const char* name) {
  if (v > INT32_MAX) bad(PyExc_ValueError, name, " does not fit 32 bits");
  return static_cast<int>(v);
}

// The call's device made current, and its stream: the current one of the device, or the torch.cuda.Stream given.
struct Place {
  c10::cuda::OptionalCUDAGuard guard;
  zmoe_stream_t stream;

  Place(int dev, PyObject* s) {
    if (s == Py_None) {
      stream = reinterpret_cast<zmoe_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
    } else {
      const long on = number(s, "device_index");
      if (on != dev) bad(PyExc_ValueError, "the stream is on cuda:", on, ", the call's tensors are on cuda:", dev);
      stream = reinterpret_cast<zmoe_stream_t>(number(s, "cuda_stream"));
    }
    if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
  }

  static long number(PyObject* s, const char* what) {
    PyObject* v = PyObject_GetAttrString(s, what);
    const long n = v ? PyLong_AsLong(v) : -1;
    Py_XDECREF(v);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      bad(PyExc_TypeError, "stream must be a torch.cuda.Stream");
    }
    return n;
  }
};

template <typename F>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, F f) {
  try {
    if (got != want) bad(PyExc_TypeError, want, " arguments wanted, got ", got);
    return PyLong_FromLong(f());
  } catch (const Bad& b) {
    PyErr_SetString(b.type, b.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (h, gamma, delta, eps, h_out, x, x_code, codes, scales, group, stream)
PyObject* add_rmsnorm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const at::Tensor& h = contiguous(a[0], "h", 2);
    const int dev = h.get_device(), group = integer(a[9], "group");
    const int64_t T = h.size(0), d = h.size(1);
    if (group < 0) bad(PyExc_ValueError, "group must not be negative");
    const void* delta = address(a[2], "delta", dev, {T, d}, at::kFloat, true);
    void* x = address(a[5], "outs['x']", dev, {T, d}, at::kFloat, true);
    const zmoe_dtype x_type = x ? code_of(THPVariable_Unpack(a[5])) : ZMOE_BF16;
    const zmoe_dtype d_type = delta ? code_of(THPVariable_Unpack(a[2])) : ZMOE_F32;
    const void* gamma = address(a[1], "gamma", dev, {d}, at::kFloat);
    void* ho = address(a[4], "outs['h']", dev, {T, d}, h.scalar_type());
    void* codes = address(a[7], "outs['codes']", dev, {T, d}, at::kByte);
    void* scales = address(a[8], "outs['scales']", dev, {T, group ? d / group : 1}, at::kFloat);
    const Place at(dev, a[10]);
    return zmoe_add_rmsnorm(h.data_ptr(), code_of(h), delta, d_type, static_cast<const float*>(gamma), real(a[3], "eps"),
                            size32(T, "T"), size32(d, "d"), ho, x, x_type, static_cast<uint8_t*>(codes),
                            static_cast<float*>(scales), group, at.stream);
  });
}

struct Cache {
  zmoe_dtype type;
  int dev;
  int64_t n_pages, Hkv, page_size, D;
  void *k, *v;
  const float *k_scale, *v_scale;

  Cache(PyObject* ko, PyObject* vo, PyObject* ks, PyObject* vs) {
    const at::Tensor& t = contiguous(ko, "k_cache", 4);
    if (t.scalar_type() == at::kBFloat16) type = ZMOE_BF16;
    else if (t.scalar_type() == at::kByte) type = ZMOE_E4M3;
    else bad(PyExc_TypeError, "k_cache must be bfloat16 or uint8 (E4M3 codes), got ", c10::toString(t.scalar_type()));
    dev = t.get_device();
    n_pages = t.size(0); Hkv = t.size(1); page_size = t.size(2); D = t.size(3);
    k = t.data_ptr();
    v = address(vo, "v_cache", dev, {n_pages, Hkv, page_size, D}, t.scalar_type());
    k_scale = static_cast<const float*>(address(ks, "k_scale", dev, {Hkv}, at::kFloat));
    v_scale = static_cast<const float*>(address(vs, "v_scale", dev, {Hkv}, at::kFloat));
  }
};

struct Table {
  const int32_t* p;
  int rows, cols;

  Table(PyObject* o, int dev) {
    const at::Tensor& t = contiguous(o, "page_table", 2);
    need_type(t, "page_table", at::kInt);
    need_device(t, "page_table", dev);
    p = static_cast<const int32_t*>(t.data_ptr());
    rows = size32(t.size(0), "page_table");
    cols = size32(t.size(1), "page_table");
  }
};

// A [T, H, D] view whose heads are contiguous: its address and the elements between its tokens.
struct Heads {
  const void* p = nullptr;
  int64_t stride = 0;

  Heads(PyObject* o, const char* name, int64_t T, int64_t H, int64_t D, at::ScalarType type, int dev) {
    const at::Tensor& t = cuda_tensor(o, name);
    need_type(t, name, type);
    need_shape(t, name, {T, H, D});
    need_device(t, name, dev);
    if (T && ((D > 1 && t.stride(2) != 1) || (H > 1 && t.stride(1) != D)))
      bad(PyExc_ValueError, name, ": the heads of a token must be contiguous, got strides ", dims(t.strides()));
    p = t.data_ptr();
    stride = T > 1 ? t.stride(0) : H * D;
  }
  Heads() = default;
};

// (k, v, pos, k_cache, v_cache, page_table, q, seq, inv_freq, interleaved, q_gamma, k_gamma, eps, k_scale, v_scale,
//  q_out, stream)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&] {
    const Cache c(a[3], a[4], a[13], a[14]);
    const at::Tensor& k = cuda_tensor(a[0], "k");
    if (k.dim() != 3) bad(PyExc_ValueError, "k must have 3 dims");
    const int64_t T = k.size(0);
    const zmoe_dtype type = code_of(k);
    const Heads kh(a[0], "k", T, c.Hkv, c.D, k.scalar_type(), c.dev), vh(a[1], "v", T, c.Hkv, c.D, k.scalar_type(), c.dev);
    Heads qh;
    int64_t Hq = 0;
    if (a[6] != Py_None) {
      const at::Tensor& q = cuda_tensor(a[6], "q");
      if (q.dim() != 3) bad(PyExc_ValueError, "q must have 3 dims");
      Hq = q.size(1);
      qh = Heads(a[6], "q", T, Hq, c.D, k.scalar_type(), c.dev);
    }
    const Table table(a[5], c.dev);
    int rot = 0;
    const void* freq = nullptr;
    if (a[8] != Py_None) {
      const at::Tensor& f = contiguous(a[8], "inv_freq", 1);
      need_type(f, "inv_freq", at::kDouble);
      need_device(f, "inv_freq", c.dev);
      rot = size32(2 * f.size(0), "inv_freq");
      freq = rot ? f.data_ptr() : nullptr;
    }
    void* q_out = address(a[15], "q_out", c.dev, {T, Hq, c.D}, at::kBFloat16);
    const void* seq = address(a[7], "seq", c.dev, {T}, at::kInt);
    const void* pos = address(a[2], "pos", c.dev, {T}, at::kInt);
    const void* qg = address(a[10], "q_gamma", c.dev, {c.D}, at::kFloat);
    const void* kg = address(a[11], "k_gamma", c.dev, {c.D}, at::kFloat);
    const Place at(c.dev, a[16]);
    return zmoe_kv_append(qh.p, kh.p, vh.p, type, qh.stride, kh.stride, vh.stride, static_cast<const int32_t*>(seq),
                          static_cast<const int32_t*>(pos), static_cast<const double*>(freq), rot, truth(a[9], "interleaved"),
                          static_cast<const float*>(qg), static_cast<const float*>(kg), real(a[12], "eps"), size32(T, "T"),
                          size32(Hq, "Hq"), size32(c.Hkv, "Hkv"), size32(c.D, "D"), q_out, c.k, c.v, c.type, c.k_scale,
                          c.v_scale, table.p, table.rows, table.cols, size32(c.n_pages, "n_pages"),
                          size32(c.page_size, "page_size"), at.stream);
  });
}

// (q, k_cache, v_cache, page_table, lens, scale or None, k_scale, v_scale, gate, out, lse, workspace, stream)
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&] {
    const Cache c(a[1], a[2], a[6], a[7]);
    const at::Tensor& q = contiguous(a[0], "q", 3);
    need_type(q, "q", at::kBFloat16);
    need_device(q, "q", c.dev);
    const int64_t B = q.size(0), Hq = q.size(1);
    need_shape(q, "q", {B, Hq, c.D});
    const Table table(a[3], c.dev);
    if (table.rows != B) bad(PyExc_ValueError, "page_table has ", table.rows, " rows for ", B, " sequences");
    const void* lens = address(a[4], "lens", c.dev, {B}, at::kInt);
    const void* gate = address(a[8], "gate", c.dev, {B, Hq}, at::kFloat);
    void* out = address(a[9], "out", c.dev, {B, Hq, c.D}, at::kFloat, true);
    void* lse = address(a[10], "lse", c.dev, {B, Hq}, at::kFloat);
    const zmoe_dtype out_type = code_of(cuda_tensor(a[9], "out"));
    const at::Tensor& ws = contiguous(a[11], "workspace", -1);
    need_device(ws, "workspace", c.dev);
    const double scale = a[5] == Py_None ? 1.0 / std::sqrt(static_cast<double>(c.D)) : real(a[5], "scale");
    const Place at(c.dev, a[12]);
    return zmoe_paged_attention(q.data_ptr(), c.k, c.v, c.type, c.k_scale, c.v_scale, table.p,
                                static_cast<const int32_t*>(lens), static_cast<const float*>(gate), static_cast<float>(scale),
                                size32(B, "B"), size32(Hq, "Hq"), size32(c.Hkv, "Hkv"), size32(c.D, "D"), table.cols,
                                size32(c.n_pages, "n_pages"), size32(c.page_size, "page_size"), out,
                                out_type, static_cast<float*>(lse), ws.data_ptr(), ws.nbytes(),
                                at.stream);
  });
}

// (logits, history, hist_lens, repetition, presence, frequency, bias, mask, out, ids, stream)
PyObject* adjust_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&] {
    const at::Tensor& z = contiguous(a[0], "logits", 3);
    const int dev = z.get_device();
    const int64_t T = z.size(0), N = z.size(1), V = z.size(2);
    const zmoe_dtype type = code_of(z);
    int64_t L = 0;
    if (a[1] != Py_None) L = contiguous(a[1], "history", 3).size(1);
    const void* hist = address(a[1], "history", dev, {T, L, N}, at::kInt);
    static const int32_t no_frames = 0;   // a history of no frames has no address, and is none the less one; never read
    if (a[1] != Py_None && L == 0) hist = &no_frames;
    const void* lens = address(a[2], "hist_lens", dev, {T}, at::kInt);
    const void* rep = address(a[3], "repetition", dev, {T}, at::kFloat);
    const void* pre = address(a[4], "presence", dev, {T}, at::kFloat);
    const void* frq = address(a[5], "frequency", dev, {T}, at::kFloat);
    const void* bias = address(a[6], "bias", dev, {N, V}, at::kFloat);
    const void* mask = address(a[7], "mask", dev, {T, N, (V + 31) / 32}, at::kInt);
    void* out = address(a[8], "out", dev, {T, N, V}, z.scalar_type());
    void* ids = address(a[9], "ids", dev, {T, N}, at::kInt);
    const Place at(dev, a[10]);
    return zmoe_adjust_logits(z.data_ptr(), type, static_cast<const int32_t*>(hist), static_cast<const int32_t*>(lens),
                              static_cast<const float*>(rep), static_cast<const float*>(pre), static_cast<const float*>(frq),
                              static_cast<const float*>(bias), static_cast<const uint32_t*>(mask), size32(T, "T"),
                              size32(N, "N"), size32(V, "V"), size32(L, "L"), out, static_cast<int32_t*>(ids), at.stream);
  });
}

#define ZMOE_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ZMOE_METHOD(add_rmsnorm), ZMOE_METHOD(kv_append), ZMOE_METHOD(paged_attention),
                         ZMOE_METHOD(adjust_logits), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Checked calls of libzmoe's decode-step operators.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&module); }
