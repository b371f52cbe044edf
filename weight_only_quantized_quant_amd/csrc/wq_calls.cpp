// The calls that a decode step makes for each layer, from tensors to the C entry
// points without a step in Python: there the host's part of such a call is longer
// than its kernel (append of 128 tokens: 8.3 us a call through ctypes, 4.0 us from
// here, which is the kernel's time).  Each function takes a call whose arguments are as the entry point
// needs them and returns NotImplemented for any other, having done nothing: the
// Python function of the same operator then says what is wrong with it, or
// makes the call itself (tensors of another device than the current one).  A
// launch that fails is not tried again: it raises what the Python function would.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include <cfloat>
#include <cmath>
#include <cstring>

#include "wq.h"

namespace {

using at::Tensor;

struct Refused {};                            // thrown by the readers below, caught at the entry
struct Failed {                               // a launch that may have run
  wq_status status;
};

const Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw Refused();
  const Tensor& t = THPVariable_Unpack(o);
  if (!t.defined() || !t.is_cuda() || t.layout() != at::kStrided) throw Refused();
  return t;
}

// Tokens x heads x channels, the heads of a token dense.
struct Rows {
  void* at;
  int64_t tokens, heads, dim, stride;
  at::ScalarType type;
  int dev;
  explicit Rows(const Tensor& t) {
    if (t.dim() != 3) throw Refused();
    tokens = t.size(0);
    heads = t.size(1);
    dim = t.size(2);
    if (t.stride(2) != 1 || (t.stride(1) != dim && heads > 1)) throw Refused();
    stride = tokens > 1 ? t.stride(0) : heads * dim;
    at = t.data_ptr();
    type = t.scalar_type();
    dev = t.get_device();
  }
};

// A contiguous tensor of a type, on device dev.
const Tensor& dense(PyObject* o, at::ScalarType type, int dev) {
  const Tensor& t = tensor(o);
  if (t.scalar_type() != type || t.get_device() != dev || !t.is_contiguous()) throw Refused();
  return t;
}
template <typename T>
T* dense_at(PyObject* o, at::ScalarType type, int dev, at::IntArrayRef sizes) {
  const Tensor& t = dense(o, type, dev);
  if (t.sizes() != sizes) throw Refused();
  return (T*)t.data_ptr();
}

struct Cache {
  int64_t pages, heads, page, dim;
  bool four;
  uint8_t *kc, *ks, *vc, *vs;
  Cache(PyObject* const* a, int dev) {        // k_codes, k_scales, v_codes, v_scales
    const Tensor &k = dense(a[0], at::kByte, dev), &s = dense(a[1], at::kByte, dev);
    if (k.dim() != 4) throw Refused();
    four = s.dim() == 4;
    pages = k.size(0);
    heads = k.size(1);
    page = k.size(2);
    const int64_t row = k.size(3);
    dim = four ? 2 * row : row;
    const std::array<int64_t, 4> sizes = {pages, heads, dim / 32, page};
    const at::IntArrayRef scales(sizes.data(), four ? 4 : 2);
    kc = (uint8_t*)k.data_ptr();
    ks = dense_at<uint8_t>(a[1], at::kByte, dev, scales);
    vc = dense_at<uint8_t>(a[2], at::kByte, dev, {pages, heads, row, page});
    vs = dense_at<uint8_t>(a[3], at::kByte, dev, scales);
  }
};

int type_of(const Rows& r) {
  if (r.type == at::kBFloat16) return WQ_BF16;
  if (r.type == at::kFloat) return WQ_F32;
  throw Refused();
}
hipStream_t stream_on(int dev) {
  if (c10::hip::current_device() != dev) throw Refused();
  return c10::hip::getCurrentHIPStream((c10::DeviceIndex)dev).stream();
}
int64_t whole(PyObject* o) {
  if (!PyLong_Check(o)) throw Refused();
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
float number(PyObject* o) {
  const double v = PyFloat_Check(o) ? PyFloat_AS_DOUBLE(o) : (double)whole(o);
  if (std::fabs(v) > FLT_MAX) throw Refused();
  return (float)v;
}
bool small(int64_t v) { return v >= 0 && v <= INT32_MAX; }
void done(wq_status s) {
  if (s == WQ_EHIP) throw Failed{s};
  if (s != WQ_OK) throw Refused();
}
// The interpreter's lock is given back while memory is allocated and kernels are
// launched: either may wait for the device.  Arguments are read before and results
// made after; what is thrown between takes the lock again on its way.
class Unlocked {
  PyThreadState* const state = PyEval_SaveThread();

 public:
  Unlocked() = default;
  Unlocked(const Unlocked&) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};
PyObject* raise(wq_status s, const char* where) {
  PyObject* m = PyImport_ImportModule("weight_only_quantized_quant_amd");
  PyObject* r = m ? PyObject_CallMethod(m, "_check", "is", (int)s, where) : nullptr;
  Py_XDECREF(m);
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
  return nullptr;
}

template <typename F>
PyObject* call(const char* name, Py_ssize_t given, Py_ssize_t wanted, F f) {
  try {
    if (given == wanted) return f();
  } catch (const Failed& e) {
    return raise(e.status, name);
  } catch (...) {                             // a refusal, or an error that the Python function will meet too
  }
  PyErr_Clear();
  Py_RETURN_NOTIMPLEMENTED;
}

// (k, v, slots, k_codes, k_scales, v_codes, v_scales)
PyObject* kv4_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("wq_kv4_append", n, 7, [&]() -> PyObject* {
    const Rows k(tensor(a[0])), v(tensor(a[1]));
    const Cache c(a + 3, k.dev);
    if (!c.four || k.heads != c.heads || k.dim != c.dim || v.tokens != k.tokens || v.heads != k.heads || v.dim != k.dim ||
        v.type != k.type || v.dev != k.dev || !small(k.heads))
      throw Refused();
    const int64_t* slots = dense_at<int64_t>(a[2], at::kLong, k.dev, {k.tokens});
    const int type = type_of(k);
    hipStream_t stream = stream_on(k.dev);
    {
      const Unlocked unlocked;
      done(wq_kv4_append(k.at, k.stride, v.at, v.stride, type, slots, k.tokens, (int32_t)k.heads, (int32_t)k.dim,
                         (int32_t)c.page, c.pages, c.kc, c.ks, c.vc, c.vs, stream));
    }
    Py_RETURN_NONE;
  });
}

// (q or None, k, v, positions, cos_sin, slots, k_codes, k_scales, v_codes, v_scales, interleaved, q_out or None)
PyObject* kv_append_rotary(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("wq_kv_append_rotary", n, 12, [&]() -> PyObject* {
    const Rows k(tensor(a[1])), v(tensor(a[2]));
    const Cache c(a + 6, k.dev);
    if (k.heads != c.heads || k.dim != c.dim || v.tokens != k.tokens || v.heads != k.heads || v.dim != k.dim ||
        v.type != k.type || v.dev != k.dev || !small(k.heads))
      throw Refused();
    const int32_t* positions = dense_at<int32_t>(a[3], at::kInt, k.dev, {k.tokens});
    const Tensor& angles = dense(a[4], at::kFloat, k.dev);
    if (angles.dim() != 2 || !small(angles.size(1))) throw Refused();
    const int64_t* slots = dense_at<int64_t>(a[5], at::kLong, k.dev, {k.tokens});
    const int inter = PyObject_IsTrue(a[10]);
    if (inter < 0) throw Refused();
    Tensor out;
    const void* qp = nullptr;
    uint16_t* op = nullptr;
    int64_t q_heads = 0, q_stride = 0, o_stride = 0;
    const int type = type_of(k);
    hipStream_t stream = stream_on(k.dev);
    const float* cos_sin = (const float*)angles.data_ptr();
    const int64_t max_pos = angles.size(0), rot = angles.size(1);
    at::TensorOptions made;
    if (a[0] != Py_None) {
      const Tensor& q = tensor(a[0]);
      const Rows r(q);
      if (r.tokens != k.tokens || r.dim != k.dim || r.type != k.type || r.dev != k.dev || !small(r.heads)) throw Refused();
      qp = r.at;
      q_heads = r.heads;
      q_stride = r.stride;
      made = q.options().dtype(at::kBFloat16);
      if (a[11] != Py_None) {
        const Rows o(tensor(a[11]));
        if (o.tokens != r.tokens || o.heads != r.heads || o.dim != r.dim || o.type != at::kBFloat16 || o.dev != k.dev) throw Refused();
        op = (uint16_t*)o.at;
        o_stride = o.stride;
      }
    } else if (a[11] != Py_None) {
      throw Refused();
    }
    {
      const Unlocked unlocked;
      if (a[0] != Py_None && a[11] == Py_None) {
        out = at::empty({k.tokens, q_heads, k.dim}, made);
        op = (uint16_t*)out.data_ptr();
        o_stride = q_heads * k.dim;
      }
      done(wq_kv_append_rotary(qp, q_stride, (int32_t)q_heads, k.at, k.stride, v.at, v.stride, type, positions, cos_sin,
                               max_pos, (int32_t)rot, inter, slots, k.tokens, (int32_t)k.heads, (int32_t)k.dim,
                               c.four ? WQ_E2M1X2 : WQ_E4M3, (int32_t)c.page, c.pages, c.kc, c.ks, c.vc, c.vs, op, o_stride,
                               stream));
    }
    if (a[11] != Py_None || a[0] == Py_None) {
      Py_INCREF(a[11]);
      return a[11];
    }
    return THPVariable_Wrap(out);
  });
}

// (q, k_codes, k_scales, v_codes, v_scales, block_table, cu_q, kv_lens, sm_scale or None, softcap, window, max_q,
//  out or None, return_lse, workspace or None)
PyObject* kv4_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call("wq_kv4_attention", n, 15, [&]() -> PyObject* {
    const Tensor& q = tensor(a[0]);
    const Rows r(q);
    const Cache c(a + 1, r.dev);
    if (!c.four || r.type != at::kBFloat16 || r.dim != c.dim || !small(r.heads) || !small(c.heads)) throw Refused();
    const Tensor& table = dense(a[5], at::kInt, r.dev);
    if (table.dim() != 2) throw Refused();
    const int64_t batch = table.size(0), width = table.size(1);
    const int32_t* cu = dense_at<int32_t>(a[6], at::kInt, r.dev, {batch + 1});
    const int32_t* lens = dense_at<int32_t>(a[7], at::kInt, r.dev, {batch});
    const float sm_scale = a[8] == Py_None ? (float)std::pow((double)r.dim, -0.5) : number(a[8]), softcap = number(a[9]);
    const int64_t window = whole(a[10]), max_q = whole(a[11]);
    const int with_lse = PyObject_IsTrue(a[13]);
    if (with_lse < 0) throw Refused();
    hipStream_t stream = stream_on(r.dev);
    const int32_t* table_at = (const int32_t*)table.data_ptr();
    const at::TensorOptions like = q.options();
    Tensor out, lse, ws;
    if (a[12] != Py_None) {
      out = dense(a[12], at::kBFloat16, r.dev);
      if (out.sizes() != q.sizes()) throw Refused();
    }
    void* ws_at = nullptr;
    size_t ws_bytes = 0;
    if (a[14] != Py_None) {
      ws = tensor(a[14]);
      if (ws.get_device() != r.dev || !ws.is_contiguous()) throw Refused();
      ws_bytes = ws.nbytes();
      ws_at = ws.data_ptr();
    }
    {
      const Unlocked unlocked;
      if (!out.defined()) out = at::empty({r.tokens, r.heads, r.dim}, like);
      if (with_lse) lse = at::empty({r.tokens, r.heads}, like.dtype(at::kFloat));
      if (!ws.defined()) {
        ws_bytes = wq_kv4_attention_workspace_size(batch, r.tokens, max_q, (int32_t)r.heads, (int32_t)c.heads, (int32_t)r.dim,
                                                   (int32_t)c.page, width, window);
        if (ws_bytes) {
          ws = at::empty({(int64_t)ws_bytes}, like.dtype(at::kByte));
          ws_at = ws.data_ptr();
        }
      }
      done(wq_kv4_attention(r.at, r.stride, cu, lens, batch, r.tokens, max_q, (int32_t)r.heads, (int32_t)c.heads,
                            (int32_t)r.dim, c.kc, c.ks, c.vc, c.vs, (int32_t)c.page, c.pages, table_at, width, sm_scale, softcap,
                            window, (uint16_t*)out.data_ptr(), with_lse ? (float*)lse.data_ptr() : nullptr, ws_at, ws_bytes,
                            stream));
    }
    PyObject* o = a[12];
    if (o == Py_None) o = THPVariable_Wrap(out);
    else Py_INCREF(o);
    if (!with_lse || !o) return o;
    PyObject* l = THPVariable_Wrap(lse);
    PyObject* both = l ? PyTuple_Pack(2, o, l) : nullptr;
    Py_DECREF(o);
    Py_XDECREF(l);
    return both;
  });
}

PyMethodDef methods[] = {
    {"kv4_append", (PyCFunction)(void*)kv4_append, METH_FASTCALL, nullptr},
    {"kv_append_rotary", (PyCFunction)(void*)kv_append_rotary, METH_FASTCALL, nullptr},
    {"kv4_attention", (PyCFunction)(void*)kv4_attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

// What lies inside a tensor is the torch's that this was compiled against, and the calling
// convention its Python's; under another of either the module must not be used.
bool built_for_this_process() {
  static const char python[] = Py_STRINGIFY(PY_MAJOR_VERSION) "." Py_STRINGIFY(PY_MINOR_VERSION) ".";
  if (strncmp(Py_GetVersion(), python, sizeof python - 1) != 0) {
    PyErr_Format(PyExc_ImportError, "_calls.so was built for Python %s* and runs under %.20s", python, Py_GetVersion());
    return false;
  }
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* version = torch ? PyObject_GetAttrString(torch, "__version__") : nullptr;
  PyObject* text = version ? PyObject_Str(version) : nullptr;
  const char* now = text ? PyUnicode_AsUTF8(text) : nullptr;
  const bool same = now && strcmp(now, WQ_TORCH) == 0;
  if (now && !same) PyErr_Format(PyExc_ImportError, "_calls.so was built for torch %s and runs under torch %s", WQ_TORCH, now);
  Py_XDECREF(text);
  Py_XDECREF(version);
  Py_XDECREF(torch);
  return same;
}

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return built_for_this_process() ? PyModule_Create(&module) : nullptr; }
