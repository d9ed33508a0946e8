// The Python calls of the FP8 cache's operators and of qk_norm_rope on tensors
// that are exactly as they should be: the same checks as in _lib.py, on the
// tensors themselves instead of through some 80 attribute reads in Python (5 us
// of a 10 us call whose kernel takes 3), then the C ABI.  Whatever is not plain
// (a wrong type, shape, stride or device, an explicit stream, an argument of
// another Python type) returns None: _lib.py then looks again, refuses with the
// reason, or makes the call through ctypes.

#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <climits>
#include <cstdint>

#include "../../include/kvint4.h"

namespace {

decltype(&kv_fp8_write) g_write = nullptr;
decltype(&kv_fp8_read) g_read = nullptr;
decltype(&kv_fp8_attention) g_attention = nullptr;
decltype(&kv_qk_norm_rope) g_norm_rope = nullptr;

struct NotPlain {};

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) throw NotPlain{};
  return THPVariable_Unpack(o);
}
void need(bool ok) {
  if (!ok) throw NotPlain{};
}
int integer(PyObject* o) {
  need(PyLong_Check(o));
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  need(!over && v >= INT_MIN && v <= INT_MAX);
  return (int)v;
}
float real(PyObject* o) {
  need(PyFloat_Check(o));
  return (float)PyFloat_AS_DOUBLE(o);
}

// device pointers of tensors that are all on one device, the current one
struct Device {
  int dev = -1;
  void* of(const at::Tensor& t) {
    need(t.is_cuda() && t.layout() == at::kStrided);
    if (dev < 0) {
      dev = t.get_device();
      need(dev == c10::cuda::current_device());
    }
    need(t.get_device() == dev);
    return t.data_ptr();
  }
  int32_t* status(PyObject* o) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    need(t.scalar_type() == at::kInt && t.numel() >= 1);
    return static_cast<int32_t*>(of(t));
  }
  void* stream(PyObject* o) {
    need(o == Py_None);
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  }
};

// token stride of bf16 head vectors [tokens, heads, d]
int64_t rows(const at::Tensor& x, int64_t tokens, int64_t heads, int64_t d) {
  need(x.dim() == 3 && x.size(0) == tokens && x.size(1) == heads && x.size(2) == d);
  need(x.scalar_type() == at::kBFloat16 && x.stride(2) == 1 && (heads == 1 || x.stride(1) == d));
  return tokens > 0 ? x.stride(0) : heads * d;
}

struct Caches {
  uint8_t *k, *v;
  float *ks, *vs;
  int64_t nb, bs, hkv, d;
  Caches(Device& dev, PyObject* const* a) {
    const at::Tensor &kc = tensor(a[0]), &vc = tensor(a[1]), &kt = tensor(a[2]), &vt = tensor(a[3]);
    need((kc.scalar_type() == at::kFloat8_e4m3fn || kc.scalar_type() == at::kByte) && vc.scalar_type() == kc.scalar_type());
    need(kc.dim() == 4 && kc.sizes() == vc.sizes() && kc.is_contiguous() && vc.is_contiguous());
    nb = kc.size(0), bs = kc.size(1), hkv = kc.size(2), d = kc.size(3);
    for (const at::Tensor* s : {&kt, &vt})
      need(s->scalar_type() == at::kFloat && s->dim() == 2 && s->size(0) == nb && s->size(1) == hkv && s->is_contiguous());
    need(nb <= INT_MAX && hkv <= INT_MAX);
    k = static_cast<uint8_t*>(dev.of(kc));
    v = static_cast<uint8_t*>(dev.of(vc));
    ks = static_cast<float*>(dev.of(kt));
    vs = static_cast<float*>(dev.of(vt));
  }
};

struct Sequences {
  int32_t *table, *lens, *start;
  int num, width;
  Sequences(Device& dev, PyObject* const* a) {
    const at::Tensor &t = tensor(a[0]), &l = tensor(a[1]), &s = tensor(a[2]);
    need(t.scalar_type() == at::kInt && t.dim() == 2 && t.is_contiguous());
    need(l.scalar_type() == at::kInt && s.scalar_type() == at::kInt && l.is_contiguous() && s.is_contiguous());
    need(l.dim() == 1 && l.size(0) == t.size(0) && s.dim() == 1 && s.size(0) == t.size(0) + 1);
    need(t.size(0) < INT_MAX && t.size(1) <= INT_MAX);
    num = (int)t.size(0), width = (int)t.size(1);
    table = static_cast<int32_t*>(dev.of(t));
    lens = static_cast<int32_t*>(dev.of(l));
    start = static_cast<int32_t*>(dev.of(s));
  }
};

// f() without the interpreter lock, its status as an int; None if the arguments
// are not plain
template <typename F>
PyObject* call(F&& prepare) {
  int code;
  try {
    auto launch = prepare();
    Py_BEGIN_ALLOW_THREADS;
    code = launch();
    Py_END_ALLOW_THREADS;
  } catch (const NotPlain&) {
    Py_RETURN_NONE;
  } catch (const std::exception&) {  // a tensor without memory of its own, say
    Py_RETURN_NONE;
  }
  return PyLong_FromLong(code);
}

// (k, v, block_table, seq_lens, start_loc, max_len, k_cache, v_cache, k_scale, v_scale, dev_status, stream)
PyObject* fp8_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 12 && g_write);
    Device dev;
    const Caches c(dev, a + 6);
    const Sequences s(dev, a + 2);
    const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
    need(k.dim() == 3 && k.size(0) <= INT_MAX);
    const int tokens = (int)k.size(0), max_len = integer(a[5]);
    const int64_t ks = rows(k, tokens, c.hkv, c.d), vs = rows(v, tokens, c.hkv, c.d);
    void *kp = dev.of(k), *vp = dev.of(v);
    int32_t* st = dev.status(a[10]);
    void* stream = dev.stream(a[11]);
    return [=] {
      return g_write(kp, ks, vp, vs, s.table, s.width, s.lens, s.start, s.num, tokens, max_len, c.k, c.v, c.ks, c.vs,
                     (int)c.nb, (int)c.bs, (int)c.hkv, (int)c.d, st, stream);
    };
  });
}

// (k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, start_loc, max_len, k, v, dev_status, stream)
PyObject* fp8_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 12 && g_read);
    Device dev;
    const Caches c(dev, a);
    const Sequences s(dev, a + 4);
    const at::Tensor &k = tensor(a[8]), &v = tensor(a[9]);
    need(k.dim() == 3 && k.size(0) <= INT_MAX);
    const int tokens = (int)k.size(0), max_len = integer(a[7]);
    const int64_t ks = rows(k, tokens, c.hkv, c.d), vs = rows(v, tokens, c.hkv, c.d);
    void *kp = dev.of(k), *vp = dev.of(v);
    int32_t* st = dev.status(a[10]);
    void* stream = dev.stream(a[11]);
    return [=] {
      return g_read(c.k, c.v, c.ks, c.vs, s.table, s.width, s.lens, s.start, s.num, tokens, max_len, kp, ks, vp, vs,
                    (int)c.nb, (int)c.bs, (int)c.hkv, (int)c.d, st, stream);
    };
  });
}

// (q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, query_start_loc, max_query_len, max_seq_len,
//  softmax_scale, causal, out, workspace, dev_status, stream, sliding_window)
PyObject* fp8_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 17 && g_attention);
    Device dev;
    const Caches c(dev, a + 1);
    const Sequences s(dev, a + 5);
    const at::Tensor &q = tensor(a[0]), &out = tensor(a[12]), &ws = tensor(a[13]);
    need(q.dim() == 3 && q.size(0) <= INT_MAX && q.size(1) <= INT_MAX);
    const int tokens = (int)q.size(0), hq = (int)q.size(1);
    const int64_t qs = rows(q, tokens, hq, c.d), os = rows(out, tokens, hq, c.d);
    need(ws.scalar_type() == at::kByte && ws.is_contiguous());
    const int max_q = integer(a[8]), max_len = integer(a[9]), window = integer(a[16]);
    const float scale = real(a[10]);
    need(PyBool_Check(a[11]));
    const int causal = a[11] == Py_True;
    void *qp = dev.of(q), *op = dev.of(out), *wp = dev.of(ws);
    const size_t bytes = (size_t)ws.numel();
    int32_t* st = dev.status(a[14]);
    void* stream = dev.stream(a[15]);
    return [=] {
      return g_attention(qp, qs, c.k, c.v, c.ks, c.vs, s.table, s.width, s.lens, s.start, s.num, tokens, max_q, max_len,
                         hq, (int)c.hkv, (int)c.d, (int)c.bs, (int)c.nb, scale, causal, window, op, os, wp, bytes, st,
                         stream);
    };
  });
}

// (q, k, positions, cos_sin, q_weight, k_weight, eps, q_out, k_out, interleaved, dev_status, stream)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 12 && g_norm_rope);
    Device dev;
    const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &qo = tensor(a[7]), &ko = tensor(a[8]);
    need(q.dim() == 3 && k.dim() == 3 && q.size(0) <= INT_MAX && q.size(1) <= INT_MAX && k.size(1) <= INT_MAX &&
         q.size(2) <= INT_MAX);
    const int tokens = (int)q.size(0), hq = (int)q.size(1), hkv = (int)k.size(1), d = (int)q.size(2);
    const int64_t qs = rows(q, tokens, hq, d), ks = rows(k, tokens, hkv, d);
    const int64_t qos = rows(qo, tokens, hq, d), kos = rows(ko, tokens, hkv, d);
    void *qp = dev.of(q), *kp = dev.of(k), *qop = dev.of(qo), *kop = dev.of(ko);
    void *qw = nullptr, *kw = nullptr;
    int64_t* pos = nullptr;
    float* table = nullptr;
    int max_pos = 0, rot = 0;
    need((a[4] == Py_None) == (a[5] == Py_None) && (a[2] == Py_None) == (a[3] == Py_None));
    if (a[4] != Py_None) {
      const at::Tensor &w = tensor(a[4]), &x = tensor(a[5]);
      for (const at::Tensor* t : {&w, &x})
        need(t->scalar_type() == at::kBFloat16 && t->dim() == 1 && t->size(0) == d && t->is_contiguous());
      qw = dev.of(w);
      kw = dev.of(x);
    }
    if (a[2] != Py_None) {
      const at::Tensor &p = tensor(a[2]), &t = tensor(a[3]);
      need(t.scalar_type() == at::kFloat && t.dim() == 2 && t.is_contiguous() && t.size(0) <= INT_MAX &&
           t.size(1) <= INT_MAX);
      need(p.scalar_type() == at::kLong && p.dim() == 1 && p.size(0) == tokens && p.is_contiguous());
      max_pos = (int)t.size(0), rot = (int)t.size(1);
      pos = static_cast<int64_t*>(dev.of(p));
      table = static_cast<float*>(dev.of(t));
    }
    const float eps = real(a[6]);
    need(PyBool_Check(a[9]));
    const int inter = a[9] == Py_True;
    int32_t* st = dev.status(a[10]);
    void* stream = dev.stream(a[11]);
    return [=] {
      return g_norm_rope(qp, qs, kp, ks, tokens, hq, hkv, d, qw, kw, eps, pos, table, max_pos, rot, inter, qop, qos, kop,
                         kos, st, stream);
    };
  });
}

// bind(write, read, attention, norm_rope): the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  void* f[4];
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "four addresses");
    return nullptr;
  }
  for (int i = 0; i < 4; i++) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_write = reinterpret_cast<decltype(g_write)>(f[0]);
  g_read = reinterpret_cast<decltype(g_read)>(f[1]);
  g_attention = reinterpret_cast<decltype(g_attention)>(f[2]);
  g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(f[3]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<bind>("bind"),           method<fp8_write>("write"),
                           method<fp8_read>("read"),       method<fp8_attention>("attention"),
                           method<norm_rope>("norm_rope"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp8_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_binding() { return PyModule_Create(&g_module); }
