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
decltype(&kv_qk_norm_rope_axes) g_norm_rope_axes = nullptr;
decltype(&kv_fp8_attention_mass) g_mass = nullptr;
decltype(&kv_fp8_evict) g_evict = nullptr;
decltype(&kv_fp8_attention_shared) g_shared = nullptr;

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

// the head vectors, their outputs and weights of the rotary calls
struct Vectors {
  int tokens, hq, hkv, d;
  int64_t qs, ks, qos, kos;
  void *q, *k, *qo, *ko, *qw = nullptr, *kw = nullptr;
  Vectors(Device& dev, PyObject* aq, PyObject* ak, PyObject* wq, PyObject* wk, PyObject* oq, PyObject* ok) {
    const at::Tensor &x = tensor(aq), &y = tensor(ak), &xo = tensor(oq), &yo = tensor(ok);
    need(x.dim() == 3 && y.dim() == 3 && x.size(0) <= INT_MAX && x.size(1) <= INT_MAX && y.size(1) <= INT_MAX &&
         x.size(2) <= INT_MAX);
    tokens = (int)x.size(0), hq = (int)x.size(1), hkv = (int)y.size(1), d = (int)x.size(2);
    qs = rows(x, tokens, hq, d), ks = rows(y, tokens, hkv, d);
    qos = rows(xo, tokens, hq, d), kos = rows(yo, tokens, hkv, d);
    q = dev.of(x), k = dev.of(y), qo = dev.of(xo), ko = dev.of(yo);
    need((wq == Py_None) == (wk == Py_None));
    if (wq != Py_None) {
      const at::Tensor &w = tensor(wq), &v = tensor(wk);
      for (const at::Tensor* t : {&w, &v})
        need(t->scalar_type() == at::kBFloat16 && t->dim() == 1 && t->size(0) == d && t->is_contiguous());
      qw = dev.of(w);
      kw = dev.of(v);
    }
  }
};

// a table of cosines and sines
struct Table {
  float* of;
  int max_pos, rot;
  Table(Device& dev, const at::Tensor& t) {
    need(t.scalar_type() == at::kFloat && t.dim() == 2 && t.is_contiguous() && t.size(0) <= INT_MAX &&
         t.size(1) <= INT_MAX);
    max_pos = (int)t.size(0), rot = (int)t.size(1);
    of = static_cast<float*>(dev.of(t));
  }
};

// (q, k, positions, cos_sin, q_weight, k_weight, eps, q_out, k_out, interleaved, dev_status, stream)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 12 && g_norm_rope);
    Device dev;
    const Vectors x(dev, a[0], a[1], a[4], a[5], a[7], a[8]);
    int64_t* pos = nullptr;
    float* table = nullptr;
    int max_pos = 0, rot = 0;
    need((a[2] == Py_None) == (a[3] == Py_None));
    if (a[2] != Py_None) {
      const at::Tensor& p = tensor(a[2]);
      need(p.scalar_type() == at::kLong && p.dim() == 1 && p.size(0) == x.tokens && p.is_contiguous());
      const Table t(dev, tensor(a[3]));
      max_pos = t.max_pos, rot = t.rot, table = t.of;
      pos = static_cast<int64_t*>(dev.of(p));
    }
    const float eps = real(a[6]);
    need(PyBool_Check(a[9]));
    const int inter = a[9] == Py_True;
    int32_t* st = dev.status(a[10]);
    void* stream = dev.stream(a[11]);
    return [=] {
      return g_norm_rope(x.q, x.qs, x.k, x.ks, x.tokens, x.hq, x.hkv, x.d, x.qw, x.kw, eps, pos, table, max_pos, rot,
                         inter, x.qo, x.qos, x.ko, x.kos, st, stream);
    };
  });
}

// (q, k, positions, cos_sin, pair_axis, q_weight, k_weight, eps, q_out, k_out, interleaved, dev_status, stream)
PyObject* norm_rope_axes(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 13 && g_norm_rope_axes);
    Device dev;
    const Vectors x(dev, a[0], a[1], a[5], a[6], a[8], a[9]);
    const at::Tensor& p = tensor(a[2]);
    need(p.scalar_type() == at::kLong && p.dim() == 2 && p.size(0) <= INT_MAX && p.size(1) == x.tokens &&
         (x.tokens <= 1 || p.stride(1) == 1));
    const Table t(dev, tensor(a[3]));
    need(PyBytes_Check(a[4]) && PyBytes_GET_SIZE(a[4]) == t.rot / 2);
    const uint8_t* axes = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(a[4]));  // the caller holds it
    const int num_axes = (int)p.size(0);
    const int64_t axis_stride = p.stride(0);
    int64_t* pos = static_cast<int64_t*>(dev.of(p));
    const float eps = real(a[7]);
    need(PyBool_Check(a[10]));
    const int inter = a[10] == Py_True;
    int32_t* st = dev.status(a[11]);
    void* stream = dev.stream(a[12]);
    return [=] {
      return g_norm_rope_axes(x.q, x.qs, x.k, x.ks, x.tokens, x.hq, x.hkv, x.d, x.qw, x.kw, eps, pos, axis_stride,
                              num_axes, axes, t.of, t.max_pos, t.rot, inter, x.qo, x.qos, x.ko, x.kos, st, stream);
    };
  });
}

// token stride of fp32 [tokens, q heads]
int64_t lse_stride(const at::Tensor& x, int64_t tokens, int64_t heads) {
  need(x.scalar_type() == at::kFloat && x.dim() == 2 && x.size(0) == tokens && x.size(1) == heads &&
       (heads <= 1 || x.stride(1) == 1));
  return tokens > 1 ? x.stride(0) : heads;
}

// (q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, query_start_loc, max_query_len, max_seq_len, group_start,
//  prefix_lens, max_group_tokens, softmax_scale, out, workspace, lse, dev_status, stream)
PyObject* fp8_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 19 && g_shared);
    Device dev;
    const Caches c(dev, a + 1);
    const Sequences s(dev, a + 5);
    const at::Tensor &q = tensor(a[0]), &out = tensor(a[14]), &ws = tensor(a[15]);
    need(q.dim() == 3 && q.size(0) <= INT_MAX && q.size(1) <= INT_MAX);
    const int tokens = (int)q.size(0), hq = (int)q.size(1);
    const int64_t qs = rows(q, tokens, hq, c.d), os = rows(out, tokens, hq, c.d);
    const at::Tensor &gs = tensor(a[10]), &pl = tensor(a[11]);
    need(pl.scalar_type() == at::kInt && pl.dim() == 1 && pl.is_contiguous() && pl.size(0) < INT_MAX);
    need(gs.scalar_type() == at::kInt && gs.dim() == 1 && gs.is_contiguous() && gs.size(0) == pl.size(0) + 1);
    need(ws.scalar_type() == at::kByte && ws.is_contiguous());
    const int groups = (int)pl.size(0), max_q = integer(a[8]), max_len = integer(a[9]), max_group = integer(a[12]);
    const float scale = real(a[13]);
    float* lp = nullptr;
    int64_t ls = 0;
    if (a[16] != Py_None) {
      const at::Tensor& lse = tensor(a[16]);
      ls = lse_stride(lse, tokens, hq);
      lp = static_cast<float*>(dev.of(lse));
    }
    void *qp = dev.of(q), *op = dev.of(out), *wp = dev.of(ws);
    int32_t *gp = static_cast<int32_t*>(dev.of(gs)), *pp = static_cast<int32_t*>(dev.of(pl));
    const size_t bytes = (size_t)ws.numel();
    int32_t* st = dev.status(a[17]);
    void* stream = dev.stream(a[18]);
    return [=] {
      return g_shared(qp, qs, c.k, c.v, c.ks, c.vs, s.table, s.width, s.lens, s.start, s.num, tokens, max_q, max_len, gp,
                      pp, groups, max_group, hq, (int)c.hkv, (int)c.d, (int)c.bs, (int)c.nb, scale, op, os, lp, ls, wp,
                      bytes, st, stream);
    };
  });
}

// masses [sequences, kv heads, positions]
struct Mass {
  float* of;
  int64_t seq, head;
  int room;
  Mass(Device& dev, const at::Tensor& t, int64_t seqs, int64_t heads) {
    need(t.scalar_type() == at::kFloat && t.dim() == 3 && t.size(0) == seqs && t.size(1) == heads &&
         t.size(2) <= INT_MAX && (t.size(2) <= 1 || t.stride(2) == 1));
    seq = t.stride(0), head = t.stride(1), room = (int)t.size(2);
    of = static_cast<float*>(dev.of(t));
  }
};

// (q, lse, k_cache, k_scale, block_table, seq_lens, query_start_loc, max_query_len, max_seq_len, softmax_scale, mass,
//  dev_status, stream)
PyObject* fp8_mass(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 13 && g_mass);
    Device dev;
    PyObject* const caches[4] = {a[2], a[2], a[3], a[3]};
    const Caches c(dev, caches);
    const Sequences s(dev, a + 4);
    const at::Tensor &q = tensor(a[0]), &lse = tensor(a[1]);
    need(q.dim() == 3 && q.size(0) <= INT_MAX && q.size(1) <= INT_MAX);
    const int tokens = (int)q.size(0), hq = (int)q.size(1);
    const int64_t qs = rows(q, tokens, hq, c.d);
    const int64_t ls = lse_stride(lse, tokens, hq);
    const Mass m(dev, tensor(a[10]), s.num, c.hkv);
    const int max_q = integer(a[7]), max_len = integer(a[8]);
    const float scale = real(a[9]);
    void* qp = dev.of(q);
    float* lp = static_cast<float*>(dev.of(lse));
    int32_t* st = dev.status(a[11]);
    void* stream = dev.stream(a[12]);
    return [=] {
      return g_mass(qp, qs, lp, ls, c.k, c.ks, s.table, s.width, s.lens, s.start, s.num, tokens, max_q, max_len, hq,
                    (int)c.hkv, (int)c.d, (int)c.bs, (int)c.nb, scale, m.of, m.seq, m.head, m.room, st, stream);
    };
  });
}

// (k_cache, v_cache, k_scale, v_scale, mass, block_table, seq_lens, budget, recent, dst_block_table, mass_out, new_lens,
//  kept, dev_status, stream)
PyObject* fp8_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return call([&] {
    need(n == 15 && g_evict);
    Device dev;
    const Caches c(dev, a);
    const int budget = integer(a[7]), recent = integer(a[8]);
    const at::Tensor &t = tensor(a[5]), &to = tensor(a[9]), &l = tensor(a[6]), &nl = tensor(a[11]), &kept = tensor(a[12]);
    for (const at::Tensor* x : {&t, &to})
      need(x->scalar_type() == at::kInt && x->dim() == 2 && x->is_contiguous() && x->size(0) < INT_MAX &&
           x->size(1) <= INT_MAX);
    const int num = (int)t.size(0), width = (int)t.size(1), to_width = (int)to.size(1);
    need(to.size(0) == num);
    for (const at::Tensor* x : {&l, &nl})
      need(x->scalar_type() == at::kInt && x->dim() == 1 && x->size(0) == num && x->is_contiguous());
    need(kept.scalar_type() == at::kInt && kept.dim() == 3 && kept.size(0) == num && kept.size(1) == c.hkv &&
         kept.size(2) == budget && kept.is_contiguous());
    const Mass m(dev, tensor(a[4]), num, c.hkv), mo(dev, tensor(a[10]), num, c.hkv);
    need(mo.room >= (m.room < budget ? m.room : budget));
    int32_t *tp = static_cast<int32_t*>(dev.of(t)), *top = static_cast<int32_t*>(dev.of(to));
    int32_t *lp = static_cast<int32_t*>(dev.of(l)), *nlp = static_cast<int32_t*>(dev.of(nl));
    int32_t* kp = static_cast<int32_t*>(dev.of(kept));
    need(num == 0 || lp != nlp);
    int32_t* st = dev.status(a[13]);
    void* stream = dev.stream(a[14]);
    return [=] {
      return g_evict(c.k, c.v, c.ks, c.vs, (int)c.nb, (int)c.bs, (int)c.hkv, (int)c.d, m.of, m.seq, m.head, m.room, tp,
                     width, lp, num, budget, recent, top, to_width, mo.of, mo.seq, mo.head, nlp, kp, st, stream);
    };
  });
}

// bind(write, read, attention, norm_rope, norm_rope_axes, mass, evict, shared): the library's functions
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int N = 8;
  void* f[N];
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "an address for each function");
    return nullptr;
  }
  for (int i = 0; i < N; i++) {
    f[i] = PyLong_AsVoidPtr(a[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_write = reinterpret_cast<decltype(g_write)>(f[0]);
  g_read = reinterpret_cast<decltype(g_read)>(f[1]);
  g_attention = reinterpret_cast<decltype(g_attention)>(f[2]);
  g_norm_rope = reinterpret_cast<decltype(g_norm_rope)>(f[3]);
  g_norm_rope_axes = reinterpret_cast<decltype(g_norm_rope_axes)>(f[4]);
  g_mass = reinterpret_cast<decltype(g_mass)>(f[5]);
  g_evict = reinterpret_cast<decltype(g_evict)>(f[6]);
  g_shared = reinterpret_cast<decltype(g_shared)>(f[7]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<bind>("bind"),           method<fp8_write>("write"),
                           method<fp8_read>("read"),       method<fp8_attention>("attention"),
                           method<norm_rope>("norm_rope"), method<norm_rope_axes>("norm_rope_axes"),
                           method<fp8_mass>("mass"),       method<fp8_evict>("evict"),
                           method<fp8_shared>("shared"),   {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_fp8_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_binding() { return PyModule_Create(&g_module); }
