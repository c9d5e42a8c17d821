// The short way into the library from Python for the gated delta rule and the norms around a
// block: checks, allocations and the C call of one operator call, in one go. Each function takes
// what its Python namesake (gdr.py, norm_gate.py) has checked nothing of, on the current stream,
// and returns NotImplemented when anything at all is not as it should be; the Python function then
// goes the long way, which explains the refusal or handles the unusual (another device). That is so
// while nothing has been launched: a failure after that is raised from here, since a call that works
// in place would do so twice. A decode call of one sequence costs 10 us the long way and 4 this way,
// two of them the launch.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <initializer_list>

#include "wkv.h"

namespace {

// Thrown for everything that is left to the long way: nothing has been launched.
struct LongWay {};
// Thrown with a Python error set.
struct Raised {};

using at::Tensor;

const Tensor* tensor(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw LongWay();
  return &THPVariable_Unpack(o);
}
const Tensor& required(PyObject* o) {
  const Tensor* t = tensor(o);
  if (t == nullptr) throw LongWay();
  return *t;
}
void need(const Tensor& t, at::ScalarType dtype, at::IntArrayRef shape, int dev) {
  if (t.scalar_type() != dtype || t.sizes() != shape || !t.is_cuda() || t.get_device() != dev ||
      !t.is_contiguous())
    throw LongWay();
}
void* at_(const Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw LongWay();
  return x;
}
int type_of(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return WKV_DTYPE_BF16;
  if (t.scalar_type() == at::kFloat) return WKV_DTYPE_F32;
  throw LongWay();
}
// The device, which has to be the current one.
int own_device_of(const Tensor& t) {
  if (!t.is_cuda()) throw LongWay();
  const int dev = int(t.get_device());
  if (dev != int(c10::cuda::current_device())) throw LongWay();
  return dev;
}
cudaStream_t stream_of(int dev) {
  return c10::cuda::getCurrentCUDAStream(c10::DeviceIndex(dev)).stream();
}
Tensor floats(at::IntArrayRef shape, const Tensor& like) {
  return at::empty(shape, like.options().dtype(at::kFloat));
}
Tensor bytes(size_t n, const Tensor& like) {
  return at::empty({int64_t(n)}, like.options().dtype(at::kByte));
}
// The outcome of a call into the library: its refusals come before any launch, a CUDA error may
// come after one.
void done(const char* name, int rc) {
  if (rc == WKV_OK) return;
  if (rc != WKV_ERR_CUDA) throw LongWay();
  PyObject* const module = PyImport_ImportModule("rwkv_linear_attention_wkv_b200");
  PyObject* const type = module == nullptr ? nullptr : PyObject_GetAttrString(module, "WkvError");
  PyObject* const error = type == nullptr ? nullptr : PyObject_CallFunction(type, "si", name, rc);
  if (error != nullptr) PyErr_SetObject(type, error);
  Py_XDECREF(error);
  Py_XDECREF(type);
  Py_XDECREF(module);
  throw Raised();
}
// What is made of the results, after the call.
PyObject* made(PyObject* o) {
  if (o == nullptr) throw Raised();
  return o;
}
PyObject* wrap(const Tensor& t) {
  PyObject* o = nullptr;
  try {
    o = THPVariable_Wrap(t);
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, "a result could not be wrapped");
  }
  return made(o);
}
// A given result checked, or a new one.
Tensor result(PyObject* given, const Tensor& like, int dev) {
  if (given == Py_None) return at::empty_like(like);
  const Tensor& t = required(given);
  need(t, like.scalar_type(), like.sizes(), dev);
  return t;
}
void put(PyObject* dict, const char* name, PyObject* value) {
  const int rc = PyDict_SetItemString(dict, name, value);
  Py_DECREF(value);
  if (rc != 0) throw Raised();
}
PyObject* none() { Py_RETURN_NONE; }

// Calls f and turns everything that goes wrong before a launch into the long way.
template <class F>
PyObject* in_short(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n == want) {
    try {
      return f();
    } catch (const Raised&) {
      return nullptr;
    } catch (...) {
      PyErr_Clear();
    }
  }
  Py_RETURN_NOTIMPLEMENTED;
}

// ---- the gated delta rule ----

struct Rule {
  const Tensor &q, &k, &v, &g, &beta;
  wkv_gdr_problem p;
  int dev;
  // a: q, k, v, g, beta; lead: dimensions before the heads
  Rule(PyObject* const* a, int lead, PyObject* scale, PyObject* offsets)
      : q(required(a[0])), k(required(a[1])), v(required(a[2])), g(required(a[3])),
        beta(required(a[4])) {
    if (q.dim() != lead + 2 || v.dim() != lead + 2) throw LongWay();
    dev = own_device_of(v);
    const at::IntArrayRef s = v.sizes();
    p = wkv_gdr_problem{};
    p.B = s[0];
    p.T = lead == 2 ? s[1] : 1;
    p.Hk = q.size(lead);
    p.H = s[lead];
    p.N = s[lead + 1];
    p.dtype = type_of(v);
    p.scale = float(number(scale));
    std::array<int64_t, 4> qk{s[0], lead == 2 ? s[1] : p.Hk, lead == 2 ? p.Hk : p.N, p.N};
    const at::IntArrayRef qk_shape(qk.data(), size_t(lead) + 2), heads = s.slice(0, size_t(lead) + 1);
    need(v, v.scalar_type(), s, dev);
    need(q, v.scalar_type(), qk_shape, dev);
    need(k, v.scalar_type(), qk_shape, dev);
    need(g, at::kFloat, heads, dev);
    need(beta, at::kFloat, heads, dev);
    if (const Tensor* o = tensor(offsets)) {
      if (o->dim() != 1 || o->size(0) < 1 || p.B != 1) throw LongWay();
      need(*o, at::kInt, o->sizes(), dev);
      p.n_seqs = o->size(0) - 1;
      p.seq_offsets = static_cast<const int32_t*>(o->data_ptr());
    }
  }
  std::array<int64_t, 4> states() const {
    return {p.seq_offsets != nullptr ? p.n_seqs : p.B, p.H, p.N, p.N};
  }
  const float* state(PyObject* o) const {
    const Tensor* t = tensor(o);
    if (t != nullptr) need(*t, at::kFloat, states(), dev);
    return static_cast<const float*>(at_(t));
  }
  const float* gp() const { return static_cast<const float*>(g.data_ptr()); }
  const float* bp() const { return static_cast<const float*>(beta.data_ptr()); }
};

// q, k, v, g, beta, state, slots, scale, y -> y
PyObject* gdr_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return in_short(n, 9, [&] {
    Rule r(a, 1, a[7], Py_None);
    const Tensor& state = required(a[5]);
    if (state.dim() != 4) throw LongWay();
    const int64_t slots = state.size(0);
    need(state, at::kFloat, {slots, r.p.H, r.p.N, r.p.N}, r.dev);
    const Tensor* at_slots = tensor(a[6]);
    if (at_slots != nullptr) need(*at_slots, at::kInt, {r.p.B}, r.dev);
    const Tensor y = result(a[8], r.v, r.dev);
    done("wkv_gdr_decode_step",
         wkv_gdr_decode_step(&r.p, r.q.data_ptr(), r.k.data_ptr(), r.v.data_ptr(), r.gp(), r.bp(),
                             y.data_ptr(), static_cast<float*>(state.data_ptr()), slots,
                             static_cast<const int32_t*>(at_(at_slots)), stream_of(r.dev)));
    return wrap(y);
  });
}

// q, k, v, g, beta, state, scale, seq_offsets, y, state_out, want_state[, workspace]
// -> (y, state[, workspace])
PyObject* forward(PyObject* const* a, bool keep) {
  Rule r(a, 2, a[6], a[7]);
  const float* s0 = r.state(a[5]);
  const Tensor y = result(a[8], r.v, r.dev);
  Tensor last;
  const int want = PyObject_IsTrue(a[10]);
  if (want < 0) throw LongWay();
  if (want && a[9] == Py_None) {
    last = floats(r.states(), r.v);
  } else if (want) {
    r.state(a[9]);
    last = required(a[9]);
  }
  Tensor scratch;
  if (r.p.T >= 1024) {
    if (const size_t need_bytes = wkv_gdr_forward_workspace_bytes(&r.p)) {
      scratch = bytes(need_bytes, r.v);
      r.p.workspace = scratch.data_ptr();
      r.p.workspace_bytes = need_bytes;
    }
  }
  float* s1 = want ? static_cast<float*>(last.data_ptr()) : nullptr;
  Tensor kept;
  if (keep) {
    const size_t need_bytes = wkv_gdr_checkpoint_bytes(&r.p);
    if (a[11] == Py_None) {
      kept = bytes(need_bytes, r.v);
    } else {
      kept = required(a[11]);
      if (!kept.is_cuda() || kept.get_device() != r.dev || !kept.is_contiguous() ||
          kept.nbytes() < need_bytes)
        throw LongWay();
    }
    done("wkv_gdr_forward_checkpointed",
         wkv_gdr_forward_checkpointed(&r.p, r.q.data_ptr(), r.k.data_ptr(), r.v.data_ptr(), r.gp(),
                                      r.bp(), y.data_ptr(), s0, s1, kept.data_ptr(), kept.nbytes(),
                                      stream_of(r.dev)));
  } else {
    done("wkv_gdr_forward",
         wkv_gdr_forward(&r.p, r.q.data_ptr(), r.k.data_ptr(), r.v.data_ptr(), r.gp(), r.bp(),
                         y.data_ptr(), s0, s1, stream_of(r.dev)));
  }
  PyObject* const py = wrap(y);
  PyObject* const ps = want ? wrap(last) : none();
  return made(keep ? Py_BuildValue("NNN", py, ps, wrap(kept)) : Py_BuildValue("NN", py, ps));
}
PyObject* gdr_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return in_short(n, 11, [&] { return forward(a, false); });
}
PyObject* gdr_forward_checkpointed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return in_short(n, 12, [&] { return forward(a, true); });
}

// q, k, v, g, beta, dy, workspace, grad_state, scale, seq_offsets, want_dstate -> dict
PyObject* gdr_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return in_short(n, 11, [&] {
    Rule r(a, 2, a[8], a[9]);
    const Tensor &dy = required(a[5]), &kept = required(a[6]);
    need(dy, r.v.scalar_type(), r.v.sizes(), r.dev);
    const float* ds1 = r.state(a[7]);
    const int want = PyObject_IsTrue(a[10]);
    if (want < 0 || !kept.is_cuda() || kept.get_device() != r.dev || !kept.is_contiguous())
      throw LongWay();
    const Tensor dq = at::empty_like(r.q), dk = at::empty_like(r.k), dv = at::empty_like(r.v),
                 dg = at::empty_like(r.g), db = at::empty_like(r.beta);
    Tensor ds;
    if (want) ds = floats(r.states(), r.v);
    const Tensor scratch = bytes(wkv_gdr_backward_workspace_bytes(&r.p), r.v);
    done("wkv_gdr_backward",
         wkv_gdr_backward(&r.p, r.q.data_ptr(), r.k.data_ptr(), r.v.data_ptr(), r.gp(), r.bp(),
                          dy.data_ptr(), kept.data_ptr(), kept.nbytes(), ds1, dq.data_ptr(),
                          dk.data_ptr(), dv.data_ptr(), static_cast<float*>(dg.data_ptr()),
                          static_cast<float*>(db.data_ptr()),
                          want ? static_cast<float*>(ds.data_ptr()) : nullptr, scratch.data_ptr(),
                          scratch.nbytes(), stream_of(r.dev)));
    PyObject* const d = made(PyDict_New());
    put(d, "dq", wrap(dq));
    put(d, "dk", wrap(dk));
    put(d, "dv", wrap(dv));
    put(d, "dg", wrap(dg));
    put(d, "dbeta", wrap(db));
    put(d, "dstate", want ? wrap(ds) : none());
    return d;
  });
}

// ---- the norms around a block ----

struct Norm {
  const Tensor& h;
  const Tensor *weight, *gate, *x, *scale, *next_weight;
  wkv_norm_gate_problem p;
  int dev;
  Norm(PyObject* h_, PyObject* w_, PyObject* z_, PyObject* x_, PyObject* s_, PyObject* n_,
       PyObject* group, PyObject* act, PyObject* eps)
      : h(required(h_)), weight(tensor(w_)), gate(tensor(z_)), x(tensor(x_)), scale(tensor(s_)),
        next_weight(tensor(n_)) {
    if (h.dim() < 1 || !PyUnicode_Check(act)) throw LongWay();
    dev = own_device_of(h);
    const int64_t C = h.size(-1);
    if (C == 0) throw LongWay();
    p = wkv_norm_gate_problem{};
    p.C = C;
    p.R = h.numel() / C;
    p.dtype = type_of(h);
    p.act = PyUnicode_CompareWithASCIIString(act, "silu") == 0      ? WKV_ACT_SILU
            : PyUnicode_CompareWithASCIIString(act, "sigmoid") == 0 ? WKV_ACT_SIGMOID
                                                                    : WKV_ACT_NONE;
    if (p.act == WKV_ACT_NONE && PyUnicode_CompareWithASCIIString(act, "none") != 0)
      throw LongWay();
    if ((gate == nullptr) != (p.act == WKV_ACT_NONE) || (scale != nullptr && x == nullptr))
      throw LongWay();
    p.eps = float(number(eps));
    p.group = C;
    if (group != Py_None) {
      p.group = PyLong_Check(group) ? PyLong_AsLongLong(group) : 0;
      if (p.group <= 0 || C % p.group != 0) throw LongWay();
    }
    need(h, h.scalar_type(), h.sizes(), dev);
    for (const Tensor* t : {gate, x})
      if (t != nullptr) need(*t, h.scalar_type(), h.sizes(), dev);
    for (const Tensor* t : {weight, scale, next_weight})
      if (t != nullptr) need(*t, at::kFloat, {C}, dev);
  }
  static const float* fp(const Tensor* t) { return static_cast<const float*>(at_(t)); }
};

// h, weight, gate, x, scale, next_weight, group, act, eps, out, y -> (out, y)
PyObject* norm_gate_forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return in_short(n, 11, [&] {
    Norm m(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8]);
    if (m.next_weight == nullptr && a[10] != Py_None) throw LongWay();
    const Tensor out = result(a[9], m.h, m.dev);
    Tensor y;
    if (m.next_weight != nullptr) y = result(a[10], m.h, m.dev);
    done("wkv_norm_gate_forward",
         wkv_norm_gate_forward(&m.p, m.h.data_ptr(), m.fp(m.weight), at_(m.gate), at_(m.x),
                               m.fp(m.scale), m.fp(m.next_weight), out.data_ptr(),
                               m.next_weight != nullptr ? y.data_ptr() : nullptr,
                               stream_of(m.dev)));
    PyObject* const po = wrap(out);
    return made(Py_BuildValue("NN", po, m.next_weight != nullptr ? wrap(y) : none()));
  });
}

// h, weight, dout, gate, x, scale, next_weight, dy, group, act, eps -> dict
PyObject* norm_gate_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return in_short(n, 11, [&] {
    Norm m(a[0], a[1], a[3], a[4], a[5], a[6], a[8], a[9], a[10]);
    const Tensor *dout = tensor(a[2]), *dy = tensor(a[7]);
    if ((dout == nullptr && dy == nullptr) || (dy != nullptr && m.next_weight == nullptr))
      throw LongWay();
    for (const Tensor* t : {dout, dy})
      if (t != nullptr) need(*t, m.h.scalar_type(), m.h.sizes(), m.dev);
    auto like = [](const Tensor* t) { return t == nullptr ? Tensor() : at::empty_like(*t); };
    auto ptr = [](const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
    auto fptr = [](const Tensor& t) {
      return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr;
    };
    const Tensor dh = at::empty_like(m.h), dw = like(m.weight), dz = like(m.gate), dx = like(m.x),
                 ds = like(m.scale), dn = dy == nullptr ? Tensor() : like(m.next_weight);
    const Tensor scratch = bytes(wkv_norm_gate_workspace_bytes(m.p.R, m.p.C), m.h);
    done("wkv_norm_gate_backward",
         wkv_norm_gate_backward(&m.p, m.h.data_ptr(), m.fp(m.weight), at_(m.gate), at_(m.x),
                                m.fp(m.scale), m.fp(m.next_weight), at_(dout), at_(dy),
                                dh.data_ptr(), fptr(dw), ptr(dz), ptr(dx), fptr(ds), fptr(dn),
                                scratch.data_ptr(), scratch.nbytes(), stream_of(m.dev)));
    PyObject* const d = made(PyDict_New());
    auto give = [&](const char* name, const Tensor& t) {
      put(d, name, t.defined() ? wrap(t) : none());
    };
    give("dh", dh);
    give("dweight", dw);
    give("dgate", dz);
    give("dx", dx);
    give("dscale", ds);
    give("dnext_weight", dn);
    return d;
  });
}

#define FAST(f) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr }
PyMethodDef kMethods[] = {FAST(gdr_decode),   FAST(gdr_forward),
                          FAST(gdr_forward_checkpointed), FAST(gdr_backward),
                          FAST(norm_gate_forward), FAST(norm_gate_backward),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

// (build.py looks for these words, gdr.py compares the version with the torch that runs)
const char kBuiltFor[] = "built for torch " TORCH_BUILT_FOR;

PyMODINIT_FUNC PyInit__binding() {
  PyObject* const m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version",
                                                 kBuiltFor + sizeof("built for torch ") - 1) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
