// Python binding of the rotated cache writes and the 8-bit cache.
//
// A decode step makes these calls once per layer with about fifteen tensors each.
// Reading shapes, strides, types, devices and addresses from Python and handing
// thirty numbers to ctypes takes 15-22 us of host time a call; here a call takes 3 us,
// its launches included.  The checks are of what the C entry points cannot see: that every tensor is
// on the current device, and that shapes, types and strides fit one another.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <stdexcept>
#include <string>

#include "../../include/pagedattn.h"

namespace {

using at::Tensor;
constexpr auto kInt = at::ScalarType::Int;
constexpr auto kFloat = at::ScalarType::Float;

struct Bad : std::invalid_argument {
  using std::invalid_argument::invalid_argument;
};

// One call's arguments.
struct Args {
  const char* where;
  PyObject* const* v;
  const Tensor* seen[20] = {};
  int count = 0;
  unsigned dense = 0;              // which of them must be contiguous

  [[noreturn]] void fail(const char* what) const {
    throw Bad(std::string(where) + ": " + what);
  }
  void need(bool ok, const char* what) const {
    if (!ok) fail(what);
  }
  // A tensor; null for None where that is allowed.
  const Tensor* tensor(int i, bool optional = false) {
    if (v[i] == Py_None && optional) return nullptr;
    need(THPVariable_Check(v[i]), "expected a tensor");
    return seen[count++] = &THPVariable_Unpack(v[i]);
  }
  const Tensor* packed(int i, bool optional = false) {
    const Tensor* t = tensor(i, optional);
    if (t) dense |= 1u << (count - 1);
    return t;
  }
  const Tensor* index(int i, bool optional = false) {
    const Tensor* t = packed(i, optional);
    need(!t || t->scalar_type() == kInt, "index arrays are contiguous int32");
    return t;
  }
  const Tensor* status(int i) {
    const Tensor* t = index(i, true);
    need(!t || t->numel() >= 1, "status is one int32");
    return t;
  }
  // What is left to see of every tensor, before any address is taken.
  void placed() const {
    for (int i = 0; i < count; ++i) {
      need(!(dense >> i & 1) || seen[i]->is_contiguous(), "tensors must be contiguous");
      need(seen[i]->is_cuda(), "every tensor must be on the current CUDA device");
      for (const int64_t n : seen[i]->sizes())
        need(n <= 0x7FFFFFFF, "a size does not fit 32 bits");
    }
    const int device = c10::cuda::current_device();
    for (int i = 0; i < count; ++i)
      need(seen[i]->get_device() == device, "every tensor must be on the current CUDA device");
  }
  cudaStream_t stream(int i) const {
    if (v[i] == Py_None) return c10::cuda::getCurrentCUDAStream().stream();
    PyObject* n = PyLong_Check(v[i]) ? Py_NewRef(v[i]) : PyObject_GetAttrString(v[i], "cuda_stream");
    if (!n) throw Bad("");
    void* p = PyLong_AsVoidPtr(n);
    Py_DECREF(n);
    if (PyErr_Occurred()) throw Bad("");
    return static_cast<cudaStream_t>(p);
  }
  double number(int i) const {
    const double x = PyFloat_AsDouble(v[i]);
    if (PyErr_Occurred()) throw Bad("");
    return x;
  }
  int dtype(const Tensor& t) const {
    if (t.scalar_type() == at::ScalarType::Half) return PA_FLOAT16;
    if (t.scalar_type() == at::ScalarType::BFloat16) return PA_BFLOAT16;
    fail("unsupported dtype; use float16 or bfloat16");
  }
};

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }
template <typename T>
T* ptr_as(const Tensor* t) { return static_cast<T*>(ptr(t)); }

// Elements from token to token of [T, heads, D] with packed heads (0: packed).
int64_t token_stride(const Args& a, const Tensor& t) {
  a.need(t.stride(2) == 1 && (t.size(1) == 1 || t.stride(1) == t.size(2)),
         "the heads of a token must be packed");
  if (t.size(0) <= 1) return 0;
  a.need(t.stride(0) > 0, "tokens that share one row (a stride of 0) are no token rows");
  return t.stride(0);
}

void check_q8(const Args& a, const Tensor& k, const Tensor& v, const Tensor& ks, const Tensor& vs) {
  auto eight = [](const Tensor& t) {
    return t.scalar_type() == at::ScalarType::Float8_e4m3fn ||
           t.scalar_type() == at::ScalarType::Byte;
  };
  a.need(eight(k) && eight(v), "8-bit pools are float8_e4m3fn (or its bytes, uint8)");
  a.need(k.dim() == 4 && v.sizes() == k.sizes(), "8-bit pools are [NB, Hkv, bs, D], both alike");
  a.need(ks.scalar_type() == kFloat && vs.scalar_type() == kFloat &&
             ks.sizes() == k.sizes().slice(0, 2) && vs.sizes() == k.sizes().slice(0, 2),
         "scales are fp32 [num_blocks, num_kv_heads]");
}

// What both rotated writes take: q_out, pools (and scales), q, key, value, cos_sin,
// block_tables, seq_lens, q_start, q_weight, k_weight, eps, interleaved, positions,
// status, stream.
long rope(Args a, bool q8) {
  int i = 0;
  const Tensor& out = *a.packed(i++);
  const Tensor& kp = *a.packed(i++);
  const Tensor& vp = *a.packed(i++);
  const Tensor* ks = q8 ? a.packed(i++) : nullptr;
  const Tensor* vs = q8 ? a.packed(i++) : nullptr;
  const Tensor& q = *a.tensor(i++);
  const Tensor& k = *a.tensor(i++);
  const Tensor& v = *a.tensor(i++);
  const Tensor* cs = a.packed(i++, true);
  const Tensor& tables = *a.index(i++);
  const Tensor& lens = *a.index(i++);
  const Tensor* q_start = a.index(i++, true);
  const Tensor* qw = a.packed(i++, true);
  const Tensor* kw = a.packed(i++, true);
  const double eps = a.number(i++);
  const int interleaved = PyObject_IsTrue(a.v[i++]);
  if (interleaved < 0) throw Bad("");
  const Tensor* pos = a.index(i++, true);
  const Tensor* status = a.status(i++);
  a.need(q.dim() == 3 && k.dim() == 3 && v.dim() == 3 && tables.dim() == 2,
         "q, key and value are [T, heads, D], block_tables [B, MB]");
  const int64_t T = q.size(0), Hq = q.size(1), D = q.size(2), H = k.size(1);
  const int64_t B = tables.size(0), MB = tables.size(1);
  a.need(out.sizes() == q.sizes() && k.size(0) == T && k.size(2) == D && v.sizes() == k.sizes(),
         "q_out as q [T, Hq, D], key and value [T, Hkv, D]");
  const auto dt = q.scalar_type();
  a.need(out.scalar_type() == dt && k.scalar_type() == dt && v.scalar_type() == dt,
         "q_out, q, key and value share one dtype");
  for (const Tensor* w : {qw, kw})
    a.need(!w || (w->dim() == 1 && w->size(0) == D && w->scalar_type() == dt),
           "norm weights are [head_dim], of q's dtype");
  a.need(!cs || (cs->dim() == 2 && cs->scalar_type() == kFloat),
         "cos_sin is fp32 [max_position, rotary_dim]");
  a.need(lens.numel() == B && (!q_start || q_start->numel() == B + 1) &&
             (!pos || pos->numel() == T),
         "seq_lens [B], q_start [B + 1], positions [T]");
  const int64_t sq = token_stride(a, q), sk = token_stride(a, k);
  a.need(token_stride(a, v) == sk, "key and value need the same token stride");
  int64_t bs;
  if (q8) {
    check_q8(a, kp, vp, *ks, *vs);
    bs = kp.size(2);
    a.need(kp.size(1) == H && kp.size(3) == D, "pools are [NB, Hkv, bs, D]");
  } else {
    a.need(kp.dim() == 4 && vp.sizes() == kp.sizes() && kp.size(2) == H && kp.size(3) == D &&
               kp.scalar_type() == dt && vp.scalar_type() == dt,
           "pools are [NB, bs, Hkv, D] of q's dtype");
    bs = kp.size(1);
  }
  const int P = cs ? (int)cs->size(0) : 0, R = cs ? (int)cs->size(1) : 0;
  a.placed();
  const int code = a.dtype(q);
  const cudaStream_t stream = a.stream(i++);
  if (q8)
    return pa_rope_append_q8(
        ptr(&out), ptr(&kp), ptr(&vp), ptr_as<float>(ks), ptr_as<float>(vs), ptr(&q), ptr(&k),
        ptr(&v), ptr(qw), ptr(kw), (float)eps, ptr_as<float>(cs), P, R, interleaved,
        ptr_as<int32_t>(pos), ptr_as<int32_t>(&tables), ptr_as<int32_t>(&lens),
        ptr_as<int32_t>(q_start), (int)B, (int)T, sq, sk, (int)Hq, (int)H, (int)D, (int)bs,
        (int)MB, (int)kp.size(0), code, ptr_as<int32_t>(status), stream);
  return pa_rope_append(ptr(&out), ptr(&kp), ptr(&vp), ptr(&q), ptr(&k), ptr(&v), ptr(qw), ptr(kw),
                        (float)eps, ptr_as<float>(cs), P, R, interleaved, ptr_as<int32_t>(pos),
                        ptr_as<int32_t>(&tables), ptr_as<int32_t>(&lens),
                        ptr_as<int32_t>(q_start), (int)B, (int)T, sq, sk, (int)Hq, (int)H, (int)D,
                        (int)bs, (int)MB, (int)kp.size(0), code, ptr_as<int32_t>(status), stream);
}

// out, q, k_pool, v_pool, k_scale, v_scale, block_tables, seq_lens, scale, max_seq_len
// (None: the tables' capacity), workspace, status, stream.
long decode_q8(Args a) {
  const Tensor& out = *a.packed(0);
  const Tensor& q = *a.packed(1);
  const Tensor& k = *a.packed(2);
  const Tensor& v = *a.packed(3);
  const Tensor& ks = *a.packed(4);
  const Tensor& vs = *a.packed(5);
  const Tensor& tables = *a.index(6);
  const Tensor& lens = *a.index(7);
  const double scale = a.number(8);
  const Tensor& ws = *a.packed(10);
  const Tensor* status = a.status(11);
  check_q8(a, k, v, ks, vs);
  a.need(q.dim() == 3 && out.sizes() == q.sizes() && out.scalar_type() == q.scalar_type() &&
             q.size(2) == k.size(3) && tables.dim() == 2 && tables.size(0) == q.size(0) &&
             lens.numel() == q.size(0),
         "out as q [B, Hq, D], block_tables [B, MB], seq_lens [B]");
  const int64_t MB = tables.size(1), bs = k.size(2);
  int64_t most = MB * bs;
  if (a.v[9] != Py_None) {
    most = PyLong_AsLongLong(a.v[9]);
    if (PyErr_Occurred()) throw Bad("");
  }
  a.need(most <= 0x7FFFFFFF, "max_seq_len does not fit 32 bits");
  a.placed();
  return pa_decode_q8(ptr(&out), ptr(&q), ptr(&k), ptr(&v), ptr_as<float>(&ks), ptr_as<float>(&vs),
                      ptr_as<int32_t>(&tables), ptr_as<int32_t>(&lens), (int)q.size(0),
                      (int)q.size(1), (int)k.size(1), (int)q.size(2), (int)bs, (int)MB,
                      (int)k.size(0), (int)most, (float)scale, a.dtype(q), ptr(&ws),
                      ws.numel() * ws.element_size(), ptr_as<int32_t>(status), a.stream(12));
}

// k_pool, v_pool, k_pool8, v_pool8, k_scale, v_scale, block_pairs, status, stream.
long expand_q8(Args a) {
  const Tensor& kp = *a.packed(0);
  const Tensor& vp = *a.packed(1);
  const Tensor& k8 = *a.packed(2);
  const Tensor& v8 = *a.packed(3);
  const Tensor& ks = *a.packed(4);
  const Tensor& vs = *a.packed(5);
  const Tensor& pairs = *a.index(6);
  const Tensor* status = a.status(7);
  check_q8(a, k8, v8, ks, vs);
  const int64_t H = k8.size(1), bs = k8.size(2), D = k8.size(3);
  a.need(kp.dim() == 4 && vp.sizes() == kp.sizes() && kp.size(1) == bs && kp.size(2) == H &&
             kp.size(3) == D && kp.scalar_type() == vp.scalar_type(),
         "16-bit pools are [NB', bs, Hkv, D]");
  a.placed();
  a.need(pairs.numel() == 0 || (pairs.dim() == 2 && pairs.size(1) == 2), "block_pairs is [n, 2]");
  const int64_t n = pairs.numel() / 2;
  return pa_expand_blocks_q8(ptr(&kp), ptr(&vp), ptr(&k8), ptr(&v8), ptr_as<float>(&ks),
                             ptr_as<float>(&vs), n ? ptr_as<int32_t>(&pairs) : nullptr, (int)n,
                             (int)H, (int)D, (int)bs, (int)k8.size(0), (int)kp.size(0),
                             a.dtype(kp), ptr_as<int32_t>(status), a.stream(8));
}

template <typename F>
PyObject* call(const char* where, PyObject* const* v, Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s: %zd arguments, %zd wanted", where, n, want);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f(Args{where, v}));
  } catch (const Bad& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* py_rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call("pa_rope_append", v, n, 17, [](Args a) { return rope(a, false); });
}
PyObject* py_rope_q8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call("pa_rope_append_q8", v, n, 19, [](Args a) { return rope(a, true); });
}
PyObject* py_decode_q8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call("pa_decode_q8", v, n, 13, decode_q8);
}
PyObject* py_expand_q8(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return call("pa_expand_blocks_q8", v, n, 9, expand_q8);
}

PyMethodDef kMethods[] = {
    {"rope_append", (PyCFunction)(void (*)(void))py_rope, METH_FASTCALL, nullptr},
    {"rope_append_q8", (PyCFunction)(void (*)(void))py_rope_q8, METH_FASTCALL, nullptr},
    {"decode_q8", (PyCFunction)(void (*)(void))py_decode_q8, METH_FASTCALL, nullptr},
    {"expand_blocks_q8", (PyCFunction)(void (*)(void))py_expand_q8, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
