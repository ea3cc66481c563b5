// Python side of the calls whose kernels take a few microseconds (QK-norm with
// RoPE, shared-prefix attention, policy loss): checks torch tensors and hands
// their addresses and strides to libnc.so (include/nc.h).  The same checks in
// Python take 7 to 10 us per call, here less than one.  nc.py holds the
// functions that users call; every error is an nc.NcError.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/nc.h"

namespace {

PyObject* g_error = nullptr;  // nc.NcError

struct Refused {
  std::string why;
};

std::string list_of(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + (v[i] < 0 ? std::string("any") : std::to_string(v[i]));
  return s + ")";
}

// The operands of one call, which must all be on the current CUDA device: the
// call runs there, on one of its streams.
struct Operands {
  const char* what;
  int device = -1;

  explicit Operands(const char* w) : what(w) {}

  [[noreturn]] void refuse(const std::string& why) const { throw Refused{std::string(what) + ": " + why}; }

  const at::Tensor& tensor(PyObject* o, const char* name) const {
    if (!THPVariable_Check(o)) refuse(std::string(name) + (o == Py_None ? " is missing" : " is not a tensor"));
    return THPVariable_Unpack(o);
  }

  // A tensor of this type and shape (-1: any size), strided, its dimensions
  // from `packed` on without gaps.
  const at::Tensor& take(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int packed) {
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != type)
      refuse(std::string(name) + " is " + c10::toString(t.scalar_type()) + ", expected " + c10::toString(type));
    bool same = t.dim() == (int64_t)shape.size();
    for (int64_t i = 0; same && i < t.dim(); ++i) same = shape[i] < 0 || t.size(i) == shape[i];
    if (!same) refuse(std::string(name) + " has shape " + list_of(t.sizes()) + ", expected " + list_of(shape));
    if (!t.is_cuda() || t.layout() != at::kStrided) refuse(std::string(name) + " is not a strided tensor on a CUDA device");
    if (device < 0) {
      c10::DeviceIndex now = -1;
      if (c10::cuda::GetDevice(&now) != cudaSuccess) refuse("no current CUDA device");
      device = now;
    }
    if (t.get_device() != device)
      refuse(std::string(name) + " is on cuda:" + std::to_string(t.get_device()) + ", the current device is cuda:" +
             std::to_string(device));
    int64_t want = 1;
    for (int64_t i = t.dim() - 1; i >= packed; --i) {
      if (t.size(i) > 1 && t.stride(i) != want)
        refuse(std::string(name) + " has strides " + list_of(t.strides()) + ": its dimensions from " +
               std::to_string(packed) + " on must have no gaps");
      want *= t.size(i);
    }
    return t;
  }

  // the address, or null for None
  template <typename T>
  T* optional(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    return o == Py_None ? nullptr : static_cast<T*>(take(o, name, type, shape, 0).data_ptr());
  }
  template <typename T>
  T* dense(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
    return static_cast<T*>(take(o, name, type, shape, 0).data_ptr());
  }

  at::ScalarType act_type(const at::Tensor& t) const {
    if (t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kFloat)
      refuse(std::string(c10::toString(t.scalar_type())) + " is not supported (bfloat16 or float32)");
    return t.scalar_type();
  }
};

// stride between rows of t [outer, inner, ...], which must be evenly spaced
int64_t even_rows(const Operands& op, const char* name, const at::Tensor& t, int64_t width) {
  const int64_t outer = t.size(0), inner = t.size(1);
  const int64_t ld = inner > 1 ? t.stride(1) : (outer > 1 ? t.stride(0) : width);
  if (outer > 1 && inner > 1 && t.stride(0) != inner * ld)
    op.refuse(std::string(name) + "'s rows must be evenly spaced (strides " + list_of(t.strides()) + ")");
  return ld;
}

int as_int(const Operands& op, int64_t v, const char* name) {
  if (v < 0 || v > 0x7fffffff) op.refuse(std::string(name) + " is out of range");
  return (int)v;
}

float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{""};
  return (float)v;
}

int as_index(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{""};
  if (v < -0x7fffffffL || v > 0x7fffffffL) throw Refused{"an integer argument is out of range"};
  return (int)v;
}

// The call's stream (a torch.cuda.Stream, or None for the current one) and its
// scratch: the caller's tensor, or a new one.  The new one comes from the call's
// stream's own pool: a block of the current stream's may have been freed while
// that stream still has work queued on it, which the call's stream does not wait
// for.
struct Launch {
  void* stream;
  void* workspace = nullptr;
  size_t bytes = 0;
  at::Tensor own;

  Launch(const Operands& op, PyObject* stream_obj) {
    if (stream_obj == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)op.device).stream();
      return;
    }
    PyObject* h = PyObject_GetAttrString(stream_obj, "cuda_stream");
    if (h == nullptr) throw Refused{""};
    stream = PyLong_AsVoidPtr(h);
    Py_DECREF(h);
    if (PyErr_Occurred()) throw Refused{""};
  }

  void scratch(const Operands& op, PyObject* o, size_t need) {
    if (o == Py_None) {
      if (need == 0) return;
      const c10::cuda::CUDAStreamGuard on(
          c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), (c10::DeviceIndex)op.device));
      own = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)op.device));
      workspace = own.data_ptr();
      bytes = need;
      return;
    }
    const at::Tensor& t = op.tensor(o, "workspace");
    if (!t.is_cuda() || t.get_device() != op.device || !t.is_contiguous())
      op.refuse("workspace: a contiguous tensor on the operands' device is needed");
    workspace = t.data_ptr();
    bytes = t.nbytes();
  }
};

PyObject* done(const char* what, int rc) {
  if (rc == NC_OK) Py_RETURN_NONE;
  static const char* names[] = {"NC_OK",       "NC_ERR_ARG",  "NC_ERR_SHAPE",   "NC_ERR_ALIGN",
                                "NC_ERR_CUDA", "NC_ERR_DATA", "NC_ERR_TIMEOUT", "NC_ERR_WORKSPACE"};
  PyErr_Format(g_error, "%s: %s (%s) %s", what, rc > 0 && rc < 8 ? names[rc] : "?", nc_status_string(rc), nc_last_error());
  return nullptr;
}

// Runs `call` and turns what it throws into a Python exception.
template <typename F>
PyObject* guarded(const char* what, Py_ssize_t n, Py_ssize_t want, F call) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, got %zd", what, want, n);
    return nullptr;
  }
  try {
    return done(what, call());
  } catch (const Refused& r) {
    if (!PyErr_Occurred()) PyErr_SetString(g_error, r.why.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(g_error, (std::string(what) + ": " + e.what()).c_str());
  } catch (...) {
    PyErr_SetString(g_error, what);
  }
  return nullptr;
}

// libnc's call itself runs without the interpreter's lock, as under ctypes
template <typename F>
int unlocked(F f) {
  int rc;
  Py_BEGIN_ALLOW_THREADS rc = f();
  Py_END_ALLOW_THREADS return rc;
}

struct Rows {
  void* p = nullptr;
  int64_t ld = 0;
};
// [rows, heads, D], heads and D without gaps
Rows rows_of(Operands& op, PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape) {
  const at::Tensor& t = op.take(o, name, type, shape, 1);
  return {t.data_ptr(), shape[0] > 1 ? t.stride(0) : shape[1] * shape[2]};
}

int dtype_of(at::ScalarType t) { return t == at::kBFloat16 ? NC_BF16 : NC_FP32; }

// q, k, positions, q_out, k_out, v, v_out, slots, alpha, rope_base, reverse, eps, stream
PyObject* qk_norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* what = "nc_qk_norm_rope";
  return guarded(what, n, 13, [&]() -> int {
    Operands op(what);
    const at::Tensor &q = op.tensor(a[0], "q"), &k = op.tensor(a[1], "k"), &ko = op.tensor(a[4], "k_out");
    if (q.dim() != 3 || k.dim() != 3 || ko.dim() != 3) op.refuse("q, k and k_out are [rows, heads, D]");
    const at::ScalarType ty = op.act_type(q);
    const int64_t N = q.size(0), H = q.size(1), D = q.size(2), Hkv = k.size(1), rows = ko.size(0);
    if ((a[5] == Py_None) != (a[6] == Py_None)) op.refuse("v and v_out come together");
    const Rows rq = rows_of(op, a[0], "q", ty, {N, H, D}), rk = rows_of(op, a[1], "k", ty, {N, Hkv, D});
    const Rows ro = rows_of(op, a[3], "q_out", ty, {N, H, D}), rc = rows_of(op, a[4], "k_out", ty, {rows, Hkv, D});
    Rows rv, rd;
    if (a[5] != Py_None) {
      rv = rows_of(op, a[5], "v", ty, {N, Hkv, D});
      rd = rows_of(op, a[6], "v_out", ty, {rows, Hkv, D});
    }
    const int32_t* pos = op.dense<int32_t>(a[2], "positions", at::kInt, {N});
    const int32_t* slots = op.optional<int32_t>(a[7], "slots", at::kInt, {N});
    const float alpha = as_float(a[8]), base = as_float(a[9]), eps = as_float(a[11]);
    const int reverse = as_index(a[10]);
    if (N == 0) return NC_OK;
    const Launch l(op, a[12]);
    const int n32 = as_int(op, N, "N"), h = as_int(op, H, "H"), hkv = as_int(op, Hkv, "H_kv"), d = as_int(op, D, "D");
    return unlocked([&] {
      return nc_qk_norm_rope(rq.p, rq.ld, rk.p, rk.ld, rv.p, rv.ld, pos, slots, n32, h, hkv, d, ro.p, ro.ld, rc.p, rc.ld,
                             rd.p, rd.ld, rows, alpha, base, reverse, eps, dtype_of(ty), l.stream);
    });
  });
}

// q, k, positions, dq_hat, dk_hat, out_dq, out_dk, alpha, rope_base, reverse, eps, stream
PyObject* qk_norm_rope_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* what = "nc_qk_norm_rope_backward";
  return guarded(what, n, 12, [&]() -> int {
    Operands op(what);
    const at::Tensor &q = op.tensor(a[0], "q"), &k = op.tensor(a[1], "k");
    if (q.dim() != 3 || k.dim() != 3) op.refuse("q and k are [N, heads, D]");
    const at::ScalarType ty = op.act_type(q);
    const int64_t N = q.size(0), H = q.size(1), D = q.size(2), Hkv = k.size(1);
    const Rows rq = rows_of(op, a[0], "q", ty, {N, H, D}), rk = rows_of(op, a[1], "k", ty, {N, Hkv, D});
    const Rows gq = rows_of(op, a[3], "dq_hat", ty, {N, H, D}), gk = rows_of(op, a[4], "dk_hat", ty, {N, Hkv, D});
    const Rows dq = rows_of(op, a[5], "out_dq", ty, {N, H, D}), dk = rows_of(op, a[6], "out_dk", ty, {N, Hkv, D});
    const int32_t* pos = op.dense<int32_t>(a[2], "positions", at::kInt, {N});
    const float alpha = as_float(a[7]), base = as_float(a[8]), eps = as_float(a[10]);
    const int reverse = as_index(a[9]);
    if (N == 0) return NC_OK;
    const Launch l(op, a[11]);
    const int n32 = as_int(op, N, "N"), h = as_int(op, H, "H"), hkv = as_int(op, Hkv, "H_kv"), d = as_int(op, D, "D");
    return unlocked([&] {
      return nc_qk_norm_rope_backward(rq.p, rq.ld, rk.p, rk.ld, pos, gq.p, gq.ld, gk.p, gk.ld, n32, h, hkv, d, dq.p, dq.ld,
                                      dk.p, dk.ld, alpha, base, reverse, eps, dtype_of(ty), l.stream);
    });
  });
}

// one side's caches [sequences, keys, H_kv, D] and lengths
struct Side {
  const void *k = nullptr, *v = nullptr;
  const int32_t* lens = nullptr;
  int64_t ld = 0, ls = 0, seqs = 1, cap = 0, heads = -1;
};
Side side_of(Operands& op, const char* side, PyObject* k, PyObject* v, PyObject* lens, int64_t seqs, int64_t D) {
  Side s;
  if ((k == Py_None) != (v == Py_None) || (k == Py_None) != (lens == Py_None))
    op.refuse(std::string("k, v and lengths of the ") + side + " come together");
  if (k == Py_None) return s;
  const std::string of = side, nk = "k_" + of, nv = "v_" + of, nl = of + "_lens";
  const at::Tensor &tk = op.take(k, nk.c_str(), at::kBFloat16, {seqs, -1, -1, D}, 2),
                   &tv = op.take(v, nv.c_str(), at::kBFloat16, tk.sizes(), 2);
  s.seqs = tk.size(0), s.cap = tk.size(1), s.heads = tk.size(2);
  s.lens = op.dense<int32_t>(lens, nl.c_str(), at::kInt, {s.seqs});
  if ((s.cap > 1 && tk.stride(1) != tv.stride(1)) || (s.seqs > 1 && tk.stride(0) != tv.stride(0)))
    op.refuse(nk + " and " + nv + " must have the same strides");
  s.k = tk.data_ptr(), s.v = tv.data_ptr();
  s.ld = s.cap > 1 ? tk.stride(1) : s.heads * D;
  s.ls = s.seqs > 1 ? tk.stride(0) : s.ld * s.cap;
  return s;
}

// q, k_prefix, v_prefix, prefix_lens, k_suffix, v_suffix, suffix_lens, out, out_lse, window, scale, workspace, stream
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* what = "nc_prefix_attention";
  return guarded(what, n, 13, [&]() -> int {
    Operands op(what);
    if (op.tensor(a[0], "q").dim() != 4) op.refuse("q is [B, Tq, H, D]");
    const at::Tensor& q = op.take(a[0], "q", at::kBFloat16, {-1, -1, -1, -1}, 2);
    const int64_t B = q.size(0), Tq = q.size(1), H = q.size(2), D = q.size(3);
    const Side p = side_of(op, "prefix", a[1], a[2], a[3], -1, D), s = side_of(op, "suffix", a[4], a[5], a[6], B, D);
    if (p.heads < 0 && s.heads < 0) op.refuse("there are no keys");
    if (p.heads >= 0 && s.heads >= 0 && p.heads != s.heads) op.refuse("prefix and suffix differ in key heads");
    void* out = op.dense<void>(a[7], "out", at::kBFloat16, q.sizes());
    float* lse = op.optional<float>(a[8], "out_lse", at::kFloat, {B, Tq, H});
    const int64_t ldq = even_rows(op, "q", q, H * D);
    const int window = as_index(a[9]);
    const float scale = a[10] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : as_float(a[10]);
    const int b = as_int(op, B, "B"), g = as_int(op, p.seqs, "G"), tq = as_int(op, Tq, "Tq"), h = as_int(op, H, "H"),
              hkv = as_int(op, p.heads < 0 ? s.heads : p.heads, "H_kv"), d = as_int(op, D, "D"),
              pm = as_int(op, p.cap, "P_max"), sm = as_int(op, s.cap, "S_max");
    Launch l(op, a[12]);
    l.scratch(op, a[11], nc_prefix_attention_workspace_bytes(b, g, tq, h, hkv, pm, sm, window));
    return unlocked([&] {
      return nc_prefix_attention(q.data_ptr(), ldq, p.k, p.v, p.ld, p.ls, p.lens, s.k, s.v, s.ld, s.ls, s.lens, out, lse, b, g,
                                 tq, h, hkv, d, pm, sm, window, scale, l.workspace, l.bytes, l.stream);
    });
  });
}

// logits, targets, advantages, out_stats, out_logp, out_dlogits, old_logp, ref_logp, clip_low, clip_high, kl_beta,
// norm, workspace, stream
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const char* what = "nc_policy_loss";
  return guarded(what, n, 14, [&]() -> int {
    Operands op(what);
    if (op.tensor(a[0], "logits").dim() != 3) op.refuse("logits are [B, T, V]");
    const at::ScalarType ty = op.act_type(op.tensor(a[0], "logits"));
    const at::Tensor& z = op.take(a[0], "logits", ty, {-1, -1, -1}, 2);
    const int64_t B = z.size(0), T = z.size(1), V = z.size(2);
    const int32_t* y = op.dense<int32_t>(a[1], "targets", at::kInt, {B, T});
    const bool per_token = op.tensor(a[2], "advantages").dim() == 2;
    const int64_t bt[2] = {B, T};
    const float* adv = op.dense<float>(a[2], "advantages", at::kFloat, at::IntArrayRef(bt, per_token ? 2 : 1));
    float *stats = op.dense<float>(a[3], "out_stats", at::kFloat, {3}), *logp = op.dense<float>(a[4], "out_logp", at::kFloat, bt);
    void* dz = nullptr;
    int64_t lddl = 0;
    if (a[5] != Py_None) {
      const at::Tensor& t = op.take(a[5], "out_dlogits", ty, z.sizes(), 2);
      dz = t.data_ptr();
      lddl = even_rows(op, "out_dlogits", t, V);
    }
    const float* old = op.optional<float>(a[6], "old_logp", at::kFloat, bt);
    const float* ref = op.optional<float>(a[7], "ref_logp", at::kFloat, bt);
    const int64_t ldl = even_rows(op, "logits", z, V);
    const float low = as_float(a[8]), high = as_float(a[9]), beta = as_float(a[10]);
    const int norm = as_index(a[11]), b = as_int(op, B, "B"), t = as_int(op, T, "T"), v = as_int(op, V, "V");
    Launch l(op, a[13]);
    l.scratch(op, a[12], nc_policy_loss_workspace_bytes());
    return unlocked([&] {
      return nc_policy_loss(z.data_ptr(), ldl, y, adv, per_token, old, ref, b, t, v, low, high, beta, norm, stats, logp, dz,
                            lddl, dtype_of(ty), l.workspace, l.bytes, l.stream);
    });
  });
}

// the exception class that errors are raised as
PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef g_methods[] = {{"set_error", set_error, METH_O, nullptr},
                           {"qk_norm_rope", fast(qk_norm_rope), METH_FASTCALL, nullptr},
                           {"qk_norm_rope_backward", fast(qk_norm_rope_backward), METH_FASTCALL, nullptr},
                           {"prefix_attention", fast(prefix_attention), METH_FASTCALL, nullptr},
                           {"policy_loss", fast(policy_loss), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ncpy", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__ncpy() { return PyModule_Create(&g_module); }
