// Tensor marshalling of the norm + rotation and chunk attention calls for
// binding.py: checks shapes, types, devices and layouts, makes the outputs that
// the caller did not give, and passes pointers and the current stream to the C
// ABI (include/parallax.h). A decode step makes these calls once per layer, with
// 16 tensors each; in Python the checks and the ctypes conversion take 20 us, the
// kernels 3. Errors: ValueError for a bad argument, RuntimeError for a status.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/core/grad_mode.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <stdexcept>
#include <string>

#include "internal.h"
#include "parallax.h"

namespace {

using at::Tensor;

[[noreturn]] void bad(const std::string& what) { throw std::invalid_argument(what); }

const Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) bad(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = tensor_or_none(o, name);
  if (!t) bad(std::string(name) + " must be a tensor, not None");
  return *t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    bad("expected a number");
  }
  return v;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad("expected an integer");
  }
  return v;
}
int to_int(int64_t v, const char* name) {
  if (v < 0 || v > 0x7fffffff) bad(std::string(name) + " is out of range");
  return (int)v;
}

int dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return PARALLAX_DTYPE_BF16;
  if (t.scalar_type() == at::kFloat) return PARALLAX_DTYPE_F32;
  bad("q, r, k must be bf16 or fp32");
}

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// The call's first tensor: its device and type are everyone's.
struct Call {
  const Tensor& q;
  c10::cuda::OptionalCUDAGuard guard;
  explicit Call(const Tensor& q_) : q(q_) {
    if (!q.is_cuda()) bad("expected CUDA tensors");
    guard.set_index(q.get_device());
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream(q.get_device()).stream(); }

  void dense(const Tensor& t, const char* name, at::IntArrayRef shape, at::ScalarType type) const {
    if (t.sizes() != shape || t.scalar_type() != type || t.get_device() != q.get_device() ||
        !t.is_contiguous()) {
      std::string s = std::string(name) + " must be a contiguous " + at::toString(type) + " tensor [";
      for (size_t i = 0; i < shape.size(); ++i) s += (i ? ", " : "") + std::to_string(shape[i]);
      bad(s + "] on q's device");
    }
  }
  // Token rows [tokens, H, D] whose heads are contiguous: their token stride.
  long long rows(const Tensor& t, const char* name, int64_t heads = -1) const {
    if (t.dim() != 3 || t.scalar_type() != q.scalar_type() || t.get_device() != q.get_device() ||
        t.size(0) != q.size(0) || t.size(2) != q.size(2) || (heads >= 0 && t.size(1) != heads))
      bad(std::string(name) + " must be [tokens, H, D], matching q in tokens, D, type and device");
    const int64_t H = t.size(1), D = t.size(2);
    if (t.stride(2) != 1 || (H > 1 && t.stride(1) != D))
      bad(std::string(name) + ": the heads of a token must be contiguous");
    return t.size(0) > 1 ? t.stride(0) : H * D;
  }
  void* weight(PyObject* o, const char* name) const {
    const Tensor* w = tensor_or_none(o, name);
    if (w) dense(*w, name, {q.size(2)}, q.scalar_type());
    return ptr(w);
  }
  const int32_t* ints(PyObject* o, const char* name, at::IntArrayRef shape) const {
    const Tensor* t = tensor_or_none(o, name);
    if (t) dense(*t, name, shape, at::kInt);
    return static_cast<const int32_t*>(ptr(t));
  }
  // A new tensor on q's device, from the allocator without the dispatcher (a call
  // makes up to seven, 0.25 us less each).
  Tensor fresh(at::IntArrayRef shape, at::ScalarType type) const {
    return Tensor(at::detail::empty_cuda(shape, type, q.device(), std::nullopt));
  }
  Tensor output(PyObject* o, const char* name, at::IntArrayRef shape) const {
    const Tensor* t = tensor_or_none(o, name);
    if (!t) return fresh(shape, q.scalar_type());
    dense(*t, name, shape, q.scalar_type());
    return *t;
  }
  // The caller's workspace, or one of `bytes` bytes with a zeroed status header.
  Tensor workspace(PyObject* o, size_t bytes) const {
    if (const Tensor* t = tensor_or_none(o, "workspace")) {
      if (t->scalar_type() != at::kByte || t->get_device() != q.get_device() || !t->is_contiguous())
        bad("workspace must be a contiguous uint8 tensor on q's device");
      return *t;
    }
    if (bytes == 0) bad("invalid arguments for a workspace size");
    Tensor t = fresh({(int64_t)bytes}, at::kByte);
    t.narrow(0, 0, 256).zero_();
    return t;
  }
};

struct Status : std::runtime_error {
  using std::runtime_error::runtime_error;
};
void check(int status, const char* what) {
  if (status != PARALLAX_OK)
    throw Status(std::string(what) + " failed: " + parallax_status_string(status) + " (status " +
                 std::to_string(status) + ")");
}

// What the norm and rotation calls share.
struct Rope {
  Call c;
  const Tensor *r, &k, &cs;
  int n, Hq, Hkv, D, rot, max_pos, dtype, L;
  long long sq, sr, sk;
  const int32_t* pos;
  void *qw, *rw, *kw;
  Rope(PyObject* q_, PyObject* r_, PyObject* k_, PyObject* cs_, PyObject* pos_, PyObject* const* w,
       long long seq_len)
      : c(tensor(q_, "q")),
        r(tensor_or_none(r_, "r")),
        k(tensor(k_, "k")),
        cs(tensor(cs_, "cos_sin")) {
    const Tensor& q = c.q;
    dtype = dtype_code(q);
    sq = c.rows(q, "q");
    sr = r ? c.rows(*r, "r", q.size(1)) : 0;
    sk = c.rows(k, "k");
    if (cs.dim() != 2) bad("cos_sin must be [max_positions, rotary_dim]");
    c.dense(cs, "cos_sin", cs.sizes(), at::kFloat);
    n = to_int(q.size(0), "tokens");
    Hq = to_int(q.size(1), "Hq");
    Hkv = to_int(k.size(1), "Hkv");
    D = to_int(q.size(2), "D");
    rot = to_int(cs.size(1), "rotary_dim");
    max_pos = to_int(cs.size(0), "max_positions");
    pos = c.ints(pos_, "positions", {n});
    qw = c.weight(w[0], "q_weight");
    rw = r ? c.weight(w[1], "r_weight") : nullptr;
    kw = c.weight(w[2], "k_weight");
    L = to_int(seq_len, "seq_len");
    if (L > 0 && n % L != 0) bad("tokens must be a multiple of seq_len");
  }
  // [tokens, H, D], or [tokens / L, H, L, D]
  c10::SmallVector<int64_t, 4> shape(int H) const {
    if (L == 0) return {n, H, D};
    return {n / L, H, L, D};
  }
};

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* none() { Py_RETURN_NONE; }
PyObject* tuple(std::initializer_list<PyObject*> xs) {
  PyObject* t = PyTuple_New((Py_ssize_t)xs.size());
  Py_ssize_t i = 0;
  for (PyObject* x : xs) PyTuple_SET_ITEM(t, i++, x);
  return t;
}

// out: None, or a tuple or list of three
struct Out3 {
  PyObject* at[3];
  explicit Out3(PyObject* o) : at{Py_None, Py_None, Py_None} {
    if (o == Py_None) return;
    if (!(PyTuple_Check(o) || PyList_Check(o)) || PySequence_Size(o) != 3)
      bad("out must be three tensors");
    for (int i = 0; i < 3; ++i)
      at[i] = PyTuple_Check(o) ? PyTuple_GET_ITEM(o, i) : PyList_GET_ITEM(o, i);
  }
};

// Whether autograd has to follow a call on these arguments.
bool wants_grad(std::initializer_list<PyObject*> xs) {
  if (!at::GradMode::is_enabled()) return false;
  for (PyObject* o : xs)
    if (THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad()) return true;
  return false;
}

// q, r, k, cos_sin, positions, 3 weights, eps, interleaved, seq_len, out, workspace;
// returns None, and does nothing, where autograd has to follow the call.
PyObject* qk_norm_rope(PyObject* const* a) {
  if (wants_grad({a[0], a[1], a[2], a[3], a[5], a[6], a[7]})) return none();
  Rope x(a[0], a[1], a[2], a[3], a[4], a + 5, integer(a[10]));
  const Out3 out(a[11]);
  const auto sq = x.shape(x.Hq), sk = x.shape(x.Hkv);
  const Tensor qo = x.c.output(out.at[0], "out[0]", sq);
  const Tensor ro = x.r ? x.c.output(out.at[1], "out[1]", sq) : Tensor();
  const Tensor ko = x.c.output(out.at[2], "out[2]", sk);
  const Tensor ws = x.c.workspace(a[12], 256);
  check(parallax_qk_norm_rope(
            x.c.q.data_ptr(), ptr(x.r), x.k.data_ptr(), x.qw, x.rw, x.kw,
            static_cast<const float*>(x.cs.data_ptr()), x.pos, qo.data_ptr(),
            x.r ? ro.data_ptr() : nullptr, ko.data_ptr(), x.n, x.Hq, x.Hkv, x.D, x.rot,
            integer(a[9]) != 0, x.max_pos, (float)number(a[8]), x.sq, x.sr, x.sk, x.L, x.dtype,
            x.c.stream(), ws.data_ptr(), (size_t)ws.numel()),
        "parallax_qk_norm_rope");
  return tuple({wrap(qo), x.r ? wrap(ro) : none(), wrap(ko)});
}

// dq_out, dr_out, dk_out, then as qk_norm_rope
PyObject* qk_norm_rope_backward(PyObject* const* a) {
  PyObject* const* b = a + 3;
  Rope x(b[0], b[1], b[2], b[3], b[4], b + 5, integer(b[10]));
  const auto sq = x.shape(x.Hq), sk = x.shape(x.Hkv);
  const auto type = x.c.q.scalar_type();
  const Tensor &gq = tensor(a[0], "dq_out"), &gk = tensor(a[2], "dk_out");
  const Tensor* gr = x.r ? &tensor(a[1], "dr_out") : nullptr;
  x.c.dense(gq, "dq_out", sq, type);
  x.c.dense(gk, "dk_out", sk, type);
  if (gr) x.c.dense(*gr, "dr_out", sq, type);
  const Out3 out(b[11]);
  const auto grad = [&](PyObject* o, const char* name, int H) {
    const Tensor* t = tensor_or_none(o, name);
    return t ? *t : x.c.fresh({x.n, H, x.D}, type);
  };
  const Tensor dq = grad(out.at[0], "out[0]", x.Hq), dk = grad(out.at[2], "out[2]", x.Hkv);
  const Tensor dr = x.r ? grad(out.at[1], "out[1]", x.Hq) : Tensor();
  const long long tq = x.c.rows(dq, "out[0]", x.Hq), tk = x.c.rows(dk, "out[2]", x.Hkv);
  const long long tr = x.r ? x.c.rows(dr, "out[1]", x.Hq) : 0;
  const auto dweight = [&](void* w) {
    return w ? x.c.fresh({x.D}, at::kFloat) : Tensor();
  };
  const Tensor dqw = dweight(x.qw), drw = dweight(x.rw), dkw = dweight(x.kw);
  const auto fp = [](const Tensor& t) {
    return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr;
  };
  const Tensor ws =
      x.c.workspace(b[12], b[12] == Py_None ? parallax_qk_norm_rope_backward_workspace_bytes(
                                                  x.n, x.Hq, x.Hkv, x.D)
                                            : 0);
  check(parallax_qk_norm_rope_backward(
            gq.data_ptr(), ptr(gr), gk.data_ptr(), x.c.q.data_ptr(), ptr(x.r), x.k.data_ptr(), x.qw,
            x.rw, x.kw, static_cast<const float*>(x.cs.data_ptr()), x.pos, dq.data_ptr(),
            x.r ? dr.data_ptr() : nullptr, dk.data_ptr(), fp(dqw), fp(drw), fp(dkw), x.n, x.Hq,
            x.Hkv, x.D, x.rot, integer(b[9]) != 0, x.max_pos, (float)number(b[8]), x.sq, x.sr, x.sk,
            tq, tr, tk, x.L, x.dtype, x.c.stream(), ws.data_ptr(), (size_t)ws.numel()),
        "parallax_qk_norm_rope_backward");
  const auto opt = [](const Tensor& t) { return t.defined() ? wrap(t) : none(); };
  return tuple({wrap(dq), opt(dr), wrap(dk), opt(dqw), opt(drw), opt(dkw)});
}

// The pools [pages, page_size, Hkv, D] and the table [B, max_pages].
struct Pool {
  const Tensor &k, &v, &table;
  Pool(const Call& c, PyObject* k_, PyObject* v_, PyObject* t_, int64_t B, int64_t Hkv)
      : k(tensor(k_, "k_pages")), v(tensor(v_, "v_pages")), table(tensor(t_, "block_table")) {
    if (k.dim() != 4 || k.size(2) != Hkv || k.size(3) != c.q.size(2))
      bad("k_pages must be [num_pages, page_size, Hkv, D]");
    c.dense(k, "k_pages", k.sizes(), c.q.scalar_type());
    c.dense(v, "v_pages", k.sizes(), c.q.scalar_type());
    if (table.dim() != 2 || table.size(0) != B) bad("block_table must be [B, max_pages_per_seq]");
    c.dense(table, "block_table", table.sizes(), at::kInt);
  }
  int pages() const { return to_int(k.size(0), "num_pages"); }
  int page_size() const { return to_int(k.size(1), "page_size"); }
  int max_pages() const { return to_int(table.size(1), "max_pages_per_seq"); }
  const int32_t* ids() const { return static_cast<const int32_t*>(table.data_ptr()); }
};

// The batch of cache_seqlens, and cu_seqlens_q [B + 1] or None.
struct Lengths {
  int B;
  const int32_t *lens, *cu;
  Lengths(const Call& c, PyObject* lens_, PyObject* cu_) {
    const Tensor& t = tensor(lens_, "cache_seqlens");
    B = to_int(t.numel(), "B");
    c.dense(t, "cache_seqlens", {B}, at::kInt);
    lens = static_cast<const int32_t*>(t.data_ptr());
    cu = c.ints(cu_, "cu_seqlens_q", {B + 1});
  }
};

// q, r, k, v, cos_sin, k_pages, v_pages, block_table, cache_seqlens,
// cu_seqlens_q, positions, 3 weights, eps, interleaved, q_out, r_out, workspace
PyObject* norm_rope_append(PyObject* const* a) {
  Rope x(a[0], a[1], a[2], a[4], a[10], a + 11, 0);
  const Tensor& v = tensor(a[3], "v");
  const long long sv = x.c.rows(v, "v", x.Hkv);
  const Lengths len(x.c, a[8], a[9]);
  const Pool pool(x.c, a[5], a[6], a[7], len.B, x.Hkv);
  const Tensor qo = x.c.output(a[16], "q_out", {x.n, x.Hq, x.D});
  const Tensor ro = x.r ? x.c.output(a[17], "r_out", {x.n, x.Hq, x.D}) : Tensor();
  // rows without a token: zeros in an output made here, untouched in a given one
  const int clear = (a[16] == Py_None ? 1 : 0) | (x.r && a[17] == Py_None ? 2 : 0);
  const Tensor ws = x.c.workspace(a[18], 256);
  check(parallax_internal_norm_rope_append(
            x.c.q.data_ptr(), ptr(x.r), x.k.data_ptr(), v.data_ptr(), x.qw, x.rw, x.kw,
            static_cast<const float*>(x.cs.data_ptr()), x.pos, len.cu, len.lens, pool.ids(),
            qo.data_ptr(), x.r ? ro.data_ptr() : nullptr, pool.k.data_ptr(), pool.v.data_ptr(),
            len.B, x.n, x.Hq, x.Hkv, x.D, x.rot, integer(a[15]) != 0, x.max_pos,
            (float)number(a[14]), x.sq, x.sr, x.sk, sv, pool.pages(), pool.page_size(),
            pool.max_pages(), x.dtype, x.c.stream(), ws.data_ptr(), (size_t)ws.numel(), clear),
        "parallax_norm_rope_append");
  return tuple({wrap(qo), x.r ? wrap(ro) : none()});
}

// q, r, k_pages, v_pages, block_table, cache_seqlens, cu_seqlens_q, scale,
// causal, probe, out, workspace
PyObject* prefill_paged(PyObject* const* a) {
  const Call c(tensor(a[0], "q"));
  if (c.q.dim() != 3 || c.q.scalar_type() != at::kBFloat16) bad("q must be [tokens, Hq, D] bf16");
  c.dense(c.q, "q", c.q.sizes(), at::kBFloat16);
  const bool probe = integer(a[9]) != 0;
  const Tensor* r = probe ? &tensor(a[1], "r") : nullptr;
  if (r) c.dense(*r, "r", c.q.sizes(), at::kBFloat16);
  const int n = to_int(c.q.size(0), "tokens"), Hq = to_int(c.q.size(1), "Hq"),
            D = to_int(c.q.size(2), "D");
  const Tensor& kp = tensor(a[2], "k_pages");
  if (kp.dim() != 4) bad("k_pages must be [num_pages, page_size, Hkv, D]");
  const int Hkv = to_int(kp.size(2), "Hkv");
  const Lengths len(c, a[5], a[6]);
  const Pool pool(c, a[2], a[3], a[4], len.B, Hkv);
  Tensor out;
  if (a[10] == Py_None && len.cu)  // rows past the last sequence are not written
    out = c.fresh(c.q.sizes(), at::kBFloat16).zero_();
  else
    out = c.output(a[10], "out", c.q.sizes());
  const Tensor ws = c.workspace(
      a[11], a[11] == Py_None ? parallax_prefill_paged_workspace_bytes(len.B, n, Hq, Hkv, D) : 0);
  const float scale = a[7] == Py_None ? 1.f / std::sqrt((float)D) : (float)number(a[7]);
  check(parallax_prefill_paged(c.q.data_ptr(), ptr(r), pool.k.data_ptr(), pool.v.data_ptr(),
                               pool.ids(), len.cu, len.lens, out.data_ptr(), len.B, n, Hq, Hkv, D,
                               scale, integer(a[8]) != 0, c.stream(), pool.pages(),
                               pool.page_size(), pool.max_pages(), probe ? 1 : 0, ws.data_ptr(),
                               (size_t)ws.numel()),
        "parallax_prefill_paged");
  return wrap(out);
}

template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  if (nargs != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define PLX_METHOD(name, n) \
  { #name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr }
PyMethodDef methods[] = {PLX_METHOD(qk_norm_rope, 13), PLX_METHOD(qk_norm_rope_backward, 16),
                         PLX_METHOD(norm_rope_append, 19), PLX_METHOD(prefill_paged, 12),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

// build.py looks for this text in the built module, binding.py asks for the version.
constexpr char kBuiltFor[] = "built for torch " PLX_TORCH_VERSION;

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "built_for", kBuiltFor) != 0) Py_CLEAR(m);
  return m;
}
