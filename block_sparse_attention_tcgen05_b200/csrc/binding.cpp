// Native marshalling of the per-head norm and paged-cache entry points.
//
// These calls run once or more per layer and step, down to single tokens, where the kernels
// take a few microseconds: checking six to eleven tensors and allocating outputs from Python
// took 20 to 40 microseconds a call, in front of them. Here the same checks, allocations and
// the call of libbsa's C entry point take about five. Nothing is kept between calls.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>
#include <string>

#include "../../include/bsa.h"

namespace {

struct ArgError {
  std::string msg;
};
struct PyError {};  // a Python error is already set
struct LibError {
  const char* fn;
  int status;
};

[[noreturn]] void bad(const std::string& msg) { throw ArgError{msg}; }

std::string show(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

std::string show(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kByte: return "torch.uint8";
    default: return std::string("torch.") + at::toString(t);
  }
}

const at::Tensor* optional(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: expected a tensor, got %s", name, Py_TYPE(o)->tp_name);
    throw PyError{};
  }
  return &THPVariable_Unpack(o);
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  const at::Tensor* t = optional(o, name);
  if (!t) bad(std::string(name) + " is required");
  return *t;
}

long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyError{};
  return v;
}

int integer32(PyObject* o, const char* name) {
  const long long v = integer(o);
  if (v > INT32_MAX || v < INT32_MIN) bad(std::string(name) + ": " + std::to_string(v) + " is out of range");
  return static_cast<int>(v);
}

float number(PyObject* o) {
  if (o == Py_None) return 0.f;
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyError{};
  return static_cast<float>(v);
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw PyError{};
  return v != 0;
}

void expect_type(const at::Tensor& t, const char* name, std::initializer_list<at::ScalarType> types) {
  for (at::ScalarType x : types)
    if (t.scalar_type() == x) return;
  std::string want;
  for (at::ScalarType x : types) want += (want.empty() ? "" : ", ") + show(x);
  bad(std::string(name) + ": dtype " + show(t.scalar_type()) + ", expected one of [" + want + "]");
}

void expect_dim(const at::Tensor& t, const char* name, int64_t dim) {
  if (t.dim() != dim)
    bad(std::string(name) + ": " + std::to_string(t.dim()) + " dimensions, expected " + std::to_string(dim));
}

void expect_shape(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) bad(std::string(name) + ": shape " + show(t.sizes()) + ", expected " + show(shape));
}

void expect_contiguous(const at::Tensor& t, const char* name) {
  if (!t.is_contiguous()) bad(std::string(name) + ": must be contiguous");
}

void expect_i32(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  expect_type(t, name, {at::kInt});
  expect_shape(t, name, shape);
  expect_contiguous(t, name);
}

int32_t as_int(int64_t v, const char* what) {
  if (v > INT32_MAX) bad(std::string(what) + ": size " + std::to_string(v) + " is out of range");
  return static_cast<int32_t>(v);
}

// Every tensor of one call on one CUDA device (the library reads plain pointers and launches on
// the current device).
c10::Device same_device(std::initializer_list<const at::Tensor*> ts) {
  const at::Tensor* first = nullptr;
  for (const at::Tensor* t : ts) {
    if (!t) continue;
    if (!first) first = t;
    else if (t->device() != first->device())
      bad("all tensors of one call must be on the same device, got " + first->device().str() + " and " +
          t->device().str());
  }
  if (!first->is_cuda()) bad("libbsa operates on CUDA tensors only");
  return first->device();
}

int dtype_code(at::ScalarType t) {
  return t == at::kBFloat16 ? BSA_BF16 : (t == at::kHalf ? BSA_F16 : BSA_F32);
}

// bsa_heads of a (B, H, S, D) or packed (H, T, D) tensor. The stride of a dimension of size 1 is
// never used and passed as 0; an output may not be broadcast.
bsa_heads heads(const at::Tensor& t, const char* name, bool written = false) {
  const int64_t n = t.dim();
  bsa_heads h{t.data_ptr(), 0, 0, 0};
  if (t.numel() == 0) return h;
  const int64_t unit = 16 / static_cast<int64_t>(t.element_size());
  if (t.stride(n - 1) != 1) bad(std::string(name) + ": the last dimension must be contiguous");
  int64_t st[3] = {0, 0, 0};
  bool ok = reinterpret_cast<uintptr_t>(h.ptr) % 16 == 0;
  for (int64_t i = 0; i < n - 1; ++i) {
    if (t.size(i) == 1) continue;
    const int64_t s = t.stride(i);
    st[i + (4 - n)] = s;
    ok = ok && s % unit == 0;
    if (written && s == 0) bad(std::string(name) + ": an output may not be broadcast");
  }
  if (!ok) bad(std::string(name) + ": pointer and strides must be multiples of 16 bytes");
  h.stride_b = st[0];
  h.stride_h = st[1];
  h.stride_s = st[2];
  return h;
}

struct Norm {
  bsa_shape shape;
  int w_f32;
  int64_t pos_b = 0;
  int n_pos;
};

void expect_table(const at::Tensor& cos, const at::Tensor& sin, int64_t D) {
  expect_type(cos, "cos", {at::kFloat});
  expect_dim(cos, "cos", 2);
  if (cos.size(1) != D / 2)
    bad("cos: shape " + show(cos.sizes()) + ", expected (positions, " + std::to_string(D / 2) + ")");
  expect_type(sin, "sin", {at::kFloat});
  expect_shape(sin, "sin", cos.sizes());
  const at::Tensor* ts[2] = {&cos, &sin};
  const char* names[2] = {"cos", "sin"};
  for (int i = 0; i < 2; ++i) {
    expect_contiguous(*ts[i], names[i]);
    if (ts[i]->numel() && reinterpret_cast<uintptr_t>(ts[i]->data_ptr()) % 16)
      bad(std::string(names[i]) + ": pointer must be a multiple of 16 bytes");
  }
}

int expect_weights(const at::Tensor& qw, const at::Tensor& kw, at::ScalarType dt, int64_t D) {
  expect_type(qw, "q_weight", {at::kFloat, dt});
  expect_shape(qw, "q_weight", {D});
  expect_type(kw, "k_weight", {qw.scalar_type()});
  expect_shape(kw, "k_weight", {D});
  expect_contiguous(qw, "q_weight");
  expect_contiguous(kw, "k_weight");
  return qw.scalar_type() == at::kFloat ? 1 : 0;
}

// Checks shared by the forward and backward calls.
Norm expect_norm(const at::Tensor& q, const at::Tensor& k, const at::Tensor& qw, const at::Tensor& kw,
                 const at::Tensor& cos, const at::Tensor& sin, const at::Tensor* positions) {
  expect_type(q, "q", {at::kBFloat16, at::kHalf, at::kFloat});
  expect_dim(q, "q", 4);
  expect_type(k, "k", {q.scalar_type()});
  expect_dim(k, "k", 4);
  const int64_t B = q.size(0), S = q.size(2), D = q.size(3);
  if (k.size(0) != B || k.size(2) != S || k.size(3) != D || k.size(1) <= 0)
    bad("k: shape " + show(k.sizes()) + " does not fit q " + show(q.sizes()));
  expect_table(cos, sin, D);
  if (!positions && cos.size(0) < S)
    bad("cos: " + std::to_string(cos.size(0)) + " positions for " + std::to_string(S) + " tokens");
  Norm n{};
  n.w_f32 = expect_weights(qw, kw, q.scalar_type(), D);
  if (positions) {
    expect_type(*positions, "positions", {at::kInt});
    const bool each = positions->dim() == 2;
    if (!(positions->dim() == 1 && positions->size(0) == S) &&
        !(each && positions->size(0) == B && positions->size(1) == S))
      bad("positions: shape " + show(positions->sizes()) + ", expected (" + std::to_string(S) + ",) or (" +
          std::to_string(B) + ", " + std::to_string(S) + ")");
    expect_contiguous(*positions, "positions");
    n.pos_b = each ? S : 0;
  }
  n.n_pos = as_int(cos.size(0), "cos");
  n.shape = bsa_shape{as_int(B, "q"), as_int(q.size(1), "q"), as_int(k.size(1), "k"), as_int(S, "q"),
                      as_int(S, "q"), as_int(D, "q"), dtype_code(q.scalar_type())};
  return n;
}

template <class T>
T* ptr(const at::Tensor* t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

// Uninitialised tensors straight from the CUDA allocator (the dispatcher costs as much again).
at::Tensor empty(at::IntArrayRef size, at::ScalarType dt, c10::Device dev) {
  return at::Tensor(at::detail::empty_cuda(size, dt, dev, std::nullopt));
}
at::Tensor empty_strided(at::IntArrayRef size, at::IntArrayRef stride, at::ScalarType dt, c10::Device dev) {
  return at::Tensor(at::detail::empty_strided_cuda(size, stride, dt, dev));
}

at::Tensor workspace_or_new(const at::Tensor* ws, size_t need, c10::Device dev) {
  if (ws && static_cast<size_t>(ws->numel()) >= need) return *ws;
  return empty({static_cast<int64_t>(std::max<size_t>(need, 256))}, at::kByte, dev);
}

void expect_workspace(const at::Tensor* ws) {
  if (!ws) return;
  expect_type(*ws, "workspace", {at::kByte});
  expect_dim(*ws, "workspace", 1);
  expect_contiguous(*ws, "workspace");
}

// The library call itself, on the device and current stream of the tensors, without the GIL.
template <class F>
void launch(const char* fn, c10::Device dev, F&& f) {
  c10::cuda::CUDAGuard guard(dev);
  void* stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  struct WithoutGil {  // taken back also when f throws
    PyThreadState* state = PyEval_SaveThread();
    ~WithoutGil() { PyEval_RestoreThread(state); }
  };
  const int st = [&] {
    WithoutGil g;
    return f(stream);
  }();
  if (st != BSA_OK) throw LibError{fn, st};
}

PyObject* wrap(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  if (!r) throw PyError{};
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
  return r;
}

// Whether autograd is to record a call on these tensors.
bool wants_grad(std::initializer_list<const at::Tensor*> ts) {
  return c10::GradMode::is_enabled() &&
         std::any_of(ts.begin(), ts.end(), [](const at::Tensor* t) { return t && t->requires_grad(); });
}

// (q_out, k_out), or None where autograd is to record the call: then the caller goes through its
// autograd function, which calls again with gradients off.
PyObject* norm(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &qw = tensor(a[2], "q_weight"),
                   &kw = tensor(a[3], "k_weight"), &cos = tensor(a[4], "cos"), &sin = tensor(a[5], "sin");
  const at::Tensor *pos = optional(a[6], "positions"), *qo = optional(a[9], "q_out"), *ko = optional(a[10], "k_out");
  if (wants_grad({&q, &k, &qw, &kw, &cos, &sin, qo, ko})) {
    if (cos.requires_grad() || sin.requires_grad()) bad("cos, sin: no gradient is computed for the rotation");
    if (qo || ko)
      bad("q_out, k_out: given outputs are written outside autograd, but a tensor of the call requires a gradient "
          "(leave them out, or call it under torch.no_grad())");
    Py_RETURN_NONE;
  }
  const Norm n = expect_norm(q, k, qw, kw, cos, sin, pos);
  if (qo) {
    expect_type(*qo, "q_out", {q.scalar_type()});
    expect_shape(*qo, "q_out", q.sizes());
  }
  if (ko) {
    expect_type(*ko, "k_out", {k.scalar_type()});
    expect_shape(*ko, "k_out", k.sizes());
  }
  const bsa_heads hq = heads(q, "q"), hk = heads(k, "k");
  const c10::Device dev = same_device({&q, &k, &qw, &kw, &cos, &sin, pos, qo, ko});
  const at::Tensor q_out = qo ? *qo : empty(q.sizes(), q.scalar_type(), dev);
  const at::Tensor k_out = ko ? *ko : empty(k.sizes(), k.scalar_type(), dev);
  const bsa_heads oq = heads(q_out, "q_out", true), ok = heads(k_out, "k_out", true);
  const float eps = number(a[7]);
  const int inter = truth(a[8]);
  launch("bsa_qk_norm_rotation", dev, [&](void* st) {
    return bsa_qk_norm_rotation(hq, hk, n.shape, qw.data_ptr(), kw.data_ptr(), n.w_f32, ptr<float>(&cos),
                                ptr<float>(&sin), n.n_pos, ptr<int32_t>(pos), n.pos_b, eps, inter, oq, ok, st);
  });
  return wrap({q_out, k_out});
}

// An empty tensor of t's shape, token-major in memory where t is, else contiguous.
at::Tensor like_layout(const at::Tensor& t) {
  const int64_t H = t.size(1), S = t.size(2), D = t.size(3);
  if (H > 1 && S > 1 && t.stride(1) < t.stride(2))
    return empty_strided(t.sizes(), {H * S * D, D, H * D, 1}, t.scalar_type(), t.device());
  return empty(t.sizes(), t.scalar_type(), t.device());
}

PyObject* norm_back(PyObject* const* a) {
  const at::Tensor &dqo = tensor(a[0], "dq_out"), &dko = tensor(a[1], "dk_out"), &q = tensor(a[2], "q"),
                   &k = tensor(a[3], "k"), &qw = tensor(a[4], "q_weight"), &kw = tensor(a[5], "k_weight"),
                   &cos = tensor(a[6], "cos"), &sin = tensor(a[7], "sin");
  const at::Tensor *pos = optional(a[8], "positions"), *ws = optional(a[11], "workspace");
  const Norm n = expect_norm(q, k, qw, kw, cos, sin, pos);
  expect_type(dqo, "dq_out", {q.scalar_type()});
  expect_shape(dqo, "dq_out", q.sizes());
  expect_type(dko, "dk_out", {k.scalar_type()});
  expect_shape(dko, "dk_out", k.sizes());
  expect_workspace(ws);
  const bsa_heads hdq = heads(dqo, "dq_out"), hdk = heads(dko, "dk_out"), hq = heads(q, "q"), hk = heads(k, "k");
  const c10::Device dev = same_device({&dqo, &dko, &q, &k, &qw, &kw, &cos, &sin, pos, ws});
  const at::Tensor work = workspace_or_new(ws, bsa_qk_norm_rotation_workspace_bytes(n.shape), dev);
  const at::Tensor dq = like_layout(q), dk = like_layout(k);
  const at::Tensor dqw = empty({q.size(3)}, at::kFloat, dev), dkw = empty({q.size(3)}, at::kFloat, dev);
  const bsa_heads oq = heads(dq, "dq", true), ok = heads(dk, "dk", true);
  const float eps = number(a[9]);
  const int inter = truth(a[10]);
  launch("bsa_qk_norm_rotation_backward", dev, [&](void* st) {
    return bsa_qk_norm_rotation_backward(hdq, hdk, hq, hk, n.shape, qw.data_ptr(), kw.data_ptr(), n.w_f32,
                                         ptr<float>(&cos), ptr<float>(&sin), n.n_pos, ptr<int32_t>(pos), n.pos_b,
                                         eps, inter, oq, ok, ptr<float>(&dqw), ptr<float>(&dkw), work.data_ptr(),
                                         static_cast<size_t>(work.numel()), st);
  });
  return wrap({dq, dk, dqw, dkw});
}

int64_t expect_block_table(const at::Tensor& t, int64_t R) {
  expect_type(t, "block_table", {at::kInt});
  expect_dim(t, "block_table", 2);
  if (t.size(0) != R)
    bad("block_table: " + std::to_string(t.size(0)) + " rows for " + std::to_string(R) + " requests");
  if (t.numel() && t.size(1) > 1 && t.stride(1) != 1) bad("block_table: rows must be contiguous");
  return R > 1 ? t.stride(0) : t.size(1);
}

PyObject* tables(PyObject* const* a) {
  const at::Tensor &ctx = tensor(a[0], "context_lens"), &nl = tensor(a[1], "new_lens"),
                   &bt = tensor(a[2], "block_table"), &fp = tensor(a[3], "free_pages");
  expect_type(ctx, "context_lens", {at::kInt});
  expect_dim(ctx, "context_lens", 1);
  expect_contiguous(ctx, "context_lens");
  const int64_t R = ctx.size(0);
  expect_i32(nl, "new_lens", {R});
  const int64_t stride = expect_block_table(bt, R);
  if (R > 1 && bt.size(1) > 0 && stride < bt.size(1)) bad("block_table: rows may not overlap");
  expect_type(fp, "free_pages", {at::kInt});
  expect_dim(fp, "free_pages", 1);
  expect_contiguous(fp, "free_pages");
  const int T = integer32(a[4], "n_tokens"), page = integer32(a[5], "page_size"), n_pages = integer32(a[6], "n_pages");
  if (T < 0) bad("n_tokens < 0");
  const c10::Device dev = same_device({&ctx, &nl, &bt, &fp});
  const at::Tensor slots = empty({T}, at::kInt, dev), positions = empty({T}, at::kInt, dev),
                   cu = empty({R + 1}, at::kInt, dev), taken = empty({1}, at::kInt, dev);
  launch("bsa_paged_block_tables", dev, [&](void* st) {
    return bsa_paged_block_tables(ptr<int32_t>(&ctx), ptr<int32_t>(&nl), as_int(R, "context_lens"), ptr<int32_t>(&bt),
                                  as_int(bt.size(1), "block_table"), stride, ptr<int32_t>(&fp),
                                  as_int(fp.size(0), "free_pages"), T, page, n_pages, ptr<int32_t>(&slots),
                                  ptr<int32_t>(&positions), ptr<int32_t>(&cu), ptr<int32_t>(&taken), st);
  });
  return wrap({slots, positions, cu, taken});
}

// bsa_paged_cache of k_cache and v_cache (n_pages, Hkv, page, D); Hkv < 0 and D < 0: any.
bsa_paged_cache paged_cache(const at::Tensor& k, const at::Tensor& v, int64_t Hkv, int64_t D,
                            const at::ScalarType* dt) {
  if (dt) expect_type(k, "k_cache", {*dt});
  expect_type(k, "k_cache", {at::kBFloat16, at::kHalf});
  expect_dim(k, "k_cache", 4);
  expect_type(v, "v_cache", {k.scalar_type()});
  expect_shape(v, "v_cache", k.sizes());
  if ((Hkv >= 0 && k.size(1) != Hkv) || (D >= 0 && k.size(3) != D))
    bad("k_cache: shape " + show(k.sizes()) + ", expected (pages, " + (Hkv >= 0 ? std::to_string(Hkv) : "heads") +
        ", page, " + std::to_string(D) + ")");
  if (k.numel() == 0) bad("k_cache: empty, shape " + show(k.sizes()));
  bsa_paged_cache c{};
  c.k = k.data_ptr();
  c.v = v.data_ptr();
  c.n_pages = as_int(k.size(0), "k_cache");
  c.Hkv = as_int(k.size(1), "k_cache");
  c.page = as_int(k.size(2), "k_cache");
  c.D = as_int(k.size(3), "k_cache");
  c.dtype = dtype_code(k.scalar_type());
  const at::Tensor* ts[2] = {&k, &v};
  const char* names[2] = {"k_cache", "v_cache"};
  int64_t* st[2][3] = {{&c.k_page_stride, &c.k_head_stride, &c.k_row_stride},
                       {&c.v_page_stride, &c.v_head_stride, &c.v_row_stride}};
  for (int i = 0; i < 2; ++i) {
    const at::Tensor& t = *ts[i];
    if (t.stride(3) != 1) bad(std::string(names[i]) + ": the last dimension must be contiguous");
    bool ok = reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0;
    for (int j = 0; j < 3; ++j) {
      const int64_t s = t.size(j) > 1 ? t.stride(j) : 8;  // unused for one entry
      if (s <= 0) bad(std::string(names[i]) + ": may not be broadcast");
      ok = ok && s % 8 == 0;
      *st[i][j] = s;
    }
    if (!ok) bad(std::string(names[i]) + ": pointer and strides must be multiples of 16 bytes");
  }
  return c;
}

PyObject* append(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v"),
                   &qw = tensor(a[3], "q_weight"), &kw = tensor(a[4], "k_weight"), &cos = tensor(a[5], "cos"),
                   &sin = tensor(a[6], "sin"), &pos = tensor(a[7], "positions"), &slots = tensor(a[8], "slots"),
                   &kc = tensor(a[9], "k_cache"), &vc = tensor(a[10], "v_cache");
  const at::Tensor* qo = optional(a[13], "q_out");
  expect_type(q, "q", {at::kBFloat16, at::kHalf});
  expect_dim(q, "q", 3);
  const at::ScalarType dt = q.scalar_type();
  const int64_t Hq = q.size(0), T = q.size(1), D = q.size(2);
  expect_type(k, "k", {dt});
  expect_dim(k, "k", 3);
  if (k.size(1) != T || k.size(2) != D || k.size(0) <= 0)
    bad("k: shape " + show(k.sizes()) + " does not fit q " + show(q.sizes()));
  expect_type(v, "v", {dt});
  expect_shape(v, "v", k.sizes());
  expect_table(cos, sin, D);
  const int f32 = expect_weights(qw, kw, dt, D);
  expect_i32(pos, "positions", {T});
  expect_i32(slots, "slots", {T});
  const bsa_paged_cache cache = paged_cache(kc, vc, k.size(0), D, &dt);
  if (qo) {
    expect_type(*qo, "q_out", {dt});
    expect_shape(*qo, "q_out", q.sizes());
  }
  const bsa_heads hq = heads(q, "q"), hk = heads(k, "k"), hv = heads(v, "v");
  const c10::Device dev = same_device({&q, &k, &v, &qw, &kw, &cos, &sin, &pos, &slots, &kc, &vc, qo});
  const at::Tensor q_out = qo ? *qo : empty(q.sizes(), q.scalar_type(), dev);
  const bsa_heads oq = heads(q_out, "q_out", true);
  const float eps = number(a[11]);
  const int inter = truth(a[12]);
  const int n_pos = as_int(cos.size(0), "cos");
  launch("bsa_paged_qk_norm_append", dev, [&](void* st) {
    return bsa_paged_qk_norm_append(hq, hk, hv, as_int(T, "q"), as_int(Hq, "q"), qw.data_ptr(), kw.data_ptr(), f32,
                                    ptr<float>(&cos), ptr<float>(&sin), n_pos, ptr<int32_t>(&pos),
                                    ptr<int32_t>(&slots), eps, inter, oq, cache, st);
  });
  return THPVariable_Wrap(q_out);
}

PyObject* attend(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache"),
                   &bt = tensor(a[3], "block_table"), &cu = tensor(a[4], "cu_new"), &ctx = tensor(a[5], "context_lens");
  const at::Tensor *mask = optional(a[8], "page_mask"), *po = optional(a[10], "out"), *ws = optional(a[11], "workspace");
  expect_type(q, "q", {at::kBFloat16, at::kHalf});
  expect_dim(q, "q", 3);
  const at::ScalarType dt = q.scalar_type();
  const int64_t Hq = q.size(0), T = q.size(1), D = q.size(2);
  expect_type(bt, "block_table", {at::kInt});
  expect_dim(bt, "block_table", 2);
  const int64_t R = bt.size(0), width = bt.size(1);
  const int64_t stride = expect_block_table(bt, R);
  expect_i32(cu, "cu_new", {R + 1});
  expect_i32(ctx, "context_lens", {R});
  const bsa_paged_cache cache = paged_cache(kc, vc, -1, D, &dt);
  if (Hq <= 0 || Hq % cache.Hkv)
    bad("q: " + std::to_string(Hq) + " heads, not a multiple of the cache's " + std::to_string(cache.Hkv));
  at::Tensor copy;
  int64_t mr = 0, mg = 0;
  if (mask) {
    const int64_t d = mask->dim();
    if ((mask->scalar_type() != at::kByte && mask->scalar_type() != at::kBool) || (d != 2 && d != 3))
      bad("page_mask must be bool or uint8 with 2 or 3 dimensions");
    const int64_t heads_of = d == 3 ? mask->size(1) : 1;
    if ((mask->size(0) != 1 && mask->size(0) != R) || (heads_of != 1 && heads_of != cache.Hkv) ||
        mask->size(d - 1) != width)
      bad("page_mask: shape " + show(mask->sizes()) + ", expected (" + std::to_string(R) + ", " +
          std::to_string(cache.Hkv) + ", " + std::to_string(width) + ") or (" + std::to_string(R) + ", " +
          std::to_string(width) + ")");
    if (width > 1 && mask->stride(d - 1) != 1) {
      copy = mask->contiguous();
      mask = &copy;
    }
    mr = mask->size(0) > 1 ? mask->stride(0) : 0;
    mg = d == 3 && mask->size(1) > 1 ? mask->stride(1) : 0;
  }
  if (po) {
    expect_type(*po, "out", {dt});
    expect_shape(*po, "out", q.sizes());
  }
  expect_workspace(ws);
  const bsa_heads hq = heads(q, "q");
  const c10::Device dev = same_device({&q, &kc, &vc, &bt, &cu, &ctx, mask, po, ws});
  const int causal = truth(a[6]);
  // A bound of 0 counts as 1: the library would return without looking at the lengths, and the
  // rows of a request that has tokens all the same would stay uninitialised, unrecorded.
  int max_new = a[7] == Py_None ? as_int(T, "q") : integer32(a[7], "max_new");
  if (max_new == 0) max_new = 1;
  const float scale = number(a[9]);
  const int iR = as_int(R, "block_table"), iT = as_int(T, "q"), iH = as_int(Hq, "q"), iW = as_int(width, "block_table");
  const size_t need = bsa_paged_attention_workspace_bytes(cache, iR, iT, iH, max_new, iW);
  if (need == 0) throw LibError{"bsa_paged_attention_workspace_bytes", BSA_ERR_UNSUPPORTED};
  const at::Tensor out = po ? *po : empty(q.sizes(), q.scalar_type(), dev);
  const bsa_heads ho = heads(out, "out", true);
  const at::Tensor work = workspace_or_new(ws, need, dev);
  launch("bsa_paged_chunk_attention", dev, [&](void* st) {
    return bsa_paged_chunk_attention(hq, cache, ptr<int32_t>(&bt), iW, stride, ptr<int32_t>(&cu), ptr<int32_t>(&ctx), iR,
                                     iT, iH, max_new, ptr<uint8_t>(mask), mr, mg, scale, causal, ho, work.data_ptr(),
                                     static_cast<size_t>(work.numel()), st);
  });
  return THPVariable_Wrap(out);
}

// Argument errors become ValueError, library errors the package's BsaError.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const ArgError& e) {
    PyErr_SetString(PyExc_ValueError, e.msg.c_str());
  } catch (const PyError&) {
  } catch (const LibError& e) {
    char detail[512] = "";
    bsa_last_error_detail(detail, sizeof(detail));
    PyObject* mod = PyImport_ImportModule("block_sparse_attention_tcgen05_b200._lib");
    PyObject* cls = mod ? PyObject_GetAttrString(mod, "BsaError") : nullptr;
    PyObject* exc = cls ? PyObject_CallFunction(cls, "sis", e.fn, e.status, detail) : nullptr;
    if (exc) PyErr_SetObject(cls, exc);
    Py_XDECREF(exc);
    Py_XDECREF(cls);
    Py_XDECREF(mod);
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* mod = PyImport_ImportModule("torch");
    PyObject* cls = mod ? PyObject_GetAttrString(mod, "OutOfMemoryError") : nullptr;
    if (cls) PyErr_SetString(cls, e.what_without_backtrace());
    Py_XDECREF(cls);
    Py_XDECREF(mod);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define BSA_METHOD(name, fn, n) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<fn, n>)), METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {
    BSA_METHOD("qk_norm_rotation", norm, 11),
    BSA_METHOD("qk_norm_rotation_backward", norm_back, 12),
    BSA_METHOD("paged_block_tables", tables, 7),
    BSA_METHOD("paged_qk_norm_append", append, 14),
    BSA_METHOD("paged_chunk_attention", attend, 12),
    {nullptr, nullptr, 0, nullptr}};

// What the module was compiled against; build.py and the loader look for it in the file.
[[gnu::used]] const char kNativeId[] = BSA_NATIVE_ID;

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", "Native marshalling of libbsa calls.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&kModule); }
