// vg_torch.cpp -- the verify round's calls from torch tensors: checks of the
// tensors, their outputs' allocation and the call into libvgemm's C ABI.  No
// computation happens here.
//
// These operators take 3 to 12 us on the device for a single token, so the
// way to them counts.  Reading the tensors and filling the descriptors in
// Python took 6 to 10 us a call beside the launch; from here a whole call, launch
// and Python's part included, takes the host 3.4 to 4 us, verification 5.7.
//
// A function returns its output, or the vg_status of a call that was refused;
// a tensor of the wrong kind raises ValueError, and so do tensors of several
// devices.  libvgemm launches on the current device: a call makes its tensors'
// device current.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/vgemm.h"

namespace {

using at::Tensor;

struct Bad {                                   // an argument of the wrong kind
  std::string what;
};

bool given(PyObject *o) { return o != Py_None; }

const Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw Bad{std::string(name) + ": expected a CUDA tensor"};
  const Tensor &t = THPVariable_Unpack(o);
  if (!t.is_cuda()) throw Bad{std::string(name) + ": expected a CUDA tensor"};
  return t;
}

// A contiguous CUDA tensor of that type and shape.
const Tensor &exact(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name) {
  const Tensor &t = tensor(o, name);
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous()) {
    std::string s;
    for (const int64_t d : shape) s += (s.empty() ? "" : ", ") + std::to_string(d);
    throw Bad{std::string(name) + ": expected a contiguous CUDA " + c10::toString(type) +
              " tensor of shape (" + s + ")"};
  }
  return t;
}
template <typename T = void>
const T *at_of(PyObject *o, at::ScalarType type, at::IntArrayRef shape, const char *name) {
  return given(o) ? static_cast<const T *>(exact(o, type, shape, name).const_data_ptr()) : nullptr;
}

// [batch, n, heads, head_dim] whose last dimension is contiguous.  The stride of a
// dimension of one is arbitrary: 0 is aligned to everything.
const Tensor &heads(PyObject *o, const char *name, int64_t (&stride)[3]) {
  const Tensor &t = tensor(o, name);
  if (t.dim() != 4 || t.stride(3) != 1)
    throw Bad{std::string(name) + ": expected a CUDA tensor [batch, n, heads, head_dim] whose last "
                                  "dimension is contiguous"};
  for (int i = 0; i < 3; ++i) stride[i] = t.size(i) > 1 ? t.stride(i) : 0;
  return t;
}

int32_t type_of(const Tensor &t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return VG_TYPE_BF16;
    case at::kHalf: return VG_TYPE_FP16;
    case at::kFloat: return VG_TYPE_FP32;
    default: return -1;
  }
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
float number(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return float(v);
}

// The device of a call's tensors, which must be one; those not given are passed
// over, but for the first.
struct Argument {
  PyObject *o;
  const char *name;
};
c10::DeviceIndex one_device(std::initializer_list<Argument> all, PyObject *cache_device = nullptr) {
  int64_t device = cache_device ? integer(cache_device) : -1;
  for (const Argument &x : all) {
    if (!given(x.o) && &x != all.begin()) continue;
    const int64_t its = tensor(x.o, x.name).get_device();
    if (device < 0) device = its;
    if (its != device)
      throw Bad{std::string(x.name) + ": on device " + std::to_string(its) + ", and others of the call on device " +
                std::to_string(device)};
  }
  return c10::DeviceIndex(device);
}

const vg_kv_cache *cache_of(PyObject *o) { return reinterpret_cast<const vg_kv_cache *>(integer(o)); }

// Work and the tensors made for it go to the current stream.
vg_stream_t stream_of(const Tensor &t) {
  return reinterpret_cast<vg_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}

// The given output, which must be like `like` (of type `type`), or a new one.
Tensor output(PyObject *o, const Tensor &like, at::ScalarType type, const char *name) {
  if (given(o)) return exact(o, type, like.sizes(), name);
  return at::empty(like.sizes(), like.options().dtype(type));
}

PyObject *result(vg_status s, const Tensor &t) {
  return s ? PyLong_FromLong(s) : THPVariable_Wrap(t);
}

#define VG_BEGIN(count)                                                               \
  HANDLE_TH_ERRORS                                                                    \
  if (n_args != count) {                                                              \
    PyErr_SetString(PyExc_TypeError, "expected " #count " arguments");                \
    return nullptr;                                                                   \
  }                                                                                   \
  try {
#define VG_END                                                                        \
  }                                                                                   \
  catch (const Bad &e) {                                                              \
    PyErr_SetString(PyExc_ValueError, e.what.c_str());                                \
    return nullptr;                                                                   \
  }                                                                                   \
  END_HANDLE_TH_ERRORS

// Fills `d` from q, k, v, inv_freq, cache, lens, depth, counts, layout, factor and q_out; returns the output.
Tensor rope_desc(PyObject *const *a, vg_rope_desc &d) {
  const Tensor &q = heads(a[0], "q", d.q_stride), &k = heads(a[1], "k", d.k_stride),
               &v = heads(a[2], "v", d.v_stride), &f = tensor(a[3], "inv_freq");
  const vg_kv_cache *cache = cache_of(a[4]);
  const int64_t B = q.size(0), n = q.size(1);
  const int64_t kv[4] = {B, n, cache->heads, cache->head_dim};
  if (B != cache->batch || q.size(3) != cache->head_dim || k.sizes() != at::IntArrayRef(kv) ||
      v.sizes() != at::IntArrayRef(kv))
    throw Bad{"q, k, v and the cache do not fit together"};
  if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
    throw Bad{"q, k and v must have the same type"};
  if (f.scalar_type() != at::kDouble || !f.is_contiguous())
    throw Bad{"inv_freq: expected a contiguous CUDA float64 tensor"};
  if (n > INT32_MAX || 2 * f.numel() > INT32_MAX) throw Bad{"q or inv_freq is too long"};
  const Tensor out = output(a[10], q, q.scalar_type(), "q_out");
  d.q = q.const_data_ptr();
  d.k = k.const_data_ptr();
  d.v = v.const_data_ptr();
  d.q_out = out.data_ptr();
  d.inv_freq = static_cast<const double *>(f.const_data_ptr());
  d.lens = static_cast<const int32_t *>(exact(a[5], at::kInt, {B}, "lens").const_data_ptr());
  d.depth = at_of<int32_t>(a[6], at::kInt, {B, n}, "depth");
  d.counts = at_of<int32_t>(a[7], at::kInt, {B}, "counts");
  d.type = type_of(q);
  d.layout = int32_t(integer(a[8]));
  d.n = int32_t(n);
  d.q_heads = int32_t(q.size(2));
  d.rot = int32_t(2 * f.numel());
  d.factor = number(a[9]);
  return out;
}

// q, k, v, inv_freq, cache, lens, depth, counts, layout, factor, q_out, the cache's device
PyObject *rope_append(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  VG_BEGIN(12)
  const c10::cuda::CUDAGuard guard(one_device({{a[0], "q"}, {a[1], "k"}, {a[2], "v"}, {a[3], "inv_freq"}, {a[5], "lens"},
                                               {a[6], "depth"}, {a[7], "counts"}, {a[10], "q_out"}}, a[11]));
  vg_rope_desc d;
  const Tensor out = rope_desc(a, d);
  return result(vg_rope_append(&d, cache_of(a[4]), stream_of(out)), out);
  VG_END
}

// rope_append's, then q_weight, k_weight, eps
PyObject *qk_norm_rope_append(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  VG_BEGIN(15)
  const c10::cuda::CUDAGuard guard(one_device({{a[0], "q"}, {a[1], "k"}, {a[2], "v"}, {a[3], "inv_freq"}, {a[5], "lens"},
                                               {a[6], "depth"}, {a[7], "counts"}, {a[10], "q_out"}, {a[12], "q_weight"},
                                               {a[13], "k_weight"}}, a[11]));
  vg_qk_norm_rope_desc d;
  const Tensor out = rope_desc(a, d.rope);
  d.weight_type = d.rope.type;
  d.q_weight = d.k_weight = nullptr;
  bool some = false;
  for (const bool k : {false, true}) {
    const char *name = k ? "k_weight" : "q_weight";
    if (!given(a[12 + k])) continue;
    const Tensor &w = tensor(a[12 + k], name);
    const at::ScalarType type = w.scalar_type() == at::kFloat ? at::kFloat : out.scalar_type();
    if (w.scalar_type() != type || w.dim() != 1 || w.size(0) != out.size(3) || !w.is_contiguous())
      throw Bad{std::string(name) + ": expected a contiguous CUDA tensor [head_dim] of float32 or of q's type"};
    if (some && type_of(w) != d.weight_type) throw Bad{"q_weight and k_weight must have the same type"};
    some = true;
    d.weight_type = type_of(w);
    (k ? d.k_weight : d.q_weight) = w.const_data_ptr();
  }
  d.eps = number(a[14]);
  return result(vg_qk_norm_rope_append(&d, cache_of(a[4]), stream_of(out)), out);
  VG_END
}

// Fills `d` from q, cache, lens, tree, counts, scale, out, lse; returns the output.
Tensor attention_desc(PyObject *const *a, vg_attention_desc &d) {
  const Tensor &q = heads(a[0], "q", d.q_stride);
  const vg_kv_cache *cache = cache_of(a[1]);
  const int64_t B = q.size(0), n = q.size(1), hq = q.size(2);
  if (B != cache->batch || q.size(3) != cache->head_dim) throw Bad{"q and the cache do not fit together"};
  if (n > INT32_MAX || hq > INT32_MAX) throw Bad{"q is too long"};
  const Tensor out = output(a[6], q, q.scalar_type(), "out");
  d.q = q.const_data_ptr();
  d.out = out.data_ptr();
  d.lse = given(a[7]) ? static_cast<float *>(exact(a[7], at::kFloat, {B, n, hq}, "lse").data_ptr()) : nullptr;
  d.lens = static_cast<const int32_t *>(exact(a[2], at::kInt, {B}, "lens").const_data_ptr());
  d.tree = at_of<uint64_t>(a[3], at::kLong, {B, n}, "tree");
  d.counts = at_of<int32_t>(a[4], at::kInt, {B}, "counts");
  d.type = type_of(q);
  d.n = int32_t(n);
  d.q_heads = int32_t(hq);
  d.scale = number(a[5]);
  return out;
}

const Tensor &workspace_of(PyObject *o, const char *maker) {
  const Tensor &ws = tensor(o, "workspace");
  if (ws.scalar_type() != at::kByte || !ws.is_contiguous())
    throw Bad{std::string("workspace: expected a tensor from ") + maker};
  return ws;
}

// q, cache, lens, tree, counts, scale, out, lse, workspace, the cache's device
PyObject *tree_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  VG_BEGIN(10)
  const c10::cuda::CUDAGuard guard(one_device({{a[0], "q"}, {a[2], "lens"}, {a[3], "tree"}, {a[4], "counts"},
                                               {a[6], "out"}, {a[7], "lse"}, {a[8], "workspace"}}, a[9]));
  vg_attention_desc d;
  const Tensor &ws = workspace_of(a[8], "tree_attention_workspace");
  const Tensor out = attention_desc(a, d);
  return result(vg_tree_attention(&d, cache_of(a[1]), ws.data_ptr(), size_t(ws.numel()), stream_of(out)), out);
  VG_END
}

// tree_attention's, then prefix, prefix_pages
PyObject *prefix_attention(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  VG_BEGIN(12)
  const c10::cuda::CUDAGuard guard(one_device({{a[0], "q"}, {a[2], "lens"}, {a[3], "tree"}, {a[4], "counts"},
                                               {a[6], "out"}, {a[7], "lse"}, {a[8], "workspace"}, {a[10], "prefix"},
                                               {a[11], "prefix_pages"}}, a[9]));
  vg_attention_desc d;
  const Tensor &ws = workspace_of(a[8], "prefix_attention_workspace");
  const Tensor &prefix = exact(a[10], at::kInt, {1}, "prefix"), &pages = tensor(a[11], "prefix_pages");
  if (pages.scalar_type() != at::kInt || pages.dim() != 1 || !pages.is_contiguous() || pages.numel() > INT32_MAX)
    throw Bad{"prefix_pages: expected a contiguous CUDA int32 tensor [pages]"};
  const Tensor out = attention_desc(a, d);
  return result(vg_prefix_attention(&d, cache_of(a[1]), static_cast<const int32_t *>(prefix.const_data_ptr()),
                                    static_cast<const int32_t *>(pages.const_data_ptr()), int(pages.numel()),
                                    ws.data_ptr(), size_t(ws.numel()), stream_of(out)),
                out);
  VG_END
}

// logits, temperature, out
PyObject *probabilities(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  VG_BEGIN(3)
  const c10::cuda::CUDAGuard guard(one_device({{a[0], "logits"}, {a[1], "temperature"}, {a[2], "out"}}));
  const Tensor &x = tensor(a[0], "logits");
  if (x.dim() < 1 || !x.numel() || !x.is_contiguous())
    throw Bad{"logits: expected a contiguous CUDA tensor that is not empty"};
  const int64_t vocab = x.size(-1), rows = x.numel() / vocab;
  const float *t = nullptr;
  if (given(a[1])) {
    const Tensor &tt = tensor(a[1], "temperature");
    if (tt.scalar_type() != at::kFloat || !tt.is_contiguous() || tt.numel() != rows)
      throw Bad{"temperature: expected a contiguous CUDA float32 tensor, one for each row"};
    t = static_cast<const float *>(tt.const_data_ptr());
  }
  const Tensor out = output(a[2], x, at::kFloat, "out");
  return result(vg_probabilities(x.const_data_ptr(), type_of(x), rows, vocab, t,
                                 static_cast<float *>(out.data_ptr()), stream_of(x)),
                out);
  VG_END
}

// logits, u, temperature, top_k, top_p, min_p, out -> tokens
PyObject *sample(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  VG_BEGIN(7)
  const c10::cuda::CUDAGuard guard(one_device({{a[0], "logits"}, {a[1], "u"}, {a[2], "temperature"}, {a[3], "top_k"},
                                               {a[4], "top_p"}, {a[5], "min_p"}, {a[6], "out"}}));
  const Tensor &x = tensor(a[0], "logits"), &u = tensor(a[1], "u");
  const bool one = x.dim() == 1;
  if (x.dim() < 1 || x.dim() > 2 || !x.numel() || (x.size(-1) > 1 && x.stride(-1) != 1))
    throw Bad{"logits: expected a CUDA tensor [rows, vocab] or [vocab] that is not empty and whose last dimension is "
              "contiguous"};
  vg_sample_desc d;
  d.rows = one ? 1 : x.size(0);
  d.vocab = x.size(-1);
  d.row_stride = d.rows > 1 ? x.stride(0) : d.vocab;
  // [rows] or [rows, draws], without rows where the logits have none
  if (u.scalar_type() != at::kFloat || !u.is_contiguous() || (!one && u.dim() < 1) ||
      u.dim() > (one ? 1 : 2) || (!one && u.size(0) != d.rows) || !u.numel() || u.numel() / d.rows > INT32_MAX)
    throw Bad{"u: expected a contiguous CUDA float32 tensor [rows] or [rows, draws]"};
  d.draws = int32_t(u.numel() / d.rows);
  auto each = [&](PyObject *o, at::ScalarType type, const char *name) -> const void * {
    if (!given(o)) return nullptr;
    const Tensor &t = tensor(o, name);
    if (t.scalar_type() != type || !t.is_contiguous() || t.numel() != d.rows)
      throw Bad{std::string(name) + ": expected a contiguous CUDA " + c10::toString(type) + " tensor, one for each row"};
    return t.const_data_ptr();
  };
  d.temperature = static_cast<const float *>(each(a[2], at::kFloat, "temperature"));
  d.top_k = static_cast<const int32_t *>(each(a[3], at::kInt, "top_k"));
  d.top_p = static_cast<const float *>(each(a[4], at::kFloat, "top_p"));
  d.min_p = static_cast<const float *>(each(a[5], at::kFloat, "min_p"));
  d.out = given(a[6]) ? static_cast<float *>(exact(a[6], at::kFloat, x.sizes(), "out").data_ptr()) : nullptr;
  d.x = x.const_data_ptr();
  d.u = static_cast<const float *>(u.const_data_ptr());
  d.type = type_of(x);
  const Tensor tokens = at::empty(u.sizes(), u.options().dtype(at::kInt));
  d.tokens = static_cast<int32_t *>(tokens.data_ptr());
  return result(vg_sample(&d, stream_of(x)), tokens);
  VG_END
}

// p, q, tokens, parents, u, counts -> (accepted, path, out)
PyObject *verify_tree(PyObject *, PyObject *const *a, Py_ssize_t n_args) {
  VG_BEGIN(6)
  const c10::cuda::CUDAGuard guard(one_device({{a[0], "p"}, {a[1], "q"}, {a[2], "tokens"}, {a[3], "parents"}, {a[4], "u"},
                                               {a[5], "counts"}}));
  const Tensor &p = tensor(a[0], "p");
  if (p.scalar_type() != at::kFloat || p.dim() != 3 || !p.is_contiguous())
    throw Bad{"p: expected a contiguous CUDA float32 tensor [batch, n, vocab]"};
  const int64_t B = p.size(0), n = p.size(1), V = p.size(2);
  if (B > INT32_MAX || n > INT32_MAX) throw Bad{"p is too long"};
  const float *q = nullptr;
  int64_t rows = 0;
  if (given(a[1])) {
    const Tensor &t = tensor(a[1], "q");
    if (t.scalar_type() != at::kFloat || t.dim() != 3 || !t.is_contiguous() || t.size(0) != B ||
        t.size(2) != V || t.size(1) > INT32_MAX)
      throw Bad{"q: expected a contiguous CUDA float32 tensor [batch, rows, vocab]"};
    q = static_cast<const float *>(t.const_data_ptr());
    rows = t.size(1);
  }
  const int32_t *tokens = static_cast<const int32_t *>(exact(a[2], at::kInt, {B, n}, "tokens").const_data_ptr());
  const int32_t *parents = static_cast<const int32_t *>(exact(a[3], at::kInt, {B, n}, "parents").const_data_ptr());
  const float *u = static_cast<const float *>(exact(a[4], at::kFloat, {B, n}, "u").const_data_ptr());
  const int32_t *counts = at_of<int32_t>(a[5], at::kInt, {B}, "counts");
  const auto opt = p.options().dtype(at::kInt);
  const Tensor accepted = at::empty({B}, opt), path = at::empty({B, n}, opt), out = at::empty({B, n + 1}, opt);
  const vg_status s = vg_verify_tree(
      static_cast<const float *>(p.const_data_ptr()), q, tokens, parents, counts, u, int(B), int(n),
      int(rows), V, static_cast<int32_t *>(accepted.data_ptr()), static_cast<int32_t *>(path.data_ptr()),
      static_cast<int32_t *>(out.data_ptr()), stream_of(p));
  if (s) return PyLong_FromLong(s);
  PyObject *r = PyTuple_New(3);
  if (!r) return nullptr;
  PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(accepted));
  PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(path));
  PyTuple_SET_ITEM(r, 2, THPVariable_Wrap(out));
  return r;
  VG_END
}

#define VG_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {VG_METHOD(rope_append), VG_METHOD(tree_attention), VG_METHOD(probabilities),
                         VG_METHOD(verify_tree), VG_METHOD(qk_norm_rope_append), VG_METHOD(prefix_attention),
                         VG_METHOD(sample), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_vgtorch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__vgtorch(void) { return PyModule_Create(&module); }
