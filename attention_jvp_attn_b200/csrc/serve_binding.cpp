// serve_binding.cpp - Python binding of the serving operators (module _serving):
// checks tensors, allocates outputs and workspace on the current stream, and
// calls the C ABI (include/attn_jvp.h) through addresses that bind() gets, so
// that the library loaded by the package is the only one.
//
// These calls are short (3 to 8 us on the GPU for a decode step), and reading some
// forty sizes, strides and pointers through Python objects took longer than that.
// Calls among others, that way and this: rotation 17.2 and 5.6 us, append 15.1 and
// 8.2, one short sequence's attention 19.1 and 10.2 (the last two: GPU time now).
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdint>

#include "attn_jvp.h"

namespace {

using at::Tensor;

decltype(&attn_jvp_rope_at) g_rope_at;
decltype(&attn_jvp_cache_append) g_cache_append;
decltype(&attn_jvp_cache_attn) g_cache_attn;
decltype(&attn_jvp_cache_attn_workspace_bytes) g_workspace_bytes;
decltype(&attn_jvp_prompt_attn) g_prompt_attn;
PyObject* g_check;  // check(code, name): raises the package's error

const Tensor& tensor(PyObject* o, const char* what) {
  TORCH_CHECK_VALUE(THPVariable_Check(o), what, " must be a tensor");
  return THPVariable_Unpack(o);
}

// Strides of a [T, heads, d] CUDA tensor whose d elements are adjacent.
attn_jvp_strides rows(const Tensor& t, const char* what, const Tensor* like = nullptr) {
  TORCH_CHECK_VALUE(t.dim() == 3, what, " must be [T, heads, d]");
  TORCH_CHECK_VALUE(t.is_cuda(), what, " must be a CUDA tensor");
  if (like)
    TORCH_CHECK_VALUE(t.size(0) == like->size(0) && t.size(2) == like->size(2) &&
                          t.scalar_type() == like->scalar_type() && t.device() == like->device(),
                      what, " must share tokens, head dim, dtype and device with the others");
  TORCH_CHECK_VALUE(t.stride(2) == 1, "the last dimension of ", what, " must be contiguous");
  return {t.stride(0), t.stride(1)};
}

const int32_t* int32s(PyObject* o, const char* what, c10::Device device, int64_t n) {
  const Tensor& t = tensor(o, what);
  TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == n && t.scalar_type() == at::kInt &&
                        t.device() == device && t.is_contiguous(),
                    what, " must be a contiguous int32 [", n, "] tensor on the inputs' device");
  return static_cast<const int32_t*>(t.data_ptr());
}

const Tensor& page_table(PyObject* o, int64_t B, c10::Device device) {
  const Tensor& t = tensor(o, "page_table");
  TORCH_CHECK_VALUE(t.dim() == 2 && t.scalar_type() == at::kInt && t.device() == device &&
                        t.size(0) == B && t.size(1) >= 1 && (t.size(1) == 1 || t.stride(1) == 1),
                    "page_table must be int32 [B, pages] with contiguous rows on the inputs' device");
  return t;
}

attn_jvp_rope_tables rope_tables(PyObject* cos_o, PyObject* sin_o, PyObject* layout, c10::Device device) {
  const Tensor &c = tensor(cos_o, "cos"), &s = tensor(sin_o, "sin");
  for (const Tensor* t : {&c, &s})
    TORCH_CHECK_VALUE(t->dim() == 2 && t->sizes() == c.sizes() && t->scalar_type() == at::kFloat &&
                          t->device() == device && t->is_contiguous(),
                      "cos and sin must be contiguous fp32 [positions, rot/2] on the inputs' device");
  attn_jvp_rope_tables r = {static_cast<const float*>(c.data_ptr()), static_cast<const float*>(s.data_ptr()),
                            c.size(0), 2 * c.size(1), ATTN_JVP_ROPE_INTERLEAVED};
  const bool text = PyUnicode_Check(layout);
  if (text && PyUnicode_CompareWithASCIIString(layout, "half") == 0)
    r.layout = ATTN_JVP_ROPE_HALF;
  else
    TORCH_CHECK_VALUE(text && PyUnicode_CompareWithASCIIString(layout, "interleaved") == 0,
                      "layout is 'interleaved' or 'half'");
  return r;
}

struct Cache {
  const Tensor *k, *v, *k_scale, *v_scale;
  explicit Cache(PyObject* o) {
    TORCH_CHECK_VALUE(PyTuple_Check(o) && PyTuple_GET_SIZE(o) == 4, "cache must be a PagedCache");
    k = &tensor(PyTuple_GET_ITEM(o, 0), "cache k");
    v = &tensor(PyTuple_GET_ITEM(o, 1), "cache v");
    k_scale = &tensor(PyTuple_GET_ITEM(o, 2), "cache k_scale");
    v_scale = &tensor(PyTuple_GET_ITEM(o, 3), "cache v_scale");
    TORCH_CHECK_VALUE(k->dim() == 4, "cache k must be [pages, Hkv, page_tokens, d]");
  }
  attn_jvp_cache checked(c10::Device device) const {
    TORCH_CHECK_VALUE(k->scalar_type() == at::kFloat8_e4m3fn && v->scalar_type() == at::kFloat8_e4m3fn &&
                          v->sizes() == k->sizes() && v->strides() == k->strides() && k->stride(3) == 1 &&
                          k->device() == device && v->device() == device,
                      "cache k and v must be float8_e4m3fn [pages, Hkv, page_tokens, d] of the "
                      "same strides, d contiguous, on the inputs' device");
    TORCH_CHECK_VALUE(k_scale->sizes() == k->sizes().slice(0, 2) && v_scale->sizes() == k_scale->sizes() &&
                          k_scale->scalar_type() == at::kFloat && v_scale->scalar_type() == at::kFloat &&
                          v_scale->strides() == k_scale->strides() && k_scale->device() == device &&
                          v_scale->device() == device,
                      "cache scales must be fp32 [pages, Hkv] of the same strides on the inputs' device");
    return {k->data_ptr(), v->data_ptr(), static_cast<float*>(k_scale->data_ptr()),
            static_cast<float*>(v_scale->data_ptr()), k->size(0), k->size(2), k->stride(0), k->stride(1),
            k->stride(2), k_scale->stride(0), k_scale->stride(1)};
  }
};

int32_t dtype(const Tensor& t, bool with_f32) {
  const auto s = t.scalar_type();
  if (s == at::kBFloat16) return ATTN_JVP_BF16;
  if (s == at::kHalf) return ATTN_JVP_F16;
  TORCH_CHECK_TYPE(s == at::kFloat && with_f32, "unsupported dtype ", s);
  return ATTN_JVP_F32;
}

// A Python number; 0 for None (the default scale).
float scale_of(PyObject* o) {
  if (o == Py_None) return 0.f;
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  const float f = static_cast<float>(x);
  TORCH_CHECK_VALUE(f > 0.f && std::isfinite(f), "scale must be positive and finite (in 32 bits)");
  return f;
}

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw python_error();
  return r != 0;
}

// The two tensors of `out`, which may be any sequence; held, as another thread
// may change it during the call.
struct Pair {
  PyObject *a = nullptr, *b = nullptr;
  explicit Pair(PyObject* out) {
    PyObject* fast = PySequence_Fast(out, "out must be a pair");
    if (!fast) throw python_error();
    const bool two = PySequence_Fast_GET_SIZE(fast) == 2;
    if (two) {
      a = PySequence_Fast_GET_ITEM(fast, 0), b = PySequence_Fast_GET_ITEM(fast, 1);
      Py_INCREF(a);
      Py_INCREF(b);
    }
    Py_DECREF(fast);
    TORCH_CHECK_VALUE(two, "out must be a pair");
  }
  ~Pair() {
    Py_DECREF(a);
    Py_DECREF(b);
  }
  Pair(const Pair&) = delete;
};

PyObject* pair(PyObject* a, PyObject* b) {  // takes both references
  PyObject* r = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return r;
}
PyObject* pair(const Tensor& a, const Tensor& b) { return pair(THPVariable_Wrap(a), THPVariable_Wrap(b)); }
PyObject* given(PyObject* a, PyObject* b) {
  Py_INCREF(a);
  Py_INCREF(b);
  return pair(a, b);
}

// f(current stream) on the tensors' device, other Python threads running
// meanwhile: a launch may wait for room in the queue.
template <typename F>
void call(const char* name, c10::Device device, F f) {
  const c10::cuda::CUDAGuard guard(device);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  PyThreadState* state = PyEval_SaveThread();
  const int rc = f(stream);
  PyEval_RestoreThread(state);
  if (rc != ATTN_JVP_OK) {
    PyObject* r = PyObject_CallFunction(g_check, "is", rc, name);
    Py_XDECREF(r);
    if (!r) throw python_error();
  }
}

// A tensor of the caller's was written over: autograd, which may have saved it,
// goes by its version (inference tensors have none).
void written(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

// rope_at(q, k, positions, cos, sin, layout, transpose, out)
PyObject* rope_at(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 8, "rope_at takes 8 arguments");
  const Tensor& q = tensor(a[0], "q");
  const Tensor* k = a[1] == Py_None ? nullptr : &tensor(a[1], "k");
  const attn_jvp_strides sq = rows(q, "q"), sk = k ? rows(*k, "k", &q) : attn_jvp_strides{0, 0};
  const int64_t T = q.size(0), H = q.size(1), d = q.size(2), Hkv = k ? k->size(1) : 0;
  const Tensor& at_ = tensor(a[2], "positions");
  TORCH_CHECK_VALUE(at_.dim() == 1 && at_.size(0) == T && (at_.scalar_type() == at::kInt || at_.scalar_type() == at::kLong) &&
                        at_.device() == q.device() && at_.is_contiguous(),
                    "positions must be contiguous int32 or int64 [T] on the inputs' device");
  const attn_jvp_rope_tables tables = rope_tables(a[3], a[4], a[5], q.device());
  const attn_jvp_tokens shape = {T, H, Hkv, d, dtype(q, true), 0.f};
  const bool transpose = truth(a[6]);
  auto run = [&](const Tensor& qo, attn_jvp_strides so, const Tensor* ko, attn_jvp_strides sko) {
    call("attn_jvp_rope_at", q.device(), [&](cudaStream_t stream) {
      return g_rope_at(&shape, q.data_ptr(), sq, k ? k->data_ptr() : nullptr, sk, at_.data_ptr(),
                       static_cast<int32_t>(at_.element_size()), &tables, transpose, qo.data_ptr(), so,
                       ko ? ko->data_ptr() : nullptr, sko, stream);
    });
  };
  if (a[7] == Py_None) {
    const Tensor qo = at::empty({T, H, d}, q.options());
    if (!k) {
      run(qo, {H * d, d}, nullptr, {0, 0});
      Py_INCREF(Py_None);
      return pair(THPVariable_Wrap(qo), Py_None);
    }
    const Tensor ko = at::empty({T, Hkv, d}, q.options());
    run(qo, {H * d, d}, &ko, {Hkv * d, d});
    return pair(qo, ko);
  }
  const Pair out(a[7]);
  const Tensor& qo = tensor(out.a, "out");
  const Tensor* ko = out.b == Py_None ? nullptr : &tensor(out.b, "out");
  TORCH_CHECK_VALUE(qo.sizes() == q.sizes() && !k == !ko && (!k || ko->sizes() == k->sizes()),
                    "out must give tensors of q's and k's shapes");
  run(qo, rows(qo, "out", &q), ko, ko ? rows(*ko, "out", &q) : attn_jvp_strides{0, 0});
  written(qo);
  if (ko) written(*ko);
  return given(out.a, out.b);
  END_HANDLE_TH_ERRORS
}

// cache_append(cache, k, v, starts, cached, page_table, cos, sin, layout)
PyObject* cache_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 9, "cache_append takes 9 arguments");
  const Cache cache(a[0]);
  const Tensor &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const attn_jvp_strides sk = rows(k, "k"), sv = rows(v, "v", &k);
  TORCH_CHECK_VALUE(v.sizes() == k.sizes(), "k and v must have the same shape");
  const int64_t T = k.size(0), heads = k.size(1), d = k.size(2);
  TORCH_CHECK_VALUE(cache.k->size(1) == heads && cache.k->size(3) == d,
                    "the cache must have the heads and head dim of k and v");
  const Tensor& cached = tensor(a[4], "cached");
  TORCH_CHECK_VALUE(cached.dim() == 1, "cached must be [B]");
  const int64_t B = cached.size(0);
  TORCH_CHECK_VALUE((a[6] == Py_None) == (a[7] == Py_None), "cos and sin go together");
  attn_jvp_rope_tables tables;
  const bool turn = a[6] != Py_None;
  if (turn) tables = rope_tables(a[6], a[7], a[8], k.device());
  const attn_jvp_cache desc = cache.checked(k.device());
  const attn_jvp_tokens shape = {T, heads, heads, d, dtype(k, true), 0.f};
  const int32_t* starts = int32s(a[3], "starts", k.device(), B + 1);
  const int32_t* old = int32s(a[4], "cached", k.device(), B);
  const Tensor& table = page_table(a[5], B, k.device());
  call("attn_jvp_cache_append", k.device(), [&](cudaStream_t stream) {
    return g_cache_append(&shape, k.data_ptr(), sk, v.data_ptr(), sv, &desc, B, starts, old,
                          static_cast<const int32_t*>(table.data_ptr()), table.size(1), table.stride(0),
                          turn ? &tables : nullptr, stream);
  });
  for (const Tensor* t : {cache.k, cache.v, cache.k_scale, cache.v_scale}) written(*t);
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

void check_out(const Tensor& o, const Tensor& lse, const Tensor& q, at::IntArrayRef lse_shape) {
  TORCH_CHECK_VALUE(o.sizes() == q.sizes() && o.scalar_type() == q.scalar_type() && o.device() == q.device() &&
                        o.is_contiguous() && lse.sizes() == lse_shape && lse.scalar_type() == at::kFloat &&
                        lse.device() == q.device() && lse.is_contiguous(),
                    "out must be contiguous: o ", q.sizes(), " of q's type, lse fp32 ", lse_shape,
                    ", on q's device");
}

// cache_attn(q, cache, seq_lens, page_table, causal, scale, max_len, out)
PyObject* cache_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 8, "cache_attn takes 8 arguments");
  const Tensor& q = tensor(a[0], "q");
  TORCH_CHECK_VALUE(q.dim() == 4 && q.is_cuda(), "q must be a CUDA tensor [B, n, H, d]");
  TORCH_CHECK_VALUE(q.stride(3) == 1, "the last dimension of q must be contiguous");
  const int64_t B = q.size(0), L = q.size(1), H = q.size(2), d = q.size(3);
  const Cache cache(a[1]);
  const int64_t Hkv = cache.k->size(1);
  TORCH_CHECK_VALUE(Hkv >= 1 && cache.k->size(3) == d && H % Hkv == 0,
                    "the cache must have q's head dim and a number of heads that divides q's");
  const attn_jvp_cache desc = cache.checked(q.device());
  const int32_t* lens = int32s(a[2], "seq_lens", q.device(), B);
  const Tensor& table = page_table(a[3], B, q.device());
  const bool causal = truth(a[4]);
  const attn_jvp_shape shape = {B, L, H, d, dtype(q, false), scale_of(a[5])};
  const int64_t max_len = PyLong_AsLongLong(a[6]);
  if (max_len == -1 && PyErr_Occurred()) throw python_error();
  int64_t most = table.size(1) * cache.k->size(2);
  if (max_len > 0 && max_len < most) most = max_len;
  const int64_t strides[3] = {q.stride(0), q.stride(1), q.stride(2)};
  auto run = [&](const Tensor& o, const Tensor& lse) {
    int64_t bytes;
    {
      const c10::cuda::CUDAGuard guard(q.device());
      bytes = g_workspace_bytes(&shape, Hkv, most);
    }
    TORCH_CHECK_VALUE(bytes >= 0, "bad shape, or no usable device");
    const Tensor work = bytes ? at::empty({bytes}, q.options().dtype(at::kByte)) : Tensor();
    call("attn_jvp_cache_attn", q.device(), [&](cudaStream_t stream) {
      return g_cache_attn(&shape, Hkv, q.data_ptr(), strides, &desc, lens,
                          static_cast<const int32_t*>(table.data_ptr()), table.size(1), table.stride(0),
                          max_len, causal, bytes ? work.data_ptr() : nullptr, bytes, o.data_ptr(),
                          static_cast<float*>(lse.data_ptr()), stream);
    });
  };
  if (a[7] == Py_None) {
    const Tensor o = at::empty({B, L, H, d}, q.options());
    const Tensor lse = at::empty({B, H, L}, q.options().dtype(at::kFloat));
    run(o, lse);
    return pair(o, lse);
  }
  const Pair out(a[7]);
  const Tensor &o = tensor(out.a, "out"), &lse = tensor(out.b, "out");
  check_out(o, lse, q, {B, H, L});
  run(o, lse);
  written(o);
  written(lse);
  return given(out.a, out.b);
  END_HANDLE_TH_ERRORS
}

// prompt_attn(q, k, v, starts, scale, out)
PyObject* prompt_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  TORCH_CHECK_VALUE(n == 6, "prompt_attn takes 6 arguments");
  const Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k"), &v = tensor(a[2], "v");
  const attn_jvp_strides sq = rows(q, "q"), sk = rows(k, "k", &q), sv = rows(v, "v", &q);
  const int64_t T = q.size(0), H = q.size(1), d = q.size(2), Hkv = k.size(1);
  TORCH_CHECK_VALUE(v.sizes() == k.sizes() && Hkv >= 1 && H % Hkv == 0,
                    "k and v must have the same number of heads, which divides q's");
  const Tensor& starts_t = tensor(a[3], "starts");
  TORCH_CHECK_VALUE(starts_t.dim() == 1 && starts_t.size(0) >= 1, "starts must be [B + 1]");
  const int64_t B = starts_t.size(0) - 1;
  const attn_jvp_tokens shape = {T, H, Hkv, d, dtype(q, false), scale_of(a[4])};
  const int32_t* starts = int32s(a[3], "starts", q.device(), B + 1);
  auto run = [&](const Tensor& o, const Tensor& lse) {
    call("attn_jvp_prompt_attn", q.device(), [&](cudaStream_t stream) {
      return g_prompt_attn(&shape, q.data_ptr(), sq, k.data_ptr(), sk, v.data_ptr(), sv, B, starts,
                           o.data_ptr(), static_cast<float*>(lse.data_ptr()), stream);
    });
  };
  if (a[5] == Py_None) {
    const Tensor o = at::empty({T, H, d}, q.options());
    const Tensor lse = at::empty({H, T}, q.options().dtype(at::kFloat));
    run(o, lse);
    return pair(o, lse);
  }
  const Pair out(a[5]);
  const Tensor &o = tensor(out.a, "out"), &lse = tensor(out.b, "out");
  check_out(o, lse, q, {H, T});
  run(o, lse);
  written(o);
  written(lse);
  return given(out.a, out.b);
  END_HANDLE_TH_ERRORS
}

// bind(check, rope_at, cache_append, cache_attn, cache_attn_workspace_bytes, prompt_attn):
// the error check and the functions' addresses.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return PyErr_Format(PyExc_ValueError, "bind takes 6 arguments");
  void* at[5];
  for (int i = 0; i < 5; ++i) {
    at[i] = PyLong_AsVoidPtr(a[i + 1]);
    if (!at[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "no address");
  }
  g_rope_at = reinterpret_cast<decltype(g_rope_at)>(at[0]);
  g_cache_append = reinterpret_cast<decltype(g_cache_append)>(at[1]);
  g_cache_attn = reinterpret_cast<decltype(g_cache_attn)>(at[2]);
  g_workspace_bytes = reinterpret_cast<decltype(g_workspace_bytes)>(at[3]);
  g_prompt_attn = reinterpret_cast<decltype(g_prompt_attn)>(at[4]);
  Py_INCREF(a[0]);
  Py_XSETREF(g_check, a[0]);
  Py_RETURN_NONE;
}

#define FAST(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(bind), FAST(rope_at), FAST(cache_append), FAST(cache_attn), FAST(prompt_attn),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_serving", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__serving() {
  PyObject* m = PyModule_Create(&module);
  // the torch and the Python that this was compiled against (build.py)
  if (m && PyModule_AddStringConstant(m, "built_for", AJVP_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
