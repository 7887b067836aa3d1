// prompt_bind.cpp -- marshalling of the prompt side's three calls from torch tensors to the C ABI of
// include/pkv.h (the functions of prompt.py, which documents them): checks of types, shapes,
// strides and devices, addresses, the output's and the workspace's memory, and nothing of the
// computation.  In C++ because the calls last a few microseconds for one token on the GPU and
// the same checks in Python with ctypes took 16 to 22 on the host.
//
// Every function returns its output tensor (or tensors), or the status of the C call as an int, for
// prompt.py to raise.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/pkv.h"

namespace {

struct Refused {
  PyObject* type;
  std::string message;
};

[[noreturn]] void value_error(std::string m) { throw Refused{PyExc_ValueError, std::move(m)}; }
[[noreturn]] void type_error(std::string m) { throw Refused{PyExc_TypeError, std::move(m)}; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// a tensor on the pool's device, or NULL for None
const at::Tensor* beside(PyObject* o, const char* name, int64_t dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name);
  if (t.get_device() != dev)
    value_error(std::string(name) + " is on " + t.device().str() + ", the cache on cuda:" + std::to_string(dev));
  return &t;
}
const at::Tensor& needed(PyObject* o, const char* name, int64_t dev) {
  const at::Tensor* t = beside(o, name, dev);
  if (!t) type_error(std::string(name) + " must be a tensor");
  return *t;
}

// the pool, on the current device
pkv_cache_desc pool_of(PyObject* ko, PyObject* vo, PyObject* so, int64_t* device) {
  const at::Tensor &k = tensor(ko, "k_cache"), &v = tensor(vo, "v_cache");
  if (!k.is_cuda()) value_error("k_cache and v_cache must be on one CUDA device");
  const int64_t dev = k.get_device();
  if (!v.is_cuda() || v.get_device() != dev) value_error("k_cache and v_cache must be on one CUDA device");
  if (dev != c10::cuda::current_device())
    value_error("tensors are on cuda:" + std::to_string(dev) + ", the current device is cuda:" +
                std::to_string(static_cast<int>(c10::cuda::current_device())));
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type())
    value_error("k_cache and v_cache must be [num_blocks, block_size, num_kv_heads, head_dim], of one shape and dtype");
  if (!k.is_contiguous() || !v.is_contiguous()) value_error("caches must be contiguous");
  const at::ScalarType st = k.scalar_type();
  const bool bf16 = st == at::kBFloat16;
  if (!bf16 && st != at::kByte && st != at::kFloat8_e4m3fn)
    type_error("the cache's dtype is neither bfloat16 nor E4M3 bytes");
  const at::Tensor* s = beside(so, "scales", dev);
  if (s && (s->scalar_type() != at::kFloat || s->dim() != 2 || s->size(0) != 2 || s->size(1) != k.size(2) ||
            !s->is_contiguous()))
    value_error("scales must be a contiguous float32 tensor [2, num_kv_heads]");
  for (int i = 1; i < 4; ++i)
    if (k.size(i) > 0x7fffffff) value_error("a dimension of the cache is too large");
  *device = dev;
  return pkv_cache_desc{k.data_ptr(),
                        v.data_ptr(),
                        k.size(0),
                        static_cast<int32_t>(k.size(1)),
                        static_cast<int32_t>(k.size(2)),
                        static_cast<int32_t>(k.size(3)),
                        bf16 ? PKV_KV_BF16 : PKV_KV_FP8_E4M3,
                        s ? static_cast<const float*>(s->data_ptr()) : nullptr};
}

// token stride of [T, heads, d] bf16 rows whose heads are contiguous (heads < 0: any number)
int64_t token_rows(const at::Tensor& t, const char* name, int64_t heads, int64_t d) {
  if (t.scalar_type() != at::kBFloat16) type_error(std::string(name) + " must be bfloat16");
  if (t.dim() != 3 || t.size(2) != d || (heads >= 0 && t.size(1) != heads))
    value_error(std::string(name) + " must be [num_tokens, heads, " + std::to_string(d) + "]" +
                (heads >= 0 ? " with " + std::to_string(heads) + " heads" : ""));
  const int64_t tokens = t.size(0), n = t.size(1);
  if (tokens > 0 && (t.stride(2) != 1 || (n > 1 && t.stride(1) != d)))
    value_error(std::string(name) + "'s heads must be contiguous (only the tokens may be strided)");
  return tokens > 1 ? t.stride(0) : n * d;
}

template <typename T>
T* vector(const at::Tensor* t, const char* name, at::ScalarType type, int64_t n) {
  if (!t) return nullptr;
  if (t->scalar_type() != type || t->dim() != 1 || t->size(0) != n || !t->is_contiguous())
    value_error(std::string(name) + " must be a contiguous " + c10::toString(type) + " tensor [" + std::to_string(n) +
                "]");
  return static_cast<T*>(t->data_ptr());
}

const int32_t* tables_of(const at::Tensor& t, int32_t* batch, int32_t* blocks) {
  if (t.scalar_type() != at::kInt || t.dim() != 2 || !t.is_contiguous())
    type_error("block_tables must be a contiguous int32 tensor [B, max_blocks]");
  if (t.size(0) > 0x7fffffff || t.size(1) > 0x7fffffff) value_error("block_tables is too large");
  *batch = static_cast<int32_t>(t.size(0));
  *blocks = static_cast<int32_t>(t.size(1));
  return static_cast<const int32_t*>(t.data_ptr());
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be an integer");
  }
  return v;
}
int32_t int32(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) value_error(std::string(name) + " does not fit in 32 bits");
  return static_cast<int32_t>(v);
}
float number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    type_error(std::string(name) + " must be a number");
  }
  return static_cast<float>(v);
}
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    type_error(std::string(name) + " must be true or false");
  }
  return v == 1;
}

void arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(got));
}

pkv_stream_t current_stream(int64_t dev) {
  return reinterpret_cast<pkv_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, int64_t dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
}

// q, k, v, positions, slot_mapping, k_cache, v_cache, q_out, q_weight, k_weight, eps, inv_freq,
// interleaved, rope_scale, scales
PyObject* append(PyObject* const* a) {
  int64_t dev;
  const pkv_cache_desc cache = pool_of(a[5], a[6], a[14], &dev);
  const int64_t d = cache.head_dim, hkv = cache.num_kv_heads;
  const at::Tensor &q = needed(a[0], "q", dev), &k = needed(a[1], "k", dev), &v = needed(a[2], "v", dev);
  pkv_rope_append_desc x{};
  x.q_stride = token_rows(q, "q", -1, d);
  x.k_stride = token_rows(k, "k", hkv, d);
  x.v_stride = token_rows(v, "v", hkv, d);
  const int64_t tokens = q.size(0), hq = q.size(1);
  if (k.size(0) != tokens || v.size(0) != tokens) value_error("q, k and v must have the same number of tokens");
  if (hq > 0x7fffffff) value_error("too many heads");
  x.q = q.data_ptr();
  x.k = k.data_ptr();
  x.v = v.data_ptr();
  const at::Tensor& slots = needed(a[4], "slot_mapping", dev);
  x.slot_mapping = vector<const int64_t>(&slots, "slot_mapping", at::kLong, tokens);
  x.num_tokens = tokens;
  x.num_q_heads = static_cast<int32_t>(hq);
  x.q_weight = vector<const void>(beside(a[8], "q_weight", dev), "q_weight", at::kBFloat16, d);
  x.k_weight = vector<const void>(beside(a[9], "k_weight", dev), "k_weight", at::kBFloat16, d);
  x.eps = number(a[10], "eps");
  const at::Tensor* freq = beside(a[11], "inv_freq", dev);
  const at::Tensor* positions = beside(a[3], "positions", dev);
  if (freq) {
    const int64_t half = freq->dim() == 1 ? freq->size(0) : 0;
    if (half > 0x3fffffff) value_error("inv_freq is too long");
    x.inv_freq = vector<const double>(freq, "inv_freq", at::kDouble, half);
    if (!positions) value_error("a rotation needs positions");
    x.positions = vector<const int32_t>(positions, "positions", at::kInt, tokens);
    x.rotary_dim = static_cast<int32_t>(2 * half);
  }
  x.interleaved = truth(a[12], "interleaved");
  x.rope_scale = number(a[13], "rope_scale");
  const at::Tensor* given = beside(a[7], "q_out", dev);
  at::Tensor out = given ? *given : fresh({tokens, hq, d}, at::kBFloat16, dev);
  x.q_out_stride = token_rows(out, "q_out", hq, d);
  if (out.size(0) != tokens) value_error("q_out must have q's shape");
  x.q_out = out.data_ptr();
  pkv_status st;
  const pkv_stream_t stream = current_stream(dev);
  Py_BEGIN_ALLOW_THREADS;
  st = pkv_qk_norm_rope_append(&cache, &x, stream);
  Py_END_ALLOW_THREADS;
  return st == PKV_OK ? THPVariable_Wrap(std::move(out)) : PyLong_FromLong(st);
}

// q, q_indptr, k_cache, v_cache, block_tables, context_lens, softmax_scale, out, causal, lse, scales,
// max_context_len, workspace
PyObject* prefill(PyObject* const* a) {
  int64_t dev;
  const pkv_cache_desc cache = pool_of(a[2], a[3], a[10], &dev);
  const int64_t d = cache.head_dim;
  const at::Tensor& q = needed(a[0], "q", dev);
  const int64_t q_stride = token_rows(q, "q", -1, d);
  const int64_t tokens = q.size(0), hq = q.size(1);
  if (tokens > 0x7fffffff || hq > 0x7fffffff) value_error("q is too large");
  int32_t batch, blocks;
  const int32_t* tables = tables_of(needed(a[4], "block_tables", dev), &batch, &blocks);
  const int32_t* lens =
      vector<const int32_t>(&needed(a[5], "context_lens", dev), "context_lens", at::kInt, batch);
  const int32_t* indptr =
      vector<const int32_t>(&needed(a[1], "q_indptr", dev), "q_indptr", at::kInt, static_cast<int64_t>(batch) + 1);
  const int64_t most = static_cast<int64_t>(blocks) * cache.block_size;
  const int32_t max_len =
      a[11] == Py_None ? static_cast<int32_t>(std::min<int64_t>(most, INT32_MAX)) : int32(a[11], "max_context_len");
  const at::Tensor* given = beside(a[7], "out", dev);
  at::Tensor out = given ? *given : fresh({tokens, hq, d}, at::kBFloat16, dev);
  if (given && (out.scalar_type() != at::kBFloat16 || out.sizes() != q.sizes() || !out.is_contiguous()))
    value_error("out must be a contiguous bfloat16 tensor [T, Hq, D]");
  const at::Tensor* lse = beside(a[9], "lse", dev);
  if (lse && (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != tokens || lse->size(1) != hq ||
              !lse->is_contiguous()))
    value_error("lse must be a contiguous float32 tensor [T, Hq]");
  const int32_t t32 = static_cast<int32_t>(tokens), hq32 = static_cast<int32_t>(hq);
  // a workspace of the call's own, unless one is given: calls on several streams and captured
  // graphs share none
  const size_t need = batch > 0 && tokens > 0 ? pkv_prefill_workspace_size(batch, t32, hq32, cache.num_kv_heads,
                                                                           cache.head_dim, max_len)
                                              : 0;
  const at::Tensor* ws = beside(a[12], "workspace", dev);
  // (its size is counted in elements, which an expanded tensor shares)
  if (ws && !ws->is_contiguous()) value_error("workspace must be contiguous");
  at::Tensor own;
  if (need > 0 && !ws) {
    own = fresh({static_cast<int64_t>(need)}, at::kByte, dev);
    ws = &own;
  }
  const float scale = number(a[6], "softmax_scale");
  const int32_t causal = truth(a[8], "causal");
  void* const ws_ptr = need > 0 ? ws->data_ptr() : nullptr;
  const size_t ws_bytes = need > 0 ? ws->numel() * ws->element_size() : 0;
  void *const qp = q.data_ptr(), *const op = out.data_ptr();
  float* const lp = lse ? static_cast<float*>(lse->data_ptr()) : nullptr;
  pkv_status st;
  const pkv_stream_t stream = current_stream(dev);
  Py_BEGIN_ALLOW_THREADS;
  st = pkv_paged_prefill_attention(&cache, qp, q_stride, indptr, t32, tables, blocks, lens, batch, hq32, max_len,
                                   causal, scale, op, lp, ws_ptr, ws_bytes, stream);
  Py_END_ALLOW_THREADS;
  return st == PKV_OK ? THPVariable_Wrap(std::move(out)) : PyLong_FromLong(st);
}

// k_cache, v_cache, block_tables, kv_indptr, k_out, v_out, starts, scales
PyObject* gather(PyObject* const* a) {
  int64_t dev;
  const pkv_cache_desc cache = pool_of(a[0], a[1], a[7], &dev);
  int32_t batch, blocks;
  const int32_t* tables = tables_of(needed(a[2], "block_tables", dev), &batch, &blocks);
  const int32_t* indptr =
      vector<const int32_t>(&needed(a[3], "kv_indptr", dev), "kv_indptr", at::kInt, static_cast<int64_t>(batch) + 1);
  const int32_t* starts = vector<const int32_t>(beside(a[6], "starts", dev), "starts", at::kInt, batch);
  const at::Tensor &k = needed(a[4], "k_out", dev), &v = needed(a[5], "v_out", dev);
  const at::ScalarType type = k.scalar_type();
  if (v.scalar_type() != type || (type != at::kBFloat16 && type != at::kFloat))
    type_error("k_out and v_out must be both bfloat16 or both float32");
  if (k.dim() != 3 || k.size(1) != cache.num_kv_heads || k.size(2) != cache.head_dim || v.sizes() != k.sizes() ||
      !k.is_contiguous() || !v.is_contiguous())
    value_error("k_out and v_out must be contiguous [rows, num_kv_heads, head_dim]");
  void *const kp = k.data_ptr(), *const vp = v.data_ptr();
  const int64_t rows = k.size(0);
  pkv_status st;
  const pkv_stream_t stream = current_stream(dev);
  Py_BEGIN_ALLOW_THREADS;
  st = pkv_paged_kv_gather(&cache, tables, blocks, indptr, starts, batch, rows, kp, vp,
                           type == at::kFloat ? PKV_OUT_FP32 : PKV_OUT_BF16, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(st);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    arguments(n, N);
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.message.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<append, 15>("append"), method<prefill, 13>("prefill"), method<gather, 8>("gather"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkv_prompt", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__pkv_prompt() { return PyModule_Create(&module); }
