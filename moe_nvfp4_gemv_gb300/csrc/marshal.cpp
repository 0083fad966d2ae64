// marshal.cpp -- argument checks and marshalling of the decode step's
// operators (a CPython extension module on torch's tensors; the operators are
// the C entry points of fp4gemv_decode.h, whose addresses the binding hands
// over once).
//
// Why not ctypes, as for the products: these calls are short.  Reading three to
// seven tensors' types, shapes and addresses as Python objects and converting
// 14 to 19 arguments took longer than the launch itself (2.1 us) and, for a few
// tokens, than the kernel.  Host time of a call with ctypes and so, us:
// moe_route 6.6 / 3.1, token_logprobs 8.0 / 3.7, attend 8.0 / 3.4, append 8.0 /
// 3.2; a token's routing one call after another 6.1 / 2.8.
//
// Every function takes its arguments by position, raises ValueError for what a
// tensor may not be, and returns the status of the C call (0 where there is
// nothing to do).  No C++ exception leaves a function.
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <exception>

#include "fp4gemv_decode.h"

namespace {

decltype(&fp4gemv_kv_append) g_append;
decltype(&fp4gemv_kv_attention) g_attention;
decltype(&fp4gemv_kv_attention_sinks) g_attention_sinks;
decltype(&fp4gemv_kv_attention_shared) g_attention_shared;
decltype(&fp4gemv_kv_read) g_read;
decltype(&fp4gemv_add_norm) g_add_norm;
decltype(&fp4gemv_moe_route) g_route;
decltype(&fp4gemv_token_logprobs) g_logprobs;

struct Raised {};  // a Python error is set

template <class... A>
[[noreturn]] void refuse(const char* format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %.100s", name, Py_TYPE(o)->tp_name);
    throw Raised();
  }
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
int int32(PyObject* o) {
  const int64_t v = integer(o);
  if (v < INT_MIN || v > INT_MAX) refuse("%lld is out of range", static_cast<long long>(v));
  return static_cast<int>(v);
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
int flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v;
}
const void* address(const at::Tensor& t) { return t.const_data_ptr(); }
template <class T>
T* address_as(const at::Tensor& t) {
  return static_cast<T*>(const_cast<void*>(t.const_data_ptr()));
}
// a contiguous tensor of the type on CUDA device `index`
bool plain(const at::Tensor& t, at::ScalarType type, int64_t index) {
  return t.scalar_type() == type && t.is_cuda() && t.get_device() == index && t.is_contiguous();
}
int half_code(const at::Tensor& t) {  // -1: neither bf16 nor f16
  return t.scalar_type() == at::kBFloat16 ? FP4GEMV_BF16 : t.scalar_type() == at::kHalf ? FP4GEMV_F16 : -1;
}
int type_code(const at::Tensor& t) {  // -1: none of bf16, f16, f32
  return t.scalar_type() == at::kFloat ? static_cast<int>(FP4GEMV_F32) : half_code(t);
}
bool shaped(const at::Tensor& t, int64_t rows) { return t.dim() == 1 && t.size(0) == rows; }
bool shaped(const at::Tensor& t, int64_t rows, int64_t columns) {
  return t.dim() == 2 && t.size(0) == rows && t.size(1) == columns;
}
cudaStream_t stream_of(int64_t index) {
  return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
}
// `body` with what it throws turned into Python errors; its status.
template <class Body>
PyObject* guarded(Py_ssize_t got, Py_ssize_t want, Body body) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments instead of %zd", got, want);
    return nullptr;
  }
  try {
    return PyLong_FromLong(body());
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
// `call` without the interpreter's lock
template <class Call>
int unlocked(Call call) {
  PyThreadState* const state = PyEval_SaveThread();
  const int status = call();
  PyEval_RestoreThread(state);
  return status;
}

// block_table and seq_lens
void sequences(const at::Tensor& table, const at::Tensor& lens, int64_t index, int* B, int* max_blocks) {
  if (table.dim() != 2 || !plain(table, at::kInt, index))
    refuse("block_table must be a contiguous int32 [B, max_blocks] tensor on the cache's device");
  const int64_t b = table.size(0), m = table.size(1);
  if (b > INT_MAX || m > INT_MAX) refuse("block_table is too large");
  if (lens.numel() != b || !plain(lens, at::kInt, index))
    refuse("seq_lens must be a contiguous int32 [%d] tensor on the cache's device", static_cast<int>(b));
  *B = static_cast<int>(b);
  *max_blocks = static_cast<int>(m);
}

// kv_append(cache, device, kv_heads, head_dim, k, v, block_table, seq_lens, cu_new, pdl)
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> int {
    const auto* cache = reinterpret_cast<const fp4gemv_kv_cache*>(integer(a[0]));
    const int64_t index = integer(a[1]), H = integer(a[2]), D = integer(a[3]);
    const at::Tensor &k = tensor(a[4], "k"), &v = tensor(a[5], "v"), &table = tensor(a[6], "block_table"),
                     &lens = tensor(a[7], "seq_lens");
    int B, max_blocks;
    sequences(table, lens, index, &B, &max_blocks);
    const int dtype = half_code(k);
    auto fits = [&](const at::Tensor& t) {
      return t.scalar_type() == k.scalar_type() && t.dim() == 3 && t.size(1) == H && t.size(2) == D && t.is_cuda() &&
             t.get_device() == index && t.stride(2) == 1 && (H == 1 || t.stride(1) == D);
    };
    if (dtype < 0 || !fits(k) || !fits(v) || v.size(0) != k.size(0))
      refuse("k and v must be bf16 or f16 [T, %d, %d] tensors of one type on the cache's device with contiguous heads",
             static_cast<int>(H), static_cast<int>(D));
    const int64_t T = k.size(0);
    const int32_t* cu = nullptr;
    if (a[8] != Py_None) {
      const at::Tensor& t = tensor(a[8], "cu_new");
      if (t.numel() != static_cast<int64_t>(B) + 1 || !plain(t, at::kInt, index))
        refuse("cu_new must be a contiguous int32 [%d] tensor on the cache's device", B + 1);
      cu = address_as<int32_t>(t);
    }
    const int pdl = flag(a[9]);
    if (T == 0) return FP4GEMV_OK;
    if (B == 0) refuse("new tokens for no sequence");
    if (T > INT_MAX) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
    const int64_t ldk = T > 1 ? k.stride(0) : H * D, ldv = T > 1 ? v.stride(0) : H * D;
    const void *pk = address(k), *pv = address(v);
    const int32_t *pt = address_as<int32_t>(table), *pl = address_as<int32_t>(lens);
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(index));
    const cudaStream_t stream = stream_of(index);
    return unlocked([&] {
      return g_append(cache, pk, ldk, pv, ldv, dtype, static_cast<int>(T), cu, pt, max_blocks, pl, B, pdl, stream);
    });
  });
}

// kv_read(cache, device, kv_heads, head_dim, block_table, seq_lens, cu, k, v, pdl)
PyObject* kv_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> int {
    const auto* cache = reinterpret_cast<const fp4gemv_kv_cache*>(integer(a[0]));
    const int64_t index = integer(a[1]), H = integer(a[2]), D = integer(a[3]);
    const at::Tensor &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "seq_lens"), &k = tensor(a[7], "k"),
                     &v = tensor(a[8], "v");
    int B, max_blocks;
    sequences(table, lens, index, &B, &max_blocks);
    const int dtype = type_code(k);
    auto fits = [&](const at::Tensor& t) {
      return t.scalar_type() == k.scalar_type() && t.dim() == 3 && t.size(1) == H && t.size(2) == D && t.is_cuda() &&
             t.get_device() == index && t.stride(2) == 1 && (H == 1 || t.stride(1) == D);
    };
    if (dtype < 0 || !fits(k) || !fits(v) || v.size(0) != k.size(0))
      refuse("k and v must be bf16, f16 or fp32 [T, %d, %d] tensors of one type on the cache's device with contiguous heads",
             static_cast<int>(H), static_cast<int>(D));
    const int64_t T = k.size(0);
    const int32_t* cu = nullptr;
    if (a[6] != Py_None) {
      const at::Tensor& t = tensor(a[6], "cu");
      if (t.numel() != static_cast<int64_t>(B) + 1 || !plain(t, at::kInt, index))
        refuse("cu must be a contiguous int32 [%d] tensor on the cache's device", B + 1);
      cu = address_as<int32_t>(t);
    }
    const int pdl = flag(a[9]);
    if (T == 0) return FP4GEMV_OK;
    if (B == 0) refuse("tokens of no sequence");
    if (T > INT_MAX) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
    const int64_t ldk = T > 1 ? k.stride(0) : H * D, ldv = T > 1 ? v.stride(0) : H * D;
    void *pk = address_as<void>(k), *pv = address_as<void>(v);
    const int32_t *pt = address_as<int32_t>(table), *pl = address_as<int32_t>(lens);
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(index));
    const cudaStream_t stream = stream_of(index);
    return unlocked([&] {
      return g_read(cache, pk, ldk, pv, ldv, dtype, static_cast<int>(T), cu, pt, max_blocks, pl, B, pdl, stream);
    });
  });
}

// add_norm(x, y, weight, post_weight, gate, gate_sigmoid, scale, eps, weight_offset, residual, out, pdl)
PyObject* add_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const at::Tensor &x = tensor(a[0], "x"), &weight = tensor(a[2], "weight"), &out = tensor(a[10], "out");
    const bool block = a[1] != Py_None;
    if (x.dim() != 2 || !x.is_cuda() || x.stride(1) != 1) refuse("x must be a 2-D CUDA tensor with unit inner stride");
    const int64_t M = x.size(0), H = x.size(1), index = x.get_device();
    const at::ScalarType half = out.scalar_type();
    const int dtype = half_code(out), x_type = type_code(x);
    auto rows = [&](const at::Tensor& t) {
      return t.dim() == 2 && t.size(0) == M && t.size(1) == H && t.stride(1) == 1 && t.is_cuda() && t.get_device() == index;
    };
    auto stride = [&](const at::Tensor& t) { return M > 1 ? t.stride(0) : H; };
    if (dtype < 0 || !rows(out)) refuse("out must be a bf16 or f16 tensor of x's shape and device with unit inner stride");
    auto kind = [&](const at::Tensor& t) { return t.scalar_type() == half || t.scalar_type() == at::kFloat; };
    if (!kind(x)) refuse("x must be of out's type or fp32");
    auto is_weight = [&](const at::Tensor& t) { return shaped(t, H) && kind(t) && plain(t, t.scalar_type(), index); };
    if (!is_weight(weight)) refuse("weight must be a contiguous [%lld] tensor of out's type or fp32 on x's device", static_cast<long long>(H));
    const void *py = nullptr, *post = nullptr, *gate = nullptr;
    int64_t ldy = H, ldg = 0, ldr = H;
    int gate_type = dtype, gate_kind = FP4GEMV_GATE_CHANNEL;
    void* pr = nullptr;
    if (block) {
      const at::Tensor &y = tensor(a[1], "y"), &residual = tensor(a[9], "residual");
      if (y.scalar_type() != half || !rows(y)) refuse("y must be a tensor of out's type and x's shape with unit inner stride");
      if (residual.scalar_type() != x.scalar_type() || !rows(residual))
        refuse("residual must be a tensor of x's type and shape with unit inner stride");
      py = address(y);
      ldy = stride(y);
      pr = address_as<void>(residual);
      ldr = stride(residual);
    }
    if (a[3] != Py_None) {
      const at::Tensor& t = tensor(a[3], "post_weight");
      if (!is_weight(t) || t.scalar_type() != weight.scalar_type()) refuse("post_weight must be a tensor like weight");
      post = address(t);
    }
    if (a[4] != Py_None) {
      const at::Tensor& t = tensor(a[4], "gate");
      const bool channel = t.dim() == 1 && t.size(0) == H && (H == 1 || t.stride(0) == 1);
      const bool token = t.dim() == 2 && t.size(0) == M && t.size(1) == 1 && H != 1;
      if (!kind(t) || !t.is_cuda() || t.get_device() != index || !(channel || token || rows(t)))
        refuse("gate must be an [H], [M, H] or [M, 1] tensor of out's type or fp32 on x's device with unit inner stride");
      gate = address(t);
      gate_type = type_code(t);
      gate_kind = token ? FP4GEMV_GATE_TOKEN : FP4GEMV_GATE_CHANNEL;
      ldg = channel ? 0 : token ? (M > 1 ? t.stride(0) : 0) : stride(t);
    }
    if (!block && (post || gate)) refuse("post_weight and gate need y");
    const int sigmoid = flag(a[5]), pdl = flag(a[11]);
    const float scale = static_cast<float>(real(a[6])), eps = static_cast<float>(real(a[7])),
                offset = static_cast<float>(real(a[8]));
    if (M == 0) return FP4GEMV_OK;
    if (M > INT_MAX || H > INT_MAX) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
    const void *px = address(x), *pw = address(weight);
    const int w_type = type_code(weight);
    const int64_t ldx = stride(x), ldo = stride(out);
    void* po = address_as<void>(out);
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(index));
    const cudaStream_t stream = stream_of(index);
    return unlocked([&] {
      return g_add_norm(px, ldx, x_type, py, ldy, dtype, pw, post, w_type, gate, ldg, gate_type, gate_kind, sigmoid, scale,
                        eps, offset, pr, ldr, po, ldo, static_cast<int>(M), static_cast<int>(H), pdl, stream);
    });
  });
}

// The one stride between tokens of a [B, n, heads, dim] tensor.
int64_t token_stride(const at::Tensor& t, const char* name) {
  const int64_t B = t.size(0), n = t.size(1), heads = t.size(2), dim = t.size(3);
  if (t.is_contiguous()) return heads * dim;
  if (t.stride(3) != 1 || (t.stride(2) != dim && heads > 1) || (n > 1 && B > 1 && t.stride(0) != n * t.stride(1)))
    refuse("%s must have contiguous heads and one stride between all its tokens", name);
  return n > 1 ? t.stride(1) : B > 1 ? t.stride(0) : heads * dim;
}

// The arguments of an attention call as the C calls take them; empty: there is nothing to do.
struct Attention {
  const fp4gemv_kv_cache* cache;
  const void* q;
  int64_t ldq, ldo, index;
  int dtype, heads, q_len, B, max_blocks, window, pdl;
  const int32_t *table, *lens;
  float sm_scale;
  void *out, *workspace;
  float* lse;
  size_t bytes;
  bool empty, large;
};
// a: cache, device, head_dim, q, block_table, seq_lens, sm_scale, window, out, lse, workspace, pdl
Attention attention_of(PyObject* const* a) {
  const auto* cache = reinterpret_cast<const fp4gemv_kv_cache*>(integer(a[0]));
  const int64_t index = integer(a[1]), D = integer(a[2]);
  const at::Tensor &q = tensor(a[3], "q"), &table = tensor(a[4], "block_table"), &lens = tensor(a[5], "seq_lens"),
                   &out = tensor(a[8], "out"), &workspace = tensor(a[10], "workspace");
  int B, max_blocks;
  sequences(table, lens, index, &B, &max_blocks);
  const int dtype = half_code(q);
  if (dtype < 0 || q.dim() != 4 || q.size(0) != B || q.size(3) != D || !q.is_cuda() || q.get_device() != index)
    refuse("q must be a bf16 or f16 [%d, q_len, heads, %d] tensor on the cache's device", B, static_cast<int>(D));
  if (out.scalar_type() != q.scalar_type() || out.sizes() != q.sizes() || !out.is_cuda() || out.get_device() != index)
    refuse("out must have q's shape, type and device");
  const int64_t ldq = token_stride(q, "q"), ldo = token_stride(out, "out"), q_len = q.size(1), heads = q.size(2);
  float* lse = nullptr;
  if (a[9] != Py_None) {
    const at::Tensor& t = tensor(a[9], "lse");
    if (t.numel() != B * q_len * heads || !plain(t, at::kFloat, index))
      refuse("lse must be a contiguous fp32 [%d, %d, %d] tensor on the cache's device", B, static_cast<int>(q_len),
             static_cast<int>(heads));
    lse = address_as<float>(t);
  }
  if (!workspace.is_cuda() || workspace.get_device() != index || !workspace.is_contiguous())
    refuse("workspace must be a contiguous tensor on the cache's device");
  const float sm_scale = static_cast<float>(real(a[6]));
  const int window = int32(a[7]), pdl = flag(a[11]);
  const void* pq = address(q);
  void *po = address_as<void>(out), *pw = address_as<void>(workspace);
  const int32_t *pt = address_as<int32_t>(table), *pl = address_as<int32_t>(lens);
  const size_t bytes = workspace.nbytes();
  return {cache, pq, ldq, ldo, index, dtype, static_cast<int>(heads), static_cast<int>(q_len), B, max_blocks, window, pdl,
          pt, pl, sm_scale, po, pw, lse, bytes, B == 0, q_len > INT_MAX || heads > INT_MAX};
}

// kv_attention(cache, device, head_dim, q, block_table, seq_lens, sm_scale, window, out, lse, workspace, pdl)
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const Attention c = attention_of(a);
    if (c.empty) return FP4GEMV_OK;
    if (c.large) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.index));
    const cudaStream_t stream = stream_of(c.index);
    return unlocked([&] {
      return g_attention(c.cache, c.q, c.ldq, c.dtype, c.heads, c.q_len, c.table, c.max_blocks, c.lens, c.B, c.sm_scale,
                         c.window, c.out, c.ldo, c.lse, c.workspace, c.bytes, c.pdl, stream);
    });
  });
}

// kv_attention_sinks(kv_attention's, sinks)
PyObject* kv_attention_sinks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> int {
    const Attention c = attention_of(a);
    const int sinks = int32(a[12]);
    if (c.empty) return FP4GEMV_OK;
    if (c.large) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.index));
    const cudaStream_t stream = stream_of(c.index);
    return unlocked([&] {
      return g_attention_sinks(c.cache, c.q, c.ldq, c.dtype, c.heads, c.q_len, c.table, c.max_blocks, c.lens, c.B,
                               c.sm_scale, c.window, sinks, c.out, c.ldo, c.lse, c.workspace, c.bytes, c.pdl, stream);
    });
  });
}

// kv_attention_shared(kv_attention's, prefix_len, scratch, always); the window is none
PyObject* kv_attention_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> int {
    const Attention c = attention_of(a);
    const at::Tensor &prefix = tensor(a[12], "prefix_len"), &scratch = tensor(a[13], "scratch");
    if (prefix.numel() != 1 || !plain(prefix, at::kInt, c.index))
      refuse("prefix_len must be an int32 [1] tensor on the cache's device");
    if (!scratch.is_cuda() || scratch.get_device() != c.index || !scratch.is_contiguous())
      refuse("scratch must be a contiguous tensor on the cache's device");
    const int always = flag(a[14]);
    if (c.window != 0) refuse("no window together with a shared beginning");
    if (c.empty) return FP4GEMV_OK;
    if (c.large) return FP4GEMV_ERR_UNSUPPORTED_SHAPE;
    const int32_t* pp = address_as<int32_t>(prefix);
    void* ps = address_as<void>(scratch);
    const size_t scratch_bytes = scratch.nbytes();
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(c.index));
    const cudaStream_t stream = stream_of(c.index);
    return unlocked([&] {
      return g_attention_shared(c.cache, c.q, c.ldq, c.dtype, c.heads, c.q_len, c.table, c.max_blocks, c.lens, c.B, pp,
                                c.sm_scale, c.out, c.ldo, c.lse, c.workspace, c.bytes, ps, scratch_bytes, always, c.pdl,
                                stream);
    });
  });
}

// The logits' type, rows, row length and row stride.
struct Logits {
  int dtype;
  int64_t rows, width, ld, index;
};
Logits logits_of(const at::Tensor& t) {
  Logits l;
  l.dtype = type_code(t);
  if (l.dtype < 0 || t.dim() != 2 || !t.is_cuda() || t.stride(1) != 1)
    refuse("logits must be a 2-D bf16, f16 or fp32 CUDA tensor with unit inner stride");
  l.rows = t.size(0);
  l.width = t.size(1);
  l.ld = l.rows > 1 ? t.stride(0) : l.width;
  l.index = t.get_device();
  if (l.rows > INT_MAX || l.width > INT_MAX) refuse("logits are too large");
  return l;
}

// moe_route(logits, topk, scores, bias, n_group, topk_group, group_top, renormalize, scale, ids, weights, pdl)
PyObject* moe_route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> int {
    const at::Tensor& logits = tensor(a[0], "logits");
    const Logits l = logits_of(logits);
    const int topk = int32(a[1]);
    int scores;
    auto is = [&](const char* name) { return PyUnicode_Check(a[2]) && PyUnicode_CompareWithASCIIString(a[2], name) == 0; };
    if (is("softmax")) scores = FP4GEMV_ROUTE_SOFTMAX;
    else if (is("sigmoid")) scores = FP4GEMV_ROUTE_SIGMOID;
    else refuse("scores must be 'softmax' or 'sigmoid', not %R", a[2]);
    const float* bias = nullptr;
    if (a[3] != Py_None) {
      const at::Tensor& t = tensor(a[3], "bias");
      if (!shaped(t, l.width) || !plain(t, at::kFloat, l.index))
        refuse("bias must be a contiguous fp32 [%d] tensor on the logits' device", static_cast<int>(l.width));
      bias = address_as<float>(t);
    }
    const int n_group = int32(a[4]), topk_group = int32(a[5]), group_top = int32(a[6]), renormalize = flag(a[7]);
    const float scale = static_cast<float>(real(a[8]));
    const at::Tensor &ids = tensor(a[9], "ids"), &weights = tensor(a[10], "weights");
    if (!shaped(ids, l.rows, topk) || !plain(ids, at::kInt, l.index))
      refuse("ids must be a contiguous int32 [%d, %d] tensor on the logits' device", static_cast<int>(l.rows), topk);
    if (!shaped(weights, l.rows, topk) || !plain(weights, at::kFloat, l.index))
      refuse("weights must be a contiguous fp32 [%d, %d] tensor on the logits' device", static_cast<int>(l.rows), topk);
    const int pdl = flag(a[11]);
    if (l.rows == 0) return FP4GEMV_OK;
    const void* px = address(logits);
    int32_t* pi = address_as<int32_t>(ids);
    float* pw = address_as<float>(weights);
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(l.index));
    const cudaStream_t stream = stream_of(l.index);
    return unlocked([&] {
      return g_route(px, l.ld, l.dtype, static_cast<int>(l.rows), static_cast<int>(l.width), topk, scores, bias, n_group,
                     topk_group, group_top, renormalize, scale, pi, pw, pdl, stream);
    });
  });
}

// token_logprobs(logits, tokens, top_n, temperature, logprob, rank, entropy, top_ids, top_logprobs, pdl)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> int {
    const at::Tensor &logits = tensor(a[0], "logits"), &tokens = tensor(a[1], "tokens");
    const Logits l = logits_of(logits);
    if (!shaped(tokens, l.rows) || !plain(tokens, at::kInt, l.index))
      refuse("tokens must be a contiguous int32 [%d] tensor on the logits' device", static_cast<int>(l.rows));
    const int top_n = int32(a[2]);
    const double temperature = real(a[3]);
    if (!(temperature > 0)) refuse("temperature must be positive");
    const at::Tensor &logprob = tensor(a[4], "logprob"), &rank = tensor(a[5], "rank"),
                     &entropy = tensor(a[6], "entropy"), &top_ids = tensor(a[7], "top_ids"),
                     &top_logprobs = tensor(a[8], "top_logprobs");
    if (!shaped(logprob, l.rows) || !shaped(rank, l.rows) || !shaped(entropy, l.rows) ||
        !shaped(top_ids, l.rows, top_n) || !shaped(top_logprobs, l.rows, top_n) ||
        !plain(logprob, at::kFloat, l.index) || !plain(rank, at::kInt, l.index) || !plain(entropy, at::kFloat, l.index) || !plain(top_ids, at::kInt, l.index) ||
        !plain(top_logprobs, at::kFloat, l.index))
      refuse("out must hold contiguous logprob fp32 [T], rank int32 [T], entropy fp32 [T], top_ids int32 [T, top_n] and "
             "top_logprobs fp32 [T, top_n] on the logits' device");
    const int pdl = flag(a[9]);
    if (l.rows == 0) return FP4GEMV_OK;
    const void* px = address(logits);
    const int32_t* pt = address_as<int32_t>(tokens);
    float *plp = address_as<float>(logprob), *pe = address_as<float>(entropy);
    int32_t* pr = address_as<int32_t>(rank);
    int32_t* pti = top_n > 0 ? address_as<int32_t>(top_ids) : nullptr;
    float* ptl = top_n > 0 ? address_as<float>(top_logprobs) : nullptr;
    const c10::cuda::CUDAGuard on(static_cast<c10::DeviceIndex>(l.index));
    const cudaStream_t stream = stream_of(l.index);
    return unlocked([&] {
      return g_logprobs(px, l.ld, l.dtype, static_cast<int>(l.rows), static_cast<int>(l.width), pt,
                        static_cast<float>(1.0 / temperature), top_n, plp, pr, pe, pti, ptl, pdl, stream);
    });
  });
}

// bind(kv_append, kv_attention, moe_route, token_logprobs): the C entry points' addresses
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> int {
    g_append = reinterpret_cast<decltype(g_append)>(integer(a[0]));
    g_attention = reinterpret_cast<decltype(g_attention)>(integer(a[1]));
    g_route = reinterpret_cast<decltype(g_route)>(integer(a[2]));
    g_logprobs = reinterpret_cast<decltype(g_logprobs)>(integer(a[3]));
    return 0;
  });
}

// bind_more(kv_read, add_norm, kv_attention_sinks, kv_attention_shared): the others'
PyObject* bind_more(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> int {
    g_read = reinterpret_cast<decltype(g_read)>(integer(a[0]));
    g_add_norm = reinterpret_cast<decltype(g_add_norm)>(integer(a[1]));
    g_attention_sinks = reinterpret_cast<decltype(g_attention_sinks)>(integer(a[2]));
    g_attention_shared = reinterpret_cast<decltype(g_attention_shared)>(integer(a[3]));
    return 0;
  });
}

template <PyObject* (*kFunction)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(kFunction)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<bind>("bind"),           method<kv_append>("kv_append"),
                           method<kv_attention>("kv_attention"), method<moe_route>("moe_route"),
                           method<token_logprobs>("token_logprobs"), method<bind_more>("bind_more"),
                           method<kv_read>("kv_read"),     method<add_norm>("add_norm"),
                           method<kv_attention_sinks>("kv_attention_sinks"),
                           method<kv_attention_shared>("kv_attention_shared"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&g_module); }
