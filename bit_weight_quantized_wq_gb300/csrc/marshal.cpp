// Argument marshalling of the attention-block and 8-bit-cache operators for Python, compiled: a decode call's
// kernels run for a few microseconds, and checking ten tensors attribute by attribute from Python
// and passing thirty ctypes arguments took 20 and more (measured on the Grace host; about 5 here).
// Checks types, devices, shapes and contiguity, allocates the outputs, finds the workspace of the
// current stream, and calls the C ABI (include/wq.h).  binding.py gives these calls their keyword
// arguments and documentation.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <map>
#include <optional>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include "../../include/wq.h"

namespace {

struct Refused {      // -> ValueError
  std::string what;
};

[[noreturn]] void refuse(const std::string& what) { throw Refused{what}; }

std::string list(at::IntArrayRef v) {
  std::string s = "[";
  for (size_t i = 0; i < v.size(); ++i) s += (i ? ", " : "") + std::to_string(v[i]);
  return s + "]";
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

at::Tensor optional(PyObject* o, const char* name) { return o == Py_None ? at::Tensor() : tensor(o, name); }

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be an integer");
  }
  return v;
}

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(std::string(name) + " must be a number");
  }
  return v;
}

int truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(std::string(name) + " must be true or false");
  }
  return v;
}

// `t` on device `dev` with the given type and shape, contiguous.
void need(const at::Tensor& t, const char* name, int dev, at::ScalarType dtype, at::IntArrayRef shape, bool contiguous = true) {
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(std::string(name) + " must be on the same CUDA device as the other tensors");
  if (t.scalar_type() != dtype)
    refuse(std::string(name) + " must be " + c10::toString(dtype) + ", got " + c10::toString(t.scalar_type()));
  if (t.sizes() != shape) refuse(std::string(name) + " must be " + list(shape) + ", got " + list(t.sizes()));
  if (contiguous && !t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
}

void dims(const at::Tensor& t, const char* name, int64_t n, const char* layout) {
  if (t.dim() != n) refuse(std::string(name) + " must be " + layout);
}

wq_dtype dtype16(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  if (t.scalar_type() == at::kBFloat16) return WQ_DTYPE_BF16;
  if (t.scalar_type() == at::kHalf) return WQ_DTYPE_F16;
  refuse(std::string(name) + " must be bfloat16 or float16, got " + c10::toString(t.scalar_type()));
}

// Token stride of a [T, heads, d] tensor whose heads are contiguous within a token.
int64_t head_stride(const at::Tensor& t, const char* name) {
  if (t.dim() != 3 || t.numel() == 0) refuse(std::string(name) + " must be [T, heads, d], none of them 0");
  if (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != t.size(2)))
    refuse(std::string(name) + ": a token's heads must be contiguous");
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

uint16_t* u16(const at::Tensor& t) { return t.defined() ? static_cast<uint16_t*>(t.data_ptr()) : nullptr; }
int32_t* i32(const at::Tensor& t) { return t.defined() ? static_cast<int32_t*>(t.data_ptr()) : nullptr; }
float* f32(const at::Tensor& t) { return t.defined() ? static_cast<float*>(t.data_ptr()) : nullptr; }

// Device and current stream of a call.
struct On {
  int dev;
  c10::cuda::CUDAGuard guard;
  cudaStream_t stream;
  explicit On(const at::Tensor& t)
      : dev(t.get_device()), guard(static_cast<c10::DeviceIndex>(dev)),
        stream(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream()) {}
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType dtype) const {
    // straight to the caching allocator: the dispatcher's way there costs most of a microsecond more
    return at::detail::empty_cuda(shape, dtype, c10::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
  }
  // The caller's workspace, or the zeroed one kept for this stream, grown when a call needs more.  One
  // that a captured call took stays when a larger one takes its place: the graph holds its address.
  at::Tensor workspace(PyObject* given, size_t bytes) const {
    if (given != Py_None) {
      const at::Tensor& t = tensor(given, "workspace");
      if (!t.is_cuda() || t.get_device() != dev || !t.is_contiguous())
        refuse("workspace must be a contiguous CUDA tensor on the inputs' device");
      return t;
    }
    struct Kept {
      at::Tensor now;
      bool captured = false;
      std::vector<at::Tensor> before;
    };
    static auto* all = new std::map<std::pair<int, cudaStream_t>, Kept>;   // outlives the interpreter's tear-down
    Kept& k = (*all)[{dev, stream}];
    cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
    bool capturing = true;
    if (cudaStreamIsCapturing(stream, &st) == cudaSuccess) capturing = st != cudaStreamCaptureStatusNone;
    else cudaGetLastError();                   // the default stream while another one is captured: the call itself will say so
    if (!k.now.defined() || static_cast<size_t>(k.now.numel()) < bytes) {
      if (capturing)
        refuse("no workspace of this size on this stream yet: make one call of this size before capturing, or pass one");
      at::Tensor grown = at::zeros({static_cast<int64_t>((bytes + 255) / 256 * 256)}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev));
      if (k.captured) k.before.push_back(k.now);
      k.now = std::move(grown), k.captured = false;
    }
    k.captured |= capturing;
    return k.now;
  }
};

void done(wq_status st, const char* what) {
  if (st == WQ_OK) return;
  const std::string msg = std::string(what) + " failed: " + wq_status_str(st);
  if (st == WQ_ERR_UNSUPPORTED_ARCH || st == WQ_ERR_CUDA) throw std::runtime_error(msg);
  refuse(msg);
}

void arity(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw std::runtime_error("internal: wrong number of arguments");
}

// ------------------------------------------------------------------------------- rotation
struct Rope {
  at::Tensor Q, K, positions, cos_sin, wq, wk;
  wq_dtype dt;
  int64_t T, Hq, Hkv, d, qs, ks;
  float eps;
  int interleaved;
};

// Q, K, positions, cos_sin, q_weight, k_weight, eps, interleaved
Rope rope_inputs(PyObject* const* a) {
  Rope r;
  r.Q = tensor(a[0], "Q"), r.K = tensor(a[1], "K");
  r.positions = tensor(a[2], "positions"), r.cos_sin = tensor(a[3], "cos_sin");
  r.wq = optional(a[4], "q_weight"), r.wk = optional(a[5], "k_weight");
  r.eps = static_cast<float>(number(a[6], "eps"));
  r.interleaved = truth(a[7], "interleaved");
  r.dt = dtype16(r.Q, "Q");
  r.qs = head_stride(r.Q, "Q"), r.ks = head_stride(r.K, "K");
  r.T = r.Q.size(0), r.Hq = r.Q.size(1), r.d = r.Q.size(2), r.Hkv = r.K.size(1);
  const int dev = r.Q.get_device();
  const at::ScalarType ty = r.Q.scalar_type();
  need(r.K, "K", dev, ty, {r.T, r.Hkv, r.d}, false);
  need(r.positions, "positions", dev, at::kInt, {r.T});
  dims(r.cos_sin, "cos_sin", 2, "[positions, rot]");
  need(r.cos_sin, "cos_sin", dev, at::kFloat, r.cos_sin.sizes());
  if (r.wq.defined()) need(r.wq, "q_weight", dev, ty, {r.d});
  if (r.wk.defined()) need(r.wk, "k_weight", dev, ty, {r.d});
  return r;
}

// ..., out Q, out K -> (Q', K')
PyObject* rope(PyObject* const* a, Py_ssize_t n) {
  arity(n, 10);
  const Rope r = rope_inputs(a);
  const On on(r.Q);
  at::Tensor qo = optional(a[8], "out Q"), ko = optional(a[9], "out K");
  if (qo.defined()) need(qo, "out Q", on.dev, r.Q.scalar_type(), {r.T, r.Hq, r.d});
  else qo = on.empty({r.T, r.Hq, r.d}, r.Q.scalar_type());
  if (ko.defined()) need(ko, "out K", on.dev, r.Q.scalar_type(), {r.T, r.Hkv, r.d});
  else ko = on.empty({r.T, r.Hkv, r.d}, r.Q.scalar_type());
  done(wq_qk_norm_rope(r.dt, r.T, r.Hq, r.Hkv, r.d, u16(r.Q), r.qs, u16(r.K), r.ks, u16(r.wq), u16(r.wk), r.eps, f32(r.cos_sin),
                       r.cos_sin.size(0), r.cos_sin.size(1), r.interleaved, i32(r.positions), u16(qo), u16(ko), on.stream),
       "wq_qk_norm_rope");
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(qo));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(ko));
  return t;
}

// ..., V, k_cache, v_cache, slots, out -> Q'
PyObject* rope_cache(PyObject* const* a, Py_ssize_t n) {
  arity(n, 13);
  const Rope r = rope_inputs(a);
  const On on(r.Q);
  const at::ScalarType ty = r.Q.scalar_type();
  const at::Tensor &V = tensor(a[8], "V"), &kc = tensor(a[9], "k_cache"), &vc = tensor(a[10], "v_cache"),
                   &slots = tensor(a[11], "slots");
  const int64_t vs = head_stride(V, "V");
  need(V, "V", on.dev, ty, {r.T, r.Hkv, r.d}, false);
  dims(kc, "k_cache", 4, "[pages, Hkv, page_size, d]");
  need(kc, "k_cache", on.dev, ty, {kc.size(0), r.Hkv, kc.size(2), r.d});
  need(vc, "v_cache", on.dev, ty, kc.sizes());
  need(slots, "slots", on.dev, at::kInt, {r.T});
  at::Tensor qo = optional(a[12], "out");
  if (qo.defined()) need(qo, "out", on.dev, ty, {r.T, r.Hq, r.d});
  else qo = on.empty({r.T, r.Hq, r.d}, ty);
  done(wq_qk_norm_rope_cache(r.dt, r.T, r.Hq, r.Hkv, r.d, u16(r.Q), r.qs, u16(r.K), r.ks, u16(V), vs, u16(r.wq), u16(r.wk), r.eps,
                             f32(r.cos_sin), r.cos_sin.size(0), r.cos_sin.size(1), r.interleaved, i32(r.positions), u16(qo),
                             u16(kc), u16(vc), kc.size(0), kc.size(2), i32(slots), on.stream),
       "wq_qk_norm_rope_cache");
  return THPVariable_Wrap(qo);
}

// ------------------------------------------------------------------------------- attention
// Q, k_cache, v_cache, prefix_pages, prefix_len, block_table, suffix_lens, q_start, max_new, scale, out O, out lse,
// workspace -> (O, lse)
PyObject* attn(PyObject* const* a, Py_ssize_t n) {
  arity(n, 13);
  const at::Tensor &Q = tensor(a[0], "Q"), &kc = tensor(a[1], "k_cache"), &vc = tensor(a[2], "v_cache");
  const wq_dtype dt = dtype16(Q, "Q");
  const at::ScalarType ty = Q.scalar_type();
  const int64_t qs = head_stride(Q, "Q"), T = Q.size(0), Hq = Q.size(1), d = Q.size(2);
  const On on(Q);
  dims(kc, "k_cache", 4, "[pages, Hkv, page_size, d]");
  need(kc, "k_cache", on.dev, ty, {kc.size(0), kc.size(1), kc.size(2), d});
  need(vc, "v_cache", on.dev, ty, kc.sizes());
  const int64_t Hkv = kc.size(1), page = kc.size(2);
  const at::Tensor pp = optional(a[3], "prefix_pages"), bt = optional(a[5], "block_table"), sl = optional(a[6], "suffix_lens"),
                   q0 = optional(a[7], "q_start");
  const int64_t prefix = integer(a[4], "prefix_len"), max_new = integer(a[8], "max_new");
  int64_t R = T, blocks = 0;
  if (q0.defined()) {
    dims(q0, "q_start", 1, "[R + 1]");
    need(q0, "q_start", on.dev, at::kInt, q0.sizes());
    R = q0.size(0) - 1;
  }
  if (bt.defined() != sl.defined()) refuse("block_table and suffix_lens go together");
  if (bt.defined()) {
    dims(bt, "block_table", 2, "[R, blocks]");
    blocks = bt.size(1);
    need(bt, "block_table", on.dev, at::kInt, {R, blocks});
    need(sl, "suffix_lens", on.dev, at::kInt, {R});
  }
  if (prefix > 0) {
    if (!pp.defined()) refuse("prefix_pages is required when prefix_len > 0");
    dims(pp, "prefix_pages", 1, "[pages of the prefix]");
    need(pp, "prefix_pages", on.dev, at::kInt, pp.sizes());
    if (pp.numel() * page < prefix) refuse("prefix_pages must hold prefix_len tokens");
  }
  const float scale = a[9] == Py_None ? 1.0f / std::sqrt(static_cast<float>(d)) : static_cast<float>(number(a[9], "scale"));
  at::Tensor o = optional(a[10], "out O"), lse = optional(a[11], "out lse");
  if (o.defined()) need(o, "out O", on.dev, ty, {T, Hq, d});
  else o = on.empty({T, Hq, d}, ty);
  if (lse.defined()) need(lse, "out lse", on.dev, at::kFloat, {T, Hq});
  else lse = on.empty({T, Hq}, at::kFloat);
  const at::Tensor ws = on.workspace(a[12], wq_attn_workspace_bytes(T, R, Hq, Hkv, d, max_new));
  done(wq_attn_shared_prefix(dt, u16(Q), qs, T, R, Hq, Hkv, d, u16(kc), u16(vc), kc.size(0), page, prefix > 0 ? i32(pp) : nullptr,
                             prefix, blocks ? i32(bt) : nullptr, blocks, blocks ? i32(sl) : nullptr, i32(q0), max_new, scale, u16(o),
                             f32(lse), ws.data_ptr(), ws.nbytes(), on.stream),
       "wq_attn_shared_prefix");
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(o));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(lse));
  return t;
}

// -------------------------------------------------------------------------------- adapters
struct Lora {
  at::Tensor X, A, B, adapter, scales, ranks;
  int64_t M, K, N, L, r;
};

// X, A, B, adapter, scales, ranks
Lora lora_inputs(PyObject* const* a) {
  Lora l;
  l.X = tensor(a[0], "X"), l.A = tensor(a[1], "A"), l.B = tensor(a[2], "B");
  l.adapter = tensor(a[3], "adapter"), l.scales = tensor(a[4], "scales"), l.ranks = optional(a[5], "ranks");
  dims(l.X, "X", 2, "[M, K]"), dims(l.A, "A", 3, "[L, r, K]"), dims(l.B, "B", 3, "[L, N, r]");
  dtype16(l.X, "X");
  const at::ScalarType ty = l.X.scalar_type();
  const int dev = l.X.get_device();
  l.M = l.X.size(0), l.K = l.X.size(1), l.L = l.A.size(0), l.r = l.A.size(1), l.N = l.B.size(1);
  need(l.X, "X", dev, ty, l.X.sizes());
  need(l.A, "A", dev, ty, {l.L, l.r, l.K});
  need(l.B, "B", dev, ty, {l.L, l.N, l.r});
  need(l.adapter, "adapter", dev, at::kInt, {l.M});
  need(l.scales, "scales", dev, at::kFloat, {l.L});
  if (l.ranks.defined()) need(l.ranks, "ranks", dev, at::kInt, {l.L});
  return l;
}

// ..., base, out, workspace -> Y
PyObject* lora_add(PyObject* const* a, Py_ssize_t n) {
  arity(n, 9);
  const Lora l = lora_inputs(a);
  const On on(l.X);
  const at::Tensor& base = tensor(a[6], "base");
  need(base, "base", on.dev, l.X.scalar_type(), {l.M, l.N});
  at::Tensor y = optional(a[7], "out");
  if (y.defined()) need(y, "out", on.dev, l.X.scalar_type(), {l.M, l.N});
  else y = on.empty({l.M, l.N}, l.X.scalar_type());
  const at::Tensor ws = on.workspace(a[8], wq_lora_workspace_bytes(l.M, l.K, l.N, l.r));
  done(wq_lora_add(dtype16(l.X, "X"), u16(base), u16(l.X), l.M, l.K, l.N, u16(l.A), u16(l.B), l.L, l.r, i32(l.ranks),
                   i32(l.adapter), f32(l.scales), u16(y), ws.data_ptr(), ws.nbytes(), on.stream),
       "wq_lora_add");
  return THPVariable_Wrap(y);
}

// ..., format, Wq, scales, zeros, out, workspace -> Y
PyObject* gemm_lora(PyObject* const* a, Py_ssize_t n) {
  arity(n, 12);
  const Lora l = lora_inputs(a);
  if (l.X.scalar_type() != at::kBFloat16) refuse("X must be BFloat16");
  const On on(l.X);
  const wq_fmt fmt = static_cast<wq_fmt>(integer(a[6], "format"));
  const bool int4 = fmt == WQ_FMT_INT4_G128_ASYM;
  const at::Tensor &Wq = tensor(a[7], "Wq"), &sc = tensor(a[8], "scales");
  const at::Tensor z = optional(a[9], "zeros");
  need(Wq, "Wq", on.dev, at::kInt, {l.N, l.K / 8});
  need(sc, "scales", on.dev, int4 ? at::kHalf : at::kByte, {l.N, l.K / (int4 ? 128 : 32)});
  if (int4 != z.defined()) refuse(int4 ? "zeros is required for INT4 g128" : "zeros must be None for MXFP4");
  if (int4) need(z, "zeros", on.dev, at::kHalf, sc.sizes());
  at::Tensor y = optional(a[10], "out");
  if (y.defined()) need(y, "out", on.dev, at::kBFloat16, {l.M, l.N});
  else y = on.empty({l.M, l.N}, at::kBFloat16);
  const at::Tensor ws = on.workspace(a[11], wq_gemm_w4a16_lora_workspace_bytes(fmt, l.M, l.K, l.N, l.r));
  done(wq_gemm_w4a16_lora(fmt, u16(l.X), l.M, l.K, l.N, i32(Wq), sc.data_ptr(), u16(z), u16(l.A), u16(l.B), l.L, l.r, i32(l.ranks),
                          i32(l.adapter), f32(l.scales), u16(y), ws.data_ptr(), ws.nbytes(), on.stream),
       "wq_gemm_w4a16_lora");
  return THPVariable_Wrap(y);
}

// ------------------------------------------------------------------------------- the cache in 8 bits
uint8_t* u8(const at::Tensor& t) { return static_cast<uint8_t*>(t.data_ptr()); }

struct Cache8 {
  at::Tensor k, v, ks, vs, table;
  int64_t pages, Hkv, page, d, blocks;
};

// k_cache, v_cache, k_scales, v_scales, block_table
Cache8 cache8(PyObject* const* a, int dev) {
  Cache8 c;
  c.k = tensor(a[0], "k_cache"), c.v = tensor(a[1], "v_cache");
  c.ks = tensor(a[2], "k_scales"), c.vs = tensor(a[3], "v_scales"), c.table = tensor(a[4], "block_table");
  dims(c.k, "k_cache", 4, "[pages, Hkv, page_size, d]");
  c.pages = c.k.size(0), c.Hkv = c.k.size(1), c.page = c.k.size(2), c.d = c.k.size(3);
  need(c.k, "k_cache", dev, at::kByte, c.k.sizes());
  need(c.v, "v_cache", dev, at::kByte, c.k.sizes());
  need(c.ks, "k_scales", dev, at::kByte, {c.pages, c.Hkv});
  need(c.vs, "v_scales", dev, at::kByte, {c.pages, c.Hkv});
  dims(c.table, "block_table", 2, "[R, blocks]");
  need(c.table, "block_table", dev, at::kInt, c.table.sizes());
  c.blocks = c.table.size(1);
  return c;
}

// The requests' lengths and first rows: T tokens of table.size(0) requests.
void rows_of(const at::Tensor& lens, const at::Tensor& q0, const Cache8& c, int dev, int64_t T) {
  const int64_t R = c.table.size(0);
  need(lens, "lens", dev, at::kInt, {R});
  if (q0.defined()) need(q0, "q_start", dev, at::kInt, {R + 1});
  else if (T != R) refuse("q_start is required unless there is one token a request");
}

// K, V, k_cache, v_cache, k_scales, v_scales, block_table, lens, q_start, max_new
PyObject* kv_append(PyObject* const* a, Py_ssize_t n) {
  arity(n, 10);
  const at::Tensor &K = tensor(a[0], "K"), &V = tensor(a[1], "V"), &lens = tensor(a[7], "lens");
  const at::Tensor q0 = optional(a[8], "q_start");
  const wq_dtype dt = dtype16(K, "K");
  const int64_t ks = head_stride(K, "K"), vs = head_stride(V, "V"), T = K.size(0);
  const On on(K);
  const Cache8 c = cache8(a + 2, on.dev);
  need(K, "K", on.dev, K.scalar_type(), {T, c.Hkv, c.d}, false);
  need(V, "V", on.dev, K.scalar_type(), {T, c.Hkv, c.d}, false);
  rows_of(lens, q0, c, on.dev, T);
  done(wq_kv_append_e4m3(dt, u16(K), ks, u16(V), vs, T, c.table.size(0), c.Hkv, c.d, u8(c.k), u8(c.v), u8(c.ks), u8(c.vs), c.pages,
                         c.page, i32(c.table), c.blocks, i32(lens), i32(q0), integer(a[9], "max_new"), on.stream),
       "wq_kv_append_e4m3");
  Py_RETURN_NONE;
}

// k_cache, v_cache, k_scales, v_scales, block_table, starts, tokens, float16, out K, out V -> (K, V)
PyObject* kv_read(PyObject* const* a, Py_ssize_t n) {
  arity(n, 10);
  const at::Tensor& k = tensor(a[0], "k_cache");
  if (!k.is_cuda()) refuse("k_cache must be a CUDA tensor");
  const On on(k);
  const Cache8 c = cache8(a, on.dev);
  const at::Tensor& starts = tensor(a[5], "starts");
  const int64_t T = integer(a[6], "tokens"), R = c.table.size(0);
  const bool f16 = truth(a[7], "float16");
  const at::ScalarType ty = f16 ? at::kHalf : at::kBFloat16;
  need(starts, "starts", on.dev, at::kInt, {R + 1});
  if (T < 1) refuse("tokens must be at least 1");
  at::Tensor ko = optional(a[8], "out K"), vo = optional(a[9], "out V");
  if (ko.defined()) need(ko, "out K", on.dev, ty, {T, c.Hkv, c.d});
  else ko = on.empty({T, c.Hkv, c.d}, ty);
  if (vo.defined()) need(vo, "out V", on.dev, ty, {T, c.Hkv, c.d});
  else vo = on.empty({T, c.Hkv, c.d}, ty);
  done(wq_kv_read_e4m3(f16 ? WQ_DTYPE_F16 : WQ_DTYPE_BF16, u8(c.k), u8(c.v), u8(c.ks), u8(c.vs), c.pages, c.page, c.Hkv, c.d,
                       i32(c.table), c.blocks, i32(starts), R, T, u16(ko), u16(vo), on.stream),
       "wq_kv_read_e4m3");
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(ko));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(vo));
  return t;
}

// Q, k_cache, v_cache, k_scales, v_scales, block_table, lens, q_start, max_new, scale, out O, out lse, workspace -> (O, lse)
PyObject* attn8(PyObject* const* a, Py_ssize_t n) {
  arity(n, 13);
  const at::Tensor &Q = tensor(a[0], "Q"), &lens = tensor(a[6], "lens");
  const at::Tensor q0 = optional(a[7], "q_start");
  const wq_dtype dt = dtype16(Q, "Q");
  const at::ScalarType ty = Q.scalar_type();
  const int64_t qs = head_stride(Q, "Q"), T = Q.size(0), Hq = Q.size(1), d = Q.size(2);
  const On on(Q);
  const Cache8 c = cache8(a + 1, on.dev);
  if (c.d != d) refuse("Q and k_cache must have heads of the same size");
  rows_of(lens, q0, c, on.dev, T);
  const int64_t R = c.table.size(0), max_new = integer(a[8], "max_new");
  const float scale = a[9] == Py_None ? 1.0f / std::sqrt(static_cast<float>(d)) : static_cast<float>(number(a[9], "scale"));
  at::Tensor o = optional(a[10], "out O"), lse = optional(a[11], "out lse");
  if (o.defined()) need(o, "out O", on.dev, ty, {T, Hq, d});
  else o = on.empty({T, Hq, d}, ty);
  if (lse.defined()) need(lse, "out lse", on.dev, at::kFloat, {T, Hq});
  else lse = on.empty({T, Hq}, at::kFloat);
  const at::Tensor ws = on.workspace(a[12], wq_attn_e4m3_workspace_bytes(T, R, Hq, c.Hkv, d, max_new));
  done(wq_attn_e4m3(dt, u16(Q), qs, T, R, Hq, c.Hkv, d, u8(c.k), u8(c.v), u8(c.ks), u8(c.vs), c.pages, c.page, i32(c.table), c.blocks,
                    i32(lens), i32(q0), max_new, scale, u16(o), f32(lse), ws.data_ptr(), ws.nbytes(), on.stream),
       "wq_attn_e4m3");
  PyObject* t = PyTuple_New(2);
  if (!t) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(o));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(lse));
  return t;
}

// Raw stream -> the number of the graph capture that it takes part in, 0: none.
PyObject* capture_id(PyObject* const* a, Py_ssize_t n) {
  arity(n, 1);
  cudaStreamCaptureStatus st = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  if (cudaStreamGetCaptureInfo(reinterpret_cast<cudaStream_t>(integer(a[0], "stream")), &st, &id) != cudaSuccess)
    throw std::runtime_error("cudaStreamGetCaptureInfo failed");
  return PyLong_FromUnsignedLongLong(st == cudaStreamCaptureStatusNone ? 0 : id);
}

// No C++ exception leaves a Python entry.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(a, n);
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

#define WQ_ENTRY(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<f>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {WQ_ENTRY("qk_norm_rope", rope), WQ_ENTRY("qk_norm_rope_cache", rope_cache),
                         WQ_ENTRY("attn_shared_prefix", attn), WQ_ENTRY("lora_add", lora_add),
                         WQ_ENTRY("gemm_w4a16_lora", gemm_lora), WQ_ENTRY("kv_append_e4m3", kv_append), WQ_ENTRY("kv_read_e4m3", kv_read),
                         WQ_ENTRY("attn_e4m3", attn8), WQ_ENTRY("capture_id", capture_id), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module); }
