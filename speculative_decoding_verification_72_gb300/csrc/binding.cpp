// Python binding of the verify step's operators (the 8-bit cache, its attention
// and eviction, token log-probs) over the C ABI of include/spec_verify.h.
//
// Argument marshalling only. These calls take a few microseconds on the GPU at
// their smallest, less than the same checks and allocations cost from Python
// (measured for one append: 24.5 us through ctypes, of which the C call is
// 2.7 us), so shapes, types, strides and devices are checked here on tensors
// directly, outputs are allocated here, and one Python call is one C call.
// Every C++ exception becomes a Python one at the entry (guarded()).

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <algorithm>
#include <cstdint>
#include <string>
#include <unordered_map>
#include <utility>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "spec_verify.h"

namespace {

PyObject* g_error = nullptr;       // SpecVerifyError
PyObject* g_as_tensor = nullptr;   // torch.as_tensor

struct Refused {
  std::string why;
};

[[noreturn]] void refuse(std::string why) { throw Refused{std::move(why)}; }

struct PyFailed {};   // a Python error is already set

std::string show(c10::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

bool given(PyObject* o) { return o != nullptr && o != Py_None; }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!o || !THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw PyFailed{};
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PyFailed{};
  return v;
}

bool same_shape(c10::IntArrayRef a, c10::IntArrayRef b) { return a == b; }

// int32 contiguous tensor on dev: the caller's own where it is one, else a copy.
// Wider integers are brought into int32's range, not cut off to its bits: past
// it a position, length or token is as far out of range as at its end.
at::Tensor ints(PyObject* o, const char* name, c10::IntArrayRef shape, at::Device dev) {
  at::Tensor t;
  if (THPVariable_Check(o)) {
    t = THPVariable_Unpack(o);
  } else {
    PyObject* r = PyObject_CallFunctionObjArgs(g_as_tensor, o, nullptr);
    if (!r) throw PyFailed{};
    t = THPVariable_Unpack(r);
    Py_DECREF(r);
  }
  if (!same_shape(t.sizes(), shape)) refuse(std::string(name) + " must have shape " + show(shape) + ", got " + show(t.sizes()));
  if (t.scalar_type() == at::kInt && t.device() == dev && t.is_contiguous()) return t;
  if (t.scalar_type() == at::kLong) t = t.clamp(INT32_MIN, INT32_MAX);
  return t.to(dev, at::kInt).contiguous();
}

void check_dense(const at::Tensor& t, const char* name, c10::IntArrayRef shape, at::ScalarType dt, at::Device dev) {
  if (!same_shape(t.sizes(), shape) || t.scalar_type() != dt || t.device() != dev || !t.is_contiguous())
    refuse(std::string(name) + " must be a contiguous " + c10::toString(dt) + " " + show(shape) + " tensor on " + dev.str());
}

int32_t dtype_code(const at::Tensor& t, bool f32, bool f16, const char* name) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return SV_BF16;
    case at::kFloat: if (f32) return SV_F32; break;
    case at::kHalf: if (f16) return SV_F16; break;
    default: break;
  }
  refuse(std::string(name) + " has an element type this call does not take: " + c10::toString(t.scalar_type()));
}

void check(sv_status rc) {
  if (rc != SV_OK) refuse("libspecverify returned " + std::to_string(rc) + ": " + spec_verify_status_string(rc));
}

// ------------------------------------------------------- outputs, workspace

struct Outputs {
  PyObject* given_;   // the caller's dict, borrowed, or null
  PyObject* dict;     // owned
  at::Device dev;
  Outputs(PyObject* out, at::Device d) : given_(given(out) ? out : nullptr), dict(nullptr), dev(d) {
    if (given_ && !PyDict_Check(given_)) refuse("out must be a dict of tensors");
    dict = given_ ? (Py_INCREF(given_), given_) : PyDict_New();
    if (!dict) throw PyFailed{};
  }
  ~Outputs() { Py_XDECREF(dict); }
  at::Tensor get(const char* name, c10::IntArrayRef shape, at::ScalarType dt) {
    if (given_) {
      PyObject* o = PyDict_GetItemString(given_, name);
      if (!o || !THPVariable_Check(o)) refuse(std::string("out[\"") + name + "\"] must be a tensor");
      const at::Tensor& t = THPVariable_Unpack(o);
      check_dense(t, name, shape, dt, dev);
      return t;
    }
    at::Tensor t = at::empty(shape, at::TensorOptions().dtype(dt).device(dev));
    PyObject* o = THPVariable_Wrap(t);
    if (!o || PyDict_SetItemString(dict, name, o) != 0) {
      Py_XDECREF(o);
      throw PyFailed{};
    }
    Py_DECREF(o);
    return t;
  }
  PyObject* release() { return std::exchange(dict, nullptr); }
};

// One workspace per device and stream, grown as needed (never shared by calls
// that can overlap); kept for the life of the process. A call that is being
// captured in a graph gets one of its own from the graph's memory: replays go on
// using its address, whatever becomes of the kept one.
at::Tensor workspace(PyObject* own, size_t need, at::Device dev, void* stream) {
  if (need == 0) refuse("invalid sizes");
  if (given(own)) {
    const at::Tensor& t = tensor(own, "workspace");
    if (t.device() != dev || t.nbytes() < need || !t.is_contiguous())
      refuse("workspace must be a contiguous CUDA tensor of at least " + std::to_string(need) + " bytes");
    return t;
  }
  auto fresh = [&] { return at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(dev)); };
  if (c10::cuda::currentStreamCaptureStatusMayInitCtx() != c10::cuda::CaptureStatus::None) return fresh();
  struct Key {
    int dev;
    void* stream;
    bool operator==(const Key& o) const { return dev == o.dev && stream == o.stream; }
  };
  struct Hash {
    size_t operator()(const Key& k) const { return std::hash<void*>()(k.stream) * 31 + k.dev; }
  };
  static auto* kept = new std::unordered_map<Key, at::Tensor, Hash>();   // guarded by the GIL
  at::Tensor& t = (*kept)[Key{dev.index(), stream}];
  if (!t.defined() || t.nbytes() < need) t = fresh();
  return t;
}

void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
int32_t* iptr(const at::Tensor& t) { return static_cast<int32_t*>(ptr(t)); }
float* fptr(const at::Tensor& t) { return static_cast<float*>(ptr(t)); }

// ------------------------------------------------------------------- cache

struct Cache {
  sv_q8_cache c;
  at::Tensor table;
  at::Device dev{at::kCPU};
  int64_t H = 0, P = 0, D = 0;
};

Cache cache_of(PyObject* o, PyObject* table, int64_t B) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 4) refuse("cache must be a Q8Cache");
  const at::Tensor& k = tensor(PyTuple_GET_ITEM(o, 0), "cache.k");
  const at::Tensor& v = tensor(PyTuple_GET_ITEM(o, 1), "cache.v");
  const at::Tensor& ks = tensor(PyTuple_GET_ITEM(o, 2), "cache.k_scale");
  const at::Tensor& vs = tensor(PyTuple_GET_ITEM(o, 3), "cache.v_scale");
  if (k.dim() != 4 || !k.is_cuda()) refuse("cache.k must be a CUDA tensor [pages, kv heads, page size, head dim]");
  Cache r;
  r.dev = k.device();
  check_dense(k, "cache.k", k.sizes(), at::kFloat8_e4m3fn, r.dev);
  check_dense(v, "cache.v", k.sizes(), at::kFloat8_e4m3fn, r.dev);
  check_dense(ks, "cache.k_scale", k.sizes().slice(0, 2), at::kFloat, r.dev);
  check_dense(vs, "cache.v_scale", k.sizes().slice(0, 2), at::kFloat, r.dev);
  r.H = k.size(1);
  r.P = k.size(2);
  r.D = k.size(3);
  if (r.P != 16 && r.P != 32 && r.P != 64 && r.P != 128) refuse("page size must be 16, 32, 64 or 128, got " + std::to_string(r.P));
  if (r.D != 64 && r.D != 128) refuse("head dim must be 64 or 128, got " + std::to_string(r.D));
  const at::Tensor& t = tensor(table, "page_table");
  if (t.dim() != 2) refuse("page_table must be [B, max_pages]");
  r.table = ints(table, "page_table", {B, t.size(1)}, r.dev);
  r.c = sv_q8_cache{k.data_ptr(), v.data_ptr(), fptr(ks), fptr(vs), iptr(r.table), static_cast<int32_t>(k.size(0)),
                    static_cast<int32_t>(r.H), static_cast<int32_t>(r.P), static_cast<int32_t>(r.D),
                    static_cast<int32_t>(t.size(1))};
  return r;
}

// A [B, N, heads, D] tensor as it lies, or a copy where the kernels cannot read it so. The stride of a dimension of
// one is never taken, whatever it is.
std::pair<sv_rows, at::Tensor> rows_of(const at::Tensor& given_t, const char* name, int64_t heads, int64_t D, at::Device dev) {
  at::Tensor t = given_t;
  if (t.dim() != 4 || t.size(2) != heads || t.size(3) != D || t.device() != dev)
    refuse(std::string(name) + " must be [B, N, " + std::to_string(heads) + ", " + std::to_string(D) + "] on " + dev.str() +
           ", got " + show(t.sizes()) + " on " + t.device().str());
  const int64_t es = t.element_size();
  auto stride = [&](int64_t d) { return t.size(d) == 1 ? 0 : t.stride(d); };
  auto lies_well = [&] {
    return t.stride(3) == 1 && reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && stride(0) * es % 16 == 0 &&
           stride(1) * es % 16 == 0 && stride(2) * es % 16 == 0;
  };
  if (!lies_well()) {
    t = t.contiguous();
    if (!lies_well()) t = t.clone();
  }
  return {sv_rows{t.data_ptr(), stride(0), stride(1), stride(2)}, t};
}

struct Path {
  at::Tensor nodes, n;
  int32_t cols = 0;
};

Path path_of(PyObject* nodes, PyObject* n, int64_t B, at::Device dev) {
  Path p;
  if (given(nodes)) {
    if (!given(n)) refuse("path_nodes needs num_accepted");
    const at::Tensor& t = tensor(nodes, "path_nodes");
    if (t.dim() != 2) refuse("path_nodes must be [B, columns]");
    p.cols = static_cast<int32_t>(t.size(1));
    p.nodes = ints(nodes, "path_nodes", {B, t.size(1)}, dev);
  }
  if (given(n)) p.n = ints(n, "num_accepted", {B}, dev);
  return p;
}

// ------------------------------------------------------------- entry points

// cache, k_new, v_new, page_table, seq_base, path_nodes, num_accepted, out
PyObject* kv_append(PyObject* const* a) {
  const at::Tensor &k = tensor(a[1], "k_new"), &v = tensor(a[2], "v_new");
  if (k.dim() != 4 || k.size(1) < 1 || !same_shape(k.sizes(), v.sizes()) || k.scalar_type() != v.scalar_type())
    refuse("k_new and v_new must be [B, N, kv heads, head dim] of one shape and type, N at least 1");
  const int64_t B = k.size(0), N = k.size(1);
  const Cache c = cache_of(a[0], a[3], B);
  const c10::cuda::CUDAGuard guard(c.dev);
  const int32_t dt = dtype_code(k, true, true, "k_new");
  const auto [kr, kt] = rows_of(k, "k_new", c.H, c.D, c.dev);
  const auto [vr, vt] = rows_of(v, "v_new", c.H, c.D, c.dev);
  const at::Tensor base = ints(a[4], "seq_base", {B}, c.dev);
  const Path p = path_of(a[5], a[6], B, c.dev);
  Outputs out(a[7], c.dev);
  const at::Tensor len = out.get("out_len", {B}, at::kInt), st = out.get("status", {B}, at::kInt);
  check(spec_kv_append_q8(&c.c, &kr, &vr, dt, static_cast<int32_t>(B), static_cast<int32_t>(N), iptr(base), iptr(p.nodes), p.cols,
                          iptr(p.n), iptr(len), iptr(st), c10::cuda::getCurrentCUDAStream(c.dev.index()).stream()));
  return out.release();
}

// q, cache, page_table, seq_base, parents, n_nodes, sm_scale, workspace, out
PyObject* attention(PyObject* const* a) {
  const at::Tensor& q0 = tensor(a[0], "q");
  if (q0.dim() != 4 || q0.size(1) < 1) refuse("q must be [B, N, heads, head dim], N at least 1");
  const int64_t B = q0.size(0), N = q0.size(1), Hq = q0.size(2);
  const Cache c = cache_of(a[1], a[2], B);
  const c10::cuda::CUDAGuard guard(c.dev);
  if (Hq == 0 || Hq % c.H != 0) refuse("q's heads must be a multiple of the cache's");
  const int32_t dt = dtype_code(q0, false, true, "q");
  const auto [qr, q] = rows_of(q0, "q", Hq, c.D, c.dev);
  const at::Tensor base = ints(a[3], "seq_base", {B}, c.dev);
  const at::Tensor par = given(a[4]) ? ints(a[4], "parents", {B, N}, c.dev) : at::Tensor();
  const at::Tensor nn = given(a[5]) ? ints(a[5], "n_nodes", {B}, c.dev) : at::Tensor();
  const double sm = given(a[6]) ? real(a[6]) : c.D == 64 ? 0.125 : 0.08838834764831845;
  Outputs out(a[8], c.dev);
  const at::Tensor o = out.get("out", {B, N, Hq, c.D}, q0.scalar_type()), lse = out.get("lse", {B, N, Hq}, at::kFloat),
                   st = out.get("status", {B}, at::kInt);
  void* stream = c10::cuda::getCurrentCUDAStream(c.dev.index()).stream();
  const auto i = [](int64_t x) { return static_cast<int32_t>(x); };
  const at::Tensor ws = workspace(a[7], spec_attention_q8_workspace_size(i(B), i(N), i(Hq), i(c.H), i(c.D)), c.dev, stream);
  check(spec_attention_q8(&qr, dt, &c.c, i(B), i(N), i(Hq), iptr(base), iptr(par), iptr(nn), static_cast<float>(sm), ptr(o),
                          fptr(lse), iptr(st), ptr(ws), ws.nbytes(), stream));
  return out.release();
}

// q, lse, cache, page_table, seq_base, scores, path_nodes, num_accepted, sm_scale, decay, out
PyObject* attention_weights(PyObject* const* a) {
  const at::Tensor& q0 = tensor(a[0], "q");
  if (q0.dim() != 4 || q0.size(1) < 1) refuse("q must be [B, N, heads, head dim], N at least 1");
  const int64_t B = q0.size(0), N = q0.size(1), Hq = q0.size(2);
  const Cache c = cache_of(a[2], a[3], B);
  const c10::cuda::CUDAGuard guard(c.dev);
  if (Hq == 0 || Hq % c.H != 0) refuse("q's heads must be a multiple of the cache's");
  const int32_t dt = dtype_code(q0, false, true, "q");
  const auto [qr, q] = rows_of(q0, "q", Hq, c.D, c.dev);
  const at::Tensor base = ints(a[4], "seq_base", {B}, c.dev);
  const Path p = path_of(a[6], a[7], B, c.dev);
  const at::Tensor &lse = tensor(a[1], "lse"), &scores = tensor(a[5], "scores");
  if (scores.dim() != 3) refuse("scores must be [B, kv heads, S]");
  const int64_t S = scores.size(2);
  check_dense(lse, "lse", {B, N, Hq}, at::kFloat, c.dev);
  check_dense(scores, "scores", {B, c.H, S}, at::kFloat, c.dev);
  const double sm = given(a[8]) ? real(a[8]) : c.D == 64 ? 0.125 : 0.08838834764831845;
  const double decay = real(a[9]);
  Outputs out(a[10], c.dev);
  const at::Tensor os = out.get("scores", {B, c.H, S}, at::kFloat), st = out.get("status", {B}, at::kInt);
  const auto i = [](int64_t x) { return static_cast<int32_t>(x); };
  check(spec_attention_weights_q8(&qr, dt, fptr(lse), &c.c, i(B), i(N), i(Hq), iptr(base), iptr(p.nodes), p.cols, iptr(p.n),
                                  static_cast<float>(sm), static_cast<float>(decay), fptr(scores), fptr(os), i(S), iptr(st),
                                  c10::cuda::getCurrentCUDAStream(c.dev.index()).stream()));
  return out.release();
}

// cache, page_table, seq_len, scores, positions, keep, sinks, protect_from, workspace, out
PyObject* kv_evict(PyObject* const* a) {
  const at::Tensor &scores = tensor(a[3], "scores"), &positions = tensor(a[4], "positions");
  if (scores.dim() != 3) refuse("scores must be [B, kv heads, S]");
  const int64_t B = scores.size(0), S = scores.size(2);
  const Cache c = cache_of(a[0], a[1], B);
  const c10::cuda::CUDAGuard guard(c.dev);
  check_dense(scores, "scores", {B, c.H, S}, at::kFloat, c.dev);
  check_dense(positions, "positions", {B, c.H, S}, at::kInt, c.dev);
  const int64_t keep = integer(a[5]), sinks = std::min<int64_t>(std::max<int64_t>(integer(a[6]), INT32_MIN), INT32_MAX);
  if (keep < c.P || keep % c.P != 0 || keep > S)
    refuse("keep must be a positive multiple of the page size " + std::to_string(c.P) + ", at most " + std::to_string(S));
  const at::Tensor n = ints(a[2], "seq_len", {B}, c.dev);
  const at::Tensor from = given(a[7]) ? ints(a[7], "protect_from", {B}, c.dev) : at::Tensor();
  Outputs out(a[9], c.dev);
  const at::Tensor os = out.get("scores", {B, c.H, S}, at::kFloat), op = out.get("positions", {B, c.H, S}, at::kInt),
                   len = out.get("out_len", {B}, at::kInt), st = out.get("status", {B}, at::kInt);
  void* stream = c10::cuda::getCurrentCUDAStream(c.dev.index()).stream();
  const auto i = [](int64_t x) { return static_cast<int32_t>(x); };
  const at::Tensor ws = workspace(a[8], spec_kv_evict_q8_workspace_size(i(B), i(c.H), i(keep)), c.dev, stream);
  check(spec_kv_evict_q8(&c.c, i(B), iptr(n), fptr(scores), iptr(positions), i(S), i(keep), i(sinks), iptr(from), fptr(os),
                         iptr(op), iptr(len), iptr(st), ptr(ws), ws.nbytes(), stream));
  return out.release();
}

// [B, R, V] logits and the stride of their evenly strided rows, or a contiguous copy.
std::pair<at::Tensor, int64_t> logit_rows(const at::Tensor& t, const char* name, bool may_copy) {
  if (t.dim() != 3 || !t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor [B, rows, V]");
  const int64_t B = t.size(0), R = t.size(1), V = t.size(2);
  const int64_t stride = R > 1 ? t.stride(1) : B > 1 ? t.stride(0) : V;
  const bool even = (V <= 1 || t.stride(2) == 1) && (R <= 1 || B <= 1 || t.stride(0) == R * t.stride(1)) && stride >= V;
  if (even) return {t, stride};
  if (!may_copy) refuse(std::string(name) + " must have evenly strided rows of unit stride");
  return {t.contiguous(), V};
}

// logits, tokens, temperature, n_top, workspace, out
PyObject* token_logprobs(PyObject* const* a) {
  const auto [x, stride] = logit_rows(tensor(a[0], "logits"), "logits", true);
  const int64_t B = x.size(0), R = x.size(1), V = x.size(2);
  const at::Device dev = x.device();
  const c10::cuda::CUDAGuard guard(dev);
  const int32_t dt = dtype_code(x, true, false, "logits");
  const at::Tensor tok = ints(a[1], "tokens", {B, R}, dev);
  const double T = real(a[2]);
  const int64_t n_top = integer(a[3]);
  if (n_top < 0 || n_top > SV_MAX_TOP_ALTERNATIVES)
    refuse("n_top must lie in [0, " + std::to_string(SV_MAX_TOP_ALTERNATIVES) + "]");
  Outputs out(a[5], dev);
  const at::Tensor lp = out.get("logprob", {B, R}, at::kFloat), ent = out.get("entropy", {B, R}, at::kFloat),
                   lse = out.get("lse", {B, R}, at::kFloat), saved = out.get("saved", {B, R, 4}, at::kFloat),
                   st = out.get("status", {B, R}, at::kInt);
  at::Tensor tt, tl;
  if (n_top > 0) {
    tt = out.get("top_tokens", {B, R, n_top}, at::kInt);
    tl = out.get("top_logprobs", {B, R, n_top}, at::kFloat);
  }
  void* stream = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  const auto i = [](int64_t v) { return static_cast<int32_t>(v); };
  if (B * R > INT32_MAX || V > INT32_MAX) refuse("too many rows or logits");
  const at::Tensor ws = workspace(a[4], spec_token_logprobs_workspace_size(i(B * R), i(V), dt, i(n_top)), dev, stream);
  check(spec_token_logprobs(ptr(x), dt, stride, iptr(tok), i(B * R), i(V), static_cast<float>(T), i(n_top), fptr(lp), fptr(ent),
                            fptr(lse), fptr(saved), iptr(tt), fptr(tl), iptr(st), ptr(ws), ws.nbytes(), stream));
  return out.release();
}

// logits, tokens, saved, grad_logprob, grad_entropy, temperature, out
PyObject* token_logprobs_backward(PyObject* const* a) {
  const auto [x, stride] = logit_rows(tensor(a[0], "logits"), "logits", true);
  const int64_t B = x.size(0), R = x.size(1), V = x.size(2);
  const at::Device dev = x.device();
  const c10::cuda::CUDAGuard guard(dev);
  const int32_t dt = dtype_code(x, true, false, "logits");
  const at::Tensor tok = ints(a[1], "tokens", {B, R}, dev);
  const at::Tensor& saved = tensor(a[2], "saved");
  check_dense(saved, "saved", {B, R, 4}, at::kFloat, dev);
  auto upstream = [&](PyObject* o, const char* name) {
    at::Tensor t = tensor(o, name);
    if (!same_shape(t.sizes(), {B, R})) refuse(std::string(name) + " must have shape " + show({B, R}) + ", got " + show(t.sizes()));
    return t.to(dev, at::kFloat).contiguous();
  };
  const at::Tensor g = upstream(a[3], "grad_logprob");
  const at::Tensor h = given(a[4]) ? upstream(a[4], "grad_entropy") : at::Tensor();
  const double T = real(a[5]);
  at::Tensor d;
  int64_t dstride = V;
  if (given(a[6])) {
    const at::Tensor& o = tensor(a[6], "out");
    if (!same_shape(o.sizes(), x.sizes()) || o.scalar_type() != x.scalar_type() || o.device() != dev)
      refuse("out must have the logits' shape, type and device");
    std::tie(d, dstride) = logit_rows(o, "out", false);
  } else {
    d = at::empty({B, R, V}, at::TensorOptions().dtype(x.scalar_type()).device(dev));
  }
  if (B * R > INT32_MAX || V > INT32_MAX) refuse("too many rows or logits");
  check(spec_token_logprobs_backward(ptr(x), dt, stride, iptr(tok), fptr(saved), fptr(g), fptr(h), static_cast<int32_t>(B * R),
                                     static_cast<int32_t>(V), static_cast<float>(T), ptr(d), dstride,
                                     c10::cuda::getCurrentCUDAStream(dev.index()).stream()));
  if (given(a[6])) return Py_NewRef(a[6]);
  return THPVariable_Wrap(d);
}

// ------------------------------------------------------------------- module

template <PyObject* (*F)(PyObject* const*), int kArgs>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", kArgs, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PyFailed&) {
    return nullptr;
  } catch (const Refused& r) {
    PyErr_SetString(g_error ? g_error : PyExc_RuntimeError, r.why.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_up(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "expected the error class and torch.as_tensor");
    return nullptr;
  }
  g_error = Py_NewRef(args[0]);
  g_as_tensor = Py_NewRef(args[1]);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"set_up", fast(set_up), METH_FASTCALL, nullptr},
    {"kv_append", fast(guarded<kv_append, 8>), METH_FASTCALL, nullptr},
    {"attention", fast(guarded<attention, 9>), METH_FASTCALL, nullptr},
    {"attention_weights", fast(guarded<attention_weights, 11>), METH_FASTCALL, nullptr},
    {"kv_evict", fast(guarded<kv_evict, 10>), METH_FASTCALL, nullptr},
    {"token_logprobs", fast(guarded<token_logprobs, 6>), METH_FASTCALL, nullptr},
    {"token_logprobs_backward", fast(guarded<token_logprobs_backward, 7>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
