// fa_binding.cpp -- argument checks, output tensors and stream of the entry
// points that a decode step makes several times per layer, compiled.
//
// The calls take a few microseconds of GPU time each; marshalled in Python
// they took 9 to 33 us of the host's.  Nothing is computed here: every
// function checks its tensors, makes the outputs that were not given, and
// calls the C ABI of include/fa.h (whose addresses Python hands over, from the
// libfa.so that it has loaded) on the tensors' device and current stream.  It
// returns the status and the outputs.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <memory>
#include <optional>
#include <stdexcept>
#include <string>

#include "fa.h"

namespace py = pybind11;

namespace {

using at::Tensor;
using Maybe = std::optional<Tensor>;

struct Entries {
  decltype(&fa_qk_norm_rope) norm_rope = nullptr;
  decltype(&fa_qk_norm_rope_bwd) norm_rope_bwd = nullptr;
  decltype(&fa_qk_norm_rope_bwd_workspace_size) norm_rope_bwd_size = nullptr;
  decltype(&fa_cache4_plan) plan = nullptr;
  decltype(&fa_cache4_append) append = nullptr;
  decltype(&fa_cache4_attn) attn = nullptr;
  decltype(&fa_cache4_attn_workspace_size) attn_size = nullptr;
  bool host = false;  // CPU tensors pass (to entry points that only record)
};
// The table in use.  It is not changed but replaced, under the GIL; a call
// takes it once, before it lets go of the GIL, and keeps it to its end.
std::shared_ptr<const Entries> g_entries;
std::shared_ptr<const Entries> entries() {
  if (!g_entries) throw std::runtime_error("_fa_binding is not connected to libfa.so");
  return g_entries;
}

template <typename F>
void entry(const py::dict& from, const char* name, F& to) {
  to = reinterpret_cast<F>(py::cast<uintptr_t>(from[name]));
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

// A contiguous tensor of this type, device and shape, or an error.
void want(const char* name, const Tensor& t, at::ScalarType type, const at::Device& device,
          at::IntArrayRef shape) {
  if (t.scalar_type() == type && t.device() == device && t.sizes() == shape && t.is_contiguous())
    return;
  if (t.sizes() != shape)
    throw py::value_error(std::string(name) + " has shape " + shape_of(t.sizes()) + ", expected " +
                          shape_of(shape));
  throw py::value_error(std::string(name) + " must be a contiguous " + c10::toString(type) +
                        " tensor on " + device.str());
}
// A CUDA tensor of this type and number of axes (its device and sizes are
// then the call's).
void want_cuda(const Entries& g, const char* name, const Tensor& t, at::ScalarType type,
               int64_t axes, const char* what) {
  if (t.scalar_type() != type || !(t.is_cuda() || (g.host && t.is_cpu())) || t.dim() != axes)
    throw py::value_error(std::string(name) + " must be a " + what);
}
void want(const char* name, const Maybe& t, at::ScalarType type, const at::Device& device,
          at::IntArrayRef shape) {
  if (t) want(name, *t, type, device, shape);
}
// The caller's output (checked) or a new one.
Tensor output(const char* name, const Maybe& t, at::ScalarType type, const at::Device& device,
              at::IntArrayRef shape) {
  if (!t) return at::empty(shape, at::TensorOptions().dtype(type).device(device));
  want(name, *t, type, device, shape);
  return *t;
}
// The caller's workspace (its size is checked by the library) or a new one.
Tensor workspace_of(const Maybe& t, size_t size, const at::Device& device) {
  if (!t) return at::empty({(int64_t)size}, at::TensorOptions().dtype(at::kByte).device(device));
  if (t->device() != device || !t->is_contiguous())
    throw py::value_error("workspace must be a contiguous tensor on " + device.str());
  return *t;
}

template <typename T = void>
T* at_of(const Tensor& t) { return static_cast<T*>(t.data_ptr()); }
template <typename T = void>
T* at_of(const Maybe& t) { return t ? static_cast<T*>(t->data_ptr()) : nullptr; }

int to_int(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) throw py::value_error(std::string(name) + " is out of range");
  return (int)v;
}

// Runs `call(stream)` with the tensors' device current, on its current stream.
template <typename Call>
int launch(const at::Device& device, Call call) {
  py::gil_scoped_release release;
  if (!device.is_cuda()) return (int)call(nullptr);
  const c10::cuda::CUDAGuard guard(device);
  return (int)call(c10::cuda::getCurrentCUDAStream(device.index()).stream());
}

// ------------------------------------------------------ norm and rotation
// Strides of the batch and token axes of a [B,N,heads,d] tensor whose tokens
// are contiguous rows (axes of length one may have any).
struct TokenStrides {
  long long b, n;
  TokenStrides(const char* name, const Tensor& t) {
    if (t.numel() && ((t.size(3) > 1 && t.stride(3) != 1) ||
                      (t.size(2) > 1 && t.stride(2) != t.size(3))))
      throw py::value_error(std::string(name) + " must have contiguous tokens [heads, d]");
    b = t.size(0) > 1 ? t.stride(0) : 0;
    n = t.size(1) > 1 ? t.stride(1) : 0;
  }
};

struct RopeCall {
  at::Device device;
  int B, N, H, Hkv, d, rows, rot, weight_bf16 = 0;
  TokenStrides s;
  RopeCall(const Entries& g, const Tensor& qkv, int64_t h, int64_t hkv, const Tensor& rope,
           const Maybe& positions, const Maybe& qw, const Maybe& kw)
      : device(qkv.device()), s(check(g, "qkv", qkv), qkv) {
    if (h < 0 || hkv < 0 || qkv.size(2) != h + 2 * hkv)
      throw py::value_error("qkv has " + std::to_string(qkv.size(2)) +
                            " heads, expected H + 2 * Hkv = " + std::to_string(h + 2 * hkv));
    B = to_int(qkv.size(0), "B"), N = to_int(qkv.size(1), "N");
    H = to_int(h, "H"), Hkv = to_int(hkv, "Hkv"), d = to_int(qkv.size(3), "d");
    want_cuda(g, "rope", rope, at::kFloat, 2, "fp32 CUDA tensor [positions, rot]");
    want("rope", rope, at::kFloat, device, rope.sizes());
    rows = to_int(rope.size(0), "positions"), rot = to_int(rope.size(1), "rot");
    want("positions", positions, at::kInt, device, {B, N});
    if (qw.has_value() != kw.has_value())
      throw py::value_error("q_weight and k_weight come together");
    if (qw) {
      weight_bf16 = qw->scalar_type() == at::kBFloat16;
      const at::ScalarType type = weight_bf16 ? at::kBFloat16 : at::kFloat;
      want("q_weight", *qw, type, device, {d});
      want("k_weight", *kw, type, device, {d});
    }
  }
  static const char* check(const Entries& g, const char* name, const Tensor& t) {
    want_cuda(g, name, t, at::kBFloat16, 4, "bf16 CUDA tensor [B,N,heads,d]");
    return name;
  }
};

py::tuple qk_norm_rope(const Tensor& qkv, int64_t H, int64_t Hkv, const Tensor& rope,
                       const Maybe& positions, const Maybe& qw, const Maybe& kw, double eps,
                       bool interleaved, const Maybe& q_, const Maybe& k_, const Maybe& v_) {
  const auto held = entries();
  const Entries& g = *held;
  const RopeCall c(g, qkv, H, Hkv, rope, positions, qw, kw);
  const Tensor q = output("q", q_, at::kBFloat16, c.device, {c.B, c.H, c.N, c.d});
  const Tensor k = output("k", k_, at::kBFloat16, c.device, {c.B, c.Hkv, c.N, c.d});
  const Tensor v = output("v", v_, at::kBFloat16, c.device, {c.B, c.Hkv, c.N, c.d});
  const int status = launch(c.device, [&](void* stream) {
    return g.norm_rope(at_of(qkv), c.s.b, c.s.n, at_of<float>(rope), c.rows, c.rot,
                       at_of<int>(positions), at_of(qw), at_of(kw), c.weight_bf16, (float)eps,
                       interleaved, at_of(q), at_of(k), at_of(v), c.B, c.N, c.H, c.Hkv, c.d, stream);
  });
  return py::make_tuple(status, q, k, v);
}

py::tuple qk_norm_rope_bwd(const Tensor& qkv, int64_t H, int64_t Hkv, const Tensor& rope,
                           const Tensor& dq, const Tensor& dk, const Tensor& dv,
                           const Maybe& positions, const Maybe& qw, const Maybe& kw, double eps,
                           bool interleaved, const Maybe& dqkv_, const Maybe& workspace_) {
  const auto held = entries();
  const Entries& g = *held;
  const RopeCall c(g, qkv, H, Hkv, rope, positions, qw, kw);
  want("dq", dq, at::kBFloat16, c.device, {c.B, c.H, c.N, c.d});
  want("dk", dk, at::kBFloat16, c.device, {c.B, c.Hkv, c.N, c.d});
  want("dv", dv, at::kBFloat16, c.device, {c.B, c.Hkv, c.N, c.d});
  if (dqkv_) {
    RopeCall::check(g, "dqkv", *dqkv_);
    if (dqkv_->sizes() != qkv.sizes() || dqkv_->device() != c.device)
      throw py::value_error("dqkv must have qkv's shape and device");
  }
  const auto options = at::TensorOptions().device(c.device);
  const Tensor dqkv = dqkv_ ? *dqkv_ : at::empty(qkv.sizes(), options.dtype(at::kBFloat16));
  const TokenStrides s("dqkv", dqkv);
  Maybe dqw, dkw, workspace;
  size_t size = 0;
  if (qw) {
    dqw = at::empty({c.d}, options.dtype(at::kFloat));
    dkw = at::empty({c.d}, options.dtype(at::kFloat));
    workspace = workspace_of(workspace_, std::max<size_t>(g.norm_rope_bwd_size(c.d), 16), c.device);
    size = workspace->nbytes();
  }
  const int status = launch(c.device, [&](void* stream) {
    return g.norm_rope_bwd(at_of(qkv), c.s.b, c.s.n, at_of<float>(rope), c.rows, c.rot,
                           at_of<int>(positions), at_of(qw), at_of(kw), c.weight_bf16, (float)eps,
                           interleaved, at_of(dq), at_of(dk), at_of(dv), at_of(dqkv), s.b, s.n,
                           at_of<float>(dqw), at_of<float>(dkw), at_of(workspace), size, c.B, c.N,
                           c.H, c.Hkv, c.d, stream);
  });
  return py::make_tuple(status, dqkv, dqw, dkw);
}

// ------------------------------------------------------------------ cache
// A 4-bit cache, uint8 [pages, Hkv, page_size / 16, 18 d].
struct Cache {
  int pages, Hkv, page, d;
  Cache(const Entries& g, const Tensor& t) {
    want_cuda(g, "cache", t, at::kByte, 4, "uint8 CUDA tensor [pages, Hkv, page_size / 16, 18 * d]");
    if (t.size(3) % 18 || !t.is_contiguous())
      throw py::value_error("cache must be contiguous, its last axis 18 * d");
    pages = to_int(t.size(0), "pages"), Hkv = to_int(t.size(1), "Hkv");
    page = to_int(16 * t.size(2), "page_size"), d = to_int(t.size(3) / 18, "d");
  }
};

py::tuple cache4_plan(const Tensor& fresh, const Tensor& lens, const Tensor& table,
                      const Tensor& free_list, const Tensor& free_count, int64_t page_size,
                      int64_t T_, const Maybe& slots_, const Maybe& positions_,
                      const Maybe& granted_) {
  const auto held = entries();
  const Entries& g = *held;
  want_cuda(g, "new_tokens", fresh, at::kInt, 1, "int32 CUDA tensor [R]");
  want_cuda(g, "block_table", table, at::kInt, 2, "int32 CUDA tensor [R, max_blocks]");
  want_cuda(g, "free_list", free_list, at::kInt, 1, "int32 CUDA tensor [pages]");
  const at::Device device = fresh.device();
  const int R = to_int(fresh.size(0), "R"), M = to_int(table.size(1), "max_blocks");
  const int P = to_int(free_list.size(0), "pages"), T = to_int(T_, "T");
  if (T < 0) throw py::value_error("T must not be negative");
  want("new_tokens", fresh, at::kInt, device, {R});
  want("lens", lens, at::kInt, device, {R});
  want("block_table", table, at::kInt, device, {R, M});
  want("free_list", free_list, at::kInt, device, {P});
  want("free_count", free_count, at::kInt, device, {1});
  const Tensor slots = output("slots", slots_, at::kInt, device, {R, T});
  const Tensor positions = output("positions", positions_, at::kInt, device, {R, T});
  const Tensor granted = output("granted", granted_, at::kInt, device, {R});
  const int page = to_int(page_size, "page_size");
  const int status = launch(device, [&](void* stream) {
    return g.plan(at_of<int>(fresh), at_of<int>(lens), at_of<int>(table), at_of<int>(free_list),
                  at_of<int>(free_count), at_of<int>(slots), at_of<int>(positions),
                  at_of<int>(granted), R, M, P, page, T, stream);
  });
  return py::make_tuple(status, slots, positions, granted);
}

int cache4_append(const Tensor& k, const Tensor& v, const Tensor& cache, const Tensor& slots,
                  double k_scale, double v_scale, const Maybe& k_out, const Maybe& v_out) {
  const auto held = entries();
  const Entries& g = *held;
  const Cache c(g, cache);
  want_cuda(g, "k", k, at::kBFloat16, 4, "bf16 CUDA tensor [B,Hkv,N,d]");
  const at::Device device = cache.device();
  const int B = to_int(k.size(0), "B"), N = to_int(k.size(2), "N");
  const int64_t shape[4] = {B, c.Hkv, N, c.d};
  want("k", k, at::kBFloat16, device, shape);
  want("v", v, at::kBFloat16, device, shape);
  want("slots", slots, at::kInt, device, {B, N});
  if (k_out.has_value() != v_out.has_value()) throw py::value_error("k_out and v_out come together");
  want("k_out", k_out, at::kBFloat16, device, shape);
  want("v_out", v_out, at::kBFloat16, device, shape);
  return launch(device, [&](void* stream) {
    return g.append(at_of(k), at_of(v), at_of(cache), at_of<int>(slots), (float)k_scale,
                    (float)v_scale, at_of(k_out), at_of(v_out), B, c.Hkv, N, c.d, c.pages, c.page,
                    stream);
  });
}

py::tuple cache4_attn(const Tensor& q, const Tensor& cache, const Tensor& table,
                      const Tensor& seq_lens, double scale, const Maybe& q_lens, int64_t window,
                      double k_scale, double v_scale, const Maybe& out_, const Maybe& lse_,
                      const Maybe& workspace_) {
  const auto held = entries();
  const Entries& g = *held;
  const Cache c(g, cache);
  want_cuda(g, "q", q, at::kBFloat16, 4, "bf16 CUDA tensor [B,H,T,d]");
  want_cuda(g, "block_table", table, at::kInt, 2, "int32 CUDA tensor [B, max_blocks]");
  const at::Device device = cache.device();
  const int B = to_int(q.size(0), "B"), H = to_int(q.size(1), "H"), T = to_int(q.size(2), "T");
  const int M = to_int(table.size(1), "max_blocks"), w = to_int(window, "window");
  want("q", q, at::kBFloat16, device, {B, H, T, c.d});
  want("block_table", table, at::kInt, device, {B, M});
  want("seq_lens", seq_lens, at::kInt, device, {B});
  want("q_lens", q_lens, at::kInt, device, {B});
  const Tensor out = output("out", out_, at::kBFloat16, device, {B, H, T, c.d});
  const Tensor lse = output("lse", lse_, at::kFloat, device, {B, H, T});
  const Tensor ws =
      workspace_of(workspace_, std::max<size_t>(g.attn_size(B, H, c.Hkv, T, c.d), 256), device);
  const int status = launch(device, [&](void* stream) {
    return g.attn(at_of(q), at_of(cache), at_of<int>(table), at_of<int>(seq_lens),
                  at_of<int>(q_lens), at_of(out), at_of<float>(lse), at_of(ws), ws.nbytes(), B, H,
                  c.Hkv, T, c.d, M, c.pages, c.page, w, (float)scale, (float)k_scale, (float)v_scale,
                  stream);
  });
  return py::make_tuple(status, out, lse);
}

}  // namespace

PYBIND11_MODULE(_fa_binding, m) {
  m.def("connect", [](const py::dict& from, bool host) {
    Entries e;
    entry(from, "fa_qk_norm_rope", e.norm_rope);
    entry(from, "fa_qk_norm_rope_bwd", e.norm_rope_bwd);
    entry(from, "fa_qk_norm_rope_bwd_workspace_size", e.norm_rope_bwd_size);
    entry(from, "fa_cache4_plan", e.plan);
    entry(from, "fa_cache4_append", e.append);
    entry(from, "fa_cache4_attn", e.attn);
    entry(from, "fa_cache4_attn_workspace_size", e.attn_size);
    e.host = host;
    g_entries = std::make_shared<const Entries>(e);
  });
  m.def("qk_norm_rope", &qk_norm_rope);
  m.def("qk_norm_rope_bwd", &qk_norm_rope_bwd);
  m.def("cache4_plan", &cache4_plan);
  m.def("cache4_append", &cache4_append);
  m.def("cache4_attn", &cache4_attn);
}
