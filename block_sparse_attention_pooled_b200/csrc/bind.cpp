// Compiled binding of the windowed-attention and paged-cache entry points of
// include/sparge.h: the checks of the tensors, the outputs and workspace that
// the caller does not bring, and the call. A single token's kernels take a few
// microseconds; checking and marshalling the same in Python took 4 to 8 more.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <optional>
#include <string>

#include "sparge.h"

namespace py = pybind11;

namespace {

using Tensor = at::Tensor;
using MaybeTensor = std::optional<Tensor>;

// The stream that the caller gave: its device's index and its handle.
using StreamArg = std::optional<std::pair<int, uintptr_t>>;

PyObject* error_class = nullptr;  // SpargeError(code, where); a reference that the module keeps

struct Failed {
  int code;
  const char* where;
};

// The calls below run without the interpreter's lock, so they raise C++ exceptions only.
[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

void check(int rc, const char* where) {
  if (rc != SPARGE_OK) throw Failed{rc, where};
}

int32_t i32(int64_t n) {
  if (n < INT32_MIN || n > INT32_MAX) refuse("a size of " + std::to_string(n) + " does not fit in 32 bits");
  return (int32_t)n;
}

bool is(const Tensor& t, at::ScalarType dtype, const at::Device& device) {
  return t.scalar_type() == dtype && t.device() == device && t.is_contiguous();
}

// Address of a contiguous tensor of that type and shape; refused if it is not one.
void* want(const Tensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape, const at::Device& device) {
  if (!is(t, dtype, device) || t.sizes() != shape) {
    std::string s;
    for (auto n : shape) s += (s.empty() ? "" : ", ") + std::to_string(n);
    refuse(std::string(name) + " must be a contiguous " + c10::toString(dtype) + " tensor of shape [" + s + "] on " +
           device.str());
  }
  return t.data_ptr();
}

// The stream to launch on, with the tensors' device current. Memory is taken
// from that stream's pool: what the current stream has freed may still be
// written by work that is queued there. An output made for a stream that is
// not the current one is also kept until the current one, where the caller
// goes on, is done with it.
class Launch {
 public:
  Launch(const at::Device& device, const StreamArg& stream) : device_(device) {
    if (c10::cuda::current_device() != device.index()) guard_.emplace(device);
    current_ = c10::cuda::getCurrentCUDAStream(device.index());
    handle_ = current_->stream();
    if (stream) {
      if (stream->first != device.index()) refuse("the stream belongs to another device than the tensors");
      auto h = reinterpret_cast<cudaStream_t>(stream->second);
      if (h != handle_) {
        handle_ = h;
        foreign_.emplace(c10::cuda::getStreamFromExternal(h, device.index()));
      }
    }
  }
  void* stream() const { return handle_; }
  Tensor make(at::IntArrayRef shape, at::ScalarType dtype) {
    return at::empty(shape, at::TensorOptions().dtype(dtype).device(device_));
  }
  // The caller's tensor, or one made here.
  Tensor out(const MaybeTensor& t, const char* name, at::ScalarType dtype, at::IntArrayRef shape) {
    if (!t) {
      Tensor made = make(shape, dtype);
      if (foreign_) made.record_stream(*current_);
      return made;
    }
    want(*t, name, dtype, shape, device_);
    return *t;
  }
  // Address and bytes of the workspace: the caller's, or query() bytes made here and held by `keep`.
  template <class Need>
  std::pair<void*, size_t> space(const MaybeTensor& t, Need query, Tensor& keep) {
    if (t) {
      if (t->device() != device_ || !t->is_contiguous()) refuse("workspace must be a contiguous tensor on the inputs' device");
      return {t->data_ptr(), t->nbytes()};
    }
    const size_t need = query();
    if (need == 0) return {nullptr, 0};
    keep = make({(int64_t)need}, at::kByte);
    return {keep.data_ptr(), need};
  }

 private:
  at::Device device_;
  cudaStream_t handle_;
  std::optional<c10::cuda::CUDAStream> current_;
  std::optional<c10::cuda::CUDAGuard> guard_;
  std::optional<c10::cuda::CUDAStreamGuard> foreign_;
};

// ---------------------------------------------------------------- whole sequences
struct WindowArgs {
  sparge_window_shape shape;
  sparge_window window;
  const int32_t* lens;
};

WindowArgs window_args(const Tensor& Q, const Tensor& K, const Tensor& V, int left, int right, int sinks, int unit,
                       const MaybeTensor& lens) {
  const at::Device device = Q.device();
  if (!device.is_cuda() || Q.dim() != 4 || K.dim() != 4 || !is(Q, at::kBFloat16, device) ||
      !is(K, at::kBFloat16, device) || !is(V, at::kBFloat16, device) || K.sizes() != V.sizes() ||
      K.size(0) != Q.size(0) || K.size(2) != Q.size(2) || K.size(3) != Q.size(3))
    refuse("Q, K, V must be contiguous bf16 CUDA tensors of shape [B,H,N,d] and [B,Hkv,N,d]");
  WindowArgs a;
  a.shape = {i32(Q.size(0)), i32(Q.size(1)), i32(K.size(1)), i32(Q.size(2)), i32(Q.size(3))};
  a.window = {left, right, sinks, unit};
  a.lens = lens ? static_cast<const int32_t*>(want(*lens, "lens", at::kInt, {Q.size(0)}, device)) : nullptr;
  return a;
}

Tensor window_fwd(const Tensor& Q, const Tensor& K, const Tensor& V, int left, int right, int sinks, int unit,
                  const MaybeTensor& lens, const MaybeTensor& O, const MaybeTensor& lse, const MaybeTensor& workspace,
                  const StreamArg& stream) {
  const WindowArgs a = window_args(Q, K, V, left, right, sinks, unit, lens);
  Launch on(Q.device(), stream);
  Tensor out = on.out(O, "O", at::kBFloat16, Q.sizes()), keep;
  float* l = lse ? static_cast<float*>(want(*lse, "lse", at::kFloat, Q.sizes().slice(0, 3), Q.device())) : nullptr;
  auto ws = on.space(
      workspace, [&] { return sparge_window_workspace_bytes(SPARGE_OP_WINDOW_FWD, &a.shape, &a.window); }, keep);
  check(sparge_window_fwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), &a.shape, &a.window, a.lens, out.data_ptr(), l,
                          ws.first, ws.second, on.stream()),
        "sparge_window_fwd");
  return out;
}

std::tuple<Tensor, Tensor, Tensor> window_bwd(const Tensor& Q, const Tensor& K, const Tensor& V, const Tensor& O, const Tensor& lse,
                     const Tensor& dO, int left, int right, int sinks, int unit, const MaybeTensor& lens,
                     const MaybeTensor& dQ, const MaybeTensor& dK, const MaybeTensor& dV, const MaybeTensor& workspace,
                     const StreamArg& stream) {
  const WindowArgs a = window_args(Q, K, V, left, right, sinks, unit, lens);
  want(O, "O", at::kBFloat16, Q.sizes(), Q.device());
  want(dO, "dO", at::kBFloat16, Q.sizes(), Q.device());
  want(lse, "lse", at::kFloat, Q.sizes().slice(0, 3), Q.device());
  Launch on(Q.device(), stream);
  Tensor q = on.out(dQ, "dQ", at::kBFloat16, Q.sizes()), k = on.out(dK, "dK", at::kBFloat16, K.sizes()),
         v = on.out(dV, "dV", at::kBFloat16, V.sizes()), keep;
  auto ws = on.space(
      workspace, [&] { return sparge_window_workspace_bytes(SPARGE_OP_WINDOW_BWD, &a.shape, &a.window); }, keep);
  check(sparge_window_bwd(Q.data_ptr(), K.data_ptr(), V.data_ptr(), &a.shape, &a.window, a.lens, O.data_ptr(),
                          static_cast<const float*>(lse.data_ptr()), dO.data_ptr(), q.data_ptr(), k.data_ptr(),
                          v.data_ptr(), ws.first, ws.second, on.stream()),
        "sparge_window_bwd");
  return {q, k, v};
}

// ---------------------------------------------------------------- the paged cache
struct CacheArgs {
  sparge_cache cache;
  sparge_cache_batch batch;
};

CacheArgs cache_args(const Tensor& k_pages, const Tensor& v_pages, const MaybeTensor& k_exp, const MaybeTensor& v_exp,
                     const Tensor& page_table, const Tensor& first, const Tensor& cu, int64_t tokens) {
  const at::Device device = k_pages.device();
  const at::ScalarType dtype = k_pages.scalar_type();
  if (!device.is_cuda() || k_pages.dim() != 4 || !is(k_pages, dtype, device) || !is(v_pages, dtype, device) ||
      k_pages.sizes() != v_pages.sizes())
    refuse("the cache's pages must be contiguous CUDA tensors of one type and of shape [pages, Hkv, page, d]");
  CacheArgs a{};
  if (dtype == at::kBFloat16) {
    if (k_exp || v_exp) refuse("a bf16 cache has no exponents");
    a.cache.type = SPARGE_CACHE_BF16;
  } else if (dtype == at::kFloat8_e4m3fn) {
    if (!k_exp || !v_exp) refuse("an e4m3 cache needs k_exp and v_exp");
    a.cache.type = SPARGE_CACHE_E4M3;
    a.cache.k_exp = static_cast<uint8_t*>(want(*k_exp, "k_exp", at::kByte, k_pages.sizes().slice(0, 3), device));
    a.cache.v_exp = static_cast<uint8_t*>(want(*v_exp, "v_exp", at::kByte, k_pages.sizes().slice(0, 3), device));
  } else {
    refuse("a cache holds bfloat16 or float8_e4m3fn");
  }
  if (page_table.dim() != 2 || first.dim() != 1 || cu.dim() != 1 || !is(page_table, at::kInt, device) ||
      !is(first, at::kInt, device) || !is(cu, at::kInt, device) || first.size(0) != page_table.size(0) ||
      cu.size(0) != page_table.size(0) + 1)
    refuse("page_table [B, max_pages], first [B] and cu [B + 1] must be contiguous int32 tensors on " + device.str());
  a.cache.k = k_pages.data_ptr();
  a.cache.v = v_pages.data_ptr();
  a.cache.pages = i32(k_pages.size(0));
  a.cache.Hkv = i32(k_pages.size(1));
  a.cache.page = i32(k_pages.size(2));
  a.cache.d = i32(k_pages.size(3));
  a.batch = {static_cast<const int32_t*>(page_table.data_ptr()),
             static_cast<const int32_t*>(first.data_ptr()),
             static_cast<const int32_t*>(cu.data_ptr()),
             i32(page_table.size(0)),
             i32(page_table.size(1)),
             i32(tokens)};
  return a;
}

// Token stride of packed tokens [T, heads, d]: heads and channels contiguous, tokens any stride.
int64_t token_stride(const Tensor& t, const char* name, int64_t heads, int64_t d, const at::Device& device) {
  if (t.scalar_type() != at::kBFloat16 || t.device() != device || t.dim() != 3 || t.size(1) != heads || t.size(2) != d ||
      (t.size(0) && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != d))))
    refuse(std::string(name) + " must be a bf16 tensor of shape [tokens, " + std::to_string(heads) + ", " +
           std::to_string(d) + "] on " + device.str() + ", contiguous within a token");
  return t.size(0) > 1 ? t.stride(0) : heads * d;
}

void cache_write(const Tensor& k, const Tensor& v, const Tensor& k_pages, const Tensor& v_pages, const Tensor& page_table,
                 const Tensor& first, const Tensor& cu, const MaybeTensor& k_exp, const MaybeTensor& v_exp,
                 const StreamArg& stream) {
  if (k.dim() != 3 || v.dim() != 3 || k.size(0) != v.size(0)) refuse("k and v must hold the same tokens, [T, Hkv, d]");
  const CacheArgs a = cache_args(k_pages, v_pages, k_exp, v_exp, page_table, first, cu, k.size(0));
  const int64_t ks = token_stride(k, "k", a.cache.Hkv, a.cache.d, k_pages.device());
  const int64_t vs = token_stride(v, "v", a.cache.Hkv, a.cache.d, k_pages.device());
  Launch on(k_pages.device(), stream);
  check(sparge_cache_write(&a.cache, &a.batch, k.data_ptr(), ks, v.data_ptr(), vs, on.stream()), "sparge_cache_write");
}

std::tuple<Tensor, Tensor> cache_read(const Tensor& k_pages, const Tensor& v_pages, const Tensor& page_table, const Tensor& first,
                     const Tensor& cu, int64_t tokens, const MaybeTensor& k_exp, const MaybeTensor& v_exp,
                     const MaybeTensor& K, const MaybeTensor& V, const StreamArg& stream) {
  if (tokens < 0) refuse("tokens must not be negative");
  const CacheArgs a = cache_args(k_pages, v_pages, k_exp, v_exp, page_table, first, cu, tokens);
  Launch on(k_pages.device(), stream);
  const int64_t shape[3] = {tokens, a.cache.Hkv, a.cache.d};
  Tensor k = on.out(K, "K", at::kBFloat16, shape), v = on.out(V, "V", at::kBFloat16, shape);
  check(sparge_cache_read(&a.cache, &a.batch, k.data_ptr(), v.data_ptr(), on.stream()), "sparge_cache_read");
  return {k, v};
}

Tensor cache_attn(const Tensor& Q, const Tensor& k_pages, const Tensor& v_pages, const Tensor& page_table,
                  const Tensor& first, const Tensor& cu, int max_new, int max_len, int left, int right, int sinks,
                  int unit, const MaybeTensor& k_exp, const MaybeTensor& v_exp, const MaybeTensor& O,
                  const MaybeTensor& lse, const MaybeTensor& workspace, const StreamArg& stream) {
  if (Q.dim() != 3) refuse("Q must be a tensor of shape [T, H, d]");
  const CacheArgs a = cache_args(k_pages, v_pages, k_exp, v_exp, page_table, first, cu, Q.size(0));
  const at::Device device = k_pages.device();
  const int64_t T = Q.size(0), H = Q.size(1), qs = token_stride(Q, "Q", H, a.cache.d, device);
  const sparge_window w = {left, right, sinks, unit};
  Launch on(device, stream);
  Tensor out = on.out(O, "O", at::kBFloat16, Q.sizes()), keep;
  float* l = lse ? static_cast<float*>(want(*lse, "lse", at::kFloat, {T, H}, device)) : nullptr;
  auto ws = on.space(
      workspace, [&] { return sparge_cache_attn_workspace_bytes(&a.cache, &a.batch, i32(H), max_new, max_len, &w); }, keep);
  check(sparge_cache_attn(&a.cache, &a.batch, Q.data_ptr(), qs, i32(H), max_new, max_len, &w, out.data_ptr(), l,
                          ws.first, ws.second, on.stream()),
        "sparge_cache_attn");
  return out;
}

}  // namespace

PYBIND11_MODULE(_bind, m) {
  m.def("set_error", [](py::object cls) { error_class = cls.release().ptr(); });
  py::register_local_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const Failed& e) {
      py::object error = py::handle(error_class)(e.code, e.where);
      PyErr_SetObject(error_class, error.ptr());
    }
  });
  using unlocked = py::call_guard<py::gil_scoped_release>;
  m.def("window_fwd", &window_fwd, unlocked());
  m.def("window_bwd", &window_bwd, unlocked());
  m.def("cache_write", &cache_write, unlocked());
  m.def("cache_read", &cache_read, unlocked());
  m.def("cache_attn", &cache_attn, unlocked());
}
