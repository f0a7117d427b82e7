// The calls of the normed and shared-prefix operators for Python: their checks of arguments, the tensors that they
// allocate, the current stream and the call of libsta, without an interpreter's step for each (64 single tokens behind
// a shared prefix: some 40 us of host time a call through ctypes, whose kernels take as long).
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/pybind.h>

#include <pybind11/numpy.h>

#include <algorithm>
#include <cmath>
#include <optional>
#include <string>
#include <tuple>

#include "sta.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

[[noreturn]] void refuse(const std::string& what) { throw py::value_error(what); }

// A status other than STA_OK becomes the package's StaError.
void check(const char* fn, sta_status status) {
  if (status != STA_OK) py::module_::import("split_kv_decode_bsr_gb300").attr("_check")(fn, status);
}

// A call of the library without the interpreter's lock, as through ctypes: where the stream has no room for another launch it
// waits, and other threads, and what the stream may be waiting for in one of them, go on.
template <class F>
sta_status unlocked(const F& call) {
  py::gil_scoped_release free;
  return call();
}

void on_cuda(const Tensor& t) {
  if (!t.is_cuda()) refuse("tensors must be on a CUDA device, not " + t.device().str());
}

int dtype_code(const Tensor& t) {
  if (t.scalar_type() == at::kBFloat16) return STA_BF16;
  if (t.scalar_type() == at::kFloat) return STA_F32;
  throw py::type_error(std::string("unsupported dtype ") + at::toString(t.scalar_type()));
}

// [n, H, d] with contiguous heads: the token stride.
int64_t token_stride(const Tensor& t, const char* what) {
  if (t.dim() != 3) refuse(std::string(what) + ": [tokens, heads, d]");
  const int64_t n = t.size(0), H = t.size(1), d = t.size(2);
  if (t.is_contiguous()) return H * d;
  if (!(n == 0 || ((d == 1 || t.stride(2) == 1) && (H == 1 || t.stride(1) == d))))
    refuse(std::string(what) + ": a token's heads must be contiguous");
  return n > 1 ? t.stride(0) : H * d;
}

// A new contiguous tensor beside `like`, without the dispatcher's steps (0.5 us less for each, in calls of 7 to 15).
Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(sizes, type, like.device(), std::nullopt));
}

struct Heads {
  void* at = nullptr;
  int H = 0;
  int64_t stride = 0;
};
Heads heads(const Maybe& x, const char* what, const Tensor& like) {
  Heads h;
  if (!x) return h;
  h.stride = token_stride(*x, what);
  if (!(x->size(0) == like.size(0) && x->size(2) == like.size(2) && x->scalar_type() == like.scalar_type() &&
        x->device() == like.device()))
    refuse(std::string(what) + ": the tokens, head size, dtype and device of the others");
  h.at = x->data_ptr();
  h.H = (int)x->size(1);
  return h;
}
// Where a result shaped like x goes: the given tensor, or a new contiguous one.
Heads result(Maybe& given, const Maybe& x, const char* what) {
  Heads h;
  if (!x) {
    if (given) refuse(std::string(what) + ": nothing to write there");
    return h;
  }
  if (!given) {
    given = fresh(x->sizes(), x->scalar_type(), *x);
    h.stride = x->size(1) * x->size(2);
  } else {
    if (!(given->sizes() == x->sizes() && given->scalar_type() == x->scalar_type() && given->device() == x->device()))
      refuse(std::string(what) + ": the shape, dtype and device of what it is for");
    h.stride = token_stride(*given, what);
  }
  h.at = given->data_ptr();
  h.H = (int)x->size(1);
  return h;
}

const float* norm_weight(const Maybe& w, const char* what, const Tensor& like) {
  if (!w) return nullptr;
  const int64_t d = like.size(2);
  if (!(w->scalar_type() == at::kFloat && w->dim() == 1 && w->size(0) == d && w->is_contiguous() && w->device() == like.device()))
    refuse(std::string(what) + ": contiguous float32 [" + std::to_string(d) + "] on " + like.device().str());
  return w->data_ptr<float>();
}

const int32_t* indices(const Tensor& t, const char* what, const Tensor& like) {
  if (!(t.scalar_type() == at::kInt && t.is_contiguous() && t.device() == like.device()))
    refuse(std::string(what) + ": contiguous int32 on " + like.device().str());
  return t.data_ptr<int32_t>();
}
const int32_t* token_positions(const Maybe& t, const Tensor& like, bool needed) {
  if (!t) {
    if (needed) refuse("positions: one a token");
    return nullptr;
  }
  const int32_t* at = indices(*t, "positions", like);
  if (!(t->dim() == 1 && t->size(0) == like.size(0))) refuse("positions: one a token");
  return at;
}

// The first of q and k, by whose tokens, head size, dtype and device the others go.
const Tensor& first(const Maybe& q, const Maybe& k) {
  const Maybe& x = q ? q : k;
  if (!x || x->dim() != 3) refuse("q or k: [tokens, heads, d]");
  on_cuda(*x);
  return *x;
}

// A Rope's parameters: the bytes of the C struct (aligned: what precedes them in a bytes object is whole words), or None.
const sta_rope_params* params(const py::object& rope) {
  if (rope.is_none()) return nullptr;
  if (!PyBytes_Check(rope.ptr()) || PyBytes_GET_SIZE(rope.ptr()) != (Py_ssize_t)sizeof(sta_rope_params)) refuse("rope: a Rope");
  return reinterpret_cast<const sta_rope_params*>(PyBytes_AS_STRING(rope.ptr()));
}

// The tensors' device, made current where it is not, and its current stream.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  sta_stream stream;
  explicit On(const Tensor& t) {
    if (c10::cuda::current_device() != t.device().index()) guard.set_device(t.device());
    stream = c10::cuda::getCurrentCUDAStream(t.device().index()).stream();
  }
};

// Scratch of the current device's current stream, to which it goes back; without a tensor around it.
void* workspace_at(const Maybe& given, size_t need, const Tensor& like, c10::DataPtr& own, size_t& bytes) {
  if (!given) {
    own = c10::cuda::CUDACachingAllocator::get()->allocate(need);
    bytes = need;
    return own.get();
  }
  if (!(given->scalar_type() == at::kByte && given->is_contiguous() && given->device() == like.device()))
    refuse("workspace: contiguous uint8 on " + like.device().str());
  if ((size_t)given->numel() < need)
    refuse("workspace: " + std::to_string(need) + " bytes needed, " + std::to_string(given->numel()) + " given");
  bytes = (size_t)given->numel();
  return given->data_ptr();
}

std::tuple<Maybe, Maybe> norm_rope(const Maybe& q, const Maybe& k, const Maybe& positions, const py::object& rope, const Maybe& q_weight,
                                   const Maybe& k_weight, double eps, Maybe q_out, Maybe k_out) {
  const Tensor& x = first(q, k);
  const int code = dtype_code(x);
  const sta_rope_params* turn = params(rope);
  const int32_t* pos = turn ? token_positions(positions, x, true) : nullptr;
  const Heads a = heads(q, "q", x), b = heads(k, "k", x);
  const float *qw = norm_weight(q_weight, "q_weight", x), *kw = norm_weight(k_weight, "k_weight", x);
  On on(x);
  const Heads c = result(q_out, q, "q_out"), d = result(k_out, k, "k_out");
  check("sta_norm_rope", unlocked([&] {
    return sta_norm_rope(a.at, b.at, a.stride, b.stride, c.at, d.at, c.stride, d.stride, qw, kw, (float)eps, pos, turn, x.size(0),
                         a.H, b.H, (int)x.size(2), code, on.stream);
  }));
  return {q_out, k_out};
}

std::tuple<Maybe, Maybe, Maybe, Maybe> norm_rope_bwd(const Maybe& dq_out, const Maybe& dk_out, const Maybe& q, const Maybe& k,
                                                     const Maybe& positions, const py::object& rope, const Maybe& q_weight,
                                                     const Maybe& k_weight, double eps, Maybe dq, Maybe dk,
                                                     const Maybe& workspace) {
  const Tensor& x = first(q, k);
  const int code = dtype_code(x);
  const sta_rope_params* turn = params(rope);
  const int32_t* pos = turn ? token_positions(positions, x, true) : nullptr;
  const Heads a = heads(q, "q", x), b = heads(k, "k", x), y = heads(dq_out, "dq_out", x), z = heads(dk_out, "dk_out", x);
  if (!(y.H == a.H && z.H == b.H)) refuse("dq_out, dk_out: the shapes of q and k");
  const float *qw = norm_weight(q_weight, "q_weight", x), *kw = norm_weight(k_weight, "k_weight", x);
  const int d = (int)x.size(2);
  On on(x);
  const Heads g = result(dq, q, "dq"), h = result(dk, k, "dk");
  Maybe dqw, dkw;
  if (q) dqw = fresh({d}, at::kFloat, x);
  if (k) dkw = fresh({d}, at::kFloat, x);
  size_t need = 0, bytes = 0;
  check("sta_norm_rope_bwd", sta_norm_rope_bwd(nullptr, nullptr, d, 0, nullptr, nullptr, d, 0, nullptr, nullptr, d, 0, nullptr,
                                               nullptr, nullptr, nullptr, 1.f, nullptr, nullptr, 0, 1, 0, d, STA_BF16, nullptr,
                                               &need, nullptr));
  c10::DataPtr own;
  void* ws = workspace_at(workspace, need, x, own, bytes);
  float *dqw_at = dqw ? dqw->data_ptr<float>() : nullptr, *dkw_at = dkw ? dkw->data_ptr<float>() : nullptr;
  check("sta_norm_rope_bwd", unlocked([&] {
    return sta_norm_rope_bwd(y.at, z.at, y.stride, z.stride, a.at, b.at, a.stride, b.stride, g.at, h.at, g.stride, h.stride, qw, kw,
                             dqw_at, dkw_at, (float)eps, pos, turn, x.size(0), a.H, b.H, d, code, ws, &bytes, on.stream);
  }));
  return {dq, dk, dqw, dkw};
}

void pages_of(const Tensor& k_pages, const Tensor& v_pages) {
  if (!(k_pages.dim() == 4 && v_pages.sizes() == k_pages.sizes() && k_pages.is_contiguous() && v_pages.is_contiguous()))
    refuse("k_pages, v_pages: contiguous [n_pages, page_size, Hkv, d]");
}

Maybe norm_rope_append_paged(const Maybe& q, const Tensor& k, const Tensor& v, const Tensor& k_pages, const Tensor& v_pages,
                             const Tensor& page_indptr, const Tensor& page_indices, const Tensor& q_indptr,
                             const Tensor& kv_indptr, const py::object& rope, const Maybe& q_weight, const Maybe& k_weight, double eps,
                             const Maybe& positions, Maybe q_out) {
  on_cuda(k);
  pages_of(k_pages, v_pages);
  const int64_t ks = token_stride(k, "k"), vs = token_stride(v, "v");
  const int64_t n = k.size(0), Hkv = k_pages.size(2), d = k_pages.size(3);
  if (!(k.size(1) == Hkv && k.size(2) == d && v.sizes() == k.sizes())) refuse("k, v: [n, Hkv, d]");
  for (const Tensor* t : {&k, &v, &k_pages, &v_pages}) {
    if (t->device() != k.device()) refuse("tensors on different devices");
    if (t->scalar_type() != at::kBFloat16) refuse("bf16 only");
  }
  const Heads a = heads(q, "q", k);
  const float *qw = norm_weight(q_weight, "q_weight", k), *kw = norm_weight(k_weight, "k_weight", k);
  const int32_t *pp = indices(page_indptr, "page_indptr", k), *pi = indices(page_indices, "page_indices", k),
                *qp = indices(q_indptr, "q_indptr", k), *kp = indices(kv_indptr, "kv_indptr", k);
  const int64_t n_req = q_indptr.numel() - 1;
  if (!(kv_indptr.numel() == n_req + 1 && page_indptr.numel() == n_req + 1)) refuse("indptr: n_req + 1 values each");
  const int32_t* pos = token_positions(positions, k, false);
  if (q_out && !(q && q_out->is_contiguous())) refuse("q_out: contiguous, q's shape");
  On on(k);
  const Heads c = result(q_out, q, "q_out");
  const sta_rope_params* turn = params(rope);
  check("sta_norm_rope_append_paged", unlocked([&] {
    return sta_norm_rope_append_paged(a.at, k.data_ptr(), v.data_ptr(), a.stride, ks, vs, c.at, k_pages.data_ptr(), v_pages.data_ptr(),
                                      (int)k_pages.size(1), (int)k_pages.size(0), pp, pi, qp, kp, pos, qw, kw, (float)eps, turn, n,
                                      (int)n_req, a.H, (int)Hkv, (int)d, STA_BF16, on.stream);
  }));
  return q_out;
}

// Host int32 values [n]: their address, kept alive by this object and the argument.
struct HostInts {
  using Array = py::array_t<int32_t, py::array::c_style>;
  const int32_t* at = nullptr;
  int64_t n = 0;
  py::object kept;
  HostInts(py::handle x, int64_t want, const char* what) {
    auto numbers = [&](py::handle o) {
      if (!Array::check_(o)) return false;
      const auto& a = reinterpret_cast<const py::array&>(o);
      if (a.ndim() != 1) return false;
      at = static_cast<const int32_t*>(a.data());
      n = a.shape(0);
      return true;
    };
    if (THPVariable_Check(x.ptr())) {
      const Tensor& t = THPVariable_Unpack(x.ptr());
      if (t.scalar_type() == at::kInt && t.is_cpu() && t.is_contiguous() && t.dim() == 1) {
        at = t.data_ptr<int32_t>();
        n = t.size(0);
      }
    }
    if (!at && !numbers(x)) {
      kept = py::module_::import("numpy").attr("ascontiguousarray")(x, py::arg("dtype") = "int32");
      if (!numbers(kept)) refuse(std::string(what) + ": a list of whole numbers");
    }
    if (want < 1 || n != want) refuse(std::string(what) + ": " + std::to_string(want) + " values, at least one");
  }
};

std::tuple<Tensor, Tensor> prefix_fwd_paged(const Tensor& q, const Tensor& k_pages, const Tensor& v_pages,
                                            const Tensor& page_indptr, const Tensor& page_indices, const Tensor& q_indptr,
                                            py::handle q_indptr_host, const Tensor& kv_indptr, py::handle kv_indptr_host,
                                            py::handle group_indptr_host, py::handle prefix_host, std::optional<double> scale,
                                            int num_splits, Maybe o, Maybe lse, const Maybe& workspace) {
  const int64_t qs = token_stride(q, "q");
  on_cuda(q);
  const int64_t n = q.size(0), Hq = q.size(1), d = q.size(2);
  pages_of(k_pages, v_pages);
  if (k_pages.size(3) != d) refuse("k_pages, v_pages: contiguous [n_pages, page_size, Hkv, d]");
  for (const Tensor* t : {&k_pages, &v_pages}) {
    if (t->device() != q.device()) refuse("tensors on different devices");
    if (t->scalar_type() != q.scalar_type()) refuse("q, k_pages, v_pages: one dtype");
  }
  const int code = dtype_code(q);
  const int32_t *pp = indices(page_indptr, "page_indptr", q), *pi = indices(page_indices, "page_indices", q),
                *qp = indices(q_indptr, "q_indptr", q), *kp = indices(kv_indptr, "kv_indptr", q);
  const int64_t n_req = q_indptr.numel() - 1;
  if (!(kv_indptr.numel() == n_req + 1 && page_indptr.numel() == n_req + 1)) refuse("indptr: n_req + 1 values each");
  const HostInts qh(q_indptr_host, n_req + 1, "q_indptr_host"), kh(kv_indptr_host, n_req + 1, "kv_indptr_host");
  const Py_ssize_t n_groups = PyObject_Size(group_indptr_host.ptr()) - 1;
  if (PyErr_Occurred()) throw py::error_already_set();
  const HostInts gh(group_indptr_host, n_groups + 1, "group_indptr_host"), ph(prefix_host, n_groups, "prefix_host");
  const int64_t rows = qh.at[n_req];
  if (!(rows >= 0 && rows <= n)) refuse("q_indptr: past q's rows");
  const float by = scale ? (float)*scale : 1.f / std::sqrt((float)d);
  On on(q);
  if (!o) o = fresh(q.sizes(), q.scalar_type(), q);
  else if (!(o->sizes() == q.sizes() && o->scalar_type() == q.scalar_type() && o->is_contiguous() && o->device() == q.device()))
    refuse("o: contiguous, q's shape, dtype and device");
  if (!lse) lse = fresh({n, Hq}, at::kFloat, q);
  else if (!(lse->dim() == 2 && lse->size(0) == n && lse->size(1) == Hq && lse->scalar_type() == at::kFloat && lse->is_contiguous() &&
             lse->device() == q.device()))
    refuse("lse: contiguous float32 [n, Hq]");
  // scratch for 16 pieces a row, which does for most calls; one that needs more says how much
  size_t bytes = 0;
  c10::DataPtr own;
  void* ws = workspace_at(workspace, workspace ? 256 : std::max<int64_t>(256, std::min<int64_t>(16 * rows * Hq * (d + 2) * 4, 1 << 26)), q,
                          own, bytes);
  auto call = [&]() {
    return sta_prefix_fwd_paged(q.data_ptr(), qs, k_pages.data_ptr(), v_pages.data_ptr(), (int)k_pages.size(1), (int)k_pages.size(0),
                                pp, pi, qp, qh.at, kp, kh.at, (int)n_req, gh.at, ph.at, (int)n_groups, (int)Hq, (int)k_pages.size(2),
                                (int)d, code, by, num_splits, o->data_ptr(), lse->data_ptr<float>(), ws, &bytes, on.stream);
  };
  sta_status status = unlocked(call);
  if (status == STA_ERR_WORKSPACE) {
    const size_t need = bytes;
    ws = workspace_at(workspace, need, q, own, bytes);
    status = unlocked(call);
  }
  check("sta_prefix_fwd_paged", status);
  return {*o, *lse};
}

}  // namespace

PYBIND11_MODULE(_bind, m) {
  m.def("norm_rope", &norm_rope);
  m.def("norm_rope_bwd", &norm_rope_bwd);
  m.def("norm_rope_append_paged", &norm_rope_append_paged);
  m.def("prefix_fwd_paged", &prefix_fwd_paged);
}
