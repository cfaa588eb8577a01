// The torch side of the calls that a training or serving step makes for every
// layer (norm and rotation, append to the paged cache, attention over it): checks
// of the tensors, their outputs and workspaces from torch's allocator, and the C
// calls of include/moba.h on the current stream.  Through ctypes the same work
// took 13 us of a thread's time for the norm and 19 us for the attention, several
// times the kernels of a small step.  No arithmetic lives here.
#include <ATen/cuda/CUDAContext.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/forward_grad.h>
#include <torch/extension.h>

#include "moba.h"

namespace {

using at::Tensor;
using std::optional;

struct Failed : std::runtime_error {
  int status;
  std::string where;
  Failed(int s, const char* w) : std::runtime_error(std::string(w) + ": " + moba_status_string((moba_status_t)s)), status(s), where(w) {}
};
void check(moba_status_t s, const char* where) {
  if (s != MOBA_OK) throw Failed((int)s, where);
}

#define REQUIRE(cond, where, ...) TORCH_CHECK_VALUE(cond, where, ": ", __VA_ARGS__)

int32_t dtype_of(const Tensor& t, const char* where) {
  const auto s = t.scalar_type();
  REQUIRE(s == at::kBFloat16 || s == at::kFloat, where, "bf16 or fp32 tensors");
  return s == at::kBFloat16 ? MOBA_BF16 : MOBA_F32;
}
void same(const Tensor& t, const Tensor& ref, at::ScalarType type, const char* where, const char* name) {
  REQUIRE(t.scalar_type() == type && t.device() == ref.device(), where, name, " must be ", type, " on ", ref.device(), ", not ",
          t.scalar_type(), " on ", t.device());
}
void dense(const Tensor& t, const char* where, const char* name) {
  REQUIRE(t.is_contiguous(), where, name, " must be contiguous");
}
int32_t i32(int64_t v, const char* where) {
  REQUIRE(v >= 0 && v <= INT32_MAX, where, "a size beyond 32 bits");
  return (int32_t)v;
}
// a tangent (forward-mode AD) does not make a tensor require a gradient, and would be lost;
// outside a dual level no tensor has one (asking each took 0.1 to 0.2 us of a call's 6)
void no_tangents(std::initializer_list<const Tensor*> ts, const char* where) {
  if (torch::autograd::ForwardADLevel::try_get_by_idx(0) == nullptr) return;
  for (const Tensor* t : ts)
    TORCH_CHECK(t == nullptr || !t->_fw_grad(/*level=*/0).defined(), where, ": has no forward-mode derivative");
}
// the cache's calls have no backward pass: an input that asks for a gradient would be cut off
void no_gradients(std::initializer_list<const Tensor*> ts, const char* where) {
  no_tangents(ts, where);
  if (!at::GradMode::is_enabled()) return;
  for (const Tensor* t : ts)
    TORCH_CHECK(t == nullptr || !t->requires_grad(), where, ": has no gradient; call it under torch.no_grad() or detach its inputs");
}
const Tensor* ptr_or_null(const optional<Tensor>& t) { return t.has_value() ? &*t : nullptr; }
// tensors of the caller that a call wrote: autograd finds out by their versions
// (which inference tensors do not keep) that a value it saved is gone
void written(std::initializer_list<const Tensor*> ts) {
  for (const Tensor* t : ts)
    if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}
const void* ptr(const optional<Tensor>& t) { return t.has_value() ? t->const_data_ptr() : nullptr; }

// x [..., h, d]: itself where its rows lie one stride apart on 16-byte borders
// (part of a fused projection), else a dense copy; `step` elements between tokens.
// Dimensions of size 1 are stepped over: their strides say nothing about the rows.
Tensor rows(const Tensor& x, int64_t& step, const char* where, const char* name) {
  REQUIRE(x.dim() >= 3 && x.is_cuda(), where, name, " must be a CUDA tensor [..., heads, head_dim]");
  const auto size = x.sizes(), st = x.strides();
  const int64_t n = x.dim(), h = size[n - 2], d = size[n - 1];
  step = h * d;
  bool ok = st[n - 1] == 1 && (h == 1 || st[n - 2] == d);
  bool first = true;
  int64_t next = 0;   // the stride that the dimension before must have
  for (int64_t i = n - 3; i >= 0 && ok; --i) {
    if (size[i] == 1) continue;
    if (first)
      step = st[i];
    else
      ok = st[i] == next;
    first = false;
    next = st[i] * size[i];
  }
  ok = ok && step >= h * d && step * x.element_size() % 16 == 0 && reinterpret_cast<uintptr_t>(x.const_data_ptr()) % 16 == 0;
  if (ok) return x;
  step = h * d;
  return x.clone(at::MemoryFormat::Contiguous);
}
Tensor dense_like(const Tensor& x) { return at::empty(x.sizes(), x.options()); }

moba_stream_t stream() { return at::cuda::getCurrentCUDAStream().stream(); }

// ---- norm and rotation ---------------------------------------------------------
struct NormRopeArgs {
  Tensor q, k;   // as read
  moba_rope_shape_t shape;
};

NormRopeArgs norm_rope_args(const Tensor& q, const Tensor& k, const Tensor& q_weight, const Tensor& k_weight,
                            const Tensor& positions, const Tensor& inv_freq, double eps, bool interleaved) {
  const char* where = "moba_norm_rope";
  NormRopeArgs a;
  int64_t qs, ks;
  a.q = rows(q, qs, where, "q");
  a.k = rows(k, ks, where, "k");
  const int32_t dt = dtype_of(q, where), wt = dtype_of(q_weight, where);
  same(k, q, q.scalar_type(), where, "k");
  same(q_weight, q, q_weight.scalar_type(), where, "q_weight");
  same(k_weight, q, q_weight.scalar_type(), where, "k_weight");
  same(positions, q, at::kInt, where, "positions");
  same(inv_freq, q, at::kDouble, where, "inv_freq");
  dense(q_weight, where, "q_weight");
  dense(k_weight, where, "k_weight");
  dense(positions, where, "positions");
  dense(inv_freq, where, "inv_freq");
  const int64_t n = q.dim(), hq = q.size(n - 2), hkv = k.size(-2), d = q.size(n - 1);
  REQUIRE(k.dim() == n && k.size(-1) == d && q.sizes().slice(0, n - 2) == k.sizes().slice(0, n - 2), where,
          "q and k must hold the same tokens and head_dim");
  REQUIRE(q_weight.dim() == 1 && q_weight.numel() == d && k_weight.dim() == 1 && k_weight.numel() == d, where,
          "the weights must be [head_dim]");
  REQUIRE(hq > 0 && d > 0, where, "empty heads");
  const int64_t tokens = q.numel() / (hq * d);
  REQUIRE(positions.numel() == tokens, where, "one position a token");
  a.shape = {i32(tokens, where), i32(hq, where), i32(hkv, where), i32(d, where), dt, tokens ? qs : 0, tokens ? ks : 0,
             {i32(2 * inv_freq.numel(), where), interleaved ? 1 : 0, wt, (float)eps}};
  return a;
}

std::tuple<Tensor, Tensor> norm_rope_forward(const NormRopeArgs& a, const Tensor& q_weight, const Tensor& k_weight,
                                             const Tensor& positions, const Tensor& inv_freq) {
  c10::DeviceGuard guard(a.q.device());
  Tensor q_out = dense_like(a.q), k_out = dense_like(a.k);
  check(moba_qk_norm_rope(&a.shape, a.q.const_data_ptr(), a.k.const_data_ptr(), q_weight.const_data_ptr(),
                          k_weight.const_data_ptr(), positions.const_data_ptr<int32_t>(), inv_freq.const_data_ptr<double>(),
                          q_out.mutable_data_ptr(), k_out.mutable_data_ptr(), stream()),
        "moba_norm_rope");
  return {q_out, k_out};
}

struct NormRope : torch::autograd::Function<NormRope> {
  static torch::autograd::variable_list forward(torch::autograd::AutogradContext* ctx, const Tensor& q, const Tensor& k,
                                                const Tensor& q_weight, const Tensor& k_weight, const Tensor& positions,
                                                const Tensor& inv_freq, double eps, bool interleaved) {
    const NormRopeArgs a = norm_rope_args(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved);
    auto [q_out, k_out] = norm_rope_forward(a, q_weight, k_weight, positions, inv_freq);
    ctx->save_for_backward({a.q, a.k, q_weight, k_weight, positions, inv_freq});
    ctx->saved_data["eps"] = eps;
    ctx->saved_data["interleaved"] = interleaved;
    return {q_out, k_out};
  }
  static torch::autograd::variable_list backward(torch::autograd::AutogradContext* ctx, torch::autograd::variable_list grads) {
    const char* where = "moba_norm_rope";
    TORCH_CHECK(!at::GradMode::is_enabled(), where, ": its gradients are not differentiable (create_graph)");
    no_tangents({&grads[0], &grads[1]}, where);
    const auto saved = ctx->get_saved_variables();
    const Tensor &qw = saved[2], &kw = saved[3], &positions = saved[4], &inv_freq = saved[5];
    const NormRopeArgs a = norm_rope_args(saved[0], saved[1], qw, kw, positions, inv_freq, ctx->saved_data["eps"].toDouble(),
                                          ctx->saved_data["interleaved"].toBool());
    c10::DeviceGuard guard(a.q.device());
    auto given = [&](const Tensor& g, const Tensor& x) {   // a gradient as the kernel reads it
      if (!g.defined()) return at::zeros(x.sizes(), x.options());
      const Tensor c = g.contiguous();
      return reinterpret_cast<uintptr_t>(c.const_data_ptr()) % 16 == 0 ? c : c.clone();
    };
    const Tensor dq_out = given(grads[0], a.q), dk_out = given(grads[1], a.k);
    Tensor dq = dense_like(a.q), dk = dense_like(a.k), dqw = dense_like(qw), dkw = dense_like(kw);
    const size_t bytes = moba_qk_norm_rope_bwd_workspace_size(&a.shape);
    Tensor ws = at::empty({(int64_t)bytes}, a.q.options().dtype(at::kByte));
    check(moba_qk_norm_rope_bwd(&a.shape, a.q.const_data_ptr(), a.k.const_data_ptr(), qw.const_data_ptr(), kw.const_data_ptr(),
                                positions.const_data_ptr<int32_t>(), inv_freq.const_data_ptr<double>(), dq_out.const_data_ptr(),
                                dk_out.const_data_ptr(), dq.mutable_data_ptr(), dk.mutable_data_ptr(), dqw.mutable_data_ptr(),
                                dkw.mutable_data_ptr(), ws.mutable_data_ptr(), bytes, stream()),
          where);
    return {dq, dk, dqw, dkw, Tensor(), Tensor(), Tensor(), Tensor()};
  }
};

std::tuple<Tensor, Tensor> norm_rope(const Tensor& q, const Tensor& k, const Tensor& q_weight, const Tensor& k_weight,
                                     const Tensor& positions, const Tensor& inv_freq, double eps, bool interleaved) {
  no_tangents({&q, &k, &q_weight, &k_weight, &inv_freq}, "moba_norm_rope");
  TORCH_CHECK(!at::GradMode::is_enabled() || !inv_freq.requires_grad(), "moba_norm_rope: inv_freq has no gradient; detach it");
  if (at::GradMode::is_enabled() &&
      (q.requires_grad() || k.requires_grad() || q_weight.requires_grad() || k_weight.requires_grad())) {
    const auto out = NormRope::apply(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved);
    return {out[0], out[1]};
  }
  return norm_rope_forward(norm_rope_args(q, k, q_weight, k_weight, positions, inv_freq, eps, interleaved), q_weight, k_weight,
                           positions, inv_freq);
}

// ---- paged cache ----------------------------------------------------------------
// Pages one after another that do not overlap: a page's offset is its number times
// the stride, and a stride of 0 (a page expanded over all) is the C call's "dense".
void check_pools(const Tensor& k_pool, const Tensor& v_pool, const char* where) {
  REQUIRE(k_pool.dim() == 4 && k_pool.sizes() == v_pool.sizes(), where,
          "the pools must be [num_pages, heads, page_size, head_dim], alike");
  const int64_t pages = k_pool.size(0), hkv = k_pool.size(1), page = k_pool.size(2), d = k_pool.size(3);
  for (const Tensor* p : {&k_pool, &v_pool}) {
    REQUIRE((hkv == 1 || p->stride(1) == page * d) && p->stride(2) == d && p->stride(3) == 1, where,
            "a page of the pools must be dense");
    REQUIRE(pages <= 1 || p->stride(0) >= hkv * page * d, where, "pages of the pools must not overlap");
  }
}

moba_paged_shape_t paged_shape(const char* where, const Tensor& ref, int64_t hq, const Tensor& k_pool, const Tensor& v_pool,
                               const Tensor& cu_new, const Tensor& kv_len, const Tensor& table, const optional<Tensor>& status,
                               double scale) {
  const int64_t pages = k_pool.size(0), hkv = k_pool.size(1), page = k_pool.size(2), d = k_pool.size(3);
  same(k_pool, ref, ref.scalar_type(), where, "k_pool");
  same(v_pool, ref, ref.scalar_type(), where, "v_pool");
  same(cu_new, ref, at::kInt, where, "cu_new");
  same(kv_len, ref, at::kInt, where, "kv_len");
  same(table, ref, at::kInt, where, "table");
  dense(cu_new, where, "cu_new");
  dense(kv_len, where, "kv_len");
  dense(table, where, "table");
  if (status.has_value()) {
    same(*status, ref, at::kInt, where, "status");
    REQUIRE(status->numel() == 1, where, "status must be one int32");
  }
  REQUIRE(table.dim() == 2 && kv_len.dim() == 1 && cu_new.dim() == 1 && kv_len.numel() == table.size(0) &&
              cu_new.numel() == table.size(0) + 1,
          where, "table must be [batch, max_pages], kv_len [batch], cu_new [batch + 1]");
  REQUIRE(ref.size(-1) == d && hkv > 0 && hq % hkv == 0, where, "the heads must match the pools'");
  moba_paged_shape_t s = {i32(table.size(0), where), i32(ref.size(0), where), i32(hq, where), i32(hkv, where), i32(d, where),
                          i32(page, where), i32(pages, where), i32(table.size(1), where), dtype_of(ref, where), (float)scale,
                          0, 0, 0, pages > 1 ? k_pool.stride(0) : 0, pages > 1 ? v_pool.stride(0) : 0};
  return s;
}

optional<Tensor> cache_append(const Tensor& k_in, const Tensor& v_in, const Tensor& cu_new, const Tensor& kv_len,
                              const Tensor& table, Tensor k_pool, Tensor v_pool, const optional<Tensor>& inv_freq,
                              const optional<Tensor>& q_in, const optional<Tensor>& q_weight, const optional<Tensor>& k_weight,
                              double eps, bool interleaved, const optional<Tensor>& status, optional<Tensor> q_out) {
  const char* where = "moba_cache_append";
  no_gradients({&k_in, &v_in, ptr_or_null(q_in), ptr_or_null(q_weight), ptr_or_null(k_weight), &k_pool, &v_pool,
                ptr_or_null(inv_freq), ptr_or_null(q_out)},
               where);
  check_pools(k_pool, v_pool, where);
  int64_t qs = 0, ks, vs;
  const Tensor k = rows(k_in, ks, where, "k"), v = rows(v_in, vs, where, "v");
  REQUIRE(k.dim() == 3 && k.sizes() == v.sizes() && k.size(1) == k_pool.size(1) && k.size(2) == k_pool.size(3),
          where, "k and v must be [tokens, heads, head_dim] with the pools' heads");
  c10::DeviceGuard guard(k.device());
  same(v, k, k.scalar_type(), where, "v");
  optional<Tensor> q;
  if (q_in.has_value()) {
    same(*q_in, k, k.scalar_type(), where, "q");
    q = rows(*q_in, qs, where, "q");
    REQUIRE(q->dim() == 3 && q->size(0) == k.size(0) && q->size(2) == k.size(2), where, "q must hold the same tokens as k");
    if (!q_out.has_value()) q_out = dense_like(*q);
    same(*q_out, k, k.scalar_type(), where, "q_out");
    dense(*q_out, where, "q_out");
    REQUIRE(q_out->sizes() == q->sizes(), where, "q_out must have q's shape");
  }
  REQUIRE(q.has_value() || (!q_weight.has_value() && !q_out.has_value()), where, "q_weight and q_out go with q");
  int32_t wt = MOBA_BF16;
  const Tensor* weight = q_weight.has_value() ? &*q_weight : k_weight.has_value() ? &*k_weight : nullptr;
  if (weight != nullptr) wt = dtype_of(*weight, where);
  for (const auto* w : {&q_weight, &k_weight}) {
    if (!w->has_value()) continue;
    same(**w, k, weight->scalar_type(), where, "a weight");
    dense(**w, where, "a weight");
    REQUIRE((*w)->dim() == 1 && (*w)->numel() == k.size(2), where, "the weights must be [head_dim]");
  }
  if (inv_freq.has_value()) {
    same(*inv_freq, k, at::kDouble, where, "inv_freq");
    dense(*inv_freq, where, "inv_freq");
  }
  moba_paged_shape_t s = paged_shape(where, k, q.has_value() ? q->size(1) : k.size(1), k_pool, v_pool, cu_new, kv_len, table,
                                     status, 0.0);
  if (s.tokens > 0) {
    s.q_stride = qs;
    s.k_stride = ks;
    s.v_stride = vs;
  }
  const moba_rope_t rope = {inv_freq.has_value() ? i32(2 * inv_freq->numel(), where) : 0, interleaved ? 1 : 0, wt, (float)eps};
  check(moba_paged_append(&s, &rope, ptr(q), k.const_data_ptr(), v.const_data_ptr(), ptr(q_weight), ptr(k_weight),
                          (const double*)ptr(inv_freq), cu_new.const_data_ptr<int32_t>(), kv_len.const_data_ptr<int32_t>(),
                          table.const_data_ptr<int32_t>(), q_out.has_value() ? q_out->mutable_data_ptr() : nullptr,
                          k_pool.mutable_data_ptr(), v_pool.mutable_data_ptr(),
                          status.has_value() ? (int*)status->mutable_data_ptr() : nullptr, stream()),
        where);
  written({&k_pool, &v_pool, ptr_or_null(q_out), ptr_or_null(status)});
  return q_out;
}

std::tuple<Tensor, optional<Tensor>> cache_attention(const Tensor& q_in, const Tensor& k_pool, const Tensor& v_pool,
                                                     const Tensor& cu_new, const Tensor& kv_len, const Tensor& table,
                                                     optional<double> scale, bool return_lse, optional<Tensor> out,
                                                     const optional<Tensor>& status) {
  const char* where = "moba_cache_attention";
  no_gradients({&q_in, &k_pool, &v_pool, ptr_or_null(out)}, where);
  check_pools(k_pool, v_pool, where);
  int64_t qs;
  const Tensor q = rows(q_in, qs, where, "q");
  REQUIRE(q.dim() == 3, where, "q must be [tokens, heads, head_dim]");
  c10::DeviceGuard guard(q.device());
  moba_paged_shape_t s = paged_shape(where, q, q.size(1), k_pool, v_pool, cu_new, kv_len, table, status, scale.value_or(0.0));
  if (s.tokens > 0) s.q_stride = qs;
  check(moba_check_paged_shape(&s), where);
  if (out.has_value()) {
    same(*out, q, q.scalar_type(), where, "out");
    dense(*out, where, "out");
    REQUIRE(out->sizes() == q.sizes(), where, "out must have q's shape");
  } else {
    out = dense_like(q);
  }
  optional<Tensor> lse;
  if (return_lse) lse = at::empty({q.size(1), q.size(0)}, q.options().dtype(at::kFloat));
  const size_t bytes = moba_paged_attn_workspace_size(&s);
  Tensor ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
  check(moba_paged_attn(&s, q.const_data_ptr(), k_pool.const_data_ptr(), v_pool.const_data_ptr(), cu_new.const_data_ptr<int32_t>(),
                        kv_len.const_data_ptr<int32_t>(), table.const_data_ptr<int32_t>(), out->mutable_data_ptr(),
                        lse.has_value() ? lse->mutable_data_ptr<float>() : nullptr,
                        status.has_value() ? (int*)status->mutable_data_ptr() : nullptr, ws.mutable_data_ptr(), bytes, stream()),
        where);
  written({&*out, ptr_or_null(status)});
  return {*out, lse};
}

}  // namespace

PYBIND11_MODULE(TORCH_EXTENSION_NAME, m) {
  namespace py = pybind11;
  py::register_exception_translator([](std::exception_ptr p) {
    try {
      if (p) std::rethrow_exception(p);
    } catch (const Failed& e) {
      const py::object type = py::module_::import("long_context_prefill_moba_b200").attr("MobaError");
      PyErr_SetObject(type.ptr(), type(e.status, e.where).ptr());
    } catch (const c10::ValueError& e) {
      PyErr_SetString(PyExc_ValueError, e.what_without_backtrace());
    }
  });
  const py::call_guard<py::gil_scoped_release> no_gil;
  m.def("norm_rope", &norm_rope, no_gil);
  m.def("cache_append", &cache_append, no_gil);
  m.def("cache_attention", &cache_attention, no_gil);
}
