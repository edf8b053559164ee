// Python binding of the serving operators (lk_serving.h) for torch tensors.
//
// Marshalling only: checks what the C ABI cannot see (shapes, strides, types,
// devices), allocates outputs and scratch memory from torch's allocator on the
// current stream of the tensors' device, and calls the library.  It stands in
// C++ because the calls it serves take a few microseconds: the same checks in
// Python cost 5 to 8 us a call.
#include <torch/extension.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <optional>
#include <vector>

#include "lk_serving.h"

namespace {

using at::Tensor;
using OptTensor = std::optional<Tensor>;

[[noreturn]] void raise_lk(lk_status s) {
  py::object cls = py::module_::import("rank_latent_kv_lk_b200._lib").attr("LkError");
  py::object err = cls((int)s, std::string(lk_last_error()));
  PyErr_SetObject(cls.ptr(), err.ptr());
  throw py::error_already_set();
}
void check(lk_status s) {
  if (s != LK_OK) raise_lk(s);
}

lk_dtype dtype_of(const char* name, at::ScalarType t, bool half_only) {
  switch (t) {
    case at::kBFloat16: return LK_BF16;
    case at::kHalf: return LK_F16;
    case at::kFloat:
      if (!half_only) return LK_F32;
      [[fallthrough]];
    default: break;
  }
  TORCH_CHECK_TYPE(false, name, ": unsupported dtype ", t);
}

// A contiguous tensor of this shape, type and device.
void same(const char* name, const Tensor& t, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  TORCH_CHECK_TYPE(t.scalar_type() == type, name, ": dtype ", t.scalar_type(), ", not ", type);
  TORCH_CHECK_VALUE(t.sizes() == shape && t.device() == dev && t.is_contiguous(), name,
                    ": a contiguous tensor of shape ", shape, " on ", dev, " is needed, not ", t.sizes(),
                    " with strides ", t.strides(), " on ", t.device());
}
void same(const char* name, const OptTensor& t, at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  if (t) same(name, *t, shape, type, dev);
}

template <typename T = void>
T* ptr(const OptTensor& t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
template <typename T = void>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}

lk_stream_t stream_of(const at::Device& dev) {
  return reinterpret_cast<lk_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
}

// An uninitialised tensor from torch's allocator (without the dispatcher's microsecond).
Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& dev) {
  return Tensor(at::detail::empty_cuda(shape, type, dev, std::nullopt));
}
Tensor scratch(size_t bytes, const at::Device& dev) { return empty({(int64_t)bytes}, at::kByte, dev); }

struct PagedCache {
  Tensor k, v;
  OptTensor k_scale, v_scale, mass, pos;
  at::Device dev;
  lk_paged_cache d;

  PagedCache(Tensor k_, Tensor v_, OptTensor ks, OptTensor vs, OptTensor m, OptTensor p)
      : k(std::move(k_)), v(std::move(v_)), k_scale(std::move(ks)), v_scale(std::move(vs)), mass(std::move(m)),
        pos(std::move(p)), dev(k.device()) {
    describe();
  }

  // The descriptor, from the tensors as they are: a call that kept the pointers and sizes of an earlier one would
  // miss a tensor whose storage or shape was changed in place.
  void describe() {
    const auto t = k.scalar_type();
    TORCH_CHECK_VALUE(k.dim() == 4 && k.is_cuda(),
                      "k: a CUDA tensor [n_pages, n_kv_heads, page_size, head_dim] is needed");
    TORCH_CHECK_TYPE(t == at::kBFloat16 || t == at::kHalf || t == at::kChar, "a paged cache holds bf16, fp16 or int8");
    same("k", k, k.sizes(), t, dev);
    same("v", v, k.sizes(), t, dev);
    TORCH_CHECK_VALUE((t == at::kChar) == k_scale.has_value() && k_scale.has_value() == v_scale.has_value(),
                      "k_scale and v_scale belong to an int8 cache, and only to it");
    TORCH_CHECK_VALUE(mass.has_value() == pos.has_value(), "mass and pos come together");
    const auto rows = k.sizes().slice(0, 3);
    same("k_scale", k_scale, rows, at::kFloat, dev);
    same("v_scale", v_scale, rows, at::kFloat, dev);
    same("mass", mass, rows, at::kFloat, dev);
    same("pos", pos, rows, at::kInt, dev);
    for (int i = 0; i < 4; ++i) TORCH_CHECK_VALUE(k.size(i) < (int64_t)1 << 31, "k: a size of 2^31 or more");
    d = {(int32_t)k.size(0), (int32_t)k.size(2), (int32_t)k.size(1), (int32_t)k.size(3),
         t == at::kChar ? LK_I8 : (t == at::kHalf ? LK_F16 : LK_BF16), k.data_ptr(), v.data_ptr(),
         ptr<float>(k_scale), ptr<float>(v_scale), ptr<float>(mass), ptr<int32_t>(pos)};
  }

  // The page table's width.
  int32_t width(const Tensor& table, int64_t batch) const {
    TORCH_CHECK_VALUE(table.dim() == 2 && table.size(0) == batch && table.scalar_type() == at::kInt &&
                          table.device() == dev && table.is_contiguous() && table.size(1) < (int64_t)1 << 31,
                      "page_table: a contiguous int32 [", batch, ", width] on ", dev, " is needed, not ",
                      table.scalar_type(), " ", table.sizes(), " on ", table.device());
    return (int32_t)table.size(1);
  }
  // An int32 vector of the batch.
  void counts(const char* name, const Tensor& t, int64_t batch) const {
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == batch && t.scalar_type() == at::kInt && t.device() == dev &&
                          t.is_contiguous(),
                      name, ": a contiguous int32 [", batch, "] on ", dev, " is needed, not ", t.scalar_type(), " ",
                      t.sizes(), " on ", t.device());
  }
  void counts(const char* name, const OptTensor& t, int64_t batch) const {
    if (t) counts(name, *t, batch);
  }
  // Elements between the tokens of [batch, n_new, n_kv_heads, head_dim].
  int64_t token_step(const char* name, const Tensor& t) const {
    TORCH_CHECK_VALUE(t.dim() == 4 && t.size(2) == d.n_kv_heads && t.size(3) == d.head_dim && t.device() == dev, name,
                      ": [batch, n_new, ", d.n_kv_heads, ", ", d.head_dim, "] on ", dev, " is needed, not ", t.sizes(),
                      " on ", t.device());
    const int64_t b = t.size(0), n = t.size(1), h = t.size(2);
    const int64_t step = n > 1 ? t.stride(1) : (b > 1 ? t.stride(0) : h * d.head_dim);
    TORCH_CHECK_VALUE(t.stride(3) == 1 && (h == 1 || t.stride(2) == d.head_dim) &&
                          (b == 1 || n == 1 || t.stride(0) == n * step),
                      name, ": heads must be contiguous within a token and tokens evenly spaced, strides are ",
                      t.strides());
    return step;
  }
};

// Scratch of a call over a page table; none for lengths beyond it, which the library then refuses.
Tensor scratch_for(size_t bytes, int32_t max_seq_len, int32_t width, const PagedCache& c) {
  return scratch(max_seq_len <= (int64_t)width * c.d.page_size ? bytes : 0, c.dev);
}

int32_t as_i32(const char* name, int64_t v) {
  TORCH_CHECK_VALUE(v >= INT32_MIN && v <= INT32_MAX, name, ": ", v, " does not fit in 32 bits");
  return (int32_t)v;
}

void paged_append(PagedCache& c, const Tensor& table, const Tensor& k_new, const Tensor& v_new,
                  const Tensor& seq_len, const OptTensor& next_pos, const OptTensor& new_len,
                  const OptTensor& seq_len_out, const OptTensor& next_pos_out) {
  c.describe();
  const c10::cuda::CUDAGuard guard(c.dev);
  const int64_t step = c.token_step("k_new", k_new);
  TORCH_CHECK_VALUE(v_new.sizes() == k_new.sizes() && v_new.scalar_type() == k_new.scalar_type() &&
                        c.token_step("v_new", v_new) == step,
                    "k_new and v_new must have the same shape, type and token spacing");
  const int64_t batch = k_new.size(0);
  const int32_t width = c.width(table, batch);
  c.counts("seq_len", seq_len, batch);
  c.counts("next_pos", next_pos, batch);
  c.counts("new_len", new_len, batch);
  c.counts("seq_len_out", seq_len_out, batch);
  c.counts("next_pos_out", next_pos_out, batch);
  if (batch == 0) return;
  check(lk_paged_append(&c.d, ptr<int32_t>(table), as_i32("batch", batch), width, ptr(k_new), ptr(v_new),
                        dtype_of("k_new", k_new.scalar_type(), true), as_i32("token spacing", step),
                        as_i32("n_new", k_new.size(1)), ptr<int32_t>(new_len), ptr<int32_t>(seq_len),
                        seq_len_out ? ptr<int32_t>(seq_len_out) : ptr<int32_t>(seq_len), ptr<int32_t>(next_pos),
                        next_pos_out ? ptr<int32_t>(next_pos_out) : ptr<int32_t>(next_pos), stream_of(c.dev)));
}

Tensor paged_decode_attn(PagedCache& c, const Tensor& table, const Tensor& q, const Tensor& seq_len,
                         int64_t max_seq_len, std::optional<double> softmax_scale, bool accumulate,
                         const OptTensor& out, std::optional<at::ScalarType> out_dtype) {
  c.describe();
  const c10::cuda::CUDAGuard guard(c.dev);
  TORCH_CHECK_VALUE(q.dim() == 3 && q.size(2) == c.d.head_dim && q.device() == c.dev, "q: [batch, n_heads, ",
                    c.d.head_dim, "] on ", c.dev, " is needed, not ", q.sizes(), " on ", q.device());
  const int64_t batch = q.size(0), heads = q.size(1), dim = q.size(2);
  TORCH_CHECK_VALUE(q.stride(2) == 1 && (heads == 1 || q.stride(1) == dim),
                    "q: heads must be contiguous within a sequence, strides are ", q.strides());
  const int32_t width = c.width(table, batch);
  c.counts("seq_len", seq_len, batch);
  if (out) same("out", *out, q.sizes(), out->scalar_type(), c.dev);
  Tensor o = out ? *out : empty(q.sizes(), out_dtype.value_or(q.scalar_type()), c.dev);
  const lk_dtype qt = dtype_of("q", q.scalar_type(), true), ot = dtype_of("out", o.scalar_type(), false);
  const int32_t b = as_i32("batch", batch), h = as_i32("n_heads", heads), m = as_i32("max_seq_len", max_seq_len);
  if (b == 0) return o;
  const size_t need = lk_paged_decode_workspace_bytes(&c.d, b, h, m, accumulate);
  const Tensor ws = scratch_for(need, m, width, c);
  check(lk_paged_decode_attn(&c.d, ptr<int32_t>(table), b, width, ptr(q), qt, h,
                             as_i32("stride of q", batch > 1 ? q.stride(0) : heads * dim), ptr<int32_t>(seq_len), m,
                             (float)softmax_scale.value_or(1.0 / std::sqrt((double)dim)), accumulate, ptr(o), ot,
                             ptr(ws), need, stream_of(c.dev)));
  return o;
}

void paged_evict(PagedCache& c, const Tensor& table, const Tensor& seq_len, const Tensor& next_pos,
                 int64_t max_seq_len, int64_t budget, int64_t window, int64_t n_sink, const OptTensor& mass_out,
                 const OptTensor& pos_out, const OptTensor& seq_len_out) {
  c.describe();
  const c10::cuda::CUDAGuard guard(c.dev);
  TORCH_CHECK_VALUE(c.mass.has_value(), "eviction needs a cache with mass and pos");
  TORCH_CHECK_VALUE(seq_len.dim() == 1, "seq_len: [batch] is needed");
  const int64_t batch = seq_len.size(0);
  const int32_t width = c.width(table, batch);
  c.counts("seq_len", seq_len, batch);
  c.counts("next_pos", next_pos, batch);
  c.counts("seq_len_out", seq_len_out, batch);
  const auto rows = c.k.sizes().slice(0, 3);
  same("mass_out", mass_out, rows, at::kFloat, c.dev);
  same("pos_out", pos_out, rows, at::kInt, c.dev);
  const int32_t b = as_i32("batch", batch), m = as_i32("max_seq_len", max_seq_len), n = as_i32("budget", budget);
  if (b == 0) return;
  const size_t need = lk_paged_evict_workspace_bytes(&c.d, b, m, n);
  const Tensor ws = scratch_for(need, m, width, c);
  check(lk_paged_evict(&c.d, ptr<int32_t>(table), b, width, ptr<int32_t>(seq_len), ptr<int32_t>(next_pos), m, n,
                       as_i32("window", window), as_i32("n_sink", n_sink),
                       mass_out ? ptr<float>(mass_out) : ptr<float>(c.mass),
                       pos_out ? ptr<int32_t>(pos_out) : ptr<int32_t>(c.pos),
                       seq_len_out ? ptr<int32_t>(seq_len_out) : ptr<int32_t>(seq_len), ptr(ws), need,
                       stream_of(c.dev)));
}

struct W4 {
  Tensor packed;
  at::Device dev;
  int32_t n_out, k_in, group, gated;

  W4(const Tensor& codes, const Tensor& scales, const OptTensor& up_codes, const OptTensor& up_scales)
      : dev(codes.device()) {
    TORCH_CHECK_VALUE(codes.dim() == 2 && scales.dim() == 2 && codes.is_cuda() && scales.size(1) > 0,
                      "codes and scales must be CUDA matrices");
    const c10::cuda::CUDAGuard guard(dev);
    n_out = as_i32("n_out", codes.size(0));
    k_in = as_i32("k_in", 2 * codes.size(1));
    group = (int32_t)(k_in / scales.size(1));
    TORCH_CHECK_VALUE(group * scales.size(1) == k_in, scales.size(1), " scale groups do not divide ", k_in, " inputs");
    TORCH_CHECK_VALUE(up_codes.has_value() == up_scales.has_value(), "up_codes and up_scales come together");
    gated = up_codes.has_value();
    const int64_t s[2] = {n_out, scales.size(1)};
    same("codes", codes, codes.sizes(), at::kByte, dev);
    same("scales", scales, s, at::kHalf, dev);
    same("up_codes", up_codes, codes.sizes(), at::kByte, dev);
    same("up_scales", up_scales, s, at::kHalf, dev);
    const size_t need = lk_w4_packed_bytes(n_out, k_in, group, gated);
    packed = scratch(need, dev);
    check(lk_w4_pack(ptr<uint8_t>(codes), ptr<uint16_t>(scales), ptr<uint8_t>(up_codes), ptr<uint16_t>(up_scales),
                     n_out, k_in, group, ptr(packed), need, stream_of(dev)));
  }
};

Tensor w4_linear(const W4& w, const Tensor& x, const OptTensor& residual, const OptTensor& y,
                 std::optional<at::ScalarType> y_dtype) {
  const c10::cuda::CUDAGuard guard(w.dev);
  TORCH_CHECK_VALUE(x.dim() == 2 && x.size(1) == w.k_in && x.stride(1) == 1 && x.device() == w.dev, "x: [m, ", w.k_in,
                    "] with contiguous rows on ", w.dev, " is needed, not ", x.sizes(), " with strides ", x.strides(),
                    " on ", x.device());
  TORCH_CHECK_VALUE((size_t)w.packed.nbytes() == lk_w4_packed_bytes(w.n_out, w.k_in, w.group, w.gated),
                    "the packed weight was resized");
  const int64_t m = x.size(0);
  const int64_t shape[2] = {m, w.n_out};
  same("residual", residual, shape, x.scalar_type(), w.dev);
  if (y) same("y", *y, shape, y->scalar_type(), w.dev);
  Tensor o = y ? *y : empty(shape, y_dtype.value_or(x.scalar_type()), w.dev);
  check(lk_w4_linear(ptr(w.packed), w.n_out, w.k_in, w.group, w.gated, ptr(x),
                     dtype_of("x", x.scalar_type(), true), as_i32("m", m),
                     as_i32("stride of x", m > 1 ? x.stride(0) : w.k_in), ptr(residual), ptr(o),
                     dtype_of("y", o.scalar_type(), false), stream_of(w.dev)));
  return o;
}

std::pair<Tensor, OptTensor> rmsnorm_gate_residual(const Tensor& y, const Tensor& x, const OptTensor& w_post,
                                                   const OptTensor& gate, double scale, const OptTensor& w_pre,
                                                   double eps, const OptTensor& x_out, const OptTensor& h) {
  const at::Device dev = y.device();
  TORCH_CHECK_VALUE(y.dim() == 2 && y.is_cuda(), "y: a CUDA matrix [m, width] is needed");
  const c10::cuda::CUDAGuard guard(dev);
  const auto t = y.scalar_type();
  const lk_dtype dt = dtype_of("y", t, false);
  const auto shape = y.sizes();
  const auto row = shape.slice(1, 1);
  const bool per_row = gate && gate->dim() == 2;
  same("y", y, shape, t, dev);
  same("x", x, shape, t, dev);
  same("w_post", w_post, row, t, dev);
  same("gate", gate, per_row ? shape : row, t, dev);
  same("w_pre", w_pre, row, t, dev);
  same("x_out", x_out, shape, t, dev);
  same("h", h, shape, t, dev);
  TORCH_CHECK_VALUE(w_pre.has_value() || !h.has_value(), "h needs w_pre");
  Tensor xo = x_out ? *x_out : empty(shape, t, dev);
  OptTensor ho = h;
  if (w_pre && !h) ho = empty(shape, t, dev);
  if (shape[0] > 0)
    check(lk_rmsnorm_gate_residual(ptr(y), ptr(x), ptr(w_post), ptr(gate), per_row, ptr(w_pre), dt,
                                   as_i32("m", shape[0]), as_i32("width", shape[1]), (float)scale, (float)eps, ptr(xo),
                                   ptr(ho), stream_of(dev)));
  return {xo, ho};
}

}  // namespace

PYBIND11_MODULE(_serving_ext, m) {
  py::class_<PagedCache>(m, "PagedCache")
      .def(py::init<Tensor, Tensor, OptTensor, OptTensor, OptTensor, OptTensor>())
      .def_readonly("k", &PagedCache::k)
      .def_readonly("v", &PagedCache::v)
      .def_readonly("k_scale", &PagedCache::k_scale)
      .def_readonly("v_scale", &PagedCache::v_scale)
      .def_readonly("mass", &PagedCache::mass)
      .def_readonly("pos", &PagedCache::pos);
  py::class_<W4>(m, "W4")
      .def(py::init<const Tensor&, const Tensor&, const OptTensor&, const OptTensor&>())
      .def_readonly("packed", &W4::packed)
      .def_readonly("n_out", &W4::n_out)
      .def_readonly("k_in", &W4::k_in)
      .def_readonly("group", &W4::group)
      .def_property_readonly("gated", [](const W4& w) { return w.gated != 0; });
  m.def("paged_append", &paged_append);
  m.def("paged_decode_attn", &paged_decode_attn);
  m.def("paged_evict", &paged_evict);
  m.def("w4_linear", &w4_linear);
  m.def("rmsnorm_gate_residual", &rmsnorm_gate_residual);
}
