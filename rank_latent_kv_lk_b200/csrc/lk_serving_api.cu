// C ABI of the serving operators: host-side validation and dispatch for every
// entry point in lk_serving.h.  Nothing is launched and nothing is written
// unless every check passes.
#include <cstdarg>
#include <cstdio>

#include "lk_serving_internal.h"

namespace lk {
lk_status set_error(lk_status s, const char* msg);  // for lk_last_error()
}

namespace {

lk_status fail(lk_status s, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return lk::set_error(s, msg);
}

lk_status cuda_fail(cudaError_t e, const char* where) {
  return fail(LK_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether two buffers (null: none) share a byte.
bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + b_bytes && y < x + a_bytes;
}

size_t size_of(lk_dtype t) { return t == LK_F32 ? 4 : (t == LK_I8 ? 1 : 2); }

int num_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------- paged key-value cache
namespace {
constexpr int64_t kMaxSlots = (int64_t)1 << 30;  // of a sequence: sizes made from it stay within 32 bits

bool is_16bit(lk_dtype t) { return t == LK_BF16 || t == LK_F16; }

lk_status check_paged(const lk_paged_cache* c, int32_t batch, int32_t table_width) {
  if (!c) return fail(LK_ERR_INVALID_ARG, "null paged cache");
  if (c->dtype != LK_BF16 && c->dtype != LK_F16 && c->dtype != LK_I8)
    return fail(LK_ERR_DTYPE, "paged cache dtype must be LK_BF16, LK_F16 or LK_I8");
  if (c->n_pages < 1) return fail(LK_ERR_SHAPE, "n_pages %d < 1", c->n_pages);
  if (c->page_size < 1 || c->page_size > LK_MAX_PAGE_SIZE || (c->page_size & (c->page_size - 1)) != 0)
    return fail(LK_ERR_SHAPE, "page_size %d must be a power of two up to %d", c->page_size, LK_MAX_PAGE_SIZE);
  if (c->n_kv_heads < 1 || c->n_kv_heads > LK_MAX_HEADS)
    return fail(LK_ERR_SHAPE, "n_kv_heads %d outside [1, %d]", c->n_kv_heads, LK_MAX_HEADS);
  if (c->head_dim < 16 || c->head_dim > LK_MAX_HEAD_DIM || c->head_dim % 16 != 0)
    return fail(LK_ERR_SHAPE, "head_dim %d must be a multiple of 16 in [16, %d]", c->head_dim, LK_MAX_HEAD_DIM);
  if ((int64_t)c->n_pages * c->n_kv_heads * c->page_size >= (int64_t)1 << 31)
    return fail(LK_ERR_SHAPE, "n_pages * n_kv_heads * page_size must stay below 2^31");
  if (batch < 1 || table_width < 1) return fail(LK_ERR_SHAPE, "batch %d or table_width %d < 1", batch, table_width);
  if ((int64_t)table_width * c->page_size > kMaxSlots)
    return fail(LK_ERR_SHAPE, "table_width * page_size must be at most 2^30");
  if ((int64_t)batch * LK_MAX_HEADS >= (int64_t)1 << 31) return fail(LK_ERR_SHAPE, "batch %d too large", batch);
  return LK_OK;
}

lk_status check_paged_buffers(const lk_paged_cache* c, const int32_t* page_table) {
  if (!c->k || !c->v || !page_table) return fail(LK_ERR_INVALID_ARG, "null k, v or page_table");
  if ((c->dtype == LK_I8) != (c->k_scale != nullptr) || (c->dtype == LK_I8) != (c->v_scale != nullptr))
    return fail(LK_ERR_INVALID_ARG, "k_scale and v_scale belong to an int8 cache, and only to it");
  if ((c->mass != nullptr) != (c->pos != nullptr)) return fail(LK_ERR_INVALID_ARG, "mass and pos come together");
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
      !aligned(c->mass, 16) || !aligned(c->pos, 16) || !aligned(page_table, 4))
    return fail(LK_ERR_ALIGN, "the cache's arrays must be 16-byte aligned");
  return LK_OK;
}

lk::PagedCacheView paged_view(const lk_paged_cache* c, const int32_t* page_table, int batch, int width) {
  return {c->k,       c->v,        c->k_scale,    c->v_scale,  c->mass,    c->pos, (int)c->dtype,
          c->n_pages, c->page_size, c->n_kv_heads, c->head_dim, page_table, batch,  width};
}

lk_status check_max_len(const lk_paged_cache* c, int32_t table_width, int32_t max_seq_len) {
  if (max_seq_len < 0 || max_seq_len > (int64_t)table_width * c->page_size)
    return fail(LK_ERR_SHAPE, "max_seq_len %d outside [0, table_width * page_size]", max_seq_len);
  return LK_OK;
}

lk_status check_decode_heads(const lk_paged_cache* c, int32_t batch, int32_t n_heads, int32_t max_seq_len) {
  if (n_heads < 1 || n_heads > LK_MAX_HEADS || n_heads % c->n_kv_heads != 0)
    return fail(LK_ERR_SHAPE, "n_heads %d must be a multiple of n_kv_heads %d, at most %d", n_heads, c->n_kv_heads,
                LK_MAX_HEADS);
  if (lk::paged_decode_max_blocks(batch, c->n_kv_heads, n_heads / c->n_kv_heads, c->head_dim, max_seq_len) >=
      (int64_t)1 << 30)
    return fail(LK_ERR_SHAPE, "batch * heads * max_seq_len too large");
  return LK_OK;
}
}  // namespace

lk_status lk_paged_append(const lk_paged_cache* cache, const int32_t* page_table, int32_t batch, int32_t table_width,
                          const void* k_new, const void* v_new, lk_dtype x_dtype, int32_t token_stride, int32_t n_new,
                          const int32_t* new_len, const int32_t* seq_len, int32_t* seq_len_out,
                          const int32_t* next_pos, int32_t* next_pos_out, lk_stream_t stream) {
  lk_status s;
  if ((s = check_paged(cache, batch, table_width)) != LK_OK) return s;
  if ((s = check_paged_buffers(cache, page_table)) != LK_OK) return s;
  if (!is_16bit(x_dtype) || (cache->dtype != LK_I8 && x_dtype != cache->dtype))
    return fail(LK_ERR_DTYPE, "x dtype must be the cache's (LK_BF16 or LK_F16 for an int8 cache)");
  if (n_new < 1) return fail(LK_ERR_SHAPE, "n_new %d < 1", n_new);
  if ((int64_t)batch * n_new >= (int64_t)1 << 31) return fail(LK_ERR_SHAPE, "batch * n_new too large");
  if (!k_new || !v_new || !seq_len || !seq_len_out)
    return fail(LK_ERR_INVALID_ARG, "null k_new, v_new, seq_len or seq_len_out");
  if (token_stride % 8 != 0) return fail(LK_ERR_ALIGN, "token_stride %d must be a multiple of 8", token_stride);
  if (token_stride < cache->n_kv_heads * cache->head_dim)
    return fail(LK_ERR_SHAPE, "token_stride %d < n_kv_heads * head_dim", token_stride);
  if (!aligned(k_new, 16) || !aligned(v_new, 16)) return fail(LK_ERR_ALIGN, "k_new and v_new must be 16-byte aligned");
  const size_t len_b = (size_t)batch * 4;
  if ((seq_len_out != seq_len && overlap(seq_len_out, len_b, seq_len, len_b)) ||
      (next_pos_out != next_pos && overlap(next_pos_out, len_b, next_pos, len_b)) ||
      overlap(seq_len_out, len_b, next_pos, len_b) || overlap(seq_len_out, len_b, next_pos_out, len_b) ||
      overlap(next_pos_out, len_b, seq_len, len_b) || overlap(seq_len_out, len_b, new_len, len_b) ||
      overlap(next_pos_out, len_b, new_len, len_b))
    return fail(LK_ERR_INVALID_ARG, "seq_len_out is seq_len and next_pos_out is next_pos, or they overlap no other");
  if ((cache->mass != nullptr) != (next_pos != nullptr) || (next_pos != nullptr) != (next_pos_out != nullptr))
    return fail(LK_ERR_INVALID_ARG, "next_pos and next_pos_out belong to a cache with mass, and only to it");
  lk::PagedAppendLaunch a{};
  a.c = paged_view(cache, page_table, batch, table_width);
  a.k_new = k_new;
  a.v_new = v_new;
  a.x_f16 = x_dtype == LK_F16;
  a.token_stride = token_stride;
  a.n_new = n_new;
  a.new_len = new_len;
  a.seq_len = seq_len;
  a.seq_len_out = seq_len_out;
  a.next_pos = next_pos;
  a.next_pos_out = next_pos_out;
  cudaError_t e = lk::launch_paged_append(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lk_paged_append");
  return LK_OK;
}

size_t lk_paged_decode_workspace_bytes(const lk_paged_cache* cache, int32_t batch, int32_t n_heads,
                                       int32_t max_seq_len, int32_t accumulate) {
  if (check_paged(cache, batch, 1) != LK_OK || max_seq_len < 0 || max_seq_len > kMaxSlots ||
      check_decode_heads(cache, batch, n_heads, max_seq_len) != LK_OK)
    return 0;
  return lk::paged_decode_workspace_bytes(batch, cache->n_kv_heads, n_heads, cache->head_dim, cache->dtype,
                                          max_seq_len, accumulate, num_sms());
}

lk_status lk_paged_decode_attn(const lk_paged_cache* cache, const int32_t* page_table, int32_t batch,
                               int32_t table_width, const void* q, lk_dtype q_dtype, int32_t n_heads,
                               int32_t q_stride, const int32_t* seq_len, int32_t max_seq_len, float softmax_scale,
                               int32_t accumulate, void* out, lk_dtype out_dtype, void* workspace,
                               size_t workspace_bytes, lk_stream_t stream) {
  lk_status s;
  if ((s = check_paged(cache, batch, table_width)) != LK_OK) return s;
  if ((s = check_paged_buffers(cache, page_table)) != LK_OK) return s;
  if ((s = check_max_len(cache, table_width, max_seq_len)) != LK_OK) return s;
  if ((s = check_decode_heads(cache, batch, n_heads, max_seq_len)) != LK_OK) return s;
  if (!is_16bit(q_dtype) || (cache->dtype != LK_I8 && q_dtype != cache->dtype))
    return fail(LK_ERR_DTYPE, "q dtype must be the cache's (LK_BF16 or LK_F16 for an int8 cache)");
  if (out_dtype != LK_F32 && !is_16bit(out_dtype))
    return fail(LK_ERR_DTYPE, "out dtype must be LK_F32, LK_BF16 or LK_F16");
  if (!q || !seq_len || !out) return fail(LK_ERR_INVALID_ARG, "null q, seq_len or out");
  if (q_stride % 8 != 0) return fail(LK_ERR_ALIGN, "q_stride %d must be a multiple of 8", q_stride);
  if (q_stride < n_heads * cache->head_dim) return fail(LK_ERR_SHAPE, "q_stride %d < n_heads * head_dim", q_stride);
  if (!aligned(q, 16) || !aligned(out, 16)) return fail(LK_ERR_ALIGN, "q and out must be 16-byte aligned");
  if (overlap(q, ((size_t)(batch - 1) * q_stride + (size_t)n_heads * cache->head_dim) * 2, out,
              (size_t)batch * n_heads * cache->head_dim * size_of(out_dtype)))
    return fail(LK_ERR_INVALID_ARG, "out must not overlap q");
  if (accumulate != 0 && accumulate != 1) return fail(LK_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  if (accumulate && !cache->mass) return fail(LK_ERR_INVALID_ARG, "accumulate needs a cache with mass");
  if (!(softmax_scale == softmax_scale)) return fail(LK_ERR_INVALID_ARG, "softmax_scale is NaN");
  const int sms = num_sms();
  const size_t need = lk::paged_decode_workspace_bytes(batch, cache->n_kv_heads, n_heads, cache->head_dim,
                                                       cache->dtype, max_seq_len, accumulate, sms);
  if (!workspace || workspace_bytes < need)
    return fail(LK_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace_bytes);
  if (!aligned(workspace, 256)) return fail(LK_ERR_ALIGN, "workspace must be 256-byte aligned");
  lk::PagedDecodeLaunch a{};
  a.c = paged_view(cache, page_table, batch, table_width);
  a.q = q;
  a.q_f16 = q_dtype == LK_F16;
  a.n_heads = n_heads;
  a.q_stride = q_stride;
  a.seq_len = seq_len;
  a.max_len = max_seq_len;
  a.accumulate = accumulate;
  a.softmax_scale = softmax_scale;
  a.out = out;
  a.out_dtype = out_dtype;
  a.workspace = workspace;
  a.num_sms = sms;
  cudaError_t e = lk::launch_paged_decode(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lk_paged_decode_attn");
  return LK_OK;
}

size_t lk_paged_evict_workspace_bytes(const lk_paged_cache* cache, int32_t batch, int32_t max_seq_len,
                                      int32_t budget) {
  if (check_paged(cache, batch, 1) != LK_OK || max_seq_len < 0 || max_seq_len > kMaxSlots || budget < 1) return 0;
  return lk::paged_evict_workspace_bytes(batch * cache->n_kv_heads, max_seq_len, budget);
}

lk_status lk_paged_evict(const lk_paged_cache* cache, const int32_t* page_table, int32_t batch, int32_t table_width,
                         const int32_t* seq_len, const int32_t* next_pos, int32_t max_seq_len, int32_t budget,
                         int32_t window, int32_t n_sink, float* mass_out, int32_t* pos_out, int32_t* seq_len_out,
                         void* workspace, size_t workspace_bytes, lk_stream_t stream) {
  lk_status s;
  if ((s = check_paged(cache, batch, table_width)) != LK_OK) return s;
  if ((s = check_paged_buffers(cache, page_table)) != LK_OK) return s;
  if (!cache->mass) return fail(LK_ERR_INVALID_ARG, "eviction needs a cache with mass and pos");
  if ((s = check_max_len(cache, table_width, max_seq_len)) != LK_OK) return s;
  if (budget < 1) return fail(LK_ERR_SHAPE, "budget %d < 1", budget);
  if (window < 0 || n_sink < 0) return fail(LK_ERR_SHAPE, "window %d or n_sink %d < 0", window, n_sink);
  if (!seq_len || !next_pos || !mass_out || !pos_out || !seq_len_out)
    return fail(LK_ERR_INVALID_ARG, "null seq_len, next_pos, mass_out, pos_out or seq_len_out");
  if ((mass_out == cache->mass) != (pos_out == cache->pos))
    return fail(LK_ERR_INVALID_ARG, "either both or neither of mass_out and pos_out are the cache's own");
  if (!aligned(mass_out, 16) || !aligned(pos_out, 16))
    return fail(LK_ERR_ALIGN, "mass_out and pos_out must be 16-byte aligned");
  const size_t len_b = (size_t)batch * 4;
  if ((seq_len_out != seq_len && overlap(seq_len_out, len_b, seq_len, len_b)) ||
      overlap(seq_len_out, len_b, next_pos, len_b))
    return fail(LK_ERR_INVALID_ARG, "seq_len_out is seq_len or overlaps neither it nor next_pos");
  const size_t row_bytes = (size_t)cache->n_pages * cache->n_kv_heads * cache->page_size * 4;
  if ((mass_out != cache->mass && overlap(mass_out, row_bytes, cache->mass, row_bytes)) ||
      (pos_out != cache->pos && overlap(pos_out, row_bytes, cache->pos, row_bytes)) ||
      overlap(mass_out, row_bytes, cache->pos, row_bytes) || overlap(pos_out, row_bytes, cache->mass, row_bytes) ||
      overlap(mass_out, row_bytes, pos_out, row_bytes))
    return fail(LK_ERR_INVALID_ARG, "mass_out and pos_out are the cache's own or overlap neither them nor each other");
  const size_t need = lk::paged_evict_workspace_bytes(batch * cache->n_kv_heads, max_seq_len, budget);
  if (!workspace || workspace_bytes < need)
    return fail(LK_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu", need, workspace_bytes);
  if (!aligned(workspace, 256)) return fail(LK_ERR_ALIGN, "workspace must be 256-byte aligned");
  lk::PagedEvictLaunch a{};
  a.c = paged_view(cache, page_table, batch, table_width);
  a.seq_len = seq_len;
  a.next_pos = next_pos;
  a.max_len = max_seq_len;
  a.budget = budget;
  a.window = window;
  a.n_sink = n_sink;
  a.mass_out = mass_out;
  a.pos_out = pos_out;
  a.seq_len_out = seq_len_out;
  a.workspace = workspace;
  a.num_sms = num_sms();
  cudaError_t e = lk::launch_paged_evict(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lk_paged_evict");
  return LK_OK;
}

// ---------------------------------------------------------------- 4-bit weights
namespace {
lk_status check_w4(int32_t n_out, int32_t k_in, int32_t group) {
  if (group != 32 && group != 64 && group != 128) return fail(LK_ERR_SHAPE, "group %d must be 32, 64 or 128", group);
  if (n_out < 1 || k_in < 1 || k_in % group != 0)
    return fail(LK_ERR_SHAPE, "n_out %d must be positive and k_in %d a positive multiple of the group", n_out, k_in);
  if (n_out > (1 << 24) || k_in > (1 << 24)) return fail(LK_ERR_SHAPE, "n_out %d or k_in %d too large", n_out, k_in);
  return LK_OK;
}
}  // namespace

size_t lk_w4_packed_bytes(int32_t n_out, int32_t k_in, int32_t group, int32_t gated) {
  if (check_w4(n_out, k_in, group) != LK_OK) return 0;
  return lk::w4_packed_bytes(n_out, k_in, group, gated != 0);
}

lk_status lk_w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* up_codes, const uint16_t* up_scales,
                     int32_t n_out, int32_t k_in, int32_t group, void* packed, size_t packed_bytes,
                     lk_stream_t stream) {
  lk_status s;
  if ((s = check_w4(n_out, k_in, group)) != LK_OK) return s;
  if (!codes || !scales || !packed) return fail(LK_ERR_INVALID_ARG, "null codes, scales or packed");
  if ((up_codes != nullptr) != (up_scales != nullptr))
    return fail(LK_ERR_INVALID_ARG, "up_codes and up_scales come together");
  if (!aligned(codes, 4) || !aligned(up_codes, 4) || !aligned(scales, 2) || !aligned(up_scales, 2))
    return fail(LK_ERR_ALIGN, "codes must be 4-byte and scales 2-byte aligned");
  if (!aligned(packed, 256)) return fail(LK_ERR_ALIGN, "packed must be 256-byte aligned");
  const size_t need = lk::w4_packed_bytes(n_out, k_in, group, up_codes != nullptr);
  if (packed_bytes < need) return fail(LK_ERR_WORKSPACE, "packed needs %zu bytes, got %zu", need, packed_bytes);
  cudaError_t e = lk::launch_w4_pack(codes, scales, up_codes, up_scales, n_out, k_in, group, packed,
                                     reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lk_w4_pack");
  return LK_OK;
}

lk_status lk_w4_linear(const void* packed, int32_t n_out, int32_t k_in, int32_t group, int32_t gated, const void* x,
                       lk_dtype x_dtype, int32_t m, int32_t x_stride, const void* residual, void* y, lk_dtype y_dtype,
                       lk_stream_t stream) {
  lk_status s;
  if ((s = check_w4(n_out, k_in, group)) != LK_OK) return s;
  if (gated != 0 && gated != 1) return fail(LK_ERR_INVALID_ARG, "gated must be 0 or 1");
  if (!is_16bit(x_dtype)) return fail(LK_ERR_DTYPE, "x dtype must be LK_BF16 or LK_F16");
  if (y_dtype != LK_F32 && !is_16bit(y_dtype)) return fail(LK_ERR_DTYPE, "y dtype must be LK_F32, LK_BF16 or LK_F16");
  if (m < 0 || m > 65535 * 32) return fail(LK_ERR_SHAPE, "m %d outside [0, %d]", m, 65535 * 32);
  if (!packed || (m > 0 && (!x || !y))) return fail(LK_ERR_INVALID_ARG, "null packed, x or y");
  if (x_stride < k_in) return fail(LK_ERR_SHAPE, "x_stride %d < k_in %d", x_stride, k_in);
  if (x_stride % 8 != 0) return fail(LK_ERR_ALIGN, "x_stride %d must be a multiple of 8", x_stride);
  if (residual && gated) return fail(LK_ERR_UNSUPPORTED, "a gated weight takes no residual");
  if (residual && residual == y && x_dtype != y_dtype)
    return fail(LK_ERR_INVALID_ARG, "residual can be y only in y's type");
  if (!aligned(packed, 256)) return fail(LK_ERR_ALIGN, "packed must be 256-byte aligned");
  if (!aligned(x, 16) || !aligned(y, 16) || !aligned(residual, 16))
    return fail(LK_ERR_ALIGN, "x, y and residual must be 16-byte aligned");
  const size_t y_bytes = (size_t)m * n_out * size_of(y_dtype);
  if (m > 0 && overlap(x, ((size_t)(m - 1) * x_stride + k_in) * 2, y, y_bytes))
    return fail(LK_ERR_INVALID_ARG, "y must not overlap x");
  if (residual != y && overlap(residual, (size_t)m * n_out * 2, y, y_bytes))
    return fail(LK_ERR_INVALID_ARG, "residual is y or does not overlap it");
  lk::W4Launch a{};
  a.packed = packed;
  a.n_out = n_out;
  a.k_in = k_in;
  a.group = group;
  a.gated = gated;
  a.x = x;
  a.x_f16 = x_dtype == LK_F16;
  a.m = m;
  a.x_stride = x_stride;
  a.residual = residual;
  a.y = y;
  a.y_dtype = y_dtype;
  a.num_sms = num_sms();
  cudaError_t e = lk::launch_w4_linear(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lk_w4_linear");
  return LK_OK;
}

lk_status lk_rmsnorm_gate_residual(const void* y, const void* x, const void* w_post, const void* gate,
                                   int32_t gate_per_row, const void* w_pre, lk_dtype dtype, int32_t m, int32_t width,
                                   float scale, float eps, void* x_out, void* h, lk_stream_t stream) {
  if (dtype != LK_F32 && !is_16bit(dtype)) return fail(LK_ERR_DTYPE, "dtype must be LK_F32, LK_BF16 or LK_F16");
  if (m < 0 || width < 1 || width > 32768) return fail(LK_ERR_SHAPE, "m %d / width %d outside range", m, width);
  if (m > 0 && (!y || !x || !x_out)) return fail(LK_ERR_INVALID_ARG, "null y, x or x_out");
  if ((w_pre != nullptr) != (h != nullptr)) return fail(LK_ERR_INVALID_ARG, "w_pre and h come together");
  if (h && (h == x_out || h == x)) return fail(LK_ERR_INVALID_ARG, "h can be y, not x or x_out");
  if (gate_per_row != 0 && gate_per_row != 1) return fail(LK_ERR_INVALID_ARG, "gate_per_row must be 0 or 1");
  if (!(eps >= 0.0f)) return fail(LK_ERR_INVALID_ARG, "eps must be >= 0");
  if (!(scale == scale)) return fail(LK_ERR_INVALID_ARG, "scale is NaN");
  const size_t es = dtype == LK_F32 ? 4 : 2;
  for (const void* t : {y, x, w_post, gate, w_pre, (const void*)x_out, (const void*)h})
    if (!aligned(t, es)) return fail(LK_ERR_ALIGN, "pointers must be aligned to their elements");
  const size_t rows_b = (size_t)m * width * es, row_b = (size_t)width * es;
  for (const void* o : {(const void*)x_out, (const void*)h}) {
    if ((o != y && overlap(o, rows_b, y, rows_b)) || (o != x && overlap(o, rows_b, x, rows_b)) ||
        overlap(o, rows_b, w_post, row_b) || overlap(o, rows_b, w_pre, row_b) ||
        overlap(o, rows_b, gate, gate_per_row ? rows_b : row_b))
      return fail(LK_ERR_INVALID_ARG, "an output is y or x (h: y) or overlaps no input");
  }
  if (overlap(x_out, rows_b, h, rows_b)) return fail(LK_ERR_INVALID_ARG, "x_out and h overlap");
  lk::BlockNormLaunch a{};
  a.y = y;
  a.x = x;
  a.w_post = w_post;
  a.gate = gate;
  a.w_pre = w_pre;
  a.x_out = x_out;
  a.h = h;
  a.gate_per_row = gate_per_row;
  a.dtype = dtype;
  a.m = m;
  a.width = width;
  a.scale = scale;
  a.eps = eps;
  cudaError_t e = lk::launch_block_norm(a, reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "lk_rmsnorm_gate_residual");
  return LK_OK;
}

}  // extern "C"
