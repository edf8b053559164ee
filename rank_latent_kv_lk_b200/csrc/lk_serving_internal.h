// Internal launch interfaces of the serving operators, between the C-ABI layer
// (lk_serving_api.cu) and the kernel translation units.
#pragma once

#include "lk_internal.h"
#include "lk_serving.h"

namespace lk {

// Launches with programmatic stream serialisation: the kernel may start while
// the previous one on its stream still runs, and waits for it
// (lk_grid_dep_wait) before it touches global memory.
template <typename... KArgs, typename P>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, cudaStream_t stream, const P& p,
                       size_t smem = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) count_launch();
  return e;
}

// ---------------------------------------------------------------- paged key-value cache
struct PagedCacheView {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  float* mass;
  int32_t* pos;
  int dtype;  // lk_dtype: LK_BF16, LK_F16 or LK_I8
  int n_pages, page_size, n_kv_heads, head_dim;
  const int32_t* page_table;
  int batch, table_width;
};
struct PagedAppendLaunch {
  PagedCacheView c;
  const void* k_new;
  const void* v_new;
  int x_f16;
  int token_stride, n_new;
  const int32_t* new_len;
  const int32_t* seq_len;
  int32_t* seq_len_out;
  const int32_t* next_pos;
  int32_t* next_pos_out;
};
cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t stream);

struct PagedDecodeLaunch {
  PagedCacheView c;
  const void* q;
  int q_f16;
  int n_heads, q_stride;
  const int32_t* seq_len;
  int max_len;
  int accumulate;
  float softmax_scale;
  void* out;
  int out_dtype;
  void* workspace;
  int num_sms;
};
// Work items (16-token blocks over all units) of the longest possible call.
int64_t paged_decode_max_blocks(int batch, int n_kv_heads, int group, int head_dim, int max_len);
size_t paged_decode_workspace_bytes(int batch, int n_kv_heads, int n_heads, int head_dim, int dtype, int max_len,
                                    int accumulate, int num_sms);
cudaError_t launch_paged_decode(const PagedDecodeLaunch& a, cudaStream_t stream);

struct PagedEvictLaunch {
  PagedCacheView c;
  const int32_t* seq_len;
  const int32_t* next_pos;
  int max_len, budget, window, n_sink;
  float* mass_out;
  int32_t* pos_out;
  int32_t* seq_len_out;
  void* workspace;
  int num_sms;
};
size_t paged_evict_workspace_bytes(int units, int max_len, int budget);
cudaError_t launch_paged_evict(const PagedEvictLaunch& a, cudaStream_t stream);

// ---------------------------------------------------------------- 4-bit weights
size_t w4_packed_bytes(int n_out, int k_in, int group, int gated);
cudaError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* up_codes,
                           const uint16_t* up_scales, int n_out, int k_in, int group, void* packed,
                           cudaStream_t stream);
struct W4Launch {
  const void* packed;
  int n_out, k_in, group, gated;
  const void* x;
  int x_f16, m, x_stride;
  const void* residual;
  void* y;
  int y_dtype;
  int num_sms;
};
cudaError_t launch_w4_linear(const W4Launch& a, cudaStream_t stream);

// ---------------------------------------------------------------- norms around a block
struct BlockNormLaunch {
  const void* y;
  const void* x;
  const void* w_post;
  const void* gate;
  const void* w_pre;
  void* x_out;
  void* h;
  int gate_per_row, dtype, m, width;
  float scale, eps;
};
cudaError_t launch_block_norm(const BlockNormLaunch& a, cudaStream_t stream);

}  // namespace lk
