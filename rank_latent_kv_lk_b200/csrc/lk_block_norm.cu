// The norms around a block with its gate and residual scale (sm_100a):
//   x_out = x + scale * gate . (RMSNorm(y) . w_post),  h = RMSNorm(x_out) . w_pre
// HBM-bound: y, x (and a gate per row) are read once, x_out and h written once.
// One CTA per row: a thread keeps its elements of the row in registers between
// the two block-wide sums of squares, so nothing is read twice, and the row is
// read whole before any of it is written (x_out may be x or y, h may be y).
#include "lk_serving.cuh"

namespace {

struct NormParams {
  const void* y;
  const void* x;
  const void* w_post;
  const void* gate;
  const void* w_pre;
  void* x_out;
  void* h;
  int width, gate_per_row;
  float scale, eps;
};

enum { T_F32 = 0, T_BF16 = 1, T_F16 = 2 };

// VEC consecutive elements as fp32: one 16-byte access (VEC 8 of 16 bits, 4
// of 32) or, for widths and pointers that do not allow it, single ones.
template <int T, int VEC>
LK_DEVICE void load_vec(const void* p, int64_t at, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (T == T_F32) f[0] = static_cast<const float*>(p)[at];
    else if constexpr (T == T_BF16) f[0] = lk_bf16_to_f32(static_cast<const uint16_t*>(p)[at]);
    else f[0] = lk_f16_to_f32(static_cast<const uint16_t*>(p)[at]);
  } else if constexpr (T == T_F32) {
    const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (T == T_BF16) {
        f[2 * e] = lk_bf16lo(u[e]);
        f[2 * e + 1] = lk_bf16hi(u[e]);
      } else {
        const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&u[e]));
        f[2 * e] = g.x;
        f[2 * e + 1] = g.y;
      }
    }
  }
}

template <int T, int VEC>
LK_DEVICE void store_vec(void* p, int64_t at, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (T == T_F32) static_cast<float*>(p)[at] = f[0];
    else if constexpr (T == T_BF16) static_cast<uint16_t*>(p)[at] = lk_f32_to_bf16(f[0]);
    else static_cast<uint16_t*>(p)[at] = lk_f32_to_f16_bits(f[0]);
  } else if constexpr (T == T_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    uint32_t u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      u[e] = T == T_BF16 ? lk_pack_bf16x2(f[2 * e], f[2 * e + 1]) : lk_pack_f16x2(f[2 * e], f[2 * e + 1]);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

LK_DEVICE float block_sum(float v, float* buf) {
  v = lk_warp_sum(v);
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < warps; ++w) s += buf[w];
  return s;
}

// The row's elements of thread t: vectors t, t + blockDim, ...
template <int T, int VEC, int R>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float buf[2][32];
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const int64_t row = (int64_t)blockIdx.x * p.width;
  float y[R][VEC], x[R][VEC];
  float ss = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC;
#pragma unroll
    for (int e = 0; e < VEC; ++e) y[r][e] = x[r][e] = 0.0f;
    if (c < p.width) {
      load_vec<T, VEC>(p.y, row + c, y[r]);
      load_vec<T, VEC>(p.x, row + c, x[r]);
    }
  }
  float rstd = 1.0f;
  if (p.w_post) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(y[r][e], y[r][e], ss);
    rstd = 1.0f / sqrtf(block_sum(ss, buf[0]) / (float)p.width + p.eps);
  }
  ss = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC;
    if (c < p.width) {
      float w[VEC];
      if (p.w_post) {
        load_vec<T, VEC>(p.w_post, c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[r][e] *= rstd * w[e];
      }
      if (p.gate) {
        load_vec<T, VEC>(p.gate, p.gate_per_row ? row + c : c, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) y[r][e] *= w[e];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        x[r][e] = fmaf(p.scale, y[r][e], x[r][e]);
        ss = fmaf(x[r][e], x[r][e], ss);
      }
    }
  }
  __syncthreads();  // every thread has read its part of the row
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC;
    if (c < p.width) store_vec<T, VEC>(p.x_out, row + c, x[r]);
  }
  if (!p.h) return;
  rstd = 1.0f / sqrtf(block_sum(ss, buf[1]) / (float)p.width + p.eps);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC;
    if (c < p.width) {
      float w[VEC];
      load_vec<T, VEC>(p.w_pre, c, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) x[r][e] *= rstd * w[e];
      store_vec<T, VEC>(p.h, row + c, x[r]);
    }
  }
}

template <int T, int VEC>
cudaError_t launch_t(const NormParams& p, int m, cudaStream_t stream) {
  // one vector a thread up to 1024 threads, then several
  const int vecs = (p.width + VEC - 1) / VEC;
  const int threads = std::min(1024, (vecs + 31) / 32 * 32);
  const int r = (vecs + threads - 1) / threads;
  const dim3 g(m), b(threads);
  if (r <= 1) return lk::launch_pdl(block_norm_kernel<T, VEC, 1>, g, b, stream, p);
  if (r <= 2) return lk::launch_pdl(block_norm_kernel<T, VEC, 2>, g, b, stream, p);
  if (r <= 4) return lk::launch_pdl(block_norm_kernel<T, VEC, 4>, g, b, stream, p);
  if constexpr (VEC < 8) {
    if (r <= 8) return lk::launch_pdl(block_norm_kernel<T, VEC, 8>, g, b, stream, p);
    if constexpr (VEC == 1) return lk::launch_pdl(block_norm_kernel<T, VEC, 32>, g, b, stream, p);
  }
  return cudaErrorInvalidValue;  // width <= 32768 is checked by the caller
}

template <int T>
cudaError_t launch_v(const NormParams& p, int m, cudaStream_t stream) {
  constexpr int V = T == T_F32 ? 4 : 8;
  auto ok = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  const bool wide = p.width % V == 0 && ok(p.y) && ok(p.x) && ok(p.w_post) && ok(p.gate) && ok(p.w_pre) &&
                    ok(p.x_out) && ok(p.h);
  return wide ? launch_t<T, V>(p, m, stream) : launch_t<T, 1>(p, m, stream);
}

}  // namespace

namespace lk {

cudaError_t launch_block_norm(const BlockNormLaunch& a, cudaStream_t stream) {
  if (a.m == 0) return cudaSuccess;
  NormParams p{a.y, a.x, a.w_post, a.gate, a.w_pre, a.x_out, a.h, a.width, a.gate_per_row, a.scale, a.eps};
  if (a.dtype == LK_F32) return launch_v<T_F32>(p, a.m, stream);
  if (a.dtype == LK_BF16) return launch_v<T_BF16>(p, a.m, stream);
  return launch_v<T_F16>(p, a.m, stream);
}

}  // namespace lk
