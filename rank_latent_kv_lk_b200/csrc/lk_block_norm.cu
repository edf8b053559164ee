// The norms around a block with its gate and residual scale (sm_100a):
//   x_out = x + scale * gate . (RMSNorm(y) . w_post),  h = RMSNorm(x_out) . w_pre
// HBM-bound: y, x (and a gate per row) are read once, x_out and h written once
// (4096 rows of 4096, fp16, gate per row, 168 MB: 28.9 us a call, 90 % of the
// measured copy bandwidth, 26.8 in a captured graph; 32 rows: 5.6 us a call, the
// host's part of it, 2.2 in a graph, the latency of one row).
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
  float scale, eps, inv_width;
};

enum { T_F32 = 0, T_BF16 = 1, T_F16 = 2 };

// VEC consecutive elements as they lie in memory: one 16-byte access (VEC 8 of
// 16 bits, 4 of 32) or, for widths and pointers that do not allow it, one.
template <int T, int VEC>
struct Raw {
  uint32_t u[VEC == 1 ? 1 : 4];
  LK_DEVICE void load(const void* p, int64_t at) {
    if constexpr (VEC > 1) {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + at * (16 / VEC));
      u[0] = v.x; u[1] = v.y; u[2] = v.z; u[3] = v.w;
    } else if constexpr (T == T_F32) {
      u[0] = static_cast<const uint32_t*>(p)[at];
    } else {
      u[0] = static_cast<const uint16_t*>(p)[at];
    }
  }
  LK_DEVICE void zero() {
#pragma unroll
    for (int e = 0; e < (VEC == 1 ? 1 : 4); ++e) u[e] = 0;
  }
  LK_DEVICE void unpack(float (&f)[VEC]) const {
    if constexpr (T == T_F32) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] = __uint_as_float(u[e]);
    } else if constexpr (VEC == 1) {
      f[0] = T == T_BF16 ? lk_bf16_to_f32((uint16_t)u[0]) : lk_f16_to_f32((uint16_t)u[0]);
    } else {
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
};

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
  const int lane = threadIdx.x & 31;
  if (lane == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  return lk_warp_sum(lane < (int)(blockDim.x >> 5) ? buf[lane] : 0.0f);
}

// Elements [c, c + VEC) of a vector whose start is 16-byte aligned, c a multiple
// of VEC plus s (the same for the whole block): two aligned accesses, shifted.
template <int T, int VEC>
LK_DEVICE void load_shifted(Raw<T, VEC>& r, const void* p, int c, int s) {
  if constexpr (VEC > 1) {
    Raw<T, VEC> a, b;
    a.load(p, c - s);
    b.load(p, c - s + VEC);
    uint32_t u[8] = {a.u[0], a.u[1], a.u[2], a.u[3], b.u[0], b.u[1], b.u[2], b.u[3]};
    const int words = T == T_F32 ? s : s >> 1;
    if (words & 2)
#pragma unroll
      for (int e = 0; e < 6; ++e) u[e] = u[e + 2];
    if (words & 1)
#pragma unroll
      for (int e = 0; e < 6; ++e) u[e] = u[e + 1];
    if (T != T_F32 && (s & 1))
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = __funnelshift_r(u[e], u[e + 1], 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) r.u[e] = u[e];
  }
}

// The row's elements of thread t: vectors t, t + blockDim, ...  Everything a
// row reads is requested at once (up to two vectors a thread; more keep the
// weights and gate for when they are used, to save registers).
template <int T, int VEC, int R>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr bool kEarly = R <= 2;
  using V = Raw<T, VEC>;
  __shared__ float buf[2][32];
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const int64_t row = (int64_t)blockIdx.x * p.width;
  const int64_t gate_row = p.gate_per_row ? row : 0;
  V y[R], x[R], g[kEarly ? R : 1], wq[kEarly ? R : 1], wp[kEarly ? R : 1];
  float z[R][VEC];
  float ss = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC;
    y[r].zero();
    if (c < p.width) {
      y[r].load(p.y, row + c);
      x[r].load(p.x, row + c);
      if constexpr (kEarly) {
        if (p.gate) g[r].load(p.gate, gate_row + c);
        if (p.w_post) wp[r].load(p.w_post, c);
        if (p.w_pre) wq[r].load(p.w_pre, c);
      }
    }
  }
  float rstd = 1.0f;
  if (p.w_post) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float f[VEC];
      y[r].unpack(f);
#pragma unroll
      for (int e = 0; e < VEC; ++e) ss = fmaf(f[e], f[e], ss);
    }
    rstd = rsqrtf(fmaf(block_sum(ss, buf[0]), p.inv_width, p.eps));
  }
  ss = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC;
    if (c < p.width) {
      V& w1 = wp[kEarly ? r : 0];
      V& w2 = g[kEarly ? r : 0];
      if constexpr (!kEarly) {
        if (p.w_post) w1.load(p.w_post, c);
        if (p.gate) w2.load(p.gate, gate_row + c);
      }
      float f[VEC], w[VEC];
      y[r].unpack(f);
      if (p.w_post) {
        w1.unpack(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] *= rstd * w[e];
      }
      if (p.gate) {
        w2.unpack(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] *= w[e];
      }
      x[r].unpack(w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        z[r][e] = fmaf(p.scale, f[e], w[e]);
        ss = fmaf(z[r][e], z[r][e], ss);
      }
    }
  }
  // every thread has read its part of the row before any of it is written
  if (p.h) rstd = rsqrtf(fmaf(block_sum(ss, buf[1]), p.inv_width, p.eps));
  else __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC;
    if (c < p.width) {
      store_vec<T, VEC>(p.x_out, row + c, z[r]);
      if (p.h) {
        V& w3 = wq[kEarly ? r : 0];
        if constexpr (!kEarly) w3.load(p.w_pre, c);
        float w[VEC];
        w3.unpack(w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) z[r][e] *= rstd * w[e];
        store_vec<T, VEC>(p.h, row + c, z[r]);
      }
    }
  }
}

// The same for widths that are no multiple of a vector (tensors 16-byte
// aligned): vectors start at the aligned element at or before the row's first,
// so rows are read and written with whole accesses except for a vector at each
// end, which goes element by element.  The weights are met at an offset that
// is the same for the whole row (load_shifted).
template <int T, int VEC, int R>
__global__ void __launch_bounds__(1024) block_norm_odd_kernel(const __grid_constant__ NormParams p) {
  using V = Raw<T, VEC>;
  __shared__ float buf[2][32];
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const int64_t row = (int64_t)blockIdx.x * p.width;
  const int mis = (int)(row % VEC);        // elements of the first vector that belong to the row before
  const int s = (VEC - mis) % VEC;         // column of the first whole vector
  V y[R], x[R];
  float z[R][VEC];
  // elements c .. c + VEC - 1 of a row's tensor one by one, 0 outside the row
  auto get_each = [&](V& v, const void* t, int64_t base, int c) {
    v.zero();
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (c + e >= 0 && c + e < p.width) {
        Raw<T, 1> one;
        one.load(t, base + c + e);
        if constexpr (T == T_F32) v.u[e] = one.u[0];
        else v.u[e >> 1] |= one.u[0] << (16 * (e & 1));
      }
    }
  };
  auto get = [&](V& v, const void* t, int64_t base, int c) {
    if (c >= 0 && c + VEC <= p.width) v.load(t, base + c);
    else get_each(v, t, base, c);
  };
  auto get_weight = [&](V& v, const void* t, int c) {
    if (s == 0) get(v, t, 0, c);
    else if (c >= s && c - s + 2 * VEC <= p.width) load_shifted<T, VEC>(v, t, c, s);
    else get_each(v, t, 0, c);
  };
  auto put = [&](void* t, int c, const float (&f)[VEC]) {
    if (c >= 0 && c + VEC <= p.width) {
      store_vec<T, VEC>(t, row + c, f);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (c + e >= 0 && c + e < p.width) {
          const float g[1] = {f[e]};
          store_vec<T, 1>(t, row + c + e, g);
        }
    }
  };
  float ss = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC - mis;
    get(y[r], p.y, row, c);
    get(x[r], p.x, row, c);
    float f[VEC];
    y[r].unpack(f);
#pragma unroll
    for (int e = 0; e < VEC; ++e) ss = fmaf(f[e], f[e], ss);
  }
  const float rstd = p.w_post ? rsqrtf(fmaf(block_sum(ss, buf[0]), p.inv_width, p.eps)) : 1.0f;
  ss = 0.0f;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC - mis;
    if (c >= p.width) continue;
    float f[VEC], w[VEC];
    V v;
    y[r].unpack(f);
    if (p.w_post) {
      get_weight(v, p.w_post, c);
      v.unpack(w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] *= rstd * w[e];
    }
    if (p.gate) {
      if (p.gate_per_row) get(v, p.gate, row, c);
      else get_weight(v, p.gate, c);
      v.unpack(w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f[e] *= w[e];
    }
    x[r].unpack(w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      z[r][e] = fmaf(p.scale, f[e], w[e]);
      if (c + e >= 0 && c + e < p.width) ss = fmaf(z[r][e], z[r][e], ss);
    }
  }
  float rstd2 = 0.0f;
  if (p.h) rstd2 = rsqrtf(fmaf(block_sum(ss, buf[1]), p.inv_width, p.eps));
  else __syncthreads();
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int c = (r * blockDim.x + threadIdx.x) * VEC - mis;
    if (c >= p.width) continue;
    put(p.x_out, c, z[r]);
    if (p.h) {
      float w[VEC];
      V v;
      get_weight(v, p.w_pre, c);
      v.unpack(w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) z[r][e] *= rstd2 * w[e];
      put(p.h, c, z[r]);
    }
  }
}

template <int T, int VEC>
cudaError_t launch_odd(const NormParams& p, int m, cudaStream_t stream) {
  const int vecs = (p.width + 2 * VEC - 2) / VEC;  // a vector more where both ends are cut
  const int threads = std::min(1024, (vecs + 31) / 32 * 32);
  const int r = (vecs + threads - 1) / threads;
  const dim3 g(m), b(threads);
  if (r <= 1) return lk::launch_pdl(block_norm_odd_kernel<T, VEC, 1>, g, b, stream, p);
  if (r <= 2) return lk::launch_pdl(block_norm_odd_kernel<T, VEC, 2>, g, b, stream, p);
  if (r <= 5) return lk::launch_pdl(block_norm_odd_kernel<T, VEC, 5>, g, b, stream, p);
  if constexpr (T == T_F32) return lk::launch_pdl(block_norm_odd_kernel<T, VEC, 9>, g, b, stream, p);
  return cudaErrorInvalidValue;  // width <= 32768 is checked by the caller
}

template <int T, int VEC>
cudaError_t launch_t(const NormParams& p, int m, cudaStream_t stream) {
  // few rows: one vector a thread, for the shortest way through a row; many: two, for fewer warps to wait for at
  // the sums (4096 rows of 4096, fp16, gate per row: 26.8 us against 30.8)
  const int vecs = (p.width + VEC - 1) / VEC;
  const int each = m >= 256 && vecs >= 128 ? 2 : 1;
  const int threads = std::min(1024, ((vecs + each - 1) / each + 31) / 32 * 32);
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
  const bool all = ok(p.y) && ok(p.x) && ok(p.w_post) && ok(p.gate) && ok(p.w_pre) && ok(p.x_out) && ok(p.h);
  if (!all) return launch_t<T, 1>(p, m, stream);
  if (p.width % V == 0) return launch_t<T, V>(p, m, stream);
  // Cut vectors pay from some width or size on.  In a graph, against element by element, fp16: 64 rows of 1023 3.3 us
  // against 1.9, of 2051 3.4 against 2.7, of 4099 3.6 against 4.2, of 8197 6.0 against 11.6; 256 of 2051 3.6 against
  // 4.0; 1024 of 515 3.7 against 3.3, of 1023 6.0 against 5.1, of 1541 6.1 against 8.3; 4096 of 1023 12.5 against 17.0.
  // fp32: 64 rows of 2051 2.8 against 2.6, of 8197 7.2 against 12.1; 1024 of 1023 4.7 against 5.0.
  return p.width >= 2048 || (int64_t)m * p.width >= 1 << 20 ? launch_odd<T, V>(p, m, stream)
                                                            : launch_t<T, 1>(p, m, stream);
}

}  // namespace

namespace lk {

cudaError_t launch_block_norm(const BlockNormLaunch& a, cudaStream_t stream) {
  if (a.m == 0) return cudaSuccess;
  NormParams p{a.y,     a.x,     a.w_post,       a.gate,  a.w_pre, a.x_out,
               a.h,     a.width, a.gate_per_row, a.scale, a.eps,   1.0f / (float)a.width};
  if (a.dtype == LK_F32) return launch_v<T_F32>(p, a.m, stream);
  if (a.dtype == LK_BF16) return launch_v<T_BF16>(p, a.m, stream);
  return launch_v<T_F16>(p, a.m, stream);
}

}  // namespace lk
