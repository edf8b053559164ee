// Products of a few rows with 4-bit weights under group scales (sm_100a).
//
//   y[m, n] = sum_g s[n, g] sum_{k in g} c[n, k] x[m, k]  (+ residual), or
//   silu(y_gate) * y_up for a gated weight.
// Bound by the weights' bytes (n k / 2 of codes and 2 n k / group of scales)
// up to the 32 rows of one pass.
//
// Layout (lk_w4_pack).  A tile is 16 outputs x 64 inputs: one 16-byte word
// group per lane, in the order of the operand A of four m16n8k16 products, so
// a warp's load of a tile is 512 consecutive bytes and needs no shuffle.  Lane
// (gid, tig) holds outputs gid and gid + 8 at inputs 8 tig .. 8 tig + 7 of each
// 32 (a sum over inputs may take them in any order inside its scale group, and
// eight consecutive inputs of x are one 16-byte load); word q belongs to
// product q, and nibble i of its low and high half are the two inputs of
// register a_i.  Nibbles hold
// code + 8, so that one and-or makes a register: 128 + n in bf16, 1024 + n in
// fp16, and one exact subtract takes the offset off.  K is padded to 128
// inputs, outputs to 16, with zero codes and scales.  Tiles of gate and up of
// the same outputs are neighbours.  Scales follow the codes: per (16 outputs,
// group, matrix) eight pairs (outputs gid, gid + 8).
//
// Codes and x are exact operands, sums run in fp32, and a group's sum is
// scaled in fp32, so the result is rounded once.
//
// One CTA per 16 outputs (and both matrices), its 8 warps taking 128 inputs in
// turn; the warps' sums meet in shared memory.
#include "lk_serving.cuh"

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStep = 128;  // inputs a warp takes at a time

struct W4Params {
  const uint4* codes;      // [tiles][kc][mats][32]
  const uint32_t* scales;  // [tiles][groups][mats][8]
  const uint16_t* x;
  const uint16_t* residual;
  void* y;
  int n_out, k_in, steps, m, x_stride, y_dtype;
};

template <bool F16>
LK_DEVICE uint32_t codes16(uint32_t w, int i) {
  uint32_t h, r;
  if constexpr (F16) {
    h = ((w >> (4 * i)) & 0x000F000Fu) | 0x64006400u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64086408u));
  } else {
    h = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x43084308u));
  }
  return r;
}

template <bool F16>
LK_DEVICE float from16(uint16_t u) {
  if constexpr (F16) return lk_f16_to_f32(u);
  else return lk_bf16_to_f32(u);
}

template <int GROUP, int MT, int MATS, bool F16>
__global__ void __launch_bounds__(kThreads) w4_kernel(const __grid_constant__ W4Params p) {
  __shared__ float red[kWarps][MATS][8 * MT][17];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int tile = blockIdx.x, m0 = blockIdx.y * 32;
  constexpr int kGroups = kStep / GROUP;  // scale groups of a step
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const uint4* codes = p.codes + (int64_t)tile * p.steps * 2 * MATS * 32 + lane;
  const uint32_t* scales = p.scales + (int64_t)tile * p.steps * kGroups * MATS * 8 + gid;

  float acc[MATS][MT][4] = {};
  uint4 w[2][MATS];
  auto load_codes = [&](int s) {
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int a = 0; a < MATS; ++a) w[c][a] = __ldcg(codes + ((int64_t)(2 * s + c) * MATS + a) * 32);
  };
  int s = warp;
  if (s < p.steps) load_codes(s);
  for (; s < p.steps; s += kWarps) {
    uint4 cur[2][MATS];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int a = 0; a < MATS; ++a) cur[c][a] = w[c][a];
    if (s + kWarps < p.steps) load_codes(s + kWarps);
    uint32_t sc[kGroups][MATS];
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int a = 0; a < MATS; ++a) sc[g][a] = __ldcg(scales + ((int64_t)(s * kGroups + g) * MATS + a) * 8);
    float part[MATS][MT][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t xr[MT][8];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int row = m0 + 8 * t + gid;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int k = s * kStep + c * 64 + 32 * j + 8 * tig;
          uint4 v = make_uint4(0, 0, 0, 0);
          if (row < p.m && k < p.k_in) v = *reinterpret_cast<const uint4*>(p.x + (int64_t)row * p.x_stride + k);
          xr[t][4 * j] = v.x;
          xr[t][4 * j + 1] = v.y;
          xr[t][4 * j + 2] = v.z;
          xr[t][4 * j + 3] = v.w;
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = c * 64 + q * 16;  // inputs of the step before this product
        const bool first = at % GROUP == 0, last = (at + 16) % GROUP == 0;
#pragma unroll
        for (int a = 0; a < MATS; ++a) {
          const uint32_t word = q == 0 ? cur[c][a].x : (q == 1 ? cur[c][a].y : (q == 2 ? cur[c][a].z : cur[c][a].w));
          const uint32_t a0 = codes16<F16>(word, 0), a1 = codes16<F16>(word, 1);
          const uint32_t a2 = codes16<F16>(word, 2), a3 = codes16<F16>(word, 3);
          const uint32_t sw = sc[at / GROUP][a];
          const float s0 = lk_f16_to_f32((uint16_t)sw), s1 = lk_f16_to_f32((uint16_t)(sw >> 16));
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            float (&pt)[4] = part[a][t];
            if (first) pt[0] = pt[1] = pt[2] = pt[3] = 0.0f;
            if constexpr (F16) lk_mma_f16_16816(pt, a0, a1, a2, a3, xr[t][2 * q], xr[t][2 * q + 1]);
            else lk_mma_bf16_16816(pt, a0, a1, a2, a3, xr[t][2 * q], xr[t][2 * q + 1]);
            if (last) {
              acc[a][t][0] = fmaf(s0, pt[0], acc[a][t][0]);
              acc[a][t][1] = fmaf(s0, pt[1], acc[a][t][1]);
              acc[a][t][2] = fmaf(s1, pt[2], acc[a][t][2]);
              acc[a][t][3] = fmaf(s1, pt[3], acc[a][t][3]);
            }
          }
        }
      }
    }
  }

  // ---- the warps' sums, [row of x][output]
#pragma unroll
  for (int a = 0; a < MATS; ++a)
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      red[warp][a][8 * t + 2 * tig][gid] = acc[a][t][0];
      red[warp][a][8 * t + 2 * tig + 1][gid] = acc[a][t][1];
      red[warp][a][8 * t + 2 * tig][gid + 8] = acc[a][t][2];
      red[warp][a][8 * t + 2 * tig + 1][gid + 8] = acc[a][t][3];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 8 * MT * 16; i += kThreads) {
    const int r = i >> 4, c = i & 15;
    const int row = m0 + r, n = tile * 16 + c;
    if (row >= p.m || n >= p.n_out) continue;
    float v = 0.0f;
#pragma unroll
    for (int wp = 0; wp < kWarps; ++wp) v += red[wp][0][r][c];
    if constexpr (MATS == 2) {
      float u = 0.0f;
#pragma unroll
      for (int wp = 0; wp < kWarps; ++wp) u += red[wp][1][r][c];
      v = v / (1.0f + expf(-v)) * u;
    }
    const int64_t at = (int64_t)row * p.n_out + n;
    if (p.residual) v += from16<F16>(p.residual[at]);
    if (p.y_dtype == LK_F32) reinterpret_cast<float*>(p.y)[at] = v;
    else reinterpret_cast<uint16_t*>(p.y)[at] = p.y_dtype == LK_BF16 ? lk_f32_to_bf16(v) : lk_f32_to_f16_bits(v);
  }
}

// ---------------------------------------------------------------- layout
// One thread per 32-bit word of the packed codes, then one per scale pair.
__global__ void w4_pack_kernel(const uint8_t* __restrict__ codes0, const uint8_t* __restrict__ codes1,
                               const uint16_t* __restrict__ scales0, const uint16_t* __restrict__ scales1, int n_out,
                               int k_in, int group, int mats, int tiles, int steps, uint32_t* __restrict__ out) {
  const int64_t words = (int64_t)tiles * steps * 2 * mats * 128;
  const int groups = steps * (kStep / group);
  const int64_t pairs = (int64_t)tiles * groups * mats * 8;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words + pairs;
       i += (int64_t)gridDim.x * blockDim.x) {
    if (i < words) {
      const int q = (int)(i & 3), lane = (int)((i >> 2) & 31);
      int64_t r = i >> 7;
      const int a = (int)(r % mats);
      r /= mats;
      const int c = (int)(r % (2 * steps)), tile = (int)(r / (2 * steps));
      const int gid = lane >> 2, tig = lane & 3;
      const int k = c * 64 + 32 * (q >> 1) + 8 * tig + 4 * (q & 1);  // inputs k .. k + 3 of two outputs
      const uint8_t* src = a ? codes1 : codes0;
      uint32_t w = 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int n = tile * 16 + gid + 8 * half;
        // two bytes, four codes; code + 8 is the nibble with its top bit flipped
        uint32_t four = 0x8888u;
        if (n < n_out && k < k_in) {
          const uint8_t* b = src + (int64_t)n * (k_in / 2) + k / 2;
          four = ((uint32_t)b[0] | ((uint32_t)b[1] << 8)) ^ 0x8888u;
        }
        // register a_half: inputs k, k + 1; a_(2 + half): k + 2, k + 3
        w |= (four & 15u) << (4 * half) | ((four >> 4) & 15u) << (4 * half + 16);
        w |= ((four >> 8) & 15u) << (4 * half + 8) | ((four >> 12) & 15u) << (4 * half + 24);
      }
      out[i] = w;
    } else {
      int64_t r = i - words;
      const int gid = (int)(r & 7);
      r >>= 3;
      const int a = (int)(r % mats);
      r /= mats;
      const int g = (int)(r % groups), tile = (int)(r / groups);
      const uint16_t* src = a ? scales1 : scales0;
      uint32_t w = 0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int n = tile * 16 + gid + 8 * half;
        if (n < n_out && g * group < k_in) w |= (uint32_t)src[(int64_t)n * (k_in / group) + g] << (16 * half);
      }
      out[i] = w;
    }
  }
}

int tiles_of(int n_out) { return (n_out + 15) / 16; }
int steps_of(int k_in) { return (k_in + kStep - 1) / kStep; }
size_t code_bytes(int n_out, int k_in, int gated) {
  return (size_t)tiles_of(n_out) * steps_of(k_in) * 2 * (gated ? 2 : 1) * 512;
}

template <int GROUP, int MT, int MATS>
cudaError_t launch2(const W4Params& p, dim3 grid, bool f16, cudaStream_t stream) {
  if (f16) return lk::launch_pdl(w4_kernel<GROUP, MT, MATS, true>, grid, dim3(kThreads), stream, p);
  return lk::launch_pdl(w4_kernel<GROUP, MT, MATS, false>, grid, dim3(kThreads), stream, p);
}
template <int GROUP, int MATS>
cudaError_t launch1(const W4Params& p, dim3 grid, bool f16, cudaStream_t stream) {
  if (p.m <= 8) return launch2<GROUP, 1, MATS>(p, grid, f16, stream);
  if (p.m <= 16) return launch2<GROUP, 2, MATS>(p, grid, f16, stream);
  return launch2<GROUP, 4, MATS>(p, grid, f16, stream);
}
template <int GROUP>
cudaError_t launch0(const W4Params& p, dim3 grid, bool f16, bool gated, cudaStream_t stream) {
  return gated ? launch1<GROUP, 2>(p, grid, f16, stream) : launch1<GROUP, 1>(p, grid, f16, stream);
}

}  // namespace

namespace lk {

size_t w4_packed_bytes(int n_out, int k_in, int group, int gated) {
  return code_bytes(n_out, k_in, gated) +
         (size_t)tiles_of(n_out) * steps_of(k_in) * (kStep / group) * (gated ? 2 : 1) * 32;
}

cudaError_t launch_w4_pack(const uint8_t* codes, const uint16_t* scales, const uint8_t* up_codes,
                           const uint16_t* up_scales, int n_out, int k_in, int group, void* packed,
                           cudaStream_t stream) {
  const int mats = up_codes ? 2 : 1;
  const size_t items = w4_packed_bytes(n_out, k_in, group, mats == 2) / 4;
  const unsigned grid = (unsigned)std::min<size_t>((items + 255) / 256, 65536);
  w4_pack_kernel<<<grid, 256, 0, stream>>>(codes, up_codes, scales, up_scales, n_out, k_in, group, mats,
                                           tiles_of(n_out), steps_of(k_in), static_cast<uint32_t*>(packed));
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) count_launch();
  return e;
}

cudaError_t launch_w4_linear(const W4Launch& a, cudaStream_t stream) {
  if (a.m == 0) return cudaSuccess;
  W4Params p{};
  p.codes = static_cast<const uint4*>(a.packed);
  p.scales = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.packed) +
                                               code_bytes(a.n_out, a.k_in, a.gated));
  p.x = static_cast<const uint16_t*>(a.x);
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.y = a.y;
  p.n_out = a.n_out;
  p.k_in = a.k_in;
  p.steps = steps_of(a.k_in);
  p.m = a.m;
  p.x_stride = a.x_stride;
  p.y_dtype = a.y_dtype;
  const dim3 grid(tiles_of(a.n_out), (a.m + 31) / 32);
  if (a.group == 32) return launch0<32>(p, grid, a.x_f16, a.gated, stream);
  if (a.group == 64) return launch0<64>(p, grid, a.x_f16, a.gated, stream);
  return launch0<128>(p, grid, a.x_f16, a.gated, stream);
}

}  // namespace lk
