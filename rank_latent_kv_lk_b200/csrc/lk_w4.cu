// Products of a few rows with 4-bit weights under group scales (sm_100a).
//
//   y[m, n] = sum_g s[n, g] sum_{k in g} c[n, k] x[m, k]  (+ residual), or
//   silu(y_gate) * y_up for a gated weight.
// The floor is the weights' bytes (n k / 2 of codes and 2 n k / group of
// scales) up to the 32 rows of one pass.  No one unit is full: one row,
// SwiGLU, 2 x 11008 x 4096 12.6 us a call, 4.0 TB/s: schedulers issue in 56 % of
// the cycles (most of it the expansion of the codes) at 23 % of the warps an SM
// holds; eight rows, 4096 x 11008 11.1 us: the same 56 %, every CTA copies all
// of x, as many bytes as its weights, and 20 SMs have no CTA; 32 rows of the
// first 28.0 us: warps wait most for the tensor and arithmetic pipes.  bf16, one
// row, 4096 x 4096 4.7 us a call, 4.2 in a captured graph.
//
// Layout (lk_w4_pack).  A tile is 16 outputs x 64 inputs: one 16-byte word
// group per lane, in the order of the operand A of four m16n8k16 products, so
// that a lane uses exactly the 16 bytes it fetched.  Lane (gid, tig) holds
// outputs gid and gid + 8 at inputs 8 tig .. 8 tig + 7 of each 32 (a sum over
// inputs may take them in any order inside its scale group, and eight
// consecutive inputs of x are one 16-byte access); word q belongs to product
// q, and nibble i of its low and high half are the two inputs of register
// a_i.  Nibbles hold code + 8, so that one and-or makes a register: 128 + n in
// bf16, 1024 + n in fp16, and one exact subtract takes the offset off.  A step
// is 128 inputs: per matrix (gate, then up) two tiles, then per matrix and
// group eight pairs of scales (outputs gid, gid + 8).  The steps of 16 outputs
// follow one another; inputs are padded to 128 and outputs to 16 with zero
// codes and scales.
//
// Codes and x are exact operands, sums run in fp32, and a group's sum is
// scaled in fp32, so the result is rounded once.
//
// One CTA an SM where that is one wave: tn tiles of 16 outputs by kn parts of
// K, a warp each.  A warp's steps stream through its own ring in shared memory
// (cp.async, no barrier), and with them its part of a single row of x; more
// rows are staged once for the tn warps of a part of K, which one named
// barrier a step keeps together.  The parts' sums meet in shared memory.
#include <atomic>
#include <climits>

#include "lk_serving.cuh"

namespace {

constexpr int kMaxWarps = 16;
constexpr int kMaxTiles = 8;   // tiles of 16 outputs a CTA
constexpr int kStep = 128;     // inputs a warp takes at a time
constexpr int kMaxSmem = 226 * 1024;
constexpr int kXStride = 320;  // bytes between x rows of a step: eight lanes of two rows read 32 banks

struct W4Params {
  const uint8_t* packed;
  const uint16_t* x;
  const uint16_t* residual;
  void* y;
  int n_out, k_in, steps, full_steps, tiles, tn, kn, m, x_stride, y_dtype;
};

__host__ __device__ constexpr int record_bytes(int group, int mats) { return mats * (1024 + (kStep / group) * 32); }

// R: rows of x at most (1, 8, 16 or 32).
template <int GROUP, int R, int MATS>
struct W4Shape {
  static constexpr int kMT = R <= 8 ? 1 : R / 8;   // products side by side
  static constexpr bool kShared = R > 1;           // x is staged for several warps
  static constexpr int kRec = record_bytes(GROUP, MATS);
  static constexpr int kStages = R <= 8 ? (MATS == 2 ? 4 : (R == 1 ? 6 : 5)) : 3;
  static constexpr int kXStage = R * kXStride;
  static constexpr int kStage = kRec + (kShared ? 0 : kXStage);  // a warp's own
  static constexpr int kRedRow = 17;
  static constexpr int kRed = MATS * 8 * kMT * kRedRow * 4;  // one warp's sums
  static constexpr int kMaxParts = kShared ? 8 : kMaxWarps;  // parts of K that stage x: one named barrier each
  static int smem(int tn, int kn) {
    const int ring = tn * kn * kStages * kStage + (kShared ? kn * kStages * kXStage : 0);
    return std::max(ring, tn * kn * kRed);
  }
};

LK_DEVICE void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
LK_DEVICE void cp16_zfill(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
LK_DEVICE uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
LK_DEVICE uint32_t lds4(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// (a & b) | c
LK_DEVICE uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// The four registers of a product from a word of codes.  fp16: nibbles 1 and 3
// are taken where they lie (1024 + 16 n), and a multiply-add brings them down,
// which saves two shifts; bf16's mantissa has room for the lowest nibble only.
template <bool F16>
LK_DEVICE void codes16(uint32_t w, uint32_t (&a)[4]) {
  if constexpr (F16) {
    const uint32_t v = w >> 8;
    const uint32_t h[4] = {and_or(w, 0x000F000Fu, 0x64006400u), and_or(w, 0x00F000F0u, 0x64006400u),
                           and_or(v, 0x000F000Fu, 0x64006400u), and_or(v, 0x00F000F0u, 0x64006400u)};
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(a[i]) : "r"(h[i]), "r"(0x64086408u));
      // (1024 + 16 n) / 16 - 72
      asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(a[i + 1]) : "r"(h[i + 1]), "r"(0x2C002C00u), "r"(0xD480D480u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("sub.rn.bf16x2 %0, %1, %2;"
          : "=r"(a[i])
          : "r"(and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u)), "r"(0x43084308u));
  }
}

template <bool F16>
LK_DEVICE float from16(uint16_t u) {
  if constexpr (F16) return lk_f16_to_f32(u);
  else return lk_bf16_to_f32(u);
}

// D = A B (+ C): the first product of a group starts from zero.
template <bool F16>
LK_DEVICE void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

template <int GROUP, int R, int MATS, bool F16>
__global__ void __launch_bounds__(kMaxWarps * 32, 1) w4_kernel(const __grid_constant__ W4Params p) {
  using S = W4Shape<GROUP, R, MATS>;
  constexpr int MT = S::kMT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int wk = warp / p.tn, wn = warp - wk * p.tn;  // part of K, tile
  const int tile = blockIdx.x * p.tn + wn, m0 = blockIdx.y * 32;
  const bool mine = tile < p.tiles;
  const int rows = min(R, p.m - m0);
  const uint32_t ring = lk_smem_addr(smem) + warp * (S::kStages * S::kStage);
  // x of stage i: behind the warp's record, or in the part's own buffer
  const uint32_t xbuf = S::kShared ? lk_smem_addr(smem) + p.tn * p.kn * (S::kStages * S::kStage) +
                                         wk * (S::kStages * S::kXStage)
                                   : ring + S::kRec;
  constexpr int kXStep = S::kShared ? S::kXStage : S::kStage;
  // While the kernel before still runs: the records that the ring will ask for first, into L2 (no value is used, so
  // that it does not matter who wrote them when).  Rows of 11008: 13.5 us -> 12.5; eight or more records ahead 13.3.
  if (mine) {
    const uint8_t* first = p.packed + ((int64_t)tile * p.steps + wk) * S::kRec;
    for (int i = 0; i < S::kStages - 1 && wk + i * p.kn < p.steps; ++i, first += (int64_t)p.kn * S::kRec)
      if (lane * 128 < S::kRec) asm volatile("prefetch.global.L2 [%0];" ::"l"(first + lane * 128));
  }
  lk_grid_dep_wait();
  lk_grid_dep_launch();

  // the next step's record and x into a stage of the ring
  const uint8_t* src = p.packed + ((int64_t)(mine ? tile : 0) * p.steps + wk) * S::kRec + 16 * lane;
  const int64_t src_step = (int64_t)p.kn * S::kRec;
  int next = wk;
  // this lane's 16 bytes of x: chunk lane % 16 of every (2 tn)th (its own ring: 2nd) row.  Rows behind the last are
  // never filled: a column of a product is one row, and theirs are not stored.
  const int x_c = lane & 15, x_r = (S::kShared ? 2 * wn : 0) + (lane >> 4), x_rows = S::kShared ? 2 * p.tn : 2;
  const uint16_t* xsrc = p.x + (int64_t)(m0 + min(x_r, rows - 1)) * p.x_stride + 8 * x_c + wk * kStep;
  const int64_t x_next = (int64_t)x_rows * p.x_stride;
  auto fetch = [&](int stage) {
    if (next < p.steps) {
      if (mine) {
        const uint32_t dst = ring + stage * S::kStage + 16 * lane;
#pragma unroll
        for (int i = 0; i < S::kRec; i += 512)
          if (i + 512 <= S::kRec || i + 16 * lane < S::kRec) cp16(dst + i, src + i);
      }
      const uint32_t xd = xbuf + stage * kXStep;
      const uint32_t xl = xd + x_r * kXStride + 16 * x_c;
      const uint16_t* xs = xsrc;
      if (next < p.full_steps) {
        if constexpr (S::kShared) {
          for (int r = x_r; r < rows; r += x_rows, xs += x_next) cp16(xl + (r - x_r) * kXStride, xs);
        } else {
#pragma unroll
          for (int i = 0; i < (R + 1) / 2; ++i, xs += x_next)
            if (x_r + 2 * i < rows) cp16(xl + 2 * i * kXStride, xs);
        }
      } else {  // inputs end inside the step
        const bool in = next * kStep + 8 * x_c < p.k_in;
        for (int r = x_r; r < rows; r += x_rows, xs += x_next)
          cp16_zfill(xl + (r - x_r) * kXStride, in ? xs : p.x, in);
      }
      xsrc += p.kn * kStep;
      src += src_step;
      next += p.kn;
    }
    lk_cp_async_commit();
  };

  float acc[MATS][MT][4] = {};
  int stage = 0;
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) fetch(i);
  for (int s = wk; s < p.steps; s += p.kn) {
    lk_cp_async_wait<S::kStages - 2>();  // this step has arrived
    if constexpr (S::kShared) asm volatile("bar.sync %0, %1;" ::"r"(1 + wk), "r"(p.tn * 32) : "memory");
    else __syncwarp();                   // and every lane is done with the one before
    fetch(stage == 0 ? S::kStages - 1 : stage - 1);
    if (mine) {
      const uint32_t rec = ring + stage * S::kStage;
      const uint32_t xs = xbuf + stage * kXStep + (R > 1 ? gid * kXStride : 0) + 16 * tig;
      float part[MATS][MT][4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint4 code[MATS];
#pragma unroll
        for (int a = 0; a < MATS; ++a) code[a] = lds16(rec + (2 * a + c) * 512 + 16 * lane);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint4 xr[MT];
#pragma unroll
          for (int t = 0; t < MT; ++t) {
            // one row: all eight columns hold it, and the first is used
            xr[t] = lds16(xs + t * 8 * kXStride + (2 * c + j) * 64);
          }
#pragma unroll
          for (int qq = 0; qq < 2; ++qq) {
            const int q = 2 * j + qq;
            const int at = c * 64 + q * 16;  // inputs of the step before this product
            const bool first = at % GROUP == 0, last = (at + 16) % GROUP == 0;
#pragma unroll
            for (int a = 0; a < MATS; ++a) {
              const uint32_t word = q == 0 ? code[a].x : (q == 1 ? code[a].y : (q == 2 ? code[a].z : code[a].w));
              uint32_t A[4];
              codes16<F16>(word, A);
              float s0 = 0.0f, s1 = 0.0f;
              if (last) {
                const uint32_t sw = lds4(rec + MATS * 1024 + (a * (kStep / GROUP) + at / GROUP) * 32 + 4 * gid);
                s0 = lk_f16_to_f32((uint16_t)sw);
                s1 = lk_f16_to_f32((uint16_t)(sw >> 16));
              }
#pragma unroll
              for (int t = 0; t < MT; ++t) {
                float (&pt)[4] = part[a][t];
                const uint32_t b0 = qq ? xr[t].z : xr[t].x, b1 = qq ? xr[t].w : xr[t].y;
                if (first) mma_first<F16>(pt, A[0], A[1], A[2], A[3], b0, b1);
                else if constexpr (F16) lk_mma_f16_16816(pt, A[0], A[1], A[2], A[3], b0, b1);
                else lk_mma_bf16_16816(pt, A[0], A[1], A[2], A[3], b0, b1);
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
    }
    if (++stage == S::kStages) stage = 0;
  }

  // ---- the parts' sums, [row of x][output]
  lk_cp_async_wait<0>();
  __syncthreads();
  float* red = reinterpret_cast<float*>(smem);
  {
    float* r = red + warp * (S::kRed / 4);
#pragma unroll
    for (int a = 0; a < MATS; ++a)
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        float* q = r + ((a * MT + t) * 8 + 2 * tig) * S::kRedRow + gid;
        q[0] = acc[a][t][0];
        q[S::kRedRow] = acc[a][t][1];
        q[8] = acc[a][t][2];
        q[S::kRedRow + 8] = acc[a][t][3];
      }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.tn * 16 * rows; i += blockDim.x) {
    const int r = i / (p.tn * 16), o = i - r * (p.tn * 16), t = o >> 4, c = o & 15;
    const int n = blockIdx.x * p.tn * 16 + o, row = m0 + r;
    if (n >= p.n_out) continue;
    const float* q = red + t * (S::kRed / 4) + r * S::kRedRow + c;
    float v = 0.0f, u = 0.0f;
    for (int k = 0; k < p.kn; ++k) {
      v += q[k * p.tn * (S::kRed / 4)];
      if constexpr (MATS == 2) u += q[k * p.tn * (S::kRed / 4) + MT * 8 * S::kRedRow];
    }
    if constexpr (MATS == 2) v = v / (1.0f + expf(-v)) * u;
    const int64_t at = (int64_t)row * p.n_out + n;
    if (p.residual) v += from16<F16>(p.residual[at]);
    if (p.y_dtype == LK_F32) reinterpret_cast<float*>(p.y)[at] = v;
    else reinterpret_cast<uint16_t*>(p.y)[at] = p.y_dtype == LK_BF16 ? lk_f32_to_bf16(v) : lk_f32_to_f16_bits(v);
  }
}

// ---------------------------------------------------------------- layout
// One thread per 32-bit word of the packed weight.
__global__ void w4_pack_kernel(const uint8_t* __restrict__ codes0, const uint8_t* __restrict__ codes1,
                               const uint16_t* __restrict__ scales0, const uint16_t* __restrict__ scales1, int n_out,
                               int k_in, int group, int mats, int tiles, int steps, uint32_t* __restrict__ out) {
  const int groups = kStep / group, rec = record_bytes(group, mats) / 4;
  const int64_t words = (int64_t)tiles * steps * rec;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t ts = i / rec;
    const int at = (int)(i - ts * rec), tile = (int)(ts / steps), step = (int)(ts - (int64_t)tile * steps);
    uint32_t w = 0;
    if (at < mats * 256) {
      const int a = at >> 8, c = (at >> 7) & 1, lane = (at >> 2) & 31, q = at & 3;
      const int gid = lane >> 2, tig = lane & 3;
      // inputs k .. k + 3 of two outputs
      const int k = step * kStep + c * 64 + 32 * (q >> 1) + 8 * tig + 4 * (q & 1);
      const uint8_t* src = a ? codes1 : codes0;
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
    } else {
      const int r = at - mats * 256, gid = r & 7, g = step * groups + (r >> 3) % groups, a = (r >> 3) / groups;
      const uint16_t* src = a ? scales1 : scales0;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int n = tile * 16 + gid + 8 * half;
        if (n < n_out && g * group < k_in) w |= (uint32_t)src[(int64_t)n * (k_in / group) + g] << (16 * half);
      }
    }
    out[i] = w;
  }
}

int tiles_of(int n_out) { return (n_out + 15) / 16; }
int steps_of(int k_in) { return (k_in + kStep - 1) / kStep; }

template <int GROUP, int R, int MATS, bool F16>
cudaError_t launch3(W4Params p, dim3 grid, cudaStream_t stream) {
  using S = W4Shape<GROUP, R, MATS>;
  p.kn = std::max(1, std::min({kMaxWarps / p.tn, p.steps, S::kMaxParts}));
  while (p.kn > 1 && S::smem(p.tn, p.kn) > kMaxSmem) --p.kn;
  static std::atomic<uint64_t> ready{0};  // devices whose shared memory limit is raised (bit = number)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(w4_kernel<GROUP, R, MATS, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  return lk::launch_pdl(w4_kernel<GROUP, R, MATS, F16>, grid, dim3(p.tn * p.kn * 32), stream, p,
                        S::smem(p.tn, p.kn));
}
template <int GROUP, int R, int MATS>
cudaError_t launch2(const W4Params& p, dim3 grid, bool f16, cudaStream_t stream) {
  return f16 ? launch3<GROUP, R, MATS, true>(p, grid, stream) : launch3<GROUP, R, MATS, false>(p, grid, stream);
}
template <int GROUP, int MATS>
cudaError_t launch1(const W4Params& p, dim3 grid, bool f16, cudaStream_t stream) {
  if (p.m == 1) return launch2<GROUP, 1, MATS>(p, grid, f16, stream);
  if (p.m <= 8) return launch2<GROUP, 8, MATS>(p, grid, f16, stream);
  if (p.m <= 16) return launch2<GROUP, 16, MATS>(p, grid, f16, stream);
  return launch2<GROUP, 32, MATS>(p, grid, f16, stream);
}
template <int GROUP>
cudaError_t launch0(const W4Params& p, dim3 grid, bool f16, bool gated, cudaStream_t stream) {
  return gated ? launch1<GROUP, 2>(p, grid, f16, stream) : launch1<GROUP, 1>(p, grid, f16, stream);
}

}  // namespace

namespace lk {

size_t w4_packed_bytes(int n_out, int k_in, int group, int gated) {
  return (size_t)tiles_of(n_out) * steps_of(k_in) * record_bytes(group, gated ? 2 : 1);
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
  p.packed = static_cast<const uint8_t*>(a.packed);
  p.x = static_cast<const uint16_t*>(a.x);
  p.residual = static_cast<const uint16_t*>(a.residual);
  p.y = a.y;
  p.n_out = a.n_out;
  p.k_in = a.k_in;
  p.steps = steps_of(a.k_in);
  p.full_steps = a.k_in / kStep;
  p.m = a.m;
  p.x_stride = a.x_stride;
  p.y_dtype = a.y_dtype;
  p.tiles = tiles_of(a.n_out);
  // tiles a CTA so that the busiest SM has the fewest (of equals the most a CTA: x is fetched once for them)
  int best = INT_MAX;
  for (int tn = 1; tn <= kMaxTiles; ++tn) {
    const int ctas = (p.tiles + tn - 1) / tn;
    const int load = (ctas + a.num_sms - 1) / a.num_sms * tn;
    if (load <= best) {
      best = load;
      p.tn = tn;
    }
  }
  p.tn = std::min(p.tn, p.tiles);
  const dim3 grid((p.tiles + p.tn - 1) / p.tn, (a.m + 31) / 32);
  if (a.group == 32) return launch0<32>(p, grid, a.x_f16, a.gated, stream);
  if (a.group == 64) return launch0<64>(p, grid, a.x_f16, a.gated, stream);
  return launch0<128>(p, grid, a.x_f16, a.gated, stream);
}

}  // namespace lk
