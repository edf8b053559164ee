// Paged key-value cache: append of new tokens, and attention of one new token
// per sequence over its pages (sm_100a).
//
// Attention.  For kv head h and the heads j of its group, over t < len:
//   s_t = scale q_j . k_t,  p = softmax(s),  out_j = sum_t p_t v_t,
//   and with accumulate  mass_t += sum_j p_t.
// HBM-bound: every K and V row is read once (2 D element bytes a token and kv
// head against 4 D flops a head of the group).
//
// Split.  A unit is (sequence, kv head, chunk of up to 8 NT heads of its
// group); a unit's tokens are cut into blocks of 16, and the blocks of all
// units, in order, are dealt out in equal ranges to a fixed grid, so ragged
// batches and single sequences fill the GPU alike.  A CTA's range that spans
// units is handled segment by segment; each segment leaves one partial
// (maximum, sum, weighted V) in the slot CTA + unit (both only grow along the
// list, so the slot is its own), and a second kernel joins a unit's partials.
//
// Inside a CTA each of the 4 warps takes every fourth block, straight from
// global memory to registers: 16-byte loads that arrive as operands of
// m16n8k16 products, so no shared-memory stage and no barrier stand between a
// load and its use, and the next block's K and V are requested as soon as the
// current one's registers are free.  Both products have the tokens or the
// head dim as their 16 rows and 8 heads of the group as their columns:
//   S^T [16 tokens x 8 heads] = K Q^T: lane (gid, tig) loads dims
//     32 j + 8 tig .. + 7 of tokens gid and gid + 8.  A product's sum over
//     dims does not depend on their order, so the eight values serve as they
//     lie as the k indices {2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9} of two
//     products, and Q is laid out in shared memory in the same order.
//   O^T [dims x 8 heads] = V^T P^T: lane (gid, tig) loads dims
//     64 j + 8 gid .. + 7 of tokens 2 tig, 2 tig + 1, 2 tig + 8, 2 tig + 9;
//     one byte-permute per register pairs two tokens of one dim, row gid of
//     product i being dim 8 gid + 2 i and row gid + 8 dim 8 gid + 2 i + 1.
//   The weights of S^T become the operand P^T by movmatrix (a transpose of
//     8 x 8 16-bit values across the warp).
// The weights are split into two 16-bit terms (high and remainder), so their
// rounding is 2^-16 (bf16) or 2^-22 (fp16) relative.  fp16 weights are held
// 2^14 times larger, which keeps small ones out of the subnormals: the largest
// weight is 2^14 and the smallest step 2^-24.
// int8 caches: codes are exact in fp16 (byte permute into the mantissa of
// 1024, one exact subtract); bf16 queries are first scaled by a power of two
// per head so that the largest lies in [2^14, 2^15) (values below 2^-39 of
// it round, which fp32 sums do not show); V weights are p times the token's
// scale over a running power of two, so that they too stay at most 2^14.
//
// Masked slots (behind the length, or on a page outside the pool) are not
// read: their K and V registers are zero and their score is -infinity.
#include "lk_serving.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kTok = 16;  // tokens per block

enum { DT_BF16 = 0, DT_F16 = 1, DT_I8 = 2 };

struct PagedParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* ks;
  const float* vs;
  const int32_t* table;
  const int32_t* seq_len;
  const uint16_t* q;
  int32_t* starts;  // [batch + 1] first block of each sequence, in blocks per (head, chunk)
  float* stats;     // [slots][HP][2]
  float* part;      // [slots][HP][D]
  float* scores;    // [blocks][HS][16] log2-scaled scores, or null
  float qscale;     // softmax_scale * log2(e)
  int n_pages, page_shift, n_kv, D, batch, width, group, nch, max_len, q_stride, q_f16;
  int hs;           // score rows per block
};

LK_DEVICE uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// Codes lo, hi (byte selectors in prmt form) of a word of codes + 128 as fp16.
template <uint32_t SEL>
LK_DEVICE uint32_t codes_f16(uint32_t wx) {
  const uint32_t h = __byte_perm(wx, 0x64646464u, SEL);  // 1024 + code + 128
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
  return r;
}

template <int DT>
LK_DEVICE void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (DT == DT_BF16) lk_mma_bf16_16816(c, a0, a1, a2, a3, b0, b1);
  else lk_mma_f16_16816(c, a0, a1, a2, a3, b0, b1);
}

// Two weights as 16-bit high terms and remainders.
template <int DT>
LK_DEVICE void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  if constexpr (DT == DT_BF16) {
    hi = lk_pack_bf16x2(a, b);
    lo = lk_pack_bf16x2(a - lk_bf16lo(hi), b - lk_bf16hi(hi));
  } else {
    hi = lk_pack_f16x2(a, b);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = lk_pack_f16x2(a - f.x, b - f.y);
  }
}

// CTAs that N blocks are dealt out to: each gets a block for every warp, and
// none is empty (a unit's pieces are then consecutive CTAs).
LK_DEVICE int64_t working_ctas(int64_t N, int grid) { return max((int64_t)1, min((int64_t)grid, N / kWarps)); }

// Blocks of one (head, chunk) of sequence b.
LK_DEVICE int seq_blocks(const PagedParams& p, int b) {
  const int len = max(0, min(__ldcg(p.seq_len + b), p.max_len));
  return (len + kTok - 1) / kTok;
}

template <int VC, int NT, int DT>
struct Shape {
  static constexpr int kKDims = DT == DT_I8 ? 64 : 32;       // dims of a K chunk (16 bytes a lane, 4 lanes a row)
  static constexpr int kKCh = VC * 64 / kKDims;
  static constexpr int kVDims = DT == DT_I8 && VC % 2 == 0 ? 16 : 8;  // dims a lane holds of a V chunk
  static constexpr int kVCh = VC * 8 / kVDims;
  static constexpr int kVRegs = (DT == DT_I8 ? kVDims : 2 * kVDims) / 4;
  static constexpr int kMT = VC * 4;                         // products of 16 dims
  static constexpr int kHP = 8 * NT;
  static constexpr int kOStride = VC * 64 + 4;
  static constexpr int kQVec = (DT == DT_I8 ? 2 : 1) * kKCh;  // uint4 a lane and 8 heads
  // registers a lane: accumulators, K and V in flight, and about 70 besides
  static constexpr int kRegs = 16 * VC * NT + (DT == DT_I8 ? 16 : 32) * VC + 64;
  static constexpr int kMinCtas = kRegs <= 128 ? 4 : (kRegs <= 168 ? 3 : 2);
};

template <int VC, int NT, int DT>
__global__ void __launch_bounds__(kThreads, Shape<VC, NT, DT>::kMinCtas)
    paged_decode_kernel(const __grid_constant__ PagedParams p) {
  using S = Shape<VC, NT, DT>;
  __shared__ uint4 Qs[NT][S::kQVec][32];
  __shared__ float ost[kWarps][S::kHP][S::kOStride];
  __shared__ float mst[kWarps][S::kHP][2];
  __shared__ float qf[S::kHP];
  __shared__ int sh[4];  // sequence, its first block, blocks in all, blocks of this sequence

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int D = p.D, rows_b = DT == DT_I8 ? D : 2 * D;
  const int per_seq = p.n_kv * p.nch;
  lk_grid_dep_wait();
  lk_grid_dep_launch();

  // blocks in all, then this CTA's range and the sequence it starts in
  int64_t i0, i1;
  if (warp == 0) {
    int tot = 0;
    for (int b = lane; b < p.batch; b += 32) tot += seq_blocks(p, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    const int64_t N = (int64_t)tot * per_seq;
    const int64_t first = (int64_t)blockIdx.x * N / working_ctas(N, gridDim.x);
    int run = 0;
    if (lane == 0) sh[0] = p.batch;
    __syncwarp();
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      const int b = b0 + lane;
      const int nb = b < p.batch ? seq_blocks(p, b) : 0;
      int inc = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const int at = run + inc - nb;
      if (blockIdx.x == 0 && b < p.batch) p.starts[b] = at;
      if (nb > 0 && first >= (int64_t)at * per_seq && first < (int64_t)(at + nb) * per_seq) {
        sh[0] = b;
        sh[1] = at;
        sh[3] = nb;
      }
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      sh[2] = tot;
      if (blockIdx.x == 0) p.starts[p.batch] = tot;
    }
  }
  __syncthreads();
  {
    const int64_t N = (int64_t)sh[2] * per_seq;
    const int64_t G = working_ctas(N, gridDim.x);
    if (blockIdx.x >= G) return;
    i0 = (int64_t)blockIdx.x * N / G;
    i1 = (int64_t)(blockIdx.x + 1) * N / G;
  }
  int b = sh[0], b_start = sh[1], nb = sh[3];

  while (i0 < i1) {
    while (i0 >= (int64_t)(b_start + nb) * per_seq) {  // next sequence with tokens
      b_start += nb;
      nb = seq_blocks(p, ++b);
    }
    const int in_seq = (int)(i0 - (int64_t)b_start * per_seq);
    const int hc = in_seq / nb, s0 = in_seq - hc * nb;
    const int s1 = (int)min((int64_t)nb, s0 + (i1 - i0));
    const int h = hc / p.nch, n0 = (hc - h * p.nch) * S::kHP;
    const int heads = min(p.group - n0, S::kHP);
    const int unit = b * per_seq + hc;
    const int len = max(0, min(__ldcg(p.seq_len + b), p.max_len));
    const int32_t* trow = p.table + (int64_t)b * p.width;

    // ---- page and row look-ups: lane l holds token l % 16 of a block
    auto page_of = [&](int blk) {
      const int t = blk * kTok + (lane & 15);
      return blk < s1 && t < len ? __ldcg(trow + (t >> p.page_shift)) : -1;
    };
    auto row_of = [&](int blk, int page) {
      const int t = blk * kTok + (lane & 15);
      return blk < s1 && t < len ? lk_paged_row(page, t, h, p.n_pages, p.n_kv, p.page_shift) : -1;
    };
    uint32_t kr[2][S::kKCh][4], vr[4][S::kVCh][S::kVRegs];
    float sc = 0.0f;  // int8: K scale of token l (l < 16) or V scale of token l - 16
    auto load_k = [&](int row) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = __shfl_sync(0xffffffffu, row, gid + 8 * i);
        const uint8_t* base = p.k + (int64_t)r * rows_b;
#pragma unroll
        for (int j = 0; j < S::kKCh; ++j) {
          const int off = 64 * j + 16 * tig;
          lk_ldcg16(kr[i][j], base + off, r >= 0 && off < rows_b);
        }
      }
      if constexpr (DT == DT_I8) sc = row >= 0 ? __ldcg((lane < 16 ? p.ks : p.vs) + row) : 0.0f;
    };
    auto load_v = [&](int row) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = __shfl_sync(0xffffffffu, row, 2 * tig + (i & 1) + 8 * (i >> 1));
        const uint8_t* base = p.v + (int64_t)r * rows_b;
#pragma unroll
        for (int j = 0; j < S::kVCh; ++j) {
          const int off = (8 * j + gid) * (4 * S::kVRegs);
          if constexpr (S::kVRegs == 4) lk_ldcg16(vr[i][j], base + off, r >= 0 && off < rows_b);
          else lk_ldcg8(vr[i][j], base + off, r >= 0 && off < rows_b);
        }
      }
    };

    int blk = s0 + warp;
    int row = row_of(blk, page_of(blk));
    load_k(row);
    load_v(row);
    int page_next = page_of(blk + kWarps);

    // ---- the group's queries, in the order of the K registers
    if constexpr (DT == DT_I8) {
      for (int j = warp; j < heads; j += kWarps) {
        const uint16_t* src = p.q + (int64_t)b * p.q_stride + (int64_t)(h * p.group + n0 + j) * D;
        float f = 1.0f;
        if (!p.q_f16) {
          float a = 0.0f;
          for (int d = lane; d < D; d += 32) a = fmaxf(a, fabsf(lk_bf16_to_f32(__ldcg(src + d))));
          a = lk_warp_max(a);
          // 2^(14 - exponent of the largest), within fp32's normal range
          const int e = (int)(__float_as_uint(a) >> 23);
          f = e == 255 || a == 0.0f ? 1.0f : __uint_as_float((uint32_t)max(1, min(254, 127 + 14 + 127 - e)) << 23);
        }
        if (lane == 0) qf[j] = f;
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < NT * S::kQVec * 32; i += kThreads) {
      const int l = i & 31, x = i >> 5, nt = x / S::kQVec, v = x - nt * S::kQVec;
      const int j = nt * 8 + (l >> 2);
      const int dim = DT == DT_I8 ? 64 * (v >> 1) + 16 * (l & 3) + 8 * (v & 1) : 32 * v + 8 * (l & 3);
      uint4 w = make_uint4(0, 0, 0, 0);
      if (j < heads && dim < D) {
        w = __ldcg(reinterpret_cast<const uint4*>(p.q + (int64_t)b * p.q_stride +
                                                  (int64_t)(h * p.group + n0 + j) * D + dim));
        if (DT == DT_I8 && !p.q_f16) {
          const float f = qf[j];
          w.x = lk_pack_f16x2(lk_bf16lo(w.x) * f, lk_bf16hi(w.x) * f);
          w.y = lk_pack_f16x2(lk_bf16lo(w.y) * f, lk_bf16hi(w.y) * f);
          w.z = lk_pack_f16x2(lk_bf16lo(w.z) * f, lk_bf16hi(w.z) * f);
          w.w = lk_pack_f16x2(lk_bf16lo(w.w) * f, lk_bf16hi(w.w) * f);
        }
      }
      Qs[nt][v][l] = w;
    }
    __syncthreads();

    float o[S::kMT][NT][4], m[NT][2], l[NT][2], sf[NT][2];
    float vref = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < S::kMT; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 8 * nt + 2 * tig + e;
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.0f;
        sf[nt][e] = p.qscale;
        if constexpr (DT == DT_I8) sf[nt][e] = j < heads ? p.qscale / qf[j] : 0.0f;
      }
    }

    for (; blk < s1; blk += kWarps) {
      // ---- scores of 16 tokens
      float c[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < S::kKCh; ++j) {
        if constexpr (DT == DT_I8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x = kr[0][j][i] ^ 0x80808080u, y = kr[1][j][i] ^ 0x80808080u;
            const uint32_t a0 = codes_f16<0x4140>(x), a2 = codes_f16<0x4342>(x);
            const uint32_t a1 = codes_f16<0x4140>(y), a3 = codes_f16<0x4342>(y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 qv = reinterpret_cast<const uint2*>(&Qs[nt][2 * j + (i >> 1)][lane])[i & 1];
              mma16816<DT>(c[nt], a0, a1, a2, a3, qv.x, qv.y);
            }
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 qv = Qs[nt][j][lane];
            mma16816<DT>(c[nt], kr[0][j][0], kr[1][j][0], kr[0][j][1], kr[1][j][1], qv.x, qv.y);
            mma16816<DT>(c[nt], kr[0][j][2], kr[1][j][2], kr[0][j][3], kr[1][j][3], qv.z, qv.w);
          }
        }
      }
      const bool live0 = __shfl_sync(0xffffffffu, row, gid) >= 0;
      const bool live1 = __shfl_sync(0xffffffffu, row, gid + 8) >= 0;
      float ks0 = 1.0f, ks1 = 1.0f, vs0 = 1.0f, vs1 = 1.0f;
      if constexpr (DT == DT_I8) {
        ks0 = __shfl_sync(0xffffffffu, sc, gid);
        ks1 = __shfl_sync(0xffffffffu, sc, gid + 8);
        vs0 = __shfl_sync(0xffffffffu, sc, gid + 16);
        vs1 = __shfl_sync(0xffffffffu, sc, gid + 24);
      }
      // ---- the next block's K
      const int row_next = row_of(blk + kWarps, page_next);
      page_next = page_of(blk + 2 * kWarps);
      load_k(row_next);

      // ---- running maximum and weights
      float alpha[NT][2];
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        c[nt][0] = live0 ? c[nt][0] * (sf[nt][0] * ks0) : -INFINITY;
        c[nt][1] = live0 ? c[nt][1] * (sf[nt][1] * ks0) : -INFINITY;
        c[nt][2] = live1 ? c[nt][2] * (sf[nt][0] * ks1) : -INFINITY;
        c[nt][3] = live1 ? c[nt][3] * (sf[nt][1] * ks1) : -INFINITY;
        if (p.scores) {
          const int64_t g = ((int64_t)b_start * per_seq + (int64_t)hc * nb + blk) * p.hs;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 8 * nt + 2 * tig + e;
            if (j < heads) {
              float* dst = p.scores + (g + j) * kTok + gid;
              dst[0] = c[nt][e];
              dst[8] = c[nt][2 + e];
            }
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(c[nt][e], c[nt][2 + e]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[nt][e], mx);
          const float use = mn == -INFINITY ? 0.0f : mn;
          alpha[nt][e] = exp2f(m[nt][e] - use);
          moved |= mn != m[nt][e];
          m[nt][e] = mn;
          // fp16 weights are held 2^14 times larger (the sum with them)
          const float ref = DT == DT_BF16 ? use : use - 14.0f;
          c[nt][e] = exp2f(c[nt][e] - ref);
          c[nt][2 + e] = exp2f(c[nt][2 + e] - ref);
          l[nt][e] = l[nt][e] * alpha[nt][e] + (c[nt][e] + c[nt][2 + e]);
        }
      }
      float grow = 1.0f;
      if constexpr (DT == DT_I8) {
        // the largest V scale of the block, as the power of two above it
        float a = fmaxf(fabsf(vs0), fabsf(vs1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
        if (a > vref) {
          const float up = __uint_as_float(min((__float_as_uint(a) & 0x7F800000u) + 0x00800000u, 0x7E800000u));
          grow = vref / up;
          vref = up;
          moved = true;
        }
        const float inv = vref > 0.0f ? 1.0f / vref : 0.0f;
        vs0 *= inv;
        vs1 *= inv;
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float f0 = alpha[nt][0] * grow, f1 = alpha[nt][1] * grow;
#pragma unroll
          for (int i = 0; i < S::kMT; ++i) {
            o[i][nt][0] *= f0;
            o[i][nt][1] *= f1;
            o[i][nt][2] *= f0;
            o[i][nt][3] *= f1;
          }
        }
      }
      uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (DT == DT_I8) {
          c[nt][0] *= vs0;
          c[nt][1] *= vs0;
          c[nt][2] *= vs1;
          c[nt][3] *= vs1;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          split2<DT>(c[nt][2 * i], c[nt][2 * i + 1], ph[nt][i], pl[nt][i]);
          ph[nt][i] = movmatrix_trans(ph[nt][i]);
          pl[nt][i] = movmatrix_trans(pl[nt][i]);
        }
      }

      // ---- weighted V
#pragma unroll
      for (int j = 0; j < S::kVCh; ++j) {
#pragma unroll
        for (int w = 0; w < S::kVRegs; ++w) {
          if constexpr (DT == DT_I8) {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // dims 4 w + 2 half, + 1 of token pairs (0, 1) and (2, 3): [t0 d, t1 d, t0 d + 1, t1 d + 1]
              const uint32_t sel = half ? 0x7362u : 0x5140u;
              const uint32_t x = __byte_perm(vr[0][j][w], vr[1][j][w], sel) ^ 0x80808080u;
              const uint32_t y = __byte_perm(vr[2][j][w], vr[3][j][w], sel) ^ 0x80808080u;
              const uint32_t a0 = codes_f16<0x4140>(x), a1 = codes_f16<0x4342>(x);
              const uint32_t a2 = codes_f16<0x4140>(y), a3 = codes_f16<0x4342>(y);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float (&acc)[4] = o[j * (S::kVDims / 2) + 2 * w + half][nt];
                mma16816<DT>(acc, a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
                mma16816<DT>(acc, a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
              }
            }
          } else {
            const uint32_t a0 = __byte_perm(vr[0][j][w], vr[1][j][w], 0x5410);
            const uint32_t a1 = __byte_perm(vr[0][j][w], vr[1][j][w], 0x7632);
            const uint32_t a2 = __byte_perm(vr[2][j][w], vr[3][j][w], 0x5410);
            const uint32_t a3 = __byte_perm(vr[2][j][w], vr[3][j][w], 0x7632);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float (&acc)[4] = o[j * 4 + w][nt];
              mma16816<DT>(acc, a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
              mma16816<DT>(acc, a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
            }
          }
        }
      }
      load_v(row_next);
      row = row_next;
    }

    // ---- the warps' states, then the segment's partial
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[nt][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int j = 8 * nt + 2 * tig + e;
        if (gid == 0) {
          mst[warp][j][0] = m[nt][e];
          mst[warp][j][1] = x;
        }
        if (j < heads) {
          const float f = DT == DT_I8 ? vref : 1.0f;
#pragma unroll
          for (int i = 0; i < S::kMT; ++i) {
            constexpr int kPer = S::kVDims / 2;
            const int dim = (i / kPer) * 8 * S::kVDims + S::kVDims * gid + 2 * (i % kPer);
            ost[warp][j][dim] = o[i][nt][e] * f;
            ost[warp][j][dim + 1] = o[i][nt][2 + e] * f;
          }
        }
      }
    }
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + unit;
    for (int i = threadIdx.x; i < heads * (D / 4); i += kThreads) {
      const int j = i / (D / 4), d = 4 * (i - j * (D / 4));
      float M = mst[0][j][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, mst[w][j][0]);
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float L = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        // a warp without a live token has weight 0 (and the sum 0)
        const float f = mst[w][j][0] == -INFINITY ? 0.0f : exp2f(mst[w][j][0] - M);
        const float4 x = *reinterpret_cast<const float4*>(&ost[w][j][d]);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
        // a NaN score leaves the maximum alone; its sum carries it on
        L = fmaf(f, mst[w][j][1], L);
      }
      *reinterpret_cast<float4*>(p.part + (slot * S::kHP + j) * D + d) = acc;
      if (d == 0) {
        p.stats[(slot * S::kHP + j) * 2] = M;
        p.stats[(slot * S::kHP + j) * 2 + 1] = L;
      }
    }
    __syncthreads();
    i0 += s1 - s0;
  }
}

// ---------------------------------------------------------------- joining the partials
// CTAs [0, batch * n_heads): one (sequence, head) each: its pieces' weights,
// then out = sum_c w_c O_c / sum_c w_c l_c, the pieces dealt out to groups of
// D / 4 threads.  CTAs behind them (accumulate): kMassTok slots of one
// (sequence, kv head): mass += sum over the heads of exp2(s - M) / L.
constexpr int kJoinThreads = 256;
constexpr int kMassTok = 1024;

struct JoinParams {
  const int32_t* starts;
  const float* stats;
  const float* part;
  const float* scores;
  float* mass;
  const int32_t* table;
  const int32_t* seq_len;
  void* out;
  int grid;  // CTAs of the split kernel
  int n_pages, page_shift, n_kv, D, batch, width, group, nch, max_len, hp, hs, out_dtype, mass_chunks;
  float offset;  // log2 of the factor the sums are held with
};

// The pieces of a unit: CTAs [c0, c1] of the split kernel, slots c + unit.
struct Pieces {
  int c0, c1;
};
LK_DEVICE Pieces unit_pieces(const JoinParams& p, int64_t start, int nb, int64_t N) {
  Pieces r;
  const int64_t G = working_ctas(N, p.grid);
  r.c0 = (int)(((start + 1) * G - 1) / N);
  r.c1 = (int)(((start + nb) * G - 1) / N);
  return r;
}

// Maximum and sum of one head over a unit's pieces (one warp; every lane gets both).
LK_DEVICE float2 warp_stats(const JoinParams& p, const Pieces& pc, int unit, int j) {
  const int lane = threadIdx.x & 31;
  float M = -INFINITY, L = 0.0f;
  for (int c = pc.c0 + lane; c <= pc.c1; c += 32) {
    const float2 s = __ldcg(reinterpret_cast<const float2*>(p.stats + (((int64_t)c + unit) * p.hp + j) * 2));
    const float mn = fmaxf(M, s.x);
    if (mn != -INFINITY) {
      L = (M == -INFINITY ? 0.0f : L * exp2f(M - mn)) + (s.x == -INFINITY ? 0.0f : s.y * exp2f(s.x - mn));
      M = mn;
    }
    if (s.y != s.y) L = s.y;
  }
  const float top = lk_warp_max(M);
  const float part = L != L ? L : (M == -INFINITY ? 0.0f : L * exp2f(M - top));
  return make_float2(top, lk_warp_sum(part));
}

__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float red[kJoinThreads * 4];
  __shared__ float2 st[LK_MAX_HEADS];
  const int per_seq = p.n_kv * p.nch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_heads = p.n_kv * p.group;
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const int64_t N = (int64_t)__ldcg(p.starts + p.batch) * per_seq;
  const int n_out = p.batch * n_heads;
  if ((int)blockIdx.x < n_out) {
    const int b = blockIdx.x / n_heads, j = blockIdx.x - b * n_heads;
    const int h = j / p.group, jg = j - h * p.group;
    const int ch = jg / p.hp, jc = jg - ch * p.hp;
    const int hc = h * p.nch + ch, unit = b * per_seq + hc;
    const int b0 = __ldcg(p.starts + b), nb = __ldcg(p.starts + b + 1) - b0;
    float* red4 = red;
    const int vec = p.D / 4;                 // float4 columns
    const int groups = kJoinThreads / vec;   // D <= 256: at least 4
    const int g = threadIdx.x / vec, d = threadIdx.x - g * vec;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float inv = 0.0f;
    if (nb > 0) {
      const Pieces pc = unit_pieces(p, (int64_t)b0 * per_seq + (int64_t)hc * nb, nb, N);
      const float2 s = warp_stats(p, pc, unit, jc);
      // every score -infinity (L = 0): zeros
      inv = s.y == 0.0f ? 0.0f : 1.0f / s.y;
      if (g < groups) {
#pragma unroll 4
        for (int c = pc.c0 + g; c <= pc.c1; c += groups) {
          const int64_t at = ((int64_t)c + unit) * p.hp + jc;
          const float mc = __ldcg(p.stats + at * 2);
          const float4 x = __ldcg(reinterpret_cast<const float4*>(p.part + at * p.D) + d);
          const float f = mc == -INFINITY ? 0.0f : exp2f(mc - s.x);
          acc.x = fmaf(f, x.x, acc.x);
          acc.y = fmaf(f, x.y, acc.y);
          acc.z = fmaf(f, x.z, acc.z);
          acc.w = fmaf(f, x.w, acc.w);
        }
      }
    }
    if (g < groups) reinterpret_cast<float4*>(red4)[g * vec + d] = acc;
    __syncthreads();
    if ((int)threadIdx.x < vec) {
      for (int i = 1; i < groups; ++i) {
        const float4 x = reinterpret_cast<float4*>(red4)[i * vec + d];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
      }
      acc.x *= inv;
      acc.y *= inv;
      acc.z *= inv;
      acc.w *= inv;
      const int64_t at = (int64_t)blockIdx.x * vec + d;
      if (p.out_dtype == LK_F32) {
        reinterpret_cast<float4*>(p.out)[at] = acc;
      } else {
        uint2 w;
        if (p.out_dtype == LK_BF16) {
          w.x = lk_pack_bf16x2(acc.x, acc.y);
          w.y = lk_pack_bf16x2(acc.z, acc.w);
        } else {
          w.x = lk_pack_f16x2(acc.x, acc.y);
          w.y = lk_pack_f16x2(acc.z, acc.w);
        }
        reinterpret_cast<uint2*>(p.out)[at] = w;
      }
    }
    return;
  }
  // ---- accumulated weights
  const int i = blockIdx.x - n_out;
  const int bh = i / p.mass_chunks, t0 = (i - bh * p.mass_chunks) * kMassTok;
  const int b = bh / p.n_kv, h = bh - b * p.n_kv;
  const int len = max(0, min(__ldcg(p.seq_len + b), p.max_len));
  if (t0 >= len) return;
  const int b0 = __ldcg(p.starts + b), nb = __ldcg(p.starts + b + 1) - b0;
  for (int j = warp; j < p.group; j += kJoinThreads / 32) {
    const int ch = j / p.hp, hc = h * p.nch + ch;
    const Pieces pc = unit_pieces(p, (int64_t)b0 * per_seq + (int64_t)hc * nb, nb, N);
    const float2 s = warp_stats(p, pc, b * per_seq + hc, j - ch * p.hp);
    // exp2(score - M') / L with the sum's factor taken out of L
    if (lane == 0) st[j] = make_float2(s.x == -INFINITY ? 0.0f : s.x, s.y == 0.0f ? 0.0f : exp2f(p.offset) / s.y);
  }
  __syncthreads();
  const int32_t* trow = p.table + (int64_t)b * p.width;
  for (int t = t0 + threadIdx.x; t < min(len, t0 + kMassTok); t += kJoinThreads) {
    const int row = lk_paged_row(__ldcg(trow + (t >> p.page_shift)), t, h, p.n_pages, p.n_kv, p.page_shift);
    if (row < 0) continue;
    float add = 0.0f;
    for (int ch = 0; ch < p.nch; ++ch) {
      const int heads = min(p.group - ch * p.hp, p.hp);
      const float* src = p.scores +
          (((int64_t)b0 * per_seq + (int64_t)(h * p.nch + ch) * nb + t / kTok) * p.hs) * kTok + t % kTok;
#pragma unroll 4
      for (int j = 0; j < heads; ++j) {
        const float2 s = st[ch * p.hp + j];
        add = fmaf(exp2f(__ldcg(src + j * kTok) - s.x), s.y, add);
      }
    }
    p.mass[row] = __ldcg(p.mass + row) + add;
  }
}

// ---------------------------------------------------------------- append
// One CTA per (new token, sequence); a warp takes a (K or V, head) row.  A
// 16-bit row is copied with one 16-byte access per lane (D <= 256); an int8
// row is quantised with the row rule (absmax / 127, round half to even).  A
// call of one token advances the lengths itself (no other CTA reads them).
constexpr int kAppThreads = 256;

struct AppendParams {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  float* mass;
  int32_t* pos;
  const int32_t* table;
  const uint16_t* k_new;
  const uint16_t* v_new;
  const int32_t* new_len;
  const int32_t* seq_len;
  int32_t* seq_len_out;
  const int32_t* next_pos;
  int32_t* next_pos_out;
  int n_pages, page_shift, n_kv, D, batch, width, n_new, token_stride, x_f16, is_i8;
};

// Tokens sequence b takes; 0 (and the status word) where they do not fit.
LK_DEVICE int append_count(const AppendParams& p, int b, int len) {
  const int n = p.new_len ? max(0, min(__ldcg(p.new_len + b), p.n_new)) : p.n_new;
  const bool fits = len >= 0 && (int64_t)len + n <= ((int64_t)p.width << p.page_shift);
  if (!fits) lk_dev_fail(LK_DEV_BAD_LENGTH);
  return fits ? n : 0;
}

__global__ void __launch_bounds__(kAppThreads) paged_append_kernel(const __grid_constant__ AppendParams p) {
  const int b = blockIdx.x / p.n_new, i = blockIdx.x - b * p.n_new;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const int len = __ldcg(p.seq_len + b);
  const int n = append_count(p, b, len);
  const int pos = p.next_pos ? __ldcg(p.next_pos + b) : 0;
  if (i < n) {
    const int slot = len + i;
    const int page = __ldcg(p.table + (int64_t)b * p.width + (slot >> p.page_shift));
    const int row0 = lk_paged_row(page, slot, 0, p.n_pages, p.n_kv, p.page_shift);
    if (row0 >= 0) {
      const int64_t src0 = ((int64_t)b * p.n_new + i) * p.token_stride;
      for (int r = warp; r < 2 * p.n_kv; r += kAppThreads / 32) {
        const int kv = r >= p.n_kv, h = kv ? r - p.n_kv : r;
        const int64_t row = row0 + ((int64_t)h << p.page_shift);
        const uint16_t* src = (kv ? p.v_new : p.k_new) + src0 + (int64_t)h * p.D;
        uint8_t* dst = kv ? p.v : p.k;
        uint4 w = make_uint4(0, 0, 0, 0);
        const bool live = 8 * lane < p.D;
        if (live) w = __ldcg(reinterpret_cast<const uint4*>(src) + lane);
        if (!p.is_i8) {
          if (live) reinterpret_cast<uint4*>(dst + row * p.D * 2)[lane] = w;
          continue;
        }
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
        float f[8], a = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[2 * e] = p.x_f16 ? lk_f16_to_f32((uint16_t)u[e]) : lk_bf16lo(u[e]);
          f[2 * e + 1] = p.x_f16 ? lk_f16_to_f32((uint16_t)(u[e] >> 16)) : lk_bf16hi(u[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(f[e]));
        const float s = lk_q8_scale(lk_warp_max(a));
        uint2 q = make_uint2(0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          q.x |= ((uint32_t)lk_q8_code(f[e], s) & 255u) << (8 * e);
          q.y |= ((uint32_t)lk_q8_code(f[4 + e], s) & 255u) << (8 * e);
        }
        if (live) reinterpret_cast<uint2*>(dst + row * p.D)[lane] = q;
        if (lane == 0) (kv ? p.vs : p.ks)[row] = s;
      }
      if (p.mass) {
        for (int h = threadIdx.x; h < p.n_kv; h += kAppThreads) {
          const int64_t row = row0 + ((int64_t)h << p.page_shift);
          p.mass[row] = 0.0f;
          p.pos[row] = pos + i;
        }
      }
    }
  }
  if (p.n_new == 1) {
    __syncthreads();  // every thread has read the lengths
    if (threadIdx.x == 0) {
      p.seq_len_out[b] = len + n;
      if (p.next_pos) p.next_pos_out[b] = pos + n;
    }
  }
}

__global__ void paged_advance_kernel(const __grid_constant__ AppendParams p) {
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= p.batch) return;
  const int len = __ldcg(p.seq_len + b);
  const int n = append_count(p, b, len);
  p.seq_len_out[b] = len + n;
  if (p.next_pos) p.next_pos_out[b] = __ldcg(p.next_pos + b) + n;
}

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// ---------------------------------------------------------------- dispatch
// 8 heads of a group are the columns of one product; groups of more share a
// unit's K and V registers between two products up to D = 128, where the
// accumulators of 16 heads still fit.
int heads_per_chunk(int group, int D) { return group > 8 && D <= 128 ? 16 : 8; }

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Plan {
  int hp, nch, units, hs, vc, nt, grid;
  int64_t blocks;
  size_t off_stats, off_part, off_scores, bytes;
};

template <int VC, int NT>
int min_ctas(int dt) {
  return dt == DT_BF16 ? Shape<VC, NT, DT_BF16>::kMinCtas
                       : (dt == DT_F16 ? Shape<VC, NT, DT_F16>::kMinCtas : Shape<VC, NT, DT_I8>::kMinCtas);
}

int ctas_per_sm(int vc, int nt, int dt) {
  switch (vc * 2 + (nt - 1)) {
    case 2: return min_ctas<1, 1>(dt);
    case 3: return min_ctas<1, 2>(dt);
    case 4: return min_ctas<2, 1>(dt);
    case 5: return min_ctas<2, 2>(dt);
    case 6: return min_ctas<3, 1>(dt);
    default: return min_ctas<4, 1>(dt);
  }
}

Plan make_plan(int batch, int n_kv, int n_heads, int D, int dtype, int max_len, int accumulate, int num_sms) {
  Plan r;
  const int group = n_heads / n_kv;
  const int dt = dtype == LK_BF16 ? DT_BF16 : (dtype == LK_F16 ? DT_F16 : DT_I8);
  r.hp = heads_per_chunk(group, D);
  r.nt = r.hp / 8;
  r.vc = (D + 63) / 64;
  r.nch = (group + r.hp - 1) / r.hp;
  r.units = batch * n_kv * r.nch;
  r.hs = std::min(group, r.hp);
  r.blocks = (int64_t)r.units * ((max_len + kTok - 1) / kTok);
  // every warp of a CTA gets a block, and the grid is resident at once
  r.grid = (int)std::max<int64_t>(
      1, std::min<int64_t>((int64_t)num_sms * ctas_per_sm(r.vc, r.nt, dt), (r.blocks + kWarps - 1) / kWarps));
  const size_t slots = (size_t)r.grid + r.units;
  r.off_stats = round256((size_t)(batch + 1) * 4);
  r.off_part = r.off_stats + round256(slots * r.hp * 2 * 4);
  r.off_scores = r.off_part + round256(slots * r.hp * D * 4);
  r.bytes = r.off_scores + (accumulate ? (size_t)r.blocks * r.hs * kTok * 4 : 0);
  return r;
}

template <int VC, int NT>
cudaError_t launch_split(int dt, int grid, const PagedParams& p, cudaStream_t stream) {
  if (dt == DT_BF16) return lk::launch_pdl(paged_decode_kernel<VC, NT, DT_BF16>, dim3(grid), dim3(kThreads), stream, p);
  if (dt == DT_F16) return lk::launch_pdl(paged_decode_kernel<VC, NT, DT_F16>, dim3(grid), dim3(kThreads), stream, p);
  return lk::launch_pdl(paged_decode_kernel<VC, NT, DT_I8>, dim3(grid), dim3(kThreads), stream, p);
}

}  // namespace

LK_DEFINE_STATUS_ACCESSOR(lk_paged_status_word)

namespace lk {

int64_t paged_decode_max_blocks(int batch, int n_kv_heads, int group, int head_dim, int max_len) {
  const int hp = heads_per_chunk(group, head_dim);
  return (int64_t)batch * n_kv_heads * ((group + hp - 1) / hp) * (((int64_t)max_len + kTok - 1) / kTok);
}

size_t paged_decode_workspace_bytes(int batch, int n_kv_heads, int n_heads, int head_dim, int dtype, int max_len,
                                    int accumulate, int num_sms) {
  return make_plan(batch, n_kv_heads, n_heads, head_dim, dtype, max_len, accumulate, num_sms).bytes;
}

cudaError_t launch_paged_decode(const PagedDecodeLaunch& a, cudaStream_t stream) {
  const PagedCacheView& c = a.c;
  const Plan r = make_plan(c.batch, c.n_kv_heads, a.n_heads, c.head_dim, c.dtype, a.max_len, a.accumulate, a.num_sms);
  const int dt = c.dtype == LK_BF16 ? DT_BF16 : (c.dtype == LK_F16 ? DT_F16 : DT_I8);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  PagedParams p{};
  p.k = static_cast<const uint8_t*>(c.k);
  p.v = static_cast<const uint8_t*>(c.v);
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.table = c.page_table;
  p.seq_len = a.seq_len;
  p.q = static_cast<const uint16_t*>(a.q);
  p.starts = reinterpret_cast<int32_t*>(ws);
  p.stats = reinterpret_cast<float*>(ws + r.off_stats);
  p.part = reinterpret_cast<float*>(ws + r.off_part);
  p.scores = a.accumulate ? reinterpret_cast<float*>(ws + r.off_scores) : nullptr;
  p.qscale = a.softmax_scale * 1.44269504088896340736f;
  p.n_pages = c.n_pages;
  p.page_shift = log2_of(c.page_size);
  p.n_kv = c.n_kv_heads;
  p.D = c.head_dim;
  p.batch = c.batch;
  p.width = c.table_width;
  p.group = a.n_heads / c.n_kv_heads;
  p.nch = r.nch;
  p.max_len = a.max_len;
  p.q_stride = a.q_stride;
  p.q_f16 = a.q_f16;
  p.hs = r.hs;
  cudaError_t e;
  switch (r.vc * 2 + (r.nt - 1)) {
    case 2: e = launch_split<1, 1>(dt, r.grid, p, stream); break;
    case 3: e = launch_split<1, 2>(dt, r.grid, p, stream); break;
    case 4: e = launch_split<2, 1>(dt, r.grid, p, stream); break;
    case 5: e = launch_split<2, 2>(dt, r.grid, p, stream); break;
    case 6: e = launch_split<3, 1>(dt, r.grid, p, stream); break;
    default: e = launch_split<4, 1>(dt, r.grid, p, stream); break;
  }
  if (e != cudaSuccess) return e;
  JoinParams j{};
  j.starts = p.starts;
  j.stats = p.stats;
  j.part = p.part;
  j.scores = p.scores;
  j.mass = a.accumulate ? c.mass : nullptr;
  j.table = p.table;
  j.seq_len = p.seq_len;
  j.out = a.out;
  j.grid = r.grid;
  j.n_pages = p.n_pages;
  j.page_shift = p.page_shift;
  j.n_kv = p.n_kv;
  j.D = p.D;
  j.batch = p.batch;
  j.width = p.width;
  j.group = p.group;
  j.nch = p.nch;
  j.max_len = p.max_len;
  j.hp = r.hp;
  j.hs = r.hs;
  j.out_dtype = a.out_dtype;
  j.offset = dt == DT_BF16 ? 0.0f : 14.0f;
  j.mass_chunks = a.accumulate ? (a.max_len + kMassTok - 1) / kMassTok : 0;
  const unsigned ctas = (unsigned)(c.batch * a.n_heads) + (unsigned)(c.batch * c.n_kv_heads) * (unsigned)j.mass_chunks;
  return lk::launch_pdl(paged_join_kernel, dim3(ctas), dim3(kJoinThreads), stream, j);
}

cudaError_t launch_paged_append(const PagedAppendLaunch& a, cudaStream_t stream) {
  const PagedCacheView& c = a.c;
  AppendParams p{};
  p.k = static_cast<uint8_t*>(c.k);
  p.v = static_cast<uint8_t*>(c.v);
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.mass = c.mass;
  p.pos = c.pos;
  p.table = c.page_table;
  p.k_new = static_cast<const uint16_t*>(a.k_new);
  p.v_new = static_cast<const uint16_t*>(a.v_new);
  p.new_len = a.new_len;
  p.seq_len = a.seq_len;
  p.seq_len_out = a.seq_len_out;
  p.next_pos = a.next_pos;
  p.next_pos_out = a.next_pos_out;
  p.n_pages = c.n_pages;
  p.page_shift = log2_of(c.page_size);
  p.n_kv = c.n_kv_heads;
  p.D = c.head_dim;
  p.batch = c.batch;
  p.width = c.table_width;
  p.n_new = a.n_new;
  p.token_stride = a.token_stride;
  p.x_f16 = a.x_f16;
  p.is_i8 = c.dtype == LK_I8;
  cudaError_t e = launch_pdl(paged_append_kernel, dim3(c.batch * a.n_new), dim3(kAppThreads), stream, p);
  if (e != cudaSuccess || a.n_new == 1) return e;
  return lk::launch_pdl(paged_advance_kernel, dim3((c.batch + 127) / 128), dim3(128), stream, p);
}

}  // namespace lk
