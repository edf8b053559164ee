// Paged key-value cache: append of new tokens, and attention of one new token
// per sequence over its pages (sm_100a).
//
// Attention.  For kv head h and the heads j of its group, over t < len:
//   s_t = scale q_j . k_t,  p = softmax(s),  out_j = sum_t p_t v_t,
//   and with accumulate  mass_t += sum_j p_t.
// HBM-bound: every K and V row is read once (2 D element bytes a token and kv
// head against 4 D flops a head of the group).  bf16, D = 128, a call (in a
// captured graph): 8 ragged sequences to 16384, group 4, 53.9 us (53.0), 78 %
// of the measured copy bandwidth; one of 4224, 32 kv heads, 21.0 us (20.3),
// 51 %: two launches and the ramp, schedulers issue in 23 % of their cycles and
// wait for memory otherwise.
//
// Split.  A unit is (sequence, kv head, chunk of up to 8 NT heads of its
// group); a unit's tokens are cut into blocks of 16, and the blocks of all
// units, in order, are dealt out in equal ranges to a fixed grid, so ragged
// batches and single sequences fill the GPU alike.  A CTA's range that spans
// units is handled segment by segment; each segment leaves one partial
// (maximum, sum, weighted V) in the slot CTA + unit (both only grow along the
// list, so the slot is its own), and a second kernel joins a unit's partials.
//
// Inside a CTA each of the 4 warps takes every fourth block through a ring of
// its own in shared memory: cp.async (16 bytes a lane) keeps the next blocks'
// K and V rows in flight while one is computed, and since no other warp
// touches the ring, no barrier does more than order the lanes.  (Loading the
// operands straight into registers held 8 KB a warp in flight, and only
// between a block's products; the ring holds twice that throughout.)  Rows are
// swizzled (16-byte chunks exclusive-or the row) so that ldmatrix reads eight
// rows without bank conflicts.  Both products have the tokens or the head dim
// as their 16 rows and 8 heads of the group as their columns (m16n8k16):
//   S^T [16 tokens x 8 heads] = K Q^T, K by ldmatrix;
//   O^T [16 dims x 8 heads] = V^T P^T, V^T by ldmatrix.trans;
//   the weights of S^T become the operand P^T by movmatrix (a transpose of
//   8 x 8 16-bit values across the warp).
// int8 rows go the same way as pairs of bytes: ldmatrix gives a lane four
// codes of a token (Q is laid out in that order of dims), ldmatrix.trans two
// dims of two tokens, whose even and odd bytes are the rows of one product.
// The weights are split into two 16-bit terms (high and remainder), so their
// rounding is 2^-16 (bf16) or 2^-22 (fp16) relative.  An fp32 output of a bf16
// cache gets a third term (2^-24) for 2 to 5 % of the time (ragged to 16384
// 53.9 us in a graph against 52.7); a 16-bit one would round it away: its error
// against 64 bits is the same without (relative 1.68e-3 in 2-norm, 9.5e-7 of
// it from the two terms).  fp16 weights are held
// 2^10 times larger, which keeps small ones out of the subnormals: the largest
// weight is 2^14, the sum at least 2^10 and the smallest step 2^-24.
// int8 caches: codes are exact in fp16 (byte permute into the mantissa of
// 1024, one exact subtract); bf16 queries are first scaled by a power of two
// per head so that the largest lies in [2^14, 2^15) (values below about 2^-31
// of it meet fp16's smallest step and are off by up to 2^-39 of the largest,
// which fp32 sums do not show); V weights are p times the token's
// scale over a running power of two, so that they too stay at most 2^14.
//
// Masked slots (behind the length, or on a page outside the pool) are not
// read: their K and V are zero-filled and their score is -infinity.
#include <algorithm>
#include <atomic>

#include "lk_serving.cuh"

namespace {

constexpr int kWarps = 4;  // of a CTA of the split
constexpr int kWideStage = 12 * 1024 + 128;  // largest stage of a CTA of eight warps (two of them each fit)
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
  int resident;     // CTAs the GPU holds
  // one CTA a unit (grid = units): the output and mass are written here
  int direct, unit_blocks, out_dtype;
  int third;        // bf16 weights in three terms
  int ring;         // bytes of a warp's ring
  void* out;
  float* mass;
  float offset;     // log2 of the factor weights and sums are held with
};

// The reference a head's weights are taken relative to follows the running
// maximum only once a score lies more than kSlack (log2) above it: the warp
// then reduces the maximum and rescales, otherwise one vote does.  Weights are
// so at most 2^kSlack; fp16 ones are held 2^kHeld times larger.
constexpr float kSlack = 4.0f, kHeld = 10.0f;

// 2^x; results below 2^-126 are 0 (such weights are nothing beside the sum).
LK_DEVICE float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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

// CTAs that N blocks are dealt out to: all resident at once, each with a block
// for every warp, none empty (a unit's pieces are then consecutive CTAs).
// (More and smaller ranges, for SMs that are served faster to take more, cost
// 4 to 10 % on long caches: their start-up is not hidden.  Ranges that end
// with a unit where all sequences are equally long gain nothing.)
__host__ __device__ inline int64_t working_ctas(int64_t N, int64_t resident) {
  const int64_t ctas = N / kWarps < resident ? N / kWarps : resident;
  return ctas < 1 ? 1 : ctas;
}

// a / c of numbers that are not negative, in 32 bits where they fit (a 64-bit division is 0.2 us on the way to a
// CTA's first load).
LK_DEVICE int64_t quotient(int64_t a, int64_t c) {
  if (((a | c) >> 32) == 0) return (uint32_t)a / (uint32_t)c;
  return a / c;
}

// What the two bf16 terms of a weight leave.
LK_DEVICE float third_term(float a) {
  const float r = a - lk_bf16_to_f32(lk_f32_to_bf16(a));
  return r - lk_bf16_to_f32(lk_f32_to_bf16(r));
}

// Four outputs in the call's type.
LK_DEVICE void store_out(void* out, int64_t at, const float4& v, int dtype) {
  if (dtype == LK_F32) {
    reinterpret_cast<float4*>(out)[at] = v;
  } else {
    uint2 w;
    if (dtype == LK_BF16) {
      w.x = lk_pack_bf16x2(v.x, v.y);
      w.y = lk_pack_bf16x2(v.z, v.w);
    } else {
      w.x = lk_pack_f16x2(v.x, v.y);
      w.y = lk_pack_f16x2(v.z, v.w);
    }
    reinterpret_cast<uint2*>(out)[at] = w;
  }
}

// The output of an empty sequence.
LK_DEVICE void zero_rows(const PagedParams& p, int b, int tid, int threads) {
  const int n = p.n_kv * p.group * (p.D / 4);
  for (int i = tid; i < n; i += threads)
    store_out(p.out, (int64_t)b * n + i, make_float4(0.0f, 0.0f, 0.0f, 0.0f), p.out_dtype);
}

// Blocks of one (head, chunk) of sequence b.
LK_DEVICE int seq_blocks(const PagedParams& p, int b) {
  const int len = max(0, min(__ldcg(p.seq_len + b), p.max_len));
  return (len + kTok - 1) / kTok;
}

LK_DEVICE void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
LK_DEVICE void cp_async16_zfill(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
LK_DEVICE void cp_async4_zfill(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(live ? 4 : 0) : "memory");
}
template <bool TRANS>
LK_DEVICE void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// Head dims up to 64 VC, 8 NT heads, W warps.
template <int VC, int NT, int DT, int W>
struct Shape {
  static constexpr int kCh = VC * 64 * (DT == DT_I8 ? 1 : 2) / 16;  // 16-byte chunks of a row
  static constexpr int kRowB = kCh * 16;
  static constexpr int kScaleB = DT == DT_I8 ? 2 * kTok * 4 : 0;
  static constexpr int kStageB = 2 * kTok * kRowB + kScaleB;        // K rows, V rows, scales
  static constexpr int kSteps = VC * 4;                              // products of 16 dims
  static constexpr int kHP = 8 * NT;
  static constexpr int kOStride = VC * 64 + 4;
  static constexpr int kRowsPer = 32 / kCh;                          // rows a warp copies at a time
  // Stages and CTAs an SM.  Rows of 256 bytes, one sequence of 4224 tokens: 2 stages and 3 CTAs 20.5 us, 3 and 2
  // 22.1, 4 and 1 24.9; rows of 128 bytes, fp16 with weights: 2 and 5 29.1 us, 3 and 4 29.2, 4 and 3 30.2.
  static constexpr int kStages = kStageB <= 2200 ? 4 : (kStageB <= 12288 ? 2 : 3);
  static constexpr int kMinCtas = W > kWarps          ? 1
                                  : kStageB <= 2200  ? 4
                                  : kStageB <= 4300  ? (NT == 1 ? 5 : 3)
                                  : kStageB <= 9000  ? 3
                                  : kStageB <= 12288 ? 2
                                                     : 1;
  static constexpr int kQB = NT * (kSteps / 2) * 32 * 16;
  static constexpr int kPartialB = kHP * kOStride * 4;
  // A warp's ring: no more stages than it has blocks, and room for its partial.
  static int ring(int blocks) {
    return std::max(std::min(kStages, std::max(blocks, 1)) * kStageB, (kPartialB + 127) / 128 * 128);
  }
  static int smem(int blocks) { return W * ring(blocks) + kQB; }
  static_assert(kStages <= 4, "live masks of the stages fit in 64 bits");
};

// Exclusive-or of a row's chunk index: eight consecutive rows of one chunk
// fall in distinct banks for rows of a multiple of 128 bytes, and of 64.
template <int CH>
LK_DEVICE int swizzle(int row) {
  return CH % 8 == 0 ? row & 7 : (row >> 1) & 3;
}

// FULL: the head dim is 64 VC (else products behind it are skipped).
template <int VC, int NT, int DT, int W, bool FULL>
__global__ void __launch_bounds__(W * 32, Shape<VC, NT, DT, W>::kMinCtas)
    paged_decode_kernel(const __grid_constant__ PagedParams p) {
  using S = Shape<VC, NT, DT, W>;
  constexpr int kThreads = W * 32, kWarps = W;
  extern __shared__ __align__(128) uint8_t smem[];
  uint4 (*Qs)[S::kSteps / 2][32] = reinterpret_cast<uint4 (*)[S::kSteps / 2][32]>(smem + kWarps * p.ring);
  __shared__ float mst[kWarps][S::kHP][2];
  __shared__ float unit_st[S::kHP][2];
  __shared__ float qf[S::kHP];
  __shared__ int sh[4];  // sequence, its first block, blocks in all, length of this sequence

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gid = lane >> 2, tig = lane & 3;
  const int D = FULL ? VC * 64 : p.D, rows_b = DT == DT_I8 ? D : 2 * D;
  const int per_seq = p.n_kv * p.nch;
  // products along the head dim; what a row's padding holds is not used
  const int steps = FULL ? S::kSteps : D / 16;
  uint8_t* ring = smem + warp * p.ring;
  const uint32_t ring_a = lk_smem_addr(ring);
  lk_grid_dep_wait();
  lk_grid_dep_launch();

  // blocks in all, then this CTA's range and the sequence it starts in
  int64_t i0, i1;
  int b, b_start, nb, len;
  if (p.direct) {
    b = blockIdx.x / per_seq;
    b_start = 0;
    len = max(0, min(__ldcg(p.seq_len + b), p.max_len));
    nb = (len + kTok - 1) / kTok;
    const int hc = blockIdx.x - b * per_seq;
    i0 = (int64_t)hc * nb;
    i1 = i0 + nb;
    if (nb == 0 && hc == 0) zero_rows(p, b, threadIdx.x, kThreads);
  } else {
    if (warp == 0) {
      // (the lengths of the first 32 sequences are read once: a second look is 0.3 us before the first load)
      const int len0 = lane < p.batch ? max(0, min(__ldcg(p.seq_len + lane), p.max_len)) : 0;
      const int n0 = (len0 + kTok - 1) / kTok;
      int tot = n0;
      for (int e = lane + 32; e < p.batch; e += 32) tot += seq_blocks(p, e);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
      const int64_t N = (int64_t)tot * per_seq;
      const int64_t first = quotient(blockIdx.x * N, working_ctas(N, p.resident));
      int run = 0;
      if (lane == 0) sh[0] = p.batch;
      __syncwarp();
      for (int e0 = 0; e0 < p.batch; e0 += 32) {
        const int e = e0 + lane;
        const int l = e0 == 0 ? len0 : (e < p.batch ? max(0, min(__ldcg(p.seq_len + e), p.max_len)) : 0);
        const int n = (l + kTok - 1) / kTok;
        int inc = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        const int at = run + inc - n;
        if (blockIdx.x == 0 && e < p.batch) p.starts[e] = at;
        if (n > 0 && first >= (int64_t)at * per_seq && first < (int64_t)(at + n) * per_seq) {
          sh[0] = e;
          sh[1] = at;
          sh[3] = l;
        }
        run += __shfl_sync(0xffffffffu, inc, 31);
      }
      if (lane == 0) {
        sh[2] = tot;
        if (blockIdx.x == 0) p.starts[p.batch] = tot;
      }
    }
    __syncthreads();
    const int64_t N = (int64_t)sh[2] * per_seq;
    const int64_t G = working_ctas(N, p.resident);
    if (blockIdx.x >= G) return;
    i0 = quotient(blockIdx.x * N, G);
    i1 = quotient((blockIdx.x + 1) * N, G);
    b = sh[0];
    b_start = sh[1];
    len = sh[3];
    nb = (len + kTok - 1) / kTok;
  }

  while (i0 < i1) {
    while (i0 >= (int64_t)(b_start + nb) * per_seq) {  // next sequence with tokens
      b_start += nb;
      len = max(0, min(__ldcg(p.seq_len + ++b), p.max_len));
      nb = (len + kTok - 1) / kTok;
    }
    const int in_seq = (int)(i0 - (int64_t)b_start * per_seq);
    const int hc = in_seq / nb, s0 = in_seq - hc * nb;
    const int s1 = (int)min((int64_t)nb, s0 + (i1 - i0));
    const int h = hc / p.nch, n0 = (hc - h * p.nch) * S::kHP;
    const int heads = min(p.group - n0, S::kHP);
    const int unit = b * per_seq + hc;
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
    // copies a block's rows into a stage; lane l holds the row of token l % 16
    const int c_row = lane / S::kCh, c_ch = lane - c_row * S::kCh;
    const bool c_in = (FULL && S::kRowsPer * S::kCh == 32) || (c_row < S::kRowsPer && 16 * c_ch < rows_b);
    auto issue = [&](int stage, int row) {
      const uint32_t st = ring_a + stage * S::kStageB;
#pragma unroll
      for (int i = 0; i < kTok / S::kRowsPer; ++i) {
        const int t = i * S::kRowsPer + (c_in ? c_row : 0);
        const int r = __shfl_sync(0xffffffffu, row, t);
        const bool live = r >= 0;
        const int64_t off = live ? (int64_t)r * rows_b + 16 * c_ch : 0;
        const uint32_t dst = st + t * S::kRowB + ((c_ch ^ swizzle<S::kCh>(t)) << 4);
        if (c_in) {
          cp_async16_zfill(dst, p.k + off, live);
          cp_async16_zfill(dst + kTok * S::kRowB, p.v + off, live);
        }
      }
      if constexpr (DT == DT_I8) {
        const float* src = lane < 16 ? p.ks : p.vs;
        cp_async4_zfill(st + 2 * kTok * S::kRowB + 4 * lane, src + max(row, 0), row >= 0);
      }
    };

    // The same for 16 live tokens of one page: their rows are consecutive, so
    // the addresses are one base and constant steps.
    const uint32_t c_dst = c_row * S::kRowB + ((c_ch ^ swizzle<S::kCh>(c_row)) << 4);
    auto issue_page = [&](int stage, int row) {
      const uint32_t st = ring_a + stage * S::kStageB;
      const int64_t off = (int64_t)__shfl_sync(0xffffffffu, row, 0) * rows_b + (c_in ? c_row * rows_b + 16 * c_ch : 0);
      const uint8_t* ks = p.k + off;
      const uint8_t* vs = p.v + off;
      if (c_in) {
#pragma unroll
        for (int i = 0; i < kTok / S::kRowsPer; ++i) {
          const uint32_t dst = st + i * S::kRowsPer * S::kRowB + (c_dst ^ (swizzle<S::kCh>(i * S::kRowsPer) << 4));
          // (constant offsets where the rows fill the chunks)
          const int step = rows_b == S::kRowB ? i * S::kRowsPer * S::kRowB : i * S::kRowsPer * rows_b;
          cp_async16(dst, ks + step);
          cp_async16(dst + kTok * S::kRowB, vs + step);
        }
      }
      if constexpr (DT == DT_I8)
        cp_async4_zfill(st + 2 * kTok * S::kRowB + 4 * lane, (lane < 16 ? p.ks : p.vs) + row, true);
    };

    int blk = s0 + warp, stage = 0, page_next;
    uint64_t live_bits = 0;  // 16 bits a stage in flight, the next to be computed lowest
    {
      int pages[S::kStages];
#pragma unroll
      for (int i = 0; i < S::kStages; ++i) pages[i] = page_of(blk + i * kWarps);
#pragma unroll
      for (int i = 0; i < S::kStages - 1; ++i) {
        const int row = row_of(blk + i * kWarps, pages[i]);
        live_bits |= (uint64_t)(__ballot_sync(0xffffffffu, row >= 0) & 0xFFFFu) << (16 * i);
        if (blk + i * kWarps < s1) issue(i, row);
        lk_cp_async_commit();
      }
      page_next = pages[S::kStages - 1];
    }

    // ---- the group's queries, in the order of the K registers
    if constexpr (DT == DT_I8) {
      for (int j = warp; j < heads; j += kWarps) {
        const uint16_t* src = p.q + (int64_t)b * p.q_stride + (int64_t)(h * p.group + n0 + j) * D;
        float f = 1.0f;
        if (!p.q_f16) {
          float a = 0.0f;
          if (8 * lane < D) {
            const uint4 w = __ldcg(reinterpret_cast<const uint4*>(src) + lane);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) a = fmaxf(a, fmaxf(fabsf(lk_bf16lo(u[e])), fabsf(lk_bf16hi(u[e]))));
          }
          a = lk_warp_max(a);
          // 2^(14 - exponent of the largest), within fp32's normal range
          const int e = (int)(__float_as_uint(a) >> 23);
          f = e == 255 || a == 0.0f ? 1.0f : __uint_as_float((uint32_t)max(1, min(254, 127 + 14 + 127 - e)) << 23);
        }
        if (lane == 0) qf[j] = f;
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < NT * S::kSteps * 32; i += kThreads) {
      // one product's two registers: 16-bit dims 2 tig, + 1, 2 tig + 8, + 9; int8 dims 4 tig .. 4 tig + 3
      const int l = i & 31, x = i >> 5, nt = x / S::kSteps, st = x - nt * S::kSteps;
      const int j = nt * 8 + (l >> 2), t4 = l & 3;
      const int d0 = 16 * st + (DT == DT_I8 ? 4 * t4 : 2 * t4), d1 = d0 + (DT == DT_I8 ? 2 : 8);
      uint32_t w[2] = {0, 0};
      if (j < heads && 16 * st < D) {
        const uint16_t* src = p.q + (int64_t)b * p.q_stride + (int64_t)(h * p.group + n0 + j) * D;
        w[0] = __ldcg(reinterpret_cast<const uint32_t*>(src + d0));
        w[1] = __ldcg(reinterpret_cast<const uint32_t*>(src + d1));
        if (DT == DT_I8 && !p.q_f16) {
          const float f = qf[j];
#pragma unroll
          for (int e = 0; e < 2; ++e) w[e] = lk_pack_f16x2(lk_bf16lo(w[e]) * f, lk_bf16hi(w[e]) * f);
        }
      }
      reinterpret_cast<uint2*>(&Qs[nt][st >> 1][l])[st & 1] = make_uint2(w[0], w[1]);
    }
    __syncthreads();

    float o[S::kSteps][NT][4], m[NT][2], l[NT][2], sf[NT][2];
    float vref = 0.0f, vinv = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < S::kSteps; ++i) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 8 * nt + 2 * tig + e;
        m[nt][e] = -INFINITY;
        l[nt][e] = 0.0f;
        sf[nt][e] = p.qscale;
        if constexpr (DT == DT_I8) sf[nt][e] = j < heads ? p.qscale / qf[j] : 0.0f;
      }
    }

    const int f_row = (lane & 7) + (lane & 8);  // ldmatrix: this lane's row and chunk of a pair
    const uint32_t f_at = f_row * S::kRowB;
    const uint32_t f_ch = ((lane >> 4) ^ swizzle<S::kCh>(f_row)) << 4;
    // the block's scores of heads 2 tig, tokens gid
    const int64_t first_block =
        p.direct ? (int64_t)unit * p.unit_blocks : (int64_t)b_start * per_seq + (int64_t)hc * nb;
    float* sp = p.scores + ((first_block + blk) * p.hs + 2 * tig) * kTok + gid;
    for (; blk < s1; blk += kWarps, sp += kWarps * p.hs * kTok) {
      // ---- request the block S::kStages - 1 ahead, then wait for this one
      {
        const int ahead = blk + (S::kStages - 1) * kWarps;
        const int row = row_of(ahead, page_next);
        page_next = page_of(ahead + kWarps);
        const uint32_t live = __ballot_sync(0xffffffffu, row >= 0) & 0xFFFFu;
        live_bits |= (uint64_t)live << (16 * (S::kStages - 1));
        const int to = stage == 0 ? S::kStages - 1 : stage - 1;
        if (live == 0xFFFFu && p.page_shift >= 4) issue_page(to, row);
        else if (ahead < s1) issue(to, row);
        lk_cp_async_commit();
      }
      lk_cp_async_wait<S::kStages - 1>();
      __syncwarp();
      const uint32_t live = (uint32_t)live_bits & 0xFFFFu;
      live_bits >>= 16;
      const uint32_t st = ring_a + stage * S::kStageB;

      // ---- scores of 16 tokens
      float c[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.0f;
#pragma unroll
      for (int v = 0; v < S::kSteps / 2; ++v) {
        if (2 * v >= steps) break;
        uint4 qv[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) qv[nt] = Qs[nt][v][lane];
        if constexpr (DT == DT_I8) {
          uint32_t k4[4];
          ldmatrix4<false>(k4, st + f_at + (f_ch ^ (v << 5)));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t x = k4[2 * i] ^ 0x80808080u, y = k4[2 * i + 1] ^ 0x80808080u;
            const uint32_t a0 = codes_f16<0x4140>(x), a2 = codes_f16<0x4342>(x);
            const uint32_t a1 = codes_f16<0x4140>(y), a3 = codes_f16<0x4342>(y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              if (2 * v + i < steps)
                mma16816<DT>(c[nt], a0, a1, a2, a3, i ? qv[nt].z : qv[nt].x, i ? qv[nt].w : qv[nt].y);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (2 * v + i >= steps) break;
            uint32_t k4[4];
            ldmatrix4<false>(k4, st + f_at + (f_ch ^ ((2 * v + i) << 5)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<DT>(c[nt], k4[0], k4[1], k4[2], k4[3], i ? qv[nt].z : qv[nt].x, i ? qv[nt].w : qv[nt].y);
          }
        }
      }
      float ks0 = 1.0f, ks1 = 1.0f, vs0 = 1.0f, vs1 = 1.0f;
      if constexpr (DT == DT_I8) {
        const float* sc = reinterpret_cast<const float*>(ring + stage * S::kStageB + 2 * kTok * S::kRowB);
        ks0 = sc[gid];
        ks1 = sc[gid + 8];
        vs0 = sc[gid + 16];
        vs1 = sc[gid + 24];
      }

      // ---- weights relative to a reference near the maximum
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        c[nt][0] *= sf[nt][0] * ks0;
        c[nt][1] *= sf[nt][1] * ks0;
        c[nt][2] *= sf[nt][0] * ks1;
        c[nt][3] *= sf[nt][1] * ks1;
        if (live != 0xFFFFu) {
          if (!((live >> gid) & 1)) c[nt][0] = c[nt][1] = -INFINITY;
          if (!((live >> (gid + 8)) & 1)) c[nt][2] = c[nt][3] = -INFINITY;
        }
        if (p.scores) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (8 * nt + 2 * tig + e < heads) {
              sp[(8 * nt + e) * kTok] = c[nt][e];
              sp[(8 * nt + e) * kTok + 8] = c[nt][2 + e];
            }
        }
        moved |= fmaxf(c[nt][0], c[nt][2]) > m[nt][0] + kSlack || fmaxf(c[nt][1], c[nt][3]) > m[nt][1] + kSlack;
      }
      if constexpr (DT == DT_I8) moved |= fmaxf(fabsf(vs0), fabsf(vs1)) > vref;
      float alpha[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) alpha[nt][0] = alpha[nt][1] = 1.0f;
      moved = __any_sync(0xffffffffu, moved);
      if (moved) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(c[nt][e], c[nt][2 + e]);
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const float mn = fmaxf(m[nt][e], mx);
            alpha[nt][e] = ex2(m[nt][e] - (mn == -INFINITY ? 0.0f : mn));
            m[nt][e] = mn;
            l[nt][e] *= alpha[nt][e];
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float ref = (m[nt][e] == -INFINITY ? 0.0f : m[nt][e]) - (DT == DT_BF16 ? 0.0f : kHeld);
          c[nt][e] = ex2(c[nt][e] - ref);
          c[nt][2 + e] = ex2(c[nt][2 + e] - ref);
          l[nt][e] += c[nt][e] + c[nt][2 + e];
        }
      }
      float grow = 1.0f;
      if constexpr (DT == DT_I8) {
        if (moved) {
          // the largest V scale of the block, as the power of two above it
          float a = fmaxf(fabsf(vs0), fabsf(vs1));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 4));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 8));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 16));
          if (a > vref) {  // the same in every lane
            const float up = __uint_as_float(min((__float_as_uint(a) & 0x7F800000u) + 0x00800000u, 0x7E800000u));
            grow = vref / up;
            vref = up;
            vinv = 1.0f / up;
          }
        }
        vs0 *= vinv;
        vs1 *= vinv;
      }
      if (moved) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float f0 = alpha[nt][0] * grow, f1 = alpha[nt][1] * grow;
#pragma unroll
          for (int i = 0; i < S::kSteps; ++i) {
            o[i][nt][0] *= f0;
            o[i][nt][1] *= f1;
            o[i][nt][2] *= f0;
            o[i][nt][3] *= f1;
          }
        }
      }
      uint32_t ph[NT][2], pl[NT][2], px[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (DT == DT_BF16) {
          if (p.third) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              px[nt][i] =
                  movmatrix_trans(lk_pack_bf16x2(third_term(c[nt][2 * i]), third_term(c[nt][2 * i + 1])));
          }
        }
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
      for (int v = 0; v < S::kCh / 2; ++v) {
        if ((DT == DT_I8 ? 2 * v : v) >= steps) break;
        uint32_t v4[4];
        ldmatrix4<true>(v4, st + kTok * S::kRowB + f_at + (f_ch ^ (v << 5)));
        if constexpr (DT == DT_I8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            // bytes: token 2 tig dims 2 gid, + 1, then token 2 tig + 1
            const uint32_t x = v4[2 * i] ^ 0x80808080u, y = v4[2 * i + 1] ^ 0x80808080u;
            const uint32_t a0 = codes_f16<0x4240>(x), a1 = codes_f16<0x4341>(x);
            const uint32_t a2 = codes_f16<0x4240>(y), a3 = codes_f16<0x4341>(y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if (2 * v + i >= steps) continue;
              float (&acc)[4] = o[2 * v + i][nt];
              mma16816<DT>(acc, a0, a1, a2, a3, ph[nt][0], ph[nt][1]);
              mma16816<DT>(acc, a0, a1, a2, a3, pl[nt][0], pl[nt][1]);
            }
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float (&acc)[4] = o[v][nt];
            mma16816<DT>(acc, v4[0], v4[2], v4[1], v4[3], ph[nt][0], ph[nt][1]);
            mma16816<DT>(acc, v4[0], v4[2], v4[1], v4[3], pl[nt][0], pl[nt][1]);
          }
        }
      }
      if constexpr (DT == DT_BF16) {
        if (p.third) {  // in a loop of its own: the one above keeps its registers and instructions
#pragma unroll
          for (int v = 0; v < S::kCh / 2; ++v) {
            if (v >= steps) break;
            uint32_t v4[4];
            ldmatrix4<true>(v4, st + kTok * S::kRowB + f_at + (f_ch ^ (v << 5)));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<DT>(o[v][nt], v4[0], v4[2], v4[1], v4[3], px[nt][0], px[nt][1]);
          }
        }
      }
      __syncwarp();  // the stage is read: the next request may fill it
      if (++stage == S::kStages) stage = 0;
    }

    // ---- the warps' states (in the drained ring), then the segment's partial
    lk_cp_async_wait<0>();
    __syncwarp();
    float* ost = reinterpret_cast<float*>(ring);
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
          for (int i = 0; i < S::kSteps; ++i) {
            // rows gid and gid + 8 of a product: 16-bit dims gid, gid + 8, int8 dims 2 gid, 2 gid + 1
            const int d0 = 16 * i + (DT == DT_I8 ? 2 * gid : gid), d1 = d0 + (DT == DT_I8 ? 1 : 8);
            ost[j * S::kOStride + d0] = o[i][nt][e] * f;
            ost[j * S::kOStride + d1] = o[i][nt][2 + e] * f;
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
        const float f = mst[w][j][0] == -INFINITY ? 0.0f : ex2(mst[w][j][0] - M);
        const float4 x = *reinterpret_cast<const float4*>(
            reinterpret_cast<const float*>(smem + w * p.ring) + j * S::kOStride + d);
        acc.x = fmaf(f, x.x, acc.x);
        acc.y = fmaf(f, x.y, acc.y);
        acc.z = fmaf(f, x.z, acc.z);
        acc.w = fmaf(f, x.w, acc.w);
        // a NaN score leaves the maximum alone; its sum carries it on
        L = fmaf(f, mst[w][j][1], L);
      }
      if (p.direct) {
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;  // every score -infinity: zeros
        store_out(p.out, ((int64_t)b * p.n_kv * p.group + h * p.group + n0) * (D / 4) + i,
                  make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv), p.out_dtype);
        if (d == 0) {
          unit_st[j][0] = M == -INFINITY ? 0.0f : M;
          unit_st[j][1] = L == 0.0f ? 0.0f : exp2f(p.offset) / L;
        }
      } else {
        *reinterpret_cast<float4*>(p.part + (slot * S::kHP + j) * D + d) = acc;
        if (d == 0) {
          p.stats[(slot * S::kHP + j) * 2] = M;
          p.stats[(slot * S::kHP + j) * 2 + 1] = L;
        }
      }
    }
    if (p.direct && p.scores) {  // (a single chunk of heads)
      __syncthreads();
      for (int t = threadIdx.x; t < len; t += kThreads) {
        const int row = lk_paged_row(__ldcg(trow + (t >> p.page_shift)), t, h, p.n_pages, p.n_kv, p.page_shift);
        if (row < 0) continue;
        const float* src = p.scores + (first_block + t / kTok) * p.hs * kTok + t % kTok;
        float add = 0.0f;
#pragma unroll 4
        for (int j = 0; j < heads; ++j) add = fmaf(ex2(__ldcg(src + j * kTok) - unit_st[j][0]), unit_st[j][1], add);
        p.mass[row] = __ldcg(p.mass + row) + add;
      }
    }
    __syncthreads();
    i0 += s1 - s0;
  }
}

// ---------------------------------------------------------------- joining the partials
// CTAs [0, n_out): a warp per (sequence, head), or a whole CTA where a unit
// has many pieces: their weights, then out = sum_c w_c O_c / sum_c w_c l_c.
// CTAs behind them (accumulate): kMassTok slots of one
// (sequence, kv head), four a thread: mass += sum over the heads of
// exp2(s - M) / L.  Latency-bound: what does not depend on the statistics
// (pieces, scores, page table, mass) is requested before they are reduced.
constexpr int kJoinThreads = 256;
constexpr int kMassTok = 4 * kJoinThreads;

struct JoinParams {
  const int32_t* starts;
  const float* stats;
  const float* part;
  const float* scores;
  float* mass;
  const int32_t* table;
  const int32_t* seq_len;
  void* out;
  int resident;  // CTAs of the split kernel the GPU holds
  int n_pages, page_shift, n_kv, D, batch, width, group, nch, max_len, hp, hs, out_dtype, mass_chunks;
  int n_out, wph;  // CTAs for the outputs, warps a head
  float offset;  // log2 of the factor the sums are held with
};

// The pieces of a unit: CTAs [c0, c1] of the split kernel, slots c + unit.
struct Pieces {
  int c0, c1;
};
LK_DEVICE Pieces unit_pieces(const JoinParams& p, int64_t start, int nb, int64_t N) {
  Pieces r;
  const int64_t G = working_ctas(N, p.resident);
  r.c0 = (int)quotient((start + 1) * G - 1, N);
  r.c1 = (int)quotient((start + nb) * G - 1, N);
  return r;
}

// Maximum and sum of one head over a unit's pieces (one warp; every lane gets
// both).  NaN sums stay NaN; a maximum of -infinity has the sum 0.
LK_DEVICE float2 warp_stats(const JoinParams& p, const Pieces& pc, int unit, int j) {
  const int lane = threadIdx.x & 31;
  float M = -INFINITY, L = 0.0f;
  for (int c = pc.c0 + lane; c <= pc.c1; c += 32) {
    const float2 s = __ldcg(reinterpret_cast<const float2*>(p.stats + (((int64_t)c + unit) * p.hp + j) * 2));
    const float mn = fmaxf(M, s.x);
    if (mn != -INFINITY) {
      L = (M == -INFINITY ? 0.0f : L * ex2(M - mn)) + (s.x == -INFINITY ? 0.0f : s.y * ex2(s.x - mn));
      M = mn;
    }
    if (s.y != s.y) L = s.y;
  }
  const float top = lk_warp_max(M);
  const float part = L != L ? L : (M == -INFINITY ? 0.0f : L * ex2(M - top));
  return make_float2(top, lk_warp_sum(part));
}

__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ float4 red[kJoinThreads];
  __shared__ float2 st[LK_MAX_HEADS];
  const int per_seq = p.n_kv * p.nch;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n_heads = p.n_kv * p.group;
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  if ((int)blockIdx.x < p.n_out) {
    // p.wph warps a head: lanes over float4 columns, the pieces dealt out to the warps (and, up to D = 64, to the
    // halves of a warp or more)
    const int per_cta = (kJoinThreads / 32) / p.wph;
    const int head = blockIdx.x * per_cta + warp / p.wph;
    const int64_t N = (int64_t)__ldcg(p.starts + p.batch) * per_seq;
    const bool on = head < p.batch * n_heads;
    const int b = on ? head / n_heads : 0, j = on ? head - b * n_heads : 0;
    const int b0 = __ldcg(p.starts + b), nb = on ? __ldcg(p.starts + b + 1) - b0 : 0;
    const int h = j / p.group, jg = j - h * p.group;
    const int ch = jg / p.hp, jc = jg - ch * p.hp;
    const int hc = h * p.nch + ch, unit = b * per_seq + hc;
    const int vec = p.D / 4;                   // float4 columns, up to 64
    const int threads = p.wph * 32, tid = (warp % p.wph) * 32 + lane;
    const int groups = max(1, threads / vec);  // a single warp takes more than 32 columns in turns
    const int g = threads < vec ? 0 : tid / vec;
    float2 s = make_float2(-INFINITY, 0.0f);
    Pieces pc{0, -1};
    if (nb > 0) pc = unit_pieces(p, (int64_t)b0 * per_seq + (int64_t)hc * nb, nb, N);
    constexpr int kAhead = 4;
    float4 x[kAhead];
    float mc[kAhead];
    for (int d = threads < vec ? tid : tid - g * vec, turn = 0; turn == 0 || d < vec; d += threads, ++turn) {
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      auto load = [&](int c, float4& xv, float& mv) {
        xv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        mv = -INFINITY;
        if (g < groups && d < vec && c <= pc.c1) {
          const int64_t at = ((int64_t)c + unit) * p.hp + jc;
          mv = __ldcg(p.stats + at * 2);
          xv = __ldcg(reinterpret_cast<const float4*>(p.part + at * p.D) + d);
        }
      };
#pragma unroll
      for (int i = 0; i < kAhead; ++i) load(pc.c0 + g + i * groups, x[i], mc[i]);
      if (turn == 0) s = warp_stats(p, pc, unit, jc);  // while the pieces travel
      // every score -infinity (L = 0): zeros
      const float inv = s.y == 0.0f ? 0.0f : 1.0f / s.y;
      for (int c = pc.c0 + g; c <= pc.c1; c += kAhead * groups) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const float f = mc[i] == -INFINITY ? 0.0f : ex2(mc[i] - s.x);
          acc.x = fmaf(f, x[i].x, acc.x);
          acc.y = fmaf(f, x[i].y, acc.y);
          acc.z = fmaf(f, x[i].z, acc.z);
          acc.w = fmaf(f, x[i].w, acc.w);
          load(c + (i + kAhead) * groups, x[i], mc[i]);
        }
      }
      if (groups > 1) {  // the same for every warp of the launch
        float4* r = red + (warp / p.wph) * threads;
        if (g < groups) r[g * vec + d] = acc;
        __syncthreads();
        if (g == 0)
          for (int i = 1; i < groups; ++i) {
            const float4 y = r[i * vec + d];
            acc.x += y.x;
            acc.y += y.y;
            acc.z += y.z;
            acc.w += y.w;
          }
      }
      if (on && g == 0 && d < vec) {
        acc.x *= inv;
        acc.y *= inv;
        acc.z *= inv;
        acc.w *= inv;
        const int64_t at = (int64_t)head * vec + d;
        store_out(p.out, at, acc, p.out_dtype);
      }
      if (threads >= vec) break;
    }
    return;
  }
  // ---- accumulated weights
  const int i = blockIdx.x - p.n_out;
  const int bh = i / p.mass_chunks, t0 = (i - bh * p.mass_chunks) * kMassTok;
  const int b = bh / p.n_kv, h = bh - b * p.n_kv;
  const int len = max(0, min(__ldcg(p.seq_len + b), p.max_len));
  if (t0 >= len) return;
  const int64_t N = (int64_t)__ldcg(p.starts + p.batch) * per_seq;
  const int b0 = __ldcg(p.starts + b), nb = __ldcg(p.starts + b + 1) - b0;
  // this thread's four slots: their rows, mass and first scores
  const int t = t0 + 4 * threadIdx.x;
  const int32_t* trow = p.table + (int64_t)b * p.width;
  const bool whole = p.page_shift >= 2 && t + 4 <= len;  // four slots of one page, 16-byte aligned
  int row[4];
  float4 m = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (whole) {
    row[0] = lk_paged_row(__ldcg(trow + (t >> p.page_shift)), t, h, p.n_pages, p.n_kv, p.page_shift);
    if (row[0] >= 0) m = __ldcg(reinterpret_cast<const float4*>(p.mass + row[0]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      row[e] = t + e < len ? lk_paged_row(__ldcg(trow + ((t + e) >> p.page_shift)), t + e, h, p.n_pages, p.n_kv,
                                          p.page_shift)
                           : -1;
      if (row[e] >= 0) (&m.x)[e] = __ldcg(p.mass + row[e]);
    }
  }
  // scores of four tokens of head j: t < len lies in a written block, whose 16 tokens are all there
  auto score = [&](int j) {
    const int ch = j / p.hp;
    const float* src = p.scores +
        (((int64_t)b0 * per_seq + (int64_t)(h * p.nch + ch) * nb + t / kTok) * p.hs + (j - ch * p.hp)) * kTok +
        t % kTok;
    return __ldcg(reinterpret_cast<const float4*>(src));
  };
  constexpr int kAhead = 4;
  float4 sc[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (t < len && j < p.group) sc[j] = score(j);
  for (int j = warp; j < p.group; j += kJoinThreads / 32) {
    const int ch = j / p.hp, hc = h * p.nch + ch;
    const Pieces pc = unit_pieces(p, (int64_t)b0 * per_seq + (int64_t)hc * nb, nb, N);
    const float2 s = warp_stats(p, pc, b * per_seq + hc, j - ch * p.hp);
    // exp2(score - M) / L with the sum's factor taken out of L
    if (lane == 0) st[j] = make_float2(s.x == -INFINITY ? 0.0f : s.x, s.y == 0.0f ? 0.0f : exp2f(p.offset) / s.y);
  }
  __syncthreads();
  if (t >= len) return;
  float4 add = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int j0 = 0; j0 < p.group; j0 += kAhead) {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int j = j0 + e;
      if (j < p.group) {
        const float2 s = st[j];
        add.x = fmaf(ex2(sc[e].x - s.x), s.y, add.x);
        add.y = fmaf(ex2(sc[e].y - s.x), s.y, add.y);
        add.z = fmaf(ex2(sc[e].z - s.x), s.y, add.z);
        add.w = fmaf(ex2(sc[e].w - s.x), s.y, add.w);
      }
      if (j + kAhead < p.group) sc[e] = score(j + kAhead);
    }
  }
  m.x += add.x;
  m.y += add.y;
  m.z += add.z;
  m.w += add.w;
  if (whole) {
    if (row[0] >= 0) *reinterpret_cast<float4*>(p.mass + row[0]) = m;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (row[e] >= 0) p.mass[row[e]] = (&m.x)[e];
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

// Up to so many tokens (more with more units, which share the GPU) a unit is one CTA's: one launch and no join.  The
// lengths are the device's, so the rule knows only their bound.  256-byte rows, group 4, in a graph, direct against
// split: equal lengths: 4 units of 512 tokens 6.7 us against 7.9; 32 of 768 8.4 against 10.7; 128 of 1024 14.2 against
// 21.1, of 2048 23.8 against 31.2; 256 of 2048 50.5 against 50.7.  Lengths spread over (0, max]: 128 units to 1024
// 11.6 against 27.5, to 2048 18.2 against 30.7, 256 to 2048 32.4 against 43.7.  The split gains where one sequence is
// much longer than all others (64 tokens): 128 units, one sequence of 1024 9.9 against 10.5, of 2048 15.9 against
// 13.0; 256 units, of 2048 23.6 against 15.8.
constexpr int kDirect = 512, kDirectPer = 24, kDirectMost = 2048;

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Plan {
  int hp, nch, units, hs, vc, nt, grid, resident, unit_blocks;
  bool direct, wide;
  int64_t blocks;
  size_t off_stats, off_part, off_scores, bytes;
};

template <int VC, int NT>
int min_ctas(int dt) {
  if (dt == DT_BF16) return Shape<VC, NT, DT_BF16, kWarps>::kMinCtas;
  return dt == DT_F16 ? Shape<VC, NT, DT_F16, kWarps>::kMinCtas : Shape<VC, NT, DT_I8, kWarps>::kMinCtas;
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
  r.resident = num_sms * ctas_per_sm(r.vc, r.nt, dt);
  r.grid = (int)working_ctas(r.blocks, r.resident);
  r.unit_blocks = (max_len + kTok - 1) / kTok;
  r.direct = max_len <= std::max(kDirect, (int)std::min<int64_t>(kDirectMost, (int64_t)kDirectPer * r.units)) && (!accumulate || r.nch == 1);
  // Eight warps a CTA where every CTA has an SM to itself (128 units of 1024 tokens: 15.2 us against 20.0; 256
  // units: 28.5 against 25.4), if there are blocks for them.
  r.wide = r.direct && r.units <= num_sms && r.unit_blocks > kWarps &&
           2 * kTok * (r.vc * 64 * (dt == DT_I8 ? 1 : 2)) <= kWideStage;
  if (r.direct) {
    r.grid = r.units;
    r.off_stats = r.off_part = r.off_scores = 0;
    r.bytes = std::max<size_t>(accumulate ? (size_t)r.blocks * r.hs * kTok * 4 : 0, 256);
    return r;
  }
  const size_t slots = (size_t)r.grid + r.units;
  r.off_stats = round256((size_t)(batch + 1) * 4);
  r.off_part = r.off_stats + round256(slots * r.hp * 2 * 4);
  r.off_scores = r.off_part + round256(slots * r.hp * D * 4);
  r.bytes = r.off_scores + (accumulate ? (size_t)r.blocks * r.hs * kTok * 4 : 0);
  return r;
}

// `blocks`: at most so many for a warp.  Raises the kernel's dynamic shared memory limit once per device.
template <int VC, int NT, int DT, int W, bool FULL>
cudaError_t launch_one(int grid, int blocks, PagedParams p, cudaStream_t stream) {
  using S = Shape<VC, NT, DT, W>;
  static std::atomic<uint64_t> ready{0};  // devices (bit = number)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(paged_decode_kernel<VC, NT, DT, W, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             S::smem(S::kStages));
    if (e != cudaSuccess) return e;
    if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
  }
  p.ring = S::ring(blocks);
  return lk::launch_pdl(paged_decode_kernel<VC, NT, DT, W, FULL>, dim3(grid), dim3(W * 32), stream, p, S::smem(blocks));
}

template <int VC, int NT, int DT, int W>
cudaError_t launch_dim(int grid, int blocks, const PagedParams& p, cudaStream_t stream) {
  return p.D == VC * 64 ? launch_one<VC, NT, DT, W, true>(grid, blocks, p, stream)
                        : launch_one<VC, NT, DT, W, false>(grid, blocks, p, stream);
}

template <int VC, int NT, int DT>
cudaError_t launch_warps(const Plan& r, const PagedParams& p, cudaStream_t stream) {
  if constexpr (Shape<VC, NT, DT, 8>::kStageB <= kWideStage) {
    if (r.wide) return launch_dim<VC, NT, DT, 8>(r.grid, (r.unit_blocks + 7) / 8, p, stream);
  }
  return launch_dim<VC, NT, DT, kWarps>(r.grid, r.direct ? (r.unit_blocks + kWarps - 1) / kWarps : 1 << 20, p, stream);
}

template <int VC, int NT>
cudaError_t launch_split(int dt, const Plan& r, const PagedParams& p, cudaStream_t stream) {
  if (dt == DT_BF16) return launch_warps<VC, NT, DT_BF16>(r, p, stream);
  if (dt == DT_F16) return launch_warps<VC, NT, DT_F16>(r, p, stream);
  return launch_warps<VC, NT, DT_I8>(r, p, stream);
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
  p.resident = r.resident;
  p.direct = r.direct;
  p.unit_blocks = r.unit_blocks;
  p.out = a.out;
  p.out_dtype = a.out_dtype;
  p.third = dt == DT_BF16 && a.out_dtype == LK_F32;
  p.mass = a.accumulate ? c.mass : nullptr;
  p.offset = dt == DT_BF16 ? 0.0f : kHeld;
  cudaError_t e;
  switch (r.vc * 2 + (r.nt - 1)) {
    case 2: e = launch_split<1, 1>(dt, r, p, stream); break;
    case 3: e = launch_split<1, 2>(dt, r, p, stream); break;
    case 4: e = launch_split<2, 1>(dt, r, p, stream); break;
    case 5: e = launch_split<2, 2>(dt, r, p, stream); break;
    case 6: e = launch_split<3, 1>(dt, r, p, stream); break;
    default: e = launch_split<4, 1>(dt, r, p, stream); break;
  }
  if (e != cudaSuccess || r.direct) return e;
  JoinParams j{};
  j.starts = p.starts;
  j.stats = p.stats;
  j.part = p.part;
  j.scores = p.scores;
  j.mass = a.accumulate ? c.mass : nullptr;
  j.table = p.table;
  j.seq_len = p.seq_len;
  j.out = a.out;
  j.resident = r.resident;
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
  j.offset = p.offset;
  j.mass_chunks = a.accumulate ? (a.max_len + kMassTok - 1) / kMassTok : 0;
  // about grid / units pieces a unit: one warp reads eight in two turns
  j.wph = r.grid > 8 * r.units ? kJoinThreads / 32 : 1;
  const int per_cta = (kJoinThreads / 32) / j.wph;
  j.n_out = (c.batch * a.n_heads + per_cta - 1) / per_cta;
  const unsigned ctas = (unsigned)j.n_out + (unsigned)(c.batch * c.n_kv_heads) * (unsigned)j.mass_chunks;
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
