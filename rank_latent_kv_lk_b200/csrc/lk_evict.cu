// Eviction from a paged key-value cache by accumulated attention weight
// (sm_100a).
//
// Per (sequence, kv head) with n tokens > budget: tokens are ordered by
// (protected, mass, lower slot), the first `budget` stay.  Kept tokens behind
// the budget move into the evicted slots below it, so only rows that have to
// move are copied, and the sequence's first `budget` slots stay dense.
//
// select_kernel: one CTA a (sequence, kv head).  The mass becomes an
// order-preserving 32-bit key in shared memory (NaN 1, below every number;
// protected tokens 0xFFFFFFFF, or, when they alone exceed the budget, all
// others 0).  The budget-th largest key is found by narrowing an interval of
// keys: 2048 bins over the current interval, then the bin that holds it, so at
// most three passes (32 bits = 11 + 11 + 10), and fewer where a bin stays as
// a whole; the first bins are counted as the keys are made.  Which slots stay becomes a bit each;
// a thread then takes a word of 32, and prefix sums over the threads number
// the equal keys (ties go to the lowest slots), the holes and the moving
// tokens.  The CTA also writes the kept mass and positions.  Bound by latency,
// a chain of block-wide steps (schedulers issue in 39 to 46 % of their cycles,
// barriers and loads are what warps wait for most): hence four tokens an
// access, and no look at ties where there are none.  A cluster of eight CTAs a
// unit that each read all the others' bins over distributed shared memory took
// 98 us for 16384 tokens a unit where one CTA took 36, a pair gained 3 %; one
// whose CTAs each sum a part of the bins was not built.  With the moves, a call
// (in a captured graph): 32 x 8 units from 2112 to 2048 slots 10.8 us (11.1),
// 8 x 8 of up to 16384 to 4096 41.2 us (40.1), 20 of them the rows' bytes both
// ways, near the copy bandwidth, and 20 with 64 of the SMs at work.
// move_kernel: the listed rows of K and V (and int8 scales), 16 bytes a lane,
// and the new lengths (which select_kernel's CTAs still read).  Where few rows
// can move, select_kernel moves them itself.
// The holes lie below the budget and the moving rows at or above it, so the
// moves cannot meet.
#include "lk_serving.cuh"

namespace {

constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kAhead = 4;      // moves a thread has in flight
constexpr int kMostFused = 256;  // moves of a unit that select_kernel makes itself: no more than its threads

struct EvictParams {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  float* mass;
  int32_t* pos;
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* next_pos;
  float* mass_out;
  int32_t* pos_out;
  int32_t* seq_len_out;
  int32_t* counts;  // [units] moves
  int32_t* src;     // [units][cap] row moved from (-1: outside the pool)
  int32_t* dst;     // [units][cap]
  uint32_t* keys;   // [units][n_keys] where they do not fit in shared memory, else null
  int n_pages, page_shift, n_kv, row_bytes, is_i8, batch, width;
  int max_len, budget, window, n_sink, cap, n_keys, seg_max, in_place, lanes;
  int fused;          // select_kernel moves the rows too
  int lengths_apart;  // and writes the lengths (seq_len_out is another array)
};

// Larger mass, larger key; +0 and -0 alike.
LK_DEVICE uint32_t mass_key(float x) {
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix of one value a warp over the block's warps, and the sum of all.  `slots` is used once.
template <int WARPS>
LK_DEVICE int warp_prefix(int x, int* slots, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) slots[warp] = x;
  __syncthreads();
  const int v = lane < WARPS ? slots[lane] : 0;
  int inc = v;
#pragma unroll
  for (int o = 1; o < WARPS; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  all = __shfl_sync(0xffffffffu, inc, WARPS - 1);
  return __shfl_sync(0xffffffffu, inc - v, warp);
}

// Exclusive prefix of one value a thread over the block.
template <int WARPS>
LK_DEVICE int block_scan(int x, int* slots, int* sum = nullptr) {
  const int lane = threadIdx.x & 31;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  int all;
  const int before = warp_prefix<WARPS>(__shfl_sync(0xffffffffu, inc, 31), slots, all);
  if (sum) *sum = all;
  return before + inc - x;
}

LK_DEVICE void new_length(const EvictParams& p, int b) {
  p.seq_len_out[b] = min(max(0, min(__ldcg(p.seq_len + b), p.max_len)), p.budget);
}

// Rows of K and V (and scales) of `count` moves, this CTA being `part` of `parts` for the unit.  `lanes` lanes per
// move (the power of two above its 16-byte pieces, K's then V's; 32 take turns), kAhead moves a thread at a time; the
// next ones' rows are looked up while these travel.
LK_DEVICE void move_rows(const EvictParams& p, const int32_t* src, const int32_t* dst, int count, int part, int parts,
                         int threads) {
  const int vec = p.row_bytes / 16, pieces = 2 * vec;
  const int sub = (int)threadIdx.x & (p.lanes - 1), per = threads / p.lanes;
  const int stride = parts * per * kAhead;
  int s[kAhead], d[kAhead];
  auto look_up = [&](int m0) {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const int m = m0 + e * per;
      s[e] = m < count ? src[m] : -1;
      d[e] = m < count ? dst[m] : -1;
    }
  };
  int m0 = part * per * kAhead + (int)threadIdx.x / p.lanes;
  look_up(m0);
  for (; m0 < count; m0 += stride) {
    int64_t from[kAhead], to[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      const bool in = s[e] >= 0 && d[e] >= 0;
      from[e] = in ? (int64_t)s[e] * p.row_bytes : -1;
      to[e] = (int64_t)d[e] * p.row_bytes;
    }
    for (int c = sub; c < pieces; c += p.lanes) {
      uint8_t* base = (c < vec ? p.k : p.v) + 16 * (c < vec ? c : c - vec);
      uint4 x[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (from[e] >= 0) x[e] = __ldcg(reinterpret_cast<const uint4*>(base + from[e]));
      if (p.is_i8 && (c == 0 || c == vec)) {
        float* sc = c < vec ? p.ks : p.vs;
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (from[e] >= 0) sc[d[e]] = __ldcg(sc + s[e]);
      }
      if (c + p.lanes >= pieces) look_up(m0 + stride);
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (from[e] >= 0) *reinterpret_cast<uint4*>(base + to[e]) = x[e];
    }
    if (sub >= pieces) look_up(m0 + stride);
  }
}

// (At least 1024 threads an SM: 32 x 8 units of 2112 slots 12.1 us with two CTAs of 512, 18.6 with one.)
template <int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) select_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ __align__(16) uint32_t smem_keys[];  // keys, then two bits a slot: kept, equal
  // the first pass of long sequences counts in four, one for every fourth lane: weights crowd in few of its bins
  constexpr int kCopies = kThreads == 1024 ? 4 : 1, kHists = kCopies == 4 ? 4 : 3;
  __shared__ __align__(16) int hist[kHists][kBins];
  __shared__ int slots[7][kWarps];
  __shared__ int pick[3][3];
  const int unit = blockIdx.x;
  const int b = unit / p.n_kv, h = unit - b * p.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto clear_bins = [&] {
    for (int i = tid; i < kHists * kBins / 4; i += kThreads) reinterpret_cast<int4*>(hist)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
  };
  clear_bins();
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  if (p.lengths_apart && h == 0 && tid == 0) new_length(p, b);
  const int n = max(0, min(__ldcg(p.seq_len + b), p.max_len));
  const int newest = __ldcg(p.next_pos + b) - p.window;
  const int32_t* trow = p.table + (int64_t)b * p.width;
  const bool quads = p.page_shift >= 2;  // four slots from a multiple of four lie in one page
  auto row_of = [&](int t) { return lk_paged_row(trow[t >> p.page_shift], t, h, p.n_pages, p.n_kv, p.page_shift); };
  // rows (-1: none), mass and positions of the slots t .. t + 3 below `end`
  auto load4 = [&](int t, int end, int (&row)[4], float (&m)[4], int (&ps)[4]) {
    if (quads) {
      const int r = t < end ? row_of(t) : -1;
      float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      int4 i = make_int4(0, 0, 0, 0);
      if (r >= 0) {
        f = __ldcg(reinterpret_cast<const float4*>(p.mass + r));
        i = __ldcg(reinterpret_cast<const int4*>(p.pos + r));
      }
      m[0] = f.x; m[1] = f.y; m[2] = f.z; m[3] = f.w;
      ps[0] = i.x; ps[1] = i.y; ps[2] = i.z; ps[3] = i.w;
#pragma unroll
      for (int e = 0; e < 4; ++e) row[e] = r >= 0 && t + e < end ? r + e : -1;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        row[e] = t + e < end ? row_of(t + e) : -1;
        m[e] = row[e] >= 0 ? __ldcg(p.mass + row[e]) : 0.0f;
        ps[e] = row[e] >= 0 ? __ldcg(p.pos + row[e]) : 0;
      }
    }
  };
  auto is_safe = [&](int ps) { return ps < p.n_sink || ps >= newest; };

  if (n <= p.budget) {  // nothing leaves
    if (tid == 0) p.counts[unit] = 0;
    if (!p.in_place)
      for (int t = 4 * tid; t < n; t += 4 * kThreads) {
        int row[4], ps[4];
        float m[4];
        load4(t, n, row, m, ps);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (row[e] >= 0) {
            p.mass_out[row[e]] = m[e];
            p.pos_out[row[e]] = ps[e];
          }
      }
    return;
  }
  uint32_t* keys = p.keys ? p.keys + (int64_t)unit * p.n_keys : smem_keys;
  uint32_t* kept = keys + p.seg_max;
  uint32_t* ties_at = kept + p.seg_max / 32;

  // ---- keys, as if fewer tokens than the budget were protected.  With outputs apart, the slots below the budget are
  // written as they come (as many moving tokens as holes overwrite the evicted ones later): reading them again once
  // the kept ones are known took 1 us more.
  int prot = 0;
  auto count_first = [&](uint32_t key) { atomicAdd(&hist[lane & (kCopies - 1)][key >> 21], 1); };
  auto put_keys = [&](int i, const int (&row)[4], const float (&m)[4], const int (&ps)[4]) {
    uint32_t key[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool safe = row[e] >= 0 && is_safe(ps[e]);
      key[e] = safe ? 0xFFFFFFFFu : (row[e] >= 0 ? mass_key(m[e]) : 1u);
      prot += safe;
    }
    const int t = 4 * (i * kThreads + tid);
    *reinterpret_cast<uint4*>(keys + t) = make_uint4(key[0], key[1], key[2], key[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (t + e < n) count_first(key[e]);
    if (!p.in_place) {
      if (quads && row[0] >= 0 && t + 4 <= p.budget) {
        *reinterpret_cast<float4*>(p.mass_out + row[0]) = make_float4(m[0], m[1], m[2], m[3]);
        *reinterpret_cast<int4*>(p.pos_out + row[0]) = make_int4(ps[0], ps[1], ps[2], ps[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (row[e] >= 0 && t + e < p.budget) {
            p.mass_out[row[e]] = m[e];
            p.pos_out[row[e]] = ps[e];
          }
      }
    }
  };
  if (quads) {  // the page look-ups of four turns, then their mass and positions, are in flight together
    constexpr int kTurns = 4;
    for (int i0 = 0; 4 * (i0 * kThreads + tid) < n; i0 += kTurns) {
      int first[kTurns];
      float4 f[kTurns];
      int4 q[kTurns];
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int t = 4 * ((i0 + i) * kThreads + tid);
        first[i] = t < n ? row_of(t) : -1;
      }
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        f[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        q[i] = make_int4(0, 0, 0, 0);
        if (first[i] >= 0) {
          f[i] = __ldcg(reinterpret_cast<const float4*>(p.mass + first[i]));
          q[i] = __ldcg(reinterpret_cast<const int4*>(p.pos + first[i]));
        }
      }
#pragma unroll
      for (int i = 0; i < kTurns; ++i) {
        const int t = 4 * ((i0 + i) * kThreads + tid);
        if (t < n) {
          int row[4];
          const float m[4] = {f[i].x, f[i].y, f[i].z, f[i].w};
          const int ps[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) row[e] = first[i] >= 0 && t + e < n ? first[i] + e : -1;
          put_keys(i0 + i, row, m, ps);
        }
      }
    }
  } else {
    for (int i = 0; 4 * (i * kThreads + tid) < n; ++i) {
      int row[4], ps[4];
      float m[4];
      load4(4 * (i * kThreads + tid), n, row, m, ps);
      put_keys(i, row, m, ps);
    }
  }
  int n_prot;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) prot += __shfl_xor_sync(0xffffffffu, prot, o);
  warp_prefix<kWarps>(prot, slots[0], n_prot);
  if (n_prot >= p.budget) {  // select among the protected alone: the keys and the first bins again
    clear_bins();
    for (int t = 4 * tid; t < n; t += 4 * kThreads) {
      int row[4], ps[4];
      float m[4];
      uint32_t key[4];
      load4(t, n, row, m, ps);
#pragma unroll
      for (int e = 0; e < 4; ++e) key[e] = row[e] >= 0 && is_safe(ps[e]) ? mass_key(m[e]) : 0u;
      *reinterpret_cast<uint4*>(keys + t) = make_uint4(key[0], key[1], key[2], key[3]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t + e < n) count_first(key[e]);
    }
    __syncthreads();
  }

  // ---- the budget-th largest key: `need` of the keys in [lo, lo + 2^bits) are still wanted, `equal` there are
  uint32_t lo = 0;
  int bits = 32, need = p.budget, equal = 0;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    if (pass > 0) {  // (the first bins are counted with the keys)
#pragma unroll 2
      for (int t = 4 * tid; t < n; t += 4 * kThreads) {
        const uint4 k4 = *reinterpret_cast<const uint4*>(keys + t);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t d = k[e] - lo;  // keys below lo wrap around to at least 2^bits
          if (t + e < n && (d >> bits) == 0) atomicAdd(&hist[pass][d >> shift], 1);
        }
      }
      __syncthreads();
    }
    // consecutive bins a thread, from the top
    constexpr int kPer = kBins / kThreads;
    const int top = kBins - kPer * (tid + 1);
    int bin[kPer];
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      bin[e] = hist[pass][top + e];
      if constexpr (kCopies == 4) if (pass == 0) {  // and made ready for the next passes
        bin[e] += hist[1][top + e] + hist[2][top + e] + hist[kHists - 1][top + e];
        hist[1][top + e] = hist[2][top + e] = 0;
      }
    }
    int mine = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) mine += bin[e];
    int above = block_scan<kWarps>(mine, slots[1 + pass]);
    if (above < need && above + mine >= need) {
#pragma unroll
      for (int e = kPer - 1; e >= 0; --e) {
        if (above < need && above + bin[e] >= need) {
          pick[pass][0] = top + e;
          pick[pass][1] = above;
          pick[pass][2] = bin[e];
        }
        above += bin[e];
      }
    }
    __syncthreads();
    lo += (uint32_t)pick[pass][0] << shift;
    need -= pick[pass][1];
    equal = pick[pass][2];
    bits = shift;
    if (need == equal) break;  // the bin stays as a whole
  }

  // ---- a bit a slot: kept, and where ties are to be told apart, equal.  Four slots a lane; eight lanes make a word.
  const bool ties = need < equal;
  const int words = (n + 31) / 32;
  for (int t = 4 * tid; t - 4 * lane < n; t += 4 * kThreads) {
    uint32_t k = 0, q = 0;
    if (t < n) {
      const uint4 k4 = *reinterpret_cast<const uint4*>(keys + t);
      const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        k |= (uint32_t)(t + e < n && (ties ? key[e] > lo : key[e] >= lo)) << e;
        q |= (uint32_t)(t + e < n && key[e] == lo) << e;
      }
    }
    k <<= 4 * (lane & 7);
    q <<= 4 * (lane & 7);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      k |= __shfl_xor_sync(0xffffffffu, k, o);
      if (ties) q |= __shfl_xor_sync(0xffffffffu, q, o);
    }
    if ((lane & 7) == 0 && t < n) {
      kept[t >> 5] = k;
      if (ties) ties_at[t >> 5] = q;
    }
  }
  __syncthreads();
  // ---- a thread a word: the first `need` of the ties are kept too; holes and moving tokens are counted and listed.
  // The lists of slots take the keys' place: as many of each, so at most half of all.
  int n_holes = 0, n_movers = 0, n_seen = 0;
  auto low_of = [&](int w) {  // slots of the word below the budget (which lies below n: such slots are all live)
    const int in_budget = min(32, max(0, p.budget - 32 * w));
    return in_budget == 32 ? 0xffffffffu : (1u << in_budget) - 1;
  };
  if (ties) {
    for (int w0 = 0; w0 < words; w0 += kThreads) {
      const int w = w0 + tid;
      uint32_t q = w < words ? ties_at[w] : 0;
      int all;
      int left = need - n_seen - block_scan<kWarps>(__popc(q), slots[4], &all);  // of this word's ties are kept
      while (q && left < __popc(q)) q &= ~(0x80000000u >> __clz(q));  // the highest go
      if (w < words && left > 0) kept[w] |= q;
      n_seen += all;
      __syncthreads();  // slots are read
    }
  }
  uint32_t* hole_slot = keys;
  uint32_t* mover_slot = keys + p.seg_max / 2;
  for (int w0 = 0; w0 < words; w0 += kThreads) {
    const int w = w0 + tid;
    const uint32_t k = w < words ? kept[w] : 0, low = w < words ? low_of(w) : 0;
    uint32_t hb = ~k & low, mb = k & ~low;
    // both counts in one sum: a round of words holds at most 32 kThreads = 2^15 slots
    int all;
    const uint32_t at = (uint32_t)block_scan<kWarps>(__popc(hb) | __popc(mb) << 16, slots[6], &all);
    int hole = n_holes + (int)(at & 0xFFFFu), mover = n_movers + (int)(at >> 16);
    n_holes += (int)((uint32_t)all & 0xFFFFu);
    n_movers += (int)((uint32_t)all >> 16);
    for (; hb; hb &= hb - 1) hole_slot[hole++] = 32 * w + __ffs(hb) - 1;
    for (; mb; mb &= mb - 1) mover_slot[mover++] = 32 * w + __ffs(mb) - 1;
    __syncthreads();  // slots are read
  }
  if (tid == 0) p.counts[unit] = n_holes;
  __syncthreads();  // the lists are written
  // ---- the moves: slots become rows, and their mass and positions go along
  if (p.fused) {  // at most kMostFused, one a thread; mass and position travel while K and V do
    int d = -1, ps = 0;
    float m = 0.0f;
    if (tid < n_holes) {
      d = row_of((int)hole_slot[tid]);
      const int f = row_of((int)mover_slot[tid]);
      if (f < 0) d = -1;
      hole_slot[tid] = (uint32_t)d;
      mover_slot[tid] = (uint32_t)f;
      if (d >= 0) {
        m = __ldcg(p.mass + f);
        ps = __ldcg(p.pos + f);
      }
    }
    __syncthreads();
    move_rows(p, reinterpret_cast<const int32_t*>(mover_slot), reinterpret_cast<const int32_t*>(hole_slot), n_holes, 0,
              1, kThreads);
    if (d >= 0) {
      p.mass_out[d] = m;
      p.pos_out[d] = ps;
    }
    return;
  }
  int32_t* src = p.src + (int64_t)unit * p.cap;
  int32_t* dst = p.dst + (int64_t)unit * p.cap;
#pragma unroll 4
  for (int j = tid; j < n_holes; j += kThreads) {
    int d = row_of((int)hole_slot[j]);
    const int f = row_of((int)mover_slot[j]);
    if (f < 0) d = -1;
    dst[j] = d;
    src[j] = f;
    if (d >= 0) {
      p.mass_out[d] = __ldcg(p.mass + f);
      p.pos_out[d] = __ldcg(p.pos + f);
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictParams p) {
  const int unit = blockIdx.x;
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  if (blockIdx.y == 0 && unit % p.n_kv == 0 && threadIdx.x == 0) new_length(p, unit / p.n_kv);
  move_rows(p, p.src + (int64_t)unit * p.cap, p.dst + (int64_t)unit * p.cap, __ldcg(p.counts + unit), blockIdx.y,
            gridDim.y, kMoveThreads);
}

// The lengths alone, where the rows are moved already and other CTAs still had the lengths to read.
__global__ void length_kernel(const __grid_constant__ EvictParams p) {
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < p.batch) new_length(p, b);
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Slots a CTA holds keys for in shared memory; longer sequences keep theirs in the workspace.
constexpr int kSmemKeys = 40 * 1024;
int seg_of(int max_len) { return (max_len + 127) & ~127; }
size_t spill_words(int max_len) { return (size_t)seg_of(max_len) / 32 * 34; }  // keys and bits
bool spills(int max_len, int budget) { return max_len > budget && seg_of(max_len) > kSmemKeys; }

int move_cap(int max_len, int budget) { return std::max(0, std::min(budget, max_len - budget)); }

template <int THREADS>
cudaError_t launch_select(int units, size_t smem, const EvictParams& p, cudaStream_t stream) {
  if (smem > 14 * 1024) {  // with the 33 KB of bins beyond the default limit
    const cudaError_t e = cudaFuncSetAttribute(select_kernel<THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmemKeys / 32 * 34 * 4);
    if (e != cudaSuccess) return e;
  }
  return lk::launch_pdl(select_kernel<THREADS>, dim3(units), dim3(THREADS), stream, p, smem);
}

}  // namespace

LK_DEFINE_STATUS_ACCESSOR(lk_evict_status_word)

namespace lk {

size_t paged_evict_workspace_bytes(int units, int max_len, int budget) {
  const size_t lists = round256((size_t)units * move_cap(max_len, budget) * 4);
  return round256((size_t)units * 4) + 2 * lists +
         (spills(max_len, budget) ? (size_t)units * spill_words(max_len) * 4 : 0);
}

cudaError_t launch_paged_evict(const PagedEvictLaunch& a, cudaStream_t stream) {
  const PagedCacheView& c = a.c;
  const int units = c.batch * c.n_kv_heads;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  EvictParams p{};
  p.k = static_cast<uint8_t*>(c.k);
  p.v = static_cast<uint8_t*>(c.v);
  p.ks = c.k_scale;
  p.vs = c.v_scale;
  p.mass = c.mass;
  p.pos = c.pos;
  p.table = c.page_table;
  p.seq_len = a.seq_len;
  p.next_pos = a.next_pos;
  p.mass_out = a.mass_out;
  p.pos_out = a.pos_out;
  p.seq_len_out = a.seq_len_out;
  p.n_pages = c.n_pages;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  p.n_kv = c.n_kv_heads;
  p.is_i8 = c.dtype == LK_I8;
  p.row_bytes = c.head_dim * (p.is_i8 ? 1 : 2);
  p.lanes = 2;
  while (p.lanes < 32 && p.lanes < p.row_bytes / 8) p.lanes *= 2;
  p.batch = c.batch;
  p.width = c.table_width;
  p.max_len = a.max_len;
  p.budget = a.budget;
  p.window = a.window;
  p.n_sink = a.n_sink;
  p.cap = move_cap(a.max_len, a.budget);
  p.in_place = a.mass_out == c.mass;
  // Few rows can move: the selecting CTA moves them itself (32 x 8 units, 2112 slots to 2048: 11.0 us
  // against 13.0).
  p.fused = p.cap <= kMostFused;
  p.lengths_apart = p.fused && a.seq_len_out != a.seq_len;
  const size_t lists = round256((size_t)units * p.cap * 4);
  p.counts = reinterpret_cast<int32_t*>(ws);
  p.src = reinterpret_cast<int32_t*>(ws + round256((size_t)units * 4));
  p.dst = reinterpret_cast<int32_t*>(ws + round256((size_t)units * 4) + lists);
  const bool spill = spills(a.max_len, a.budget);
  p.keys = spill ? reinterpret_cast<uint32_t*>(ws + round256((size_t)units * 4) + 2 * lists) : nullptr;
  p.n_keys = (int)spill_words(a.max_len);
  p.seg_max = seg_of(a.max_len);
  const size_t smem = spill || a.max_len <= a.budget ? 0 : (size_t)p.seg_max / 32 * 34 * 4;
  cudaError_t e;
  // threads for about four slots each
  if (a.max_len <= 1024) e = launch_select<256>(units, smem, p, stream);
  else if (a.max_len <= 4096) e = launch_select<512>(units, smem, p, stream);
  else e = launch_select<1024>(units, smem, p, stream);
  if (e != cudaSuccess || p.lengths_apart) return e;
  if (p.fused) return launch_pdl(length_kernel, dim3((c.batch + 127) / 128), dim3(128), stream, p);
  // CTAs for a unit's most moves, but no more in all than four times what stays resident (dealing all units' moves
  // out in equal ranges needs a prefix sum per CTA, which cost more than ragged batches gain)
  const int rows = kMoveThreads / p.lanes * kAhead;
  const int chunks = std::max(1, std::min((p.cap + rows - 1) / rows, 16 * a.num_sms / units));
  return launch_pdl(move_kernel, dim3(units, chunks), dim3(kMoveThreads), stream, p);
}

}  // namespace lk
