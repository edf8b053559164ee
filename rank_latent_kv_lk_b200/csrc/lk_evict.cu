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
// keys: 2048 bins over the current interval, then the bin that holds it, so
// three passes (32 bits = 11 + 11 + 10).  Ties at that key go to the lowest slots: each thread owns
// consecutive slots, so block-wide prefix sums over the threads give every
// equal key, every hole and every moving token its number.  The CTA also
// writes the kept mass and positions.
// move_kernel: the listed rows of K and V (and int8 scales), 16 bytes a lane,
// and the new lengths (which select_kernel's CTAs still read).
// The holes lie below the budget and the moving rows at or above it, so the
// moves cannot meet.
#include "lk_serving.cuh"

namespace {

constexpr int kBins = 2048;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;  // moves a CTA takes at a time
constexpr int kAhead = 8;      // moves a thread has in flight

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
  int max_len, budget, window, n_sink, cap, n_keys, in_place, lanes;
};

// Larger mass, larger key; +0 and -0 alike.
LK_DEVICE uint32_t mass_key(float x) {
  if (x != x) return 1u;
  const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block (every thread); total in `sum`.
template <int THREADS>
LK_DEVICE int block_scan(int x, int* warp_sums, int& sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // warp_sums of an earlier scan are read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  int base = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int s = warp_sums[w];
    if (w < warp) base += s;
    tot += s;
  }
  sum = tot;
  return base + inc - x;
}

// Sum of the values of the warps before this one; the sum of all in `sum`.
template <int WARPS>
LK_DEVICE int warp_prefix(int x, int* warp_sums, int* sum = nullptr) {
  __syncthreads();  // warp_sums of an earlier use are read
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = x;
  __syncthreads();
  int base = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const int v = warp_sums[w];
    if (w < (int)(threadIdx.x >> 5)) base += v;
    tot += v;
  }
  if (sum) *sum = tot;
  return base;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t smem_keys[];
  __shared__ int hist[kBins];
  __shared__ int warp_sums[THREADS / 32];
  __shared__ int pick[2];
  const int unit = blockIdx.x, b = unit / p.n_kv, h = unit - b * p.n_kv;
  const int tid = threadIdx.x;
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  const int n = max(0, min(__ldcg(p.seq_len + b), p.max_len));
  const int32_t* trow = p.table + (int64_t)b * p.width;
  auto row_of = [&](int t) {
    return lk_paged_row(trow[t >> p.page_shift], t, h, p.n_pages, p.n_kv, p.page_shift);
  };
  if (n <= p.budget) {  // nothing leaves
    if (tid == 0) p.counts[unit] = 0;
    if (!p.in_place)
      for (int t = tid; t < n; t += THREADS) {
        const int row = row_of(t);
        if (row < 0) continue;
        p.mass_out[row] = __ldcg(p.mass + row);
        p.pos_out[row] = __ldcg(p.pos + row);
      }
    return;
  }
  uint32_t* keys = p.keys ? p.keys + (int64_t)unit * p.n_keys : smem_keys;
  const int newest = __ldcg(p.next_pos + b) - p.window;

  // ---- keys, kBatch tokens' look-ups at a time; which are protected stays in `safe` (bit i: this thread's
  // i-th token) for the first 64 a thread, and is read again for those behind
  constexpr int kBatch = THREADS == 1024 ? 16 : 8;
  auto is_safe = [&](int ps) { return ps < p.n_sink || ps >= newest; };
  uint64_t safe = 0;
  int prot = 0;
  for (int i0 = 0; i0 * THREADS + tid < n; i0 += kBatch) {
    int row[kBatch], ps[kBatch];
    float m[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = (i0 + i) * THREADS + tid;
      row[i] = t < n ? row_of(t) : -1;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      m[i] = row[i] >= 0 ? __ldcg(p.mass + row[i]) : NAN;
      ps[i] = row[i] >= 0 ? __ldcg(p.pos + row[i]) : 0;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int t = (i0 + i) * THREADS + tid;
      if (t < n) keys[t] = mass_key(m[i]);
      if (row[i] >= 0 && is_safe(ps[i])) {
        ++prot;
        if (i0 + i < 64) safe |= 1ull << (i0 + i);
      }
    }
  }
  int n_prot;
  block_scan<THREADS>(prot, warp_sums, n_prot);
  const bool among = n_prot >= p.budget;  // select among the protected alone
  if (n_prot > 0) {
    for (int i = 0, t = tid; t < n; ++i, t += THREADS) {
      bool s = i < 64 && (safe >> i & 1);
      if (i >= 64) {
        const int row = row_of(t);
        s = row >= 0 && is_safe(__ldcg(p.pos + row));
      }
      if (s && !among) keys[t] = 0xFFFFFFFFu;
      if (!s && among) keys[t] = 0u;
    }
  }

  // ---- the budget-th largest key: `need` of the keys in [lo, lo + 2^bits) are still wanted
  uint32_t lo = 0;
  int bits = 32, need = p.budget;
  while (bits > 0) {
    const int shift = max(0, bits - 11);
    for (int i = tid; i < kBins; i += THREADS) hist[i] = 0;
    __syncthreads();
    for (int t = tid; t < n; t += THREADS) {
      const uint32_t d = keys[t] - lo;
      if (keys[t] >= lo && (bits == 32 || d < (1u << bits))) atomicAdd(&hist[d >> shift], 1);
    }
    __syncthreads();
    // bins from the top: thread i owns bins [kPer i', ...) with i' counted from the top
    constexpr int kPer = kBins / THREADS;
    int mine = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) mine += hist[kBins - 1 - (tid * kPer + e)];
    int all;
    int above = block_scan<THREADS>(mine, warp_sums, all);
    if (above < need && above + mine >= need) {
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int bin = kBins - 1 - (tid * kPer + e), x = hist[bin];
        if (above < need && above + x >= need) {
          pick[0] = bin;
          pick[1] = above;
        }
        above += x;
      }
    }
    __syncthreads();
    lo += (uint32_t)pick[0] << shift;
    need -= pick[1];
    bits = shift;
    __syncthreads();  // hist and pick are read
  }

  // ---- consecutive slots per warp, 32 at a time; each key makes room for a flag: 1 = kept
  const int lane = tid & 31, warp = tid >> 5;
  const uint32_t below = (1u << lane) - 1;
  constexpr int kWarps = THREADS / 32;
  const int seg = ((n + THREADS - 1) / THREADS) * 32;
  const int t0 = warp * seg, t1 = min(n, t0 + seg);
  int eq = 0;
#pragma unroll 4
  for (int t = t0 + lane; t - lane < t1; t += 32) eq += __popc(__ballot_sync(0xffffffffu, t < t1 && keys[t] == lo));
  int seen = warp_prefix<kWarps>(eq, warp_sums), holes = 0, movers = 0;
#pragma unroll 4
  for (int t = t0 + lane; t - lane < t1; t += 32) {
    const uint32_t key = t < t1 ? keys[t] : 0u;
    const uint32_t e = __ballot_sync(0xffffffffu, t < t1 && key == lo);
    const bool kept = t < t1 && (key > lo || (key == lo && seen + __popc(e & below) < need));
    seen += __popc(e);
    if (t < t1) keys[t] = kept;
    holes += __popc(__ballot_sync(0xffffffffu, t < t1 && t < p.budget && !kept));
    movers += __popc(__ballot_sync(0xffffffffu, t >= p.budget && kept));
  }
  int n_holes;
  int hole = warp_prefix<kWarps>(holes, warp_sums, &n_holes);
  int mover = warp_prefix<kWarps>(movers, warp_sums);
  int32_t* src = p.src + (int64_t)unit * p.cap;
  int32_t* dst = p.dst + (int64_t)unit * p.cap;
#pragma unroll 4
  for (int t = t0 + lane; t - lane < t1; t += 32) {
    const bool kept = t < t1 && keys[t];
    const uint32_t hb = __ballot_sync(0xffffffffu, t < t1 && t < p.budget && !kept);
    const uint32_t mb = __ballot_sync(0xffffffffu, t >= p.budget && kept);
    if (hb >> lane & 1) dst[hole + __popc(hb & below)] = t;
    if (mb >> lane & 1) src[mover + __popc(mb & below)] = t;
    hole += __popc(hb);
    mover += __popc(mb);
  }
  __syncthreads();  // the lists (of slots so far) and flags are written
  if (tid == 0) p.counts[unit] = n_holes;
  if (!p.in_place) {
    for (int i0 = 0; i0 * THREADS + tid < p.budget; i0 += kBatch) {
      int row[kBatch], ps[kBatch];
      float m[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int t = (i0 + i) * THREADS + tid;
        row[i] = t < p.budget && keys[t] ? row_of(t) : -1;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (row[i] >= 0) {
          m[i] = __ldcg(p.mass + row[i]);
          ps[i] = __ldcg(p.pos + row[i]);
        }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (row[i] >= 0) {
          p.mass_out[row[i]] = m[i];
          p.pos_out[row[i]] = ps[i];
        }
    }
  }
  // the moves: slots become rows, and their mass and positions go along
  constexpr int kPairs = 4;
  for (int i0 = 0; i0 * THREADS + tid < n_holes; i0 += kPairs) {
    int d[kPairs], f[kPairs], ps[kPairs];
    float m[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int j = (i0 + i) * THREADS + tid;
      d[i] = j < n_holes ? dst[j] : -1;
      f[i] = j < n_holes ? src[j] : -1;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      if (d[i] >= 0) {
        d[i] = row_of(d[i]);
        f[i] = row_of(f[i]);
        if (f[i] < 0) d[i] = -1;
      } else {
        d[i] = -2;  // behind the list
      }
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
      if (d[i] >= 0) {
        m[i] = __ldcg(p.mass + f[i]);
        ps[i] = __ldcg(p.pos + f[i]);
      }
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int j = (i0 + i) * THREADS + tid;
      if (d[i] >= 0) {
        p.mass_out[d[i]] = m[i];
        p.pos_out[d[i]] = ps[i];
      }
      if (d[i] >= -1) {
        dst[j] = d[i];
        src[j] = f[i];
      }
    }
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ EvictParams p) {
  const int unit = blockIdx.x;
  lk_grid_dep_wait();
  lk_grid_dep_launch();
  if (blockIdx.y == 0 && unit % p.n_kv == 0 && threadIdx.x == 0) {
    const int b = unit / p.n_kv;
    p.seq_len_out[b] = min(max(0, min(__ldcg(p.seq_len + b), p.max_len)), p.budget);
  }
  const int count = __ldcg(p.counts + unit);
  const int32_t* src = p.src + (int64_t)unit * p.cap;
  const int32_t* dst = p.dst + (int64_t)unit * p.cap;
  // `lanes` lanes per move (the power of two above its 16-byte pieces, K's then V's; 32 take two turns)
  const int vec = p.row_bytes / 16, pieces = 2 * vec;
  const int sub = (int)threadIdx.x & (p.lanes - 1), per = kMoveThreads / p.lanes;
  for (int m0 = blockIdx.y * kMoveRows; m0 < count; m0 += gridDim.y * kMoveRows) {
    for (int m1 = m0 + (int)threadIdx.x / p.lanes; m1 < min(m0 + kMoveRows, count); m1 += kAhead * per) {
      int s[kAhead], d[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) {
        const int m = m1 + e * per;
        const bool in = m < min(m0 + kMoveRows, count);
        s[e] = in ? __ldcg(src + m) : -1;
        d[e] = in ? __ldcg(dst + m) : -1;
      }
      for (int c = sub; c < pieces; c += p.lanes) {
        uint8_t* base = c < vec ? p.k : p.v;
        const int off = 16 * (c < vec ? c : c - vec);
        uint4 x[kAhead];
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (s[e] >= 0 && d[e] >= 0) x[e] = __ldcg(reinterpret_cast<const uint4*>(base + (int64_t)s[e] * p.row_bytes + off));
#pragma unroll
        for (int e = 0; e < kAhead; ++e)
          if (s[e] >= 0 && d[e] >= 0) *reinterpret_cast<uint4*>(base + (int64_t)d[e] * p.row_bytes + off) = x[e];
        if (p.is_i8 && off == 0) {
          float* sc = c < vec ? p.ks : p.vs;
#pragma unroll
          for (int e = 0; e < kAhead; ++e)
            if (s[e] >= 0 && d[e] >= 0) sc[d[e]] = __ldcg(sc + s[e]);
        }
      }
    }
  }
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Keys a CTA holds in shared memory; longer sequences keep theirs in the workspace.
constexpr int kSmemKeys = 48 * 1024;
constexpr int kSmallKeys = 4096;  // up to here 512 threads a CTA

int move_cap(int max_len, int budget) { return std::max(0, std::min(budget, max_len - budget)); }

}  // namespace

LK_DEFINE_STATUS_ACCESSOR(lk_evict_status_word)

namespace lk {

size_t paged_evict_workspace_bytes(int units, int max_len, int budget) {
  const size_t lists = round256((size_t)units * move_cap(max_len, budget) * 4);
  return round256((size_t)units * 4) + 2 * lists +
         (max_len > budget && max_len > kSmemKeys ? (size_t)units * max_len * 4 : 0);
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
  const size_t lists = round256((size_t)units * p.cap * 4);
  p.counts = reinterpret_cast<int32_t*>(ws);
  p.src = reinterpret_cast<int32_t*>(ws + round256((size_t)units * 4));
  p.dst = reinterpret_cast<int32_t*>(ws + round256((size_t)units * 4) + lists);
  const bool spill = a.max_len > a.budget && a.max_len > kSmemKeys;
  p.keys = spill ? reinterpret_cast<uint32_t*>(ws + round256((size_t)units * 4) + 2 * lists) : nullptr;
  p.n_keys = a.max_len;
  const size_t smem = spill || a.max_len <= a.budget ? 0 : (size_t)a.max_len * 4;
  cudaError_t e;
  if (a.max_len <= kSmallKeys) {
    e = launch_pdl(select_kernel<512>, dim3(units), dim3(512), stream, p, smem);
  } else {
    if (smem > 36 * 1024) {
      e = cudaFuncSetAttribute(select_kernel<1024>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemKeys * 4);
      if (e != cudaSuccess) return e;
    }
    e = launch_pdl(select_kernel<1024>, dim3(units), dim3(1024), stream, p, smem);
  }
  if (e != cudaSuccess) return e;
  const int chunks = std::max(1, std::min(1024, (p.cap + kMoveRows - 1) / kMoveRows));
  return launch_pdl(move_kernel, dim3(units, chunks), dim3(kMoveThreads), stream, p);
}

}  // namespace lk
