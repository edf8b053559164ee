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
constexpr int kMoveRows = 32;  // moves per CTA

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
  int max_len, budget, window, n_sink, cap, n_keys, in_place;
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
    return lk_paged_row(__ldcg(trow + (t >> p.page_shift)), t, h, p.n_pages, p.n_kv, p.page_shift);
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

  // ---- keys; a protected token's top bit pattern is set once their number is known
  int prot = 0;
  for (int t = tid; t < n; t += THREADS) {
    const int row = row_of(t);
    uint32_t key = 1u;
    if (row >= 0) {
      key = mass_key(__ldcg(p.mass + row));
      const int ps = __ldcg(p.pos + row);
      prot += ps < p.n_sink || ps >= newest;
    }
    keys[t] = key;
  }
  int n_prot;
  block_scan<THREADS>(prot, warp_sums, n_prot);
  const bool among = n_prot >= p.budget;  // select among the protected alone
  if (n_prot > 0) {
    for (int t = tid; t < n; t += THREADS) {
      const int row = row_of(t);
      const int ps = row >= 0 ? __ldcg(p.pos + row) : 0;
      const bool safe = row >= 0 && (ps < p.n_sink || ps >= newest);
      if (safe && !among) keys[t] = 0xFFFFFFFFu;
      if (!safe && among) keys[t] = 0u;
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

  // ---- consecutive slots per thread (an odd number: distinct banks)
  const int per = ((n + THREADS - 1) / THREADS) | 1;
  const int t0 = min(n, tid * per), t1 = min(n, t0 + per);
  int eq = 0;
  for (int t = t0; t < t1; ++t) eq += keys[t] == lo;
  int dummy;
  const int eq0 = block_scan<THREADS>(eq, warp_sums, dummy);
  int seen = eq0, holes = 0, movers = 0;
  for (int t = t0; t < t1; ++t) {
    const uint32_t key = keys[t];
    bool kept = key > lo;
    if (key == lo) kept = seen++ < need;
    holes += t < p.budget && !kept;
    movers += t >= p.budget && kept;
  }
  int n_holes, n_movers;
  int hole = block_scan<THREADS>(holes, warp_sums, n_holes);
  int mover = block_scan<THREADS>(movers, warp_sums, n_movers);
  int32_t* src = p.src + (int64_t)unit * p.cap;
  int32_t* dst = p.dst + (int64_t)unit * p.cap;
  seen = eq0;
  for (int t = t0; t < t1; ++t) {
    const uint32_t key = keys[t];
    bool kept = key > lo;
    if (key == lo) kept = seen++ < need;
    if (t < p.budget && !kept) dst[hole++] = row_of(t);
    else if (t >= p.budget && kept) src[mover++] = row_of(t);
    else if (t < p.budget && !p.in_place) {
      const int row = row_of(t);
      if (row >= 0) {
        p.mass_out[row] = __ldcg(p.mass + row);
        p.pos_out[row] = __ldcg(p.pos + row);
      }
    }
  }
  __syncthreads();  // the lists are written
  if (tid == 0) p.counts[unit] = n_holes;
  for (int i = tid; i < n_holes; i += THREADS) {
    const int d = dst[i], s = src[i];
    if (d < 0 || s < 0) continue;
    p.mass_out[d] = __ldcg(p.mass + s);
    p.pos_out[d] = __ldcg(p.pos + s);
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
  const int vec = p.row_bytes / 16;
  const int64_t total = 2 * (int64_t)count * vec;
  const int64_t step = (int64_t)gridDim.y * kMoveThreads;
  for (int64_t i = (int64_t)blockIdx.y * kMoveThreads + threadIdx.x; i < total; i += step) {
    const int r = (int)(i / vec), c = (int)(i - (int64_t)r * vec), m = r >> 1;
    const int s = __ldcg(src + m), d = __ldcg(dst + m);
    if (s < 0 || d < 0) continue;
    uint8_t* base = (r & 1) ? p.v : p.k;
    reinterpret_cast<uint4*>(base + (int64_t)d * p.row_bytes)[c] =
        __ldcg(reinterpret_cast<const uint4*>(base + (int64_t)s * p.row_bytes) + c);
    if (p.is_i8 && c == 0) {
      float* sc = (r & 1) ? p.vs : p.ks;
      sc[d] = __ldcg(sc + s);
    }
  }
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Keys a CTA holds in shared memory; longer sequences keep theirs in the workspace.
constexpr int kSmemKeys = 48 * 1024;
constexpr int kSmallKeys = 4096;  // up to here 256 threads a CTA

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
    e = launch_pdl(select_kernel<256>, dim3(units), dim3(256), stream, p, smem);
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
