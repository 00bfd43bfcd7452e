// Scaled token embedding and its gradient by sorted tokens.
//
//   forward   y[r] = scale * table[ids[r]]
//   backward  d_table[v] (+)= scale * sum_{r : ids[r] = v} dy[r]
//
// Both are bound by HBM: the forward reads the used table rows and writes y, the backward reads
// dy once and reads and writes (or only writes) the table rows.
#include <type_traits>

#include "sbp_internal.cuh"

namespace sbp {

namespace {

inline int64_t nblk(int64_t n, int64_t t) { return (n + t - 1) / t; }

constexpr int kThreads = 256;

// ---------------------------------------------------------------- vectors of V elements
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};
// stored to be evicted first: the result is not read again here
template <typename T, int V>
__device__ __forceinline__ void store_last(Vec<T, V>* p, const Vec<T, V>& x) {
  if constexpr (sizeof(x) == 16)
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&x));
  else
    *p = x;
}

// widest vector of fp32 with which a row of cols elements stays aligned
int vec_width(int64_t cols) {
  int v = 4;
  while (cols % v) v /= 2;
  return v;
}

// n / d and n % d by a multiplication, for n and d below 2^31: the quotient by floor(2^32 / d) is
// at most one short.
struct Divisor {
  unsigned d, m;
  explicit Divisor(unsigned d_) : d(d_), m((unsigned)(((uint64_t)1 << 32) / d_ - (d_ == 1))) {}
  __device__ __forceinline__ unsigned divide(unsigned n, unsigned& rest) const {
    unsigned q = __umulhi(n, m);
    rest = n - q * d;
    if (rest >= d) {
      rest -= d;
      ++q;
    }
    return q;
  }
};

// ---------------------------------------------------------------- forward
// The rows are one list of cols / V vectors each; a CTA takes kFwdUnroll * 256 consecutive
// vectors, so that a thread has kFwdUnroll independent loads in flight whatever the row length.
// y goes past the table rows in L2, of which the frequent ones are read again: 64K x 4096 in bf16
// 120 us, 123 without.
constexpr int kFwdUnroll = 4;
template <typename T, int V>
__global__ void __launch_bounds__(kThreads)
embed_scaled_fwd_kernel(int64_t rows, Divisor by_nv, int64_t vocab, float scale,
                        const int* __restrict__ ids, const T* __restrict__ table,
                        T* __restrict__ y) {
  const unsigned nv = by_nv.d;
  const int64_t first = (int64_t)blockIdx.x * (kFwdUnroll * kThreads);
  const int64_t r0 = first / nv;
  const unsigned o0 = (unsigned)(first - r0 * nv) + threadIdx.x;
  const Vec<T, V>* tv = reinterpret_cast<const Vec<T, V>*>(table);
  Vec<T, V>* yv = reinterpret_cast<Vec<T, V>*>(y);
  Vec<T, V> x[kFwdUnroll];
  bool ok[kFwdUnroll];
#pragma unroll
  for (int k = 0; k < kFwdUnroll; ++k) {
    unsigned c;
    const int64_t r = r0 + by_nv.divide(o0 + k * kThreads, c);
    const int64_t v = r < rows ? ids[r] : -1;
    ok[k] = v >= 0 && v < vocab;
    if (ok[k]) x[k] = tv[v * nv + c];
  }
#pragma unroll
  for (int k = 0; k < kFwdUnroll; ++k) {
    const int64_t i = first + threadIdx.x + k * kThreads;
    if (i >= rows * nv) break;
#pragma unroll
    for (int j = 0; j < V; ++j) st_f(x[k].v, j, ok[k] ? scale * ld_f(x[k].v, j) : 0.f);
    store_last(yv + i, x[k]);
  }
}

// Rows that are no whole number of 16-byte vectors: kLanes threads take a row, or four vectors each
// of it.  They write the vectors that are aligned in y; the elements of one lie in two aligned
// vectors of the table, `by` elements behind the first one's start, and `by` is the same for the
// whole row.  The elements before and behind y's vectors are moved one by one.  A warp's stores
// begin at a 128-byte line where they can (60180 x 3209 in bf16: 92 us, 97 without; with element-
// wise loads 147, with vectors of the whole list that shift by a variable 166: those two are bound
// by the instructions they issue).
template <typename T, int kBy>
__device__ __forceinline__ uint4 shifted(uint4 lo, uint4 hi) {
  const unsigned w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  constexpr int word = kBy * sizeof(T) / 4;
  if constexpr (kBy * sizeof(T) % 4 != 0)
    return make_uint4(__funnelshift_r(w[word], w[word + 1], 16),
                      __funnelshift_r(w[word + 1], w[word + 2], 16),
                      __funnelshift_r(w[word + 2], w[word + 3], 16),
                      __funnelshift_r(w[word + 3], w[word + 4], 16));
  else
    return make_uint4(w[word], w[word + 1], w[word + 2], w[word + 3]);
}

// f(integral_constant n), for n in [kFrom, kTo)
template <int kFrom, int kTo, typename F>
__device__ __forceinline__ void with_constant(int n, F&& f) {
  if constexpr (kFrom + 1 == kTo) {
    f(std::integral_constant<int, kFrom>());
  } else {
    if (n == kFrom)
      f(std::integral_constant<int, kFrom>());
    else
      with_constant<kFrom + 1, kTo>(n, f);
  }
}

template <typename T, int kLanes>
__global__ void __launch_bounds__(kThreads)
embed_scaled_fwd_odd_kernel(int64_t rows, int64_t cols, int64_t vocab, float scale, int lines,
                            const int* __restrict__ ids, const T* __restrict__ table,
                            T* __restrict__ y) {
  constexpr int kV = 16 / sizeof(T);
  const int64_t r = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
  if (r >= rows) return;
  const int lane = threadIdx.x % kLanes;
  const int64_t v = ids[r];
  const bool in = v >= 0 && v < vocab;
  // columns [0, head) and [tail, cols) one by one
  const int head = (int)imin(cols, -(r * cols) & (kV - 1));
  const int vectors = (int)(cols - head) / kV, tail = head + vectors * kV;
  // the first vector: with lines = 7 a warp's first one begins a line
  const int j0 = (int)blockIdx.y * (kLanes * kFwdUnroll) + lane -
                 (int)((r * cols + head) / kV & lines);
  const T* src = table + (in ? v * cols : 0);
  T* dst = y + r * cols;
  if (blockIdx.y == 0) {
    for (int i = lane; i < head + (int)cols - tail; i += kLanes) {
      const int c = i < head ? i : tail + i - head;
      st_f(dst, c, in ? scale * ld_f(src, c) : 0.f);
    }
  }
  Vec<T, kV>* out = reinterpret_cast<Vec<T, kV>*>(dst + head);
  if (!in) {
    const Vec<T, kV> zero = {};
#pragma unroll
    for (int k = 0; k < kFwdUnroll; ++k) {
      const int j = j0 + kLanes * k;
      if (j >= 0 && j < vectors) store_last(out + j, zero);
    }
    return;
  }
  const int by = (int)((v * cols + head) & (kV - 1));
  const uint4* t = reinterpret_cast<const uint4*>(src + head - by);
  // the last vector of the table's last row may have its second half behind the table's end
  const bool ends = by != 0 && v * cols + head - by + (int64_t)(vectors + 1) * kV > vocab * cols;
  uint4 lo[kFwdUnroll], hi[kFwdUnroll];
#pragma unroll
  for (int k = 0; k < kFwdUnroll; ++k) {
    const int j = j0 + kLanes * k;
    lo[k] = hi[k] = make_uint4(0, 0, 0, 0);
    if (j < 0 || j >= vectors) continue;
    lo[k] = t[j];
    if (ends && j == vectors - 1) {
      T* h = reinterpret_cast<T*>(&hi[k]);
      for (int e = 0; e < by; ++e) h[e] = src[tail - by + e];
    } else if (by != 0) {
      hi[k] = t[j + 1];
    }
  }
  with_constant<0, kV>(by, [&](auto n) {
#pragma unroll
    for (int k = 0; k < kFwdUnroll; ++k) {
      const int j = j0 + kLanes * k;
      if (j < 0 || j >= vectors) continue;
      Vec<T, kV> x;
      *reinterpret_cast<uint4*>(&x) = shifted<T, decltype(n)::value>(lo[k], hi[k]);
#pragma unroll
      for (int i = 0; i < kV; ++i) st_f(x.v, i, scale * ld_f(x.v, i));
      store_last(out + j, x);
    }
  });
}

// ---------------------------------------------------------------- sort by id
// What the accumulation reads of a sorted position: its row, and its run (the positions with the
// same id): where it starts and how long it is, and the id.
//   sorted[p] = {row, start, length, id},  p in [0, *n_valid); rows of ids outside [0, vocab)
// are left out.

// Up to 4096 rows: the sorted position of every row by counting.  A run starts at the number of
// rows with a smaller id, and a row stands behind the earlier rows of its own id.  Sixteen
// threads share a row; the ids pass through shared memory, four at a time.  Rows before and
// behind the CTA's own are counted apart, so two comparisons per id give all three numbers.
// rows^2 comparisons: 4096 rows take 7 us, 6857 rows 16, more than the digit sort below.
constexpr int kRankRows = 4096;
constexpr int kRankShare = 16, kRankPerCta = kThreads / kRankShare;
static_assert(kRankPerCta == kRankShare, "each of a row's threads takes one of the CTA's rows");
__global__ void __launch_bounds__(kThreads)
embed_rank_kernel(int rows, int vocab, const int* __restrict__ ids, int4* __restrict__ sorted,
                  int* __restrict__ n_valid, int* __restrict__ n_long) {
  release_next();
  __shared__ __align__(16) int key[kRankRows];
  const int rows4 = (rows + 3) / 4, padded = (rows + 15) / 16 * 16;
  int4* keys = reinterpret_cast<int4*>(key);
  auto key_of = [&](int v) { return v < 0 || v >= vocab ? vocab : v; };
  constexpr int kLoads = kRankRows / 4 / kThreads;
  int4 v[kLoads];
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int i = threadIdx.x + k * kThreads;
    if (i < rows / 4) v[k] = reinterpret_cast<const int4*>(ids)[i];
  }
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int i = threadIdx.x + k * kThreads;
    if (i < rows / 4)
      keys[i] = make_int4(key_of(v[k].x), key_of(v[k].y), key_of(v[k].z), key_of(v[k].w));
  }
  for (int i = rows / 4 * 4 + threadIdx.x; i < padded; i += kThreads)
    key[i] = i < rows ? key_of(ids[i]) : vocab;
  __syncthreads();
  const int r0 = blockIdx.x * kRankPerCta, own = threadIdx.x / kRankShare;
  const int part = threadIdx.x % kRankShare;
  const int mine = key[r0 + own];
  const int4* key4 = reinterpret_cast<const int4*>(key);
  auto count = [&](int i, int& less, int& upto) {
    const int4 k = key4[i];
    less += (k.x < mine) + (k.y < mine) + (k.z < mine) + (k.w < mine);
    upto += (k.x <= mine) + (k.y <= mine) + (k.z <= mine) + (k.w <= mine);
  };
  int less = 0, upto = 0, rank = 0;
  const int b = r0 / 4, e = b + kRankPerCta / 4;    // the CTA's own rows, in fours
#pragma unroll 4
  for (int i = part; i < b; i += kRankShare) count(i, less, upto);
  rank = upto - less;
#pragma unroll 4
  for (int i = e + part; i < rows4; i += kRankShare) count(i, less, upto);
  const int k = key[r0 + part];
  less += k < mine;
  upto += k <= mine;
  rank += k == mine && part < own;
#pragma unroll
  for (int o = 1; o < kRankShare; o <<= 1) {
    less += __shfl_xor_sync(0xffffffffu, less, o);
    upto += __shfl_xor_sync(0xffffffffu, upto, o);
    rank += __shfl_xor_sync(0xffffffffu, rank, o);
  }
  if (part == 0 && mine < vocab)
    sorted[less + rank] = make_int4(r0 + own, less, upto - less, mine);
  if (blockIdx.x == 0) {
    __shared__ int red[kThreads / 32];
    int n = 0;
    for (int i = threadIdx.x; i < rows; i += kThreads) n += key[i] < vocab;
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = n;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < kThreads / 32; ++w) n += red[w];
      *n_valid = n;
      n_long[0] = n_long[1] = 0;
    }
  }
}

// Many rows: the rows are dealt to kBuckets buckets by the low digit of their id, then each
// bucket is sorted by the rest of the id by one CTA (neighbouring ids, of which a vocabulary
// numbered by frequency has its most frequent at the low end, fall into different buckets).
// Both steps are counting sorts that keep the rows' order: every warp takes a contiguous piece,
// counts its keys in a histogram of its own, and after a scan over (key, warp) places them; inside
// a warp equal keys are ranked by lane.  (Atomics only count: integers, in shared memory.)
constexpr int kBuckets = 512, kDealThreads = 512, kDealWarps = kDealThreads / 32;
// Rows of a block: few, as its steps over them follow one another, but each block reads the others'
// counts (16000 rows: 17.8 us for the gradient of 64 columns with 512, 18.2 with 1024, 21.3 with
// 2048; 32000: 27.6, 24.7, 25.9)
constexpr int64_t kDealRows = 512, kDealManyRows = 1024, kDealMany = 16384, kDealMaxBlocks = 128;
constexpr int64_t kWideRows = 32768;      // above: buckets' CTAs of twice the threads

__device__ __forceinline__ bool valid_id(int v, int vocab) { return v >= 0 && v < vocab; }

// counts[block][bucket]
__global__ void __launch_bounds__(kDealThreads)
embed_count_kernel(int rows, int per_block, int vocab, const int* __restrict__ ids,
                   int* __restrict__ counts, int* __restrict__ n_long) {
  __shared__ int hist[kBuckets];
  release_next();
  if (blockIdx.x == 0 && threadIdx.x < 2) n_long[threadIdx.x] = 0;
  hist[threadIdx.x] = 0;
  __syncthreads();
  const int r0 = blockIdx.x * per_block, r1 = min(rows, r0 + per_block);
  for (int r = r0 + threadIdx.x; r < r1; r += kDealThreads) {
    const int v = ids[r];
    if (valid_id(v, vocab)) atomicAdd(&hist[v % kBuckets], 1);
  }
  __syncthreads();
  counts[blockIdx.x * kBuckets + threadIdx.x] = hist[threadIdx.x];
}

// exclusive scan of one value per thread over the block (any multiple of 32 threads)
__device__ __forceinline__ int block_exclusive_scan(int v, int* red) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();
  if (lane == 31) red[wid] = s;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < wid; ++w) base += red[w];
  return base + s - v;
}

// dealt[...] = {id, row} by bucket, rows in order; base[b] = start of bucket b, base[kBuckets] =
// number of valid rows
__global__ void __launch_bounds__(kDealThreads)
embed_deal_kernel(int rows, int per_block, int vocab, const int* __restrict__ ids,
                  const int* counts, int2* __restrict__ dealt, int* __restrict__ base) {
  __shared__ int hist[kDealWarps][kBuckets];
  __shared__ int red[kDealWarps];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int b = threadIdx.x;                      // one bucket per thread in the scans
  const int per_warp = per_block / kDealWarps;    // per_block is a multiple of 512
  const int r0 = blockIdx.x * per_block + wid * per_warp;
  // the first 64 ids of the warp's piece (all of them up to 131072 rows), read at once
  constexpr int kHeld = (int)kDealManyRows / kDealThreads;
  int held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int o = 32 * i;
    held[i] = o < per_warp && r0 + o + lane < rows ? ids[r0 + o + lane] : -1;
  }
#pragma unroll
  for (int w = 0; w < kDealWarps; ++w) hist[w][b] = 0;
  release_next();
  await_previous();
  int total = 0, before = 0;
  auto add = [&](int k, int c) {
    total += c;
    if (k < (int)blockIdx.x) before += c;
  };
  int k = 0;
  for (; k + 16 <= (int)gridDim.x; k += 16) {      // sixteen loads in flight
    int c[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) c[i] = counts[(k + i) * kBuckets + b];
#pragma unroll
    for (int i = 0; i < 16; ++i) add(k + i, c[i]);
  }
  if (k < (int)gridDim.x) {                        // the rest too: 48000 rows 28.2 us, 30.1
    int c[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
      c[i] = k + i < (int)gridDim.x ? counts[(k + i) * kBuckets + b] : 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) add(k + i, c[i]);
  }
  const int start = block_exclusive_scan(total, red);
  if (blockIdx.x == 0) {
    base[b] = start;
    if (b == kBuckets - 1) base[kBuckets] = start + total;
  }
  __syncthreads();
  auto tally = [&](int v) {
    if (valid_id(v, vocab)) atomicAdd(&hist[wid][v % kBuckets], 1);
  };
  auto place = [&](int v, int r) {
    const int key = valid_id(v, vocab) ? v % kBuckets : kBuckets;
    const unsigned same = __match_any_sync(0xffffffffu, key);
    const int rank = __popc(same & ((1u << lane) - 1));
    int pos = 0;
    if (key < kBuckets) pos = hist[wid][key] + rank;
    __syncwarp();
    if (key < kBuckets) {
      if (rank == 0) hist[wid][key] = pos + __popc(same);
      dealt[pos] = make_int2(v, r);
    }
    __syncwarp();
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) tally(held[i]);
  for (int i = 32 * kHeld; i < per_warp; i += 32)
    tally(r0 + i + lane < rows ? ids[r0 + i + lane] : -1);
  __syncthreads();
  int at = start + before;
#pragma unroll
  for (int w = 0; w < kDealWarps; ++w) {
    const int c = hist[w][b];
    hist[w][b] = at;
    at += c;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kHeld; ++i) place(held[i], r0 + 32 * i + lane);
  for (int i = 32 * kHeld; i < per_warp; i += 32)
    place(r0 + i + lane < rows ? ids[r0 + i + lane] : -1, r0 + i + lane);
}

// One CTA per bucket: a counting sort by bin = id / kBuckets with `warps` histograms.  Shared
// memory: hist[warps][bins], start[bins], len[bins].  present[v] (where it is wanted) tells
// whether id v occurs.
__global__ void __launch_bounds__(2 * kThreads)
embed_bucket_kernel(int vocab, int bins, int warps, const int* base, const int2* dealt,
                    int4* __restrict__ sorted, unsigned char* __restrict__ present) {
  extern __shared__ int sm[];
  __shared__ int red[2 * kThreads / 32];
  int* start = sm + warps * bins;
  int* len = start + bins;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < warps * bins; i += blockDim.x) sm[i] = 0;
  release_next();
  await_previous();
  const int b0 = base[blockIdx.x], n = base[blockIdx.x + 1] - b0;
  __syncthreads();
  const int per_warp = (n + warps * 32 - 1) / (warps * 32) * 32;
  const int i0 = b0 + wid * per_warp, i1 = min(b0 + n, i0 + per_warp);
  int* hist = sm + wid * bins;
  if (wid < warps) {
    for (int i = i0; i < i1; i += 32) {
      if (i + lane < i1) atomicAdd(&hist[dealt[i + lane].x / kBuckets], 1);
    }
  }
  __syncthreads();
  const int per = (bins + (int)blockDim.x - 1) / (int)blockDim.x;
  const int k0 = min(bins, (int)threadIdx.x * per), k1 = min(bins, k0 + per);
  int mine = 0;
  for (int k = k0; k < k1; ++k) {
    int c = 0;
    for (int w = 0; w < warps; ++w) c += sm[w * bins + k];
    len[k] = c;
    mine += c;
  }
  int at = b0 + block_exclusive_scan(mine, red);
  for (int k = k0; k < k1; ++k) {
    start[k] = at;
    for (int w = 0; w < warps; ++w) {
      const int c = sm[w * bins + k];
      sm[w * bins + k] = at;
      at += c;
    }
    const int v = k * kBuckets + blockIdx.x;
    if (present && v < vocab) present[v] = len[k] > 0;
  }
  __syncthreads();
  if (wid < warps) {
    for (int i = i0; i < i1; i += 32) {
      const int2 d = i + lane < i1 ? dealt[i + lane] : make_int2(0, 0);
      const int key = i + lane < i1 ? d.x / kBuckets : bins;
      const unsigned same = __match_any_sync(0xffffffffu, key);
      const int rank = __popc(same & ((1u << lane) - 1));
      int pos = 0;
      if (key < bins) pos = hist[key] + rank;
      __syncwarp();
      if (key < bins) {
        if (rank == 0) hist[key] = pos + __popc(same);
        sorted[pos] = make_int4(d.y, start[key], len[key], d.x);
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------- accumulate
// A run is cut into units of `unit` rows counted from its start.  A group of `group` threads
// takes `window` consecutive sorted positions and adds every unit that begins there, all of its
// rows in order, four columns per thread (as 4 / V vectors a group apart).  The unit of a run of
// one unit goes into the table; those of longer runs go to partial rows, which embed_join_kernel
// adds in order (the runs' starts are left in two lists for it, in no particular order: the few
// of more than kLongUnits units from the back).  Of the units that go to partial rows at most two
// begin within `unit` positions: one that continues a run and one that begins the next (a run
// longer than a unit leaves room for no third), which gives the slot
// 2 (p / unit) + (p is its run's start).
constexpr int kMaxUnit = 64, kMinUnit = 8, kLongUnits = 8;

template <int V>
__device__ __forceinline__ void vload(const float* p, float (&x)[V]) {
  const Vec<float, V> t = *reinterpret_cast<const Vec<float, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = t.v[i];
}
template <int V>
__device__ __forceinline__ void vstore(float* p, const float (&x)[V]) {
  Vec<float, V> t;
#pragma unroll
  for (int i = 0; i < V; ++i) t.v[i] = x[i];
  *reinterpret_cast<Vec<float, V>*>(p) = t;
}

struct AccumArgs {
  int64_t cols;
  int rows, vocab;
  float scale;
  int accumulate, group, window, unit, clear_rows;
  int64_t acc_blocks;      // CTAs that accumulate; the ones behind them clear absent rows
  const int4* sorted;
  const int* n_valid;
  const int* ids;          // the ids where they are few, else null:
  const unsigned char* present;
  const float* dy;
  float *d_table, *partial;
  int *n_long, *longs, max_longs;     // n_long[0], n_long[1]: entries of the two lists
};

// The CTAs behind the accumulating ones clear the table rows whose id does not occur, in pieces
// dealt in turn: by the flags of the sort, or by marking the few ids in shared memory (four loads
// of four ids in flight: 4000 rows, 100000 x 1024: 77 us, 88 with one id at a time).  Many short
// CTAs write faster than few long ones (2.2 GB: 8 per SM 428 us, 64 per SM 393).
constexpr int kClearRows = 512, kClearPerSm = 64;

// kLanes threads per row: its vectors are written side by side
template <int V, int kLanes>
__device__ __forceinline__ void clear_rows(float* d, int64_t cols, int n,
                                           const unsigned char* here) {
  const int64_t nv = cols / V;
  const float zero[V] = {};
  for (int i = threadIdx.x / kLanes; i < n; i += blockDim.x / kLanes) {
    if (here[i]) continue;
    for (int64_t c = threadIdx.x % kLanes; c < nv; c += kLanes)
      vstore<V>(d + i * cols + c * V, zero);
  }
}

template <int V>
__device__ void clear_absent(const AccumArgs& a, int64_t b, int64_t nb) {
  __shared__ unsigned char here[kClearRows];
  const int piece = a.clear_rows;
  for (int64_t v0 = b * piece; v0 < a.vocab; v0 += nb * piece) {
    const int n = (int)imin(piece, a.vocab - v0);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) here[i] = a.ids ? 0 : a.present[v0 + i];
    __syncthreads();
    if (a.ids) {
      auto mark = [&](int id) {
        const int64_t v = id - v0;
        if (v >= 0 && v < n) here[v] = 1;
      };
      const int4* ids4 = reinterpret_cast<const int4*>(a.ids);
      const int rows4 = a.rows / 4;
#pragma unroll 4
      for (int i = threadIdx.x; i < rows4; i += blockDim.x) {
        const int4 q = ids4[i];
        mark(q.x);
        mark(q.y);
        mark(q.z);
        mark(q.w);
      }
      if ((int)threadIdx.x < a.rows % 4) mark(a.ids[4 * rows4 + threadIdx.x]);
      __syncthreads();
    }
    // rows of up to 16 vectors by part of a warp (100000 x 64: 6.7 us, 9.5 by a warp per row)
    float* d = a.d_table + v0 * a.cols;
    if (a.cols / V > 16)
      clear_rows<V, 32>(d, a.cols, n, here);
    else if (a.cols / V > 8)
      clear_rows<V, 16>(d, a.cols, n, here);
    else
      clear_rows<V, 8>(d, a.cols, n, here);
  }
}

// d_table row v (+)= scale * sum
template <int V>
__device__ __forceinline__ void put_row(const AccumArgs& a, int v, int64_t c, float (&sum)[V]) {
  float* d = a.d_table + (int64_t)v * a.cols + c;
  if (a.accumulate) {
    float old[V];
    vload<V>(d, old);
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = fmaf(a.scale, sum[j], old[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] *= a.scale;
  }
  vstore<V>(d, sum);
}

template <int V>
__global__ void __launch_bounds__(kThreads)
embed_accum_kernel(AccumArgs a) {
  if ((int64_t)blockIdx.x >= a.acc_blocks) {
    if (!a.ids) await_previous();       // by the ids, the clearing need not wait for the sort
    if (blockIdx.y == 0) clear_absent<V>(a, blockIdx.x - a.acc_blocks, gridDim.x - a.acc_blocks);
    return;
  }
  // the thread's columns: kV vectors, a group apart
  constexpr int kV = 4 / V;
  const int64_t c = ((int64_t)blockIdx.y * kV * a.group + threadIdx.x % a.group) * V;
  const int64_t apart = (int64_t)a.group * V;
  const int g = threadIdx.x / a.group, groups = blockDim.x / a.group;
  // the sorted positions that the CTA's groups read, at once: their loads would otherwise stand
  // before those of the rows in every turn (64K of 4096: 492 us, 502)
  extern __shared__ int4 staged[];
  const int64_t first = (int64_t)blockIdx.x * groups * a.window;
  const int4* sorted = staged - first;
  await_previous();
  const int n = *a.n_valid;
  for (int i = threadIdx.x; i < groups * a.window + a.unit; i += blockDim.x)
    staged[i] = a.sorted[imin(first + i, a.rows - 1)];
  __syncthreads();
  const int64_t p0 = first + (int64_t)g * a.window;
  const int p1 = (int)imin(n, p0 + a.window);
  if (c >= a.cols || p0 >= p1) return;
  // positions [b, e): the units that begin in the window, the last of them to its end
  const int4 s0 = sorted[p0], s1 = sorted[p1 - 1];
  const int into = ((int)p0 - s0.y) & (a.unit - 1);
  const int b = into ? min((int)p0 + a.unit - into, s0.y + s0.z) : (int)p0;
  if (b >= p1) return;
  const int last = p1 - 1 - ((p1 - 1 - s1.y) & (a.unit - 1));
  const int e = min(last + a.unit, s1.y + s1.z);
  float sum[kV][V];
  int4 run = sorted[b];       // of the unit in hand, and where the unit begins
  int from = b;
  auto flush = [&]() {
    const bool whole = run.z <= a.unit;
    float* part = a.partial + (2 * (int64_t)(from / a.unit) + (from == run.y)) * a.cols;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      if (c + v * apart >= a.cols) break;
      if (whole)
        put_row<V>(a, run.w, c + v * apart, sum[v]);
      else
        vstore<V>(part + c + v * apart, sum[v]);
    }
    if (!whole && from == run.y && c == 0) {
      if (run.z <= a.unit * kLongUnits)
        a.longs[atomicAdd(a.n_long, 1)] = from;
      else
        a.longs[a.max_longs - 1 - atomicAdd(a.n_long + 1, 1)] = from;
    }
  };
  // four rows in flight, whatever units they belong to
  constexpr int kRows = 4;
  for (int p = b; p < e; p += kRows) {
    int4 s[kRows];
    float x[kRows][kV][V] = {};
#pragma unroll
    for (int k = 0; k < kRows; ++k) s[k] = sorted[min(p + k, e - 1)];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const float* row = a.dy + (int64_t)s[k].x * a.cols + c;
#pragma unroll
      for (int v = 0; v < kV; ++v)
        if (c + v * apart < a.cols) vload<V>(row + v * apart, x[k][v]);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (p + k >= e) break;
      const bool begins = ((p + k - s[k].y) & (a.unit - 1)) == 0;
      if (begins) {
        if (p + k > b) flush();
        run = s[k];
        from = p + k;
      }
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int j = 0; j < V; ++j) sum[v][j] = begins ? x[k][v][j] : sum[v][j] + x[k][v][j];
    }
  }
  flush();
}

// At most kFewRows rows: no sort.  A warp takes (row, 32 V columns); it marks the rows of the
// same id by ballots over all ids and, where its own row is the first of them, adds them in
// order.  One launch, where the sorted form takes three.
constexpr int kFewRows = 256;
template <int V>
__global__ void __launch_bounds__(kThreads)
embed_few_kernel(AccumArgs a, int slabs) {
  if ((int64_t)blockIdx.x >= a.acc_blocks) {
    clear_absent<V>(a, blockIdx.x - a.acc_blocks, gridDim.x - a.acc_blocks);
    return;
  }
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t r = item / slabs, c = ((item - r * slabs) * 32 + lane) * V;
  if (r >= a.rows) return;
  const int mine = a.ids[r];
  if (!valid_id(mine, a.vocab)) return;
  unsigned same[kFewRows / 32];
#pragma unroll
  for (int q = 0; q < kFewRows / 32; ++q) {
    const int i = q * 32 + lane;
    same[q] = __ballot_sync(0xffffffffu, i < a.rows && a.ids[i] == mine);
    // an earlier row has this id: that row's warp adds it
    if (q * 32 < r && (same[q] & (r >= q * 32 + 32 ? ~0u : (1u << (r & 31)) - 1))) return;
  }
  if (c >= a.cols) return;
  float sum[V] = {};
#pragma unroll
  for (int q = 0; q < kFewRows / 32; ++q) {
    const float* dy = a.dy + q * 32 * a.cols + c;
    unsigned m = same[q];
    while (m) {
      float x[4][V] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (m) vload<V>(dy + (int64_t)(__ffs(m) - 1) * a.cols, x[k]);
        m &= m - 1;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += x[k][j];
    }
  }
  put_row<V>(a, mine, c, sum);
}

// Runs longer than a unit, by the lists: a warp takes (run, 32 V columns) and adds the run's
// partial rows in order, V columns per lane.  Of runs of more than kLongUnits units a whole CTA
// takes it: each warp adds an eighth of the units, warp 0 the eight sums.
template <int V>
__global__ void __launch_bounds__(kThreads)
embed_join_kernel(AccumArgs a) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float sums[kWarps][32 * V];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int slabs = (int)((a.cols + 32 * V - 1) / (32 * V));
  // units [u0, u1) of the run that starts at `start`, eight of them in flight
  auto add = [&](int start, int u0, int u1, int64_t c, float (&sum)[V]) {
    const float* first = a.partial + 2 * (int64_t)(start / a.unit) * a.cols + c;
    for (int u = u0; u < u1; u += 8) {
      float x[8][V] = {};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (u + k < u1) vload<V>(first + (2 * (int64_t)(u + k) + (u + k == 0)) * a.cols, x[k]);
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += x[k][j];
    }
  };
  const int64_t items = (int64_t)a.n_long[0] * slabs, heavy = (int64_t)a.n_long[1] * slabs;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + wid; i < items;
       i += (int64_t)gridDim.x * kWarps) {
    const int64_t run = i / slabs, c = ((i - run * slabs) * 32 + lane) * V;
    const int4 s = a.sorted[a.longs[run]];
    if (c >= a.cols) continue;
    float sum[V] = {};
    add(s.y, 0, (s.z + a.unit - 1) / a.unit, c, sum);
    put_row<V>(a, s.w, c, sum);
  }
  for (int64_t i = blockIdx.x; i < heavy; i += gridDim.x) {
    const int64_t run = i / slabs, c = ((i - run * slabs) * 32 + lane) * V;
    const int4 s = a.sorted[a.longs[a.max_longs - 1 - run]];
    const int units = (s.z + a.unit - 1) / a.unit, per = (units + kWarps - 1) / kWarps;
    float sum[V] = {};
    if (c < a.cols) add(s.y, min(units, wid * per), min(units, wid * per + per), c, sum);
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) sums[wid][lane * V + j] = sum[j];
    __syncthreads();
    if (wid == 0 && c < a.cols) {
      for (int w = 1; w < kWarps; ++w)
#pragma unroll
        for (int j = 0; j < V; ++j) sum[j] += sums[w][lane * V + j];
      put_row<V>(a, s.w, c, sum);
    }
  }
}

// ---------------------------------------------------------------- workspace
struct Plan {
  int* head;                // number of valid rows, or the buckets' starts with it behind them,
                            // and the entries of the lists of long runs
  int4* sorted;
  unsigned char* present;
  int2* dealt;
  int* counts;
  float* partial;
  int* longs;
  int64_t max_longs;
  size_t bytes;
};

// slabs of columns that the groups of the accumulation take, 4 columns a thread
int64_t slabs_of(int64_t cols) { return nblk(cols, 4 * kThreads); }

// Rows of a unit: long units write few partial rows, short ones leave few sums in a row for a
// group to wait for; a power of two that gives every SM eight groups' worth of full units
// (overwritten tables, Zipf ids, in all: 65536 rows of 4096 into 128256: 64, 485 us, 492 with 32,
// 528 with 8; 48890 of 440 into 32000: 64, 47.9, 51.0 with 8; 600 of 64 into 512: 8, 8.0, 9.7 with
// 32.  In between half the unit is up to 6 % faster: 11132 of 1112 into 30000: 32, 49.8, 46.7 with
// 16).
int unit_rows(int64_t rows, int64_t cols) {
  const int64_t slabs = slabs_of(cols);
  int unit = kMinUnit;
  while (unit < kMaxUnit && rows * slabs >= (int64_t)sm_count() * 8 * unit) unit *= 2;
  return unit;
}

int64_t deal_rows(int64_t rows) {     // rows of a block of the deal, a multiple of 512
  const int64_t r = nblk(nblk(rows, kDealMaxBlocks), kDealThreads) * kDealThreads;
  return imax(rows > kDealMany ? kDealManyRows : kDealRows, r);
}

Plan plan(void* ws, int64_t rows, int64_t cols, int64_t vocab) {
  Plan p;
  size_t off = 0;
  auto take = [&](size_t n) {
    void* q = ws ? static_cast<char*>(ws) + off : nullptr;
    off += (n + 255) & ~size_t(255);
    return q;
  };
  p.head = static_cast<int*>(take(sizeof(int) * (kBuckets + 3)));
  p.sorted = static_cast<int4*>(take(sizeof(int4) * rows));
  const bool deal = rows > kRankRows;
  p.present = static_cast<unsigned char*>(take(deal ? vocab : 0));
  p.dealt = static_cast<int2*>(take(deal ? sizeof(int2) * rows : 0));
  p.counts =
      static_cast<int*>(take(deal ? sizeof(int) * kBuckets * nblk(rows, deal_rows(rows)) : 0));
  const int64_t units = rows > kFewRows ? nblk(rows, unit_rows(rows, cols)) : 0;
  p.partial = static_cast<float*>(take(sizeof(float) * 2 * units * cols));
  p.longs = static_cast<int*>(take(sizeof(int) * units));
  p.max_longs = units;
  p.bytes = off;
  return p;
}

template <typename T, int V>
cudaError_t fwd(int64_t rows, int64_t cols, int64_t vocab, float scale, const int* ids,
                const void* table, void* y, cudaStream_t st) {
  const int64_t nv = cols / V;
  launch(embed_scaled_fwd_kernel<T, V>, dim3((unsigned)nblk(rows * nv, kFwdUnroll * kThreads)),
         dim3(kThreads), 0, st, rows, Divisor((unsigned)nv), vocab, scale, ids,
         static_cast<const T*>(table), static_cast<T*>(y));
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd_odd(int64_t rows, int64_t cols, int64_t vocab, float scale, const int* ids,
                    const void* table, void* y, cudaStream_t st) {
  const int64_t vectors = cols * (int64_t)sizeof(T) / 16;
  auto go = [&](auto kernel, int lanes) {
    const int64_t take = lanes * kFwdUnroll, parts = imax(1, nblk(vectors, take));
    // from lines on where that needs no further part of the row
    const int lines = lanes == 32 && vectors + 7 <= parts * take ? 7 : 0;
    launch(kernel, dim3((unsigned)nblk(rows, kThreads / lanes), (unsigned)parts), dim3(kThreads),
           0, st, rows, cols, vocab, scale, lines, ids, static_cast<const T*>(table),
           static_cast<T*>(y));
  };
  // short rows by a quarter of a warp (60180 x 65: 6.7 us, 13.4 by a warp)
  if (vectors <= 64)
    go(embed_scaled_fwd_odd_kernel<T, 8>, 8);
  else
    go(embed_scaled_fwd_odd_kernel<T, 32>, 32);
  return cudaGetLastError();
}

// CTAs that clear absent rows.  A piece holds 64 KB, so that its marking costs little beside it
// (32 KB where the ids are few), but no more rows than leave every SM two pieces (256 rows into
// 8000 x 64: 3.3 us, 6.7 with 64 KB).
int64_t clear_blocks(AccumArgs& a) {
  const bool few = a.rows <= kFewRows;
  const int64_t most = imin((few ? 8192 : 16384) / a.cols, a.vocab / (sm_count() * 2));
  a.clear_rows = (int)imax(few ? 8 : 16, imin(kClearRows, most));
  return a.accumulate ? 0 : imin(nblk(a.vocab, a.clear_rows), (int64_t)sm_count() * kClearPerSm);
}

template <int V>
cudaError_t accum_few(AccumArgs a, cudaStream_t st) {
  const int64_t slabs = nblk(a.cols, 32 * V);
  a.acc_blocks = nblk(a.rows * slabs, kThreads / 32);
  const int64_t clear = clear_blocks(a);
  launch(embed_few_kernel<V>, dim3((unsigned)(a.acc_blocks + clear)), dim3(kThreads), 0, st, a,
         (int)slabs);
  return cudaGetLastError();
}

template <int V>
cudaError_t accum(AccumArgs a, cudaStream_t st) {
  // the columns in equal slabs of at most 1024; a group of whole warps takes one (of 8 or 16
  // threads where a slab is shorter than a warp), a CTA as many groups as 256 threads hold
  const int64_t slabs = slabs_of(a.cols);
  const int64_t threads = nblk(nblk(a.cols, slabs), 4);
  a.group = threads <= 8 ? 8 : threads <= 16 ? 16 : (int)nblk(threads, 32) * 32;
  const int groups = kThreads / a.group;
  // positions per group: four at least, which are in flight together (4058 rows of 280: 13.4 us
  // in all, 15.6 with one), and as many as leave every SM twelve CTAs' worth of groups
  const int64_t fill = (int64_t)sm_count() * 12 * groups;
  a.window = (int)imax(4, imin(64, a.rows * slabs / fill));
  a.acc_blocks = nblk(nblk(a.rows, a.window), groups);
  const int64_t clear = clear_blocks(a);
  a.unit = unit_rows(a.rows, a.cols);
  launch_next(embed_accum_kernel<V>, dim3((unsigned)(a.acc_blocks + clear), (unsigned)slabs),
              dim3(a.group * groups), sizeof(int4) * (groups * a.window + a.unit), st, a);
  // not set up early: its CTAs would hold the places of accumulating ones (11132 rows of 1112:
  // 33.9 us in all, 37.5 with them; 64K of 4096: 501, 502)
  // two columns a lane: twice the parts of a frequent id's run, and eight loads of it in flight
  // (48890 rows of 440: 49.2 us in all, 55.0 with four; rare ids, 12043 rows of 2568: 51.4, 49.8)
  launch(embed_join_kernel<V < 2 ? V : 2>, dim3(sm_count() * 4), dim3(kThreads), 0, st, a);
  return cudaGetLastError();
}

// sorted, n_valid, and what tells the absent ids
cudaError_t sort_by_id(int64_t rows, int64_t vocab, const int* ids, const Plan& p, AccumArgs& a,
                       cudaStream_t st) {
  a.sorted = p.sorted;
  a.n_valid = p.head;
  if (rows <= kRankRows) {
    launch(embed_rank_kernel, dim3((unsigned)nblk(rows, kRankPerCta)), dim3(kThreads), 0, st,
           (int)rows, (int)vocab, ids, p.sorted, p.head, a.n_long);
    return cudaGetLastError();
  }
  const int bins = (int)((vocab - 1) / kBuckets + 1);
  // 512 threads where a frequent id may fill a bucket with thousands of rows (64K rows: 502 us in
  // all, 505 with 256; 8570 rows: 26.5, 25.9)
  const int threads = rows > kWideRows ? 2 * kThreads : kThreads;
  int warps = threads / 32;      // as many histograms as 96 KB hold
  while (warps > 1 && (size_t)bins * (warps + 2) * 4 > 96 * 1024) warps /= 2;
  const size_t smem = sizeof(int) * (size_t)bins * (warps + 2);
  // asked for below 48 KB already, which have to hold the kernel's static arrays too; before the
  // first launch, as it may fail
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        embed_bucket_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 1024);
    if (e != cudaSuccess) return e;
  }
  const int per_block = (int)deal_rows(rows);
  const dim3 grid((unsigned)nblk(rows, per_block));
  int* base = p.head;
  launch(embed_count_kernel, grid, dim3(kDealThreads), 0, st, (int)rows, per_block, (int)vocab,
         ids, p.counts, a.n_long);
  launch_next(embed_deal_kernel, grid, dim3(kDealThreads), 0, st, (int)rows, per_block,
              (int)vocab, ids, (const int*)p.counts, p.dealt, base);
  launch_next(embed_bucket_kernel, dim3(kBuckets), dim3(threads), smem, st, (int)vocab, bins,
              warps, (const int*)base, (const int2*)p.dealt, p.sorted,
              a.accumulate ? static_cast<unsigned char*>(nullptr) : p.present);
  a.n_valid = base + kBuckets;
  a.ids = nullptr;
  a.present = p.present;
  return cudaGetLastError();
}

}  // namespace

cudaError_t embed_scaled_fwd(int64_t rows, int64_t cols, int64_t vocab, int dt, float scale,
                             const int* ids, const void* table, void* y, cudaStream_t st) {
  using bf16 = __nv_bfloat16;
  if (dt == DT_BF16)
    return cols % 8 == 0 ? fwd<bf16, 8>(rows, cols, vocab, scale, ids, table, y, st)
                         : fwd_odd<bf16>(rows, cols, vocab, scale, ids, table, y, st);
  return cols % 4 == 0 ? fwd<float, 4>(rows, cols, vocab, scale, ids, table, y, st)
                       : fwd_odd<float>(rows, cols, vocab, scale, ids, table, y, st);
}

size_t embed_scaled_bwd_ws_bytes(int64_t rows, int64_t cols, int64_t vocab) {
  return plan(nullptr, rows, cols, vocab).bytes;
}

cudaError_t embed_scaled_bwd(int64_t rows, int64_t cols, int64_t vocab, float scale,
                             const int* ids, const float* dy, float* d_table, int accumulate,
                             void* ws, cudaStream_t st) {
  const Plan p = plan(ws, rows, cols, vocab);
  AccumArgs a = {};
  a.cols = cols;
  a.rows = (int)rows;
  a.vocab = (int)vocab;
  a.scale = scale;
  a.accumulate = accumulate;
  a.ids = ids;
  a.dy = dy;
  a.d_table = d_table;
  a.partial = p.partial;
  a.n_long = p.head + kBuckets + 1;
  a.longs = p.longs;
  a.max_longs = (int)p.max_longs;
  const int v = vec_width(cols);
  if (rows <= kFewRows)
    return v == 4 ? accum_few<4>(a, st) : v == 2 ? accum_few<2>(a, st) : accum_few<1>(a, st);
  const cudaError_t e = sort_by_id(rows, vocab, ids, p, a, st);
  if (e != cudaSuccess) return e;
  return v == 4 ? accum<4>(a, st) : v == 2 ? accum<2>(a, st) : accum<1>(a, st);
}

}  // namespace sbp
