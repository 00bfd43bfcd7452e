// Global gradient norm over many tensors, and clipping.
//
//   sqsum = sum over tensors and elements of g^2,  norm = sqrt(sqsum)
//   out = g * min(1, max_norm / (norm + 1e-6))
//
// Products and sums are formed in 64 bits: the square of an fp32 value neither overflows nor
// vanishes there.  Both passes are bound by HBM (4 bytes read per element, then 8 moved where
// the clipping bites).  The tensors' pointers travel as kernel parameters, so a call copies
// nothing to the device and can be captured.
//
// The tensors are one list of units of four elements (the last unit of a tensor may hold fewer),
// which is shared out without regard to the tensors' borders, so that many small and few large
// tensors load the GPU alike.
#include <cooperative_groups.h>

#include "sbp_internal.cuh"

namespace sbp {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
// CTAs per SM of the summing pass and of the clipping.  In place under the limit the clipping's
// CTAs only read the sum and end, so they are kept few where the list is short (38 M elements:
// 3 us at 8 per SM, 13 with a CTA per piece); a long list goes faster with a CTA per piece
// (218 M elements: 248 us, 266 at 32 per SM).
constexpr int kSumBlocks = 16, kClipBlocks = 32, kManyPieces = 128;
// Up to this many pieces per SM every CTA of the clipping joins the partial sums itself; above,
// a launch of its own does.
constexpr int kJoinPieces = 8;
// tensors of one launch: the small table where it is enough, as a launch copies its parameters
constexpr int kSmallTable = 64, kLargeTable = 1024;

constexpr int kIndex = 64;     // entries of a table's index

template <int N>
struct Tensors {
  int n;
  int64_t units;          // of all n tensors
  int64_t end[N];         // units up to and including tensor i, times 4, plus the number of
                          // elements that its last unit lacks
  const float* src[N];
  float* dst[N];
  // the tensor of every (1 << shift)-th unit: a search through 300 tensors starts between two of
  // these and takes about three dependent loads, not nine (30 M elements: 61.4 us, 62.6 without;
  // 2 M in 50 tensors: 10.0, 10.4)
  int shift;
  short first[kIndex + 1];
};

// the tensor in [lo, n) that unit u belongs to, by the table of ends
__device__ __forceinline__ int tensor_of(const int64_t* end, int lo, int n, int64_t u) {
  int hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if ((end[mid] >> 2) <= u)
      lo = mid + 1;
    else
      hi = mid;
  }
  return lo;
}

// One unit: where its elements are and how many it has.
struct Unit {
  int64_t at;       // element index in the tensor
  int have;
  __device__ __forceinline__ Unit(const int64_t* end, int i, int64_t u)
      : at(4 * (u - (i ? end[i - 1] >> 2 : 0))),
        have(u == (end[i] >> 2) - 1 ? 4 - (int)(end[i] & 3) : 4) {}
};
__device__ __forceinline__ float4 load_unit(const float* p, int have) {
  if (have == 4) return *reinterpret_cast<const float4*>(p);
  return make_float4(p[0], have > 1 ? p[1] : 0.f, have > 2 ? p[2] : 0.f, 0.f);
}
__device__ __forceinline__ void store_unit(float* p, int have, float4 v) {
  if (have == 4) {
    *reinterpret_cast<float4*>(p) = v;
    return;
  }
  p[0] = v.x;
  if (have > 1) p[1] = v.y;
  if (have > 2) p[2] = v.z;
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// the block's sum in thread 0 (two levels of shuffles; red holds a value per warp)
__device__ __forceinline__ double block_sum(double v, double* red) {
  v = warp_sum64(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) v = warp_sum64(threadIdx.x < blockDim.x / 32 ? red[threadIdx.x] : 0.0);
  return v;
}

__device__ __forceinline__ double square(float v) { return (double)v * (double)v; }
__device__ __forceinline__ double square(float4 v) {
  return square(v.x) + square(v.y) + (square(v.z) + square(v.w));
}

// coefficient of the clipping; 1 where the norm is not finite (no right one exists)
__device__ __forceinline__ float clip_coef(double norm, float max_norm) {
  if (!isfinite(norm)) return 1.f;
  const double c = (double)max_norm / (norm + 1e-6);
  return c < 1.0 ? (float)c : 1.f;
}

// The list is taken in pieces of kPiece units, dealt to the CTAs in turn, so that the GPU moves
// through one neighbourhood of memory at a time (an equal contiguous range per CTA, 1184 streams
// at once, took 490 instead of 442 us for 218 M elements).  A piece that lies in one tensor and
// does not hold its last unit takes the direct path; one with a border looks each unit's tensor up.
constexpr int kPiece = 4 * kThreads;

// the tensor that a thread's last piece was in, and its units [from, to)
struct Place {
  int i = 0;
  int64_t from = 0, to = 0;
  template <int N>
  __device__ __forceinline__ void find(const Tensors<N>& t, int64_t u) {
    if (u >= from && u < to) return;
    const int k = (int)(u >> t.shift);
    i = tensor_of(t.end, t.first[k], t.first[k + 1] + 1, u);
    from = i ? t.end[i - 1] >> 2 : 0;
    to = t.end[i] >> 2;
  }
  // behind the tensors that a unit of the piece at c can be in: mostly this one and the next; a
  // short range keeps the units' own searches short (1 M elements in 200 tensors: 8.4 us, 10.4
  // with a search to the list's end)
  template <int N>
  __device__ __forceinline__ int behind(const Tensors<N>& t, int64_t c) const {
    if (i + 1 < t.n && (t.end[i + 1] >> 2) >= c + kPiece) return i + 2;
    const int64_t u = imin(c + kPiece, t.units) - 1;
    const int k = (int)(u >> t.shift);
    return tensor_of(t.end, max(i, t.first[k]), t.first[k + 1] + 1, u) + 1;
  }
};

template <int N>
__global__ void __launch_bounds__(kThreads)
sqsum_kernel(const __grid_constant__ Tensors<N> t, double* __restrict__ partial) {
  __shared__ double red[kThreads / 32];
  release_next();
  double s[4] = {};
  Place at, next;
  next.find(t, (int64_t)blockIdx.x * kPiece);
  for (int64_t c = (int64_t)blockIdx.x * kPiece; c < t.units;) {
    at = next;
    float4 v[4];
    if (c + kPiece < at.to) {
      const float4* g = reinterpret_cast<const float4*>(t.src[at.i]) + (c - at.from) + threadIdx.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = g[k * kThreads];
    } else {
      const int hi = at.behind(t, c);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t u = c + threadIdx.x + k * kThreads;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (u >= t.units) continue;
        const int j = tensor_of(t.end, at.i, hi, u);
        const Unit x(t.end, j, u);
        v[k] = load_unit(t.src[j] + x.at, x.have);
      }
    }
    c += (int64_t)gridDim.x * kPiece;
    if (c < t.units) next.find(t, c);      // while the loads are on their way
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] += square(v[k]);
  }
  const double v = block_sum((s[0] + s[1]) + (s[2] + s[3]), red);
  if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// sum of the partial sums in thread 0, the same bits in every CTA
__device__ __forceinline__ double join(int64_t n, const double* partial, double* red) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) s += partial[i];
  return block_sum(s, red);
}

constexpr int kFinishThreads = 1024;
__global__ void __launch_bounds__(kFinishThreads)
sqsum_finish_kernel(int64_t n, const double* partial, double* __restrict__ sqsum) {
  __shared__ double red[kFinishThreads / 32];
  release_next();
  await_previous();
  const double s = join(n, partial, red);
  if (threadIdx.x == 0) *sqsum = s;
}

__device__ __forceinline__ float4 scaled(float4 v, float c) {
  return make_float4(v.x * c, v.y * c, v.z * c, v.w * c);
}

// The pieces are taken from the end of the list: what was summed last is still in L2.
template <int N>
__global__ void __launch_bounds__(kThreads)
clip_kernel(const __grid_constant__ Tensors<N> t, int64_t parts, const double* partial,
            float max_norm, bool in_place, float* __restrict__ norm_out) {
  __shared__ double red[kThreads / 32];
  __shared__ float shared_coef;
  release_next();
  await_previous();
  const double sum = join(parts, partial, red);
  if (threadIdx.x == 0) {      // one thread's square root and division
    const double norm = sqrt(sum);
    shared_coef = clip_coef(norm, max_norm);
    if (norm_out && blockIdx.x == 0) *norm_out = (float)norm;
  }
  __syncthreads();
  const float coef = shared_coef;
  if (in_place && coef == 1.f) return;
  Place at;
  for (int64_t p = (t.units + kPiece - 1) / kPiece - 1 - blockIdx.x; p >= 0; p -= gridDim.x) {
    const int64_t c = p * kPiece;
    at.find(t, c);
    float4 v[4];
    if (c + kPiece < at.to) {
      const int64_t o = c - at.from + threadIdx.x;
      const float4* g = reinterpret_cast<const float4*>(t.src[at.i]) + o;
      float4* d = reinterpret_cast<float4*>(t.dst[at.i]) + o;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = g[k * kThreads];
#pragma unroll
      for (int k = 0; k < 4; ++k) d[k * kThreads] = scaled(v[k], coef);
      continue;
    }
    const int hi = at.behind(t, c);
    float* d[4];
    int have[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t u = c + threadIdx.x + k * kThreads;
      have[k] = 0;
      if (u >= t.units) continue;
      const int j = tensor_of(t.end, at.i, hi, u);
      const Unit x(t.end, j, u);
      d[k] = t.dst[j] + x.at;
      have[k] = x.have;
      v[k] = load_unit(t.src[j] + x.at, x.have);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (have[k] > 0) store_unit(d[k], have[k], scaled(v[k], coef));
  }
}

// Few elements: one cluster holds them in registers, joins its CTAs' sums over distributed
// shared memory and writes, in a single launch and with every element read once.
constexpr int kFewCtas = 8, kFewThreads = 1024, kFewUnits = 4;
constexpr int64_t kFewMax = (int64_t)kFewCtas * kFewThreads * kFewUnits;
template <int N>
__global__ void __cluster_dims__(kFewCtas, 1, 1) __launch_bounds__(kFewThreads)
clip_few_kernel(const __grid_constant__ Tensors<N> t, float max_norm,
                float* __restrict__ norm_out) {
  __shared__ double red[kFewThreads / 32], sum;
  __shared__ float shared_coef;
  __shared__ int64_t end[N];
  cg::cluster_group cluster = cg::this_cluster();
  for (int i = threadIdx.x; i < t.n; i += kFewThreads) end[i] = t.end[i];
  __syncthreads();
  float4 v[kFewUnits];
  const float* src[kFewUnits];
  float* dst[kFewUnits];
  int have[kFewUnits];      // elements of the unit, 0 behind the last one
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < kFewUnits; ++k) {
    const int64_t u = blockIdx.x * kFewThreads + threadIdx.x + k * (kFewCtas * kFewThreads);
    have[k] = 0;
    if (u >= t.units) continue;
    const int i = tensor_of(end, 0, t.n, u);
    const Unit x(end, i, u);
    src[k] = t.src[i] + x.at;
    dst[k] = t.dst[i] + x.at;
    have[k] = x.have;
    v[k] = load_unit(src[k], x.have);
    s += square(v[k]);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) sum = s;
  cluster.sync();
  if (threadIdx.x == 0) {
    s = 0.0;
#pragma unroll
    for (int c = 0; c < kFewCtas; ++c) s += *cluster.map_shared_rank(&sum, c);
    const double norm = sqrt(s);
    shared_coef = clip_coef(norm, max_norm);
    if (blockIdx.x == 0) *norm_out = (float)norm;
  }
  cluster.sync();           // the coefficient; and no CTA ends while another reads its sum
  const float coef = shared_coef;
#pragma unroll
  for (int k = 0; k < kFewUnits; ++k)
    if (have[k] > 0 && (dst[k] != src[k] || coef != 1.f))
      store_unit(dst[k], have[k], scaled(v[k], coef));
}

// the next launch's tensors: up to N non-empty ones from index i on
template <int N>
int64_t take(Tensors<N>& t, int64_t i, const GradTensors& g) {
  t.n = 0;
  t.units = 0;
  for (; i < g.n && t.n < N; ++i) {
    const int64_t m = g.numel[i];
    if (m == 0) continue;
    t.units += (m + 3) / 4;
    t.src[t.n] = g.src[i];
    t.dst[t.n] = g.dst ? g.dst[i] : const_cast<float*>(g.src[i]);
    t.end[t.n] = 4 * t.units + (4 - m % 4) % 4;
    ++t.n;
  }
  return i;
}

// the index of a table of at least one unit (of none: zeros, which no kernel reads)
template <int N>
void index(Tensors<N>& t) {
  t.shift = 0;
  while (((t.units - 1) >> t.shift) >= kIndex) ++t.shift;
  int i = 0;
  for (int k = 0; k <= kIndex; ++k) {
    const int64_t u = imin((int64_t)k << t.shift, t.units - 1);
    while (i + 1 < t.n && (t.end[i] >> 2) <= u) ++i;
    t.first[k] = (short)i;
  }
}

int64_t pieces_of(int64_t units) { return imax(1, (units + kPiece - 1) / kPiece); }

template <int N>
int64_t launch_sqsum(const GradTensors& g, double* partial, cudaStream_t st) {
  int64_t parts = 0;
  Tensors<N> t;
  for (int64_t i = 0; i < g.n;) {
    i = take(t, i, g);
    if (t.n == 0) break;
    index(t);
    const int64_t grid = imin(pieces_of(t.units), (int64_t)sm_count() * kSumBlocks);
    launch(sqsum_kernel<N>, dim3((unsigned)grid), dim3(kThreads), 0, st, t, partial + parts);
    parts += grid;
  }
  return parts;
}

template <int N>
void launch_clip(const GradTensors& g, int64_t parts, const double* partial, float max_norm,
                 float* norm_out, bool after_sum, cudaStream_t st) {
  Tensors<N> t;
  bool in_place = true;
  for (int64_t i = 0; g.dst && i < g.n; ++i) in_place &= g.dst[i] == g.src[i] || g.numel[i] == 0;
  for (int64_t i = 0; i == 0 || i < g.n;) {     // one launch at least: it writes the norm
    i = imax(1, take(t, i, g));
    index(t);
    int64_t grid = pieces_of(t.units);
    if (grid <= (int64_t)sm_count() * kManyPieces)
      grid = imin(grid, (int64_t)sm_count() * kClipBlocks);
    if (after_sum)
      launch_next(clip_kernel<N>, dim3((unsigned)grid), dim3(kThreads), 0, st, t, parts, partial,
                  max_norm, in_place, norm_out);
    else
      launch(clip_kernel<N>, dim3((unsigned)grid), dim3(kThreads), 0, st, t, parts, partial,
             max_norm, in_place, norm_out);
    norm_out = nullptr;
  }
}

template <int N>
void launch_few(const GradTensors& g, float max_norm, float* norm_out, cudaStream_t st) {
  Tensors<N> t;
  take(t, 0, g);
  launch(clip_few_kernel<N>, dim3(kFewCtas), dim3(kFewThreads), 0, st, t, max_norm, norm_out);
}

// the workspace: the joined sum, then the partial sums
constexpr size_t kPartialOffset = 256;
double* partials(void* ws) {
  return reinterpret_cast<double*>(static_cast<char*>(ws) + kPartialOffset);
}

int64_t sqsum_parts(const GradTensors& g, void* ws, cudaStream_t st) {
  return g.n <= kSmallTable ? launch_sqsum<kSmallTable>(g, partials(ws), st)
                            : launch_sqsum<kLargeTable>(g, partials(ws), st);
}

void sqsum_join(int64_t parts, void* ws, double* sqsum, cudaStream_t st) {
  launch_next(sqsum_finish_kernel, dim3(1), dim3(kFinishThreads), 0, st, parts,
         (const double*)partials(ws), sqsum);
}

void clip_parts(const GradTensors& g, int64_t parts, const double* partial, float max_norm,
                float* norm_out, bool after_sum, cudaStream_t st) {
  if (g.n <= kSmallTable)
    launch_clip<kSmallTable>(g, parts, partial, max_norm, norm_out, after_sum, st);
  else
    launch_clip<kLargeTable>(g, parts, partial, max_norm, norm_out, after_sum, st);
}

}  // namespace

size_t grad_norm_ws_bytes(int64_t n) {
  const int64_t launches = n / kLargeTable + 1;
  return kPartialOffset + sizeof(double) * (size_t)(launches * sm_count() * kSumBlocks);
}

cudaError_t grad_sqsum(const GradTensors& g, double* sqsum, void* ws, cudaStream_t st) {
  sqsum_join(sqsum_parts(g, ws, st), ws, sqsum, st);
  return cudaGetLastError();
}

cudaError_t grad_clip(const GradTensors& g, const double* sqsum, float max_norm, float* norm_out,
                      cudaStream_t st) {
  clip_parts(g, 1, sqsum, max_norm, norm_out, false, st);
  return cudaGetLastError();
}

cudaError_t grad_clip_norm(const GradTensors& g, float max_norm, float* norm_out, void* ws,
                           cudaStream_t st) {
  int64_t units = 0, n = 0;
  for (int64_t i = 0; i < g.n; ++i) {
    units += (g.numel[i] + 3) / 4;
    n += g.numel[i] > 0;
  }
  if (units <= kFewMax && n <= kLargeTable) {
    if (n <= kSmallTable)
      launch_few<kSmallTable>(g, max_norm, norm_out, st);
    else
      launch_few<kLargeTable>(g, max_norm, norm_out, st);
    return cudaGetLastError();
  }
  const int64_t parts = sqsum_parts(g, ws, st);
  if (pieces_of(units) <= (int64_t)sm_count() * kJoinPieces) {
    clip_parts(g, parts, partials(ws), max_norm, norm_out, true, st);
  } else {
    double* sqsum = static_cast<double*>(ws);
    sqsum_join(parts, ws, sqsum, st);
    clip_parts(g, 1, sqsum, max_norm, norm_out, true, st);
  }
  return cudaGetLastError();
}

}  // namespace sbp
