// Global gradient norm over many tensors, and clipping.
//
//   sqsum = sum over tensors and elements of g^2,  norm = sqrt(sqsum)
//   out = g * min(1, max_norm / (norm + 1e-6))
//
// Products and sums are formed in 64 bits: the square of an fp32 value neither overflows nor
// vanishes there.  Both passes are bound by HBM (4 bytes read per element, then 8 moved where
// the clipping bites).  The tensors' pointers travel as kernel parameters, so a call copies
// nothing to the device and can be captured; tensors are cut into chunks of kChunk elements.
#include <cmath>

#include "sbp_internal.cuh"

namespace sbp {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kChunk = 16384;        // elements of a chunk
constexpr int kMaxTensors = 256;         // tensors of one launch
constexpr int kBlocksPerSm = 8;

struct Tensors {
  int n;
  int64_t chunks;                        // first[n]
  const float* src[kMaxTensors];
  float* dst[kMaxTensors];
  int64_t numel[kMaxTensors];
  int64_t first[kMaxTensors + 1];        // chunk index at which each tensor begins
};

// the tensor that chunk c belongs to: the last one with first[i] <= c
__device__ __forceinline__ int tensor_of(const Tensors& t, int64_t c) {
  int lo = 0, hi = t.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int i = 0; i < (int)(blockDim.x >> 5); ++i) s += red[i];
  return s;
}

__device__ __forceinline__ double square(float v) { return (double)v * (double)v; }

__global__ void __launch_bounds__(kThreads)
sqsum_kernel(const __grid_constant__ Tensors t, double* __restrict__ partial) {
  __shared__ double red[32];
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t o = (c - t.first[i]) * kChunk;
    const int n = (int)imin(kChunk, t.numel[i] - o);
    const float* g = t.src[i] + o;
    const float4* g4 = reinterpret_cast<const float4*>(g);
    for (int k = threadIdx.x; k < n / 4; k += kThreads) {
      const float4 v = g4[k];
      s += square(v.x) + square(v.y) + (square(v.z) + square(v.w));
    }
    for (int k = n / 4 * 4 + threadIdx.x; k < n; k += kThreads) s += square(g[k]);
  }
  s = block_sum(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kThreads)
sqsum_finish_kernel(int64_t n, const double* __restrict__ partial, double* __restrict__ sqsum) {
  __shared__ double red[32];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) s += partial[i];
  s = block_sum(s, red);
  if (threadIdx.x == 0) *sqsum = s;
}

// coefficient of the clipping; 1 where the norm is not finite (no right one exists)
__device__ __forceinline__ float clip_coef(double norm, float max_norm) {
  if (!isfinite(norm)) return 1.f;
  const double c = (double)max_norm / (norm + 1e-6);
  return c < 1.0 ? (float)c : 1.f;
}

__global__ void __launch_bounds__(kThreads)
clip_kernel(const __grid_constant__ Tensors t, const double* __restrict__ sqsum, float max_norm,
            float* __restrict__ norm_out) {
  const double norm = sqrt(*sqsum);
  const float coef = clip_coef(norm, max_norm);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t o = (c - t.first[i]) * kChunk;
    const int n = (int)imin(kChunk, t.numel[i] - o);
    const float* g = t.src[i] + o;
    float* d = t.dst[i] + o;
    if (g == d && coef == 1.f) continue;
    const float4* g4 = reinterpret_cast<const float4*>(g);
    float4* d4 = reinterpret_cast<float4*>(d);
    for (int k = threadIdx.x; k < n / 4; k += kThreads) {
      float4 v = g4[k];
      v.x *= coef; v.y *= coef; v.z *= coef; v.w *= coef;
      d4[k] = v;
    }
    for (int k = n / 4 * 4 + threadIdx.x; k < n; k += kThreads) d[k] = g[k] * coef;
  }
}

// the next launch's tensors: up to kMaxTensors non-empty ones from index i on
int64_t take(Tensors& t, int64_t i, int64_t n, const float* const* grads, float* const* outs,
             const int64_t* numel) {
  t.n = 0;
  t.chunks = 0;
  for (; i < n && t.n < kMaxTensors; ++i) {
    if (numel[i] == 0) continue;
    t.src[t.n] = grads[i];
    t.dst[t.n] = outs ? outs[i] : const_cast<float*>(grads[i]);
    t.numel[t.n] = numel[i];
    t.first[t.n] = t.chunks;
    t.chunks += (numel[i] + kChunk - 1) / kChunk;
    ++t.n;
  }
  t.first[t.n] = t.chunks;
  return i;
}

unsigned grid_of(const Tensors& t) {
  return (unsigned)imin(t.chunks, (int64_t)sm_count() * kBlocksPerSm);
}

}  // namespace

size_t grad_norm_ws_bytes(int64_t n) {
  const int64_t launches = n > 0 ? (n + kMaxTensors - 1) / kMaxTensors : 1;
  return 256 + sizeof(double) * (size_t)(launches * sm_count() * kBlocksPerSm);
}

cudaError_t grad_sqsum(int64_t n, const float* const* grads, const int64_t* numel, double* sqsum,
                       void* ws, cudaStream_t st) {
  double* partial = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
  int64_t parts = 0;
  Tensors t;
  for (int64_t i = 0; i < n;) {
    i = take(t, i, n, grads, nullptr, numel);
    if (t.n == 0) break;
    launch(sqsum_kernel, dim3(grid_of(t)), dim3(kThreads), 0, st, t, partial + parts);
    parts += grid_of(t);
  }
  launch(sqsum_finish_kernel, dim3(1), dim3(kThreads), 0, st, parts, (const double*)partial,
         sqsum);
  return cudaGetLastError();
}

cudaError_t grad_clip(int64_t n, const float* const* grads, float* const* outs,
                      const int64_t* numel, const double* sqsum, float max_norm, float* norm_out,
                      cudaStream_t st) {
  Tensors t;
  bool first = true;
  for (int64_t i = 0; first || i < n;) {
    i = take(t, i, n, grads, outs, numel);
    if (t.n == 0 && !first) break;
    launch(clip_kernel, dim3(t.n ? grid_of(t) : 1u), dim3(kThreads), 0, st, t, sqsum, max_norm,
           first ? norm_out : static_cast<float*>(nullptr));
    first = false;
  }
  return cudaGetLastError();
}

}  // namespace sbp
