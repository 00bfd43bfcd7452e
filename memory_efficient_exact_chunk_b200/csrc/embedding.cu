// Scaled token embedding and its gradient by sorted tokens.
//
//   forward   y[r] = scale * table[ids[r]]
//   backward  d_table[v] (+)= scale * sum_{r : ids[r] = v} dy[r]
//
// Both are bound by HBM: the forward reads the used table rows and writes y, the backward reads
// dy once and reads and writes (or only writes) the table rows.
#include "sbp_internal.cuh"

namespace sbp {

namespace {

inline unsigned nblk(int64_t n, int64_t t) { return (unsigned)((n + t - 1) / t); }

// ---------------------------------------------------------------- forward
// One CTA per row; a row whose id is outside [0, vocab) becomes zero.
template <typename T>
__global__ void embed_scaled_fwd_kernel(int64_t cols, int64_t vocab, float scale,
                                        const int* __restrict__ ids, const T* __restrict__ table,
                                        T* __restrict__ y) {
  const int64_t r = blockIdx.x;
  const int64_t v = ids[r];
  const bool ok = v >= 0 && v < vocab;
  for (int64_t c = threadIdx.x; c < cols; c += blockDim.x)
    st_f(y, r * cols + c, ok ? scale * ld_f(table, v * cols + c) : 0.f);
}

// ---------------------------------------------------------------- sort by id
// Sorted position of every row by counting: a row's run starts at the number of rows with a
// smaller id and the row stands behind the earlier rows of its own id (a stable sort).  Ids
// outside [0, vocab) take the key vocab and end up last.  Four threads share a row; the ids
// pass through shared memory.
constexpr int kRankThreads = 256, kRankRows = kRankThreads / 4, kRankTile = 4096;
__global__ void __launch_bounds__(kRankThreads)
embed_rank_kernel(int rows, int vocab, const int* __restrict__ ids, int4* __restrict__ sorted) {
  __shared__ __align__(16) int key[kRankTile];
  const int r = blockIdx.x * kRankRows + threadIdx.x / 4, part = threadIdx.x % 4;
  int mine = -1;
  if (r < rows) {
    mine = ids[r];
    if (mine < 0 || mine >= vocab) mine = vocab;
  }
  int less = 0, equal = 0, before = 0;
  for (int t0 = 0; t0 < rows; t0 += kRankTile) {
    const int n = min(kRankTile, rows - t0);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kRankThreads) {
      const int v = ids[t0 + i];
      key[i] = v < 0 || v >= vocab ? vocab : v;
    }
    __syncthreads();
    for (int i = part; i < n; i += 4) {
      const int k = key[i];
      less += k < mine;
      equal += k == mine;
      before += k == mine && t0 + i < r;
    }
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    less += __shfl_xor_sync(0xffffffffu, less, o);
    equal += __shfl_xor_sync(0xffffffffu, equal, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (r < rows && part == 0) sorted[less + before] = make_int4(r, less, equal, mine);
}

// ---------------------------------------------------------------- accumulate
// One CTA per sorted position; the first of each run adds the run's rows in order.
__global__ void embed_run_kernel(int64_t cols, int vocab, float scale,
                                 const int4* __restrict__ sorted, const float* __restrict__ dy,
                                 float* __restrict__ d_table) {
  const int p = blockIdx.x;
  const int4 s = sorted[p];
  if (s.y != p || s.w == vocab) return;
  for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) {
    float a = 0.f;
    for (int i = 0; i < s.z; ++i) a += dy[(int64_t)sorted[p + i].x * cols + c];
    d_table[(int64_t)s.w * cols + c] += scale * a;
  }
}

}  // namespace

cudaError_t embed_scaled_fwd(int64_t rows, int64_t cols, int64_t vocab, int dt, float scale,
                             const int* ids, const void* table, void* y, cudaStream_t st) {
  if (dt == DT_BF16)
    launch(embed_scaled_fwd_kernel<__nv_bfloat16>, dim3((unsigned)rows), dim3(256), 0, st, cols,
           vocab, scale, ids, static_cast<const __nv_bfloat16*>(table),
           static_cast<__nv_bfloat16*>(y));
  else
    launch(embed_scaled_fwd_kernel<float>, dim3((unsigned)rows), dim3(256), 0, st, cols, vocab,
           scale, ids, static_cast<const float*>(table), static_cast<float*>(y));
  return cudaGetLastError();
}

size_t embed_scaled_bwd_ws_bytes(int64_t rows, int64_t cols, int64_t vocab) {
  (void)cols;
  (void)vocab;
  return (size_t)rows * sizeof(int4);
}

cudaError_t embed_scaled_bwd(int64_t rows, int64_t cols, int64_t vocab, float scale,
                             const int* ids, const float* dy, float* d_table, int accumulate,
                             void* ws, cudaStream_t st) {
  if (!accumulate) {
    const cudaError_t e = cudaMemsetAsync(d_table, 0, sizeof(float) * (size_t)vocab * cols, st);
    if (e != cudaSuccess) return e;
  }
  int4* sorted = static_cast<int4*>(ws);
  launch(embed_rank_kernel, dim3(nblk(rows, kRankRows)), dim3(kRankThreads), 0, st, (int)rows,
         (int)vocab, ids, sorted);
  launch(embed_run_kernel, dim3((unsigned)rows), dim3(256), 0, st, cols, (int)vocab, scale,
         (const int4*)sorted, dy, d_table);
  return cudaGetLastError();
}

}  // namespace sbp
