// Per-head RMS norm of queries and keys with the rotate-half RoPE in the same pass, forward and
// backward.  For one head x of hd elements at position p (h = hd / 2):
//   n = x rstd g,  rstd = 1 / sqrt(mean(x^2) + eps)
//   y_j = n_j c_j - n_{j+h} s_j,  y_{j+h} = n_{j+h} c_j + n_j s_j
// and for an upstream gradient dy, with u its inverse rotation and xh = x rstd:
//   dg += sum u xh,   dx = rstd (g u - xh mean(xh g u)).
// A head is read once into registers, so both directions move each element once; they are bound
// by HBM.
#include "sbp_internal.cuh"

namespace sbp {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs = 4;   // pairs (j, j + hd / 2) of one lane: hd <= 256

inline int64_t nblk(int64_t n, int64_t t) { return (n + t - 1) / t; }

struct RowMap {
  const int* positions;
  int64_t seq_len, pos0, table_len, k_T;
  __device__ __forceinline__ int64_t pos(int64_t r) const {
    return positions ? (int64_t)positions[r] : pos0 + r % seq_len;
  }
  // row of the keys' output that row r goes to
  __device__ __forceinline__ int64_t k_row(int64_t r) const {
    return k_T > 0 ? (r / seq_len) * k_T + pos0 + r % seq_len : r;
  }
};

template <typename T>
struct Heads {        // one of the two tensors (queries or keys)
  int n;              // heads per row
  const T* x;
  int64_t ldx;
  const T* g;
  T* y;
  int64_t ldy;
  const float* dy;
  int64_t lddy;
  float* dx;
  int64_t lddx;
};

// One warp per (row, head); lane l holds the pairs l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(kThreads)
qk_fwd_kernel(int64_t rows, int hd, Heads<T> q, Heads<T> k, RowMap map,
              const float* __restrict__ cosb, const float* __restrict__ sinb, float eps) {
  const int lane = threadIdx.x & 31, half = hd / 2;
  const int64_t heads = q.n + k.n;
  for (int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); item < rows * heads;
       item += (int64_t)gridDim.x * kWarps) {
  const int64_t r = item / heads;
  int hh = (int)(item - r * heads);
  const bool is_k = hh >= q.n;
  const Heads<T>& t = is_k ? k : q;
  if (is_k) hh -= q.n;
  const T* x = t.x + r * t.ldx + (int64_t)hh * hd;
  T* y = t.y + (is_k ? map.k_row(r) : r) * t.ldy + (int64_t)hh * hd;
  const int64_t p = map.pos(r);
  const bool ok = p >= 0 && p < map.table_len;
  float a[kMaxPairs], b[kMaxPairs], ss = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxPairs; ++i) {
    const int j = lane + 32 * i;
    a[i] = j < half ? ld_f(x, j) : 0.f;
    b[i] = j < half ? ld_f(x, j + half) : 0.f;
    ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
  }
  const float rs = rsqrtf(warp_sum(ss) / (float)hd + eps);
#pragma unroll
  for (int i = 0; i < kMaxPairs; ++i) {
    const int j = lane + 32 * i;
    if (j >= half) continue;
    float y1 = 0.f, y2 = 0.f;
    if (ok) {
      const float c = cosb[p * half + j], s = sinb[p * half + j];
      const float n1 = a[i] * rs * ld_f(t.g, j), n2 = b[i] * rs * ld_f(t.g, j + half);
      y1 = n1 * c - n2 * s;
      y2 = n2 * c + n1 * s;
    }
    st_f(y, j, y1);
    st_f(y, j + half, y2);
  }
  }
}

// Blocks [0, q_blocks) take the queries, the others the keys; a block's warps take (row, head)
// items in turn, keep the gain gradient of their pairs in registers and leave the block's sum
// in partial[block].
template <typename T>
__global__ void __launch_bounds__(kThreads)
qk_bwd_kernel(int64_t rows, int hd, int q_blocks, Heads<T> q, Heads<T> k, RowMap map,
              const float* __restrict__ cosb, const float* __restrict__ sinb, float eps,
              float* __restrict__ partial) {
  __shared__ float red[kWarps][256];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, half = hd / 2;
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const Heads<T>& t = is_k ? k : q;
  const int64_t b0 = is_k ? blockIdx.x - q_blocks : blockIdx.x;
  const int64_t nb = is_k ? gridDim.x - q_blocks : q_blocks;
  float ga[kMaxPairs], gb[kMaxPairs], da[kMaxPairs], db[kMaxPairs];
#pragma unroll
  for (int i = 0; i < kMaxPairs; ++i) {
    const int j = lane + 32 * i;
    ga[i] = j < half ? ld_f(t.g, j) : 0.f;
    gb[i] = j < half ? ld_f(t.g, j + half) : 0.f;
    da[i] = db[i] = 0.f;
  }
  for (int64_t item = b0 * kWarps + wid; item < rows * t.n; item += nb * kWarps) {
    const int64_t r = item / t.n, hh = item - r * t.n;
    const T* x = t.x + r * t.ldx + hh * hd;
    const float* dy = t.dy + r * t.lddy + hh * hd;
    float* dx = t.dx + r * t.lddx + hh * hd;
    const int64_t p = map.pos(r);
    const bool ok = p >= 0 && p < map.table_len;
    float a[kMaxPairs], b[kMaxPairs], u[kMaxPairs], v[kMaxPairs], ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < kMaxPairs; ++i) {
      const int j = lane + 32 * i;
      a[i] = b[i] = u[i] = v[i] = 0.f;
      if (j < half && ok) {
        a[i] = ld_f(x, j);
        b[i] = ld_f(x, j + half);
        const float d1 = dy[j], d2 = dy[j + half];
        const float c = cosb[p * half + j], s = sinb[p * half + j];
        u[i] = d1 * c + d2 * s;
        v[i] = d2 * c - d1 * s;
      }
      ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
    }
    const float rs = rsqrtf(warp_sum(ss) / (float)hd + eps);
#pragma unroll
    for (int i = 0; i < kMaxPairs; ++i) {
      if (ok) {
        a[i] *= rs;
        b[i] *= rs;
        da[i] = fmaf(u[i], a[i], da[i]);
        db[i] = fmaf(v[i], b[i], db[i]);
      }
      u[i] *= ga[i];
      v[i] *= gb[i];
      dot = fmaf(a[i], u[i], fmaf(b[i], v[i], dot));
    }
    dot = warp_sum(dot) / (float)hd;
#pragma unroll
    for (int i = 0; i < kMaxPairs; ++i) {
      const int j = lane + 32 * i;
      if (j >= half) continue;
      dx[j] = ok ? rs * (u[i] - a[i] * dot) : 0.f;
      dx[j + half] = ok ? rs * (v[i] - b[i] * dot) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kMaxPairs; ++i) {
    const int j = lane + 32 * i;
    if (j < half) {
      red[wid][j] = da[i];
      red[wid][j + half] = db[i];
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < hd; c += kThreads) {
    float s = red[0][c];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += red[w][c];
    partial[(int64_t)blockIdx.x * hd + c] = s;
  }
}

// dst[c] += sum of the blocks' partials in order (block 0: queries, block 1: keys)
__global__ void qk_gain_kernel(int hd, int q_blocks, int blocks, const float* __restrict__ partial,
                               float* __restrict__ dq_g, float* __restrict__ dk_g) {
  const int b0 = blockIdx.x ? q_blocks : 0, b1 = blockIdx.x ? blocks : q_blocks;
  float* dst = blockIdx.x ? dk_g : dq_g;
  for (int c = threadIdx.x; c < hd; c += blockDim.x) {
    float s = 0.f;
    for (int b = b0; b < b1; ++b) s += partial[(int64_t)b * hd + c];
    dst[c] += s;
  }
}

// blocks of the backward for the queries and the keys, in proportion to their items
void bwd_blocks(const QkNorm& a, int& qb, int& kb) {
  const int64_t cap = (int64_t)sm_count() * 4;
  const int64_t qi = nblk(a.rows * a.q.n, kWarps), ki = nblk(a.rows * a.k.n, kWarps);
  if (qi + ki <= cap) {
    qb = (int)qi;
    kb = (int)ki;
  } else {
    kb = a.k.n ? (int)imax(1, cap * ki / (qi + ki)) : 0;
    qb = (int)(cap - kb);
  }
}

template <typename T>
Heads<T> heads_of(const QkNormHeads& h) {
  return Heads<T>{(int)h.n, static_cast<const T*>(h.x), h.ldx, static_cast<const T*>(h.g),
                  static_cast<T*>(h.y), h.ldy, h.dy, h.lddy, h.dx, h.lddx};
}
RowMap map_of(const QkNorm& a) {
  return RowMap{a.positions, a.seq_len, a.pos0, a.table_len, a.k_T};
}

template <typename T>
cudaError_t fwd(const QkNorm& a, cudaStream_t st) {
  const int64_t n = nblk(a.rows * (a.q.n + a.k.n), kWarps);
  launch(qk_fwd_kernel<T>, dim3((unsigned)imin(n, (int64_t)sm_count() * 8)), dim3(kThreads), 0,
         st, a.rows, (int)a.hd, heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb,
         a.eps);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const QkNorm& a, float* dq_g, float* dk_g, float* partial, cudaStream_t st) {
  int qb, kb;
  bwd_blocks(a, qb, kb);
  launch(qk_bwd_kernel<T>, dim3(qb + kb), dim3(kThreads), 0, st, a.rows, (int)a.hd, qb,
         heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb, a.eps, partial);
  launch(qk_gain_kernel, dim3(kb ? 2 : 1), dim3(256), 0, st, (int)a.hd, qb, qb + kb,
         (const float*)partial, dq_g, dk_g);
  return cudaGetLastError();
}

}  // namespace

cudaError_t qk_norm_rope_fwd(const QkNorm& a, cudaStream_t st) {
  return a.dt == DT_BF16 ? fwd<__nv_bfloat16>(a, st) : fwd<float>(a, st);
}

size_t qk_norm_bwd_partial_floats(int64_t rows, int64_t n_heads, int64_t n_kv, int64_t hd) {
  QkNorm a;
  a.rows = rows;
  a.q.n = n_heads;
  a.k.n = n_kv;
  int qb, kb;
  bwd_blocks(a, qb, kb);
  return (size_t)(qb + kb) * hd;
}

cudaError_t qk_norm_rope_bwd(const QkNorm& a, float* dq_g, float* dk_g, float* partial,
                             cudaStream_t st) {
  return a.dt == DT_BF16 ? bwd<__nv_bfloat16>(a, dq_g, dk_g, partial, st)
                         : bwd<float>(a, dq_g, dk_g, partial, st);
}

}  // namespace sbp
