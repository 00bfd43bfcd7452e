// Per-head RMS norm of queries and keys with the rotate-half RoPE in the same pass, forward and
// backward.  For one head x of hd elements at position p (h = hd / 2):
//   n = x rstd g,  rstd = 1 / sqrt(mean(x^2) + eps)
//   y_j = n_j c_j - n_{j+h} s_j,  y_{j+h} = n_{j+h} c_j + n_j s_j
// and for an upstream gradient dy, with u its inverse rotation and xh = x rstd:
//   dg += sum u xh,   dx = rstd (g u - xh mean(xh g u)).
// A head is read once into registers, so both directions move each element once; they are bound
// by HBM (bf16: 4 bytes an element forward, 10 backward).
#include "sbp_internal.cuh"

namespace sbp {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxPairs = 4;   // pairs (j, j + hd / 2) of one lane: hd <= 256

inline int64_t nblk(int64_t n, int64_t t) { return (n + t - 1) / t; }

struct RowMap {      // rows are below 2^30, so their division is a 32-bit one
  const int* positions;
  unsigned seq_len;
  int64_t pos0, table_len, k_T;
  __device__ __forceinline__ int64_t pos(int64_t r) const {
    return positions ? (int64_t)positions[r] : pos0 + (unsigned)r % seq_len;
  }
  // row of the keys' output that row r goes to
  __device__ __forceinline__ int64_t k_row(int64_t r) const {
    const unsigned b = (unsigned)r / seq_len;
    return k_T > 0 ? b * k_T + pos0 + ((unsigned)r - b * seq_len) : r;
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

// ---------------------------------------------------------------- vector path
// head_dim a multiple of 16 and 16-byte aligned rows: a lane holds 8 elements of the first half
// of a head and the 8 that they are rotated with, so the rotation needs no exchange and every
// access has 16 bytes.  `1 << lw` lanes share a head (8 at head_dim 128; the next power of two
// where hd / 16 is none, the lanes past the head's end idle).
struct Lanes {
  int j;            // first of the lane's elements in either half
  int sub, per;     // which of the warp's `per` heads
  bool in;          // the lane has elements
  __device__ __forceinline__ Lanes(int lane, int lw, int half)
      : j(8 * (lane & ((1 << lw) - 1))), sub(lane >> lw), per(32 >> lw), in(j < half) {}
};
__device__ __forceinline__ float lanes_sum(float v, int lw) {
  for (int o = 1; o < (1 << lw); o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A warp takes kFwdHeads x (heads per warp) heads of one row, all of their loads in flight
// together; the warps of a CTA take neighbouring items, which share the row's angles in L1.
constexpr int kFwdHeads = 2;
template <typename T>
__global__ void __launch_bounds__(kThreads)
qk_fwd_vec_kernel(int64_t rows, int hd, int lw, int q_items, int row_items, Heads<T> q,
                  Heads<T> k, RowMap map, const float* __restrict__ cosb,
                  const float* __restrict__ sinb, float eps) {
  const int half = hd / 2;
  const int64_t item0 = (int64_t)blockIdx.x * kWarps, r0 = item0 / row_items;
  const unsigned rem = (unsigned)(item0 - r0 * row_items) + (threadIdx.x >> 5);
  const int64_t r = r0 + rem / (unsigned)row_items;
  int it = rem % (unsigned)row_items;
  if (r >= rows) return;
  const bool is_k = it >= q_items;
  const Heads<T>& t = is_k ? k : q;
  if (is_k) it -= q_items;
  const Lanes ln(threadIdx.x & 31, lw, half);
  const int h0 = it * kFwdHeads * ln.per + ln.sub;
  float a[kFwdHeads][8], b[kFwdHeads][8];
#pragma unroll
  for (int u = 0; u < kFwdHeads; ++u) {
    const int h = h0 + u * ln.per;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[u][i] = b[u][i] = 0.f;
    if (ln.in && h < t.n) {
      const T* x = t.x + r * t.ldx + (int64_t)h * hd + ln.j;
      load8(x, a[u]);
      load8(x + half, b[u]);
    }
  }
  const int64_t p = map.pos(r);
  const bool ok = p >= 0 && p < map.table_len;
  float c[8], s[8], ga[8], gb[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = s[i] = ga[i] = gb[i] = 0.f;
  if (ln.in && ok) {
    load8(cosb + p * half + ln.j, c);
    load8(sinb + p * half + ln.j, s);
    load8(t.g + ln.j, ga);
    load8(t.g + ln.j + half, gb);
  }
  T* yr = t.y + (is_k ? map.k_row(r) : r) * t.ldy;
#pragma unroll
  for (int u = 0; u < kFwdHeads; ++u) {
    const int h = h0 + u * ln.per;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[u][i], a[u][i], fmaf(b[u][i], b[u][i], ss));
    const float rs = rsqrtf(lanes_sum(ss, lw) / (float)hd + eps);
    if (!ln.in || h >= t.n) continue;
    float y1[8], y2[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n1 = a[u][i] * rs * ga[i], n2 = b[u][i] * rs * gb[i];
      y1[i] = ok ? n1 * c[i] - n2 * s[i] : 0.f;
      y2[i] = ok ? n2 * c[i] + n1 * s[i] : 0.f;
    }
    store8(yr + (int64_t)h * hd + ln.j, y1);
    store8(yr + (int64_t)h * hd + ln.j + half, y2);
  }
}

// Blocks [0, q_blocks) take the queries, the others the keys.  Warps take items of `per` heads
// of one row in turn and keep the gain gradient of their elements in registers; the block's sum
// goes to partial[block].
template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
qk_bwd_vec_kernel(int64_t rows, int hd, int lw, int q_blocks, Heads<T> q, Heads<T> k, RowMap map,
                  const float* __restrict__ cosb, const float* __restrict__ sinb, float eps,
                  float* __restrict__ partial) {
  __shared__ float red[kWarps][256];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, half = hd / 2;
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const Heads<T>& t = is_k ? k : q;
  const int64_t b0 = is_k ? blockIdx.x - q_blocks : blockIdx.x;
  const int64_t nb = is_k ? gridDim.x - q_blocks : q_blocks;
  const Lanes ln(lane, lw, half);
  const int row_items = (t.n + ln.per - 1) / ln.per;
  float ga[8], gb[8], da[8], db[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) ga[i] = gb[i] = da[i] = db[i] = 0.f;
  if (ln.in) {
    load8(t.g + ln.j, ga);
    load8(t.g + ln.j + half, gb);
  }
  for (int64_t item = b0 * kWarps + wid; item < rows * row_items; item += nb * kWarps) {
    const int64_t r = item / row_items;
    const int h = (int)(item - r * row_items) * ln.per + ln.sub;
    const int64_t p = map.pos(r);
    const bool ok = p >= 0 && p < map.table_len;
    const bool in = ln.in && h < t.n;
    float a[8], b[8], u[8], v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = b[i] = u[i] = v[i] = 0.f;
    if (in && ok) {
      const T* x = t.x + r * t.ldx + (int64_t)h * hd + ln.j;
      const float* dy = t.dy + r * t.lddy + (int64_t)h * hd + ln.j;
      float c[8], s[8], d1[8], d2[8];
      load8(x, a);
      load8(x + half, b);
      load8(dy, d1);
      load8(dy + half, d2);
      load8(cosb + p * half + ln.j, c);
      load8(sinb + p * half + ln.j, s);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = d1[i] * c[i] + d2[i] * s[i];
        v[i] = d2[i] * c[i] - d1[i] * s[i];
      }
    }
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
    const float rs = rsqrtf(lanes_sum(ss, lw) / (float)hd + eps);
    if (in && ok) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] *= rs;
        b[i] *= rs;
        da[i] = fmaf(u[i], a[i], da[i]);
        db[i] = fmaf(v[i], b[i], db[i]);
        u[i] *= ga[i];
        v[i] *= gb[i];
        dot = fmaf(a[i], u[i], fmaf(b[i], v[i], dot));
      }
    }
    dot = lanes_sum(dot, lw) / (float)hd;
    if (in) {
      float* dx = t.dx + r * t.lddx + (int64_t)h * hd + ln.j;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[i] = ok ? rs * (u[i] - a[i] * dot) : 0.f;
        v[i] = ok ? rs * (v[i] - b[i] * dot) : 0.f;
      }
      store8(dx, u);
      store8(dx + half, v);
    }
  }
  // the warp's heads, then the block's warps in order
  for (int o = 1 << lw; o < 32; o <<= 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      da[i] += __shfl_xor_sync(0xffffffffu, da[i], o);
      db[i] += __shfl_xor_sync(0xffffffffu, db[i], o);
    }
  }
  if (ln.sub == 0 && ln.in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      red[wid][ln.j + i] = da[i];
      red[wid][ln.j + half + i] = db[i];
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

// ---------------------------------------------------------------- any even head_dim, any stride
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

// dst[c] += sum of the blocks' partials (CTA 0: queries, CTA 1: keys).  Four threads share a
// column, each adds a quarter of the partials, and the first adds the four sums in order.
constexpr int kGainThreads = 1024;
__global__ void __launch_bounds__(kGainThreads)
qk_gain_kernel(int hd, int q_blocks, int blocks, const float* __restrict__ partial,
               float* __restrict__ dq_g, float* __restrict__ dk_g) {
  __shared__ float red[4][256];
  const int b0 = blockIdx.x ? q_blocks : 0, b1 = blockIdx.x ? blocks : q_blocks;
  float* dst = blockIdx.x ? dk_g : dq_g;
  const int c = threadIdx.x % 256, part = threadIdx.x / 256;
  const int per = (b1 - b0 + 3) / 4, e = min(b1, b0 + (part + 1) * per);
  if (c < hd) {
    float s = 0.f;
#pragma unroll 8
    for (int b = b0 + part * per; b < e; ++b) s += partial[(int64_t)b * hd + c];
    red[part][c] = s;
  }
  __syncthreads();
  if (part == 0 && c < hd) dst[c] += red[0][c] + red[1][c] + red[2][c] + red[3][c];
}

// blocks of the backward for the queries and the keys, in proportion to their items; the cap is
// two resident CTAs per SM, all in one wave
void bwd_blocks(const QkNorm& a, int& qb, int& kb) {
  const int64_t cap = (int64_t)sm_count() * 2;
  const int64_t qi = nblk(a.rows * a.q.n, kWarps), ki = nblk(a.rows * a.k.n, kWarps);
  if (qi + ki <= cap) {
    qb = (int)qi;
    kb = (int)ki;
  } else {
    kb = a.k.n ? (int)imax(1, cap * ki / (qi + ki)) : 0;
    qb = (int)(cap - kb);
  }
}

// log2 of the lanes that share a head on the vector path
int lanes_log2(int64_t hd) {
  int lw = 0;
  while ((16 << lw) < hd) ++lw;
  return lw;
}

// whether the vector path takes this tensor (see qk_fwd_vec_kernel)
bool vec_ok(const QkNormHeads& h, int dt, bool backward) {
  auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
  if (h.n == 0) return true;
  const int64_t unit = dt == DT_BF16 ? 8 : 4;
  if (!al(h.x) || !al(h.g) || h.ldx % unit) return false;
  if (backward) return al(h.dy) && al(h.dx) && h.lddy % 4 == 0 && h.lddx % 4 == 0;
  return al(h.y) && h.ldy % unit == 0;
}
bool vec_ok(const QkNorm& a, bool backward) {
  return a.hd % 16 == 0 && vec_ok(a.q, a.dt, backward) && vec_ok(a.k, a.dt, backward);
}

template <typename T>
Heads<T> heads_of(const QkNormHeads& h) {
  return Heads<T>{(int)h.n, static_cast<const T*>(h.x), h.ldx, static_cast<const T*>(h.g),
                  static_cast<T*>(h.y), h.ldy, h.dy, h.lddy, h.dx, h.lddx};
}
RowMap map_of(const QkNorm& a) {
  return RowMap{a.positions, (unsigned)imin(a.seq_len, (int64_t)1 << 30), a.pos0, a.table_len,
                a.k_T};
}

template <typename T>
cudaError_t fwd(const QkNorm& a, cudaStream_t st) {
  if (vec_ok(a, false)) {
    const int lw = lanes_log2(a.hd);
    const int64_t per = kFwdHeads * (32 >> lw);
    const int64_t qi = nblk(a.q.n, per), ki = nblk(a.k.n, per);
    launch(qk_fwd_vec_kernel<T>, dim3((unsigned)nblk(a.rows * (qi + ki), kWarps)),
           dim3(kThreads), 0, st, a.rows, (int)a.hd, lw, (int)qi, (int)(qi + ki),
           heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb, a.eps);
    return cudaGetLastError();
  }
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
  if (vec_ok(a, true))
    launch(qk_bwd_vec_kernel<T>, dim3(qb + kb), dim3(kThreads), 0, st, a.rows, (int)a.hd,
           lanes_log2(a.hd), qb, heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb,
           a.eps, partial);
  else
    launch(qk_bwd_kernel<T>, dim3(qb + kb), dim3(kThreads), 0, st, a.rows, (int)a.hd, qb,
         heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb, a.eps, partial);
  launch(qk_gain_kernel, dim3(kb ? 2 : 1), dim3(kGainThreads), 0, st, (int)a.hd, qb, qb + kb,
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
