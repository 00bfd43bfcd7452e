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
// 1 << kLw lanes share a head (8 at head_dim 128; the next power of two where hd / 16 is none).
// A lane holds 8 elements of the first half of a head and the 8 that they are rotated with, so
// the rotation needs no exchange.  The 8 are neighbours (kWide: one 16-byte access in bf16), or
// two groups of 4 a group of lanes apart: then the 16-byte accesses of neighbouring lanes to
// fp32 values lie side by side too (with 8 neighbours they touch half of each sector twice).
template <int kLw, bool kWide>
struct Lanes {
  static constexpr int per = 32 >> kLw;     // heads of a warp
  int sub;          // which of them
  int j0, j1;       // first elements of the lane's two groups of 4 in either half
  bool in0, in1;    // they lie in the head
  __device__ __forceinline__ Lanes(int lane, int half) : sub(lane >> kLw) {
    const int l = lane & ((1 << kLw) - 1);
    j0 = kWide ? 8 * l : 4 * l;
    j1 = kWide ? j0 + 4 : j0 + (4 << kLw);
    in0 = j0 < half;
    in1 = j1 < half;
  }
};
template <int kLw>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < (1 << kLw); o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Two fp32 values in a 64-bit register, for the two-wide fp32 instructions.  Both kernels were
// bounded by the instructions that they issue as much as by HBM (two thirds of the slots): these,
// no division per item and a width known to the compiler took the forward of 4096 x (32 + 8)
// heads of 128 from 23 to 19 us and the backward of 16384 x (28 + 4) from 130 to 118 us.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 pair(F2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 neg(F2 a) { return F2{a.v ^ 0x8000000080000000ull}; }
__device__ __forceinline__ float total(F2 a) {
  const float2 p = pair(a);
  return p.x + p.y;
}

// Four elements as they lie in memory, and as two pairs.
template <typename T>
struct alignas(4 * sizeof(T)) Pack {
  unsigned w[sizeof(T)];
};
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16>& x, F2* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    f[i] = f2(__uint_as_float(x.w[i] << 16), __uint_as_float(x.w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const Pack<float>& x, F2* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    f[i] = f2(__uint_as_float(x.w[2 * i]), __uint_as_float(x.w[2 * i + 1]));
}
__device__ __forceinline__ Pack<__nv_bfloat16> pack(const F2* f, __nv_bfloat16) {
  Pack<__nv_bfloat16> x;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(x.w);
#pragma unroll
  for (int i = 0; i < 2; ++i) h[i] = __float22bfloat162_rn(pair(f[i]));
  return x;
}
__device__ __forceinline__ Pack<float> pack(const F2* f, float) {
  Pack<float> x;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x.w[2 * i] = __float_as_uint(pair(f[i]).x);
    x.w[2 * i + 1] = __float_as_uint(pair(f[i]).y);
  }
  return x;
}

// A lane's 8 elements of one half of a head.
template <typename T>
struct Eight {
  Pack<T> lo, hi;
};
template <typename T, int kLw, bool kWide>
__device__ __forceinline__ Eight<T> load(const T* p, const Lanes<kLw, kWide>& ln) {
  Eight<T> x = {};
  if constexpr (kWide) {
    if (ln.in0) *reinterpret_cast<uint4*>(&x) = *reinterpret_cast<const uint4*>(p + ln.j0);
  } else {
    if (ln.in0) x.lo = *reinterpret_cast<const Pack<T>*>(p + ln.j0);
    if (ln.in1) x.hi = *reinterpret_cast<const Pack<T>*>(p + ln.j1);
  }
  return x;
}
// fp32 tables, whatever the lanes' layout
template <int kLw, bool kWide>
__device__ __forceinline__ void load_table(const float* p, const Lanes<kLw, kWide>& ln, F2 (&f)[4]) {
  Eight<float> x = {};
  if (ln.in0) x.lo = *reinterpret_cast<const Pack<float>*>(p + ln.j0);
  if (ln.in1) x.hi = *reinterpret_cast<const Pack<float>*>(p + ln.j1);
  unpack(x.lo, f);
  unpack(x.hi, f + 2);
}
template <typename T>
__device__ __forceinline__ void unpack(const Eight<T>& x, F2 (&f)[4]) {
  unpack(x.lo, f);
  unpack(x.hi, f + 2);
}
template <typename T, int kLw, bool kWide>
__device__ __forceinline__ void store(T* p, const Lanes<kLw, kWide>& ln, const F2 (&f)[4]) {
  Eight<T> x;
  x.lo = pack(f, T());
  x.hi = pack(f + 2, T());
  if constexpr (kWide) {
    if (ln.in0) *reinterpret_cast<uint4*>(p + ln.j0) = *reinterpret_cast<const uint4*>(&x);
  } else {
    if (ln.in0) *reinterpret_cast<Pack<T>*>(p + ln.j0) = x.lo;
    if (ln.in1) *reinterpret_cast<Pack<T>*>(p + ln.j1) = x.hi;
  }
}

template <typename T>
constexpr bool kFwdWide = sizeof(T) == 2;

// A warp takes U x (heads per warp) heads of one row (2 x 4 in bf16 at head_dim 128), all of
// their loads in flight together and held as they came until their turn; the warps of a CTA take
// neighbouring items, which share the row's angles in L1.  Gain and angle are multiplied once per
// row, so a pair costs y1 = rs (a (g c) - b (g' s)), y2 = rs (b (g' c) + a (g s)).
template <typename T>
constexpr int kFwdHeads = 4 / sizeof(T);
template <typename T, int U, int kLw>
__global__ void __launch_bounds__(kThreads, 3)
qk_fwd_vec_kernel(unsigned rows, int hd, float inv_hd, unsigned q_items, unsigned row_items, Heads<T> q,
                  Heads<T> k, RowMap map, const float* __restrict__ cosb,
                  const float* __restrict__ sinb, float eps) {
  const int half = hd / 2;
  const unsigned item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const unsigned r = item / row_items;
  unsigned it = item - r * row_items;
  if (r >= rows) return;
  const bool is_k = it >= q_items;
  const Heads<T>& t = is_k ? k : q;
  if (is_k) it -= q_items;
  const Lanes<kLw, kFwdWide<T>> ln(threadIdx.x & 31, half);
  const int h0 = it * U * ln.per + ln.sub, step = ln.per * hd;
  const T* x = t.x + r * t.ldx + (int64_t)h0 * hd;
  Eight<T> a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (h0 + u * ln.per < t.n) {
      a[u] = load(x + u * step, ln);
      b[u] = load(x + u * step + half, ln);
    } else {
      a[u] = b[u] = Eight<T>{};
    }
  }
  T* y = t.y + (is_k ? map.k_row(r) : r) * t.ldy + (int64_t)h0 * hd;
  const int64_t p = map.pos(r);
  F2 gc[4], gs[4], hc[4], hs[4];       // g c, -g' s, g' c, g s
  if (p < 0 || p >= map.table_len) {   // the whole warp: it is the row's position
#pragma unroll
    for (int i = 0; i < 4; ++i) gc[i] = f2(0.f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u * ln.per < t.n) {
        store(y + u * step, ln, gc);
        store(y + u * step + half, ln, gc);
      }
    }
    return;
  }
  F2 c[4], s[4];
  load_table(cosb + p * half, ln, c);
  load_table(sinb + p * half, ln, s);
  unpack(load(t.g, ln), gc);
  unpack(load(t.g + half, ln), hc);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hs[i] = gc[i] * s[i];
    gs[i] = neg(hc[i] * s[i]);
    gc[i] = gc[i] * c[i];
    hc[i] = hc[i] * c[i];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    F2 fa[4], fb[4], s2 = f2(0.f);
    unpack(a[u], fa);
    unpack(b[u], fb);
#pragma unroll
    for (int i = 0; i < 4; ++i) s2 = fma2(fa[i], fa[i], fma2(fb[i], fb[i], s2));
    const F2 rs = f2(rsqrtf(fmaf(lanes_sum<kLw>(total(s2)), inv_hd, eps)));
    if (h0 + u * ln.per >= t.n) continue;
    F2 y1[4], y2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y1[i] = fma2(fa[i], gc[i], fb[i] * gs[i]) * rs;
      y2[i] = fma2(fb[i], hc[i], fa[i] * hs[i]) * rs;
    }
    store(y + u * step, ln, y1);
    store(y + u * step + half, ln, y2);
  }
}

// Backward.  Blocks [0, q_blocks) take the queries, the others the keys.  Warps take items of
// `per` heads of one row in turn and keep the gain gradient of their elements in registers; the
// block's sum goes to partial[block].
template <typename T, int kLw>
__global__ void __launch_bounds__(kThreads, 2)
qk_bwd_vec_kernel(int rows, int hd, float inv_hd, int q_blocks, Heads<T> q, Heads<T> k,
                  RowMap map, const float* __restrict__ cosb, const float* __restrict__ sinb,
                  float eps, float* __restrict__ partial) {
  __shared__ float red[kWarps][256];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, half = hd / 2;
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const Heads<T>& t = is_k ? k : q;
  const int first = (is_k ? blockIdx.x - q_blocks : blockIdx.x) * kWarps + wid;
  const int stride = (is_k ? gridDim.x - q_blocks : q_blocks) * kWarps;
  const Lanes<kLw, false> ln(lane, half);
  // item `first`, and the step to the warp's next item, as row and item of the row
  const int row_items = (t.n + ln.per - 1) / ln.per;
  const int step_r = stride / row_items, step_it = stride - step_r * row_items;
  int r = first / row_items, it = first - r * row_items;
  F2 ga[4], gb[4], da[4], db[4];
  unpack(load(t.g, ln), ga);
  unpack(load(t.g + half, ln), gb);
#pragma unroll
  for (int i = 0; i < 4; ++i) da[i] = db[i] = f2(0.f);
  while (r < rows) {
    const int h = it * ln.per + ln.sub;
    const int64_t p = map.pos(r);
    const bool ok = p >= 0 && p < map.table_len, in = h < t.n;
    F2 a[4], b[4], u[4], v[4], s2 = f2(0.f);
    if (in && ok) {
      const T* x = t.x + r * t.ldx + h * hd;
      const float* dy = t.dy + r * t.lddy + h * hd;
      const Eight<T> xa = load(x, ln), xb = load(x + half, ln);
      const Eight<float> d1p = load(dy, ln), d2p = load(dy + half, ln);
      F2 c[4], s[4], d1[4], d2[4];
      load_table(cosb + p * half, ln, c);
      load_table(sinb + p * half, ln, s);
      unpack(xa, a);
      unpack(xb, b);
      unpack(d1p, d1);
      unpack(d2p, d2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = fma2(d1[i], c[i], d2[i] * s[i]);
        v[i] = fma2(d2[i], c[i], neg(d1[i] * s[i]));
        s2 = fma2(a[i], a[i], fma2(b[i], b[i], s2));
      }
    }
    const float rs = rsqrtf(fmaf(lanes_sum<kLw>(total(s2)), inv_hd, eps));
    F2 dot2 = f2(0.f);
    if (in && ok) {
      const F2 r2 = f2(rs);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = a[i] * r2;
        b[i] = b[i] * r2;
        da[i] = fma2(u[i], a[i], da[i]);
        db[i] = fma2(v[i], b[i], db[i]);
        u[i] = u[i] * ga[i];
        v[i] = v[i] * gb[i];
        dot2 = fma2(a[i], u[i], fma2(b[i], v[i], dot2));
      }
    }
    const float dot = lanes_sum<kLw>(total(dot2)) * inv_hd;
    if (in) {
      float* dx = t.dx + r * t.lddx + h * hd;
      const F2 r2 = f2(rs), m = f2(-dot);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        u[i] = ok ? fma2(a[i], m, u[i]) * r2 : f2(0.f);
        v[i] = ok ? fma2(b[i], m, v[i]) * r2 : f2(0.f);
      }
      store(dx, ln, u);
      store(dx + half, ln, v);
    }
    r += step_r;
    it += step_it;
    if (it >= row_items) {
      it -= row_items;
      ++r;
    }
  }
  // the warp's heads, then the block's warps in order
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 p = pair(da[i]), o = pair(db[i]);
    #pragma unroll
    for (int x = 1 << kLw; x < 32; x <<= 1) {
      p.x += __shfl_xor_sync(0xffffffffu, p.x, x);
      p.y += __shfl_xor_sync(0xffffffffu, p.y, x);
      o.x += __shfl_xor_sync(0xffffffffu, o.x, x);
      o.y += __shfl_xor_sync(0xffffffffu, o.y, x);
    }
    const int j = (i < 2 ? ln.j0 : ln.j1) + 2 * (i & 1);
    if (ln.sub == 0 && (i < 2 ? ln.in0 : ln.in1)) {
      red[wid][j] = p.x;
      red[wid][j + 1] = p.y;
      red[wid][j + half] = o.x;
      red[wid][j + half + 1] = o.y;
    }
  }
  __syncthreads();
  for (int col = threadIdx.x; col < hd; col += kThreads) {
    float sum = red[0][col];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) sum += red[i][col];
    partial[(int64_t)blockIdx.x * hd + col] = sum;
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

// dst[c] += sum of the blocks' partials, 32 columns of the queries' (y = 0) or the keys' (y = 1)
// gain per CTA: each warp adds a 32nd of the partials, warp 0 the 32 sums in order.
__global__ void __launch_bounds__(1024)
qk_gain_kernel(int hd, int q_blocks, int blocks, const float* __restrict__ partial,
               float* __restrict__ dq_g, float* __restrict__ dk_g) {
  __shared__ float red[32][33];
  const int b0 = blockIdx.y ? q_blocks : 0, b1 = blockIdx.y ? blocks : q_blocks;
  float* dst = blockIdx.y ? dk_g : dq_g;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < hd) {
#pragma unroll 8
    for (int b = b0 + wid; b < b1; b += 32) s += partial[(int64_t)b * hd + c];
  }
  red[wid][lane] = s;
  __syncthreads();
  if (wid != 0 || c >= hd) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) s += red[w][lane];
  dst[c] += s;
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
  return a.hd % (a.dt == DT_BF16 && !backward ? 16 : 8) == 0 && vec_ok(a.q, a.dt, backward) && vec_ok(a.k, a.dt, backward);
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

template <typename T, int kLw>
void launch_fwd_vec(const QkNorm& a, cudaStream_t st) {
  constexpr int U = kFwdHeads<T>, per = U * (32 >> kLw);
  const int64_t qi = nblk(a.q.n, per), ki = nblk(a.k.n, per);
  launch(qk_fwd_vec_kernel<T, U, kLw>, dim3((unsigned)nblk(a.rows * (qi + ki), kWarps)),
         dim3(kThreads), 0, st, (unsigned)a.rows, (int)a.hd, 1.f / a.hd, (unsigned)qi,
         (unsigned)(qi + ki), heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb,
         a.eps);
}

template <typename T, int kLw>
void launch_bwd_vec(const QkNorm& a, int qb, int kb, float* partial, cudaStream_t st) {
  launch(qk_bwd_vec_kernel<T, kLw>, dim3(qb + kb), dim3(kThreads), 0, st, (int)a.rows, (int)a.hd,
         1.f / a.hd, qb, heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb, a.eps,
         partial);
}

template <typename T>
cudaError_t fwd(const QkNorm& a, cudaStream_t st) {
  if (vec_ok(a, false)) {
    switch (lanes_log2(a.hd)) {
      case 0: launch_fwd_vec<T, 0>(a, st); break;
      case 1: launch_fwd_vec<T, 1>(a, st); break;
      case 2: launch_fwd_vec<T, 2>(a, st); break;
      case 3: launch_fwd_vec<T, 3>(a, st); break;
      default: launch_fwd_vec<T, 4>(a, st);
    }
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
  if (vec_ok(a, true)) {
    switch (lanes_log2(a.hd)) {
      case 0: launch_bwd_vec<T, 0>(a, qb, kb, partial, st); break;
      case 1: launch_bwd_vec<T, 1>(a, qb, kb, partial, st); break;
      case 2: launch_bwd_vec<T, 2>(a, qb, kb, partial, st); break;
      case 3: launch_bwd_vec<T, 3>(a, qb, kb, partial, st); break;
      default: launch_bwd_vec<T, 4>(a, qb, kb, partial, st);
    }
  } else {
    launch(qk_bwd_kernel<T>, dim3(qb + kb), dim3(kThreads), 0, st, a.rows, (int)a.hd, qb,
           heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb, a.eps, partial);
  }
  launch(qk_gain_kernel, dim3((unsigned)nblk(a.hd, 32), kb ? 2 : 1), dim3(1024), 0, st,
         (int)a.hd, qb, qb + kb, (const float*)partial, dq_g, dk_g);
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
