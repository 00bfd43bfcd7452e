// Per-head RMS norm of queries and keys with the rotate-half RoPE in the same pass, forward and
// backward.  For one head x of hd elements at position p (h = hd / 2):
//   n = x rstd g,  rstd = 1 / sqrt(mean(x^2) + eps)
//   y_j = n_j c_j - n_{j+h} s_j,  y_{j+h} = n_{j+h} c_j + n_j s_j
// and for an upstream gradient dy, with u its inverse rotation and xh = x rstd:
//   dg += sum u xh,   dx = rstd (g u - xh mean(xh g u)).
// A head is read once into registers, so both directions move each element once; they are bound
// by HBM (bf16: 4 bytes an element forward, 10 backward).
#include <type_traits>

#include "sbp_internal.cuh"

namespace sbp {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;

inline int64_t nblk(int64_t n, int64_t t) { return (n + t - 1) / t; }

struct RowMap {      // rows are below 2^30, so their division is a 32-bit one
  const int* positions;
  unsigned seq_len;
  int64_t pos0, table_len, k_T;
  __device__ __forceinline__ int64_t pos(int r) const {
    return positions ? (int64_t)positions[r] : pos0 + (unsigned)r % seq_len;
  }
  // row of the keys' output that row r goes to
  __device__ __forceinline__ int64_t k_row(int r) const {
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

// kN lanes share a head: a power of two (8 at head_dim 128; the next one where hd / 16 is none), but
// 5 and 6 for heads of 65 to 96 in the vector layouts: a warp takes 6 or 5 heads there, 4 with 8
// lanes a head.  16384 x (28 + 4) heads, us, with 8 lanes behind the stroke:
//              72          80           88          96
//   fwd bf16   -           42.0 / 46.5  -           43.1 / 47.6
//   fwd fp32   49.9 / 57.8 53.4 / 60.2  59.2 / 63.7 62.3 / 65.7
//   bwd bf16   83.6 / 93.0 87.6 / 94.7  98.3 / 98.3 103.0 / 100.7
//   bwd fp32   80.8 / 97.4 85.5 / 101   95.1 / 105  100.5 / 108
// Heads of 48 gain nothing from 3 lanes (fp32 forward 45 us, 37 with 4).  9 and 10 lanes for heads to
// 160 would take 3 heads for 2; they need kernels of their own.
// A lane holds 8 elements of the first half of a head and the 8 that they are rotated with, so
// the rotation needs no exchange.  Which 8:
//   kWide    neighbours: one 16-byte access in bf16
//   kSplit   two groups of 4, a group of lanes apart: the 16-byte accesses of neighbouring lanes
//            to fp32 values lie side by side too (8 neighbours touch half of each sector twice)
//   kScalar  every kN-th element, one by one: any even head_dim, any alignment
enum Layout { kWide, kSplit, kScalar };
template <int kN, Layout kL>
struct Lanes {
  static constexpr int per = 32 / kN;       // heads of a warp
  int sub, l, half;                         // which of them (per: a lane left over), the lane in it
  __device__ __forceinline__ Lanes(int lane, int half_)
      : sub(lane / kN), l(lane % kN), half(half_) {}
  // the lane's e-th element of either half
  __device__ __forceinline__ int at(int e) const {
    if constexpr (kL == kWide) return 8 * l + e;
    if constexpr (kL == kSplit) return 4 * l + e + (e < 4 ? 0 : 4 * kN - 4);
    return l + e * kN;
  }
  __device__ __forceinline__ bool in(int e) const { return at(e) < half; }
  __device__ __forceinline__ bool left_over() const { return 32 % kN != 0 && sub == per; }
  // the sum over the lanes of the head
  __device__ __forceinline__ float sum(float v) const {
    if constexpr ((kN & (kN - 1)) == 0) {
#pragma unroll
      for (int o = 1; o < kN; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    }
    // v becomes the sum of w lanes from the own one on; those of kN's bits are strung together
    auto from = [&](float x, int k) {
      const int j = l + k;
      return __shfl_sync(0xffffffffu, x, sub * kN + (j < kN ? j : j - kN));
    };
    float s = 0.f;
    int have = 0;
#pragma unroll
    for (int w = 1; w <= kN; w <<= 1) {
      if (kN & w) {
        s += have ? from(v, have) : v;
        have += w;
      }
      if (2 * w <= kN) v += from(v, w);
    }
    return s;
  }
  // over the heads of the warp, for the lanes of the first
  __device__ __forceinline__ float sum_heads(float v) const {
    float s = v;
    if constexpr ((kN & (kN - 1)) == 0) {
#pragma unroll
      for (int x = kN; x < 32; x <<= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    } else {
#pragma unroll
      for (int h = 1; h < per; ++h) s += __shfl_down_sync(0xffffffffu, v, h * kN);
    }
    return s;
  }
};

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
  T v[4];
};
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16>& x, F2* f) {
  const unsigned* w = reinterpret_cast<const unsigned*>(x.v);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const Pack<float>& x, F2* f) {
  f[0] = f2(x.v[0], x.v[1]);
  f[1] = f2(x.v[2], x.v[3]);
}
__device__ __forceinline__ void pack(const F2* f, Pack<__nv_bfloat16>& x) {
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(x.v);
#pragma unroll
  for (int i = 0; i < 2; ++i) h[i] = __float22bfloat162_rn(pair(f[i]));
}
__device__ __forceinline__ void pack(const F2* f, Pack<float>& x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x.v[2 * i] = pair(f[i]).x;
    x.v[2 * i + 1] = pair(f[i]).y;
  }
}

// A lane's 8 elements of one half of a head; zeros past the half's end.
template <typename T>
struct alignas(16) Eight {
  Pack<T> lo, hi;
};
template <typename T, int kN, Layout kL>
__device__ __forceinline__ Eight<T> load(const T* p, const Lanes<kN, kL>& ln) {
  Eight<T> x = {};
  if constexpr (kL == kWide && sizeof(T) == 2) {
    if (ln.in(0)) *reinterpret_cast<uint4*>(&x) = *reinterpret_cast<const uint4*>(p + ln.at(0));
  } else if constexpr (kL != kScalar) {
    if (ln.in(0)) x.lo = *reinterpret_cast<const Pack<T>*>(p + ln.at(0));
    if (ln.in(4)) x.hi = *reinterpret_cast<const Pack<T>*>(p + ln.at(4));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (ln.in(e)) (e < 4 ? x.lo : x.hi).v[e & 3] = p[ln.at(e)];
  }
  return x;
}
template <typename T>
__device__ __forceinline__ void unpack(const Eight<T>& x, F2 (&f)[4]) {
  unpack(x.lo, f);
  unpack(x.hi, f + 2);
}
template <typename T, int kN, Layout kL>
__device__ __forceinline__ void store(T* p, const Lanes<kN, kL>& ln, const F2 (&f)[4]) {
  Eight<T> x;
  pack(f, x.lo);
  pack(f + 2, x.hi);
  if constexpr (kL == kWide && sizeof(T) == 2) {
    if (ln.in(0)) *reinterpret_cast<uint4*>(p + ln.at(0)) = *reinterpret_cast<const uint4*>(&x);
  } else if constexpr (kL != kScalar) {
    if (ln.in(0)) *reinterpret_cast<Pack<T>*>(p + ln.at(0)) = x.lo;
    if (ln.in(4)) *reinterpret_cast<Pack<T>*>(p + ln.at(4)) = x.hi;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (ln.in(e)) p[ln.at(e)] = (e < 4 ? x.lo : x.hi).v[e & 3];
  }
}

// Forward.  U = 1: the heads of all rows are one list, of which a warp takes `per` neighbours.
// U = 2: a warp takes up to 2 x per heads of one row, all of their loads in flight together and
// held as they came until their turn (4096 rows of 32 + 8 heads of 128: 17.3 us, 25 with U = 1).
// Gain and angle are multiplied once per row, so a pair of elements costs
//   y1 = rs (a (g c) - b (g' s)),  y2 = rs (b (g' c) + a (g s)).
// Small CTAs fill the SM's places sooner, and as many warps as the registers of their loads leave
// room for hide more of the latency (16384 x (28 + 4) heads of 128 in bf16: 28 warps per SM 50.4
// us, 24 53.7; U = 1, heads of 80: 32 warps 42.0, 24 48.3; scalar bf16, heads of 102: 28 warps 88,
// 32 97).
constexpr int kFwdThreads = 64, kFwdWarps = kFwdThreads / 32;
template <typename T, int U, Layout kL>
constexpr int fwd_blocks() {
  return U == 1 && (kL != kScalar || sizeof(T) == 4) ? 16 : 14;
}
template <typename T, int U, int kN, Layout kL>
__global__ void __launch_bounds__(kFwdThreads, (fwd_blocks<T, U, kL>()))
qk_fwd_kernel(int rows, int hd, float inv_hd, unsigned q_warps, unsigned warps, Heads<T> q,
              Heads<T> k, RowMap map, const float* __restrict__ cosb,
              const float* __restrict__ sinb, float eps) {
  const int half = hd / 2;
  unsigned item = blockIdx.x * kFwdWarps + (threadIdx.x >> 5);
  if (item >= warps) return;
  const bool is_k = item >= q_warps;
  const Heads<T>& t = is_k ? k : q;
  if (is_k) item -= q_warps;
  const Lanes<kN, kL> ln(threadIdx.x & 31, half);
  // the lane's heads: h of row r, and with U = 2 also h + per of the same row
  int r, h;
  if constexpr (U == 1) {
    const unsigned first = item * ln.per;
    r = first / (unsigned)t.n;
    h = first - (unsigned)r * t.n + ln.sub;
    if (h >= t.n) {        // a division only where a row ends
      const int more = (unsigned)h / (unsigned)t.n;
      r += more;
      h -= more * t.n;
    }
  } else {
    const unsigned row_items = (unsigned)(t.n + U * ln.per - 1) / (U * ln.per);
    r = item / row_items;
    h = (item - (unsigned)r * row_items) * (U * ln.per) + ln.sub;
  }
  // heads of the lane: none behind the last row, one where the row has no second; places without
  // a head load the row's last one instead of branching, and store nothing
  const int have = r >= rows || ln.left_over() ? 0 : U == 1 || h + ln.per >= t.n ? (h < t.n) : U;
  r = min(r, rows - 1);
  const T* x = t.x + r * t.ldx;
  Eight<T> a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const T* xh = x + min(h + u * ln.per, t.n - 1) * hd;
    a[u] = load(xh, ln);
    b[u] = load(xh + half, ln);
  }
  const int64_t p = map.pos(r);
  const bool ok = p >= 0 && p < map.table_len;
  F2 gc[4], gs[4], hc[4], hs[4];       // g c, -g' s, g' c, g s
  if (ok) {
    F2 c[4], s[4];
    unpack(load(cosb + p * half, ln), c);
    unpack(load(sinb + p * half, ln), s);
    unpack(load(t.g, ln), gc);
    unpack(load(t.g + half, ln), hc);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      hs[i] = gc[i] * s[i];
      gs[i] = neg(hc[i] * s[i]);
      gc[i] = gc[i] * c[i];
      hc[i] = hc[i] * c[i];
    }
  }
  T* y = t.y + (is_k ? map.k_row(r) : r) * t.ldy + h * hd;
  const int step = ln.per * hd;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    F2 fa[4], fb[4], s2 = f2(0.f);
    unpack(a[u], fa);
    unpack(b[u], fb);
#pragma unroll
    for (int i = 0; i < 4; ++i) s2 = fma2(fa[i], fa[i], fma2(fb[i], fb[i], s2));
    const F2 rs = f2(rsqrtf(fmaf(ln.sum(total(s2)), inv_hd, eps)));
    if (u >= have) continue;
    if (ok) {
      F2 y1[4], y2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y1[i] = fma2(fa[i], gc[i], fb[i] * gs[i]) * rs;
        y2[i] = fma2(fb[i], hc[i], fa[i] * hs[i]) * rs;
      }
      store(y + u * step, ln, y1);
      store(y + u * step + half, ln, y2);
    } else {
      const F2 zero[4] = {};
      store(y + u * step, ln, zero);
      store(y + u * step + half, ln, zero);
    }
  }
}

// Backward.  Blocks [0, q_blocks) take the queries, the others the keys.  Warps take `per`
// neighbours of the list of heads in turn and keep the gain gradient of their elements in
// registers; the block's sum goes to partial[block].  One wave of CTAs: 20 warps per SM where the
// registers of their loads leave room (16384 x (28 + 4) heads of 128: bf16 111 us, 115 with 16;
// fp32 136, 125 with 16).
constexpr int kBwdBlocks = 5;
constexpr int bwd_blocks_per_sm(bool bf16, bool vec) { return bf16 && vec ? kBwdBlocks : 4; }
template <typename T, int kN, Layout kL>
__global__ void __launch_bounds__(kThreads, bwd_blocks_per_sm(sizeof(T) == 2, kL != kScalar))
qk_bwd_kernel(int rows, int hd, float inv_hd, int q_blocks, Heads<T> q, Heads<T> k, RowMap map,
              const float* __restrict__ cosb, const float* __restrict__ sinb, float eps,
              float* __restrict__ partial) {
  __shared__ float red[kWarps][256];
  release_next();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, half = hd / 2;
  const bool is_k = (int)blockIdx.x >= q_blocks;
  const Heads<T>& t = is_k ? k : q;
  const Lanes<kN, kL> ln(lane, half);
  const int warp = (is_k ? blockIdx.x - q_blocks : blockIdx.x) * kWarps + wid;
  const int stride = (is_k ? gridDim.x - q_blocks : q_blocks) * kWarps * ln.per;
  // the lane's first head, and the step to its next one, as row and head of the row
  const int first = warp * ln.per + ln.sub, step_r = stride / t.n, step_h = stride - step_r * t.n;
  int r = first / t.n, h = first - r * t.n;
  if (ln.left_over()) r = rows;
  F2 ga[4], gb[4], da[4], db[4];
  unpack(load(t.g, ln), ga);
  unpack(load(t.g + half, ln), gb);
#pragma unroll
  for (int i = 0; i < 4; ++i) da[i] = db[i] = f2(0.f);
  while (__any_sync(0xffffffffu, r < rows)) {
    const bool in = r < rows;
    bool ok = false;
    F2 a[4], b[4], u[4], v[4], s2 = f2(0.f);
    if (in) {
      const int64_t p = map.pos(r);
      ok = p >= 0 && p < map.table_len;
      if (ok) {
        const T* x = t.x + r * t.ldx + h * hd;
        const float* dy = t.dy + r * t.lddy + h * hd;
        const Eight<T> xa = load(x, ln), xb = load(x + half, ln);
        const Eight<float> d1p = load(dy, ln), d2p = load(dy + half, ln);
        F2 c[4], s[4], d1[4], d2[4];
        unpack(load(cosb + p * half, ln), c);
        unpack(load(sinb + p * half, ln), s);
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
    }
    const float rs = rsqrtf(fmaf(ln.sum(total(s2)), inv_hd, eps));
    F2 dot2 = f2(0.f);
    if (ok) {
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
    const float dot = ln.sum(total(dot2)) * inv_hd;
    if (in) {
      float* dx = t.dx + r * t.lddx + h * hd;
      const F2 r2 = f2(rs), m = f2(-dot);
      F2 o1[4] = {}, o2[4] = {};
      if (ok) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o1[i] = fma2(a[i], m, u[i]) * r2;
          o2[i] = fma2(b[i], m, v[i]) * r2;
        }
      }
      store(dx, ln, o1);
      store(dx + half, ln, o2);
    }
    r += step_r;
    h += step_h;
    if (h >= t.n) {
      h -= t.n;
      ++r;
    }
  }
  // the warp's heads, then the block's warps in order
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 da2 = pair(da[i]), db2 = pair(db[i]);
    const float2 p = make_float2(ln.sum_heads(da2.x), ln.sum_heads(da2.y));
    const float2 o = make_float2(ln.sum_heads(db2.x), ln.sum_heads(db2.y));
    if (ln.sub == 0 && ln.in(2 * i)) {
      red[wid][ln.at(2 * i)] = p.x;
      red[wid][ln.at(2 * i) + half] = o.x;
    }
    if (ln.sub == 0 && ln.in(2 * i + 1)) {
      red[wid][ln.at(2 * i + 1)] = p.y;
      red[wid][ln.at(2 * i + 1) + half] = o.y;
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

// dst[c] += sum of the blocks' partials, 32 columns of the queries' (y = 0) or the keys' (y = 1)
// gain per CTA: each warp adds a 32nd of the partials, warp 0 the 32 sums in order.  Where both
// have one gradient, y = 0 adds the partials of all blocks.
__global__ void __launch_bounds__(1024)
qk_gain_kernel(int hd, int q_blocks, int blocks, const float* partial,
               float* __restrict__ dq_g, float* __restrict__ dk_g) {
  __shared__ float red[32][33];
  const int b0 = blockIdx.y ? q_blocks : 0, b1 = blockIdx.y ? blocks : q_blocks;
  float* dst = blockIdx.y ? dk_g : dq_g;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  await_previous();
  if (c < hd) {
    for (int b = b0 + wid; b < b1; b += 8 * 32) {      // eight loads in flight, always
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = b + 32 * i < b1 ? partial[(int64_t)(b + 32 * i) * hd + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
  }
  red[wid][lane] = s;
  __syncthreads();
  if (wid != 0 || c >= hd) return;
#pragma unroll
  for (int w = 1; w < 32; ++w) s += red[w][lane];
  dst[c] += s;
}

// lanes that share a head
int lanes_of(int64_t hd, bool vec) {
  if (vec && hd > 64 && hd <= 96) return (int)nblk(hd, 16);
  int n = 1;
  while (16 * n < hd) n *= 2;
  return n;
}

// whether the tensor's rows keep accesses of four elements (eight: bf16 forward) aligned
bool vec_ok(const QkNormHeads& h, int dt, bool backward) {
  auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
  if (h.n == 0) return true;
  const int64_t unit = dt == DT_BF16 ? 8 : 4;
  if (!al(h.x) || !al(h.g) || h.ldx % unit) return false;
  if (backward) return al(h.dy) && al(h.dx) && h.lddy % 4 == 0 && h.lddx % 4 == 0;
  return al(h.y) && h.ldy % unit == 0;
}
bool vec_ok(const QkNorm& a, bool backward) {
  return a.hd % (a.dt == DT_BF16 && !backward ? 16 : 8) == 0 && vec_ok(a.q, a.dt, backward) &&
         vec_ok(a.k, a.dt, backward);
}

// blocks of the backward for the queries and the keys, in proportion to their heads; one wave
void bwd_blocks(const QkNorm& a, int& qb, int& kb) {
  const bool vec = vec_ok(a, true);
  const int64_t cap = (int64_t)sm_count() * bwd_blocks_per_sm(a.dt == DT_BF16, vec);
  const int64_t per = kWarps * (32 / lanes_of(a.hd, vec));
  const int64_t qi = nblk(a.rows * a.q.n, per), ki = nblk(a.rows * a.k.n, per);
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
  return RowMap{a.positions, (unsigned)imin(a.seq_len, (int64_t)1 << 30), a.pos0, a.table_len,
                a.k_T};
}

struct Backward {
  int qb, kb;
  float* partial;
};

template <typename T, int kN, Layout kL>
void launch_fwd(const QkNorm& a, const Backward&, cudaStream_t st) {
  constexpr int per = 32 / kN;
  auto go = [&](auto kernel, int64_t qw, int64_t kw) {
    launch(kernel, dim3((unsigned)nblk(qw + kw, kFwdWarps)), dim3(kFwdThreads), 0, st,
           (int)a.rows, (int)a.hd, 1.f / a.hd, (unsigned)qw, (unsigned)(qw + kw),
           heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb, a.sinb, a.eps);
  };
  if constexpr (kL == kWide) {
    // two heads per lane unless more than a fifth of the places would be empty
    const int64_t qi = nblk(a.q.n, 2 * per), ki = nblk(a.k.n, 2 * per);
    if (8 * per * (qi + ki) <= 5 * (a.q.n + a.k.n))
      return go(qk_fwd_kernel<T, 2, kN, kL>, a.rows * qi, a.rows * ki);
  }
  go(qk_fwd_kernel<T, 1, kN, kL>, nblk(a.rows * a.q.n, per), nblk(a.rows * a.k.n, per));
}

template <typename T, int kN, Layout kL>
void launch_bwd(const QkNorm& a, const Backward& b, cudaStream_t st) {
  launch(qk_bwd_kernel<T, kN, kL>, dim3(b.qb + b.kb), dim3(kThreads), 0, st, (int)a.rows,
         (int)a.hd, 1.f / a.hd, b.qb, heads_of<T>(a.q), heads_of<T>(a.k), map_of(a), a.cosb,
         a.sinb, a.eps, b.partial);
}

template <typename T, Layout kL, bool kBwd>
void launch_width(const QkNorm& a, const Backward& b, cudaStream_t st) {
  auto go = [&](auto lanes) {
    constexpr int kN = decltype(lanes)::value;
    if constexpr (kBwd)
      launch_bwd<T, kN, kL>(a, b, st);
    else
      launch_fwd<T, kN, kL>(a, b, st);
  };
  const int lanes = lanes_of(a.hd, kL != kScalar);
  if constexpr (kL != kScalar) {
    if (lanes == 5) return go(std::integral_constant<int, 5>());
    if (lanes == 6) return go(std::integral_constant<int, 6>());
  }
  switch (lanes) {
    case 1: return go(std::integral_constant<int, 1>());
    case 2: return go(std::integral_constant<int, 2>());
    case 4: return go(std::integral_constant<int, 4>());
    case 8: return go(std::integral_constant<int, 8>());
    default: return go(std::integral_constant<int, 16>());
  }
}

template <typename T, bool kBwd>
void launch_type(const QkNorm& a, const Backward& b, cudaStream_t st) {
  if (vec_ok(a, kBwd))
    launch_width<T, sizeof(T) == 2 && !kBwd ? kWide : kSplit, kBwd>(a, b, st);
  else
    launch_width<T, kScalar, kBwd>(a, b, st);
}

}  // namespace

cudaError_t qk_norm_rope_fwd(const QkNorm& a, cudaStream_t st) {
  if (a.dt == DT_BF16)
    launch_type<__nv_bfloat16, false>(a, {}, st);
  else
    launch_type<float, false>(a, {}, st);
  return cudaGetLastError();
}

size_t qk_norm_bwd_partial_floats(int64_t hd) { return (size_t)sm_count() * kBwdBlocks * hd; }

cudaError_t qk_norm_rope_bwd(const QkNorm& a, float* dq_g, float* dk_g, float* partial,
                             cudaStream_t st) {
  Backward b;
  bwd_blocks(a, b.qb, b.kb);
  b.partial = partial;
  if (a.dt == DT_BF16)
    launch_type<__nv_bfloat16, true>(a, b, st);
  else
    launch_type<float, true>(a, b, st);
  const bool apart = b.kb > 0 && dk_g != dq_g;
  launch_next(qk_gain_kernel, dim3((unsigned)nblk(a.hd, 32), apart ? 2 : 1), dim3(1024), 0, st,
         (int)a.hd, apart ? b.qb : b.qb + b.kb, b.qb + b.kb, (const float*)partial, dq_g, dk_g);
  return cudaGetLastError();
}

}  // namespace sbp
