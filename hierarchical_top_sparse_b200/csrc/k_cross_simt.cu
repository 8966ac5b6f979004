// k_cross_simt.cu -- cross attention on the CUDA cores (fp32 FMA), forward and
// backward, bf16 or fp32 tokens, any d up to 128.
//
//   z_ij = scale q_i . k_j over the batch row's valid keys,  P = softmax_j(z),
//   O = P V,  LSE_i = log sum_j exp z_ij;
//   D_i = dO_i . O_i,  dV = P^T dO,  dS = scale P o (dO V^T - D),
//   dQ = dS K,  dK = dS^T Q  (summed over the query heads that share a key head).
//
// 8 heads of 4096 queries and 4096 keys in fp32: forward 24 and 25 TFLOP/s (64 and 128
// channels: 1.42 and 2.74 ms), backward 27 and 25 of the seven products it computes
// (4.49 and 9.49 ms), a third of the FMA rate: two 16-byte shared-memory reads feed 16 FMAs,
// and no load is on its way during a product.  12 heads of 1024 queries and 77 keys, where
// the tiles fill the device once: 8 and 9 TFLOP/s.
//
// Tiles of 64 queries x 64 keys (32 queries in the dK / dV pass), 256 threads
// with 4 x 4 products each; both operands of a product stand in shared memory
// with the contracted index outermost, so that a step reads two float4 and
// does 16 FMAs.  The softmax runs online (one pass over the keys, running
// maximum and sum in registers).  Few tiles are made up for by splitting the
// other axis: keys in the forward and in dQ, queries in dK / dV; the splits'
// results are fp32 and joined in a fixed order, without atomics, so that a
// call gives the same bits every time.
#include <math.h>

#include "cross.cuh"

namespace llsa {
namespace cross {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int BM = 64, BN = 64, BQ = 32, THREADS = 256;
constexpr int LD = 68;         // row of 64 values and 4 of padding: spreads the transposed stores over the banks
constexpr int LQ = 36;         // row of 32 values and 4 of padding

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  __nv_bfloat162 lo = __floats2bfloat162_rn(x.x, x.y), hi = __floats2bfloat162_rn(x.z, x.w);
  uint2 w;
  w.x = *reinterpret_cast<uint32_t*>(&lo);
  w.y = *reinterpret_cast<uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p) = w;
}

// ROWS rows from row0 on as [channel][row] (leading dimension ld) and / or as
// [row][channel]; rows at or behind n, masked rows and channels at or behind d
// are zero.  Eight rows by four 4-channel chunks per warp: the transposed
// stores then meet two to a bank.
template <typename T, int DP, int ROWS>
__device__ __forceinline__ void load_tile(float* t, int ld, float* nrm, const T* base, int64_t stride, int row0, int n,
                                          int d, const uint8_t* mask) {
  constexpr int C4 = DP / 4, N = ROWS * C4 / THREADS;
  float4 x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {                          // all of a thread's loads first: one latency, not N
    const int i = threadIdx.x + k * THREADS;
    const int c = ((i >> 3) % C4) * 4, row = row0 + (i & 7) + 8 * ((i >> 3) / C4);
    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (row < n && c < d && (!mask || mask[row])) x[k] = load4(base + (int64_t)row * stride + c);
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const int i = threadIdx.x + k * THREADS;
    const int c = ((i >> 3) % C4) * 4, r = (i & 7) + 8 * ((i >> 3) / C4);
    if (t) {
      t[(c + 0) * ld + r] = x[k].x;
      t[(c + 1) * ld + r] = x[k].y;
      t[(c + 2) * ld + r] = x[k].z;
      t[(c + 3) * ld + r] = x[k].w;
    }
    if (nrm) store4(nrm + r * (DP + 4) + c, x[k]);
  }
}

template <int DP>
__device__ __forceinline__ void product_4x4(float acc[4][4], const float* a, const float* b) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll 8
  for (int c = 0; c < DP; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(a + c * LD);
    const float4 y = *reinterpret_cast<const float4*>(b + c * LD);
    const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
  }
}

// ------------------------------------------------------------------ forward

template <int DP>
struct FwdSmem {
  float qt[DP * LD], kt[DP * LD], vn[BN * (DP + 4)], pt[BN * LD];
};

template <typename T, int DP>
__global__ void __launch_bounds__(THREADS) fwd_kernel(const __grid_constant__ Geo g, Keys keys, int ks,
                                                      const T* __restrict__ q, const T* __restrict__ k,
                                                      const T* __restrict__ v, T* __restrict__ o,
                                                      float* __restrict__ lse, FwdWork part) {
  extern __shared__ __align__(16) unsigned char raw[];
  FwdSmem<DP>& s = *reinterpret_cast<FwdSmem<DP>*>(raw);
  const int nqt = (g.nq + BM - 1) / BM;
  const int split = (int)(blockIdx.x % ks);
  const int qt = (int)((blockIdx.x / ks) % nqt);
  const int bh = (int)(blockIdx.x / ks / nqt);
  const int b = bh / g.h, h = bh % g.h, hk = h / g.group;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const bool busy = qt * BM + (int)(threadIdx.x >> 5) * 8 < g.nq;    // of the warp's eight queries
  const int n = key_count(g, keys, b);
  const uint8_t* mask = keys.mask ? keys.mask + (int64_t)b * g.nk : nullptr;
  const int ntiles = (n + BN - 1) / BN;
  const int t0 = (int)((int64_t)ntiles * split / ks), t1 = (int)((int64_t)ntiles * (split + 1) / ks);
  const T* kb = k + b * g.k.b + hk * g.k.h;
  const T* vb = v + b * g.v.b + hk * g.v.h;
  const float sc2 = g.scale * kLog2e;
  load_tile<T, DP, BM>(s.qt, LD, nullptr, q + b * g.q.b + h * g.q.h, g.q.n, qt * BM, g.nq, g.d, nullptr);
  float m[4], l[4], acc[4][DP / 64][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int j = 0; j < DP / 64; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
  }
  for (int t = t0; t < t1; ++t) {
    const int key0 = t * BN;
    __syncthreads();
    load_tile<T, DP, BN>(s.kt, LD, nullptr, kb, g.k.n, key0, n, g.d, mask);
    load_tile<T, DP, BN>(nullptr, 0, s.vn, vb, g.v.n, key0, n, g.d, mask);
    __syncthreads();
    if (!busy) continue;                                 // (barriers count warps: the two above are all of a step)
    float z[4][4];
    product_4x4<DP>(z, s.qt + ty * 4, s.kt + tx * 4);
    bool ok[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = key0 + tx * 4 + j;
      ok[j] = key < n && (!mask || mask[key]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[i][j] = ok[j] ? z[i][j] * sc2 : -INFINITY;
        mx = fmaxf(mx, z[i][j]);
      }
#pragma unroll
      for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;      // no valid key so far: every weight is 2^-inf = 0
      const float a = exp2f(m[i] - ref);
      m[i] = mn;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        z[i][j] = exp2f(z[i][j] - ref);
        sum += z[i][j];
      }
      l[i] = l[i] * a + sum;                             // this thread's columns; joined over tx at the end
#pragma unroll
      for (int j = 0; j < DP / 64; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] *= a;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      store4(s.pt + (tx * 4 + j) * LD + ty * 4, make_float4(z[0][j], z[1][j], z[2][j], z[3][j]));
    __syncwarp();                                        // a warp's weights are its own rows'
    const int live = min(BN, n - key0);                  // the weights behind are zero
#pragma unroll 4
    for (int key = 0; key < live; ++key) {
      const float4 p = *reinterpret_cast<const float4*>(s.pt + key * LD + ty * 4);
      const float ps[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(s.vn + key * (DP + 4) + 64 * j + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][j][0] = fmaf(ps[i], x.x, acc[i][j][0]);
          acc[i][j][1] = fmaf(ps[i], x.y, acc[i][j][1]);
          acc[i][j][2] = fmaf(ps[i], x.z, acc[i][j][2]);
          acc[i][j][3] = fmaf(ps[i], x.w, acc[i][j][3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int w = 8; w; w >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    const int row = qt * BM + ty * 4 + i;
    if (row >= g.nq) continue;
    // a row without a valid key: O = 0, LSE = -inf; NaN sums pass through
    const bool none = m[i] == -INFINITY && !(l[i] > 0.f) && l[i] == l[i];
    const float inv = none ? 0.f : 1.f / l[i];
    const float ls = none ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
    const int64_t r = (int64_t)bh * g.nq + row;
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
      const int c = 64 * j + tx * 4;
      if (c >= g.d) continue;
      const float4 x = make_float4(acc[i][j][0] * inv, acc[i][j][1] * inv, acc[i][j][2] * inv, acc[i][j][3] * inv);
      if (ks > 1)
        store4(part.o + ((int64_t)split * rows_of(g) + r) * g.d + c, x);
      else
        store4(o + b * g.o.b + h * g.o.h + (int64_t)row * g.o.n + c, x);
    }
    if (tx == 0) {
      if (ks > 1)
        part.lse[(int64_t)split * rows_of(g) + r] = ls;
      else if (lse)
        lse[r] = ls;
    }
  }
}

// One thread per four channels of a row: O = sum_s w_s O_s / sum_s w_s with
// w_s = exp(LSE_s - max LSE), splits in order.
template <typename T>
__global__ void join_fwd_kernel(const __grid_constant__ Geo g, int ks, FwdWork part, T* __restrict__ o,
                                float* __restrict__ lse) {
  const int c4 = g.d / 4;
  const int64_t rows = rows_of(g);
  const int64_t total = rows * c4;
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / c4;
    const int c = (int)(i % c4) * 4;
    float mx = -INFINITY;
    for (int s = 0; s < ks; ++s) mx = fmaxf(mx, part.lse[s * rows + r]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < ks; ++s) {
      const float ls = part.lse[s * rows + r];
      if (ls == -INFINITY) continue;                     // a split without keys has written no O
      const float w = exp2f((ls - ref) * kLog2e);
      const float4 y = load4(part.o + (s * rows + r) * g.d + c);
      sum += w;
      x.x = fmaf(w, y.x, x.x);
      x.y = fmaf(w, y.y, x.y);
      x.z = fmaf(w, y.z, x.z);
      x.w = fmaf(w, y.w, x.w);
    }
    const bool none = mx == -INFINITY && sum == 0.f;
    const float inv = none ? 0.f : 1.f / sum;
    const int64_t bh = r / g.nq;
    const int n = (int)(r % g.nq), b = (int)(bh / g.h), h = (int)(bh % g.h);
    store4(o + b * g.o.b + h * g.o.h + n * g.o.n + c, make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv));
    if (lse && c == 0) lse[r] = none ? -INFINITY : mx + log2f(sum) * kLn2;
  }
}

// ------------------------------------------------------------------ backward

// D = rowsum(dO * O).  Eight threads per row, 16 bytes of it each at a time;
// two rows per thread group are on their way at once.
template <typename T>
__device__ __forceinline__ float dot16(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float r = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      r = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), r);
      r = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), r);
    } else {
      r = fmaf(__uint_as_float(x[i]), __uint_as_float(y[i]), r);
    }
  }
  return r;
}
template <typename T>
__global__ void __launch_bounds__(256) row_dot_kernel(const __grid_constant__ Geo g, Divisor by_nq, Divisor by_h,
                                                      const T* __restrict__ o, const T* __restrict__ dO,
                                                      float* __restrict__ D) {
  constexpr int V = 16 / sizeof(T), STEPS = 128 / (8 * V);     // d <= 128: 2 or 4 loads of 16 bytes a thread
  const int64_t rows = rows_of(g);
  const int sub = threadIdx.x & 7;
  for (int64_t r0 = (int64_t)blockIdx.x * 64; r0 < rows; r0 += (int64_t)gridDim.x * 64) {
    uint4 a[2][STEPS], e[2][STEPS];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t r = r0 + 32 * k + (threadIdx.x >> 3);
      if (r >= rows) continue;
      // rows are fewer than 2^34: batch row by the 64-bit quotient, the rest in 32 bits
      const int64_t bh64 = rows <= 0xffffffffll ? (int64_t)over((uint32_t)r, by_nq) : r / g.nq;
      const int64_t n = r - bh64 * g.nq;
      const uint32_t b = over((uint32_t)bh64, by_h);
      const int64_t h = bh64 - (int64_t)b * g.h;
      const T* po = o + b * g.o.b + h * g.o.h + n * g.o.n;
      const T* pg = dO + b * g.dO.b + h * g.dO.h + n * g.dO.n;
#pragma unroll
      for (int i = 0; i < STEPS; ++i) {
        const int c = (8 * i + sub) * V;
        if (c < g.d) {
          a[k][i] = *reinterpret_cast<const uint4*>(po + c);
          e[k][i] = *reinterpret_cast<const uint4*>(pg + c);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t r = r0 + 32 * k + (threadIdx.x >> 3);
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < STEPS; ++i)
        if (r < rows && (8 * i + sub) * V < g.d) x += dot16<T>(a[k][i], e[k][i]);
#pragma unroll
      for (int w = 4; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      if (r < rows && sub == 0) D[r] = x;
    }
  }
}

template <int DP>
struct DqSmem {
  float qt[DP * LD], gt[DP * LD], kt[DP * LD], vt[DP * LD], kn[BN * (DP + 4)], st[BN * LD];
};

template <typename T, int DP>
__global__ void __launch_bounds__(THREADS) dq_kernel(const __grid_constant__ Geo g, Keys keys, int ks,
                                                     const T* __restrict__ q, const T* __restrict__ k,
                                                     const T* __restrict__ v, const T* __restrict__ dO,
                                                     const float* __restrict__ lse, const float* __restrict__ D,
                                                     T* __restrict__ dq, float* __restrict__ part) {
  extern __shared__ __align__(16) unsigned char raw[];
  DqSmem<DP>& s = *reinterpret_cast<DqSmem<DP>*>(raw);
  const int nqt = (g.nq + BM - 1) / BM;
  const int split = (int)(blockIdx.x % ks);
  const int qt = (int)((blockIdx.x / ks) % nqt);
  const int bh = (int)(blockIdx.x / ks / nqt);
  const int b = bh / g.h, h = bh % g.h, hk = h / g.group;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const bool busy = qt * BM + (int)(threadIdx.x >> 5) * 8 < g.nq;    // of the warp's eight queries
  const int n = key_count(g, keys, b);
  const uint8_t* mask = keys.mask ? keys.mask + (int64_t)b * g.nk : nullptr;
  const int ntiles = (n + BN - 1) / BN;
  const int t0 = (int)((int64_t)ntiles * split / ks), t1 = (int)((int64_t)ntiles * (split + 1) / ks);
  const T* kb = k + b * g.k.b + hk * g.k.h;
  const T* vb = v + b * g.v.b + hk * g.v.h;
  const float sc2 = g.scale * kLog2e;
  load_tile<T, DP, BM>(s.qt, LD, nullptr, q + b * g.q.b + h * g.q.h, g.q.n, qt * BM, g.nq, g.d, nullptr);
  load_tile<T, DP, BM>(s.gt, LD, nullptr, dO + b * g.dO.b + h * g.dO.h, g.dO.n, qt * BM, g.nq, g.d, nullptr);
  float ls[4], dd[4], acc[4][DP / 64][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = qt * BM + ty * 4 + i;
    const int64_t r = (int64_t)bh * g.nq + row;
    const float x = row < g.nq ? lse[r] : -INFINITY;
    ls[i] = x == -INFINITY ? INFINITY : x * kLog2e;      // rows without keys: 2^(z - inf) = 0
    dd[i] = row < g.nq ? D[r] : 0.f;
#pragma unroll
    for (int j = 0; j < DP / 64; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
  }
  for (int t = t0; t < t1; ++t) {
    const int key0 = t * BN;
    __syncthreads();
    load_tile<T, DP, BN>(s.kt, LD, s.kn, kb, g.k.n, key0, n, g.d, mask);
    load_tile<T, DP, BN>(s.vt, LD, nullptr, vb, g.v.n, key0, n, g.d, mask);
    __syncthreads();
    if (!busy) continue;
    float z[4][4], dp[4][4];
    product_4x4<DP>(z, s.qt + ty * 4, s.kt + tx * 4);
    product_4x4<DP>(dp, s.gt + ty * 4, s.vt + tx * 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = key0 + tx * 4 + j;
      const bool ok = key < n && (!mask || mask[key]);
      float x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = ok ? exp2f(fmaf(z[i][j], sc2, -ls[i])) * (dp[i][j] - dd[i]) * g.scale : 0.f;
      store4(s.st + (tx * 4 + j) * LD + ty * 4, make_float4(x[0], x[1], x[2], x[3]));
    }
    __syncwarp();
    const int live = min(BN, n - key0);
#pragma unroll 4
    for (int key = 0; key < live; ++key) {
      const float4 p = *reinterpret_cast<const float4*>(s.st + key * LD + ty * 4);
      const float ps[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(s.kn + key * (DP + 4) + 64 * j + tx * 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i][j][0] = fmaf(ps[i], x.x, acc[i][j][0]);
          acc[i][j][1] = fmaf(ps[i], x.y, acc[i][j][1]);
          acc[i][j][2] = fmaf(ps[i], x.z, acc[i][j][2]);
          acc[i][j][3] = fmaf(ps[i], x.w, acc[i][j][3]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = qt * BM + ty * 4 + i;
    if (row >= g.nq) continue;
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
      const int c = 64 * j + tx * 4;
      if (c >= g.d) continue;
      const float4 x = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
      if (ks > 1)
        store4(part + ((int64_t)split * rows_of(g) + (int64_t)bh * g.nq + row) * g.d + c, x);
      else
        store4(dq + b * g.dq.b + h * g.dq.h + (int64_t)row * g.dq.n + c, x);
    }
  }
}

template <int DP>
struct DkvSmem {
  float kt[DP * LD], vt[DP * LD], qt[DP * LQ], gt[DP * LQ], qn[BQ * (DP + 4)], gn[BQ * (DP + 4)], p[BQ * LD], ds[BQ * LD];
};

// Two keys-by-queries products of this thread's 4 keys and 2 queries.
template <int DP>
__device__ __forceinline__ void product_4x2(float acc[4][2], const float* a, const float* b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i][0] = acc[i][1] = 0.f;
#pragma unroll 8
  for (int c = 0; c < DP; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(a + c * LD);
    const float2 y = *reinterpret_cast<const float2*>(b + c * LQ);
    const float xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[i][0] = fmaf(xs[i], y.x, acc[i][0]);
      acc[i][1] = fmaf(xs[i], y.y, acc[i][1]);
    }
  }
}

template <typename T, int DP>
__global__ void __launch_bounds__(THREADS) dkv_kernel(const __grid_constant__ Geo g, Keys keys, int qs,
                                                      const T* __restrict__ q, const T* __restrict__ k,
                                                      const T* __restrict__ v, const T* __restrict__ dO,
                                                      const float* __restrict__ lse, const float* __restrict__ D,
                                                      T* __restrict__ dk, T* __restrict__ dv,
                                                      float* __restrict__ partk, float* __restrict__ partv) {
  extern __shared__ __align__(16) unsigned char raw[];
  DkvSmem<DP>& s = *reinterpret_cast<DkvSmem<DP>*>(raw);
  const int nkt = (g.nk + BN - 1) / BN;
  const int split = (int)(blockIdx.x % qs);
  const int kt = (int)((blockIdx.x / qs) % nkt);
  const int bk = (int)(blockIdx.x / qs / nkt);
  const int b = bk / g.hk, hk = bk % g.hk;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int n = key_count(g, keys, b);
  const uint8_t* mask = keys.mask ? keys.mask + (int64_t)b * g.nk : nullptr;
  const int key0 = kt * BN;
  const float sc2 = g.scale * kLog2e;
  const int nqt = (g.nq + BQ - 1) / BQ;
  const int64_t units = (int64_t)g.group * nqt;          // (query head of the group, query tile)
  const int64_t u0 = units * split / qs, u1 = key0 < n ? units * (split + 1) / qs : u0;
  load_tile<T, DP, BN>(s.kt, LD, nullptr, k + b * g.k.b + hk * g.k.h, g.k.n, key0, n, g.d, mask);
  load_tile<T, DP, BN>(s.vt, LD, nullptr, v + b * g.v.b + hk * g.v.h, g.v.n, key0, n, g.d, mask);
  bool ok[4];
  float ak[4][DP / 64][4], av[4][DP / 64][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = key0 + ty * 4 + i;
    ok[i] = key < n && (!mask || mask[key]);
#pragma unroll
    for (int j = 0; j < DP / 64; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) ak[i][j][e] = av[i][j][e] = 0.f;
  }
  for (int64_t u = u0; u < u1; ++u) {
    const int h = hk * g.group + (int)(u / nqt), row0 = (int)(u % nqt) * BQ;
    __syncthreads();
    load_tile<T, DP, BQ>(s.qt, LQ, s.qn, q + b * g.q.b + h * g.q.h, g.q.n, row0, g.nq, g.d, nullptr);
    load_tile<T, DP, BQ>(s.gt, LQ, s.gn, dO + b * g.dO.b + h * g.dO.h, g.dO.n, row0, g.nq, g.d, nullptr);
    __syncthreads();
    float z[4][2], dp[4][2];
    product_4x2<DP>(z, s.kt + ty * 4, s.qt + tx * 2);
    product_4x2<DP>(dp, s.vt + ty * 4, s.gt + tx * 2);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = row0 + tx * 2 + j;
      const int64_t r = ((int64_t)b * g.h + h) * g.nq + row;
      const float x = row < g.nq ? lse[r] : -INFINITY;
      const float ls = x == -INFINITY ? INFINITY : x * kLog2e;
      const float dd = row < g.nq ? D[r] : 0.f;
      float p[4], ds[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = ok[i] ? exp2f(fmaf(z[i][j], sc2, -ls)) : 0.f;
        ds[i] = ok[i] ? p[i] * (dp[i][j] - dd) * g.scale : 0.f;
      }
      store4(s.p + (tx * 2 + j) * LD + ty * 4, make_float4(p[0], p[1], p[2], p[3]));
      store4(s.ds + (tx * 2 + j) * LD + ty * 4, make_float4(ds[0], ds[1], ds[2], ds[3]));
    }
    __syncthreads();
    const int live = min(BQ, g.nq - row0);
#pragma unroll 2
    for (int r = 0; r < live; ++r) {
      const float4 p = *reinterpret_cast<const float4*>(s.p + r * LD + ty * 4);
      const float4 e = *reinterpret_cast<const float4*>(s.ds + r * LD + ty * 4);
      const float ps[4] = {p.x, p.y, p.z, p.w}, es[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
      for (int j = 0; j < DP / 64; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(s.gn + r * (DP + 4) + 64 * j + tx * 4);
        const float4 y = *reinterpret_cast<const float4*>(s.qn + r * (DP + 4) + 64 * j + tx * 4);
        const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            av[i][j][c] = fmaf(ps[i], xs[c], av[i][j][c]);
            ak[i][j][c] = fmaf(es[i], ys[c], ak[i][j][c]);
          }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = key0 + ty * 4 + i;
    if (key >= g.nk) continue;
#pragma unroll
    for (int j = 0; j < DP / 64; ++j) {
      const int c = 64 * j + tx * 4;
      if (c >= g.d) continue;
      float4 x = make_float4(ak[i][j][0], ak[i][j][1], ak[i][j][2], ak[i][j][3]);
      float4 y = make_float4(av[i][j][0], av[i][j][1], av[i][j][2], av[i][j][3]);
      if (!ok[i]) x = y = make_float4(0.f, 0.f, 0.f, 0.f);   // (whatever its zero weights met)
      if (qs > 1) {
        const int64_t at = ((int64_t)split * keys_of(g) + (int64_t)bk * g.nk + key) * g.d + c;
        store4(partk + at, x);
        store4(partv + at, y);
      } else {
        store4(dk + b * g.dk.b + hk * g.dk.h + (int64_t)key * g.dk.n + c, x);
        store4(dv + b * g.dv.b + hk * g.dv.h + (int64_t)key * g.dv.n + c, y);
      }
    }
  }
}

// out = sum of the parts, in order; one thread per four channels; the second
// row of the grid takes the second tensor.
struct Sums {
  const float* part[2];
  void* out[2];
  Lay lay[2];
};
template <typename T>
__global__ void sum_parts_kernel(int parts, const __grid_constant__ Sums a, int heads, int n, int d, int64_t rows) {
  const int c4 = d / 4;
  const int64_t total = rows * c4;
  const int which = blockIdx.y;
  const float* part = a.part[which];
  T* out = static_cast<T*>(a.out[which]);
  const Lay lay = a.lay[which];
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < total; i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t r = i / c4;
    const int c = (int)(i % c4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int s = 0; s < parts; ++s) {
      const float4 y = load4(part + (s * rows + r) * d + c);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    const int64_t bh = r / n;
    store4(out + (bh / heads) * lay.b + (bh % heads) * lay.h + (r % n) * lay.n + c, x);
  }
}

// ------------------------------------------------------------------ host

static int grid_for(int64_t threads_needed, int per_block) {
  const int64_t blocks = (threads_needed + per_block - 1) / per_block;
  return (int)(blocks < 148 * 16 ? (blocks < 1 ? 1 : blocks) : 148 * 16);
}

cudaError_t launch_join_fwd(const Geo& g, int ks, const FwdWork& w, void* o, float* lse, cudaStream_t s) {
  const int grid = grid_for(rows_of(g) * (g.d / 4), 128);
  if (g.bf16)
    join_fwd_kernel<<<grid, 128, 0, s>>>(g, ks, w, (__nv_bfloat16*)o, lse);
  else
    join_fwd_kernel<<<grid, 128, 0, s>>>(g, ks, w, (float*)o, lse);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_row_dot(const Geo& g, const void* o, const void* dO, float* D, cudaStream_t s) {
  const int grid = grid_for(rows_of(g), 64);
  const Divisor n = divisor(g.nq), h = divisor(g.h);
  if (g.bf16)
    row_dot_kernel<<<grid, 256, 0, s>>>(g, n, h, (const __nv_bfloat16*)o, (const __nv_bfloat16*)dO, D);
  else
    row_dot_kernel<<<grid, 256, 0, s>>>(g, n, h, (const float*)o, (const float*)dO, D);
  note_launches(1);
  return cudaGetLastError();
}

static cudaError_t sum_parts(const Geo& g, int parts, const Sums& a, int tensors, int heads, int n, cudaStream_t s) {
  const int64_t rows = (int64_t)g.b * heads * n;
  const dim3 grid((unsigned)grid_for(rows * (g.d / 4), 128), (unsigned)tensors);
  if (g.bf16)
    sum_parts_kernel<__nv_bfloat16><<<grid, 128, 0, s>>>(parts, a, heads, n, g.d, rows);
  else
    sum_parts_kernel<float><<<grid, 128, 0, s>>>(parts, a, heads, n, g.d, rows);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_sum_q(const Geo& g, int parts, const float* part, void* dq, cudaStream_t s) {
  return sum_parts(g, parts, Sums{{part, nullptr}, {dq, nullptr}, {g.dq, Lay{}}}, 1, g.h, g.nq, s);
}

cudaError_t launch_sum_kv(const Geo& g, int parts, const float* partk, const float* partv, void* dk, void* dv,
                          cudaStream_t s) {
  return sum_parts(g, parts, Sums{{partk, partv}, {dk, dv}, {g.dk, g.dv}}, 2, g.hk, g.nk, s);
}

// Splits fill the device two to three times over when the tiles alone do not
// fill it once (two blocks an SM, rounded up to whole splits: fewer than three),
// 64 at most, and no split with less than one tile.
static int splits_for(int64_t blocks, int64_t units, int sms) {
  if (blocks >= sms) return 1;
  int64_t s = (2 * sms + blocks - 1) / blocks;
  if (s > units) s = units;
  if (s > 64) s = 64;
  return (int)(s < 1 ? 1 : s);
}

Plan plan_simt(const Geo& g, int sms) {
  const int64_t qtiles = (int64_t)g.b * g.h * ((g.nq + BM - 1) / BM);
  const int64_t nkt = (g.nk + BN - 1) / BN;
  Plan p;
  p.fwd_ks = splits_for(qtiles, nkt, sms);
  p.dq_ks = p.fwd_ks;
  p.dkv_qs = splits_for((int64_t)g.b * g.hk * nkt, (int64_t)g.group * ((g.nq + BQ - 1) / BQ), sms);
  return p;
}

static BwdWork carve_bwd(const Geo& g, const Plan& p, void* work, size_t* bytes) {
  char* w = static_cast<char*>(work);
  size_t at = 0;
  auto take = [&](size_t n) {
    float* ptr = reinterpret_cast<float*>(w + at);
    at += round256(n);
    return ptr;
  };
  BwdWork out;
  out.D = take((size_t)rows_of(g) * 4);
  out.dq = p.dq_ks > 1 ? take((size_t)p.dq_ks * rows_of(g) * g.d * 4) : nullptr;
  out.dk = p.dkv_qs > 1 ? take((size_t)p.dkv_qs * keys_of(g) * g.d * 4) : nullptr;
  out.dv = p.dkv_qs > 1 ? take((size_t)p.dkv_qs * keys_of(g) * g.d * 4) : nullptr;
  if (bytes) *bytes = at;
  return out;
}

size_t bwd_work_bytes_simt(const Geo& g, const Plan& p) {
  size_t n = 0;
  carve_bwd(g, p, nullptr, &n);
  return n;
}

template <typename K>
static cudaError_t allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

template <typename T, int DP>
static cudaError_t fwd(const Geo& g, const Plan& p, const void* q, const void* k, const void* v, const Keys& keys,
                       void* o, float* lse, void* work, cudaStream_t s) {
  cudaError_t e = allow_smem(fwd_kernel<T, DP>, sizeof(FwdSmem<DP>));
  if (e != cudaSuccess) return e;
  const FwdWork w = carve_fwd(g, p.fwd_ks, work);
  const int64_t grid = (int64_t)g.b * g.h * ((g.nq + BM - 1) / BM) * p.fwd_ks;
  fwd_kernel<T, DP><<<(unsigned)grid, THREADS, sizeof(FwdSmem<DP>), s>>>(g, keys, p.fwd_ks, (const T*)q, (const T*)k,
                                                                        (const T*)v, (T*)o, lse, w);
  note_launches(1);
  e = cudaGetLastError();
  if (e == cudaSuccess && p.fwd_ks > 1) e = launch_join_fwd(g, p.fwd_ks, w, o, lse, s);
  return e;
}

cudaError_t launch_fwd_simt(const Geo& g, const Plan& p, const void* q, const void* k, const void* v,
                            const Keys& keys, void* o, float* lse, void* work, cudaStream_t s) {
  if (g.bf16)
    return g.d <= 64 ? fwd<__nv_bfloat16, 64>(g, p, q, k, v, keys, o, lse, work, s)
                     : fwd<__nv_bfloat16, 128>(g, p, q, k, v, keys, o, lse, work, s);
  return g.d <= 64 ? fwd<float, 64>(g, p, q, k, v, keys, o, lse, work, s)
                   : fwd<float, 128>(g, p, q, k, v, keys, o, lse, work, s);
}

template <typename T, int DP>
static cudaError_t bwd(const Geo& g, const Plan& p, const void* q, const void* k, const void* v, const Keys& keys,
                       const void* o, const void* dO, const float* lse, void* dq, void* dk, void* dv, void* work,
                       cudaStream_t s) {
  cudaError_t e = allow_smem(dq_kernel<T, DP>, sizeof(DqSmem<DP>));
  if (e == cudaSuccess) e = allow_smem(dkv_kernel<T, DP>, sizeof(DkvSmem<DP>));
  if (e != cudaSuccess) return e;
  const BwdWork w = carve_bwd(g, p, work, nullptr);
  e = launch_row_dot(g, o, dO, w.D, s);
  if (e != cudaSuccess) return e;
  const int64_t gq = (int64_t)g.b * g.h * ((g.nq + BM - 1) / BM) * p.dq_ks;
  dq_kernel<T, DP><<<(unsigned)gq, THREADS, sizeof(DqSmem<DP>), s>>>(g, keys, p.dq_ks, (const T*)q, (const T*)k,
                                                                    (const T*)v, (const T*)dO, lse, w.D, (T*)dq, w.dq);
  note_launches(1);
  e = cudaGetLastError();
  if (e == cudaSuccess && p.dq_ks > 1) e = launch_sum_q(g, p.dq_ks, w.dq, dq, s);
  if (e != cudaSuccess) return e;
  const int64_t gk = (int64_t)g.b * g.hk * ((g.nk + BN - 1) / BN) * p.dkv_qs;
  dkv_kernel<T, DP><<<(unsigned)gk, THREADS, sizeof(DkvSmem<DP>), s>>>(
      g, keys, p.dkv_qs, (const T*)q, (const T*)k, (const T*)v, (const T*)dO, lse, w.D, (T*)dk, (T*)dv, w.dk, w.dv);
  note_launches(1);
  e = cudaGetLastError();
  if (e == cudaSuccess && p.dkv_qs > 1) e = launch_sum_kv(g, p.dkv_qs, w.dk, w.dv, dk, dv, s);
  return e;
}

cudaError_t launch_bwd_simt(const Geo& g, const Plan& p, const void* q, const void* k, const void* v,
                            const Keys& keys, const void* o, const void* dO, const float* lse, void* dq, void* dk,
                            void* dv, void* work, cudaStream_t s) {
  if (g.bf16)
    return g.d <= 64 ? bwd<__nv_bfloat16, 64>(g, p, q, k, v, keys, o, dO, lse, dq, dk, dv, work, s)
                     : bwd<__nv_bfloat16, 128>(g, p, q, k, v, keys, o, dO, lse, dq, dk, dv, work, s);
  return g.d <= 64 ? bwd<float, 64>(g, p, q, k, v, keys, o, dO, lse, dq, dk, dv, work, s)
                   : bwd<float, 128>(g, p, q, k, v, keys, o, dO, lse, dq, dk, dv, work, s);
}

}  // namespace cross
}  // namespace llsa
