// k_norm.cu -- layer norm of token rows, forward and backward.
//
//   y = (x - mean) rstd w + b;
//   g = dy w,  xhat = (x - mean) rstd,
//   dx = rstd (g - mean_c(g) - xhat mean_c(g xhat)),  dw = sum_rows dy xhat,  db = sum_rows dy.
//
// Bound by memory: every row is read once and kept in registers as it came (the
// variance is the mean of the squared deviations from the mean, in a second
// pass over the registers, and xhat is formed from the deviation in both
// directions, so that an offset costs what rounding it costs the mean, 2^-24 of
// itself, and no more).  G threads
// work on a row, each on IT vectors of 16 bytes (narrower ones, down to single
// values, where the width, a stride or an address does not allow them).  Rows of up to
// 2 KB take a part of a warp or a warp (in the backward of bf16 up to 1 KB, and up to 1 KB
// or less by narrower loads), wider ones a block.  R rows are taken at a time,
// and the next R are on their way while these are worked on: an SM needs some
// 40 KB in flight.  Rows are walked in the order of x's memory.
//
// In the backward every thread keeps the same channels for all its rows and
// sums dy xhat and dy in registers; a block adds up its row groups (by
// shuffles, then through shared memory, in a fixed order) and writes one
// partial row, and a second kernel adds the partial rows: no atomics, the same
// bits every time.  786432 rows of 64 bf16 channels: 44 us forward, 65 backward
// (4.6 TB/s; the issue slots are two thirds full); 16384 rows of 8192: 113 us.
#include "norm.cuh"
#include "packed.cuh"

namespace llsa {
namespace norm {

template <typename T, int V> struct Raw;
template <> struct Raw<__nv_bfloat16, 8> { uint4 w; };
template <> struct Raw<__nv_bfloat16, 4> { uint2 w; };
template <> struct Raw<__nv_bfloat16, 2> { uint32_t w; };
template <> struct Raw<float, 2> { float2 w; };
template <> struct Raw<float, 4> { float4 w; };
template <> struct Raw<__nv_bfloat16, 1> { __nv_bfloat16 w; };
template <> struct Raw<float, 1> { float w; };

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 8>& r, float* f) {
  const uint32_t w[4] = {r.w.x, r.w.y, r.w.z, r.w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 4>& r, float* f) {
  f[0] = __uint_as_float(r.w.x << 16);
  f[1] = __uint_as_float(r.w.x & 0xffff0000u);
  f[2] = __uint_as_float(r.w.y << 16);
  f[3] = __uint_as_float(r.w.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const Raw<float, 4>& r, float* f) {
  f[0] = r.w.x;
  f[1] = r.w.y;
  f[2] = r.w.z;
  f[3] = r.w.w;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 2>& r, float* f) {
  f[0] = __uint_as_float(r.w << 16);
  f[1] = __uint_as_float(r.w & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const Raw<float, 2>& r, float* f) {
  f[0] = r.w.x;
  f[1] = r.w.y;
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, 1>& r, float* f) { f[0] = __bfloat162float(r.w); }
__device__ __forceinline__ void unpack(const Raw<float, 1>& r, float* f) { f[0] = r.w; }

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void pack(Raw<__nv_bfloat16, 8>& r, const float* f) {
  r.w = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void pack(Raw<__nv_bfloat16, 4>& r, const float* f) {
  r.w = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3]));
}
__device__ __forceinline__ void pack(Raw<float, 4>& r, const float* f) { r.w = make_float4(f[0], f[1], f[2], f[3]); }
__device__ __forceinline__ void pack(Raw<__nv_bfloat16, 2>& r, const float* f) { r.w = pack2(f[0], f[1]); }
__device__ __forceinline__ void pack(Raw<float, 2>& r, const float* f) { r.w = make_float2(f[0], f[1]); }
__device__ __forceinline__ void pack(Raw<__nv_bfloat16, 1>& r, const float* f) { r.w = __float2bfloat16_rn(f[0]); }
__device__ __forceinline__ void pack(Raw<float, 1>& r, const float* f) { r.w = f[0]; }

// V weights from column c on, of either type.
template <int V>
__device__ __forceinline__ void load_param(const void* p, int bf16, int64_t at, float* f) {
  if (bf16) {
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p) + at;
    if constexpr (V == 8) {
      Raw<__nv_bfloat16, 8> r;
      r.w = *reinterpret_cast<const uint4*>(w);
      unpack(r, f);
    } else if constexpr (V == 4) {
      const uint2 u = *reinterpret_cast<const uint2*>(w);
      f[0] = __uint_as_float(u.x << 16);
      f[1] = __uint_as_float(u.x & 0xffff0000u);
      f[2] = __uint_as_float(u.y << 16);
      f[3] = __uint_as_float(u.y & 0xffff0000u);
    } else if constexpr (V == 2) {
      const uint32_t u = *reinterpret_cast<const uint32_t*>(w);
      f[0] = __uint_as_float(u << 16);
      f[1] = __uint_as_float(u & 0xffff0000u);
    } else {
      f[0] = __bfloat162float(*w);
    }
  } else {
    const float* w = static_cast<const float*>(p) + at;
    if constexpr (V >= 4) {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 u = *reinterpret_cast<const float4*>(w + i);
        f[i] = u.x;
        f[i + 1] = u.y;
        f[i + 2] = u.z;
        f[i + 3] = u.w;
      }
    } else if constexpr (V == 2) {
      const float2 u = *reinterpret_cast<const float2*>(w);
      f[0] = u.x;
      f[1] = u.y;
    } else {
      f[0] = *w;
    }
  }
}

struct At {
  int64_t i0, i1, i2;
};
__device__ __forceinline__ At place(const Geo& g, int64_t row) {
  const uint32_t r = (uint32_t)row;         // rows of a group are fewer than 2^31
  const uint32_t q = over(r, g.n2), p = over(q, g.n1);
  return At{(int64_t)p, (int64_t)(q - p * g.n1.d), (int64_t)(r - q * g.n2.d)};
}
__device__ __forceinline__ int64_t offset(const At& a, const int64_t* st, int group) {
  return a.i0 * st[0] + a.i1 * st[1] + a.i2 * st[2] + group * st[3];
}

// V values as pairs (of one value: its other half is zero).
template <int V> constexpr int pairs() { return (V + 1) / 2; }
template <typename T, int V>
__device__ __forceinline__ void unpack2(const Raw<T, V>& r, f2* f) {
  float x[V + 1];
  unpack(r, x);
  if (V == 1) x[1] = 0.f;
#pragma unroll
  for (int i = 0; i < pairs<V>(); ++i) f[i] = pair(x[2 * i], x[2 * i + 1]);
}
template <typename T, int V>
__device__ __forceinline__ void pack2(Raw<T, V>& r, const f2* f) {
  float x[V + 1];
#pragma unroll
  for (int i = 0; i < pairs<V>(); ++i) split(f[i], x[2 * i], x[2 * i + 1]);
  pack(r, x);
}

// Sums N values over the G threads of a row.  Rows that span a block use
// `red` ([2][N][32] floats, used in turn, so that one barrier per sum suffices).
template <int G, int N>
__device__ __forceinline__ void row_sum(float* v, float* red, int& turn) {
  constexpr int W = G < 32 ? G : 32;
#pragma unroll
  for (int w = W / 2; w; w >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], w);
  if constexpr (G > 32) {
    float* buf = red + turn * N * 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) buf[i * 32 + warp] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float x = lane < G / 32 ? buf[i * 32 + lane] : 0.f;
#pragma unroll
      for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
      v[i] = x;
    }
    turn ^= 1;
  }
}

template <int G> constexpr int threads() { return G <= 32 ? 256 : G; }

// Rows of a step and thread group.  Two where a thread holds one vector of each (with four the registers leave too few
// blocks: 51 us against 44 for 786432 rows of 64 bf16 channels).
template <int G, int IT, int V> constexpr int rows_at_once() {
  if (G > 32) return 1;
  if (V <= 2) return IT <= 2 ? 4 : (IT <= 4 ? 2 : 1);
  return IT > 1 ? 1 : 2;
}

template <typename T, int V, int G, int IT>
__global__ void __launch_bounds__(threads<G>()) fwd_kernel(const __grid_constant__ Geo g, const T* x, const void* w,
                                                           const void* b, T* y, float* mean, float* rstd) {
  constexpr int RPB = threads<G>() / G;              // thread groups of a block
  constexpr int R = rows_at_once<G, IT, V>();
  constexpr bool KEEP = G <= 32;                     // weights in registers; a block-wide row reads them again (from L1)
  __shared__ float red[G > 32 ? 2 * R * 32 : 1];
  int turn = 0;
  const int sub = threadIdx.x % G, slot = threadIdx.x / G;
  const int group = blockIdx.y;
  const float inv_c = 1.f / (float)g.c;
  constexpr int P = pairs<V>();
  f2 wv[KEEP ? IT * P : 1], bv[KEEP ? IT * P : 1];
  auto params = [&](int i, f2* ww, f2* bb) {
    const int c = (i * G + sub) * V;
    float fw[V + 1], fb[V + 1];
#pragma unroll
    for (int e = 0; e < V + 1; ++e) {
      fw[e] = 1.f;
      fb[e] = 0.f;
    }
    if (c < g.c) {
      if (w) load_param<V>(w, g.param_bf16, group * g.ws + c, fw);
      if (b) load_param<V>(b, g.param_bf16, group * g.bs + c, fb);
    }
#pragma unroll
    for (int e = 0; e < P; ++e) {
      ww[e] = pair(fw[2 * e], fw[2 * e + 1]);
      bb[e] = pair(fb[2 * e], fb[2 * e + 1]);
    }
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < IT; ++i) params(i, wv + i * P, bv + i * P);
  }
  auto at_x = [&](int64_t r) { return g.flat_fwd ? r * g.x[2] + group * g.x[3] : offset(place(g, r), g.x, group); };
  auto at_y = [&](int64_t r) { return g.flat_fwd ? r * g.y[2] + group * g.y[3] : offset(place(g, r), g.y, group); };
  const int64_t step = (int64_t)gridDim.x * RPB * R;
  Raw<T, V> next[R][IT];
  auto fetch = [&](int64_t r0) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t r = r0 + k * RPB + slot;
      if (r >= g.rows) continue;
      const T* px = x + at_x(r);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * G + sub) * V;
        if (c < g.c) next[k][i] = *reinterpret_cast<const Raw<T, V>*>(px + c);
      }
    }
  };
  fetch((int64_t)blockIdx.x * RPB * R);
  for (int64_t r0 = (int64_t)blockIdx.x * RPB * R; r0 < g.rows; r0 += step) {
    f2 f[R][IT * P];
    float mu[R], rs[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      f2 sum = twice(0.f);
      const bool live = r0 + k * RPB + slot < g.rows;
#pragma unroll
      for (int i = 0; i < IT; ++i)
        if (live && (i * G + sub) * V < g.c) {
          unpack2(next[k][i], f[k] + i * P);
#pragma unroll
          for (int e = 0; e < P; ++e) sum = add2(sum, f[k][i * P + e]);
        }
      mu[k] = both(sum);
    }
    fetch(r0 + step);
    row_sum<G, R>(mu, red, turn);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mu[k] *= inv_c;
      const f2 minus = V == 1 ? pair(-mu[k], 0.f) : twice(-mu[k]);
      f2 sum = twice(0.f);
      const bool live = r0 + k * RPB + slot < g.rows;
#pragma unroll
      for (int i = 0; i < IT; ++i)
        if (live && (i * G + sub) * V < g.c) {
#pragma unroll
          for (int e = 0; e < P; ++e) {
            f[k][i * P + e] = add2(f[k][i * P + e], minus);
            sum = fma2(f[k][i * P + e], f[k][i * P + e], sum);
          }
        }
      rs[k] = both(sum);
    }
    row_sum<G, R>(rs, red, turn);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t r = r0 + k * RPB + slot;
      rs[k] = rsqrtf(fmaf(rs[k], inv_c, g.eps));
      if (r >= g.rows) continue;
      const f2 rk = twice(rs[k]);
      T* py = y + at_y(r);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * G + sub) * V;
        if (c >= g.c) continue;
        f2 ww[P], bb[P];
        if constexpr (KEEP) {
#pragma unroll
          for (int e = 0; e < P; ++e) {
            ww[e] = wv[i * P + e];
            bb[e] = bv[i * P + e];
          }
        } else {
          params(i, ww, bb);
        }
#pragma unroll
        for (int e = 0; e < P; ++e) f[k][i * P + e] = fma2(mul2(f[k][i * P + e], rk), ww[e], bb[e]);
        Raw<T, V> o;
        pack2(o, f[k] + i * P);
        *reinterpret_cast<Raw<T, V>*>(py + c) = o;
      }
    }
    if (mean || rstd) {                              // thread k of a row's threads: the k-th row's statistics
      float m = mu[0], v = rs[0];
#pragma unroll
      for (int k = 1; k < R; ++k)
        if (sub == k) {
          m = mu[k];
          v = rs[k];
        }
      const int64_t r = r0 + sub * RPB + slot;
      if (sub < R && r < g.rows) {
        const int64_t st = offset(place(g, r), g.s, group);
        if (mean) mean[st] = m;
        if (rstd) rstd[st] = v;
      }
    }
  }
}

template <typename T, int V, int G, int IT>
__global__ void __launch_bounds__(threads<G>()) bwd_kernel(const __grid_constant__ Geo g, const T* x, const T* dy,
                                                           const void* w, const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, T* dx,
                                                           float* __restrict__ part) {
  constexpr int RPB = threads<G>() / G;
  // Rows of a step and thread group.  Block-wide rows: two a barrier where that paid (50 M bf16 values, 768, 1024, 4096
  // channels: 129, 111, 125 us against 151, 122, 151), not with 256 threads (1152, 2048 channels: 165, 113 against 138,
  // 99) nor in fp32 (25 M values, 1024, 2048 channels: 103, 114 against 83, 86).
  constexpr int R = G > 32 ? ((V == 1 && G == 128) || (V == 8 && IT == 1 && G != 256) ? 2 : 1)
                           : (V <= 2 ? (IT <= 2 ? 4 : (IT <= 4 ? 2 : 1)) : (IT > 1 ? 1 : 2));
  constexpr int NV = IT * V;
  // A block-wide row's xhat stays in registers between its two uses, up to 16 registers of it, which undoes what the
  // subtraction costs (50 M bf16 values of 1152, 2048, 8192 channels: 138, 99, 125 us against 149, 107, 128).  Not of
  // single values, whose pairs are half empty (25 M fp32 values of 1001: 168 against 113), nor of narrow rows (the same).
  constexpr bool HOLD = G > 32 && V > 1 && IT * ((V + 1) / 2) <= 8;
  __shared__ float red[G > 32 ? 2 * 2 * R * 32 : 1];
  __shared__ float cols[G <= 32 ? 8 * G * NV : 1];   // a block's eight warps' sums
  int turn = 0;
  const int sub = threadIdx.x % G, slot = threadIdx.x / G;
  const int group = blockIdx.y;
  const float inv_c = 1.f / (float)g.c;
  constexpr int P = pairs<V>();
  constexpr bool KEEP = G <= 32;
  f2 wv[KEEP ? IT * P : 1];
  auto weights = [&](int i, f2* ww) {
    const int c = (i * G + sub) * V;
    float fw[V + 1];
#pragma unroll
    for (int e = 0; e < V + 1; ++e) fw[e] = 1.f;
    if (w && c < g.c) load_param<V>(w, g.param_bf16, group * g.ws + c, fw);
#pragma unroll
    for (int e = 0; e < P; ++e) ww[e] = pair(fw[2 * e], fw[2 * e + 1]);
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < IT; ++i) weights(i, wv + i * P);
  }
  auto weights_of = [&](int i, f2* ww) {
    if constexpr (KEEP) {
#pragma unroll
      for (int e = 0; e < P; ++e) ww[e] = wv[i * P + e];
    } else {
      weights(i, ww);
    }
  };
  f2 dw[IT * P], db[IT * P];
#pragma unroll
  for (int i = 0; i < IT * P; ++i) dw[i] = db[i] = twice(0.f);
  const int64_t step = (int64_t)gridDim.x * RPB * R;
  Raw<T, V> nx[R][IT], ng[R][IT];
  float nmu[R], nrs[R];
  auto fetch = [&](int64_t r0) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int64_t r = r0 + k * RPB + slot;
      if (r >= g.rows) continue;
      const At at = place(g, r);
      const T* px = x + (g.flat_bwd ? r * g.x[2] + group * g.x[3] : offset(at, g.x, group));
      const T* pg = dy + (g.flat_bwd ? r * g.dy[2] + group * g.dy[3] : offset(at, g.dy, group));
      const int64_t st = offset(at, g.s, group);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * G + sub) * V;
        if (c < g.c) {
          nx[k][i] = *reinterpret_cast<const Raw<T, V>*>(px + c);
          ng[k][i] = *reinterpret_cast<const Raw<T, V>*>(pg + c);
        }
      }
      nmu[k] = mean[st];
      nrs[k] = rstd[st];
    }
  };
  fetch((int64_t)blockIdx.x * RPB * R);
  for (int64_t r0 = (int64_t)blockIdx.x * RPB * R; r0 < g.rows; r0 += step) {
    Raw<T, V> rx[R][IT], rg[R][IT];
    float mu[R], rs[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mu[k] = nmu[k];
      rs[k] = nrs[k];
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        rx[k][i] = nx[k][i];
        rg[k][i] = ng[k][i];
      }
    }
    fetch(r0 + step);
    float sum[2 * R];
    // xhat = (x - mean) rstd, as in the forward: x rstd - mean rstd would leave the rounding of mean rstd in rows far from 0
    f2 minus[R], scale[R];
    f2 held[HOLD ? R : 1][HOLD ? IT * P : 1];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      scale[k] = twice(rs[k]);
      minus[k] = V == 1 ? pair(-mu[k], 0.f) : twice(-mu[k]);
      f2 s0 = twice(0.f), s1 = twice(0.f);
      const bool live = r0 + k * RPB + slot < g.rows;
#pragma unroll
      for (int i = 0; i < IT; ++i)
        if (live && (i * G + sub) * V < g.c) {
          f2 fx[P], fg[P], ww[P];
          unpack2(rx[k][i], fx);
          unpack2(rg[k][i], fg);
          weights_of(i, ww);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const f2 xh = mul2(add2(fx[e], minus[k]), scale[k]), gw = mul2(fg[e], ww[e]);
            if constexpr (HOLD) held[k][i * P + e] = xh;
            s0 = add2(s0, gw);
            s1 = fma2(gw, xh, s1);
            dw[i * P + e] = fma2(fg[e], xh, dw[i * P + e]);
            db[i * P + e] = add2(db[i * P + e], fg[e]);
          }
        }
      sum[2 * k] = both(s0);                           // (the empty half of a single value has dy = 0)
      sum[2 * k + 1] = both(s1);
    }
    if (dx) {                                          // uniform over the grid
      row_sum<G, 2 * R>(sum, red, turn);
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int64_t r = r0 + k * RPB + slot;
        if (r >= g.rows) continue;
        const f2 c1 = twice(-sum[2 * k] * inv_c * rs[k]), c2 = twice(-sum[2 * k + 1] * inv_c);
        T* po = dx + (g.flat_bwd ? r * g.dx[2] + group * g.dx[3] : offset(place(g, r), g.dx, group));
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int c = (i * G + sub) * V;
          if (c >= g.c) continue;
          f2 fx[P], fg[P], ww[P];
          unpack2(rx[k][i], fx);
          unpack2(rg[k][i], fg);
          weights_of(i, ww);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const f2 xh = HOLD ? held[k][i * P + e] : mul2(add2(fx[e], minus[k]), scale[k]);
            fx[e] = fma2(fma2(xh, c2, mul2(fg[e], ww[e])), scale[k], c1);   // rstd (g - xhat c2) - rstd c1
          }
          Raw<T, V> o;
          pack2(o, fx);
          *reinterpret_cast<Raw<T, V>*>(po + c) = o;
        }
      }
    }
  }
  if (!part) return;
  float* out = part + ((int64_t)group * gridDim.x + blockIdx.x) * 2 * g.c;
  float sw[IT * P * 2], sb[IT * P * 2];                // value e of vector i at 2 P i + e
#pragma unroll
  for (int i = 0; i < IT * P; ++i) {
    split(dw[i], sw[2 * i], sw[2 * i + 1]);
    split(db[i], sb[2 * i], sb[2 * i + 1]);
  }
  if constexpr (G > 32) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
      if (c < g.c)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          out[c + e] = sw[2 * P * i + e];
          out[g.c + c + e] = sb[2 * P * i + e];
        }
    }
  } else {
    // the row groups of a warp by shuffles, then the eight warps in order
#pragma unroll
    for (int i = 0; i < IT * P * 2; ++i)
#pragma unroll
      for (int s = 16; s >= G; s >>= 1) {
        sw[i] += __shfl_xor_sync(0xffffffffu, sw[i], s);
        sb[i] += __shfl_xor_sync(0xffffffffu, sb[i], s);
      }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
      if (lane < G)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int at = (i / V) * 2 * P + i % V;
          cols[(warp * NV + i) * G + lane] = which ? sb[at] : sw[at];
        }
      __syncthreads();
      for (int j = threadIdx.x; j < G * NV; j += 256) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) x += cols[k * NV * G + j];
        const int i = j / G, l = j % G;                // value i of lane l: channel ((i / V) G + l) V + i % V
        const int c = ((i / V) * G + l) * V + i % V;
        if (c < g.c) out[which * g.c + c] = x;
      }
    }
  }
}

// Adds the partial rows: 32 channels per block, 32 threads per channel.
__global__ void __launch_bounds__(1024) finish_kernel(const float* __restrict__ part, int parts, int c, int param_bf16,
                                                      void* dw, void* db) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane, group = blockIdx.y, which = blockIdx.z;
  void* out = which ? db : dw;
  if (!out) return;
  const float* p = part + (int64_t)group * parts * 2 * c + which * c;
  float x = 0.f;
  if (col < c)
#pragma unroll 8
    for (int k = y; k < parts; k += 32) x += p[(int64_t)k * 2 * c + col];
  s[y][lane] = x;
  __syncthreads();
  x = s[lane][y];                                      // thread (lane, y): part lane of channel y
#pragma unroll
  for (int w = 16; w; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
  const int cc = blockIdx.x * 32 + y;
  if (lane == 0 && cc < c) {
    const int64_t at = (int64_t)group * c + cc;
    if (param_bf16)
      static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
    else
      static_cast<float*>(out)[at] = x;
  }
}

// ------------------------------------------------------------------ host

// Values per load (16 bytes, or what a width, stride or address that is no
// multiple of that allows), threads per row and loads per thread.  A row's threads are
// the fewest that hold it in a few registers: in the backward, which keeps two
// sums for each channel of a thread, about 16 channels each, in the forward up
// to 32.  257 to 384 bf16 channels take 8-byte loads, which fill a warp where
// 16-byte ones would leave a quarter of it (or, with 16 threads a row, need the
// registers of 24 channels: 150, and one block an SM).
struct Shape {
  int v, g, it;
};
static Shape shape_of(const Geo& g, bool bwd) {
  if (g.vec * (g.bf16 ? 2 : 4) == 16) {
    const int v = g.vec, n = g.c / v;
    if (n <= 8) return {v, 8, 1};
    if (n <= 16) return {v, 16, 1};
    if (n <= 32) return {v, 32, 1};
    if (n <= 48) return g.bf16 ? Shape{4, 32, 3} : Shape{4, 16, 3};
    if (n <= 64) return {v, 32, 2};
    if (bwd) {
      if (!g.bf16 && n <= 96) return {v, 32, 3};
      if (!g.bf16 && n <= 128) return {v, 32, 4};
      if (n <= 128) return {v, 128, 1};
      if (n <= 256) return {v, 256, 1};
      if (n <= 512) return {v, 512, 1};
    } else {
      if (n <= 96) return {v, 32, 3};
      if (n <= 128) return {v, 32, 4};
      if (n <= 256) return {v, 128, 2};
      if (n <= 512) return {v, 256, 2};
    }
    if (n <= 1024) return {v, 512, 2};
    if (n <= 2048) return {v, 512, 4};
    return {v, 1024, 4};
  }
  if (g.vec > 1) {                             // 8-byte loads of bf16, or pairs
    const int v = g.vec, n = g.c / v;
    if (n <= 8) return {v, 8, 1};
    if (n <= 16) return {v, 8, 2};
    if (n <= 32) return {v, 8, 4};
    if (n <= 64) return {v, 16, 4};
    if (n <= 128) return {v, 32, 4};
    if (n <= 256) return {v, 128, 2};
    if (n <= 512) return {v, 128, 4};
    if (n <= 1024) return {v, 256, 4};
    if (n <= 2048) return {v, 512, 4};
    if (n <= 4096) return {v, 512, 8};
    return {v, 1024, 8};
  }
  if (g.c <= 8) return {1, 8, 1};
  if (g.c <= 16) return {1, 8, 2};
  if (g.c <= 32) return {1, 8, 4};
  if (g.c <= 64) return {1, 8, 8};
  if (g.c <= 128) return {1, 16, 8};
  if (g.c <= 256) return {1, 32, 8};
  if (g.c <= 512) return {1, 128, 4};
  if (g.c <= 1024) return bwd ? Shape{1, 256, 4} : Shape{1, 128, 8};
  if (g.c <= 2048) return {1, 512, 4};
  if (g.c <= 4096) return {1, 512, 8};
  if (g.c <= 8192) return bwd ? Shape{1, 512, 16} : Shape{1, 1024, 8};
  return {1, 1024, 16};
}

static int rows_per_block(const Shape& s) { return s.g <= 32 ? 256 / s.g : 1; }

// Blocks per group in the backward: enough to fill the device, no more than there are row steps.
int bwd_parts(const Geo& g) {
  const Shape s = shape_of(g, true);
  const int rows = rows_per_block(s);
  const int64_t steps = (g.rows + rows - 1) / rows;
  const int per_sm = s.g <= 32 ? 2 : (s.g <= 256 ? 4 : (s.g <= 512 ? 2 : 1));
  const int64_t want = (kSms * per_sm + g.groups - 1) / g.groups;
  return (int)(steps < want ? steps : want);
}

#define NORM_BOTH_SHAPES(F, T, V) \
  F(T, V, 8, 1) F(T, V, 16, 1) F(T, V, 32, 1) F(T, V, 32, 2) F(T, V, 512, 2) F(T, V, 512, 4)
#define NORM_FWD_SHAPES(F, T, V) NORM_BOTH_SHAPES(F, T, V) F(T, V, 32, 3) F(T, V, 32, 4) F(T, V, 128, 2) F(T, V, 256, 2)
#define NORM_BWD_SHAPES(F, T, V) NORM_BOTH_SHAPES(F, T, V) F(T, V, 256, 1) F(T, V, 512, 1)
#define NORM_FEW_SHAPES(F, T, V) \
  F(T, V, 8, 1) F(T, V, 8, 2) F(T, V, 8, 4) F(T, V, 16, 4) F(T, V, 32, 4) F(T, V, 128, 2) F(T, V, 128, 4) \
  F(T, V, 256, 4) F(T, V, 512, 4) F(T, V, 512, 8)
#define NORM_ONE_SHAPES(F, T) \
  F(T, 1, 8, 1) F(T, 1, 8, 2) F(T, 1, 8, 4) F(T, 1, 8, 8) F(T, 1, 16, 8) F(T, 1, 32, 8) F(T, 1, 128, 4) \
  F(T, 1, 512, 4) F(T, 1, 512, 8) F(T, 1, 1024, 16)

cudaError_t launch_fwd(const Geo& g, const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                       cudaStream_t s) {
  const Shape sh = shape_of(g, false);
  const int rows = rows_per_block(sh);
  const int64_t steps = (g.rows + rows - 1) / rows;
  const int64_t most = (int64_t)kSms * (sh.g <= 256 ? 8 : (sh.g <= 512 ? 4 : 2));
  const int64_t want = (most + g.groups - 1) / g.groups;
  const dim3 grid((unsigned)(steps < want ? steps : want), (unsigned)g.groups);
#define NORM_FWD(T, VV, GG, II)                                                                              \
  if (sh.v == VV && sh.g == GG && sh.it == II) {                                                                           \
    fwd_kernel<T, VV, GG, II><<<grid, threads<GG>(), 0, s>>>(g, (const T*)x, w, b, (T*)y, mean, rstd);       \
    note_launches(1);                                                                                        \
    return cudaGetLastError();                                                                               \
  }
  if (g.bf16) {
    NORM_FWD_SHAPES(NORM_FWD, __nv_bfloat16, 8) NORM_FWD(__nv_bfloat16, 4, 32, 3)
    NORM_FEW_SHAPES(NORM_FWD, __nv_bfloat16, 4) NORM_FEW_SHAPES(NORM_FWD, __nv_bfloat16, 2)
    NORM_FWD(__nv_bfloat16, 2, 1024, 8)
    NORM_ONE_SHAPES(NORM_FWD, __nv_bfloat16) NORM_FWD(__nv_bfloat16, 1, 128, 8) NORM_FWD(__nv_bfloat16, 1, 1024, 8)
  } else {
    NORM_FWD_SHAPES(NORM_FWD, float, 4) NORM_FWD(float, 4, 16, 3) NORM_FWD(float, 4, 1024, 4)
    NORM_FEW_SHAPES(NORM_FWD, float, 2) NORM_FWD(float, 2, 1024, 8)
    NORM_ONE_SHAPES(NORM_FWD, float) NORM_FWD(float, 1, 128, 8) NORM_FWD(float, 1, 1024, 8)
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_bwd(const Geo& g, const void* x, const void* dy, const void* w, const float* mean,
                       const float* rstd, void* dx, void* dw, void* db, void* work, cudaStream_t s) {
  const Shape sh = shape_of(g, true);
  const int parts = bwd_parts(g);
  const dim3 grid((unsigned)parts, (unsigned)g.groups);
  float* part = (dw || db) ? static_cast<float*>(work) : nullptr;
  cudaError_t e = cudaErrorInvalidValue;
#define NORM_BWD(T, VV, GG, II)                                                                                     \
  if (sh.v == VV && sh.g == GG && sh.it == II) {                                                                                  \
    bwd_kernel<T, VV, GG, II>                                                                                       \
        <<<grid, threads<GG>(), 0, s>>>(g, (const T*)x, (const T*)dy, w, mean, rstd, (T*)dx, part);                 \
    note_launches(1);                                                                                               \
    e = cudaGetLastError();                                                                                         \
  }
  if (g.bf16) {
    NORM_BWD_SHAPES(NORM_BWD, __nv_bfloat16, 8) NORM_BWD(__nv_bfloat16, 8, 128, 1) NORM_BWD(__nv_bfloat16, 4, 32, 3)
    NORM_FEW_SHAPES(NORM_BWD, __nv_bfloat16, 4) NORM_FEW_SHAPES(NORM_BWD, __nv_bfloat16, 2)
    NORM_BWD(__nv_bfloat16, 2, 1024, 8)
    NORM_ONE_SHAPES(NORM_BWD, __nv_bfloat16) NORM_BWD(__nv_bfloat16, 1, 256, 4) NORM_BWD(__nv_bfloat16, 1, 512, 16)
  } else {
    NORM_BWD_SHAPES(NORM_BWD, float, 4) NORM_BWD(float, 4, 16, 3) NORM_BWD(float, 4, 32, 3) NORM_BWD(float, 4, 32, 4) NORM_BWD(float, 4, 1024, 4)
    NORM_FEW_SHAPES(NORM_BWD, float, 2) NORM_BWD(float, 2, 1024, 8)
    NORM_ONE_SHAPES(NORM_BWD, float) NORM_BWD(float, 1, 256, 4) NORM_BWD(float, 1, 512, 16)
  }
  if (e != cudaSuccess || !part) return e;
  const dim3 fgrid((unsigned)((g.c + 31) / 32), (unsigned)g.groups, 2);
  finish_kernel<<<fgrid, 1024, 0, s>>>(part, parts, g.c, g.param_bf16, dw, db);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace norm
}  // namespace llsa
