// k_norm.cu -- layer norm of token rows, forward and backward.
//
//   y = (x - mean) rstd w + b;
//   g = dy w,  xhat = (x - mean) rstd,
//   dx = rstd (g - mean_c(g) - xhat mean_c(g xhat)),  dw = sum_rows dy xhat,  db = sum_rows dy.
//
// Bound by memory: every row is read once and kept in registers (the variance
// is the mean of the squared deviations from the mean, in a second pass over
// the registers, so that large offsets cost no digits).  G threads work on a
// row, each on IT vectors of 16 bytes (single values where the width, a stride
// or an address does not allow vectors); rows of up to 4 KB take a part of a warp or
// a warp, wider ones a block.  Rows are walked in the order of x's memory.
//
// In the backward every thread keeps the same channels for all its rows and
// sums dy xhat and dy in registers; a block adds up its row groups (by
// shuffles, then through shared memory, in a fixed order) and writes one
// partial row, and a second kernel adds the partial rows: no atomics, the same
// bits every time.
#include "norm.cuh"

namespace llsa {
namespace norm {

template <typename T, int V> struct Raw;
template <> struct Raw<__nv_bfloat16, 8> { uint4 w; };
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
__device__ __forceinline__ void unpack(const Raw<float, 4>& r, float* f) {
  f[0] = r.w.x;
  f[1] = r.w.y;
  f[2] = r.w.z;
  f[3] = r.w.w;
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
__device__ __forceinline__ void pack(Raw<float, 4>& r, const float* f) { r.w = make_float4(f[0], f[1], f[2], f[3]); }
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
  const uint32_t q = r / g.n2;
  return At{(int64_t)(q / g.n1), (int64_t)(q % g.n1), (int64_t)(r % g.n2)};
}
__device__ __forceinline__ int64_t offset(const At& a, const int64_t* st, int group) {
  return a.i0 * st[0] + a.i1 * st[1] + a.i2 * st[2] + group * st[3];
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

template <typename T, int V, int G, int IT>
__global__ void __launch_bounds__(threads<G>()) fwd_kernel(const __grid_constant__ Geo g, const T* x, const void* w,
                                                           const void* b, T* y, float* mean, float* rstd) {
  constexpr int RPB = threads<G>() / G;              // rows per block and step
  __shared__ float red[G > 32 ? 2 * 32 : 1];
  int turn = 0;
  const int sub = threadIdx.x % G, slot = threadIdx.x / G;
  const int group = blockIdx.y;
  const float inv_c = 1.f / (float)g.c;
  float wv[IT * V], bv[IT * V];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * G + sub) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      wv[i * V + e] = 1.f;
      bv[i * V + e] = 0.f;
    }
    if (c < g.c) {
      if (w) load_param<V>(w, g.param_bf16, group * g.ws + c, wv + i * V);
      if (b) load_param<V>(b, g.param_bf16, group * g.bs + c, bv + i * V);
    }
  }
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < g.rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = r0 + slot;
    const bool live = r < g.rows;
    const At at = place(g, live ? r : 0);
    const T* px = x + offset(at, g.x, group);
    Raw<T, V> raw[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
      if (live && c < g.c) raw[i] = *reinterpret_cast<const Raw<T, V>*>(px + c);
    }
    float f[IT * V];
    float sum[1] = {0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
      if (live && c < g.c) {
        unpack(raw[i], f + i * V);
#pragma unroll
        for (int e = 0; e < V; ++e) sum[0] += f[i * V + e];
      }
    }
    row_sum<G, 1>(sum, red, turn);
    const float mu = sum[0] * inv_c;
    float sq[1] = {0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
      if (live && c < g.c)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[i * V + e] -= mu;
          sq[0] = fmaf(f[i * V + e], f[i * V + e], sq[0]);
        }
    }
    row_sum<G, 1>(sq, red, turn);
    const float rs = 1.f / sqrtf(fmaf(sq[0], inv_c, g.eps));
    if (!live) continue;
    T* py = y + offset(at, g.y, group);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
      if (c >= g.c) continue;
      float out[V];
#pragma unroll
      for (int e = 0; e < V; ++e) out[e] = fmaf(f[i * V + e] * rs, wv[i * V + e], bv[i * V + e]);
      Raw<T, V> o;
      pack(o, out);
      *reinterpret_cast<Raw<T, V>*>(py + c) = o;
    }
    if (sub == 0) {
      const int64_t st = offset(at, g.s, group);
      if (mean) mean[st] = mu;
      if (rstd) rstd[st] = rs;
    }
  }
}

template <typename T, int V, int G, int IT>
__global__ void __launch_bounds__(threads<G>()) bwd_kernel(const __grid_constant__ Geo g, const T* x, const T* dy,
                                                           const void* w, const float* __restrict__ mean,
                                                           const float* __restrict__ rstd, T* dx,
                                                           float* __restrict__ part) {
  constexpr int RPB = threads<G>() / G;
  constexpr int NV = IT * V;
  __shared__ float red[G > 32 ? 2 * 2 * 32 : 1];
  __shared__ float cols[G <= 32 ? 8 * G * NV : 1];   // a block's eight warps' sums
  int turn = 0;
  const int sub = threadIdx.x % G, slot = threadIdx.x / G;
  const int group = blockIdx.y;
  const float inv_c = 1.f / (float)g.c;
  // narrow rows keep the weights in registers; a block-wide row reads them again (from L1)
  float wv[G <= 32 ? NV : 1];
  if constexpr (G <= 32) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
#pragma unroll
      for (int e = 0; e < V; ++e) wv[i * V + e] = 1.f;
      if (w && c < g.c) load_param<V>(w, g.param_bf16, group * g.ws + c, wv + i * V);
    }
  }
  float dw[NV], db[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) dw[i] = db[i] = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < g.rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = r0 + slot;
    const bool live = r < g.rows;
    const At at = place(g, live ? r : 0);
    const T* px = x + offset(at, g.x, group);
    const T* pg = dy + offset(at, g.dy, group);
    const int64_t st = offset(at, g.s, group);
    Raw<T, V> rx[IT], rg[IT];
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
      if (live && c < g.c) {
        rx[i] = *reinterpret_cast<const Raw<T, V>*>(px + c);
        rg[i] = *reinterpret_cast<const Raw<T, V>*>(pg + c);
      }
    }
    const float mu = live ? mean[st] : 0.f, rs = live ? rstd[st] : 0.f;
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
      if (live && c < g.c) {
        float fx[V], fg[V], ww[V];
        unpack(rx[i], fx);
        unpack(rg[i], fg);
        if constexpr (G <= 32) {
#pragma unroll
          for (int e = 0; e < V; ++e) ww[e] = wv[i * V + e];
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) ww[e] = 1.f;
          if (w) load_param<V>(w, g.param_bf16, group * g.ws + c, ww);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float xh = (fx[e] - mu) * rs, gw = fg[e] * ww[e];
          sum[0] += gw;
          sum[1] = fmaf(gw, xh, sum[1]);
          dw[i * V + e] = fmaf(fg[e], xh, dw[i * V + e]);
          db[i * V + e] += fg[e];
        }
      }
    }
    if (dx) {                                          // uniform over the grid
      row_sum<G, 2>(sum, red, turn);
      const float c1 = sum[0] * inv_c, c2 = sum[1] * inv_c;
      T* po = dx + offset(at, g.dx, group);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * G + sub) * V;
        if (live && c < g.c) {
          float fx[V], fg[V], ww[V];
          unpack(rx[i], fx);
          unpack(rg[i], fg);
          if constexpr (G <= 32) {
#pragma unroll
            for (int e = 0; e < V; ++e) ww[e] = wv[i * V + e];
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) ww[e] = 1.f;
            if (w) load_param<V>(w, g.param_bf16, group * g.ws + c, ww);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float xh = (fx[e] - mu) * rs, gw = fg[e] * ww[e];
            fx[e] = rs * (gw - c1 - xh * c2);
          }
          Raw<T, V> o;
          pack(o, fx);
          *reinterpret_cast<Raw<T, V>*>(po + c) = o;
        }
      }
    }
  }
  if (!part) return;
  float* out = part + ((int64_t)group * gridDim.x + blockIdx.x) * 2 * g.c;
  if constexpr (G > 32) {
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * G + sub) * V;
      if (c < g.c)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          out[c + e] = dw[i * V + e];
          out[g.c + c + e] = db[i * V + e];
        }
    }
  } else {
    // the row groups of a warp by shuffles, then the eight warps in order
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int s = 16; s >= G; s >>= 1) {
        dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], s);
        db[i] += __shfl_xor_sync(0xffffffffu, db[i], s);
      }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
      if (lane < G)
#pragma unroll
        for (int i = 0; i < NV; ++i) cols[(warp * NV + i) * G + lane] = which ? db[i] : dw[i];
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
#pragma unroll 4
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

// Threads per row and vectors per thread.  Vectors: the narrowest set of
// threads whose registers hold the row with at most 4 vectors each; single
// values: up to 16 of them.
struct Shape {
  int g, it;
};
static Shape shape_of(const Geo& g) {
  if (g.vec) {
    const int n = g.c / (g.bf16 ? 8 : 4);
    if (n <= 8) return {8, 1};
    if (n <= 16) return {16, 1};
    if (n <= 32) return {32, 1};
    if (n <= 48) return {16, 3};
    if (n <= 64) return {32, 2};
    if (n <= 96) return {32, 3};
    if (n <= 128) return {32, 4};
    if (n <= 256) return {128, 2};
    if (n <= 512) return {256, 2};
    if (n <= 1024) return {512, 2};
    if (n <= 2048) return {512, 4};
    return {1024, 4};
  }
  if (g.c <= 8) return {8, 1};
  if (g.c <= 32) return {32, 1};
  if (g.c <= 128) return {32, 4};
  if (g.c <= 256) return {32, 8};
  if (g.c <= 1024) return {128, 8};
  if (g.c <= 4096) return {512, 8};
  return {1024, 16};
}

static int rows_per_block(const Shape& s) { return s.g <= 32 ? 256 / s.g : 1; }

// Blocks per group in the backward: enough to fill the device, no more than there are row steps.
int bwd_parts(const Geo& g) {
  const Shape s = shape_of(g);
  const int64_t steps = (g.rows + rows_per_block(s) - 1) / rows_per_block(s);
  const int per_sm = s.g <= 32 ? 4 : (s.g <= 256 ? 4 : (s.g <= 512 ? 2 : 1));
  const int64_t want = (kSms * per_sm + g.groups - 1) / g.groups;
  return (int)(steps < want ? steps : want);
}

#define NORM_VEC_SHAPES(F, T, V) \
  F(T, V, 8, 1) F(T, V, 16, 1) F(T, V, 32, 1) F(T, V, 16, 3) F(T, V, 32, 2) F(T, V, 32, 3) F(T, V, 32, 4) \
  F(T, V, 128, 2) F(T, V, 256, 2) F(T, V, 512, 2) F(T, V, 512, 4)
#define NORM_ONE_SHAPES(F, T) \
  F(T, 1, 8, 1) F(T, 1, 32, 1) F(T, 1, 32, 4) F(T, 1, 32, 8) F(T, 1, 128, 8) F(T, 1, 512, 8) F(T, 1, 1024, 16)

cudaError_t launch_fwd(const Geo& g, const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                       cudaStream_t s) {
  const Shape sh = shape_of(g);
  const int64_t steps = (g.rows + rows_per_block(sh) - 1) / rows_per_block(sh);
  const int64_t most = (int64_t)kSms * (sh.g <= 256 ? 8 : (sh.g <= 512 ? 4 : 2));
  const int64_t want = (most + g.groups - 1) / g.groups;
  const dim3 grid((unsigned)(steps < want ? steps : want), (unsigned)g.groups);
#define NORM_FWD(T, VV, GG, II)                                                                              \
  if (sh.g == GG && sh.it == II) {                                                                           \
    fwd_kernel<T, VV, GG, II><<<grid, threads<GG>(), 0, s>>>(g, (const T*)x, w, b, (T*)y, mean, rstd);       \
    note_launches(1);                                                                                        \
    return cudaGetLastError();                                                                               \
  }
  if (g.bf16) {
    if (g.vec) { NORM_VEC_SHAPES(NORM_FWD, __nv_bfloat16, 8) } else { NORM_ONE_SHAPES(NORM_FWD, __nv_bfloat16) }
  } else {
    if (g.vec) { NORM_VEC_SHAPES(NORM_FWD, float, 4) NORM_FWD(float, 4, 1024, 4) } else { NORM_ONE_SHAPES(NORM_FWD, float) }
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_bwd(const Geo& g, const void* x, const void* dy, const void* w, const float* mean,
                       const float* rstd, void* dx, void* dw, void* db, void* work, cudaStream_t s) {
  const Shape sh = shape_of(g);
  const int parts = bwd_parts(g);
  const dim3 grid((unsigned)parts, (unsigned)g.groups);
  float* part = (dw || db) ? static_cast<float*>(work) : nullptr;
  cudaError_t e = cudaErrorInvalidValue;
#define NORM_BWD(T, VV, GG, II)                                                                                     \
  if (sh.g == GG && sh.it == II) {                                                                                  \
    bwd_kernel<T, VV, GG, II>                                                                                       \
        <<<grid, threads<GG>(), 0, s>>>(g, (const T*)x, (const T*)dy, w, mean, rstd, (T*)dx, part);                 \
    note_launches(1);                                                                                               \
    e = cudaGetLastError();                                                                                         \
  }
  if (g.bf16) {
    if (g.vec) { NORM_VEC_SHAPES(NORM_BWD, __nv_bfloat16, 8) } else { NORM_ONE_SHAPES(NORM_BWD, __nv_bfloat16) }
  } else {
    if (g.vec) { NORM_VEC_SHAPES(NORM_BWD, float, 4) NORM_BWD(float, 4, 1024, 4) } else { NORM_ONE_SHAPES(NORM_BWD, float) }
  }
  if (e != cudaSuccess || !part) return e;
  const dim3 fgrid((unsigned)((g.c + 31) / 32), (unsigned)g.groups, 2);
  finish_kernel<<<fgrid, 1024, 0, s>>>(part, parts, g.c, g.param_bf16, dw, db);
  note_launches(1);
  return cudaGetLastError();
}

}  // namespace norm
}  // namespace llsa
