// k_cross_bwd_kv_tc.cu -- dK and dV of cross attention on the 5th-generation
// tensor cores, for encoders of more than one tile of keys.
//
// An item is one tile of 128 keys of a key head against a run of query tiles
// (of all query heads that share it).  The scores are computed transposed,
// keys in the rows, so that P and dS come out as the left operands of the
// second products and never leave tensor memory:
//   S^T = K Q^T, dP^T = V dO^T            (M = 128 keys, N = 128 queries)
//   P^T = 2^(z - lse), dS^T = P^T o (dP^T - D)   bf16, over the columns they came from
//   dV += P^T dO, dK += dS^T Q            (A from TMEM, accumulated in TMEM over the item)
// lse and D of a tile's queries stand in shared memory, one pair per column.
// Two threads share a key's row, each half of the query columns.  Two warps
// issue MMAs, one the products around P, one those around dS: while one pair
// runs, the softmax works on the other.  A key that takes no part has weights
// of zero whatever its row holds (rows do not mix), and its gradients are
// written as zero.
//
// Items that split a key tile's queries leave fp32 partial sums, added in
// order by a second kernel: no atomics.
//
// 4096 queries of 16 heads on 4 key heads, 589 states, 128 channels, batch 2
// (a key mask): 113 us, 760 TFLOP/s; bound by the two chains of
// scores, weights and product, which overlap only with each other.
//
// Warps: 0-7 softmax, 8-11 epilogue, 12 producer of Q and dO (TMA), 13 MMA issue
// of S and dV, 14 of dP and dK, 15 K and V, lse and D; also gathers Q and dO
// where heads are packed.
#include <math.h>

#include "cross_tc.cuh"

namespace llsa {
namespace cross {
namespace bwdkv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int THREADS = 512;
constexpr int EPI0 = 8, PRODUCER = 12, MMA0 = 13, STATS = 15;
constexpr int NSTAT = 4;                       // tiles of lse and D in flight
constexpr uint32_t TMEM_COLS = 512;

struct Args {
  Geo g;
  Keys keys;
  Where wq, wk, wv, wg;
  int packed, qs, nqt, units, tiles;           // query splits, query tiles per head and per key head, key tiles
  int items;
  Divisor by_qs, by_tiles, by_hk, by_nqt, by_nq;
  const void *q, *dO;
  const float *lse, *D;
  void *dk, *dv;
  float *partk, *partv;
  int* err;
};

template <int NP>
struct Smem {
  static constexpr int ST = NP == 1 ? 4 : 2;   // tiles of Q and dO in flight
  alignas(1024) unsigned char k[NP * kPanel];
  alignas(1024) unsigned char v[NP * kPanel];
  alignas(1024) unsigned char q[ST][NP * kPanel];
  alignas(1024) unsigned char dO[ST][NP * kPanel];
  alignas(16) float ls[NSTAT][kTile], dd[NSTAT][kTile];
  alignas(8) uint64_t kvfull, kvempty, acc_full, acc_empty;
  uint64_t full[ST], empty[ST], st_full[NSTAT], st_empty[NSTAT];
  uint64_t s_full[2], w_full[2], w_done[2], drain[2];    // scores, weights, their second product: of P and of dS
  uint32_t tmem_base;
};
static_assert(sizeof(Smem<1>) + 1024 <= 232448 && sizeof(Smem<2>) + 1024 <= 232448, "shared memory of one CTA");

struct Item {
  int b, hk, split, key0, u0, n;               // first key, first query tile and tiles (none behind the length)
  int len;
};
__device__ __forceinline__ Item item_of(const Args& a, int it) {
  Item x;
  int tile;
  x.b = divide(divide(divide(it, a.by_qs, x.split), a.by_tiles, tile), a.by_hk, x.hk);
  x.len = key_count(a.g, a.keys, x.b);
  x.key0 = tile * kTile;
  x.u0 = (int)((int64_t)a.units * x.split / a.qs);
  x.n = x.key0 < x.len ? (int)((int64_t)a.units * (x.split + 1) / a.qs) - x.u0 : 0;
  return x;
}
// Row r of query tile u: its head and token; false behind the last row.
__device__ __forceinline__ bool row_of(const Args& a, int hk, int u, int r, int& h, int& n) {
  if (a.packed) {
    const int rr = u * kTile + r;
    h = hk * a.g.group + divide(rr, a.by_nq, n);
    return rr < a.g.group * a.g.nq;
  }
  int tile;
  h = hk * a.g.group + divide(u, a.by_nqt, tile);
  n = tile * kTile + r;
  return n < a.g.nq;
}
// Columns of query tile u that are computed: its rows, rounded up to 32.
__device__ __forceinline__ int tile_cols(const Args& a, int u) {
  int tile = u;
  if (!a.packed) divide(u, a.by_nqt, tile);
  const int left = (a.packed ? a.g.group * a.g.nq : a.g.nq) - tile * kTile;
  return left >= kTile ? kTile : (left + 31) & ~31;
}

template <int NP>
__global__ void __launch_bounds__(THREADS, 1)
bwd_kv_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tq,
              const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
              const __grid_constant__ CUtensorMap tg) {
  using Sm = Smem<NP>;
  constexpr int ST = Sm::ST;
  constexpr uint32_t kBytes = NP * kPanel;
  // TMEM columns: scores r (S^T, dP^T; bf16 weights over them), accumulators r (dV, dK)
  auto col_s = [](int r) { return 128u * r; };
  auto col_a = [](int r) { return 256u + 64u * NP * r; };
  extern __shared__ __align__(1024) unsigned char raw[];
  Sm& s = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const Geo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&s.kvfull, 1);
    ptx::mbar_init(&s.kvempty, 2);
    ptx::mbar_init(&s.acc_full, 2);
    ptx::mbar_init(&s.acc_empty, 4);
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 2);
    }
    for (int i = 0; i < NSTAT; ++i) {
      ptx::mbar_init(&s.st_full[i], 1);
      ptx::mbar_init(&s.st_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s.s_full[i], 1);
      ptx::mbar_init(&s.w_full[i], 8);
      ptx::mbar_init(&s.w_done[i], 1);
      ptx::mbar_init(&s.drain[i], 1);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 0) {
    tc::tmem_alloc(&s.tmem_base, TMEM_COLS);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tbase = s.tmem_base;
  bool ok = true;
  // Every lane of a warp waits, and all go on together or all give up together.
  auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
    if (!ok) return false;
    ok = warp_wait(bar, parity);
    if (!ok && lane == 0) report(a.err, code);
    return ok;
  };
  auto arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
    __syncwarp();
  };

  if (warp < 8) {
    // ============================================================ softmax: half of the queries of a key
    const int half = warp >> 2, sub = warp & 3;
    const uint32_t tl = tbase + ((uint32_t)(sub * 32) << 16);
    const float sc2 = g.scale * kLog2e;
    uint32_t tc_ = 0;                          // query tiles so far
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.n == 0) continue;
      const int key = x.key0 + sub * 32 + lane;
      const bool valid = key < x.len && (!a.keys.mask || a.keys.mask[(int64_t)x.b * g.nk + key]);
      for (int i = 0; i < x.n; ++i, ++tc_) {
        const int chunks = tile_cols(a, x.u0 + i) >> 5;  // 16 columns each, in this half
        const uint32_t col0 = 16u * chunks * half;
        const uint32_t ph = tc_ & 1, si = tc_ % NSTAT;
        if (!wait(&s.st_full[si], (tc_ / NSTAT) & 1, 141)) break;
        if (!wait(&s.s_full[0], ph, 141)) break;
        tc::fence_after_sync();
        const uint32_t cs = tl + col_s(0) + col0, cd = tl + col_s(1) + col0;
        float p[64];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) {
            uint32_t r[16], w[8];
            tc::tmem_ld16(cs + 16u * c, r);
            const float4* l4 = reinterpret_cast<const float4*>(&s.ls[si][col0 + 16 * c]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 l = l4[e];
              const float ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
              for (int f = 0; f < 4; ++f) {
                const float y = ptx::ex2(fmaf(__uint_as_float(r[4 * e + f]), sc2, -ls[f]));
                p[16 * c + 4 * e + f] = valid ? y : 0.f;
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = ptx::pack_bf16(p[16 * c + 2 * e], p[16 * c + 2 * e + 1]);
            tc::tmem_st8(cs + 8u * c, w);      // (over columns of this thread's own that are in registers)
          }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        arrive(&s.w_full[0]);
        if (!wait(&s.s_full[1], ph, 142)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) {
            uint32_t r[16], w[8];
            tc::tmem_ld16(cd + 16u * c, r);
            const float4* d4 = reinterpret_cast<const float4*>(&s.dd[si][col0 + 16 * c]);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 d = d4[e];
              const float* pe = p + 16 * c + 4 * e;
              const float y0 = pe[0] * (__uint_as_float(r[4 * e]) - d.x), y1 = pe[1] * (__uint_as_float(r[4 * e + 1]) - d.y);
              const float y2 = pe[2] * (__uint_as_float(r[4 * e + 2]) - d.z),
                          y3 = pe[3] * (__uint_as_float(r[4 * e + 3]) - d.w);
              w[2 * e] = valid ? ptx::pack_bf16(y0, y1) : 0u;
              w[2 * e + 1] = valid ? ptx::pack_bf16(y2, y3) : 0u;
            }
            tc::tmem_st8(cd + 8u * c, w);
          }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&s.w_full[1]);
          ptx::mbar_arrive(&s.st_empty[si]);
        }
        __syncwarp();
      }
    }
  } else if (warp < EPI0 + 4) {
    // ============================================================ epilogue
    const int sub = warp & 3;
    const uint32_t tl = tbase + ((uint32_t)(sub * 32) << 16);
    const int c16 = (g.d + 15) >> 4;
    uint32_t ac = 0;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      const bool none = x.n == 0;
      if (!none) {
        if (!wait(&s.acc_full, ac & 1, 143)) break;
        tc::fence_after_sync();
        ++ac;
      }
      const int key = x.key0 + sub * 32 + lane;
      const bool live = key < g.nk;
      const bool valid = key < x.len && (!a.keys.mask || a.keys.mask[(int64_t)x.b * g.nk + key]);
      const int64_t at = ((int64_t)x.split * keys_of(g) + ((int64_t)x.b * g.hk + x.hk) * g.nk + key) * g.d;
#pragma unroll 1
      for (int r = 0; r < 2; ++r) {
        __nv_bfloat16* out = r ? static_cast<__nv_bfloat16*>(a.dk) + x.b * g.dk.b + x.hk * g.dk.h + key * g.dk.n
                               : static_cast<__nv_bfloat16*>(a.dv) + x.b * g.dv.b + x.hk * g.dv.h + key * g.dv.n;
        float* part = (r ? a.partk : a.partv) + at;
        const float f = r ? g.scale : 1.f;
#pragma unroll 1
        for (int c = 0; c < c16; ++c) {
          uint32_t w[16];
          if (!none) {
            tc::tmem_ld16(tl + col_a(r) + 16u * c, w);
            tc::tmem_wait_ld();
          }
          float y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = none || !valid ? 0.f : __uint_as_float(w[e]) * f;
          if (live) store16(y, a.qs > 1 ? nullptr : out + 16 * c, part + 16 * c, 16 * c + 8 < g.d);
          __syncwarp();
        }
      }
      if (!none) {
        tc::fence_before_sync();
        arrive(&s.acc_empty);
      }
    }
  } else if (warp == PRODUCER) {
    // ============================================================ producer of Q and dO
    if (lane == 0) {
      auto wait1 = [&](uint64_t* bar, uint32_t parity, int code) {
        if (ok && !ptx::mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
          ok = false;
          report(a.err, code);
        }
        return ok;
      };
      uint32_t tc_ = 0;
      for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
        const Item x = item_of(a, it);
        for (int i = 0; i < x.n && !a.packed; ++i) {
          const uint32_t st = tc_ % ST;
          if (!wait1(&s.empty[st], ((tc_ / ST) & 1) ^ 1, 144)) break;
          int n0;
          const int h = x.hk * g.group + divide(x.u0 + i, a.by_nqt, n0);
          n0 *= kTile;
          ptx::mbar_arrive_expect_tx(&s.full[st], 2 * kBytes);
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            tma_load_4d(s.q[st] + p * kPanel, &tq, 64 * p, n0, h * a.wq.h, x.b * a.wq.b, &s.full[st]);
            tma_load_4d(s.dO[st] + p * kPanel, &tg, 64 * p, n0, h * a.wg.h, x.b * a.wg.b, &s.full[st]);
          }
          ++tc_;
        }
      }
      // After a timeout, do not leave while copies issued here may still be landing.
      if (!ok) {
        for (uint32_t c = tc_ > ST ? tc_ - ST : 0; c < tc_; ++c)
          ptx::mbar_wait_bounded(&s.full[c % ST], (c / ST) & 1, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == STATS) {
    // ============================================================ K and V; lse and D; packed rows of Q and dO
    uint32_t tc_ = 0, ic = 0;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.n == 0) continue;
      if (!wait(&s.kvempty, (ic & 1) ^ 1, 144)) break;
      ++ic;
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&s.kvfull, 2 * kBytes);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          tma_load_4d(s.k + p * kPanel, &tk, 64 * p, x.key0, x.hk * a.wk.h, x.b * a.wk.b, &s.kvfull);
          tma_load_4d(s.v + p * kPanel, &tv, 64 * p, x.key0, x.hk * a.wv.h, x.b * a.wv.b, &s.kvfull);
        }
      }
      __syncwarp();
      for (int i = 0; i < x.n; ++i, ++tc_) {
        const uint32_t st = tc_ % ST, si = tc_ % NSTAT;
        auto at = [&](int r, int& h, int& n) { return row_of(a, x.hk, x.u0 + i, r, h, n); };
        float l[4], d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          int h, n;
          const bool live = at(32 * e + lane, h, n);
          const int64_t row = ((int64_t)x.b * g.h + h) * g.nq + n;
          l[e] = live ? a.lse[row] : -INFINITY;
          l[e] = l[e] == -INFINITY ? INFINITY : l[e] * kLog2e;     // no key, or no row: every weight is 2^-inf = 0
          d[e] = live ? a.D[row] : 0.f;
        }
        if (!wait(&s.st_empty[si], ((tc_ / NSTAT) & 1) ^ 1, 145)) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s.ls[si][32 * e + lane] = l[e];
          s.dd[si][32 * e + lane] = d[e];
        }
        arrive(&s.st_full[si]);
        if (a.packed) {
          if (!wait(&s.empty[st], ((tc_ / ST) & 1) ^ 1, 145)) break;
          gather_rows<NP>(s.q[st], static_cast<const __nv_bfloat16*>(a.q) + x.b * g.q.b, g.q, g.d, lane, at);
          gather_rows<NP>(s.dO[st], static_cast<const __nv_bfloat16*>(a.dO) + x.b * g.dO.b, g.dO, g.d, lane, at);
          ptx::fence_proxy_async();
          arrive(&s.full[st]);
        }
      }
    }
    if (!ok && lane == 0 && ic) ptx::mbar_wait_bounded(&s.kvfull, (ic - 1) & 1, kWaitLimitNs);   // (as above)
    __syncwarp();
  } else {
    // ============================================================ MMA issue: r = 0: S^T and dV, r = 1: dP^T and dK
    const int r = warp - MMA0;
    const uint64_t first = tc::sw128_desc(ptx::smem_u32(r ? s.v : s.k), 16, 1024);
    const uint64_t second = tc::sw128_desc(ptx::smem_u32(r ? s.dO[0] : s.q[0]), 16, 1024);       // N = queries, K-major
    const uint64_t third = tc::sw128_desc(ptx::smem_u32(r ? s.q[0] : s.dO[0]), kPanel, 1024);    // N = channels, MN-major
    const int dsteps = (g.d + 15) >> 4;
    const uint32_t id_acc = tc::idesc_bf16(128, 16 * dsteps, 0, 1);
    const uint32_t cs = tbase + col_s(r), ca = tbase + col_a(r);
    constexpr uint64_t kStep = kBytes >> 4;
    uint32_t tc_ = 0, ic = 0;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.n == 0) continue;
      if (!wait(&s.kvfull, ic & 1, 146)) break;
      for (int i = 0; i < x.n; ++i) {
        const uint32_t c = tc_ + i, ph = c & 1, st = c % ST;
        const int cols = tile_cols(a, x.u0 + i);
        if (!wait(&s.full[st], (c / ST) & 1, 146)) break;
        if (!wait(&s.w_done[r], ph ^ 1, 146)) break;     // the weights of the tile before, in these columns, are used
        tc::fence_after_sync();
        const uint32_t id = tc::idesc_bf16(128, cols, 0, 0);
        if (tc::elect_one()) {
          for (int k = 0; k < dsteps; ++k) {
            const uint64_t o = (uint64_t)(k >> 2) * (kPanel >> 4) + 2u * (k & 3);
            tc::mma_bf16(cs, first + o, second + st * kStep + o, id, k > 0);
          }
          tc::commit(&s.s_full[r]);
        }
        __syncwarp();
        if (!wait(&s.w_full[r], ph, 146)) break;
        if (i == 0 && !wait(&s.acc_empty, (ic & 1) ^ 1, 146)) break;
        tc::fence_after_sync();
        const int steps = cols >> 4, mid = steps >> 1;
        if (tc::elect_one()) {
          for (int k = 0; k < steps; ++k)      // 16 queries: 8 columns of weights (the second half's at its own scores)
            tc::mma_bf16_ta(ca, cs + (k < mid ? 8u * k : 16u * mid + 8u * (k - mid)), third + st * kStep + 128u * k,
                            id_acc, i > 0 || k > 0);
          tc::commit(&s.w_done[r]);
          tc::commit(&s.empty[st]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (tc::elect_one()) {
        tc::commit(&s.acc_full);
        tc::commit(&s.kvempty);
      }
      __syncwarp();
      tc_ += x.n;
      ++ic;
    }
    // every MMA issued here has finished before TMEM is released
    if (tc::elect_one()) tc::commit(&s.drain[r]);
    __syncwarp();
    ptx::mbar_wait_bounded(&s.drain[r], 0, kWaitLimitNs);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, TMEM_COLS);
  }
}

}  // namespace bwdkv

// Query splits as for one tile of keys (fewest tiles one after the other on an SM).
DkvPlan plan_bwd_kv(const Geo& g, int sms) {
  DkvPlan p;
  p.packed = g.group > 1 && g.nq < kTile;
  p.nqt = (g.nq + kTile - 1) / kTile;
  p.units = (int)(p.packed ? ((int64_t)g.group * g.nq + kTile - 1) / kTile : (int64_t)g.group * p.nqt);
  p.tiles = (g.nk + kTile - 1) / kTile;
  const int64_t slices = (int64_t)g.b * g.hk * p.tiles;
  p.qs = splits_of_queries(slices, p.units, sms);
  p.items = slices * p.qs;
  return p;
}

template <int NP>
static cudaError_t launch(const bwdkv::Args& a, const CUtensorMap* t, int grid, cudaStream_t s) {
  const size_t smem = sizeof(bwdkv::Smem<NP>) + 1024;
  cudaError_t e =
      cudaFuncSetAttribute(bwdkv::bwd_kv_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  bwdkv::bwd_kv_kernel<NP><<<grid, bwdkv::THREADS, smem, s>>>(a, t[0], t[1], t[2], t[3]);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_bwd_kv(const Geo& g, const DkvPlan& p, const CUtensorMap* t, const Where* w, const void* q,
                          const Keys& keys, const void* dO, const float* lse, const float* D, void* dk, void* dv,
                          float* partk, float* partv, cudaStream_t s) {
  bwdkv::Args a;
  a.g = g;
  a.keys = keys;
  a.wq = w[0];
  a.wk = w[1];
  a.wv = w[2];
  a.wg = w[3];
  a.packed = p.packed;
  a.qs = p.qs;
  a.nqt = p.nqt;
  a.units = p.units;
  a.tiles = p.tiles;
  a.items = (int)p.items;
  a.by_qs = divisor(p.qs);
  a.by_tiles = divisor(p.tiles);
  a.by_hk = divisor(g.hk);
  a.by_nqt = divisor(p.nqt);
  a.by_nq = divisor(g.nq);
  a.q = q;
  a.dO = dO;
  a.lse = lse;
  a.D = D;
  a.dk = dk;
  a.dv = dv;
  a.partk = partk;
  a.partv = partv;
  a.err = device_error_word();
  const int sms = sm_count();
  const int grid = a.items < sms ? a.items : sms;
  const cudaError_t e = g.d <= 64 ? launch<1>(a, t, grid, s) : launch<2>(a, t, grid, s);
  if (e != cudaSuccess || p.qs == 1) return e;
  return launch_sum_kv(g, p.qs, partk, partv, dk, dv, s);
}

// ------------------------------------------------------------------ the whole backward

bool bwd_tc_supported(const Geo& g) {
  return g.bf16 && tokens_apart(g.q, g.nq) && tokens_apart(g.k, g.nk) && tokens_apart(g.v, g.nk) &&
         tokens_apart(g.dO, g.nq);
}

namespace {
struct TcBwdWork {
  float *D, *dq, *dk, *dv;
};
TcBwdWork carve_tc(const Geo& g, void* work, size_t* bytes, int sms) {
  char* w = static_cast<char*>(work);
  size_t at = 0;
  auto take = [&](size_t n) {
    float* ptr = reinterpret_cast<float*>(w + at);
    at += round256(n);
    return ptr;
  };
  TcBwdWork out{nullptr, nullptr, nullptr, nullptr};
  const size_t kv = (size_t)keys_of(g) * g.d * 4;
  if (g.nk <= kTile) {
    const OnePlan p = plan_bwd_one(g, sms);
    if (p.qs > 1) {
      out.dk = take(p.qs * kv);
      out.dv = take(p.qs * kv);
    }
  } else {
    const DqPlan pq = plan_bwd_q(g, sms);
    const DkvPlan pk = plan_bwd_kv(g, sms);
    out.D = take((size_t)rows_of(g) * 4);
    if (pq.ks > 1) out.dq = take((size_t)pq.ks * rows_of(g) * g.d * 4);
    if (pk.qs > 1) {
      out.dk = take(pk.qs * kv);
      out.dv = take(pk.qs * kv);
    }
  }
  if (bytes) *bytes = at;
  return out;
}
}  // namespace

size_t bwd_work_bytes_tc(const Geo& g, int sms) {
  size_t n = 0;
  carve_tc(g, nullptr, &n, sms);
  return n;
}

cudaError_t launch_bwd_tc(const Geo& g, int sms, const void* q, const void* k, const void* v, const Keys& keys,
                          const void* o, const void* dO, const float* lse, void* dq, void* dk, void* dv, void* work,
                          cudaStream_t s) {
  const TcBwdWork w = carve_tc(g, work, nullptr, sms);
  CUtensorMap t[4];
  Where at[4];
  cudaError_t e = make_map4(&t[0], &at[0], q, g.q, g.h, g.b, g.nq, g.d, kTile);
  if (e == cudaSuccess) e = make_map4(&t[1], &at[1], k, g.k, g.hk, g.b, g.nk, g.d, kTile);
  if (e == cudaSuccess) e = make_map4(&t[2], &at[2], v, g.v, g.hk, g.b, g.nk, g.d, kTile);
  if (e == cudaSuccess) e = make_map4(&t[3], &at[3], dO, g.dO, g.h, g.b, g.nq, g.d, kTile);
  if (e != cudaSuccess) return e;
  if (g.nk <= kTile)
    return launch_bwd_one(g, plan_bwd_one(g, sms), t, at, q, keys, dO, lse, dq, dk, dv, w.dk, w.dv, s);
  e = launch_row_dot(g, o, dO, w.D, s);
  if (e == cudaSuccess) e = launch_bwd_q(g, plan_bwd_q(g, sms), t, at, q, keys, dO, lse, w.D, dq, w.dq, s);
  if (e == cudaSuccess)
    e = launch_bwd_kv(g, plan_bwd_kv(g, sms), t, at, q, keys, dO, lse, w.D, dk, dv, w.dk, w.dv, s);
  return e;
}

}  // namespace cross
}  // namespace llsa
