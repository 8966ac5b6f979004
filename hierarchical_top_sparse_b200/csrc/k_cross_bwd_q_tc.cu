// k_cross_bwd_q_tc.cu -- dQ of cross attention on the 5th-generation tensor
// cores, for encoders of more than one tile of keys.
//
// An item is one tile of 128 query rows against the key tiles of one split:
//   S = Q K^T, dP = dO V^T              (M = 128 queries, N = the tile's keys)
//   dS = 2^(z - lse) o (dP - D)         as two bf16 (the value and what rounding left) over S
//   dQ += dS K                          (A = dS from TMEM, accumulated in TMEM)
// Two threads share a row, each half of a tile's key columns.  S has two
// buffers: the next tile's S is computed while this one's softmax runs, its dP
// while the next exponentials do (116 us for 4096 queries of 16 heads on 4 key
// heads, 589 states, 128 channels, batch 2: 560 TFLOP/s, the rest of dS apart).  D comes from the rounded O; with dS rounded
// as well dQ was 2.6e-3 off (relative to its norm) where the result's own
// rounding makes 1.7e-3; the second bf16 costs products that the tensor cores
// have time for.  Bound by one tile's chain of hand-offs (load S, exponentials, wait for
// dP, dS, hand over): some 6400 cycles a tile in that case, where its exponentials take
// 1024 and its four products 2850, and no second tile of queries fills the gaps.
//
// Warps: 0-7 softmax, 8-11 epilogue, 12 producer of K and V (TMA), 13 MMA
// issue, 14 fetches Q and dO (where heads are packed by plain loads) and clears
// masked rows of K and V.  (One producer for all would hold the next item's
// keys back until this one's queries are done with.)
#include <math.h>

#include "cross_tc.cuh"

namespace llsa {
namespace cross {
namespace bwdq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int THREADS = 480;
constexpr int EPI0 = 8, PRODUCER = 12, MMA = 13, FIXER = 14;
constexpr uint32_t TMEM_COLS = 512, COL_S = 0, COL_DP = 256, COL_DQ = 384;   // two buffers of S

struct Args {
  Geo g;
  Keys keys;
  Where wq, wk, wv, wg;
  int packed, ks, ct, tiles;                   // key splits, key tiles per split, query tiles per slice
  int items;
  Divisor by_ks, by_tiles, by_heads, by_group, by_nq;
  const void *q, *dO;
  const float *lse, *D;
  void* dq;
  float* part;
  int* err;
};

template <int NP>
struct Smem {
  static constexpr int QST = NP == 1 ? 2 : 1, NK = NP == 1 ? 4 : 3, NV = NP == 1 ? 4 : 2;
  alignas(1024) unsigned char q[QST][NP * kPanel];
  alignas(1024) unsigned char dO[QST][NP * kPanel];
  alignas(1024) unsigned char k[NK][NP * kPanel];
  alignas(1024) unsigned char v[NV][NP * kPanel];
  alignas(8) uint64_t qfull[QST], qempty[QST];
  uint64_t kfull[NK], kready[NK], kempty[NK], vfull[NV], vready[NV], vempty[NV];
  uint64_t s_full[2], s_free[2], dp_full, dp_free, ds_full[2], dq_full, dq_free, drain;
  uint32_t tmem_base;
};
static_assert(sizeof(Smem<1>) + 1024 <= 232448 && sizeof(Smem<2>) + 1024 <= 232448, "shared memory of one CTA");

struct Item {
  int b, hk, h, row0, rows, split, key0, n, len;
};
__device__ __forceinline__ Item item_of(const Args& a, int it) {
  Item x;
  int tile, h;
  x.b = divide(divide(divide(it, a.by_ks, x.split), a.by_tiles, tile), a.by_heads, h);
  x.h = a.packed ? h * a.g.group : h;
  x.hk = a.packed ? h : over(h, a.by_group);
  x.rows = a.packed ? a.g.group * a.g.nq : a.g.nq;
  x.row0 = tile * kTile;
  x.len = key_count(a.g, a.keys, x.b);
  const int t0 = x.split * a.ct;
  x.n = max(min(t0 + a.ct, (x.len + kTile - 1) / kTile) - t0, 0);
  x.key0 = t0 * kTile;
  return x;
}
__device__ __forceinline__ int tile_cols(const Item& x, int j) {
  const int left = x.len - (x.key0 + j * kTile);
  return left >= kTile ? kTile : (left + 31) & ~31;
}
// Row r of the item: head and token; false behind the last row.
__device__ __forceinline__ bool row_of(const Args& a, const Item& x, int r, int& h, int& n) {
  const int rr = x.row0 + r;
  h = x.h;
  n = rr;
  if (a.packed) h += divide(rr, a.by_nq, n);
  return rr < x.rows;
}

template <int NP>
__global__ void __launch_bounds__(THREADS, 1)
bwd_q_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tq,
             const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
             const __grid_constant__ CUtensorMap tg) {
  using Sm = Smem<NP>;
  constexpr int QST = Sm::QST, NK = Sm::NK, NV = Sm::NV;
  constexpr uint32_t kBytes = NP * kPanel;
  extern __shared__ __align__(1024) unsigned char raw[];
  Sm& s = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const Geo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < QST; ++i) {
      ptx::mbar_init(&s.qfull[i], 1);
      ptx::mbar_init(&s.qempty[i], 1);
    }
    for (int i = 0; i < NK; ++i) {
      ptx::mbar_init(&s.kfull[i], 1);
      ptx::mbar_init(&s.kready[i], 1);
      ptx::mbar_init(&s.kempty[i], 1);
    }
    for (int i = 0; i < NV; ++i) {
      ptx::mbar_init(&s.vfull[i], 1);
      ptx::mbar_init(&s.vready[i], 1);
      ptx::mbar_init(&s.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&s.s_full[i], 1);
      ptx::mbar_init(&s.s_free[i], 1);
      ptx::mbar_init(&s.ds_full[i], 8);
    }
    for (uint64_t* b : {&s.dp_full, &s.dq_full, &s.drain}) ptx::mbar_init(b, 1);
    ptx::mbar_init(&s.dp_free, 8);
    ptx::mbar_init(&s.dq_free, 4);
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
    // ============================================================ softmax: a row's half of the keys
    const int half = warp >> 2, sub = warp & 3;
    const uint32_t tl = tbase + ((uint32_t)(sub * 32) << 16);
    const float sc2 = g.scale * kLog2e;
    uint32_t tc_ = 0;                          // key tiles so far
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.n == 0) continue;
      const uint8_t* mask = a.keys.mask ? a.keys.mask + (int64_t)x.b * g.nk : nullptr;
      int h, n;
      const bool live = row_of(a, x, sub * 32 + lane, h, n);
      const int64_t at = ((int64_t)x.b * g.h + h) * g.nq + n;
      float ls = live ? a.lse[at] : -INFINITY;
      ls = ls == -INFINITY ? INFINITY : ls * kLog2e;     // no key, or no row: every weight is 2^-inf = 0
      const float D = live ? a.D[at] : 0.f;
      for (int j = 0; j < x.n; ++j, ++tc_) {
        const int key0 = x.key0 + j * kTile;
        const int chunks = tile_cols(x, j) >> 5;         // 16 columns each, in this half
        const uint32_t col0 = 16u * chunks * half;
        const bool whole = !mask && key0 + kTile <= x.len;
        uint64_t bits = ~0ull;
        if (!whole) {
          uint32_t w[4];
          key_bits(mask, key0, x.len, lane, w);
          const uint64_t lo = (uint64_t)w[1] << 32 | w[0], hi = (uint64_t)w[3] << 32 | w[2];
          bits = col0 == 0 ? lo : (col0 == 64 ? hi : (lo >> col0) | (hi << (64 - col0)));
        }
        const uint32_t sb = tc_ & 1, sp = (tc_ >> 1) & 1;
        if (!wait(&s.s_full[sb], sp, 121)) break;
        tc::fence_after_sync();
        const uint32_t cs = tl + COL_S + 128u * sb;
        float p[64];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) {
            uint32_t r[16];
            tc::tmem_ld16(cs + col0 + 16u * c, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) p[16 * c + e] = ptx::ex2(fmaf(__uint_as_float(r[e]), sc2, -ls));
            if (!whole)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!((bits >> (16 * c + e)) & 1u)) p[16 * c + e] = 0.f;
          }
        if (!wait(&s.dp_full, tc_ & 1, 122)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) {
            uint32_t r[16], w[16];               // 16 columns of S become 8 of dS and 8 of what the rounding left
            tc::tmem_ld16(tl + COL_DP + col0 + 16u * c, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float x0 = p[16 * c + 2 * e] * (__uint_as_float(r[2 * e]) - D);
              const float x1 = p[16 * c + 2 * e + 1] * (__uint_as_float(r[2 * e + 1]) - D);
              w[e] = ptx::pack_bf16(x0, x1);
              w[8 + e] = ptx::pack_bf16(x0 - __uint_as_float(w[e] << 16), x1 - __uint_as_float(w[e] & 0xffff0000u));
            }
            tc::tmem_st16(cs + col0 + 16u * c, w);
          }
        tc::fence_before_sync();
        arrive(&s.dp_free);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        arrive(&s.ds_full[sb]);
      }
    }
  } else if (warp < EPI0 + 4) {
    // ============================================================ epilogue
    const int sub = warp & 3;
    const uint32_t tl = tbase + ((uint32_t)(sub * 32) << 16);
    const int c16 = (g.d + 15) >> 4;
    uint32_t ic = 0;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      int h, n;
      const bool live = row_of(a, x, sub * 32 + lane, h, n);
      const bool none = x.n == 0;
      const int64_t at = ((int64_t)x.b * g.h + h) * g.nq + n;
      // a query whose keys are all masked has gradient zero, whatever its zero weights met
      bool any = true;
      if (a.keys.mask && live) any = a.lse[at] != -INFINITY;
      if (!none) {
        if (!wait(&s.dq_full, ic & 1, 123)) break;
        tc::fence_after_sync();
        ++ic;
      }
      __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dq) + x.b * g.dq.b + h * g.dq.h + n * g.dq.n;
      float* part = a.part + ((int64_t)x.split * rows_of(g) + at) * g.d;
#pragma unroll 1
      for (int c = 0; c < c16; ++c) {
        uint32_t w[16];
        if (!none) {
          tc::tmem_ld16(tl + COL_DQ + 16u * c, w);
          tc::tmem_wait_ld();
        }
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = none || !any ? 0.f : __uint_as_float(w[e]) * g.scale;
        if (live) store16(f, a.ks > 1 ? nullptr : out + 16 * c, part + 16 * c, 16 * c + 8 < g.d);
        __syncwarp();
      }
      if (!none) {
        tc::fence_before_sync();
        arrive(&s.dq_free);
      }
    }
  } else if (warp == PRODUCER) {
    // ============================================================ producer of K and V
    if (lane == 0) {
      auto wait1 = [&](uint64_t* bar, uint32_t parity, int code) {
        if (ok && !ptx::mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
          ok = false;
          report(a.err, code);
        }
        return ok;
      };
      uint32_t kc = 0, vc = 0;
      for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
        const Item x = item_of(a, it);
        if (x.n == 0) continue;
        for (int j = 0; j < x.n; ++j) {
          const int n0 = x.key0 + j * kTile;
          const uint32_t ki = kc % NK, vi = vc % NV;
          if (!wait1(&s.kempty[ki], ((kc / NK) & 1) ^ 1, 125)) break;
          ++kc;
          ptx::mbar_arrive_expect_tx(&s.kfull[ki], kBytes);
#pragma unroll
          for (int p = 0; p < NP; ++p)
            tma_load_4d(s.k[ki] + p * kPanel, &tk, 64 * p, n0, x.hk * a.wk.h, x.b * a.wk.b, &s.kfull[ki]);
          if (!wait1(&s.vempty[vi], ((vc / NV) & 1) ^ 1, 125)) break;
          ++vc;
          ptx::mbar_arrive_expect_tx(&s.vfull[vi], kBytes);
#pragma unroll
          for (int p = 0; p < NP; ++p)
            tma_load_4d(s.v[vi] + p * kPanel, &tv, 64 * p, n0, x.hk * a.wv.h, x.b * a.wv.b, &s.vfull[vi]);
        }
      }
      // After a timeout, do not leave while copies issued here may still be landing.
      if (!ok) {
        for (uint32_t c = kc > NK ? kc - NK : 0; c < kc; ++c)
          ptx::mbar_wait_bounded(&s.kfull[c % NK], (c / NK) & 1, kWaitLimitNs);
        for (uint32_t c = vc > NV ? vc - NV : 0; c < vc; ++c)
          ptx::mbar_wait_bounded(&s.vfull[c % NV], (c / NV) & 1, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == FIXER) {
    // ============================================================ Q and dO; rows of K and V
    uint32_t kc = 0, qc = 0;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.n == 0) continue;
      const uint32_t st = qc % QST;
      if (!wait(&s.qempty[st], ((qc / QST) & 1) ^ 1, 126)) break;
      ++qc;
      if (a.packed) {
        auto at = [&](int r, int& h, int& n) { return row_of(a, x, r, h, n); };
        gather_rows<NP>(s.q[st], static_cast<const __nv_bfloat16*>(a.q) + x.b * g.q.b, g.q, g.d, lane, at);
        gather_rows<NP>(s.dO[st], static_cast<const __nv_bfloat16*>(a.dO) + x.b * g.dO.b, g.dO, g.d, lane, at);
        ptx::fence_proxy_async();
        arrive(&s.qfull[st]);
      } else if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&s.qfull[st], 2 * kBytes);
#pragma unroll
        for (int p = 0; p < NP; ++p)
          tma_load_4d(s.q[st] + p * kPanel, &tq, 64 * p, x.row0, x.h * a.wq.h, x.b * a.wq.b, &s.qfull[st]);
#pragma unroll
        for (int p = 0; p < NP; ++p)
          tma_load_4d(s.dO[st] + p * kPanel, &tg, 64 * p, x.row0, x.h * a.wg.h, x.b * a.wg.b, &s.qfull[st]);
      }
      __syncwarp();
      const uint8_t* mask = a.keys.mask ? a.keys.mask + (int64_t)x.b * g.nk : nullptr;
      for (int j = 0; j < x.n; ++j, ++kc) {
        const int key0 = x.key0 + j * kTile;
        const bool whole = !mask && key0 + kTile <= x.len;
        uint32_t bits[4];
        if (!whole) key_bits(mask, key0, x.len, lane, bits);
        const uint32_t ki = kc % NK, vi = kc % NV;
        if (!wait(&s.kfull[ki], (kc / NK) & 1, 127)) break;
        if (!whole) {
          clear_rows<NP>(s.k[ki], bits, lane);
          ptx::fence_proxy_async();
        }
        arrive(&s.kready[ki]);
        if (!wait(&s.vfull[vi], (kc / NV) & 1, 127)) break;
        if (!whole) {
          clear_rows<NP>(s.v[vi], bits, lane);
          ptx::fence_proxy_async();
        }
        arrive(&s.vready[vi]);
      }
    }
    if (!ok && lane == 0 && !a.packed)         // (as above)
      for (uint32_t c = qc > QST ? qc - QST : 0; c < qc; ++c)
        ptx::mbar_wait_bounded(&s.qfull[c % QST], (c / QST) & 1, kWaitLimitNs);
    __syncwarp();
  } else if (warp == MMA) {
    // ============================================================ MMA issue
    const uint64_t qd = tc::sw128_desc(ptx::smem_u32(s.q[0]), 16, 1024);
    const uint64_t gd = tc::sw128_desc(ptx::smem_u32(s.dO[0]), 16, 1024);
    const uint64_t kd = tc::sw128_desc(ptx::smem_u32(s.k[0]), 16, 1024);
    const uint64_t kd_mn = tc::sw128_desc(ptx::smem_u32(s.k[0]), kPanel, 1024);
    const uint64_t vd = tc::sw128_desc(ptx::smem_u32(s.v[0]), 16, 1024);
    const int dsteps = (g.d + 15) >> 4;
    const uint32_t id_q = tc::idesc_bf16(128, 16 * dsteps, 0, 1);    // dQ += dS K: A from TMEM, B = K (MN-major)
    constexpr uint64_t kStep = kBytes >> 4;
    uint32_t tc_ = 0, qc = 0, ic = 0;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.n == 0) continue;
      auto panel = [](int k) { return (uint64_t)(k >> 2) * (kPanel >> 4) + 2u * (k & 3); };   // 16 channels on
      const uint64_t qo = (uint64_t)(qc % QST) * kStep;
      auto scores = [&](int j) {
        const uint32_t c = tc_ + j, sb = c & 1;
        if (!wait(&s.kready[c % NK], (c / NK) & 1, 128)) return;
        if (!wait(&s.s_free[sb], ((c >> 1) & 1) ^ 1, 128)) return;    // dQ of the tile before the last has read dS
        tc::fence_after_sync();
        const uint32_t id = tc::idesc_bf16(128, tile_cols(x, j), 0, 0);
        if (tc::elect_one()) {
          for (int k = 0; k < dsteps; ++k)
            tc::mma_bf16(tbase + COL_S + 128u * sb, qd + qo + panel(k), kd + (c % NK) * kStep + panel(k), id, k > 0);
          tc::commit(&s.s_full[sb]);
        }
        __syncwarp();
      };
      auto dps = [&](int j) {
        const uint32_t c = tc_ + j;
        if (!wait(&s.vready[c % NV], (c / NV) & 1, 128)) return;
        if (!wait(&s.dp_free, (c & 1) ^ 1, 128)) return;
        tc::fence_after_sync();
        const uint32_t id = tc::idesc_bf16(128, tile_cols(x, j), 0, 0);
        if (tc::elect_one()) {
          for (int k = 0; k < dsteps; ++k)
            tc::mma_bf16(tbase + COL_DP, gd + qo + panel(k), vd + (c % NV) * kStep + panel(k), id, k > 0);
          tc::commit(&s.dp_full);
          tc::commit(&s.vempty[c % NV]);
          if (j == x.n - 1) tc::commit(&s.qempty[qc % QST]);          // (its S was issued before)
        }
        __syncwarp();
      };
      auto grads = [&](int j) {
        const uint32_t c = tc_ + j, sb = c & 1;
        if (!wait(&s.ds_full[sb], (c >> 1) & 1, 128)) return;
        if (j == 0 && !wait(&s.dq_free, (ic & 1) ^ 1, 128)) return;
        tc::fence_after_sync();
        const int steps = tile_cols(x, j) >> 4;
        const uint32_t ds = tbase + COL_S + 128u * sb;
        if (tc::elect_one()) {
          for (int k = 0; k < steps; ++k)      // 16 keys: 8 columns of dS, then 8 of its rest
#pragma unroll
            for (int e = 0; e < 2; ++e)
              tc::mma_bf16_ta(tbase + COL_DQ, ds + 16u * k + 8u * e, kd_mn + (c % NK) * kStep + 128u * k, id_q,
                              j > 0 || k > 0 || e > 0);
          tc::commit(&s.s_free[sb]);
          tc::commit(&s.kempty[c % NK]);
        }
        __syncwarp();
      };
      if (!wait(&s.qfull[qc % QST], (qc / QST) & 1, 128)) break;
      scores(0);
      if (ok) dps(0);
      for (int j = 0; j < x.n && ok; ++j) {
        const bool more = j + 1 < x.n;
        if (more) scores(j + 1);
        if (ok && more) dps(j + 1);
        if (ok) grads(j);
      }
      if (!ok) break;
      if (tc::elect_one()) tc::commit(&s.dq_full);
      __syncwarp();
      tc_ += x.n;
      ++qc;
      ++ic;
    }
    // every MMA issued here has finished before TMEM is released
    if (tc::elect_one()) tc::commit(&s.drain);
    __syncwarp();
    ptx::mbar_wait_bounded(&s.drain, 0, kWaitLimitNs);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, TMEM_COLS);
  }
}

}  // namespace bwdq

// Key splits as in the forward, into two items an SM, rounded up: when the query
// tiles alone do not fill the device.
DqPlan plan_bwd_q(const Geo& g, int sms) {
  DqPlan p;
  p.packed = g.group > 1 && g.nq < kTile;
  const int64_t rows = p.packed ? (int64_t)g.group * g.nq : g.nq;
  p.tiles = (int)((rows + kTile - 1) / kTile);
  const int64_t items = (int64_t)g.b * (p.packed ? g.hk : g.h) * p.tiles;
  const int64_t nkt = (g.nk + kTile - 1) / kTile;
  int64_t ks = 1;
  if (items < sms && nkt >= 4) {
    ks = (2 * sms + items - 1) / items;
    if (ks > nkt / 2) ks = nkt / 2;
    if (ks > 64) ks = 64;
  }
  p.ct = (int)((nkt + ks - 1) / ks);
  p.ks = (int)((nkt + p.ct - 1) / p.ct);
  p.items = items * p.ks;
  return p;
}

template <int NP>
static cudaError_t launch(const bwdq::Args& a, const CUtensorMap* t, int grid, cudaStream_t s) {
  const size_t smem = sizeof(bwdq::Smem<NP>) + 1024;
  cudaError_t e = cudaFuncSetAttribute(bwdq::bwd_q_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  bwdq::bwd_q_kernel<NP><<<grid, bwdq::THREADS, smem, s>>>(a, t[0], t[1], t[2], t[3]);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_bwd_q(const Geo& g, const DqPlan& p, const CUtensorMap* t, const Where* w, const void* q,
                         const Keys& keys, const void* dO, const float* lse, const float* D, void* dq, float* part,
                         cudaStream_t s) {
  bwdq::Args a;
  a.g = g;
  a.keys = keys;
  a.wq = w[0];
  a.wk = w[1];
  a.wv = w[2];
  a.wg = w[3];
  a.packed = p.packed;
  a.ks = p.ks;
  a.ct = p.ct;
  a.tiles = p.tiles;
  a.items = (int)p.items;
  a.by_ks = divisor(p.ks);
  a.by_tiles = divisor(p.tiles);
  a.by_heads = divisor(p.packed ? g.hk : g.h);
  a.by_group = divisor(g.group);
  a.by_nq = divisor(g.nq);
  a.q = q;
  a.dO = dO;
  a.lse = lse;
  a.D = D;
  a.dq = dq;
  a.part = part;
  a.err = device_error_word();
  const int sms = sm_count();
  const int grid = a.items < sms ? a.items : sms;
  const cudaError_t e = g.d <= 64 ? launch<1>(a, t, grid, s) : launch<2>(a, t, grid, s);
  if (e != cudaSuccess || p.ks == 1) return e;
  return launch_sum_q(g, p.ks, part, dq, s);
}

}  // namespace cross
}  // namespace llsa
