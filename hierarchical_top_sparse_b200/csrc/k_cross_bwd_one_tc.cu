// k_cross_bwd_one_tc.cu -- cross attention backward on the 5th-generation
// tensor cores where the encoder has at most 128 states: one tile of keys,
// kept in shared memory, and one pass over the queries for all three gradients.
//
// An item is a run of query tiles (128 rows) of one key head.  Per tile:
//   S = Q K^T, dP = dO V^T                        (M = 128 queries, N = keys)
//   P = 2^(z - lse);  D = rowsum(P o dP);  dS = P o (dP - D)
//   dV += P^T dO, dK += dS^T Q                    (M = 128 keys, accumulated in TMEM over the item)
//   dQ = scale dS K                               (M = 128 queries, complete: there is no other key tile)
// With all keys of a row at hand D needs no O (rowsum(P o dP) = dO . O), so the
// pass reads q, d_o and lse and writes dq: 46 us of bytes for 786432 rows of 64
// channels, where it takes 128 us (lengths of 120 and 60 states: 377 TFLOP/s of the columns computed): the
// chain from scores to dS and on, about 6000 cycles a tile, is longer.  P and dS are rounded to bf16 for the products and stand in shared
// memory, read transposed for dV and dK (rows are then the contracted index)
// and as they are for dQ.
//
// Two threads share a query row (each half of the key columns, P kept in
// registers between the two passes over dP) and exchange their parts of D.
// The scores of the next tile are computed while the gradients of this one
// are.  Items that split a key head's queries leave fp32 partial dK and dV,
// added in order by a second kernel: no atomics.
//
// Warps: 0-7 softmax, 8-11 epilogue, 12 producer (TMA), 13 MMA issue, 14
// clears masked rows of K and V, and gathers Q and dO where heads are packed.
#include <math.h>

#include "cross_tc.cuh"

namespace llsa {
namespace cross {
namespace bwdone {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int THREADS = 480;
constexpr int EPI0 = 8, PRODUCER = 12, MMA = 13, FIXER = 14;
constexpr uint32_t TMEM_COLS = 512;
// TMEM columns: S, dP, dV, dK, dQ.  Above 64 channels dQ takes the columns of dP.
template <int NP> struct Cols {
  static constexpr uint32_t S = 0, DP = 128, DV = 256, DK = 256 + 64 * NP, DQ = NP == 1 ? 384 : 128;
};

struct Args {
  Geo g;
  Keys keys;
  Where wq, wk, wv, wg;
  int packed, qs, nqt, units;                  // query splits, query tiles per head, tiles per key head
  int items;
  Divisor by_qs, by_hk, by_nqt, by_nq;
  const void *q, *dO;
  const float* lse;
  void *dq, *dk, *dv;
  float *partk, *partv;
  int* err;
};

template <int NP>
struct Smem {
  static constexpr int ST = NP == 1 ? 3 : 1;   // tiles of Q and dO in flight
  alignas(1024) unsigned char k[NP * kPanel];
  alignas(1024) unsigned char v[NP * kPanel];
  alignas(1024) unsigned char p[2 * kPanel];   // [128 queries][2 x 64 keys]
  alignas(1024) unsigned char ds[2 * kPanel];
  alignas(1024) unsigned char q[ST][NP * kPanel];
  alignas(1024) unsigned char dO[ST][NP * kPanel];
  float dpart[2][2][128];                      // by tile parity and half: a row's part of D
  alignas(8) uint64_t kvfull, kvready, kvempty, acc_full, acc_empty;
  uint64_t full[ST], empty[ST];                // Q and dO of a tile
  uint64_t s_full, s_free, dp_full, dp_free, p_full, p_free, ds_full, ds_free, dq_full, dq_free;
  uint64_t xbar[4], drain;
  uint32_t tmem_base;
};
static_assert(sizeof(Smem<1>) + 1024 <= 232448 && sizeof(Smem<2>) + 1024 <= 232448, "shared memory of one CTA");

struct Item {
  int b, hk, split, u0, n, len;                // first tile and tiles, keys of the batch row
};
__device__ __forceinline__ Item item_of(const Args& a, int it) {
  Item x;
  x.b = divide(divide(it, a.by_qs, x.split), a.by_hk, x.hk);
  x.u0 = (int)((int64_t)a.units * x.split / a.qs);
  x.n = (int)((int64_t)a.units * (x.split + 1) / a.qs) - x.u0;
  x.len = key_count(a.g, a.keys, x.b);
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

template <int NP>
__global__ void __launch_bounds__(THREADS, 1)
bwd_one_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tq,
               const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
               const __grid_constant__ CUtensorMap tg) {
  using Sm = Smem<NP>;
  using C = Cols<NP>;
  constexpr int ST = Sm::ST;
  constexpr uint32_t kBytes = NP * kPanel;
  extern __shared__ __align__(1024) unsigned char raw[];
  Sm& s = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const Geo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (uint64_t* b : {&s.kvfull, &s.kvready, &s.kvempty, &s.acc_full, &s.s_full, &s.dp_full, &s.p_free, &s.ds_free,
                        &s.dq_full, &s.drain})
      ptx::mbar_init(b, 1);
    for (uint64_t* b : {&s.acc_empty, &s.dq_free}) ptx::mbar_init(b, 4);
    for (uint64_t* b : {&s.s_free, &s.dp_free, &s.p_full, &s.ds_full}) ptx::mbar_init(b, 8);
    for (int i = 0; i < ST; ++i) {
      ptx::mbar_init(&s.full[i], 1);
      ptx::mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) ptx::mbar_init(&s.xbar[i], 2);
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
    const int row = sub * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(sub * 32) << 16);
    const float sc2 = g.scale * kLog2e;
    uint32_t tc_ = 0;                          // tiles so far
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.len == 0) continue;
      const uint8_t* mask = a.keys.mask ? a.keys.mask + (int64_t)x.b * g.nk : nullptr;
      const int chunks = ((x.len + 31) >> 5);  // 16 columns each, in this half
      const int col0 = 16 * chunks * half;
      const bool whole = !mask && (x.len & 31) == 0;
      uint64_t bits = ~0ull;                   // of the half's 64 columns
      if (!whole) {
        uint32_t w[4];
        key_bits(mask, 0, x.len, lane, w);
        const uint64_t lo = (uint64_t)w[1] << 32 | w[0], hi = (uint64_t)w[3] << 32 | w[2];
        bits = col0 == 0 ? lo : (col0 == 64 ? hi : (lo >> col0) | (hi << (64 - col0)));
      }
      auto lse_of = [&](int i) {
        int h, n;
        const bool live = i < x.n && row_of(a, x.hk, x.u0 + i, row, h, n);
        const float v = live ? a.lse[((int64_t)x.b * g.h + h) * g.nq + n] : -INFINITY;
        return v == -INFINITY ? INFINITY : v * kLog2e;
      };
      float next = lse_of(0);
      for (int i = 0; i < x.n; ++i, ++tc_) {
        const float ls = next;
        next = lse_of(i + 1);
        const uint32_t ph = tc_ & 1;
        if (!wait(&s.s_full, ph, 101)) break;
        tc::fence_after_sync();
        float p[64];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) {
            uint32_t r[16];
            tc::tmem_ld16(tl + C::S + col0 + 16u * c, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) p[16 * c + e] = ptx::ex2(fmaf(__uint_as_float(r[e]), sc2, -ls));
            if (!whole)
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!((bits >> (16 * c + e)) & 1u)) p[16 * c + e] = 0.f;
          }
        tc::fence_before_sync();
        arrive(&s.s_free);
        if (!wait(&s.p_free, ph ^ 1, 102)) break;    // dV of the tile before has read P
        auto put = [&](unsigned char* tile, int c, const float* f) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = col0 + 16 * c + 8 * e;
            *reinterpret_cast<uint4*>(tile + (col >> 6) * kPanel + row * 128 +
                                      ((((col >> 3) & 7) ^ (row & 7)) << 4)) =
                make_uint4(ptx::pack_bf16(f[8 * e], f[8 * e + 1]), ptx::pack_bf16(f[8 * e + 2], f[8 * e + 3]),
                           ptx::pack_bf16(f[8 * e + 4], f[8 * e + 5]), ptx::pack_bf16(f[8 * e + 6], f[8 * e + 7]));
          }
        };
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) put(s.p, c, p + 16 * c);
        ptx::fence_proxy_async();
        arrive(&s.p_full);
        if (!wait(&s.dp_full, ph, 103)) break;
        tc::fence_after_sync();
        float d0 = 0.f, d1 = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) {
            uint32_t r[16];
            tc::tmem_ld16(tl + C::DP + col0 + 16u * c, r);
            tc::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              d0 = fmaf(p[16 * c + e], __uint_as_float(r[e]), d0);
              d1 = fmaf(p[16 * c + e + 1], __uint_as_float(r[e + 1]), d1);
            }
          }
        // the other half's part (by tile parity, so that a slow partner still reads this tile's)
        s.dpart[ph][half][row] = d0 + d1;
        arrive(&s.xbar[sub]);
        if (!wait(&s.xbar[sub], ph, 104)) break;
        const float D = s.dpart[ph][0][row] + s.dpart[ph][1][row];
        if (!wait(&s.ds_free, ph ^ 1, 105)) break;   // dK and dQ of the tile before have read dS
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) {
            uint32_t r[16];
            tc::tmem_ld16(tl + C::DP + col0 + 16u * c, r);
            tc::tmem_wait_ld();
            float f[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = p[16 * c + e] * (__uint_as_float(r[e]) - D);
            put(s.ds, c, f);
          }
        tc::fence_before_sync();
        ptx::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(&s.dp_free);
          ptx::mbar_arrive(&s.ds_full);
        }
        __syncwarp();
      }
    }
  } else if (warp < EPI0 + 4) {
    // ============================================================ epilogue
    const int sub = warp & 3;
    const int row = sub * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(sub * 32) << 16);
    const int c16 = (g.d + 15) >> 4;
    uint32_t tc_ = 0, ac = 0;
    // 16 channels of chunk c from TMEM column `col` on, times f (zero where !keep), to global memory
    auto store = [&](uint32_t col, int c, bool none, bool keep, float f, __nv_bfloat16* out, float* part, bool live) {
      uint32_t w[16];
      if (!none) {
        tc::tmem_ld16(tl + col + 16u * c, w);
        tc::tmem_wait_ld();
      }
      float v[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = none || !keep ? 0.f : __uint_as_float(w[e]) * f;
      if (live) store16(v, part ? nullptr : out + 16 * c, part + 16 * c, 16 * c + 8 < g.d);
      __syncwarp();
    };
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      const bool none = x.len == 0;
      for (int i = 0; i < x.n; ++i) {
        int h, n;
        const bool live = row_of(a, x.hk, x.u0 + i, row, h, n);
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.dq) + x.b * g.dq.b + h * g.dq.h + n * g.dq.n;
        // a query whose keys are all masked has gradient zero, whatever its zero weights met
        bool any = true;
        if (a.keys.mask && live) any = a.lse[((int64_t)x.b * g.h + h) * g.nq + n] != -INFINITY;
        if (!none) {
          if (!wait(&s.dq_full, tc_ & 1, 106)) break;
          tc::fence_after_sync();
          ++tc_;
        }
#pragma unroll 1
        for (int c = 0; c < c16; ++c) store(C::DQ, c, none, any, g.scale, out, nullptr, live);
        if (!none) {
          tc::fence_before_sync();
          arrive(&s.dq_free);
        }
      }
      if (!ok) break;
      if (!none) {
        if (!wait(&s.acc_full, ac & 1, 107)) break;
        tc::fence_after_sync();
        ++ac;
      }
      const bool live = row < g.nk;
      bool valid = row < x.len;
      if (valid && a.keys.mask) valid = a.keys.mask[(int64_t)x.b * g.nk + row] != 0;
      const int64_t at = ((int64_t)x.split * keys_of(g) + ((int64_t)x.b * g.hk + x.hk) * g.nk + row) * g.d;
      __nv_bfloat16* ov = static_cast<__nv_bfloat16*>(a.dv) + x.b * g.dv.b + x.hk * g.dv.h + row * g.dv.n;
      __nv_bfloat16* ok_ = static_cast<__nv_bfloat16*>(a.dk) + x.b * g.dk.b + x.hk * g.dk.h + row * g.dk.n;
      // (a key that takes no part has gradient zero whatever its zero weights met)
#pragma unroll 1
      for (int c = 0; c < c16; ++c) {
        store(C::DV, c, none, valid, 1.f, ov, a.qs > 1 ? a.partv + at : nullptr, live);
        store(C::DK, c, none, valid, g.scale, ok_, a.qs > 1 ? a.partk + at : nullptr, live);
      }
      if (!none) {
        tc::fence_before_sync();
        arrive(&s.acc_empty);
      }
    }
  } else if (warp == PRODUCER) {
    // ============================================================ producer
    if (lane == 0) {
      auto wait1 = [&](uint64_t* bar, uint32_t parity, int code) {
        if (ok && !ptx::mbar_wait_bounded(bar, parity, kWaitLimitNs)) {
          ok = false;
          report(a.err, code);
        }
        return ok;
      };
      uint32_t tc_ = 0, ic = 0;
      for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
        const Item x = item_of(a, it);
        if (x.len == 0) continue;
        if (!wait1(&s.kvempty, (ic & 1) ^ 1, 108)) break;
        ++ic;
        ptx::mbar_arrive_expect_tx(&s.kvfull, 2 * kBytes);
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          tma_load_4d(s.k + p * kPanel, &tk, 64 * p, 0, x.hk * a.wk.h, x.b * a.wk.b, &s.kvfull);
          tma_load_4d(s.v + p * kPanel, &tv, 64 * p, 0, x.hk * a.wv.h, x.b * a.wv.b, &s.kvfull);
        }
        for (int i = 0; i < x.n && !a.packed; ++i) {
          const uint32_t st = tc_ % ST;
          if (!wait1(&s.empty[st], ((tc_ / ST) & 1) ^ 1, 108)) break;
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
        if (ic) ptx::mbar_wait_bounded(&s.kvfull, (ic - 1) & 1, kWaitLimitNs);
        for (uint32_t c = tc_ > ST ? tc_ - ST : 0; c < tc_; ++c)
          ptx::mbar_wait_bounded(&s.full[c % ST], (c / ST) & 1, kWaitLimitNs);
      }
    }
    __syncwarp();
  } else if (warp == FIXER) {
    // ============================================================ rows of K and V; packed rows of Q and dO
    uint32_t ic = 0, tc_ = 0;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.len == 0) continue;
      const uint8_t* mask = a.keys.mask ? a.keys.mask + (int64_t)x.b * g.nk : nullptr;
      uint32_t bits[4];
      key_bits(mask, 0, x.len, lane, bits);
      if (!wait(&s.kvfull, ic & 1, 109)) break;
      ++ic;
      clear_rows<NP>(s.k, bits, lane);
      clear_rows<NP>(s.v, bits, lane);
      ptx::fence_proxy_async();
      arrive(&s.kvready);
      for (int i = 0; i < x.n && a.packed; ++i, ++tc_) {
        const uint32_t st = tc_ % ST;
        if (!wait(&s.empty[st], ((tc_ / ST) & 1) ^ 1, 109)) break;
        auto at = [&](int r, int& h, int& n) { return row_of(a, x.hk, x.u0 + i, r, h, n); };
        gather_rows<NP>(s.q[st], static_cast<const __nv_bfloat16*>(a.q) + x.b * g.q.b, g.q, g.d, lane, at);
        gather_rows<NP>(s.dO[st], static_cast<const __nv_bfloat16*>(a.dO) + x.b * g.dO.b, g.dO, g.d, lane, at);
        ptx::fence_proxy_async();
        arrive(&s.full[st]);
      }
    }
  } else if (warp == MMA) {
    // ============================================================ MMA issue
    const uint64_t kd = tc::sw128_desc(ptx::smem_u32(s.k), 16, 1024);          // K-major
    const uint64_t kd_mn = tc::sw128_desc(ptx::smem_u32(s.k), kPanel, 1024);   // MN-major
    const uint64_t vd = tc::sw128_desc(ptx::smem_u32(s.v), 16, 1024);
    const uint64_t qd = tc::sw128_desc(ptx::smem_u32(s.q[0]), 16, 1024);
    const uint64_t qd_mn = tc::sw128_desc(ptx::smem_u32(s.q[0]), kPanel, 1024);
    const uint64_t gd = tc::sw128_desc(ptx::smem_u32(s.dO[0]), 16, 1024);
    const uint64_t gd_mn = tc::sw128_desc(ptx::smem_u32(s.dO[0]), kPanel, 1024);
    const uint64_t pd_mn = tc::sw128_desc(ptx::smem_u32(s.p), kPanel, 1024);
    const uint64_t dsd = tc::sw128_desc(ptx::smem_u32(s.ds), 16, 1024);
    const uint64_t dsd_mn = tc::sw128_desc(ptx::smem_u32(s.ds), kPanel, 1024);
    const int dsteps = (g.d + 15) >> 4;
    const uint32_t id_acc = tc::idesc_bf16(128, 16 * dsteps, 1, 1), id_q = tc::idesc_bf16(128, 16 * dsteps, 0, 1);
    uint32_t tc_ = 0, ic = 0;
    for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      if (x.len == 0) continue;
      const int cols = (x.len + 31) & ~31;
      const uint32_t id_s = tc::idesc_bf16(128, cols, 0, 0);
      auto stage = [&](int i) { return (uint64_t)((tc_ + i) % ST) * (kBytes >> 4); };
      auto panel = [](int k) { return (uint64_t)(k >> 2) * (kPanel >> 4) + 2u * (k & 3); };   // 16 channels on
      auto scores = [&](int i) {               // S
        const uint32_t c = tc_ + i;
        if (!wait(&s.full[c % ST], (c / ST) & 1, 110)) return;
        if (!wait(&s.s_free, (c & 1) ^ 1, 110)) return;
        tc::fence_after_sync();
        const uint64_t so = stage(i);
        if (tc::elect_one()) {
          for (int k = 0; k < dsteps; ++k) tc::mma_bf16(tbase + C::S, qd + so + panel(k), kd + panel(k), id_s, k > 0);
          tc::commit(&s.s_full);
        }
        __syncwarp();
      };
      auto dps = [&](int i) {                  // dP
        const uint32_t c = tc_ + i;
        if (!wait(&s.dp_free, (c & 1) ^ 1, 110)) return;
        if (NP == 2 && !wait(&s.dq_free, (c & 1) ^ 1, 110)) return;    // dQ of the tile before, in these columns, is out
        tc::fence_after_sync();
        const uint64_t so = stage(i);
        if (tc::elect_one()) {
          for (int k = 0; k < dsteps; ++k) tc::mma_bf16(tbase + C::DP, gd + so + panel(k), vd + panel(k), id_s, k > 0);
          tc::commit(&s.dp_full);
        }
        __syncwarp();
      };
      auto grad_v = [&](int i) {
        const uint32_t c = tc_ + i;
        if (!wait(&s.p_full, c & 1, 110)) return;
        if (i == 0 && !wait(&s.acc_empty, (ic & 1) ^ 1, 110)) return;
        tc::fence_after_sync();
        const uint64_t so = stage(i);
        if (tc::elect_one()) {
          for (int k = 0; k < 8; ++k)          // 16 queries: 2 KB of a panel
            tc::mma_bf16(tbase + C::DV, pd_mn + 128u * k, gd_mn + so + 128u * k, id_acc, i > 0 || k > 0);
          tc::commit(&s.p_free);
        }
        __syncwarp();
      };
      auto grad_kq = [&](int i) {
        const uint32_t c = tc_ + i;
        if (!wait(&s.ds_full, c & 1, 110)) return;
        if (NP == 1 && !wait(&s.dq_free, (c & 1) ^ 1, 110)) return;
        tc::fence_after_sync();
        const uint64_t so = stage(i);
        if (tc::elect_one()) {
          for (int k = 0; k < cols / 16; ++k)  // 16 keys: 32 bytes of dS's rows, 2 KB of K's panel
            tc::mma_bf16(tbase + C::DQ, dsd + panel(k), kd_mn + 128u * k, id_q, k > 0);
          tc::commit(&s.dq_full);
          for (int k = 0; k < 8; ++k)
            tc::mma_bf16(tbase + C::DK, dsd_mn + 128u * k, qd_mn + so + 128u * k, id_acc, i > 0 || k > 0);
          tc::commit(&s.ds_free);
          tc::commit(&s.empty[c % ST]);
        }
        __syncwarp();
      };
      if (!wait(&s.kvready, ic & 1, 110)) break;
      scores(0);
      if (ok) dps(0);
      for (int i = 0; i < x.n && ok; ++i) {
        const bool more = i + 1 < x.n;
        if (ST > 1 && more) scores(i + 1);
        if (ok) grad_v(i);
        if (NP == 1 && ok && more) dps(i + 1);
        if (ok) grad_kq(i);
        if (ST == 1 && ok && more) scores(i + 1);
        if (NP == 2 && ok && more) dps(i + 1);
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

}  // namespace bwdone

// The number of splits that needs the fewest tiles one after the other on an
// SM.  A run of tiles costs about two tiles more (filling, storing the
// accumulators), and a split's partial sums about an eighth of a tile.
int splits_of_queries(int64_t slices, int units, int sms) {
  double best = 0;
  int splits = 1;
  for (int qs = 1; qs <= sms && qs <= units; ++qs) {
    const int64_t waves = (slices * qs + sms - 1) / sms;
    const double cost =
        (double)waves * ((units + qs - 1) / qs + 2) + (qs > 1 ? 2.0 + 0.125 * qs * (double)slices / sms : 0.0);
    if (qs == 1 || cost < best) {
      best = cost;
      splits = qs;
    }
  }
  return splits;
}

OnePlan plan_bwd_one(const Geo& g, int sms) {
  OnePlan p;
  p.packed = g.group > 1 && g.nq < kTile;
  p.nqt = (g.nq + kTile - 1) / kTile;
  p.units = (int)(p.packed ? ((int64_t)g.group * g.nq + kTile - 1) / kTile : (int64_t)g.group * p.nqt);
  const int64_t slices = (int64_t)g.b * g.hk;
  p.qs = splits_of_queries(slices, p.units, sms);
  p.items = slices * p.qs;
  return p;
}

template <int NP>
static cudaError_t launch(const bwdone::Args& a, const CUtensorMap* t, int grid, cudaStream_t s) {
  const size_t smem = sizeof(bwdone::Smem<NP>) + 1024;
  cudaError_t e =
      cudaFuncSetAttribute(bwdone::bwd_one_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  bwdone::bwd_one_kernel<NP><<<grid, bwdone::THREADS, smem, s>>>(a, t[0], t[1], t[2], t[3]);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_bwd_one(const Geo& g, const OnePlan& p, const CUtensorMap* t, const Where* w, const void* q,
                           const Keys& keys, const void* dO, const float* lse, void* dq, void* dk, void* dv,
                           float* partk, float* partv, cudaStream_t s) {
  bwdone::Args a;
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
  a.items = (int)p.items;
  a.by_qs = divisor(p.qs);
  a.by_hk = divisor(g.hk);
  a.by_nqt = divisor(p.nqt);
  a.by_nq = divisor(g.nq);
  a.q = q;
  a.dO = dO;
  a.lse = lse;
  a.dq = dq;
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

}  // namespace cross
}  // namespace llsa
