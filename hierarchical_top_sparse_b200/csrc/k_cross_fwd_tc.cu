// k_cross_fwd_tc.cu -- cross attention forward on the 5th-generation tensor
// cores (tcgen05, accumulators in tensor memory), bf16, d a multiple of 8 up
// to 128.
//
// An item is up to two tiles of 128 query rows of one key head against the
// key tiles of one split, 128 keys each:
//   S = Q K^T                     (M = 128 rows, N = the tile's keys, K = d)
//   one thread per row takes its 128 logits from TMEM, with the running
//   maximum m and sum l of the softmax, and writes P = 2^(z - m) as bf16 back;
//   O += P V                      (A = P from TMEM, N = d, K = the tile's keys)
// The maximum is lazy: O (in TMEM) is rescaled only when a logit exceeds m by
// more than 2^8, so weights stay below 256.  The bound is the exponential (16
// a cycle and SM): the two tiles of an item run on warpgroups of their own, so
// that one works while the other waits.  16384 queries of 48 heads against 512
// states, 64 channels (6 heads, batch 8): 212 us where the exponentials alone take 89; the rest of
// a tile's chain (load, maximum, hand-offs) is about 1600 of its 4000 cycles.
//
// Rows: the tokens of one query head, or, where a head has fewer than 128, the
// tokens of all heads of a key head, one after the other (each key head's keys
// are then read once).  Few items are made up for by splitting the keys; the
// splits' results are fp32 and joined by their LSE.
//
// Key tiles that are not whole (the length ends inside, or keys are masked):
// such keys' logits are replaced, never computed with, and their rows of V are
// cleared in shared memory, so that 0 * V is 0 whatever V holds.
//
// Warps (one CTA per SM, items dealt round robin): 0-3 and 4-7 softmax of tile
// 0 and 1, 8-11 epilogue, 12 producer of K and V (TMA), 13 MMA issue of S,
// 14 of O, 15 fetches Q (where heads are packed by plain loads) and clears rows
// of V.  (One producer for all would hold the next item's keys back until this
// one's queries are done with.)
// Up to 64 channels, P has columns of its own and S of the next key tile is
// computed while P of this one is made; above, P takes S's columns.
#include <math.h>

#include "cross_tc.cuh"

namespace llsa {
namespace cross {
namespace fwdtc {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kHeadroom = 8.f;               // log2 of the largest weight before O is rescaled
constexpr int THREADS = 512;
constexpr int EPI0 = 8, PRODUCER = 12, MMA_S = 13, FIXER = 15;
constexpr uint32_t TMEM_COLS = 512;
// Registers of a thread: at launch, then of the softmax warps and of the others.  (A share that the block was not
// launched with would be waited for without end.)
constexpr int REGS = 65536 / THREADS / 8 * 8, SOFT_REGS = 184, OTHER_REGS = 72;
static_assert(EPI0 * 32 * SOFT_REGS + (THREADS - EPI0 * 32) * OTHER_REGS <= THREADS * REGS, "register shares");

struct Args {
  Geo g;
  Keys keys;
  Where wq, wk, wv;
  int ks, ct;                                  // key splits, key tiles per split
  int tpi;                                     // query tiles per item: 1, or 2 (the last of a slice may be empty)
  int packed;                                  // rows: all heads of a key head
  int slices, pairs;                           // slices of rows; items' row groups per slice
  int items;
  Divisor by_ks, by_pairs, by_heads, by_group, by_nq;    // heads: of a batch row's slices
  const void* q;                               // where heads are packed
  void* o;
  float* lse;
  FwdWork part;
  int* err;
};

template <int NP>
struct Smem {
  static constexpr int QST = NP == 1 ? 2 : 1, NS = NP == 1 ? 4 : 2;
  alignas(1024) unsigned char q[2][QST][NP * kPanel];
  alignas(1024) unsigned char k[NS][NP * kPanel];
  alignas(1024) unsigned char v[NS][NP * kPanel];
  float stat_m[2][128], stat_l[2][128];        // an item's row maxima and sums: softmax -> epilogue
  alignas(8) uint64_t qfull[2][QST], qempty[2][QST];
  uint64_t kfull[NS], kempty[NS], vfull[NS], vempty[NS], vready[NS];
  uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2], o_full[2], o_empty[2], st_full[2], drain[2];
  uint32_t tmem_base;
};
static_assert(sizeof(Smem<1>) + 1024 <= 232448 && sizeof(Smem<2>) + 1024 <= 232448, "shared memory of one CTA");

struct Item {
  int b, hk, h, row0, rows;                    // batch row, key head, query head (not packed), first row, rows of the slice
  int split, key0, n, len;                     // first key, key tiles, keys of the batch row
};

__device__ __forceinline__ Item item_of(const Args& a, int it) {
  Item x;
  int p, h;
  const int slice = divide(divide(it, a.by_ks, x.split), a.by_pairs, p);
  x.b = divide(slice, a.by_heads, h);
  if (a.packed) {
    x.hk = h;
    x.h = h * a.g.group;
    x.rows = a.g.group * a.g.nq;
  } else {
    x.h = h;
    x.hk = over(h, a.by_group);
    x.rows = a.g.nq;
  }
  x.row0 = p * a.tpi * kTile;
  x.len = key_count(a.g, a.keys, x.b);
  const int t0 = x.split * a.ct;
  const int all = (x.len + kTile - 1) / kTile;
  const int t1 = min(t0 + a.ct, all);
  x.n = max(t1 - t0, 0);
  x.key0 = t0 * kTile;
  return x;
}
// Columns of a key tile that are computed: its keys up to the length, rounded up to 32.
__device__ __forceinline__ int tile_cols(const Item& x, int j) {
  const int left = x.len - (x.key0 + j * kTile);
  return left >= kTile ? kTile : (left + 31) & ~31;
}

// The logits of masked keys become -inf, whatever they are.
__device__ __forceinline__ void keep_keys(uint32_t r[32], uint32_t bits) {
  if (bits == 0xffffffffu) return;
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!((bits >> i) & 1u)) r[i] = 0xff800000u;
}

template <int NP>
__global__ void __launch_bounds__(THREADS, 1) fwd_tc_kernel(const __grid_constant__ Args a,
                                                            const __grid_constant__ CUtensorMap tq,
                                                            const __grid_constant__ CUtensorMap tk,
                                                            const __grid_constant__ CUtensorMap tv) {
  using S = Smem<NP>;
  constexpr int QST = S::QST, NS = S::NS;
  constexpr uint32_t kBytes = NP * kPanel;
  extern __shared__ __align__(1024) unsigned char raw[];
  S& s = *reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  const Geo& g = a.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      for (int i = 0; i < QST; ++i) {
        ptx::mbar_init(&s.qfull[t][i], 1);
        ptx::mbar_init(&s.qempty[t][i], 1);
      }
      ptx::mbar_init(&s.s_full[t], 1);
      ptx::mbar_init(&s.s_empty[t], 4);
      ptx::mbar_init(&s.p_full[t], 4);
      ptx::mbar_init(&s.p_empty[t], 1);
      ptx::mbar_init(&s.o_full[t], 1);
      ptx::mbar_init(&s.o_empty[t], 4);
      ptx::mbar_init(&s.st_full[t], 4);
      ptx::mbar_init(&s.drain[t], 1);
    }
    for (int i = 0; i < NS; ++i) {
      ptx::mbar_init(&s.kfull[i], 1);
      ptx::mbar_init(&s.kempty[i], 1);
      ptx::mbar_init(&s.vfull[i], 1);
      ptx::mbar_init(&s.vempty[i], 1);
      ptx::mbar_init(&s.vready[i], 1);
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
  // TMEM columns of tile t: S, P (bf16 pairs), O
  auto col_s = [](int t) { return 128u * t; };
  auto col_p = [](int t) { return NP == 1 ? 256u + 64u * t : 128u * t; };
  auto col_o = [](int t) { return NP == 1 ? 384u + 64u * t : 256u + 128u * t; };
  bool ok = true;
  // Every lane of a warp waits, and all go on together or all give up together.
  auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
    if (!ok) return false;
    ok = warp_wait(bar, parity);
    if (!ok && lane == 0) report(a.err, code);
    return ok;
  };

  if (warp < EPI0) {
    // ============================================================ softmax: one row a thread
    more_registers<SOFT_REGS>();
    const int t = warp >> 2, sub = warp & 3;
    const int items = t < a.tpi ? a.items : 0;
    const int row = sub * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(sub * 32) << 16);
    const float sc2 = g.scale * kLog2e;        // logits in the log2 domain
    const f2 scale2 = twice(sc2);
    uint32_t sc = 0, oc = 0;
    for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
      const Item x = item_of(a, it);
      const uint8_t* mask = a.keys.mask ? a.keys.mask + (int64_t)x.b * g.nk : nullptr;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < x.n; ++j, ++sc) {
        const int key0 = x.key0 + j * kTile;
        const int blocks = tile_cols(x, j) >> 5;
        const bool whole = !mask && key0 + kTile <= x.len;
        uint32_t bits[4];
        if (!whole) key_bits(mask, key0, x.len, lane, bits);
        if (!wait(&s.s_full[t], sc & 1, 91)) break;
        tc::fence_after_sync();
        // the whole row of S in registers (columns behind `blocks` hold anything: their bits are clear)
        uint32_t r[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tl + col_s(t) + 32u * c, r + 32 * c);
        tc::tmem_wait_ld();
        if (NP == 1) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&s.s_empty[t]);
          __syncwarp();
        }
        if (!whole) {
#pragma unroll
          for (int c = 0; c < 4; ++c) keep_keys(r + 32 * c, bits[c]);
        }
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaxf(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
#pragma unroll
        for (int i = 16; i < 128; i += 2)
          y[(i >> 1) & 7] = max3(y[(i >> 1) & 7], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
        const float mx = max3(max3(y[0], y[1], y[2]), max3(y[3], y[4], y[5]), fmaxf(y[6], y[7]));
        const float mn = fmaxf(m, mx * sc2);
        bool resc = false;
        float f = 1.f;
        if (m == -INFINITY) {
          m = mn;
        } else if (mn > m + kHeadroom) {
          resc = true;
          f = ptx::ex2(m - mn);
          m = mn;
          l *= f;
        }
        const float ref = m == -INFINITY ? 0.f : m;      // no key so far: every weight is 2^-inf = 0
        if (__any_sync(0xffffffffu, resc)) {
          if (!wait(&s.p_empty[t], (sc & 1) ^ 1, 92)) break;     // every earlier update is in O
          tc::fence_after_sync();
          const int oc16 = (g.d + 15) >> 4;
#pragma unroll 1
          for (int c = 0; c < oc16; ++c) {
            uint32_t w[16];
            tc::tmem_ld16(tl + col_o(t) + 16u * c, w);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * f);
            tc::tmem_st16(tl + col_o(t) + 16u * c, w);
          }
        }
        const f2 ref2 = twice(-ref);
        f2 sum = twice(0.f);
        auto weights = [&](int c, uint32_t* w) {         // of 32 keys
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float p0, p1;
            split(fma2(pair(__uint_as_float(r[32 * c + 2 * i]), __uint_as_float(r[32 * c + 2 * i + 1])), scale2, ref2),
                  p0, p1);
            p0 = ptx::ex2(p0);
            p1 = ptx::ex2(p1);
            sum = add2(sum, pair(p0, p1));
            w[i] = ptx::pack_bf16(p0, p1);
          }
        };
        // the first half of the weights before P is free: the O update of the tile before is still reading it
        uint32_t w0[16], w1[16];
        weights(0, w0);
        if (1 < blocks) weights(1, w1);
        if (!wait(&s.p_empty[t], (sc & 1) ^ 1, 92)) break;
        tc::fence_after_sync();
        tc::tmem_st16(tl + col_p(t), w0);
        if (1 < blocks) tc::tmem_st16(tl + col_p(t) + 16u, w1);
        if (2 < blocks) {
          weights(2, w0);
          tc::tmem_st16(tl + col_p(t) + 32u, w0);
        }
        if (3 < blocks) {
          weights(3, w1);
          tc::tmem_st16(tl + col_p(t) + 48u, w1);
        }
        l += both(sum);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&s.p_full[t]);
        __syncwarp();
      }
      if (!wait(&s.o_empty[t], (oc & 1) ^ 1, 93)) break;    // the epilogue has read the last item's statistics
      s.stat_m[t][row] = m;
      s.stat_l[t][row] = l;
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&s.st_full[t]);
      __syncwarp();
      ++oc;
    }
  } else {
    fewer_registers<OTHER_REGS>();
    if (warp < EPI0 + 4) {
      // ============================================================ epilogue
      const int sub = warp & 3;
      const uint32_t tl = tbase + ((uint32_t)(sub * 32) << 16);
      uint32_t oc[2] = {0, 0};
      for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
        const Item x = item_of(a, it);
#pragma unroll 1
        for (int t = 0; t < a.tpi; ++t) {
          const uint32_t c0 = t ? oc[1] : oc[0];
          if (t) ++oc[1]; else ++oc[0];
          if (!wait(&s.st_full[t], c0 & 1, 94) || !wait(&s.o_full[t], c0 & 1, 94)) break;
          tc::fence_after_sync();
          const float m = s.stat_m[t][sub * 32 + lane];
          const float l = s.stat_l[t][sub * 32 + lane];
          const int r = x.row0 + t * kTile + sub * 32 + lane;
          const bool live = r < x.rows;
          int h = x.h, n = r;
          if (a.packed && live) {
            h = x.h + divide(r, a.by_nq, n);
          }
          const bool none = m == -INFINITY && !(l > 0.f) && l == l;    // NaN sums pass through
          const float inv = none ? 0.f : 1.f / l;
          const float ls = none ? -INFINITY : (m + log2f(l)) * kLn2;
          const int64_t at = ((int64_t)x.b * g.h + h) * g.nq + n;
          __nv_bfloat16* po = static_cast<__nv_bfloat16*>(a.o) + x.b * g.o.b + h * g.o.h + n * g.o.n;
          float* pp = a.part.o + ((int64_t)x.split * rows_of(g) + at) * g.d;
#pragma unroll 1
          for (int c = 0; c < g.d; c += 16) {
            uint32_t w[16];
            tc::tmem_ld16(tl + col_o(t) + c, w);
            tc::tmem_wait_ld();
            float f[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] = none ? 0.f : __uint_as_float(w[e]) * inv;
            if (live) store16(f, a.ks > 1 ? nullptr : po + c, pp + c, c + 8 < g.d);
            __syncwarp();
          }
          if (live) {
            if (a.ks > 1)
              a.part.lse[(int64_t)x.split * rows_of(g) + at] = ls;
            else if (a.lse)
              a.lse[at] = ls;
          }
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&s.o_empty[t]);
        }
      }
    } else if (warp == PRODUCER) {
      // ============================================================ producer of K and V
      uint32_t kc = 0;
      bool k_alone = false;                    // a K was asked for, its V not yet
      if (lane == 0) {
        auto wait = [&](uint64_t* bar, uint32_t parity, int code) {
          if (ok && !lane_wait(bar, parity)) {
            ok = false;
            report(a.err, code);
          }
          return ok;
        };
        for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
          const Item x = item_of(a, it);
          if (x.n == 0) continue;
          for (int j = 0; j < x.n && ok; ++j) {
            const uint32_t i = kc % NS, ph = ((kc / NS) & 1) ^ 1;
            if (!wait(&s.kempty[i], ph, 96)) break;
            ptx::mbar_arrive_expect_tx(&s.kfull[i], kBytes);
#pragma unroll
            for (int p = 0; p < NP; ++p)
              tma_load_4d(s.k[i] + p * kPanel, &tk, 64 * p, x.key0 + j * kTile, x.hk * a.wk.h, x.b * a.wk.b,
                          &s.kfull[i]);
            k_alone = true;
            if (!wait(&s.vempty[i], ph, 96)) break;
            k_alone = false;
            ptx::mbar_arrive_expect_tx(&s.vfull[i], kBytes);
#pragma unroll
            for (int p = 0; p < NP; ++p)
              tma_load_4d(s.v[i] + p * kPanel, &tv, 64 * p, x.key0 + j * kTile, x.hk * a.wv.h, x.b * a.wv.b,
                          &s.vfull[i]);
            ++kc;
          }
        }
        // After a timeout, do not leave while copies issued here may still be landing.
        if (!ok) {
          for (uint32_t c = kc > NS ? kc - NS : 0; c < kc; ++c) {
            lane_wait(&s.kfull[c % NS], (c / NS) & 1);
            lane_wait(&s.vfull[c % NS], (c / NS) & 1);
          }
          if (k_alone) lane_wait(&s.kfull[kc % NS], (kc / NS) & 1);
        }
      }
      __syncwarp();
    } else if (warp == FIXER) {
      // ============================================================ Q; rows of V
      uint32_t kc = 0, qc = 0;
      for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x) {
        const Item x = item_of(a, it);
        if (x.n == 0) continue;
#pragma unroll 1
        for (int t = 0; t < a.tpi; ++t) {
          uint64_t* full = &s.qfull[t][qc % QST];
          if (!wait(&s.qempty[t][qc % QST], ((qc / QST) & 1) ^ 1, 97)) break;
          if (a.packed) {
            gather_rows<NP>(s.q[t][qc % QST], static_cast<const __nv_bfloat16*>(a.q) + x.b * g.q.b, g.q, g.d, lane,
                            [&](int r, int& h, int& n) {
                              const int rr = x.row0 + t * kTile + r;
                              h = x.h + divide(rr, a.by_nq, n);
                              return rr < x.rows;
                            });
            ptx::fence_proxy_async();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full);
          } else if (lane == 0) {
            ptx::mbar_arrive_expect_tx(full, kBytes);
#pragma unroll
            for (int p = 0; p < NP; ++p)
              tma_load_4d(s.q[t][qc % QST] + p * kPanel, &tq, 64 * p, x.row0 + t * kTile, x.h * a.wq.h, x.b * a.wq.b,
                          full);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++qc;
        const uint8_t* mask = a.keys.mask ? a.keys.mask + (int64_t)x.b * g.nk : nullptr;
        for (int j = 0; j < x.n; ++j, ++kc) {
          const int key0 = x.key0 + j * kTile;
          const uint32_t i = kc % NS;
          const bool whole = !mask && key0 + kTile <= x.len;
          uint32_t bits[4];
          if (!whole) key_bits(mask, key0, x.len, lane, bits);
          if (!wait(&s.vfull[i], (kc / NS) & 1, 98)) break;
          if (!whole) {
            clear_rows<NP>(s.v[i], bits, lane);
            ptx::fence_proxy_async();
            __syncwarp();
          }
          if (lane == 0) ptx::mbar_arrive(&s.vready[i]);
        }
      }
      if (!ok && lane == 0 && !a.packed)       // (as above; the last item's copies may not all have been asked for)
        for (int t = 0; t < a.tpi; ++t)
          for (uint32_t c = qc >= QST ? qc + 1 - QST : 0; c <= qc; ++c) lane_wait(&s.qfull[t][c % QST], (c / QST) & 1);
      __syncwarp();
    } else {
      // ============================================================ MMA issue: one warp S, one O
      const bool is_s = warp == MMA_S;
      const uint64_t dk0 = tc::sw128_desc(ptx::smem_u32(s.k[0]), 16, 1024);
      const uint64_t dv0 = tc::sw128_desc(ptx::smem_u32(s.v[0]), kPanel, 1024);
      const uint64_t dq0 = tc::sw128_desc(ptx::smem_u32(s.q[0][0]), 16, 1024);
      constexpr uint64_t kStep = kBytes >> 4;
      const int dsteps = (g.d + 15) >> 4;
      const uint32_t id_o = tc::idesc_bf16(128, 16 * dsteps, 0, 1);      // O += P V: A = P (TMEM), B = V (MN-major)
      uint32_t kc = 0, qc = 0, oc = 0;         // key tiles, items with keys, items
      for (int it = blockIdx.x; it < a.items && ok; it += gridDim.x, ++oc) {
        const Item x = item_of(a, it);
        if (x.n == 0) {                        // no keys: O is not there, the epilogue goes on
          for (int t = 0; t < a.tpi && !is_s; ++t) {
            if (!wait(&s.o_empty[t], (oc & 1) ^ 1, 99)) break;
            if (tc::elect_one()) tc::commit(&s.o_full[t]);
            __syncwarp();
          }
          continue;
        }
        for (int j = 0; j < x.n && ok; ++j, ++kc) {
          const uint32_t i = kc % NS, ph = kc & 1;
          const int cols = tile_cols(x, j);
          if (!wait(is_s ? &s.kfull[i] : &s.vready[i], (kc / NS) & 1, 99)) break;
          if (is_s) {
            const uint32_t id = tc::idesc_bf16(128, cols, 0, 0);
#pragma unroll 1
            for (int t = 0; t < a.tpi; ++t) {
              const uint32_t qs = qc % QST;
              if (j == 0 && !wait(&s.qfull[t][qs], (qc / QST) & 1, 99)) break;
              // NP == 1: the softmax has read the last S; NP == 2: the O update has read P from these columns
              if (!wait(NP == 1 ? &s.s_empty[t] : &s.p_empty[t], ph ^ 1, 99)) break;
              tc::fence_after_sync();
              const uint64_t qd = dq0 + (t * QST + qs) * kStep, kd = dk0 + i * kStep;
              if (tc::elect_one()) {
#pragma unroll
                for (int k = 0; k < 4 * NP; ++k)
                  if (k < dsteps) {
                    const uint64_t o = (uint64_t)(k >> 2) * (kPanel >> 4) + 2u * (k & 3);
                    tc::mma_bf16(tbase + col_s(t), qd + o, kd + o, id, k > 0);
                  }
                tc::commit(&s.s_full[t]);
                if (j == x.n - 1) tc::commit(&s.qempty[t][qs]);
                if (t == a.tpi - 1) tc::commit(&s.kempty[i]);
              }
              __syncwarp();
            }
          } else {
            const int steps = cols >> 4;
#pragma unroll 1
            for (int t = 0; t < a.tpi; ++t) {
              if (!wait(&s.p_full[t], ph, 99)) break;
              if (j == 0 && !wait(&s.o_empty[t], (oc & 1) ^ 1, 99)) break;   // the last item's O has been read
              tc::fence_after_sync();
              const uint64_t vd = dv0 + i * kStep;
              if (tc::elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)    // 16 keys: 8 columns of P, 2 KB of V's panel
                  if (k < steps)
                    tc::mma_bf16_ta(tbase + col_o(t),
                                    tbase + col_p(t) + 8u * k, vd + 128u * k, id_o, j > 0 || k > 0);
                tc::commit(&s.p_empty[t]);
                if (j == x.n - 1) tc::commit(&s.o_full[t]);
                if (t == a.tpi - 1) tc::commit(&s.vempty[i]);
              }
              __syncwarp();
            }
          }
        }
        ++qc;
      }
      // every MMA issued here has finished before TMEM is released
      if (tc::elect_one()) tc::commit(&s.drain[is_s]);
      __syncwarp();
      warp_wait(&s.drain[is_s], 0);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tbase, TMEM_COLS);
  }
}

}  // namespace fwdtc

bool fwd_tc_supported(const Geo& g) {
  return g.bf16 && tokens_apart(g.q, g.nq) && tokens_apart(g.k, g.nk) && tokens_apart(g.v, g.nk);
}

// Items: two query tiles each where that still fills the device; the keys are
// split (whole tiles, as even as they come, two at least, 64 splits at most) when
// there are fewer items than SMs, into four items an SM, rounded up to whole
// splits (fewer than five), so that rows of unlike length even out.
TcPlan plan_fwd_tc(const Geo& g, int sms) {
  TcPlan p;
  p.packed = g.group > 1 && g.nq < kTile;
  p.slices = p.packed ? g.b * g.hk : g.b * g.h;
  const int64_t rows = p.packed ? (int64_t)g.group * g.nq : g.nq;
  const int64_t tiles = (rows + kTile - 1) / kTile;
  p.tpi = tiles > 1 && p.slices * ((tiles + 1) / 2) >= sms ? 2 : 1;
  p.pairs = (int)((tiles + p.tpi - 1) / p.tpi);
  const int64_t items = (int64_t)p.slices * p.pairs;
  const int64_t nkt = (g.nk + kTile - 1) / kTile;
  int64_t ks = 1;
  if (items < sms && nkt >= 4) {
    ks = (4 * sms + items - 1) / items;
    if (ks > nkt / 2) ks = nkt / 2;
    if (ks > 64) ks = 64;
  }
  p.ct = (int)((nkt + ks - 1) / ks);
  p.ks = (int)((nkt + p.ct - 1) / p.ct);
  p.items = items * p.ks;
  return p;
}

template <int NP>
static cudaError_t launch(const fwdtc::Args& a, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                          int grid, cudaStream_t s) {
  const size_t smem = sizeof(fwdtc::Smem<NP>) + 1024;
  cudaError_t e =
      cudaFuncSetAttribute(fwdtc::fwd_tc_kernel<NP>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  fwdtc::fwd_tc_kernel<NP><<<grid, fwdtc::THREADS, smem, s>>>(a, tq, tk, tv);
  note_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_fwd_tc(const Geo& g, const TcPlan& p, const void* q, const void* k, const void* v,
                          const Keys& keys, void* o, float* lse, void* work, cudaStream_t s) {
  fwdtc::Args a;
  CUtensorMap tq, tk, tv;
  cudaError_t e = make_map4(&tq, &a.wq, q, g.q, g.h, g.b, g.nq, g.d, kTile);
  if (e == cudaSuccess) e = make_map4(&tk, &a.wk, k, g.k, g.hk, g.b, g.nk, g.d, kTile);
  if (e == cudaSuccess) e = make_map4(&tv, &a.wv, v, g.v, g.hk, g.b, g.nk, g.d, kTile);
  if (e != cudaSuccess) return e;
  a.g = g;
  a.keys = keys;
  a.q = q;
  a.ks = p.ks;
  a.ct = p.ct;
  a.tpi = p.tpi;
  a.packed = p.packed;
  a.slices = p.slices;
  a.pairs = p.pairs;
  a.items = (int)p.items;
  a.by_ks = divisor(p.ks);
  a.by_pairs = divisor(p.pairs);
  a.by_heads = divisor(p.packed ? g.hk : g.h);
  a.by_group = divisor(g.group);
  a.by_nq = divisor(g.nq);
  a.o = o;
  a.lse = lse;
  a.part = carve_fwd(g, p.ks, work);
  a.err = device_error_word();
  const int sms = sm_count();
  const int grid = a.items < sms ? a.items : sms;
  e = g.d <= 64 ? launch<1>(a, tq, tk, tv, grid, s) : launch<2>(a, tq, tk, tv, grid, s);
  if (e == cudaSuccess && p.ks > 1) e = launch_join_fwd(g, p.ks, a.part, o, lse, s);
  return e;
}

}  // namespace cross
}  // namespace llsa
