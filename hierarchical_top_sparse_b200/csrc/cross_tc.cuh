// cross_tc.cuh -- what the tensor-core cross-attention kernels share.
#pragma once

#include "cross.cuh"
#include "packed.cuh"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace llsa {
namespace cross {

constexpr uint64_t kWaitLimitNs = 4000000000ull;
constexpr int kTile = 128;           // queries or keys of a tile
constexpr int kPanel = kTile * 128;  // bytes of a [128][64] bf16 panel, 128-byte swizzle

// A token tensor as TMA sees it: channels, tokens, heads, batch rows.  A head
// or batch dimension that the tensor repeats (stride 0), or of one, is left
// out: its coordinate is always 0.
struct Where {
  int h, b;                          // factors of the head and batch coordinates: 1, or 0 where left out
};
cudaError_t make_map4(CUtensorMap* map, Where* w, const void* base, const Lay& lay, int heads, int batch, int n, int d,
                      int box_rows);

// Whether the tensor-core kernels take a tensor: its tokens must lie apart.
inline bool tokens_apart(const Lay& lay, int n) { return n == 1 || lay.n != 0; }

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int n, int h, int b,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(ptx::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(n), "r"(h), "r"(b), "r"(ptx::smem_u32(bar))
      : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// A whole warp waits for a barrier, at most 4 s (the longest wait of a run that
// goes well, the epilogue's for an item of the most tiles, stays under 2 s): all lanes ask, and go on or
// give up together.  The vote before the branch keeps the ready case short
// (about 70 cycles; a branch on each lane's own answer took about 190, and one
// lane asking for all of them longer still).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
  uint32_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1;; ++n) {
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
    if (n & 63u) continue;
    uint32_t now;
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(now));    // (wraps after 4.3 s)
    now = __shfl_sync(0xffffffffu, now, 0);
    if (n == 64u) t0 = now;
    if (now - t0 > 4000000000u) return false;
  }
}

// The same for one lane.  (Neither is a call: a kernel that moves registers
// between its warps cannot make one.)
__device__ __forceinline__ bool lane_wait(uint64_t* bar, uint32_t parity) {
  uint32_t t0 = 0;
#pragma unroll 1
  for (uint32_t n = 1; !ptx::mbar_try_wait(bar, parity); ++n) {
    if (n & 63u) continue;
    uint32_t now;
    asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(now));
    if (n == 64u) t0 = now;
    if (now - t0 > 4000000000u) return false;
  }
  return true;
}

// The registers of a thread, for all warps of a warpgroup at once.
template <int N> __device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N> __device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ void report(int* err, int code) {
  if (err) atomicExch(err, code);
}

// n / v.d, and n modulo v.d into rest.
__device__ __forceinline__ int divide(int n, const Divisor& v, int& rest) {
  const uint32_t q = over((uint32_t)n, v);
  rest = (int)((uint32_t)n - q * v.d);
  return (int)q;
}

// Bits of the 128 keys from key0 on that take part; lane i of the returned
// words' warp holds nothing of its own: all four words in every lane.
__device__ __forceinline__ void key_bits(const uint8_t* mask, int key0, int n, int lane, uint32_t bits[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int key = key0 + 32 * i + lane;
    const bool ok = key < n && (!mask || mask[key]);
    bits[i] = __ballot_sync(0xffffffffu, ok);
  }
}

// Zeros the rows of a swizzled [128][64 x panels] tile whose bit is clear
// (every lane of one warp): four rows at a time, eight lanes a row.
template <int PANELS>
__device__ __forceinline__ void clear_rows(unsigned char* tile, const uint32_t bits[4], int lane) {
  unsigned char* at = tile + (lane >> 3) * 128 + (lane & 7) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t off = ~bits[i] >> (lane >> 3);
    if (bits[i] == 0xffffffffu) continue;
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if ((off >> (4 * r)) & 1u)
#pragma unroll
        for (int p = 0; p < PANELS; ++p)
          *reinterpret_cast<uint4*>(at + p * kPanel + (32 * i + 4 * r) * 128) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Gathers the 128 rows that at(r, head, token) names (zeros where it says
// false) from a batch row at `base` into a swizzled tile (every lane of a warp).
template <int PANELS, typename At>
__device__ __forceinline__ void gather_rows(unsigned char* tile, const __nv_bfloat16* base, const Lay& lay, int d,
                                            int lane, At at) {
#pragma unroll 4
  for (int e = lane; e < kTile * 8 * PANELS; e += 32) {
    const int r = e / (8 * PANELS), ch = e % (8 * PANELS);
    int h, n;
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (at(r, h, n) && ch * 8 < d) w = *reinterpret_cast<const uint4*>(base + h * lay.h + n * lay.n + ch * 8);
    *reinterpret_cast<uint4*>(tile + (ch >> 3) * kPanel + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = w;
  }
}

// 16 channels (8 unless `both`) as bf16 to `out`, or, where that is null, as fp32 to `part`.
__device__ __forceinline__ void store16(const float* f, __nv_bfloat16* out, float* part, bool both) {
  if (out) {
    uint4* d4 = reinterpret_cast<uint4*>(out);
    d4[0] = make_uint4(ptx::pack_bf16(f[0], f[1]), ptx::pack_bf16(f[2], f[3]), ptx::pack_bf16(f[4], f[5]),
                       ptx::pack_bf16(f[6], f[7]));
    if (both)
      d4[1] = make_uint4(ptx::pack_bf16(f[8], f[9]), ptx::pack_bf16(f[10], f[11]), ptx::pack_bf16(f[12], f[13]),
                         ptx::pack_bf16(f[14], f[15]));
  } else {
    float4* d4 = reinterpret_cast<float4*>(part);
    d4[0] = make_float4(f[0], f[1], f[2], f[3]);
    d4[1] = make_float4(f[4], f[5], f[6], f[7]);
    if (both) {
      d4[2] = make_float4(f[8], f[9], f[10], f[11]);
      d4[3] = make_float4(f[12], f[13], f[14], f[15]);
    }
  }
}

inline int sm_count() {
  int dev = 0, sms = 148;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms;
}

int splits_of_queries(int64_t slices, int units, int sms);

// The backward where all keys fit one tile (nk <= 128).
struct OnePlan {
  int packed, qs, nqt, units;
  int64_t items;
};
OnePlan plan_bwd_one(const Geo& g, int sms);
cudaError_t launch_bwd_one(const Geo& g, const OnePlan& p, const CUtensorMap* t, const Where* w, const void* q,
                           const Keys& keys, const void* dO, const float* lse, void* dq, void* dk, void* dv,
                           float* partk, float* partv, cudaStream_t s);

// The parts of the backward for more than one tile of keys.  t, w: maps of q,
// k, v, dO with boxes of 128 tokens.
struct DqPlan {
  int packed, ks, ct, tiles;
  int64_t items;
};
DqPlan plan_bwd_q(const Geo& g, int sms);
cudaError_t launch_bwd_q(const Geo& g, const DqPlan& p, const CUtensorMap* t, const Where* w, const void* q,
                         const Keys& keys, const void* dO, const float* lse, const float* D, void* dq, float* part,
                         cudaStream_t s);
struct DkvPlan {
  int packed, qs, nqt, units, tiles;
  int64_t items;
};
DkvPlan plan_bwd_kv(const Geo& g, int sms);
cudaError_t launch_bwd_kv(const Geo& g, const DkvPlan& p, const CUtensorMap* t, const Where* w, const void* q,
                          const Keys& keys, const void* dO, const float* lse, const float* D, void* dk, void* dv,
                          float* partk, float* partv, cudaStream_t s);

}  // namespace cross
}  // namespace llsa
