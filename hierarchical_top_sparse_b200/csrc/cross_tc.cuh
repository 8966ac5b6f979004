// cross_tc.cuh -- what the tensor-core cross-attention kernels share.
#pragma once

#include "cross.cuh"
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
struct Map4 {
  CUtensorMap map;
};
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

__device__ __forceinline__ void report(int* err, int code) {
  if (err) atomicExch(err, code);
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
// (every lane of one warp).
template <int PANELS>
__device__ __forceinline__ void clear_rows(unsigned char* tile, const uint32_t bits[4], int lane) {
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    uint32_t off = ~bits[i];
    while (off) {
      // four rows at a time: eight lanes write a row's eight 16-byte chunks
      int row = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int first = off ? __ffs(off) - 1 : -1;
        if (lane >> 3 == k) row = first;
        off &= off - 1;
      }
      if (row >= 0)
#pragma unroll
        for (int p = 0; p < PANELS; ++p)
          *reinterpret_cast<uint4*>(tile + p * kPanel + (32 * i + row) * 128 + (lane & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

}  // namespace cross
}  // namespace llsa
