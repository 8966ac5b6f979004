// cross.cuh -- shared definitions of the cross-attention kernels.
#pragma once

#include "divisor.cuh"
#include "llsa_internal.cuh"

namespace llsa {
namespace cross {

struct Lay {                 // element strides of a [batch][heads][tokens][d] tensor
  int64_t b, h, n;
};

struct Geo {
  int b, h, hk, group;       // batch rows, query heads, key heads, query heads per key head
  int nq, nk, d;
  float scale;
  int bf16;
  Lay q, k, v, o, dO, dq, dk, dv;
};

// Keys per tile of a split's unit and the splits of one problem.  A split of
// the keys takes whole key tiles, a split of the queries whole query tiles.
struct Plan {
  int fwd_ks;                // key splits of the forward (1: O is written directly)
  int dq_ks;                 // key splits of dQ
  int dkv_qs;                // query splits of dK / dV
};

// The keys that take part: the first len(b) of the batch row, less those whose mask byte is zero.
struct Keys {
  const int32_t* len;
  const uint8_t* mask;
};

__device__ __forceinline__ int key_count(const Geo& g, const Keys& keys, int b) {
  if (!keys.len) return g.nk;
  const int n = keys.len[b];
  return n < 0 ? 0 : (n > g.nk ? g.nk : n);
}

__host__ __device__ inline int64_t rows_of(const Geo& g) { return (int64_t)g.b * g.h * g.nq; }
__host__ __device__ inline int64_t keys_of(const Geo& g) { return (int64_t)g.b * g.hk * g.nk; }

inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

struct FwdWork {
  float* o;                  // [splits][rows][d] normalised partial outputs
  float* lse;                // [splits][rows]
};
struct BwdWork {
  float* D;                  // [rows] rowsum(dO * O)
  float* dq;                 // [splits][rows][d]
  float* dk;                 // [splits][keys][d]
  float* dv;
};

inline size_t fwd_work_bytes(const Geo& g, int ks) {
  if (ks <= 1) return 0;
  return round256((size_t)ks * rows_of(g) * g.d * 4) + round256((size_t)ks * rows_of(g) * 4);
}
inline FwdWork carve_fwd(const Geo& g, int ks, void* work) {
  if (ks <= 1) return FwdWork{nullptr, nullptr};
  char* w = static_cast<char*>(work);
  return FwdWork{reinterpret_cast<float*>(w),
                 reinterpret_cast<float*>(w + round256((size_t)ks * rows_of(g) * g.d * 4))};
}

// Joins the key splits of the forward; sums the splits of a gradient.
cudaError_t launch_join_fwd(const Geo& g, int ks, const FwdWork& w, void* o, float* lse, cudaStream_t s);
cudaError_t launch_row_dot(const Geo& g, const void* o, const void* dO, float* D, cudaStream_t s);
cudaError_t launch_sum_q(const Geo& g, int parts, const float* part, void* dq, cudaStream_t s);
cudaError_t launch_sum_kv(const Geo& g, int parts, const float* partk, const float* partv, void* dk, void* dv,
                          cudaStream_t s);

// Tensor-core forward (bf16).  The plan follows from the sizes alone.
struct TcPlan {
  int ks, ct, tpi, packed, slices, pairs;
  int64_t items;
};
bool fwd_tc_supported(const Geo& g);
TcPlan plan_fwd_tc(const Geo& g, int sms);
cudaError_t launch_fwd_tc(const Geo& g, const TcPlan& p, const void* q, const void* k, const void* v,
                          const Keys& keys, void* o, float* lse, void* work, cudaStream_t s);

// Forward for at most 16 query rows a key head (bf16).
bool token_supported(const Geo& g);
size_t token_work_bytes(const Geo& g, int sms);
cudaError_t launch_fwd_token(const Geo& g, int sms, const void* q, const void* k, const void* v, const Keys& keys,
                             void* o, float* lse, void* work, cudaStream_t s);

// Tensor-core backward (bf16).
bool bwd_tc_supported(const Geo& g);
size_t bwd_work_bytes_tc(const Geo& g, int sms);
cudaError_t launch_bwd_tc(const Geo& g, int sms, const void* q, const void* k, const void* v, const Keys& keys,
                          const void* o, const void* dO, const float* lse, void* dq, void* dk, void* dv, void* work,
                          cudaStream_t s);

// CUDA-core kernels (fp32 FMA), either type.
Plan plan_simt(const Geo& g, int sms);
size_t bwd_work_bytes_simt(const Geo& g, const Plan& p);
cudaError_t launch_fwd_simt(const Geo& g, const Plan& p, const void* q, const void* k, const void* v,
                            const Keys& keys, void* o, float* lse, void* work, cudaStream_t s);
cudaError_t launch_bwd_simt(const Geo& g, const Plan& p, const void* q, const void* k, const void* v,
                            const Keys& keys, const void* o, const void* dO, const float* lse, void* dq, void* dk,
                            void* dv, void* work, cudaStream_t s);

}  // namespace cross
}  // namespace llsa
