// norm.cuh -- shared definitions of the layer-norm kernels.
#pragma once

#include "divisor.cuh"
#include "llsa_internal.cuh"

namespace llsa {
namespace norm {

// Rows in the order of x's memory: three nested runs, the innermost last, with
// the element strides of every tensor (s: of mean / rstd) in each run; where
// the rows of all tensors of a call lie a fixed stride apart it is flat, and
// row r is at r times that stride.  Rows are dealt out in groups that share
// weight and bias (one group, or one per batch row).
struct Geo {
  int groups;
  int64_t rows;              // per group
  Divisor n1, n2;            // rows = n0 * n1 * n2 (n0 implied)
  int64_t x[4], y[4], dy[4], dx[4], s[4];   // [0..2]: runs, outermost first; [3]: group
  int flat_fwd, flat_bwd;    // flat: the stride is that of the innermost run
  int64_t ws, bs;            // between the groups' weights and biases
  int c;
  float eps;
  int bf16, param_bf16;
  int vec;                   // values a load: the most, up to 16 bytes, that c, every stride and every address allow
};

constexpr int kSms = 148;

// Partial sums per group in the backward, and the bytes of the most that any
// strides of the same sizes need (the sizes alone give the workspace).
int bwd_parts(const Geo& g);
inline size_t bwd_work_bytes(Geo g) {
  int most = 0;
  for (g.vec = g.bf16 ? 8 : 4; g.vec; g.vec /= 2) most = bwd_parts(g) > most ? bwd_parts(g) : most;
  return (size_t)g.groups * most * 2 * g.c * sizeof(float);
}

cudaError_t launch_fwd(const Geo& g, const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                       cudaStream_t s);
cudaError_t launch_bwd(const Geo& g, const void* x, const void* dy, const void* w, const float* mean,
                       const float* rstd, void* dx, void* dw, void* db, void* work, cudaStream_t s);

}  // namespace norm
}  // namespace llsa
