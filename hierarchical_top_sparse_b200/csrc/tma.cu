// tma.cu -- TMA tensor-map encoding through the driver entry point (no libcuda link).
#include <cudaTypedefs.h>

#include <mutex>

#include "cross_tc.cuh"
#include "llsa_internal.cuh"

namespace llsa {

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

cudaError_t make_token_map_box(CUtensorMap* map, const void* base, int64_t rows, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  if (((uintptr_t)base & 15u) != 0 || box_rows < 1 || box_rows > 256) return cudaErrorInvalidValue;
  cuuint64_t dims[2] = {64, (cuuint64_t)rows};
  cuuint64_t strides[1] = {64 * sizeof(__nv_bfloat16)};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
  cuuint32_t estr[2] = {1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_run_maps(RunMaps* maps, const void* base, int64_t rows) {
  for (int r = 0; r < kRunMax; ++r) {
    cudaError_t e = make_token_map_box(&maps->m[r], base, rows, 16 * (r + 1));
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

namespace cross {

cudaError_t make_map4(CUtensorMap* map, Where* w, const void* base, const Lay& lay, int heads, int batch, int n, int d,
                      int box_rows) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  w->h = heads > 1 && lay.h != 0;
  w->b = batch > 1 && lay.b != 0;
  const cuuint64_t es = sizeof(__nv_bfloat16);
  const cuuint64_t plain = (cuuint64_t)d * es;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)n, w->h ? (cuuint64_t)heads : 1, w->b ? (cuuint64_t)batch : 1};
  cuuint64_t strides[3] = {n > 1 ? (cuuint64_t)lay.n * es : plain, w->h ? (cuuint64_t)lay.h * es : plain,
                           w->b ? (cuuint64_t)lay.b * es : plain};
  cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace cross

}  // namespace llsa
