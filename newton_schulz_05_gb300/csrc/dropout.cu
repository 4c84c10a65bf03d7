// Dropout from a counter-based generator, alone or added to a residual.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "random.cuh"

namespace muon {

namespace {

template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(int64_t n, const T* x, const T* residual,
                                                      Drop d, T* y) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * blockDim.x) {
    float v = drop_one(to_f(x[i]), (uint64_t)i, d);
    if (residual) v += to_f(residual[i]);
    y[i] = from_f<T>(v);
  }
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_dropout(int64_t n, int dtype, const void* x, const void* residual,
                                    float p, uint64_t seed, uint64_t offset, void* y,
                                    void* stream) {
  if (n < 0 || (n > 0 && (!x || !y)) || !(p >= 0.f && p <= 1.f)) return MUON_ERR_INVALID_ARG;
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_DTYPE;
  const size_t es = dtype == MUON_BF16 ? 2 : 4;
  if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
       reinterpret_cast<uintptr_t>(y)) % es)
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (n == 0) return MUON_OK;
  NvtxRange range("muon_dropout");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Drop d = make_drop(p, seed, offset);
  const int64_t want = (n + 255) / 256;
  const int grid = (int)(want < 152 * 8 ? want : 152 * 8);
  if (dtype == MUON_BF16)
    dropout_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
        n, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(residual), d,
        static_cast<__nv_bfloat16*>(y));
  else
    dropout_kernel<float><<<grid, 256, 0, s>>>(n, static_cast<const float*>(x),
                                               static_cast<const float*>(residual), d,
                                               static_cast<float*>(y));
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
