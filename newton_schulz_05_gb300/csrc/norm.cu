// Layer norm, alone or behind dropout and the residual add, and its gradient
// with the reduction of the weight's and the bias's.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "random.cuh"

namespace muon {

namespace {

constexpr int kNormThreads = 256;
constexpr int kNormParts = 304;      // partial column sums of a gradient

struct NormFwd {
  int64_t rows, cols, ldx, ldr;
  const void *x, *residual, *weight, *bias;
  void *sum, *y;
  float *mean, *rstd;
  float eps;
  int drop;
  Drop d;
};

struct NormBwd {
  int64_t rows, cols, lddy, lds, ldds;
  const void *dy, *sum, *dsum, *weight;
  const float *mean, *rstd;
  void *dx, *dresidual;
  float* part;      // [parts][2][cols]
  int drop;
  Drop d;
};

// sum over the block, the same value in every thread
template <int NT>
__device__ __forceinline__ float block_all_sum(float v, float* red /* NT/32 + 1 floats */) {
  const float s = block_sum<NT>(v, red);
  if (threadIdx.x == 0) red[NT / 32] = s;
  __syncthreads();
  const float r = red[NT / 32];
  __syncthreads();
  return r;
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kNormThreads) norm_fwd_kernel(const __grid_constant__ NormFwd a) {
  __shared__ float red[kNormThreads / 32 + 1];
  const T* x = static_cast<const T*>(a.x);
  const T* r = static_cast<const T*>(a.residual);
  const WT* w = static_cast<const WT*>(a.weight);
  const WT* b = static_cast<const WT*>(a.bias);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    auto value = [&](int64_t c) {
      float v = to_f(x[row * a.ldx + c]);
      if (a.drop) v = drop_one(v, (uint64_t)(row * a.cols + c), a.d);
      return r ? v + to_f(r[row * a.ldr + c]) : v;
    };
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) s += value(c);
    const float mean = block_all_sum<kNormThreads>(s, red) / (float)a.cols;
    float q = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
      const float e = value(c) - mean;
      q = fmaf(e, e, q);
    }
    const float rstd = 1.f / sqrtf(block_all_sum<kNormThreads>(q, red) / (float)a.cols + a.eps);
    for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
      const float v = value(c);
      const float h = (v - mean) * rstd;
      static_cast<T*>(a.y)[row * a.cols + c] =
          from_f<T>(fmaf(h, w ? to_f(w[c]) : 1.f, b ? to_f(b[c]) : 0.f));
      if (a.sum) static_cast<T*>(a.sum)[row * a.cols + c] = from_f<T>(v);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kNormThreads) norm_bwd_kernel(const __grid_constant__ NormBwd a) {
  __shared__ float red[kNormThreads / 32 + 1];
  const T* dy = static_cast<const T*>(a.dy);
  const T* sum = static_cast<const T*>(a.sum);
  const T* ds = static_cast<const T*>(a.dsum);
  const WT* w = static_cast<const WT*>(a.weight);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    float sg = 0.f, sh = 0.f;
    for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
      const float g = to_f(dy[row * a.lddy + c]) * (w ? to_f(w[c]) : 1.f);
      sg += g;
      sh = fmaf(g, (to_f(sum[row * a.lds + c]) - mean) * rstd, sh);
    }
    sg = block_all_sum<kNormThreads>(sg, red) / (float)a.cols;
    sh = block_all_sum<kNormThreads>(sh, red) / (float)a.cols;
    for (int64_t c = threadIdx.x; c < a.cols; c += kNormThreads) {
      const float g = to_f(dy[row * a.lddy + c]) * (w ? to_f(w[c]) : 1.f);
      const float h = (to_f(sum[row * a.lds + c]) - mean) * rstd;
      float d = rstd * (g - sg - h * sh);
      if (ds) d += to_f(ds[row * a.ldds + c]);
      if (a.dresidual) static_cast<T*>(a.dresidual)[row * a.cols + c] = from_f<T>(d);
      if (a.drop) d = drop_one(d, (uint64_t)(row * a.cols + c), a.d);
      if (a.dx) static_cast<T*>(a.dx)[row * a.cols + c] = from_f<T>(d);
    }
  }
}

// partial column sums: block (part, column tile) adds up rows part, part + parts, ...
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_cols_kernel(const __grid_constant__ NormBwd a) {
  const T* dy = static_cast<const T*>(a.dy);
  const T* sum = static_cast<const T*>(a.sum);
  for (int64_t c = (int64_t)blockIdx.y * kNormThreads + threadIdx.x; c < a.cols;
       c += (int64_t)gridDim.y * kNormThreads) {
    float w = 0.f, b = 0.f;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
      const float g = to_f(dy[row * a.lddy + c]);
      w = fmaf(g, (to_f(sum[row * a.lds + c]) - a.mean[row]) * a.rstd[row], w);
      b += g;
    }
    a.part[(int64_t)blockIdx.x * 2 * a.cols + c] = w;
    a.part[((int64_t)blockIdx.x * 2 + 1) * a.cols + c] = b;
  }
}

template <typename WT>
__global__ void __launch_bounds__(kNormThreads) norm_join_kernel(int64_t cols, int parts,
                                                                 const float* part, WT* dweight,
                                                                 WT* dbias) {
  for (int64_t c = (int64_t)blockIdx.x * kNormThreads + threadIdx.x; c < cols;
       c += (int64_t)gridDim.x * kNormThreads) {
    float w = 0.f, b = 0.f;
    for (int i = 0; i < parts; ++i) {
      w += part[(int64_t)i * 2 * cols + c];
      b += part[((int64_t)i * 2 + 1) * cols + c];
    }
    if (dweight) dweight[c] = from_f<WT>(w);
    if (dbias) dbias[c] = from_f<WT>(b);
  }
}

int norm_parts(int64_t rows) { return (int)(rows < kNormParts ? rows : kNormParts); }

bool misaligned(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

muon_status check_common(int64_t rows, int64_t cols, int dtype, int wdtype, float p) {
  if (rows < 0 || !(p >= 0.f && p <= 1.f)) return MUON_ERR_INVALID_ARG;
  if (cols < 1 || cols > (int64_t)1 << 30 || rows > (int64_t)1 << 40)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  if ((dtype != MUON_BF16 && dtype != MUON_F32) || (wdtype != MUON_BF16 && wdtype != MUON_F32))
    return MUON_ERR_DTYPE;
  return MUON_OK;
}

template <typename F>
void by_types(int dtype, int wdtype, F f) {
  if (dtype == MUON_BF16) {
    if (wdtype == MUON_BF16) f(__nv_bfloat16(), __nv_bfloat16());
    else f(__nv_bfloat16(), float());
  } else {
    if (wdtype == MUON_BF16) f(float(), __nv_bfloat16());
    else f(float(), float());
  }
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_layer_norm(int64_t rows, int64_t cols, int dtype, int wdtype,
                                       const void* x, int64_t ldx, const void* residual,
                                       int64_t ldr, const void* weight, const void* bias,
                                       float eps, float p, uint64_t seed, uint64_t offset,
                                       void* sum, void* y, float* mean, float* rstd,
                                       void* stream) {
  const muon_status st = check_common(rows, cols, dtype, wdtype, p);
  if (st != MUON_OK) return st;
  if (!std::isfinite(eps) || eps < 0.f || ldx < 0 || ldr < 0 || (rows > 0 && (!x || !y)))
    return MUON_ERR_INVALID_ARG;
  const size_t es = dtype == MUON_BF16 ? 2 : 4, ws = wdtype == MUON_BF16 ? 2 : 4;
  if (misaligned(x, es) || misaligned(residual, es) || misaligned(sum, es) || misaligned(y, es) ||
      misaligned(weight, ws) || misaligned(bias, ws) || misaligned(mean, 4) || misaligned(rstd, 4))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (rows == 0) return MUON_OK;
  NvtxRange range("muon_layer_norm");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const NormFwd a = {rows, cols, ldx, ldr, x, residual, weight, bias, sum, y, mean, rstd, eps,
                     p > 0.f, make_drop(p, seed, offset)};
  const int grid = (int)(rows < 152 * 8 ? rows : 152 * 8);
  by_types(dtype, wdtype, [&](auto t, auto wt) {
    norm_fwd_kernel<decltype(t), decltype(wt)><<<grid, kNormThreads, 0, s>>>(a);
  });
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" muon_status muon_layer_norm_workspace_bytes(int64_t rows, int64_t cols, size_t* out) {
  if (!out || rows < 0) return MUON_ERR_INVALID_ARG;
  if (cols < 1 || cols > (int64_t)1 << 30) return MUON_ERR_UNSUPPORTED_SHAPE;
  *out = (size_t)norm_parts(rows) * 2 * (size_t)cols * sizeof(float) + 256;
  return MUON_OK;
}

extern "C" muon_status muon_layer_norm_backward(
    int64_t rows, int64_t cols, int dtype, int wdtype, const void* dy, int64_t lddy,
    const void* sum, int64_t ldsum, const float* mean, const float* rstd, const void* weight,
    const void* dsum, int64_t ldds, float p, uint64_t seed, uint64_t offset, void* dx,
    void* dresidual, void* dweight, void* dbias, void* workspace, size_t ws_bytes, void* stream) {
  const muon_status st = check_common(rows, cols, dtype, wdtype, p);
  if (st != MUON_OK) return st;
  if (lddy < 0 || ldsum < 0 || ldds < 0 || (rows > 0 && (!dy || !sum || !mean || !rstd)))
    return MUON_ERR_INVALID_ARG;
  const size_t es = dtype == MUON_BF16 ? 2 : 4, ws = wdtype == MUON_BF16 ? 2 : 4;
  if (misaligned(dy, es) || misaligned(sum, es) || misaligned(dsum, es) || misaligned(dx, es) ||
      misaligned(dresidual, es) || misaligned(weight, ws) || misaligned(dweight, ws) ||
      misaligned(dbias, ws) || misaligned(mean, 4) || misaligned(rstd, 4))
    return MUON_ERR_ALIGNMENT;
  const bool cols_wanted = dweight || dbias;
  if (cols_wanted && rows > 0) {
    size_t need = 0;
    muon_layer_norm_workspace_bytes(rows, cols, &need);
    if (!workspace) return MUON_ERR_INVALID_ARG;
    if (misaligned(workspace, 256)) return MUON_ERR_ALIGNMENT;
    if (ws_bytes < need) return MUON_ERR_WORKSPACE;
  }
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  NvtxRange range("muon_layer_norm_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // empty sums
    if (dweight && cudaMemsetAsync(dweight, 0, (size_t)cols * ws, s) != cudaSuccess)
      return MUON_ERR_CUDA;
    if (dbias && cudaMemsetAsync(dbias, 0, (size_t)cols * ws, s) != cudaSuccess)
      return MUON_ERR_CUDA;
    return MUON_OK;
  }
  const NormBwd a = {rows, cols, lddy, ldsum, ldds, dy, sum, dsum, weight, mean, rstd, dx,
                     dresidual, static_cast<float*>(workspace), p > 0.f,
                     make_drop(p, seed, offset)};
  const int parts = norm_parts(rows);
  const int tiles = (int)((cols + kNormThreads - 1) / kNormThreads < 65535
                              ? (cols + kNormThreads - 1) / kNormThreads : 65535);
  by_types(dtype, wdtype, [&](auto t, auto wt) {
    using T = decltype(t);
    using WT = decltype(wt);
    if (dx || dresidual)
      norm_bwd_kernel<T, WT><<<(int)(rows < 152 * 8 ? rows : 152 * 8), kNormThreads, 0, s>>>(a);
    if (cols_wanted) {
      norm_cols_kernel<T><<<dim3(parts, tiles), kNormThreads, 0, s>>>(a);
      norm_join_kernel<WT><<<tiles, kNormThreads, 0, s>>>(
          cols, parts, a.part, static_cast<WT*>(dweight), static_cast<WT*>(dbias));
    }
  });
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
