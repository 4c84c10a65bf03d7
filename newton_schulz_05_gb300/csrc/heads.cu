// Norms of query and key heads with the rotation of positions, and the gradient.
#include "sequence.cuh"

namespace muon {

namespace {

constexpr int kHeadThreads = 256, kHeadWarps = kHeadThreads / 32;
constexpr int kHeadMaxDim = 1024;
constexpr int kHeadParts = 304;       // blocks of the gradient, images of its weight sums

// Queries or keys: heads `step` elements apart, tokens `ld`
struct HeadSide {
  const void *x, *dy, *weight;
  int64_t ld, step, lddy, stepdy;
  void *out, *dweight;
  int heads;
};
struct Heads {
  int64_t tokens, table, period;
  int dim, rotary, neighbours;
  float eps;
  const float *cos, *sin;
  const int64_t* positions;
  HeadSide side[2];
  float* part;
};

__device__ __forceinline__ float warp_sum(float v) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// row of the table, or -1: no token
__device__ __forceinline__ int64_t position_of(const Heads& a, int64_t t) {
  if (!a.rotary) return 0;
  const int64_t p = a.positions ? a.positions[t] : t % a.period;
  return p >= 0 && p < a.table ? p : -1;
}
// f(i, j, c, s): each of a lane's pairs; f1(i): each of its other elements
template <typename F, typename F1>
__device__ __forceinline__ void pairs(const Heads& a, int64_t pos, F f, F1 f1) {
  const int half = a.rotary / 2, lane = threadIdx.x & 31;
  for (int m = lane; m < half; m += 32)
    f(a.neighbours ? 2 * m : m, a.neighbours ? 2 * m + 1 : m + half, a.cos[pos * half + m],
      a.sin[pos * half + m]);
  for (int i = a.rotary + lane; i < a.dim; i += 32) f1(i);
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kHeadThreads) heads_kernel(const __grid_constant__ Heads a) {
  pdl_wait();
  const int lane = threadIdx.x & 31, all = a.side[0].heads + a.side[1].heads;
  for (int64_t u = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); u < a.tokens * all;
       u += (int64_t)gridDim.x * kHeadWarps) {
    const int64_t t = u / all;
    int hd = (int)(u % all);
    const bool key = hd >= a.side[0].heads;
    const HeadSide& s = a.side[key];
    if (key) hd -= a.side[0].heads;
    const T* x = static_cast<const T*>(s.x) + t * s.ld + hd * s.step;
    T* out = static_cast<T*>(s.out) + (t * s.heads + hd) * a.dim;
    const WT* w = static_cast<const WT*>(s.weight);
    const int64_t pos = position_of(a, t);
    if (pos < 0) {
      for (int i = lane; i < a.dim; i += 32) out[i] = from_f<T>(0.f);
      continue;
    }
    float sq = 0.f;
    for (int i = lane; i < a.dim; i += 32) sq = fmaf(to_f(x[i]), to_f(x[i]), sq);
    const float rstd = 1.f / sqrtf(warp_sum(sq) / a.dim + a.eps);
    auto n = [&](int i) { return to_f(x[i]) * rstd * (w ? to_f(w[i]) : 1.f); };
    pairs(a, pos,
          [&](int i, int j, float c, float sn) {
            const float u = n(i), v = n(j);
            out[i] = from_f<T>(u * c - v * sn);
            out[j] = from_f<T>(v * c + u * sn);
          },
          [&](int i) { out[i] = from_f<T>(n(i)); });
  }
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kHeadThreads) heads_bwd_kernel(const __grid_constant__ Heads a) {
  extern __shared__ float sums[];     // a warp: [2][dim], then [dim] of g
  pdl_wait();
  const int lane = threadIdx.x & 31, all = a.side[0].heads + a.side[1].heads;
  float* mine = sums + (threadIdx.x >> 5) * 3 * a.dim;
  float* g = mine + 2 * a.dim;
  for (int i = lane; i < 2 * a.dim; i += 32) mine[i] = 0.f;
  for (int64_t u = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); u < a.tokens * all;
       u += (int64_t)gridDim.x * kHeadWarps) {
    const int64_t t = u / all;
    int hd = (int)(u % all);
    const int key = hd >= a.side[0].heads;
    const HeadSide& s = a.side[key];
    if (key) hd -= a.side[0].heads;
    const T* x = static_cast<const T*>(s.x) + t * s.ld + hd * s.step;
    const T* dy = static_cast<const T*>(s.dy) + t * s.lddy + hd * s.stepdy;
    T* out = static_cast<T*>(s.out) + (t * s.heads + hd) * a.dim;
    const WT* w = static_cast<const WT*>(s.weight);
    const int64_t pos = position_of(a, t);
    if (pos < 0) {
      if (s.out)
        for (int i = lane; i < a.dim; i += 32) out[i] = from_f<T>(0.f);
      continue;
    }
    __syncwarp();
    pairs(a, pos,
          [&](int i, int j, float c, float sn) {
            const float u = to_f(dy[i]), v = to_f(dy[j]);
            g[i] = u * c + v * sn;
            g[j] = v * c - u * sn;
          },
          [&](int i) { g[i] = to_f(dy[i]); });
    __syncwarp();
    float sq = 0.f, dot = 0.f;
    for (int i = lane; i < a.dim; i += 32) {
      const float v = to_f(x[i]);
      sq = fmaf(v, v, sq);
      dot = fmaf(g[i] * (w ? to_f(w[i]) : 1.f), v, dot);
    }
    const float rstd = 1.f / sqrtf(warp_sum(sq) / a.dim + a.eps);
    const float mean = warp_sum(dot) * rstd / a.dim;
    for (int i = lane; i < a.dim; i += 32) {
      const float h = to_f(x[i]) * rstd;
      mine[key * a.dim + i] += g[i] * h;
      if (s.out) out[i] = from_f<T>((g[i] * (w ? to_f(w[i]) : 1.f) - h * mean) * rstd);
    }
  }
  __syncthreads();
  if (!a.part) return;
  for (int i = threadIdx.x; i < 2 * a.dim; i += kHeadThreads) {
    float v = 0.f;
    for (int k = 0; k < kHeadWarps; ++k) v += sums[k * 3 * a.dim + i];
    a.part[(int64_t)blockIdx.x * 2 * a.dim + i] = v;
  }
}

template <typename WT>
__global__ void __launch_bounds__(kHeadThreads)
heads_join_kernel(int dim, int parts, const float* part, WT* dq, WT* dk) {
  pdl_wait();
  const int i = blockIdx.x * kHeadThreads + threadIdx.x;
  if (i >= 2 * dim) return;
  float v = 0.f;
  for (int p = 0; p < parts; ++p) v += part[(int64_t)p * 2 * dim + i];
  WT* out = i < dim ? dq : dk;
  if (out) out[i < dim ? i : i - dim] = from_f<WT>(v);
}

// --------------------------------------------------------------------- host

int64_t head_parts(int64_t tokens, int heads) {
  const int64_t want = (tokens * heads + kHeadWarps - 1) / kHeadWarps;
  return want < kHeadParts ? want : kHeadParts;
}

muon_status check_heads(int64_t tokens, int q_heads, int k_heads, int dim, int rotary, int dtype,
                        int wdtype, float eps, const float* cos, const float* sin, int64_t table,
                        const int64_t* positions, int64_t period) {
  if (tokens < 0 || q_heads < 0 || k_heads < 0 || rotary < 0 || !(eps >= 0.f) || std::isinf(eps))
    return MUON_ERR_INVALID_ARG;
  if (tokens >= (int64_t)1 << 31 || q_heads > 65536 || k_heads > 65536 || dim < 1 ||
      dim > kHeadMaxDim || rotary > dim || rotary % 2)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  if (!known(dtype) || !known(wdtype)) return MUON_ERR_DTYPE;
  if (rotary && (table < 0 || (table > 0 && (!cos || !sin)) || (!positions && period < 1)))
    return MUON_ERR_INVALID_ARG;
  if (off(cos, 4) || off(sin, 4) || off(positions, 8)) return MUON_ERR_ALIGNMENT;
  return MUON_OK;
}

template <typename F> cudaError_t by_both(int dtype, int wdtype, F f) {
  return by_type(dtype, [&](auto t) { return by_type(wdtype, [&](auto w) { return f(t, w); }); });
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_norm_rotate_heads(
    int64_t tokens, int q_heads, int k_heads, int dim, int rotary, int dtype, int wdtype,
    const void* q, int64_t ldq, int64_t q_step, const void* k, int64_t ldk, int64_t k_step,
    const void* q_weight, const void* k_weight, float eps, const float* cos, const float* sin,
    int64_t table, const int64_t* positions, int64_t period, int neighbours, void* q_out,
    void* k_out, void* stream) {
  const muon_status st = check_heads(tokens, q_heads, k_heads, dim, rotary, dtype, wdtype, eps, cos, sin,
                                     table, positions, period);
  if (st != MUON_OK) return st;
  if (ldq < 0 || ldk < 0 || q_step < 0 || k_step < 0 || (tokens > 0 && q_heads > 0 && (!q || !q_out)) ||
      (tokens > 0 && k_heads > 0 && (!k || !k_out)))
    return MUON_ERR_INVALID_ARG;
  if (any_off(size_of(dtype), q, k, q_out, k_out) || any_off(size_of(wdtype), q_weight, k_weight))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (tokens == 0 || q_heads + k_heads == 0) return MUON_OK;
  NvtxRange range("muon_norm_rotate_heads");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Heads a = {tokens, table, period, dim, rotary, neighbours, eps, cos, sin, positions,
                   {{q, nullptr, q_weight, ldq, q_step, 0, 0, q_out, nullptr, q_heads},
                    {k, nullptr, k_weight, ldk, k_step, 0, 0, k_out, nullptr, k_heads}},
                   nullptr};
  const int64_t want = (tokens * (q_heads + k_heads) + kHeadWarps - 1) / kHeadWarps;
  const cudaError_t e = by_both(dtype, wdtype, [&](auto t, auto w) {
    return launch_k(heads_kernel<decltype(t), decltype(w)>, dim3((unsigned)(want < 152 * 8 ? want : 152 * 8)),
                    dim3(kHeadThreads), 0, s, true, a);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" muon_status muon_norm_rotate_heads_workspace_bytes(int64_t tokens, int q_heads,
                                                              int k_heads, int dim, size_t* out) {
  if (!out || tokens < 0 || q_heads < 0 || k_heads < 0) return MUON_ERR_INVALID_ARG;
  if (tokens >= (int64_t)1 << 31 || q_heads > 65536 || k_heads > 65536 || dim < 1 || dim > kHeadMaxDim)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  *out = (size_t)head_parts(tokens, q_heads + k_heads) * 2 * dim * sizeof(float) + 256;
  return MUON_OK;
}

extern "C" muon_status muon_norm_rotate_heads_backward(
    int64_t tokens, int q_heads, int k_heads, int dim, int rotary, int dtype, int wdtype,
    const void* dq, int64_t lddq, int64_t dq_step, const void* dk, int64_t lddk, int64_t dk_step,
    const void* q, int64_t ldq, int64_t q_step, const void* k, int64_t ldk, int64_t k_step,
    const void* q_weight, const void* k_weight, float eps, const float* cos, const float* sin,
    int64_t table, const int64_t* positions, int64_t period, int neighbours, void* q_grad,
    void* k_grad, void* q_dweight, void* k_dweight, void* workspace, size_t ws_bytes,
    void* stream) {
  const muon_status st = check_heads(tokens, q_heads, k_heads, dim, rotary, dtype, wdtype, eps, cos, sin,
                                     table, positions, period);
  if (st != MUON_OK) return st;
  if (lddq < 0 || lddk < 0 || dq_step < 0 || dk_step < 0 || ldq < 0 || ldk < 0 || q_step < 0 ||
      k_step < 0 || (tokens > 0 && q_heads > 0 && (!q || !dq)) ||
      (tokens > 0 && k_heads > 0 && (!k || !dk)))
    return MUON_ERR_INVALID_ARG;
  const size_t es = size_of(dtype), ws = size_of(wdtype);
  if (any_off(es, dq, dk, q, k, q_grad, k_grad) || any_off(ws, q_weight, k_weight, q_dweight, k_dweight))
    return MUON_ERR_ALIGNMENT;
  const bool none = tokens == 0 || q_heads + k_heads == 0, sums = q_dweight || k_dweight;
  if (sums && !none) {
    size_t need = 0;
    muon_norm_rotate_heads_workspace_bytes(tokens, q_heads, k_heads, dim, &need);
    if (!workspace) return MUON_ERR_INVALID_ARG;
    if (off(workspace, 256)) return MUON_ERR_ALIGNMENT;
    if (ws_bytes < need) return MUON_ERR_WORKSPACE;
  }
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  NvtxRange range("muon_norm_rotate_heads_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (none) {     // empty sums
    for (void* d : {q_dweight, k_dweight})
      if (d && cudaMemsetAsync(d, 0, dim * ws, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  const Heads a = {tokens, table, period, dim, rotary, neighbours, eps, cos, sin, positions,
                   {{q, dq, q_weight, ldq, q_step, lddq, dq_step, q_grad, q_dweight, q_heads},
                    {k, dk, k_weight, ldk, k_step, lddk, dk_step, k_grad, k_dweight, k_heads}},
                   sums ? static_cast<float*>(workspace) : nullptr};
  const int parts = (int)head_parts(tokens, q_heads + k_heads);
  const cudaError_t e = by_both(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using WT = decltype(w);
    const size_t smem = (size_t)kHeadWarps * 3 * dim * sizeof(float);
    cudaError_t e = allow_shared<heads_bwd_kernel<T, WT>>(kHeadWarps * 3 * kHeadMaxDim * sizeof(float));
    if (e == cudaSuccess)
      e = launch_k(heads_bwd_kernel<T, WT>, dim3(parts), dim3(kHeadThreads), smem, s, true, a);
    if (e == cudaSuccess && sums)
      e = launch_k(heads_join_kernel<WT>, dim3((2 * dim + kHeadThreads - 1) / kHeadThreads),
                   dim3(kHeadThreads), 0, s, true, dim, parts, (const float*)a.part,
                   static_cast<WT*>(q_dweight), static_cast<WT*>(k_dweight));
    return e;
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
