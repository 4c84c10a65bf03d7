// Expert router: top-k choice, combine weights, per-expert counts and the
// balance loss of a token batch, and the gradient of weights and loss.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace muon {

namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteParts = 304;      // blocks of the forward pass, partial sums of each
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 32;
constexpr int kLane = kRouteMaxExperts / 32;

struct RouteArgs {
  int64_t tokens, ld;
  int experts, k, normalize;
  const void* logits;
  const uint8_t* mask;
  float* weights;
  int32_t* index;
  float* part_p;       // [parts][experts]
  int32_t* part_c;     // [parts][experts + 1]
};

// A key whose unsigned order is the order of the logits: NaN above +inf,
// -0 equal to +0.  0 is below the key of every value.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // order_key(-inf)

__device__ __forceinline__ float warp_sum(float v) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One warp a token; expert e belongs to lane e % 32.
template <typename T>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const __grid_constant__ RouteArgs a) {
  __shared__ float sp[kRouteMaxExperts];
  __shared__ int sc[kRouteMaxExperts + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e <= a.experts; e += kRouteThreads) {
    sc[e] = 0;
    if (e < a.experts) sp[e] = 0.f;
  }
  __syncthreads();
  float acc[kLane];
  #pragma unroll
  for (int j = 0; j < kLane; ++j) acc[j] = 0.f;
  const T* logits = static_cast<const T*>(a.logits);
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens;
       t += (int64_t)gridDim.x * kRouteWarps) {
    const bool masked = a.mask && !a.mask[t];
    float v[kLane];
    uint32_t key[kLane];
    #pragma unroll
    for (int j = 0; j < kLane; ++j) {
      const int e = j * 32 + lane;
      v[j] = e < a.experts ? to_f(logits[t * a.ld + e]) : -INFINITY;
      key[j] = e < a.experts ? order_key(v[j]) : 0u;
    }
    float top = 0.f, norm = 0.f, p_norm = 0.f;
    bool routed = !masked;
    float mine = 0.f;        // lane j holds pick j
    int mine_e = -1;
    for (int pick = 0; pick < a.k; ++pick) {
      uint32_t best = 0;
      int best_j = 0;
      #pragma unroll
      for (int j = 0; j < kLane; ++j)
        if (key[j] > best) { best = key[j]; best_j = j; }
      const uint32_t win = __reduce_max_sync(0xffffffffu, best);
      const uint32_t e = __reduce_min_sync(
          0xffffffffu, best == win ? (uint32_t)(best_j * 32 + lane) : 0xffffffffu);
      if (pick == 0) {
        routed = routed && win > kKeyNegInf;
        top = win > kKeyNegInf
            ? __uint_as_float(win == 0xffffffffu ? 0x7fc00000u
                              : win & 0x80000000u ? win & 0x7fffffffu : ~win)
            : 0.f;
        float s = 0.f;
        #pragma unroll
        for (int j = 0; j < kLane; ++j) {
          v[j] = routed ? expf(v[j] - top) : 0.f;
          s += v[j];
        }
        p_norm = warp_sum(s);
        #pragma unroll
        for (int j = 0; j < kLane; ++j)
          if (routed && j * 32 + lane < a.experts) acc[j] += v[j] / p_norm;
      }
      const bool ok = routed && win > kKeyNegInf;
      float x = 0.f;
      #pragma unroll
      for (int j = 0; j < kLane; ++j)
        if (j * 32 + lane == (int)e) {
          key[j] = 0;
          x = v[j];
        }
      x = __shfl_sync(0xffffffffu, x, (int)(e & 31));
      if (ok) norm += x;
      if (lane == pick) {
        mine = ok ? x : 0.f;
        mine_e = ok ? (int)e : -1;
      }
    }
    if (lane < a.k) {
      const float z = a.normalize ? norm : p_norm;
      a.weights[t * a.k + lane] = mine_e >= 0 ? mine / z : 0.f;
      a.index[t * a.k + lane] = mine_e;
      if (mine_e >= 0) atomicAdd(&sc[mine_e], 1);
    }
    if (lane == 0 && routed) atomicAdd(&sc[a.experts], 1);
  }
  // the block's sums, warp after warp
  for (int w = 0; w < kRouteWarps; ++w) {
    if (w == warp) {
      #pragma unroll
      for (int j = 0; j < kLane; ++j)
        if (j * 32 + lane < a.experts) sp[j * 32 + lane] += acc[j];
    }
    __syncthreads();
  }
  for (int e = threadIdx.x; e <= a.experts; e += kRouteThreads) {
    if (e < a.experts) a.part_p[(int64_t)blockIdx.x * a.experts + e] = sp[e];
    a.part_c[(int64_t)blockIdx.x * (a.experts + 1) + e] = sc[e];
  }
}

// counts, mean probabilities and the loss from the blocks' partial sums
__global__ void __launch_bounds__(kRouteThreads) route_join_kernel(
    int experts, int k, int parts, const float* part_p, const int32_t* part_c, int32_t* counts,
    float* mean_prob, float* loss) {
  __shared__ float red[kRouteWarps];
  __shared__ int routed;
  int c = 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < parts; ++i) c += part_c[(int64_t)i * (experts + 1) + experts];
    routed = c;
    counts[experts] = c;
  }
  __syncthreads();
  const float n = (float)(routed > 0 ? routed : 1);
  float l = 0.f;
  for (int e = threadIdx.x; e < experts; e += kRouteThreads) {
    int ce = 0;
    float p = 0.f;
    for (int i = 0; i < parts; ++i) {
      ce += part_c[(int64_t)i * (experts + 1) + e];
      p += part_p[(int64_t)i * experts + e];
    }
    p /= n;
    counts[e] = ce;
    mean_prob[e] = p;
    l = fmaf((float)ce / ((float)k * n), p, l);
  }
  l = block_sum<kRouteThreads>(l, red);
  if (threadIdx.x == 0) *loss = (float)experts * l;
}

struct RouteBwd {
  int64_t tokens, ld;
  int experts, k, normalize;
  const void* logits;
  const uint8_t* mask;
  const int32_t *index, *counts;
  const float *dweights, *dloss;
  void* dlogits;
};

template <typename T>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_kernel(
    const __grid_constant__ RouteBwd a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* logits = static_cast<const T*>(a.logits);
  const float n = (float)(a.counts[a.experts] > 0 ? a.counts[a.experts] : 1);
  const float c = a.dloss ? *a.dloss * (float)a.experts / ((float)a.k * n * n) : 0.f;
  for (int64_t t = (int64_t)blockIdx.x * kRouteWarps + warp; t < a.tokens;
       t += (int64_t)gridDim.x * kRouteWarps) {
    const bool masked = a.mask && !a.mask[t];
    float v[kLane], g[kLane];
    float top = -INFINITY;
    bool nan = false;
    #pragma unroll
    for (int j = 0; j < kLane; ++j) {
      const int e = j * 32 + lane;
      v[j] = e < a.experts ? to_f(logits[t * a.ld + e]) : -INFINITY;
      g[j] = e < a.experts ? c * (float)a.counts[e] : 0.f;
      top = fmaxf(top, v[j]);
      nan = nan || v[j] != v[j];
    }
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    nan = __any_sync(0xffffffffu, nan);
    const bool routed = !masked && (nan || top > -INFINITY);
    float s = 0.f;
    #pragma unroll
    for (int j = 0; j < kLane; ++j) {
      v[j] = routed ? expf(v[j] - top) : 0.f;
      s += v[j];
    }
    s = warp_sum(s);
    // picks: lane j holds pick j
    int e = -1;
    float dw = 0.f;
    if (lane < a.k) {
      e = a.index[t * a.k + lane];
      if (e < 0 || e >= a.experts) e = -1;
      if (e >= 0 && a.dweights) dw = a.dweights[t * a.k + lane];
    }
    float w = 0.f, add = dw;
    if (a.normalize) {
      if (e >= 0) w = expf(to_f(logits[t * a.ld + e]) - top);
      if (nan && e >= 0) w = NAN;
      const float z = warp_sum(w);
      w = z != 0.f ? w / z : 0.f;
      add = w * (dw - warp_sum(w * dw));
    } else {
      for (int i = 0; i < a.k; ++i) {
        const int ei = __shfl_sync(0xffffffffu, e, i);
        const float di = __shfl_sync(0xffffffffu, dw, i);
        #pragma unroll
        for (int j = 0; j < kLane; ++j)
          if (j * 32 + lane == ei) g[j] += di;
      }
    }
    float dot = 0.f;
    #pragma unroll
    for (int j = 0; j < kLane; ++j) {
      v[j] = routed ? v[j] / s : 0.f;
      dot = fmaf(v[j], g[j], dot);
    }
    dot = warp_sum(dot);
    #pragma unroll
    for (int j = 0; j < kLane; ++j) v[j] *= g[j] - dot;
    if (a.normalize) {
      for (int i = 0; i < a.k; ++i) {
        const int ei = __shfl_sync(0xffffffffu, e, i);
        const float di = __shfl_sync(0xffffffffu, add, i);
        #pragma unroll
        for (int j = 0; j < kLane; ++j)
          if (j * 32 + lane == ei) v[j] += di;
      }
    }
    #pragma unroll
    for (int j = 0; j < kLane; ++j) {
      const int o = j * 32 + lane;
      if (o < a.experts)
        static_cast<T*>(a.dlogits)[t * a.experts + o] = from_f<T>(routed ? v[j] : 0.f);
    }
  }
}

int route_blocks(int64_t tokens) {
  const int64_t b = (tokens + kRouteWarps - 1) / kRouteWarps;
  return (int)(b < kRouteParts ? b : kRouteParts);
}

bool misaligned(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

muon_status check_route(int64_t tokens, int experts, int k, int dtype, int64_t ld) {
  if (tokens < 0 || k < 1 || ld < 0) return MUON_ERR_INVALID_ARG;
  if (experts < 1 || experts > kRouteMaxExperts || k > kRouteMaxK || k > experts ||
      tokens > 0x7fffffff / k)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_DTYPE;
  return MUON_OK;
}

size_t counts_offset(int64_t tokens, int experts) {
  return ((size_t)route_blocks(tokens) * experts * sizeof(float) + 255) / 256 * 256;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_route_workspace_bytes(int64_t tokens, int experts, size_t* out) {
  if (!out || tokens < 0) return MUON_ERR_INVALID_ARG;
  if (experts < 1 || experts > kRouteMaxExperts) return MUON_ERR_UNSUPPORTED_SHAPE;
  *out = counts_offset(tokens, experts) +
         (size_t)route_blocks(tokens) * (experts + 1) * sizeof(int32_t) + 256;
  return MUON_OK;
}

extern "C" muon_status muon_route(int64_t tokens, int experts, int k, int dtype,
                                  const void* logits, int64_t ld, const uint8_t* token_mask,
                                  int normalize, float* weights, int32_t* index, int32_t* counts,
                                  float* mean_prob, float* loss, void* workspace, size_t ws_bytes,
                                  void* stream) {
  const muon_status st = check_route(tokens, experts, k, dtype, ld);
  if (st != MUON_OK) return st;
  if (!counts || !mean_prob || !loss || !workspace ||
      (tokens > 0 && (!logits || !weights || !index)))
    return MUON_ERR_INVALID_ARG;
  if (misaligned(logits, dtype == MUON_BF16 ? 2 : 4) || misaligned(weights, 4) ||
      misaligned(index, 4) || misaligned(counts, 4) || misaligned(mean_prob, 4) ||
      misaligned(loss, 4) || misaligned(workspace, 256))
    return MUON_ERR_ALIGNMENT;
  size_t need = 0;
  muon_route_workspace_bytes(tokens, experts, &need);
  if (ws_bytes < need) return MUON_ERR_WORKSPACE;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  NvtxRange range("muon_route");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int blocks = route_blocks(tokens);
  RouteArgs a = {tokens, ld, experts, k, normalize, logits, token_mask, weights, index,
                 static_cast<float*>(workspace),
                 reinterpret_cast<int32_t*>(static_cast<char*>(workspace) +
                                            counts_offset(tokens, experts))};
  if (blocks > 0) {
    if (dtype == MUON_BF16) route_kernel<__nv_bfloat16><<<blocks, kRouteThreads, 0, s>>>(a);
    else route_kernel<float><<<blocks, kRouteThreads, 0, s>>>(a);
  }
  route_join_kernel<<<1, kRouteThreads, 0, s>>>(experts, k, blocks, a.part_p, a.part_c, counts,
                                                mean_prob, loss);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" muon_status muon_route_backward(int64_t tokens, int experts, int k, int dtype,
                                           const void* logits, int64_t ld,
                                           const uint8_t* token_mask, int normalize,
                                           const int32_t* index, const int32_t* counts,
                                           const float* dweights, const float* dloss,
                                           void* dlogits, void* stream) {
  const muon_status st = check_route(tokens, experts, k, dtype, ld);
  if (st != MUON_OK) return st;
  if (tokens > 0 && (!logits || !index || !counts || !dlogits)) return MUON_ERR_INVALID_ARG;
  const size_t es = dtype == MUON_BF16 ? 2 : 4;
  if (misaligned(logits, es) || misaligned(dlogits, es) || misaligned(index, 4) ||
      misaligned(counts, 4) || misaligned(dweights, 4) || misaligned(dloss, 4))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (tokens == 0) return MUON_OK;
  NvtxRange range("muon_route_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RouteBwd a = {tokens, ld, experts, k, normalize, logits, token_mask, index, counts,
                      dweights, dloss, dlogits};
  const int64_t want = (tokens + kRouteWarps - 1) / kRouteWarps;
  const int blocks = (int)(want < 152 * 4 ? want : 152 * 4);
  if (dtype == MUON_BF16) route_bwd_kernel<__nv_bfloat16><<<blocks, kRouteThreads, 0, s>>>(a);
  else route_bwd_kernel<float><<<blocks, kRouteThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
