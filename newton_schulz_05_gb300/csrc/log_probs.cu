// Log probabilities of given tokens under a softmax over the vocabulary, and
// their gradient.
#include <cfloat>

#include "sequence.cuh"

namespace muon {

namespace {

constexpr int kVocabThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

// A running maximum (not under the lowest finite number, so that a difference to it is
// not NaN for a -inf) and the sum of exp2((l - max) * c), joined with another.
struct Mass { float top, sum; };
__device__ __forceinline__ Mass join(Mass a, Mass b, float c) {
  const float top = fmaxf(a.top, b.top);
  return {top, a.sum * exp2f((a.top - top) * c) + b.sum * exp2f((b.top - top) * c)};
}

template <typename T>
__global__ void __launch_bounds__(kVocabThreads)
log_probs_kernel(int64_t vocab, const T* logits, int64_t ld, const int64_t* index, float scale,
                 float* log_probs, float* lse) {
  __shared__ Mass slots[kVocabThreads / 32];
  pdl_wait();
  const int64_t t = blockIdx.x, y = index[t];
  if (y < 0 || y >= vocab) {
    if (threadIdx.x == 0) log_probs[t] = lse[t] = 0.f;
    return;
  }
  const T* row = logits + t * ld;
  const float c = scale * kLog2e;
  Mass m = {-FLT_MAX, 0.f};
  for (int64_t v = threadIdx.x; v < vocab; v += kVocabThreads) {
    const float l = to_f(row[v]);
    if (l > m.top) {
      m.sum *= exp2f((m.top - l) * c);
      m.top = l;
    }
    m.sum += exp2f((l - m.top) * c);
  }
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    m = join(m, Mass{__shfl_xor_sync(~0u, m.top, o), __shfl_xor_sync(~0u, m.sum, o)}, c);
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kVocabThreads / 32; ++i) m = join(m, slots[i], c);
    const float rest = logf(m.sum);
    log_probs[t] = (to_f(row[y]) - m.top) * scale - rest;
    lse[t] = fmaf(m.top, scale, rest);
  }
}

template <typename T>
__global__ void __launch_bounds__(kVocabThreads)
log_probs_bwd_kernel(int64_t vocab, const float* dlp, const T* logits, int64_t ld,
                     const int64_t* index, const float* lse, float scale, T* dlogits) {
  pdl_wait();
  const int64_t t = blockIdx.x, y = index[t];
  const float d = y < 0 || y >= vocab ? 0.f : dlp[t] * scale;
  const float s = lse[t];
  for (int64_t v = threadIdx.x; v < vocab; v += kVocabThreads) {
    float g = 0.f;
    if (d != 0.f) g = d * ((v == y ? 1.f : 0.f) - expf(fmaf(to_f(logits[t * ld + v]), scale, -s)));
    dlogits[t * vocab + v] = from_f<T>(g);
  }
}

muon_status check_vocab(int64_t tokens, int64_t vocab, int dtype, int64_t ld, float scale) {
  if (tokens < 0 || ld < 0 || !(scale > 0.f) || std::isinf(scale)) return MUON_ERR_INVALID_ARG;
  if (vocab < 1 || vocab > (int64_t)1 << 30 || tokens >= (int64_t)1 << 31)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  return known(dtype) ? MUON_OK : MUON_ERR_DTYPE;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_token_log_probs(int64_t tokens, int64_t vocab, int dtype,
                                            const void* logits, int64_t ld, const int64_t* index,
                                            float scale, float* log_probs, float* lse,
                                            void* stream) {
  const muon_status st = check_vocab(tokens, vocab, dtype, ld, scale);
  if (st != MUON_OK) return st;
  if (tokens > 0 && (!logits || !index || !log_probs || !lse)) return MUON_ERR_INVALID_ARG;
  if (off(logits, size_of(dtype)) || off(index, 8) || any_off(4, log_probs, lse))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (tokens == 0) return MUON_OK;
  NvtxRange range("muon_token_log_probs");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return launch_k(log_probs_kernel<T>, dim3((unsigned)tokens), dim3(kVocabThreads), 0, s, true, vocab,
                    static_cast<const T*>(logits), ld, index, scale, log_probs, lse);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" muon_status muon_token_log_probs_backward(int64_t tokens, int64_t vocab, int dtype,
                                                     const float* dlog_probs, const void* logits,
                                                     int64_t ld, const int64_t* index,
                                                     const float* lse, float scale, void* dlogits,
                                                     void* stream) {
  const muon_status st = check_vocab(tokens, vocab, dtype, ld, scale);
  if (st != MUON_OK) return st;
  if (tokens > 0 && (!dlog_probs || !logits || !index || !lse || !dlogits)) return MUON_ERR_INVALID_ARG;
  if (any_off(size_of(dtype), logits, dlogits) || off(index, 8) || any_off(4, dlog_probs, lse))
    return MUON_ERR_ALIGNMENT;
  if (dlogits == logits && tokens > 1 && ld != vocab) return MUON_ERR_INVALID_ARG;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (tokens == 0) return MUON_OK;
  NvtxRange range("muon_token_log_probs_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = by_type(dtype, [&](auto t) {
    using T = decltype(t);
    return launch_k(log_probs_bwd_kernel<T>, dim3((unsigned)tokens), dim3(kVocabThreads), 0, s, true,
                    vocab, dlog_probs, static_cast<const T*>(logits), ld, index, lse, scale,
                    static_cast<T*>(dlogits));
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
