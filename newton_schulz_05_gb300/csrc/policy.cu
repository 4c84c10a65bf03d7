// Clipped policy loss with a KL term over the log probabilities of tokens, and
// its gradient.
#include "sequence.cuh"

namespace muon {

namespace {

constexpr int kPolicyThreads = 256;
constexpr int kPolicyChunk = 4096;      // tokens of one sequence that a block takes

struct Policy {
  int64_t batch, length, ldl, ldo, lda, ldr;
  const float *lp, *old, *adv, *ref;
  const uint8_t* mask;
  float high, high_rest, low, low_rest;     // log(1 + clip_high) and log(1 - clip_low): value and rest
  float most, least;                        // 1 + clip_high, 1 - clip_low
  float kl_weight;
  int by_sequence;
};

// Whether the exact difference lp - old lies past a bound given as a value and its
// rest (to far below fp32's step): the rounded difference decides unless it equals the
// value, and then what the rounding left out does.
__device__ __forceinline__ float left_out(float lp, float old, float d) {
  const float b = lp - d, a = d + b;
  return (lp - a) - (old - b);
}

// exp(e) - e - 1 without the cancellation at small e: its Taylor series where 12
// terms are exact to fp32
__device__ __forceinline__ float excess(float e) {
  if (fabsf(e) > 1.f) return expf(e) - 1.f - e;
  float s = 1.f / 479001600.f;                 // 1 / 12!
  s = fmaf(s, e, 1.f / 39916800.f);
  s = fmaf(s, e, 1.f / 3628800.f);
  s = fmaf(s, e, 1.f / 362880.f);
  s = fmaf(s, e, 1.f / 40320.f);
  s = fmaf(s, e, 1.f / 5040.f);
  s = fmaf(s, e, 1.f / 720.f);
  s = fmaf(s, e, 1.f / 120.f);
  s = fmaf(s, e, 1.f / 24.f);
  s = fmaf(s, e, 1.f / 6.f);
  s = fmaf(s, e, 0.5f);
  return s * e * e;
}

struct Token { float lp, old, adv, d; bool cut; };
__device__ __forceinline__ Token token_of(const Policy& a, int64_t b, int64_t t) {
  Token k;
  k.lp = a.lp[b * a.ldl + t];
  k.old = a.old[b * a.ldo + t];
  k.adv = a.lda < 0 ? a.adv[b] : a.adv[b * a.lda + t];
  k.d = k.lp - k.old;
  if (k.adv >= 0.f) k.cut = k.d > a.high || (k.d == a.high && left_out(k.lp, k.old, k.d) > a.high_rest);
  else k.cut = k.d < a.low || (k.d == a.low && left_out(k.lp, k.old, k.d) < a.low_rest);
  return k;
}

// one block a chunk: sums of each, of k, of the cut tokens and of all
__global__ void __launch_bounds__(kPolicyThreads)
policy_kernel(const __grid_constant__ Policy a, int64_t chunks, float4* part) {
  __shared__ float red[kPolicyThreads / 32];
  pdl_wait();
  const int64_t b = blockIdx.x / chunks, t0 = blockIdx.x % chunks * kPolicyChunk;
  const int64_t t1 = t0 + kPolicyChunk < a.length ? t0 + kPolicyChunk : a.length;
  float each = 0.f, kl = 0.f, cut = 0.f, n = 0.f;
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kPolicyThreads) {
    if (a.mask && !a.mask[b * a.length + t]) continue;
    const Token k = token_of(a, b, t);
    const float r = k.cut ? (k.adv >= 0.f ? a.most : a.least) : expf(k.d);
    const float e = a.ref ? excess(a.ref[b * a.ldr + t] - k.lp) : 0.f;
    each += fmaf(-r, k.adv, a.kl_weight * e);
    kl += e;
    cut += k.cut ? 1.f : 0.f;
    n += 1.f;
  }
  each = block_sum<kPolicyThreads>(each, red);
  kl = block_sum<kPolicyThreads>(kl, red);
  cut = block_sum<kPolicyThreads>(cut, red);
  n = block_sum<kPolicyThreads>(n, red);
  if (threadIdx.x == 0) part[blockIdx.x] = make_float4(each, kl, cut, n);
}

constexpr int kPolicyJoin = 512;
// sum over the block of a 64-bit value, in every thread
__device__ double join_sum(double v, double* red) {
  __syncthreads();
  red[threadIdx.x] = v;
  __syncthreads();
  for (int o = kPolicyJoin / 2; o > 0; o >>= 1) {
    if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  return red[0];
}

// one block: the sequences' weights and the three means
__global__ void __launch_bounds__(kPolicyJoin)
policy_join_kernel(int64_t batch, int64_t chunks, int by_sequence, const float4* part, float* loss,
                   float* kl, float* clipped, float* weights) {
  __shared__ double red[kPolicyJoin];
  pdl_wait();
  double tokens = 0, filled = 0;
  for (int64_t b = threadIdx.x; b < batch; b += kPolicyJoin) {
    double n = 0;
    for (int64_t c = 0; c < chunks; ++c) n += part[b * chunks + c].w;
    tokens += n;
    filled += n > 0;
  }
  tokens = join_sum(tokens, red);
  filled = join_sum(filled, red);
  double s[3] = {0, 0, 0};
  for (int64_t b = threadIdx.x; b < batch; b += kPolicyJoin) {
    double n = 0, v[3] = {0, 0, 0};
    for (int64_t c = 0; c < chunks; ++c) {
      const float4 p = part[b * chunks + c];
      v[0] += p.x;
      v[1] += p.y;
      v[2] += p.z;
      n += p.w;
    }
    const double w = n > 0 ? 1.0 / (by_sequence ? n * filled : tokens) : 0.0;
    weights[b] = (float)w;
    for (int i = 0; i < 3; ++i) s[i] += w * v[i];
  }
  for (int i = 0; i < 3; ++i) s[i] = join_sum(s[i], red);
  if (threadIdx.x == 0) {
    *loss = (float)s[0];
    if (kl) *kl = (float)s[1];
    if (clipped) *clipped = (float)s[2];
  }
}

__global__ void __launch_bounds__(kPolicyThreads)
policy_bwd_kernel(const __grid_constant__ Policy a, int64_t chunks, const float* weights,
                  const float* dloss, float* dlp) {
  pdl_wait();
  const int64_t b = blockIdx.x / chunks, t0 = blockIdx.x % chunks * kPolicyChunk;
  const int64_t t1 = t0 + kPolicyChunk < a.length ? t0 + kPolicyChunk : a.length;
  const float w = weights[b] * (dloss ? *dloss : 1.f);
  for (int64_t t = t0 + threadIdx.x; t < t1; t += kPolicyThreads) {
    float g = 0.f;
    if (!a.mask || a.mask[b * a.length + t]) {
      const Token k = token_of(a, b, t);
      g = k.cut ? 0.f : -expf(k.d) * k.adv;
      if (a.ref) g = fmaf(-a.kl_weight, expm1f(a.ref[b * a.ldr + t] - k.lp), g);
      g *= w;
    }
    dlp[b * a.length + t] = g;
  }
}

// --------------------------------------------------------------------- host

int64_t policy_chunks(int64_t length) { return (length + kPolicyChunk - 1) / kPolicyChunk; }

muon_status check_policy(int64_t batch, int64_t length, double clip_low, double clip_high, float kl_weight,
                         int64_t ldl, int64_t ldo, int64_t ldr) {
  if (batch < 0 || length < 0 || !(clip_low >= 0 && clip_low < 1) || !(clip_high >= 0) ||
      std::isinf(clip_high) || !std::isfinite(kl_weight) || ldl < 0 || ldo < 0 || ldr < 0)
    return MUON_ERR_INVALID_ARG;
  if (batch >= (int64_t)1 << 31 || length >= (int64_t)1 << 31 ||
      (length > 0 && batch >= ((int64_t)1 << 40) / length) ||
      batch * policy_chunks(length) >= (int64_t)1 << 31)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  return MUON_OK;
}

Policy policy_of(int64_t batch, int64_t length, const float* lp, int64_t ldl, const float* old,
                 int64_t ldo, const float* adv, int64_t lda, const float* ref, int64_t ldr,
                 const uint8_t* mask, double clip_low, double clip_high, float kl_weight, int by_sequence) {
  const double high = std::log1p(clip_high), low = std::log1p(-clip_low);
  Policy a = {batch, length, ldl, ldo, lda, ldr, lp, old, adv, ref, mask, (float)high, 0.f, (float)low,
              0.f, (float)(1 + clip_high), (float)(1 - clip_low), kl_weight, by_sequence};
  a.high_rest = (float)(high - (double)a.high);
  a.low_rest = (float)(low - (double)a.low);
  return a;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_policy_loss_workspace_bytes(int64_t batch, int64_t length, size_t* out) {
  if (!out) return MUON_ERR_INVALID_ARG;
  const muon_status st = check_policy(batch, length, 0, 0, 0.f, 0, 0, 0);
  if (st != MUON_OK) return st;
  *out = (size_t)batch * policy_chunks(length) * sizeof(float4) + 256;
  return MUON_OK;
}

extern "C" muon_status muon_policy_loss(int64_t batch, int64_t length, const float* log_probs,
                                        int64_t ldl, const float* old, int64_t ldo,
                                        const float* advantages, int64_t lda, const float* ref,
                                        int64_t ldr, const uint8_t* token_mask, double clip_low,
                                        double clip_high, float kl_weight, int by_sequence,
                                        float* loss, float* kl, float* clipped, float* weights,
                                        void* workspace, size_t ws_bytes, void* stream) {
  const muon_status st = check_policy(batch, length, clip_low, clip_high, kl_weight, ldl, ldo, ldr);
  if (st != MUON_OK) return st;
  const bool any = batch > 0 && length > 0;
  if (!loss || !workspace || (batch > 0 && !weights) || (any && (!log_probs || !old || !advantages)))
    return MUON_ERR_INVALID_ARG;
  if (any_off(4, log_probs, old, advantages, ref, loss, kl, clipped, weights) || off(workspace, 256))
    return MUON_ERR_ALIGNMENT;
  size_t need = 0;
  muon_policy_loss_workspace_bytes(batch, length, &need);
  if (ws_bytes < need) return MUON_ERR_WORKSPACE;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  NvtxRange range("muon_policy_loss");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Policy a = policy_of(batch, length, log_probs, ldl, old, ldo, advantages, lda, ref, ldr, token_mask,
                             clip_low, clip_high, kl_weight, by_sequence);
  const int64_t chunks = policy_chunks(length);
  float4* part = static_cast<float4*>(workspace);
  cudaError_t e = cudaSuccess;
  if (any)
    e = launch_k(policy_kernel, dim3((unsigned)(batch * chunks)), dim3(kPolicyThreads), 0, s, true, a,
                 chunks, part);
  if (e == cudaSuccess)
    e = launch_k(policy_join_kernel, dim3(1), dim3(kPolicyJoin), 0, s, true, batch, chunks, by_sequence,
                 (const float4*)part, loss, kl, clipped, weights);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" muon_status muon_policy_loss_backward(
    int64_t batch, int64_t length, const float* log_probs, int64_t ldl, const float* old,
    int64_t ldo, const float* advantages, int64_t lda, const float* ref, int64_t ldr,
    const uint8_t* token_mask, double clip_low, double clip_high, float kl_weight,
    const float* weights, const float* dloss, float* dlog_probs, void* stream) {
  const muon_status st = check_policy(batch, length, clip_low, clip_high, kl_weight, ldl, ldo, ldr);
  if (st != MUON_OK) return st;
  const bool any = batch > 0 && length > 0;
  if (any && (!log_probs || !old || !advantages || !weights || !dlog_probs)) return MUON_ERR_INVALID_ARG;
  if (any_off(4, log_probs, old, advantages, ref, weights, dloss, dlog_probs)) return MUON_ERR_ALIGNMENT;
  if (batch > 1 && ((dlog_probs == log_probs && ldl != length) || (dlog_probs == old && ldo != length) ||
                    (dlog_probs == ref && ldr != length)))
    return MUON_ERR_INVALID_ARG;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (!any) return MUON_OK;
  NvtxRange range("muon_policy_loss_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Policy a = policy_of(batch, length, log_probs, ldl, old, ldo, advantages, lda, ref, ldr, token_mask,
                             clip_low, clip_high, kl_weight, 0);
  const int64_t chunks = policy_chunks(length);
  const cudaError_t e = launch_k(policy_bwd_kernel, dim3((unsigned)(batch * chunks)), dim3(kPolicyThreads),
                                 0, s, true, a, chunks, weights, dloss, dlog_probs);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
