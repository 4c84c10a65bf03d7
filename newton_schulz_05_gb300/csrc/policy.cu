// Clipped policy loss with a KL term over the log probabilities of tokens, and
// its gradient.
//
// Both passes read 12 or 16 bytes a token and a mask byte once, the gradient writes 4; what
// they compute (two exponentials or a series of 11 terms) is near what the SMs have time for
// meanwhile.  The forward pass leaves the sums of parts of sequences, which a cluster of blocks
// joins into the means and the sequences' weights; few tokens are summed and joined by one
// cluster in one launch.
//
// Measured: gradient of [2048, 8192] with mask and reference 57 us, 6.1 TB/s, the loss itself 53
// us, of which the join takes about 5; [1024, 1000] 5.0 and 8.0 us, with one advantage a sequence
// 4.0 and 6.9; [64, 513] in one launch 6.7 us.
#include "sequence.cuh"

#include <cstddef>
#include <type_traits>

namespace muon {

namespace {

constexpr int kPolicyThreads = 256;

struct Policy {
  int64_t batch, length, ldl, ldo, lda, ldr;
  const float *lp, *old, *adv, *ref;
  const uint8_t* mask;
  float high, high_rest, low, low_rest;     // log(1 + clip_high) and log(1 - clip_low): value and rest
  float most, least;                        // 1 + clip_high, 1 - clip_low
  float kl_weight;
  int by_sequence;
  bool vec;                                 // fours of tokens lie alike in all operands
};

// Whether the exact difference lp - old lies past a bound given as a value and its
// rest (to far below fp32's step): the rounded difference decides unless it equals the
// value, and then what the rounding left out does.
__device__ __forceinline__ float left_out(float lp, float old, float d) {
  const float b = lp - d, a = d + b;
  return (lp - a) - (old - b);
}

// exp(e) - e - 1 for |e| <= 1, without the cancellation at small e: its Taylor series, of
// which 12 terms are exact to fp32
__device__ __forceinline__ float near_excess(float e) {
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
// exp(e) - e - 1, and exp(e) - 1: not as the former plus e, which has no digits left for the
// 1 where e is below -2^24 (references that forbid a token), and is NaN for -inf
__device__ __forceinline__ float excess(float e) { return fabsf(e) > 1.f ? expf(e) - 1.f - e : near_excess(e); }
__device__ __forceinline__ float change(float e) { return fabsf(e) > 1.f ? expf(e) - 1.f : near_excess(e) + e; }

// The loss of one token and its slope in log_probs.  cut: the minimum is the clipped side.
struct Token { float each, kl, slope; bool cut; };
template <bool GRAD>
__device__ __forceinline__ Token token_of(const Policy& a, float lp, float old, float adv, float ref) {
  Token k;
  const float d = lp - old;
  const bool up = adv >= 0.f;
  const float bound = up ? a.high : a.low, rest = up ? a.high_rest : a.low_rest;
  k.cut = up ? d > bound : d < bound;
  if (d == bound) {
    const float out = left_out(lp, old, d);
    k.cut = up ? out > rest : out < rest;
  }
  const float r = expf(d);
  if (GRAD) {
    k.slope = k.cut ? 0.f : -r * adv;
    if (a.ref && a.kl_weight != 0.f) k.slope = fmaf(-a.kl_weight, change(ref - lp), k.slope);
  } else {
    k.kl = a.ref ? excess(ref - lp) : 0.f;
    // without a weight not even an infinite k counts
    k.each = fmaf(k.cut ? (up ? -a.most : -a.least) : -r, adv, a.kl_weight != 0.f ? a.kl_weight * k.kl : 0.f);
  }
  return k;
}

// Tokens go four at a time (16 bytes of each operand, 4 mask bytes), aligned in memory: a
// sequence that does not start at an aligned address has parts of fours at its ends.
// TPR threads take a unit of kPolicyFours fours each, a part of one sequence.
constexpr int kPolicyFours = 2;
template <int TPR> constexpr int kUnit = TPR * kPolicyFours * 4;

struct Four { float lp[4], old[4], adv[4], ref[4]; uint32_t live; };     // live: a byte a token

__device__ __forceinline__ void get(float (&to)[4], const float* p) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  to[0] = f.x;
  to[1] = f.y;
  to[2] = f.z;
  to[3] = f.w;
}
// tokens t .. t + 3 of sequence b, those inside it
__device__ __forceinline__ void get(Four& f, const Policy& a, int64_t b, int64_t t, float adv) {
  f.live = 0;
  if (t >= a.length) return;
  if (a.vec && t >= 0 && t + 4 <= a.length) {
    get(f.lp, a.lp + b * a.ldl + t);
    get(f.old, a.old + b * a.ldo + t);
    if (a.lda >= 0) get(f.adv, a.adv + b * a.lda + t);
    if (a.ref) get(f.ref, a.ref + b * a.ldr + t);
    f.live = a.mask ? *reinterpret_cast<const uint32_t*>(a.mask + b * a.length + t) : ~0u;
  } else {
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = t + j;
      if (i < 0 || i >= a.length || (a.mask && !a.mask[b * a.length + i])) continue;
      f.live |= 0xffu << 8 * j;
      f.lp[j] = a.lp[b * a.ldl + i];
      f.old[j] = a.old[b * a.ldo + i];
      if (a.lda >= 0) f.adv[j] = a.adv[b * a.lda + i];
      if (a.ref) f.ref[j] = a.ref[b * a.ldr + i];
    }
  }
  if (a.lda < 0) {
    #pragma unroll
    for (int j = 0; j < 4; ++j) f.adv[j] = adv;
  }
}
// the first token of a thread's first four in a unit, and where its sequence begins in it
template <int TPR> __device__ __forceinline__ int64_t first_of(const Policy& a, int64_t b, int64_t chunk) {
  const int64_t phase = a.vec ? b * a.length & 3 : 0;
  return chunk * kUnit<TPR> + 4 * (threadIdx.x % TPR) - phase;
}

// A sum and what its roundings have left out (Knuth's two-sum), for sums over many parts of
// either sign in a row.  Sums in 64 bits took most of a small call (12.2 us of [64, 513]) on
// this GPU's few units for them.
struct Sum { float hi, lo; };
__device__ __forceinline__ void add(Sum& s, float x) {
  const float t = s.hi + x, b = t - s.hi;
  s.lo += (s.hi - (t - b)) + (x - b);
  s.hi = t;
}

// (what is left out of an infinite sum is NaN)
__device__ __forceinline__ float value(const Sum& s) { return isfinite(s.hi) ? s.hi + s.lo : s.hi; }

// What a thread, a warp and in the end all know of the sequences: tokens, sequences that have
// one, and the sums of each, of k and of clipped tokens (by_sequence: of their means)
struct alignas(16) Total {
  unsigned long long tokens;
  float sum[3];
  unsigned filled;
};
__device__ __forceinline__ void add(Total& v, const Total& x) {
  v.tokens += x.tokens;
  v.filled += x.filled;
  #pragma unroll
  for (int i = 0; i < 3; ++i) v.sum[i] += x.sum[i];
}
__device__ __forceinline__ void add_lanes(Total& v) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Total x;
    x.tokens = __shfl_xor_sync(~0u, v.tokens, o);
    x.filled = __shfl_xor_sync(~0u, v.filled, o);
    #pragma unroll
    for (int i = 0; i < 3; ++i) x.sum[i] = __shfl_xor_sync(~0u, v.sum[i], o);
    add(v, x);
  }
}
// Over kPolicyJoin threads of each of CL blocks, in every thread; all: a slot a rank and warp
constexpr int kPolicyJoin = 256;
template <int CL> __device__ __forceinline__ void add_all(Total& v, Total (*all)[kPolicyJoin / 32]) {
  constexpr int W = kPolicyJoin / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = CL > 1 ? cluster_rank() : 0;
  add_lanes(v);
  if constexpr (CL == 1) {
    if (lane == 0) all[0][warp] = v;
  } else if (lane < CL) {      // lane r tells block r
    const uint32_t to = at_rank(&all[rank][warp], lane);
    const float2 n = *reinterpret_cast<const float2*>(&v.tokens);
    put_at(to, make_float4(n.x, n.y, v.sum[0], v.sum[1]));
    put_at(to + 16, v.sum[2]);
    put_at(to + 20, (int)v.filled);
  }
  __syncwarp();
  if constexpr (CL > 1) cluster_barrier();
  else asm volatile("barrier.sync 1, %0;\n" ::"n"(kPolicyJoin) : "memory");
  static_assert(CL * W <= 64 && sizeof(Total) == 32 && offsetof(Total, filled) == 20, "slots");
  v = Total{};
  #pragma unroll
  for (int i = lane; i < CL * W; i += 32) add(v, all[i / W][i % W]);
  add_lanes(v);
}

struct PolicyOut { float *loss, *kl, *clipped, *weights; };

// CL blocks: the sequences' weights and the three means from their units, each of which has
// its sums of each and of k, its clipped tokens and all of them.
template <int CL>
__device__ __forceinline__ void join_units(const float4* __restrict__ part, int64_t batch, int64_t chunks,
                                           int by_sequence, const PolicyOut& out) {
  __shared__ Total all[CL][kPolicyJoin / 32];
  const int rank = CL > 1 ? cluster_rank() : 0;
  const int64_t first = (int64_t)rank * kPolicyJoin + threadIdx.x, step = (int64_t)CL * kPolicyJoin;
  Total t = {};
  Sum s[3] = {};
  unsigned kept = 0;        // the first sequence's tokens, all that most threads have
  #pragma unroll 4
  for (int64_t b = first; b < batch; b += step) {
    Sum v[3] = {};
    unsigned n = 0;
    for (int64_t c = 0; c < chunks; ++c) {
      const float4 p = part[b * chunks + c];
      add(v[0], p.x);
      add(v[1], p.y);
      add(v[2], p.z);
      n += (unsigned)p.w;
    }
    if (b == first) kept = n;
    t.tokens += n;
    t.filled += n > 0;
    const float w = by_sequence ? 1.f / (float)(n ? n : 1) : 1.f;
    #pragma unroll
    for (int i = 0; i < 3; ++i) add(s[i], w * value(v[i]));
  }
  #pragma unroll
  for (int i = 0; i < 3; ++i) t.sum[i] = value(s[i]);
  add_all<CL>(t, all);
  const unsigned long long over = by_sequence ? t.filled : t.tokens;
  const float share = 1.f / (float)(over ? over : 1);
  #pragma unroll 4
  for (int64_t b = first; b < batch; b += step) {
    unsigned n = kept;
    if (b != first) {
      n = 0;
      for (int64_t c = 0; c < chunks; ++c) n += (unsigned)part[b * chunks + c].w;
    }
    out.weights[b] = n == 0 ? 0.f : by_sequence ? 1.f / ((float)n * (float)over) : share;
  }
  if (rank == 0 && threadIdx.x < 3) {
    float* const to = threadIdx.x == 0 ? out.loss : threadIdx.x == 1 ? out.kl : out.clipped;
    const float v = threadIdx.x == 0 ? t.sum[0] : threadIdx.x == 1 ? t.sum[1] : t.sum[2];
    if (to) *to = v / (float)(over ? over : 1);
  }
}

constexpr int kFusedBlocks = 8, kFusedThreads = 512, kFusedUnits = 256;

// FUSED: one cluster takes all units and joins them in its first block's shared memory
template <int TPR, bool FUSED, int NT>
__global__ void __launch_bounds__(NT)
policy_kernel(const __grid_constant__ Policy a, int64_t units, int64_t chunks, float4* part,
              const __grid_constant__ PolicyOut out) {
  __shared__ alignas(16) float4 slots[FUSED ? kFusedUnits : 1];
  __shared__ float4 red[NT / 32];
  constexpr int groups = NT / TPR;
  static_assert(TPR <= 32 || TPR == NT, "a unit's threads are lanes of a warp, or the block");
  pdl_wait();
  if (FUSED) cluster_barrier();      // the first block has begun
  // the block's groups go on together: shuffles and barriers in each turn
  for (int64_t unit0 = (int64_t)blockIdx.x * groups; unit0 < units; unit0 += (int64_t)gridDim.x * groups) {
    const int64_t unit = unit0 + threadIdx.x / TPR;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (unit < units) {
      const int64_t b = unit / chunks, t0 = first_of<TPR>(a, b, unit % chunks);
      const float adv = a.lda < 0 ? a.adv[b] : 0.f;
      Four f[kPolicyFours];
      #pragma unroll
      for (int k = 0; k < kPolicyFours; ++k) get(f[k], a, b, t0 + k * 4 * TPR, adv);
      #pragma unroll
      for (int k = 0; k < kPolicyFours; ++k)
        #pragma unroll
        for (int j = 0; j < 4; ++j)
          if (f[k].live >> 8 * j & 0xff) {
            const Token v = token_of<false>(a, f[k].lp[j], f[k].old[j], f[k].adv[j], f[k].ref[j]);
            s.x += v.each;
            s.y += v.kl;
            s.z += v.cut ? 1.f : 0.f;
            s.w += 1.f;
          }
    }
    #pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
      s.x += __shfl_xor_sync(~0u, s.x, o);
      s.y += __shfl_xor_sync(~0u, s.y, o);
      s.z += __shfl_xor_sync(~0u, s.z, o);
      s.w += __shfl_xor_sync(~0u, s.w, o);
    }
    if constexpr (TPR > 32) {
      __syncthreads();
      if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
      __syncthreads();
      s = red[0];
      #pragma unroll
      for (int i = 1; i < NT / 32; ++i) {
        s.x += red[i].x;
        s.y += red[i].y;
        s.z += red[i].z;
        s.w += red[i].w;
      }
    }
    if (threadIdx.x % TPR == 0 && unit < units) {
      if constexpr (FUSED) put_at(at_rank(&slots[unit], 0), s);
      else part[unit] = s;
    }
  }
  if constexpr (FUSED) {
    __syncthreads();
    cluster_barrier();
    if (blockIdx.x == 0 && threadIdx.x < kPolicyJoin) join_units<1>(slots, a.batch, chunks, a.by_sequence, out);
  }
}

__global__ void __launch_bounds__(kPolicyJoin)
policy_join_kernel(int64_t batch, int64_t chunks, int by_sequence, const float4* part,
                   const __grid_constant__ PolicyOut out) {
  pdl_wait();
  cluster_barrier();      // every block has begun
  join_units<kFusedBlocks>(part, batch, chunks, by_sequence, out);
}

template <int TPR>
__global__ void __launch_bounds__(kPolicyThreads)
policy_bwd_kernel(const __grid_constant__ Policy a, int64_t units, int64_t chunks, const float* weights,
                  const float* dloss, float* dlp) {
  pdl_wait();
  const int64_t unit = (int64_t)blockIdx.x * (kPolicyThreads / TPR) + threadIdx.x / TPR;
  if (unit >= units) return;
  const int64_t b = unit / chunks, t0 = first_of<TPR>(a, b, unit % chunks);
  const float adv = a.lda < 0 ? a.adv[b] : 0.f, w = weights[b] * (dloss ? *dloss : 1.f);
  Four f[kPolicyFours];
  #pragma unroll
  for (int k = 0; k < kPolicyFours; ++k) get(f[k], a, b, t0 + k * 4 * TPR, adv);
  #pragma unroll
  for (int k = 0; k < kPolicyFours; ++k) {
    const int64_t t = t0 + k * 4 * TPR;
    float g[4];
    #pragma unroll
    for (int j = 0; j < 4; ++j)
      g[j] = f[k].live >> 8 * j & 0xff
                 ? w * token_of<true>(a, f[k].lp[j], f[k].old[j], f[k].adv[j], f[k].ref[j]).slope : 0.f;
    float* out = dlp + b * a.length + t;
    if (a.vec && t >= 0 && t + 4 <= a.length) {
      *reinterpret_cast<float4*>(out) = make_float4(g[0], g[1], g[2], g[3]);
    } else {
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t + j >= 0 && t + j < a.length) out[j] = g[j];
    }
  }
}

// --------------------------------------------------------------------- host

// threads a unit, and units of a sequence (three tokens may lie ahead of its first four)
int policy_threads(int64_t length) { return length <= kUnit<8> ? 8 : length <= 4 * kUnit<32> ? 32 : 256; }
int64_t policy_chunks(int64_t length, int threads) {
  const int64_t unit = (int64_t)threads * kPolicyFours * 4;
  return (length + (length % 4 ? 3 : 0) + unit - 1) / unit;
}
int64_t policy_chunks(int64_t length) { return policy_chunks(length, policy_threads(length)); }
// f(threads a unit)
template <typename F> auto by_threads(int64_t length, F f) {
  const int n = policy_threads(length);
  if (n == 8) return f(std::integral_constant<int, 8>());
  if (n == 32) return f(std::integral_constant<int, 32>());
  return f(std::integral_constant<int, 256>());
}
// Whether fours of tokens lie alike in all operands, sequence by sequence: aligned first
// rows, and strides that are that of the dense rows but for whole fours
bool in_fours(const Policy& a, const float* out) {
  auto like = [&](const float* p, int64_t ld) {
    return !p || (!off(p, 16) && (a.batch <= 1 || (ld - a.length) % 4 == 0));
  };
  return like(a.lp, a.ldl) && like(a.old, a.ldo) && (a.lda < 0 || like(a.adv, a.lda)) && like(a.ref, a.ldr) &&
         like(out, a.length) && !off(a.mask, 4);
}

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
              0.f, (float)(1 + clip_high), (float)(1 - clip_low), kl_weight, by_sequence, false};
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
  Policy a = policy_of(batch, length, log_probs, ldl, old, ldo, advantages, lda, ref, ldr, token_mask,
                       clip_low, clip_high, kl_weight, by_sequence);
  a.vec = in_fours(a, nullptr);
  const int64_t chunks = policy_chunks(length), units = batch * chunks;
  float4* part = static_cast<float4*>(workspace);
  const PolicyOut out = {loss, kl, clipped, weights};
  cudaError_t e = cudaSuccess;
  // One launch saves the host's time for the other, about 2 us of a call that the host bounds up
  // to some 60 Ki tokens; beyond, eight blocks take longer ([256, 512] 11.2 us, 5.5 in two).
  const int64_t few = policy_chunks(length, 32);
  if (any && batch * few <= kFusedUnits) {
    e = launch_cluster(policy_kernel<32, true, kFusedThreads>, kFusedBlocks, kFusedBlocks, kFusedThreads, 0, s, a,
                       batch * few, few, part, out);
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  }
  if (units > 0)
    e = by_threads(length, [&](auto n) {
      constexpr int TPR = decltype(n)::value, groups = kPolicyThreads / TPR;
      return launch_k(policy_kernel<TPR, false, kPolicyThreads>, dim3((unsigned)((units + groups - 1) / groups)),
                      dim3(kPolicyThreads), 0, s, true, a, units, chunks, part, out);
    });
  if (e == cudaSuccess)
    e = launch_cluster(policy_join_kernel, kFusedBlocks, kFusedBlocks, kPolicyJoin, 0, s, batch, chunks,
                       by_sequence, (const float4*)part, out);
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
  Policy a = policy_of(batch, length, log_probs, ldl, old, ldo, advantages, lda, ref, ldr, token_mask,
                       clip_low, clip_high, kl_weight, 0);
  a.vec = in_fours(a, dlog_probs);
  const int64_t chunks = policy_chunks(length), units = batch * chunks;
  const cudaError_t e = by_threads(length, [&](auto n) {
    constexpr int TPR = decltype(n)::value, groups = kPolicyThreads / TPR;
    return launch_k(policy_bwd_kernel<TPR>, dim3((unsigned)((units + groups - 1) / groups)), dim3(kPolicyThreads),
                    0, s, true, a, units, chunks, weights, dloss, dlog_probs);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
