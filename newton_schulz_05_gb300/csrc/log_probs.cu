// Log probabilities of given tokens under a softmax over the vocabulary, and
// their gradient.
//
// Both passes are bound by HBM: the logits are read once, with a running maximum and a
// sum of exponentials to it a thread, and the gradient reads them once more and writes
// theirs.  A row is cut into 16-byte pieces that are aligned in memory, so a row that does
// not start at an aligned address has parts of pieces at its ends, taken element by
// element.  A thread has four pieces in flight; the maximum of all of them is taken first,
// in pairs of bf16, so that the sum is scaled once for 32 elements.
//
// Measured: [8192, 131072] bf16 294 us, 7.3 TB/s (reading alone is faster than a copy), the
// gradient of three rows in four 556 us, 6.8 TB/s; [4096, 50021] 66 us and 116 us; [20000, 2048]
// 15.5 and 25 us, 5.3 and 5.7 TB/s; one row of 262144 3.8 us in a cluster of eight blocks.
// Few rows are uneven: 509 of 50021 fp32, a quarter of them ignored, take 15.8 us where their
// bytes take 11.3, as the blocks of an SM end apart.
#include <cfloat>

#include "sequence.cuh"

namespace muon {

namespace {

constexpr int kVocabThreads = 256;
constexpr int kVocabPieces = 4;      // of a thread in flight
constexpr float kLog2e = 1.4426950408889634f;

// A row as pieces of E elements: piece i begins at column i * E - phase
template <typename T> __device__ __forceinline__ int phase_of(const T* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) & (kEl<T> - 1));
}

// A running maximum (not under the lowest finite number, so that a difference to it is
// not NaN for a -inf) and the sum of exp2((l - top) * c).  The difference is taken
// first: it is exact next to the maximum, where the terms count, and does not overflow
// to NaN where all logits are the type's lowest value.
struct Mass { float top, sum; };
__device__ __forceinline__ Mass join(const Mass& a, const Mass& b, float c) {
  const float top = fmaxf(a.top, b.top);
  return {top, a.sum * exp2_fast((a.top - top) * c) + b.sum * exp2_fast((b.top - top) * c)};
}
// the largest of a piece's elements (NaN counts as none)
__device__ __forceinline__ float largest(const uint4& u, __nv_bfloat16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&w[0]);
  #pragma unroll
  for (int j = 1; j < 4; ++j) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[j]));
  return fmaxf(__low2float(m), __high2float(m));
}
__device__ __forceinline__ float largest(const uint4& u, float) {
  return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
               fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
}
template <typename T, int N> __device__ __forceinline__ void take(Mass& m, const uint4 (&u)[N], float c) {
  constexpr int E = kEl<T>;
  float top = m.top;
  #pragma unroll
  for (int k = 0; k < N; ++k) top = fmaxf(top, largest(u[k], T()));
  float2 s = make_float2(m.sum * exp2_fast((m.top - top) * c), 0.f);
  #pragma unroll
  for (int k = 0; k < N; ++k) {
    Piece<E> v;
    widen(v, u[k]);
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float2 d = mul2(add2(v.v[j], both(-top)), both(c));
      s = add2(s, make_float2(exp2_fast(d.x), exp2_fast(d.y)));
    }
  }
  m = {top, s.x + s.y};
}
// A piece's elements, those inside the columns [0, vocab), the others -inf.  col: of its first
template <typename T>
__device__ __forceinline__ uint4 piece_at(const T* row, int64_t col, int64_t vocab) {
  constexpr int E = kEl<T>;
  if (col >= 0 && col + E <= vocab) return *reinterpret_cast<const uint4*>(row + col);
  Piece<E> v;
  #pragma unroll
  for (int j = 0; j < E; ++j)
    elem(v, j) = col + j >= 0 && col + j < vocab ? to_f(row[col + j]) : -INFINITY;
  return narrow(v);
}

// TPR threads a row, or CL blocks of TPR = kVocabThreads
template <typename T, int TPR, int CL>
__global__ void __launch_bounds__(kVocabThreads, 4)
log_probs_kernel(int64_t tokens, int64_t vocab, const T* logits, int64_t ld, const int64_t* index,
                 float scale, float* log_probs, float* lse) {
  constexpr int E = kEl<T>, N = kVocabPieces, kWarps = kVocabThreads / 32;
  __shared__ alignas(8) Mass slots[kWarps], blocks[CL];
  pdl_wait();
  const int64_t row = TPR < kVocabThreads ? (int64_t)blockIdx.x * (kVocabThreads / TPR) + threadIdx.x / TPR
                                          : blockIdx.x / CL;
  const int rank = CL > 1 ? (int)(blockIdx.x % CL) : 0, thread = threadIdx.x % TPR;
  const bool any = TPR == kVocabThreads || row < tokens;
  const int64_t y = any ? index[row] : -1;
  const T* l = logits + (any ? row * ld : 0);
  const int phase = phase_of(l);
  const float c = scale * kLog2e;
  // The blocks of a cluster take turns of N pieces a thread.  The first is read before it is
  // known whether the token counts.
  constexpr int64_t kTurn = (int64_t)TPR * N * E;
  int64_t col = rank * kTurn + thread * E - phase;
  uint4 u[N];
  auto fetch = [&] {
    #pragma unroll
    for (int k = 0; k < N; ++k) u[k] = piece_at(l, col + k * (TPR * E), vocab);
    col += kTurn * CL;
  };
  if (any) fetch();
  const bool live = y >= 0 && y < vocab;
  if (TPR == kVocabThreads && !live) {        // in every block of the row
    if (rank == 0 && thread == 0) log_probs[row] = lse[row] = 0.f;
    return;
  }
  Mass m = {-FLT_MAX, 0.f};
  if (live) {
    take<T>(m, u, c);
    while (col < vocab) {
      fetch();
      take<T>(m, u, c);
    }
  }
  #pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
    m = join(m, Mass{__shfl_xor_sync(~0u, m.top, o), __shfl_xor_sync(~0u, m.sum, o)}, c);
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = m;
    __syncthreads();
    m = slots[0];
    #pragma unroll
    for (int i = 1; i < kWarps; ++i) m = join(m, slots[i], c);
    if constexpr (CL > 1) {
      cluster_barrier();      // rank 0 has begun
      if (threadIdx.x == 0) {
        put_at(at_rank(&blocks[rank].top, 0), m.top);
        put_at(at_rank(&blocks[rank].sum, 0), m.sum);
      }
      __syncwarp();
      cluster_barrier();
      if (rank > 0) return;
      m = blocks[0];
      #pragma unroll
      for (int i = 1; i < CL; ++i) m = join(m, blocks[i], c);
    }
  }
  if (any && thread == 0) {
    const float rest = logf(m.sum);
    log_probs[row] = live ? (to_f(l[y]) - m.top) * scale - rest : 0.f;
    lse[row] = live ? fmaf(m.top, scale, rest) : 0.f;
  }
}

// The smaller one; NaN where either is
__device__ __forceinline__ float least(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// TPR threads take a unit of kVocabPieces pieces each of one row.  As in the forward pass the
// difference is taken before the base is changed, so that it does not overflow where logits
// and log sum are near the type's lowest value; a softmax is at most 1, whatever digits the log
// sum of a row far from zero has lost.
template <typename T, int TPR>
__global__ void __launch_bounds__(kVocabThreads)
log_probs_bwd_kernel(int64_t units, int units_a_row, int64_t vocab, const float* dlp, const T* logits, int64_t ld,
                     const int64_t* index, const float* lse, float scale, T* dlogits) {
  constexpr int E = kEl<T>, N = kVocabPieces;
  pdl_wait();
  const int64_t unit = (int64_t)blockIdx.x * (kVocabThreads / TPR) + threadIdx.x / TPR;
  if (TPR < kVocabThreads && unit >= units) return;
  const int64_t row = unit / units_a_row;
  const int64_t y = index[row];
  const float d = y < 0 || y >= vocab ? 0.f : dlp[row] * scale;
  const float less = -lse[row];
  const T* l = logits + row * ld;
  T* out = dlogits + row * vocab;
  const int phase = phase_of(out);
  const bool vec = phase == phase_of(l);
  const int64_t p0 = unit % units_a_row * (TPR * N) + threadIdx.x % TPR;
  uint4 u[N];
  bool whole[N];
  #pragma unroll
  for (int k = 0; k < N; ++k) {
    const int64_t p = p0 + k * TPR;
    whole[k] = vec && p * E >= phase && (p + 1) * E <= vocab + phase;
    u[k] = make_uint4(0, 0, 0, 0);
    if (whole[k] && d != 0.f) u[k] = *reinterpret_cast<const uint4*>(l + (p * E - phase));
  }
  #pragma unroll
  for (int k = 0; k < N; ++k) {
    const int64_t col = (p0 + k * TPR) * E - phase;
    if (col >= vocab) break;
    Piece<E> v;
    if (whole[k]) {
      widen(v, u[k]);
    } else {
      #pragma unroll
      for (int j = 0; j < E; ++j)
        elem(v, j) = d != 0.f && col + j >= 0 && col + j < vocab ? to_f(l[col + j]) : 0.f;
    }
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      float2 e = fma2(v.v[j], both(scale), both(less));
      e = mul2(make_float2(least(e.x, 0.f), least(e.y, 0.f)), both(kLog2e));
      v.v[j] = d != 0.f ? mul2(make_float2(exp2_fast(e.x), exp2_fast(e.y)), both(-d)) : both(0.f);
    }
    if (d != 0.f && y >= col && y < col + E) {
      #pragma unroll
      for (int j = 0; j < E; ++j)
        if (col + j == y) elem(v, j) += d;
    }
    if (whole[k]) {
      *reinterpret_cast<uint4*>(out + col) = narrow(v);
    } else {
      #pragma unroll
      for (int j = 0; j < E; ++j)
        if (col + j >= 0 && col + j < vocab) out[col + j] = from_f<T>(elem(v, j));
    }
  }
}

// --------------------------------------------------------------------- host

muon_status check_vocab(int64_t tokens, int64_t vocab, int dtype, int64_t ld, float scale) {
  // (beyond 2^127 the scale in base 2 is infinite, and every row NaN)
  if (tokens < 0 || ld < 0 || !(scale > 0.f) || scale > 0x1p127f) return MUON_ERR_INVALID_ARG;
  if (vocab < 1 || vocab > (int64_t)1 << 30 || tokens >= (int64_t)1 << 31 || tokens > ((int64_t)1 << 40) / vocab)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  return known(dtype) ? MUON_OK : MUON_ERR_DTYPE;
}

template <typename T, int TPR, int CL>
cudaError_t log_probs_with(int64_t tokens, int64_t vocab, const void* logits, int64_t ld, const int64_t* index,
                           float scale, float* log_probs, float* lse, cudaStream_t s) {
  constexpr int rows = kVocabThreads / TPR;
  return launch_cluster(log_probs_kernel<T, TPR, CL>, (tokens + rows - 1) / rows * CL, CL, kVocabThreads, 0, s, tokens,
                        vocab, static_cast<const T*>(logits), ld, index, scale, log_probs, lse);
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
    const int64_t turn = (int64_t)kVocabThreads * kVocabPieces * kEl<T>;      // elements of a block's turn
    // 8 lanes a row, or a warp (65536 rows of 256 bf16: 8.1 us, 46 with a warp); from there on a
    // block, or a cluster where blocks alone do not fill the SMs (300 rows of 50021: 9.4 us with
    // two blocks a row, 19.3 with eight)
    auto with = vocab * 32 <= turn ? log_probs_with<T, 8, 1>
                : vocab * 4 <= turn ? log_probs_with<T, 32, 1>
                : tokens > 304 || vocab <= turn ? log_probs_with<T, kVocabThreads, 1>
                : tokens > 152 || vocab <= 2 * turn ? log_probs_with<T, kVocabThreads, 2>
                : tokens > 76 || vocab <= 4 * turn ? log_probs_with<T, kVocabThreads, 4>
                                                   : log_probs_with<T, kVocabThreads, 8>;
    return with(tokens, vocab, logits, ld, index, scale, log_probs, lse, s);
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
    constexpr int E = kEl<T>;
    const int64_t lane = kVocabPieces * E;       // elements of a thread
    // 8 lanes a unit, or a warp, where a block would be wider than the row (65536 rows of 256
    // bf16: 16.7 us, 22.0 with a warp)
    const int tpr = vocab <= 8 * lane ? 8 : vocab <= 64 * lane ? 32 : kVocabThreads;
    const int groups = kVocabThreads / tpr;
    const int64_t ahead = vocab % E || off(dlogits, 16) ? E - 1 : 0;      // of a row in its first piece
    const int per_row = (int)((vocab + ahead + tpr * lane - 1) / (tpr * lane));
    const int64_t units = tokens * per_row;
    return launch_k(tpr == 8 ? log_probs_bwd_kernel<T, 8>
                    : tpr == 32 ? log_probs_bwd_kernel<T, 32> : log_probs_bwd_kernel<T, kVocabThreads>,
                    dim3((unsigned)((units + groups - 1) / groups)), dim3(kVocabThreads), 0, s, true, units,
                    per_row, vocab, dlog_probs, static_cast<const T*>(logits), ld, index, lse, scale,
                    static_cast<T*>(dlogits));
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
