// Layer norm, alone or behind dropout and the residual add: the forward pass.
#include "norm.cuh"

namespace muon {

namespace {

struct NormFwd {
  int64_t rows, cols, ldx, ldr;
  const void *x, *residual, *weight, *bias;
  void *sum, *y;
  float *mean, *rstd;
  float eps;
  int wbf16;        // weight and bias are bf16
  int drop;
  int vec;          // every operand's rows share one phase
  int depth;        // of the ring
  Drop d;
};

// TPR threads a row (0: the block), C chunks a thread.  FUSED: residual and
// dropout may be present.
template <typename T, int TPR, int C, int NT, bool FUSED, bool REG>
__global__ void __launch_bounds__(NT, fwd_blocks(TPR, C, NT))
norm_fwd_kernel(const __grid_constant__ NormFwd a) {
  extern __shared__ uint4 ring[];
  __shared__ alignas(16) float slots[2][32];
  constexpr int OPS = FUSED ? 2 : 1, PER = C * kPieces<T>;
  const Place<TPR> at;
  const int nt = blockDim.x, warps = nt >> 5, cols = (int)a.cols;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  if constexpr (TPR == 0) {
    for (int i = threadIdx.x; i < 64; i += nt) (&slots[0][0])[i] = 0.f;
    __syncthreads();
  }
  const bool vec = REG || a.vec;
  const Visits go = visits(at, a.rows);
  const int phase =
      REG || !vec ? 0
                  : (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T) + (uint64_t)go.first * a.ldx) & 7);
  const int col = at.t * 8 - phase;             // chunk i begins at column col + i * span
  const int span = at.width * 8;
  // this thread's place in the next row to copy in, and in the current row
  const T *fx = x + go.first * a.ldx + col, *fr = res + go.first * a.ldr + col;
  const T *cx = fx, *cr = fr;
  int64_t out = go.first * a.cols + col;
  const int stage_len = OPS * PER * nt;
  uint4* const ring0 = ring + threadIdx.x;
  uint4* fill = ring0;
  int ahead = 0;
  auto start = [&] {
    if (vec && ahead < go.mine) {
      #pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c0 = col + i * span;
        fetch<T, REG>(fill + i * kPieces<T> * nt, nt, fx + i * span, x, c0, cols);
        if (FUSED && res)
          fetch<T, REG>(fill + (PER + i * kPieces<T>) * nt, nt, fr + i * span, res, c0, cols);
      }
    }
    copy_commit();
    ++ahead;
    fx += go.step * a.ldx;
    if constexpr (FUSED) fr += go.step * a.ldr;
    fill += stage_len;
    if (fill == ring0 + a.depth * stage_len) fill = ring0;
  };
  for (int s = 0; s + 1 < a.depth; ++s) start();
  Chunk w[C], b[C];
  #pragma unroll
  for (int i = 0; i < C; ++i) {
    columns(w[i], a.weight, a.wbf16, col + i * span, cols, 1.f);
    columns(b[i], a.bias, a.wbf16, col + i * span, cols, 0.f);
  }
  const float inv = 1.f / (float)cols;
  const uint4* from = ring0;
  int64_t row = go.first;
  for (int visit = 0; visit < go.all; ++visit) {
    start();                              // into the slot read in the last visit
    copy_wait(a.depth - 1);
    const bool live = TPR == 0 || visit < go.mine;
    Chunk v[C];
    float2 s2 = both(0.f);
    #pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c0 = col + i * span;
      if (live) {
        take<T, REG>(v[i], from + i * kPieces<T> * nt, nt, cx + i * span, x, c0, cols, vec);
        if constexpr (FUSED) {
          if (a.drop) drop8(v[i].v, out + i * span, a.d);
          if (res) {
            Chunk r;
            take<T, REG>(r, from + (PER + i * kPieces<T>) * nt, nt, cr + i * span, res, c0, cols, vec);
            #pragma unroll
            for (int j = 0; j < 4; ++j) v[i].v[j] = add2(v[i].v[j], r.v[j]);
          }
          if (a.sum) put<T, REG>(static_cast<T*>(a.sum) + out + i * span, c0, cols, v[i], vec);
        }
      } else {
        clear(v[i]);
      }
      #pragma unroll
      for (int j = 0; j < 4; ++j) s2 = add2(s2, v[i].v[j]);
    }
    const float mean = row_sum<TPR>(s2.x + s2.y, slots[0], warps) * inv;
    const float2 m2 = both(-mean);
    float2 q2 = both(0.f);
    #pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c0 = col + i * span;
      #pragma unroll
      for (int j = 0; j < 4; ++j) v[i].v[j] = add2(v[i].v[j], m2);
      if (whole<REG>(c0, cols)) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) q2 = fma2(v[i].v[j], v[i].v[j], q2);
      } else if (!REG) {
        #pragma unroll
        for (int j = 0; j < 8; ++j)
          if (inside(c0 + j, cols)) q2.x = fmaf(elem(v[i], j), elem(v[i], j), q2.x);
      }
    }
    const float rstd = rsqrtf(row_sum<TPR>(q2.x + q2.y, slots[1], warps) * inv + a.eps);
    if (live) {
      const float2 r2 = both(rstd);
      #pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c0 = col + i * span;
        #pragma unroll
        for (int j = 0; j < 4; ++j) v[i].v[j] = fma2(mul2(v[i].v[j], r2), w[i].v[j], b[i].v[j]);
        put<T, REG>(static_cast<T*>(a.y) + out + i * span, c0, cols, v[i], vec);
      }
      if (at.t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
    row += go.step;
    out += go.step * a.cols;
    if constexpr (!REG) {
      cx += go.step * a.ldx;
      cr += go.step * a.ldr;
    }
    from += stage_len;
    if (from == ring0 + a.depth * stage_len) from = ring0;
  }
}

// ------------------------------------------------- rows longer than a block

template <typename T, typename WT>
__global__ void __launch_bounds__(kNormThreads) norm_long_fwd_kernel(const __grid_constant__ NormFwd a) {
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

// --------------------------------------------------------------------- host

template <typename T, bool FUSED, bool REG>
cudaError_t forward(NormFwd a, int64_t chunks, cudaStream_t s) {
  const Shape sh = norm_shape(chunks, false);
  size_t smem;
  ring_of(sh, sizeof(T), FUSED ? 2 : 1, &a.depth, &smem);
  const int64_t grid = norm_grid(sh, a.rows);
  if (sh.tpr == 8)
    return launch_rows(norm_fwd_kernel<T, 8, 1, 256, FUSED, REG>, a, grid, sh.nt, smem, s);
  if (sh.tpr == 32 && sh.c == 1)
    return launch_rows(norm_fwd_kernel<T, 32, 1, 256, FUSED, REG>, a, grid, sh.nt, smem, s);
  if (sh.tpr == 32)
    return launch_rows(norm_fwd_kernel<T, 32, 2, 256, FUSED, REG>, a, grid, sh.nt, smem, s);
  if (sh.c == 1)
    return launch_rows(norm_fwd_kernel<T, 0, 1, 128, FUSED, REG>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 128)
    return launch_rows(norm_fwd_kernel<T, 0, 2, 128, FUSED, REG>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 256)
    return launch_rows(norm_fwd_kernel<T, 0, 2, 256, FUSED, REG>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 512)
    return launch_rows(norm_fwd_kernel<T, 0, 2, 512, FUSED, REG>, a, grid, sh.nt, smem, s);
  return launch_rows(norm_fwd_kernel<T, 0, 2, 1024, FUSED, REG>, a, grid, sh.nt, smem, s);
}

template <typename T>
cudaError_t forward(const NormFwd& a, const Phases& ph, bool fused, cudaStream_t s) {
  if (ph.regular())
    return fused ? forward<T, true, true>(a, ph.chunks(), s) : forward<T, false, true>(a, ph.chunks(), s);
  return fused ? forward<T, true, false>(a, ph.chunks(), s) : forward<T, false, false>(a, ph.chunks(), s);
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
  Phases ph{rows, cols, es};
  ph.add(x, ldx);
  ph.add(residual, ldr);
  ph.add(sum, cols);
  ph.add(y, cols);
  const bool fused = residual || sum || p > 0.f;
  const NormFwd a = {rows, cols, ldx, ldr, x, residual, weight, bias, sum, y, mean, rstd, eps,
                     wdtype == MUON_BF16, p > 0.f, ph.same, 1, make_drop(p, seed, offset)};
  cudaError_t e;
  if (ph.chunks() > kMaxChunks) {
    const int grid = (int)(rows < kSMs * 8 ? rows : kSMs * 8);
    e = by_types(dtype, wdtype, [&](auto t, auto wt) {
      norm_long_fwd_kernel<decltype(t), decltype(wt)><<<grid, kNormThreads, 0, s>>>(a);
      return cudaGetLastError();
    });
  } else {
    e = dtype == MUON_BF16 ? forward<__nv_bfloat16>(a, ph, fused, s) : forward<float>(a, ph, fused, s);
  }
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
