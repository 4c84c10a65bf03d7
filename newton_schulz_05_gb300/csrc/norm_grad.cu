// Layer norm, alone or behind dropout and the residual add: the gradient.
#include "norm.cuh"

namespace muon {

namespace {

struct NormBwd {
  int64_t rows, cols, lddy, lds, ldds;
  const void *dy, *sum, *dsum, *weight;
  const float *mean, *rstd;
  void *dx, *dresidual;
  float* part;      // [parts][2][cols], or null
  int wbf16;
  int drop;
  int vec;
  int depth;
  Drop d;
};

// KEEP: the row's values stay in registers between the reduction and the
// output; otherwise (blocks of 1024 threads, 64 registers each) they are read
// from the ring twice, and the weight from memory.
template <typename T, int TPR, int C, int NT, bool FUSED, bool KEEP, bool REG>
__global__ void __launch_bounds__(NT, bwd_blocks(NT))
norm_bwd_kernel(const __grid_constant__ NormBwd a) {
  extern __shared__ uint4 ring[];
  __shared__ alignas(16) float slots[2][2][32];
  constexpr int OPS = FUSED ? 3 : 2, PER = C * kPieces<T>;
  const Place<TPR> at;
  const int nt = blockDim.x, warps = nt >> 5, cols = (int)a.cols;
  const T* dy = static_cast<const T*>(a.dy);
  const T* sum = static_cast<const T*>(a.sum);
  const T* ds = static_cast<const T*>(a.dsum);
  if constexpr (TPR == 0) {
    for (int i = threadIdx.x; i < 128; i += nt) (&slots[0][0][0])[i] = 0.f;
    __syncthreads();
  }
  const bool vec = REG || a.vec;
  const Visits go = visits(at, a.rows);
  const int phase =
      REG || !vec ? 0
                  : (int)((reinterpret_cast<uintptr_t>(dy) / sizeof(T) + (uint64_t)go.first * a.lddy) & 7);
  const int col = at.t * 8 - phase;             // chunk i begins at column col + i * span
  const int span = at.width * 8;
  // this thread's place in the next row to copy in, and in the current row
  const T *fy = dy + go.first * a.lddy + col, *fs = sum + go.first * a.lds + col,
          *fd = ds + go.first * a.ldds + col;
  const T *cy = fy, *cs = fs, *cd = fd;
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
        fetch<T, REG>(fill + i * kPieces<T> * nt, nt, fy + i * span, dy, c0, cols);
        fetch<T, REG>(fill + (PER + i * kPieces<T>) * nt, nt, fs + i * span, sum, c0, cols);
        if (FUSED && ds)
          fetch<T, REG>(fill + (2 * PER + i * kPieces<T>) * nt, nt, fd + i * span, ds, c0, cols);
      }
    }
    copy_commit();
    ++ahead;
    fy += go.step * a.lddy;
    fs += go.step * a.lds;
    if constexpr (FUSED) fd += go.step * a.ldds;
    fill += stage_len;
    if (fill == ring0 + a.depth * stage_len) fill = ring0;
  };
  for (int s = 0; s + 1 < a.depth; ++s) start();
  Chunk w[KEEP ? C : 1], accw[C], accb[C];
  #pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (KEEP) columns(w[i], a.weight, a.wbf16, col + i * span, cols, 1.f);
    clear(accw[i]);
    clear(accb[i]);
  }
  const float inv = 1.f / (float)cols;
  const float *pm = a.mean + go.first, *pr = a.rstd + go.first;
  float mean_next = 0.f, rstd_next = 0.f;
  if (go.mine > 0) { mean_next = *pm; rstd_next = *pr; }
  const uint4* from = ring0;
  int turn = 0;
  for (int visit = 0; visit < go.all; ++visit) {
    start();                              // into the slot read in the last visit
    const bool live = TPR == 0 || visit < go.mine;
    const float2 mean = both(-mean_next), rstd = both(rstd_next);
    pm += go.step;
    pr += go.step;
    if (visit + 1 < go.mine) { mean_next = *pm; rstd_next = *pr; }
    copy_wait(a.depth - 1);
    // dy and h = (sum - mean) * rstd of chunk i
    auto value = [&](int i, Chunk& y, Chunk& h) {
      const int c0 = col + i * span;
      take<T, REG>(y, from + i * kPieces<T> * nt, nt, cy + i * span, dy, c0, cols, vec);
      take<T, REG>(h, from + (PER + i * kPieces<T>) * nt, nt, cs + i * span, sum, c0, cols, vec);
      #pragma unroll
      for (int j = 0; j < 4; ++j) h.v[j] = mul2(add2(h.v[j], mean), rstd);
      if (!REG && !whole<REG>(c0, cols)) {     // dy is 0 there, but h may be infinite
        #pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!inside(c0 + j, cols)) elem(h, j) = 0.f;
      }
    };
    Chunk g[KEEP ? C : 1], h[KEEP ? C : 1];
    float2 sg2 = both(0.f), sh2 = both(0.f);
    #pragma unroll
    for (int i = 0; i < C; ++i) {
      Chunk& gi = g[KEEP ? i : 0];
      Chunk& hi = h[KEEP ? i : 0];
      Chunk& wi = w[KEEP ? i : 0];
      if (live && (!REG || col + i * span < cols)) {
        value(i, gi, hi);
      } else {
        clear(gi);
        clear(hi);
      }
      if constexpr (!KEEP) columns(wi, a.weight, a.wbf16, col + i * span, cols, 1.f);
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        accw[i].v[j] = fma2(gi.v[j], hi.v[j], accw[i].v[j]);
        accb[i].v[j] = add2(gi.v[j], accb[i].v[j]);
        gi.v[j] = mul2(gi.v[j], wi.v[j]);
        sg2 = add2(sg2, gi.v[j]);
        sh2 = fma2(gi.v[j], hi.v[j], sh2);
      }
    }
    // the two sums share a barrier; a slot pair is rewritten two rows later,
    // after the barrier of the row between
    float sg = sg2.x + sg2.y, sh = sh2.x + sh2.y;
    float* s2 = slots[turn][0];
    turn ^= 1;
    #pragma unroll
    for (int o = (TPR == 0 ? 32 : TPR) / 2; o > 0; o >>= 1) {
      sg += __shfl_xor_sync(0xffffffffu, sg, o);
      sh += __shfl_xor_sync(0xffffffffu, sh, o);
    }
    if constexpr (TPR == 0) {
      if ((threadIdx.x & 31) == 0) {
        s2[threadIdx.x >> 5] = sg;
        s2[32 + (threadIdx.x >> 5)] = sh;
      }
      __syncthreads();
      sg = sh = 0.f;
      for (int i = 0; i < warps; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(s2 + i);
        const float4 e = *reinterpret_cast<const float4*>(s2 + 32 + i);
        sg += (f.x + f.y) + (f.z + f.w);
        sh += (e.x + e.y) + (e.z + e.w);
      }
    }
    const float2 mg = both(-sg * inv), mh = both(-sh * inv);
    if (live) {
      #pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c0 = col + i * span;
        Chunk d;
        Chunk& gi = g[KEEP ? i : 0];
        Chunk& hi = h[KEEP ? i : 0];
        if constexpr (!KEEP) {
          value(i, gi, hi);
          columns(w[0], a.weight, a.wbf16, c0, cols, 1.f);
          #pragma unroll
          for (int j = 0; j < 4; ++j) gi.v[j] = mul2(gi.v[j], w[0].v[j]);
        }
        #pragma unroll
        for (int j = 0; j < 4; ++j)
          d.v[j] = mul2(rstd, fma2(hi.v[j], mh, add2(gi.v[j], mg)));
        if constexpr (FUSED) {
          if (ds) {
            Chunk e;
            take<T, REG>(e, from + (2 * PER + i * kPieces<T>) * nt, nt, cd + i * span, ds, c0, cols, vec);
            #pragma unroll
            for (int j = 0; j < 4; ++j) d.v[j] = add2(d.v[j], e.v[j]);
          }
          if (a.dresidual)
            put<T, REG>(static_cast<T*>(a.dresidual) + out + i * span, c0, cols, d, vec);
          if (a.drop) drop8(d.v, out + i * span, a.d);
        }
        if (a.dx) put<T, REG>(static_cast<T*>(a.dx) + out + i * span, c0, cols, d, vec);
      }
    }
    out += go.step * a.cols;
    if constexpr (!REG) {
      cy += go.step * a.lddy;
      cs += go.step * a.lds;
      cd += go.step * a.ldds;
    }
    from += stage_len;
    if (from == ring0 + a.depth * stage_len) from = ring0;
  }
  if (!a.part) return;
  // this block's column sums
  float* pw = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  float* pb = pw + a.cols;
  if constexpr (TPR == 0) {
    #pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c0 = col + i * span;
      #pragma unroll
      for (int j = 0; j < 8; ++j)
        if (inside(c0 + j, cols)) {
          pw[c0 + j] = elem(accw[i], j);
          pb[c0 + j] = elem(accb[i], j);
        }
    }
  } else {
    // row groups in order, through the ring's memory (every copy has landed
    // and been read)
    copy_wait(0);
    __syncthreads();
    float* buf = reinterpret_cast<float*>(ring);
    for (int c = threadIdx.x; c < 2 * cols; c += nt) buf[c] = 0.f;
    __syncthreads();
    for (int r = 0; r < at.rows; ++r) {
      if (r == at.g) {
        #pragma unroll
        for (int i = 0; i < C; ++i) {
          const int c0 = col + i * span;
          #pragma unroll
          for (int j = 0; j < 8; ++j)
            if (inside(c0 + j, cols)) {
              buf[c0 + j] += elem(accw[i], j);
              buf[cols + c0 + j] += elem(accb[i], j);
            }
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * cols; c += nt) pw[c] = buf[c];
  }
}

// dweight and dbias from the blocks' column sums: 32 columns a block, eight
// threads a column, then the eight in order
template <typename WT>
__global__ void __launch_bounds__(256) norm_join_kernel(int64_t cols, int parts, const float* part,
                                                        WT* dweight, WT* dbias) {
  __shared__ float red[2][8][32];
  pdl_wait();
  const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const int k = threadIdx.x >> 5;
  float w = 0.f, b = 0.f;
  if (c < cols) {
    #pragma unroll 4
    for (int i = k; i < parts; i += 8) {
      w += part[(int64_t)i * 2 * cols + c];
      b += part[((int64_t)i * 2 + 1) * cols + c];
    }
  }
  red[0][k][threadIdx.x & 31] = w;
  red[1][k][threadIdx.x & 31] = b;
  __syncthreads();
  if (k < 2 && c < cols) {
    float s = 0.f;
    #pragma unroll
    for (int i = 0; i < 8; ++i) s += red[k][i][threadIdx.x & 31];
    WT* out = k == 0 ? dweight : dbias;
    if (out) out[c] = from_f<WT>(s);
  }
}

// ------------------------------------------------- rows longer than a block

template <typename T, typename WT>
__global__ void __launch_bounds__(kNormThreads) norm_long_bwd_kernel(const __grid_constant__ NormBwd a) {
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

// --------------------------------------------------------------------- host

template <typename T, bool FUSED, bool REG>
cudaError_t backward(NormBwd a, int64_t chunks, int* parts, cudaStream_t s) {
  const Shape sh = norm_shape(chunks, true);
  size_t smem;
  ring_of(sh, sizeof(T), FUSED ? 3 : 2, &a.depth, &smem);
  const int64_t grid = norm_grid(sh, a.rows);
  *parts = (int)grid;
  if (sh.tpr == 8)
    return launch_rows(norm_bwd_kernel<T, 8, 1, 256, FUSED, true, REG>, a, grid, sh.nt, smem, s);
  if (sh.tpr == 32 && sh.c == 1)
    return launch_rows(norm_bwd_kernel<T, 32, 1, 256, FUSED, true, REG>, a, grid, sh.nt, smem, s);
  if (sh.tpr == 32)
    return launch_rows(norm_bwd_kernel<T, 32, 2, 256, FUSED, true, REG>, a, grid, sh.nt, smem, s);
  if (sh.c == 1)
    return launch_rows(norm_bwd_kernel<T, 0, 1, 128, FUSED, true, REG>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 128)
    return launch_rows(norm_bwd_kernel<T, 0, 2, 128, FUSED, true, REG>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 256)
    return launch_rows(norm_bwd_kernel<T, 0, 2, 256, FUSED, true, REG>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 512)
    return launch_rows(norm_bwd_kernel<T, 0, 2, 512, FUSED, true, REG>, a, grid, sh.nt, smem, s);
  return launch_rows(norm_bwd_kernel<T, 0, 2, 1024, FUSED, false, REG>, a, grid, sh.nt, smem, s);
}

template <typename T>
cudaError_t backward(const NormBwd& a, const Phases& ph, bool fused, int* parts, cudaStream_t s) {
  if (ph.regular())
    return fused ? backward<T, true, true>(a, ph.chunks(), parts, s)
                 : backward<T, false, true>(a, ph.chunks(), parts, s);
  return fused ? backward<T, true, false>(a, ph.chunks(), parts, s)
               : backward<T, false, false>(a, ph.chunks(), parts, s);
}

template <typename WT>
cudaError_t join(int64_t cols, int parts, const float* part, void* dweight, void* dbias,
                 cudaStream_t s) {
  return launch_k(norm_join_kernel<WT>, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, s, true,
                  cols, parts, part, static_cast<WT*>(dweight), static_cast<WT*>(dbias));
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_layer_norm_workspace_bytes(int64_t rows, int64_t cols, size_t* out) {
  if (!out || rows < 0) return MUON_ERR_INVALID_ARG;
  if (cols < 1 || cols > (int64_t)1 << 30) return MUON_ERR_UNSUPPORTED_SHAPE;
  *out = (size_t)norm_parts(rows, cols) * 2 * (size_t)cols * sizeof(float) + 256;
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
  Phases ph{rows, cols, es};
  ph.add(dy, lddy);
  ph.add(sum, ldsum);
  ph.add(dsum, ldds);
  ph.add(dx, cols);
  ph.add(dresidual, cols);
  const bool fused = dsum || dresidual || p > 0.f;
  const NormBwd a = {rows, cols, lddy, ldsum, ldds, dy, sum, dsum, weight, mean, rstd, dx,
                     dresidual, cols_wanted ? static_cast<float*>(workspace) : nullptr,
                     wdtype == MUON_BF16, p > 0.f, ph.same, 1, make_drop(p, seed, offset)};
  cudaError_t e;
  int parts = (int)(rows < kLongParts ? rows : kLongParts);
  if (ph.chunks() > kMaxChunks) {
    const int64_t tiles = (cols + kNormThreads - 1) / kNormThreads;
    e = by_types(dtype, wdtype, [&](auto t, auto wt) {
      using T = decltype(t);
      if (dx || dresidual)
        norm_long_bwd_kernel<T, decltype(wt)>
            <<<(int)(rows < kSMs * 8 ? rows : kSMs * 8), kNormThreads, 0, s>>>(a);
      if (cols_wanted)
        norm_cols_kernel<T><<<dim3(parts, (unsigned)(tiles < 65535 ? tiles : 65535)), kNormThreads,
                              0, s>>>(a);
      return cudaGetLastError();
    });
  } else {
    e = dtype == MUON_BF16 ? backward<__nv_bfloat16>(a, ph, fused, &parts, s)
                           : backward<float>(a, ph, fused, &parts, s);
  }
  if (e == cudaSuccess && cols_wanted)
    e = wdtype == MUON_BF16 ? join<__nv_bfloat16>(cols, parts, a.part, dweight, dbias, s)
                            : join<float>(cols, parts, a.part, dweight, dbias, s);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
