// Layer norm, alone or behind dropout and the residual add: the forward pass.
//
// Measured: [16384, 4096] bf16 44.9 us, 6.0 TB/s of x and y (42.6 us, 6.3 TB/s, of the
// kernel alone); behind dropout and the residual add [8192, 10240] 118 us, 5.7 TB/s;
// [4096, 10240] fp32 54 us, 6.2 TB/s; [9000, 3001] fp32 36 us, 5.9 TB/s; one row
// 2.5 us.  16-bit rows behind dropout are bound by instructions, 30 an element.
#include "norm.cuh"

#include <type_traits>

namespace muon {

namespace {

struct NormFwd {
  int64_t rows, cols, ldx, ldr;
  const void *x, *residual, *weight, *bias;
  void *sum, *y;
  float *mean, *rstd;
  float eps;
  int wbf16;        // weight and bias are bf16 ...
  int wvec;         // ... and 16-byte aligned
  int drop;
  Drop d;
};

// blocks of NT threads an SM: 24 warps, 80 registers a thread
__host__ __device__ constexpr int fwd_blocks(int nt) { return nt <= 768 ? 768 / nt : 1; }

// TPR threads a row (0: the block), C eights of elements a thread.  FUSED:
// residual and dropout may be present.
template <typename T, int TPR, int C, int NT, bool FUSED, bool REG>
__global__ void __launch_bounds__(NT, fwd_blocks(NT))
norm_fwd_kernel(const __grid_constant__ NormFwd a) {
  extern __shared__ uint4 ring[];
  __shared__ alignas(16) float slots[2][32];
  constexpr int E = kEl<T>, OPS = FUSED ? 2 : 1, PER = C * 8 / E;   // pieces a thread and operand
  constexpr int D = ring_depth(NT, C, sizeof(T), OPS, fwd_blocks(NT), 0);
  constexpr int nt = NT;
  constexpr int width = TPR ? TPR : nt, groups = TPR ? NT / (TPR ? TPR : 1) : 1;
  const int t = TPR ? (int)threadIdx.x % (TPR ? TPR : 1) : (int)threadIdx.x;
  const int g = TPR ? (int)threadIdx.x / (TPR ? TPR : 1) : 0;
  const int cols = (int)a.cols;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  if constexpr (TPR == 0) {
    for (int i = threadIdx.x; i < 64; i += nt) (&slots[0][0])[i] = 0.f;
    __syncthreads();
  }
  pdl_wait();
  const Visits go = visits(groups, g, a.rows);
  const int phase = REG ? 0 : (int)(((uint64_t)go.first * a.ldx) & (E - 1));
  int c0[PER];               // first column of each of the thread's pieces
  uint32_t in[PER];          // which of its elements are inside the row
  #pragma unroll
  for (int k = 0; k < PER; ++k) {
    c0[k] = (t + k * width) * E - phase;
    in[k] = inside<E, REG>(c0[k], cols);
  }
  const uint4 front = front_mask<T, REG>(c0[0]);
  // 1 for the elements inside the row, 0 for the others
  float2 one[REG ? 1 : PER][E / 2];
  if constexpr (!REG) {
    #pragma unroll
    for (int k = 0; k < PER; ++k)
      #pragma unroll
      for (int j = 0; j < E / 2; ++j)
        one[k][j] = make_float2(in[k] >> 2 * j & 1 ? 1.f : 0.f, in[k] >> (2 * j + 1) & 1 ? 1.f : 0.f);
  }
  // the next row to copy in, and the current row's elements in the outputs
  const T *fx = x + go.first * a.ldx, *fr = res + go.first * a.ldr;
  int64_t out = go.first * a.cols;
  const int stage_len = OPS * PER * nt;
  uint4* const ring0 = ring + threadIdx.x;
  uint4* fill = ring0;
  int ahead = 0;
  auto start = [&] {
    if (ahead < go.mine) {
      #pragma unroll
      for (int k = 0; k < PER; ++k) {
        fetch<T, REG>(fill + k * nt, fx + c0[k], in[k]);
        if (FUSED && res) fetch<T, REG>(fill + (PER + k) * nt, fr + c0[k], in[k]);
      }
    }
    copy_commit();
    ++ahead;
    fx += go.step * a.ldx;
    if constexpr (FUSED) fr += go.step * a.ldr;
    fill += stage_len;
    if (fill == ring0 + D * stage_len) fill = ring0;
  };
  #pragma unroll
  for (int s = 0; s + 1 < D; ++s) start();
  Piece<E> w[PER], b[PER];
  #pragma unroll
  for (int k = 0; k < PER; ++k) {
    columns<T, REG>(w[k], a.weight, a.wbf16, c0[k], in[k], 1.f, a.wvec);
    columns<T, REG>(b[k], a.bias, a.wbf16, c0[k], in[k], 0.f, a.wvec);
  }
  const float inv = 1.f / (float)cols;
  const uint4* from = ring0;
  int64_t row = go.first;
  for (int visit = 0; visit < go.all; ++visit) {
    start();                              // into the slot read in the last visit
    copy_wait<D - 1>();
    const bool live = TPR == 0 || visit < go.mine;
    Piece<E> v[PER];
    float2 s2 = both(0.f);
    #pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (live) {
        take<T, REG>(v[k], from + k * nt, in[k], k == 0, front);
        if constexpr (FUSED) {
          // without a branch the generator blocks of a thread's pieces overlap, where
          // there are registers for it: [8192, 10240] bf16 117.9 against 127.0 us,
          // [8192, 4096] fp32 92.7 against 93.7, [65536, 256] fp32 49.2 against 50.8; but
          // [4096, 16384] bf16 108.0 against 97.1, [4096, 10240] fp32 116.4 against 108.4
          if (a.drop)
            drop<E, REG && NT <= (sizeof(T) == 2 ? 704 : 512)>(v[k].v, out + c0[k], a.d);
          if (res) {
            Piece<E> r;
            take<T, REG>(r, from + (PER + k) * nt, in[k], k == 0, front);
            #pragma unroll
            for (int j = 0; j < E / 2; ++j) v[k].v[j] = add2(v[k].v[j], r.v[j]);
          }
          if (a.sum) put<T, REG>(static_cast<T*>(a.sum) + out + c0[k], v[k], in[k]);
        }
      } else {
        clear(v[k]);
      }
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) s2 = add2(s2, v[k].v[j]);
    }
    // The mean: the sum times a rounded 1 / cols, and one step of iterative refinement
    // by what that leaves of the sum (nothing to refine where the sum is infinite).
    // Without it the mean of a constant row of 1000 was off by its last bit and y by
    // 0.02; a division cost [32768, 1024] bf16 26.3 against 25.3 us
    // (24.9 without either).
    const float total = row_sum<TPR, sizeof(T) == 2>(s2.x + s2.y, slots[0], nt >> 5);
    const float near = total * inv, left = fmaf(-near, (float)cols, total);
    const float mean = fabsf(left) < INFINITY ? fmaf(left, inv, near) : near;
    const float2 m2 = both(-mean);
    float2 q2 = both(0.f);
    #pragma unroll
    for (int k = 0; k < PER; ++k) {
      // outside the row the zeros stay
      #pragma unroll
      for (int j = 0; j < E / 2; ++j)
        v[k].v[j] = REG ? add2(v[k].v[j], m2) : fma2(one[REG ? 0 : k][j], m2, v[k].v[j]);
      if (!REG || in[k]) {
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) q2 = fma2(v[k].v[j], v[k].v[j], q2);
      }
    }
    // rsqrtf is within two units of its last place, the sum within a few of its own
    const float rstd = rsqrtf(row_sum<TPR, sizeof(T) == 2>(q2.x + q2.y, slots[1], nt >> 5) * inv + a.eps);
    if (live) {
      const float2 r2 = both(rstd);
      #pragma unroll
      for (int k = 0; k < PER; ++k) {
        #pragma unroll
        for (int j = 0; j < E / 2; ++j)
          v[k].v[j] = fma2(mul2(v[k].v[j], r2), w[k].v[j], b[k].v[j]);
        put<T, REG>(static_cast<T*>(a.y) + out + c0[k], v[k], in[k]);
      }
      if (t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
    row += go.step;
    out += go.step * a.cols;
    from += stage_len;
    if (from == ring0 + D * stage_len) from = ring0;
  }
}

// ------- rows longer than a block, and operands whose phases differ

// Eight neighbours a thread, so that a generator block serves them all.  KEPT: the row's sums stay in shared memory (fp32) between the three
// passes; otherwise each pass reads and computes them again.
template <typename T, typename WT, bool KEPT, bool VEC>
__global__ void __launch_bounds__(kNormThreads) norm_long_fwd_kernel(const __grid_constant__ NormFwd a) {
  extern __shared__ uint4 ring[];
  __shared__ float red[kNormThreads / 32 + 1];
  Piece<8>* const kept = reinterpret_cast<Piece<8>*>(ring);
  const T* x = static_cast<const T*>(a.x);
  const T* r = static_cast<const T*>(a.residual);
  const WT* w = static_cast<const WT*>(a.weight);
  const WT* b = static_cast<const WT*>(a.bias);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    // the sums of eight columns from c; zeros past the row
    auto value = [&](Piece<8>& v, int64_t c) {
      load8<VEC>(v, x + row * a.ldx + c, a.cols - c);
      if (a.drop) drop<8, false>(v.v, row * a.cols + c, a.d);
      if (r) {
        Piece<8> e;
        load8<VEC>(e, r + row * a.ldr + c, a.cols - c);
        #pragma unroll
        for (int j = 0; j < 4; ++j) v.v[j] = add2(v.v[j], e.v[j]);
      }
    };
    auto again = [&](Piece<8>& v, int64_t c) {
      if (KEPT) v = kept[c >> 3];
      else value(v, c);
    };
    float s = 0.f;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += kNormThreads * 8) {
      Piece<8> v;
      value(v, c);
      if (KEPT) kept[c >> 3] = v;       // read by this thread alone
      #pragma unroll
      for (int j = 0; j < 8; ++j) s += elem(v, j);
    }
    const float mean = block_all_sum<kNormThreads>(s, red) / (float)a.cols;
    float q = 0.f;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += kNormThreads * 8) {
      Piece<8> v;
      again(v, c);
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = c + j < a.cols ? elem(v, j) - mean : 0.f;
        q = fmaf(e, e, q);
      }
    }
    const float rstd = rsqrtf(block_all_sum<kNormThreads>(q, red) / (float)a.cols + a.eps);
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += kNormThreads * 8) {
      Piece<8> v;
      again(v, c);
      if (a.sum) store8<VEC>(static_cast<T*>(a.sum) + row * a.cols + c, v, a.cols - c);
      Piece<8> wc, bc;
      weight8<VEC>(wc, w, c, a.cols, 1.f, a.wvec);
      weight8<VEC>(bc, b, c, a.cols, 0.f, a.wvec);
      const float2 m2 = both(-mean), r2 = both(rstd);
      #pragma unroll
      for (int j = 0; j < 4; ++j) v.v[j] = fma2(mul2(add2(v.v[j], m2), r2), wc.v[j], bc.v[j]);
      store8<VEC>(static_cast<T*>(a.y) + row * a.cols + c, v, a.cols - c);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// --------------------------------------------------------------------- host

template <typename T, int TPR, int C, int NT, bool FUSED, bool REG>
cudaError_t launch_fwd(const NormFwd& a, cudaStream_t s) {
  constexpr int D = ring_depth(NT, C, sizeof(T), FUSED ? 2 : 1, fwd_blocks(NT), 0);
  return launch_rows<norm_fwd_kernel<T, TPR, C, NT, FUSED, REG>>(
      a, blocks_for(a.rows, TPR ? NT / (TPR ? TPR : 1) : 1, fwd_blocks(NT)), NT,
      (size_t)D * NT * C * 8 * sizeof(T) * (FUSED ? 2 : 1), s);
}

// Rows of up to 64 columns take 8 lanes, of up to 512 a warp ([100000, 400] bf16
// 28.0 against 35.1 us with two, but behind dropout [65536, 512] 60.3 against
// 47.1), longer ones a block of the next size compiled in: eight elements a thread
// up to 1536 columns, sixteen beyond.  Ragged fp32 keeps eight up to 4096: one row of
// 3001 2.4 against 2.6 us, 500 rows 5.2 against 5.9, 9000 36.1 against 37.7, behind
// dropout 2.9, 8.2 and 73.8 against 3.6, 8.9 and 76.9; near the end of its block
// sixteen are faster ([9000, 4093] 53.0 against 58.1, behind dropout 97.3 against 110.8).
template <typename T, bool FUSED, bool REG>
cudaError_t forward(const NormFwd& a, int64_t chunks, cudaStream_t s) {
  if (chunks <= 8) return launch_fwd<T, 8, 1, 256, FUSED, REG>(a, s);
  if (chunks <= 32) return launch_fwd<T, 32, 1, 256, FUSED, REG>(a, s);
  if (chunks <= 64) {     // the random bits want registers: two warps a row where they are drawn
    if constexpr (FUSED) return launch_fwd<T, 0, 1, 64, FUSED, REG>(a, s);
    else return launch_fwd<T, 32, 2, 256, FUSED, REG>(a, s);
  }
  if (chunks <= 128) return launch_fwd<T, 0, 1, 128, FUSED, REG>(a, s);
  if (chunks <= 160) return launch_fwd<T, 0, 1, 160, FUSED, REG>(a, s);
  if (chunks <= 192) return launch_fwd<T, 0, 1, 192, FUSED, REG>(a, s);
  if constexpr (!REG && sizeof(T) == 4) {
    if (chunks <= 256) return launch_fwd<T, 0, 1, 256, FUSED, REG>(a, s);
    if (chunks <= 384) return launch_fwd<T, 0, 1, 384, FUSED, REG>(a, s);
    if (chunks <= 512) return launch_fwd<T, 0, 1, 512, FUSED, REG>(a, s);
  } else {
    if (chunks <= 256) return launch_fwd<T, 0, 2, 128, FUSED, REG>(a, s);
    if (chunks <= 384) return launch_fwd<T, 0, 2, 192, FUSED, REG>(a, s);
    if (chunks <= 512) return launch_fwd<T, 0, 2, 256, FUSED, REG>(a, s);
  }
  if (chunks <= 768) return launch_fwd<T, 0, 2, 384, FUSED, REG>(a, s);
  if (chunks <= 1024) return launch_fwd<T, 0, 2, 512, FUSED, REG>(a, s);
  if (chunks <= 1408) return launch_fwd<T, 0, 2, 704, FUSED, REG>(a, s);
  return launch_fwd<T, 0, 2, 1024, FUSED, REG>(a, s);
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
  ldx = row_stride(rows, ldx);
  ldr = row_stride(rows, ldr);
  Phases ph{rows, cols, es};
  ph.add(x, ldx);
  ph.add(residual, ldr);
  ph.add(sum, cols);
  ph.add(y, cols);
  const bool fused = residual || sum || p > 0.f;
  const NormFwd a = {rows, cols, ldx, ldr, x, residual, weight, bias, sum, y, mean, rstd, eps,
                     wdtype == MUON_BF16, !misaligned(weight, 16) && !misaligned(bias, 16), drop_threshold(p) > 0,
                     make_drop(p, seed, offset)};
  cudaError_t e;
  if (!ph.same || ph.chunks() > kMaxChunks) {
    constexpr size_t kMost = 200u << 10;      // of a row kept in shared memory
    const size_t row = ((size_t)cols + 7) / 8 * sizeof(Piece<8>);
    const int per_sm = row > kMost || row < 24u << 10 ? 4 : (int)((220u << 10) / row);
    const int64_t grid = blocks_for(rows, 1, per_sm);
    e = by_types(dtype, wdtype, [&](auto t, auto wt) {
      using T = decltype(t);
      using WT = decltype(wt);
      auto run = [&](auto vec) {
        constexpr bool VEC = decltype(vec)::value;
        if (row > kMost)
          return launch_k(norm_long_fwd_kernel<T, WT, false, VEC>, dim3((unsigned)grid),
                          dim3(kNormThreads), 0, s, false, a);
        const cudaError_t set = allow_shared<norm_long_fwd_kernel<T, WT, true, VEC>>(kMost);
        if (set != cudaSuccess) return set;
        return launch_k(norm_long_fwd_kernel<T, WT, true, VEC>, dim3((unsigned)grid),
                        dim3(kNormThreads), row, s, false, a);
      };
      return ph.eights() ? run(std::true_type()) : run(std::false_type());
    });
  } else {
    e = dtype == MUON_BF16 ? forward<__nv_bfloat16>(a, ph, fused, s) : forward<float>(a, ph, fused, s);
  }
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
