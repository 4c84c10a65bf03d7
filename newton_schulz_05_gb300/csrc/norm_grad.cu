// Layer norm, alone or behind dropout and the residual add: the gradient.
//
// With g = dy weight and h = (sum - mean) rstd a row needs the means of g and of
// g h before its first output: one reduction of two sums, after which the row is
// still in registers.  dy h and dy add up by column in registers over all the rows
// a thread visits; the row groups of a block are added through shared memory, the
// blocks' sums by a second kernel (norm_join_kernel) in a fixed order, so results
// do not depend on scheduling and nothing is added atomically.
//
// Measured: [16384, 4096] bf16 71 us, 5.7 TB/s of dy, sum and dx (67 us here, 4 in
// the join); with dropout and dsum [8192, 4096] 58 us, 5.7 TB/s; [8192, 4096] fp32
// 64 us, 6.3 TB/s; [9000, 3001] fp32 57 us, 5.6 TB/s.  16-bit rows are bound by
// instructions at sixteen warps an SM (the column sums take the registers of more):
// 18 an element, 35 with the random bits.
#include "norm.cuh"

namespace muon {

namespace {

struct NormBwd {
  int64_t rows, cols, lddy, lds, ldds;
  const void *dy, *sum, *dsum, *weight;
  const float *mean, *rstd;
  void *dx, *dresidual;
  float* part;      // [parts][2][cols], or null
  void *dweight, *dbias;     // written here where there is one block
  int wbf16;        // the weight is bf16 ...
  int wvec;         // ... and 16-byte aligned
  int drop;
  Drop d;
};

// waits for the threads of row group g alone
__device__ __forceinline__ void group_sync(int g, int width) {
  asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(width) : "memory");
}

constexpr int kBwdThreads = 512;     // one block an SM, 128 registers a thread

// shared memory for the weight of C eights of columns a thread, where the ring
// leaves room for it
__host__ __device__ constexpr int weight_bytes(int c, int es, int ops) {
  const int w = kBwdThreads * c * 8 * 4;
  return kBwdThreads * c * 8 * es * ops + w <= 220 << 10 ? w : 0;
}

// One block an SM, cut into row groups of TPR lanes or (TPR 0) of W threads, so
// that an SM leaves one partial column sum; C eights of elements a thread.  KEEP: the row's values and the weight stay in registers
// between the reduction and the output; otherwise (long rows) the values are
// read from the ring twice, and the weight from shared memory.
template <typename T, int TPR, int C, int W, bool FUSED, bool KEEP, bool REG>
__global__ void __launch_bounds__(kBwdThreads, 1)
norm_bwd_kernel(const __grid_constant__ NormBwd a) {
  extern __shared__ uint4 ring[];
  __shared__ alignas(16) float slots[2][2][40];
  constexpr int E = kEl<T>, OPS = FUSED ? 3 : 2, PER = C * 8 / E;
  constexpr int WB = KEEP ? 0 : weight_bytes(C, sizeof(T), OPS);
  constexpr int D = ring_depth(kBwdThreads, C, sizeof(T), OPS, 1, WB);
  constexpr int width = TPR ? TPR : W, groups = kBwdThreads / width, nt = groups * width;
  const int g = (int)threadIdx.x / width, t = (int)threadIdx.x - g * width;
  constexpr int warps = ((width >> 5) + 3) & ~3;  // of a row group, in whole float4s
  const int cols = (int)a.cols;
  const T* dy = static_cast<const T*>(a.dy);
  const T* sum = static_cast<const T*>(a.sum);
  const T* ds = static_cast<const T*>(a.dsum);
  if constexpr (TPR == 0) {
    for (int i = threadIdx.x; i < 160; i += nt) (&slots[0][0][0])[i] = 0.f;
    __syncthreads();
  }
  pdl_wait();
  const Visits go = visits(groups, g, a.rows);
  const int phase = REG ? 0 : (int)(((uint64_t)go.first * a.lddy) & (E - 1));
  int c0[PER];               // first column of each of the thread's pieces
  uint32_t in[PER];          // which of its elements are inside the row
  #pragma unroll
  for (int k = 0; k < PER; ++k) {
    c0[k] = (t + k * width) * E - phase;
    in[k] = inside<E, REG>(c0[k], cols);
  }
  const uint4 front = front_mask<T, REG>(c0[0]);
  // the next row to copy in, and the current row's elements in the outputs
  const T *fy = dy + go.first * a.lddy, *fs = sum + go.first * a.lds, *fd = ds + go.first * a.ldds;
  int64_t out = go.first * a.cols;
  const int stage_len = OPS * PER * nt;
  uint4* const ring0 = ring + threadIdx.x;
  uint4* fill = ring0;
  int ahead = 0;
  auto start = [&] {
    if (ahead < go.mine) {
      #pragma unroll
      for (int k = 0; k < PER; ++k) {
        fetch<T, REG>(fill + k * nt, fy + c0[k], in[k]);
        fetch<T, REG>(fill + (PER + k) * nt, fs + c0[k], in[k]);
        if (FUSED && ds) fetch<T, REG>(fill + (2 * PER + k) * nt, fd + c0[k], in[k]);
      }
    }
    copy_commit();
    ++ahead;
    fy += go.step * a.lddy;
    fs += go.step * a.lds;
    if constexpr (FUSED) fd += go.step * a.ldds;
    fill += stage_len;
    if (fill == ring0 + D * stage_len) fill = ring0;
  };
  #pragma unroll
  for (int s = 0; s + 1 < D; ++s) start();
  Piece<E> w[KEEP ? PER : 1], accw[PER], accb[PER];
  // the weight's place in shared memory, two pairs at a time
  float4* const ws = reinterpret_cast<float4*>(ring + D * stage_len) + threadIdx.x;
  #pragma unroll
  for (int k = 0; k < PER; ++k) {
    Piece<E>& wk = w[KEEP ? k : 0];
    if (KEEP || WB) columns<T, REG>(wk, a.weight, a.wbf16, c0[k], in[k], 1.f, a.wvec);
    if (!KEEP && WB) {
      #pragma unroll
      for (int j = 0; j < E / 4; ++j)
        ws[(k * (E / 4) + j) * nt] = make_float4(wk.v[2 * j].x, wk.v[2 * j].y, wk.v[2 * j + 1].x,
                                                 wk.v[2 * j + 1].y);
    }
    clear(accw[k]);
    clear(accb[k]);
  }
  auto weight = [&](int k) {      // into w[0], where it is not kept
    if constexpr (WB) {
      #pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        const float4 q = ws[(k * (E / 4) + j) * nt];
        w[0].v[2 * j] = make_float2(q.x, q.y);
        w[0].v[2 * j + 1] = make_float2(q.z, q.w);
      }
    } else {
      columns<T, REG>(w[0], a.weight, a.wbf16, c0[k], in[k], 1.f, a.wvec);
    }
  };
  const float inv = 1.f / (float)cols;
  const float *pm = a.mean + go.first, *pr = a.rstd + go.first;
  float mean_next = 0.f, rstd_next = 0.f;
  if (go.mine > 0) { mean_next = *pm; rstd_next = *pr; }
  const uint4* from = ring0;
  int turn = 0;
  // groups of whole warps meet only among themselves, so each makes its own
  // visits; lanes that share a warp make the block's
  const int visits_made = TPR == 0 ? go.mine : go.all;
  for (int visit = 0; visit < visits_made; ++visit) {
    start();                              // into the slot read in the last visit
    const bool live = TPR == 0 || visit < go.mine;
    const float2 mean = both(-mean_next), rstd = both(rstd_next);
    pm += go.step;
    pr += go.step;
    if (visit + 1 < go.mine) { mean_next = *pm; rstd_next = *pr; }
    copy_wait<D - 1>();
    // dy and h = (sum - mean) * rstd of piece k; outside the row dy is 0 and h is
    // -mean * rstd, so products with dy vanish there while that is finite
    auto value = [&](int k, Piece<E>& y, Piece<E>& h) {
      take<T, REG>(y, from + k * nt, in[k], k == 0, front);
      take<T, REG>(h, from + (PER + k) * nt, in[k], k == 0, front);
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) h.v[j] = mul2(add2(h.v[j], mean), rstd);
    };
    Piece<E> gk[KEEP ? PER : 1], hk[KEEP ? PER : 1];
    float2 sg2 = both(0.f), sh2 = both(0.f);
    #pragma unroll
    for (int k = 0; k < PER; ++k) {
      Piece<E>& gi = gk[KEEP ? k : 0];
      Piece<E>& hi = hk[KEEP ? k : 0];
      if (live && (!REG || in[k])) {
        value(k, gi, hi);
      } else {
        clear(gi);
        clear(hi);
      }
      if constexpr (!KEEP) weight(k);
      const Piece<E>& wi = w[KEEP ? k : 0];
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        accw[k].v[j] = fma2(gi.v[j], hi.v[j], accw[k].v[j]);
        accb[k].v[j] = add2(gi.v[j], accb[k].v[j]);
        gi.v[j] = mul2(gi.v[j], wi.v[j]);
        sg2 = add2(sg2, gi.v[j]);
        sh2 = fma2(gi.v[j], hi.v[j], sh2);
      }
    }
    float sg = sg2.x + sg2.y, sh = sh2.x + sh2.y;
    // mean * rstd may be infinite where no h of the row is: that of a constant row of
    // 2^120 whose rstd is 512.  The sum is then made again, of the row's columns alone.
    // Masking h in every edge piece instead cost [100000, 401] bf16 63.1 against 59.6 us
    if (!REG && live && !(fabsf(mean.x * rstd.x) < INFINITY)) {
      sh = 0.f;
      if constexpr (KEEP) {
        #pragma unroll
        for (int k = 0; k < PER; ++k)
          #pragma unroll
          for (int j = 0; j < E; ++j)
            if (in[k] >> j & 1) sh = fmaf(elem(gk[k], j), elem(hk[k], j), sh);
      } else {
        // an element at a time, which takes few registers: whole pieces, unrolled, made
        // the common path spill ([2097, 16001] bf16 84.9 against 62.8 us)
        #pragma unroll 1
        for (int i = 0; i < PER * E; ++i) {
          const int k = i / E, j = i % E, c = (t + k * width) * E + j - phase;
          if (c < 0 || c >= cols) continue;
          float gw = to_f(reinterpret_cast<const T*>(from + k * nt)[j]);
          if (a.weight)
            gw *= a.wbf16 ? to_f(static_cast<const __nv_bfloat16*>(a.weight)[c])
                          : static_cast<const float*>(a.weight)[c];
          const float s = to_f(reinterpret_cast<const T*>(from + (PER + k) * nt)[j]);
          sh = fmaf(gw, (s + mean.x) * rstd.x, sh);
        }
      }
    }
    if constexpr (TPR == 8) {
      #pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        sg += __shfl_xor_sync(0xffffffffu, sg, o);
        sh += __shfl_xor_sync(0xffffffffu, sh, o);
      }
    } else {
      // half a warp adds up one sum, half the other
      const bool low = (threadIdx.x & 16) == 0;
      float v = (low ? sg : sh) + __shfl_xor_sync(0xffffffffu, low ? sh : sg, 16);
      #pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if constexpr (TPR == 32) {
        sg = __shfl_sync(0xffffffffu, v, 0);
        sh = __shfl_sync(0xffffffffu, v, 16);
      } else {
        // a slot pair is rewritten two rows later, after the barrier of the
        // row between
        float* s2 = slots[turn][0] + g * warps;
        turn ^= 1;
        if ((threadIdx.x & 15) == 0) s2[(low ? 0 : 40) + (t >> 5)] = v;
        group_sync(g, width);
        sg = sh = 0.f;
        #pragma unroll
        for (int i = 0; i < warps; i += 4) {
          const float4 f = *reinterpret_cast<const float4*>(s2 + i);
          const float4 e = *reinterpret_cast<const float4*>(s2 + 40 + i);
          sg += (f.x + f.y) + (f.z + f.w);
          sh += (e.x + e.y) + (e.z + e.w);
        }
      }
    }
    const float2 mg = both(-sg * inv), mh = both(-sh * inv);
    if (live) {
      #pragma unroll
      for (int k = 0; k < PER; ++k) {
        Piece<E> d;
        Piece<E>& gi = gk[KEEP ? k : 0];
        Piece<E>& hi = hk[KEEP ? k : 0];
        if constexpr (!KEEP) {
          value(k, gi, hi);
          weight(k);
          #pragma unroll
          for (int j = 0; j < E / 2; ++j) gi.v[j] = mul2(gi.v[j], w[0].v[j]);
        }
        #pragma unroll
        for (int j = 0; j < E / 2; ++j)
          d.v[j] = mul2(rstd, fma2(hi.v[j], mh, add2(gi.v[j], mg)));
        if constexpr (FUSED) {
          if (ds) {
            Piece<E> e;
            take<T, REG>(e, from + (2 * PER + k) * nt, in[k], false, front);
            #pragma unroll
            for (int j = 0; j < E / 2; ++j) d.v[j] = add2(d.v[j], e.v[j]);
          }
          if (a.dresidual)
            put<T, REG>(static_cast<T*>(a.dresidual) + out + c0[k], d, in[k]);
          // without a branch the generator blocks of a thread's pieces overlap: [8192,
          // 4096] bf16 58.5 against 60.0 us, fp32 114.8 against 123.8; the long forms
          // [3276, 10240] 78.4 against 85.3, 128.5 against 129.9, [2048, 16384] 98.8
          // against 101.1, 166.0 against 168.0; from 64 columns on none is slower by
          // more than 1%
          if (a.drop) drop<E, REG>(d.v, out + c0[k], a.d);
        }
        if (a.dx) put<T, REG>(static_cast<T*>(a.dx) + out + c0[k], d, in[k]);
      }
    }
    out += go.step * a.cols;
    from += stage_len;
    if (from == ring0 + D * stage_len) from = ring0;
  }
  // the join may be set up while the column sums are put together
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!a.part) return;
  float* const pw = a.part + (int64_t)blockIdx.x * 2 * a.cols;
  float* const pb = pw + a.cols;
  if (TPR == 0 && groups == 1) {
    #pragma unroll
    for (int k = 0; k < PER; ++k) {
      #pragma unroll
      for (int j = 0; j < E; ++j)
        if (in[k] >> j & 1) {
          pw[c0[k] + j] = elem(accw[k], j);
          pb[c0[k] + j] = elem(accb[k], j);
        }
    }
  } else {
    // through the ring's memory (every copy has landed and been read): each group
    // leaves its sums as an image of its row, `phase` elements late, and columns
    // are added over the groups in order
    copy_wait<0>();
    __syncthreads();
    constexpr int kImage = PER * E;      // floats a thread and sum
    float* const image = reinterpret_cast<float*>(ring) + (size_t)g * 2 * width * kImage;
    #pragma unroll
    for (int k = 0; k < PER; ++k)
      #pragma unroll
      for (int q = 0; q < E / 4; ++q) {
        if (!in[k]) continue;
        float4* to = reinterpret_cast<float4*>(image + c0[k] + phase) + q;
        to[0] = make_float4(accw[k].v[2 * q].x, accw[k].v[2 * q].y, accw[k].v[2 * q + 1].x,
                            accw[k].v[2 * q + 1].y);
        to[width * kImage / 4] = make_float4(accb[k].v[2 * q].x, accb[k].v[2 * q].y,
                                             accb[k].v[2 * q + 1].x, accb[k].v[2 * q + 1].y);
      }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += nt) {
      float sw = 0.f, sb = 0.f;
      for (int r = 0; r < groups; ++r) {
        const int late =
            REG ? 0 : (int)((((uint64_t)blockIdx.x * groups + r) * a.lddy) & (E - 1));
        const float* from =
            reinterpret_cast<const float*>(ring) + (size_t)r * 2 * width * kImage + c + late;
        sw += from[0];
        sb += from[width * kImage];
      }
      pw[c] = sw;
      pb[c] = sb;
    }
  }
  // a block alone joins its sums itself.  A loop of its own: written into the
  // unrolled stores above the choice of types cost [2000, 7001] fp32 9 of 40 us
  if (gridDim.x > 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < cols; c += nt) {
    const float sw = pw[c], sb = pb[c];
    if (a.wbf16) {
      if (a.dweight) static_cast<__nv_bfloat16*>(a.dweight)[c] = from_f<__nv_bfloat16>(sw);
      if (a.dbias) static_cast<__nv_bfloat16*>(a.dbias)[c] = from_f<__nv_bfloat16>(sb);
    } else {
      if (a.dweight) static_cast<float*>(a.dweight)[c] = sw;
      if (a.dbias) static_cast<float*>(a.dbias)[c] = sb;
    }
  }
}

// dweight (blockIdx.y 0) and dbias (1) from the blocks' column sums: 32 columns a
// block, eight threads a column, then the eight in order
template <typename WT>
__global__ void __launch_bounds__(256) norm_join_kernel(int64_t cols, int parts, const float* part,
                                                        WT* dweight, WT* dbias) {
  __shared__ float red[8][32];
  WT* out = blockIdx.y == 0 ? dweight : dbias;
  if (!out) return;
  const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const int k = threadIdx.x >> 5;
  const float* p = part + blockIdx.y * cols + c;
  float s = 0.f;
  pdl_wait();
  if (c < cols) {
    #pragma unroll 10
    for (int i = k; i < parts; i += 8) s += p[(int64_t)i * 2 * cols];
  }
  red[k][threadIdx.x & 31] = s;
  __syncthreads();
  if (k == 0 && c < cols) {
    s = 0.f;
    #pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i][threadIdx.x];
    out[c] = from_f<WT>(s);
  }
}

// ------- rows longer than a block, and operands whose phases differ

// Eight neighbours a thread, so that a generator block serves them all; the
// second pass finds the row in L2.
template <typename T, typename WT, bool VEC>
__global__ void __launch_bounds__(kNormThreads) norm_long_bwd_kernel(const __grid_constant__ NormBwd a) {
  __shared__ float red[kNormThreads / 32 + 1];
  const T* dy = static_cast<const T*>(a.dy);
  const T* sum = static_cast<const T*>(a.sum);
  const T* ds = static_cast<const T*>(a.dsum);
  const WT* w = static_cast<const WT*>(a.weight);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float mean = a.mean[row], rstd = a.rstd[row];
    // g = dy weight and h = (sum - mean) rstd of eight columns from c; both are 0 past
    // the row
    auto value = [&](int64_t c, Piece<8>& g, Piece<8>& h) {
      Piece<8> wc;
      load8<VEC>(g, dy + row * a.lddy + c, a.cols - c);
      load8<VEC>(h, sum + row * a.lds + c, a.cols - c);
      weight8<VEC>(wc, w, c, a.cols, 1.f, a.wvec);
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        g.v[j] = mul2(g.v[j], wc.v[j]);
        h.v[j] = mul2(add2(h.v[j], both(-mean)), both(rstd));
      }
      if (!VEC && c + 8 > a.cols) {
        #pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j >= a.cols) elem(h, j) = 0.f;
      }
    };
    float2 sg2 = both(0.f), sh2 = both(0.f);
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += kNormThreads * 8) {
      Piece<8> g, h;
      value(c, g, h);
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        sg2 = add2(sg2, g.v[j]);
        sh2 = fma2(g.v[j], h.v[j], sh2);
      }
    }
    const float sg = block_all_sum<kNormThreads>(sg2.x + sg2.y, red) / (float)a.cols;
    const float sh = block_all_sum<kNormThreads>(sh2.x + sh2.y, red) / (float)a.cols;
    for (int64_t c = threadIdx.x * 8; c < a.cols; c += kNormThreads * 8) {
      Piece<8> g, h;
      value(c, g, h);
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        g.v[j] = mul2(both(rstd), fma2(h.v[j], both(-sh), add2(g.v[j], both(-sg))));
      if (ds) {
        Piece<8> e;
        load8<VEC>(e, ds + row * a.ldds + c, a.cols - c);
        #pragma unroll
        for (int j = 0; j < 4; ++j) g.v[j] = add2(g.v[j], e.v[j]);
      }
      if (a.dresidual) store8<VEC>(static_cast<T*>(a.dresidual) + row * a.cols + c, g, a.cols - c);
      if (a.drop) drop<8, false>(g.v, row * a.cols + c, a.d);
      if (a.dx) store8<VEC>(static_cast<T*>(a.dx) + row * a.cols + c, g, a.cols - c);
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

// partial column sums of a gradient, whatever its width and the phases of its operands
int64_t norm_parts(int64_t rows) { return rows < kLongParts ? rows : kLongParts; }

template <typename T, int TPR, int C, int W, bool FUSED, bool KEEP, bool REG>
cudaError_t launch_bwd(const NormBwd& a, int* parts, cudaStream_t s) {
  constexpr int OPS = FUSED ? 3 : 2, WB = KEEP ? 0 : weight_bytes(C, sizeof(T), OPS);
  constexpr int D = ring_depth(kBwdThreads, C, sizeof(T), OPS, 1, WB);
  constexpr int width = TPR ? TPR : W, groups = kBwdThreads / width, nt = groups * width;
  const int64_t grid = blocks_for(a.rows, groups, 1);
  *parts = (int)grid;
  return launch_rows<norm_bwd_kernel<T, TPR, C, W, FUSED, KEEP, REG>>(
      a, grid, nt, (size_t)nt * C * 8 * sizeof(T) * OPS * D + (WB ? (size_t)nt * C * 32 : 0), s);
}

// Rows of up to 64 columns take 8 lanes, of up to 512 a warp, of up to 8192 the
// next number of threads that is compiled in, sixteen elements each, longer ones
// the whole block.
template <typename T, bool FUSED, bool REG>
cudaError_t backward(const NormBwd& a, int64_t chunks, int* parts, cudaStream_t s) {
  if (chunks <= 8) return launch_bwd<T, 8, 1, 0, FUSED, true, REG>(a, parts, s);
  if (chunks <= 32) return launch_bwd<T, 32, 1, 0, FUSED, true, REG>(a, parts, s);
  if (chunks <= 64) {     // as in the forward pass
    if constexpr (FUSED) return launch_bwd<T, 0, 1, 64, FUSED, true, REG>(a, parts, s);
    else return launch_bwd<T, 32, 2, 0, FUSED, true, REG>(a, parts, s);
  }
  // Ragged fp32 rows with dsum or dropout: sixteen elements a thread spill, so eight
  // ([9000, 3001] p .1 107.6 against 126.9 us, dsum alone 81.2 against 96.8; [1000, 1023]
  // 13.0 against 14.7, 11.2 against 12.4), unless there are few rows and more groups a
  // block count for more ([517, 1023] 10.5 against 9.0, 8.8 against 7.6).  Without them
  // sixteen fit ([9000, 3001] 57.5 against 68.1, [2000, 3001] 20.7 against 22.6).
  if constexpr (!REG && sizeof(T) == 4 && FUSED) {
    if (a.rows > 4 * kSMs) {
      if (chunks <= 128) return launch_bwd<T, 0, 1, 128, FUSED, true, REG>(a, parts, s);
      if (chunks <= 160) return launch_bwd<T, 0, 1, 160, FUSED, true, REG>(a, parts, s);
      if (chunks <= 256) return launch_bwd<T, 0, 1, 256, FUSED, true, REG>(a, parts, s);
      if (chunks <= 512) return launch_bwd<T, 0, 1, 512, FUSED, true, REG>(a, parts, s);
    }
  }
  if (chunks <= 128) return launch_bwd<T, 0, 2, 64, FUSED, true, REG>(a, parts, s);
  if (chunks <= 192) return launch_bwd<T, 0, 2, 96, FUSED, true, REG>(a, parts, s);
  if (chunks <= 256) return launch_bwd<T, 0, 2, 128, FUSED, true, REG>(a, parts, s);
  if (chunks <= 512) return launch_bwd<T, 0, 2, 256, FUSED, true, REG>(a, parts, s);
  if (chunks <= 1024) return launch_bwd<T, 0, 2, 512, FUSED, true, REG>(a, parts, s);
  if (chunks <= 1536) return launch_bwd<T, 0, 3, 512, FUSED, false, REG>(a, parts, s);
  return launch_bwd<T, 0, 4, 512, FUSED, false, REG>(a, parts, s);
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
  return launch_k(norm_join_kernel<WT>, dim3((unsigned)((cols + 31) / 32), 2), dim3(256), 0, s, true,
                  cols, parts, part, static_cast<WT*>(dweight), static_cast<WT*>(dbias));
}

}  // namespace

}  // namespace muon

using namespace muon;

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
  lddy = row_stride(rows, lddy);
  ldsum = row_stride(rows, ldsum);
  ldds = row_stride(rows, ldds);
  Phases ph{rows, cols, es};
  ph.add(dy, lddy);
  ph.add(sum, ldsum);
  ph.add(dsum, ldds);
  ph.add(dx, cols);
  ph.add(dresidual, cols);
  const bool fused = dsum || dresidual || p > 0.f;
  const NormBwd a = {rows, cols, lddy, ldsum, ldds, dy, sum, dsum, weight, mean, rstd, dx,
                     dresidual, cols_wanted ? static_cast<float*>(workspace) : nullptr, dweight, dbias,
                     wdtype == MUON_BF16, !misaligned(weight, 16), drop_threshold(p) > 0,
                     make_drop(p, seed, offset)};
  cudaError_t e;
  int parts = (int)norm_parts(rows);
  bool joined = false;
  if (!ph.same || ph.chunks() > kMaxChunks) {
    const int64_t tiles = (cols + kNormThreads - 1) / kNormThreads;
    e = by_types(dtype, wdtype, [&](auto t, auto wt) {
      using T = decltype(t);
      using WT = decltype(wt);
      cudaError_t e = cudaSuccess;
      if (dx || dresidual)
        e = launch_k(ph.eights() ? norm_long_bwd_kernel<T, WT, true> : norm_long_bwd_kernel<T, WT, false>,
                     dim3((unsigned)blocks_for(rows, 1, 4)), dim3(kNormThreads), 0, s, false, a);
      if (cols_wanted && e == cudaSuccess)
        e = launch_k(norm_cols_kernel<T>, dim3(parts, (unsigned)(tiles < 65535 ? tiles : 65535)),
                     dim3(kNormThreads), 0, s, false, a);
      return e;
    });
  } else {
    e = dtype == MUON_BF16 ? backward<__nv_bfloat16>(a, ph, fused, &parts, s)
                           : backward<float>(a, ph, fused, &parts, s);
    joined = parts == 1;
  }
  if (e == cudaSuccess && cols_wanted && !joined)
    e = wdtype == MUON_BF16 ? join<__nv_bfloat16>(cols, parts, a.part, dweight, dbias, s)
                            : join<float>(cols, parts, a.part, dweight, dbias, s);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
