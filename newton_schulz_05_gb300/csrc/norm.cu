// Layer norm, alone or behind dropout and the residual add, and its gradient
// with the reduction of the weight's and the bias's.
//
// Both passes are bound by HBM: forward reads x (and the residual) and writes
// y (and the sum) once, backward reads dy, the sum (and dsum) and writes dx
// (and dresidual) once.  A row lives in the registers of 8 lanes, a warp or a
// block (by its length), so its statistics take no second trip to memory: the
// mean first, then the centred squares, both over registers in fp32.
//
// Layout.  A row is cut into chunks of eight elements that are aligned in
// memory, not in the row: a row that starts `phase` elements past an aligned
// address has its first chunk begin `phase` elements early, and what falls
// outside the row is masked.  So rows of odd width move in 16-byte accesses
// too.  A thread takes the same chunks of every row it visits (row steps are
// multiples of eight, which keeps the phase), so weights stay in registers and
// the column sums of the gradient accumulate there.  Operands whose phases
// differ are read element by element.
//
// Rows stream through a ring of asynchronous copies into shared memory.  Each
// thread copies, waits for and reads only its own chunks, so the ring needs no
// barrier; its depth holds enough bytes in flight to cover the HBM latency
// while a row is reduced.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "random.cuh"

namespace muon {

namespace {

constexpr int kNormThreads = 256;    // of the kernels for rows longer than a block holds
constexpr int kSMs = 152;
constexpr int kRingDepth = 4;        // rows in flight per block, when shared memory allows
constexpr size_t kRingBytes = 220u << 10;   // shared memory of an SM given to rings

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

// ------------------------------------------------------------ chunks of rows

// pairs of fp32 in one instruction each (two round-to-nearest operations)
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{.reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

struct Chunk { float2 v[4]; };   // eight consecutive elements
__device__ __forceinline__ float& elem(Chunk& c, int j) { return j & 1 ? c.v[j >> 1].y : c.v[j >> 1].x; }
__device__ __forceinline__ void clear(Chunk& c) {
  #pragma unroll
  for (int j = 0; j < 4; ++j) c.v[j] = make_float2(0.f, 0.f);
}

// 16-byte pieces of a chunk
template <typename T> constexpr int kPieces = (int)sizeof(T) / 2;

__device__ __forceinline__ void copy16(void* smem, const void* global, int bytes) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(smem);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(s), "l"(global), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copy16(void* smem, const void* global) {
  const uint32_t s = (uint32_t)__cvta_generic_to_shared(smem);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(s), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
// until at most `n` (0 .. kRingDepth - 1) of the newest groups are in flight
__device__ __forceinline__ void copy_wait(int n) {
  if (n >= 3) asm volatile("cp.async.wait_group 3;\n" ::: "memory");
  else if (n == 2) asm volatile("cp.async.wait_group 2;\n" ::: "memory");
  else if (n == 1) asm volatile("cp.async.wait_group 1;\n" ::: "memory");
  else asm volatile("cp.async.wait_group 0;\n" ::: "memory");
}

// What a chunk that begins at column c0 holds of its row
__device__ __forceinline__ bool whole(int c0, int cols) { return c0 >= 0 && c0 + 8 <= cols; }
__device__ __forceinline__ bool inside(int c, int cols) { return c >= 0 && c < cols; }

// Start the copy of the chunk whose first element is base[at], column c0 of
// its row, into slot[0], slot[stride].  Bytes past the row are not read; bytes
// ahead of it are, when they lie inside the tensor (at >= 0), and masked later.
template <typename T>
__device__ __forceinline__ void fetch(uint4* slot, int stride, const T* base, int64_t at, int c0,
                                      int cols) {
  constexpr int per = 8 / kPieces<T>;
  if (whole(c0, cols)) {
    #pragma unroll
    for (int q = 0; q < kPieces<T>; ++q) copy16(slot + q * stride, base + at + q * per);
  } else if (at >= 0) {
    #pragma unroll
    for (int q = 0; q < kPieces<T>; ++q) {
      const int left = cols - c0 - q * per;
      if (left > 0)
        copy16(slot + q * stride, base + at + q * per, (left < per ? left : per) * (int)sizeof(T));
    }
  }
}

__device__ __forceinline__ void unpack(const uint4* slot, int, Chunk& c, __nv_bfloat16) {
  const uint4 u = slot[0];
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  #pragma unroll
  for (int j = 0; j < 4; ++j)
    c.v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}
__device__ __forceinline__ void unpack(const uint4* slot, int stride, Chunk& c, float) {
  const float4 a = *reinterpret_cast<const float4*>(slot);
  const float4 b = *reinterpret_cast<const float4*>(slot + stride);
  c.v[0] = make_float2(a.x, a.y);
  c.v[1] = make_float2(a.z, a.w);
  c.v[2] = make_float2(b.x, b.y);
  c.v[3] = make_float2(b.z, b.w);
}

// The chunk in fp32, zeros outside the row: from its ring slot, or from memory
// where fetch() made no copy.
template <typename T>
__device__ __forceinline__ void take(Chunk& c, const uint4* slot, int stride, const T* base,
                                     int64_t at, int c0, int cols, bool vec) {
  if (vec && whole(c0, cols)) {
    unpack(slot, stride, c, T());
  } else if (vec && at >= 0 && c0 < cols) {
    unpack(slot, stride, c, T());
    #pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!inside(c0 + j, cols)) elem(c, j) = 0.f;
  } else {
    #pragma unroll
    for (int j = 0; j < 8; ++j) elem(c, j) = inside(c0 + j, cols) ? to_f(base[at + j]) : 0.f;
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const Chunk& c) {
  uint32_t w[4];
  #pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __float22bfloat162_rn(c.v[j]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const Chunk& c) {
  reinterpret_cast<float4*>(p)[0] = make_float4(c.v[0].x, c.v[0].y, c.v[1].x, c.v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(c.v[2].x, c.v[2].y, c.v[3].x, c.v[3].y);
}

template <typename T>
__device__ __forceinline__ void put(T* base, int64_t at, int c0, int cols, Chunk& c, bool vec) {
  if (vec && whole(c0, cols)) {
    store8(base + at, c);
  } else {
    #pragma unroll
    for (int j = 0; j < 8; ++j)
      if (inside(c0 + j, cols)) base[at + j] = from_f<T>(elem(c, j));
  }
}

// weight (or bias) of the chunk's columns; `none` where there is no vector
__device__ __forceinline__ void columns(Chunk& c, const void* w, int bf16, int c0, int cols,
                                        float none) {
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    float v = none;
    if (w && inside(c0 + j, cols))
      v = bf16 ? to_f(static_cast<const __nv_bfloat16*>(w)[c0 + j])
               : static_cast<const float*>(w)[c0 + j];
    elem(c, j) = v;
  }
}

// Sum over the threads of a row (TPR lanes, or the block where TPR is 0), the
// same value in each; slots: one float a warp, zeros up to a multiple of four.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* slots, int warps) {
  #pragma unroll
  for (int o = (TPR == 0 ? 32 : TPR) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR == 0) {
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int i = 0; i < warps; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(slots + i);
      v += (f.x + f.y) + (f.z + f.w);
    }
  }
  return v;
}

// A thread's place: row group g of the block, thread t of the row
template <int TPR> struct Place {
  int t, g, rows, width;       // rows: row groups in a block; width: threads a row
  __device__ __forceinline__ Place() {
    width = TPR == 0 ? (int)blockDim.x : TPR;
    t = TPR == 0 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
    g = TPR == 0 ? 0 : (int)threadIdx.x / TPR;
    rows = TPR == 0 ? 1 : (int)blockDim.x / TPR;
  }
};

// registers a thread that a block of NT threads is held to: blocks an SM
constexpr int fwd_blocks(int nt) { return nt <= 128 ? 6 : nt <= 256 ? 3 : 1; }
constexpr int bwd_blocks(int nt) { return nt <= 128 ? 4 : nt <= 256 ? 2 : 1; }

// ------------------------------------------------------------------ forward

// TPR threads a row (0: the block), C chunks a thread.  FUSED: residual and
// dropout may be present.
template <typename T, int TPR, int C, int NT, bool FUSED>
__global__ void __launch_bounds__(NT, fwd_blocks(NT))
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
  const bool vec = a.vec;
  const int64_t step = (int64_t)gridDim.x * at.rows;
  const int64_t first = (int64_t)blockIdx.x * at.rows + at.g;
  const int phase =
      vec ? (int)((reinterpret_cast<uintptr_t>(x) / sizeof(T) + (uint64_t)first * a.ldx) & 7) : 0;
  const int col = at.t * 8 - phase;             // chunk i begins at column col + i * span
  const int span = at.width * 8;
  auto slot = [&](int stage, int op, int i) {
    return ring + ((stage * OPS + op) * PER + i * kPieces<T>) * nt + threadIdx.x;
  };
  auto start = [&](int64_t row, int stage) {
    if (vec && row < a.rows) {
      #pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c0 = col + i * span;
        fetch<T>(slot(stage, 0, i), nt, x, row * a.ldx + c0, c0, cols);
        if (FUSED && res) fetch<T>(slot(stage, OPS - 1, i), nt, res, row * a.ldr + c0, c0, cols);
      }
    }
    copy_commit();
  };
  for (int s = 0; s + 1 < a.depth; ++s) start(first + s * step, s);
  Chunk w[C], b[C];
  #pragma unroll
  for (int i = 0; i < C; ++i) {
    columns(w[i], a.weight, a.wbf16, col + i * span, cols, 1.f);
    columns(b[i], a.bias, a.wbf16, col + i * span, cols, 0.f);
  }
  const float inv = 1.f / (float)cols;
  int stage = 0;
  for (int64_t base = (int64_t)blockIdx.x * at.rows; base < a.rows; base += step) {
    const int64_t row = base + at.g;
    const bool live = row < a.rows;
    int into = stage + a.depth - 1;       // the slot read in the last iteration
    if (into >= a.depth) into -= a.depth;
    start(row + (a.depth - 1) * step, into);
    copy_wait(a.depth - 1);
    Chunk v[C];
    float2 s2 = both(0.f);
    #pragma unroll
    for (int i = 0; i < C; ++i) {
      const int c0 = col + i * span;
      if (live) {
        take<T>(v[i], slot(stage, 0, i), nt, x, row * a.ldx + c0, c0, cols, vec);
        if constexpr (FUSED) {
          if (a.drop) drop8(v[i].v, row * a.cols + c0, a.d);
          if (res) {
            Chunk r;
            take<T>(r, slot(stage, 1, i), nt, res, row * a.ldr + c0, c0, cols, vec);
            #pragma unroll
            for (int j = 0; j < 4; ++j) v[i].v[j] = add2(v[i].v[j], r.v[j]);
          }
          if (a.sum) put<T>(static_cast<T*>(a.sum), row * a.cols + c0, c0, cols, v[i], vec);
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
      if (whole(c0, cols)) {
        #pragma unroll
        for (int j = 0; j < 4; ++j) q2 = fma2(v[i].v[j], v[i].v[j], q2);
      } else {
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
        put<T>(static_cast<T*>(a.y), row * a.cols + c0, c0, cols, v[i], vec);
      }
      if (at.t == 0) {
        if (a.mean) a.mean[row] = mean;
        if (a.rstd) a.rstd[row] = rstd;
      }
    }
    if (++stage == a.depth) stage = 0;
  }
}

// ----------------------------------------------------------------- backward

// KEEP: the row's values stay in registers between the reduction and the
// output; otherwise (blocks of 1024 threads, 64 registers each) they are read
// from the ring twice, and the weight from memory.
template <typename T, int TPR, int C, int NT, bool FUSED, bool KEEP>
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
  const bool vec = a.vec;
  const int64_t step = (int64_t)gridDim.x * at.rows;
  const int64_t first = (int64_t)blockIdx.x * at.rows + at.g;
  const int phase =
      vec ? (int)((reinterpret_cast<uintptr_t>(dy) / sizeof(T) + (uint64_t)first * a.lddy) & 7) : 0;
  const int col = at.t * 8 - phase;
  const int span = at.width * 8;
  auto slot = [&](int stage, int op, int i) {
    return ring + ((stage * OPS + op) * PER + i * kPieces<T>) * nt + threadIdx.x;
  };
  auto start = [&](int64_t row, int stage) {
    if (vec && row < a.rows) {
      #pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c0 = col + i * span;
        fetch<T>(slot(stage, 0, i), nt, dy, row * a.lddy + c0, c0, cols);
        fetch<T>(slot(stage, 1, i), nt, sum, row * a.lds + c0, c0, cols);
        if (FUSED && ds) fetch<T>(slot(stage, OPS - 1, i), nt, ds, row * a.ldds + c0, c0, cols);
      }
    }
    copy_commit();
  };
  for (int s = 0; s + 1 < a.depth; ++s) start(first + s * step, s);
  Chunk w[KEEP ? C : 1], accw[C], accb[C];
  #pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (KEEP) columns(w[i], a.weight, a.wbf16, col + i * span, cols, 1.f);
    clear(accw[i]);
    clear(accb[i]);
  }
  const float inv = 1.f / (float)cols;
  float mean_next = 0.f, rstd_next = 0.f;
  if (first < a.rows) { mean_next = a.mean[first]; rstd_next = a.rstd[first]; }
  int stage = 0, turn = 0;
  for (int64_t base = (int64_t)blockIdx.x * at.rows; base < a.rows; base += step) {
    const int64_t row = base + at.g;
    const bool live = row < a.rows;
    int into = stage + a.depth - 1;
    if (into >= a.depth) into -= a.depth;
    start(row + (a.depth - 1) * step, into);
    const float2 mean = both(-mean_next), rstd = both(rstd_next);
    if (row + step < a.rows) { mean_next = a.mean[row + step]; rstd_next = a.rstd[row + step]; }
    copy_wait(a.depth - 1);
    // dy and h = (sum - mean) * rstd of chunk i
    auto value = [&](int i, Chunk& y, Chunk& h) {
      const int c0 = col + i * span;
      take<T>(y, slot(stage, 0, i), nt, dy, row * a.lddy + c0, c0, cols, vec);
      take<T>(h, slot(stage, 1, i), nt, sum, row * a.lds + c0, c0, cols, vec);
      #pragma unroll
      for (int j = 0; j < 4; ++j) h.v[j] = mul2(add2(h.v[j], mean), rstd);
      if (!whole(c0, cols)) {
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
      if (live) {
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
            take<T>(e, slot(stage, 2, i), nt, ds, row * a.ldds + c0, c0, cols, vec);
            #pragma unroll
            for (int j = 0; j < 4; ++j) d.v[j] = add2(d.v[j], e.v[j]);
          }
          if (a.dresidual)
            put<T>(static_cast<T*>(a.dresidual), row * a.cols + c0, c0, cols, d, vec);
          if (a.drop) drop8(d.v, row * a.cols + c0, a.d);
        }
        if (a.dx) put<T>(static_cast<T*>(a.dx), row * a.cols + c0, c0, cols, d, vec);
      }
    }
    if (++stage == a.depth) stage = 0;
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

// sum over the block, the same value in every thread
template <int NT>
__device__ __forceinline__ float block_all_sum(float v, float* red /* NT/32 + 1 floats */) {
  const float s = block_sum<NT>(v, red);
  if (threadIdx.x == 0) red[NT / 32] = s;
  __syncthreads();
  const float r = red[NT / 32];
  __syncthreads();
  return r;
}

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

// How rows of `chunks` chunks are laid out: threads a row (0: the block),
// chunks a thread, threads a block, blocks an SM.
struct Shape { int tpr, c, nt, per_sm; };
constexpr int64_t kMaxChunks = 2048;

Shape norm_shape(int64_t chunks, bool backward) {
  if (chunks <= 8) return {8, 1, 256, 4};
  if (chunks <= 32) return {32, 1, 256, 4};
  if (chunks <= 64) return {32, 2, 256, 2};
  if (chunks <= 128) return {0, 1, (int)(chunks + 31) / 32 * 32, 8};
  const int nt = (int)(((chunks + 1) / 2 + 31) / 32 * 32);
  return {0, 2, nt, backward ? bwd_blocks(nt) : fwd_blocks(nt)};
}

int64_t norm_grid(const Shape& s, int64_t rows) {
  const int64_t per = s.tpr == 0 ? 1 : s.nt / s.tpr;
  const int64_t want = (rows + per - 1) / per;
  return want < kSMs * s.per_sm ? want : kSMs * s.per_sm;
}

constexpr int kLongParts = 304;

// partial column sums of a gradient, whatever the phases of its operands
int64_t norm_parts(int64_t rows, int64_t cols) {
  const int64_t most = norm_grid(norm_shape((cols + 7) / 8, true), rows);
  const int64_t odd = norm_grid(norm_shape((cols + 14) / 8, true), rows);
  const int64_t large = rows < kLongParts ? rows : kLongParts;
  int64_t p = most > odd ? most : odd;
  if ((cols + 14) / 8 > kMaxChunks) p = p > large ? p : large;
  return p;
}

bool misaligned(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

// Collects the phases of the operands' rows: `same` while they all agree,
// `chunks` the chunks of the longest row.
struct Phases {
  int64_t rows, cols;
  size_t es;
  bool same = true, any = false;
  int phase = 0, ld = 0;
  void add(const void* p, int64_t stride) {
    if (!p) return;
    const int f = (int)(reinterpret_cast<uintptr_t>(p) / es & 7);
    const int l = rows > 1 ? (int)(stride & 7) : 0;
    if (any && (f != phase || l != ld)) same = false;
    if (!any) { any = true; phase = f; ld = l; }
  }
  int64_t chunks() const {
    const int most = !same ? 0 : ld ? 7 : phase;
    return (cols + most + 7) / 8;
  }
};

muon_status check_common(int64_t rows, int64_t cols, int dtype, int wdtype, float p) {
  if (rows < 0 || !(p >= 0.f && p <= 1.f)) return MUON_ERR_INVALID_ARG;
  if (cols < 1 || cols > (int64_t)1 << 30 || rows > (int64_t)1 << 40)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  if ((dtype != MUON_BF16 && dtype != MUON_F32) || (wdtype != MUON_BF16 && wdtype != MUON_F32))
    return MUON_ERR_DTYPE;
  return MUON_OK;
}

// ring depth and bytes for `ops` operands
void ring_of(const Shape& s, size_t es, int ops, int* depth, size_t* bytes) {
  const size_t row = (size_t)s.nt * s.c * 8 * es * ops;
  const size_t room = kRingBytes / s.per_sm;
  size_t d = room / row;
  *depth = d < 1 ? 1 : d > (size_t)kRingDepth ? kRingDepth : (int)d;
  *bytes = row * *depth;
}

template <typename K, typename A>
cudaError_t launch_rows(K kernel, const A& a, int64_t grid, int nt, size_t smem, cudaStream_t s) {
  if (smem > 40u << 10) {     // 48 KB with the static part, without the attribute
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(224u << 10));
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)grid, nt, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool FUSED>
cudaError_t forward(NormFwd a, int64_t chunks, cudaStream_t s) {
  const Shape sh = norm_shape(chunks, false);
  size_t smem;
  ring_of(sh, sizeof(T), FUSED ? 2 : 1, &a.depth, &smem);
  const int64_t grid = norm_grid(sh, a.rows);
  if (sh.tpr == 8) return launch_rows(norm_fwd_kernel<T, 8, 1, 256, FUSED>, a, grid, sh.nt, smem, s);
  if (sh.tpr == 32 && sh.c == 1)
    return launch_rows(norm_fwd_kernel<T, 32, 1, 256, FUSED>, a, grid, sh.nt, smem, s);
  if (sh.tpr == 32) return launch_rows(norm_fwd_kernel<T, 32, 2, 256, FUSED>, a, grid, sh.nt, smem, s);
  if (sh.c == 1) return launch_rows(norm_fwd_kernel<T, 0, 1, 128, FUSED>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 128) return launch_rows(norm_fwd_kernel<T, 0, 2, 128, FUSED>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 256) return launch_rows(norm_fwd_kernel<T, 0, 2, 256, FUSED>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 512) return launch_rows(norm_fwd_kernel<T, 0, 2, 512, FUSED>, a, grid, sh.nt, smem, s);
  return launch_rows(norm_fwd_kernel<T, 0, 2, 1024, FUSED>, a, grid, sh.nt, smem, s);
}

template <typename T, bool FUSED>
cudaError_t backward(NormBwd a, int64_t chunks, int* parts, cudaStream_t s) {
  const Shape sh = norm_shape(chunks, true);
  size_t smem;
  ring_of(sh, sizeof(T), FUSED ? 3 : 2, &a.depth, &smem);
  const int64_t grid = norm_grid(sh, a.rows);
  *parts = (int)grid;
  if (sh.tpr == 8)
    return launch_rows(norm_bwd_kernel<T, 8, 1, 256, FUSED, true>, a, grid, sh.nt, smem, s);
  if (sh.tpr == 32 && sh.c == 1)
    return launch_rows(norm_bwd_kernel<T, 32, 1, 256, FUSED, true>, a, grid, sh.nt, smem, s);
  if (sh.tpr == 32)
    return launch_rows(norm_bwd_kernel<T, 32, 2, 256, FUSED, true>, a, grid, sh.nt, smem, s);
  if (sh.c == 1)
    return launch_rows(norm_bwd_kernel<T, 0, 1, 128, FUSED, true>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 128)
    return launch_rows(norm_bwd_kernel<T, 0, 2, 128, FUSED, true>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 256)
    return launch_rows(norm_bwd_kernel<T, 0, 2, 256, FUSED, true>, a, grid, sh.nt, smem, s);
  if (sh.nt <= 512)
    return launch_rows(norm_bwd_kernel<T, 0, 2, 512, FUSED, true>, a, grid, sh.nt, smem, s);
  return launch_rows(norm_bwd_kernel<T, 0, 2, 1024, FUSED, false>, a, grid, sh.nt, smem, s);
}

template <typename WT>
cudaError_t join(int64_t cols, int parts, const float* part, void* dweight, void* dbias,
                 cudaStream_t s) {
  return launch_k(norm_join_kernel<WT>, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, s, true,
                  cols, parts, part, static_cast<WT*>(dweight), static_cast<WT*>(dbias));
}

template <typename F>
auto by_types(int dtype, int wdtype, F f) {
  if (dtype == MUON_BF16) {
    if (wdtype == MUON_BF16) return f(__nv_bfloat16(), __nv_bfloat16());
    return f(__nv_bfloat16(), float());
  }
  if (wdtype == MUON_BF16) return f(float(), __nv_bfloat16());
  return f(float(), float());
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
  } else if (dtype == MUON_BF16) {
    e = fused ? forward<__nv_bfloat16, true>(a, ph.chunks(), s)
              : forward<__nv_bfloat16, false>(a, ph.chunks(), s);
  } else {
    e = fused ? forward<float, true>(a, ph.chunks(), s) : forward<float, false>(a, ph.chunks(), s);
  }
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

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
  } else if (dtype == MUON_BF16) {
    e = fused ? backward<__nv_bfloat16, true>(a, ph.chunks(), &parts, s)
              : backward<__nv_bfloat16, false>(a, ph.chunks(), &parts, s);
  } else {
    e = fused ? backward<float, true>(a, ph.chunks(), &parts, s)
              : backward<float, false>(a, ph.chunks(), &parts, s);
  }
  if (e == cudaSuccess && cols_wanted)
    e = wdtype == MUON_BF16 ? join<__nv_bfloat16>(cols, parts, a.part, dweight, dbias, s)
                            : join<float>(cols, parts, a.part, dweight, dbias, s);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
