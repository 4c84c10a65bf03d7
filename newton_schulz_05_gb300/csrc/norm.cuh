// Layer norm, alone or behind dropout and the residual add (norm.cu), and its
// gradient with the reduction of the weight's and the bias's (norm_grad.cu):
// what the two share.
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
#pragma once

#include <cmath>

#include "chunk.cuh"
#include "common.cuh"
#include "internal.h"
#include "random.cuh"

namespace muon {

namespace {

constexpr int kNormThreads = 256;    // of the kernels for rows longer than a block holds
constexpr int kSMs = 152;
constexpr int kRingDepth = 4;        // rows in flight per block, when shared memory allows
constexpr size_t kRingBytes = 220u << 10;   // shared memory of an SM given to rings

// ------------------------------------------------------------ chunks of rows

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

// REG (regular): every chunk of every row lies wholly inside the row or wholly
// past its end, so one comparison says which.  Otherwise a chunk may begin
// ahead of the row, end past it, or (operands of different phases) be read
// element by element.
template <bool REG>
__device__ __forceinline__ bool whole(int c0, int cols) {
  return REG ? c0 < cols : c0 >= 0 && c0 + 8 <= cols;
}
__device__ __forceinline__ bool inside(int c, int cols) { return c >= 0 && c < cols; }

// Start the copy of the chunk at p, column c0 of its row, into slot[0],
// slot[stride].  Bytes past the row are not read; bytes ahead of it are, when
// they lie inside the tensor (from `base`), and masked later.
template <typename T, bool REG>
__device__ __forceinline__ void fetch(uint4* slot, int stride, const T* p, const T* base, int c0,
                                      int cols) {
  constexpr int per = 8 / kPieces<T>;
  if (whole<REG>(c0, cols)) {
    #pragma unroll
    for (int q = 0; q < kPieces<T>; ++q) copy16(slot + q * stride, p + q * per);
  } else if (!REG && p >= base) {
    #pragma unroll
    for (int q = 0; q < kPieces<T>; ++q) {
      const int left = cols - c0 - q * per;
      if (left > 0)
        copy16(slot + q * stride, p + q * per, (left < per ? left : per) * (int)sizeof(T));
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
template <typename T, bool REG>
__device__ __forceinline__ void take(Chunk& c, const uint4* slot, int stride, const T* p,
                                     const T* base, int c0, int cols, bool vec) {
  if (REG) {
    if (c0 < cols) unpack(slot, stride, c, T());
    else clear(c);
  } else if (vec && whole<REG>(c0, cols)) {
    unpack(slot, stride, c, T());
  } else if (vec && p >= base && c0 < cols) {
    unpack(slot, stride, c, T());
    #pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!inside(c0 + j, cols)) elem(c, j) = 0.f;
  } else {
    #pragma unroll
    for (int j = 0; j < 8; ++j) elem(c, j) = inside(c0 + j, cols) ? to_f(p[j]) : 0.f;
  }
}

template <typename T, bool REG>
__device__ __forceinline__ void put(T* p, int c0, int cols, Chunk& c, bool vec) {
  if (REG) {
    if (c0 < cols) store8(p, c);
  } else if (vec && whole<REG>(c0, cols)) {
    store8(p, c);
  } else {
    #pragma unroll
    for (int j = 0; j < 8; ++j)
      if (inside(c0 + j, cols)) p[j] = from_f<T>(elem(c, j));
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

// Row visits of a thread's row group: `mine` of its own, `all` of the block's
// longest group.
struct Visits { int64_t first, step; int mine, all; };
template <int TPR>
__device__ __forceinline__ Visits visits(const Place<TPR>& at, int64_t rows) {
  Visits v;
  v.step = (int64_t)gridDim.x * at.rows;
  v.first = (int64_t)blockIdx.x * at.rows + at.g;
  v.mine = v.first < rows ? (int)((rows - 1 - v.first) / v.step) + 1 : 0;
  v.all = (int)((rows - 1 - (int64_t)blockIdx.x * at.rows) / v.step) + 1;
  return v;
}

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

// --------------------------------------------------------------------- host

// blocks of NT threads an SM, which caps their registers
constexpr int fwd_blocks(int tpr, int c, int nt) {
  return nt <= 128 ? 6 : nt <= 256 ? (tpr == 32 && c == 2 ? 2 : 3) : 1;
}
constexpr int bwd_blocks(int nt) { return nt <= 128 ? 4 : nt <= 256 ? 2 : 1; }

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
  return {0, 2, nt, backward ? bwd_blocks(nt) : fwd_blocks(0, 2, nt)};
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
  // every chunk wholly inside or past its row
  bool regular() const { return same && phase == 0 && ld == 0 && cols % 8 == 0; }
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
