// Layer norm, alone or behind dropout and the residual add (norm.cu), and its
// gradient with the reduction of the weight's and the bias's (norm_grad.cu):
// what the two share.
//
// Both passes are bound by HBM: forward reads x (and the residual) and writes
// y (and the sum) once, backward reads dy, the sum (and dsum) and writes dx
// (and dresidual) once.  A row lives in the registers of 8 lanes, a warp, or a
// group of warps (by its length), so its statistics take no second trip to
// memory: the mean first, then the centred squares, both over registers in
// fp32.
//
// Layout.  A row is cut into 16-byte pieces that are aligned in memory, not in
// the row: a row that starts `phase` elements past an aligned address has its
// first piece begin `phase` elements early, and what falls outside the row is
// masked.  So rows of odd width move in 16-byte accesses too.  Neighbouring
// threads take neighbouring pieces, and a thread takes the same pieces of every
// row it visits (row steps are multiples of eight, which keeps the phase), so
// weights stay in registers and the column sums of the gradient accumulate
// there.  Operands whose phases differ, or whose first row is not aligned, take the
// kernels for rows longer than a block holds, which move single elements then:
// 12 to 13% of the copy rate at 16381 bf16 columns, 22 to 42% for long rows of
// whole eights.
//
// Rows stream through a ring of asynchronous copies into shared memory.  Each
// thread copies, waits for and reads only its own pieces, so the ring needs no
// barrier; its depth holds enough bytes in flight to cover the HBM latency
// while a row is reduced.
#pragma once

#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "pieces.cuh"
#include "random.cuh"

namespace muon {

namespace {

constexpr int kNormThreads = 512;    // of the kernels for rows longer than a block holds
constexpr int kSMs = 152;

// ------------------------------------------------------------ pieces of rows

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
// until at most N of the newest groups are in flight
template <int N> __device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Which of a thread's E elements are inside the row: bit j for column c0 + j.
// REG (regular): every piece of every row lies wholly inside the row or wholly
// past its end.  Otherwise a piece may begin ahead of the row or end past it.
template <int E> constexpr uint32_t kFull = (1u << E) - 1;
template <int E, bool REG> __device__ __forceinline__ uint32_t inside(int c0, int cols) {
  if (REG) return c0 < cols ? kFull<E> : 0u;
  if (c0 >= cols || c0 + E <= 0) return 0u;
  const uint32_t tail = cols - c0 < E ? (1u << (cols - c0)) - 1 : kFull<E>;
  return c0 < 0 ? tail & (kFull<E> << -c0) : tail;
}

// Start the copy of the piece at p.  Bytes past the row are not read and arrive
// as zeros; bytes ahead of it are read (they lie inside the tensor, whose first
// row begins at an aligned address) and masked when the piece is taken.
template <typename T, bool REG>
__device__ __forceinline__ void fetch(uint4* slot, const T* p, uint32_t in) {
  if (!REG) copy16(slot, p, (32 - __clz(in)) * (int)sizeof(T));
  else if (in) copy16(slot, p);
}

// A thread's first piece ANDed with this has nothing from ahead of the row
template <typename T, bool REG> __device__ __forceinline__ uint4 front_mask(int c0) {
  uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
  if (!REG && c0 < 0) {
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ahead = -c0 * (int)sizeof(T) - 4 * j;      // bytes of word j
      w[j] = ahead >= 4 ? 0u : ahead > 0 ? ~0u << 8 * ahead : ~0u;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The piece in fp32, zeros outside the row
template <typename T, bool REG>
__device__ __forceinline__ void take(Piece<kEl<T>>& v, const uint4* slot, uint32_t in, bool first,
                                     const uint4& front) {
  if (REG && !in) {
    clear(v);
    return;
  }
  uint4 u = *slot;
  if (!REG && first) {
    u.x &= front.x;
    u.y &= front.y;
    u.z &= front.z;
    u.w &= front.w;
  }
  widen(v, u);
}

template <typename T, bool REG>
__device__ __forceinline__ void put(T* p, Piece<kEl<T>>& v, uint32_t in) {
  if (in == kFull<kEl<T>>) {
    *reinterpret_cast<uint4*>(p) = narrow(v);
  } else if (!REG && in) {
    if constexpr (sizeof(T) == 2) {
      const uint4 u = narrow(v);         // the piece's words are aligned
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      #pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t two = in >> 2 * j & 3;
        if (two == 3) reinterpret_cast<uint32_t*>(p)[j] = w[j];
        else if (two) reinterpret_cast<uint16_t*>(p)[2 * j + (two >> 1)] = (uint16_t)(two == 2 ? w[j] >> 16 : w[j]);
      }
    } else {
      #pragma unroll
      for (int j = 0; j < kEl<T>; ++j)
        if (in >> j & 1) p[j] = from_f<T>(elem(v, j));
    }
  }
}

// weight (or bias) of the piece's columns; `none` where there is no vector.
// `vec`: the vector is 16-byte aligned.
template <typename T, bool REG>
__device__ __forceinline__ void columns(Piece<kEl<T>>& v, const void* w, int bf16, int c0,
                                        uint32_t in, float none, bool vec) {
  constexpr int E = kEl<T>;
  #pragma unroll
  for (int j = 0; j < E / 2; ++j) v.v[j] = both(none);
  if (!w) return;
  if (REG && vec) {
    if (!in) return;
    if (bf16) {
      const uint2* q = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(w) + c0);
      #pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        const uint2 u = q[j];
        v.v[2 * j] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
        v.v[2 * j + 1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
      }
    } else {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(w) + c0);
      #pragma unroll
      for (int j = 0; j < E / 4; ++j) {
        const float4 u = q[j];
        v.v[2 * j] = make_float2(u.x, u.y);
        v.v[2 * j + 1] = make_float2(u.z, u.w);
      }
    }
    return;
  }
  #pragma unroll
  for (int j = 0; j < E; ++j)
    if (in >> j & 1)
      elem(v, j) = bf16 ? to_f(static_cast<const __nv_bfloat16*>(w)[c0 + j])
                        : static_cast<const float*>(w)[c0 + j];
}

// Sum over the threads of a row (TPR lanes, or the block where TPR is 0), the
// same value in each; slots: one float a warp, zeros past the last.
// SHORT: the warps' sums are added by shuffles, in fewer instructions but more
// latency than four at a time from shared memory.  It pays for 16-bit rows, which
// have the more instructions a byte, of more than 16 warps: [4096, 11008] 36.1
// against 39.0 us, [4096, 16384] 50.5 against 63.3, [8192, 10240] behind dropout 118
// against 125; at 16 warps ([8192, 8192]) 54.2 against 53.0, for fp32 [4096, 10240]
// 56.7 against 53.3.
template <int TPR, bool SHORT>
__device__ __forceinline__ float row_sum(float v, float* slots, int warps) {
  #pragma unroll
  for (int o = (TPR == 0 ? 32 : TPR) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR == 0) {
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    if (SHORT && warps > 16) {
      v = slots[threadIdx.x & 31];
      #pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    } else {
      v = 0.f;
      #pragma unroll 8
      for (int i = 0; i < warps; i += 4) {
        const float4 f = *reinterpret_cast<const float4*>(slots + i);
        v += (f.x + f.y) + (f.z + f.w);
      }
    }
  }
  return v;
}

// Row visits of a thread's row group: `mine` of its own, `all` of the block's
// longest group.
struct Visits { int64_t first, step; int mine, all; };
__device__ __forceinline__ Visits visits(int groups, int g, int64_t rows) {
  Visits v;
  v.step = (int64_t)gridDim.x * groups;
  v.first = (int64_t)blockIdx.x * groups + g;
  v.mine = v.first < rows ? (int)((rows - 1 - v.first) / v.step) + 1 : 0;
  v.all = (int)((rows - 1 - (int64_t)blockIdx.x * groups) / v.step) + 1;
  return v;
}

// Eight columns of a long row: `left` of them inside it.  VEC: whole, aligned
// eights; else single elements.
template <bool VEC, typename T>
__device__ __forceinline__ void load8(Piece<8>& v, const T* p, int64_t left) {
  if constexpr (VEC && sizeof(T) == 2) {
    widen(v, *reinterpret_cast<const uint4*>(p));
  } else if constexpr (VEC) {
    #pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float4 u = reinterpret_cast<const float4*>(p)[q];
      v.v[2 * q] = make_float2(u.x, u.y);
      v.v[2 * q + 1] = make_float2(u.z, u.w);
    }
  } else {
    #pragma unroll
    for (int j = 0; j < 8; ++j) elem(v, j) = j < left ? to_f(p[j]) : 0.f;
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, Piece<8>& v, int64_t left) {
  if constexpr (VEC && sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) = narrow(v);
  } else if constexpr (VEC) {
    #pragma unroll
    for (int q = 0; q < 2; ++q)
      reinterpret_cast<float4*>(p)[q] =
          make_float4(v.v[2 * q].x, v.v[2 * q].y, v.v[2 * q + 1].x, v.v[2 * q + 1].y);
  } else {
    #pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) p[j] = from_f<T>(elem(v, j));
  }
}
// weight or bias of eight columns; `none` where there is no vector.  vec: the
// vector is aligned
template <bool VEC, typename WT>
__device__ __forceinline__ void weight8(Piece<8>& v, const WT* p, int64_t c, int64_t cols, float none,
                                        bool vec) {
  if (VEC && vec && p) {
    load8<true>(v, p + c, 8);
  } else {
    #pragma unroll
    for (int j = 0; j < 8; ++j) elem(v, j) = p && c + j < cols ? to_f(p[c + j]) : none;
  }
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

// rows in flight in a block's ring: as many as an SM's shared memory gives each
// of its blocks, at most four
__host__ __device__ constexpr int ring_depth(int nt, int c, int es, int ops, int per_sm, int extra) {
  const int row = nt * c * 8 * es * ops;
  const int room = (220 << 10) / per_sm - extra;
  return room / row < 1 ? 1 : room / row > 4 ? 4 : room / row;
}

constexpr int64_t kMaxChunks = 2048;     // eights of elements of the longest row a block holds
constexpr int kLongParts = 304;

inline int64_t blocks_for(int64_t rows, int groups, int per_sm) {
  const int64_t want = (rows + groups - 1) / groups;
  return want < kSMs * per_sm ? want : kSMs * per_sm;
}

bool misaligned(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

// The stride the kernels are given.  That of a single row has no meaning and is 0:
// a row group without a row of its own then takes the phase that the first row
// has, for which the layout was chosen, in its column sums.
inline int64_t row_stride(int64_t rows, int64_t ld) { return rows > 1 ? ld : 0; }

// Collects the phases of the operands' rows (in elements of a 16-byte piece):
// `same` while they all agree and every first row is aligned.
struct Phases {
  int64_t rows, cols;
  size_t es;
  bool same = true, any = false;
  int ld = 0;
  void add(const void* p, int64_t stride) {
    if (!p) return;
    const int last = (int)(16 / es) - 1;
    const int f = (int)(reinterpret_cast<uintptr_t>(p) / es & last);
    const int l = rows > 1 ? (int)(stride & last) : 0;
    if (f || (any && l != ld)) same = false;
    if (!any) { any = true; ld = l; }
  }
  // every piece wholly inside or past its row
  bool regular() const { return same && ld == 0 && cols % (int64_t)(16 / es) == 0; }
  // whole, aligned eights of elements
  bool eights() const { return regular() && cols % 8 == 0; }
  // eights of elements that the pieces of the longest row span
  int64_t chunks() const {
    const int64_t e = (int64_t)(16 / es);
    const int64_t most = ld ? e - 1 : 0;
    return ((cols + most + e - 1) / e * e + 7) / 8;
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

// smem: the same for every launch of the kernel
template <auto Kernel, typename A>
cudaError_t launch_rows(const A& a, int64_t grid, int nt, size_t smem, cudaStream_t s) {
  if (smem > 40u << 10) {     // 48 KB with the static part, without the attribute
    const cudaError_t e = allow_shared<Kernel>(smem);
    if (e != cudaSuccess) return e;
  }
  return launch_k(Kernel, dim3((unsigned)grid), dim3(nt), smem, s, true, a);
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
