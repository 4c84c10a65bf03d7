// Expert router: top-k choice, combine weights, per-expert counts and the
// balance loss of a token batch, and the gradient of weights and loss.
//
// A token's logits live in the registers of G lanes, eight consecutive experts
// a lane (two or four times eight for more than 256 experts), so one warp takes
// 32 / G tokens at once and every reduction over experts is log2 G shuffles.  An
// expert stays with its lane for all of a warp's tokens: probabilities add up
// in registers, and the gradient's per-expert factors are loaded once.
//
// The choice.  Logits map to unsigned keys of the same order, and a key and the
// complement of its index share a word (sixteen bits each for bf16, 32 for
// fp32), so one unsigned maximum settles value and tie.  Each lane sorts its
// eight words once; a pick is then the largest head of the G lists, whose owner
// drops it.  From 48 Ki tokens on a lane takes a whole token instead
// (route_rows_kernel).
//
// Both passes read the logits once from HBM.  The forward pass of [131072, 64] bf16,
// k = 6, takes 21.3 us where its 23 MB would take 3.4.  No pipe is full (issue 62%,
// integer pipe 53%, 38% of the warps active): a lane waits on its own chain of copy,
// sort and merge; a join of the blocks' partial sums costs 3 us of that and of every
// call of more than one block.  The gradient comes nearer HBM: [65537, 160] fp32,
// k = 8, 18.3 us, 4.8 TB/s.
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "pieces.cuh"

namespace muon {

namespace {

constexpr int kRouteThreads = 512;
constexpr int kRouteWarps = kRouteThreads / 32;
constexpr int kRouteParts = 152 * 2;  // blocks of a pass, partial sums of the forward one
constexpr int kJoinExperts = 8;       // experts of a block of the join
constexpr int kRouteMaxExperts = 1024;
constexpr int kRouteMaxK = 32;
constexpr uint32_t kAll = 0xffffffffu;

struct RouteFwd {
  int64_t tokens, ld;
  int experts, k, normalize;
  int vec;              // rows of whole, aligned chunks
  int wide;             // weights and index are 16-byte aligned
  const void* logits;
  const uint8_t* mask;
  float* weights;
  int32_t* index;
  float* part_p;        // [parts][experts]
  int32_t* part_c;      // [parts][experts + 1]
  unsigned* ticket;     // zeroed here for the join
  int32_t* counts;      // written here when one block does it all
  float *mean_prob, *loss;
};

struct RouteJoin {
  int experts, k, parts;
  const float* part_p;
  const int32_t* part_c;
  int32_t* counts;
  float *mean_prob, *loss;
  float* part_loss;     // one a block
  unsigned* ticket;
};

struct RouteBwd {
  int64_t tokens, ld;
  int experts, k, normalize;
  int vec;
  const void* logits;
  const uint8_t* mask;
  const int32_t *index, *counts;
  const float *dweights, *dloss;
  void* dlogits;
};

// 16-byte pieces of eight logits, as loaded, and the eight in fp32
template <typename T> constexpr int kPieces = 8 / kEl<T>;
__device__ __forceinline__ void widen8(float (&v)[8], const uint4 (&u)[1]) {
  Piece<8> p;
  widen(p, u[0]);
  #pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = elem(p, j);
}
__device__ __forceinline__ void widen8(float (&v)[8], const uint4 (&u)[2]) {
  const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
  #pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
}

// A key whose unsigned order is the order of the logits; 0 is below every
// key.  Adding 0 turns -0 into +0 and every NaN into the canonical positive
// one, which ranks above +inf.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;   // order_key(-inf)
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// exp(v - top) as 2^x, x = (v - top) log2 e.  The difference, the product and log2 e
// are rounded to 24 bits, each of which moves the result by up to |v - top| 2^-24 of
// itself (bf16 logits: the difference is mostly exact), and 2^x adds two units: 7 units
// at 8 below the top, 15 at 20 below.  Below 2^-126 the result is 0.
__device__ __forceinline__ float exp_below(float v, float top) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((v - top) * 1.4426950408889634f));
  return y;
}

// Sum or maximum over the G lanes of a token
template <int G> __device__ __forceinline__ float group_sum(float v) {
  #pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int G> __device__ __forceinline__ uint32_t group_max(uint32_t v) {
  if constexpr (G == 32) return __reduce_max_sync(kAll, v);
  #pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int G> __device__ __forceinline__ unsigned long long group_max(unsigned long long v) {
  if constexpr (G == 32) {
    const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
    return (unsigned long long)hi << 32 | lo;
  }
  #pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) {
    const unsigned long long x = __shfl_xor_sync(kAll, v, o);
    v = x > v ? x : v;
  }
  return v;
}

__device__ __forceinline__ float2 exp_below2(float2 v, float top) {
  const float2 x = mul2(add2(v, both(-top)), both(1.4426950408889634f));
  float2 y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
  return y;
}

// Words that order logits and carry the expert, larger for the larger logit and
// for the lower index: key and complement of the index, sixteen bits each for
// bf16, 32 for fp32.
template <typename T> struct WordOf;
template <> struct WordOf<__nv_bfloat16> { using type = uint32_t; };
template <> struct WordOf<float> { using type = unsigned long long; };
template <typename T> using Word = typename WordOf<T>::type;

// of eight logits as loaded, experts e0, e0 + step, ...: two bf16 at a time
__device__ __forceinline__ void keys8(uint32_t (&k)[8], const uint4 (&u)[1], int e0, int step) {
  const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
  #pragma unroll
  for (int j = 0; j < 4; ++j) {
    // adding 0 turns -0 into +0 and a NaN into the canonical positive one
    uint32_t x;
    asm("{.reg .b32 z;\n mov.b32 z, 0;\n add.rn.bf16x2 %0, %1, z;}" : "=r"(x) : "r"(w[j]));
    // a set sign flips all sixteen bits, a clear one the sign alone
    x ^= ((x >> 15) & 0x00010001u) * 0x7fffu | 0x80008000u;
    k[2 * j] = x * 65536u + (uint32_t)(0xffff - (e0 + 2 * j * step));
    k[2 * j + 1] = (x & 0xffff0000u) | (uint32_t)(0xffff - (e0 + (2 * j + 1) * step));
  }
}
__device__ __forceinline__ void keys8(unsigned long long (&k)[8], const uint4 (&u)[2], int e0,
                                      int step) {
  const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
  #pragma unroll
  for (int j = 0; j < 8; ++j)
    k[j] = (unsigned long long)order_key(__uint_as_float(w[j])) << 32 | (uint32_t)~(e0 + j * step);
}
// the logit's own key (a bf16 value's low sixteen bits are zeros, in the key's
// own sense) and the expert
__device__ __forceinline__ uint32_t key_of(uint32_t w) {
  return w & 0x80000000u ? w & 0xffff0000u : w | 0xffffu;
}
__device__ __forceinline__ uint32_t key_of(unsigned long long w) { return (uint32_t)(w >> 32); }
__device__ __forceinline__ int expert_of(uint32_t w) { return 0xffff - (int)(w & 0xffffu); }
__device__ __forceinline__ int expert_of(unsigned long long w) { return (int)~(uint32_t)w; }

// a, b = the larger, the smaller
__device__ __forceinline__ void exchange(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
__device__ __forceinline__ void exchange(unsigned long long& a, unsigned long long& b) {
  const bool s = b > a;
  const unsigned long long hi = s ? b : a;
  b = s ? a : b;
  a = hi;
}
// descending order in nineteen exchanges (two sorted fours and Batcher's
// odd-even merge)
template <typename W> __device__ __forceinline__ void sort8(W (&k)[8]) {
  exchange(k[0], k[1]); exchange(k[2], k[3]); exchange(k[4], k[5]); exchange(k[6], k[7]);
  exchange(k[0], k[2]); exchange(k[1], k[3]); exchange(k[4], k[6]); exchange(k[5], k[7]);
  exchange(k[1], k[2]); exchange(k[5], k[6]);
  exchange(k[0], k[4]); exchange(k[1], k[5]); exchange(k[2], k[6]); exchange(k[3], k[7]);
  exchange(k[2], k[4]); exchange(k[3], k[5]);
  exchange(k[1], k[2]); exchange(k[3], k[4]); exchange(k[5], k[6]);
}

// The candidates of one lane, a sorted list where there are eight: next() gives
// the largest word over the group that has not been given yet.
template <typename T, int G, int N> struct Choice {
  Word<T> k[N];
  // eight logits as loaded, experts e0, e0 + step, ...
  __device__ __forceinline__ void set(int c, const uint4 (&u)[kPieces<T>], int e0, int step) {
    Word<T> w[8];
    keys8(w, u, e0, step);
    #pragma unroll
    for (int j = 0; j < 8; ++j) k[c * 8 + j] = w[j];
  }
  __device__ __forceinline__ void order() {
    if constexpr (N == 8) sort8(k);
  }
  // `left` (known at compile time): picks that may still follow
  __device__ __forceinline__ Word<T> next(int left) {
    Word<T> head = k[0];
    if constexpr (N != 8) {
      #pragma unroll
      for (int j = 1; j < N; ++j) head = head > k[j] ? head : k[j];
    }
    const Word<T> win = group_max<G>(head);
    if constexpr (N == 8) {
      if (head == win) {
        #pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < left) k[j] = k[j + 1];
        if (left > 7) k[7] = 0;
      }
    } else {
      #pragma unroll
      for (int j = 0; j < N; ++j) k[j] = k[j] == win ? 0 : k[j];
    }
    return win;
  }
};

// A lane's logits of one token in flight, so that the next token's load while
// this one is worked on.  VEC: rows of whole, aligned 16-byte pieces, a lane's
// chunk of eight being eight consecutive experts; else single logits, the eight
// G experts apart, so that the lanes of a load are neighbours in memory all the
// same.  -inf where there is no expert; a token past the end or masked keeps
// what was there: its results are thrown away.
template <typename T, int G, int NCH, bool VEC> struct Logits {
  static constexpr int P = kPieces<T>, STEP = VEC ? 1 : G;
  uint4 u[VEC ? NCH : 1][P];
  uint32_t w[VEC ? 1 : NCH * 8];
  bool live;
  static __device__ __forceinline__ int first(int c, int gl) { return VEC ? (c * G + gl) * 8 : c * 8 * G + gl; }
  __device__ __forceinline__ void clear() {
    const uint32_t m = sizeof(T) == 2 ? (VEC ? 0xff80ff80u : 0xff80u) : 0xff800000u;
    if constexpr (VEC) {
      #pragma unroll
      for (int c = 0; c < NCH; ++c)
        #pragma unroll
        for (int q = 0; q < P; ++q) u[c][q] = make_uint4(m, m, m, m);
    } else {
      #pragma unroll
      for (int j = 0; j < NCH * 8; ++j) w[j] = m;
    }
  }
  __device__ __forceinline__ void load(const RouteFwd& a, int64_t t, int gl) {
    live = t < a.tokens && !(a.mask && !a.mask[t]);
    if (t >= a.tokens) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    #pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int e0 = first(c, gl);
      if constexpr (VEC) {
        if (e0 < a.experts) {
          #pragma unroll
          for (int q = 0; q < P; ++q) u[c][q] = __ldg(reinterpret_cast<const uint4*>(row + e0) + q);
        }
      } else {
        #pragma unroll
        for (int j = 0; j < 8; ++j)
          if (e0 + j * G < a.experts) w[c * 8 + j] = raw(row + e0 + j * G);
      }
    }
  }
  static __device__ __forceinline__ uint32_t raw(const __nv_bfloat16* p) {
    return __ldg(reinterpret_cast<const unsigned short*>(p));
  }
  static __device__ __forceinline__ uint32_t raw(const float* p) {
    return __ldg(reinterpret_cast<const unsigned*>(p));
  }
  __device__ __forceinline__ void get(uint4 (&to)[NCH][P]) const {
    #pragma unroll
    for (int c = 0; c < NCH; ++c)
      #pragma unroll
      for (int q = 0; q < P; ++q) {
        if constexpr (VEC) {
          to[c][q] = u[c][q];
        } else if constexpr (sizeof(T) == 2) {
          const uint32_t* x = w + c * 8;
          to[c][q] = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
        } else {
          const uint32_t* x = w + c * 8 + q * 4;
          to[c][q] = make_uint4(x[0], x[1], x[2], x[3]);
        }
      }
  }
};

// The end of a forward block: its probabilities (`sums` rows of `stride` floats
// to add up in order), counts sc and n routed tokens become its partial sums.  The
// whole block calls it, after a barrier.
__device__ __forceinline__ void finish(const RouteFwd& a, const float* sums, int rows, int stride,
                                       const int* sc, int n) {
  for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
    float p = 0.f;
    for (int i = 0; i < rows; ++i) p += sums[i * stride + e];
    a.part_p[(int64_t)blockIdx.x * a.experts + e] = p;
    a.part_c[(int64_t)blockIdx.x * (a.experts + 1) + e] = sc[e];
  }
  if (threadIdx.x == 0) a.part_c[(int64_t)blockIdx.x * (a.experts + 1) + a.experts] = n;
}
// The same where the block, of kRouteThreads, is the only one: they become the results.
__device__ __forceinline__ void finish_alone(const RouteFwd& a, const float* sums, int rows, int stride,
                                             const int* sc, int n) {
  __shared__ float red[kRouteWarps];
  const float fn = (float)(n > 0 ? n : 1);
  float l = 0.f;
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
    float p = 0.f;
    for (int i = 0; i < rows; ++i) p += sums[i * stride + e];
    p /= fn;
    a.counts[e] = sc[e];
    a.mean_prob[e] = p;
    l = fmaf((float)sc[e] / ((float)a.k * fn), p, l);
  }
  l = block_sum<kRouteThreads>(l, red);
  if (threadIdx.x == 0) {
    a.counts[a.experts] = n;
    *a.loss = (float)a.experts * l;
  }
}

// A token takes G lanes, NCH eights of experts a lane.
template <typename T, int G, int NCH, bool VEC>
__global__ void __launch_bounds__(kRouteThreads, NCH == 1 ? 2 : 1)
route_kernel(const __grid_constant__ RouteFwd a) {
  using Row = Logits<T, G, NCH, VEC>;
  constexpr int TPW = 32 / G, N = NCH * 8, E = G * N;
  constexpr int kStage = TPW * (E < kRouteMaxK ? E : kRouteMaxK);
  // warps whose sums are added side by side
  constexpr int kRows = E <= 256 ? kRouteWarps : 2;
  __shared__ float sp[kRows][E];
  __shared__ int sc[E + 1];
  __shared__ uint2 picks[kRouteWarps][kStage];     // the winning words, then weight and expert
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % G, grp = lane / G;
  for (int e = threadIdx.x; e <= E; e += kRouteThreads) sc[e] = 0;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  __syncthreads();
  float acc[N];
  #pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;
  int routed_count = 0;
  const int64_t stride = (int64_t)gridDim.x * kRouteWarps * TPW;
  const int64_t begin = ((int64_t)blockIdx.x * kRouteWarps + warp) * TPW;
  Row next;
  next.clear();
  next.load(a, begin + grp, gl);
  uint2* const mine = picks[warp] + grp * a.k;
  for (int64_t t0 = begin; t0 < a.tokens; t0 += stride) {
    const int64_t t = t0 + grp;
    const bool live = next.live;
    uint4 now[NCH][kPieces<T>];
    next.get(now);
    next.load(a, t + stride, gl);
    Choice<T, G, N> choice;
    #pragma unroll
    for (int c = 0; c < NCH; ++c) choice.set(c, now[c], Row::first(c, gl), Row::STEP);
    choice.order();
    Word<T> most = 0;
    auto pick = [&](int p, int left) {
      const Word<T> win = choice.next(left);
      if (p == 0) most = win;
      if (gl == 0) *reinterpret_cast<Word<T>*>(mine + p) = win;
    };
    if (a.k <= 8) {
      #pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p < a.k) pick(p, 7 - p);
    } else {
      for (int p = 0; p < a.k; ++p) pick(p, 8);
    }
    const uint32_t first = key_of(most);
    const bool routed = live && first > kKeyNegInf;
    const float top = key_value(first);
    float v[N];
    float2 s2 = both(0.f);
    #pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float u[8];
      widen8(u, now[c]);
      #pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float2 e = exp_below2(make_float2(u[j], u[j + 1]), top);
        v[c * 8 + j] = e.x;
        v[c * 8 + j + 1] = e.y;
        s2 = add2(s2, e);
      }
    }
    const float total = group_sum<G>(s2.x + s2.y);
    if (routed) {
      const float inv = __frcp_rn(total);
      #pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = fmaf(v[j], inv, acc[j]);
      if (gl == 0) ++routed_count;
    }
    // the picks, a lane each
    __syncwarp();
    float picked = 0.f;
    for (int p = gl; p < a.k; p += G) {
      const Word<T> win = *reinterpret_cast<const Word<T>*>(mine + p);
      const uint32_t key = key_of(win);
      const bool ok = routed && key > kKeyNegInf;
      const int e = ok ? expert_of(win) : -1;
      const float y = ok ? exp_below(key_value(key), top) : 0.f;
      picked += y;
      mine[p] = make_uint2(__float_as_uint(y), (uint32_t)e);
      if (ok) atomicAdd(&sc[e], 1);
    }
    const float z = __frcp_rn(a.normalize ? group_sum<G>(picked) : total);
    if (t < a.tokens)
      for (int p = gl; p < a.k; p += G) {
        const uint2 x = mine[p];
        a.weights[t * a.k + p] = (int)x.y >= 0 ? __uint_as_float(x.x) * z : 0.f;
        a.index[t * a.k + p] = (int)x.y;
      }
    __syncwarp();
  }
  // the join may be set up while the sums are put together
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (routed_count) atomicAdd(&sc[E], routed_count);
  // the block's sums: lanes of a warp, then warps in order
  #pragma unroll
  for (int o = G; o < 32; o <<= 1)
    #pragma unroll
    for (int j = 0; j < N; ++j) acc[j] += __shfl_xor_sync(kAll, acc[j], o);
  for (int i = 0; i < kRouteWarps; i += kRows) {
    if (grp == 0 && warp >= i && warp < i + kRows) {
      #pragma unroll
      for (int j = 0; j < N; ++j) {
        float& to = sp[warp - i][Row::first(j / 8, gl) + (j % 8) * Row::STEP];
        to = i ? to + acc[j] : acc[j];
      }
    }
    __syncthreads();
  }
  if (gridDim.x > 1) finish(a, &sp[0][0], kRows, E, sc, sc[E]);
  else finish_alone(a, &sp[0][0], kRows, E, sc, sc[E]);
}

// Many tokens: a lane a token.  A warp copies 32 rows, 128 bytes of each at a
// time, into shared memory (rows 144 bytes apart, which spreads a column over
// the banks); each lane reads its own row in eights, sorts each eight, merges it
// into its K largest so far, and keeps a running maximum and sum of
// exponentials.  No lane waits for another, and a token takes 79 instructions of
// a warp where the lanes-a-token form takes about 110 (64 experts, k = 6).  Then
// the lanes take columns and add up the 32 tokens' probabilities; rows longer
// than a slice are read again for that, from L2.
constexpr int kSlice = 128, kSliceRow = kSlice + 16, kSliceBytes = 32 * kSliceRow;

// shared memory of a warp: slices, column sums, each token's maximum and
// reciprocal sum
__host__ __device__ constexpr int rows_warp_bytes(int slices, int experts_padded) {
  return (slices > 1 ? 2 : 1) * kSliceBytes + experts_padded * 4 + 32 * 8;
}

template <typename W, int K> struct Best {
  W k[K];      // descending
  __device__ __forceinline__ void clear() {
    #pragma unroll
    for (int j = 0; j < K; ++j) k[j] = 0;
  }
  // merge eight sorted words: the larger of each opposite pair are the K
  // largest of both, in bitonic order
  __device__ __forceinline__ void merge(const W (&c)[8]) {
    #pragma unroll
    for (int j = 0; j < K; ++j) k[j] = k[j] > c[K - 1 - j] ? k[j] : c[K - 1 - j];
    #pragma unroll
    for (int o = K / 2; o > 0; o >>= 1)
      #pragma unroll
      for (int j = 0; j < K; ++j)
        if (!(j & o)) exchange(k[j], k[j + o]);
  }
};

template <typename T, int K>
__global__ void __launch_bounds__(kRouteThreads, sizeof(T) == 2 ? 2 : 1)
route_rows_kernel(const __grid_constant__ RouteFwd a) {
  constexpr int P = kPieces<T>, SE = kSlice / (int)sizeof(T);    // experts of a slice
  extern __shared__ __align__(16) char smem[];
  __shared__ int sc[kRouteMaxExperts + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int slices = (a.experts + SE - 1) / SE, padded = slices * SE;
  char* const mine = smem + warp * rows_warp_bytes(slices, padded);
  const int buffers = slices > 1 ? 2 : 1;
  float* const col = reinterpret_cast<float*>(mine + buffers * kSliceBytes);
  float2* const stat = reinterpret_cast<float2*>(col + padded);
  for (int e = threadIdx.x; e <= a.experts; e += blockDim.x) sc[e] = 0;
  for (int e = lane; e < padded; e += 32) col[e] = 0.f;
  pdl_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  __syncthreads();
  const T* logits = static_cast<const T*>(a.logits);
  const int64_t tiles = (a.tokens + 31) / 32, stride = (int64_t)gridDim.x * warps;
  const int passes = slices > 1 ? 2 : 1;        // times a tile is read
  // the slice to copy next: tile, pass and slice
  int64_t ft = (int64_t)blockIdx.x * warps + warp;
  int fp = 0, fs = 0, fb = 0;
  auto start = [&] {
    if (ft < tiles) {
      char* to = mine + fb * kSliceBytes + (lane >> 3) * kSliceRow + (lane & 7) * 16;
      const int e0 = fs * SE + (lane & 7) * kEl<T>;
      const int64_t row = ft * 32 + (lane >> 3);
      const T* from = logits + row * a.ld + e0;
      #pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4* slot = reinterpret_cast<uint4*>(to + i * 4 * kSliceRow);
        if (e0 >= a.experts) {
          const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;    // -inf
          *slot = make_uint4(w, w, w, w);
        } else if (row + 4 * i < a.tokens) {
          const uint32_t s = (uint32_t)__cvta_generic_to_shared(slot);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(s), "l"(from + 4 * i * a.ld)
                       : "memory");
        }
      }
      if (++fs == slices) {
        fs = 0;
        if (++fp == passes) { fp = 0; ft += stride; }
      }
      if (++fb == buffers) fb = 0;
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  };
  int buffer = 0;
  if (buffers == 2) start();
  // the next slice in sequence, its successor under way
  auto arrive = [&]() -> const char* {
    __syncwarp();            // the buffer filled next has been read by all lanes
    start();
    if (buffers == 2) asm volatile("cp.async.wait_group 1;\n" ::: "memory");
    else asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncwarp();
    const char* b = mine + buffer * kSliceBytes;
    if (++buffer == buffers) buffer = 0;
    return b;
  };
  int routed_count = 0;
  for (int64_t tile = (int64_t)blockIdx.x * warps + warp; tile < tiles; tile += stride) {
    const int64_t t = tile * 32 + lane;
    const bool live = t < a.tokens && !(a.mask && !a.mask[t]);
    Best<Word<T>, K> best;
    best.clear();
    float top = -INFINITY, total = 0.f;
    const char* slice = nullptr;
    for (int s = 0; s < slices; ++s) {
      slice = arrive();
      const uint4* row = reinterpret_cast<const uint4*>(slice + lane * kSliceRow);
      #pragma unroll 2
      for (int c = 0; c < SE / 8; ++c) {
        uint4 u[P];
        #pragma unroll
        for (int q = 0; q < P; ++q) u[q] = row[c * P + q];
        Word<T> w[8];
        keys8(w, u, s * SE + c * 8, 1);
        sort8(w);
        best.merge(w);
        const float higher = max_nan(top, key_value(key_of(w[0])));
        const float at = higher == -INFINITY ? 0.f : higher;
        float v[8];
        widen8(v, u);
        float2 e = make_float2(total * exp_below(top, at), 0.f);
        #pragma unroll
        for (int j = 0; j < 8; j += 2) e = add2(e, exp_below2(make_float2(v[j], v[j + 1]), at));
        total = e.x + e.y;
        top = higher;
      }
    }
    const bool routed = live && top != -INFINITY;
    const float inv = __frcp_rn(total);
    // the picks
    float y[K];
    int x[K];
    float picked = 0.f;
    #pragma unroll
    for (int p = 0; p < K; ++p) {
      const uint32_t key = key_of(best.k[p]);
      const bool ok = routed && p < a.k && key > kKeyNegInf;
      x[p] = ok ? expert_of(best.k[p]) : -1;
      y[p] = ok ? exp_below(key_value(key), top) : 0.f;
      picked += y[p];
      if (ok) atomicAdd(&sc[x[p]], 1);
    }
    const float z = a.normalize ? __frcp_rn(picked) : inv;
    if (t < a.tokens) {
      float* w = a.weights + t * a.k;
      int32_t* ix = a.index + t * a.k;
      #pragma unroll
      for (int p = 0; p < K; ++p) y[p] = x[p] >= 0 ? y[p] * z : 0.f;
      if (K >= 4 && a.k % 4 == 0 && a.wide) {
        #pragma unroll
        for (int p = 0; p + 3 < K; p += 4)
          if (p < a.k) {
            *reinterpret_cast<float4*>(w + p) = make_float4(y[p], y[p + 1], y[p + 2], y[p + 3]);
            *reinterpret_cast<int4*>(ix + p) = make_int4(x[p], x[p + 1], x[p + 2], x[p + 3]);
          }
      } else if (a.k % 2 == 0 && a.wide) {
        #pragma unroll
        for (int p = 0; p + 1 < K; p += 2)
          if (p < a.k) {
            *reinterpret_cast<float2*>(w + p) = make_float2(y[p], y[p + 1]);
            *reinterpret_cast<int2*>(ix + p) = make_int2(x[p], x[p + 1]);
          }
      } else {
        #pragma unroll
        for (int p = 0; p < K; ++p)
          if (p < a.k) { w[p] = y[p]; ix[p] = x[p]; }
      }
    }
    // column sums of the tile's probabilities
    const uint32_t which = __ballot_sync(kAll, routed);
    routed_count += __popc(which);
    stat[lane] = make_float2(top, inv);
    __syncwarp();
    for (int s = 0; s < slices; ++s) {
      if (slices > 1) slice = arrive();
      float sum[4 / sizeof(T)] = {};
      auto add = [&](int i) {
        const float2 st = stat[i];
        const uint32_t u = *reinterpret_cast<const uint32_t*>(slice + i * kSliceRow + lane * 4);
        if constexpr (sizeof(T) == 2) {
          const float2 e = exp_below2(
              make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), st.x);
          sum[0] = fmaf(e.x, st.y, sum[0]);
          sum[1] = fmaf(e.y, st.y, sum[1]);
        } else {
          sum[0] = fmaf(exp_below(__uint_as_float(u), st.x), st.y, sum[0]);
        }
      };
      if (which == kAll) {
        #pragma unroll 8
        for (int i = 0; i < 32; ++i) add(i);
      } else {
        for (uint32_t m = which; m; m &= m - 1) add(__ffs(m) - 1);
      }
      #pragma unroll
      for (int j = 0; j < 4 / (int)sizeof(T); ++j) col[s * SE + lane * (4 / (int)sizeof(T)) + j] += sum[j];
    }
    __syncwarp();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int routed_tokens;
  if (threadIdx.x == 0) routed_tokens = 0;
  __syncthreads();
  if (lane == 0) atomicAdd(&routed_tokens, routed_count);
  __syncthreads();
  finish(a, reinterpret_cast<const float*>(smem + buffers * kSliceBytes), warps,
         rows_warp_bytes(slices, padded) / 4, sc, routed_tokens);
}

// Counts, mean probabilities and the loss from the blocks' partial sums: eight
// experts a block, 32 threads an expert; the block that finishes last adds up
// the blocks' shares of the loss in order.
__global__ void __launch_bounds__(256) route_join_kernel(const __grid_constant__ RouteJoin a) {
  __shared__ float red_p[8][kJoinExperts];
  __shared__ int red_c[8][kJoinExperts], red_n[8];
  __shared__ unsigned arrived;
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col = lane % kJoinExperts, row = threadIdx.x / kJoinExperts;
  const int e = blockIdx.x * kJoinExperts + col;
  float p = 0.f;
  int c = 0, n = 0;
  if (e < a.experts) {
    #pragma unroll 5
    for (int i = row; i < a.parts; i += 256 / kJoinExperts) {
      p += a.part_p[(int64_t)i * a.experts + e];
      c += a.part_c[(int64_t)i * (a.experts + 1) + e];
    }
  }
  for (int i = threadIdx.x; i < a.parts; i += 256) n += a.part_c[(int64_t)i * (a.experts + 1) + a.experts];
  n = __reduce_add_sync(kAll, n);
  #pragma unroll
  for (int o = kJoinExperts; o < 32; o <<= 1) {
    p += __shfl_xor_sync(kAll, p, o);
    c += __shfl_xor_sync(kAll, c, o);
  }
  if (lane < kJoinExperts) {
    red_p[warp][lane] = p;
    red_c[warp][lane] = c;
  }
  if (lane == 0) red_n[warp] = n;
  __syncthreads();
  if (warp != 0) return;
  n = 0;
  p = 0.f;
  c = 0;
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    n += red_n[i];
    p += red_p[i][col];
    c += red_c[i][col];
  }
  const float fn = (float)(n > 0 ? n : 1);
  p /= fn;
  const bool mine = lane < kJoinExperts && e < a.experts;
  if (mine) {
    a.counts[e] = c;
    a.mean_prob[e] = p;
  }
  if (blockIdx.x == 0 && lane == 0) a.counts[a.experts] = n;
  const float l = group_sum<32>(mine ? (float)c / ((float)a.k * fn) * p : 0.f);
  if (lane == 0) {
    a.part_loss[blockIdx.x] = l;
    __threadfence();
    arrived = atomicAdd(a.ticket, 1u);
  }
  __syncwarp();
  if (arrived == gridDim.x - 1) {
    __threadfence();
    float s = 0.f;
    for (int i = lane; i < (int)gridDim.x; i += 32) s += __ldcg(a.part_loss + i);
    s = group_sum<32>(s);
    if (lane == 0) *a.loss = (float)a.experts * s;
  }
}

// The gradient of a logit is p (b - dot + x): b the loss's gradient by the
// probability, x what the combine weights add at a picked expert, dot the sum
// over experts of p times the rest.  Unnormalised weights are probabilities, so
// x = dw and dot counts it.  Normalised ones are w = p / sum of the picks' p, so
// x = (dw - sum of w dw) / (sum of the picks' p), whose mean under p is zero.
//
// A token takes G lanes, piece k of lane l its experts (k G + l) E .. + E - 1
// (E = 8 bf16, 4 fp32: a 16-byte piece), NP pieces a lane; rows that are not
// whole, aligned pieces take single logits G experts apart instead, so that the
// lanes of an access are neighbours in memory all the same.  The next token's
// logits and picks are in flight while this one is worked on.
constexpr int kBwdThreads = 256, kBwdWarps = kBwdThreads / 32;
// blocks an SM, by the logits a lane holds: 64, 85 or 128 registers
__host__ __device__ constexpr int bwd_blocks(int n) { return n <= 8 ? 4 : n <= 16 ? 3 : 2; }

template <typename T, int G, int NP, bool VEC>
__global__ void __launch_bounds__(kBwdThreads, bwd_blocks(NP * kEl<T>))
route_bwd_kernel(const __grid_constant__ RouteBwd a) {
  constexpr int E = kEl<T>, TPW = 32 / G, N = NP * E, KS = 2;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % G, grp = lane / G;
  // x by expert, zeros between tokens
  float* const xx = reinterpret_cast<float*>(smem) + (warp * TPW + grp) * (G * N);
  for (int i = gl; i < G * N; i += G) xx[i] = 0.f;
  __syncwarp();
  pdl_wait();
  // expert j of piece k
  auto expert = [&](int k, int j) { return VEC ? (k * G + gl) * E + j : k * G * E + j * G + gl; };
  const T* logits = static_cast<const T*>(a.logits);
  const int routed_tokens = a.counts[a.experts];
  const float n = (float)(routed_tokens > 0 ? routed_tokens : 1);
  const float f = a.dloss ? *a.dloss * (float)a.experts / ((float)a.k * n) / n : 0.f;
  float2 b[N / 2];
  #pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = expert(j / E, j % E);
    const float v = e < a.experts ? f * (float)a.counts[e] : 0.f;
    if (j & 1) b[j / 2].y = v;
    else b[j / 2].x = v;
  }
  const int64_t stride = (int64_t)gridDim.x * kBwdWarps * TPW;
  const int64_t begin = ((int64_t)blockIdx.x * kBwdWarps + warp) * TPW;
  const uint32_t minus = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;    // -inf
  uint4 next[VEC ? NP : 1];
  uint32_t single[VEC ? 1 : N];
  bool live_next;
  int e_next[KS];
  float d_next[KS];
  if constexpr (VEC) {
    #pragma unroll
    for (int k = 0; k < NP; ++k) next[k] = make_uint4(minus, minus, minus, minus);
  } else {
    #pragma unroll
    for (int j = 0; j < N; ++j) single[j] = sizeof(T) == 2 ? 0xff80u : 0xff800000u;
  }
  auto load = [&](int64_t t) {
    const bool in = t < a.tokens;
    live_next = in && !(a.mask && !a.mask[t]);
    const T* row = logits + t * a.ld;
    #pragma unroll
    for (int k = 0; k < NP; ++k) {
      if constexpr (VEC) {
        if (in && expert(k, 0) < a.experts)
          next[k] = __ldg(reinterpret_cast<const uint4*>(row + expert(k, 0)));
      } else {
        #pragma unroll
        for (int j = 0; j < E; ++j)
          if (in && expert(k, j) < a.experts)
            single[k * E + j] = Logits<T, G, 1, false>::raw(row + expert(k, j));
      }
    }
    #pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int p = gl + s * G;
      e_next[s] = -1;
      d_next[s] = 0.f;
      if (a.dweights && p < a.k && in) {
        e_next[s] = a.index[t * a.k + p];
        d_next[s] = a.dweights[t * a.k + p];
      }
    }
  };
  load(begin + grp);
  for (int64_t t0 = begin; t0 < a.tokens; t0 += stride) {
    const int64_t t = t0 + grp;
    const T* row = logits + t * a.ld;
    const bool live = live_next;
    uint4 u[NP];
    int e[KS];
    float d[KS], l[KS];
    #pragma unroll
    for (int s = 0; s < KS; ++s) {
      e[s] = e_next[s];
      d[s] = d_next[s];
      if (!live || e[s] < 0 || e[s] >= a.experts) {
        e[s] = -1;
        d[s] = 0.f;              // whatever a missing pick's gradient holds
      }
      l[s] = e[s] >= 0 ? to_f(row[e[s]]) : -INFINITY;
    }
    #pragma unroll
    for (int k = 0; k < NP; ++k) {
      if constexpr (VEC) {
        u[k] = next[k];
      } else if constexpr (sizeof(T) == 2) {
        const uint32_t* x = single + k * E;
        u[k] = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
      } else {
        u[k] = make_uint4(single[k * E], single[k * E + 1], single[k * E + 2], single[k * E + 3]);
      }
    }
    load(t + stride);
    float2 v[N / 2];
    float best = -INFINITY;
    #pragma unroll
    for (int k = 0; k < NP; ++k) {
      Piece<E> w;
      widen(w, u[k]);
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        v[k * (E / 2) + j] = w.v[j];
        best = max_nan(best, max_nan(w.v[j].x, w.v[j].y));
      }
    }
    const float top = key_value(group_max<G>(order_key(best)));
    const bool routed = live && top != -INFINITY;
    float2 s2 = both(0.f);
    #pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      v[j] = exp_below2(v[j], top);
      s2 = add2(s2, v[j]);
    }
    const float total = group_sum<G>(s2.x + s2.y);
    if (a.dweights) {
      if (a.normalize) {
        float z = 0.f, wd = 0.f;
        #pragma unroll
        for (int s = 0; s < KS; ++s) {
          const float y = exp_below(l[s], top);
          z += e[s] >= 0 ? y : 0.f;
          wd += e[s] >= 0 ? y * d[s] : 0.f;
        }
        z = __frcp_rn(group_sum<G>(z));
        wd = group_sum<G>(wd) * z;
        z *= total;
        #pragma unroll
        for (int s = 0; s < KS; ++s) d[s] = (d[s] - wd) * z;
      }
      #pragma unroll
      for (int s = 0; s < KS; ++s)
        if (e[s] >= 0) xx[e[s]] = d[s];
      __syncwarp();
    }
    const float2 inv = both(__frcp_rn(total));
    // x of piece k
    auto added = [&](int k, float2 (&x)[E / 2]) {
      if constexpr (VEC) {
        #pragma unroll
        for (int q = 0; q < E / 4; ++q) {
          const float4 w = *reinterpret_cast<const float4*>(xx + expert(k, q * 4));
          x[2 * q] = make_float2(w.x, w.y);
          x[2 * q + 1] = make_float2(w.z, w.w);
        }
      } else {
        #pragma unroll
        for (int j = 0; j < E / 2; ++j)
          x[j] = make_float2(xx[expert(k, 2 * j)], xx[expert(k, 2 * j + 1)]);
      }
    };
    float2 dot2 = both(0.f);
    #pragma unroll
    for (int k = 0; k < NP; ++k) {
      float2 x[E / 2];
      if (!a.normalize) added(k, x);
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        float2& p = v[k * (E / 2) + j];
        const float2 bj = b[k * (E / 2) + j];
        p = mul2(p, inv);
        dot2 = fma2(p, a.normalize ? bj : add2(x[j], bj), dot2);
      }
    }
    const float2 minus_dot = both(-group_sum<G>(dot2.x + dot2.y));
    #pragma unroll
    for (int k = 0; k < NP; ++k) {
      float2 x[E / 2];
      added(k, x);
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        float2& p = v[k * (E / 2) + j];
        p = mul2(p, add2(add2(x[j], b[k * (E / 2) + j]), minus_dot));
      }
    }
    if (t < a.tokens) {
      T* out = static_cast<T*>(a.dlogits) + t * a.experts;
      #pragma unroll
      for (int k = 0; k < NP; ++k) {
        Piece<E> w;
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) w.v[j] = v[k * (E / 2) + j];
        if (!routed) clear(w);
        if constexpr (VEC) {
          if (expert(k, 0) < a.experts) *reinterpret_cast<uint4*>(out + expert(k, 0)) = narrow(w);
        } else {
          #pragma unroll
          for (int j = 0; j < E; ++j)
            if (expert(k, j) < a.experts) out[expert(k, j)] = from_f<T>(elem(w, j));
        }
      }
    }
    if (a.dweights) {
      __syncwarp();
      #pragma unroll
      for (int s = 0; s < KS; ++s)
        if (e[s] >= 0) xx[e[s]] = 0.f;
      __syncwarp();
    }
  }
}

// lanes a token
int lanes_of(int experts) {
  int g = 1;
  while (g < 32 && g * 8 < experts) g *= 2;
  return g;
}

// Tokens from which the lane-a-token form is taken.  Its 32 tokens are one warp's
// serial work, so it pays once every SM has many warps: 64 experts, k = 6, bf16
// took 9.0 against 6.7 us at 4096 tokens, 11.3 against 11.8 at 32768 and 21.9
// against 25.0 at 131072; 256 experts, k = 8, fp32 28 against 20 at 16384 and 38
// against 33 at 32768; 160 experts at 65537 42 against 60.
constexpr int64_t kRowsTokens = 49152;
static_assert((kRowsTokens + 31) / 32 > kRouteWarps, "the lane-a-token form has several blocks");

// blocks of a pass: a warp for every token group, up to two blocks an SM (the
// lane-a-token form has fewer groups)
int route_blocks(int64_t tokens, int experts) {
  const int per = kRouteWarps * 32 / lanes_of(experts);
  const int64_t b = (tokens + per - 1) / per;
  return (int)(b < 1 ? 1 : b < kRouteParts ? b : kRouteParts);
}

int join_blocks(int experts) { return (experts + kJoinExperts - 1) / kJoinExperts; }

bool misaligned(const void* p, size_t es) { return reinterpret_cast<uintptr_t>(p) % es != 0; }

muon_status check_route(int64_t tokens, int experts, int k, int dtype, int64_t ld) {
  if (tokens < 0 || k < 1 || ld < 0) return MUON_ERR_INVALID_ARG;
  if (experts < 1 || experts > kRouteMaxExperts || k > kRouteMaxK || k > experts ||
      tokens > 0x7fffffff / k)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  if (dtype != MUON_BF16 && dtype != MUON_F32) return MUON_ERR_DTYPE;
  return MUON_OK;
}

// every row of p in whole, 16-byte aligned chunks
bool whole_rows(const void* p, int64_t tokens, int64_t ld, int experts, size_t es) {
  return experts % 8 == 0 && reinterpret_cast<uintptr_t>(p) % 16 == 0 &&
         (tokens <= 1 || (size_t)ld * es % 16 == 0);
}

// workspace: ticket and shares of the loss, counts, probabilities
constexpr size_t kJoinBytes = 1024;
int64_t most_blocks(int64_t tokens, int experts) {     // of either form
  return tokens >= kRowsTokens ? kRouteParts : route_blocks(tokens, experts);
}
size_t probs_offset(int64_t tokens, int experts) {
  return kJoinBytes +
         ((size_t)most_blocks(tokens, experts) * (experts + 1) * sizeof(int32_t) + 255) / 256 * 256;
}

template <typename F>
cudaError_t by_experts(int dtype, int experts, F f) {
  auto pick = [&](auto t) -> cudaError_t {
    using T = decltype(t);
    if (experts <= 8) return f.template operator()<T, 1, 1>();
    if (experts <= 16) return f.template operator()<T, 2, 1>();
    if (experts <= 32) return f.template operator()<T, 4, 1>();
    if (experts <= 64) return f.template operator()<T, 8, 1>();
    if (experts <= 128) return f.template operator()<T, 16, 1>();
    if (experts <= 256) return f.template operator()<T, 32, 1>();
    if (experts <= 512) return f.template operator()<T, 32, 2>();
    return f.template operator()<T, 32, 4>();
  };
  return dtype == MUON_BF16 ? pick(__nv_bfloat16()) : pick(float());
}

struct LaunchFwd {
  const RouteFwd& a;
  int blocks;
  cudaStream_t s;
  template <typename T, int G, int NCH> cudaError_t operator()() const {
    return launch_k(a.vec ? route_kernel<T, G, NCH, true> : route_kernel<T, G, NCH, false>, dim3(blocks),
                    dim3(kRouteThreads), 0, s, true, a);
  }
};

template <typename T, int K>
cudaError_t launch_rows_k(const RouteFwd& a, int blocks, int warps, cudaStream_t s) {
  constexpr int SE = kSlice / (int)sizeof(T);
  const int slices = (a.experts + SE - 1) / SE;
  const size_t smem = (size_t)warps * rows_warp_bytes(slices, slices * SE);
  const cudaError_t e = allow_shared<route_rows_kernel<T, K>>(
      kRouteWarps * rows_warp_bytes(2, 512));       // of the most warps and experts
  if (e != cudaSuccess) return e;
  return launch_k(route_rows_kernel<T, K>, dim3(blocks), dim3(32 * warps), smem, s, true, a);
}
template <typename T>
cudaError_t launch_rows(const RouteFwd& a, int blocks, int warps, cudaStream_t s) {
  return a.k <= 2 ? launch_rows_k<T, 2>(a, blocks, warps, s)
       : a.k <= 4 ? launch_rows_k<T, 4>(a, blocks, warps, s) : launch_rows_k<T, 8>(a, blocks, warps, s);
}

// Blocks and warps a block of the lane-a-token form: the tiles of 32 tokens are
// spread evenly, over two blocks an SM where their shared memory allows (a
// slice a row), else one.
void rows_grid(int64_t tokens, int experts, size_t es, int* blocks, int* warps) {
  const int64_t tiles = (tokens + 31) / 32;
  const int most = (size_t)experts * es <= kSlice ? kRouteParts : kRouteParts / 2;
  const int64_t w = (tiles + most - 1) / most;
  *warps = (int)(w < kRouteWarps ? w : kRouteWarps);
  const int64_t b = (tiles + *warps - 1) / *warps;
  *blocks = (int)(b < most ? b : most);
}

// the lane-a-token form: rows of whole, aligned 16-byte pieces, up to eight
// picks, and column sums that fit beside the slices in shared memory
bool rows_form(int64_t tokens, int experts, int k, const void* p, int64_t ld, size_t es) {
  return tokens >= kRowsTokens && k <= 8 && experts <= 512 && experts % (16 / es) == 0 &&
         reinterpret_cast<uintptr_t>(p) % 16 == 0 && (size_t)ld * es % 16 == 0;
}

template <typename T, int G, int NP, bool VEC>
cudaError_t launch_bwd(const RouteBwd& a, cudaStream_t s) {
  const size_t smem = (size_t)kBwdWarps * 32 * NP * kEl<T> * sizeof(float);
  if (smem > 48u << 10) {
    const cudaError_t e = allow_shared<route_bwd_kernel<T, G, NP, VEC>>(smem);
    if (e != cudaSuccess) return e;
  }
  const int per = kBwdWarps * 32 / G;
  const int64_t want = (a.tokens + per - 1) / per;
  const int64_t most = 152 * bwd_blocks(NP * kEl<T>);
  return launch_k(route_bwd_kernel<T, G, NP, VEC>, dim3((unsigned)(want < most ? want : most)),
                  dim3(kBwdThreads), smem, s, true, a);
}
template <typename T, int G, int NP> cudaError_t launch_bwd(const RouteBwd& a, cudaStream_t s) {
  return a.vec ? launch_bwd<T, G, NP, true>(a, s) : launch_bwd<T, G, NP, false>(a, s);
}

// Lanes a token: the fewest that leave a lane at most two picks and twenty fp32
// or 24 bf16 logits (more only where 32 lanes leave more), so that a warp has
// many tokens and few lanes idle.
template <typename T, int G> cudaError_t bwd_pieces(const RouteBwd& a, cudaStream_t s) {
  constexpr int kMost = sizeof(T) == 2 ? 3 : 5;
  const int pieces = (a.experts + kEl<T> - 1) / kEl<T>, np = (pieces + G - 1) / G;
  if constexpr (G < 32) {
    if (np > kMost || 2 * G < a.k) return bwd_pieces<T, 2 * G>(a, s);
  }
  switch (np) {
    case 1: return launch_bwd<T, G, 1>(a, s);
    case 2: return launch_bwd<T, G, 2>(a, s);
    case 3: return launch_bwd<T, G, 3>(a, s);
  }
  if constexpr (sizeof(T) == 4) {
    if (np == 4) return launch_bwd<T, G, 4>(a, s);
    if (np == 5) return launch_bwd<T, G, 5>(a, s);
    if constexpr (G == 32) return np <= 6 ? launch_bwd<T, G, 6>(a, s) : launch_bwd<T, G, 8>(a, s);
  } else if constexpr (G == 32) {
    return launch_bwd<T, G, 4>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_route_workspace_bytes(int64_t tokens, int experts, size_t* out) {
  if (!out || tokens < 0) return MUON_ERR_INVALID_ARG;
  if (experts < 1 || experts > kRouteMaxExperts) return MUON_ERR_UNSUPPORTED_SHAPE;
  *out = probs_offset(tokens, experts) +
         (size_t)most_blocks(tokens, experts) * experts * sizeof(float);
  return MUON_OK;
}

extern "C" muon_status muon_route(int64_t tokens, int experts, int k, int dtype,
                                  const void* logits, int64_t ld, const uint8_t* token_mask,
                                  int normalize, float* weights, int32_t* index, int32_t* counts,
                                  float* mean_prob, float* loss, void* workspace, size_t ws_bytes,
                                  void* stream) {
  const muon_status st = check_route(tokens, experts, k, dtype, ld);
  if (st != MUON_OK) return st;
  if (!counts || !mean_prob || !loss || !workspace ||
      (tokens > 0 && (!logits || !weights || !index)))
    return MUON_ERR_INVALID_ARG;
  if (misaligned(logits, dtype == MUON_BF16 ? 2 : 4) || misaligned(weights, 4) ||
      misaligned(index, 4) || misaligned(counts, 4) || misaligned(mean_prob, 4) ||
      misaligned(loss, 4) || misaligned(workspace, 256))
    return MUON_ERR_ALIGNMENT;
  size_t need = 0;
  muon_route_workspace_bytes(tokens, experts, &need);
  if (ws_bytes < need) return MUON_ERR_WORKSPACE;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  NvtxRange range("muon_route");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int blocks = route_blocks(tokens, experts);
  char* ws = static_cast<char*>(workspace);
  const size_t es = dtype == MUON_BF16 ? 2 : 4;
  const RouteFwd a = {tokens, ld, experts, k, normalize,
                      whole_rows(logits, tokens, ld, experts, es),
                      !misaligned(weights, 16) && !misaligned(index, 16), logits, token_mask, weights,
                      index, reinterpret_cast<float*>(ws + probs_offset(tokens, experts)),
                      reinterpret_cast<int32_t*>(ws + kJoinBytes), reinterpret_cast<unsigned*>(ws),
                      counts, mean_prob, loss};
  cudaError_t e;
  if (rows_form(tokens, experts, k, logits, ld, es)) {
    int warps;
    rows_grid(tokens, experts, es, &blocks, &warps);
    e = dtype == MUON_BF16 ? launch_rows<__nv_bfloat16>(a, blocks, warps, s)
                           : launch_rows<float>(a, blocks, warps, s);
  } else {
    e = by_experts(dtype, experts, LaunchFwd{a, blocks, s});
  }
  if (e == cudaSuccess && blocks > 1) {
    const RouteJoin j = {experts, k, blocks, a.part_p, a.part_c, counts, mean_prob, loss,
                         reinterpret_cast<float*>(ws) + 1, a.ticket};
    e = launch_k(route_join_kernel, dim3(join_blocks(experts)), dim3(256), 0, s, true, j);
  }
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" muon_status muon_route_backward(int64_t tokens, int experts, int k, int dtype,
                                           const void* logits, int64_t ld,
                                           const uint8_t* token_mask, int normalize,
                                           const int32_t* index, const int32_t* counts,
                                           const float* dweights, const float* dloss,
                                           void* dlogits, void* stream) {
  const muon_status st = check_route(tokens, experts, k, dtype, ld);
  if (st != MUON_OK) return st;
  if (tokens > 0 && (!logits || !index || !counts || !dlogits)) return MUON_ERR_INVALID_ARG;
  const size_t es = dtype == MUON_BF16 ? 2 : 4;
  if (misaligned(logits, es) || misaligned(dlogits, es) || misaligned(index, 4) ||
      misaligned(counts, 4) || misaligned(dweights, 4) || misaligned(dloss, 4))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (tokens == 0) return MUON_OK;
  NvtxRange range("muon_route_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RouteBwd a = {tokens, ld, experts, k, normalize,
                      experts % (int)(16 / es) == 0 && !misaligned(logits, 16) &&
                          !misaligned(dlogits, 16) && (tokens <= 1 || (size_t)ld * es % 16 == 0),
                      logits, token_mask, index, counts, dweights, dloss, dlogits};
  const cudaError_t e =
      dtype == MUON_BF16 ? bwd_pieces<__nv_bfloat16, 1>(a, s) : bwd_pieces<float, 1>(a, s);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
