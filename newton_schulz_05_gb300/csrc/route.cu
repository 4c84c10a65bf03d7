// Expert router: top-k choice, combine weights, per-expert counts and the
// balance loss of a token batch, and the gradient of weights and loss.
//
// A token's logits live in the registers of G lanes, eight consecutive experts
// a lane (two or four times eight for more than 256 experts), so one warp takes
// 32 / G tokens at once and every reduction over experts is log2 G shuffles.  An
// expert stays with its lane for all of a warp's tokens: probabilities add up
// in registers, and the gradient's per-expert factors are loaded once.
//
// The choice.  Logits map to unsigned keys of the same order.  Each lane sorts
// its eight once; a pick is then the largest head of the G lists, whose owner
// drops it.  bf16 keys leave sixteen bits for the complement of the index, so
// one unsigned maximum settles value and tie; fp32 keys carry the index beside
// them, and the lowest lane with the largest head wins, its list being sorted
// stably.
//
// Both passes read the logits once from HBM; the forward pass is bound by the
// instructions of the choice, the gradient by HBM.
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
__device__ __forceinline__ void narrow8(uint4 (&u)[1], const float (&v)[8]) {
  Piece<8> p;
  #pragma unroll
  for (int j = 0; j < 8; ++j) elem(p, j) = v[j];
  u[0] = narrow(p);
}
__device__ __forceinline__ void narrow8(uint4 (&u)[2], const float (&v)[8]) {
  #pragma unroll
  for (int q = 0; q < 2; ++q)
    u[q] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                      __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
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

// exp(v - top): the difference is rounded once, so the relative error is that
// of the difference, a few units more for 2^x; below 2^-126 the result is 0
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

// The candidates of one lane: next() gives the largest over the group that has
// not been given yet, as a word that value() and expert() read (for fp32 the
// expert comes beside it).
template <typename T, int G, int N> struct Choice;

// bf16: key and index in one word.  N == 8: a sorted list.
template <int G, int N> struct Choice<__nv_bfloat16, G, N> {
  uint32_t k[N];
  // chunk c, which begins at expert e0, as loaded: keys of two at once
  __device__ __forceinline__ void set(int c, const uint4 (&u)[1], int e0) {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
      // adding 0 turns -0 into +0 and a NaN into the canonical positive one
      uint32_t x;
      asm("{.reg .b32 z;\n mov.b32 z, 0;\n add.rn.bf16x2 %0, %1, z;}" : "=r"(x) : "r"(w[j]));
      // a set sign flips all sixteen bits, a clear one the sign alone
      x ^= ((x >> 15) & 0x00010001u) * 0x7fffu | 0x80008000u;
      k[c * 8 + 2 * j] = x * 65536u + (uint32_t)(0xffff - (e0 + 2 * j));
      k[c * 8 + 2 * j + 1] = (x & 0xffff0000u) | (uint32_t)(0xffff - (e0 + 2 * j + 1));
    }
  }
  __device__ __forceinline__ void order() {
    if constexpr (N == 8) {
      auto ce = [&](int a, int b) {
        const uint32_t hi = max(k[a], k[b]);
        k[b] = min(k[a], k[b]);
        k[a] = hi;
      };
      // nineteen exchanges (Batcher's odd-even merge of two sorted fours)
      ce(0, 1); ce(2, 3); ce(4, 5); ce(6, 7);
      ce(0, 2); ce(1, 3); ce(4, 6); ce(5, 7);
      ce(1, 2); ce(5, 6);
      ce(0, 4); ce(1, 5); ce(2, 6); ce(3, 7);
      ce(2, 4); ce(3, 5);
      ce(1, 2); ce(3, 4); ce(5, 6);
    }
  }
  // `left` (known at compile time): picks that may still follow
  __device__ __forceinline__ uint32_t next(int, int&, int left) {
    uint32_t head = k[0];
    if constexpr (N != 8) {
      #pragma unroll
      for (int j = 1; j < N; ++j) head = max(head, k[j]);
    }
    const uint32_t win = group_max<G>(head);
    if constexpr (N == 8) {
      if (head == win) {
        #pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < left) k[j] = k[j + 1];
        if (left > 7) k[7] = 0;
      }
    } else {
      #pragma unroll
      for (int j = 0; j < N; ++j) k[j] = k[j] == win ? 0u : k[j];
    }
    return win;
  }
  // the value's low sixteen bits are zeros, in the key's own sense
  static __device__ __forceinline__ uint32_t key(uint32_t win) {
    return win & 0x80000000u ? win & 0xffff0000u : win | 0xffffu;
  }
  static __device__ __forceinline__ int expert(uint32_t win, int) {
    return 0xffff - (int)(win & 0xffffu);
  }
};

// fp32: key and index side by side
template <int G, int N> struct Choice<float, G, N> {
  uint32_t k[N];
  int id[N];
  __device__ __forceinline__ void set(int c, const uint4 (&u)[2], int e0) {
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
      k[c * 8 + j] = order_key(__uint_as_float(w[j]));
      id[c * 8 + j] = e0 + j;
    }
  }
  __device__ __forceinline__ void order() {
    if constexpr (N == 8) {
      // odd-even transposition: neighbours are exchanged only when out of
      // order, so equal keys keep their order
      #pragma unroll
      for (int r = 0; r < 8; ++r)
        #pragma unroll
        for (int j = r & 1; j + 1 < 8; j += 2) {
          const bool s = k[j + 1] > k[j];
          const uint32_t a = s ? k[j + 1] : k[j], b = s ? k[j] : k[j + 1];
          const int x = s ? id[j + 1] : id[j], y = s ? id[j] : id[j + 1];
          k[j] = a; k[j + 1] = b;
          id[j] = x; id[j + 1] = y;
        }
    }
  }
  __device__ __forceinline__ uint32_t next(int group_lanes, int& e, int left) {
    uint32_t win;
    if constexpr (N == 8) {
      win = group_max<G>(k[0]);
      const uint32_t who = __ballot_sync(kAll, k[0] == win) & (uint32_t)group_lanes;
      const int lane = __ffs(who) - 1;
      e = __shfl_sync(kAll, id[0], lane);
      if ((int)(threadIdx.x & 31) == lane) {
        #pragma unroll
        for (int j = 0; j < 7; ++j)
          if (j < left) { k[j] = k[j + 1]; id[j] = id[j + 1]; }
        if (left > 7) k[7] = 0;
      }
    } else {      // a lane's experts are not consecutive: the lowest index decides
      uint32_t head = 0;
      int first = 0x7fffffff;
      #pragma unroll
      for (int j = 0; j < N; ++j)
        if (k[j] > head) { head = k[j]; first = id[j]; }
      win = group_max<G>(head);
      e = (int)__reduce_min_sync(kAll, head == win ? (uint32_t)first : 0x7fffffffu);
      #pragma unroll
      for (int j = 0; j < N; ++j)
        if (id[j] == e) k[j] = 0;
    }
    return win;
  }
  static __device__ __forceinline__ uint32_t key(uint32_t win) { return win; }
  static __device__ __forceinline__ int expert(uint32_t, int e) { return e; }
};

// One token's logits as a lane holds them: its chunks as loaded, -inf where
// there is no expert.  Rows of whole, aligned chunks are loaded ahead, so that
// the next token's are in flight while this one is worked on; others when they
// are needed.  A token past the end or masked keeps what was there: its results
// are thrown away.
template <typename T, int G, int NCH> struct Logits {
  uint4 u[NCH][kPieces<T>];
  bool live;
  __device__ __forceinline__ void clear() {
    const uint32_t w = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
    #pragma unroll
    for (int c = 0; c < NCH; ++c)
      #pragma unroll
      for (int q = 0; q < kPieces<T>; ++q) u[c][q] = make_uint4(w, w, w, w);
  }
  template <typename A>
  __device__ __forceinline__ void load(const A& a, int64_t t, int gl) {
    live = t < a.tokens && !(a.mask && !a.mask[t]);
    if (!a.vec || t >= a.tokens) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    #pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int e0 = (c * G + gl) * 8;
      if (e0 < a.experts) {
        #pragma unroll
        for (int q = 0; q < kPieces<T>; ++q) u[c][q] = __ldg(reinterpret_cast<const uint4*>(row + e0) + q);
      }
    }
  }
  template <typename A>
  __device__ __forceinline__ void arrive(const A& a, int64_t t, int gl) {
    if (a.vec || t >= a.tokens) return;
    const T* row = static_cast<const T*>(a.logits) + t * a.ld;
    #pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int e0 = (c * G + gl) * 8;
      float w[8];
      #pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = e0 + j < a.experts ? to_f(row[e0 + j]) : -INFINITY;
      narrow8(u[c], w);
    }
  }
};

// Lane l of a token's G lanes has experts (c G + l) 8 .. + 7 for c = 0 .. NCH - 1.
template <typename T, int G, int NCH>
__global__ void __launch_bounds__(kRouteThreads, NCH == 1 ? 2 : 1)
route_kernel(const __grid_constant__ RouteFwd a) {
  constexpr int TPW = 32 / G, N = NCH * 8, E = G * N;
  constexpr int kStage = TPW * (E < kRouteMaxK ? E : kRouteMaxK);
  // warps whose sums are added side by side
  constexpr int kRows = E <= 256 ? kRouteWarps : 2;
  __shared__ float sp[kRows][E];
  __shared__ int sc[E + 1];
  __shared__ uint32_t sw[kRouteWarps][kStage];     // picks: the winning words, then weights
  __shared__ int se[kRouteWarps][kStage];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % G, grp = lane / G;
  const int group_lanes = (int)((G == 32 ? kAll : ((1u << (G & 31)) - 1u) << (grp * G)));
  for (int e = threadIdx.x; e <= E; e += kRouteThreads) sc[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  __syncthreads();
  float acc[N];
  #pragma unroll
  for (int j = 0; j < N; ++j) acc[j] = 0.f;
  int routed_count = 0;
  const int64_t stride = (int64_t)gridDim.x * kRouteWarps * TPW;
  const int64_t begin = ((int64_t)blockIdx.x * kRouteWarps + warp) * TPW;
  Logits<T, G, NCH> now, next;
  next.clear();
  next.load(a, begin + grp, gl);
  uint32_t* const w = sw[warp] + grp * a.k;
  int* const x = se[warp] + grp * a.k;
  for (int64_t t0 = begin; t0 < a.tokens; t0 += stride) {
    const int64_t t = t0 + grp;
    now = next;
    now.arrive(a, t, gl);
    next.load(a, t + stride, gl);
    Choice<T, G, N> choice;
    #pragma unroll
    for (int c = 0; c < NCH; ++c) choice.set(c, now.u[c], (c * G + gl) * 8);
    choice.order();
    uint32_t first = 0;
    auto pick = [&](int p, int left) {
      int e = 0;
      const uint32_t win = choice.next(group_lanes, e, left);
      if (p == 0) first = win;
      if (gl == 0) {
        w[p] = win;
        if (sizeof(T) == 4) x[p] = e;
      }
    };
    if (a.k <= 8) {
      #pragma unroll
      for (int p = 0; p < 8; ++p)
        if (p < a.k) pick(p, 7 - p);
    } else {
      for (int p = 0; p < a.k; ++p) pick(p, 8);
    }
    float v[N];
    #pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float u[8];
      widen8(u, now.u[c]);
      #pragma unroll
      for (int j = 0; j < 8; ++j) v[c * 8 + j] = u[j];
    }
    first = choice.key(first);
    const bool routed = now.live && first > kKeyNegInf;
    const float top = key_value(first);
    float s = 0.f;
    #pragma unroll
    for (int j = 0; j < N; ++j) {
      v[j] = exp_below(v[j], top);
      s += v[j];
    }
    const float total = group_sum<G>(s);
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
      const uint32_t key = choice.key(w[p]);
      const bool ok = routed && key > kKeyNegInf;
      const int e = ok ? choice.expert(w[p], x[p]) : -1;
      const float y = ok ? exp_below(key_value(key), top) : 0.f;
      picked += y;
      w[p] = __float_as_uint(y);
      x[p] = e;
      if (ok) atomicAdd(&sc[e], 1);
    }
    const float z = __frcp_rn(a.normalize ? group_sum<G>(picked) : total);
    if (t < a.tokens)
      for (int p = gl; p < a.k; p += G) {
        const int e = x[p];
        a.weights[t * a.k + p] = e >= 0 ? __uint_as_float(w[p]) * z : 0.f;
        a.index[t * a.k + p] = e;
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
        float& to = sp[warp - i][((j / 8) * G + gl) * 8 + j % 8];
        to = i ? to + acc[j] : acc[j];
      }
    }
    __syncthreads();
  }
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e <= a.experts; e += kRouteThreads) {
      if (e < a.experts) {
        float p = 0.f;
        #pragma unroll
        for (int i = 0; i < kRows; ++i) p += sp[i][e];
        a.part_p[(int64_t)blockIdx.x * a.experts + e] = p;
      }
      a.part_c[(int64_t)blockIdx.x * (a.experts + 1) + e] = sc[e < a.experts ? e : E];
    }
    return;
  }
  // one block: the results themselves
  const int n = sc[E];
  const float fn = (float)(n > 0 ? n : 1);
  float l = 0.f;
  for (int e = threadIdx.x; e < a.experts; e += kRouteThreads) {
    float p = 0.f;
    #pragma unroll
    for (int i = 0; i < kRows; ++i) p += sp[i][e];
    p /= fn;
    a.counts[e] = sc[e];
    a.mean_prob[e] = p;
    l = fmaf((float)sc[e] / ((float)a.k * fn), p, l);
  }
  __shared__ float red[kRouteWarps];
  l = block_sum<kRouteThreads>(l, red);
  if (threadIdx.x == 0) {
    a.counts[a.experts] = n;
    *a.loss = (float)a.experts * l;
  }
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
template <typename T, int G, int NCH>
__global__ void __launch_bounds__(kRouteThreads, NCH == 1 ? 2 : 1)
route_bwd_kernel(const __grid_constant__ RouteBwd a) {
  constexpr int TPW = 32 / G, N = NCH * 8, E = G * N;
  constexpr int KS = ((E < kRouteMaxK ? E : kRouteMaxK) + G - 1) / G;   // picks a lane
  extern __shared__ float smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gl = lane % G, grp = lane / G;
  float* const px = smem + (warp * TPW + grp) * (2 * E);   // exponentials of the token's row
  float* const xx = px + E;                                // x by expert, zeros between tokens
  for (int i = gl; i < E; i += G) xx[i] = 0.f;
  __syncwarp();
  const int routed_tokens = a.counts[a.experts];
  const float n = (float)(routed_tokens > 0 ? routed_tokens : 1);
  const float f = a.dloss ? *a.dloss * (float)a.experts / ((float)a.k * n) / n : 0.f;
  float b[N];
  #pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = ((j / 8) * G + gl) * 8 + j % 8;
    b[j] = e < a.experts ? f * (float)a.counts[e] : 0.f;
  }
  const int64_t stride = (int64_t)gridDim.x * kRouteWarps * TPW;
  const int64_t begin = ((int64_t)blockIdx.x * kRouteWarps + warp) * TPW;
  Logits<T, G, NCH> now, next;
  int e_now[KS], e_next[KS];
  float d_now[KS], d_next[KS];
  auto load_picks = [&](int64_t t) {
    #pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int p = gl + s * G;
      e_next[s] = -1;
      d_next[s] = 0.f;
      if (a.dweights && p < a.k && t < a.tokens) {
        e_next[s] = a.index[t * a.k + p];
        d_next[s] = a.dweights[t * a.k + p];
      }
    }
  };
  next.clear();
  next.load(a, begin + grp, gl);
  load_picks(begin + grp);
  for (int64_t t0 = begin; t0 < a.tokens; t0 += stride) {
    const int64_t t = t0 + grp;
    now = next;
    #pragma unroll
    for (int s = 0; s < KS; ++s) { e_now[s] = e_next[s]; d_now[s] = d_next[s]; }
    now.arrive(a, t, gl);
    next.load(a, t + stride, gl);
    load_picks(t + stride);
    float v[N];
    float best = -INFINITY;
    #pragma unroll
    for (int c = 0; c < NCH; ++c) {
      float u[8];
      widen8(u, now.u[c]);
      #pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[c * 8 + j] = u[j];
        best = max_nan(best, v[c * 8 + j]);
      }
    }
    const float top = key_value(group_max<G>(order_key(best)));
    const bool routed = now.live && top != -INFINITY;
    float s = 0.f;
    #pragma unroll
    for (int c = 0; c < NCH; ++c) {
      #pragma unroll
      for (int j = c * 8; j < c * 8 + 8; ++j) {
        v[j] = exp_below(v[j], top);
        s += v[j];
      }
      float4* q = reinterpret_cast<float4*>(px + (c * G + gl) * 8);
      q[0] = make_float4(v[c * 8], v[c * 8 + 1], v[c * 8 + 2], v[c * 8 + 3]);
      q[1] = make_float4(v[c * 8 + 4], v[c * 8 + 5], v[c * 8 + 6], v[c * 8 + 7]);
    }
    const float total = group_sum<G>(s);
    __syncwarp();
    if (a.dweights) {
      float z = 0.f, wd = 0.f;
      #pragma unroll
      for (int s = 0; s < KS; ++s) {
        if (!routed || e_now[s] < 0 || e_now[s] >= a.experts) {
          e_now[s] = -1;
          d_now[s] = 0.f;      // whatever a missing pick's gradient holds
        }
        const float y = e_now[s] >= 0 ? px[e_now[s]] : 0.f;
        z += y;
        wd = fmaf(y, d_now[s], wd);
      }
      if (a.normalize) {
        z = __frcp_rn(group_sum<G>(z));
        wd = group_sum<G>(wd) * z;
        z *= total;
        #pragma unroll
        for (int s = 0; s < KS; ++s) d_now[s] = (d_now[s] - wd) * z;
      }
      #pragma unroll
      for (int s = 0; s < KS; ++s)
        if (e_now[s] >= 0) xx[e_now[s]] = d_now[s];
      __syncwarp();
    }
    const float inv = __frcp_rn(total);
    float x[N];
    float dot = 0.f;
    #pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const float4* q = reinterpret_cast<const float4*>(xx + (c * G + gl) * 8);
      const float4 q0 = q[0], q1 = q[1];
      x[c * 8 + 0] = q0.x; x[c * 8 + 1] = q0.y; x[c * 8 + 2] = q0.z; x[c * 8 + 3] = q0.w;
      x[c * 8 + 4] = q1.x; x[c * 8 + 5] = q1.y; x[c * 8 + 6] = q1.z; x[c * 8 + 7] = q1.w;
    }
    #pragma unroll
    for (int j = 0; j < N; ++j) {
      v[j] *= inv;
      const float bx = b[j] + x[j];
      dot = fmaf(v[j], a.normalize ? b[j] : bx, dot);
      x[j] = bx;
    }
    dot = group_sum<G>(dot);
    #pragma unroll
    for (int j = 0; j < N; ++j) v[j] = routed ? v[j] * (x[j] - dot) : 0.f;
    if (t < a.tokens) {
      #pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int e0 = (c * G + gl) * 8;
        T* out = static_cast<T*>(a.dlogits) + t * a.experts + e0;
        if (a.vec) {
          float o[8];
          uint4 u[kPieces<T>];
          #pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = v[c * 8 + j];
          narrow8(u, o);
          if (e0 < a.experts) {
            #pragma unroll
            for (int q = 0; q < kPieces<T>; ++q) reinterpret_cast<uint4*>(out)[q] = u[q];
          }
        } else {
          #pragma unroll
          for (int j = 0; j < 8; ++j)
            if (e0 + j < a.experts) out[j] = from_f<T>(v[c * 8 + j]);
        }
      }
    }
    __syncwarp();
    if (a.dweights) {
      #pragma unroll
      for (int s = 0; s < KS; ++s)
        if (e_now[s] >= 0) xx[e_now[s]] = 0.f;
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

// blocks of a pass: a warp for every token group, up to two blocks an SM
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
size_t probs_offset(int64_t tokens, int experts) {
  return kJoinBytes +
         ((size_t)route_blocks(tokens, experts) * (experts + 1) * sizeof(int32_t) + 255) / 256 * 256;
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
    route_kernel<T, G, NCH><<<blocks, kRouteThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
};

struct LaunchBwd {
  const RouteBwd& a;
  int blocks;
  cudaStream_t s;
  template <typename T, int G, int NCH> cudaError_t operator()() const {
    const size_t smem = (size_t)kRouteWarps * (32 / G) * 2 * G * NCH * 8 * sizeof(float);
    if (smem > 48u << 10) {
      const cudaError_t e = cudaFuncSetAttribute(route_bwd_kernel<T, G, NCH>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e != cudaSuccess) return e;
    }
    route_bwd_kernel<T, G, NCH><<<blocks, kRouteThreads, smem, s>>>(a);
    return cudaGetLastError();
  }
};

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_route_workspace_bytes(int64_t tokens, int experts, size_t* out) {
  if (!out || tokens < 0) return MUON_ERR_INVALID_ARG;
  if (experts < 1 || experts > kRouteMaxExperts) return MUON_ERR_UNSUPPORTED_SHAPE;
  *out = probs_offset(tokens, experts) +
         (size_t)route_blocks(tokens, experts) * experts * sizeof(float);
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
  const int blocks = route_blocks(tokens, experts);
  char* ws = static_cast<char*>(workspace);
  const size_t es = dtype == MUON_BF16 ? 2 : 4;
  const RouteFwd a = {tokens, ld, experts, k, normalize,
                      whole_rows(logits, tokens, ld, experts, es), logits, token_mask, weights,
                      index, reinterpret_cast<float*>(ws + probs_offset(tokens, experts)),
                      reinterpret_cast<int32_t*>(ws + kJoinBytes), reinterpret_cast<unsigned*>(ws),
                      counts, mean_prob, loss};
  cudaError_t e = by_experts(dtype, experts, LaunchFwd{a, blocks, s});
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
                      whole_rows(logits, tokens, ld, experts, es) &&
                          reinterpret_cast<uintptr_t>(dlogits) % 16 == 0,
                      logits, token_mask, index, counts, dweights, dloss, dlogits};
  const cudaError_t e =
      by_experts(dtype, experts, LaunchBwd{a, route_blocks(tokens, experts), s});
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
