// Norms of query and key heads with the rotation of positions, and the gradient.
//
// A head is read once and written once (the gradient reads two and writes one), so both are
// bound by HBM where a head's arithmetic is short enough.  A head lies in the registers of a few
// lanes of a warp, two pieces of 16 bytes each (8 where only those divide its parts), chosen so
// that a pair's two elements are in one lane: its mean square is a few shuffles, its rotation
// none.  A warp takes as many heads as fit, in passes that come through a ring of asynchronous
// copies into shared memory; a token's angles are loaded once for its heads.  Weight gradients
// add up in registers over all of a warp's heads, then over the block's warps, then over blocks,
// always in the same order.  Heads of odd widths, at odd addresses, or about 2^31 of them go
// through kernels that move single elements, a warp a head (9 to 25% of the copy rate, the
// gradient 5 to 13%).
//
// Measured: [32768, 32 + 8, 128] bf16 104 us, 6.4 TB/s, its gradient 193 us, 5.2 TB/s; in fp32
// [8192, 16 + 16, 256] 82 us, 6.6 TB/s, and 139 us, 5.9 TB/s; [8192, 16 + 4, 64] bf16 11.4 and
// 21.7 us (57 and 44% of the copy rate: about 200 instructions a pass, prologue and join); one
// token of 32 sequences 2.6 us.
#include "sequence.cuh"

#include <algorithm>
#include <type_traits>

namespace muon {

namespace {

constexpr int kHeadThreads = 256, kHeadWarps = kHeadThreads / 32;
constexpr int kHeadMaxDim = 1024;
// Blocks of the gradient and images of its weight sums, two an SM: with 152, 456 and 608 the gradient of
// [8191, 12 + 12, 80] fp32 takes 51, 47 and 44 us, with these 38; [32768, 32 + 8, 128] bf16 264, 210 and
// 183, with these 184; [8192, 16 + 16, 256] fp32 133, 138 and 136, with these 139
constexpr int kHeadParts = 304;

// Queries or keys: heads `step` elements apart, tokens `ld`
struct HeadSide {
  const void *x, *dy, *weight;
  int64_t ld, step, lddy, stepdy;
  void* out;
  int heads;
};
struct Heads {
  int64_t tokens, table, period;
  int dim, rotary, neighbours;
  float eps;
  const float *cos, *sin;
  const int64_t* positions;
  HeadSide side[2];
  float* part;
};

__device__ __forceinline__ float warp_sum(float v) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// row of the table, or -1: no token
__device__ __forceinline__ int64_t position_of(const Heads& a, int64_t t) {
  if (!a.rotary) return 0;
  const int64_t p = a.positions ? a.positions[t] : t % a.period;
  return p >= 0 && p < a.table ? p : -1;
}
// f(i, j, c, s): each of a lane's pairs; f1(i): each of its other elements
template <typename F, typename F1>
__device__ __forceinline__ void pairs(const Heads& a, int64_t pos, F f, F1 f1) {
  const int half = a.rotary / 2, lane = threadIdx.x & 31;
  for (int m = lane; m < half; m += 32)
    f(a.neighbours ? 2 * m : m, a.neighbours ? 2 * m + 1 : m + half, a.cos[pos * half + m],
      a.sin[pos * half + m]);
  for (int i = a.rotary + lane; i < a.dim; i += 32) f1(i);
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kHeadThreads) heads_kernel(const __grid_constant__ Heads a) {
  pdl_wait();
  const int lane = threadIdx.x & 31, all = a.side[0].heads + a.side[1].heads;
  for (int64_t u = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); u < a.tokens * all;
       u += (int64_t)gridDim.x * kHeadWarps) {
    const int64_t t = u / all;
    int hd = (int)(u % all);
    const bool key = hd >= a.side[0].heads;
    const HeadSide& s = a.side[key];
    if (key) hd -= a.side[0].heads;
    const T* x = static_cast<const T*>(s.x) + t * s.ld + hd * s.step;
    T* out = static_cast<T*>(s.out) + (t * s.heads + hd) * a.dim;
    const WT* w = static_cast<const WT*>(s.weight);
    const int64_t pos = position_of(a, t);
    if (pos < 0) {
      for (int i = lane; i < a.dim; i += 32) out[i] = from_f<T>(0.f);
      continue;
    }
    float sq = 0.f;
    for (int i = lane; i < a.dim; i += 32) sq = fmaf(to_f(x[i]), to_f(x[i]), sq);
    const float rstd = 1.f / sqrtf(warp_sum(sq) / a.dim + a.eps);
    auto n = [&](int i) { return to_f(x[i]) * rstd * (w ? to_f(w[i]) : 1.f); };
    pairs(a, pos,
          [&](int i, int j, float c, float sn) {
            const float u = n(i), v = n(j);
            out[i] = from_f<T>(u * c - v * sn);
            out[j] = from_f<T>(v * c + u * sn);
          },
          [&](int i) { out[i] = from_f<T>(n(i)); });
  }
}

template <typename T, typename WT>
__global__ void __launch_bounds__(kHeadThreads) heads_bwd_kernel(const __grid_constant__ Heads a) {
  extern __shared__ float sums[];     // a warp: [2][dim], then [dim] of g
  pdl_wait();
  const int lane = threadIdx.x & 31, all = a.side[0].heads + a.side[1].heads;
  float* mine = sums + (threadIdx.x >> 5) * 3 * a.dim;
  float* g = mine + 2 * a.dim;
  for (int i = lane; i < 2 * a.dim; i += 32) mine[i] = 0.f;
  for (int64_t u = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); u < a.tokens * all;
       u += (int64_t)gridDim.x * kHeadWarps) {
    const int64_t t = u / all;
    int hd = (int)(u % all);
    const int key = hd >= a.side[0].heads;
    const HeadSide& s = a.side[key];
    if (key) hd -= a.side[0].heads;
    const T* x = static_cast<const T*>(s.x) + t * s.ld + hd * s.step;
    const T* dy = static_cast<const T*>(s.dy) + t * s.lddy + hd * s.stepdy;
    T* out = static_cast<T*>(s.out) + (t * s.heads + hd) * a.dim;
    const WT* w = static_cast<const WT*>(s.weight);
    const int64_t pos = position_of(a, t);
    if (pos < 0) {
      if (s.out)
        for (int i = lane; i < a.dim; i += 32) out[i] = from_f<T>(0.f);
      continue;
    }
    __syncwarp();
    pairs(a, pos,
          [&](int i, int j, float c, float sn) {
            const float u = to_f(dy[i]), v = to_f(dy[j]);
            g[i] = u * c + v * sn;
            g[j] = v * c - u * sn;
          },
          [&](int i) { g[i] = to_f(dy[i]); });
    __syncwarp();
    float sq = 0.f, dot = 0.f;
    for (int i = lane; i < a.dim; i += 32) {
      const float v = to_f(x[i]);
      sq = fmaf(v, v, sq);
      dot = fmaf(g[i] * (w ? to_f(w[i]) : 1.f), v, dot);
    }
    const float rstd = 1.f / sqrtf(warp_sum(sq) / a.dim + a.eps);
    const float mean = warp_sum(dot) * rstd / a.dim;
    for (int i = lane; i < a.dim; i += 32) {
      const float h = to_f(x[i]) * rstd;
      mine[key * a.dim + i] += g[i] * h;
      if (s.out) out[i] = from_f<T>((g[i] * (w ? to_f(w[i]) : 1.f) - h * mean) * rstd);
    }
  }
  __syncthreads();
  if (!a.part) return;
  for (int i = threadIdx.x; i < 2 * a.dim; i += kHeadThreads) {
    float v = 0.f;
    for (int k = 0; k < kHeadWarps; ++k) v += sums[k * 3 * a.dim + i];
    a.part[(int64_t)blockIdx.x * 2 * a.dim + i] = v;
  }
}

// ------------------------------------------------------------ heads of whole pieces

// E elements as they lie in memory: 16 bytes, or 8 where only those fit a head's parts
template <typename T, int E> struct RawPiece { using type = uint4; };
template <> struct RawPiece<__nv_bfloat16, 4> { using type = uint2; };
__device__ __forceinline__ void widen(Piece<4>& p, const uint2& u) {
  p.v[0] = make_float2(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
  p.v[1] = make_float2(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
template <typename T, int E> __device__ __forceinline__ typename RawPiece<T, E>::type pack(const Piece<E>& p) {
  if constexpr (sizeof(T) == 2 && E == 4) {
    const __nv_bfloat162 a = __float22bfloat162_rn(p.v[0]), b = __float22bfloat162_rn(p.v[1]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    return narrow(p);
  }
}
// A lane's two pieces of a head.  Those of the rotated part are turned into one another,
// so no lane needs another's: m and m + rotary / 2 for one half against the other, where
// both pieces have the E pairs from E * unit on; neighbours have their pairs within a piece.
// Neighbouring lanes have neighbouring pieces throughout.
template <int E, bool NB> struct Unit {
  int a, b;              // first elements of the pieces
  int pa, pb;            // first pairs of their halves of E angles
  bool any, ta, tb;      // there is work; the pieces are turned
  __device__ __forceinline__ Unit(int dim, int rotary, int u) {
    const int units = dim / (2 * E), turned = rotary / (2 * E);
    any = u < units;
    if (NB) {
      a = E * u;
      b = E * (u + units);
      ta = a < rotary;
      tb = b < rotary;
      pa = a / 2;
      pb = b / 2;
    } else {
      ta = tb = u < turned;
      const int first = ta ? 0 : turned;       // of the turned units, or of the others
      a = E * (first + u);
      b = a + E * (ta ? turned : units - turned);
      pa = E * u;
      pb = pa + E / 2;
    }
  }
};

// (a, b) turned by the angles (c, s); s negated: turned back
template <int E, bool NB>
__device__ __forceinline__ void turn(Piece<E>& a, Piece<E>& b, const Piece<E>& c, const Piece<E>& s) {
  if constexpr (NB) {
    auto one = [](float2& v, float c, float s) {
      v = fma2(make_float2(v.y, v.x), make_float2(-s, s), mul2(v, both(c)));
    };
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      // pair j of the first piece, pair E / 2 + j of all
      one(a.v[j], j & 1 ? c.v[j / 2].y : c.v[j / 2].x, j & 1 ? s.v[j / 2].y : s.v[j / 2].x);
      const int k = j + E / 2;
      one(b.v[j], k & 1 ? c.v[k / 2].y : c.v[k / 2].x, k & 1 ? s.v[k / 2].y : s.v[k / 2].x);
    }
  } else {
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float2 x = a.v[j], y = b.v[j], t = mul2(x, c.v[j]);
      a.v[j] = make_float2(fmaf(-s.v[j].x, y.x, t.x), fmaf(-s.v[j].y, y.y, t.y));
      b.v[j] = fma2(x, s.v[j], mul2(y, c.v[j]));
    }
  }
}
// The lanes of a head: G neighbouring ones of which dim / 2E have work, or exactly dim / 2E
// (G == 0) where more heads fit in a warp so, as three of 80 fp32 elements in place of two.
template <int G> struct Lanes {
  int length, heads, group, lane;      // lanes a head, heads a warp, the lane's head and place
  __device__ __forceinline__ explicit Lanes(int units) {
    const int l = threadIdx.x & 31;
    length = G ? G : units;
    heads = 32 / length;
    group = l / length;
    lane = l - group * length;
  }
  // over the lanes of a head, the same value in each
  __device__ __forceinline__ float sum(float v) const {
    if constexpr (G > 0) {
      #pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
      return v;
    } else {
      #pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        const float u = __shfl_down_sync(~0u, v, o);
        if (lane < o && lane + o < length) v += u;
      }
      return __shfl_sync(~0u, v, group * length);
    }
  }
};

// A token's heads are numbered through, n = token * heads + head, and warps take runs of them in
// turn: a run is about a token, and what the warps read at a time lies together.  In the forward
// pass queries and keys are one row of heads (blocks[0] and run[0] are for both; in blocks of
// their own they took 130 us where together they took 112, [32768, 32 + 8, 128] bf16); in the
// gradient, with one set of weight sums a warp, the first blocks work on the queries, the others
// on the keys.
struct HeadWork { int blocks[2], run[2]; int wbf16; };      // run: passes

// One side's weights in fp32 (1 where there are none), as the lanes of a warp need them: four at a
// time, those of all lanes next to one another; staged by one warp
template <int E> struct HeadWeights { float4 v[E / 2][32]; };
template <int E, typename U>
__device__ __forceinline__ void stage_weights(HeadWeights<E>& to, const HeadSide& side, const U& un, int wbf16) {
  if (un.any) {
    #pragma unroll
    for (int q = 0; q < E / 2; ++q) {
      const int at = q < E / 4 ? un.a + 4 * q : un.b + 4 * (q - E / 4);
      float w[4];
      #pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = !side.weight ? 1.f
               : wbf16      ? to_f(static_cast<const __nv_bfloat16*>(side.weight)[at + j])
                            : static_cast<const float*>(side.weight)[at + j];
      to.v[q][threadIdx.x & 31] = make_float4(w[0], w[1], w[2], w[3]);
    }
  }
}
// of the first piece or the second
template <int E> __device__ __forceinline__ void load_weights(Piece<E>& v, const HeadWeights<E>& from, int piece) {
  #pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    const float4 f = from.v[piece * (E / 4) + q][threadIdx.x & 31];
    v.v[2 * q] = make_float2(f.x, f.y);
    v.v[2 * q + 1] = make_float2(f.z, f.w);
  }
}
__device__ __forceinline__ float rsqrt_fast(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A lane's N pieces of a pass (one head a group of lanes) and the position of its token, in a
// ring of kHeadRing passes that it copies, waits for and reads alone.  Slots of lanes without
// work hold zeros.
constexpr int kHeadRing = 4;
template <typename Raw, int N> struct HeadRing {
  Raw *at, *last;              // of the pass to use, and of the last one in the ring
  int64_t* position;
  __device__ __forceinline__ HeadRing(void* smem, bool has) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    at = static_cast<Raw*>(smem) + warp * (kHeadRing * N * 32) + lane;
    last = at + (kHeadRing - 1) * N * 32;
    position = reinterpret_cast<int64_t*>(static_cast<Raw*>(smem) + kHeadWarps * (kHeadRing * N * 32)) +
               warp * (kHeadRing * 32) + lane;
    if (!has)
      for (int i = 0; i < kHeadRing * N; ++i) at[i * 32] = Raw{};
  }
  __device__ __forceinline__ Raw& piece(int n) const { return at[n * 32]; }
  __device__ __forceinline__ void next() {
    if (at == last) {
      at -= (kHeadRing - 1) * N * 32;
      position -= (kHeadRing - 1) * 32;
    } else {
      at += N * 32;
      position += 32;
    }
  }
  static constexpr size_t kBytes = (sizeof(Raw) * N + 8) * kHeadRing * kHeadThreads;
  template <typename V> __device__ __forceinline__ static void copy(V* to, const void* p) {
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (sizeof(V) == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(s), "l"(p) : "memory");
    else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(s), "l"(p) : "memory");
  }
};

// Where a lane's group is in its walk through heads, numbered in 32 bits
struct HeadWalk {
  uint32_t n, all, stop;      // stop: the end of the run
  int token, head, heads;
  uint32_t run, jump;         // heads of a run, and from its end to that of the warp's next
  __device__ __forceinline__ void find() {
    token = (int)(n / (uint32_t)heads);
    head = (int)(n - (uint32_t)token * (uint32_t)heads);
  }
  __device__ __forceinline__ bool live() const { return n < all; }
  // by `by` heads; whether the token may be another
  __device__ __forceinline__ bool next(int by) {
    n += by;
    head += by;
    if (n >= stop) {
      n += jump;
      stop += jump + run;
    } else if (head < heads) {
      return false;
    }
    find();
    return true;
  }
};
// of a lane with work, `group` of the warp's `by`, in block `block` of `blocks`; run: passes a run;
// passes: of the warp's runs, all of them
__device__ __forceinline__ HeadWalk walk_of(const Heads& a, int heads, int block, int blocks, int run, int group,
                                            int by, bool has, int& passes) {
  const uint32_t warps = (uint32_t)blocks * kHeadWarps, warp = (uint32_t)block * kHeadWarps + (threadIdx.x >> 5);
  HeadWalk k;
  k.run = (uint32_t)(run * by);
  k.heads = heads;
  const uint32_t all = (uint32_t)a.tokens * (uint32_t)heads, runs = (all + k.run - 1) / k.run;
  k.n = warp * k.run + group;
  k.stop = (warp + 1) * k.run;
  k.all = has ? all : 0;
  k.jump = (warps - 1) * k.run;
  k.find();
  passes = warp < runs ? (int)((runs - 1 - warp) / warps + 1) * run : 0;
  return k;
}
// Heads that these walks can number without passing 2^32.  A walk's last step goes from the end of a
// run, at most that many heads and a run (a token's, 131088) further, by a run of every warp.  A run is at
// most what a warp has at all (share_out), so those are all heads again and a pass a warp.
constexpr int64_t kMostHeads = ((int64_t)1 << 31) - (1 << 20);
constexpr int kMostBlocks = 3648, kMostAPass = 16;
static_assert(2 * kMostHeads + 131088 + (kMostBlocks * kHeadWarps + 1) * kMostAPass <= (int64_t)1 << 32, "32 bits");

// the angles of the lane's pairs at a position: 1 and 0 where there are none
template <int E, bool NB>
__device__ __forceinline__ void angles(Piece<E>& c, Piece<E>& s, const Heads& a, int64_t pos, const Unit<E, NB>& un) {
  #pragma unroll
  for (int j = 0; j < E / 2; ++j) {
    c.v[j] = both(1.f);
    s.v[j] = both(0.f);
  }
  if (pos < 0) return;
  const float* const pc = a.cos + pos * (a.rotary / 2);
  const float* const ps = a.sin + pos * (a.rotary / 2);
  #pragma unroll
  for (int j = 0; j < E / 4; ++j) {      // E / 2 angles a half
    if (un.ta) {
      c.v[j] = reinterpret_cast<const float2*>(pc + un.pa)[j];
      s.v[j] = reinterpret_cast<const float2*>(ps + un.pa)[j];
    }
    if (un.tb) {
      c.v[E / 4 + j] = reinterpret_cast<const float2*>(pc + un.pb)[j];
      s.v[E / 4 + j] = reinterpret_cast<const float2*>(ps + un.pb)[j];
    }
  }
}

constexpr int kPieceDim = 512;        // widest head of these kernels

// A token's queries and keys follow one another, so that a warp reads and writes about what lies
// together.
template <typename T, int E, int G, bool NB>
__global__ void __launch_bounds__(kHeadThreads, 3)
heads_piece_kernel(const __grid_constant__ Heads a, const __grid_constant__ HeadWork w) {
  using Raw = typename RawPiece<T, E>::type;
  extern __shared__ uint4 ring[];
  __shared__ HeadWeights<E> weights[2];
  pdl_wait();
  const Lanes<G> ln(a.dim / (2 * E));
  const Unit<E, NB> un(a.dim, a.rotary, ln.lane);
  if (threadIdx.x < 64) stage_weights(weights[threadIdx.x >> 5], a.side[threadIdx.x >> 5], un, w.wbf16);
  __syncthreads();
  const float inv = 1.f / (float)a.dim;
  const bool has = un.any && ln.group < ln.heads;
  HeadRing<Raw, 2> slots(ring, has), fill = slots;
  int passes;
  const int queries = a.side[0].heads;
  HeadWalk in = walk_of(a, queries + a.side[1].heads, blockIdx.x, gridDim.x, w.run[0], ln.group, ln.heads, has, passes);
  HeadWalk at = in;
  const T* px;
  T* out;
  const int to_b = un.b - un.a;
  int64_t step;
  bool key_in, key;
  auto seek_in = [&] {
    key_in = in.head >= queries;
    const HeadSide& side = a.side[key_in];
    px = static_cast<const T*>(side.x) + in.token * side.ld + (in.head - (key_in ? queries : 0)) * side.step + un.a;
    step = ln.heads * side.step;
  };
  auto seek = [&] {
    key = at.head >= queries;
    const HeadSide& side = a.side[key];
    out = static_cast<T*>(side.out) + ((int64_t)at.token * side.heads + at.head - (key ? queries : 0)) * a.dim + un.a;
  };
  bool other_in = true, other = true;      // another token than in the pass before
  auto fetch = [&] {
    if (in.live()) {
      fill.copy(&fill.piece(0), px);
      fill.copy(&fill.piece(1), px + to_b);
      if (other_in && a.positions) fill.copy(fill.position, a.positions + in.token);
    }
    other_in = in.next(ln.heads);
    if (other_in || (!key_in && in.head >= queries)) seek_in();
    else px += step;
    fill.next();
  };
  seek_in();
  seek();
  #pragma unroll
  for (int d = 0; d < kHeadRing; ++d) {
    if (d < passes) fetch();
    copies_commit();
  }
  Piece<E> c, s;
  int64_t pos = -1;
  for (int i = 0; i < passes; ++i) {
    copies_wait<kHeadRing - 1>();
    const bool live = at.live();
    if (live && other) {
      pos = !a.rotary ? 0 : a.positions ? *slots.position : at.token % a.period;
      if (pos >= a.table && a.rotary) pos = -1;
      angles(c, s, a, pos, un);
    }
    Piece<E> x, y;      // of a group past the end: whatever was there, and goes nowhere
    widen(x, slots.piece(0));
    widen(y, slots.piece(1));
    if (i + kHeadRing < passes) fetch();
    copies_commit();
    slots.next();
    float2 sq = mul2(x.v[0], x.v[0]);
    #pragma unroll
    for (int j = 1; j < E / 2; ++j) sq = fma2(x.v[j], x.v[j], sq);
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) sq = fma2(y.v[j], y.v[j], sq);
    const float rstd = rsqrt_fast(fmaf(ln.sum(sq.x + sq.y), inv, a.eps));
    if (live) {
      Raw ra = Raw{}, rb = Raw{};
      if (pos >= 0) {
        Piece<E> wx;
        load_weights(wx, weights[key], 0);
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) x.v[j] = mul2(mul2(x.v[j], both(rstd)), wx.v[j]);
        load_weights(wx, weights[key], 1);
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) y.v[j] = mul2(mul2(y.v[j], both(rstd)), wx.v[j]);
        turn<E, NB>(x, y, c, s);
        ra = pack<T>(x);
        rb = pack<T>(y);
      }
      *reinterpret_cast<Raw*>(out) = ra;
      *reinterpret_cast<Raw*>(out + to_b) = rb;
    }
    other = at.next(ln.heads);
    if (other || (!key && at.head >= queries)) seek();
    else out += ln.heads * a.dim;
  }
}

template <typename T, int E, int G, bool NB>
__global__ void __launch_bounds__(kHeadThreads, 2)
heads_piece_bwd_kernel(const __grid_constant__ Heads a, const __grid_constant__ HeadWork w) {
  using Raw = typename RawPiece<T, E>::type;
  extern __shared__ uint4 ring[];
  __shared__ HeadWeights<E> weights;
  __shared__ alignas(16) float sums[kHeadWarps * kPieceDim];
  pdl_wait();
  const int key = (int)blockIdx.x >= w.blocks[0], warp = threadIdx.x >> 5;
  const HeadSide& side = a.side[key];
  const Lanes<G> ln(a.dim / (2 * E));
  const Unit<E, NB> un(a.dim, a.rotary, ln.lane);
  if (warp == 0) stage_weights(weights, side, un, w.wbf16);
  __syncthreads();
  const float inv = 1.f / (float)a.dim;
  const bool has = un.any && ln.group < ln.heads;
  HeadRing<Raw, 4> slots(ring, has), fill = slots;
  int passes;
  HeadWalk in = walk_of(a, side.heads, (int)blockIdx.x - (key ? w.blocks[0] : 0), w.blocks[key], w.run[key],
                        ln.group, ln.heads, has, passes);
  HeadWalk at = in;
  const T* const x0 = static_cast<const T*>(side.x) + un.a;
  const T* const d0 = static_cast<const T*>(side.dy) + un.a;
  const T* px = x0 + in.token * side.ld + in.head * side.step;
  const T* pd = d0 + in.token * side.lddy + in.head * side.stepdy;
  const int to_b = un.b - un.a;
  const int64_t step = ln.heads * side.step, step_d = ln.heads * side.stepdy;
  bool other_in = true, other = true;
  auto fetch = [&] {
    if (in.live()) {
      fill.copy(&fill.piece(0), px);
      fill.copy(&fill.piece(1), px + to_b);
      fill.copy(&fill.piece(2), pd);
      fill.copy(&fill.piece(3), pd + to_b);
      if (other_in && a.positions) fill.copy(fill.position, a.positions + in.token);
    }
    px += step;
    pd += step_d;
    other_in = in.next(ln.heads);
    if (other_in) {
      px = x0 + in.token * side.ld + in.head * side.step;
      pd = d0 + in.token * side.lddy + in.head * side.stepdy;
    }
    fill.next();
  };
  #pragma unroll
  for (int d = 0; d < kHeadRing; ++d) {
    if (d < passes) fetch();
    copies_commit();
  }
  T* const out0 = static_cast<T*>(side.out) + un.a;
  Piece<E> sa, sb, c, s;
  clear(sa);
  clear(sb);
  clear(c);      // of lanes without work, whose zeros stay zeros
  clear(s);
  int64_t pos = -1;
  for (int i = 0; i < passes; ++i) {
    copies_wait<kHeadRing - 1>();
    const bool live = at.live();
    if (live && other) {
      pos = !a.rotary ? 0 : a.positions ? *slots.position : at.token % a.period;
      if (pos >= a.table && a.rotary) pos = -1;
      angles(c, s, a, pos, un);
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) s.v[j] = make_float2(-s.v[j].x, -s.v[j].y);      // turned back
    }
    const bool counts = live && pos >= 0;
    Piece<E> x, y, g, h;
    widen(x, slots.piece(0));
    widen(y, slots.piece(1));
    widen(g, slots.piece(2));
    widen(h, slots.piece(3));
    if (i + kHeadRing < passes) fetch();
    copies_commit();
    slots.next();
    turn<E, NB>(g, h, c, s);
    float2 sq = both(0.f), dot = both(0.f);
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) sq = fma2(x.v[j], x.v[j], fma2(y.v[j], y.v[j], sq));
    const float rstd = rsqrt_fast(fmaf(ln.sum(sq.x + sq.y), inv, a.eps));
    // h = x rstd; the sums of g h; then g w in g's place
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      x.v[j] = mul2(x.v[j], both(rstd));
      y.v[j] = mul2(y.v[j], both(rstd));
    }
    if (counts) {
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        sa.v[j] = fma2(g.v[j], x.v[j], sa.v[j]);
        sb.v[j] = fma2(h.v[j], y.v[j], sb.v[j]);
      }
      Piece<E> wa;
      load_weights(wa, weights, 0);
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) g.v[j] = mul2(g.v[j], wa.v[j]);
      load_weights(wa, weights, 1);
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) h.v[j] = mul2(h.v[j], wa.v[j]);
    }
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) dot = fma2(g.v[j], x.v[j], fma2(h.v[j], y.v[j], dot));
    // dx = rstd (g w - h mean(g w h))
    const float mean = ln.sum(dot.x + dot.y) * inv;
    if (live && side.out) {
      Raw ra = Raw{}, rb = Raw{};
      if (counts) {
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          x.v[j] = mul2(fma2(x.v[j], both(-mean), g.v[j]), both(rstd));
          y.v[j] = mul2(fma2(y.v[j], both(-mean), h.v[j]), both(rstd));
        }
        ra = pack<T>(x);
        rb = pack<T>(y);
      }
      T* const out = out0 + (int64_t)at.n * a.dim;
      *reinterpret_cast<Raw*>(out) = ra;
      *reinterpret_cast<Raw*>(out + to_b) = rb;
    }
    other = at.next(ln.heads);
  }
  if (!a.part) return;
  // the warp's groups, then the block's warps in order
  __syncwarp();
  for (int group = 0; group < ln.heads; ++group) {
    if (ln.group == group && un.any) {
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        float2* const ta = reinterpret_cast<float2*>(sums + warp * a.dim + un.a) + j;
        float2* const tb = reinterpret_cast<float2*>(sums + warp * a.dim + un.b) + j;
        *ta = group ? add2(*ta, sa.v[j]) : sa.v[j];
        *tb = group ? add2(*tb, sb.v[j]) : sb.v[j];
      }
    }
    __syncwarp();
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.dim; i += kHeadThreads) {
    float v = 0.f;
    #pragma unroll
    for (int k = 0; k < kHeadWarps; ++k) v += sums[k * a.dim + i];
    a.part[(int64_t)blockIdx.x * a.dim + i] = v;
  }
}

// 32 columns of one side a block, added up by eight warps: rows of `part`
// from first[side] on, or (both_rows) each row with both sides' columns
struct HeadJoin { const float* part; int64_t ld; int first[2], parts[2]; bool both_rows; void* out[2]; };
template <typename WT>
__global__ void __launch_bounds__(kHeadThreads) heads_join_kernel(int dim, const __grid_constant__ HeadJoin j) {
  __shared__ float sums[kHeadWarps][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, key = blockIdx.y, i = blockIdx.x * 32 + lane;
  const float* part = j.part + j.first[key] * j.ld + (j.both_rows ? key * dim : 0) + i;
  float v = 0.f;
  if (i < dim) {
    #pragma unroll 4
    for (int p = warp; p < j.parts[key]; p += kHeadWarps) v += part[p * j.ld];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp > 0 || i >= dim) return;
  v = 0.f;
  #pragma unroll
  for (int k = 0; k < kHeadWarps; ++k) v += sums[k][lane];
  if (j.out[key]) static_cast<WT*>(j.out[key])[i] = from_f<WT>(v);
}

// --------------------------------------------------------------------- host

int64_t head_parts(int64_t tokens, int heads) {
  const int64_t want = (tokens * heads + kHeadWarps - 1) / kHeadWarps;
  return want < kHeadParts ? want : kHeadParts;
}

muon_status check_heads(int64_t tokens, int q_heads, int k_heads, int dim, int rotary, int dtype,
                        int wdtype, float eps, const float* cos, const float* sin, int64_t table,
                        const int64_t* positions, int64_t period) {
  if (tokens < 0 || q_heads < 0 || k_heads < 0 || rotary < 0 || !(eps >= 0.f) || std::isinf(eps))
    return MUON_ERR_INVALID_ARG;
  if (tokens >= (int64_t)1 << 31 || q_heads > 65536 || k_heads > 65536 || dim < 1 ||
      dim > kHeadMaxDim || rotary > dim || rotary % 2)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  if (!known(dtype) || !known(wdtype)) return MUON_ERR_DTYPE;
  if (rotary && (table < 0 || (table > 0 && (!cos || !sin)) || (!positions && period < 1)))
    return MUON_ERR_INVALID_ARG;
  if (off(cos, 4) || off(sin, 4) || off(positions, 8)) return MUON_ERR_ALIGNMENT;
  return MUON_OK;
}

// Whether all heads are made of whole, aligned units of two pieces of `e` elements
bool whole_units(const Heads& a, int e, size_t es) {
  const int64_t all = a.tokens * (a.side[0].heads + a.side[1].heads);
  bool ok = all < kMostHeads && a.dim % (2 * e) == 0 && a.rotary % (2 * e) == 0 && a.dim <= kPieceDim && a.dim <= 64 * e &&
            !off(a.cos, 16) && !off(a.sin, 16);
  for (const HeadSide& s : a.side) {
    if (!s.heads) continue;
    for (const void* p : {s.x, s.dy, (const void*)s.out}) ok = ok && !off(p, e * es);
    for (const int64_t n : {s.ld, s.step, s.lddy, s.stepdy}) ok = ok && n % e == 0;
  }
  return ok;
}

// f(pieces of E elements, lanes a head, heads a warp), the first two as integral constants:
// 16-byte pieces where heads allow them, else pieces of four; the least lanes that hold a head,
// a power of two of them unless fewer let more heads in.  False where neither piece fits.
template <typename T, typename F> bool by_units(const Heads& a, F f) {
  auto lanes = [&](auto e) {
    constexpr int E = decltype(e)::value;
    const int l = a.dim / (2 * E), g = l <= 2 ? 2 : l <= 4 ? 4 : l <= 8 ? 8 : l <= 16 ? 16 : 32;
    if (32 / l > 32 / g && l > 2) f(e, std::integral_constant<int, 0>(), 32 / l);
    else if (g == 2) f(e, std::integral_constant<int, 2>(), 16);
    else if (g == 4) f(e, std::integral_constant<int, 4>(), 8);
    else if (g == 8) f(e, std::integral_constant<int, 8>(), 4);
    else if (g == 16) f(e, std::integral_constant<int, 16>(), 2);
    else f(e, std::integral_constant<int, 32>(), 1);
  };
  if (whole_units(a, kEl<T>, sizeof(T))) {
    lanes(std::integral_constant<int, kEl<T>>());
    return true;
  }
  if (kEl<T> > 4 && whole_units(a, 4, sizeof(T))) {
    lanes(std::integral_constant<int, 4>());
    return true;
  }
  return false;
}

// Blocks and a run for `n` heads, of which a token has `of_token`; B heads a pass of a warp.  A run
// is a token's heads, or what a warp has at all.
void share_out(int64_t n, int of_token, int B, int most, int& blocks, int& run) {
  const int64_t passes = (n + B - 1) / B;
  const int64_t of_warp = (passes + (int64_t)most * kHeadWarps - 1) / ((int64_t)most * kHeadWarps);
  run = (int)std::min<int64_t>((of_token + B - 1) / B, of_warp);
  blocks = (int)std::min<int64_t>((passes + (int64_t)run * kHeadWarps - 1) / ((int64_t)run * kHeadWarps), most);
}
// Blocks of the forward pass: as many as are resident, three an SM, or up to eight times as many.
// Resident blocks go in step, all reading and then all writing, which wastes HBM; more blocks have
// more beginnings, which cost instructions, and bf16 has twice as many of those a byte.  So fp32 takes
// many, and bf16 from where the two cross.  In us, with 456 and with up to 3648 blocks (a warp has about
// six passes at the least: [8192, 32 + 8, 64] fp32, with 1824 blocks 28 and with 3648 33):
//   [tokens, 32 + 8, 128]  2048       4096       8192       16384      32768
//   bf16                   9.7, 9.7   18.3, 17.7 31.1, 34.2 62.0, 61.5 123.7, 103.9
//   fp32                   12.3, 14.4 31.6, 28.9 60.7, 52.7 110.8, 102 217, 200
//   bf16 [16384, 12 + 12, 192] 57.2, 70.4, [65536, 16 + 4, 64] 65.7, 73.9, [8192, 16 + 16, 256] 51.2, 52.2
//   fp32                       111.6, 95.1                     116, 102                         95.6, 82.5
// (bf16 of 2^26 to 2^27 elements would take a few percent less with 912 to 1824 at 40 heads, and a few more
// at 20 and 24.)
int forward_blocks(const Heads& a, int B, size_t es) {
  const int64_t heads = a.tokens * (a.side[0].heads + a.side[1].heads);
  if (es == 2 && heads * a.dim < (int64_t)1 << 27) return 456;
  return (int)std::max<int64_t>(456, std::min<int64_t>(kMostBlocks, heads / B / (kHeadWarps * 45 / 8)));
}
// out of `most` blocks
HeadWork work_of(const Heads& a, int B, int most, int wbf16) {
  HeadWork w = {{0, 0}, {1, 1}, wbf16};
  const int q = a.side[0].heads, k = a.side[1].heads;
  int for_q = (int)((double)most * q / (q + k) + 0.5);
  if (k && for_q > most - 1) for_q = most - 1;
  if (q) share_out(a.tokens * q, q, B, for_q < 1 ? 1 : for_q, w.blocks[0], w.run[0]);
  if (k) share_out(a.tokens * k, k, B, most - w.blocks[0], w.blocks[1], w.run[1]);
  return w;
}

template <typename F> cudaError_t by_both(int dtype, int wdtype, F f) {
  return by_type(dtype, [&](auto t) { return by_type(wdtype, [&](auto w) { return f(t, w); }); });
}

}  // namespace

}  // namespace muon

using namespace muon;

extern "C" muon_status muon_norm_rotate_heads(
    int64_t tokens, int q_heads, int k_heads, int dim, int rotary, int dtype, int wdtype,
    const void* q, int64_t ldq, int64_t q_step, const void* k, int64_t ldk, int64_t k_step,
    const void* q_weight, const void* k_weight, float eps, const float* cos, const float* sin,
    int64_t table, const int64_t* positions, int64_t period, int neighbours, void* q_out,
    void* k_out, void* stream) {
  const muon_status st = check_heads(tokens, q_heads, k_heads, dim, rotary, dtype, wdtype, eps, cos, sin,
                                     table, positions, period);
  if (st != MUON_OK) return st;
  if (ldq < 0 || ldk < 0 || q_step < 0 || k_step < 0 || (tokens > 0 && q_heads > 0 && (!q || !q_out)) ||
      (tokens > 0 && k_heads > 0 && (!k || !k_out)))
    return MUON_ERR_INVALID_ARG;
  if (any_off(size_of(dtype), q, k, q_out, k_out) || any_off(size_of(wdtype), q_weight, k_weight))
    return MUON_ERR_ALIGNMENT;
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  if (tokens == 0 || q_heads + k_heads == 0) return MUON_OK;
  NvtxRange range("muon_norm_rotate_heads");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Heads a = {tokens, table, period, dim, rotary, neighbours, eps, cos, sin, positions,
                   {{q, nullptr, q_weight, ldq, q_step, 0, 0, q_out, q_heads},
                    {k, nullptr, k_weight, ldk, k_step, 0, 0, k_out, k_heads}},
                   nullptr};
  const int64_t want = (tokens * (q_heads + k_heads) + kHeadWarps - 1) / kHeadWarps;
  const cudaError_t e = by_both(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    cudaError_t e = cudaSuccess;
    if (by_units<T>(a, [&](auto pe, auto pg, int B) {
          constexpr int E = decltype(pe)::value, G = decltype(pg)::value;
          constexpr size_t smem = HeadRing<typename RawPiece<T, E>::type, 2>::kBytes;
          HeadWork hw = {{0, 0}, {1, 1}, wdtype == MUON_BF16};
          share_out(tokens * (q_heads + k_heads), q_heads + k_heads, B, forward_blocks(a, B, sizeof(T)), hw.blocks[0],
                    hw.run[0]);
          e = launch_k(neighbours ? heads_piece_kernel<T, E, G, true> : heads_piece_kernel<T, E, G, false>,
                       dim3(hw.blocks[0]), dim3(kHeadThreads), smem, s, true, a, hw);
        }))
      return e;
    return launch_k(heads_kernel<decltype(t), decltype(w)>, dim3((unsigned)(want < 152 * 8 ? want : 152 * 8)),
                    dim3(kHeadThreads), 0, s, true, a);
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" muon_status muon_norm_rotate_heads_workspace_bytes(int64_t tokens, int q_heads,
                                                              int k_heads, int dim, size_t* out) {
  if (!out || tokens < 0 || q_heads < 0 || k_heads < 0) return MUON_ERR_INVALID_ARG;
  if (tokens >= (int64_t)1 << 31 || q_heads > 65536 || k_heads > 65536 || dim < 1 || dim > kHeadMaxDim)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  *out = (size_t)head_parts(tokens, q_heads + k_heads) * 2 * dim * sizeof(float) + 256;
  return MUON_OK;
}

extern "C" muon_status muon_norm_rotate_heads_backward(
    int64_t tokens, int q_heads, int k_heads, int dim, int rotary, int dtype, int wdtype,
    const void* dq, int64_t lddq, int64_t dq_step, const void* dk, int64_t lddk, int64_t dk_step,
    const void* q, int64_t ldq, int64_t q_step, const void* k, int64_t ldk, int64_t k_step,
    const void* q_weight, const void* k_weight, float eps, const float* cos, const float* sin,
    int64_t table, const int64_t* positions, int64_t period, int neighbours, void* q_grad,
    void* k_grad, void* q_dweight, void* k_dweight, void* workspace, size_t ws_bytes,
    void* stream) {
  const muon_status st = check_heads(tokens, q_heads, k_heads, dim, rotary, dtype, wdtype, eps, cos, sin,
                                     table, positions, period);
  if (st != MUON_OK) return st;
  if (lddq < 0 || lddk < 0 || dq_step < 0 || dk_step < 0 || ldq < 0 || ldk < 0 || q_step < 0 ||
      k_step < 0 || (tokens > 0 && q_heads > 0 && (!q || !dq)) ||
      (tokens > 0 && k_heads > 0 && (!k || !dk)))
    return MUON_ERR_INVALID_ARG;
  const size_t es = size_of(dtype), ws = size_of(wdtype);
  if (any_off(es, dq, dk, q, k, q_grad, k_grad) || any_off(ws, q_weight, k_weight, q_dweight, k_dweight))
    return MUON_ERR_ALIGNMENT;
  const bool none = tokens == 0 || q_heads + k_heads == 0, sums = q_dweight || k_dweight;
  if (sums && !none) {
    size_t need = 0;
    muon_norm_rotate_heads_workspace_bytes(tokens, q_heads, k_heads, dim, &need);
    if (!workspace) return MUON_ERR_INVALID_ARG;
    if (off(workspace, 256)) return MUON_ERR_ALIGNMENT;
    if (ws_bytes < need) return MUON_ERR_WORKSPACE;
  }
  if (fault_switch() == kFaultLaunch) return MUON_ERR_CUDA;
  NvtxRange range("muon_norm_rotate_heads_backward");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (none) {     // empty sums
    for (void* d : {q_dweight, k_dweight})
      if (d && cudaMemsetAsync(d, 0, dim * ws, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  const Heads a = {tokens, table, period, dim, rotary, neighbours, eps, cos, sin, positions,
                   {{q, dq, q_weight, ldq, q_step, lddq, dq_step, q_grad, q_heads},
                    {k, dk, k_weight, ldk, k_step, lddk, dk_step, k_grad, k_heads}},
                   sums ? static_cast<float*>(workspace) : nullptr};
  const int parts = (int)head_parts(tokens, q_heads + k_heads);
  const cudaError_t e = by_both(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using WT = decltype(w);
    cudaError_t e = cudaSuccess;
    HeadJoin j = {a.part, dim, {0, 0}, {0, 0}, false, {q_dweight, k_dweight}};
    if (!by_units<T>(a, [&](auto pe, auto pg, int B) {
          constexpr int E = decltype(pe)::value, G = decltype(pg)::value;
          constexpr size_t smem = HeadRing<typename RawPiece<T, E>::type, 4>::kBytes;
          const HeadWork hw = work_of(a, B, 2 * parts < kHeadParts ? 2 * parts : kHeadParts, wdtype == MUON_BF16);
          j.first[1] = j.parts[0] = hw.blocks[0];
          j.parts[1] = hw.blocks[1];
          e = neighbours ? allow_shared<heads_piece_bwd_kernel<T, E, G, true>>(smem)
                         : allow_shared<heads_piece_bwd_kernel<T, E, G, false>>(smem);
          if (e == cudaSuccess)
            e = launch_k(neighbours ? heads_piece_bwd_kernel<T, E, G, true> : heads_piece_bwd_kernel<T, E, G, false>,
                         dim3(hw.blocks[0] + hw.blocks[1]), dim3(kHeadThreads), smem, s, true, a, hw);
        })) {
      const size_t smem = (size_t)kHeadWarps * 3 * dim * sizeof(float);
      j = {a.part, 2 * dim, {0, 0}, {parts, parts}, true, {q_dweight, k_dweight}};
      e = allow_shared<heads_bwd_kernel<T, WT>>(kHeadWarps * 3 * kHeadMaxDim * sizeof(float));
      if (e == cudaSuccess)
        e = launch_k(heads_bwd_kernel<T, WT>, dim3(parts), dim3(kHeadThreads), smem, s, true, a);
    }
    if (e == cudaSuccess && sums)
      e = launch_k(heads_join_kernel<WT>, dim3((dim + 31) / 32, 2), dim3(kHeadThreads), 0, s, true, dim, j);
    return e;
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
