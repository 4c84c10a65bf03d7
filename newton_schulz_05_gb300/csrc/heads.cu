// Norms of query and key heads with the rotation of positions, and the gradient.
#include "sequence.cuh"

#include <type_traits>

namespace muon {

namespace {

constexpr int kHeadThreads = 256, kHeadWarps = kHeadThreads / 32;
constexpr int kHeadMaxDim = 1024;
constexpr int kHeadParts = 304;       // blocks of the gradient, images of its weight sums

// Queries or keys: heads `step` elements apart, tokens `ld`
struct HeadSide {
  const void *x, *dy, *weight;
  int64_t ld, step, lddy, stepdy;
  void *out, *dweight;
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
template <int E> __device__ __forceinline__ void load_floats(Piece<E>& v, const float* p) {
  #pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    const float4 f = reinterpret_cast<const float4*>(p)[q];
    v.v[2 * q] = make_float2(f.x, f.y);
    v.v[2 * q + 1] = make_float2(f.z, f.w);
  }
}

// A lane's two pieces of a head.  Those of the rotated part are turned into one another,
// so no lane needs another's: m and m + rotary / 2 for one half against the other, or
// neighbouring pieces, which hold their pairs whole.  Both ways they have the E pairs
// from E * unit on.  G lanes a head, of which dim / 2E have work.
template <int E> struct Unit {
  int a, b;              // first elements of the pieces
  bool any, turned;
  __device__ __forceinline__ Unit(int dim, int rotary, bool neighbours, int u) {
    any = 2 * E * u < dim;
    turned = 2 * E * u < rotary;
    const bool halves = turned && !neighbours;
    a = halves ? E * u : 2 * E * u;
    b = halves ? E * u + rotary / 2 : 2 * E * u + E;
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
      one(a.v[j], j & 1 ? c.v[j / 2].y : c.v[j / 2].x, j & 1 ? s.v[j / 2].y : s.v[j / 2].x);
      const int k = j + E / 2;
      one(b.v[j], k & 1 ? c.v[k / 2].y : c.v[k / 2].x, k & 1 ? s.v[k / 2].y : s.v[k / 2].x);
    }
  } else {
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      const float2 x = a.v[j], y = b.v[j], n = make_float2(-s.v[j].x, -s.v[j].y);
      a.v[j] = fma2(y, n, mul2(x, c.v[j]));
      b.v[j] = fma2(x, s.v[j], mul2(y, c.v[j]));
    }
  }
}
template <int G> __device__ __forceinline__ float group_sum(float v) {
  #pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// What a warp works through: `chunks` items a token, of `passes` passes over 32 / G heads.
// The passes of a token: those of the queries, then those of the keys.
struct HeadWork { int64_t items; int chunks, passes, q_passes, all_passes; };

// both sides' weights in fp32 (1 where there are none), for every thread of the block
__device__ __forceinline__ void stage_weights(float* to, const Heads& a, int wbf16) {
  for (int i = threadIdx.x; i < 2 * a.dim; i += kHeadThreads) {
    const void* w = a.side[i >= a.dim].weight;
    const int j = i >= a.dim ? i - a.dim : i;
    to[i] = !w ? 1.f : wbf16 ? to_f(static_cast<const __nv_bfloat16*>(w)[j]) : static_cast<const float*>(w)[j];
  }
  __syncthreads();
}

constexpr int kPieceDim = 512;        // widest head of these kernels

template <typename T, int E, int G, bool NB>
__global__ void __launch_bounds__(kHeadThreads, 3)
heads_piece_kernel(const __grid_constant__ Heads a, const __grid_constant__ HeadWork w, int wbf16) {
  using Raw = typename RawPiece<T, E>::type;
  constexpr int B = 32 / G, U = 2;        // heads a pass, passes in flight
  __shared__ alignas(16) float weights[2 * kPieceDim];
  pdl_wait();
  stage_weights(weights, a, wbf16);
  const int lane = threadIdx.x & 31, group = lane / G;
  const Unit<E> un(a.dim, a.rotary, NB, lane % G);
  const float inv = 1.f / (float)a.dim;
  for (int64_t item = (int64_t)blockIdx.x * kHeadWarps + (threadIdx.x >> 5); item < w.items;
       item += (int64_t)gridDim.x * kHeadWarps) {
    const int64_t t = w.chunks == 1 ? item : item / w.chunks;
    int pass = w.chunks == 1 ? 0 : (int)(item % w.chunks) * w.passes;
    const int end = min(pass + w.passes, w.all_passes);
    const int64_t pos = position_of(a, t);
    Piece<E> c, s;
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) {
      c.v[j] = both(1.f);
      s.v[j] = both(0.f);
    }
    if (un.turned && pos >= 0) {
      load_floats(c, a.cos + pos * (a.rotary / 2) + E * (lane % G));
      load_floats(s, a.sin + pos * (a.rotary / 2) + E * (lane % G));
    }
    for (; pass < end; pass += U) {
      Raw ra[U], rb[U];
      int head[U];
      bool key[U], has[U];
      #pragma unroll
      for (int k = 0; k < U; ++k) {
        key[k] = pass + k >= w.q_passes;
        head[k] = (key[k] ? pass + k - w.q_passes : pass + k) * B + group;
        has[k] = pass + k < end && un.any && head[k] < a.side[key[k]].heads;
        ra[k] = rb[k] = Raw{};
        if (has[k] && pos >= 0) {
          const T* x = static_cast<const T*>(a.side[key[k]].x) + t * a.side[key[k]].ld + head[k] * a.side[key[k]].step;
          ra[k] = *reinterpret_cast<const Raw*>(x + un.a);
          rb[k] = *reinterpret_cast<const Raw*>(x + un.b);
        }
      }
      #pragma unroll
      for (int k = 0; k < U; ++k) {
        Piece<E> x, y, wx, wy;
        widen(x, ra[k]);
        widen(y, rb[k]);
        float2 sq = both(0.f);
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) sq = fma2(x.v[j], x.v[j], fma2(y.v[j], y.v[j], sq));
        const float rstd = 1.f / sqrtf(fmaf(group_sum<G>(sq.x + sq.y), inv, a.eps));
        if (!has[k]) continue;
        load_floats(wx, weights + key[k] * a.dim + un.a);
        load_floats(wy, weights + key[k] * a.dim + un.b);
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          x.v[j] = mul2(mul2(x.v[j], both(rstd)), wx.v[j]);
          y.v[j] = mul2(mul2(y.v[j], both(rstd)), wy.v[j]);
        }
        if (un.turned) turn<E, NB>(x, y, c, s);
        if (pos < 0) {
          clear(x);
          clear(y);
        }
        T* out = static_cast<T*>(a.side[key[k]].out) + (t * a.side[key[k]].heads + head[k]) * a.dim;
        *reinterpret_cast<Raw*>(out + un.a) = pack<T>(x);
        *reinterpret_cast<Raw*>(out + un.b) = pack<T>(y);
      }
    }
  }
}

// The queries of all tokens first, then the keys: one set of weight sums in registers.
template <typename T, int E, int G, bool NB>
__global__ void __launch_bounds__(kHeadThreads, 2)
heads_piece_bwd_kernel(const __grid_constant__ Heads a, const __grid_constant__ HeadWork wq,
                       const __grid_constant__ HeadWork wk, int wbf16) {
  using Raw = typename RawPiece<T, E>::type;
  constexpr int B = 32 / G;
  __shared__ alignas(16) float weights[2 * kPieceDim], sums[kHeadWarps * kPieceDim];
  pdl_wait();
  stage_weights(weights, a, wbf16);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = lane / G;
  const Unit<E> un(a.dim, a.rotary, NB, lane % G);
  const float inv = 1.f / (float)a.dim;
  for (int key = 0; key < 2; ++key) {
    const HeadWork& w = key ? wk : wq;
    const HeadSide& side = a.side[key];
    Piece<E> sa, sb, wa, wb;
    clear(sa);
    clear(sb);
    clear(wa);
    clear(wb);
    if (un.any) {
      load_floats(wa, weights + key * a.dim + un.a);
      load_floats(wb, weights + key * a.dim + un.b);
    }
    for (int64_t item = (int64_t)blockIdx.x * kHeadWarps + warp; item < w.items;
         item += (int64_t)gridDim.x * kHeadWarps) {
      const int64_t t = w.chunks == 1 ? item : item / w.chunks;
      int pass = w.chunks == 1 ? 0 : (int)(item % w.chunks) * w.passes;
      const int end = min(pass + w.passes, w.all_passes);
      const int64_t pos = position_of(a, t);
      Piece<E> c, s;
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        c.v[j] = both(1.f);
        s.v[j] = both(0.f);
      }
      if (un.turned && pos >= 0) {
        load_floats(c, a.cos + pos * (a.rotary / 2) + E * (lane % G));
        load_floats(s, a.sin + pos * (a.rotary / 2) + E * (lane % G));
      }
      Raw xa, xb, da, db;
      auto fetch = [&](int p) {
        const int head = p * B + group;
        xa = xb = da = db = Raw{};
        if (pos < 0 || p >= end || !un.any || head >= side.heads) return;
        const T* x = static_cast<const T*>(side.x) + t * side.ld + head * side.step;
        const T* d = static_cast<const T*>(side.dy) + t * side.lddy + head * side.stepdy;
        xa = *reinterpret_cast<const Raw*>(x + un.a);
        xb = *reinterpret_cast<const Raw*>(x + un.b);
        da = *reinterpret_cast<const Raw*>(d + un.a);
        db = *reinterpret_cast<const Raw*>(d + un.b);
      };
      fetch(pass);
      for (; pass < end; ++pass) {
        Piece<E> x, y, g, h;
        widen(x, xa);
        widen(y, xb);
        widen(g, da);
        widen(h, db);
        fetch(pass + 1);
        if (un.turned) {
          Piece<E> n;
          #pragma unroll
          for (int j = 0; j < E / 2; ++j) n.v[j] = make_float2(-s.v[j].x, -s.v[j].y);
          turn<E, NB>(g, h, c, n);
        }
        float2 sq = both(0.f), dot = both(0.f);
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          sq = fma2(x.v[j], x.v[j], fma2(y.v[j], y.v[j], sq));
          dot = fma2(mul2(g.v[j], wa.v[j]), x.v[j], fma2(mul2(h.v[j], wb.v[j]), y.v[j], dot));
        }
        const int head = pass * B + group;
        const bool live = pos >= 0 && head < side.heads;      // else 1 / 0 without eps
        const float ms = fmaf(group_sum<G>(sq.x + sq.y), inv, a.eps);
        const float rstd = live ? 1.f / sqrtf(ms) : 0.f;
        // dx = rstd (g w - h mean(g w h)) with h = x rstd
        const float mean = group_sum<G>(dot.x + dot.y) * rstd * inv;
        #pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          x.v[j] = mul2(x.v[j], both(rstd));
          y.v[j] = mul2(y.v[j], both(rstd));
          sa.v[j] = fma2(g.v[j], x.v[j], sa.v[j]);
          sb.v[j] = fma2(h.v[j], y.v[j], sb.v[j]);
          x.v[j] = mul2(fma2(x.v[j], both(-mean), mul2(g.v[j], wa.v[j])), both(rstd));
          y.v[j] = mul2(fma2(y.v[j], both(-mean), mul2(h.v[j], wb.v[j])), both(rstd));
        }
        if (side.out && un.any && head < side.heads) {
          T* out = static_cast<T*>(side.out) + (t * side.heads + head) * a.dim;
          *reinterpret_cast<Raw*>(out + un.a) = pack<T>(x);
          *reinterpret_cast<Raw*>(out + un.b) = pack<T>(y);
        }
      }
    }
    if (!a.part) continue;
    // the warp's groups, then the block's warps in order
    #pragma unroll
    for (int o = G; o < 32; o <<= 1)
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        sa.v[j].x += __shfl_xor_sync(~0u, sa.v[j].x, o);
        sa.v[j].y += __shfl_xor_sync(~0u, sa.v[j].y, o);
        sb.v[j].x += __shfl_xor_sync(~0u, sb.v[j].x, o);
        sb.v[j].y += __shfl_xor_sync(~0u, sb.v[j].y, o);
      }
    __syncthreads();
    if (group == 0 && un.any) {
      #pragma unroll
      for (int j = 0; j < E / 2; ++j) {
        reinterpret_cast<float2*>(sums + warp * a.dim + un.a)[j] = sa.v[j];
        reinterpret_cast<float2*>(sums + warp * a.dim + un.b)[j] = sb.v[j];
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.dim; i += kHeadThreads) {
      float v = 0.f;
      #pragma unroll
      for (int k = 0; k < kHeadWarps; ++k) v += sums[k * a.dim + i];
      a.part[((int64_t)blockIdx.x * 2 + key) * a.dim + i] = v;
    }
  }
}

// 32 columns a block, added up by eight warps
template <typename WT>
__global__ void __launch_bounds__(kHeadThreads)
heads_join_kernel(int dim, int parts, const float* part, WT* dq, WT* dk) {
  __shared__ float sums[kHeadWarps][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (i < 2 * dim) {
    #pragma unroll 4
    for (int p = warp; p < parts; p += kHeadWarps) v += part[(int64_t)p * 2 * dim + i];
  }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp > 0 || i >= 2 * dim) return;
  v = 0.f;
  #pragma unroll
  for (int k = 0; k < kHeadWarps; ++k) v += sums[k][lane];
  WT* out = i < dim ? dq : dk;
  if (out) out[i < dim ? i : i - dim] = from_f<WT>(v);
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
  bool ok = a.dim % (2 * e) == 0 && a.rotary % (2 * e) == 0 && a.dim <= kPieceDim && a.dim <= 64 * e &&
            !off(a.cos, 16) && !off(a.sin, 16);
  for (const HeadSide& s : a.side) {
    if (!s.heads) continue;
    for (const void* p : {s.x, s.dy, (const void*)s.out}) ok = ok && !off(p, e * es);
    for (const int64_t n : {s.ld, s.step, s.lddy, s.stepdy}) ok = ok && n % e == 0;
  }
  return ok;
}

// f(pieces of E elements, lanes a head) as integral constants: 16-byte pieces where heads allow
// them, else pieces of four; the least lanes that hold a head.  False where neither fits.
template <typename T, typename F> bool by_units(const Heads& a, F f) {
  auto lanes = [&](auto e) {
    constexpr int E = decltype(e)::value;
    const int l = a.dim / (2 * E);
    if (l <= 4) f(e, std::integral_constant<int, 4>());
    else if (l <= 8) f(e, std::integral_constant<int, 8>());
    else if (l <= 16) f(e, std::integral_constant<int, 16>());
    else f(e, std::integral_constant<int, 32>());
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

// A warp takes all passes of a token where there are tokens for all warps, else fewer.
HeadWork work_of(int64_t tokens, int q_passes, int all_passes, int64_t warps) {
  int64_t chunks = (warps + tokens - 1) / tokens;
  if (chunks > all_passes) chunks = all_passes;
  if (chunks < 1) chunks = 1;
  const int passes = (int)((all_passes + chunks - 1) / chunks);
  chunks = passes ? (all_passes + passes - 1) / passes : 0;
  return {tokens * chunks, (int)chunks, passes, q_passes, all_passes};
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
                   {{q, nullptr, q_weight, ldq, q_step, 0, 0, q_out, nullptr, q_heads},
                    {k, nullptr, k_weight, ldk, k_step, 0, 0, k_out, nullptr, k_heads}},
                   nullptr};
  const int64_t want = (tokens * (q_heads + k_heads) + kHeadWarps - 1) / kHeadWarps;
  const cudaError_t e = by_both(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    cudaError_t e = cudaSuccess;
    if (by_units<T>(a, [&](auto pe, auto pg) {
          constexpr int E = decltype(pe)::value, G = decltype(pg)::value, B = 32 / G, blocks = 152 * 3;
          const int pq = (q_heads + B - 1) / B, all = pq + (k_heads + B - 1) / B;
          const HeadWork hw = work_of(tokens, pq, all, blocks * kHeadWarps);
          const int64_t need = (hw.items + kHeadWarps - 1) / kHeadWarps;
          e = launch_k(neighbours ? heads_piece_kernel<T, E, G, true> : heads_piece_kernel<T, E, G, false>,
                       dim3((unsigned)(need < blocks ? need : blocks)), dim3(kHeadThreads), 0, s, true, a, hw,
                       (int)(wdtype == MUON_BF16));
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
                   {{q, dq, q_weight, ldq, q_step, lddq, dq_step, q_grad, q_dweight, q_heads},
                    {k, dk, k_weight, ldk, k_step, lddk, dk_step, k_grad, k_dweight, k_heads}},
                   sums ? static_cast<float*>(workspace) : nullptr};
  const int parts = (int)head_parts(tokens, q_heads + k_heads);
  const cudaError_t e = by_both(dtype, wdtype, [&](auto t, auto w) {
    using T = decltype(t);
    using WT = decltype(w);
    cudaError_t e = cudaSuccess;
    int used = parts;
    if (!by_units<T>(a, [&](auto pe, auto pg) {
          constexpr int E = decltype(pe)::value, G = decltype(pg)::value, B = 32 / G;
          const int64_t warps = (int64_t)kHeadParts * kHeadWarps;
          const int pq = (q_heads + B - 1) / B, pk = (k_heads + B - 1) / B;
          const HeadWork wq = work_of(tokens, pq, pq, warps), wk = work_of(tokens, pk, pk, warps);
          const int64_t items = wq.items > wk.items ? wq.items : wk.items;
          const int64_t need = (items + kHeadWarps - 1) / kHeadWarps;
          used = (int)(need < parts ? need : parts);
          e = launch_k(neighbours ? heads_piece_bwd_kernel<T, E, G, true> : heads_piece_bwd_kernel<T, E, G, false>,
                       dim3(used), dim3(kHeadThreads), 0, s, true, a, wq, wk, (int)(wdtype == MUON_BF16));
        })) {
    const size_t smem = (size_t)kHeadWarps * 3 * dim * sizeof(float);
    e = allow_shared<heads_bwd_kernel<T, WT>>(kHeadWarps * 3 * kHeadMaxDim * sizeof(float));
    if (e == cudaSuccess)
      e = launch_k(heads_bwd_kernel<T, WT>, dim3(parts), dim3(kHeadThreads), smem, s, true, a);
    }
    if (e == cudaSuccess && sums)
      e = launch_k(heads_join_kernel<WT>, dim3((2 * dim + 31) / 32), dim3(kHeadThreads), 0, s, true, dim, used, (const float*)a.part,
                   static_cast<WT*>(q_dweight), static_cast<WT*>(k_dweight));
    return e;
  });
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
