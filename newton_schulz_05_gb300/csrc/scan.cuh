// Gated linear recurrence (scan.cu) and its gradient (scan_grad.cu): what the two
// share.
//
// The recurrence is a chain of maps p -> a p + b, and a run of tokens is one such
// map again: the state's factor and what the tokens add.  So the length is cut up: a
// thread takes S tokens of four channels and reduces them to such a run while it reads
// them, the 2 W segments of a block's warps are joined in order through shuffles
// and shared memory, the blocks of a cluster through each other's shared memory, and
// then every thread knows the state in front of its tokens and finishes them from
// registers.  Each input is read once and each output written once; the only serial
// part is the walk over chunks of 2 W S tokens (times the blocks of a cluster).  The
// order of the joins is fixed, so results are the same bits each time.
//
// a = 1 / (1 + exp(-gate)) needs no cases: exp overflows to infinity and a is 0, or
// underflows and a is 1.  A token that is masked or past the end is given the gate
// +infinity and the input 0, which changes nothing.
//
// A block has a strip of 64 channels: 16 lanes of four channels (neighbouring ones
// where rows allow pieces of four, else 16 apart), so a warp holds two segments.
#pragma once

#include "sequence.cuh"

namespace muon {

namespace {

constexpr int kStrip = 64;

// four elements as they lie in memory
template <typename T> struct Raw4;
template <> struct Raw4<__nv_bfloat16> { uint2 u; };
template <> struct Raw4<float> { uint4 u; };
// four channels in fp32
struct Quad { float2 v[2]; };

__device__ __forceinline__ void zero(Raw4<__nv_bfloat16>& r) { r.u = make_uint2(0, 0); }
__device__ __forceinline__ void zero(Raw4<float>& r) { r.u = make_uint4(0, 0, 0, 0); }
__device__ __forceinline__ void infinite(Raw4<__nv_bfloat16>& r) { r.u = make_uint2(0x7f807f80u, 0x7f807f80u); }
__device__ __forceinline__ void infinite(Raw4<float>& r) {
  r.u = make_uint4(0x7f800000u, 0x7f800000u, 0x7f800000u, 0x7f800000u);
}
__device__ __forceinline__ Quad widen(const Raw4<__nv_bfloat16>& r) {
  return {{make_float2(__uint_as_float(r.u.x << 16), __uint_as_float(r.u.x & 0xffff0000u)),
           make_float2(__uint_as_float(r.u.y << 16), __uint_as_float(r.u.y & 0xffff0000u))}};
}
__device__ __forceinline__ Quad widen(const Raw4<float>& r) {
  return {{make_float2(__uint_as_float(r.u.x), __uint_as_float(r.u.y)),
           make_float2(__uint_as_float(r.u.z), __uint_as_float(r.u.w))}};
}
__device__ __forceinline__ Quad quad(float v) { return {{both(v), both(v)}}; }
__device__ __forceinline__ Quad add(const Quad& a, const Quad& b) {
  return {{add2(a.v[0], b.v[0]), add2(a.v[1], b.v[1])}};
}
__device__ __forceinline__ Quad mul(const Quad& a, const Quad& b) {
  return {{mul2(a.v[0], b.v[0]), mul2(a.v[1], b.v[1])}};
}
__device__ __forceinline__ Quad fma(const Quad& a, const Quad& b, const Quad& c) {
  return {{fma2(a.v[0], b.v[0], c.v[0]), fma2(a.v[1], b.v[1], c.v[1])}};
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
// until at most N of the newest groups are in flight
template <int N> __device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Flags of a segment's tokens: its first S lanes hold a byte each from when they are
// asked for until they are needed.
struct Flags { uint32_t starts, live; };
template <int S>
__device__ __forceinline__ Flags ask(const uint8_t* starts, const uint8_t* mask, int64_t row0, int64_t t0,
                                     int64_t length) {
  const int l = threadIdx.x & 15;
  const int64_t t = t0 + l;
  const bool in = l < S && t >= 0 && t < length;
  return {in && starts ? starts[row0 + t] : 0u, in && mask ? mask[row0 + t] : (uint32_t)in};
}
// as bits by token: which are live, and which of those start over
__device__ __forceinline__ Flags bits(const Flags& f) {
  const int half = threadIdx.x & 16;
  const uint32_t live = __ballot_sync(~0u, f.live != 0) >> half & 0xffff;
  return {__ballot_sync(~0u, f.starts != 0) >> half & live, live};
}

// Which channels a lane has: `has` of its four are inside the row.  VEC: four
// neighbours, all inside or all outside.
template <bool VEC> struct Channels {
  int first;      // of the lane, in the row
  int left;       // channels from `first` on that are inside the row
  __device__ __forceinline__ Channels(int strip, int64_t dim) {
    const int l = threadIdx.x & 15;
    first = strip * kStrip + (VEC ? 4 * l : l);
    left = (int)dim - first;
  }
  __device__ __forceinline__ bool any() const { return left > 0; }
  __device__ __forceinline__ int at(int j) const { return VEC ? j : 16 * j; }
  __device__ __forceinline__ bool has(int j) const { return at(j) < left; }

  // p: the lane's first channel
  __device__ __forceinline__ void load(Raw4<__nv_bfloat16>& r, const __nv_bfloat16* p) const {
    if constexpr (VEC) {
      r.u = *reinterpret_cast<const uint2*>(p);
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      uint32_t w[4];
      #pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = has(j) ? q[16 * j] : 0;
      r.u = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    }
  }
  __device__ __forceinline__ void load(Raw4<float>& r, const float* p) const {
    if constexpr (VEC) {
      r.u = *reinterpret_cast<const uint4*>(p);
    } else {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
      uint32_t w[4];
      #pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = has(j) ? q[16 * j] : 0;
      r.u = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // asynchronous copy of a piece into the thread's slot of a ring
  template <typename T> __device__ __forceinline__ static void copy(Raw4<T>* slot, const T* p) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(slot);
    if constexpr (sizeof(T) == 2)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;\n" ::"r"(to), "l"(p) : "memory");
    else
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to), "l"(p) : "memory");
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, const Quad& q) const {
    const __nv_bfloat162 a = __float22bfloat162_rn(q.v[0]), b = __float22bfloat162_rn(q.v[1]);
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(p) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else {
      if (has(0)) p[0] = a.x;
      if (has(1)) p[16] = a.y;
      if (has(2)) p[32] = b.x;
      if (has(3)) p[48] = b.y;
    }
  }
  __device__ __forceinline__ void store(float* p, const Quad& q) const {
    if constexpr (VEC) {
      *reinterpret_cast<float4*>(p) = make_float4(q.v[0].x, q.v[0].y, q.v[1].x, q.v[1].y);
    } else {
      if (has(0)) p[0] = q.v[0].x;
      if (has(1)) p[16] = q.v[0].y;
      if (has(2)) p[32] = q.v[1].x;
      if (has(3)) p[48] = q.v[1].y;
    }
  }
  // fp32 states at p, whatever their alignment
  __device__ __forceinline__ Quad state(const float* p) const {
    float w[4];
    #pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = has(j) ? p[at(j)] : 0.f;
    return {{make_float2(w[0], w[1]), make_float2(w[2], w[3])}};
  }
  __device__ __forceinline__ void put_state(float* p, const Quad& q) const {
    const float w[4] = {q.v[0].x, q.v[0].y, q.v[1].x, q.v[1].y};
    #pragma unroll
    for (int j = 0; j < 4; ++j)
      if (has(j)) p[at(j)] = w[j];
  }
};

// A run of tokens as a map of the state p in front of it: H + P p.  Where P is 1/2 or
// more, m is -(1 - P), with its sign bit set, and the map is p + (H + m p); else m is P.
// 1 - P decides how much of the state a long run forgets, and P has no bits for it: with
// P alone, 3000 tokens of the gate 8 took a constant state off by 1.6e-5 of itself.
// cut: some token of the run starts over, and H is the state whatever p was.
struct Run {
  Quad m, H;
  bool cut;
};
__device__ __forceinline__ bool keeps(float m) { return __float_as_int(m) < 0; }
// from P and 1 - P
__device__ __forceinline__ Quad shares(const Quad& P, const Quad& Q) {
  Quad m;
  #pragma unroll
  for (int j = 0; j < 2; ++j)
    m.v[j] = make_float2(P.v[j].x >= 0.5f ? -Q.v[j].x : P.v[j].x, P.v[j].y >= 0.5f ? -Q.v[j].y : P.v[j].y);
  return m;
}
__device__ __forceinline__ Quad apply(const Run& r, const Quad& p) {
  Quad q = fma(r.m, p, r.H), base;
  #pragma unroll
  for (int j = 0; j < 2; ++j)
    base.v[j] = make_float2(keeps(r.m.v[j].x) ? p.v[j].x : 0.f, keeps(r.m.v[j].y) ? p.v[j].y : 0.f);
  q = add(q, base);
  if (r.cut) q = r.H;
  return q;
}
// the share of two runs, one after the other
__device__ __forceinline__ float both_shares(float a, float b) {
  const bool ka = keeps(a), kb = keeps(b);
  // (1 + a)(1 + b) - 1, a (1 + b), (1 + a) b or a b
  const float m = fmaf(a, b, (kb ? a : 0.f) + (ka ? b : 0.f));
  return ka && kb ? (m < -0.5f ? 1.f + m : -fabsf(m)) : m;
}
// first `a`, then `b`
__device__ __forceinline__ Run then(const Run& a, const Run& b) {
  Run r;
  #pragma unroll
  for (int j = 0; j < 2; ++j)
    r.m.v[j] = make_float2(both_shares(a.m.v[j].x, b.m.v[j].x), both_shares(a.m.v[j].y, b.m.v[j].y));
  r.H = apply(b, a.H);
  r.cut = a.cut || b.cut;
  return r;
}

// what the runs of a block's warps, and of a cluster's blocks, are exchanged through
template <int W, int CL> struct RunSlots {
  float4 m[2][W][16], H[2][W][16];
  float4 cm[2][CL][16], cH[2][CL][16];
  int cut[2][W], ccut[2][CL];
};
__device__ __forceinline__ float4 four(const Quad& q) {
  return make_float4(q.v[0].x, q.v[0].y, q.v[1].x, q.v[1].y);
}
__device__ __forceinline__ Quad quad(const float4& f) {
  return {{make_float2(f.x, f.y), make_float2(f.z, f.w)}};
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
// the address in block `rank` of the cluster of what is at p in this one
__device__ __forceinline__ uint32_t at_rank(const void* p, int rank) {
  uint32_t to;
  const uint32_t from = (uint32_t)__cvta_generic_to_shared(p);
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(from), "r"(rank));
  return to;
}
__device__ __forceinline__ void put_at(uint32_t to, const float4& f) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(f.x), "f"(f.y),
               "f"(f.z), "f"(f.w) : "memory");
}
__device__ __forceinline__ void put_at(uint32_t to, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(to), "r"(v) : "memory");
}

// Joins the segments of a chunk in the order of `mine`: half warp 0 of warp 0 first, and
// blocks of a cluster by rank.  carry: the state in front of the chunk, replaced by the one
// behind it.  Returns the state in front of the thread's segment.  `round` counts up.
// BACK: in the opposite order (last segment of the last warp first; ranks as before).
template <int W, int CL, bool FLAGS, bool BACK>
__device__ __forceinline__ Quad join_runs(RunSlots<W, CL>& sh, Run mine, Quad& carry, int round) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 15, buf = round & 1;
  const bool second = BACK ? lane < 16 : lane >= 16;
  // the other half's run
  Run other;
  #pragma unroll
  for (int j = 0; j < 2; ++j) {
    other.m.v[j].x = __shfl_xor_sync(~0u, mine.m.v[j].x, 16);
    other.m.v[j].y = __shfl_xor_sync(~0u, mine.m.v[j].y, 16);
    other.H.v[j].x = __shfl_xor_sync(~0u, mine.H.v[j].x, 16);
    other.H.v[j].y = __shfl_xor_sync(~0u, mine.H.v[j].y, 16);
  }
  other.cut = FLAGS ? (bool)__shfl_xor_sync(~0u, (int)mine.cut, 16) : false;
  if (!FLAGS) mine.cut = false;
  const Run whole = second ? then(other, mine) : then(mine, other);     // the same in both halves
  Quad at = carry;
  if constexpr (W == 1 && CL == 1) {
    carry = apply(whole, carry);
  } else {
    if (second) {
      sh.m[buf][warp][l] = four(whole.m);
      sh.H[buf][warp][l] = four(whole.H);
      if (FLAGS && l == 0) sh.cut[buf][warp] = whole.cut;
    }
    __syncthreads();
    auto warp_run = [&](int w) {
      return Run{quad(sh.m[buf][w][l]), quad(sh.H[buf][w][l]), FLAGS ? (bool)sh.cut[buf][w] : false};
    };
    Quad front = carry;
    if constexpr (CL > 1) {
      const int rank = cluster_rank();
      if (threadIdx.x < 16 * CL) {      // 16 threads for each block of the cluster
        const int to = threadIdx.x >> 4;
        Run all = warp_run(BACK ? W - 1 : 0);
        #pragma unroll
        for (int i = 1; i < W; ++i) all = then(all, warp_run(BACK ? W - 1 - i : i));
        put_at(at_rank(&sh.cm[buf][rank][l], to), four(all.m));
        put_at(at_rank(&sh.cH[buf][rank][l], to), four(all.H));
        if (FLAGS && l == 0) put_at(at_rank(&sh.ccut[buf][rank], to), (int)all.cut);
      }
      cluster_barrier();
      #pragma unroll
      for (int c = 0; c < CL; ++c) {
        if (c == rank) front = carry;
        carry = apply(Run{quad(sh.cm[buf][c][l]), quad(sh.cH[buf][c][l]), FLAGS ? (bool)sh.ccut[buf][c] : false},
                      carry);
      }
    }
    at = front;
    #pragma unroll
    for (int i = 0; i < W; ++i) {
      const int w = BACK ? W - 1 - i : i;
      if (w == warp) at = front;
      if (CL == 1 || i + 1 < W) front = apply(warp_run(w), front);
    }
    if constexpr (CL == 1) carry = front;
  }
  if (second) at = apply(other, at);
  return at;
}

// --------------------------------------------------------------------- host

inline muon_status check_scan(int64_t batch, int64_t length, int64_t dim, int dtype) {
  if (batch < 0 || length < 0) return MUON_ERR_INVALID_ARG;
  if (dim < 1 || dim > 1 << 20 || batch >= (int64_t)1 << 31 || length >= (int64_t)1 << 31 ||
      batch * dim >= (int64_t)1 << 33 || batch * ((dim + kStrip - 1) / kStrip) >= (int64_t)1 << 27)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  return known(dtype) ? MUON_OK : MUON_ERR_DTYPE;
}

// whether rows of `p` are made of aligned pieces of four
inline bool fours(const void* p, int64_t rows, int64_t ld, size_t es) {
  return !off(p, 4 * es) && (rows <= 1 || ld % 4 == 0);
}

// Launch with clusters of CL blocks along the length
template <int CL, typename A>
cudaError_t launch_strips(void (*kernel)(A), int64_t strips, int threads, size_t smem, cudaStream_t s,
                          const A& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(strips * CL));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CL;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

}  // namespace muon
