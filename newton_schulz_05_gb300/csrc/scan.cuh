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
// underflows and a is 1.  1 - a is what a token takes in and what the state loses; it has
// digits of its own (shares_of).  A token that is masked or past the end is given the gate
// +infinity and the input 0, which changes nothing.
//
// A block has a strip of 64 channels: 16 lanes of four channels, so a warp holds two
// segments.
#pragma once

#include "sequence.cuh"

#include <type_traits>

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
// what m (all ones or none) has of the bits
__device__ __forceinline__ float masked(float v, uint32_t m) { return __uint_as_float(__float_as_uint(v) & m); }
__device__ __forceinline__ Quad masked(const Quad& q, uint32_t m) {
  return {{make_float2(masked(q.v[0].x, m), masked(q.v[0].y, m)),
           make_float2(masked(q.v[1].x, m), masked(q.v[1].y, m))}};
}
__device__ __forceinline__ Raw4<__nv_bfloat16> masked(const Raw4<__nv_bfloat16>& r, uint32_t m) {
  return {make_uint2(r.u.x & m, r.u.y & m)};
}
__device__ __forceinline__ Raw4<float> masked(const Raw4<float>& r, uint32_t m) {
  return {make_uint4(r.u.x & m, r.u.y & m, r.u.z & m, r.u.w & m)};
}
// a gate, or the infinite one
__device__ __forceinline__ Raw4<__nv_bfloat16> gate_or(const Raw4<__nv_bfloat16>& r, uint32_t m) {
  const uint32_t n = 0x7f807f80u & ~m;
  return {make_uint2((r.u.x & m) | n, (r.u.y & m) | n)};
}
__device__ __forceinline__ Raw4<float> gate_or(const Raw4<float>& r, uint32_t m) {
  const uint32_t n = 0x7f800000u & ~m;
  return {make_uint4((r.u.x & m) | n, (r.u.y & m) | n, (r.u.z & m) | n, (r.u.w & m) | n)};
}
// all ones where bit i is set
__device__ __forceinline__ uint32_t ones(uint32_t bits, int i) { return (uint32_t)((int)(bits << (31 - i)) >> 31); }

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

__device__ __forceinline__ float reciprocal_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// keep = a = sigmoid(g) and take = 1 - a.  t = 4 exp(-g); a = 1 / (1 + t / 4), 1 - a = a t / 4,
// so that both have their own precision: 1 minus the rounded a is off by up to 3.6% at the gate 14,
// and 0 from about 17 on.  The 4 makes t infinite before a is flushed to 0, and the minimum
// drops the NaN of infinity times 0.
__device__ __forceinline__ void shares_of(const Quad& g, Quad& keep, Quad& take) {
  #pragma unroll
  for (int j = 0; j < 2; ++j) {
    float2 t = fma2(g.v[j], both(-1.4426950408889634f), both(2.f));
    t = make_float2(exp2_fast(t.x), exp2_fast(t.y));
    const float2 n = fma2(t, both(0.25f), both(1.f));
    keep.v[j] = make_float2(reciprocal_fast(n.x), reciprocal_fast(n.y));
    t = mul2(mul2(t, both(0.25f)), keep.v[j]);
    take.v[j] = make_float2(fminf(t.x, 1.f), fminf(t.y, 1.f));
  }
}

// Flags of a segment's tokens: its first S lanes hold a byte each from when they are
// asked for until they are needed.
struct Flags { uint32_t starts, live; bool quiet; };     // quiet: of the bits, none does anything in the warp
template <int S>
__device__ __forceinline__ Flags ask(const uint8_t* starts, const uint8_t* mask, int64_t row0, int64_t t0,
                                     int64_t length) {
  static_assert(S <= 16, "a lane a token");
  const int l = threadIdx.x & 15;
  const int64_t t = t0 + l;
  const bool in = l < S && t >= 0 && t < length;
  return {in && starts ? starts[row0 + t] : 0u, in && mask ? mask[row0 + t] : (uint32_t)in, false};
}
// as bits by token: which are live, and which of those start over
template <int S> __device__ __forceinline__ Flags bits(const Flags& f) {
  const int half = threadIdx.x & 16;
  const uint32_t live = __ballot_sync(~0u, f.live != 0), starts = __ballot_sync(~0u, f.starts != 0) & live;
  constexpr uint32_t whole = (S < 16 ? (1u << S) - 1 : 0xffffu) * 0x10001u;
  return {starts >> half & 0xffff, live >> half & 0xffff, live == whole && starts == 0};
}

// How a lane's four channels lie in a row: neighbours, in aligned pieces of four; two aligned
// pairs of bf16, 32 apart; or alone, 16 apart
enum { kFours, kPairs, kSingles };

template <typename T, int HOW> struct Channels {
  int strip, first;      // first channel of the strip, and of the lane, in the row
  int left;              // channels from `first` on that are inside the row
  __device__ __forceinline__ Channels(int index, int64_t dim) {
    const int l = threadIdx.x & 15;
    strip = index * kStrip;
    first = strip + (HOW == kFours ? 4 * l : HOW == kPairs ? 2 * l : l);
    left = (int)dim - first;
  }
  __device__ __forceinline__ bool any() const { return left > 0; }
  // of channel j from the first
  static __device__ __forceinline__ int at(int j) {
    return HOW == kFours ? j : HOW == kPairs ? (j >> 1) * 32 + (j & 1) : 16 * j;
  }
  __device__ __forceinline__ bool has(int j) const { return at(j) < left; }

  // p: the lane's first channel
  __device__ __forceinline__ void load(Raw4<T>& r, const T* p) const {
    if constexpr (HOW == kFours) {
      r = *reinterpret_cast<const Raw4<T>*>(p);
    } else if constexpr (HOW == kPairs) {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
      r.u = make_uint2(has(0) ? q[0] : 0, has(2) ? q[16] : 0);
    } else if constexpr (sizeof(T) == 2) {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
      uint32_t w[4];
      #pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = has(j) ? q[16 * j] : 0;
      r.u = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    } else {
      const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
      r.u = make_uint4(has(0) ? q[0] : 0, has(1) ? q[16] : 0, has(2) ? q[32] : 0, has(3) ? q[48] : 0);
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, const Quad& q) const {
    const __nv_bfloat162 a = __float22bfloat162_rn(q.v[0]), b = __float22bfloat162_rn(q.v[1]);
    const uint2 u = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    if constexpr (HOW == kFours) {
      *reinterpret_cast<uint2*>(p) = u;
    } else if constexpr (HOW == kPairs) {
      if (has(0)) *reinterpret_cast<uint32_t*>(p) = u.x;
      if (has(2)) *reinterpret_cast<uint32_t*>(p + 32) = u.y;
    } else {
      if (has(0)) p[0] = a.x;
      if (has(1)) p[16] = a.y;
      if (has(2)) p[32] = b.x;
      if (has(3)) p[48] = b.y;
    }
  }
  __device__ __forceinline__ void store(float* p, const Quad& q) const {
    if constexpr (HOW == kFours) {
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

// Rows of N operands on their way through shared memory: D chunks, S tokens a segment, 2 W
// segments.  A lane copies the piece of four that it reads.  Pairs and singles are copied by the half
// warp that reads their rows, in aligned pieces of 16 bytes, the first of which may begin ahead of
// the row and the last end behind it: only pieces that hold an element of the row are read, and an
// aligned 16 bytes lie wholly in the allocation that one of them does.  A lane's row then gets the
// piece behind its last whole one.  (Copies of single fp32 elements took 179 us for [8, 4096, 1409]
// where these take 153.)  How far a row is ahead of its first piece depends on its number
// modulo kPiece alone, and the chunks of a block are a multiple of that apart.
template <typename T, int HOW, int N, int S, int W> struct Ring {
  static constexpr int kPiece = HOW != kFours ? 16 / (int)sizeof(T) : 4;      // elements
  static constexpr int kLanes = kStrip / kPiece, kAtOnce = 16 / kLanes;   // of a row; rows
  static constexpr int kRow = 16 + (HOW != kFours ? kPiece / 4 : 0);
  static constexpr size_t kStage = sizeof(Raw4<T>) * N * S * 2 * W * kRow;
  static_assert(S <= 16, "a lane a row");
  Raw4<T>* base;
  int left;         // channels of the strip
  __device__ __forceinline__ Ring(void* smem, int strip, int64_t dim)
      : base(static_cast<Raw4<T>*>(smem) + (threadIdx.x >> 4) * kRow),
        left(min(kStrip, (int)dim - strip)) {}
  __device__ __forceinline__ Raw4<T>* row(int stage, int operand, int i) const {
    return base + ((stage * N + operand) * S + i) * (2 * W * kRow);
  }
  // of a segment's rows from..n - 1, those of i to i + kAtOnce - 1; p: the strip's first channel in
  // row 0
  __device__ __forceinline__ void copy(int stage, int operand, const T* p, uint32_t ld, int i, int from, int n) const {
    const int l = threadIdx.x & 15, mine = l & (kLanes - 1);
    if (kAtOnce > 1) i += l / kLanes;
    if (i < from || i >= n) return;
    p += (uint64_t)ld * i;
    Raw4<T>* to = row(stage, operand, i);
    if constexpr (HOW == kFours) {
      if (4 * l < left) put<4 * sizeof(T)>(to + l, p + 4 * l);
    } else {
      const Pieces s(p);
      if (kPiece * mine < left + s.ahead) put<16>(to + mine * (kPiece / 4), s.first + kPiece * mine);
    }
  }
  // the last pieces of rows from..n - 1, a lane a row
  __device__ __forceinline__ void copy_ends(int stage, int operand, const T* p, uint32_t ld, int from, int n) const {
    if constexpr (HOW != kFours) {
      const int i = threadIdx.x & 15;
      if (i < from || i >= min(S, n)) return;
      const Pieces s(p + (uint64_t)ld * i);
      if (left + s.ahead > kStrip) put<16>(row(stage, operand, i) + 16, s.first + kStrip);
    }
  }
  // rows from..n - 1, and the others as tokens that change nothing
  __device__ __forceinline__ void copy_some(int stage, int operand, const T* p, uint32_t ld, int from, int n,
                                            bool gate) const {
    for (int i = 0; i < S; i += kAtOnce) copy(stage, operand, p, ld, i, from, n);
    copy_ends(stage, operand, p, ld, from, n);
    for (int i = 0; i < S; ++i)
      if (i < from || i >= n) fill(row(stage, operand, i), gate);
  }
  // where the aligned pieces of a strip's row begin, and how many elements ahead of it
  struct Pieces {
    const T* first;
    int ahead;
    __device__ __forceinline__ Pieces(const T* p) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      first = reinterpret_cast<const T*>(at & ~(uintptr_t)15);
      ahead = (int)((uint32_t)at / sizeof(T) & (kPiece - 1));
    }
  };
  // elements of row i ahead of the strip, of a segment whose row 0 is at p
  static __device__ __forceinline__ uint32_t ahead(const T* p, uint32_t ld, int i) {
    return HOW == kFours ? 0 : ((uint32_t)(reinterpret_cast<uintptr_t>(p) / sizeof(T)) + (i & (kPiece - 1)) * ld) &
                                     (kPiece - 1);
  }
  template <int BYTES> static __device__ __forceinline__ void put(void* to, const T* p) {
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
    if constexpr (BYTES == 16)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(s), "l"(p) : "memory");
    else
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(s), "l"(p), "n"(BYTES) : "memory");
  }
  // every element of a row
  __device__ __forceinline__ void fill(Raw4<T>* to, bool gate) const {
    const int l = threadIdx.x & 15;
    Raw4<T> v;
    if (gate) infinite(v);
    else zero(v);
    to[l] = v;
    if (l < kRow - 16) to[16 + l] = v;
  }
  // the lane's channels; f: the row's elements ahead of the strip
  __device__ __forceinline__ Raw4<T> get(const Raw4<T>* from, int f) const {
    const int l = threadIdx.x & 15;
    if constexpr (HOW == kFours) {
      return from[l];
    } else if constexpr (HOW == kPairs) {
      const uint32_t* e = reinterpret_cast<const uint32_t*>(from) + f / 2 + l;
      return {make_uint2(e[0], e[16])};
    } else if constexpr (sizeof(T) == 2) {
      const uint16_t* e = reinterpret_cast<const uint16_t*>(from) + f + l;
      return {make_uint2(e[0] | (uint32_t)e[16] << 16, e[32] | (uint32_t)e[48] << 16)};
    } else {
      const uint32_t* e = reinterpret_cast<const uint32_t*>(from) + f + l;
      return {make_uint4(e[0], e[16], e[32], e[48])};
    }
  }
  // the half warp's lanes have copied for one another, and have read
  __device__ __forceinline__ void arrived() const { if (HOW != kFours) __syncwarp(); }
};

// A run of tokens as a map of the state p in front of it, H + (k + m) p: where its
// factor P is 1/2 or more, k is 1 and m is -(1 - P), else k is 0 and m is P.  1 - P
// decides how much of the state a long run forgets, and P has no bits for it: with P
// alone, 3000 tokens of the gate 8 took a constant state off by 1.6e-5 of itself.
// cut: some token of the run starts over, and H is the state whatever p was.
struct Run {
  Quad m, k, H;
  bool cut;
};
__device__ __forceinline__ Quad apply(const Run& r, const Quad& p) {
  Quad q = fma(r.k, p, fma(r.m, p, r.H));
  if (r.cut) q = r.H;
  return q;
}
// first `a`, then `b`: (k + m) (k' + m') = k k' + the rest
__device__ __forceinline__ Run then(const Run& a, const Run& b) {
  return {fma(a.m, b.k, fma(a.k, b.m, mul(a.m, b.m))), mul(a.k, b.k), apply(b, a.H), a.cut || b.cut};
}
// a segment's factor, 1 minus it, and what its tokens add.  1 minus the factor is a sum of
// positive terms, each of which has its own digits (shares_of).
struct Segment {
  Quad P, Q, H;
  bool cut;
};
__device__ __forceinline__ Run run_of(const Segment& g) {
  Run r;
  #pragma unroll
  for (int j = 0; j < 2; ++j) {
    const bool x = g.P.v[j].x >= 0.5f, y = g.P.v[j].y >= 0.5f;
    r.m.v[j] = make_float2(x ? -g.Q.v[j].x : g.P.v[j].x, y ? -g.Q.v[j].y : g.P.v[j].y);
    r.k.v[j] = make_float2(x ? 1.f : 0.f, y ? 1.f : 0.f);
  }
  r.H = g.H;
  r.cut = g.cut;
  return r;
}

// Blocks an SM: two of eight warps, or one where a thread has more tokens and needs the
// registers of two
template <typename T, int W, int OPERANDS, int S> constexpr int kScanBlocks =
    W < 8 ? 16 / W : S * (int)sizeof(T) * OPERANDS > 32 ? 1 : 2;

// what the runs of a block's warps, and of a cluster's blocks, are exchanged through
struct RunSlot { float4 m[16], k[16], H[16]; };
template <int W, int CL> struct RunSlots {
  RunSlot warp[2][W], block[2][CL];
  float4 carry[2][16];
  int cut[2][W], block_cut[2][CL];
};
__device__ __forceinline__ float4 four(const Quad& q) {
  return make_float4(q.v[0].x, q.v[0].y, q.v[1].x, q.v[1].y);
}
__device__ __forceinline__ Quad quad(const float4& f) {
  return {{make_float2(f.x, f.y), make_float2(f.z, f.w)}};
}
__device__ __forceinline__ Run run_in(const RunSlot& s, int cut) {
  const int l = threadIdx.x & 15;
  return {quad(s.m[l]), quad(s.k[l]), quad(s.H[l]), cut != 0};
}

__device__ __forceinline__ Quad from_other_half(const Quad& q) {
  Quad r;
  #pragma unroll
  for (int j = 0; j < 2; ++j) {
    r.v[j].x = __shfl_xor_sync(~0u, q.v[j].x, 16);
    r.v[j].y = __shfl_xor_sync(~0u, q.v[j].y, 16);
  }
  return r;
}

// Joins the segments of chunk `round` in order: the first half of warp 0 first, blocks of
// a cluster by rank.  BACK: the second half of the last warp first, blocks as before.
// Returns the state in front of the thread's segment.  The state in front of the chunk is
// read from sh.carry[round & 1] and the one behind it left in the other.  A warp goes
// through the runs in front of its own only; the last one knows the block's run or the
// state behind the chunk.  `meanwhile` is done while the blocks of a cluster wait.
template <int W, int CL, bool FLAGS, bool BACK, typename F>
__device__ __forceinline__ Quad join_segments(RunSlots<W, CL>& sh, const Segment& mine, int round, F meanwhile) {
  const int lane = threadIdx.x & 31, l = lane & 15, buf = round & 1;
  const int warp = BACK ? W - 1 - (threadIdx.x >> 5) : threadIdx.x >> 5;      // in order
  const bool second = BACK ? lane < 16 : lane >= 16;
  Segment other = {from_other_half(mine.P), from_other_half(mine.Q), from_other_half(mine.H), false};
  if (FLAGS) other.cut = __shfl_xor_sync(~0u, (int)mine.cut, 16) != 0;
  // both halves' segments as one; right in the second half alone
  Segment whole = {mul(other.P, mine.P), fma(other.P, mine.Q, other.Q), fma(mine.P, other.H, mine.H), false};
  if (FLAGS) {
    whole.cut = other.cut || mine.cut;
    if (mine.cut) whole.H = mine.H;
  }
  if (second) {
    const Run run = run_of(whole);
    RunSlot& to = sh.warp[buf][warp];
    to.m[l] = four(run.m);
    to.k[l] = four(run.k);
    to.H[l] = four(run.H);
    if (FLAGS && l == 0) sh.cut[buf][warp] = run.cut;
  }
  if (CL == 1) meanwhile();
  if constexpr (W > 1 || CL > 1) __syncthreads();
  else __syncwarp();
  auto warp_run = [&](int w) { return run_in(sh.warp[buf][w], FLAGS ? sh.cut[buf][w] : 0); };
  Quad p;
  if constexpr (CL > 1) {
    const int rank = cluster_rank();
    auto block_run = [&](int c) { return run_in(sh.block[buf][c], FLAGS ? sh.block_cut[buf][c] : 0); };
    Run ahead = {quad(0.f), quad(1.f), quad(0.f), false}, next = warp_run(0);
    #pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w > warp || (w == warp && w < W - 1)) break;      // the last warp takes in its own, too
      const Run now = next;
      if (w + 1 < W) next = warp_run(w + 1);
      if (w == W - 1) {
        const Run all = then(ahead, now);
        RunSlot& slot = sh.block[buf][rank];
        for (int to = lane >> 4; to < CL; to += 2) {
          put_at(at_rank(&slot.m[l], to), four(all.m));
          put_at(at_rank(&slot.k[l], to), four(all.k));
          put_at(at_rank(&slot.H[l], to), four(all.H));
          if (FLAGS && l == 0) put_at(at_rank(&sh.block_cut[buf][rank], to), (int)all.cut);
        }
      } else {
        ahead = then(ahead, now);
      }
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");
    meanwhile();
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    p = quad(sh.carry[buf][l]);
    Run run = block_run(0);
    Quad q = p;
    #pragma unroll
    for (int c = 0; c < CL; ++c) {
      if (c == rank) p = q;
      if (c >= rank && warp > 0) break;      // the first warp goes on to the state behind the chunk
      const Run now = run;
      if (c + 1 < CL) run = block_run(c + 1);
      q = apply(now, q);
    }
    if (warp == 0 && second) sh.carry[buf ^ 1][l] = four(q);
    p = apply(ahead, p);
  } else {
    p = quad(sh.carry[buf][l]);
    Run run = warp_run(0);
    #pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w >= warp && w < W - 1) break;
      const Run now = run;
      if (w + 1 < W) run = warp_run(w + 1);
      if (w == W - 1) {
        const Quad q = apply(now, p);
        if (second) sh.carry[buf ^ 1][l] = four(q);
      } else {
        p = apply(now, p);
      }
    }
  }
  if (second) p = apply(run_of(other), p);
  return p;
}

// --------------------------------------------------------------------- host

inline muon_status check_scan(int64_t batch, int64_t length, int64_t dim, int dtype) {
  if (batch < 0 || length < 0) return MUON_ERR_INVALID_ARG;
  if (dim < 1 || dim > 1 << 20 || batch >= (int64_t)1 << 31 || length >= (int64_t)1 << 31 ||
      batch * ((dim + kStrip - 1) / kStrip) >= (int64_t)1 << 27)
    return MUON_ERR_UNSUPPORTED_SHAPE;
  return known(dtype) ? MUON_OK : MUON_ERR_DTYPE;
}

// How the length is cut up: f(warps a block, S's multiple, blocks a cluster, chunks in flight)
// as integral constants.  A chunk of a block is 2 W S tokens.  (Figures taken side by side; later
// steps made all of a column up to a tenth faster.)
//   Few strips take blocks with twice the tokens a thread, one an SM, in clusters that fill
// the SMs between them; a round of joins through a cluster takes 1 us more, so it is worth it
// where it saves rounds only.  bf16, forward and gradient in us, with clusters of 8, 4, 2 and
// without, then two blocks an SM in clusters of 8, 4 and without:
//   [1, 65536, 64] 101, 181, 347 | 140: 210, 365, 698 | 328     8 from 1 strip on
//   [1, 32768, 2048] 162, 103, 185 | 111: 328, 199, 372 | 236   4 from 20 strips on
//   [2, 16384, 2048] 144, 106, 100 | 100: 283, 201, 197 | 210   2 from 39 strips on
//   [1, 16000, 5120] -, -, 196, 140 | 158: 385, 285 | 340       none from 77 strips on
//   [200, 4096, 64] -, -, 81, 74 | 79, 68: 154, 145 | 163, 136  two an SM from 153 strips on
// In fp32 39 to 76 strips are the exception: clusters of four with two blocks an SM took 158
// us for [2, 16384, 2048] where clusters of two took 178, and the gradient 318 and 354.
// Smaller blocks with less to join from 305 strips on: [16, 1024, 4096] bf16 65 and 71 us,
// gradient 133 and 136 ([16, 2048, 2048] fp32 154 and 137, 312 and 293, where the strips are
// 1.7 times as many as the larger blocks' places), and for lengths of one chunk.
template <int V> using Int = std::integral_constant<int, V>;
template <typename T, int S, typename F> cudaError_t scan_layout(int64_t length, int64_t strips, F f) {
  if (length <= 2 * S) return f(Int<1>(), Int<1>(), Int<1>(), Int<0>());
  if (length <= 8 * S || strips > 304) return f(Int<4>(), Int<1>(), Int<1>(), Int<2>());
  if (length <= 16 * S || strips > 152) return f(Int<8>(), Int<1>(), Int<1>(), Int<2>());
  if (length <= 32 * S || strips > 76) return f(Int<8>(), Int<2>(), Int<1>(), Int<2>());
  if constexpr (sizeof(T) == 4)
    if (strips > 38) return f(Int<8>(), Int<1>(), Int<4>(), Int<2>());
  if (length <= 64 * S || strips > 38) return f(Int<8>(), Int<2>(), Int<2>(), Int<2>());
  if (length <= 128 * S || strips > 19) return f(Int<8>(), Int<2>(), Int<4>(), Int<2>());
  return f(Int<8>(), Int<2>(), Int<8>(), Int<2>());
}

// the widest access that all rows allow
inline int lie(const void* p, int64_t rows, int64_t ld, size_t es) {
  auto in = [&](int n) { return !off(p, n * es) && (rows <= 1 || ld % n == 0); };
  return in(4) ? kFours : es == 2 && in(2) ? kPairs : kSingles;
}
// f(how), as an integral constant
template <typename T, typename F> cudaError_t by_how(int how, F f) {
  if (how == kFours) return f(Int<kFours>());
  if constexpr (sizeof(T) == 2)
    if (how == kPairs) return f(Int<kPairs>());
  return f(Int<kSingles>());
}

}  // namespace

}  // namespace muon
