// Counter-based random bits of dropout: Philox4x32-10 (J. Salmon, M. Moraes,
// R. Dror, D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC 2011),
// and the keep rule built on it.
//
// One block of the generator serves eight elements with 16 bits each: ten
// rounds of two 32 x 32 -> 64 bit products cost about 45 instructions, 6 an
// element, where a word an element would cost 11 and make dropout of 16-bit
// data bound by integer products instead of HBM.  The price is that the drop
// probability is a multiple of 1/65536; the kept elements are scaled by the
// exact inverse of the probability used, so the expectation stays exact.
#pragma once

#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "pieces.cuh"

namespace muon {

struct Drop {
  uint32_t key[20];    // the rounds' keys, two a round (kernel parameters: constant operands)
  uint64_t offset;     // counter of element 0
  uint32_t limit;      // an element is kept when its 16 bits, moved to a word's high half,
                       // are above this
  float scale;         // of the kept elements
};

// floor(65536 p + 1/2): an element is kept when its 16 bits are >= this
inline uint32_t drop_threshold(float p) { return (uint32_t)std::floor((double)p * 65536.0 + 0.5); }

// of a threshold above 0 (at 0 nothing is dropped and nothing need be drawn): 16
// bits h are >= threshold when h << 16 (whatever its low half) is above
// (threshold << 16) - 1
inline Drop make_drop(float p, uint64_t seed, uint64_t offset) {
  const uint32_t threshold = drop_threshold(p);
  Drop d;
  for (int r = 0; r < 10; ++r) {
    d.key[2 * r] = (uint32_t)seed + r * 0x9E3779B9u;
    d.key[2 * r + 1] = (uint32_t)(seed >> 32) + r * 0xBB67AE85u;
  }
  d.offset = offset;
  d.limit = (uint32_t)(((uint64_t)threshold << 16) - 1);
  d.scale = threshold < 65536u ? (float)(65536.0 / (65536.0 - threshold)) : 0.f;
  return d;
}

__device__ __forceinline__ uint4 philox(uint64_t counter, const Drop& d) {
  uint32_t c0 = (uint32_t)counter, c1 = (uint32_t)(counter >> 32), c2 = 0, c3 = 0;
  #pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ d.key[2 * r];
    c2 = (uint32_t)(a >> 32) ^ c3 ^ d.key[2 * r + 1];
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The sixteen-bit halves of eight consecutive elements, the first of index i
// (which may be below zero where a row's first piece begins ahead of the row:
// such elements are not used).  When i is not a multiple of eight the elements
// straddle two blocks, whose sixteen halves are shifted into place.
__device__ __forceinline__ uint4 drop_bits(int64_t i, const Drop& d) {
  const uint64_t c = d.offset + (uint64_t)(i >> 3);
  uint4 w = philox(c, d);
  const int shift = (int)(i & 7);
  if (shift) {
    const uint4 n = philox(c + 1, d);
    uint32_t a[8] = {w.x, w.y, w.z, w.w, n.x, n.y, n.z, n.w};
    if (shift & 4) {
      #pragma unroll
      for (int j = 0; j < 6; ++j) a[j] = a[j + 2];
    }
    if (shift & 2) {
      #pragma unroll
      for (int j = 0; j < 5; ++j) a[j] = a[j + 1];
    }
    const uint32_t bits = (shift & 1) * 16;
    w = make_uint4(__funnelshift_r(a[0], a[1], bits), __funnelshift_r(a[1], a[2], bits),
                   __funnelshift_r(a[2], a[3], bits), __funnelshift_r(a[3], a[4], bits));
  }
  return w;
}

// Dropout of E (4 or 8) consecutive elements, the first of index i.  ALIGNED: i is
// known to be a multiple of E.
template <int E, bool ALIGNED>
__device__ __forceinline__ void drop(float2 (&v)[E / 2], int64_t i, const Drop& d) {
  // p = 1.  The comparison below drops everything by itself; the branch keeps the
  // pieces' blocks apart where registers are short: layer norm of [4096, 10240] fp32
  // 108.4 us against 114.9 without it (of [4096, 16384] bf16 97.1 against 95.0)
  if (!ALIGNED && d.limit == 0xffffffffu) {
    #pragma unroll
    for (int j = 0; j < E / 2; ++j) v[j] = both(0.f);
    return;
  }
  uint32_t u[4];
  if (E == 4 && (ALIGNED || (i & 3) == 0)) {    // half a block
    const uint4 w = philox(d.offset + (uint64_t)(i >> 3), d);
    u[0] = i & 4 ? w.z : w.x;
    u[1] = i & 4 ? w.w : w.y;
  } else {
    const uint4 w = ALIGNED ? philox(d.offset + (uint64_t)(i >> 3), d) : drop_bits(i, d);
    u[0] = w.x; u[1] = w.y; u[2] = w.z; u[3] = w.w;
  }
  #pragma unroll
  for (int j = 0; j < E / 2; ++j) {
    const float2 k = mul2(v[j], both(d.scale));
    v[j].x = (u[j] << 16) > d.limit ? k.x : 0.f;
    v[j].y = u[j] > d.limit ? k.y : 0.f;
  }
}

}  // namespace muon
