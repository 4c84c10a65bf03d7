// Chunks of eight consecutive elements: what one thread moves in 16-byte
// accesses (one of bf16, two of fp32) and computes on in fp32 pairs.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace muon {

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

// the 16-byte pieces of a chunk, as loaded, in fp32
__device__ __forceinline__ void widen(Chunk& c, const uint4 (&u)[1]) {
  const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
  #pragma unroll
  for (int j = 0; j < 4; ++j)
    c.v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}
__device__ __forceinline__ void widen(Chunk& c, const uint4 (&u)[2]) {
  c.v[0] = make_float2(__uint_as_float(u[0].x), __uint_as_float(u[0].y));
  c.v[1] = make_float2(__uint_as_float(u[0].z), __uint_as_float(u[0].w));
  c.v[2] = make_float2(__uint_as_float(u[1].x), __uint_as_float(u[1].y));
  c.v[3] = make_float2(__uint_as_float(u[1].z), __uint_as_float(u[1].w));
}

}  // namespace muon
