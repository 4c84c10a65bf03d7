// 16-byte pieces of a row: eight bf16 or four fp32 elements, moved whole and
// computed on as fp32 pairs.
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

template <int E> struct Piece { float2 v[E / 2]; };
template <int E> __device__ __forceinline__ float& elem(Piece<E>& p, int j) {
  return j & 1 ? p.v[j >> 1].y : p.v[j >> 1].x;
}
template <int E> __device__ __forceinline__ void clear(Piece<E>& p) {
  #pragma unroll
  for (int j = 0; j < E / 2; ++j) p.v[j] = both(0.f);
}

// elements of a piece
template <typename T> constexpr int kEl = 16 / (int)sizeof(T);

__device__ __forceinline__ void widen(Piece<8>& p, const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  #pragma unroll
  for (int j = 0; j < 4; ++j)
    p.v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
}
__device__ __forceinline__ void widen(Piece<4>& p, const uint4& u) {
  p.v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
  p.v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 narrow(const Piece<8>& p) {
  uint32_t w[4];
  #pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b = __float22bfloat162_rn(p.v[j]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 narrow(const Piece<4>& p) {
  return make_uint4(__float_as_uint(p.v[0].x), __float_as_uint(p.v[0].y),
                    __float_as_uint(p.v[1].x), __float_as_uint(p.v[1].y));
}

}  // namespace muon
