// Paired fp32 arithmetic (sm_100a issues two operations as one instruction) and
// codes as floats by byte permutes.
#pragma once

#include "common.cuh"

namespace qmm {

// two fp32 operations in one instruction
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2f(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// 2^23 + code i of the words w, exactly
template <int B>
__device__ __forceinline__ float code_2p23(const uint32_t* w, int i) {
  if constexpr (B == 8) {
    return __uint_as_float(__byte_perm(w[i >> 2], 0x4B000000u, 0x7440u | (uint32_t)(i & 3)));
  } else if constexpr (B == 4) {
    const uint32_t t = (i & 1) ? (w[i >> 3] >> 4) & 0x0F0F0F0Fu : w[i >> 3] & 0x0F0F0F0Fu;
    return __uint_as_float(__byte_perm(t, 0x4B000000u, 0x7440u | (uint32_t)((i >> 1) & 3)));
  } else {
    return __uint_as_float(0x4B000000u | stream_code<B>(w, i));
  }
}

// Codes i and i + 1 as floats: 2^23 + q, less 2^23, exact.
template <int B>
__device__ __forceinline__ float2 codes2(const uint32_t* w, int i) {
  return add2(make_float2(code_2p23<B>(w, i), code_2p23<B>(w, i + 1)), make_float2(-8388608.0f, -8388608.0f));
}

}  // namespace qmm
