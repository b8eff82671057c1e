// The microscaled modes' lanes and scale bytes, decoded to fp32 ("emily 0.5.1
// lib/emily/quantization.ex"; the modes are listed at the top of mx.cu).
#pragma once

#include "common.cuh"

namespace qmm {
namespace mx {

__device__ __forceinline__ float e2m1(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  // e = 0: subnormal 0.5 m; else 2^(e - 1) (1 + m / 2)
  const float mag = e == 0 ? 0.5f * (float)m : __int_as_float((int)(e + 126u) << 23) * (1.0f + 0.5f * (float)m);
  return (c & 8u) ? -mag : mag;
}
__device__ __forceinline__ float e8m0(uint32_t s) {
  s &= 0xffu;
  // exponent field s with a zero fraction is 2^(s - 127); s = 0 is 2^-127
  // (a subnormal), s = 255 reads as +inf
  return s == 0 ? __int_as_float(0x00400000) : __int_as_float((int)(s << 23));
}
__device__ __forceinline__ float e4m3(uint32_t b) {
  const float mag = __half2float(__ushort_as_half((unsigned short)((b & 0x7fu) << 7))) * 256.0f;
  return (b & 0x80u) ? -mag : mag;
}

template <int MODE>
struct Mode;
template <>
struct Mode<QMM_MODE_MXFP4> {
  static constexpr int B = 4, GS = 32;
  __device__ static float lane(uint32_t c) { return e2m1(c); }
  __device__ static float scale(uint32_t s) { return e8m0(s); }
};
template <>
struct Mode<QMM_MODE_MXFP8> {
  static constexpr int B = 8, GS = 32;
  __device__ static float lane(uint32_t c) { return e4m3(c); }
  __device__ static float scale(uint32_t s) { return e8m0(s); }
};
template <>
struct Mode<QMM_MODE_NVFP4> {
  static constexpr int B = 4, GS = 16;
  __device__ static float lane(uint32_t c) { return e2m1(c); }
  __device__ static float scale(uint32_t s) { return e4m3(s); }
};

}  // namespace mx
}  // namespace qmm
