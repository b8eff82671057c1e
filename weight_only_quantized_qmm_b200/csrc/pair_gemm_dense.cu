// The many-token products over weights dequantized beforehand, and the pass
// that dequantizes them: w_hat = q * s + z in fp32, rounded once to the
// activations' type, [rows, K] row-major for each part.
//
// The pass writes 2 bytes a weight (4096 x 14336 gate and up: 235 MB) and is
// bound by that; one thread turns 8 codes into one 16-byte store, so that a
// warp writes 512 contiguous bytes.
#include "pair_gemm.cuh"

namespace qmm {
namespace pg {

struct DequantArgs {
  Weight w[2];
  void* out[2];
  int rows, per_row;  // per_row: 8-code pieces of a row
  int lanes;          // lanes per row: the largest power of two up to 32 and per_row
  int lgs;
};

template <int B, typename T>
__global__ void __launch_bounds__(256) dequant_rows_kernel(const __grid_constant__ DequantArgs p) {
  const Weight& w = p.w[blockIdx.y];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int rpw = 32 / p.lanes, lane = threadIdx.x & 31;
  const int64_t row = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * rpw + lane / p.lanes;
  if (row >= p.rows) return;
  const int64_t base = row * p.per_row, gbase = row * (p.per_row >> (p.lgs - 3));
  const uint8_t* src0 = reinterpret_cast<const uint8_t*>(w.packed) + base * B;
  const T* sc = reinterpret_cast<const T*>(w.scales) + gbase;
  const T* bi = reinterpret_cast<const T*>(w.biases) + gbase;
  uint4* out = reinterpret_cast<uint4*>(p.out[blockIdx.y]) + base;
#pragma unroll 4
  for (int c = lane % p.lanes; c < p.per_row; c += p.lanes) {
    // 8 codes are B bytes
    uint32_t r[2] = {0u, 0u};
    const uint8_t* src = src0 + (int64_t)c * B;
    if constexpr (B == 8) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
      r[0] = v.x;
      r[1] = v.y;
    } else if constexpr (B == 4) {
      r[0] = __ldcs(reinterpret_cast<const uint32_t*>(src));
    } else if constexpr (B == 2) {
      r[0] = __ldcs(reinterpret_cast<const uint16_t*>(src));
    } else if constexpr (B == 6) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
      r[0] = __ldg(h) | ((uint32_t)__ldg(h + 1) << 16);
      r[1] = __ldg(h + 2);
    } else {
      r[0] = __ldg(src) | ((uint32_t)__ldg(src + 1) << 8) | ((uint32_t)__ldg(src + 2) << 16);
    }
    const int g = c >> (p.lgs - 3);
    const float s = to_f32(__ldg(sc + g)), z = to_f32(__ldg(bi + g));
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // the code in the low mantissa bits of 2^23, less 2^23: exact
      v[e] = fmaf(__uint_as_float(0x4B000000u | stream_code<B>(r, e)) - 8388608.0f, s, z);
    }
    out[c] = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  }
}

template <int B>
static cudaError_t dequant_b(const DequantArgs& d, bool f16, dim3 grid, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);  // 8 warps
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return f16 ? cudaLaunchKernelEx(&cfg, dequant_rows_kernel<B, __half>, d)
             : cudaLaunchKernelEx(&cfg, dequant_rows_kernel<B, __nv_bfloat16>, d);
}

// Dequantizes the parts of `p` into ws, [N, K] each, and maps them for `op`.
cudaError_t dequant_parts(int op, int bits, const Args& p, void* ws, Maps& tm, cudaStream_t st) {
  DequantArgs d{};
  d.rows = p.N;
  d.per_row = p.K / 8;
  d.lanes = 32;
  while (d.lanes > d.per_row) d.lanes /= 2;
  d.lgs = p.lgs;
  for (int i = 0; i < 2; ++i) {
    const int part = i < p.parts ? i : 0;
    d.w[i] = p.w[part];
    d.out[i] = static_cast<char*>(ws) + (int64_t)part * p.N * p.K * 2;
    // FWD reads 128 rows x 64 k, DX 64 rows x 64 columns at a time
    if (!make_map(&tm.b[i], d.out[i], p.f16, p.N, p.K, p.K, op == FWD ? 128 : 64)) return cudaErrorInvalidValue;
  }
  const int rows_per_block = 8 * (32 / d.lanes);
  const dim3 grid((unsigned)(((int64_t)p.N + rows_per_block - 1) / rows_per_block), p.parts);
  switch (bits) {
    case 2: return dequant_b<2>(d, p.f16, grid, st);
    case 3: return dequant_b<3>(d, p.f16, grid, st);
    case 4: return dequant_b<4>(d, p.f16, grid, st);
    case 6: return dequant_b<6>(d, p.f16, grid, st);
    default: return dequant_b<8>(d, p.f16, grid, st);
  }
}

cudaError_t dispatch_dense(int op, const Args& p, const Maps& tm, int clusters, cudaStream_t st) {
  return op == FWD ? launch_t<FWD, 0, true>(p, tm, clusters, st) : launch_t<DX, 0, true>(p, tm, clusters, st);
}

}  // namespace pg
}  // namespace qmm
