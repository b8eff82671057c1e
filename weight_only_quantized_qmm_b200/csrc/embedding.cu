// Lookup in a packed table and the gradient of its scales and biases.
//
// Forward:  y[t, i] = alpha * w_hat[ids[t]][i], w_hat as in qmm_dequantize.
// Backward: a[r, i] = alpha * sum over the tokens t with ids[t] = r of dy[t, i]
//           dscales[r, g] = sum over i in group g of a[r, i] * q[r, i]
//           dbiases[r, g] = sum over i in group g of a[r, i]
// (w_hat = q * scale + bias; the codes are constants).  Rows no token names
// get zeros.
#include <algorithm>

#include "common.cuh"
#include "mx.cuh"

namespace qmm {
namespace embed {

// One thread per 32 codes of one token's row (B words, whole groups of 16 or
// part of one larger group).
template <int B, int MODE, typename TS, typename TO>
__global__ void __launch_bounds__(256)
lookup_kernel(const int32_t* __restrict__ ids, int64_t n, const uint32_t* __restrict__ packed,
              const void* __restrict__ scales, const void* __restrict__ biases, int64_t rows, int64_t cols, int gs,
              float alpha, TO* __restrict__ out, int32_t* d_status) {
  const int64_t chunks = cols / 32, G = cols / gs;
  for (int64_t idx = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; idx < n * chunks;
       idx += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = idx / chunks, c = idx - t * chunks;
    const int64_t r = __ldg(ids + t);
    __align__(16) TO vals[32];
    if (r < 0 || r >= rows) {
      if (c == 0) set_status(d_status, QMM_ERR_BAD_TOKEN_ID);
#pragma unroll
      for (int i = 0; i < 32; ++i) vals[i] = from_f32<TO>(0.0f);
    } else {
      const uint32_t* src = packed + r * (cols * B / 32) + c * B;
      uint32_t wr[B + 1];
#pragma unroll
      for (int i = 0; i < B; ++i) wr[i] = __ldg(src + i);
      wr[B] = 0u;
      if constexpr (MODE == QMM_MODE_AFFINE) {
        const float s = to_f32(reinterpret_cast<const TS*>(scales)[r * G + c * 32 / gs]);
        const float b = to_f32(reinterpret_cast<const TS*>(biases)[r * G + c * 32 / gs]);
#pragma unroll
        for (int i = 0; i < 32; ++i)
          vals[i] = from_f32<TO>(__fmul_rn(alpha, fmaf((float)stream_code<B>(wr, i), s, b)));
      } else {
        using Md = mx::Mode<MODE>;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float s = Md::scale(__ldg(reinterpret_cast<const uint8_t*>(scales) + r * G + (c * 32 + i) / Md::GS));
          vals[i] = from_f32<TO>(__fmul_rn(alpha, Md::lane(stream_code<B>(wr, i)) * s));
        }
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + t * cols + c * 32);
    const uint4* v4 = reinterpret_cast<const uint4*>(vals);
#pragma unroll
    for (int i = 0; i < (int)(32 * sizeof(TO) / 16); ++i) dst[i] = v4[i];
  }
}

// One block per token; the first token of each row sums all of the row's
// tokens in order.  One thread per 32 codes, groups joined in group order.
template <int B, typename TD>
__global__ void __launch_bounds__(256)
grad_kernel(const TD* __restrict__ dy, const int32_t* __restrict__ ids, int64_t n, const uint32_t* __restrict__ packed,
            int64_t rows, int64_t cols, int gs, float alpha, void* dscales, void* dbiases, int g_dtype,
            int32_t* d_status) {
  const int64_t t0 = blockIdx.x;
  const int64_t r = ids[t0];
  if (r < 0 || r >= rows) {
    if (threadIdx.x == 0) set_status(d_status, QMM_ERR_BAD_TOKEN_ID);
    return;
  }
  int seen = 0;
  for (int64_t t = threadIdx.x; t < t0; t += blockDim.x) seen |= ids[t] == r;
  if (__syncthreads_or(seen)) return;
  const int64_t G = cols / gs;
  for (int64_t g = threadIdx.x; g < G; g += blockDim.x) {
    float ds = 0.0f, db = 0.0f;
    for (int64_t c = g * gs / 32; c < (g + 1) * gs / 32; ++c) {
      float a[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) a[i] = 0.0f;
      for (int64_t t = t0; t < n; ++t)
        if (ids[t] == r)
          for (int i = 0; i < 32; ++i) a[i] += to_f32(dy[t * cols + c * 32 + i]);
      uint32_t wr[B + 1];
      for (int i = 0; i < B; ++i) wr[i] = packed[r * (cols * B / 32) + c * B + i];
      wr[B] = 0u;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        ds = fmaf(a[i], (float)stream_code<B>(wr, i), ds);
        db += a[i];
      }
    }
    store_as(dscales, g_dtype, r * G + g, alpha * ds);
    store_as(dbiases, g_dtype, r * G + g, alpha * db);
  }
}

template <int B, int MODE, typename TS>
static cudaError_t lookup_o(const int32_t* ids, int64_t n, const qmm_qweight* w, float alpha, void* out, int out_dtype,
                            int32_t* d_status, cudaStream_t st) {
  const int64_t items = n * (w->cols / 32);
  const int grid = (int)std::min<int64_t>((items + 255) / 256, 148 * 64);
#define QMM_L(TO)                                                                                              \
  lookup_kernel<B, MODE, TS, TO><<<grid, 256, 0, st>>>(ids, n, w->packed, w->scales, w->biases, w->rows, w->cols, \
                                                       w->group_size, alpha, (TO*)out, d_status)
  if (out_dtype == QMM_F32) QMM_L(float);
  else if (out_dtype == QMM_BF16) QMM_L(__nv_bfloat16);
  else QMM_L(__half);
#undef QMM_L
  return cudaGetLastError();
}

template <int B>
static cudaError_t lookup_s(const int32_t* ids, int64_t n, const qmm_qweight* w, float alpha, void* out, int out_dtype,
                            int32_t* d_status, cudaStream_t st) {
  if (w->sdtype == QMM_F32) return lookup_o<B, 0, float>(ids, n, w, alpha, out, out_dtype, d_status, st);
  if (w->sdtype == QMM_BF16) return lookup_o<B, 0, __nv_bfloat16>(ids, n, w, alpha, out, out_dtype, d_status, st);
  return lookup_o<B, 0, __half>(ids, n, w, alpha, out, out_dtype, d_status, st);
}

static cudaError_t launch_lookup(const int32_t* ids, int64_t n, const qmm_qweight* w, float alpha, void* out,
                                 int out_dtype, int32_t* d_status, cudaStream_t st) {
  switch (w->mode) {
    case QMM_MODE_MXFP4: return lookup_o<4, QMM_MODE_MXFP4, uint8_t>(ids, n, w, alpha, out, out_dtype, d_status, st);
    case QMM_MODE_MXFP8: return lookup_o<8, QMM_MODE_MXFP8, uint8_t>(ids, n, w, alpha, out, out_dtype, d_status, st);
    case QMM_MODE_NVFP4: return lookup_o<4, QMM_MODE_NVFP4, uint8_t>(ids, n, w, alpha, out, out_dtype, d_status, st);
    default: break;
  }
  switch (w->bits) {
    case 2: return lookup_s<2>(ids, n, w, alpha, out, out_dtype, d_status, st);
    case 3: return lookup_s<3>(ids, n, w, alpha, out, out_dtype, d_status, st);
    case 4: return lookup_s<4>(ids, n, w, alpha, out, out_dtype, d_status, st);
    case 6: return lookup_s<6>(ids, n, w, alpha, out, out_dtype, d_status, st);
    default: return lookup_s<8>(ids, n, w, alpha, out, out_dtype, d_status, st);
  }
}

template <typename TD>
static cudaError_t launch_grad(const void* dy, const int32_t* ids, int64_t n, const qmm_qweight* w, float alpha,
                               void* dscales, void* dbiases, int g_dtype, int32_t* d_status, cudaStream_t st) {
  const int64_t G = w->cols / w->group_size;
  const size_t bytes = (size_t)(w->rows * G * qmm_host::dtype_size((qmm_dtype)g_dtype));
  cudaError_t e = cudaMemsetAsync(dscales, 0, bytes, st);
  if (e == cudaSuccess) e = cudaMemsetAsync(dbiases, 0, bytes, st);
  if (e != cudaSuccess || n == 0) return e;
#define QMM_E(BB)                                                                                                  \
  grad_kernel<BB, TD><<<(unsigned)n, 256, 0, st>>>((const TD*)dy, ids, n, w->packed, w->rows, w->cols, w->group_size, \
                                                  alpha, dscales, dbiases, g_dtype, d_status)
  switch (w->bits) {
    case 2: QMM_E(2); break;
    case 3: QMM_E(3); break;
    case 4: QMM_E(4); break;
    case 6: QMM_E(6); break;
    default: QMM_E(8); break;
  }
#undef QMM_E
  return cudaGetLastError();
}

}  // namespace embed
}  // namespace qmm

using namespace qmm_host;

extern "C" {

qmm_status qmm_embedding(const int32_t* ids, int64_t n, const qmm_qweight* w, float alpha, void* out,
                         qmm_dtype out_dtype, int32_t* d_status, void* stream) {
  qmm_status s = check_qweight(w);
  if (s != QMM_OK) return s;
  if (!dtype_ok(out_dtype)) return QMM_ERR_DTYPE;
  if (n < 0 || n > (int64_t)INT32_MAX) return QMM_ERR_INVALID_ARG;
  if (d_status && !aligned4(d_status)) return QMM_ERR_ALIGNMENT;
  if (n == 0) return QMM_OK;
  if (!aligned4(ids) || !aligned16(out)) return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  return launch_status(qmm::embed::launch_lookup(ids, n, w, alpha, out, out_dtype, d_status, (cudaStream_t)stream));
}

int64_t qmm_embedding_backward_workspace_bytes(int64_t n, int64_t rows, int64_t cols) {
  if (n < 0 || n > (int64_t)INT32_MAX || rows < 0 || rows > (int64_t)INT32_MAX || cols <= 0) return -1;
  return 16;
}

qmm_status qmm_embedding_backward(const void* dy, qmm_dtype dy_dtype, const int32_t* ids, int64_t n,
                                  const qmm_qweight* w, float alpha, void* dscales, void* dbiases, qmm_dtype g_dtype,
                                  void* workspace, int64_t workspace_bytes, int32_t* d_status, void* stream) {
  qmm_status s = check_qweight(w);
  if (s != QMM_OK) return s;
  if (w->mode != QMM_MODE_AFFINE) return QMM_ERR_UNSUPPORTED;
  if (!dtype_ok(dy_dtype) || !dtype_ok(g_dtype)) return QMM_ERR_DTYPE;
  const int64_t need = qmm_embedding_backward_workspace_bytes(n, w->rows, w->cols);
  if (need < 0 || workspace_bytes < need) return QMM_ERR_INVALID_ARG;
  if (d_status && !aligned4(d_status)) return QMM_ERR_ALIGNMENT;
  if (w->rows == 0 && n == 0) return QMM_OK;
  if ((n > 0 && (!aligned16(dy) || !aligned4(ids))) || !aligned16(dscales) || !aligned16(dbiases) ||
      !aligned16(workspace))
    return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (dy_dtype == QMM_F32)
    return launch_status(qmm::embed::launch_grad<float>(dy, ids, n, w, alpha, dscales, dbiases, g_dtype, d_status, st));
  if (dy_dtype == QMM_BF16)
    return launch_status(
        qmm::embed::launch_grad<__nv_bfloat16>(dy, ids, n, w, alpha, dscales, dbiases, g_dtype, d_status, st));
  return launch_status(qmm::embed::launch_grad<__half>(dy, ids, n, w, alpha, dscales, dbiases, g_dtype, d_status, st));
}

}  // extern "C"
