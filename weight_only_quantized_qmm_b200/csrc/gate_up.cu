// The dense gated feed-forward projection and the backward passes of the
// quantized products (one weight, or gate and up together):
//   h  = SiLU(g) * u,  g = x . dequant(gate)^T,  u = x . dequant(up)^T
//   du = dh * SiLU(g),  dg = dh * u * p * (1 + g (1 - p)),  p = 1 / (1 + e^-g)
//   dx = dy . dequant(W)                      (gate and up: the two sums)
//   dW = dy^T x;  dscales[n, j] = sum over k in group j of dW[n, k] q[n, k],
//   dbiases[n, j] = sum over k in group j of dW[n, k]
// (w_hat = q * scale + bias; the codes are constants, dW is never stored).
#include <algorithm>

#include "common.cuh"

namespace qmm {
namespace ffn {

constexpr int kT = 16;  // tile of the simple kernels

template <int B>
__device__ __forceinline__ float code_at(const uint32_t* row, int64_t i) {
  const int64_t bit = i * B;
  const int sh = (int)(bit & 31);
  uint32_t v = row[bit >> 5] >> sh;
  if (sh + B > 32) v |= row[(bit >> 5) + 1] << (32 - sh);
  return (float)(v & ((1u << B) - 1u));
}

struct Weight {
  const uint32_t* packed;
  const void* scales;
  const void* biases;
};

template <int B, typename T>
__device__ __forceinline__ float w_at(const Weight& w, int64_t n, int64_t k, int64_t K, int gs) {
  const int64_t G = K / gs;
  return fmaf(code_at<B>(w.packed + n * (K * B / 32), k), to_f32(reinterpret_cast<const T*>(w.scales)[n * G + k / gs]),
              to_f32(reinterpret_cast<const T*>(w.biases)[n * G + k / gs]));
}

template <int B, typename T>
__global__ void __launch_bounds__(kT * kT)
gate_up_kernel(const T* __restrict__ x, int M, int K, int F, int gs, Weight gate, Weight up, void* h, int h_dtype, T* gp,
               T* upre) {
  __shared__ float xs[kT][kT + 1], ws[2][kT][kT + 1];
  const int tx = threadIdx.x % kT, ty = threadIdx.x / kT;
  const int64_t m = (int64_t)blockIdx.y * kT + ty, n = (int64_t)blockIdx.x * kT + tx;
  float g = 0.0f, u = 0.0f;
  for (int k0 = 0; k0 < K; k0 += kT) {
    const int64_t wr = (int64_t)blockIdx.x * kT + ty;
    xs[ty][tx] = m < M ? to_f32(x[m * K + k0 + tx]) : 0.0f;
    ws[0][ty][tx] = wr < F ? w_at<B, T>(gate, wr, k0 + tx, K, gs) : 0.0f;
    ws[1][ty][tx] = wr < F ? w_at<B, T>(up, wr, k0 + tx, K, gs) : 0.0f;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kT; ++k) {
      g = fmaf(xs[ty][k], ws[0][tx][k], g);
      u = fmaf(xs[ty][k], ws[1][tx][k], u);
    }
    __syncthreads();
  }
  if (m < M && n < F) {
    store_as(h, h_dtype, m * F + n, g / (1.0f + expf(-g)) * u);
    if (gp) {
      gp[m * F + n] = from_f32<T>(g);
      upre[m * F + n] = from_f32<T>(u);
    }
  }
}

// dg, du of one element
__device__ __forceinline__ void silu_mul_grad(float dh, float g, float u, float& dg, float& du) {
  const float p = 1.0f / (1.0f + expf(-g));
  du = dh * (g * p);
  dg = dh * u * (p * (1.0f + g * (1.0f - p)));
}

template <typename T>
__global__ void __launch_bounds__(256)
act_grad_kernel(const T* __restrict__ dh, const T* __restrict__ g, const T* __restrict__ u, int64_t n, T* dg, T* du) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    float a, b;
    silu_mul_grad(to_f32(dh[i]), to_f32(g[i]), to_f32(u[i]), a, b);
    dg[i] = from_f32<T>(a);
    du[i] = from_f32<T>(b);
  }
}

template <int B, typename T>
__global__ void __launch_bounds__(kT * kT)
dx_kernel(const T* __restrict__ dy0, const T* __restrict__ dy1, int M, int K, int N, int gs, Weight w0, Weight w1,
          int parts, T* dx) {
  __shared__ float ys[kT][kT + 1], ws[kT][kT + 1];
  const int tx = threadIdx.x % kT, ty = threadIdx.x / kT;
  const int64_t m = (int64_t)blockIdx.y * kT + ty, k = (int64_t)blockIdx.x * kT + tx;
  float acc = 0.0f;
  for (int part = 0; part < parts; ++part)
    for (int n0 = 0; n0 < N; n0 += kT) {
      ys[ty][tx] = m < M && n0 + tx < N ? to_f32((part ? dy1 : dy0)[m * N + n0 + tx]) : 0.0f;
      ws[ty][tx] = n0 + ty < N && k < K ? w_at<B, T>(part ? w1 : w0, n0 + ty, k, K, gs) : 0.0f;
      __syncthreads();
#pragma unroll
      for (int n = 0; n < kT; ++n) acc = fmaf(ys[ty][n], ws[n][tx], acc);
      __syncthreads();
    }
  if (m < M && k < K) dx[m * K + k] = from_f32<T>(acc);
}

// one warp per (row, group)
template <int B, typename T>
__global__ void __launch_bounds__(256)
param_grad_kernel(const T* __restrict__ dy, const T* __restrict__ x, int M, int K, int N, int gs,
                  const uint32_t* __restrict__ packed, void* dscales, void* dbiases, int g_dtype) {
  const int64_t G = K / gs, id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (id >= (int64_t)N * G) return;
  const int64_t n = id / G, j = id % G;
  float ds = 0.0f, db = 0.0f;
  for (int64_t k = j * gs + lane; k < (j + 1) * gs; k += 32) {
    float a = 0.0f;
    for (int64_t m = 0; m < M; ++m) a = fmaf(to_f32(dy[m * N + n]), to_f32(x[m * K + k]), a);
    ds = fmaf(a, code_at<B>(packed + n * ((int64_t)K * B / 32), k), ds);
    db += a;
  }
  for (int o = 16; o > 0; o >>= 1) {
    ds += __shfl_xor_sync(0xffffffffu, ds, o);
    db += __shfl_xor_sync(0xffffffffu, db, o);
  }
  if (lane == 0) {
    store_as(dscales, g_dtype, id, ds);
    store_as(dbiases, g_dtype, id, db);
  }
}

static Weight weight_of(const qmm_qweight* w) { return Weight{w->packed, w->scales, w->biases}; }

#define QMM_BITS(bits, CALL) \
  switch (bits) {            \
    case 2: CALL(2); break;  \
    case 3: CALL(3); break;  \
    case 4: CALL(4); break;  \
    case 6: CALL(6); break;  \
    default: CALL(8); break; \
  }

template <typename T>
static cudaError_t forward_t(const void* x, int64_t M, int64_t K, const qmm_qweight* gate, const qmm_qweight* up, void* h,
                             int h_dtype, void* gp, void* upre, cudaStream_t st) {
  const int64_t F = gate->rows;
  const dim3 grid((unsigned)((F + kT - 1) / kT), (unsigned)((M + kT - 1) / kT));
#define QMM_C(BB)                                                                                                    \
  gate_up_kernel<BB, T><<<grid, kT * kT, 0, st>>>((const T*)x, (int)M, (int)K, (int)F, gate->group_size,             \
                                                  weight_of(gate), weight_of(up), h, h_dtype, (T*)gp, (T*)upre)
  QMM_BITS(gate->bits, QMM_C)
#undef QMM_C
  return cudaGetLastError();
}

template <typename T>
static cudaError_t backward_t(const void* dy0, const void* dy1, const void* x, int64_t M, int64_t K,
                              const qmm_qweight* w0, const qmm_qweight* w1, void* dx, void* const* grads, int g_dtype,
                              cudaStream_t st) {
  const int64_t N = w0->rows;
  if (dx && M > 0) {
    const dim3 grid((unsigned)((K + kT - 1) / kT), (unsigned)((M + kT - 1) / kT));
#define QMM_C(BB)                                                                                            \
  dx_kernel<BB, T><<<grid, kT * kT, 0, st>>>((const T*)dy0, (const T*)dy1, (int)M, (int)K, (int)N, w0->group_size, \
                                             weight_of(w0), weight_of(w1 ? w1 : w0), w1 ? 2 : 1, (T*)dx)
    QMM_BITS(w0->bits, QMM_C)
#undef QMM_C
  }
  for (int p = 0; grads[0] && p < (w1 ? 2 : 1); ++p) {
    const int64_t items = N * (K / w0->group_size);
    const unsigned grid = (unsigned)((items + 7) / 8);
    if (items == 0) continue;
#define QMM_C(BB)                                                                                                   \
  param_grad_kernel<BB, T><<<grid, 256, 0, st>>>((const T*)(p ? dy1 : dy0), (const T*)x, (int)M, (int)K, (int)N,    \
                                                 w0->group_size, p ? w1->packed : w0->packed, grads[2 * p],         \
                                                 grads[2 * p + 1], g_dtype)
    QMM_BITS(w0->bits, QMM_C)
#undef QMM_C
  }
  return cudaGetLastError();
}

}  // namespace ffn
}  // namespace qmm

using namespace qmm_host;

namespace {

bool i32(int64_t v) { return v >= 0 && v <= (int64_t)INT32_MAX; }

// The rules shared by the gated block and the backward passes: affine
// weights, 16-bit activations of the scales' dtype.
qmm_status check_weight(const qmm_qweight* w, qmm_dtype x_dtype, int64_t M, int64_t K) {
  const qmm_status s = check_qweight(w);
  if (s != QMM_OK) return s;
  if (w->mode != QMM_MODE_AFFINE) return QMM_ERR_UNSUPPORTED;
  if (!dtype_ok(x_dtype) || x_dtype != w->sdtype) return QMM_ERR_DTYPE;
  if (M < 0 || K <= 0 || w->cols != K) return QMM_ERR_INVALID_ARG;
  if (x_dtype == QMM_F32) return QMM_ERR_UNSUPPORTED;  // tensor-core path only
  if (!i32(M) || !i32(K) || !i32(w->rows)) return QMM_ERR_UNSUPPORTED;
  return QMM_OK;
}

qmm_status check_pair(const qmm_qweight* gate, const qmm_qweight* up, qmm_dtype x_dtype, int64_t M, int64_t K) {
  qmm_status s = check_weight(gate, x_dtype, M, K);
  if (s != QMM_OK) return s;
  s = check_weight(up, x_dtype, M, K);
  if (s != QMM_OK) return s;
  return up->rows == gate->rows && up->group_size == gate->group_size && up->bits == gate->bits ? QMM_OK
                                                                                                : QMM_ERR_INVALID_ARG;
}

}  // namespace

extern "C" {

qmm_status qmm_gate_up_silu(const void* x, qmm_dtype x_dtype, int64_t M, int64_t K, const qmm_qweight* gate,
                            const qmm_qweight* up, void* h, qmm_dtype h_dtype, void* g_pre, void* u_pre, void* stream) {
  qmm_status s = check_pair(gate, up, x_dtype, M, K);
  if (s != QMM_OK) return s;
  if (!dtype_ok(h_dtype) || (h_dtype != x_dtype && h_dtype != QMM_F32)) return QMM_ERR_DTYPE;
  if ((g_pre == nullptr) != (u_pre == nullptr)) return QMM_ERR_INVALID_ARG;
  if (M == 0 || gate->rows == 0) return QMM_OK;
  if (!aligned16(x) || !aligned16(h) || (g_pre && (!aligned16(g_pre) || !aligned16(u_pre)))) return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  return launch_status(x_dtype == QMM_BF16
                           ? qmm::ffn::forward_t<__nv_bfloat16>(x, M, K, gate, up, h, h_dtype, g_pre, u_pre, st)
                           : qmm::ffn::forward_t<__half>(x, M, K, gate, up, h, h_dtype, g_pre, u_pre, st));
}

int64_t qmm_matmul_backward_workspace_bytes(int64_t M, int64_t K, int64_t N) {
  if (!i32(M) || !i32(K) || !i32(N)) return -1;
  return 16;
}

qmm_status qmm_matmul_backward(const void* dy, const void* x, qmm_dtype x_dtype, int64_t M, int64_t K,
                               const qmm_qweight* w, void* dx, void* dscales, void* dbiases, qmm_dtype g_dtype,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  qmm_status s = check_weight(w, x_dtype, M, K);
  if (s != QMM_OK) return s;
  if (!dtype_ok(g_dtype) || (g_dtype != x_dtype && g_dtype != QMM_F32)) return QMM_ERR_DTYPE;
  if ((dscales == nullptr) != (dbiases == nullptr) || (!dx && !dscales)) return QMM_ERR_INVALID_ARG;
  if (workspace_bytes < qmm_matmul_backward_workspace_bytes(M, K, w->rows)) return QMM_ERR_INVALID_ARG;
  if (M > 0 && w->rows > 0 && (!aligned16(dy) || !aligned16(x))) return QMM_ERR_ALIGNMENT;
  if ((dx && !aligned16(dx)) || (dscales && (!aligned16(dscales) || !aligned16(dbiases))) || !aligned16(workspace))
    return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  void* const grads[4] = {dscales, dbiases, nullptr, nullptr};
  cudaStream_t st = (cudaStream_t)stream;
  return launch_status(
      x_dtype == QMM_BF16
          ? qmm::ffn::backward_t<__nv_bfloat16>(dy, nullptr, x, M, K, w, nullptr, dx, grads, g_dtype, st)
          : qmm::ffn::backward_t<__half>(dy, nullptr, x, M, K, w, nullptr, dx, grads, g_dtype, st));
}

int64_t qmm_gate_up_silu_backward_workspace_bytes(int64_t M, int64_t K, int64_t F) {
  if (!i32(M) || !i32(K) || !i32(F)) return -1;
  return 16 + (M * F * 2 + 15) / 16 * 16 * 2;
}

qmm_status qmm_gate_up_silu_backward(const void* dh, const void* x, const void* g_pre, const void* u_pre,
                                     qmm_dtype x_dtype, int64_t M, int64_t K, const qmm_qweight* gate,
                                     const qmm_qweight* up, void* dx, void* dgate_scales, void* dgate_biases,
                                     void* dup_scales, void* dup_biases, qmm_dtype g_dtype, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
  qmm_status s = check_pair(gate, up, x_dtype, M, K);
  if (s != QMM_OK) return s;
  if (!dtype_ok(g_dtype) || (g_dtype != x_dtype && g_dtype != QMM_F32)) return QMM_ERR_DTYPE;
  void* const grads[4] = {dgate_scales, dgate_biases, dup_scales, dup_biases};
  for (int i = 1; i < 4; ++i)
    if ((grads[i] == nullptr) != (grads[0] == nullptr)) return QMM_ERR_INVALID_ARG;
  if (!dx && !grads[0]) return QMM_ERR_INVALID_ARG;
  const int64_t F = gate->rows;
  if (workspace_bytes < qmm_gate_up_silu_backward_workspace_bytes(M, K, F)) return QMM_ERR_INVALID_ARG;
  if (M > 0 && F > 0 && (!aligned16(dh) || !aligned16(x) || !aligned16(g_pre) || !aligned16(u_pre)))
    return QMM_ERR_ALIGNMENT;
  if ((dx && !aligned16(dx)) || !aligned16(workspace)) return QMM_ERR_ALIGNMENT;
  for (int i = 0; i < 4; ++i)
    if (grads[i] && !aligned16(grads[i])) return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  char* dg = static_cast<char*>(workspace);
  char* du = dg + (M * F * 2 + 15) / 16 * 16;
  const int64_t n = M * F;
  if (n > 0) {
    const int grid = (int)std::min<int64_t>((n + 255) / 256, 148 * 16);
    if (x_dtype == QMM_BF16) {
      using T = __nv_bfloat16;
      qmm::ffn::act_grad_kernel<T><<<grid, 256, 0, st>>>((const T*)dh, (const T*)g_pre, (const T*)u_pre, n, (T*)dg, (T*)du);
    } else {
      using T = __half;
      qmm::ffn::act_grad_kernel<T><<<grid, 256, 0, st>>>((const T*)dh, (const T*)g_pre, (const T*)u_pre, n, (T*)dg, (T*)du);
    }
  }
  return launch_status(
      x_dtype == QMM_BF16
          ? qmm::ffn::backward_t<__nv_bfloat16>(dg, du, x, M, K, gate, up, dx, grads, g_dtype, st)
          : qmm::ffn::backward_t<__half>(dg, du, x, M, K, gate, up, dx, grads, g_dtype, st));
}

}  // extern "C"
