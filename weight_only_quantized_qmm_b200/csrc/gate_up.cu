// The dense gated feed-forward projection and the backward passes of the
// quantized products (one weight, or gate and up together):
//   h  = SiLU(g) * u,  g = x . dequant(gate)^T,  u = x . dequant(up)^T
//   du = dh * SiLU(g),  dg = dh * u * p * (1 + g (1 - p)),  p = 1 / (1 + e^-g)
//   dx = dy . dequant(W)                      (gate and up: the two sums)
//   dW = dy^T x;  dscales[n, j] = sum over k in group j of dW[n, k] q[n, k],
//   dbiases[n, j] = sum over k in group j of dW[n, k]
// (w_hat = q * scale + bias; the codes are constants, dW is never stored).
//
// For more than 16 tokens, and for every gradient, the products run on the
// tensor cores (pair_gemm.cuh).  The gated block's gradient is three launches:
// dg and du into the workspace, the dx product over gate and up together, and
// the parameter gradients of both.
#include <algorithm>

#include "pair_gemm.cuh"
#include "qgemv.cuh"

namespace qmm {
namespace pg {
cudaError_t dispatch_b2(int, bool, Args&, Maps&, int, cudaStream_t);
cudaError_t dispatch_b3(int, bool, Args&, Maps&, int, cudaStream_t);
cudaError_t dispatch_b4(int, bool, Args&, Maps&, int, cudaStream_t);
cudaError_t dispatch_b6(int, bool, Args&, Maps&, int, cudaStream_t);
cudaError_t dispatch_b8(int, bool, Args&, Maps&, int, cudaStream_t);
cudaError_t dispatch_both_b2(Args&, Maps&, const Args&, const Maps&, int, int, cudaStream_t);
cudaError_t dispatch_both_b3(Args&, Maps&, const Args&, const Maps&, int, int, cudaStream_t);
cudaError_t dispatch_both_b4(Args&, Maps&, const Args&, const Maps&, int, int, cudaStream_t);
cudaError_t dispatch_both_b6(Args&, Maps&, const Args&, const Maps&, int, int, cudaStream_t);
cudaError_t dispatch_both_b8(Args&, Maps&, const Args&, const Maps&, int, int, cudaStream_t);
cudaError_t dispatch_dense(int, const Args&, const Maps&, int, cudaStream_t);
cudaError_t dequant_parts(int op, int bits, const Args& p, void* ws, Maps& tm, cudaStream_t st);
}  // namespace pg

namespace ffn {

// dg and du, rounded once to T (they are operands of 16-bit products), in rows
// of ld elements.  Bound by memory: 10 bytes an element.  VEC: F is a multiple
// of 8 (then ld = F, and rows need no telling apart), 16-byte loads and stores.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256)
act_grad_kernel(const T* __restrict__ dh, const T* __restrict__ g, const T* __restrict__ u, int64_t n, int F, int ld,
                T* __restrict__ dg, T* __restrict__ du) {
  auto grad = [](float a, float b, float c, float& x, float& y) {
    const float2 p = pg::logistic<T>(b);
    x = a * c * (p.x * fmaf(b, p.y, 1.0f));
    y = a * (b * p.x);
  };
  const int64_t step = (int64_t)gridDim.x * blockDim.x, first = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
  if constexpr (VEC) {
    for (int64_t i = first; i < n / 8; i += step) {
      const uint4 a = __ldcs(reinterpret_cast<const uint4*>(dh) + i), b = __ldcs(reinterpret_cast<const uint4*>(g) + i),
                  c = __ldcs(reinterpret_cast<const uint4*>(u) + i);
      __align__(16) T ta[8], tb[8], tc[8], td[8], te[8];
      memcpy(ta, &a, 16);
      memcpy(tb, &b, 16);
      memcpy(tc, &c, 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x, y;
        grad(to_f32(ta[e]), to_f32(tb[e]), to_f32(tc[e]), x, y);
        td[e] = from_f32<T>(x);
        te[e] = from_f32<T>(y);
      }
      uint4 o0, o1;
      memcpy(&o0, td, 16);
      memcpy(&o1, te, 16);
      reinterpret_cast<uint4*>(dg)[i] = o0;
      reinterpret_cast<uint4*>(du)[i] = o1;
    }
  } else {
    for (int64_t i = first; i < n; i += step) {
      const int64_t m = i / F, at = m * ld + (i - m * F);
      float x, y;
      grad(to_f32(dh[i]), to_f32(g[i]), to_f32(u[i]), x, y);
      dg[at] = from_f32<T>(x);
      du[at] = from_f32<T>(y);
    }
  }
}

template <typename T>
static cudaError_t act_grad(const void* dh, const void* g, const void* u, int64_t n, int F, int ld, void* dg, void* du,
                            cudaStream_t st) {
  const bool vec = F % 8 == 0;
  const int64_t items = vec ? n / 8 : n;
  const int grid = (int)std::min<int64_t>((items + 255) / 256, (int64_t)qmm_host::num_sms() * 8);
  if (vec)
    act_grad_kernel<T, true><<<grid, 256, 0, st>>>((const T*)dh, (const T*)g, (const T*)u, n, F, ld, (T*)dg, (T*)du);
  else
    act_grad_kernel<T, false><<<grid, 256, 0, st>>>((const T*)dh, (const T*)g, (const T*)u, n, F, ld, (T*)dg, (T*)du);
  return cudaGetLastError();
}

// rows of n elements to rows of ld
__global__ void __launch_bounds__(256)
pad_kernel(const uint16_t* __restrict__ src, int64_t n, int F, int ld, uint16_t* __restrict__ dst) {
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x)
    dst[i / F * ld + i % F] = src[i];
}

static int blocks_for(int64_t n) { return (int)std::min<int64_t>((n + 255) / 256, (int64_t)qmm_host::num_sms() * 8); }

static pg::Weight weight_of(const qmm_qweight* w) { return pg::Weight{w->packed, w->scales, w->biases}; }

static pg::Args args_of(int64_t M, int64_t K, const qmm_qweight* w0, const qmm_qweight* w1, int x_dtype) {
  pg::Args p{};
  p.M = (int)M;
  p.K = (int)K;
  p.N = (int)w0->rows;
  p.parts = w1 ? 2 : 1;
  p.w[0] = weight_of(w0);
  p.w[1] = weight_of(w1 ? w1 : w0);
  p.lgs = w0->group_size == 32 ? 5 : w0->group_size == 64 ? 6 : 7;
  p.f16 = x_dtype == QMM_F16;
  return p;
}

static int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// How a product runs: weights dequantized beforehand or in the kernel, on CTA
// pairs or single CTAs, and how many of those share a tile.
struct Plan {
  bool dense, pair;
  int splits;
  int m_tiles, n_tiles;
};

// The cheapest by the times measured for one 64-deep step (us, 4096 x 14336, 4
// bits): a pair's 256 x 256 tile 0.39 from dense weights and 0.45 dequantizing,
// a single CTA's 128 x 256 tile 0.66; 3 us to join splits; and for the
// dequantizing pass 2 us and its bytes at 4.5 TB/s.  Kernels that dequantize want
// rows of codes on 16 bytes; dx runs on pairs only, which shares a launch with the
// parameter gradients.  Clusters of 4 find room on 132 of the 148 SMs, clusters
// of 8 on 120 (cudaOccupancyMaxActiveClusters).  Other widths are priced alike: at
// each of them, 64 to 2048 tokens forward and dx, each way forced, the choice was
// within 5% of the best, but for 2048 tokens of 8-bit bf16 codes, whose conversion
// costs more (dx 222 us against 205 dense).
static Plan plan_of(int op, int64_t M, int64_t K, int64_t N, int parts, int bits) {
  const int64_t out = op == pg::FWD ? N : K;  // columns of the output
  const int tn = op == pg::FWD ? 128 : 256;
  const int steps = op == pg::FWD ? ceil_div(K, pg::kBK) : parts * ceil_div(N, pg::kBK);
  const int sms = qmm_host::num_sms();
  Plan best{};
  double cost = 1e300;
  for (int kind = 0; kind < (op == pg::FWD ? 3 : 2); ++kind) {
    const bool dense = kind == 0, pair = kind < 2;
    if (!dense && (K * bits) % 128 != 0) continue;
    const int64_t mt = ceil_div(M, pair ? 256 : 128), nt = ceil_div(out, tn);
    for (int s = 1; s <= (pair ? 4 : 8); s *= 2) {
      const int ctas = (pair ? 2 : 1) * s;
      const int room = (ctas >= 8 ? sms * 120 / 148 : ctas >= 4 ? sms * 132 / 148 : sms) / ctas;
      if (s > 1 && (mt * nt > room || steps < 4 * s)) break;
      const double waves = (double)((mt * nt + room - 1) / room);
      const double c = waves * ceil_div(steps, s) * (dense ? 0.39 : pair ? 0.45 : 0.66) + (s > 1 ? 3.0 : 0.0) +
                       (dense ? 2.0 + (double)parts * N * K * (2.0 + bits / 8.0) / 4.5e6 : 0.0);
      if (c < cost) {
        cost = c;
        best = Plan{dense, pair, s, (int)mt, (int)nt};
      }
    }
  }
  return best;
}

// bits == 0: weights dequantized beforehand
static cudaError_t run(int op, int bits, const Plan& plan, pg::Args& p, pg::Maps& tm, cudaStream_t st) {
  p.m_tiles = plan.m_tiles;
  p.n_tiles = plan.n_tiles;
  p.splits = plan.splits;
  const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles * (op == pg::DP ? p.parts : 1);
  if (tiles > INT32_MAX / 16) return cudaErrorInvalidValue;
  const int sms = qmm_host::num_sms();
  const int clusters = plan.splits > 1 ? (int)tiles : (int)std::min<int64_t>(tiles, plan.pair ? sms / 2 : sms);
  switch (bits) {
    case 0: return pg::dispatch_dense(op, p, tm, clusters, st);
    case 2: return pg::dispatch_b2(op, plan.pair, p, tm, clusters, st);
    case 3: return pg::dispatch_b3(op, plan.pair, p, tm, clusters, st);
    case 4: return pg::dispatch_b4(op, plan.pair, p, tm, clusters, st);
    case 6: return pg::dispatch_b6(op, plan.pair, p, tm, clusters, st);
    default: return pg::dispatch_b8(op, plan.pair, p, tm, clusters, st);
  }
}

// dense: room for both dequantized weights where the plan wants it
static cudaError_t forward(const void* x, int x_dtype, int64_t M, int64_t K, const qmm_qweight* gate,
                           const qmm_qweight* up, void* h, int h_dtype, void* gp, void* upre, void* dense,
                           cudaStream_t st) {
  pg::Args p = args_of(M, K, gate, up, x_dtype);
  const Plan plan = plan_of(pg::FWD, M, K, gate->rows, 2, gate->bits);
  p.steps = ceil_div(K, pg::kBK);
  p.out[0] = h;
  p.out[1] = gp;
  p.out[2] = upre;
  p.out_dtype = h_dtype;
  pg::Maps tm;
  if (!pg::make_map(&tm.a[0], x, p.f16, M, K, K, 128)) return cudaErrorInvalidValue;
  tm.a[1] = tm.b[0] = tm.b[1] = tm.s[0] = tm.s[1] = tm.z[0] = tm.z[1] = tm.a[0];
  const cudaError_t e = plan.dense ? pg::dequant_parts(pg::FWD, gate->bits, p, dense, tm, st) : cudaSuccess;
  return e != cudaSuccess ? e : run(pg::FWD, plan.dense ? 0 : gate->bits, plan, p, tm, st);
}

// dy0 (and dy1): [M, N] in rows of ld elements, ld a multiple of 8
static cudaError_t backward(const void* dy0, const void* dy1, int64_t ld, const void* x, int x_dtype, int64_t M,
                            int64_t K, const qmm_qweight* w0, const qmm_qweight* w1, void* dx, void* const* grads,
                            int g_dtype, void* dense, cudaStream_t st) {
  const int64_t N = w0->rows;
  if (M == 0 || N == 0) {  // empty sums
    cudaError_t e = cudaSuccess;
    if (dx && M > 0) e = cudaMemsetAsync(dx, 0, (size_t)(M * K * 2), st);
    const size_t bytes = (size_t)(N * (K / w0->group_size) * qmm_host::dtype_size((qmm_dtype)g_dtype));
    for (int i = 0; i < (w1 ? 4 : 2) && grads[0] && bytes && e == cudaSuccess; ++i)
      e = cudaMemsetAsync(grads[i], 0, bytes, st);
    return e;
  }
  pg::Args a = args_of(M, K, w0, w1, x_dtype), g = a;  // dx, parameter gradients
  pg::Maps am, gm;
  Plan plan{};
  if (dx) {
    plan = plan_of(pg::DX, M, K, N, a.parts, w0->bits);
    a.steps = a.parts * ceil_div(N, pg::kBK);
    a.out[0] = dx;
    a.out_dtype = x_dtype;
    if (!pg::make_map(&am.a[0], dy0, a.f16, M, N, ld, 128)) return cudaErrorInvalidValue;
    if (!w1)
      am.a[1] = am.a[0];
    else if (!pg::make_map(&am.a[1], dy1, a.f16, M, N, ld, 128))
      return cudaErrorInvalidValue;
    am.b[0] = am.b[1] = am.s[0] = am.s[1] = am.z[0] = am.z[1] = am.a[0];
  }
  const Plan gplan{true, true, 1, ceil_div(N, 256), ceil_div(K, 256)};
  if (grads[0]) {
    g.steps = ceil_div(M, pg::kBK);
    for (int i = 0; i < 4; ++i) g.out[i] = grads[i];
    g.out_dtype = g_dtype;
    if (!pg::make_map(&gm.a[0], dy0, g.f16, M, N, ld, 64) || !pg::make_map(&gm.b[0], x, g.f16, M, K, K, 64))
      return cudaErrorInvalidValue;
    if (!w1)
      gm.a[1] = gm.a[0];
    else if (!pg::make_map(&gm.a[1], dy1, g.f16, M, N, ld, 64))
      return cudaErrorInvalidValue;
    gm.b[1] = gm.s[0] = gm.s[1] = gm.z[0] = gm.z[1] = gm.b[0];
  }
  const int sms = qmm_host::num_sms();
  const int64_t tiles = (int64_t)plan.m_tiles * plan.n_tiles, gtiles = (int64_t)gplan.m_tiles * gplan.n_tiles * g.parts;
  const int pairs = (plan.splits == 4 ? sms * 120 / 148 : plan.splits == 2 ? sms * 132 / 148 : sms) / 2;
  if (dx && grads[0] && !plan.dense && tiles * plan.splits <= pairs - pairs / 4) {
    // one launch: the parameter gradients take the pairs that dx leaves (64 tokens
    // of 4096 x 14336: 138 us against 104 + 66; where dx leaves less than a quarter
    // of the SMs, two launches are as fast: 1024 tokens 497 us against 250 + 220)
    a.m_tiles = plan.m_tiles;
    a.n_tiles = plan.n_tiles;
    a.splits = plan.splits;
    g.m_tiles = gplan.m_tiles;
    g.n_tiles = gplan.n_tiles;
    g.splits = 1;
    const int clusters = (int)tiles;
    int gpairs = (int)std::min<int64_t>(gtiles, pairs - clusters * plan.splits);
    gpairs = (gpairs + plan.splits - 1) / plan.splits * plan.splits;
    if (gtiles > INT32_MAX / 16) return cudaErrorInvalidValue;
    switch (w0->bits) {
      case 2: return pg::dispatch_both_b2(a, am, g, gm, clusters, gpairs, st);
      case 3: return pg::dispatch_both_b3(a, am, g, gm, clusters, gpairs, st);
      case 4: return pg::dispatch_both_b4(a, am, g, gm, clusters, gpairs, st);
      case 6: return pg::dispatch_both_b6(a, am, g, gm, clusters, gpairs, st);
      default: return pg::dispatch_both_b8(a, am, g, gm, clusters, gpairs, st);
    }
  }
  if (dx) {
    cudaError_t e = plan.dense ? pg::dequant_parts(pg::DX, w0->bits, a, dense, am, st) : cudaSuccess;
    if (e == cudaSuccess) e = run(pg::DX, plan.dense ? 0 : w0->bits, plan, a, am, st);
    if (e != cudaSuccess) return e;
  }
  return grads[0] ? run(pg::DP, w0->bits, gplan, g, gm, st) : cudaSuccess;
}

static int64_t padded(int64_t n) { return (n + 7) / 8 * 8; }
static int64_t align16(int64_t n) { return (n + 15) / 16 * 16; }
// bytes of the weights that the plan wants dequantized
static int64_t dense_bytes(int op, int64_t M, int64_t K, int64_t N, int bits, int parts) {
  return M > 0 && N > 0 && plan_of(op, M, K, N, parts, bits).dense ? parts * N * K * 2 : 0;
}

}  // namespace ffn
}  // namespace qmm

using namespace qmm_host;

namespace {

// Tokens of the streaming kernels, which keep the weights exact.  They are ahead of
// the tensor cores up to 12 tokens (4096 x 14336 bf16, us: 9 tokens 34 against 62 at
// 4 bits, 37 against 67 at 3; 12 tokens 37 against 59, 54 against 66 at 6) but for
// 8-bit bf16 codes (74 against 69), and at 16 tokens for 2 and 3 bits (39 against 48,
// 50 against 53); 4, 6 and 8 bits lose 13%, 8% and 24% there (48, 57, 81).
constexpr int64_t kFewTokens = 16;

// sizes: 32 bits, and so are the rows and columns past the last one of a tile
bool i32(int64_t v) { return v >= 0 && v <= (int64_t)INT32_MAX - 1023; }
// M rows of n elements (padded) and n rows of K, all within 2^57 elements
bool fits(int64_t M, int64_t K, int64_t n) {
  return std::max(M, K) <= ((int64_t)1 << 57) / (n + 8);
}

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

// A gradient call whose every output is not asked for or holds no elements: the
// dx of no tokens, the parameter gradients of no rows (an empty tensor's address
// may be null, as that of an output that is not asked for is).
bool nothing_to_write(int64_t M, int64_t rows, const void* dx, const void* grad) {
  return (M == 0 && !grad) || (rows == 0 && !dx);
}

}  // namespace

extern "C" {

int64_t qmm_gate_up_silu_workspace_bytes(int64_t M, int64_t K, int64_t F, int bits) {
  if (!i32(M) || !i32(K) || !i32(F) || !fits(M, K, F) || qmm_packed_words_per_row(K, bits) < 0) return -1;
  return M > kFewTokens ? qmm::ffn::dense_bytes(qmm::pg::FWD, M, K, F, bits, 2) : 0;
}

qmm_status qmm_gate_up_silu(const void* x, qmm_dtype x_dtype, int64_t M, int64_t K, const qmm_qweight* gate,
                            const qmm_qweight* up, void* h, qmm_dtype h_dtype, void* g_pre, void* u_pre,
                            void* workspace, int64_t workspace_bytes, void* stream) {
  qmm_status s = check_pair(gate, up, x_dtype, M, K);
  if (s != QMM_OK) return s;
  if (!dtype_ok(h_dtype) || (h_dtype != x_dtype && h_dtype != QMM_F32)) return QMM_ERR_DTYPE;
  if ((g_pre == nullptr) != (u_pre == nullptr)) return QMM_ERR_INVALID_ARG;
  const int64_t need = qmm_gate_up_silu_workspace_bytes(M, K, gate->rows, gate->bits);
  if (need < 0 || workspace_bytes < need) return QMM_ERR_INVALID_ARG;
  if (M == 0 || gate->rows == 0) return QMM_OK;
  if (need > 0 && !aligned16(workspace)) return QMM_ERR_ALIGNMENT;
  if (!aligned16(x) || !aligned16(h) || (g_pre && (!aligned16(g_pre) || !aligned16(u_pre)))) return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (M <= kFewTokens) {  // the streaming kernels, both matrices in one pass
    const qmm::QgemvParams p = qmm::make_gated_params(x, x_dtype, M, K, gate, up, h, h_dtype, g_pre, u_pre);
    const cudaError_t e = qmm::launch_qgemv(p, gate->bits, gate->group_size, x_dtype, true, st);
    return e == cudaErrorInvalidValue ? QMM_ERR_UNSUPPORTED : launch_status(e);
  }
  return launch_status(qmm::ffn::forward(x, x_dtype, M, K, gate, up, h, h_dtype, g_pre, u_pre, workspace, st));
}

int64_t qmm_matmul_backward_workspace_bytes(int64_t M, int64_t K, int64_t N, int bits) {
  if (!i32(M) || !i32(K) || !i32(N) || !fits(M, K, N) || qmm_packed_words_per_row(K, bits) < 0) return -1;
  // rows of dy that do not start on 16 bytes are copied to ones that do
  return qmm::ffn::align16(N % 8 ? M * qmm::ffn::padded(N) * 2 : 0) +
         qmm::ffn::dense_bytes(qmm::pg::DX, M, K, N, bits, 1);
}

qmm_status qmm_matmul_backward(const void* dy, const void* x, qmm_dtype x_dtype, int64_t M, int64_t K,
                               const qmm_qweight* w, void* dx, void* dscales, void* dbiases, qmm_dtype g_dtype,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  qmm_status s = check_weight(w, x_dtype, M, K);
  if (s != QMM_OK) return s;
  if (!dtype_ok(g_dtype) || (g_dtype != x_dtype && g_dtype != QMM_F32)) return QMM_ERR_DTYPE;
  if ((dscales == nullptr) != (dbiases == nullptr)) return QMM_ERR_INVALID_ARG;
  if (nothing_to_write(M, w->rows, dx, dscales)) return QMM_OK;
  if (!dx && !dscales) return QMM_ERR_INVALID_ARG;
  const int64_t need = qmm_matmul_backward_workspace_bytes(M, K, w->rows, w->bits);
  if (need < 0 || workspace_bytes < need) return QMM_ERR_INVALID_ARG;
  if (M > 0 && w->rows > 0 && (!aligned16(dy) || (dscales && !aligned16(x)))) return QMM_ERR_ALIGNMENT;
  if ((dx && !aligned16(dx)) || (dscales && (!aligned16(dscales) || !aligned16(dbiases))) ||
      (need > 0 && !aligned16(workspace)))
    return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  void* const grads[4] = {dscales, dbiases, nullptr, nullptr};
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t N = w->rows, ld = qmm::ffn::padded(N), n = M * N;
  if (ld != N && n > 0) {
    qmm::ffn::pad_kernel<<<qmm::ffn::blocks_for(n), 256, 0, st>>>((const uint16_t*)dy, n, (int)N, (int)ld,
                                                                  (uint16_t*)workspace);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return launch_status(e);
    dy = workspace;
  }
  void* dense = static_cast<char*>(workspace) + qmm::ffn::align16(N % 8 ? M * ld * 2 : 0);
  return launch_status(qmm::ffn::backward(dy, nullptr, ld, x, x_dtype, M, K, w, nullptr, dx, grads, g_dtype, dense, st));
}

int64_t qmm_gate_up_silu_backward_workspace_bytes(int64_t M, int64_t K, int64_t F, int bits) {
  if (!i32(M) || !i32(K) || !i32(F) || !fits(M, K, F) || qmm_packed_words_per_row(K, bits) < 0) return -1;
  return qmm::ffn::align16(2 * M * qmm::ffn::padded(F) * 2) +
         qmm::ffn::dense_bytes(qmm::pg::DX, M, K, F, bits, 2);  // dg and du first
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
  if (nothing_to_write(M, gate->rows, dx, grads[0])) return QMM_OK;
  if (!dx && !grads[0]) return QMM_ERR_INVALID_ARG;
  const int64_t F = gate->rows;
  const int64_t need = qmm_gate_up_silu_backward_workspace_bytes(M, K, F, gate->bits);
  if (need < 0 || workspace_bytes < need) return QMM_ERR_INVALID_ARG;
  if (M > 0 && F > 0 && (!aligned16(dh) || (grads[0] && !aligned16(x)) || !aligned16(g_pre) || !aligned16(u_pre)))
    return QMM_ERR_ALIGNMENT;
  if ((dx && !aligned16(dx)) || (need > 0 && !aligned16(workspace))) return QMM_ERR_ALIGNMENT;
  for (int i = 0; i < 4; ++i)
    if (grads[i] && !aligned16(grads[i])) return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  const int64_t ld = qmm::ffn::padded(F), n = M * F;
  uint16_t* dg = static_cast<uint16_t*>(workspace);
  uint16_t* du = dg + M * ld;
  if (n > 0) {
    const cudaError_t e =
        x_dtype == QMM_BF16
            ? qmm::ffn::act_grad<__nv_bfloat16>(dh, g_pre, u_pre, n, (int)F, (int)ld, dg, du, st)
            : qmm::ffn::act_grad<__half>(dh, g_pre, u_pre, n, (int)F, (int)ld, dg, du, st);
    if (e != cudaSuccess) return launch_status(e);
  }
  void* dense = static_cast<char*>(workspace) + qmm::ffn::align16(2 * M * ld * 2);
  return launch_status(qmm::ffn::backward(dg, du, ld, x, x_dtype, M, K, gate, up, dx, grads, g_dtype, dense, st));
}

}  // extern "C"
