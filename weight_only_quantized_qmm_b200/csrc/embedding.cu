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
#include "f32x2.cuh"
#include "mx.cuh"

namespace qmm {
namespace embed {

template <typename K, typename A>
static cudaError_t launch_next(K kernel, dim3 grid, int threads, int cluster, const A& args, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args);
}

// 8 codes (B bytes, 1- or 2-byte aligned for 3- and 6-bit codes) as words
template <int B>
__device__ __forceinline__ void load8(const uint8_t* src, uint32_t (&w)[3]) {
  w[0] = w[1] = w[2] = 0u;
  if constexpr (B == 8) {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(src));
    w[0] = q.x;
    w[1] = q.y;
  } else if constexpr (B == 4) {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
  } else if constexpr (B == 2 || B == 6) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(src);
    w[0] = __ldg(h);
    if constexpr (B == 6) {
      w[0] |= (uint32_t)__ldg(h + 1) << 16;
      w[1] = __ldg(h + 2);
    }
  } else {
    w[0] = __ldg(src) | ((uint32_t)__ldg(src + 1) << 8) | ((uint32_t)__ldg(src + 2) << 16);
  }
}

constexpr int kLookThreads = 256;
constexpr int kLookTokens = 4;  // rows a thread has in flight

struct LookArgs {
  const int32_t* ids;
  const uint32_t* packed;
  const void* scales;
  const void* biases;
  int rows, n;
  int pieces, lgs;      // pieces: 8 columns each
  int lanes;            // threads of a block on one row: a power of two
  float alpha;
  void* out;
  int32_t* d_status;
};

// A thread turns 8 codes of a row into 8 outputs, so that a warp's stores are
// contiguous.  The bound is the output's bytes; what hides the two dependent
// loads (the id, then the row) is kLookTokens rows in flight per thread
// (16384 rows of 4096 columns: 45 us with 32 codes of one row a thread).
template <int B, int MODE, typename TS, typename TO>
__global__ void __launch_bounds__(kLookThreads) lookup_kernel(const LookArgs p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int per_block = kLookThreads / p.lanes;  // rows of a block at a time
  const int c = blockIdx.y * p.lanes + threadIdx.x % p.lanes;
  const int step = gridDim.x * per_block;
  if (c >= p.pieces) return;
  const int per_group = p.lgs - 3, G = p.pieces >> per_group, g0 = c >> per_group;
  const float2 alpha = make_float2(p.alpha, p.alpha);
  for (int64_t t0 = blockIdx.x * per_block + threadIdx.x / p.lanes; t0 < p.n; t0 += kLookTokens * step) {
    int row[kLookTokens];
    uint32_t w[kLookTokens][3];
    float s[kLookTokens], b[kLookTokens];
    bool ok[kLookTokens];
#pragma unroll
    for (int u = 0; u < kLookTokens; ++u) row[u] = t0 + u * step < p.n ? __ldg(p.ids + t0 + u * step) : 0;
#pragma unroll
    for (int u = 0; u < kLookTokens; ++u) {
      ok[u] = (uint32_t)row[u] < (uint32_t)p.rows;
      if (ok[u] && t0 + u * step < p.n) {
        load8<B>(reinterpret_cast<const uint8_t*>(p.packed) + ((int64_t)row[u] * p.pieces + c) * B, w[u]);
        const int64_t g = (int64_t)row[u] * G + g0;
        if constexpr (MODE == QMM_MODE_AFFINE) {
          s[u] = to_f32(__ldg(reinterpret_cast<const TS*>(p.scales) + g));
          b[u] = to_f32(__ldg(reinterpret_cast<const TS*>(p.biases) + g));
        } else {
          s[u] = mx::Mode<MODE>::scale(__ldg(reinterpret_cast<const uint8_t*>(p.scales) + g));
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kLookTokens; ++u) {
      if (t0 + u * step >= p.n) break;
      __align__(16) TO v[8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float2 x;
        if constexpr (MODE == QMM_MODE_AFFINE)
          x = mul2(alpha, fma2f(codes2<B>(w[u], i), make_float2(s[u], s[u]), make_float2(b[u], b[u])));
        else
          x = mul2(alpha, mul2(make_float2(mx::Mode<MODE>::lane(stream_code<B>(w[u], i)),
                                           mx::Mode<MODE>::lane(stream_code<B>(w[u], i + 1))),
                               make_float2(s[u], s[u])));
        v[i] = from_f32<TO>(x.x);
        v[i + 1] = from_f32<TO>(x.y);
      }
      uint4 o[sizeof(TO) / 2];
      memcpy(o, v, sizeof(o));
      if (!ok[u]) {
#pragma unroll
        for (int h = 0; h < (int)sizeof(TO) / 2; ++h) o[h] = make_uint4(0u, 0u, 0u, 0u);
        if (c == 0) set_status(p.d_status, QMM_ERR_BAD_TOKEN_ID);
      }
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<TO*>(p.out) + ((t0 + u * step) * p.pieces + c) * 8);
#pragma unroll
      for (int h = 0; h < (int)sizeof(TO) / 2; ++h) dst[h] = o[h];
    }
  }
}

// ------------------------------------------------------------------ gradient
// The tokens are sorted by row (stable, so that a row's tokens keep their
// order and the sums do not depend on timing), and the sorted list is cut into
// chunks of P tokens.  A chunk sums each of its runs (tokens of one row) over a
// slab of columns in fp32, multiplies by the row's codes and folds the groups;
// runs inside a chunk are stored at once, those that cross its ends leave
// partial group sums that the join adds in list order.  Everything is read
// once: the bound is dy's bytes (and the output's, zeros included).
constexpr int kSortThreads = 512, kSortWarps = 16;  // of each sorting CTA
constexpr int kHeld = 4;            // list entries a lane keeps between a pass's two readings
constexpr int kDigitBits = 9, kDigits = 1 << kDigitBits;
constexpr int kSlabThreads = 128;   // most of a block of sums, 16 columns each

struct SortArgs {
  const int32_t* ids;
  int n;
  int rows;
  int passes, bits;      // digits of the keys and bits of a digit
  int ctas;              // that sort: one, or a cluster of 8
  uint32_t* keys[2];     // ping-pong; pass i writes buffer i & 1
  uint32_t* perm[2];
  int32_t* d_status;
  uint4* zero[2];        // outputs to clear
  int64_t zero_bytes;    // of each
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t read_rank(const uint32_t* p, uint32_t rank) {
  uint32_t a, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(a)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// The first CTA (short lists) or cluster sorts by least significant digits, each
// warp owning a contiguous piece of the list; the other CTAs clear the outputs
// meanwhile.  A pass is a chain of latencies (count, scan over warps, CTAs and
// digits, scatter), so it keeps few warps per digit column and its list entries
// in registers.
__global__ void __launch_bounds__(kSortThreads) sort_kernel(const __grid_constant__ SortArgs p) {
  __shared__ uint32_t hist[kSortWarps][kDigits];  // counts, then running positions
  __shared__ uint32_t total[kDigits], base[kDigits], wsum[kSortWarps];
  static_assert(kSortThreads == kDigits, "one thread a digit");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if ((int)blockIdx.x >= p.ctas) {
    const int64_t step = (int64_t)(gridDim.x - p.ctas) * kSortThreads;
    const int64_t first = (int64_t)(blockIdx.x - p.ctas) * kSortThreads + tid;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
#pragma unroll 4
      for (int64_t i = first; i < p.zero_bytes / 16; i += step) p.zero[o][i] = make_uint4(0u, 0u, 0u, 0u);
      uint16_t* tail = reinterpret_cast<uint16_t*>(p.zero[o]);
      for (int64_t i = p.zero_bytes / 16 * 8 + first; i < p.zero_bytes / 2; i += step) tail[i] = 0;
    }
    return;
  }
  const uint32_t rank = cluster_rank();
  const int w = (int)rank * kSortWarps + warp, nw = p.ctas * kSortWarps;
  const int lo = (int)((int64_t)p.n * w / nw), hi = (int)((int64_t)p.n * (w + 1) / nw);
  uint32_t* mine = hist[warp];
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const uint32_t mask = (1u << p.bits) - 1u;
    const bool odd = pass & 1, last = pass == p.passes - 1;
    const uint32_t* src_k = odd ? p.keys[0] : p.keys[1];
    const uint32_t* src_p = odd ? p.perm[0] : p.perm[1];
    uint32_t* dst_k = odd ? p.keys[1] : p.keys[0];
    uint32_t* dst_p = odd ? p.perm[1] : p.perm[0];
    auto key_at = [&](int i) -> uint32_t {
      if (pass) return src_k[i];
      const int32_t id = p.ids[i];
      return id >= 0 && id < p.rows ? (uint32_t)id : (uint32_t)p.rows;  // bad ids come last
    };
    // the first kHeld rounds' entries stay in registers for the scatter
    uint32_t hk[kHeld], hp[kHeld];
#pragma unroll
    for (int r = 0; r < kHeld; ++r) {
      const int i = lo + 32 * r + lane;
      hk[r] = i < hi ? key_at(i) : 0u;
      hp[r] = i < hi ? (pass ? src_p[i] : (uint32_t)i) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kSortWarps; ++j) hist[j][tid] = 0u;
    __syncthreads();
    auto count = [&](uint32_t k) {
      if (pass == 0 && k == (uint32_t)p.rows) set_status(p.d_status, QMM_ERR_BAD_TOKEN_ID);
      atomicAdd(mine + ((k >> shift) & mask), 1u);
    };
#pragma unroll
    for (int r = 0; r < kHeld; ++r)
      if (lo + 32 * r + lane < hi) count(hk[r]);
    for (int i = lo + 32 * kHeld + lane; i < hi; i += 32) count(key_at(i));
    __syncthreads();
    // counts of this CTA's warps -> exclusive prefixes
    uint32_t col[kSortWarps], run = 0u;
#pragma unroll
    for (int j = 0; j < kSortWarps; ++j) col[j] = hist[j][tid];
#pragma unroll
    for (int j = 0; j < kSortWarps; ++j) {
      hist[j][tid] = run;
      run += col[j];
    }
    uint32_t before = 0u, all = run;
    if (p.ctas > 1) {
      total[tid] = run;
      cluster_sync();
      uint32_t c[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) c[r] = read_rank(total + tid, r);
      all = 0u;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        before += r < (int)rank ? c[r] : 0u;
        all += c[r];
      }
    }
    uint32_t incl = all;  // scan over the digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    uint32_t off = 0u;
#pragma unroll
    for (int j = 0; j < kSortWarps; ++j) off += j < warp ? wsum[j] : 0u;
    base[tid] = off + incl - all + before;
    __syncthreads();
    auto scatter = [&](bool in, uint32_t k, uint32_t t) {
      const uint32_t act = __ballot_sync(0xffffffffu, in);
      if (in) {
        const uint32_t d = (k >> shift) & mask;
        const uint32_t peers = __match_any_sync(act, d);
        const int r = __popc(peers & ((1u << lane) - 1u));
        const uint32_t at = base[d] + mine[d] + (uint32_t)r;
        __syncwarp(act);
        if (r == 0) mine[d] += (uint32_t)__popc(peers);
        dst_k[at] = k;
        dst_p[at] = t;
      }
      __syncwarp();
    };
#pragma unroll
    for (int r = 0; r < kHeld; ++r) scatter(lo + 32 * r + lane < hi, hk[r], hp[r]);
    for (int i0 = lo + 32 * kHeld; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < hi;
      scatter(in, in ? key_at(i) : 0u, in ? (pass ? src_p[i] : (uint32_t)i) : 0u);
    }
    // the list is whole (and the totals have been read)
    if (p.ctas > 1)
      cluster_sync();
    else if (!last)
      __syncthreads();
  }
}

struct GradArgs {
  const void* dy;
  const uint32_t* keys;  // sorted rows and their tokens
  const uint32_t* perm;
  const uint32_t* packed;
  int n, rows, chunk, chunks;
  int cols, lgs;
  float alpha;
  void* out[2];  // dscales, dbiases
  int g_dtype;
  float* part;  // [chunk][first run | last run][scales | biases][groups]
};

// P list entries x up to 2048 columns a block; 16 columns a thread.
template <int B, typename TD>
__global__ void __launch_bounds__(kSlabThreads) grad_kernel(const GradArgs p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, chunk = blockIdx.x;
  const int e0 = chunk * p.chunk, cnt = min(p.chunk, p.n - e0);
  // one entry a lane, with the neighbours' keys
  const uint32_t key = lane < cnt ? p.keys[e0 + lane] : 0xffffffffu;
  const uint32_t tok = lane < cnt ? p.perm[e0 + lane] : 0u;
  const uint32_t prev = e0 > 0 ? p.keys[e0 - 1] : 0xffffffffu, next = e0 + cnt < p.n ? p.keys[e0 + cnt] : 0xffffffffu;
  const int col = (blockIdx.y * blockDim.x + threadIdx.x) * 16;
  const bool live = col < p.cols;  // (threads past the row read its start and store nothing)
  const uint8_t* dy = reinterpret_cast<const uint8_t*>(p.dy) + (live ? col : 0) * (int)sizeof(TD);
  const uint32_t dy_row = (uint32_t)p.cols * (uint32_t)sizeof(TD), code_row = (uint32_t)(p.cols >> 3) * B;
  const uint8_t* codes = reinterpret_cast<const uint8_t*>(p.packed) + (int64_t)(col >> 3) * B;
  const int G = p.cols >> p.lgs, g = col >> p.lgs;
  const int lpg = 1 << (p.lgs - 4);  // threads of a group
  // after the group's sum, its first thread holds the scale's, its second the bias's
  const bool odd = threadIdx.x & 1, stores = live && (threadIdx.x & (lpg - 1)) < 2;
  const uint32_t out_row = (uint32_t)G * (p.g_dtype == QMM_F32 ? 4u : 2u);
  uint8_t* const out =
      reinterpret_cast<uint8_t*>(odd ? p.out[1] : p.out[0]) + (int64_t)g * (p.g_dtype == QMM_F32 ? 4 : 2);
  constexpr int U = sizeof(TD) == 4 ? 2 : 4;  // rows requested at a time
  const uint32_t after = __shfl_down_sync(0xffffffffu, key, 1);
  // the entries after which a run or the chunk ends
  const uint32_t ends = __ballot_sync(0xffffffffu, lane < cnt && (lane + 1 == cnt || after != key));
  float2 acc[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) acc[c] = make_float2(0.0f, 0.0f);
  int start = 0;
  for (int i0 = 0; i0 < cnt; i0 += U) {
    // U rows of dy, and the codes of the rows whose runs end among them
    uint4 raw[U][sizeof(TD)];
    uint32_t code[U][2][3];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      // (lanes past the chunk hold token 0: a valid row, and what a bad id's
      // tokens add is dropped with their run)
      const uint32_t t = __shfl_sync(0xffffffffu, tok, (i0 + j) & 31);
      const uint4* src = reinterpret_cast<const uint4*>(dy + (uint64_t)t * dy_row);
#pragma unroll
      for (int h = 0; h < (int)sizeof(TD); ++h) raw[j][h] = __ldcs(src + h);
      if (ends >> ((i0 + j) & 31) & 1u) {
        const uint32_t k = __shfl_sync(0xffffffffu, key, (i0 + j) & 31);
        if (live && k < (uint32_t)p.rows) {
          load8<B>(codes + (uint64_t)k * code_row, code[j][0]);
          load8<B>(codes + (uint64_t)k * code_row + B, code[j][1]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = i0 + j;
      if (i >= cnt) break;
      __align__(16) TD v[16];
      memcpy(v, raw[j], sizeof(v));
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] = add2(acc[c], make_float2(to_f32(v[2 * c]), to_f32(v[2 * c + 1])));
      if (!(ends >> i & 1u)) continue;  // the run goes on
      const uint32_t k = __shfl_sync(0xffffffffu, key, i);
      if (k < (uint32_t)p.rows) {
        float2 s2 = make_float2(0.0f, 0.0f), b2 = s2;
        if (live) {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            s2 = fma2f(acc[c], codes2<B>(code[j][c >> 2], 2 * (c & 3)), s2);
            b2 = add2(b2, acc[c]);
          }
        }
        const float ds = s2.x + s2.y, db = b2.x + b2.y;
        float v = (odd ? db : ds) + __shfl_xor_sync(0xffffffffu, odd ? ds : db, 1);
        if (lpg > 2) v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (lpg > 4) v += __shfl_xor_sync(0xffffffffu, v, 4);
        if (stores) {
          if ((start == 0 && prev == k) || (i + 1 == cnt && next == k))  // a piece of a longer run
            p.part[(((int64_t)chunk * 2 + (start == 0 ? 0 : 1)) * 2 + odd) * G + g] = v;
          else
            store_as(out + (uint64_t)k * out_row, p.g_dtype, 0, p.alpha * v);
        }
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) acc[c] = make_float2(0.0f, 0.0f);
      start = i + 1;
    }
  }
}

// The chunk where a run that crosses chunks begins adds its pieces in order.
__global__ void __launch_bounds__(128) join_kernel(const GradArgs p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int chunk = blockIdx.x, e0 = chunk * p.chunk, last = e0 + p.chunk - 1;
  if (last + 1 >= p.n) return;
  const uint32_t k = p.keys[last], first = p.keys[e0], prev = e0 > 0 ? p.keys[e0 - 1] : 0xffffffffu;
  // further chunks that begin with the run, 32 looked at together
  auto same_at = [&](int from) {
    const int64_t at = (int64_t)(from + (int)(threadIdx.x & 31)) * p.chunk;
    return __ballot_sync(0xffffffffu, at < p.n && p.keys[at < p.n ? at : 0] == k);
  };
  uint32_t same = same_at(chunk + 1);
  if (k >= (uint32_t)p.rows || !(same & 1u)) return;  // no run goes on
  const bool whole = first == k;                      // it fills this chunk
  if (whole && prev == k) return;                     // it began earlier
  const int64_t G = p.cols >> p.lgs;
  int pieces = 0;
  while (same == 0xffffffffu) {
    pieces += 32;
    same = same_at(chunk + 1 + pieces);
  }
  pieces += __ffs(~same) - 1;
  for (int64_t g = threadIdx.x; g < 2 * G; g += blockDim.x) {
    float sum = p.part[((int64_t)chunk * 2 + (whole ? 0 : 1)) * 2 * G + g];
#pragma unroll 16
    for (int c = 1; c <= pieces; ++c) sum += p.part[(int64_t)(chunk + c) * 4 * G + g];
    store_as(p.out[g >= G], p.g_dtype, (int64_t)k * G + (g >= G ? g - G : g), p.alpha * sum);
  }
}

// Short lists in one launch, without a sort: a warp takes one token and 256
// columns, finds the list's entries of the same row by votes, leaves the work to
// the row's first entry and sums the entries in order; then it folds the
// groups as grad_kernel does.  Every block also clears the untouched rows of its
// share of the outputs.  A row with many entries is summed by one warp per 256
// columns, 8 rows in flight, which is what bounds the list's length.
constexpr int kShort = 512;
constexpr int kShortThreads = 256, kShortBlocks = 4;  // per SM: one wave

struct ShortArgs {
  const void* dy;
  const int32_t* ids;
  const uint32_t* packed;
  int n, rows, cols, lgs;
  float alpha;
  void* out[2];
  int g_dtype;
  int32_t* d_status;
};

template <int B, typename TD>
__global__ void __launch_bounds__(kShortThreads, kShortBlocks) short_kernel(const ShortArgs p) {
  __shared__ int32_t ids[kShort];
  __shared__ uint32_t touched[1024];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.cols >> p.lgs, esize = p.g_dtype == QMM_F32 ? 4 : 2;
  // this block's rows to clear, 32768 of them at a time
  const int r_lo = (int)((int64_t)p.rows * blockIdx.x / gridDim.x);
  const int r_hi = (int)((int64_t)p.rows * (blockIdx.x + 1) / gridDim.x);
  for (int i = tid; i < p.n; i += kShortThreads) {
    ids[i] = p.ids[i];
    if (blockIdx.x == 0 && (uint32_t)ids[i] >= (uint32_t)p.rows) set_status(p.d_status, QMM_ERR_BAD_TOKEN_ID);
  }
  for (int r0 = r_lo; r0 < r_hi; r0 += 32768) {
    const int nr = min(32768, r_hi - r0);
    for (int i = tid; i < (nr + 31) / 32; i += kShortThreads) touched[i] = 0u;
    __syncthreads();
    for (int i = tid; i < p.n; i += kShortThreads) {
      const int64_t r = (int64_t)ids[i] - r0;
      if (r >= 0 && r < nr) atomicOr(touched + (r >> 5), 1u << (r & 31));
    }
    __syncthreads();
    const int row_bytes = G * esize;
    const int unit = row_bytes % 16 == 0 ? 16 : esize;
    const uint32_t per_row = (uint32_t)(row_bytes / unit);
    const int64_t items = (int64_t)nr * per_row;
    for (int64_t i = tid; i < items; i += kShortThreads) {
      const int r = (int)(items <= UINT32_MAX ? (uint32_t)i / per_row : i / per_row);
      if (touched[r >> 5] >> (r & 31) & 1u) continue;
      const int64_t at = (int64_t)r0 * row_bytes + i * unit;
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        uint8_t* dst = reinterpret_cast<uint8_t*>(p.out[o]) + at;
        if (unit == 16)
          *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
        else if (unit == 4)
          *reinterpret_cast<uint32_t*>(dst) = 0u;
        else
          *reinterpret_cast<uint16_t*>(dst) = 0;
      }
    }
    __syncthreads();
  }
  __syncthreads();  // (a block without rows to clear)
  const int slabs = (p.cols + 255) / 256, lpg = 1 << (p.lgs - 3);
  const int64_t tasks = (int64_t)p.n * slabs;
  constexpr int U = sizeof(TD) == 4 ? 4 : 8;
  for (int64_t task = (int64_t)warp * gridDim.x + blockIdx.x; task < tasks;
       task += (int64_t)gridDim.x * (kShortThreads / 32)) {
    const int t0 = (int)(task / slabs), slab = (int)(task - (int64_t)t0 * slabs);
    const int row = ids[t0];
    if ((uint32_t)row >= (uint32_t)p.rows) continue;
    // the list as 32-entry masks: lane w keeps that of entries 32 w ..
    uint32_t mask = 0u;
    for (int w = 0; w * 32 < p.n; ++w) {
      const uint32_t m = __ballot_sync(0xffffffffu, w * 32 + lane < p.n && ids[w * 32 + lane] == row);
      if (lane == w) mask = m;
    }
    const uint32_t before = __ballot_sync(0xffffffffu, lane < (t0 >> 5) && mask != 0u);
    const uint32_t here = __shfl_sync(0xffffffffu, mask, t0 >> 5);
    if (before != 0u || (here & ((1u << (t0 & 31)) - 1u)) != 0u) continue;  // not its first entry
    const int col = slab * 256 + lane * 8;
    const bool live = col < p.cols;
    const uint8_t* dy = reinterpret_cast<const uint8_t*>(p.dy) + (int64_t)(live ? col : 0) * (int)sizeof(TD);
    const int64_t dy_row = (int64_t)p.cols * (int)sizeof(TD);
    uint32_t code[3] = {0u, 0u, 0u};
    const int64_t piece = (int64_t)row * (p.cols >> 3) + (col >> 3);
    if (live) load8<B>(reinterpret_cast<const uint8_t*>(p.packed) + piece * B, code);
    float2 acc[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = make_float2(0.0f, 0.0f);
    int w = t0 >> 5;
    uint32_t m = here;
    bool more = true;
    while (more) {
      uint4 raw[U][sizeof(TD) / 2];
      int got = 0;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        while (m == 0u && (w + 1) * 32 < p.n) {
          ++w;
          m = __shfl_sync(0xffffffffu, mask, w);
        }
        if (m != 0u) {
          const uint4* src = reinterpret_cast<const uint4*>(dy + (int64_t)(w * 32 + __ffs(m) - 1) * dy_row);
          m &= m - 1u;
#pragma unroll
          for (int h = 0; h < (int)sizeof(TD) / 2; ++h) raw[j][h] = __ldcs(src + h);
          got = j + 1;
        }
      }
      more = got == U;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (j >= got) break;
        __align__(16) TD v[8];
        memcpy(v, raw[j], sizeof(v));
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = add2(acc[c], make_float2(to_f32(v[2 * c]), to_f32(v[2 * c + 1])));
      }
    }
    float2 s2 = make_float2(0.0f, 0.0f), b2 = s2;
    if (live) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s2 = fma2f(acc[c], codes2<B>(code, 2 * c), s2);
        b2 = add2(b2, acc[c]);
      }
    }
    const bool odd = lane & 1;
    const float ds = s2.x + s2.y, db = b2.x + b2.y;
    float v = (odd ? db : ds) + __shfl_xor_sync(0xffffffffu, odd ? ds : db, 1);
    v += __shfl_xor_sync(0xffffffffu, v, 2);
    if (lpg > 4) v += __shfl_xor_sync(0xffffffffu, v, 4);
    if (lpg > 8) v += __shfl_xor_sync(0xffffffffu, v, 8);
    if (live && (lane & (lpg - 1)) < 2)
      store_as(odd ? p.out[1] : p.out[0], p.g_dtype, (int64_t)row * G + (col >> p.lgs), p.alpha * v);
  }
}

// Threads of a block of sums: whole warps over the columns, up to kSlabThreads.
static int slab_threads(int64_t cols) { return (int)std::min<int64_t>(kSlabThreads, (cols + 511) / 512 * 32); }

// Tokens of a chunk: up to 32 (one a lane), fewer while that leaves SMs idle.  (148
// whatever the device: the workspace's size and the order of the sums follow it.)
static int chunk_of(int64_t n, int64_t cols) {
  const int64_t slabs = (cols + 16 * slab_threads(cols) - 1) / (16 * slab_threads(cols));
  int c = 32;
  while (c > 4 && (n + c - 1) / c * slabs < 4 * 148) c /= 2;
  return c;
}

static int64_t grad_workspace(int64_t n, int64_t cols) {
  if (n <= kShort) return 0;
  const int64_t chunks = (n + chunk_of(n, cols) - 1) / chunk_of(n, cols);
  // two lists of keys and tokens, and the pieces of two runs a chunk (groups of 32 at most)
  return 16 + (n + 3) / 4 * 16 * 4 + chunks * 4 * ((cols + 31) / 32) * 4;
}

template <int B, int MODE, typename TS>
static cudaError_t lookup_o(const int32_t* ids, int64_t n, const qmm_qweight* w, float alpha, void* out, int out_dtype,
                            int32_t* d_status, cudaStream_t st) {
  const int rows = (int)std::min<int64_t>(w->rows, INT32_MAX);  // ids are 32-bit
  LookArgs a{ids, w->packed, w->scales, w->biases, rows, (int)n, (int)(w->cols / 8), 4, kLookThreads, alpha, out, d_status};
  while ((1 << a.lgs) < w->group_size) ++a.lgs;  // 16 (nvfp4), 32, 64 or 128
  while (a.lanes / 2 >= a.pieces) a.lanes /= 2;
  const int per_block = kLookThreads / a.lanes;
  const int64_t tiles = ((int64_t)a.pieces + a.lanes - 1) / a.lanes;
  // one row a thread while SMs are idle, then up to kLookTokens
  const int64_t want = (n + per_block - 1) / per_block;
  const int64_t most = std::max<int64_t>(1, (int64_t)qmm_host::num_sms() * 16 / tiles);
  const dim3 grid((unsigned)std::min(want, most), (unsigned)tiles);
  constexpr int kThreads = kLookThreads;
  if (out_dtype == QMM_F32) return launch_next(lookup_kernel<B, MODE, TS, float>, grid, kThreads, 1, a, st);
  if (out_dtype == QMM_BF16) return launch_next(lookup_kernel<B, MODE, TS, __nv_bfloat16>, grid, kThreads, 1, a, st);
  return launch_next(lookup_kernel<B, MODE, TS, __half>, grid, kThreads, 1, a, st);
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
                               void* dscales, void* dbiases, int g_dtype, void* workspace, int32_t* d_status,
                               cudaStream_t st) {
  if (n <= kShort) {
    const int lgs = w->group_size == 32 ? 5 : w->group_size == 64 ? 6 : 7;
    const ShortArgs a{dy, ids, w->packed, (int)n, (int)w->rows, (int)w->cols, lgs, alpha, {dscales, dbiases}, g_dtype,
                      d_status};
    const dim3 grid(qmm_host::num_sms() * kShortBlocks);
    switch (w->bits) {
      case 2: return launch_next(short_kernel<2, TD>, grid, kShortThreads, 1, a, st);
      case 3: return launch_next(short_kernel<3, TD>, grid, kShortThreads, 1, a, st);
      case 4: return launch_next(short_kernel<4, TD>, grid, kShortThreads, 1, a, st);
      case 6: return launch_next(short_kernel<6, TD>, grid, kShortThreads, 1, a, st);
      default: return launch_next(short_kernel<8, TD>, grid, kShortThreads, 1, a, st);
    }
  }
  const int64_t G = w->cols / w->group_size, n4 = (n + 3) / 4 * 4;
  uint32_t* ws = static_cast<uint32_t*>(workspace);
  SortArgs sa{};
  sa.ids = ids;
  sa.n = (int)n;
  sa.rows = (int)w->rows;
  int bits = 1;
  while (bits < 32 && (w->rows >> bits) != 0) ++bits;  // keys up to rows
  sa.passes = (bits + kDigitBits - 1) / kDigitBits;
  sa.bits = (bits + sa.passes - 1) / sa.passes;
  for (int i = 0; i < 2; ++i) {
    sa.keys[i] = ws + (2 * i) * n4;
    sa.perm[i] = ws + (2 * i + 1) * n4;
    sa.zero[i] = static_cast<uint4*>(i ? dbiases : dscales);
  }
  sa.d_status = d_status;
  sa.zero_bytes = w->rows * G * qmm_host::dtype_size((qmm_dtype)g_dtype);
  // A cluster's barriers against a short list's rounds, us of the whole gradient with one
  // CTA and with eight: rows of 4096 columns, 1024 tokens 14.4 and 17.3, 2048 20.7 and
  // 20.5, 4096 34 and 28; rows of 1024 columns cross at 1000 (2048 tokens 16.6 and 13.6).
  sa.ctas = n <= 2048 ? 1 : 8;
  const int ctas = qmm_host::num_sms() * 2 / sa.ctas * sa.ctas;
  cudaError_t e = launch_next(sort_kernel, dim3(ctas), kSortThreads, sa.ctas, sa, st);
  if (e != cudaSuccess) return e;
  GradArgs ga{};
  ga.dy = dy;
  ga.keys = sa.keys[(sa.passes - 1) & 1];
  ga.perm = sa.perm[(sa.passes - 1) & 1];
  ga.packed = w->packed;
  ga.n = (int)n;
  ga.rows = (int)w->rows;
  ga.chunk = chunk_of(n, w->cols);
  ga.chunks = (int)((n + ga.chunk - 1) / ga.chunk);
  ga.cols = (int)w->cols;
  ga.lgs = w->group_size == 32 ? 5 : w->group_size == 64 ? 6 : 7;
  ga.alpha = alpha;
  ga.out[0] = dscales;
  ga.out[1] = dbiases;
  ga.g_dtype = g_dtype;
  ga.part = reinterpret_cast<float*>(ws + 4 * n4);
  const int threads = slab_threads(w->cols);
  const dim3 grid(ga.chunks, (unsigned)((w->cols + 16 * threads - 1) / (16 * threads)));
  switch (w->bits) {
    case 2: e = launch_next(grad_kernel<2, TD>, grid, threads, 1, ga, st); break;
    case 3: e = launch_next(grad_kernel<3, TD>, grid, threads, 1, ga, st); break;
    case 4: e = launch_next(grad_kernel<4, TD>, grid, threads, 1, ga, st); break;
    case 6: e = launch_next(grad_kernel<6, TD>, grid, threads, 1, ga, st); break;
    default: e = launch_next(grad_kernel<8, TD>, grid, threads, 1, ga, st); break;
  }
  if (e != cudaSuccess || ga.chunks == 1) return e;
  return launch_next(join_kernel, dim3(ga.chunks - 1), 128, 1, ga, st);
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
  if (w->cols > (1 << 25)) return QMM_ERR_UNSUPPORTED;
  if (d_status && !aligned4(d_status)) return QMM_ERR_ALIGNMENT;
  if (n == 0) return QMM_OK;
  if (!aligned4(ids) || !aligned16(out)) return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  return launch_status(qmm::embed::launch_lookup(ids, n, w, alpha, out, out_dtype, d_status, (cudaStream_t)stream));
}

int64_t qmm_embedding_backward_workspace_bytes(int64_t n, int64_t rows, int64_t cols) {
  // (rows and list entries past the last one of a block's share are counted in 32 bits)
  if (n < 0 || n > (1 << 30) || rows < 0 || rows > (1 << 30) || cols <= 0 || cols > (1 << 25)) return -1;
  return qmm::embed::grad_workspace(n, cols);
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
      (need > 0 && !aligned16(workspace)))
    return QMM_ERR_ALIGNMENT;
  s = qmm_device_check();
  if (s != QMM_OK) return s;
  cudaStream_t st = (cudaStream_t)stream;
  if (dy_dtype == QMM_F32)
    return launch_status(qmm::embed::launch_grad<float>(dy, ids, n, w, alpha, dscales, dbiases, g_dtype, workspace,
                                                        d_status, st));
  if (dy_dtype == QMM_BF16)
    return launch_status(
        qmm::embed::launch_grad<__nv_bfloat16>(dy, ids, n, w, alpha, dscales, dbiases, g_dtype, workspace,
                                                        d_status, st));
  return launch_status(qmm::embed::launch_grad<__half>(dy, ids, n, w, alpha, dscales, dbiases, g_dtype, workspace,
                                                        d_status, st));
}

}  // extern "C"
