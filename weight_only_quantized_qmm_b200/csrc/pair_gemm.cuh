// Tensor-core products of packed weights for many tokens (tcgen05, sm_100a):
//   FWD  g | u [m, n] = sum_k x[m, k] w_hat[n, k] of gate and up, then
//        h = SiLU(g) * u                               (A = x, B = w_hat)
//   DX   dx[m, k] = sum over n (and parts) of dy[m, n] w_hat[n, k]
//                                                      (A = dy, B = w_hat^T)
//   DP   dW[n, k] = sum_m dy[m, n] x[m, k], folded at once into
//        dscales[n, j] = sum_{k in j} dW q, dbiases[n, j] = sum_{k in j} dW
//                                                      (A = dy^T, B = x^T)
//
// Tokens (DP: weight rows) are the M side of the MMA, so that an accumulator
// lane is one output row and its columns are contiguous in memory: 16-byte
// stores, and a group's sum of DP stays in one thread.  256 accumulator
// columns: FWD holds 128 columns of g and the same 128 of u, so SiLU(g) * u is
// local to a thread.
//
// PAIR: two CTAs share one 256 x 256 tile (cta_group::2); each holds 128 rows
// of A and half of B, so an SM reads and writes 64 KB of shared memory per
// 64-deep step (512 tensor cycles) instead of the 96 KB of a 128 x 256 tile,
// which is what bounds that tile.  Single (FWD): one CTA per 128 x 256 tile for
// few tokens.  Where the tiles are few, a cluster of `splits` CTAs (or pairs) shares
// one by cutting the sum, and joins its partial tiles through distributed shared
// memory in rank order.
//
// FWD and DX take weights dequantized beforehand (B = 0: many tokens, where the
// extra pass is small beside the product and the two TMA-fed operands run at
// the tensor cores' rate), or dequantize in the kernel: the packed codes of each
// step arrive in a ring of their own (TMA boxes, swizzled at their width), the
// scales and biases too where their rows start on 16 bytes; sixteen warps turn 64
// codes of one row per thread into (OFF + q) - OFF and one fused q * s + z in the
// activations' type (one rounding), and write the swizzled operand tile:
// K-major for FWD, MN-major for DX (the same packed rows, read along their length
// both times).
//
// Warps: 0 TMA producer of the activations; 1 TMEM owner and MMA issuer (PAIR:
// of the leader CTA); 2.. epilogue (4 warps; DP two sets of 8, one for
// each accumulator); then the producer of the
// codes and the 16 dequant warps.
// Every wait is bounded; after one that gave up both CTAs of a pair write their
// tiles as NaN (after one of an epilogue, that CTA its rows).
#pragma once

#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "f32x2.cuh"
#include "mbarrier.cuh"

namespace qmm {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn tensor_map_encoder();

namespace pg {

enum Op { FWD = 0, DX = 1, DP = 2 };

constexpr int kBK = 64;                  // depth of a step: 128 bytes of 16-bit values
constexpr int kTile = 128 * kBK * 2;     // 128 x 64 operand tile: 16 KB
constexpr int kDeqWarps = 16;

// The widths of FWD and DX, with B = 0 for weights dequantized beforehand.
template <int OP, int B, bool PAIR>
struct Cfg {
  static constexpr bool DENSE = OP == DP || B == 0;                // both operands come by TMA
  static constexpr int EPI = OP == DP ? 16 : 4;                    // epilogue warps
  static constexpr int DEQ = DENSE ? 0 : kDeqWarps;
  static constexpr int THREADS = (2 + EPI + (DENSE ? 0 : 1) + DEQ) * 32;
  static constexpr int A_BYTES = kTile;                            // 128 rows of A per CTA
  static constexpr int B_BYTES = PAIR ? kTile : 2 * kTile;         // 128 or 256 of B
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int STAGES = DENSE ? 6 : PAIR ? 5 : 3;
  // the ring of packed codes, one slot a step.  A box: FWD, 128 rows of 64
  // codes (3-bit: of 128, whose 48 bytes TMA can copy; each step reads its
  // half); DX, 64 rows of 128 codes.  Single CTAs have two boxes.
  static constexpr int ROW = OP == FWD ? (B == 3 ? 48 : 8 * B) : 16 * B;
  static constexpr int BOX_ROWS = OP == FWD ? 128 : 64;
  static constexpr int BOX = BOX_ROWS * ROW;
  static constexpr int BOXES = PAIR ? 1 : 2;
  // swizzle: 16-byte piece c of row r sits at c ^ swz(r)
  static constexpr int SWZ = ROW == 32 || ROW == 64 || ROW == 128 ? ROW : 0;
  // scales and biases, 8 groups (16 bytes) of each row: DX, those of the step's 64
  // rows, in the slot of its codes; FWD, windows of 8 groups in a ring of two
  static constexpr int SB = BOX_ROWS * 16;                         // one array, one box
  static constexpr int SLOT = DENSE ? 1024 : (BOXES * BOX + (OP == DX ? 2 * SB : 0) + 1023) / 1024 * 1024;
  static constexpr int WINDOW = OP == FWD ? 2 * BOXES * SB : 0;
  static constexpr int OUT0 = STAGES * STAGE;                      // 4 KB a warp to turn rows for storing
  static constexpr int CODE0 = OUT0 + (OP == DP ? 0 : EPI * 4096);
  static constexpr int AVAIL = 227 * 1024 - 2048 - CODE0 - 2 * WINDOW;
  static constexpr int SLOTS = DENSE ? 0 : AVAIL / SLOT < 8 ? AVAIL / SLOT : 8;
  static constexpr int WIN0 = CODE0 + SLOTS * SLOT;
  static constexpr int BAR0 = WIN0 + (DENSE ? 0 : 2 * WINDOW);
  static constexpr int BARS = 2 * STAGES + 5 + 2 * SLOTS + 2;
  static constexpr int SMEM = 1024 + BAR0 + 512;                   // + alignment slack, barriers
  static_assert((!DENSE && OP == FWD) || PAIR, "these run on CTA pairs");
  static_assert(DENSE || SLOTS >= 3, "room for the codes");
  static_assert(8 * BARS + 8 <= 512, "barriers, TMEM slot and abort flag");
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static_assert(128 * 256 * 4 <= OUT0, "a partial tile fits the stages");
  __device__ static constexpr int swz(int r) {
    return SWZ == 32 ? (r >> 2) & 1 : SWZ == 64 ? (r >> 1) & 3 : SWZ == 128 ? r & 7 : 0;
  }
};

struct Weight {
  const uint32_t* packed;
  const void* scales;
  const void* biases;
};

struct Args {
  int M, K, N;            // tokens, weight columns, weight rows (of one part)
  int parts;              // FWD: 2; DX, DP: 1 or 2
  Weight w[2];
  int lgs;                // log2 of the group size
  int m_tiles, n_tiles;   // tiles along the output's rows and columns (DP: rows of one part)
  int steps;              // 64-deep steps of the whole sum
  int splits;             // CTAs (PAIR: pairs) that share a tile by cutting the sum; 1: persistent
  void* out[4];           // FWD: h, g, u; DX: dx; DP: dscales, dbiases of both parts
  int out_dtype;          // FWD: of h; DP
  int f16;                // operands are f16 (otherwise bf16)
  int sb_tma;             // scales and biases come by TMA (rows of a multiple of 8 groups)
};

struct Maps {
  CUtensorMap a[2];  // FWD: x; DX, DP: dy of each part
  CUtensorMap b[2];  // packed codes or dequantized weights of each part; DP: x
  CUtensorMap s[2], z[2];
};

// ------------------------------------------------------------------ PTX
__device__ __forceinline__ uint32_t su32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Arrives on a barrier of the pair's leader.  What it announces is shared
// memory of its own SM already made visible to the tensor cores by a proxy
// fence, or TMEM reads already waited for, so it releases at CTA scope: a
// cluster-scope release waits for every load in flight (measured at 1024 tokens
// of 4096 x 14336: 347 us instead of 225).
__device__ __forceinline__ void arrive_remote(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// Bounded waits of this kernel: polls that may sleep up to kNap ns each (a
// waiting warp that polls without a nap takes issue slots from the dequant
// warps), giving up after kPolls of them (measured: 0.35 to 0.7 s) or when another
// role has raised the abort flag.
constexpr uint32_t kNap = 20000, kPolls = 1u << 17;
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity), "r"(kNap)
      : "memory");
  return done != 0;
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const int* abort_flag) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (poll(bar, parity)) return true;
    if (*reinterpret_cast<const volatile int*>(abort_flag)) return false;
  }
  return false;
}
// the same, acquiring what the other CTA of the pair released
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, const int* abort_flag) {
  for (uint32_t i = 0; i < kPolls; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kNap)
        : "memory");
    if (done) return true;
    if (*reinterpret_cast<const volatile int*>(abort_flag)) return false;
  }
  return false;
}
// Waits that last as long as whole sums (the epilogue's for a tile, in turn with
// another's; the second CTA's for the last commit) get that bound for every 32768
// steps of them, which take about 13 ms: 134 million tokens of a parameter gradient
// are one tile of 0.7 s.
__device__ __forceinline__ bool wait_steps(uint32_t bar, uint32_t parity, const int* abort_flag, int64_t steps) {
  for (int64_t i = 0; i <= steps >> 15; ++i) {
    if (wait(bar, parity, abort_flag)) return true;
    if (*reinterpret_cast<const volatile int*>(abort_flag)) return false;
  }
  return false;
}
// Raises the abort flag, PAIR: of both CTAs.  The operands that one of them fails
// to deliver enter the accumulators of both, and after a failure of the issuer the
// other CTA's epilogue is signalled too: each must know before it reads its half.
template <bool PAIR>
static __device__ __noinline__ void give_up(int* abort_flag) {
  *reinterpret_cast<volatile int*>(abort_flag) = 1;
  if constexpr (PAIR) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_rank(su32(abort_flag), cta_rank() ^ 1u)), "r"(1u)
                 : "memory");
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
  }
}
// One poll is the usual case; the full bounded wait stands aside, and one that
// gives up raises the abort flag.
template <bool PAIR>
static __device__ __noinline__ void wait_slow(uint32_t bar, uint32_t parity, int* abort_flag) {
  if (!wait(bar, parity, abort_flag)) give_up<PAIR>(abort_flag);
}
template <bool PAIR>
__device__ __forceinline__ void wait_fast(uint32_t bar, uint32_t parity, int* abort_flag) {
  if (!poll(bar, parity)) wait_slow<PAIR>(bar, parity, abort_flag);
}
template <bool PAIR>
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, int c0, int c1, uint32_t bar) {
  if constexpr (PAIR)  // the barrier may be the leader CTA's
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(dst),
        "l"(m), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(m), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}
// Shared-memory descriptors of 128-byte swizzled 16-bit operands.
//   K-major: rows of 64 k, 8-row groups 1024 bytes apart;
//   MN-major: blocks of [64 k][64 rows], 8 k 1024 bytes apart (stride byte
//   offset), blocks of 64 rows 8192 bytes apart (leading byte offset).
template <bool MN>
__device__ __forceinline__ uint64_t desc(uint32_t saddr) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(MN ? 8192u >> 4 : 1u) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;  // descriptor version (sm_100)
  d |= (uint64_t)2u << 61;  // 128-byte swizzle
  return d;
}
template <bool PAIR>
__device__ __forceinline__ void mma(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
}
// arrives on `bar` (PAIR: of both CTAs) once the MMAs issued so far are done
template <bool PAIR>
__device__ __forceinline__ void commit(uint32_t bar, uint32_t lead) {
  if constexpr (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)(3u << lead))
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 16 columns of this warp's 32 lanes; tmem_wait() before the registers are read
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void sts_v4(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float4 lds_cluster(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

// ------------------------------------------------------------------ dequantize
template <typename T>
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  if constexpr (std::is_same<T, __half>::value)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  else
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)bits16(from_f32<T>(a)) | ((uint32_t)bits16(from_f32<T>(b)) << 16);
}

// Values 8c .. 8c + 7 of 32 codes as four pairs of T.
template <int B, typename T>
__device__ __forceinline__ uint4 dequant8(const uint32_t (&w)[B], uint16_t scale, uint16_t bias, int c) {
  constexpr bool H = std::is_same<T, __half>::value;
  uint32_t v[4];
  if constexpr (B == 8 && !H) {
    // 8-bit codes do not fit under a bf16 magic: exact in fp32, one rounding
    const float s = __uint_as_float((uint32_t)scale << 16), z = __uint_as_float((uint32_t)bias << 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t v4 = w[2 * c + (e >> 1)];
      const float q0 = __uint_as_float(__byte_perm(v4, 0x4B000000u, (e & 1) ? 0x7442 : 0x7440)) - 8388608.0f;
      const float q1 = __uint_as_float(__byte_perm(v4, 0x4B000000u, (e & 1) ? 0x7443 : 0x7441)) - 8388608.0f;
      v[e] = pack2<T>(fmaf(q0, s, z), fmaf(q1, s, z));
    }
  } else {
    // (OFF + q) in T with the code in the low mantissa bits; minus OFF is exact
    constexpr uint32_t OFF2 = H ? 0x64006400u : 0x43004300u;
    const uint32_t s2 = (uint32_t)scale * 0x00010001u, z2 = (uint32_t)bias * 0x00010001u;
    uint32_t p[4];
    if constexpr (B == 8) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t v4 = w[2 * c + (e >> 1)];
        p[e] = __byte_perm(v4, 0x64646464u, (e & 1) ? 0x4342 : 0x4140);
      }
    } else if constexpr (B == 4) {
      const uint32_t t0 = w[c] & 0x0F0F0F0Fu, t1 = (w[c] >> 4) & 0x0F0F0F0Fu;
      const uint32_t a = __byte_perm(t0, t1, 0x5140), b = __byte_perm(t0, t1, 0x7362);
      constexpr uint32_t M8 = H ? 0x64646464u : 0x43434343u;
      p[0] = __byte_perm(a, M8, 0x4140);
      p[1] = __byte_perm(a, M8, 0x4342);
      p[2] = __byte_perm(b, M8, 0x4140);
      p[3] = __byte_perm(b, M8, 0x4342);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        p[e] = stream_code<B>(w, 8 * c + 2 * e) | (stream_code<B>(w, 8 * c + 2 * e + 1) << 16) | OFF2;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fma2<T>(sub2<T>(p[e], OFF2), s2, z2);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// 32 codes of a row in global memory
template <int B>
__device__ __forceinline__ void load_words(const uint32_t* src, uint32_t (&w)[B]) {
  if constexpr (B % 4 == 0) {
#pragma unroll
    for (int i = 0; i < B; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(src + i));
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  } else if constexpr (B % 2 == 0) {
#pragma unroll
    for (int i = 0; i < B; i += 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(src + i));
      w[i] = v.x; w[i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < B; ++i) w[i] = __ldg(src + i);
  }
}
__device__ __forceinline__ uint4 lds_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint16_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
// 64 codes (8 B bytes) from byte `off` of the row at `row`, whose 16-byte pieces
// are swizzled by `swz`
template <int B>
__device__ __forceinline__ void read_codes(uint32_t row, int off, int swz, uint32_t (&w)[2][B]) {
  uint32_t* d = &w[0][0];
  if constexpr (B == 3) {  // 24 bytes, 8-byte aligned, never swizzled
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint2 v = lds_v2(row + off + 8 * i);
      d[2 * i] = v.x;
      d[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < B / 2; ++i) {
      const uint4 v = lds_v4(row + ((((off >> 4) + i) ^ swz) << 4));
      d[4 * i] = v.x; d[4 * i + 1] = v.y; d[4 * i + 2] = v.z; d[4 * i + 3] = v.w;
    }
  }
}

struct Tile {
  int m0, n0, part;  // first output row and column of the cluster's tile; DP: the part it belongs to
};
template <int OP, bool PAIR>
__device__ __forceinline__ Tile tile_of(const Args& p, int t) {
  constexpr int TM = PAIR ? 256 : 128;
  constexpr int TN = OP == FWD ? 128 : 256;
  // tiles along M vary fastest: the clusters running at one time share weight tiles
  const int nt = t / p.m_tiles, mt = t - nt * p.m_tiles;
  if constexpr (OP == DP) {
    const int part = nt / p.n_tiles;
    return Tile{mt * TM, (nt - part * p.n_tiles) * TN, part};
  } else {
    return Tile{mt * TM, nt * TN, 0};
  }
}

// out[0 .. 7] of one row (16-byte aligned when vec), the first `cnt` of them
template <typename T>
__device__ __forceinline__ void store8(T* dst, const float* v, bool vec, int cnt) {
  if (vec && cnt >= 8) {
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(dst) =
          make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) dst[i] = from_f32<T>(v[i]);
  }
}

// N values (2 or 4) at a multiple of N, in one store
template <int N>
__device__ __forceinline__ void store_run(void* base, int dtype, int64_t at, const float* v) {
  if (dtype == QMM_F32) {
    if constexpr (N == 4)
      *reinterpret_cast<float4*>(static_cast<float*>(base) + at) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<float2*>(static_cast<float*>(base) + at) = make_float2(v[0], v[1]);
    return;
  }
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    w[i] = dtype == QMM_BF16 ? pack2<__nv_bfloat16>(v[2 * i], v[2 * i + 1]) : pack2<__half>(v[2 * i], v[2 * i + 1]);
  if constexpr (N == 4)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(base) + at) = make_uint2(w[0], w[1]);
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(base) + at) = w[0];
}

// (1 / (1 + e^-g), 1 / (1 + e^g)) for a result rounded to T.  e^-|g| is at most
// one, so it and its sum with one stay in range for every g (1 + e^-g itself
// passes 2^126 at g = -87.4, where the fast division gives 0).  f32: expf, each
// value within 2^-21 of itself (2^-148 where it is subnormal).  16 bits: __expf,
// whose error grows with |g| but stays below 2^-16 while e^-|g| is not zero, and a
// rounding to T is 2^-11 or 2^-8 (expf for all: 2048 tokens of 256 x 14336, where
// the epilogue is half of the time, 65 -> 89 us).
template <typename T>
__device__ __forceinline__ float2 logistic(float g) {
  float e;
  if constexpr (sizeof(T) == 4)
    e = expf(-fabsf(g));
  else
    e = __expf(-fabsf(g));
  const float r = __fdividef(1.0f, 1.0f + e), er = e * r;
  return g >= 0.0f ? make_float2(r, er) : make_float2(er, r);
}

// SiLU(g) * u for a result rounded to T: within 2^-20 of itself (f32) or 2^-15
template <typename T>
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * logistic<T>(g).x * u;
}

// A warp's 32 rows of 128 bytes, row `lane` written by that lane in 16-byte
// pieces swizzled by the row, then stored so that a row's 128 bytes leave
// together: 4 rows an instruction, where a lane's own row would touch 32 lines.
template <typename T>
struct Turn {
  static constexpr int COLS = 128 / (int)sizeof(T);
  uint32_t buf;
  int lane;
  // columns c .. c + 7 of the lane's row
  __device__ __forceinline__ void put8(int c, const float* v) const {
    const uint32_t row = buf + (uint32_t)(lane * 128);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        sts_v4(row + (uint32_t)((((c >> 2) + h) ^ (lane & 7)) << 4),
               make_uint4(__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]), __float_as_uint(v[4 * h + 2]),
                          __float_as_uint(v[4 * h + 3])));
    } else {
      sts_v4(row + (uint32_t)(((c >> 3) ^ (lane & 7)) << 4),
             make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7])));
    }
  }
  // to dst (row 0, column 0 of the piece), rows of ld elements; vec: 16-byte rows
  __device__ __forceinline__ void flush(T* dst, int64_t ld, int rows, int cols, bool vec) const {
    __syncwarp();
    if (vec) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = i * 4 + (lane >> 3), c = lane & 7;
        const uint4 v = lds_v4(buf + (uint32_t)(row * 128 + ((c ^ (row & 7)) << 4)));
        if (row < rows && c * (16 / (int)sizeof(T)) < cols)
          *reinterpret_cast<uint4*>(dst + row * ld + c * (16 / (int)sizeof(T))) = v;
      }
    } else {
#pragma unroll 8
      for (int row = 0; row < 32; ++row) {
#pragma unroll
        for (int c = lane; c < COLS; c += 32) {
          const int byte = c * (int)sizeof(T);
          const uint32_t a = buf + (uint32_t)(row * 128 + (((byte >> 4) ^ (row & 7)) << 4) + (byte & 15));
          if (c < cols && row < rows) {
            if constexpr (sizeof(T) == 4) {
              float v;
              asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
              dst[row * ld + c] = v;
            } else {
              const uint16_t v = lds_u16(a);
              memcpy(dst + row * ld + c, &v, 2);
            }
          }
        }
      }
    }
    __syncwarp();
  }
};

// h (and g, u) of 8 columns from column n of row m
template <typename T>
__device__ __forceinline__ void store_h8(const Args& p, int m, int n, const float* g, const float* u, bool vec) {
  const int cnt = p.N - n;
  if (cnt <= 0) return;
  const int64_t at = (int64_t)m * p.N + n;
  float h[8];
  if (p.out_dtype == QMM_F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = silu_mul<float>(g[i], u[i]);
    store8(reinterpret_cast<float*>(p.out[0]) + at, h, vec, cnt);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = silu_mul<T>(g[i], u[i]);
    store8(reinterpret_cast<T*>(p.out[0]) + at, h, vec, cnt);
  }
  if (p.out[1]) {
    store8(reinterpret_cast<T*>(p.out[1]) + at, g, vec, cnt);
    store8(reinterpret_cast<T*>(p.out[2]) + at, u, vec, cnt);
  }
}

// One product by `blocks` CTAs, of which this is number `block`; at least
// Cfg::THREADS threads (warps past those only keep the barriers).
template <int OP, int B, typename T, bool PAIR>
__device__ __forceinline__ void product(const Args& p, const Maps& tm, int block, int blocks) {
  using C = Cfg<OP, B, PAIR>;
  constexpr int S = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (su32(smem_raw) & 1023u)) & 1023u);
  const uint32_t stage0 = su32(smem);
  const uint32_t full0 = stage0 + C::BAR0;   // [S] operands of the stage are in (PAIR: the leader's counts both CTAs)
  const uint32_t empty0 = full0 + 8 * S;     // [S] the MMAs that read the stage are done
  const uint32_t accf0 = empty0 + 8 * S;     // [2] accumulator complete
  const uint32_t tfree0 = accf0 + 16;        // [2] accumulator read out
  const uint32_t drain = tfree0 + 16;        // every issued MMA complete
  const uint32_t cfull0 = drain + 8;         // [SLOTS] the step's codes are in
  const uint32_t cempty0 = cfull0 + 8 * C::SLOTS;   // [SLOTS] and dequantized
  const uint32_t wfull0 = cempty0 + 8 * C::SLOTS;   // [2] a window of scales and biases is in (FWD)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR0 + 8 * C::BARS);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int side = PAIR ? (int)(rank & 1u) : 0;        // this CTA's half of the pair's tile
  const uint32_t lead = PAIR ? rank & ~1u : rank;      // rank of the pair's leader
  const bool leader = side == 0;
  const int splits = p.splits;
  const int cta_per = (PAIR ? 2 : 1) * splits;  // CTAs of a cluster
  const int cluster = block / cta_per, clusters = blocks / cta_per;
  const int split = splits == 1 ? 0 : PAIR ? (int)(rank >> 1) : (int)rank;
  // this CTA's range of steps, and its cluster's tiles
  const int s_lo = (int)((int64_t)p.steps * split / splits), s_hi = (int)((int64_t)p.steps * (split + 1) / splits);
  const int nk = s_hi - s_lo;
  const int T_all = p.m_tiles * p.n_tiles * (OP == DP ? p.parts : 1);
  const int my_tiles = cluster < T_all ? (T_all - 1 - cluster) / clusters + 1 : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      // the producer, and the dequant warps that fill the stage (4 of each CTA
      // of a pair, 8 of a single one)
      mbar_init(full0 + 8 * s, 1 + (C::DENSE ? 0 : 8));
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf0 + 8 * b, 1);
      mbar_init(tfree0 + 8 * b, (OP == DP ? 8 : C::EPI) * (PAIR ? 2 : 1));
    }
    mbar_init(drain, 1);
    for (int s = 0; s < C::SLOTS; ++s) {
      mbar_init(cfull0 + 8 * s, 1);
      mbar_init(cempty0 + 8 * s, PAIR ? 4 : 8);
    }
    mbar_init(wfull0, 1);
    mbar_init(wfull0 + 8, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {  // two accumulators of 256 columns
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(tmem_slot)));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(tmem_slot)));
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
  }
  fence_before();
  __syncthreads();
  cluster_sync();  // the other CTAs' barriers are initialised
  fence_after();
  const uint32_t tmem = *tmem_slot;
  // the operands may come from the previous kernel
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    if (lane == 0) {
      constexpr uint32_t kTx = (PAIR ? 2 : 1) * (C::DENSE ? C::STAGE : C::A_BYTES);
      const uint32_t lfull0 = PAIR ? map_rank(full0, lead) : full0;
      const int half = OP == DP ? 0 : p.steps / p.parts;  // DX: steps of one part
      int s = 0, u = 0, issued = 0;
      bool stop = false;
      for (int lt = 0; lt < my_tiles && !stop; ++lt) {
        const Tile tl = tile_of<OP, PAIR>(p, cluster + lt * clusters);
        const int row = tl.m0 + 128 * side;
        for (int i = s_lo; i < s_hi; ++i) {
          if (u > 0 && !wait(empty0 + 8 * s, (u - 1) & 1, abort_flag)) {
            give_up<PAIR>(abort_flag);
            stop = true;
            break;
          }
          const uint32_t a = stage0 + s * C::STAGE, bar = lfull0 + 8 * s;
          if (leader) mbar_arrive_expect_tx(full0 + 8 * s, kTx);
          if constexpr (OP == DP) {
            const CUtensorMap* ma = &tm.a[tl.part];
            const int col = tl.n0 + 128 * side;
            tma_2d<PAIR>(a, ma, row, i * kBK, bar);
            tma_2d<PAIR>(a + 8192, ma, row + 64, i * kBK, bar);
            tma_2d<PAIR>(a + C::A_BYTES, &tm.b[0], col, i * kBK, bar);
            tma_2d<PAIR>(a + C::A_BYTES + 8192, &tm.b[0], col + 64, i * kBK, bar);
          } else if constexpr (OP == DX) {
            const bool second = i >= half;
            const int n = (second ? i - half : i) * kBK;
            tma_2d<PAIR>(a, &tm.a[second], n, row, bar);
            if constexpr (C::DENSE) {
              const CUtensorMap* mb = &tm.b[second];
              const int col = tl.n0 + 128 * side;
              tma_2d<PAIR>(a + C::A_BYTES, mb, col, n, bar);
              tma_2d<PAIR>(a + C::A_BYTES + 8192, mb, col + 64, n, bar);
            }
          } else {
            tma_2d<PAIR>(a, &tm.a[0], i * kBK, row, bar);
            if constexpr (C::DENSE) tma_2d<PAIR>(a + C::A_BYTES, &tm.b[side], i * kBK, tl.n0, bar);
          }
          ++issued;
          if (++s == S) s = 0, ++u;
        }
      }
      // no copy may still be landing when the CTA exits.  Every copy of a
      // finished tile was waited for by its MMAs; after a failure the leader
      // waits for the stages it armed, and the other CTA, whose copies count on
      // the leader's barrier, sits out a time far beyond any copy's.
      if (*reinterpret_cast<volatile int*>(abort_flag)) {
        if (leader) {
          for (int i = max(0, issued - S); i < issued; ++i)
            mbar_wait_n(full0 + 8 * (i % S), (uint32_t)(i / S) & 1u, 1u << 12);
        }
        for (int i = 0; i < 1000; ++i) __nanosleep(1000);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (PAIR && lane == 0 && !leader) {
      // (the leader's last commit arrives here too: nothing is on its way after it)
      for (int64_t i = 0; i < (int64_t)kPolls * (1 + ((int64_t)my_tiles * nk >> 15)) && !poll(drain, 0); ++i) {
      }
    } else if (lane == 0) {
      constexpr bool AMN = OP == DP, BMN = OP != FWD;
      constexpr int AK = AMN ? 2048 : 32, BK_ = BMN ? 2048 : 32;  // bytes per 16 k
      const uint32_t fmt = p.f16 ? 0u : 1u;
      const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((AMN ? 1u : 0u) << 15) | ((BMN ? 1u : 0u) << 16) |
                             ((256u >> 3) << 17) | (((PAIR ? 256u : 128u) >> 4) << 24);
      int s = 0, u = 0;
      bool stop = false;
      for (int lt = 0; lt < my_tiles && !stop; ++lt) {
        const int b = lt & 1;
        if (lt >= 2 && !wait_cluster(tfree0 + 8 * b, ((lt >> 1) - 1) & 1, abort_flag)) {
          give_up<PAIR>(abort_flag);
          break;
        }
        fence_after();
        const uint32_t acc = tmem + (uint32_t)(b * 256);
        for (int i = 0; i < nk; ++i) {
          if (!wait_cluster(full0 + 8 * s, u & 1, abort_flag)) {
            give_up<PAIR>(abort_flag);
            stop = true;
            break;
          }
          fence_after();
          const uint32_t a0 = stage0 + s * C::STAGE, b0 = a0 + C::A_BYTES;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk)
            mma<PAIR>(acc, desc<AMN>(a0 + kk * AK), desc<BMN>(b0 + kk * BK_), idesc, (i | kk) != 0 ? 1u : 0u);
          commit<PAIR>(empty0 + 8 * s, lead);
          if (++s == S) s = 0, ++u;
        }
        commit<PAIR>(accf0 + 8 * b, lead);  // (also after a failure)
      }
      // TMEM is released only once every issued MMA is done
      commit<PAIR>(drain, lead);
      for (uint32_t i = 0; i < kPolls && !poll(drain, 0); ++i) {
      }
    }
  } else if (!C::DENSE && warp >= 2 + C::EPI && warp < C::THREADS / 32) {
    if constexpr (!C::DENSE) {
      const int half = p.steps / p.parts;    // DX: steps of one part
      const int spw = p.lgs - 3;             // log2 of the steps of a window: 8 groups
      if (warp == 2 + C::EPI) {
        // ---------------- producer of the codes, scales and biases ----------------
        if (lane == 0) {
          const uint32_t sb_tx = p.sb_tma ? 2 * C::SB : 0;
          int j = 0, done = 0, win = 0, win_start = 0;  // done: steps known to be dequantized
          bool stop = false;
          auto reach = [&](int upto) {
            for (; done < upto; ++done)
              if (!wait(cempty0 + 8 * (done % C::SLOTS), (done / C::SLOTS) & 1, abort_flag)) return false;
            return true;
          };
          for (int lt = 0; lt < my_tiles && !stop; ++lt) {
            const Tile tl = tile_of<OP, PAIR>(p, cluster + lt * clusters);
            for (int i = s_lo; i < s_hi; ++i, ++j) {
              if (OP == FWD && p.sb_tma && (i == s_lo || (i & ((1 << spw) - 1)) == 0)) {
                // the window before the last one makes room
                if (!reach(win_start)) {
                  stop = true;
                  break;
                }
                const uint32_t d = stage0 + C::WIN0 + (win & 1) * C::WINDOW, bar = wfull0 + 8 * (win & 1);
                const int g = ((i * kBK) >> p.lgs) & ~7;
                mbar_arrive_expect_tx(bar, C::WINDOW);
#pragma unroll
                for (int x = 0; x < C::BOXES; ++x) {
                  const int part = PAIR ? side : x;
                  tma_2d<false>(d + (2 * x) * C::SB, &tm.s[part], g, tl.n0, bar);
                  tma_2d<false>(d + (2 * x + 1) * C::SB, &tm.z[part], g, tl.n0, bar);
                }
                ++win;
                win_start = j;
              }
              if (!reach(j - C::SLOTS + 1)) {
                stop = true;
                break;
              }
              const uint32_t d = stage0 + C::CODE0 + (j % C::SLOTS) * C::SLOT, bar = cfull0 + 8 * (j % C::SLOTS);
              mbar_arrive_expect_tx(bar, C::BOXES * C::BOX + (OP == DX ? sb_tx : 0u));
              if constexpr (OP == FWD) {
                const int w = B == 3 ? (i >> 1) * 12 : i * 2 * B;  // first word
#pragma unroll
                for (int x = 0; x < C::BOXES; ++x)
                  tma_2d<false>(d + x * C::BOX, &tm.b[PAIR ? side : x], w, tl.n0, bar);
              } else {
                const int part = i >= half, n = (part ? i - half : i) * kBK;
                const int col = tl.n0 + 128 * side;
#pragma unroll
                for (int x = 0; x < C::BOXES; ++x)
                  tma_2d<false>(d + x * C::BOX, &tm.b[part], ((col + 128 * x) >> 5) * B, n, bar);
                if (p.sb_tma) {
                  const int g = (col >> p.lgs) & ~7;
                  tma_2d<false>(d + C::BOXES * C::BOX, &tm.s[part], g, n, bar);
                  tma_2d<false>(d + C::BOXES * C::BOX + C::SB, &tm.z[part], g, n, bar);
                }
              }
            }
          }
          if (stop) {
            // (as the other producer: copies may be landing)
            give_up<PAIR>(abort_flag);
            for (int q = max(0, j - C::SLOTS); q < j; ++q)
              mbar_wait_n(cfull0 + 8 * (q % C::SLOTS), (q / C::SLOTS) & 1, 1u << 12);
            for (int q = max(0, win - 2); q < win; ++q) mbar_wait_n(wfull0 + 8 * (q & 1), (q >> 1) & 1, 1u << 12);
          }
        }
      } else {
        // ---------------- dequantize ----------------
        // the sets of warps that fill a stage (PAIR: 128 rows of B, 4 warps;
        // single: 256, 8 warps) take turns
        constexpr int WPS = PAIR ? 4 : 8, SETS = kDeqWarps / WPS;
        static_assert(C::SLOTS >= SETS && C::STAGES >= SETS, "one wrap a unit; older phases than the last are over");
        const int dw = warp - 3 - C::EPI, set = dw / WPS;
        const uint32_t lfull0 = PAIR ? map_rank(full0, lead) : full0;
        // this thread's 128 bytes of the operand tile: FWD, row r of B; DX, row
        // r of the step's 64 in block blk of 64 columns.  16-byte pieces are
        // swizzled by the row, so eight lanes write eight bank groups.
        const int r = OP == FWD ? (dw % WPS) * 32 + lane : (dw & 1) * 32 + lane;
        const int blk = OP == FWD ? 0 : (dw % WPS) >> 1;
        const uint32_t at = C::A_BYTES + (uint32_t)(blk * 8192 + r * 128);
        const int swz = r & 7;
        // its codes in a slot, its scales in a window or slot
        const int crow = OP == FWD ? r & 127 : r, cbox = OP == FWD ? r >> 7 : blk >> 1;
        const uint32_t codes = stage0 + C::CODE0 + (uint32_t)(cbox * C::BOX + crow * C::ROW);
        const int cswz = C::swz(crow);
        const uint32_t sbs = OP == FWD ? stage0 + C::WIN0 + (uint32_t)(2 * cbox * C::SB + crow * 16)
                                       : stage0 + C::CODE0 + (uint32_t)(C::BOXES * C::BOX + crow * 16);
        const int nwin = ((s_hi - 1) >> spw) - (s_lo >> spw) + 1;  // windows of a tile
        const int total = my_tiles * nk;
        const int64_t G = p.K >> p.lgs;
        int li = set, lt = 0, n0 = 0;
        auto settle = [&]() {  // li to a step of tile lt
          while (li >= nk) li -= nk, ++lt;
          n0 = lt < my_tiles ? tile_of<OP, PAIR>(p, cluster + lt * clusters).n0 : 0;
        };
        // first column of the unit's 64 codes and its two halves' groups
        auto column = [&]() {
          return OP == FWD ? (s_lo + li) * kBK : n0 + 128 * side + blk * 64;
        };
        // scales and biases of the unit at the cursor, from global memory
        auto fetch = [&](uint16_t (&sv)[2], uint16_t (&zv)[2]) {
          const int i = s_lo + li, k = column();
          int row, part;
          if constexpr (OP == FWD) {
            part = PAIR ? side : r >> 7;
            row = n0 + (r & 127);
          } else {
            part = i >= half;
            row = (part ? i - half : i) * kBK + r;
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int kh = k + 32 * h;
            sv[h] = zv[h] = 0;
            if (lt < my_tiles && row < p.N && kh < p.K) {  // past the weight: zeros
              const int64_t g = row * G + (kh >> p.lgs);
              sv[h] = __ldg(reinterpret_cast<const uint16_t*>(p.w[part].scales) + g);
              zv[h] = __ldg(reinterpret_cast<const uint16_t*>(p.w[part].biases) + g);
            }
          }
        };
        uint16_t sn[2] = {0, 0}, zn[2] = {0, 0};
        if (total > 0) settle();
        if (!p.sb_tma && total > 0) fetch(sn, zn);
        int s = set % S, u = set / S, c = set % C::SLOTS, cu = set / C::SLOTS;
        uint32_t dst = stage0 + (uint32_t)(s * C::STAGE) + at + (uint32_t)(swz << 4);
        uint32_t src = codes + (uint32_t)(c * C::SLOT);
        int win_in = -1;  // FWD: the last window waited for
        for (int j = set; j < total; j += SETS) {
          const int i = s_lo + li, k = column();
          uint32_t w[2][B];
          uint16_t sv[2], zv[2];
          // Where a slot passes from set to set, this set has not seen its last codes
          // land (copies may land out of order, and the parity of the phase before last
          // would pass for this one's): those codes must be dequantized first.  That
          // barrier cannot run ahead, since its next phase needs this set.
          if constexpr (C::SLOTS % SETS != 0) {
            if (cu > 0) wait_fast<PAIR>(cempty0 + 8 * c, (cu - 1) & 1, abort_flag);
          }
          wait_fast<PAIR>(cfull0 + 8 * c, cu & 1, abort_flag);
          read_codes<B>(src, OP == FWD ? (B == 3 ? (i & 1) * 24 : 0) : (blk & 1) * 8 * B, cswz, w);
          if (p.sb_tma) {
            uint32_t o = sbs + ((k >> p.lgs) & 7) * 2;
            if constexpr (OP == FWD) {
              const int win = lt * nwin + (i >> spw) - (s_lo >> spw);
              if (win != win_in) wait_fast<PAIR>(wfull0 + 8 * (win & 1), (win >> 1) & 1, abort_flag);
              win_in = win;
              o += (uint32_t)((win & 1) * C::WINDOW);
            } else {
              o += (uint32_t)(c * C::SLOT);
            }
            sv[0] = sv[1] = lds_u16(o);
            zv[0] = zv[1] = lds_u16(o + C::SB);
            if (p.lgs == 5) {  // 64 codes are two groups
              sv[1] = lds_u16(o + 2);
              zv[1] = lds_u16(o + C::SB + 2);
            }
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) sv[h] = sn[h], zv[h] = zn[h];
          }
          li += SETS;
          if (li >= nk) settle();
          if (!p.sb_tma) fetch(sn, zn);
          // all of the unit before the wait for its stage, which the MMAs of S steps
          // ago hold: what then stands between them and the next is the store alone
          uint4 v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            v[q] = dequant8<B, T>(w[q >> 2], sv[q >> 2], zv[q >> 2], q & 3);
            asm volatile("" ::"r"(v[q].x), "r"(v[q].y), "r"(v[q].z), "r"(v[q].w));
          }
          if (u > 0) wait_fast<PAIR>(empty0 + 8 * s, (u - 1) & 1, abort_flag);
#pragma unroll
          for (int q = 0; q < 8; ++q) sts_v4(dst ^ (uint32_t)(q << 4), v[q]);
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // visible to the tensor cores
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR)
              arrive_remote(lfull0 + 8 * s);
            else
              mbar_arrive(full0 + 8 * s);
            mbar_arrive(cempty0 + 8 * c);
          }
          s += SETS, dst += SETS * C::STAGE;
          if (s >= S) s -= S, ++u, dst -= S * C::STAGE;
          c += SETS, src += SETS * C::SLOT;
          if (c >= C::SLOTS) c -= C::SLOTS, ++cu, src -= C::SLOTS * C::SLOT;
        }
      }
    }
  }

  // ---------------- epilogue ----------------
  // The epilogue warps; where each CTA has one tile, the dequant warps too once
  // they are done (a tile's columns are dealt out 16 at a time).
  const bool only = T_all <= clusters;
  if ((warp >= 2 && warp < 2 + C::EPI) || (!C::DENSE && only && warp > 2 + C::EPI && warp < C::THREADS / 32)) {
    constexpr int kEach = C::EPI / 4 + C::DEQ / 4;  // warps of a lane quarter, when all take part
    const int first = (C::DENSE || !only || warp < 2 + C::EPI) ? 0 : 16 * (1 + (warp - 3 - C::EPI) / 4);
    const int stride = (C::DENSE || !only) ? 16 : 16 * kEach;
    const int qq = warp & 3;           // the TMEM lanes this warp may read
    const int r = qq * 32 + lane;      // row of the CTA's 128
    const uint32_t lanes = tmem + ((uint32_t)(qq * 32) << 16);
    const uint32_t ltfree0 = PAIR ? map_rank(tfree0, lead) : tfree0;
    const float nan = __int_as_float(0x7fc00000);
    bool failed = false;
    // (DP: two sets of 8 warps, one for each accumulator)
    for (int lt = OP == DP ? (warp - 2) >> 3 : 0; lt < my_tiles; lt += OP == DP ? 2 : 1) {
      const Tile tl = tile_of<OP, PAIR>(p, cluster + lt * clusters);
      const int b = lt & 1;
      const int row = tl.m0 + 128 * side + r;
      // DP: the codes of the lane's row, requested while the products run: 128
      // codes are 16 B bytes, in 16-byte loads where rows start on 16 bytes
      uint32_t codes[4][B ? B : 1];
      const int c0 = OP == DP ? (((warp - 2) >> 2) & 1) * 128 : 0;
      if constexpr (OP == DP) {
        const int k0 = tl.n0 + c0;
        const uint32_t* src = p.w[tl.part].packed + ((int64_t)row * (p.K >> 5) + (k0 >> 5)) * B;
        if (row < p.N && (p.K >> 5) * B % 4 == 0 && k0 + 128 <= p.K) {
          uint32_t* flat = &codes[0][0];
#pragma unroll
          for (int i = 0; i < B; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + i);
            flat[4 * i] = v.x; flat[4 * i + 1] = v.y; flat[4 * i + 2] = v.z; flat[4 * i + 3] = v.w;
          }
        } else if (row < p.N) {
#pragma unroll
          for (int un = 0; un < 4; ++un)
            if (k0 + un * 32 < p.K) load_words<B>(src + un * B, codes[un]);
        }
      }
      if (!failed) {
        failed = !wait_steps(accf0 + 8 * b, (lt >> 1) & 1, abort_flag, nk) ||
                 *reinterpret_cast<volatile int*>(abort_flag);
        failed = __any_sync(0xffffffffu, failed);
      }
      fence_after();
      const uint32_t acc = lanes + (uint32_t)(b * 256);
      if constexpr (OP == DP) {
        // 128 columns of one weight row: sums of units of 32, then groups of 1, 2
        // or 4 units, stored together where they are aligned
        const int G = p.K >> p.lgs, k0 = tl.n0 + c0;
        const bool live = row < p.N;
        float ds[4], dz[4];
#pragma unroll
        for (int un = 0; un < 4; ++un) {
          float2 sq = make_float2(0.0f, 0.0f), sv = sq;
          if (k0 + un * 32 < p.K) {
            const uint32_t(&w)[B] = codes[un];
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float v[16];
              if (!failed) {
                tmem_ld16(acc + (uint32_t)(c0 + un * 32 + hf * 16), v);
                tmem_wait();
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = nan;
              }
              if (live) {
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                  const float2 x = make_float2(v[i], v[i + 1]);
                  sq = fma2f(x, codes2<B>(w, hf * 16 + i), sq);
                  sv = add2(sv, x);
                }
              }
            }
          }
          ds[un] = sq.x + sq.y;
          dz[un] = sv.x + sv.y;
        }
        if (live && k0 < p.K) {
          if (p.lgs > 5) {
            ds[0] += ds[1], ds[1] = ds[2] + ds[3];
            dz[0] += dz[1], dz[1] = dz[2] + dz[3];
          }
          if (p.lgs > 6) ds[0] += ds[1], dz[0] += dz[1];
          const int64_t at = (int64_t)row * G + (k0 >> p.lgs);
          const int n = min(128, p.K - k0) >> p.lgs;  // groups
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            void* dst = p.out[2 * tl.part + o];
            const float* v = o ? dz : ds;
            if (n == 4 && G % 4 == 0)
              store_run<4>(dst, p.out_dtype, at, v);
            else if (n == 2 && G % 2 == 0)
              store_run<2>(dst, p.out_dtype, at, v);
            else
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (i < n) store_as(dst, p.out_dtype, at + i, v[i]);
          }
        }
      } else if (splits > 1) {
        // a partial tile: four columns of all 128 rows are 2 KB
#pragma unroll 1
        for (int c = first; c < 256; c += stride) {
          float v[16];
          if (!failed) {
            tmem_ld16(acc + (uint32_t)c, v);
            tmem_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = nan;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            sts_v4(stage0 + (uint32_t)(((c >> 2) + i) * 2048 + r * 16),
                   make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                              __float_as_uint(v[4 * i + 3])));
        }
      } else if constexpr (OP == FWD) {
        const bool vec = p.N % 8 == 0;
        auto read = [&](int c, float (&g)[16], float (&u)[16]) {
          if (!failed) {
            tmem_ld16(acc + (uint32_t)c, g);
            tmem_ld16(acc + (uint32_t)(128 + c), u);
            tmem_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) g[i] = u[i] = nan;
          }
        };
        if (only && vec) {  // each lane stores its own row: more warps at work
#pragma unroll 1
          for (int c = first; c < 128 && tl.n0 + c < p.N; c += stride) {
            float g[16], u[16];
            read(c, g, u);
            if (row < p.M) {
              store_h8<T>(p, row, tl.n0 + c, g, u, vec);
              store_h8<T>(p, row, tl.n0 + c + 8, g + 8, u + 8, vec);
            }
          }
        } else {
          // what 0: h, 1: g, 2: u, each 128 bytes of 32 rows at a time, dealt to
          // the warps of the lane quarter (all done reading the stages, if several)
          const uint32_t buf = stage0 + (uint32_t)((only ? 0 : C::OUT0) + (warp - 2) * 4096);
          int job = -(first >> 4);
          auto piece = [&](auto type, int what) {
            using O = decltype(type);
            const Turn<O> out{buf, lane};
            const int row0 = row - lane;
#pragma unroll 1
            for (int c0 = 0; c0 < 128 && tl.n0 + c0 < p.N; c0 += Turn<O>::COLS) {
              if (job++ % (stride >> 4) != 0) continue;
#pragma unroll 1
              for (int c = 0; c < Turn<O>::COLS; c += 16) {
                float g[16], u[16];
                if (what == 0) {
                  read(c0 + c, g, u);
#pragma unroll
                  for (int i = 0; i < 16; ++i) g[i] = silu_mul<O>(g[i], u[i]);
                } else if (!failed) {
                  tmem_ld16(acc + (uint32_t)((what - 1) * 128 + c0 + c), g);
                  tmem_wait();
                } else {
#pragma unroll
                  for (int i = 0; i < 16; ++i) g[i] = nan;
                }
                out.put8(c, g);
                out.put8(c + 8, g + 8);
              }
              out.flush(reinterpret_cast<O*>(p.out[what]) + (int64_t)row0 * p.N + tl.n0 + c0, p.N, p.M - row0,
                        p.N - tl.n0 - c0, vec);
            }
          };
          if (p.out_dtype == QMM_F32)
            piece(float(), 0);
          else
            piece(T(), 0);
          if (p.out[1]) {
            piece(T(), 1);
            piece(T(), 2);
          }
        }
      } else {
        auto read = [&](int c, float (&v)[16]) {
          if (!failed) {
            tmem_ld16(acc + (uint32_t)c, v);
            tmem_wait();
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = nan;
          }
        };
        if (only) {
#pragma unroll 1
          for (int c = first; c < 256 && tl.n0 + c < p.K; c += stride) {
            float v[16];
            read(c, v);
            if (row < p.M) {
              T* dst = reinterpret_cast<T*>(p.out[0]) + (int64_t)row * p.K + tl.n0 + c;
              store8(dst, v, true, 8);
              store8(dst + 8, v + 8, true, 8);
            }
          }
        } else {
          const Turn<T> out{stage0 + (uint32_t)(C::OUT0 + (warp - 2) * 4096), lane};
          const int row0 = row - lane;
#pragma unroll 1
          for (int c0 = 0; c0 < 256 && tl.n0 + c0 < p.K; c0 += Turn<T>::COLS) {
#pragma unroll 1
            for (int c = 0; c < Turn<T>::COLS; c += 16) {
              float v[16];
              read(c0 + c, v);
              out.put8(c, v);
              out.put8(c + 8, v + 8);
            }
            out.flush(reinterpret_cast<T*>(p.out[0]) + (int64_t)row0 * p.K + tl.n0 + c0, p.K, p.M - row0,
                      p.K - tl.n0 - c0, true);
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0 && !failed && warp < 2 + C::EPI) {
        if constexpr (PAIR)
          arrive_remote(ltfree0 + 8 * b);
        else
          mbar_arrive(tfree0 + 8 * b);
      }
    }
  }

  __syncwarp();
  fence_before();
  if constexpr (OP != DP) {
    if (splits > 1) {
      // join the partial tiles: this CTA takes its share of the columns of its
      // 128 rows, adding the partials of the CTAs with the same rows in rank order
      cluster_sync();
      constexpr int COLS = OP == FWD ? 128 : 256;
      const Tile tl = tile_of<OP, PAIR>(p, cluster);
      const int per = COLS / 8 / splits;  // 8-column pieces of this CTA (splits divides 16)
      const bool vec = OP == DX || p.N % 8 == 0;
      const int m0 = tl.m0 + 128 * side, rows = min(128, p.M - m0);
      for (int it = threadIdx.x; it < per * 128; it += (int)blockDim.x) {
        const int row = it & 127, c = (split * per + (it >> 7)) * 8;
        if (row >= rows || tl.n0 + c >= (OP == FWD ? p.N : p.K)) continue;
        float v[2][8];
#pragma unroll
        for (int q = 0; q < (OP == FWD ? 2 : 1); ++q) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
          for (int src = 0; src < splits; ++src) {
            const uint32_t a = map_rank(stage0 + (uint32_t)(((q * 128 + c) >> 2) * 2048 + row * 16),
                                        PAIR ? 2 * src + side : src);
            const float4 x = lds_cluster(a), y = lds_cluster(a + 2048);
            v[q][0] += x.x; v[q][1] += x.y; v[q][2] += x.z; v[q][3] += x.w;
            v[q][4] += y.x; v[q][5] += y.y; v[q][6] += y.z; v[q][7] += y.w;
          }
        }
        if constexpr (OP == FWD)
          store_h8<T>(p, m0 + row, tl.n0 + c, v[0], v[1], vec);
        else
          store8(reinterpret_cast<T*>(p.out[0]) + (int64_t)(m0 + row) * p.K + tl.n0 + c, v[0], true, 8);
      }
    }
  }
  __syncthreads();
  cluster_sync();  // no CTA leaves while another may signal or read it
  if (warp == 1) {
    fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    else
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

template <int OP, int B, typename T, bool PAIR>
__global__ void __launch_bounds__(Cfg<OP, B, PAIR>::THREADS, 1)
pair_gemm_kernel(const __grid_constant__ Args p, const __grid_constant__ Maps tm) {
  product<OP, B, T, PAIR>(p, tm, (int)blockIdx.x, (int)gridDim.x);
}

// Both products of a backward pass in one launch: the first dx_blocks CTAs take
// dx, the others the parameter gradients, so that few tiles of the one leave no
// SM idle that the other can use.  (Both use cta_group::2, as one kernel must.)
template <int B, typename T>
__global__ void __launch_bounds__(Cfg<DX, B, true>::THREADS, 1)
backward_kernel(const __grid_constant__ Args dx, const __grid_constant__ Maps dx_maps, const __grid_constant__ Args dp,
                const __grid_constant__ Maps dp_maps, int dx_blocks) {
  static_assert(Cfg<DX, B, true>::THREADS >= Cfg<DP, B, true>::THREADS, "one block shape for both");
  if ((int)blockIdx.x < dx_blocks)
    product<DX, B, T, true>(dx, dx_maps, (int)blockIdx.x, dx_blocks);
  else
    product<DP, B, T, true>(dp, dp_maps, (int)blockIdx.x - dx_blocks, (int)gridDim.x - dx_blocks);
}

// ------------------------------------------------------------------ host
// 2-D map over 16-bit [rows, cols] (row stride ld elements): boxes of 64
// columns x box_rows rows, 128-byte swizzle, zeros outside
inline bool make_map(CUtensorMap* m, const void* base, bool f16, int64_t rows, int64_t cols, int64_t ld, int box_rows) {
  EncodeTiledFn enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * 2)};
  const cuuint32_t box[2] = {kBK, (cuuint32_t)box_rows};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of the packed side of one part: codes in boxes of Cfg's shape, and
// scales and biases in boxes of 8 groups.  False when the codes' rows do not
// start on 16 bytes.
template <int OP, int B>
bool make_code_maps(Maps* tm, int part, const Args& p) {
  using C = Cfg<OP, B, true>;
  EncodeTiledFn enc = tensor_map_encoder();
  const int64_t wpr = (int64_t)p.K / 32 * B, G = p.K >> p.lgs;
  if (!enc || wpr % 4 != 0) return false;
  const cuuint32_t estr[2] = {1, 1};
  const cuuint64_t dims[2] = {(cuuint64_t)wpr, (cuuint64_t)p.N};
  const cuuint64_t strides[1] = {(cuuint64_t)(wpr * 4)};
  const cuuint32_t box[2] = {(cuuint32_t)(C::ROW / 4), (cuuint32_t)C::BOX_ROWS};
  const CUtensorMapSwizzle swz = C::SWZ == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                                 : C::SWZ == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                 : C::SWZ == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                                 : CU_TENSOR_MAP_SWIZZLE_NONE;
  if (enc(&tm->b[part], CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<uint32_t*>(p.w[part].packed), dims, strides, box,
          estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  tm->s[part] = tm->z[part] = tm->b[part];
  if (!p.sb_tma) return true;
  const cuuint64_t gdims[2] = {(cuuint64_t)G, (cuuint64_t)p.N};
  const cuuint64_t gstrides[1] = {(cuuint64_t)(G * 2)};
  const cuuint32_t gbox[2] = {8, (cuuint32_t)C::BOX_ROWS};
  for (int a = 0; a < 2; ++a)
    if (enc(a ? &tm->z[part] : &tm->s[part], CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
            const_cast<void*>(a ? p.w[part].biases : p.w[part].scales), gdims, gstrides, gbox, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  return true;
}

// A launch of `blocks` CTAs in clusters of `per`, programmatic after the
// previous kernel; the shared-memory limit is raised once per device and kernel.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*k)(P...), int* configured, int blocks, int threads, int smem, int per, cudaStream_t st,
                          const A&... args) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = per;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = per > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

template <int OP, int B, typename T, bool PAIR>
cudaError_t launch(const Args& p, const Maps& tm, int clusters, cudaStream_t st) {
  using C = Cfg<OP, B, PAIR>;
  static int configured[64] = {0};
  const int per = (PAIR ? 2 : 1) * p.splits;
  return launch_kernel(pair_gemm_kernel<OP, B, T, PAIR>, configured, clusters * per, C::THREADS, C::SMEM, per, st, p,
                       tm);
}

template <int OP, int B, bool PAIR>
cudaError_t launch_t(const Args& p, const Maps& tm, int clusters, cudaStream_t st) {
  return p.f16 ? launch<OP, B, __half, PAIR>(p, tm, clusters, st)
               : launch<OP, B, __nv_bfloat16, PAIR>(p, tm, clusters, st);
}

// One bit width's kernels; DP does not depend on T.  cudaErrorNotSupported: FWD
// and DX want the codes' rows on 16 bytes.
template <int B>
cudaError_t dispatch(int op, bool pair, Args& p, Maps& tm, int clusters, cudaStream_t st) {
  if (op == DP) return launch<DP, B, __nv_bfloat16, true>(p, tm, clusters, st);
  p.sb_tma = (p.K >> p.lgs) % 8 == 0;
  for (int i = 0; i < p.parts; ++i)
    if (!(op == FWD ? make_code_maps<FWD, B>(&tm, i, p) : make_code_maps<DX, B>(&tm, i, p)))
      return cudaErrorNotSupported;
  if (op == DX) return launch_t<DX, B, true>(p, tm, clusters, st);
  return pair ? launch_t<FWD, B, true>(p, tm, clusters, st) : launch_t<FWD, B, false>(p, tm, clusters, st);
}

// Both products of a backward pass in one launch.  dx_clusters of dx, then
// dp_pairs CTA pairs (a multiple of dx.splits) of the parameter gradients.
template <int B>
cudaError_t dispatch_both(Args& dx, Maps& dx_maps, const Args& dp, const Maps& dp_maps, int dx_clusters, int dp_pairs,
                          cudaStream_t st) {
  dx.sb_tma = (dx.K >> dx.lgs) % 8 == 0;
  for (int i = 0; i < dx.parts; ++i)
    if (!make_code_maps<DX, B>(&dx_maps, i, dx)) return cudaErrorNotSupported;
  constexpr int kThreads = Cfg<DX, B, true>::THREADS;
  constexpr int kSmem = std::max(Cfg<DX, B, true>::SMEM, Cfg<DP, B, true>::SMEM);
  static int configured[2][64] = {{0}};
  const int per = 2 * dx.splits, dx_blocks = dx_clusters * per, blocks = dx_blocks + 2 * dp_pairs;
  if (dx.f16)
    return launch_kernel(backward_kernel<B, __half>, configured[0], blocks, kThreads, kSmem, per, st, dx, dx_maps, dp,
                         dp_maps, dx_blocks);
  return launch_kernel(backward_kernel<B, __nv_bfloat16>, configured[1], blocks, kThreads, kSmem, per, st, dx, dx_maps,
                       dp, dp_maps, dx_blocks);
}

}  // namespace pg
}  // namespace qmm
