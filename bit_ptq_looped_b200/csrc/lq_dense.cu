// Dense (unquantized) products around the looped linear, on the 5th-generation
// tensor cores (sm_100a), operands bf16 or f16:
//
//   dense        y  = act(x W^T + b) + r          (optionally z = x W^T + b)
//   gated        h  = act(x Wg^T + bg) * (x Wu^T + bu)   (optionally both factors)
//   dx           dx = dz W        (gated: [dg | du] [Wg ; Wu])
//   dw           dw = dz^T x      (gated: both weights in one product)
//
// All four are one product C = A B^T over a contraction index kept in 64-wide
// blocks; they differ in which operand is contiguous along the contraction
// (K-major: x, W, dz rows) and which across it (MN-major: W in dx, both
// operands of dw), and in the epilogue.  tcgen05.mma reads either form
// straight from the 128-byte-swizzled tile that TMA wrote, so no operand is
// ever transposed in memory.
//
// k_dense_gemm is persistent (one CTA per SM): a TMA warp fills a ring of
// stages, an MMA warp issues kind::f16 MMAs (float32 accumulators in TMEM, two
// accumulators so that a tile's epilogue overlaps the next tile's products),
// and the epilogue warps read TMEM, apply bias, activation, product and
// residual in float32, round once, and write whole 64-byte or longer row
// pieces through a swizzled shared-memory tile.  Large products are bound by the
// tensor pipe: a tile of CTA pairs takes the pipe's own 512 clocks per 64-wide
// block, 16384 x 5632 x 2048 takes 244 us (1.55 PFLOP/s) and its gated form 473
// (1.60) in a short series; in a long one the power cap sets the clock.  One elected lane runs
// the whole copy or MMA loop: an elected lane inside a loop of the whole warp took
// 350 clocks per block of a 128 x 64 tile, a plain lane test 540, this form 285.
// Where a long contraction has few tiles, a cluster of CTAs shares a tile: each takes
// a part of the contraction, sends its float32 sums to the CTA that finishes the row,
// and that one adds them in a fixed order.
//
// Up to 16 rows (decode) the product is a stream of the weights:
// k_dense_rows reads each weight once with 16-byte loads and multiplies with
// mma.sync (16 weight rows x 8 tokens), the contraction split over the warps
// of a block (1 x 49152 x 2048: 37.6 us, 5.35 TB/s, 82 % of HBM); k_rows_dx and
// k_rows_dw do the same for the gradients, in float32.
//
// Every mbarrier wait is bounded; on expiry the kernel records
// LQ_ERR_DEVICE_TIMEOUT, stops all roles, frees its TMEM and returns.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "lq_dense.cuh"

namespace lq {
namespace {

constexpr int BM = 128;  // accumulator rows of a CTA (TMEM lanes)
constexpr int BK = 64;   // contraction elements per stage: one 128-byte row of 16-bit values
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per wait

__device__ int g_dense_status = 0;

// Bounded wait on an mbarrier phase: false once `limit_ns` have passed or the
// CTA's abort flag is up (and raises it on a timeout, so that the other roles
// stop too).  The clock is read once in 1024 polls.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort,
                                             uint64_t limit_ns = kWaitLimitNs) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 1023u) == 0) {
      if (*abort) return false;
      const uint64_t t = global_timer_ns();
      if (t0 == 0) {
        t0 = t;
      } else if (t - t0 > limit_ns) {
        *abort = 1;
        atomicExch(&g_dense_status, (int)LQ_ERR_DEVICE_TIMEOUT);
        return false;
      }
    }
  }
}

// The same wait by a whole warp, with one answer: lanes may see the limit or the abort
// flag at different polls, and what follows (tcgen05.ld, shuffles) needs all of them.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort,
                                          uint64_t limit_ns = kWaitLimitNs) {
  return __all_sync(~0u, wait_bounded(bar, parity, abort, limit_ns));
}

// The same wait without the abort flag (teardown: no copy or MMA of this CTA is
// in flight when it exits).
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
  int none = 0;
  wait_bounded(bar, parity, &none);
}

// ---------------------------------------------------------------------------
// element types
// ---------------------------------------------------------------------------
template <typename T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
  static constexpr uint32_t kFormat = 1;  // instruction descriptor: bf16
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  static __device__ __forceinline__ float load(const uint16_t* p) {
    return __uint_as_float((uint32_t)*p << 16);
  }
  static __device__ __forceinline__ uint16_t round(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};
template <>
struct Elem<__half> {
  static constexpr uint32_t kFormat = 0;  // f16
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
  }
  static __device__ __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<__half2*>(&w));
  }
  static __device__ __forceinline__ float load(const uint16_t* p) {
    return __half2float(__ushort_as_half(*p));
  }
  static __device__ __forceinline__ uint16_t round(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
};

// ---------------------------------------------------------------------------
// activations, float32
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// logistic function through the hardware exponential and reciprocal (off by about
// 2^-22 + |z| 2^-23 of the value, its exponent being rounded: far below the 16-bit
// output rounding); exp overflow gives 1/inf = 0
__device__ __forceinline__ float logistic(float z) {
  return rcp(1.f + ex2(-1.4426950408889634f * z));
}
constexpr float kGeluC = 0.7978845608028654f;  // sqrt(2 / pi)
// 0.5 (1 + tanh(v)) = logistic(2 v): no cancellation for large negative v
__device__ __forceinline__ float gelu_tanh_gate(float z) {
  return logistic(2.f * kGeluC * (z + 0.044715f * z * z * z));
}
// The normal distribution function Phi(z), and e = exp(-z^2 / 2).  The upper
// tail is Q(a) = e P(1 / (1 + c a)), a = |z|, with a polynomial P without
// constant term (Q(a) / e falls off as 1 / a) fitted to 0.5 erfcx(a / sqrt 2) by
// weighted least squares over 0 <= a <= 14; Phi is Q or 1 - Q, so nothing cancels
// at large negative z.  In float32 it is off by at most 6e-7 absolute, and by 1.3e-6 of
// the value above z = -3; below, the rounded exponent adds up to z^2 2^-23 of the value
// (2.2e-6 down to -6, 7.7e-6 down to -13), against half a step of 4.9e-4 of an f16 output.
__device__ __forceinline__ float phi_cdf(float z, float& e) {
  const float a = fabsf(z);
  const float t = rcp(fmaf(0.36f, a, 1.f));
  float p = 0.04705650359392166f;
  p = fmaf(p, t, -0.17976532876491547f);
  p = fmaf(p, t, 0.18095475435256958f);
  p = fmaf(p, t, 0.026548894122242928f);
  p = fmaf(p, t, 0.1397193968296051f);
  p = fmaf(p, t, 0.14177243411540985f);
  p = fmaf(p, t, 0.14371304214000702f);
  e = ex2(-0.7213475204444817f * z * z);
  const float q = e * (p * t);
  return z > 0.f ? 1.f - q : q;
}

template <int kAct>
__device__ __forceinline__ float act_fn(float z) {
  if (kAct == LQ_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
  if (kAct == LQ_ACT_SILU) return z * logistic(z);
  if (kAct == LQ_ACT_GELU) {
    float e;
    return z * phi_cdf(z, e);
  }
  if (kAct == LQ_ACT_GELU_TANH) return z * gelu_tanh_gate(z);
  return z;
}

// act(z) and act'(z)
template <int kAct>
__device__ __forceinline__ void act_grad(float z, float& a, float& da) {
  if (kAct == LQ_ACT_RELU) {
    a = z > 0.f ? z : (z != z ? z : 0.f);
    da = z > 0.f ? 1.f : (z != z ? z : 0.f);
  } else if (kAct == LQ_ACT_SILU) {
    const float s = logistic(z);
    a = z * s;
    da = s + a * (1.f - s);
  } else if (kAct == LQ_ACT_GELU) {
    float e;
    const float p = phi_cdf(z, e);
    a = z * p;
    da = fmaf(z * e, 0.3989422804014327f, p);  // 1 / sqrt(2 pi)
  } else if (kAct == LQ_ACT_GELU_TANH) {
    const float s = gelu_tanh_gate(z);
    a = z * s;
    // past |z| = 100 the factor a (1 - s) is zero; the bound keeps z^2 finite
    da = s + 2.f * a * (1.f - s) * kGeluC * (1.f + 3.f * 0.044715f * fminf(z * z, 1e4f));
  } else {
    a = z;
    da = 1.f;
  }
}

// v[i] = act(v[i]) for n values, the activation chosen once per call
template <int kN>
__device__ __forceinline__ void apply_act(int act, float (&v)[kN]) {
  switch (act) {
    case LQ_ACT_RELU:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = act_fn<LQ_ACT_RELU>(v[i]);
      break;
    case LQ_ACT_SILU:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = act_fn<LQ_ACT_SILU>(v[i]);
      break;
    case LQ_ACT_GELU:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = act_fn<LQ_ACT_GELU>(v[i]);
      break;
    case LQ_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < kN; ++i) v[i] = act_fn<LQ_ACT_GELU_TANH>(v[i]);
      break;
    default:
      break;
  }
}

// ---------------------------------------------------------------------------
// tcgen05 wrappers
// ---------------------------------------------------------------------------
// Shared-memory descriptors of 128-byte-swizzled 16-bit tiles.
// K-major: rows of 64 contraction elements (128 B), 8-row atoms 1024 B apart
// (stride offset); the leading offset is not used.
// MN-major: the tile is a row of chunks of 64 row indices (128 B) by 64
// contraction steps; 8-step atoms are 1024 B apart (stride offset), chunks
// 8192 B apart (leading offset).
__device__ __forceinline__ uint64_t smem_desc(uint32_t saddr, bool mn_major) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((mn_major ? 8192u : 16u) >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;  // descriptor version (sm_100)
  d |= (uint64_t)2u << 61;  // 128-byte swizzle
  return d;
}

// kind::f16: F32 accumulator, operand format, operand majors, N >> 3, M >> 4
__host__ __device__ constexpr uint32_t instr_desc(uint32_t fmt, bool a_mn, bool b_mn, int m,
                                                  int n) {
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// kPair: CTAs that share one MMA (1, or 2: the pair's first CTA issues for both)
template <int kPair>
__device__ __forceinline__ void umma_f16(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t acc) {
  if (kPair == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc)
        : "memory");
}

// arrival on `bar` (the same offset in both CTAs of a pair) once every MMA
// issued so far has completed
template <int kPair>
__device__ __forceinline__ void commit_all(uint32_t bar) {
  if (kPair == 1)
    umma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

template <int kPair>
__device__ __forceinline__ void tmem_take(uint32_t dst_smem, uint32_t ncols) {
  if (kPair == 1) {
    tmem_alloc(dst_smem, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int kPair>
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t ncols) {
  if (kPair == 1)
    tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}

// a tile into this CTA's shared memory; the bytes count on `bar`, a shared::cluster
// address that may belong to the pair's first CTA
template <int kPair>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                          int c0, int c1) {
  if (kPair == 1)
    tma_load_2d(dst, map, bar, c0, c1);
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".cta_group::2 [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"((uint64_t)map), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the same shared-memory offset in the pair's first CTA
__device__ __forceinline__ uint32_t in_first_cta(uint32_t saddr) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(0));
  return r;
}
// ... in any CTA of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  cluster_arrive();
  cluster_wait();
}

// ---------------------------------------------------------------------------
// the tile kernel
// ---------------------------------------------------------------------------
enum Epi : int {
  kEpiDense = 0,  // act(acc + bias) + residual, optionally the pre-activation
  kEpiGated = 1,  // act(acc_g + bias_g) * (acc_u + bias_u), optionally both factors
  kEpiStore = 2,  // round and store
  kEpiF32 = 3,    // float32, optionally added to what is there
};

struct GemmParams {
  int64_t M, N;    // extents of the output (N per factor when gated)
  int64_t ldo;     // elements between output rows
  int n_kb, n_kb1; // contraction blocks; those of the first operand pair
  int slice_kb;    // blocks of a slice of the contraction (blockIdx.y, or the cluster's
                   // member where a cluster shares a tile), n_kb when whole
  int64_t slice_bytes;  // bytes from one slice's output to the next
  int members;     // CTAs of a cluster that share a tile
  int act;
  int accumulate;
  int vec;         // rows are 16-byte aligned: 16-byte stores
  const uint16_t* bias;
  const uint16_t* bias2;
  const uint16_t* res;
  void* out;
  // output rows from `split` on go to out2 (row r to out2 + (r - split) * ldo),
  // rows in [rows1, split) are padding and are not written
  void* out2;
  int64_t split, rows1;
  uint16_t* aux;   // z, or the gate factor g
  uint16_t* aux2;  // the up factor u
};

// Float32 sums of a 64-wide tile that a cluster shares, row by row in shared memory; 16
// bytes more per row keep the row-per-lane stores free of bank conflicts.
constexpr int kSumLd = 64 + 4;

template <int kBN, int kPair, int kEpi, bool kShared>
struct Cfg {
  static constexpr int kEpiWarps = kBN >= 128 ? 8 : 4;
  // columns an epilogue warp handles: its column half of the tile (of each
  // factor's half when gated)
  static constexpr int kCols = kBN / (kEpiWarps / 4) / (kEpi == kEpiGated ? 2 : 1);
  // columns per shared-memory unit: 128-byte rows, or 64-byte ones
  static constexpr int kUnit = (kEpi == kEpiF32 || kCols < 64) ? 32 : 64;
  // a CTA of a pair holds its own 128 rows of A and its half of B's rows
  static constexpr uint32_t kStageA = BM * BK * 2, kStageB = kBN / kPair * BK * 2;
  static constexpr uint32_t kStageBytes = kStageA + kStageB;
  // epilogue units, or the sums that a shared tile's members sent
  static constexpr uint32_t kStaging = kShared ? BM * kSumLd * 4 : kEpiWarps * 32 * 128;
  static constexpr int kStages = (int)((226u * 1024u - 1024u - 512u - kStaging) / kStageBytes);
  static constexpr uint32_t kOffB = kStages * kStageA;
  static constexpr uint32_t kOffStaging = kOffB + kStages * kStageB;
  static constexpr uint32_t kOffBar = kOffStaging + kStaging;
  static constexpr uint32_t kOffMisc = kOffBar + (2 * kStages + 5) * 8;
  static constexpr uint32_t kSmem = kOffMisc + 16 + 1024;
  static constexpr int kThreads = 32 * (kEpiWarps + 2);
  static constexpr int kTmemCols = 2 * kBN;
};

// Elements m .. m + 7 (m < 8) of the sixteen in x and y: a shift in three steps
// of 4, 2 and 1 elements.
__device__ __forceinline__ uint4 shift8(const uint4& x, const uint4& y, int m) {
  const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
  uint32_t u[6], v[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) u[i] = (m & 4) ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = (m & 2) ? u[i + 1] : u[i];
  const int b = (m & 1) * 16;
  return make_uint4(__funnelshift_r(v[0], v[1], b), __funnelshift_r(v[1], v[2], b),
                    __funnelshift_r(v[2], v[3], b), __funnelshift_r(v[3], v[4], b));
}

// Eight 16-bit elements at any element offset of a 16-byte aligned array of
// `total`: the two aligned vectors around them, shifted together.  Near the end
// of the array one by one (zero beyond it).
__device__ __forceinline__ uint4 load8_any(const uint16_t* base, int64_t at, int64_t total) {
  const int m = (int)(at & 7);
  const int64_t a0 = at - m;
  if (a0 + 16 > total) {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (at + e < total) w[e / 2] |= (uint32_t)base[at + e] << (16 * (e % 2));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  const uint4* p = reinterpret_cast<const uint4*>(base + a0);
  return shift8(p[0], p[1], m);
}

// 32 x kUnit values of one warp in shared memory: row = lane, 16-byte pieces
// XOR-swizzled so that both the row-per-lane accesses and the row-piece-per-
// lane accesses are free of bank conflicts
template <int kRowBytes>
__device__ __forceinline__ int piece_at(int row, int piece) {
  return kRowBytes == 128 ? row * 128 + ((piece ^ (row & 7)) << 4)
                          : row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
}

struct RowMap {
  int64_t M, rows1, split;
  char* out;
  char* out2;
  int64_t row_bytes;
  __device__ __forceinline__ char* operator()(int64_t r) const {
    if (r >= M) return nullptr;
    if (r < rows1) return out + r * row_bytes;
    if (r < split) return nullptr;
    return out2 + (r - split) * row_bytes;
  }
};

// shared-memory unit -> global rows.  kEsz: bytes per element
template <int kRowBytes, int kEsz>
__device__ __forceinline__ void flush_unit(const unsigned char* stg, int lane, const RowMap& map,
                                           int64_t row0, int64_t col0, int64_t N, bool vec) {
  constexpr int kPieces = kRowBytes / 16;
  constexpr int kPer = 16 / kEsz;  // elements per piece
  if (vec) {  // whole pieces: N is a multiple of a piece
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int row = j * (32 / kPieces) + lane / kPieces, pc = lane % kPieces;
      char* dst = map(row0 + row);
      const int64_t c = col0 + pc * kPer;
      if (dst && c < N && LQ_IN_RANGE(c + kPer - 1, N))
        *reinterpret_cast<uint4*>(dst + c * kEsz) =
            *reinterpret_cast<const uint4*>(stg + piece_at<kRowBytes>(row, pc));
    }
    return;
  }
  if (kEsz != 2) return;  // float32 rows are whole pieces
  constexpr int kWords = kRowBytes / 4;
  const int64_t left = N - col0;  // columns of this unit that exist
  if (left >= 2 * kWords) {
    // Rows that start anywhere: the aligned 16-byte vectors inside the row's piece,
    // each shifted together from two, and the eight elements before and after them
    // one by one (1003 x 49155 x 2048: 148 us; with 4-byte words 183, with elements
    // 199; short series, in a long one the first takes 192).
#pragma unroll 4
    for (int j = 0; j < kPieces; ++j) {
      const int row = j * (32 / kPieces) + lane / kPieces, pc = lane % kPieces;
      char* dst = map(row0 + row);
      if (!dst) continue;
      uint16_t* d = reinterpret_cast<uint16_t*>(dst) + col0;
      const int s0 = (int)((16 - ((uintptr_t)d & 15)) & 15) / 2;  // first aligned element
      const uint4 x = *reinterpret_cast<const uint4*>(stg + piece_at<kRowBytes>(row, pc));
      const uint4 y = *reinterpret_cast<const uint4*>(
          stg + piece_at<kRowBytes>(row, min(pc + 1, kPieces - 1)));
      if ((s0 == 0 || pc < kPieces - 1) && LQ_IN_RANGE(col0 + s0 + 8 * pc + 7, N))
        *reinterpret_cast<uint4*>(d + s0 + 8 * pc) = shift8(x, y, s0);
      if (s0 != 0) {
#pragma unroll
        for (int h = 0; h < 8; h += kPieces) {
          const int e = pc + h < s0 ? pc + h : 2 * kWords - 8 + pc + h;
          if (LQ_IN_RANGE(col0 + e, N))
            d[e] = *reinterpret_cast<const uint16_t*>(stg + piece_at<kRowBytes>(row, e / 8) +
                                                      (e % 8) * 2);
        }
      }
    }
    return;
  }
  // The row's last piece: lane l holds the word of elements 2l and 2l + 1.  Where
  // the row starts inside a 4-byte word the words are shifted by one element, and
  // the first and the last element go alone.
  const int n = left < 2 * kWords ? (int)left : 2 * kWords;
#pragma unroll 8
  for (int row = 0; row < 32; ++row) {
    uint32_t w = 0;
    if (lane < kWords)
      w = *reinterpret_cast<const uint32_t*>(stg + piece_at<kRowBytes>(row, lane / 4) +
                                             (lane % 4) * 4);
    const uint32_t next = __shfl_down_sync(~0u, w, 1);
    char* dst = map(row0 + row);
    if (!dst) continue;
    uint16_t* d = reinterpret_cast<uint16_t*>(dst) + col0;
    const int odd = ((uintptr_t)d & 2) ? 1 : 0;
    const int e = 2 * lane + odd;  // first element of this lane's word
    if (odd) w = __funnelshift_r(w, next, 16);
    if (e + 1 < n && LQ_IN_RANGE(col0 + e + 1, N)) *reinterpret_cast<uint32_t*>(d + e) = w;
    // what no whole word covers: the first element, and the last where one is left
    const int tail = (n - odd) & 1;
    if (lane == 0 && odd && LQ_IN_RANGE(col0, N))
      d[0] = *reinterpret_cast<const uint16_t*>(stg + piece_at<kRowBytes>(row, 0));
    if (lane == 1 && tail && LQ_IN_RANGE(col0 + n - 1, N))
      d[n - 1] = *reinterpret_cast<const uint16_t*>(
          stg + piece_at<kRowBytes>(row, (n - 1) / 8) + ((n - 1) % 8) * 2);
  }
}

// A unit of 16-bit elements of global rows, in two steps: the loads, which may
// travel while something else is done, and their pieces put into shared memory.
// Where rows start anywhere the loads take the aligned vectors around the unit,
// one more per row (lane l holds that of row l), and are shifted into place in
// the second step; what they hold beyond the row's end is not stored.
template <int kRowBytes>
struct UnitLoad {
  static constexpr int kPieces = kRowBytes / 16;
  uint4 v[kPieces], ext;
  // the aligned vector at element a; beyond the end of the array zero
  static __device__ __forceinline__ uint4 vector_at(const uint16_t* src, int64_t a, int64_t total) {
    if (a + 8 <= total) return *reinterpret_cast<const uint4*>(src + a);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (a + e < total) w[e / 2] |= (uint32_t)src[a + e] << (16 * (e % 2));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void load(int lane, const uint16_t* src, int64_t ld, int64_t row0,
                                       int64_t col0, int64_t M, int64_t N, bool vec) {
    const int64_t total = M * ld;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int64_t r = row0 + j * (32 / kPieces) + lane / kPieces;
      const int64_t c = col0 + (lane % kPieces) * 8;
      v[j] = make_uint4(0, 0, 0, 0);
      if (r >= M) continue;
      if (vec) {
        if (c < N) v[j] = *reinterpret_cast<const uint4*>(src + r * ld + c);
      } else {
        v[j] = vector_at(src, (r * ld + c) & ~(int64_t)7, total);
      }
    }
    ext = make_uint4(0, 0, 0, 0);
    if (!vec && row0 + lane < M)
      ext = vector_at(src, ((row0 + lane) * ld + col0 + kPieces * 8) & ~(int64_t)7, total);
  }
  __device__ __forceinline__ void put(unsigned char* stg, int lane, int64_t ld, int64_t row0,
                                      int64_t col0, bool vec) const {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int row = j * (32 / kPieces) + lane / kPieces, pc = lane % kPieces;
      uint4 x = v[j];
      if (!vec) {
        uint4 y;
        y.x = __shfl_down_sync(~0u, x.x, 1), y.y = __shfl_down_sync(~0u, x.y, 1);
        y.z = __shfl_down_sync(~0u, x.z, 1), y.w = __shfl_down_sync(~0u, x.w, 1);
        const uint32_t e0 = __shfl_sync(~0u, ext.x, row), e1 = __shfl_sync(~0u, ext.y, row),
                       e2 = __shfl_sync(~0u, ext.z, row), e3 = __shfl_sync(~0u, ext.w, row);
        if (pc == kPieces - 1) y = make_uint4(e0, e1, e2, e3);
        x = shift8(x, y, (int)(((row0 + row) * ld + col0) & 7));
      }
      *reinterpret_cast<uint4*>(stg + piece_at<kRowBytes>(row, pc)) = x;
    }
  }
};

// v[i] += the bias that lane i holds
__device__ __forceinline__ void add_bias(float (&v)[32], float own) {
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(~0u, own, i);
}

template <typename T, int kRowBytes>
__device__ __forceinline__ void put_row(unsigned char* stg, int lane, int c0, const float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 w;
    w.x = Elem<T>::pack(v[8 * i], v[8 * i + 1]);
    w.y = Elem<T>::pack(v[8 * i + 2], v[8 * i + 3]);
    w.z = Elem<T>::pack(v[8 * i + 4], v[8 * i + 5]);
    w.w = Elem<T>::pack(v[8 * i + 6], v[8 * i + 7]);
    *reinterpret_cast<uint4*>(stg + piece_at<kRowBytes>(lane, c0 / 8 + i)) = w;
  }
}

template <typename T, int kRowBytes>
__device__ __forceinline__ void add_row(const unsigned char* stg, int lane, int c0,
                                        float (&v)[32]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(stg + piece_at<kRowBytes>(lane, c0 / 8 + i));
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = Elem<T>::unpack(q[e]);
      v[8 * i + 2 * e] += f.x;
      v[8 * i + 2 * e + 1] += f.y;
    }
  }
}

__device__ __forceinline__ void load_acc(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld_32x32b_x32(taddr, r);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// tile t -> (tile row, tile column): bands of 16 tile rows, column by column
// inside a band, so that the tiles in flight share operand rows and columns
__device__ __forceinline__ void tile_at(int t, int tm, int tn, int& im, int& in) {
  const int band = t / (16 * tn), first = band * 16;
  const int h = min(16, tm - first), r = t - band * 16 * tn;
  im = first + r % h;
  in = r / h;
}

// Eight values of an output row at column c, each rounded once.
template <typename T>
__device__ __forceinline__ void store8(uint16_t* row, int64_t c, int64_t N, bool vec,
                                       const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = Elem<T>::pack(v[2 * i], v[2 * i + 1]);
  if (vec) {
    if (LQ_IN_RANGE(c + 7, N))
      *reinterpret_cast<uint4*>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < N && LQ_IN_RANGE(c + e, N)) row[c + e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
}

// The elements at p[c] .. p[c + 7] that lie below n, zero beyond.
__device__ __forceinline__ uint4 load8(const uint16_t* p, int64_t c, int64_t n, bool vec) {
  if (vec) return *reinterpret_cast<const uint4*>(p + c);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < n) w[e / 2] |= (uint32_t)p[c + e] << (16 * (e % 2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ void add8(const uint4& w, float (&v)[8]) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = Elem<T>::unpack(q[i]);
    v[2 * i] += f.x, v[2 * i + 1] += f.y;
  }
}

// The end of a shared tile.  Member m of the cluster finishes the tile's m-th block
// of BM / members rows: the other members send it their sums of those rows, and it
// adds the parts in the members' order, eight columns a thread.  Bias and residual
// are read while the products are under way.
template <typename T, int kEpi>
struct SharedTile {
  static constexpr int kPieces = (kEpi == kEpiGated ? 32 : 64) / 8;
  static constexpr int kStep = 128 / kPieces;
  static constexpr int kMax = BM / 2 / kStep;  // pieces of a thread, two members
  int block;              // rows of a member's block
  int64_t row_first;      // first row of this member's block
  int rows;               // rows of the block that exist
  int64_t col;
  bool live;
  uint4 bias, bias2, res[kMax];

  __device__ __forceinline__ void load(const GemmParams& P, int member, int64_t row0,
                                       int64_t col0) {
    block = BM / P.members;
    row_first = row0 + member * block;
    rows = (int)max((int64_t)0, min((int64_t)block, P.M - row_first));
    col = col0 + threadIdx.x % kPieces * 8;
    live = col < P.N;
    bias = bias2 = make_uint4(0, 0, 0, 0);
    if (kEpi == kEpiStore || !live) return;
    if (P.bias) bias = load8(P.bias, col, P.N, P.vec);
    if (kEpi == kEpiGated && P.bias2) bias2 = load8(P.bias2, col, P.N, P.vec);
    if (kEpi == kEpiDense && P.res) {
#pragma unroll
      for (int i = 0; i < kMax; ++i) {
        const int r = threadIdx.x / kPieces + i * kStep;
        if (r < rows) res[i] = load8(P.res + (row_first + r) * P.ldo, col, P.N, P.vec);
      }
    }
  }

  // row `row` of this member's sums, 32 columns from c on, to the row's owner
  __device__ __forceinline__ void send(uint32_t sums, int member, int row, int c,
                                       const float (&v)[32]) const {
    const uint32_t dst = in_cta(
        sums + ((member * block + row % block) * kSumLd + c) * 4, (uint32_t)(row / block));
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 16 * i),
                   "f"(v[4 * i]), "f"(v[4 * i + 1]), "f"(v[4 * i + 2]), "f"(v[4 * i + 3])
                   : "memory");
  }

  __device__ __forceinline__ void finish(const float* sums, const GemmParams& P) const {
    if (!live) return;
#pragma unroll
    for (int i = 0; i < kMax; ++i) {
      const int r = threadIdx.x / kPieces + i * kStep;
      if (r >= rows) break;
      float v[8] = {}, w[8] = {};
      for (int m = 0; m < P.members; ++m) {
        const float4* p = reinterpret_cast<const float4*>(sums + (m * block + r) * kSumLd +
                                                          threadIdx.x % kPieces * 8);
        const float4 x = p[0], y = p[1];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
        v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
        if (kEpi == kEpiGated) {
          const float4 g = p[8], h = p[9];
          w[0] += g.x, w[1] += g.y, w[2] += g.z, w[3] += g.w;
          w[4] += h.x, w[5] += h.y, w[6] += h.z, w[7] += h.w;
        }
      }
      const int64_t at = (row_first + r) * P.ldo;
      if (kEpi != kEpiStore) {
        if (P.bias) add8<T>(bias, v);
        if (kEpi == kEpiGated && P.bias2) add8<T>(bias2, w);
        if (P.aux) store8<T>(P.aux + at, col, P.N, P.vec, v);
        if (kEpi == kEpiGated && P.aux) store8<T>(P.aux2 + at, col, P.N, P.vec, w);
        apply_act(P.act, v);
        if (kEpi == kEpiGated) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= w[e];
        } else if (P.res) {
          add8<T>(res[i], v);
        }
      }
      store8<T>((uint16_t*)P.out + at, col, P.N, P.vec, v);
    }
  }
};

// kShared: the CTAs of a cluster share one tile, each a part of the contraction
// (gridDim.x: clusters of P.members CTAs, one tile each).
template <typename T, int kBN, int kPair, bool kAMn, bool kBMn, int kEpi, bool kShared>
__global__ void __launch_bounds__(Cfg<kBN, kPair, kEpi, kShared>::kThreads, 1)
    k_dense_gemm(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmA2,
                 const __grid_constant__ CUtensorMap tmB, const __grid_constant__ CUtensorMap tmB2,
                 const __grid_constant__ GemmParams P) {
  using C = Cfg<kBN, kPair, kEpi, kShared>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  unsigned char* gbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar_full = base + C::kOffBar;
  const uint32_t bar_empty = bar_full + C::kStages * 8;
  const uint32_t bar_accf = bar_empty + C::kStages * 8;
  const uint32_t bar_acce = bar_accf + 2 * 8;
  const uint32_t bar_drain = bar_acce + 2 * 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + C::kOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + C::kOffMisc + 4);
  constexpr int kTileN = kEpi == kEpiGated ? kBN / 2 : kBN;  // output columns of a tile
  constexpr int kTileM = BM * kPair;
  const int tm = (int)((P.M + kTileM - 1) / kTileM), tn = (int)((P.N + kTileN - 1) / kTileN);
  const int n_tiles = tm * tn;
  const int rank = kPair == 1 ? 0 : (int)cluster_rank();
  static_assert(!kShared || (kPair == 1 && kBN == 64 && kEpi != kEpiF32), "");
  const int ctas = kShared ? P.members : kPair;  // CTAs that work on one tile
  const int member = kShared ? (int)cluster_rank() : 0;
  const int t_first = blockIdx.x / ctas, t_step = gridDim.x / ctas;
  const int kb_first = (kShared ? member : (int)blockIdx.y) * P.slice_kb, kb_end = min(P.n_kb, kb_first + P.slice_kb);

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_accf + 8 * b, 1);
      mbar_init(bar_acce + 8 * b, C::kEpiWarps * kPair);
    }
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_take<kPair>(smem_u32(tmem_slot), C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  if (kPair == 2) cluster_sync_all();  // both CTAs' barriers are set up
  if (kShared) cluster_arrive();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();  // everything below reads or writes global memory
  SharedTile<T, kEpi> shared;

  if (warp == C::kEpiWarps) {
    // ---- TMA producer: one lane runs the whole loop
    if (elect_one()) {
      int it = 0, st = 0;
      uint32_t ph = 1u;  // parity to wait for: the ring starts out empty
      bool ok = true;
      for (int t = t_first; t < n_tiles && ok; t += t_step) {
        int im, in;
        tile_at(t, tm, tn, im, in);
        const int m0 = im * kTileM + rank * BM;
        const int n0 = in * kTileN + (kEpi == kEpiGated ? 0 : rank * (kBN / kPair));
        for (int kb = kb_first; kb < kb_end; ++kb, ++it) {
          if (!wait_bounded(bar_empty + 8 * st, ph, abort_flag)) {
            ok = false;
            break;
          }
          const bool first = kb < P.n_kb1;
          const CUtensorMap* a = first ? &tmA : &tmA2;
          const CUtensorMap* b = first ? &tmB : &tmB2;
          const int k0 = (first ? kb : kb - P.n_kb1) * BK;
          // a stage is full once the bytes of both CTAs have arrived at the
          // first one's barrier, where the MMAs are issued
          const uint32_t full = kPair == 1 ? bar_full + 8 * st : in_first_cta(bar_full + 8 * st);
          const uint32_t sa = base + st * C::kStageA, sb = base + C::kOffB + st * C::kStageB;
          if (rank == 0) mbar_arrive_expect_tx(bar_full + 8 * st, C::kStageBytes * kPair);
          if (kAMn) {
#pragma unroll
            for (int c = 0; c < BM / 64; ++c)
              load_tile<kPair>(sa + c * 8192, a, full, m0 + 64 * c, k0);
          } else {
            load_tile<kPair>(sa, a, full, k0, m0);
          }
          if (kBMn) {
#pragma unroll
            for (int c = 0; c < kBN / kPair / 64; ++c)
              load_tile<kPair>(sb + c * 8192, b, full, n0 + 64 * c, k0);
          } else if (kEpi == kEpiGated && kPair == 2) {
            // the first CTA holds the gate's rows of B, the second the up ones
            load_tile<kPair>(sb, rank == 0 ? &tmB : &tmB2, full, k0, n0);
          } else if (kEpi == kEpiGated) {
            load_tile<kPair>(sb, &tmB, full, k0, n0);
            load_tile<kPair>(sb + C::kStageB / 2, &tmB2, full, k0, n0);
          } else {
            load_tile<kPair>(sb, b, full, k0, n0);
          }
          if (++st == C::kStages) st = 0, ph ^= 1u;
        }
      }
      // no copy is in flight when the CTA leaves
      if (rank == 0)
        for (int i = max(0, it - C::kStages); i < it; ++i)
          wait_drain(bar_full + 8 * (i % C::kStages), (uint32_t)(i / C::kStages) & 1u);
    }
  } else if (warp == C::kEpiWarps + 1) {
    // ---- MMA issuer (of a pair: the first CTA's, for both): one lane
    if (rank == 0 && elect_one()) {
      constexpr uint32_t idesc = instr_desc(Elem<T>::kFormat, kAMn, kBMn, kTileM, kBN);
      // descriptor units (16 bytes) between consecutive 16-wide contraction steps
      constexpr uint64_t stepA = (kAMn ? 2048u : 32u) >> 4, stepB = (kBMn ? 2048u : 32u) >> 4;
      const uint64_t descA = smem_desc(base, kAMn), descB = smem_desc(base + C::kOffB, kBMn);
      int st = 0, j = 0;
      uint32_t ph = 0u;
      bool ok = true;
      for (int t = t_first; t < n_tiles && ok; t += t_step, ++j) {
        const int buf = j & 1;
        if (!wait_bounded(bar_acce + 8 * buf, ((uint32_t)(j >> 1) & 1u) ^ 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(buf * kBN);
        for (int kb = kb_first; kb < kb_end; ++kb) {
          if (!wait_bounded(bar_full + 8 * st, ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t da = descA + (uint64_t)(st * (C::kStageA >> 4));
          const uint64_t db = descB + (uint64_t)(st * (C::kStageB >> 4));
#pragma unroll
          for (int i = 0; i < BK / 16; ++i)
            umma_f16<kPair>(d, da + stepA * i, db + stepB * i, idesc,
                            (kb != kb_first || i != 0) ? 1u : 0u);
          commit_all<kPair>(bar_empty + 8 * st);
          if (++st == C::kStages) st = 0, ph ^= 1u;
        }
        if (ok) commit_all<kPair>(bar_accf + 8 * buf);
      }
      commit_all<kPair>(bar_drain);
      wait_drain(bar_drain, 0u);
    }
  } else if (kShared) {
    // ---- epilogue of a shared tile: send the sums
    int im, in;
    tile_at(t_first, tm, tn, im, in);
    shared.load(P, member, (int64_t)im * kTileM, (int64_t)in * kTileN);
    const bool ok = wait_warp(bar_accf, 0u, abort_flag);
    cluster_wait();  // every member runs, so that its shared memory may be written
    if (ok && (int64_t)im * kTileM + 32 * warp < P.M) {
      tc_fence_after();
      for (int c = 0; c < kBN; c += 32) {
        float v[32];
        load_acc(tmem_base + ((uint32_t)(32 * warp) << 16) + c, v);
        shared.send(base + C::kOffStaging, member, 32 * warp + lane, c, v);
      }
    }
  } else {
    // ---- epilogue: warp w reads TMEM lanes 32 (w % 4).. and column part w / 4
    const int q = warp & 3, part = warp >> 2;
    unsigned char* stg = gbase + C::kOffStaging + warp * 4096;
    constexpr int kRowBytes = C::kUnit * (kEpi == kEpiF32 ? 4 : 2);
    constexpr int kParts = C::kCols / 32;  // 32-column parts of this warp
    int j = 0;
    for (int t = t_first; t < n_tiles; t += t_step, ++j) {
      int im, in;
      tile_at(t, tm, tn, im, in);
      const int buf = j & 1;
      const int64_t row0 = (int64_t)im * kTileM + rank * BM + 32 * q;
      const int64_t n0 = (int64_t)in * kTileN + part * C::kCols;  // this warp's first column
      const bool live = row0 < P.M;
      // while the products are under way: the bias (lane l holds column l of every
      // part) and the first unit of the residual
      float own[kParts], own2[kParts];
      UnitLoad<kRowBytes> res;
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const int64_t c = n0 + 32 * k + lane;
        own[k] = (kEpi == kEpiDense || kEpi == kEpiGated) && P.bias && c < P.N
                     ? Elem<T>::load(P.bias + c) : 0.f;
        own2[k] = kEpi == kEpiGated && P.bias2 && c < P.N ? Elem<T>::load(P.bias2 + c) : 0.f;
      }
      if (kEpi == kEpiDense && P.res && live)
        res.load(lane, P.res, P.ldo, row0, n0, P.M, P.N, P.vec);
      auto of_part = [&](const float (&o)[kParts], int k) {
        float b = o[0];
#pragma unroll
        for (int i = 1; i < kParts; ++i) b = k == i ? o[i] : b;
        return b;
      };
      if (!wait_warp(bar_accf + 8 * buf, (uint32_t)(j >> 1) & 1u, abort_flag)) break;
      tc_fence_after();
      const uint32_t acc = tmem_base + ((uint32_t)(32 * q) << 16) +
                           (uint32_t)(buf * kBN + part * C::kCols);
      const RowMap map = {P.M, P.rows1, P.split, (char*)P.out + blockIdx.y * P.slice_bytes,
                          (char*)P.out2, P.ldo * (kEpi == kEpiF32 ? 4 : 2)};
      for (int u = 0; u < C::kCols; u += C::kUnit) {
        const int64_t col = n0 + u;
        if (!live || col >= P.N) continue;
        // accumulator columns of this warp from u + c on, with the bias
        auto take = [&](int c, float (&v)[32]) {
          load_acc(acc + u + c, v);
          if ((kEpi == kEpiDense || kEpi == kEpiGated) && P.bias)
            add_bias(v, of_part(own, (u + c) / 32));
        };
        auto take_up = [&](int c, float (&v)[32]) {
          load_acc(acc + kTileN + u + c, v);
          if (P.bias2) add_bias(v, of_part(own2, (u + c) / 32));
        };
        if ((kEpi == kEpiDense || kEpi == kEpiGated) && P.aux) {
          // what the backward pass reads
          for (int f = 0; f < (kEpi == kEpiGated ? 2 : 1); ++f) {
            for (int c = 0; c < C::kUnit; c += 32) {
              float v[32];
              if (f)
                take_up(c, v);
              else
                take(c, v);
              put_row<T, kRowBytes>(stg, lane, c, v);
            }
            __syncwarp();
            const RowMap za = {P.M, P.M, P.M, (char*)(f ? P.aux2 : P.aux), nullptr, P.ldo * 2};
            flush_unit<kRowBytes, 2>(stg, lane, za, row0, col, P.N, P.vec);
            __syncwarp();
          }
        }
        if (kEpi == kEpiDense && P.res) {
          res.put(stg, lane, P.ldo, row0, col, P.vec);
          __syncwarp();
          if (u + C::kUnit < C::kCols)
            res.load(lane, P.res, P.ldo, row0, col + C::kUnit, P.M, P.N, P.vec);
        }
        for (int c = 0; c < C::kUnit; c += 32) {
          float v[32];
          take(c, v);
          if (kEpi == kEpiDense) {
            apply_act(P.act, v);
            if (P.res) add_row<T, kRowBytes>(stg, lane, c, v);
          }
          if (kEpi == kEpiGated) {
            apply_act(P.act, v);
            float w[32];
            take_up(c, w);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= w[i];
          }
          if (kEpi == kEpiF32) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(stg + piece_at<128>(lane, i)) =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
            put_row<T, kRowBytes>(stg, lane, c, v);
          }
        }
        __syncwarp();
        if (kEpi == kEpiF32) {
          if (P.accumulate) {
            // each lane adds its own pieces of what is there
            for (int row = 0; row < 32; ++row) {
              const char* src = map(row0 + row);
              if (src && col + lane < P.N) {
                float* p = reinterpret_cast<float*>(stg + piece_at<128>(row, lane / 4)) + lane % 4;
                *p += reinterpret_cast<const float*>(src)[col + lane];
              }
            }
            __syncwarp();
          }
          flush_unit<kRowBytes, 4>(stg, lane, map, row0, col, P.N, P.vec);
        } else {
          flush_unit<kRowBytes, 2>(stg, lane, map, row0, col, P.N, P.vec);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (kPair == 1)
          mbar_arrive(bar_acce + 8 * buf);
        else
          arrive_cluster(in_first_cta(bar_acce + 8 * buf));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other's copies, MMAs or arrivals may still
  // reach its shared memory
  if (kPair == 2) cluster_sync_all();
  if (kShared) {
    if (warp >= C::kEpiWarps) cluster_wait();
    cluster_sync_all();  // all sums have arrived; no member writes another's memory now
    if (warp < C::kEpiWarps)
      shared.finish(reinterpret_cast<const float*>(gbase + C::kOffStaging), P);
    __syncwarp();
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_free<kPair>(tmem_base, C::kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// up to 16 rows: stream the weights
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1, bool bf16) {
  if (bf16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct RowsParams {
  const uint16_t* x;
  const uint16_t* w;
  const uint16_t* w2;
  const uint16_t* bias;
  const uint16_t* bias2;
  const uint16_t* res;
  uint16_t* y;
  uint16_t* aux;
  uint16_t* aux2;
  int M, N, K, act;
};

constexpr int kRowsUnroll = 4;

// A block owns 16 weight rows (of each factor when gated); its warps take
// 32-wide contraction blocks in turn.  The contraction order inside a 32-wide
// block is permuted so that every operand load is one 16-byte vector: lane
// (g, t) holds elements 8t..8t+7 of weight rows g and g + 8 and of token g,
// and calls the first four "k = 2t, 2t+1, 2t+8, 2t+9" of a first MMA, the
// others of a second; both operands use the same permutation, so the sum is
// unchanged.  The warps' partial sums are added in shared memory in warp order.
template <typename T, int kNT, bool kGated, int kRowsWarps>
__global__ void __launch_bounds__(32 * kRowsWarps) k_dense_rows(const RowsParams P) {
  constexpr int kF = kGated ? 2 : 1;
  constexpr bool kBf16 = Elem<T>::kFormat == 1;
  __shared__ float part[kRowsWarps][kF][16][8 * kNT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * 16;
  pdl_trigger();
  pdl_wait();
  float acc[kF][kNT][4];
#pragma unroll
  for (int f = 0; f < kF; ++f)
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[f][j][i] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int n_blk = (P.K + 31) / 32;
  for (int b0 = warp; b0 < n_blk; b0 += kRowsWarps * kRowsUnroll) {
    uint4 a[kRowsUnroll][kF][2], xb[kRowsUnroll][kNT];
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u) {
      // up to 48 blocks past the last one, which may pass 2^31: compared unsigned
      const int k = (int)((uint32_t)(b0 + u * kRowsWarps) * 32u) + 8 * t;
      const bool in = (uint32_t)k < (uint32_t)P.K;  // K is a multiple of 8
#pragma unroll
      for (int f = 0; f < kF; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = n0 + g + 8 * h;
          a[u][f][h] = zero;
          if (in && n < P.N)
            a[u][f][h] =
                __ldg(reinterpret_cast<const uint4*>((f ? P.w2 : P.w) + (int64_t)n * P.K + k));
        }
#pragma unroll
      for (int j = 0; j < kNT; ++j) {
        const int m = 8 * j + g;
        xb[u][j] = zero;
        if (in && m < P.M)
          xb[u][j] = __ldg(reinterpret_cast<const uint4*>(P.x + (int64_t)m * P.K + k));
      }
    }
#pragma unroll
    for (int u = 0; u < kRowsUnroll; ++u)
#pragma unroll
      for (int f = 0; f < kF; ++f)
#pragma unroll
        for (int j = 0; j < kNT; ++j) {
          const uint4 p = a[u][f][0], r = a[u][f][1], c = xb[u][j];
          mma_16x8x16(acc[f][j], p.x, r.x, p.y, r.y, c.x, c.y, kBf16);
          mma_16x8x16(acc[f][j], p.z, r.z, p.w, r.w, c.z, c.w, kBf16);
        }
  }
#pragma unroll
  for (int f = 0; f < kF; ++f)
#pragma unroll
    for (int j = 0; j < kNT; ++j) {
      float(*p)[8 * kNT + 1] = part[warp][f];
      p[g][8 * j + 2 * t] = acc[f][j][0];
      p[g][8 * j + 2 * t + 1] = acc[f][j][1];
      p[g + 8][8 * j + 2 * t] = acc[f][j][2];
      p[g + 8][8 * j + 2 * t + 1] = acc[f][j][3];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 16 * 8 * kNT; i += 32 * kRowsWarps) {
    const int r = i % 16, m = i / 16, n = n0 + r;
    if (n >= P.N || m >= P.M) continue;
    float v[1] = {0.f}, s2 = 0.f;
#pragma unroll
    for (int w = 0; w < kRowsWarps; ++w) {
      v[0] += part[w][0][r][m];
      if (kGated) s2 += part[w][kF - 1][r][m];
    }
    const int64_t o = (int64_t)m * P.N + n;
    if (P.bias) v[0] += Elem<T>::load(P.bias + n);
    const bool ok = LQ_IN_RANGE(o, (int64_t)P.M * P.N);
    if (P.aux && ok) P.aux[o] = Elem<T>::round(v[0]);
    apply_act(P.act, v);
    if (kGated) {
      if (P.bias2) s2 += Elem<T>::load(P.bias2 + n);
      if (P.aux2 && ok) P.aux2[o] = Elem<T>::round(s2);
      v[0] *= s2;
    } else if (P.res) {
      v[0] += Elem<T>::load(P.res + o);
    }
    if (ok) P.y[o] = Elem<T>::round(v[0]);
  }
}

// ---------------------------------------------------------------------------
// dz from the output gradient, and the column sums of dz
// ---------------------------------------------------------------------------
struct GradParams {
  const uint16_t* dy;
  const uint16_t* z;   // gate (or only) pre-activation; null: no activation
  const uint16_t* u;   // up factor (gated)
  uint16_t* dz;        // M x ldz, null: not wanted (sums only)
  float* sums;         // row blocks x (factors * N) partial column sums, or null
  int64_t M, N, ldz;   // gated: du starts at column ldz / 2
  int64_t rows;        // rows per row block
  int act;
};

template <typename T>
__device__ __forceinline__ void unpack_vec(const uint4& w, float (&f)[8]) {
  const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 v = Elem<T>::unpack(q[e]);
    f[2 * e] = v.x;
    f[2 * e + 1] = v.y;
  }
}
// A block covers 256 columns of one row block: a thread owns eight neighbouring
// columns and every 8th row, keeps their float32 sums in registers, and the eight
// row groups are added in shared memory in order.  kWhole: rows start on 16-byte
// boundaries (N a multiple of 8).  Bound by memory: 4096 x 5632 gated, 231 MB in 40
// us, 88 % of HBM.
template <typename T, bool kWhole, bool kGated, int kAct>
__global__ void __launch_bounds__(256) k_act_grad(const GradParams P) {
  constexpr int kF = kGated ? 2 : 1, kVec = 8;
  __shared__ float red[8][kF][32 * kVec];
  const int lane = threadIdx.x & 31, rg = threadIdx.x >> 5;
  const int64_t half = kGated ? P.ldz / 2 : P.ldz;
  const int64_t c0 = ((int64_t)blockIdx.x * 32 + lane) * kVec;
  const int64_t r0 = (int64_t)blockIdx.y * P.rows, r1 = min(P.M, r0 + P.rows);
  pdl_trigger();
  pdl_wait();
  float sum[kF][kVec];
#pragma unroll
  for (int f = 0; f < kF; ++f)
#pragma unroll
    for (int i = 0; i < kVec; ++i) sum[f][i] = 0.f;
  if (c0 < half) {
    const bool in = c0 < P.N;
    constexpr int kRows = 4;  // rows whose loads travel together
    const int64_t total = P.M * P.N;
    for (int64_t rb = r0 + rg; rb < r1; rb += 8 * kRows) {
      uint4 la[kRows], lb[kRows], lc[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int64_t r = rb + 8 * j, at = r * P.N + c0;
        la[j] = lb[j] = lc[j] = make_uint4(0, 0, 0, 0);
        if (in && r < r1) {
          auto load = [&](const uint16_t* p) {
            return kWhole ? __ldg(reinterpret_cast<const uint4*>(p + at)) : load8_any(p, at, total);
          };
          la[j] = load(P.dy);
          if (kAct != LQ_ACT_NONE || kGated) lb[j] = load(P.z);
          if (kGated) lc[j] = load(P.u);
        }
      }
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int64_t r = rb + 8 * j;
        if (r >= r1) break;
        float dy[kVec], z[kVec], u[kVec], o[kF][kVec];
        unpack_vec<T>(la[j], dy);
        unpack_vec<T>(lb[j], z);
        unpack_vec<T>(lc[j], u);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          float a, da;
          act_grad<kAct>(z[i], a, da);
          o[0][i] = kGated ? dy[i] * u[i] * da : dy[i] * da;
          if (kGated) o[kF - 1][i] = dy[i] * a;
          // columns past N are padding of the contraction: exactly zero
          if (kWhole ? !in : c0 + i >= P.N) o[0][i] = o[kF - 1][i] = 0.f;
        }
#pragma unroll
        for (int f = 0; f < kF; ++f) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) sum[f][i] += o[f][i];
          if (P.dz) {
            uint16_t* dst = P.dz + r * P.ldz + f * half + c0;
            uint4 w;
            w.x = Elem<T>::pack(o[f][0], o[f][1]);
            w.y = Elem<T>::pack(o[f][2], o[f][3]);
            w.z = Elem<T>::pack(o[f][4], o[f][5]);
            w.w = Elem<T>::pack(o[f][6], o[f][7]);
            if (LQ_IN_RANGE(dst + 7 - P.dz, P.M * P.ldz)) *reinterpret_cast<uint4*>(dst) = w;
          }
        }
      }
    }
  }
  if (!P.sums) return;
#pragma unroll
  for (int f = 0; f < kF; ++f)
#pragma unroll
    for (int i = 0; i < kVec; ++i) red[rg][f][lane * kVec + i] = sum[f][i];
  __syncthreads();
  for (int i = threadIdx.x; i < kF * 32 * kVec; i += 256) {
    const int f = i / (32 * kVec), c = i % (32 * kVec);
    const int64_t col = (int64_t)blockIdx.x * 32 * kVec + c;
    if (col >= P.N) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += red[k][f][c];
    const int64_t at = ((int64_t)blockIdx.y * kF + f) * P.N + col;
    if (LQ_IN_RANGE(at, (int64_t)gridDim.y * kF * P.N)) P.sums[at] = s;
  }
}

// the row blocks' partial sums, added in order
template <typename T>
__global__ void __launch_bounds__(256) k_col_sums(const float* __restrict__ sums, int64_t N, int nf,
                                                  int blocks, void* out, void* out2, int f32,
                                                  int accumulate) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  pdl_trigger();
  pdl_wait();
  if (c >= N * nf) return;
  float s = 0.f;
  for (int b = 0; b < blocks; ++b) s += sums[(int64_t)b * nf * N + c];
  void* o = c < N ? out : out2;
  if (!o) return;
  const int64_t i = c < N ? c : c - N;
  if (!LQ_IN_RANGE(i, N)) return;
  if (f32)
    ((float*)o)[i] = accumulate ? ((float*)o)[i] + s : s;
  else
    ((uint16_t*)o)[i] = Elem<T>::round(s);
}

// the slices of a product added up, in order: rows x cols float32 each, to
// float32 (added to what is there) or rounded; rows as in GemmParams
template <typename T>
__global__ void __launch_bounds__(256)
    k_add_slices(const float* __restrict__ part, int slices, int64_t rows, int64_t cols,
                 const GemmParams P, int f32) {
  pdl_trigger();
  pdl_wait();
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;  // cols is a multiple of 8
  if (i >= rows * cols) return;
  const int64_t r = i / cols, c = i - r * cols;
  const RowMap map = {P.M, P.rows1, P.split, (char*)P.out, (char*)P.out2, cols * (f32 ? 4 : 2)};
  char* dst = map(r);
  if (!dst || !LQ_IN_RANGE(c + 3, cols)) return;
  float4 v = *reinterpret_cast<const float4*>(part + i);
  for (int k = 1; k < slices; ++k) {
    const float4 q = *reinterpret_cast<const float4*>(part + k * rows * cols + i);
    v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
  }
  if (f32) {
    float4* o = reinterpret_cast<float4*>(dst + c * 4);
    if (P.accumulate) {
      const float4 q = *o;
      v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
    }
    *o = v;
  } else {
    *reinterpret_cast<uint2*>(dst + c * 2) =
        make_uint2(Elem<T>::pack(v.x, v.y), Elem<T>::pack(v.z, v.w));
  }
}

// ---------------------------------------------------------------------------
// backward pass of up to 4 rows: stream the weights once for dx, write the
// weights' gradients once, dz in float32 throughout.  Measured at 5632 x 2048 (dx
// and dw): 4 rows 15 + 6 us against 16 + 12 of the tiles with their dz pass, 16
// rows 39 + 20, where the products outgrow the FMA units.
// ---------------------------------------------------------------------------
struct RowsBwdParams {
  const uint16_t* dy;
  const uint16_t* z;  // gate (or only) pre-activation
  const uint16_t* u;  // up factor (gated)
  const uint16_t* x;
  const uint16_t* w;
  const uint16_t* w2;
  uint16_t* dx;
  void* dw;
  void* dw2;
  void* db;
  void* db2;
  int M, N, K, act, f32, accumulate;
};

constexpr int kBwdRowsMax = 4;  // tokens up to which these kernels run
constexpr int kBwdRows = 64;   // weight rows a block works on at a time
constexpr int kBwdSplit = 8;   // CTAs of a cluster that share the weight rows of dx
constexpr int kBwdCols = 128;  // columns of dx per cluster

__device__ __forceinline__ void act_grad_any(int act, float z, float& a, float& da) {
  switch (act) {
    case LQ_ACT_RELU: act_grad<LQ_ACT_RELU>(z, a, da); break;
    case LQ_ACT_SILU: act_grad<LQ_ACT_SILU>(z, a, da); break;
    case LQ_ACT_GELU: act_grad<LQ_ACT_GELU>(z, a, da); break;
    case LQ_ACT_GELU_TANH: act_grad<LQ_ACT_GELU_TANH>(z, a, da); break;
    default: act_grad<LQ_ACT_NONE>(z, a, da); break;
  }
}

// dz of weight rows n0 .. n0 + 63 for all tokens (zero beyond the matrix)
template <typename T, int kM, bool kGated>
__device__ __forceinline__ void rows_dz(const RowsBwdParams& P, int n0,
                                        float (&dz)[kGated ? 2 : 1][kBwdRows][kM]) {
  for (int i = threadIdx.x; i < kBwdRows * kM; i += 256) {
    const int r = i % kBwdRows, m = i / kBwdRows, n = n0 + r;
    float g = 0.f, gu = 0.f;
    if (n < P.N && m < P.M) {
      const int64_t at = (int64_t)m * P.N + n;
      const float dy = Elem<T>::load(P.dy + at);
      float a, da;
      const bool needs_z = kGated || P.act != LQ_ACT_NONE;
      act_grad_any(P.act, needs_z ? Elem<T>::load(P.z + at) : 0.f, a, da);
      g = kGated ? dy * Elem<T>::load(P.u + at) * da : dy * da;
      gu = dy * a;
    }
    dz[0][r][m] = g;
    if (kGated) dz[kGated ? 1 : 0][r][m] = gu;
  }
}

// dx = dz W: a cluster owns 128 columns, its CTAs take 64-row pieces of W in
// turn, a warp 8 rows of a piece (256 contiguous bytes each, all in flight
// together).  Partial sums are added over the warps and then, through
// distributed shared memory, over the CTAs, in order.
template <typename T, int kM, bool kGated>
__global__ void __launch_bounds__(256) __cluster_dims__(kBwdSplit, 1, 1)
    k_rows_dx(const RowsBwdParams P) {
  constexpr int kF = kGated ? 2 : 1;
  __shared__ float dz[kF][kBwdRows][kM];
  __shared__ float part[4][kM][kBwdCols];
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col0 = (int)(blockIdx.x / kBwdSplit) * kBwdCols, c = col0 + 4 * lane;
  pdl_trigger();
  pdl_wait();
  float acc[kM][4];
#pragma unroll
  for (int m = 0; m < kM; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.f;
  auto load = [&](uint2 (&w)[kF][8], int n0) {
#pragma unroll
    for (int f = 0; f < kF; ++f)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = n0 + warp * 8 + i;
        w[f][i] = make_uint2(0u, 0u);
        if (n < P.N && c < P.K)  // K is a multiple of 8
          w[f][i] = __ldg(reinterpret_cast<const uint2*>((f ? P.w2 : P.w) + (int64_t)n * P.K + c));
      }
  };
  constexpr int kStep = kBwdSplit * kBwdRows;
  uint2 w[kF][8], next[kF][8];
  load(w, rank * kBwdRows);
  for (int n0 = rank * kBwdRows; n0 < P.N; n0 += kStep) {
    load(next, n0 + kStep);  // the next piece travels while this one is used
    __syncthreads();         // the piece before has been used
    rows_dz<T, kM, kGated>(P, n0, dz);
    __syncthreads();
#pragma unroll
    for (int f = 0; f < kF; ++f)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 lo = Elem<T>::unpack(w[f][i].x), hi = Elem<T>::unpack(w[f][i].y);
        const float* g = dz[f][warp * 8 + i];
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          acc[m][0] = fmaf(g[m], lo.x, acc[m][0]);
          acc[m][1] = fmaf(g[m], lo.y, acc[m][1]);
          acc[m][2] = fmaf(g[m], hi.x, acc[m][2]);
          acc[m][3] = fmaf(g[m], hi.y, acc[m][3]);
        }
      }
#pragma unroll
    for (int f = 0; f < kF; ++f)
#pragma unroll
      for (int i = 0; i < 8; ++i) w[f][i] = next[f][i];
  }
  for (int h = 1; h >= 0; --h) {  // warps 4..7, then 0..3 on top
    if (warp / 4 == h) {
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        float4* p = reinterpret_cast<float4*>(&part[warp & 3][m][4 * lane]);
        float4 v = make_float4(acc[m][0], acc[m][1], acc[m][2], acc[m][3]);
        if (h == 0) {
          const float4 o = *p;
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        *p = v;
      }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < kM * kBwdCols; i += 256) {
    float* p = &part[0][0][0] + i;
    p[0] = (p[0] + p[kM * kBwdCols]) + (p[2 * kM * kBwdCols] + p[3 * kM * kBwdCols]);
  }
  cluster.sync();
  constexpr int kOwn = kBwdCols / kBwdSplit;  // columns this CTA finishes
  for (int i = threadIdx.x; i < kM * kOwn; i += 256) {
    const int m = i / kOwn, k = rank * kOwn + i % kOwn;
    if (m >= P.M || col0 + k >= P.K) continue;
    float v = 0.f;
    for (int r = 0; r < kBwdSplit; ++r) v += *cluster.map_shared_rank(&part[0][m][k], r);
    const int64_t at = (int64_t)m * P.K + col0 + k;
    if (LQ_IN_RANGE(at, (int64_t)P.M * P.K)) P.dx[at] = Elem<T>::round(v);
  }
  cluster.sync();  // no CTA leaves while its sums are read
}

// dw = dz^T x and db: a block owns 64 weight rows and 256 columns; a thread keeps
// its eight columns of every token of x and writes 16 bytes (or 32) of a row.
template <typename T, int kM, bool kGated>
__global__ void __launch_bounds__(256) k_rows_dw(const RowsBwdParams P) {
  constexpr int kF = kGated ? 2 : 1;
  __shared__ float dz[kF][kBwdRows][kM];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = blockIdx.y * kBwdRows, c = (int)blockIdx.x * 256 + 8 * lane;
  pdl_trigger();
  pdl_wait();
  uint4 x[kM];
#pragma unroll
  for (int m = 0; m < kM; ++m) {
    x[m] = make_uint4(0, 0, 0, 0);
    if ((P.dw || P.dw2) && m < P.M && c < P.K)
      x[m] = __ldg(reinterpret_cast<const uint4*>(P.x + (int64_t)m * P.K + c));
  }
  rows_dz<T, kM, kGated>(P, n0, dz);
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x < kBwdRows && n0 + (int)threadIdx.x < P.N) {
    const int n = n0 + threadIdx.x;
#pragma unroll
    for (int f = 0; f < kF; ++f) {
      void* db = f ? P.db2 : P.db;
      if (!db) continue;
      float v = 0.f;
#pragma unroll
      for (int m = 0; m < kM; ++m) v += dz[f][threadIdx.x][m];
      if (P.f32)
        ((float*)db)[n] = P.accumulate ? ((float*)db)[n] + v : v;
      else
        ((uint16_t*)db)[n] = Elem<T>::round(v);
    }
  }
  if (c >= P.K) return;
#pragma unroll
  for (int f = 0; f < kF; ++f) {
    void* dw = f ? P.dw2 : P.dw;
    if (!dw) continue;
    for (int i = 0; i < 8; ++i) {
      const int r = warp * 8 + i, n = n0 + r;
      if (n >= P.N) break;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int m = 0; m < kM; ++m) {
        const float g = dz[f][r][m];
        float xf[8];
        unpack_vec<T>(x[m], xf);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(g, xf[e], v[e]);
      }
      const int64_t at = (int64_t)n * P.K + c;
      if (!LQ_IN_RANGE(at + 7, (int64_t)P.N * P.K)) continue;
      if (P.f32) {
        float4* o = reinterpret_cast<float4*>((float*)dw + at);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float4 q = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
          if (P.accumulate) {
            const float4 b = o[h];
            q.x += b.x, q.y += b.y, q.z += b.z, q.w += b.w;
          }
          o[h] = q;
        }
      } else {
        *reinterpret_cast<uint4*>((uint16_t*)dw + at) =
            make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]),
                       Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7]));
      }
    }
  }
}

// Self-test of the waits: a warp waits on an mbarrier phase that nothing completes, as
// an epilogue warp does, and gives up after limit_ns.
__global__ void __launch_bounds__(32) k_dense_wait_selftest(uint64_t limit_ns) {
  __shared__ __align__(8) unsigned long long bar;
  __shared__ int abort_flag;
  const uint32_t b = smem_u32(&bar);
  if (threadIdx.x == 0) {
    mbar_init(b, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncwarp();
  wait_warp(b, 0u, &abort_flag, limit_ns);
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (PFN_cuTensorMapEncodeTiled_v12000)p;
  });
  return fn;
}

// rows x cols 16-bit matrix (cols contiguous, row stride ld elements), boxes of
// 64 columns by box_rows rows, 128-byte swizzle, zeros outside
bool make_map(CUtensorMap* map, const void* p, bool bf16, int64_t rows, int64_t cols, int64_t ld,
              int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, es[2] = {1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
            const_cast<void*>(p), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// one operand of a product: rows x contraction when K-major, contraction x
// rows when MN-major
struct Operand {
  const void* p;
  int64_t rows, k, ld;
};

bool operand_map(CUtensorMap* m, const Operand& o, bool mn, bool bf16, int tile_rows) {
  return mn ? make_map(m, o.p, bf16, o.k, o.rows, o.ld, BK)
            : make_map(m, o.p, bf16, o.rows, o.k, o.ld, tile_rows);
}

template <typename T, int kBN, int kPair, bool kAMn, bool kBMn, int kEpi, bool kShared = false>
cudaError_t run_gemm(const Operand& a, const Operand& a2, const Operand& b, const Operand& b2,
                     const GemmParams& P, int slices, cudaStream_t s) {
  using C = Cfg<kBN, kPair, kEpi, kShared>;
  constexpr bool bf16 = Elem<T>::kFormat == 1;
  constexpr int rowsB = kEpi == kEpiGated ? kBN / 2 : kBN / kPair;
  CUtensorMap mA, mA2, mB, mB2;
  if (!operand_map(&mA, a, kAMn, bf16, BM) || !operand_map(&mB, b, kBMn, bf16, rowsB))
    return cudaErrorInvalidValue;
  mA2 = mA;
  mB2 = mB;
  if ((a2.p != a.p && !operand_map(&mA2, a2, kAMn, bf16, BM)) ||
      (b2.p != b.p && !operand_map(&mB2, b2, kBMn, bf16, rowsB)))
    return cudaErrorInvalidValue;
  auto* k = k_dense_gemm<T, kBN, kPair, kAMn, kBMn, kEpi, kShared>;
  static std::atomic<uint64_t> smem_set{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((smem_set.load() >> dev) & 1u)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) smem_set.fetch_or(1ull << dev);
  }
  constexpr int kTileN = kEpi == kEpiGated ? kBN / 2 : kBN, kTileM = BM * kPair;
  const int64_t tiles = ((P.M + kTileM - 1) / kTileM) * ((P.N + kTileN - 1) / kTileN);
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  const int64_t slots = std::max(1, num_sms() / kPair / slices);
  const int ctas = kShared ? P.members : kPair;
  cfg.gridDim = kShared ? dim3((unsigned)(tiles * ctas))
                        : dim3((unsigned)(std::min<int64_t>(tiles, slots) * kPair), (unsigned)slices);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ctas == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, k, mA, mA2, mB, mB2, P);
}

// Tile shape, by the time it would take.  Clocks of one 64-wide contraction
// block: 512 for the 256 x 256 tile of a CTA pair (the tensor pipe's own time),
// 300 for its 256 x 128 tile, 330 for a CTA's own 128 x 128 and 285 for its
// 128 x 64 tile (what the operand tiles take from L2); a tile's last epilogue and
// a pair's handshakes come on top once.  Measured on 2048 x 2048 x 5632: 34.2,
// 34.7, 38.9 and 56.2 us; on 16384 x 5632 x 2048: 251, 281, 331 and 466; on
// 128 x 2048 x 2048: 14.2, 9.1, 8.9 and 8.2; on 2048 x 256 x 256: 6.4, 5.0, 4.5
// and 4.2.
// A long contraction over few tiles is cut into slices (only where the caller has
// room for their float32 outputs, which another pass adds up): that pass, with its
// launch on the host, and the slices' outputs count as well, at 6000 clocks and
// 2600 bytes a clock.  dw of 8192 x 512 x 512 25 -> 17 us.
// Where that leaves most SMs idle, a cluster of 2 or 4 CTAs shares a 128 x 64 tile
// instead and adds its parts up through distributed shared memory; the exchange costs
// 5000 clocks (256 x 1024 x 1024 would go from 5.4 to 6.2 us).  64 x 2048 x 5632 14.4
// -> 8.1 us, 128 rows 14.5 -> 9.0, 256 rows 14.6 -> 12.1, gated 14.5 -> 11; 64 x 2048 x
// 2048 7.4 -> 6.0; dx of 64 x 5632 x 2048 14.1 -> 7.8, of 128 x 49152 x 2048 112 -> 39.
// 128 x 128 tiles shared in the same way take as long.  Eight CTAs a tile gain nothing
// more and do not all fit at once (128 of them: 11.5 us against 6.8 with four a tile,
// 100 x 1003 x 2048).
struct Shape {
  int tile, slices, members;
  int64_t clocks;
};
Shape pick_shape(int64_t M, int64_t N, int n_kb, int factors, int max_slices, bool may_share) {
  const int sms = num_sms();
  struct Kind {
    int tile, bm, bn, slots, per_block, once;
  };
  const Kind kinds[4] = {{2256, 256, 256, sms / 2, 512, 7800},
                         {2128, 256, 128, sms / 2, 300, 4300},
                         {128, 128, 128, sms, 330, 3000},
                         {64, 128, 64, sms, 285, 2600}};
  Shape best{2256, 1, 1, INT64_MAX};
  for (int slices = 1; slices <= max_slices; slices *= 2) {
    const int kb = (n_kb + slices - 1) / slices;
    if (slices > 1 && (kb < 8 || (int64_t)(slices - 1) * kb >= n_kb)) break;
    for (const Kind& k : kinds) {
      const int64_t tiles = ((M + k.bm - 1) / k.bm) * ((N * factors + k.bn - 1) / k.bn) * slices;
      int64_t c = (tiles + k.slots - 1) / k.slots * kb * k.per_block + k.once;
      if (slices > 1) c += 6000 + M * N * 8 * slices / 2600;
      if (c < best.clocks) best = {k.tile, slices, 1, c};
    }
  }
  const int64_t tiles = ((M + BM - 1) / BM) * ((N * factors + 63) / 64);
  for (int members = 2; may_share && members <= 4 && tiles * members <= sms; members *= 2) {
    const int kb = (n_kb + members - 1) / members;
    if ((members - 1) * kb >= n_kb) break;  // every member has a part
    const int64_t c = (int64_t)kb * 285 + 2600 + 5000;
    if (c < best.clocks) best = {64, 1, members, c};
  }
  return best;
}

template <typename T, bool kAMn, bool kBMn, int kEpi>
cudaError_t run_shape(const Shape& sh, const Operand& a, const Operand& a2, const Operand& b,
                      const Operand& b2, const GemmParams& P, cudaStream_t s) {
  if constexpr (!kAMn && kEpi != kEpiF32) {
    if (sh.members > 1) {
      GemmParams Q = P;
      Q.members = sh.members;
      Q.slice_kb = (P.n_kb + sh.members - 1) / sh.members;
      return run_gemm<T, 64, 1, kAMn, kBMn, kEpi, true>(a, a2, b, b2, Q, 1, s);
    }
  }
  switch (sh.tile) {
    case 2256:
      return run_gemm<T, 256, 2, kAMn, kBMn, kEpi>(a, a2, b, b2, P, sh.slices, s);
    case 2128:
      return run_gemm<T, 128, 2, kAMn, kBMn, kEpi>(a, a2, b, b2, P, sh.slices, s);
    case 128:
      return run_gemm<T, 128, 1, kAMn, kBMn, kEpi>(a, a2, b, b2, P, sh.slices, s);
    default:
      return run_gemm<T, 64, 1, kAMn, kBMn, kEpi>(a, a2, b, b2, P, sh.slices, s);
  }
}

GemmParams base_params(int64_t M, int64_t N, int64_t kdim) {
  GemmParams P{};
  P.M = M;
  P.N = N;
  P.ldo = N;
  P.n_kb = P.n_kb1 = P.slice_kb = (int)((kdim + BK - 1) / BK);
  P.rows1 = P.split = M;
  P.vec = N % 8 == 0;
  return P;
}

template <typename T, int kNT, bool kGated>
cudaError_t run_rows(const RowsParams& P, cudaStream_t s) {
  // Warps that share a block's contraction: 16 where an SM has one block at most and
  // the contraction gives them work (1 x 2048 x 5632: 5.4 us against 6.9, 16 tokens
  // 7.6 against 10.8), else 8 (16 x 5632 x 2048: 6.0 against 8.4; 16 x 512 x 512:
  // 2.2 against 2.7).
  const int blocks = (P.N + 15) / 16;
  const dim3 grid((unsigned)blocks);
  if (blocks <= num_sms() && P.K > 1024)
    return launch_kernel(k_dense_rows<T, kNT, kGated, 16>, grid, dim3(512), 0, s, true, P);
  return launch_kernel(k_dense_rows<T, kNT, kGated, 8>, grid, dim3(256), 0, s, true, P);
}

template <typename T>
cudaError_t forward(const DenseForward& d, cudaStream_t s) {
  const bool gated = d.w2 != nullptr;
  if (d.M <= kDenseRowsMax) {
    RowsParams R{(const uint16_t*)d.x,    (const uint16_t*)d.w,     (const uint16_t*)d.w2,
                 (const uint16_t*)d.bias, (const uint16_t*)d.bias2, (const uint16_t*)d.res,
                 (uint16_t*)d.y,          (uint16_t*)d.aux,         (uint16_t*)d.aux2,
                 (int)d.M,                (int)d.N,                 (int)d.K,
                 d.act};
    if (gated) return d.M <= 8 ? run_rows<T, 1, true>(R, s) : run_rows<T, 2, true>(R, s);
    return d.M <= 8 ? run_rows<T, 1, false>(R, s) : run_rows<T, 2, false>(R, s);
  }
  GemmParams P = base_params(d.M, d.N, d.K);
  P.act = d.act;
  P.bias = (const uint16_t*)d.bias;
  P.bias2 = (const uint16_t*)d.bias2;
  P.res = (const uint16_t*)d.res;
  P.out = d.y;
  P.aux = (uint16_t*)d.aux;
  P.aux2 = (uint16_t*)d.aux2;
  const Operand x{d.x, d.M, d.K, d.K}, w{d.w, d.N, d.K, d.K};
  if (gated) {
    const Operand w2{d.w2, d.N, d.K, d.K};
    return run_shape<T, false, false, kEpiGated>(pick_shape(d.M, d.N, P.n_kb, 2, 1, true), x, x, w, w2, P,
                                                 s);
  }
  return run_shape<T, false, false, kEpiDense>(pick_shape(d.M, d.N, P.n_kb, 1, 1, true), x, x, w, w, P,
                                               s);
}

template <typename T, bool kWhole, bool kGated>
cudaError_t act_grad_launch(const GradParams& P, dim3 grid, cudaStream_t s) {
  switch (P.act) {
    case LQ_ACT_RELU:
      return launch_kernel(k_act_grad<T, kWhole, kGated, LQ_ACT_RELU>, grid, dim3(256), 0, s, true, P);
    case LQ_ACT_SILU:
      return launch_kernel(k_act_grad<T, kWhole, kGated, LQ_ACT_SILU>, grid, dim3(256), 0, s, true, P);
    case LQ_ACT_GELU:
      return launch_kernel(k_act_grad<T, kWhole, kGated, LQ_ACT_GELU>, grid, dim3(256), 0, s, true, P);
    case LQ_ACT_GELU_TANH:
      return launch_kernel(k_act_grad<T, kWhole, kGated, LQ_ACT_GELU_TANH>, grid, dim3(256), 0, s,
                           true, P);
    default:
      return launch_kernel(k_act_grad<T, kWhole, kGated, LQ_ACT_NONE>, grid, dim3(256), 0, s, true, P);
  }
}

// A backward product, in slices where its shape says so.
template <typename T, bool kAMn, bool kBMn>
cudaError_t run_grad(const Shape& sh, const Operand& a, const Operand& a2, const Operand& b,
                     const Operand& b2, const GemmParams& P, bool f32, float* part,
                     cudaStream_t s) {
  if (sh.slices == 1)
    return f32 ? run_shape<T, kAMn, kBMn, kEpiF32>(sh, a, a2, b, b2, P, s)
               : run_shape<T, kAMn, kBMn, kEpiStore>(sh, a, a2, b, b2, P, s);
  GemmParams Q = P;
  Q.out = part;
  Q.out2 = nullptr;
  Q.rows1 = Q.split = P.M;
  Q.accumulate = 0;
  Q.slice_kb = (P.n_kb + sh.slices - 1) / sh.slices;
  Q.slice_bytes = P.M * P.N * 4;
  cudaError_t e = run_shape<T, kAMn, kBMn, kEpiF32>(sh, a, a2, b, b2, Q, s);
  if (e != cudaSuccess) return e;
  return launch_kernel(k_add_slices<T>, dim3((unsigned)((P.M * P.N / 4 + 255) / 256)), dim3(256), 0,
                       s, true, (const float*)part, sh.slices, P.M, P.N, P, f32 ? 1 : 0);
}

// few rows: the grid's second dimension counts 64-row pieces of the weights
bool bwd_by_rows(int64_t M, int64_t N) {
  return M <= kBwdRowsMax && N <= 65535 * (int64_t)kBwdRows;
}

// shapes of the backward products (half: columns of dz of one factor)
constexpr int kMaxSlices = 8;
Shape dx_shape(int64_t M, int64_t half, int64_t K, bool gated) {
  return pick_shape(M, K, (int)((half + BK - 1) / BK) * (gated ? 2 : 1), 1, kMaxSlices, true);
}
Shape dw_shape(int64_t rows, int64_t K, int64_t M) {
  return pick_shape(rows, K, (int)((M + BK - 1) / BK), 1, kMaxSlices, false);
}

template <typename T, int kM, bool kGated>
cudaError_t run_rows_bwd(const RowsBwdParams& P, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (P.dx)
    e = launch_kernel(k_rows_dx<T, kM, kGated>,
                      dim3((unsigned)((P.K + kBwdCols - 1) / kBwdCols * kBwdSplit)), dim3(256), 0, s,
                      true, P);
  if (e == cudaSuccess && (P.dw || P.dw2 || P.db || P.db2)) {
    const bool dw = P.dw || P.dw2;
    e = launch_kernel(k_rows_dw<T, kM, kGated>,
                      dim3(dw ? (unsigned)((P.K + 255) / 256) : 1u,
                           (unsigned)((P.N + kBwdRows - 1) / kBwdRows)),
                      dim3(256), 0, s, true, P);
  }
  return e;
}

template <typename T>
cudaError_t backward(const DenseBackward& d, cudaStream_t s) {
  const bool gated = d.gated;
  if (bwd_by_rows(d.M, d.N)) {
    RowsBwdParams R{(const uint16_t*)d.dy, (const uint16_t*)d.z,  (const uint16_t*)d.u,
                    (const uint16_t*)d.x,  (const uint16_t*)d.w,  (const uint16_t*)d.w2,
                    (uint16_t*)d.dx,       d.dw,                  d.dw2,
                    d.db,                  d.db2,                 (int)d.M,
                    (int)d.N,              (int)d.K,              d.act,
                    d.f32,                 d.accumulate};
    return gated ? run_rows_bwd<T, kBwdRowsMax, true>(R, s)
                 : run_rows_bwd<T, kBwdRowsMax, false>(R, s);
  }
  const DenseBwdPlan pl = dense_bwd_plan(d.M, d.N, d.K, gated, d.act != LQ_ACT_NONE);
  const bool products = d.dx || d.dw || d.dw2;
  const bool sums = d.db || d.db2;
  uint16_t* dz = (uint16_t*)d.ws;
  float* part = (float*)((char*)d.ws + pl.dz_bytes);
  float* slices = (float*)((char*)d.ws + pl.dz_bytes + pl.sum_bytes);
  const int nf = gated ? 2 : 1;
  cudaError_t e;
  if (sums || (products && pl.copy)) {
    GradParams G{};
    G.dy = (const uint16_t*)d.dy;
    G.z = (const uint16_t*)d.z;
    G.u = (const uint16_t*)d.u;
    G.dz = products && pl.copy ? dz : nullptr;
    G.sums = sums ? part : nullptr;
    G.M = d.M;
    G.N = d.N;
    G.ldz = pl.ldz;
    G.rows = pl.rows;
    G.act = d.act;
    const bool whole = d.N % 8 == 0;
    const int64_t width = gated ? pl.ldz / 2 : pl.ldz;
    const dim3 grid((unsigned)((width + 255) / 256), (unsigned)pl.row_blocks);
    if (gated)
      e = whole ? act_grad_launch<T, true, true>(G, grid, s)
                : act_grad_launch<T, false, true>(G, grid, s);
    else
      e = whole ? act_grad_launch<T, true, false>(G, grid, s)
                : act_grad_launch<T, false, false>(G, grid, s);
    if (e != cudaSuccess) return e;
  }
  if (sums) {
    e = launch_kernel(k_col_sums<T>, dim3((unsigned)((d.N * nf + 255) / 256)), dim3(256), 0, s,
                      true, (const float*)part, d.N, nf, pl.row_blocks, d.db, d.db2, d.f32,
                      d.accumulate);
    if (e != cudaSuccess) return e;
  }
  const void* dzp = pl.copy ? (const void*)dz : d.dy;
  const int64_t half = gated ? pl.ldz / 2 : pl.ldz;
  if (d.dx) {
    GemmParams P = base_params(d.M, d.K, half);
    P.out = d.dx;
    const Operand a{dzp, d.M, half, pl.ldz};
    const Operand b{d.w, d.K, d.N, d.K};
    Operand a2 = a, b2 = b;
    if (gated) {
      a2.p = dz + half;
      b2.p = d.w2;
      P.n_kb = 2 * P.n_kb1;
    }
    P.slice_kb = P.n_kb;
    e = run_grad<T, false, true>(dx_shape(d.M, half, d.K, gated), a, a2, b, b2, P, false, slices, s);
    if (e != cudaSuccess) return e;
  }
  // Output rows of a weight gradient: the columns of dz.  Both factors are one
  // product, whose padding rows between and after them are not written, unless its
  // rows pass the 31 bits of a TMA coordinate.
  const bool both = d.dw && d.dw2 && half + d.N <= INT32_MAX - 255;
  for (int f = 0; f < 2; ++f) {
    void* dw = f ? d.dw2 : d.dw;
    if (!dw || (f && both)) continue;
    const int64_t rows = both ? half + d.N : d.N;
    GemmParams P = base_params(rows, d.K, d.M);
    P.out = dw;
    P.out2 = both ? d.dw2 : nullptr;
    P.rows1 = d.N;
    P.split = both ? half : rows;
    P.accumulate = d.accumulate;
    const Operand a{f ? (const void*)(dz + half) : dzp, rows, d.M, pl.ldz};
    const Operand b{d.x, d.K, d.M, d.K};
    e = run_grad<T, true, true>(dw_shape(rows, d.K, d.M), a, a, b, b, P, d.f32, slices, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_dense_forward(const DenseForward& d, cudaStream_t s) {
  return d.dtype == LQ_BF16 ? forward<__nv_bfloat16>(d, s) : forward<__half>(d, s);
}

DenseBwdPlan dense_bwd_plan(int64_t M, int64_t N, int64_t K, bool gated, bool act) {
  DenseBwdPlan p{};
  if (bwd_by_rows(M, N)) return p;
  // dz is its own matrix where it differs from dy, or where dy's rows do not
  // start on 16-byte boundaries (a TMA source needs that)
  p.copy = gated || act || N % 8 != 0;
  const int64_t width = (N + BK - 1) / BK * BK;
  p.ldz = p.copy ? width * (gated ? 2 : 1) : N;
  p.dz_bytes = p.copy ? (M * p.ldz * 2 + 255) / 256 * 256 : 0;
  // at most 256 row blocks of at least 64 rows
  p.rows = std::max<int64_t>(64, (M + 255) / 256);
  p.row_blocks = (int)((M + p.rows - 1) / p.rows);
  p.sum_bytes = ((int64_t)p.row_blocks * N * (gated ? 2 : 1) * 4 + 255) / 256 * 256;
  // the largest of the products' slices (dw of one or of both factors)
  const int64_t half = gated ? p.ldz / 2 : p.ldz;
  auto room = [](const Shape& sh, int64_t rows, int64_t cols) {
    return sh.slices > 1 ? (rows * cols * 4 * sh.slices + 255) / 256 * 256 : 0;
  };
  p.slice_bytes = std::max(room(dx_shape(M, half, K, gated), M, K), room(dw_shape(N, K, M), N, K));
  if (gated)
    p.slice_bytes = std::max(p.slice_bytes, room(dw_shape(half + N, K, M), half + N, K));
  return p;
}

cudaError_t launch_dense_backward(const DenseBackward& d, cudaStream_t s) {
  return d.dtype == LQ_BF16 ? backward<__nv_bfloat16>(d, s) : backward<__half>(d, s);
}

unsigned long long bounds_fail_dense() { return lq_take_bounds_fail(); }

cudaError_t launch_dense_wait_selftest(uint64_t limit_ns, cudaStream_t s) {
  k_dense_wait_selftest<<<1, 32, 0, s>>>(limit_ns);
  return cudaGetLastError();
}

cudaError_t take_dense_status(int* status) {
  int zero = 0;
  *status = 0;
  cudaError_t e = cudaMemcpyFromSymbol(status, g_dense_status, sizeof(int));
  if (e == cudaSuccess && *status) e = cudaMemcpyToSymbol(g_dense_status, &zero, sizeof(int));
  return e;
}

}  // namespace lq
