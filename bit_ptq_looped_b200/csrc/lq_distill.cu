// Distillation from a teacher's top logits: loss and gradient of the student's
// logits, row by row.
//
// Row m has V student logits z and k listed teacher logits t_i at vocabulary
// indices v_i.  With temperature T, q = softmax(z / T) and
//   no rest class:  p = softmax(t / T) over the listed entries, R = 0;
//   rest class:     p_i = exp(t_i / T - L) with the teacher's log-partition L,
//                   R = max(0, 1 - sum p) for everything that is not listed (0
//                   where the student has no mass there, Q_rest = 0);
//   loss = w (sum_i p_i (log p_i - log q_{v_i}) + R (log R - log Q_rest)),
//   dz_j = w / T (C q_j - p_j)                 j listed, C = sum p + R
//   dz_j = w / T  q_j (C - R S / S_rest)       otherwise,
// S the sum of exp(z / T) over the vocabulary and S_rest that over the entries
// that are not listed, Q_rest = S_rest / S.  With a rest class S_rest is summed
// directly (not as a difference, which loses everything when the listed entries hold
// nearly all of the student's mass) and relative to the largest logit that is not
// listed, m_rest: it keeps its digits however far those logits lie below the listed
// ones.  S is put together from it and the listed entries' sum in float64, log Q_rest
// from logarithms, and with f = w / T (C exp((m_rest - m) / T) / S - R / S_rest) an
// entry that is not listed gets f exp((z_j - m_rest) / T): no factor overflows.
//
// What bounds it is memory, each logit read once and each gradient written
// once, and next to it the exponential unit (two exponentials per logit, 16 per
// clock and SM).  A CTA, or over a cluster of 2, 4 or 8 CTAs each one, walks its
// columns twice: a first pass with a running maximum and sum, and for the
// gradient a second one that finds the row in L2, where the rows in flight (some
// 100 KB each, four per SM) stay; the gradients are stored as streaming data so
// as not to displace them.  Nothing limits the row's length, and nothing waits
// but at barriers.  Measured, 8192 x 49152 bf16 logits: 212 us for the loss
// (floor 123), 355 with the gradient (floor 246) in a short series, 384 in a long one;
// with a rest class, whose listed entries are hidden vector by vector, 239 and 387 (a
// float maximum over the unpacked vector instead of the packed one took 4 more).  Holding
// the row in shared memory between the passes (bulk copies in and out, two rows per SM) took 250
// and 342-365, and 46-56 against 26 for the loss of 255 x 100003 float32 logits;
// a ring of bulk copies running ahead across passes and rows took 600, and keeping
// part of the row in shared memory 555: what shared memory takes, the L1 lines
// of the loads in flight lack.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "lq_dense.cuh"

namespace lq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxSmem = 164 * 1024;  // 64 KB of bitmap, 96 KB of listed entries
constexpr int kMaxCluster = 8;
constexpr float kNegInf = -INFINITY;

// eight 16-bit elements, kInf where bit i of marks is set
template <uint32_t kInf>
__device__ __forceinline__ uint4 hide16(const uint4& w, uint32_t marks) {
  uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((marks >> (2 * i)) & 1u) q[i] = (q[i] & 0xFFFF0000u) | kInf;
    if ((marks >> (2 * i)) & 2u) q[i] = (q[i] & 0x0000FFFFu) | (kInf << 16);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

template <typename T>
struct Log;  // element access of a logit type
template <>
struct Log<float> {
  static constexpr int kE = 4;  // elements per 16 bytes
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[4]) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ uint4 nothing() {  // -inf throughout
    return make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
  }
  // -inf where bit i of marks is set
  static __device__ __forceinline__ uint4 hide(const uint4& w, uint32_t marks) {
    return make_uint4((marks & 1u) ? 0xFF800000u : w.x, (marks & 2u) ? 0xFF800000u : w.y,
                      (marks & 4u) ? 0xFF800000u : w.z, (marks & 8u) ? 0xFF800000u : w.w);
  }
  // running maximum of 16-byte vectors, in the type's own pairs
  using Run = float;
  static __device__ __forceinline__ float run_start() { return kNegInf; }
  static __device__ __forceinline__ float run_max(float m, const uint4& w) {
    return fmaxf(fmaxf(fmaxf(m, __uint_as_float(w.x)), __uint_as_float(w.y)),
                 fmaxf(__uint_as_float(w.z), __uint_as_float(w.w)));
  }
  static __device__ __forceinline__ float run_end(float m) { return m; }
};
template <>
struct Log<__nv_bfloat16> {
  static constexpr int kE = 8;
  static __device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(q[i] << 16);
      f[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      q[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
  }
  static __device__ __forceinline__ uint4 nothing() {
    return make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
  }
  static __device__ __forceinline__ uint4 hide(const uint4& w, uint32_t marks) {
    return hide16<0xFF80u>(w, marks);
  }
  using Run = __nv_bfloat162;
  static __device__ __forceinline__ Run run_start() { return __float2bfloat162_rn(kNegInf); }
  static __device__ __forceinline__ Run run_max(Run m, const uint4& w) {
    const Run* v = reinterpret_cast<const Run*>(&w);
    return __hmax2(__hmax2(m, __hmax2(v[0], v[1])), __hmax2(v[2], v[3]));
  }
  static __device__ __forceinline__ float run_end(Run m) {
    return fmaxf(__low2float(m), __high2float(m));
  }
};
template <>
struct Log<__half> {
  static constexpr int kE = 8;
  static __device__ __forceinline__ float get(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ void put(__half* p, float v) { *p = __float2half_rn(v); }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[8]) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&q[i]));
      f[2 * i] = v.x;
      f[2 * i + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      q[i] = *reinterpret_cast<uint32_t*>(&v);
    }
    return make_uint4(q[0], q[1], q[2], q[3]);
  }
  static __device__ __forceinline__ uint4 nothing() {
    return make_uint4(0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u, 0xFC00FC00u);
  }
  static __device__ __forceinline__ uint4 hide(const uint4& w, uint32_t marks) {
    return hide16<0xFC00u>(w, marks);
  }
  using Run = __half2;
  static __device__ __forceinline__ Run run_start() { return __float2half2_rn(kNegInf); }
  static __device__ __forceinline__ Run run_max(Run m, const uint4& w) {
    const Run* v = reinterpret_cast<const Run*>(&w);
    return __hmax2(__hmax2(m, __hmax2(v[0], v[1])), __hmax2(v[2], v[3]));
  }
  static __device__ __forceinline__ float run_end(Run m) {
    return fmaxf(__low2float(m), __high2float(m));
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct DistillParams {
  const void* z;
  void* grad;
  const void* t;
  const void* idx;
  const float* t_lse;
  const float* weight;
  float* loss;
  int64_t M, V;
  int k, t_dtype, idx64;
  int slice;   // elements per CTA, a multiple of 32
  int ahead;   // several rows per resident CTA: fetch a row's rest to L2 at once
  float temp, inv_temp;
  double c2d;  // log2(e) / temp
  float c2;    // the same, rounded: the student's exponents, and consistently its
               // log-partition, use this one
};

__device__ __forceinline__ float teacher_at(const DistillParams& P, int64_t i) {
  if (P.t_dtype == LQ_F32) return ((const float*)P.t)[i];
  if (P.t_dtype == LQ_BF16) return __bfloat162float(((const __nv_bfloat16*)P.t)[i]);
  return __half2float(((const __half*)P.t)[i]);
}
__device__ __forceinline__ int64_t index_at(const DistillParams& P, int64_t i) {
  return P.idx64 ? ((const int64_t*)P.idx)[i] : (int64_t)((const int32_t*)P.idx)[i];
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// what a slice tells the others
struct Part {
  float m, m2nd;     // maximum of its logits (rest class: of those not listed); of its
                     // teacher entries (rest class: of the listed logits)
  double s, s2nd;    // the sums of exponentials that go with them
  double p_sum;      // rest class: sum of p
};
// a row's numbers, worked out by one thread.  What the gradient waits for needs
// divisions only; the logarithms come at the end, for the loss alone.
struct RowNumbers {
  float m;       // exponents of listed entries are (z - m) c2
  float m_rest;  // of entries that are not listed (z - m_rest) c2
  float f_rest;  // gradient of an entry that is not listed, over its exponential
  float f_top;   // C / S times the scale: what q adds to a listed entry's
  float inv_ts;  // no rest class: one over the listed exponentials' sum, 0 if there is none
  float tm;      // exponents of p are (t - tm) c2 (no rest class)
};

// Running maximum and sum of exponentials.  An exponent is the difference of a logit
// and the maximum, times c2: z c2 - m c2 would be one multiply-add, but both products
// leave float32's range where logits are masked with their type's lowest value or the
// temperature is small, and inf - inf is no number.  The difference may at worst be
// -inf, which counts nothing.  ref: the maximum, 0 while there is none.  A maximum
// passes over NaN, a sum does not: where nothing but NaN was seen m is -inf and s NaN,
// and every join keeps it, so that the row's loss and gradient become NaN.
struct Run1 {
  float m, s;
};
__device__ __forceinline__ float ref(float m) { return m == kNegInf ? 0.f : m; }
__device__ __forceinline__ float ex2_from(float z, float from, float c2) {
  return ex2((z - from) * c2);
}
// the lanes' as one, in a fixed order
__device__ __forceinline__ Run1 warp_join(Run1 r, float c2) {
  const float m = warp_max(r.m);
  const float s = warp_sum(r.m == kNegInf ? r.s : r.s * ex2_from(r.m, m, c2));
  return {m, s};
}

// log2 p of a listed entry, in float64: logit and log-partition may be far larger
// than their difference, and the mass that is not listed, 1 - sum p, may be small
__device__ __forceinline__ double log2p(float t, double c2d, double lse2) {
  return (double)t * c2d - lse2;
}

// What a CTA holds of one row: its slice of the columns, counted from the
// 16-byte boundary at or before the row's start (column j of the row is
// j + lead), so that the slice's vectors are aligned in global memory.
template <typename T>
struct Slice {
  static constexpr int kE = Log<T>::kE;
  int64_t c0;      // row column of slice element 0
  int lo, hi;      // valid slice elements
  int v_lo, v_hi;  // whole 16-byte vectors
  int edge0, n_edge;
  __device__ __forceinline__ Slice(const void* z, int64_t row, int64_t V, int rank, int slice) {
    const int lead = (int)(((uintptr_t)z / sizeof(T) + (uint64_t)(row * V)) % kE);
    c0 = (int64_t)rank * slice - lead;
    lo = (int)(c0 < 0 ? -c0 : 0);
    const int64_t left = V - c0;
    hi = (int)(left < 0 ? 0 : left < slice ? left : slice);
    v_lo = (lo + kE - 1) / kE;
    v_hi = max(v_lo, hi / kE);
    // the few elements before and after the vectors
    edge0 = max(0, min(hi, v_lo * kE) - lo);
    n_edge = edge0 + max(0, hi - v_hi * kE);
  }
  // slice element of edge number i < n_edge
  __device__ __forceinline__ int edge(int i) const {
    return i < edge0 ? lo + i : v_hi * kE + (i - edge0);
  }
};

template <typename T, bool kTail, int kThreads, int kUnroll, int kCtas>
__global__ void __launch_bounds__(kThreads, kCtas)
    k_distill(const __grid_constant__ DistillParams P) {
  constexpr int kE = Log<T>::kE, kWarps = kThreads / 32;
  extern __shared__ uint32_t bits[];  // the slice's listed entries
  // the listed entries, each read and written by one thread: position in the
  // slice (-1 for none of it), teacher logit, student logit
  int* ent_e = reinterpret_cast<int*>(bits + P.slice / 32);
  float* ent_t = reinterpret_cast<float*>(ent_e + P.k);
  float* ent_z = ent_t + P.k;
  __shared__ Part parts[kMaxCluster];
  __shared__ double loss_parts[kMaxCluster];
  __shared__ float sm_m[2][32], sm_s[2][32];
  __shared__ double sm_d[2][32];
  __shared__ RowNumbers row_n;
  __shared__ int flags;  // 1: an entry is in range, 2: an index is listed again
  cg::cluster_group cluster = cg::this_cluster();
  const int n_parts = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / n_parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  pdl_trigger();
  if (tid == 0) flags = 0;
  for (int i = tid; i < P.slice / 32; i += kThreads) bits[i] = 0u;
  const Slice<T> sl(P.z, row, P.V, rank, P.slice);
  const T* zs = (const T*)P.z + row * P.V + sl.c0;  // slice element 0
  T* gs = P.grad ? (T*)P.grad + row * P.V + sl.c0 : nullptr;
  const uint4* vec = reinterpret_cast<const uint4*>(zs);
  const int64_t list = row * P.k;
  // Both passes walk the vectors in batches of kUnroll per thread, the next batch
  // on its way while one is worked on.  The last batch may be partial: what lies
  // beyond the end is -inf, which counts nothing.
  const int n_vec = sl.v_hi - sl.v_lo, n_full = n_vec / (kUnroll * kThreads);
  const int n_batch = (n_vec + kUnroll * kThreads - 1) / (kUnroll * kThreads);
  vec += sl.v_lo + tid;
  auto batch = [&](uint4 (&x)[kUnroll], int b) {
    const uint4* p = vec + b * (kUnroll * kThreads);
    if (b < n_full) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) x[u] = p[u * kThreads];
    } else {
      const int left = n_vec - tid - b * (kUnroll * kThreads);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) x[u] = u * kThreads < left ? p[u * kThreads] : Log<T>::nothing();
    }
  };
  pdl_wait();
  // the row's weight, its first batch and its list travel together
  const float w = P.weight ? P.weight[row] : 1.f;
  uint4 x[kUnroll];
  batch(x, 0);
  // with many rows, the rest of the slice towards L2 at once: more of it travels
  // than the loads of the pass alone would ask for (8192 x 49152: 372 -> 355 us;
  // where all rows are in flight anyway it costs 5 %)
  if (P.ahead && warp == 0 && n_batch > 1 && elect_one()) {
    const uint4* p = reinterpret_cast<const uint4*>(zs) + sl.v_lo + kUnroll * kThreads;
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p),
                 "r"((uint32_t)(n_vec - kUnroll * kThreads) * 16u)
                 : "memory");
  }
  bool any = false;
  for (int i0 = tid; i0 < P.k; i0 += 4 * kThreads) {
    int64_t v[4];
    float t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * kThreads;
      v[j] = i < P.k ? index_at(P, list + i) : -1;
      t[j] = i < P.k ? teacher_at(P, list + i) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * kThreads;
      if (i >= P.k) break;
      const int64_t e = v[j] - sl.c0;
      const bool in = v[j] >= 0 && v[j] < P.V;
      any |= in;
      ent_e[i] = in && e >= sl.lo && e < sl.hi ? (int)e : -1;
      ent_t[i] = t[j];
    }
  }
  auto zero_row = [&]() {
    if (rank == 0 && tid == 0) P.loss[row] = 0.f;
    if (!gs) return;
    for (int v = sl.v_lo + tid; v < sl.v_hi; v += kThreads)
      if (LQ_IN_RANGE(sl.c0 + (v + 1) * kE - 1, P.V))
        reinterpret_cast<uint4*>(gs)[v] = make_uint4(0, 0, 0, 0);
    if (tid < sl.n_edge && LQ_IN_RANGE(sl.c0 + sl.edge(tid), P.V))
      Log<T>::put(gs + sl.edge(tid), 0.f);
  };
  // a row of weight 0 counts nothing, whatever its logits hold (the same
  // decision in every CTA of the cluster)
  if (w == 0.f) {
    zero_row();
    return;
  }
  if (n_parts > 1) cluster.barrier_arrive();  // this CTA runs: its shared memory may be written
  __syncthreads();

  // mark the listed entries of the slice; an index that is listed again counts
  // at its first position only
  bool dup = false;
  for (int i0 = tid; i0 < P.k; i0 += 4 * kThreads) {
    float z[4];
    int e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j * kThreads;
      e[j] = i < P.k ? ent_e[i] : -1;
      z[j] = e[j] >= 0 ? Log<T>::get(zs + e[j]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (e[j] < 0) continue;
      const uint32_t b = 1u << (e[j] & 31);
      dup |= (atomicOr(&bits[e[j] >> 5], b) & b) != 0;
      ent_z[i0 + j * kThreads] = z[j];
    }
  }
  any = __any_sync(~0u, any);
  dup = __any_sync(~0u, dup);
  if (lane == 0 && (any || dup)) atomicOr(&flags, (any ? 1 : 0) | (dup ? 2 : 0));
  __syncthreads();
  any = flags & 1;
  if (flags & 2) {
    for (int i = tid; i < P.k; i += kThreads) {
      const int64_t v = index_at(P, list + i);
      bool first = true;
      for (int j = 0; j < i && first; ++j) first = index_at(P, list + j) != v;
      if (!first) ent_e[i] = -1;
    }
  }
  // fn(position, teacher logit, student logit) for this thread's entries
  auto for_entries = [&](auto&& fn) {
    for (int i = tid; i < P.k; i += kThreads) {
      const int e = ent_e[i];
      if (e >= 0) fn(e, ent_t[i], ent_z[i]);
    }
  };
  auto marked = [&](int e) { return (bits[e >> 5] >> (e & 31)) & 1u; };

  // First pass: running maximum and sum.  A batch first raises the maximum
  // (packed), then adds its exponentials.
  Run1 r1 = {kNegInf, 0.f};
  float2 s2 = make_float2(0.f, 0.f);
  const float2 c2v = make_float2(P.c2, P.c2);
  auto raise = [&](float to) {
    if (to > r1.m) {
      const float f = ex2_from(r1.m, to, P.c2);
      s2 = fmul2(s2, make_float2(f, f));
      r1.m = to;
    }
  };

  for (int b = 0; b < n_batch; ++b) {
    uint4 y[kUnroll];
    if (b + 1 < n_batch) batch(y, b + 1);
    if (kTail) {  // listed entries do not count here
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int e = min(sl.v_lo + tid + (b * kUnroll + u) * kThreads, sl.v_hi - 1) * kE;
        x[u] = Log<T>::hide(x[u], bits[e >> 5] >> (e & 31));
      }
    }
    typename Log<T>::Run run = Log<T>::run_start();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) run = Log<T>::run_max(run, x[u]);
    raise(Log<T>::run_end(run));
    const float2 nm = make_float2(-ref(r1.m), -ref(r1.m));
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float f[kE];
      Log<T>::unpack(x[u], f);
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        const float2 q = fmul2(fadd2(make_float2(f[i], f[i + 1]), nm), c2v);
        s2 = fadd2(s2, make_float2(ex2(q.x), ex2(q.y)));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x[u] = y[u];
  }
  float z_edge = 0.f;
  if (tid < sl.n_edge) {
    z_edge = Log<T>::get(zs + sl.edge(tid));
    if (!kTail || !marked(sl.edge(tid))) {
      raise(z_edge);
      s2.x += ex2_from(z_edge, ref(r1.m), P.c2);
    }
  }
  if (gs) batch(x, 0);  // the second pass's first batch
  r1.s = s2.x + s2.y;
  // the listed entries: their teacher's maximum and sum, or with a rest class
  // their student's exponentials, and the sum of p in float64 (1 - sum p may be
  // small)
  Run1 r2 = {kNegInf, 0.f};
  double p_sum = 0.0;
  const double lse2_t = kTail ? (double)P.t_lse[row] * 1.4426950408889634 : 0.0;
  for_entries([&](int, float t, float z) {
    const float l = kTail ? z : t;
    if (l > r2.m) {
      r2.s *= ex2_from(r2.m, l, P.c2);
      r2.m = l;
    }
    r2.s += ex2_from(l, ref(r2.m), P.c2);
    if (kTail) p_sum += (double)ex2((float)log2p(t, P.c2d, lse2_t));
  });
  r1 = warp_join(r1, P.c2);
  r2 = warp_join(r2, P.c2);
  if (kTail) p_sum = warp_sum(p_sum);
  if (lane == 0) {
    sm_m[0][warp] = r1.m, sm_s[0][warp] = r1.s;
    sm_m[1][warp] = r2.m, sm_s[1][warp] = r2.s;
    if (kTail) sm_d[0][warp] = p_sum;
  }
  __syncthreads();
  if (n_parts > 1) cluster.barrier_wait();
  if (warp == 0) {
    Part p;
    double d[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float m = lane < kWarps ? sm_m[j][lane] : kNegInf, mm = warp_max(m);
      const float f = m == kNegInf ? 1.f : ex2_from(m, mm, P.c2);
      d[j] = warp_sum(lane < kWarps ? (double)(sm_s[j][lane] * f) : 0.0);
      (j ? p.m2nd : p.m) = mm;
    }
    p.s = d[0];
    p.s2nd = d[1];
    p.p_sum = kTail ? warp_sum(lane < kWarps ? sm_d[0][lane] : 0.0) : 0.0;
    if (lane < n_parts)
      *(n_parts > 1 ? cluster.map_shared_rank(&parts[rank], lane) : &parts[0]) = p;
    __syncwarp();
  }
  if (n_parts > 1) cluster.sync();

  // the row's numbers, from the slices in order
  double S = 0.0, total = 0.0, TS = 0.0, R = 0.0;
  double to_top = 0.0;  // rest class: its largest exponent below the row's
  if (tid == 0) {
    float M = kNegInf, M2nd = kNegInf;
    for (int r = 0; r < n_parts; ++r) {
      M = fmaxf(M, parts[r].m);
      M2nd = fmaxf(M2nd, parts[r].m2nd);
    }
    auto scaled = [&](float m, double v, float to) {
      return m == kNegInf || m == to ? v : v * exp2(((double)m - (double)to) * (double)P.c2);
    };
    double second = 0.0;
    for (int r = 0; r < n_parts; ++r) {
      S += scaled(parts[r].m, parts[r].s, M);
      second += scaled(parts[r].m2nd, parts[r].s2nd, M2nd);
      TS += parts[r].p_sum;
    }
    RowNumbers n;
    if (kTail) {
      // both sums in units of the larger maximum
      const float top = fmaxf(M, M2nd);
      to_top = M == top ? 0.0 : ((double)M - (double)top) * (double)P.c2;
      const double up = to_top == 0.0 ? 1.0 : exp2(to_top);
      total = S * up + scaled(M2nd, second, top);
      // nothing outside the list: no rest class, neither in the loss nor in its gradient
      R = S != 0.0 && 1.0 - TS > 0.0 ? 1.0 - TS : 0.0;
      const double C = TS + R;
      const float scale = w * P.inv_temp, f = (float)C / (float)total;
      n.m = ref(top);
      n.m_rest = ref(M);
      n.f_rest = S != 0.0 ? scale * (f * (float)up - (float)R / (float)S) : 0.f;
      n.f_top = scale * f;
      n.inv_ts = n.tm = 0.f;
    } else {
      total = S;
      TS = second;
      n.m = n.m_rest = ref(M);
      n.inv_ts = TS != 0.0 ? 1.f / (float)TS : 0.f;
      const float C = TS > 0.0 ? 1.f : (float)TS;  // the sum of p: 1, 0 without any, or NaN
      n.f_rest = n.f_top = w * P.inv_temp / (float)total * C;
      n.tm = ref(M2nd);
    }
    row_n = n;
  }
  __syncthreads();
  const RowNumbers n = row_n;
  if (!kTail && !any) {
    // no entry in range: the row counts nothing (the same in the whole cluster)
    zero_row();
    if (n_parts > 1) cluster.sync();
    return;
  }

  // second pass: the gradient of entries that are not listed
  if (gs) {
    const float2 fr = make_float2(n.f_rest, n.f_rest), nn = make_float2(-n.m_rest, -n.m_rest);
    uint4* out = reinterpret_cast<uint4*>(gs) + sl.v_lo + tid;
    // the row's column at which a vector starts (for the bounds-check build)
    [[maybe_unused]] auto column = [&](int b, int u) {
      return sl.c0 + (int64_t)(sl.v_lo + tid + (b * kUnroll + u) * kThreads) * kE;
    };
    auto grad = [&](const uint4& x) {
      float f[kE];
      Log<T>::unpack(x, f);
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        float2 y = fmul2(fadd2(make_float2(f[i], f[i + 1]), nn), c2v);
        y = fmul2(make_float2(ex2(y.x), ex2(y.y)), fr);
        f[i] = y.x;
        f[i + 1] = y.y;
      }
      return Log<T>::pack(f);
    };

    for (int b = 0; b < n_batch; ++b) {
      uint4 y[kUnroll];
      if (b + 1 < n_batch) batch(y, b + 1);
      uint4* o = out + b * (kUnroll * kThreads);
      if (b < n_full) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (LQ_IN_RANGE(column(b, u) + kE - 1, P.V))
            __stcs(o + u * kThreads, grad(x[u]));
      } else {
        const int left = n_vec - tid - b * (kUnroll * kThreads);
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (u * kThreads < left && LQ_IN_RANGE(column(b, u) + kE - 1, P.V))
            __stcs(o + u * kThreads, grad(x[u]));
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) x[u] = y[u];
    }
    if (tid < sl.n_edge && LQ_IN_RANGE(sl.c0 + sl.edge(tid), P.V))
      Log<T>::put(gs + sl.edge(tid), n.f_rest * ex2_from(z_edge, n.m_rest, P.c2));
    __syncthreads();
  }
  // The listed entries: their gradients over it, and the loss up to the
  // logarithms of the sums: sum p (log2 p - log2 q) = sum p (a - b) + sum p lg,
  // a and b the exponents of p and q relative to their references, in float64
  // (the logits may be far larger than the difference, and the difference past
  // float32's range).
  const float scale = w * P.inv_temp;
  double part = 0.0;
  float mass = 0.f;
  for_entries([&](int e, float t, float z) {
    // without a rest class the teacher's exponents, as the student's, use the
    // rounded c2: both sides of their log-partitions then agree
    const double a = kTail ? log2p(t, P.c2d, lse2_t) : ((double)t - (double)n.tm) * (double)P.c2;
    const float p = kTail ? ex2((float)a) : n.inv_ts != 0.f ? ex2((float)a) * n.inv_ts : 0.f;
    if (p != 0.f) {
      part += (double)p * (a - ((double)z - (double)n.m) * (double)P.c2);
      mass += p;
    }
    if (gs && LQ_IN_RANGE(sl.c0 + e, P.V))
      Log<T>::put(gs + e, n.f_top * ex2_from(z, n.m, P.c2) - scale * p);
  });
  {
    const double pd = warp_sum(part);
    const float mf = warp_sum(mass);
    if (lane == 0) sm_d[0][warp] = pd, sm_d[1][warp] = mf;
  }
  __syncthreads();
  if (warp == 0) {
    const double l = warp_sum(lane < kWarps ? sm_d[0][lane] : 0.0);
    const double mass_d = warp_sum(lane < kWarps ? sm_d[1][lane] : 0.0);
    if (lane == 0) {
      // log2 q is b - log2 S; log2 p is a, less log2 of the listed exponentials'
      // sum where they are normalised here
      const double sum = mass_d > 0.0 ? l + mass_d * log2(kTail ? total : total / TS) : l;
      if (n_parts > 1)
        *cluster.map_shared_rank(&loss_parts[rank], 0) = sum;
      else
        loss_parts[0] = sum;
    }
  }
  if (n_parts > 1) cluster.sync();  // the loss parts have arrived; no CTA leaves before
  if (tid == 0 && rank == 0) {
    double l = 0.0;
    for (int r = 0; r < n_parts; ++r) l += loss_parts[r];
    l *= 0.6931471805599453;
    if (kTail && R > 0.0)
      l += R * (log(R * total / S) - to_top * 0.6931471805599453);
    P.loss[row] = (float)((double)w * l);
  }
}

template <typename T, bool kTail, int kThreads, int kUnroll, int kCtas>
cudaError_t run(const DistillParams& P, int parts, cudaStream_t s) {
  auto* k = k_distill<T, kTail, kThreads, kUnroll, kCtas>;
  const size_t smem = P.slice / 8 + (size_t)P.k * 12;
  static std::atomic<uint64_t> smem_set{0};  // one bit per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !((smem_set.load() >> dev) & 1u)) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) smem_set.fetch_or(1ull << dev);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(P.M * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, P);
}

template <typename T, bool kTail>
cudaError_t run_size(const DistillParams& P, int parts, cudaStream_t s) {
  // Threads and loads in flight by the length of a slice: a short row is all
  // latency, and small CTAs put more rows on an SM at once (4000 rows of 1003 bf16
  // logits with gradient: 70 us with 512 threads, 25 with 128, 16 with 64 and half the
  // loads in flight; 1000 rows of 8001 float32: 17 with that, 14 with 128 and all of
  // them).
  const size_t bytes = P.slice * sizeof(T);
  if (bytes <= 8 * 1024) return run<T, kTail, 64, 2, 20>(P, parts, s);
  if (bytes <= 32 * 1024) return run<T, kTail, 128, 4, 8>(P, parts, s);
  return run<T, kTail, 256, 4, 4>(P, parts, s);
}

template <typename T>
cudaError_t run_tail(const DistillParams& P, int parts, cudaStream_t s) {
  return P.t_lse ? run_size<T, true>(P, parts, s) : run_size<T, false>(P, parts, s);
}

}  // namespace

unsigned long long bounds_fail_distill() { return lq_take_bounds_fail(); }

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s) {
  const int64_t esz = a.dtype == LQ_F32 ? 4 : 2;
  // CTAs per row: one, unless the rows are too few to keep the SMs busy and a
  // slice is still worth its own CTA
  int parts = 1;
  auto slice_of = [&](int n) { return ((a.V + 8 + n - 1) / n + 31) / 32 * 32; };
  while (parts < kMaxCluster && a.M * parts < 2 * num_sms() && slice_of(parts) * esz > 8 * 1024)
    parts *= 2;
  DistillParams P{};
  P.z = a.z;
  P.grad = a.grad;
  P.t = a.t;
  P.idx = a.idx;
  P.t_lse = a.t_lse;
  P.weight = a.weight;
  P.loss = a.loss;
  P.M = a.M;
  P.V = a.V;
  P.k = a.k;
  P.t_dtype = a.t_dtype;
  P.idx64 = a.idx64;
  P.slice = (int)slice_of(parts);
  P.ahead = a.M * parts > 8 * num_sms();
  P.temp = a.temp;
  P.inv_temp = 1.f / a.temp;
  P.c2d = 1.4426950408889634 / (double)a.temp;
  P.c2 = (float)P.c2d;
  if (a.dtype == LQ_F32) return run_tail<float>(P, parts, s);
  if (a.dtype == LQ_BF16) return run_tail<__nv_bfloat16>(P, parts, s);
  return run_tail<__half>(P, parts, s);
}

}  // namespace lq
