// Distillation from a teacher's top logits: loss and gradient of the student's
// logits, row by row.
//
// Row m has V student logits z and k listed teacher logits t_i at vocabulary
// indices v_i.  With temperature T, q = softmax(z / T) and
//   no rest class:  p = softmax(t / T) over the listed entries, R = 0;
//   rest class:     p_i = exp(t_i / T - L) with the teacher's log-partition L,
//                   R = max(0, 1 - sum p) for everything that is not listed;
//   loss = w (sum_i p_i (log p_i - log q_{v_i}) + R (log R - log Q_rest)),
//   dz_j = w / T (C q_j - p_j)                 j listed, C = sum p + R
//   dz_j = w / T  q_j (C - R S / S_rest)       otherwise,
// S the sum of exp(z / T) over the vocabulary and S_rest that over the entries
// that are not listed, Q_rest = S_rest / S.  S_rest is summed directly (not as
// a difference, which loses everything when the listed entries hold nearly
// all of the student's mass).
//
// What bounds it is memory: each logit is read once and each gradient written
// once.  A row (or, over a cluster of 2, 4 or 8 CTAs, an equal slice of it) is
// brought to shared memory by one bulk copy, reduced there (maximum, sum), the
// few numbers of the slices are exchanged through distributed shared memory,
// the gradient replaces the logits in place, the listed entries' gradients are
// put over it, and one bulk copy writes the slice back.  Next to memory it is
// the exponential unit (two exponentials per logit, 16 per clock and SM) that
// sets the pace; the passes therefore use packed maxima, two-lane float32
// arithmetic and nothing per element that could be done per row.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "lq_dense.cuh"

namespace lq {
namespace {

namespace cg = cooperative_groups;

constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s
constexpr int kKeep = 2;  // listed entries a thread keeps in registers
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kNegInf = -INFINITY;

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

__device__ int g_distill_status = 0;

struct DistillParams {
  const void* z;
  void* grad;
  const void* t;
  const void* idx;
  const float* t_lse;
  const float* weight;
  float* loss;
  int64_t V;
  int k, t_dtype, idx64;
  int slice;  // elements per CTA, a multiple of 32
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
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// what a slice tells the others
struct Part {
  float m, tm;       // maximum of its logits, of its teacher entries
  double s, top;     // sum over its logits (rest class: those not listed), listed ones
  double ts;         // sum over its teacher entries (rest class: of p)
};
// a row's numbers, worked out by one thread
struct RowNumbers {
  float m2;      // exponents are z c2 - m2
  float f_rest;  // gradient of an entry that is not listed, over its exponential
  float f_top;   // C / S times the scale, the same for listed entries
  double p_sub;  // log2 of a listed p is t c2 - p_sub
  double q_sub;  // log2 q is z c2 - q_sub
  int has_p;     // the listed entries carry mass
  double tail;   // the rest class's share of the loss
};

__device__ __forceinline__ void block_max2(float& a, float& b, float* sm) {
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  a = warp_max(a);
  b = warp_max(b);
  if (l == 0) sm[w] = a, sm[kWarps + w] = b;
  __syncthreads();
  a = warp_max(sm[l % kWarps]);
  b = warp_max(sm[kWarps + l % kWarps]);
}

// log2 p of a listed entry, in float64: logit and log-partition may be far larger
// than their difference, and the mass that is not listed, 1 - sum p, may be small
__device__ __forceinline__ double log2p(float t, double c2d, double lse2) {
  return (double)t * c2d - lse2;
}

template <typename T, bool kTail>
__global__ void __launch_bounds__(kThreads, 2) k_distill(const DistillParams P) {
  constexpr int kE = Log<T>::kE;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Part parts[kMaxCluster];
  __shared__ double loss_parts[kMaxCluster];
  __shared__ double sm_d[3][kWarps];
  __shared__ float sm_f[2 * kWarps];
  __shared__ RowNumbers row_n;
  __shared__ __align__(8) unsigned long long bar;
  __shared__ int flags;  // 1: an entry is in range, 2: an index is listed again
  cg::cluster_group cluster = cg::this_cluster();
  const int n_parts = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / n_parts;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  T* zs = reinterpret_cast<T*>(smem);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + (size_t)P.slice * sizeof(T));

  pdl_trigger();
  if (tid == 0) {
    mbar_init(smem_u32(&bar), 1);
    fence_mbar_init();
    flags = 0;
  }
  for (int i = tid; i < P.slice / 32; i += kThreads) bits[i] = 0u;
  pdl_wait();
  __syncthreads();
  const float w = P.weight ? P.weight[row] : 1.f;
  // columns are counted from the 16-byte boundary at or before the row's
  // start: column j of the row is j + lead; this slice holds [c0, c0 + slice)
  const T* zrow = (const T*)P.z + row * P.V;
  T* grow = P.grad ? (T*)P.grad + row * P.V : nullptr;
  const int lead = (int)(((uintptr_t)zrow & 15u) / sizeof(T));
  const int64_t c0 = (int64_t)rank * P.slice - lead;  // row column of slice element 0
  const int lo = (int)(c0 < 0 ? -c0 : 0);             // first valid slice element
  const int64_t left = P.V - c0;
  const int hi = (int)(left < 0 ? 0 : left < P.slice ? left : P.slice);  // end of the valid ones
  // whole 16-byte vectors, and the few elements before and after them
  const int v_lo = (lo + kE - 1) / kE, v_hi = max(v_lo, hi / kE);
  const int edge0 = min(hi, v_lo * kE) - lo, edge1 = max(0, hi - v_hi * kE);
  // element of edge number i < edge0 + edge1
  auto edge_at = [&](int i) { return i < edge0 ? lo + i : v_hi * kE + (i - edge0); };
  const int n_edge = max(0, edge0) + (v_hi * kE < hi ? edge1 : 0);

  auto zero_row = [&]() {
    if (rank == 0 && tid == 0) P.loss[row] = 0.f;
    if (!grow) return;
    for (int v = v_lo + tid; v < v_hi; v += kThreads)
      *reinterpret_cast<uint4*>(grow + c0 + (int64_t)v * kE) = make_uint4(0, 0, 0, 0);
    if (tid < n_edge) Log<T>::put(grow + c0 + edge_at(tid), 0.f);
  };
  // a row of weight 0 counts nothing, whatever its logits hold
  if (w == 0.f) {
    zero_row();  // the same decision in every CTA of the cluster
    return;
  }
  if (n_parts > 1) cluster.barrier_arrive();  // this CTA runs: its shared memory may be written
  const uint32_t bar_a = smem_u32(&bar);
  const uint32_t copy_bytes = (uint32_t)(v_hi - v_lo) * 16u;
  if (tid == 0 && copy_bytes) {
    mbar_arrive_expect_tx(bar_a, copy_bytes);
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
            "r"(smem_u32(zs + v_lo * kE)),
        "l"(zrow + c0 + (int64_t)v_lo * kE), "r"(copy_bytes), "r"(bar_a)
        : "memory");
  }
  if (tid < n_edge) zs[edge_at(tid)] = zrow[c0 + edge_at(tid)];

  // While the row travels: the listed entries.  Those of this slice are marked
  // in a bitmap; a thread keeps its first ones (position in the slice, -1 for
  // none, and teacher logit).
  const int64_t list = row * P.k;
  auto slice_pos = [&](int i, bool& valid) -> int {
    const int64_t v = index_at(P, list + i);
    const int64_t e = v - c0;
    valid = v >= 0 && v < P.V;
    return valid && e >= lo && e < hi ? (int)e : -1;
  };
  int keep_e[kKeep];
  float keep_t[kKeep];
  bool any = false, dup = false;
#pragma unroll
  for (int r = 0; r < kKeep; ++r) {
    const int i = tid + r * kThreads;
    keep_e[r] = -1;
    keep_t[r] = 0.f;
    if (i < P.k) {
      bool ok;
      keep_e[r] = slice_pos(i, ok);
      keep_t[r] = teacher_at(P, list + i);
      any |= ok;
    }
  }
#pragma unroll
  for (int r = 0; r < kKeep; ++r)
    if (keep_e[r] >= 0) {
      const uint32_t b = 1u << (keep_e[r] & 31);
      dup |= (atomicOr(&bits[keep_e[r] >> 5], b) & b) != 0;
    }
  for (int i = tid + kKeep * kThreads; i < P.k; i += kThreads) {
    bool ok;
    const int e = slice_pos(i, ok);
    any |= ok;
    if (e >= 0) {
      const uint32_t b = 1u << (e & 31);
      dup |= (atomicOr(&bits[e >> 5], b) & b) != 0;
    }
  }
  any = __any_sync(~0u, any);
  dup = __any_sync(~0u, dup);
  if (lane == 0 && (any || dup)) atomicOr(&flags, (any ? 1 : 0) | (dup ? 2 : 0));
  __syncthreads();
  any = flags & 1;
  dup = flags & 2;
  // an index that is listed again counts at its first position only
  auto first_of = [&](int i) {
    const int64_t v = index_at(P, list + i);
    for (int j = 0; j < i; ++j)
      if (index_at(P, list + j) == v) return false;
    return true;
  };
  if (dup) {
#pragma unroll
    for (int r = 0; r < kKeep; ++r)
      if (keep_e[r] >= 0 && !first_of(tid + r * kThreads)) keep_e[r] = -1;
  }
  // fn(position, teacher logit) for this thread's entries of the slice
  auto for_entries = [&](auto&& fn) {
#pragma unroll
    for (int r = 0; r < kKeep; ++r)
      if (keep_e[r] >= 0) fn(keep_e[r], keep_t[r]);
    for (int i = tid + kKeep * kThreads; i < P.k; i += kThreads) {
      bool ok;
      const int e = slice_pos(i, ok);
      if (e >= 0 && (!dup || first_of(i))) fn(e, teacher_at(P, list + i));
    }
  };
  float tm = kNegInf;
  if (!kTail) for_entries([&](int, float t) { tm = fmaxf(tm, t); });

  // the row has arrived
  if (copy_bytes) {
    if (!mbar_try_wait(bar_a, 0u)) {
      uint64_t t0 = 0;
      for (uint32_t i = 1; !mbar_try_wait(bar_a, 0u); ++i) {
        if (i & 1023u) continue;
        const uint64_t t = global_timer_ns();
        if (t0 == 0) t0 = t;
        // recorded for lq_check_device; the CTA goes on (to its cluster's
        // barriers), with whatever has arrived
        if (t - t0 > kWaitLimitNs) {
          atomicExch(&g_distill_status, (int)LQ_ERR_DEVICE_TIMEOUT);
          break;
        }
      }
    }
  }

  // maxima
  uint4* vec = reinterpret_cast<uint4*>(zs);
  typename Log<T>::Run run = Log<T>::run_start();
  for (int v = v_lo + tid; v < v_hi; v += kThreads) run = Log<T>::run_max(run, vec[v]);
  float m = Log<T>::run_end(run);
  if (tid < n_edge) m = fmaxf(m, Log<T>::get(zs + edge_at(tid)));
  block_max2(m, tm, sm_f);

  // sums, relative to the slice's maxima; base-2 exponents z c2 - m2
  const float m2 = m == kNegInf ? 0.f : m * P.c2;
  const float2 c2v = make_float2(P.c2, P.c2), nm2 = make_float2(-m2, -m2);
  float2 s2 = make_float2(0.f, 0.f);
  for (int v = v_lo + tid; v < v_hi; v += kThreads) {
    float f[kE];
    Log<T>::unpack(vec[v], f);
    if (kTail) {
      const uint32_t mark = bits[(v * kE) >> 5] >> ((v * kE) & 31);
#pragma unroll
      for (int i = 0; i < kE; ++i)
        if ((mark >> i) & 1u) f[i] = kNegInf;
    }
#pragma unroll
    for (int i = 0; i < kE; i += 2) {
      const float2 x = ffma2(make_float2(f[i], f[i + 1]), c2v, nm2);
      s2 = fadd2(s2, make_float2(ex2(x.x), ex2(x.y)));
    }
  }
  float s = s2.x + s2.y;
  if (tid < n_edge) {
    const int e = edge_at(tid);
    if (!kTail || !((bits[e >> 5] >> (e & 31)) & 1u))
      s += ex2(fmaf(Log<T>::get(zs + e), P.c2, -m2));
  }
  float top = 0.f, ts = 0.f;
  const double lse2_t = kTail ? (double)P.t_lse[row] * 1.4426950408889634 : 0.0;
  for_entries([&](int e, float t) {
    if (kTail) {
      top += ex2(fmaf(Log<T>::get(zs + e), P.c2, -m2));
      ts += ex2((float)log2p(t, P.c2d, lse2_t));
    } else if (tm != kNegInf) {
      ts += ex2((t - tm) * P.c2);
    }
  });
  {
    const double sd = warp_sum((double)s), td = warp_sum((double)ts);
    const double pd = kTail ? warp_sum((double)top) : 0.0;
    if (lane == 0) sm_d[0][warp] = sd, sm_d[1][warp] = td, sm_d[2][warp] = pd;
  }
  __syncthreads();
  if (n_parts > 1) cluster.barrier_wait();
  if (warp == 0) {
    const double sd = warp_sum(lane < kWarps ? sm_d[0][lane] : 0.0);
    const double td = warp_sum(lane < kWarps ? sm_d[1][lane] : 0.0);
    const double pd = kTail ? warp_sum(lane < kWarps ? sm_d[2][lane] : 0.0) : 0.0;
    if (lane < n_parts) {
      Part* dst = n_parts > 1 ? cluster.map_shared_rank(&parts[rank], lane) : &parts[0];
      dst->m = m;
      dst->tm = tm;
      dst->s = sd;
      dst->top = pd;
      dst->ts = td;
    }
  }
  if (n_parts > 1)
    cluster.sync();
  else
    __syncthreads();

  // the row's numbers, from the slices in order
  if (tid == 0) {
    float M = kNegInf, TM = kNegInf;
    for (int r = 0; r < n_parts; ++r) {
      M = fmaxf(M, parts[r].m);
      TM = fmaxf(TM, parts[r].tm);
    }
    const float M2 = M == kNegInf ? 0.f : M * P.c2;
    double S = 0.0, Top = 0.0, TS = 0.0;
    for (int r = 0; r < n_parts; ++r) {
      const Part& q = parts[r];
      const double f = q.m == M ? 1.0 : q.m == kNegInf ? 0.0 : exp2((double)(q.m * P.c2) - M2);
      S += q.s * f;
      Top += q.top * f;
      TS += kTail          ? q.ts
            : q.tm == TM   ? q.ts
            : q.tm == kNegInf ? 0.0
                              : q.ts * exp2(((double)q.tm - TM) * P.c2d);
    }
    const double total = kTail ? S + Top : S;
    const double R = kTail && 1.0 - TS > 0.0 ? 1.0 - TS : 0.0;
    const bool has_p = TS > 0.0;
    const double C = kTail ? TS + R : (has_p ? 1.0 : 0.0);
    const bool has_rest = R > 0.0 && S > 0.0;
    const double lse2 = (double)M2 + log2(total);  // log2 sum exp(z / T)
    const double lp2 = kTail ? lse2_t : (double)TM * P.c2d + log2(TS);
    const double scale = (double)w / (double)P.temp;
    RowNumbers n;
    n.m2 = M2;
    n.f_rest = (float)(scale * (C - (has_rest ? R * total / S : 0.0)) / total);
    n.f_top = (float)(scale * C / total);
    n.p_sub = lp2;
    n.q_sub = lse2;
    n.has_p = has_p;
    n.tail = has_rest ? R * (log(R) - log(S / total)) : 0.0;
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

  // the gradient of entries that are not listed, in place; the listed ones
  // read their logits first
  const float scale = w * P.inv_temp;
  float part = 0.f;
  float keep_g[kKeep];
  auto entry_loss = [&](float t, float z) -> float {  // returns the entry's gradient
    const double lp = log2p(t, P.c2d, n.p_sub);
    const float p = !n.has_p ? 0.f : ex2((float)lp);
    if (p != 0.f) part = fmaf(p, (float)(lp - ((double)z * (double)P.c2 - n.q_sub)), part);
    return n.f_top * ex2(fmaf(z, P.c2, -n.m2)) - scale * p;
  };
#pragma unroll
  for (int r = 0; r < kKeep; ++r)
    if (keep_e[r] >= 0) keep_g[r] = entry_loss(keep_t[r], Log<T>::get(zs + keep_e[r]));
  if (grow) {
    __syncthreads();
    const float2 fr = make_float2(n.f_rest, n.f_rest), nn = make_float2(-n.m2, -n.m2);
    for (int v = v_lo + tid; v < v_hi; v += kThreads) {
      float f[kE];
      Log<T>::unpack(vec[v], f);
#pragma unroll
      for (int i = 0; i < kE; i += 2) {
        const float2 x = ffma2(make_float2(f[i], f[i + 1]), c2v, nn);
        const float2 g = fmul2(make_float2(ex2(x.x), ex2(x.y)), fr);
        f[i] = g.x;
        f[i + 1] = g.y;
      }
      vec[v] = Log<T>::pack(f);
    }
    if (tid < n_edge) {
      T* p = zs + edge_at(tid);
      Log<T>::put(p, n.f_rest * ex2(fmaf(Log<T>::get(p), P.c2, -n.m2)));
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kKeep; ++r)
      if (keep_e[r] >= 0) Log<T>::put(zs + keep_e[r], keep_g[r]);
  }
  // entries beyond those kept: their logits are read again (nothing of the
  // row has been written yet)
  for (int i = tid + kKeep * kThreads; i < P.k; i += kThreads) {
    bool ok;
    const int e = slice_pos(i, ok);
    if (e < 0 || (dup && !first_of(i))) continue;
    const float g = entry_loss(teacher_at(P, list + i), Log<T>::get(zrow + c0 + e));
    if (grow) Log<T>::put(zs + e, g);
  }
  {
    const double pd = warp_sum((double)part);
    if (lane == 0) sm_d[0][warp] = pd;
  }
  if (grow) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncthreads();
  if (tid == 0) {
    if (grow && copy_bytes) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                       grow + c0 + (int64_t)v_lo * kE),
                   "r"(smem_u32(zs + v_lo * kE)), "r"(copy_bytes)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
    double l = 0.0;
    for (int i = 0; i < kWarps; ++i) l += sm_d[0][i];
    if (n_parts > 1)
      *cluster.map_shared_rank(&loss_parts[rank], 0) = l;
    else
      loss_parts[0] = l;
  }
  if (grow && tid < n_edge) grow[c0 + edge_at(tid)] = zs[edge_at(tid)];
  if (n_parts > 1) cluster.sync();  // the loss parts have arrived; no CTA leaves before
  if (tid == 0) {
    if (rank == 0) {
      double l = 0.0;
      for (int r = 0; r < n_parts; ++r) l += loss_parts[r];
      P.loss[row] = (float)((double)w * (l * 0.6931471805599453 + n.tail));
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

template <typename T, bool kTail>
cudaError_t run(const DistillParams& P, int64_t M, int parts, cudaStream_t s) {
  auto* k = k_distill<T, kTail>;
  const size_t smem = (size_t)P.slice * sizeof(T) + P.slice / 8;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(M * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)parts;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, P);
}

template <typename T>
cudaError_t run_tail(const DistillParams& P, int64_t M, int parts, cudaStream_t s) {
  return P.t_lse ? run<T, true>(P, M, parts, s) : run<T, false>(P, M, parts, s);
}

}  // namespace

int take_distill_status() {
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_distill_status, sizeof(int)) != cudaSuccess) return 0;
  if (v) cudaMemcpyToSymbol(g_distill_status, &zero, sizeof(int));
  return v;
}

cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s) {
  const int64_t esz = a.dtype == LQ_F32 ? 4 : 2;
  // CTAs per row: as few as let two of them share an SM (their copies and
  // passes then overlap), more while the SMs are not all busy and a slice
  // still is worth its own CTA
  int parts = 1;
  auto slice_of = [&](int n) { return ((a.V + 8 + n - 1) / n + 31) / 32 * 32; };
  while (parts < kMaxCluster && slice_of(parts) * esz > 100 * 1024) parts *= 2;
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
  P.V = a.V;
  P.k = a.k;
  P.t_dtype = a.t_dtype;
  P.idx64 = a.idx64;
  P.slice = (int)slice_of(parts);
  P.temp = a.temp;
  P.inv_temp = 1.f / a.temp;
  P.c2d = 1.4426950408889634 / (double)a.temp;
  P.c2 = (float)P.c2d;
  if (a.dtype == LQ_F32) return run_tail<float>(P, a.M, parts, s);
  if (a.dtype == LQ_BF16) return run_tail<__nv_bfloat16>(P, a.M, parts, s);
  return run_tail<__half>(P, a.M, parts, s);
}

}  // namespace lq
