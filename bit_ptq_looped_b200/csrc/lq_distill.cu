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
// copied to shared memory, reduced there (maximum, sum), the few numbers of
// the slices are exchanged through distributed shared memory, and the gradient
// is written from the same copy.  Listed entries are marked in a bitmap of the
// slice; their final gradients replace their logits in shared memory, so the
// output pass writes every value once, in order.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "lq_dense.cuh"

namespace lq {
namespace {

namespace cg = cooperative_groups;

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
  int64_t V;
  int k, t_dtype, idx64;
  int slice;  // elements per CTA, a multiple of 32
  float temp, inv_temp;
  float c2;  // log2(e) / temp
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

// block-wide maximum of two values / sums of three, in a fixed order
__device__ void block_max2(float& a, float& b, float* sm) {
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  a = warp_max(a);
  b = warp_max(b);
  if (l == 0) sm[w] = a, sm[kWarps + w] = b;
  __syncthreads();
  a = sm[l % kWarps];
  b = sm[kWarps + l % kWarps];
  a = warp_max(a);
  b = warp_max(b);
  __syncthreads();
}
__device__ void block_sum3(double& a, double& b, double& c, double* sm) {
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  a = warp_sum(a);
  b = warp_sum(b);
  c = warp_sum(c);
  if (l == 0) sm[w] = a, sm[kWarps + w] = b, sm[2 * kWarps + w] = c;
  __syncthreads();
  a = warp_sum(l < kWarps ? sm[l] : 0.0);
  b = warp_sum(l < kWarps ? sm[kWarps + l] : 0.0);
  c = warp_sum(l < kWarps ? sm[2 * kWarps + l] : 0.0);
  __syncthreads();
}

template <typename T, bool kTail>
__global__ void __launch_bounds__(kThreads, 2) k_distill(const DistillParams P) {
  constexpr int kE = Log<T>::kE;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ Part parts[kMaxCluster];
  __shared__ double loss_parts[kMaxCluster];
  __shared__ double sm_d[3 * kWarps];
  __shared__ float sm_f[2 * kWarps];
  cg::cluster_group cluster = cg::this_cluster();
  const int n_parts = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / n_parts;
  const int tid = threadIdx.x;
  T* zs = reinterpret_cast<T*>(smem);
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem + (size_t)P.slice * sizeof(T));

  pdl_trigger();
  pdl_wait();
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
  const int v_lo = (lo + kE - 1) / kE, v_hi = hi / kE;  // whole 16-byte vectors

  // entries in range; without any (or with weight 0) the row counts nothing,
  // whatever its logits hold
  bool any = false;
  for (int i = tid; i < P.k; i += kThreads) {
    const int64_t v = index_at(P, row * P.k + i);
    any |= v >= 0 && v < P.V;
  }
  any = __syncthreads_or(any);
  if (w == 0.f || (!kTail && !any)) {
    if (rank == 0 && tid == 0) P.loss[row] = 0.f;
    if (grow)
      for (int e = lo + tid; e < hi; e += kThreads) Log<T>::put(grow + c0 + e, 0.f);
    return;  // the same decision in every CTA of the cluster
  }

  cluster.barrier_arrive();  // this CTA runs: its shared memory may be written
  // copy the slice; meanwhile mark the listed entries
  for (int v = v_lo + tid; v < v_hi; v += kThreads)
    cp_async16(smem_u32(zs + v * kE), zrow + c0 + (int64_t)v * kE);
  cp_async_commit();
  for (int e = lo + tid; e < min(hi, v_lo * kE); e += kThreads) zs[e] = zrow[c0 + e];
  for (int e = max(v_lo, v_hi) * kE + tid; e < hi; e += kThreads) zs[e] = zrow[c0 + e];
  for (int i = tid; i < P.slice / 32; i += kThreads) bits[i] = 0u;
  __syncthreads();
  bool dup = false;
  for (int i = tid; i < P.k; i += kThreads) {
    const int64_t v = index_at(P, row * P.k + i);
    const int64_t e = v - c0;
    if (v >= 0 && v < P.V && e >= lo && e < hi) {
      const uint32_t b = 1u << (e & 31);
      dup |= (atomicOr(&bits[e >> 5], b) & b) != 0;
    }
  }
  dup = __syncthreads_or(dup);
  // entry i of this row belongs to this slice (its position there, else -1);
  // an index that is listed again counts at its first position only
  auto entry = [&](int i) -> int {
    const int64_t v = index_at(P, row * P.k + i);
    const int64_t e = v - c0;
    if (v < 0 || v >= P.V || e < lo || e >= hi) return -1;
    if (dup)
      for (int j = 0; j < i; ++j)
        if (index_at(P, row * P.k + j) == v) return -1;
    return (int)e;
  };
  cp_async_wait<0>();
  __syncthreads();

  // maxima
  const uint4* vec = reinterpret_cast<const uint4*>(zs);
  float m = kNegInf, tm = kNegInf;
  for (int v = v_lo + tid; v < v_hi; v += kThreads) {
    float f[kE];
    Log<T>::unpack(vec[v], f);
#pragma unroll
    for (int i = 0; i < kE; ++i) m = fmaxf(m, f[i]);
  }
  for (int e = lo + tid; e < min(hi, v_lo * kE); e += kThreads) m = fmaxf(m, Log<T>::get(zs + e));
  for (int e = max(v_lo, v_hi) * kE + tid; e < hi; e += kThreads) m = fmaxf(m, Log<T>::get(zs + e));
  if (!kTail)
    for (int i = tid; i < P.k; i += kThreads)
      if (entry(i) >= 0) tm = fmaxf(tm, teacher_at(P, row * P.k + i));
  block_max2(m, tm, sm_f);

  // sums, relative to the slice's maxima; base-2 exponents z c2 - m2
  const float m2 = m == kNegInf ? 0.f : m * P.c2;
  float s = 0.f;
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
    for (int i = 0; i < kE; ++i) s += ex2(fmaf(f[i], P.c2, -m2));
  }
  for (int e = lo + tid; e < hi; e += kThreads) {
    if (e >= v_lo * kE && e < v_hi * kE) continue;
    if (kTail && ((bits[e >> 5] >> (e & 31)) & 1u)) continue;
    s += ex2(fmaf(Log<T>::get(zs + e), P.c2, -m2));
  }
  double top = 0.0, ts = 0.0;
  const float lse = kTail ? P.t_lse[row] : 0.f;
  for (int i = tid; i < P.k; i += kThreads) {
    const int e = entry(i);
    if (e < 0) continue;
    const float t = teacher_at(P, row * P.k + i);
    if (kTail) {
      top += ex2(fmaf(Log<T>::get(zs + e), P.c2, -m2));
      ts += exp((double)t / P.temp - (double)lse);
    } else if (tm != kNegInf) {
      ts += expf((t - tm) * P.inv_temp);
    }
  }
  double sd = s;
  block_sum3(sd, top, ts, sm_d);
  cluster.barrier_wait();
  if (tid < n_parts) {
    Part* dst = cluster.map_shared_rank(&parts[rank], tid);
    dst->m = m;
    dst->tm = tm;
    dst->s = sd;
    dst->top = top;
    dst->ts = ts;
  }
  cluster.sync();

  // the row's numbers, from the slices in order (every thread the same)
  float M = kNegInf, TM = kNegInf;
  for (int r = 0; r < n_parts; ++r) {
    M = fmaxf(M, parts[r].m);
    TM = fmaxf(TM, parts[r].tm);
  }
  const float M2 = M == kNegInf ? 0.f : M * P.c2;
  double S = 0.0, Top = 0.0, TS = 0.0;
  for (int r = 0; r < n_parts; ++r) {
    const float pm2 = parts[r].m == kNegInf ? 0.f : parts[r].m * P.c2;
    const double f = parts[r].m == kNegInf ? 0.0 : exp2((double)pm2 - (double)M2);
    S += parts[r].s * f;
    Top += parts[r].top * f;
    TS += kTail ? parts[r].ts
          : parts[r].tm == kNegInf ? 0.0
                                   : parts[r].ts * exp(((double)parts[r].tm - (double)TM) / P.temp);
  }
  const double rest = S, total = kTail ? S + Top : S;
  const double R = kTail ? (1.0 - TS > 0.0 ? 1.0 - TS : 0.0) : 0.0;
  const double Cm = kTail ? TS + R : (TS > 0.0 ? 1.0 : 0.0);
  const bool has_rest = kTail && R > 0.0 && rest > 0.0;
  const double lse2 = (double)M2 + log2(total);          // log2 sum exp(z / T)
  const double log_p0 = kTail ? (double)lse : (double)TM / P.temp + log(TS);
  const float scale = w * P.inv_temp;
  const float inv_total = (float)(1.0 / total);
  const float f_rest = scale * (float)((Cm - (has_rest ? R * total / rest : 0.0)) / total);
  constexpr double kLn2 = 0.6931471805599453;

  // listed entries: loss, and the final gradient in place of the logit
  double part = 0.0;
  for (int i = tid; i < P.k; i += kThreads) {
    const int e = entry(i);
    if (e < 0) continue;
    const float t = teacher_at(P, row * P.k + i), z = Log<T>::get(zs + e);
    const double log_p = (double)t / P.temp - log_p0;
    const float p = (!kTail && !(TS > 0.0)) ? 0.f : (float)exp(log_p);
    const double log_q = ((double)z * P.c2 - lse2) * kLn2;
    if (p != 0.f) part += (double)p * (log_p - log_q);
    if (grow) Log<T>::put(zs + e, scale * ((float)Cm * ex2(fmaf(z, P.c2, -M2)) * inv_total - p));
  }
  double z1 = 0.0, z2 = 0.0;
  block_sum3(part, z1, z2, sm_d);  // also orders the entries' writes before the output pass
  if (tid == 0) *cluster.map_shared_rank(&loss_parts[rank], 0) = part;

  if (grow) {
    for (int v = v_lo + tid; v < v_hi; v += kThreads) {
      float f[kE], g[kE];
      Log<T>::unpack(vec[v], f);
      const uint32_t mark = bits[(v * kE) >> 5] >> ((v * kE) & 31);
#pragma unroll
      for (int i = 0; i < kE; ++i)
        g[i] = ((mark >> i) & 1u) ? f[i] : f_rest * ex2(fmaf(f[i], P.c2, -M2));
      *reinterpret_cast<uint4*>(grow + c0 + (int64_t)v * kE) = Log<T>::pack(g);
    }
    for (int e = lo + tid; e < hi; e += kThreads) {
      if (e >= v_lo * kE && e < v_hi * kE) continue;
      const float f = Log<T>::get(zs + e);
      Log<T>::put(grow + c0 + e, ((bits[e >> 5] >> (e & 31)) & 1u)
                                     ? f
                                     : f_rest * ex2(fmaf(f, P.c2, -M2)));
    }
  }
  cluster.sync();  // the loss parts have arrived; no CTA leaves while they do
  if (rank == 0 && tid == 0) {
    double l = 0.0;
    for (int r = 0; r < n_parts; ++r) l += loss_parts[r];
    if (has_rest) l += R * (log(R) - log(rest / total));
    P.loss[row] = (float)(l * (double)w);
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
  P.c2 = (float)(1.4426950408889634 / (double)a.temp);
  if (a.dtype == LQ_F32) return run_tail<float>(P, a.M, parts, s);
  if (a.dtype == LQ_BF16) return run_tail<__nv_bfloat16>(P, a.M, parts, s);
  return run_tail<__half>(P, a.M, parts, s);
}

}  // namespace lq
