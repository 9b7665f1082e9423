// Launch interface of the dense products (lq_dense.cu) and the distillation
// loss (lq_distill.cu).
#pragma once

#include "lq_common.cuh"

namespace lq {

// one lane of a converged warp.  The roles that issue TMA copies and MMAs run
// with the whole warp and let the elected lane issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

constexpr int64_t kDenseRowsMax = 16;  // rows up to which the weight-streaming kernel runs

// y = act(x w^T + bias) + res, or with w2 y = act(x w^T + bias) * (x w2^T + bias2);
// aux (and aux2): the pre-activation (both factors), or null
struct DenseForward {
  const void *x, *w, *w2, *bias, *bias2, *res;
  void *y, *aux, *aux2;
  int64_t M, N, K;
  int dtype, act;
};
cudaError_t launch_dense_forward(const DenseForward& d, cudaStream_t s);

// workspace layout of a backward call: dz (M x ldz), then the row blocks'
// partial column sums, then the slices of a product cut along its contraction
struct DenseBwdPlan {
  bool copy;  // dz is written (else dy serves as it is)
  int64_t ldz, dz_bytes, rows, sum_bytes, slice_bytes;
  int row_blocks;
};
DenseBwdPlan dense_bwd_plan(int64_t M, int64_t N, int64_t K, bool gated, bool act);

struct DenseBackward {
  const void *dy, *z, *u, *x, *w, *w2;
  void *dx, *dw, *dw2, *db, *db2;
  void* ws;
  int64_t M, N, K;
  int dtype, act, f32, accumulate;
  bool gated;  // u, w2, dw2, db2 belong to the call
};
cudaError_t launch_dense_backward(const DenseBackward& d, cudaStream_t s);

// distillation loss and gradient (see lq_distill_loss)
struct DistillArgs {
  const void *z, *t, *idx;
  const float *t_lse, *weight;
  float* loss;
  void* grad;
  int64_t M, V;
  int k, dtype, t_dtype, idx64;
  float temp;
};
cudaError_t launch_distill(const DistillArgs& a, cudaStream_t s);

// the dense kernels' status word (LQ_ERR_DEVICE_TIMEOUT after a bounded wait
// expired), read and cleared; an error where it could not be
cudaError_t take_dense_status(int* status);
cudaError_t launch_dense_wait_selftest(uint64_t limit_ns, cudaStream_t s);

// per source file: the first index out of range of the bounds-check build (0: none)
unsigned long long bounds_fail_dense();
unsigned long long bounds_fail_distill();

}  // namespace lq
