// C ABI of the dense products and the distillation loss: argument checks and
// dispatch to the launches of lq_dense.cu and lq_distill.cu.
#include <cmath>

#include "lq_dense.cuh"

using namespace lq;

namespace {

constexpr int64_t kMaxExtent = ((int64_t)1 << 31) - 256;
constexpr int64_t kMaxElems = (int64_t)1 << 46;  // of a matrix; byte counts stay far below 2^63

bool bad_extent(int64_t M, int64_t N, int64_t K) {
  return M < 0 || N <= 0 || K <= 0 || M > kMaxExtent || N > kMaxExtent || K > kMaxExtent ||
         M * N > kMaxElems || M * K > kMaxElems || N * K > kMaxElems;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

lq_status check_dense(int32_t dtype, int64_t M, int64_t N, int64_t K, int32_t act) {
  if (dtype != LQ_BF16 && dtype != LQ_F16) {
    set_error("dense operands are bf16 or f16 (dtype %d)", dtype);
    return LQ_ERR_UNSUPPORTED;
  }
  if (act < LQ_ACT_NONE || act > LQ_ACT_GELU_TANH) {
    set_error("unknown activation %d", act);
    return LQ_ERR_UNSUPPORTED;
  }
  if (M < 0 || N <= 0 || K <= 0) {
    set_error("invalid shape M=%lld N=%lld K=%lld", (long long)M, (long long)N, (long long)K);
    return LQ_ERR_ARG;
  }
  if (K % 8) {
    set_error("K=%lld is not a multiple of 8", (long long)K);
    return LQ_ERR_SHAPE;
  }
  if (bad_extent(M, N, K)) {
    set_error("M, N and K must be below 2^31 - 256 and a matrix at most 2^46 elements");
    return LQ_ERR_SHAPE;
  }
  return LQ_OK;
}

// a buffer of the call; written ones may overlap no other
struct Buf {
  const char* name;
  const void* p;
  int64_t bytes;
  bool out;
};

template <int n>
lq_status check_bufs(const Buf (&b)[n]) {
  for (int i = 0; i < n; ++i) {
    if (!aligned16(b[i].p)) {
      set_error("%s must be 16-byte aligned", b[i].name);
      return LQ_ERR_ALIGN;
    }
  }
  for (int i = 0; i < n; ++i) {
    if (!b[i].p || !b[i].out || b[i].bytes <= 0) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || !b[j].p || b[j].bytes <= 0 || (b[j].out && j < i)) continue;
      const uintptr_t a = (uintptr_t)b[i].p, c = (uintptr_t)b[j].p;
      if (a < c + (uintptr_t)b[j].bytes && c < a + (uintptr_t)b[i].bytes) {
        set_error("%s overlaps %s", b[i].name, b[j].name);
        return LQ_ERR_ARG;
      }
    }
  }
  return LQ_OK;
}

lq_status check_ws(const void* ws, int64_t have, int64_t need) {
  if (need <= 0) return LQ_OK;
  if (!ws) {
    set_error("null workspace");
    return LQ_ERR_ARG;
  }
  if ((uintptr_t)ws & 255u) {
    set_error("the workspace must be 256-byte aligned");
    return LQ_ERR_ALIGN;
  }
  if (have < need) {
    set_error("workspace too small: %lld bytes, %lld needed", (long long)have, (long long)need);
    return LQ_ERR_WORKSPACE;
  }
  return LQ_OK;
}

lq_status check_grads(int32_t dtype, int32_t g_dtype, int32_t accumulate) {
  if (g_dtype != dtype && g_dtype != LQ_F32) {
    set_error("weight gradients are of the operands' type or float32 (g_dtype %d)", g_dtype);
    return LQ_ERR_UNSUPPORTED;
  }
  if (accumulate && g_dtype != LQ_F32) {
    set_error("only float32 weight gradients accumulate");
    return LQ_ERR_UNSUPPORTED;
  }
  return LQ_OK;
}

lq_status null_pointer(const char* what) {
  set_error("null %s", what);
  return LQ_ERR_ARG;
}

// gradients over no rows
lq_status clear(void* p, int64_t bytes, cudaStream_t s) {
  if (!p) return LQ_OK;
  cudaError_t e = cudaMemsetAsync(p, 0, (size_t)bytes, s);
  return e == cudaSuccess ? LQ_OK : cuda_error(e, "clear gradient");
}

int64_t bwd_bytes(int64_t M, int64_t N, int64_t K, bool gated, bool act) {
  const DenseBwdPlan p = dense_bwd_plan(M, N, K, gated, act);
  return p.dz_bytes + p.sum_bytes + p.slice_bytes;
}

lq_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? LQ_OK : cuda_error(e, what);
}

}  // namespace

extern "C" {

lq_status lq_dense_linear(const void* d_x, const void* d_w, const void* d_bias,
                          const void* d_residual, int32_t dtype, int64_t M, int64_t N, int64_t K,
                          int32_t act, void* d_y, void* d_z, void* stream) {
  lq_status st = check_dense(dtype, M, N, K, act);
  if (st != LQ_OK || M == 0) return st;
  if (!d_x || !d_w || !d_y) return null_pointer("x, W or y");
  const Buf bufs[] = {{"x", d_x, M * K * 2, false},
                      {"W", d_w, N * K * 2, false},
                      {"the bias", d_bias, N * 2, false},
                      {"the residual", d_residual == d_y ? nullptr : d_residual, M * N * 2, false},
                      {"y", d_y, M * N * 2, true},
                      {"z", d_z, M * N * 2, true}};
  if ((st = check_bufs(bufs)) != LQ_OK) return st;
  DenseForward d{};
  d.x = d_x;
  d.w = d_w;
  d.bias = d_bias;
  d.res = d_residual;
  d.y = d_y;
  d.aux = d_z;
  d.M = M;
  d.N = N;
  d.K = K;
  d.dtype = dtype;
  d.act = act;
  return launched(launch_dense_forward(d, (cudaStream_t)stream), "dense linear launch");
}

int64_t lq_dense_linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t act) {
  return bad_extent(M, N, K) ? -1 : bwd_bytes(M, N, K, false, act != LQ_ACT_NONE);
}

lq_status lq_dense_linear_bwd(const void* d_dy, const void* d_z, const void* d_x,
                              const void* d_w, int32_t dtype, int64_t M, int64_t N, int64_t K,
                              int32_t act, void* d_dx, void* d_dw, void* d_db, int32_t g_dtype,
                              int32_t accumulate, void* d_ws, int64_t ws_bytes, void* stream) {
  lq_status st = check_dense(dtype, M, N, K, act);
  if (st == LQ_OK) st = check_grads(dtype, g_dtype, accumulate);
  if (st != LQ_OK) return st;
  const int64_t gsz = g_dtype == LQ_F32 ? 4 : 2;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t need = lq_dense_linear_bwd_workspace_bytes(M, N, K, act);
  const Buf bufs[] = {{"dy", d_dy, M * N * 2, false},   {"z", d_z, M * N * 2, false},
                      {"x", d_x, M * K * 2, false},     {"W", d_w, N * K * 2, false},
                      {"dx", d_dx, M * K * 2, true},    {"dw", d_dw, N * K * gsz, true},
                      {"db", d_db, N * gsz, true},      {"the workspace", d_ws, ws_bytes < need ? 0 : need, true}};
  if ((st = check_bufs(bufs)) != LQ_OK) return st;
  if (M == 0) {
    if (accumulate) return LQ_OK;
    if ((st = clear(d_dw, N * K * gsz, s)) != LQ_OK) return st;
    return clear(d_db, N * gsz, s);
  }
  if (!d_dx && !d_dw && !d_db) return LQ_OK;
  if (!d_dy || (act != LQ_ACT_NONE && !d_z) || (d_dx && !d_w) || (d_dw && !d_x))
    return null_pointer("dy, z, x or W");
  if ((st = check_ws(d_ws, ws_bytes, need)) != LQ_OK) return st;
  DenseBackward d{};
  d.dy = d_dy;
  d.z = d_z;
  d.x = d_x;
  d.w = d_w;
  d.dx = d_dx;
  d.dw = d_dw;
  d.db = d_db;
  d.ws = d_ws;
  d.M = M;
  d.N = N;
  d.K = K;
  d.dtype = dtype;
  d.act = act;
  d.f32 = g_dtype == LQ_F32;
  d.accumulate = accumulate != 0;
  return launched(launch_dense_backward(d, s), "dense linear backward launch");
}

lq_status lq_gated_linear(const void* d_x, const void* d_wg, const void* d_wu,
                          const void* d_bias_g, const void* d_bias_u, int32_t dtype, int64_t M,
                          int64_t N, int64_t K, int32_t act, void* d_h, void* d_g, void* d_u,
                          void* stream) {
  lq_status st = check_dense(dtype, M, N, K, act);
  if (st != LQ_OK) return st;
  if (!d_g != !d_u) {
    set_error("g and u are saved together or not at all");
    return LQ_ERR_ARG;
  }
  if (M == 0) return LQ_OK;
  if (!d_x || !d_wg || !d_wu || !d_h) return null_pointer("x, Wg, Wu or h");
  const Buf bufs[] = {{"x", d_x, M * K * 2, false},
                      {"Wg", d_wg, N * K * 2, false},
                      {"Wu", d_wu, N * K * 2, false},
                      {"the gate's bias", d_bias_g, N * 2, false},
                      {"the up bias", d_bias_u, N * 2, false},
                      {"h", d_h, M * N * 2, true},
                      {"g", d_g, M * N * 2, true},
                      {"u", d_u, M * N * 2, true}};
  if ((st = check_bufs(bufs)) != LQ_OK) return st;
  DenseForward d{};
  d.x = d_x;
  d.w = d_wg;
  d.w2 = d_wu;
  d.bias = d_bias_g;
  d.bias2 = d_bias_u;
  d.y = d_h;
  d.aux = d_g;
  d.aux2 = d_u;
  d.M = M;
  d.N = N;
  d.K = K;
  d.dtype = dtype;
  d.act = act;
  return launched(launch_dense_forward(d, (cudaStream_t)stream), "gated linear launch");
}

int64_t lq_gated_linear_bwd_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  return bad_extent(M, N, K) ? -1 : bwd_bytes(M, N, K, true, true);
}

lq_status lq_gated_linear_bwd(const void* d_dh, const void* d_g, const void* d_u,
                              const void* d_x, const void* d_wg, const void* d_wu, int32_t dtype,
                              int64_t M, int64_t N, int64_t K, int32_t act, void* d_dx,
                              void* d_dwg, void* d_dwu, void* d_dbg, void* d_dbu,
                              int32_t g_dtype, int32_t accumulate, void* d_ws, int64_t ws_bytes,
                              void* stream) {
  lq_status st = check_dense(dtype, M, N, K, act);
  if (st == LQ_OK) st = check_grads(dtype, g_dtype, accumulate);
  if (st != LQ_OK) return st;
  const int64_t gsz = g_dtype == LQ_F32 ? 4 : 2;
  cudaStream_t s = (cudaStream_t)stream;
  const int64_t need = lq_gated_linear_bwd_workspace_bytes(M, N, K);
  const Buf bufs[] = {{"dh", d_dh, M * N * 2, false},     {"g", d_g, M * N * 2, false},
                      {"u", d_u, M * N * 2, false},       {"x", d_x, M * K * 2, false},
                      {"Wg", d_wg, N * K * 2, false},     {"Wu", d_wu, N * K * 2, false},
                      {"dx", d_dx, M * K * 2, true},      {"dwg", d_dwg, N * K * gsz, true},
                      {"dwu", d_dwu, N * K * gsz, true},  {"dbg", d_dbg, N * gsz, true},
                      {"dbu", d_dbu, N * gsz, true},      {"the workspace", d_ws, ws_bytes < need ? 0 : need, true}};
  if ((st = check_bufs(bufs)) != LQ_OK) return st;
  if (M == 0) {
    if (accumulate) return LQ_OK;
    if ((st = clear(d_dwg, N * K * gsz, s)) != LQ_OK) return st;
    if ((st = clear(d_dwu, N * K * gsz, s)) != LQ_OK) return st;
    if ((st = clear(d_dbg, N * gsz, s)) != LQ_OK) return st;
    return clear(d_dbu, N * gsz, s);
  }
  const bool dw = d_dwg || d_dwu;
  if (!d_dx && !dw && !d_dbg && !d_dbu) return LQ_OK;
  if (!d_dh || !d_g || !d_u || (d_dx && (!d_wg || !d_wu)) || (dw && !d_x))
    return null_pointer("dh, g, u, x, Wg or Wu");
  if ((st = check_ws(d_ws, ws_bytes, need)) != LQ_OK) return st;
  DenseBackward d{};
  d.dy = d_dh;
  d.z = d_g;
  d.u = d_u;
  d.x = d_x;
  d.w = d_wg;
  d.w2 = d_wu;
  d.gated = true;
  d.dx = d_dx;
  d.dw = d_dwg;
  d.dw2 = d_dwu;
  d.db = d_dbg;
  d.db2 = d_dbu;
  d.ws = d_ws;
  d.M = M;
  d.N = N;
  d.K = K;
  d.dtype = dtype;
  d.act = act;
  d.f32 = g_dtype == LQ_F32;
  d.accumulate = accumulate != 0;
  return launched(launch_dense_backward(d, s), "gated linear backward launch");
}

lq_status lq_distill_loss(const void* d_logits, int32_t dtype, int64_t M, int64_t V,
                          const void* d_t_values, int32_t t_dtype, const void* d_t_index,
                          int32_t idx_bytes, int64_t k, const float* d_t_lse,
                          const float* d_weight, float temp, float* d_loss, void* d_grad,
                          void* stream) {
  if ((dtype != LQ_F32 && dtype != LQ_BF16 && dtype != LQ_F16) ||
      (t_dtype != LQ_F32 && t_dtype != LQ_BF16 && t_dtype != LQ_F16)) {
    set_error("logits are float32, bf16 or f16 (dtype %d, t_dtype %d)", dtype, t_dtype);
    return LQ_ERR_UNSUPPORTED;
  }
  if (idx_bytes != 4 && idx_bytes != 8) {
    set_error("indices are int32 or int64 (idx_bytes %d)", idx_bytes);
    return LQ_ERR_UNSUPPORTED;
  }
  if (M < 0 || V <= 0 || k <= 0) {
    set_error("invalid shape M=%lld V=%lld k=%lld", (long long)M, (long long)V, (long long)k);
    return LQ_ERR_ARG;
  }
  // exponents are differences of logits times log2(e) / temp
  if (!(temp > 0.f) || !std::isfinite(temp) || !std::isfinite(1.4426950408889634f / temp)) {
    set_error("the temperature must be positive and finite, log2(e) over it too");
    return LQ_ERR_ARG;
  }
  const int64_t esz = dtype == LQ_F32 ? 4 : 2, tsz = t_dtype == LQ_F32 ? 4 : 2;
  if (k > V || k > LQ_DISTILL_MAX_K || V > LQ_DISTILL_MAX_V) {
    set_error("V=%lld, k=%lld: k must not exceed V nor %d, and V not %d", (long long)V,
              (long long)k, LQ_DISTILL_MAX_K, LQ_DISTILL_MAX_V);
    return LQ_ERR_SHAPE;
  }
  if (M > kMaxExtent / 8 || M * V > kMaxElems) {
    set_error("too many rows");
    return LQ_ERR_SHAPE;
  }
  if (M == 0) return LQ_OK;
  if (!d_logits || !d_t_values || !d_t_index || !d_loss)
    return null_pointer("logits, teacher list or loss");
  const Buf bufs[] = {{"the logits", d_grad == d_logits ? nullptr : d_logits, M * V * esz, false},
                      {"the teacher's values", d_t_values, M * k * tsz, false},
                      {"the teacher's indices", d_t_index, M * k * idx_bytes, false},
                      {"the teacher's log-partition", d_t_lse, M * 4, false},
                      {"the weights", d_weight, M * 4, false},
                      {"the loss", d_loss, M * 4, true},
                      {"the gradient", d_grad, M * V * esz, true}};
  lq_status st = check_bufs(bufs);
  if (st != LQ_OK) return st;
  if (!aligned16(d_logits)) {
    set_error("the logits must be 16-byte aligned");
    return LQ_ERR_ALIGN;
  }
  DistillArgs a{};
  a.z = d_logits;
  a.t = d_t_values;
  a.idx = d_t_index;
  a.t_lse = d_t_lse;
  a.weight = d_weight;
  a.loss = d_loss;
  a.grad = d_grad;
  a.M = M;
  a.V = V;
  a.k = (int)k;
  a.dtype = dtype;
  a.t_dtype = t_dtype;
  a.idx64 = idx_bytes == 8;
  a.temp = temp;
  return launched(launch_distill(a, (cudaStream_t)stream), "distillation loss launch");
}

}  // extern "C"
