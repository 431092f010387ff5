// pk_xent.cu -- softmax cross entropy of token rows over a vocabulary, without keeping the logits (pk_cross_entropy,
// pk_cross_entropy_backward in include/pk.h).
//
//     z = x W^T + b  [T, V],   lse_t = ln sum_v exp z_tv,   loss_t = lse_t - z_t,label(t)
//     dz = g_t (exp(z - lse_t) - [v = label(t)]),   dx = dz W,   dW = dz^T x,   db = sum over rows of dz
//
// Rows without a label cost nothing: the labelled ones (one in seven in masked-token training) are listed on the device,
// their x gathered, and every product runs over that count, which only the device knows.
//
// Forward: the logits live in tensor memory only. Each warp of the product's epilogue reduces its 32 rows x 128 (64)
// columns to a running maximum and a sum of exponentials, joined over the vocabulary by a second small kernel.
// Backward: the vocabulary in pieces. Of each piece the logits are computed again, turned into dz (16-bit, or three bf16
// planes for fp32) in the epilogue and written to scratch, which two products then read: dW of the piece is complete, dx
// grows piece by piece in an fp32 buffer. Six operations a (row, word, feature), none of them avoidable without the logits.
// dz is rounded to the element type once, as an operand of products of that type: bf16's dx and dw are then 2.4e-3 of their
// norm off, 1.7e-3 of it their own rounding; two planes of dz would undo that at twice the time of those products.
#include "pk_vocab.cuh"

namespace pk {

namespace {

template <int DT>
using LabelStat = StatEpi<DT, false>;
template <int DT>
using LabelGrad = GradEpi<DT, false>;

// Joins the slices of each row, in a fixed order: 8 rows x 32 strided lanes of slices a block.
__global__ void __launch_bounds__(256) pk_xent_join_kernel(const float2* part, int64_t cap, int slices, const float* picked,
                                                           const int* idx, const int* count, float* loss, float* lse) {
  __shared__ float2 s[32][8];
  const int r = threadIdx.x & 7, g = threadIdx.x >> 3;
  griddep_wait();
  const int n = __ldcg(count);
  const auto join = [](float& m, float& l, float2 q) {
    const float mn = fmaxf(m, q.x);
    l = l * exp2f((m - mn) * kLog2e) + q.y * exp2f((q.x - mn) * kLog2e);
    m = mn;
  };
  for (int64_t r0 = blockIdx.x * 8LL; r0 < n; r0 += gridDim.x * 8LL) {
    const int64_t row = r0 + r;
    float m = kFloor, l = 0.0f;
    if (row < n) {
#pragma unroll 4
      for (int i = g; i < slices; i += 32) join(m, l, __ldcg(part + i * cap + row));
    }
    s[g][r] = make_float2(m, l);
    __syncthreads();
    if (g == 0 && row < n) {
      for (int i = 1; i < 32; ++i) join(m, l, s[i][r]);
      const float rest = logf(l);
      const int t = __ldcg(idx + row);
      lse[t] = m + rest;
      loss[t] = (m - __ldcg(picked + row)) + rest;  // not lse - z: large logits would leave the loss their rounding
    }
    __syncthreads();
  }
}

struct Fwd {
  Common m;
  gemm::Shape shape;
  float2* part;
  float* picked;
  int slices;
  int64_t bytes;
};
Fwd plan_forward(int dtype, const void* x, int64_t ldx, const void* w, int64_t T, int D, int V, int sms, void* ws) {
  Fwd f = {};
  Carver c(ws);
  plan_common(c, f.m, dtype, x, ldx, w, T, D, V);
  f.shape = gemm::pick_shape(T, V, D, dtype == PK_F32 ? gemm::kTerms32 : 1, sms, false);
  f.slices = (V + 64 * f.shape.cg - 1) / (64 * f.shape.cg);
  f.part = static_cast<float2*>(c.take(f.slices * f.m.cap * 8));
  f.picked = static_cast<float*>(c.take(f.m.cap * 4));
  f.bytes = c.used;
  return f;
}

}  // namespace

namespace rows {
cudaError_t prepare_xent() {
  cudaError_t e;
  if ((e = gemm::prepare<LabelStat<PK_F32>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<LabelStat<PK_BF16>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<LabelStat<PK_F16>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<LabelGrad<PK_F32>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<LabelGrad<PK_BF16>>()) != cudaSuccess) return e;
  return gemm::prepare<LabelGrad<PK_F16>>();
}
}  // namespace rows

}  // namespace pk

extern "C" {

int pk_cross_entropy_workspace(int dtype, const void* x, int64_t ldx, const void* w, int backward, int need_db, int64_t T,
                               int D, int V, int64_t* bytes) {
  using namespace pk;
  if (!bytes || !rows::dtype_ok(dtype) || !sizes_ok(T, D, V) || ldx < D) return PK_ERR_ARG;
  *bytes = 0;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  *bytes = backward ? plan_backward(dtype, x, ldx, w, need_db != 0, T, D, V, d.sms, nullptr).bytes
                    : plan_forward(dtype, x, ldx, w, T, D, V, d.sms, nullptr).bytes;
  return PK_OK;
}

int pk_cross_entropy(int dtype, const void* x, int64_t ldx, const void* w, const void* bias, const int64_t* labels, int64_t T,
                     int D, int V, float* loss, float* lse, void* workspace, int64_t workspace_bytes, int* status,
                     struct CUstream_st* stream) {
  using namespace pk;
  if (!rows::dtype_ok(dtype) || !sizes_ok(T, D, V) || ldx < D || workspace_bytes < 0) return PK_ERR_ARG;
  if (T > 0 && (!x || !w || !labels || !loss || !lse)) return PK_ERR_ARG;
  const uintptr_t e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, e) || !rows::aligned_to(w, e) || !rows::aligned_to(bias, e) || !rows::aligned_to(labels, 8) ||
      !rows::aligned_to(loss, 4) || !rows::aligned_to(lse, 4) || !rows::aligned_to(workspace, 256) || !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) return status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess ? PK_ERR_CUDA : PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Fwd f = plan_forward(dtype, x, ldx, w, T, D, V, d.sms, workspace);
  if (!workspace || workspace_bytes < f.bytes) return PK_ERR_NOMEM;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  RowArgs r = {};
  r.labels = reinterpret_cast<const long long*>(labels);
  r.T = T;
  r.V = V;
  r.counts = f.m.counts;
  r.maxima = f.m.maxima;
  r.idx = f.m.idx;
  r.lab = f.m.lab;
  r.count = f.m.count;
  r.loss = loss;
  r.lse = lse;
  r.status = status ? status : rows::stream_status(d, stream);
  if (rows_launch(r, stream) != cudaSuccess) return PK_ERR_CUDA;
  Inputs in;
  if (lay_out(dtype, f.m, x, ldx, w, T, D, V, d.sms, stream, &in) != cudaSuccess) return PK_ERR_CUDA;
  gemm::Args a = {};
  a.M = static_cast<int>(T);
  a.N = V;
  a.K = D;
  a.dyn = f.m.count;
  a.dyn_axis = 0;
  a.alt_count = static_cast<int>(T);
  a.alt_operand = 0;
  a.status = r.status;
  a.timeout_ns = wait_limit_ns();
  StatParams sp = {};
  sp.bias = bias;
  sp.bias_vec = bias && rows::aligned_to(bias, 16);
  sp.lab = f.m.lab;
  sp.part = f.part;
  sp.picked = f.picked;
  sp.cap = f.m.cap;
  if (logits_product<LabelStat>(dtype, in.xc, in.w, in.alt ? &in.xd : nullptr, a, sp, f.shape, d.sms, stream) != cudaSuccess)
    return PK_ERR_CUDA;
  const int64_t blocks = (T + 7) / 8, most = static_cast<int64_t>(d.sms) * 8;
  rows::Launch l(blocks < most ? blocks : most, 256, stream);
  const float2* part = f.part;
  const float* picked = f.picked;
  const int *idx = f.m.idx, *count = f.m.count;
  return cudaLaunchKernelEx(&l.cfg, pk_xent_join_kernel, part, f.m.cap, f.slices, picked, idx, count, loss, lse) == cudaSuccess
             ? PK_OK
             : PK_ERR_CUDA;
}

int pk_cross_entropy_backward(int dtype, const void* x, int64_t ldx, const void* w, const void* bias, const int64_t* labels,
                              const float* lse, const float* dloss, int64_t T, int D, int V, void* dx, void* dw, void* db,
                              void* workspace, int64_t workspace_bytes, int* status, struct CUstream_st* stream) {
  using namespace pk;
  if (!rows::dtype_ok(dtype) || !sizes_ok(T, D, V) || ldx < D || workspace_bytes < 0) return PK_ERR_ARG;
  if (T > 0 && (!x || !w || !labels || !lse || !dloss)) return PK_ERR_ARG;
  const uintptr_t e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, e) || !rows::aligned_to(w, e) || !rows::aligned_to(bias, e) || !rows::aligned_to(labels, 8) ||
      !rows::aligned_to(lse, 4) || !rows::aligned_to(dloss, 4) || !rows::aligned_to(dx, e) || !rows::aligned_to(dw, e) ||
      !rows::aligned_to(db, e) || !rows::aligned_to(workspace, 256) || !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) {
    if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
    if (dw && cudaMemsetAsync(dw, 0, e * V * static_cast<size_t>(D), stream) != cudaSuccess) return PK_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, e * V, stream) != cudaSuccess) return PK_ERR_CUDA;
    return PK_OK;
  }
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Bwd b = plan_backward(dtype, x, ldx, w, db != nullptr, T, D, V, d.sms, workspace);
  if (!workspace || workspace_bytes < b.bytes) return PK_ERR_NOMEM;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  RowArgs r = {};
  r.labels = reinterpret_cast<const long long*>(labels);
  r.T = T;
  r.V = V;
  r.counts = b.m.counts;
  r.maxima = b.m.maxima;
  r.idx = b.m.idx;
  r.lab = b.m.lab;
  r.count = b.m.count;
  r.dloss = dloss;
  r.lse_in = lse;
  r.coef = b.coef;
  r.lse_rows = b.lse;
  r.unscale = b.unscale;
  r.factor = 1.0f;
  r.scaled = dtype == PK_F16;
  r.status = status ? status : rows::stream_status(d, stream);
  if (rows_launch(r, stream) != cudaSuccess) return PK_ERR_CUDA;
  Inputs in;
  if (lay_out(dtype, b.m, x, ldx, w, T, D, V, d.sms, stream, &in) != cudaSuccess) return PK_ERR_CUDA;
  GradParams gp = {};
  gp.lab = b.m.lab;
  return backward_pieces<LabelGrad>(dtype, b, in, gp, bias, T, D, V, dx, dw, db, r.status, d.sms, stream);
}

}  // extern "C"
