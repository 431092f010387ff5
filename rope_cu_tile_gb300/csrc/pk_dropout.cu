// pk_dropout.cu -- dropout of token rows from a counter-based generator, with the residual stream (pk_dropout in
// include/pk.h):  y = r + x keep / (1 - p),  keep drawn from (seed, offset, row, column) by pk_philox.cuh. The mask is
// never stored: the backward pass draws it again from the same arguments.
//
// Bound by bytes (x and r read, y written). A thread draws once for 8 columns, 20 wide multiplications for 8 elements, and
// asks for several such groups before it uses the first.
#include "pk_rows.cuh"

namespace pk {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // groups of 8 elements a thread has in flight (one, where that leaves SMs without a block)

struct DropoutArgs {
  const void* x;
  const void* res;
  void* y;
  int64_t ldx, ldr, ldy;
  uint32_t row0;  // of this launch
  uint32_t total; // groups of this launch, below 2^31
  int N;
  rows::FastDiv groups;
  DropArgs drop;
  int vec, res_vec;
};

template <int DT, int kB>
__global__ void __launch_bounds__(kThreads) pk_dropout_kernel(const __grid_constant__ DropoutArgs a) {
  griddep_wait();
  const uint32_t i0 = blockIdx.x * (kThreads * kB) + threadIdx.x;
  Raw8<DT> x[kB], res[kB];
  uint32_t r[kB], g[kB];
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const uint32_t i = i0 + b * kThreads;
    if (i >= a.total) break;
    r[b] = a.groups.div(i);
    g[b] = i - r[b] * a.groups.d;
    r[b] += a.row0;
    const int c = 8 * static_cast<int>(g[b]);
    x[b].load(a.x, r[b] * a.ldx + c, a.vec, a.N - c);
    if (a.res) res[b].load(a.res, r[b] * a.ldr + c, a.res_vec, a.N - c);
  }
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    if (i0 + b * kThreads >= a.total) break;
    const int c = 8 * static_cast<int>(g[b]), n = a.N - c;
    float v[8];
    x[b].get(v);
    if (a.drop.cut) drop8(v, r[b], g[b], a.drop);
    if (a.res) {
      float q[8];
      res[b].get(q);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += q[j];
    }
    if (a.vec && n >= 8)
      store8<DT>(a.y, r[b] * a.ldy + c, v);
    else
      store8_any<DT>(a.y, r[b] * a.ldy + c, n, v);
  }
}

template <int DT>
cudaError_t dropout_launch(const DropoutArgs& a, int sms, cudaStream_t stream) {
  const int batch = a.total >= static_cast<uint32_t>(2 * sms * kThreads * kBatch) ? kBatch : 1;
  rows::Launch l((a.total + kThreads * batch - 1) / (kThreads * batch), kThreads, stream);
  return batch == 1 ? cudaLaunchKernelEx(&l.cfg, pk_dropout_kernel<DT, 1>, a)
                    : cudaLaunchKernelEx(&l.cfg, pk_dropout_kernel<DT, kBatch>, a);
}

}  // namespace

}  // namespace pk

extern "C" int pk_dropout(int dtype, const void* x, int64_t ldx, const void* residual, int64_t ldr, double p, uint64_t seed,
                          uint64_t offset, int64_t T, int N, void* y, int64_t ldy, struct CUstream_st* stream) {
  using namespace pk;
  DropoutArgs a = {};
  if (!rows::dtype_ok(dtype) || T < 0 || T > PK_ROWS_MAX_T || N < 1 || N > PK_ROWS_MAX_DIM || !drop_args(p, seed, offset, &a.drop))
    return PK_ERR_ARG;
  if (ldx < N || ldy < N || (residual && ldr < N) || (T > 0 && (!x || !y))) return PK_ERR_ARG;
  const int e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, e) || !rows::aligned_to(y, e) || !rows::aligned_to(residual, e)) return PK_ERR_ALIGN;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  a.x = x;
  a.res = residual;
  a.y = y;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.N = N;
  a.vec = rows16(x, ldx, e) && rows16(y, ldy, e);
  a.res_vec = residual && rows16(residual, ldr, e);
  const int64_t groups = (N + 7) / 8, most = (int64_t(1) << 30) / groups;  // rows of one launch
  a.groups = rows::FastDiv(static_cast<uint32_t>(groups));
  for (int64_t r0 = 0; r0 < T; r0 += most) {
    a.row0 = static_cast<uint32_t>(r0);
    a.total = static_cast<uint32_t>((T - r0 < most ? T - r0 : most) * groups);
    const cudaError_t r = dtype == PK_F32    ? dropout_launch<PK_F32>(a, d.sms, stream)
                          : dtype == PK_BF16 ? dropout_launch<PK_BF16>(a, d.sms, stream)
                                             : dropout_launch<PK_F16>(a, d.sms, stream);
    if (r != cudaSuccess) return PK_ERR_CUDA;
  }
  return PK_OK;
}
