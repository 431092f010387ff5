// pk_dropout.cu -- dropout of token rows from a counter-based generator, with the residual stream (pk_dropout in
// include/pk.h):  y = r + x keep / (1 - p),  keep drawn from (seed, offset, row, column) by pk_philox.cuh. The mask is
// never stored: the backward pass draws it again from the same arguments.
//
// Bound by bytes (x and r read, y written); a thread draws once for the 8 columns it holds, 20 wide multiplications for
// 8 elements.
#include "pk_rows.cuh"

namespace pk {

namespace {

struct DropoutArgs {
  const void* x;
  const void* res;
  void* y;
  int64_t ldx, ldr, ldy, T;
  int N;
  DropArgs drop;
  int vec, res_vec;
};

template <int DT>
__global__ void __launch_bounds__(256) pk_dropout_kernel(const __grid_constant__ DropoutArgs a) {
  griddep_wait();
  const int64_t groups = (a.N + 7) / 8, total = a.T * groups;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = i / groups;
    const int g = static_cast<int>(i - r * groups), c = 8 * g, n = a.N - c;
    float v[8], b[8];
    const bool vec = a.vec && n >= 8;
    if (vec)
      load8<DT>(a.x, r * a.ldx + c, v);
    else
      load8_any<DT>(a.x, r * a.ldx + c, n, v);
    if (a.res) {
      if (a.res_vec && n >= 8)
        load8<DT>(a.res, r * a.ldr + c, b);
      else
        load8_any<DT>(a.res, r * a.ldr + c, n, b);
    }
    if (a.drop.cut) drop8(v, static_cast<uint32_t>(r), static_cast<uint32_t>(g), a.drop);
    if (a.res) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    if (vec)
      store8<DT>(a.y, r * a.ldy + c, v);
    else
      store8_any<DT>(a.y, r * a.ldy + c, n, v);
  }
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
  a.T = T;
  a.N = N;
  a.vec = rows16(x, ldx, e) && rows16(y, ldy, e);
  a.res_vec = residual && rows16(residual, ldr, e);
  const int64_t total = T * ((N + 7) / 8), most = static_cast<int64_t>(d.sms) * 8;
  rows::Launch l((total + 255) / 256 < most ? (total + 255) / 256 : most, 256, stream);
  cudaError_t r;
  if (dtype == PK_F32)
    r = cudaLaunchKernelEx(&l.cfg, pk_dropout_kernel<PK_F32>, a);
  else if (dtype == PK_BF16)
    r = cudaLaunchKernelEx(&l.cfg, pk_dropout_kernel<PK_BF16>, a);
  else
    r = cudaLaunchKernelEx(&l.cfg, pk_dropout_kernel<PK_F16>, a);
  return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}
