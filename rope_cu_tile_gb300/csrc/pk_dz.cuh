// pk_dz.cuh -- the backward pass of a projection from its dz on, shared by pk_linear.cu and pk_gated.cu: dz as an operand
// (one copy in the element type, its column sums, fp16's scale), the scratch of a call, and the two products
//     dx = dz W,  dW = dz^T x.
#pragma once

#include "pk_rows.cuh"

namespace pk {
namespace rows {

constexpr int kDzThreads = 256;
constexpr int kDzLeast = 16;  // rows of a block
// Rows of a block: one wave of resident blocks, all of the same length (fixed blocks of 128 rows left part of the SMs
// idle at the end). Measured: 65536 x 2048 bf16, gelu and dropout, 159 us (0.75 of the copy rate; issue slots 63 % full).
inline int dz_rows(int64_t T, int64_t ldz, int sms, int resident) {
  const int64_t blocks = resident * sms / ((ldz + 255) / 256);
  const int64_t rows = blocks > 1 ? round_up((T + blocks - 1) / blocks, 8) : T;
  return static_cast<int>(rows < kDzLeast ? kDzLeast : rows);
}

struct DzArgs {
  const void* dy;
  const void* pre;
  int64_t lddy, ldpre;
  int64_t T;
  int N;
  int act;
  DropArgs drop;
  uint16_t* dz;  // [T, ldz] operand (three planes for fp32), or null
  int64_t ldz, plane;
  float* part;  // [blocks of rows, ldz] column sums, or null
  int dy_vec, pre_vec;
  int rows;    // of a block
  float* tops;     // [blocks] fp16: each block's largest finite |dz|, or null
  float* unscale;  // the inverse of dz's scale
};

// The power of two that fp16's dz is multiplied by: 1 while the largest |dz| is within [2^-10, 65504], where it overflows
// nothing and every element within 2^-4 of it keeps its 11 bits (half a step of the smallest numbers, 2^-25, is 2^-15 of it at
// most); past either end the one that brings it to [2^14, 2^15).
__device__ __forceinline__ int dz_exponent(float top) {
  if (!(top > 0.0f) || (top >= 0.0009765625f && top <= 65504.0f)) return 0;
  return max(-100, min(100, 14 - ilogbf(top)));
}

// The largest of a block's values, in every thread; `shared` holds a value a warp.
__device__ __forceinline__ float block_top(float v, float* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = shared[0];
#pragma unroll
  for (int i = 1; i < kDzThreads / 32; ++i) v = fmaxf(v, shared[i]);
  return v;
}

struct Bwd {
  gemm::Shape dx, dw;
  void *x, *w, *dz;
  float *part, *partial;
  float *tops, *unscale;  // of a dz that may need a scale
  bool scaled;
  int rows;  // of a block of dz
  int64_t blocks, bytes;
};
// `made`: dz is not dy itself; `scaled`: fp16's dz may need a scale; `wide`: columns that the kernel which makes dz walks (dz
// itself has N), with `resident` blocks an SM.
inline Bwd plan_products(int dtype, const void* x, int64_t ldx, const void* w, bool made, bool scaled, int wide, int resident,
                         bool need_dx, bool need_dw, bool need_db, int64_t T, int N, int K, int sms, void* ws) {
  Bwd b = {};
  Carver c(ws);
  const int terms = dtype == PK_F32 ? gemm::kTerms32 : 1;
  if (need_dw && !in_place(dtype, x, ldx)) b.x = c.take(copy_bytes(dtype, T, K));
  if (need_dx && !in_place(dtype, w, K)) b.w = c.take(copy_bytes(dtype, N, K));
  if (made) b.dz = c.take(copy_bytes(dtype, T, N));
  b.rows = dz_rows(T, copy_ld(wide), sms, resident);
  b.blocks = (T + b.rows - 1) / b.rows;
  b.scaled = scaled;
  if (b.scaled) {
    b.tops = static_cast<float*>(c.take(b.blocks * ((copy_ld(wide) + 255) / 256) * 4));
    b.unscale = static_cast<float*>(c.take(4));
  }
  if (need_db) b.part = static_cast<float*>(c.take(b.blocks * copy_ld(N) * 4));
  int64_t partial = 0;
  if (need_dx) {
    b.dx = gemm::pick_shape(T, K, N, terms, sms, true);
    partial = partial_bytes(b.dx, T, K);
  }
  if (need_dw) {
    b.dw = gemm::pick_shape(N, K, T, terms, sms, true);
    const int64_t m = partial_bytes(b.dw, N, K);
    partial = m > partial ? m : partial;
  }
  b.partial = static_cast<float*>(c.take(partial));
  b.bytes = c.used;
  return b;
}

// The two products, from the dz of the plan (or dy itself). `status`: the call's word.
inline int back_products(int dtype, const Bwd& b, const void* x, int64_t ldx, const void* w, const void* dy, int64_t lddy,
                         int64_t T, int N, int K, void* dx, void* dw, int* status, int sms, cudaStream_t stream) {
  Copies copies(dtype);
  if (b.w) copies.add(w, K, N, K, b.w);
  if (b.x) copies.add(x, ldx, T, K, b.x);
  if (copies.launch(sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  gemm::Args a = {};
  a.status = status;
  a.timeout_ns = wait_limit_ns();
  if (dx) {
    const gemm::Operand A = b.dz ? operand_of_copy(dtype, b.dz, T, N, 0) : operand(dtype, dy, lddy, T, N, 0);
    const gemm::Operand B = b.w ? operand_of_copy(dtype, b.w, N, K, 1) : operand(dtype, w, K, N, K, 1);
    a.M = static_cast<int>(T);
    a.N = K;
    a.K = N;
    LinParams ep = {};
    ep.y = dx;
    ep.ldy = K;
    ep.alpha = b.scaled ? b.unscale : nullptr;
    if (product(dtype, dtype, A, B, nullptr, a, ep, b.dx, b.partial, partial_rows(b.dx, T), sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  }
  if (dw) {
    const gemm::Operand A = b.dz ? operand_of_copy(dtype, b.dz, T, N, 1) : operand(dtype, dy, lddy, T, N, 1);
    const gemm::Operand B = b.x ? operand_of_copy(dtype, b.x, T, K, 1) : operand(dtype, x, ldx, T, K, 1);
    a.M = N;
    a.N = K;
    a.K = static_cast<int>(T);
    LinParams ep = {};
    ep.y = dw;
    ep.ldy = K;
    ep.alpha = b.scaled ? b.unscale : nullptr;
    if (product(dtype, dtype, A, B, nullptr, a, ep, b.dw, b.partial, partial_rows(b.dw, N), sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  }
  return PK_OK;
}

}  // namespace rows
}  // namespace pk
