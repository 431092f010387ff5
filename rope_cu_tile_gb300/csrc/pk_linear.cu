// pk_linear.cu -- the projection of token rows and its gradients (pk_linear, pk_linear_backward in include/pk.h).
//
//     z = x W^T + b,   y = r + drop(act(z))          x [T, K], W [N, K], b [N], r and y [T, N]
//     dz = act'(z) drop(dy),  dx = dz W,  dW = dz^T x,  db = sum over rows of dz,  dr = dy
//
// The products run on the tensor cores (pk_gemm.cuh); the forward's bias, activation, dropout and residual are its
// epilogue, so z and the mask are never stored unless the caller asks for z. The backward makes dz once (pk_dz_kernel: it
// is an operand of both products, so it has to exist in memory in the operand's type) and sums its columns on the way.
#include <cstring>

#include "pk_rows.cuh"

namespace pk {

namespace {

using namespace rows;

// ------------------------------------------------------------------------------------
// dz and its column sums

constexpr int kDzThreads = 256;
constexpr int kDzBlocks = 4;  // resident blocks of an SM
constexpr int kDzLeast = 16;  // rows of a block
// Rows of a block: one wave of resident blocks, all of the same length (fixed blocks of 128 rows left part of the SMs
// idle at the end). Measured: 65536 x 2048 bf16, gelu and dropout, 159 us (0.75 of the copy rate; issue slots 63 % full).
int dz_rows(int64_t T, int64_t ldz, int sms) {
  const int64_t blocks = kDzBlocks * sms / ((ldz + 255) / 256);
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

// A warp takes 256 columns of a row (8 a lane: one draw of the generator); a block eight rows at a time.
// Moves dy, z and dz; bound by issue slots with dropout and gelu (64 % of them, 0.75 of the copy rate).
// dz is rounded to the element type once: it is an operand of tensor-core products of that type, as x and W are. bf16
// results are then off by 2.3e-3 of their norm (1.7e-3 of it their own rounding); two planes of dz would undo that at twice
// the products' time.
// fp16: a dz of ordinary size is stored as it is. How large the largest is, is known after this kernel only: a second launch
// (kScale) stores dz again, times a power of two, where that has to be, and else ends at once (some 2 us); the products' results are
// multiplied by the inverse. (A pass over dy before this one would cost its reading every time.)
template <int DT, bool kScale>
__global__ void __launch_bounds__(kDzThreads, kDzBlocks) pk_dz_kernel(const __grid_constant__ DzArgs a) {
  __shared__ float sums[8][256];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int c = blockIdx.y * 256 + lane * 8;
  const int n = a.N - c;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  griddep_wait();
  float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float top = 0.0f, scale = 1.0f;
  if constexpr (kScale) {
    const int blocks = gridDim.x * gridDim.y;
    for (int i = threadIdx.x; i < blocks; i += kDzThreads) top = fmaxf(top, __ldcg(a.tops + i));
    top = block_top(top, &sums[0][0]);
    const int e = dz_exponent(top);
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) *a.unscale = scalbnf(1.0f, -e);
    if (e == 0) return;
    scale = scalbnf(1.0f, e);
  }
  if (c < a.ldz) {
    // the next row's values are asked for before this one's are used (two rows ahead, or batches of rows, take longer: the
    // body is copied for each and no longer fits the instruction cache)
    const int64_t end = min(r0 + a.rows, a.T);
    Raw8<DT> dy, pre;
    const auto load = [&](int64_t r) {
      if (r >= end) return;
      dy.load(a.dy, r * a.lddy + c, a.dy_vec, n);
      if (a.act != PK_ACT_NONE) pre.load(a.pre, r * a.ldpre + c, a.pre_vec, n);
    };
    load(r0 + w);
#pragma unroll 1
    for (int64_t r = r0 + w; r < end; r += 8) {
      float z[8], v[8];
      dy.get(v);
      if (a.act != PK_ACT_NONE) pre.get(z);
      load(r + 8);
      if (a.drop.cut) drop8(v, static_cast<uint32_t>(r), c / 8, a.drop);
      if (a.act != PK_ACT_NONE) act_slopes<DT>(a.act, z, v);
      if (n < 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j >= n) v[j] = 0.0f;  // the operand's padding
      }
      if constexpr (kScale) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= scale;
      } else {
#pragma unroll
        for (int j = 0; j < 8; j += 2) add2(sum[j], sum[j + 1], make_float2(v[j], v[j + 1]));
        if constexpr (DT == PK_F16) {
          // (an infinite or undefined element is none that a scale could hold)
          if (a.tops) {
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fabsf(v[j]) <= 3.4e38f ? fmaxf(top, fabsf(v[j])) : top;
          }
        }
        if (!a.dz) continue;
      }
      if constexpr (DT == PK_F32) {
        uint32_t h[3][4];
        planes8(v, h);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          *reinterpret_cast<uint4*>(a.dz + k * a.plane + r * a.ldz + c) = make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
      } else {
        store8<DT>(a.dz, r * a.ldz + c, v);
      }
    }
  }
  if constexpr (kScale) return;
  if constexpr (DT == PK_F16) {
    if (a.tops) {
      top = block_top(top, &sums[0][0]);
      if (threadIdx.x == 0) a.tops[blockIdx.y * gridDim.x + blockIdx.x] = top;
      __syncthreads();
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) sums[w][lane * 8 + j] = sum[j];
  __syncthreads();
  const int col = blockIdx.y * 256 + threadIdx.x;
  if (col < a.ldz) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += sums[i][threadIdx.x];
    a.part[static_cast<int64_t>(blockIdx.x) * a.ldz + col] = v;
  }
}

cudaError_t dz_launch(int dtype, DzArgs a, cudaStream_t stream) {
  a.dy_vec = rows16(a.dy, a.lddy, elem_bytes(dtype));
  a.pre_vec = a.pre && rows16(a.pre, a.ldpre, elem_bytes(dtype));
  Launch l(1, kDzThreads, stream);
  l.cfg.gridDim = dim3(static_cast<unsigned int>((a.T + a.rows - 1) / a.rows), static_cast<unsigned int>((a.ldz + 255) / 256));
  if (dtype == PK_F32) return cudaLaunchKernelEx(&l.cfg, pk_dz_kernel<PK_F32, false>, a);
  if (dtype == PK_BF16) return cudaLaunchKernelEx(&l.cfg, pk_dz_kernel<PK_BF16, false>, a);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, pk_dz_kernel<PK_F16, false>, a);
  return e != cudaSuccess || !a.tops ? e : cudaLaunchKernelEx(&l.cfg, pk_dz_kernel<PK_F16, true>, a);
}

// ------------------------------------------------------------------------------------
// a few rows (serving)

// Bound by W's bytes, read once; x stays in L1. A warp dots kR rows of W with every row of x, 8 elements a lane and step, in
// fp32 on the CUDA cores (fp32 inputs need no planes); where N alone gives too few warps, several share the rows and split
// k, so that most of W is on its way at once. One launch, no scratch. Past a few rows its arithmetic and the reads of x
// outweigh the tensor cores' fixed costs: W [4096, 1024] in bf16 took 3.5 us at 1 row, 6.5 at 4, 11.9 at 8, and 7.3 there;
// fp32 10.5 at 8 rows here and some 19 there, with its plane copies.
constexpr int kFewThreads = 256;
bool few_rows(int dtype, int64_t T) { return T <= (dtype == PK_F32 ? PK_LINEAR_FEW_T : PK_LINEAR_FEW_T / 2); }

struct FewArgs {
  const void* x;
  const void* w;
  int64_t ldx;
  int T, N, K;
  int share;  // warps that split k: 1, 2, 4 or 8
  int vec;    // rows of x and W on 16-byte boundaries
  LinParams ep;
};

// rows of W a warp, and steps of k asked for together: as many 16-byte loads in flight as the registers of 16 warps an SM hold
__host__ __device__ constexpr int few_r(int dt, int tm) { return dt == PK_F32 && tm < 8 ? 2 : 4; }
__host__ __device__ constexpr int few_steps(int dt) { return dt == PK_F32 ? 1 : 2; }

template <int DT, int TM>
__global__ void __launch_bounds__(kFewThreads) pk_linear_few_kernel(const __grid_constant__ FewArgs a) {
  constexpr int kR = few_r(DT, TM), kFewSteps = few_steps(DT);
  __shared__ float part[8][kR * TM];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int group = w / a.share, sub = w % a.share, groups = 8 / a.share;
  const int n0 = (blockIdx.x * groups + group) * kR;
  float acc[kR][TM];
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[r][t] = 0.0f;
  griddep_wait();
  if (n0 < a.N) {
    const int step = a.share * 256;
#pragma unroll 1
    for (int k0 = sub * 256 + lane * 8; k0 < a.K; k0 += kFewSteps * step) {
      Raw8<DT> q[kFewSteps][kR];
#pragma unroll
      for (int s = 0; s < kFewSteps; ++s)
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const int k = k0 + s * step;
          if (k < a.K) q[s][r].load(a.w, static_cast<int64_t>(min(n0 + r, a.N - 1)) * a.K + k, a.vec, a.K - k);
        }
#pragma unroll
      for (int s = 0; s < kFewSteps; ++s) {
        const int k = k0 + s * step;
        if (k >= a.K) break;
        float v[kR][8];
#pragma unroll
        for (int r = 0; r < kR; ++r) q[s][r].get(v[r]);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          float x[8];
          const int64_t at = min(t, a.T - 1) * a.ldx + k;
          if (a.vec && k + 8 <= a.K)
            load8<DT, true>(a.x, at, x);
          else
            load8_any<DT>(a.x, at, a.K - k, x);
#pragma unroll
          for (int r = 0; r < kR; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[r][t] = fmaf(v[r][j], x[j], acc[r][t]);
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
      if (lane == 0) part[w][r * TM + t] = acc[r][t];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < groups * kR * TM; i += kFewThreads) {
    const int g = i / (kR * TM), e = i % (kR * TM), t = e % TM, n = (blockIdx.x * groups + g) * kR + e / TM;
    if (t >= a.T || n >= a.N) continue;
    float v = 0.0f;
    for (int s = 0; s < a.share; ++s) v += part[g * a.share + s][e];
    finish1<DT>(a.ep, v, t, n);
  }
}

template <int DT, int TM>
cudaError_t few_launch_rows(FewArgs a, int sms, cudaStream_t stream) {
  constexpr int kR = few_r(DT, TM);
  a.share = 1;
  while (a.share < 8 && static_cast<int64_t>(a.N) / kR * a.share < 16 * sms && a.K > 256 * a.share) a.share *= 2;
  const int per_block = 8 / a.share * kR;
  Launch l((a.N + per_block - 1) / per_block, kFewThreads, stream);
  return cudaLaunchKernelEx(&l.cfg, pk_linear_few_kernel<DT, TM>, a);
}
template <int DT>
cudaError_t few_launch(const FewArgs& a, int sms, cudaStream_t stream) {
  if (a.T == 1) return few_launch_rows<DT, 1>(a, sms, stream);
  if (a.T == 2) return few_launch_rows<DT, 2>(a, sms, stream);
  if constexpr (DT == PK_F32)
    if (a.T > 4) return few_launch_rows<DT, 8>(a, sms, stream);
  return few_launch_rows<DT, 4>(a, sms, stream);
}

// ------------------------------------------------------------------------------------
// plans: the scratch of a call, laid out the same way when its size is asked for and when it is used

struct Fwd {
  gemm::Shape shape;
  void *x, *w;
  float* partial;
  int64_t bytes;
};
Fwd plan_forward(int dtype, const void* x, int64_t ldx, const void* w, int64_t T, int N, int K, int sms, void* ws) {
  Fwd f = {};
  Carver c(ws);
  if (few_rows(dtype, T)) return f;
  f.x = in_place(dtype, x, ldx) ? nullptr : c.take(copy_bytes(dtype, T, K));
  f.w = in_place(dtype, w, K) ? nullptr : c.take(copy_bytes(dtype, N, K));
  f.shape = gemm::pick_shape(T, N, K, dtype == PK_F32 ? gemm::kTerms32 : 1, sms, true);
  f.partial = static_cast<float*>(c.take(partial_bytes(f.shape, T, N)));
  f.bytes = c.used;
  return f;
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
Bwd plan_backward(int dtype, const void* x, int64_t ldx, const void* w, const void* dy, int64_t lddy, int act,
                  uint32_t cut, bool need_dx, bool need_dw, bool need_db, int64_t T, int N, int K, int sms, void* ws) {
  Bwd b = {};
  Carver c(ws);
  const int terms = dtype == PK_F32 ? gemm::kTerms32 : 1;
  if (need_dw && !in_place(dtype, x, ldx)) b.x = c.take(copy_bytes(dtype, T, K));
  if (need_dx && !in_place(dtype, w, K)) b.w = c.take(copy_bytes(dtype, N, K));
  // dy itself is the operand when nothing changes it on the way
  const bool made = (need_dx || need_dw) && (act != PK_ACT_NONE || cut || !in_place(dtype, dy, lddy));
  if (made) b.dz = c.take(copy_bytes(dtype, T, N));
  b.rows = dz_rows(T, copy_ld(N), sms);
  b.blocks = (T + b.rows - 1) / b.rows;
  // (without dropout dz of relu, or of no activation, is made of dy's elements and zeros: exact)
  b.scaled = made && dtype == PK_F16 && (cut || act == PK_ACT_GELU || act == PK_ACT_SILU);
  if (b.scaled) {
    b.tops = static_cast<float*>(c.take(b.blocks * ((copy_ld(N) + 255) / 256) * 4));
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

bool sizes_ok(int64_t T, int N, int K) {
  return T >= 0 && T <= PK_ROWS_MAX_T && N >= 1 && N <= PK_ROWS_MAX_DIM && K >= 1 && K <= PK_ROWS_MAX_DIM;
}
bool act_ok(int act) { return act >= PK_ACT_NONE && act <= PK_ACT_SILU; }

}  // namespace

}  // namespace pk

extern "C" {

int pk_linear_workspace(int dtype, const void* x, int64_t ldx, const void* w, int64_t T, int N, int K, int64_t* bytes) {
  using namespace pk;
  if (!bytes || !rows::dtype_ok(dtype) || !sizes_ok(T, N, K) || ldx < K) return PK_ERR_ARG;
  *bytes = 0;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  *bytes = plan_forward(dtype, x, ldx, w, T, N, K, d.sms, nullptr).bytes;
  return PK_OK;
}

int pk_linear(int dtype, const void* x, int64_t ldx, const void* w, const void* bias, const void* residual, int64_t ldr,
              int act, double p, uint64_t seed, uint64_t offset, int64_t T, int N, int K, void* y, int64_t ldy, void* pre,
              void* workspace, int64_t workspace_bytes, int* status, struct CUstream_st* stream) {
  using namespace pk;
  LinParams ep = {};
  if (!rows::dtype_ok(dtype) || !sizes_ok(T, N, K) || !act_ok(act) || !drop_args(p, seed, offset, &ep.drop)) return PK_ERR_ARG;
  if (ldx < K || ldy < N || (residual && ldr < N) || workspace_bytes < 0) return PK_ERR_ARG;
  if (T > 0 && (!x || !w || !y)) return PK_ERR_ARG;
  const uintptr_t e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, e) || !rows::aligned_to(w, e) || !rows::aligned_to(bias, e) || !rows::aligned_to(residual, e) ||
      !rows::aligned_to(y, e) || !rows::aligned_to(pre, e) || !rows::aligned_to(workspace, 256) || !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) return status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess ? PK_ERR_CUDA : PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Fwd f = plan_forward(dtype, x, ldx, w, T, N, K, d.sms, workspace);
  if (f.bytes > 0 && (!workspace || workspace_bytes < f.bytes)) return PK_ERR_NOMEM;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  ep.bias = bias;
  ep.res = residual;
  ep.ldres = ldr;
  ep.y = y;
  ep.ldy = ldy;
  ep.pre = pre;
  ep.ldpre = N;
  ep.act = act;
  if (few_rows(dtype, T)) {
    const FewArgs fa = {x, w, ldx, static_cast<int>(T), N, K, 1, rows16(x, ldx, e) && rows16(w, K, e), ep};
    const cudaError_t r = dtype == PK_F32    ? few_launch<PK_F32>(fa, d.sms, stream)
                          : dtype == PK_BF16 ? few_launch<PK_BF16>(fa, d.sms, stream)
                                             : few_launch<PK_F16>(fa, d.sms, stream);
    return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
  }
  rows::Copies copies(dtype);
  if (f.x) copies.add(x, ldx, T, K, f.x);
  if (f.w) copies.add(w, K, N, K, f.w);
  if (copies.launch(d.sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  gemm::Args a = {};
  a.M = static_cast<int>(T);
  a.N = N;
  a.K = K;
  a.status = status ? status : rows::stream_status(d, stream);
  a.timeout_ns = wait_limit_ns();
  const gemm::Operand A = f.x ? rows::operand_of_copy(dtype, f.x, T, K, 0) : rows::operand(dtype, x, ldx, T, K, 0);
  const gemm::Operand B = f.w ? rows::operand_of_copy(dtype, f.w, N, K, 0) : rows::operand(dtype, w, K, N, K, 0);
  return rows::product(dtype, dtype, A, B, nullptr, a, ep, f.shape, f.partial, rows::partial_rows(f.shape, T), d.sms, stream) == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

int pk_linear_backward_workspace(int dtype, const void* x, int64_t ldx, const void* w, const void* dy, int64_t lddy, int act,
                                 double p, int need_dx, int need_dw, int need_db, int64_t T, int N, int K, int64_t* bytes) {
  using namespace pk;
  DropArgs drop;
  if (!bytes || !rows::dtype_ok(dtype) || !sizes_ok(T, N, K) || !act_ok(act) || !drop_args(p, 0, 0, &drop) || ldx < K ||
      lddy < N)
    return PK_ERR_ARG;
  *bytes = 0;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  *bytes = plan_backward(dtype, x, ldx, w, dy, lddy, act, drop.cut, need_dx != 0, need_dw != 0, need_db != 0, T, N, K, d.sms,
                         nullptr)
               .bytes;
  return PK_OK;
}

int pk_linear_backward(int dtype, const void* x, int64_t ldx, const void* w, const void* dy, int64_t lddy, const void* pre,
                       int act, double p, uint64_t seed, uint64_t offset, int64_t T, int N, int K, void* dx, void* dw,
                       void* db, void* workspace, int64_t workspace_bytes, int* status, struct CUstream_st* stream) {
  using namespace pk;
  DzArgs z = {};
  if (!rows::dtype_ok(dtype) || !sizes_ok(T, N, K) || !act_ok(act) || !drop_args(p, seed, offset, &z.drop)) return PK_ERR_ARG;
  if (ldx < K || lddy < N || workspace_bytes < 0) return PK_ERR_ARG;
  if (T > 0 && (!dy || (dw && !x) || (dx && !w) || (act != PK_ACT_NONE && !pre))) return PK_ERR_ARG;
  const uintptr_t e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, e) || !rows::aligned_to(w, e) || !rows::aligned_to(dy, e) || !rows::aligned_to(pre, e) ||
      !rows::aligned_to(dx, e) || !rows::aligned_to(dw, e) || !rows::aligned_to(db, e) || !rows::aligned_to(workspace, 256) ||
      !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) {
    // no rows: the gradients of the weights are zero
    if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
    if (dw && cudaMemsetAsync(dw, 0, e * N * static_cast<size_t>(K), stream) != cudaSuccess) return PK_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, e * N, stream) != cudaSuccess) return PK_ERR_CUDA;
    return PK_OK;
  }
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Bwd b = plan_backward(dtype, x, ldx, w, dy, lddy, act, z.drop.cut, dx != nullptr, dw != nullptr, db != nullptr, T, N,
                              K, d.sms, workspace);
  if (b.bytes > 0 && (!workspace || workspace_bytes < b.bytes)) return PK_ERR_NOMEM;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  if (b.dz || b.part) {
    z.dy = dy;
    z.lddy = lddy;
    z.pre = pre;
    z.ldpre = N;
    z.T = T;
    z.N = N;
    z.act = act;
    z.dz = static_cast<uint16_t*>(b.dz);
    z.ldz = rows::copy_ld(N);
    z.plane = T * z.ldz;
    z.part = b.part;
    z.rows = b.rows;
    z.tops = b.tops;
    z.unscale = b.unscale;
    if (dz_launch(dtype, z, stream) != cudaSuccess) return PK_ERR_CUDA;
    if (db && rows::sum_rows(dtype, b.part, b.blocks, nullptr, 1, N, z.ldz, nullptr, db, stream) != cudaSuccess) return PK_ERR_CUDA;
  }
  rows::Copies copies(dtype);
  if (b.w) copies.add(w, K, N, K, b.w);
  if (b.x) copies.add(x, ldx, T, K, b.x);
  if (copies.launch(d.sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  gemm::Args a = {};
  a.status = status ? status : rows::stream_status(d, stream);
  a.timeout_ns = wait_limit_ns();
  if (dx) {
    const gemm::Operand A = b.dz ? rows::operand_of_copy(dtype, b.dz, T, N, 0) : rows::operand(dtype, dy, lddy, T, N, 0);
    const gemm::Operand B = b.w ? rows::operand_of_copy(dtype, b.w, N, K, 1) : rows::operand(dtype, w, K, N, K, 1);
    a.M = static_cast<int>(T);
    a.N = K;
    a.K = N;
    LinParams ep = {};
    ep.y = dx;
    ep.ldy = K;
    ep.alpha = b.scaled ? b.unscale : nullptr;
    if (rows::product(dtype, dtype, A, B, nullptr, a, ep, b.dx, b.partial, rows::partial_rows(b.dx, T), d.sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  }
  if (dw) {
    const gemm::Operand A = b.dz ? rows::operand_of_copy(dtype, b.dz, T, N, 1) : rows::operand(dtype, dy, lddy, T, N, 1);
    const gemm::Operand B = b.x ? rows::operand_of_copy(dtype, b.x, T, K, 1) : rows::operand(dtype, x, ldx, T, K, 1);
    a.M = N;
    a.N = K;
    a.K = static_cast<int>(T);
    LinParams ep = {};
    ep.y = dw;
    ep.ldy = K;
    ep.alpha = b.scaled ? b.unscale : nullptr;
    if (rows::product(dtype, dtype, A, B, nullptr, a, ep, b.dw, b.partial, rows::partial_rows(b.dw, N), d.sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  }
  return PK_OK;
}

}  // extern "C"
