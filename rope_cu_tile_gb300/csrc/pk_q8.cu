// pk_q8.cu -- the projection of 8-bit rows (pk_linear_q8 in include/pk.h):
//
//     y = r + act(s_t v_n sum_k q[t, k] p[n, k] + b)       q [T, K] e4m3 with a scale s_t a row, p [N, K] e4m3 with a scale v_n
//
// The product runs on the tensor cores at twice the 16-bit rate, with half the operands' bytes: to the kernel of pk_gemm.cuh a
// pair of 8-bit elements is one 16-bit element of k, and only the instruction differs (kBytes). Every product of two e4m3
// numbers is exact in fp32 and the scales stand outside the sum, so they are part of the epilogue: the sum times s_t, then times v_n,
// wherever it is done (s_t v_n by itself may be past either end of fp32's range where these two are not).
#include "pk_few.cuh"

namespace pk {

namespace {

using namespace rows;

struct Q8Params {
  const float* xs;   // [M]
  const float* ws;   // [N]
  const void* bias;  // [N] in the output's type, or null
  const void* res;   // [M, N], or null
  void* y;
  int64_t ldres, ldy;
  int act;
  int ws_vec, bias_vec, res_vec, y_vec;
};
struct Q8Tiles : Q8Params {
  CUtensorMap map_y;
  int tma_y;
};

// 16384 x 1024 -> 4096, bf16 results: 50 us (the tensor cores' floor 35: at this K the operands and the 134 MB of results share
// the way through L2), 68 with bias and gelu, 89 with a residual besides. Stored from registers, 16 or 32 bytes a lane, it took
// 62 to 80 us; in tiles of 64 columns on eight warps 50 and 76 with gelu.
template <int DT>
struct Q8Epi {
  using Params = Q8Tiles;
  using S = Stage<DT>;
  static constexpr bool kBytes = true;
  static constexpr int kWarps = DT == PK_F32 ? 8 : 16;  // (as LinEpi)

  template <class Ready, class Done>
  static __device__ __forceinline__ bool run(const Params& p, uint32_t tacc, bool zero, int r0, int c0, int cols, int M, int N, int,
                                             int lane, uint8_t* stage, const Ready& ready, const Done& done) {
    if (r0 >= M || c0 >= N) {
      if (!ready()) return false;
      done();
      return true;
    }
    const int end = min(cols, N - c0);
    const float xs = r0 + lane < M ? __ldcg(p.xs + r0 + lane) : 0.0f;
#pragma unroll 1
    for (int cc = 0; cc < end; cc += 32) {
      const int c = c0 + cc;
      if (p.res) {
        stored(lane);  // the previous chunk's tile has left the staging memory
        S::fetch(stage, lane, p.res, p.ldres, p.res_vec, r0, c, M, N);
      }
      float v[32];
      {
        Bias<PK_F32, 32> ws;
        Bias<DT, 32> b;
        ws.fetch(p.ws, p.ws_vec, c, N);
        if (p.bias) b.fetch(p.bias, p.bias_vec, c, N);
        if (cc == 0 && !ready()) return false;
        read_acc(tacc + cc, zero, v);
        if (cc + 32 >= end) done();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t u[4] = {ws.q[i].x, ws.q[i].y, ws.q[i].z, ws.q[i].w};
#pragma unroll
          for (int j = 0; j < 4; j += 2) {
            const float2 f = mul2(mul2(make_float2(v[4 * i + j], v[4 * i + j + 1]), make_float2(xs, xs)),
                                  make_float2(__uint_as_float(u[j]), __uint_as_float(u[j + 1])));
            v[4 * i + j] = f.x;
            v[4 * i + j + 1] = f.y;
          }
        }
        if (p.bias) b.add(v);
      }
      act_values<DT>(p.act, v);
      if (p.res) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        S::add(stage, lane, v, 0);
      } else {
        stored(lane);  // (as late as can be: all of the above runs under the copy)
      }
      S::put(stage, lane, v);
      if (p.tma_y) {
        store_tile(&p.map_y, stage, c, r0, 0, lane);
      } else {
        __syncwarp();
        S::flush(stage, lane, p.y, p.ldy, p.y_vec, nullptr, r0, c, M, N);
        __syncwarp();
      }
    }
    return true;
  }
};

// the partial sums of the splits of k, unscaled
struct Q8Part : LinEpi<PK_F32, PK_F32> {
  static constexpr bool kBytes = true;
};

template <int DT>
__global__ void __launch_bounds__(256) pk_q8_splits_kernel(const float* part, int64_t ldp, int64_t stride, int splits, int64_t M, int N,
                                                           FastDiv groups, const __grid_constant__ Q8Params p) {
  griddep_wait();
  const int64_t n = M * static_cast<int64_t>(groups.d);
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = n < (int64_t(1) << 31) ? groups.div(static_cast<uint32_t>(i)) : i / groups.d;
    const int c = static_cast<int>(i - r * groups.d) * 8, left = N - c;
    float v[8], b[8];
    load8<PK_F32>(part, r * ldp + c, v);
#pragma unroll 4
    for (int s = 1; s < splits; ++s) {
      load8<PK_F32>(part, s * stride + r * ldp + c, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    const float xs = __ldcg(p.xs + r);
    load8_any<PK_F32>(p.ws, c, left, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * xs * b[j];
    if (p.bias) {
      load8_any<DT>(p.bias, c, left, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    act_values<DT>(p.act, v);
    if (p.res) {
      if (p.res_vec && left >= 8)
        load8<DT>(p.res, r * p.ldres + c, b);
      else
        load8_any<DT>(p.res, r * p.ldres + c, left, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    if (p.y_vec && left >= 8)
      store8<DT>(p.y, r * p.ldy + c, v);
    else
      store8_any<DT>(p.y, r * p.ldy + c, left, v);
  }
}

// ------------------------------------------------------------------------------------
// a few rows (serving): as pk_linear_few_kernel, 16 elements a lane and step. e4m3 numbers are exact in fp16, and a product of
// two of those is added to an fp32 sum by one instruction.

constexpr int kFewT = PK_LINEAR_FEW_T / 2;
constexpr int kFewRows = 4;   // of the weights, a warp
constexpr int kFewSteps = 2;  // of 512 elements, asked for together

struct FewArgs {
  const uint8_t* x;
  const uint8_t* w;
  int64_t ldx;
  int T, N, K;
  int share;
  Q8Params ep;
};

__device__ __forceinline__ void to_halves(const uint4& q, uint32_t (&h)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
        : "r"(w[i]));
}

template <int DT, int TM>
__global__ void __launch_bounds__(kFewThreads) pk_q8_few_kernel(const __grid_constant__ FewArgs a) {
  __shared__ float part[8][kFewRows * TM];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int group = w / a.share, sub = w % a.share, groups = 8 / a.share;
  const int n0 = (blockIdx.x * groups + group) * kFewRows;
  float acc[kFewRows][TM];
#pragma unroll
  for (int r = 0; r < kFewRows; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[r][t] = 0.0f;
  griddep_wait();
  if (n0 < a.N) {
    const int step = a.share * 512;
#pragma unroll 1
    for (int k0 = sub * 512 + lane * 16; k0 < a.K; k0 += kFewSteps * step) {
      uint4 q[kFewSteps][kFewRows];
#pragma unroll
      for (int s = 0; s < kFewSteps; ++s)
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
          const int k = k0 + s * step;
          if (k < a.K)
            q[s][r] = __ldcg(reinterpret_cast<const uint4*>(a.w + static_cast<int64_t>(min(n0 + r, a.N - 1)) * a.K + k));
        }
#pragma unroll
      for (int s = 0; s < kFewSteps; ++s) {
        const int k = k0 + s * step;
        if (k >= a.K) break;
        uint32_t x[TM][8];
#pragma unroll
        for (int t = 0; t < TM; ++t) to_halves(*reinterpret_cast<const uint4*>(a.x + min(t, a.T - 1) * a.ldx + k), x[t]);
#pragma unroll
        for (int r = 0; r < kFewRows; ++r) {
          uint32_t h[8];
          to_halves(q[s][r], h);
#pragma unroll
          for (int t = 0; t < TM; ++t)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[r][t] = Elem<false>::fma_hi(h[j], x[t][j], Elem<false>::fma_lo(h[j], x[t][j], acc[r][t]));
        }
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kFewRows; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
      if (lane == 0) part[w][r * TM + t] = acc[r][t];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < groups * kFewRows * TM; i += kFewThreads) {
    const int g = i / (kFewRows * TM), e = i % (kFewRows * TM), t = e % TM, n = (blockIdx.x * groups + g) * kFewRows + e / TM;
    if (t >= a.T || n >= a.N) continue;
    float v[2] = {0.0f, 0.0f};
    for (int s = 0; s < a.share; ++s) v[0] += part[g * a.share + s][e];
    v[0] = v[0] * a.ep.xs[t] * a.ep.ws[n];
    if (a.ep.bias) v[0] += Ty<DT>::get(a.ep.bias, n);
    act_values<DT>(a.ep.act, v);
    if (a.ep.res) v[0] += Ty<DT>::get(a.ep.res, t * a.ep.ldres + n);
    Ty<DT>::put(a.ep.y, t * a.ep.ldy + n, v[0]);
  }
}

template <int DT, int TM>
cudaError_t few_launch_rows(FewArgs a, int sms, cudaStream_t stream) {
  a.share = few_share(a.N / kFewRows, a.K / 2, sms);
  const int per_block = 8 / a.share * kFewRows;
  Launch l((a.N + per_block - 1) / per_block, kFewThreads, stream);
  return cudaLaunchKernelEx(&l.cfg, pk_q8_few_kernel<DT, TM>, a);
}
template <int DT>
cudaError_t few_launch(const FewArgs& a, int sms, cudaStream_t stream) {
  if (a.T == 1) return few_launch_rows<DT, 1>(a, sms, stream);
  if (a.T == 2) return few_launch_rows<DT, 2>(a, sms, stream);
  return few_launch_rows<DT, 4>(a, sms, stream);
}

// ------------------------------------------------------------------------------------

struct Plan {
  gemm::Shape shape;
  float* partial;
  int64_t bytes;
};
Plan plan(int64_t T, int N, int K, int sms, void* ws) {
  Plan p = {};
  if (T <= kFewT) return p;
  Carver c(ws);
  p.shape = gemm::pick_shape(T, N, K / 2, 1, sms, true);
  p.partial = static_cast<float*>(c.take(partial_bytes(p.shape, T, N)));
  p.bytes = c.used;
  return p;
}

template <int DT>
cudaError_t product_of(const gemm::Operand& A, const gemm::Operand& B, gemm::Args a, const Q8Params& ep, const Plan& p, int sms,
                       cudaStream_t stream) {
  const int64_t T = a.M;
  // what the sum of many terms loses on the tensor pipe (pk_gemm.cuh) counts where the result is not rounded to 16 bits
  if (DT == PK_F32) a.phase = gemm::kPhase32;
  if (p.shape.splits > 1) {
    LinTiles part = {};
    part.y = p.partial;
    part.ldy = round_up(a.N, 8);
    part.tma_y = 1;
    a.part_rows = static_cast<int>(partial_rows(p.shape, T));
    if (!gemm::make_out_map(&part.map_y, PK_F32, p.partial, a.part_rows, a.N, part.ldy, 1, 0)) return cudaErrorInvalidValue;
    const cudaError_t r = gemm::launch<Q8Part>(A, B, nullptr, a, part, p.shape, sms, stream);
    if (r != cudaSuccess) return r;
    const FastDiv groups(static_cast<uint32_t>(part.ldy / 8));
    const int64_t n = T * groups.d, most = static_cast<int64_t>(sms) * 8;
    Launch l(n / 256 + 1 < most ? n / 256 + 1 : most, 256, stream);
    const float* cp = p.partial;
    return cudaLaunchKernelEx(&l.cfg, pk_q8_splits_kernel<DT>, cp, part.ldy, round_up(T, 256) * part.ldy, p.shape.splits, T, a.N, groups, ep);
  }
  Q8Tiles t = {};
  static_cast<Q8Params&>(t) = ep;
  // (a TMA store clips a row's end to whole 16 bytes only)
  t.tma_y = ep.y_vec && (static_cast<int64_t>(a.N) * Ty<DT>::kBytes & 15) == 0;
  if (t.tma_y && !gemm::make_out_map(&t.map_y, DT, ep.y, T, a.N, ep.ldy, 1, 0)) return cudaErrorInvalidValue;
  return gemm::launch<Q8Epi<DT>>(A, B, nullptr, a, t, p.shape, sms, stream);
}

bool sizes_ok(int64_t T, int N, int K) {
  return T >= 0 && T <= PK_ROWS_MAX_T && N >= 1 && N <= PK_ROWS_MAX_DIM && K >= 16 && K <= PK_ROWS_MAX_DIM && (K & 15) == 0;
}

}  // namespace

namespace rows {
cudaError_t prepare_q8() {
  cudaError_t e;
  if ((e = gemm::prepare<Q8Part>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<Q8Epi<PK_F32>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<Q8Epi<PK_BF16>>()) != cudaSuccess) return e;
  return gemm::prepare<Q8Epi<PK_F16>>();
}
}  // namespace rows

}  // namespace pk

extern "C" {

int pk_linear_q8_workspace(int64_t T, int N, int K, int64_t* bytes) {
  using namespace pk;
  if (!bytes || !sizes_ok(T, N, K)) return PK_ERR_ARG;
  *bytes = 0;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  *bytes = plan(T, N, K, d.sms, nullptr).bytes;
  return PK_OK;
}

int pk_linear_q8(int dtype, const void* x, int64_t ldx, const float* x_scale, const void* w, const float* w_scale, const void* bias,
                 const void* residual, int64_t ldr, int act, int64_t T, int N, int K, void* y, int64_t ldy, void* workspace,
                 int64_t workspace_bytes, int* status, struct CUstream_st* stream) {
  using namespace pk;
  if (!rows::dtype_ok(dtype) || !sizes_ok(T, N, K) || act < PK_ACT_NONE || act > PK_ACT_SILU || ldx < K || (ldx & 15) != 0 || ldy < N ||
      (residual && ldr < N) || workspace_bytes < 0)
    return PK_ERR_ARG;
  if (T > 0 && (!x || !x_scale || !w || !w_scale || !y)) return PK_ERR_ARG;
  const int e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, 16) || !rows::aligned_to(w, 16) || !rows::aligned_to(x_scale, 4) || !rows::aligned_to(w_scale, 4) ||
      !rows::aligned_to(bias, e) || !rows::aligned_to(residual, e) || !rows::aligned_to(y, e) || !rows::aligned_to(workspace, 256) ||
      !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) return status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess ? PK_ERR_CUDA : PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Plan p = plan(T, N, K, d.sms, workspace);
  if (p.bytes > 0 && (!workspace || workspace_bytes < p.bytes)) return PK_ERR_NOMEM;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  Q8Params ep = {};
  ep.xs = x_scale;
  ep.ws = w_scale;
  ep.bias = bias;
  ep.res = residual;
  ep.y = y;
  ep.ldres = ldr;
  ep.ldy = ldy;
  ep.act = act;
  ep.ws_vec = rows::aligned_to(w_scale, 16);
  ep.bias_vec = bias && rows::aligned_to(bias, 16);
  ep.res_vec = residual && rows16(residual, ldr, e);
  ep.y_vec = rows16(y, ldy, e);
  cudaError_t r;
  if (T <= kFewT) {
    const FewArgs fa = {static_cast<const uint8_t*>(x), static_cast<const uint8_t*>(w), ldx, static_cast<int>(T), N, K, 1, ep};
    r = dtype == PK_F32    ? few_launch<PK_F32>(fa, d.sms, stream)
        : dtype == PK_BF16 ? few_launch<PK_BF16>(fa, d.sms, stream)
                           : few_launch<PK_F16>(fa, d.sms, stream);
    return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
  }
  gemm::Args a = {};
  a.M = static_cast<int>(T);
  a.N = N;
  a.K = K / 2;
  a.status = status ? status : rows::stream_status(d, stream);
  a.timeout_ns = wait_limit_ns();
  const gemm::Operand A = rows::operand(PK_F16, x, ldx / 2, T, K / 2, 0), B = rows::operand(PK_F16, w, K / 2, N, K / 2, 0);
  r = dtype == PK_F32    ? product_of<PK_F32>(A, B, a, ep, p, d.sms, stream)
      : dtype == PK_BF16 ? product_of<PK_BF16>(A, B, a, ep, p, d.sms, stream)
                         : product_of<PK_F16>(A, B, a, ep, p, d.sms, stream);
  return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // extern "C"
