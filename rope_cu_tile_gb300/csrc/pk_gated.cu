// pk_gated.cu -- the gated feed-forward of token rows and its gradients (pk_gated_linear, pk_gated_linear_backward in
// include/pk.h).
//
//     [g | u] = x W^T + b,   y = act(g) u                     x [T, K], W [2F, K] (the gate's rows, then the other's), y [T, F]
//     dg = dy u act'(g),  du = dy act(g),   dz = [dg | du]:   dx = dz W,  dW = dz^T x,  db = sum over rows of dz
//
// Forward: one product whose tiles hold the same columns of both halves (pk_gemm.cuh, kPair), so that the activation and
// the product of the two are its epilogue and neither half goes through memory unless the caller keeps them for the
// backward. Backward: dz is made once and is an operand of both products, as in pk_linear.cu, rounded to the element type as such
// operands are: dx and dw of fp16 are then 2.9e-4 of their norm off, 2.1e-4 of it their own rounding; db sums it unrounded.
#include "pk_dz.cuh"
#include "pk_few.cuh"

namespace pk {

namespace {

using namespace rows;

struct GluParams {
  const void* bias;  // [2 F], or null
  void* y;           // [M, F]
  void* pre;         // [M, 2 F], or null
  int64_t ldy;
  int act;
  int bias_vec, bias_up_vec, y_vec, pre_vec;
};
struct GluTiles : GluParams {
  CUtensorMap map_y, map_pre, map_up;
  int tma_y, tma_pre;
};

template <int DT>
__device__ __forceinline__ const void* up_half(const void* p, int F) {
  return static_cast<const char*>(p) + static_cast<int64_t>(F) * Ty<DT>::kBytes;
}

// A chunk of 32 columns: each half with its bias to `pre` where that is kept, then both again, 16 columns at a time, for y.
// One staging tile a warp serves the three; an accumulator read twice costs less than the registers to hold both halves.
// 16384 x 1024 -> 2 x 2624 bf16: 109 us with gelu (a plain product of that size 104; bound by its operands' way through L2 as
// that is), 121 with both halves kept. Of 96 registers a thread 116 bytes are spilled and 340 read back, the pair's tile in 16 bits. fp32
// 584 us (537 by six passes).
template <int DT>
struct GluEpi {
  using Params = GluTiles;
  using S = Stage<DT>;
  static constexpr bool kPair = true;
  static constexpr int kWarps = DT == PK_F32 ? 8 : 16;  // (as LinEpi)

  template <class Ready, class Done>
  static __device__ __forceinline__ bool run(const Params& p, uint32_t gate, uint32_t up, bool zero, int r0, int c0, int cols, int M,
                                             int F, int, int lane, uint8_t* stage, const Ready& ready, const Done& done) {
    if (r0 >= M || c0 >= F) {
      if (!ready()) return false;
      done();
      return true;
    }
    const int end = min(cols, F - c0);
#pragma unroll 1
    for (int cc = 0; cc < end; cc += 32) {
      const int c = c0 + cc;
      if (cc == 0 && !ready()) return false;
      if (p.pre) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float v[32];
          read_acc((h ? up : gate) + cc, zero, v);
          if (p.bias) {
            Bias<DT, 32> b;
            b.fetch(h ? up_half<DT>(p.bias, F) : p.bias, h ? p.bias_up_vec : p.bias_vec, c, F);
            b.add(v);
          }
          stored(lane);
          S::put(stage, lane, v);
          if (p.tma_pre) {
            store_tile(h ? &p.map_up : &p.map_pre, stage, c, r0, 0, lane);
          } else {
            __syncwarp();
            S::flush(stage, lane, const_cast<void*>(h ? up_half<DT>(p.pre, F) : p.pre), 2 * static_cast<int64_t>(F), p.pre_vec, nullptr,
                     r0, c, M, F);
            __syncwarp();
          }
        }
      }
#pragma unroll 1
      for (int q = 0; q < 32; q += 16) {
        float g[16], u[16];
        if (zero) {
#pragma unroll
          for (int i = 0; i < 16; ++i) g[i] = u[i] = 0.0f;
        } else {
          __syncwarp();  // (as in read_acc)
          tmem_ld16(gate + cc + q, g);
          tmem_ld16(up + cc + q, u);
        }
        if (q == 16 && cc + 32 >= end) done();
        if (p.bias) {
          Bias<DT, 16> b;
          b.fetch(p.bias, p.bias_vec, c + q, F);
          b.add(g);
          b.fetch(up_half<DT>(p.bias, F), p.bias_up_vec, c + q, F);
          b.add(u);
        }
        act_values<DT>(p.act, g);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 v = mul2(make_float2(g[i], g[i + 1]), make_float2(u[i], u[i + 1]));
          g[i] = v.x;
          g[i + 1] = v.y;
        }
        if (q == 0) stored(lane);
        S::put(stage, lane, g, q / S::kPer);
      }
      if (p.tma_y) {
        store_tile(&p.map_y, stage, c, r0, 0, lane);
      } else {
        __syncwarp();
        S::flush(stage, lane, p.y, p.ldy, p.y_vec, nullptr, r0, c, M, F);
        __syncwarp();
      }
    }
    return true;
  }
};

// Eight columns of one row from their sums (splits of k).
template <int DT>
__device__ __forceinline__ void glu8(const GluParams& p, float (&g)[8], float (&u)[8], int64_t row, int c, int F) {
  const int n = F - c;
  if (p.bias) {
    float b[8];
    load8_any<DT>(p.bias, c, n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] += b[i];
    load8_any<DT>(p.bias, F + c, n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] += b[i];
  }
  if (p.pre) {
    const int64_t at = row * 2 * F + c;
    if (p.pre_vec && n >= 8) {
      store8<DT>(p.pre, at, g);
      store8<DT>(p.pre, at + F, u);
    } else {
      store8_any<DT>(p.pre, at, n, g);
      store8_any<DT>(p.pre, at + F, n, u);
    }
  }
  act_values<DT>(p.act, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] *= u[i];
  if (p.y_vec && n >= 8)
    store8<DT>(p.y, row * p.ldy + c, g);
  else
    store8_any<DT>(p.y, row * p.ldy + c, n, g);
}

// y from the partial sums of the splits of k, added in order.
template <int DT>
__global__ void __launch_bounds__(256) pk_gated_splits_kernel(const float* part, int64_t ldp, int64_t stride, int splits, int64_t M, int F,
                                                              FastDiv groups, const __grid_constant__ GluParams p) {
  griddep_wait();
  const int64_t n = M * static_cast<int64_t>(groups.d);
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = n < (int64_t(1) << 31) ? groups.div(static_cast<uint32_t>(i)) : i / groups.d;
    const int c = static_cast<int>(i - r * groups.d) * 8;
    float g[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, u[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int s = 0; s < splits; ++s) {
      const int64_t at = s * stride + r * ldp + c;
      float a[8], b[8];
      if ((F & 7) == 0) {
        load8<PK_F32>(part, at, a);
        load8<PK_F32>(part, at + F, b);
      } else {
        load8_any<PK_F32>(part, at, F - c, a);
        load8_any<PK_F32>(part, at + F, F - c, b);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        g[j] += a[j];
        u[j] += b[j];
      }
    }
    glu8<DT>(p, g, u, r, c, F);
  }
}

// ------------------------------------------------------------------------------------
// a few rows (serving): as pk_linear_few_kernel, half of a warp's rows of W the gate's and half the other's

struct FewArgs {
  const void* x;
  const void* w;
  int64_t ldx;
  int T, F, K;
  int share, vec;
  GluParams ep;
};

// Bound by the bytes of W from 10 MB on, by its launch below: one row bf16 or f16, 2 x 4096 x 4096 12.2 us (0.82 of the copy rate; 16.4
// while both operands were unpacked first), 2 x 2624 x 1024 3.8. Up to two rows on 64 registers, for four blocks an SM: two rows 15 us, 17
// to 18.6 without. Four rows 23 and 7.4: a step's weights are asked for, waited for and multiplied with every row in turns.
template <int DT, int TM>
__global__ void __launch_bounds__(kFewThreads, TM > 2 ? 1 : 4) pk_gated_few_kernel(const __grid_constant__ FewArgs a) {
  constexpr int kR = few_r(DT, TM), kCols = kR / 2;
  __shared__ float part[8][kR * TM];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int group = w / a.share, sub = w % a.share, groups = 8 / a.share;
  const int n0 = (blockIdx.x * groups + group) * kCols;
  float acc[kR][TM];
  griddep_wait();
  few_dots<DT, 1>(a.x, a.ldx, a.T, a.w, a.K, a.vec, n0 < a.F, sub, a.share, lane,
               [&](int r) { return min(n0 + r % kCols, a.F - 1) + (r < kCols ? 0 : a.F); }, acc);
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][t] += __shfl_xor_sync(0xffffffffu, acc[r][t], o);
      if (lane == 0) part[w][r * TM + t] = acc[r][t];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < groups * kCols * TM; i += kFewThreads) {
    const int g = i / (kCols * TM), e = i % (kCols * TM), t = e % TM, c = (blockIdx.x * groups + g) * kCols + e / TM;
    if (t >= a.T || c >= a.F) continue;
    float v[2] = {0.0f, 0.0f};
    float u = 0.0f;
    for (int s = 0; s < a.share; ++s) {
      v[0] += part[g * a.share + s][e];
      u += part[g * a.share + s][kCols * TM + e];
    }
    if (a.ep.bias) {
      v[0] += Ty<DT>::get(a.ep.bias, c);
      u += Ty<DT>::get(a.ep.bias, a.F + c);
    }
    if (a.ep.pre) {
      const int64_t at = static_cast<int64_t>(t) * 2 * a.F + c;
      Ty<DT>::put(a.ep.pre, at, v[0]);
      Ty<DT>::put(a.ep.pre, at + a.F, u);
    }
    act_values<DT>(a.ep.act, v);
    Ty<DT>::put(a.ep.y, t * a.ep.ldy + c, v[0] * u);
  }
}

bool few_rows(int dtype, int64_t T) { return T <= (dtype == PK_F32 ? PK_LINEAR_FEW_T : PK_LINEAR_FEW_T / 2); }

template <int DT, int TM>
cudaError_t few_launch_rows(FewArgs a, int sms, cudaStream_t stream) {
  constexpr int kCols = few_r(DT, TM) / 2;
  a.share = few_share(a.F / kCols, a.K, sms);
  const int per_block = 8 / a.share * kCols;
  Launch l((a.F + per_block - 1) / per_block, kFewThreads, stream);
  return cudaLaunchKernelEx(&l.cfg, pk_gated_few_kernel<DT, TM>, a);
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
// dz

// As pk_dz_kernel (pk_linear.cu), but for a half warp to 128 columns of a row, a block sixteen rows at a time (dz_rows is asked for
// blocks of 256, so for twice the columns): widths such as 1152 leave fewer lanes without any. dy, g and u are
// read and both halves of dz written, their columns summed on the way. The activation and its slope share their
// exponentials. In fp16 always with the second launch that applies a scale where the largest element asks for one: a
// product of three factors is no element of dy.
// 65536 x 2624 bf16 272 us (0.95 of the copy rate), 16384 x 2624 74 (0.87), 16931 x 1152 f16 38 (0.77; 40 with whole
// warps to 256 columns).
constexpr int dz_resident(int dtype) { return dtype == PK_F32 ? 2 : 3; }  // blocks of an SM

template <int DT, bool kScale>
__global__ void __launch_bounds__(kDzThreads, (DT == PK_F32 ? 2 : 3)) pk_gated_dz_kernel(const __grid_constant__ DzArgs a, int F) {
  __shared__ float sums[2][16][128];
  const int lane = threadIdx.x & 15, w = threadIdx.x >> 4;  // of a half warp
  const int c = blockIdx.y * 128 + lane * 8;
  const int n = F - c;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * a.rows;
  griddep_wait();
  float sg[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, su[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  float top = 0.0f, scale = 1.0f;
  if constexpr (kScale) {
    const int blocks = gridDim.x * gridDim.y;
    for (int i = threadIdx.x; i < blocks; i += kDzThreads) top = fmaxf(top, __ldcg(a.tops + i));
    top = block_top(top, &sums[0][0][0]);
    const int e = dz_exponent(top);
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) *a.unscale = scalbnf(1.0f, -e);
    if (e == 0) return;
    scale = scalbnf(1.0f, e);
  }
  // (dz's rows begin on 16-byte boundaries, and so does every eighth column of the gate's half; the other's where F allows)
  const auto put16 = [&](uint16_t* d, const uint32_t(&q)[4], bool whole) {
    if (whole) {
      *reinterpret_cast<uint4*>(d) = make_uint4(q[0], q[1], q[2], q[3]);
    } else if ((F & 1) == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (2 * j < n) reinterpret_cast<uint32_t*>(d)[j] = q[j];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) d[j] = static_cast<uint16_t>(q[j >> 1] >> (16 * (j & 1)));
    }
  };
  const auto put = [&](int64_t r, int col, float(&v)[8]) {
    const bool whole = n >= 8 && (col == c || (F & 7) == 0);
    uint16_t* d = a.dz + r * a.ldz + col;
    if constexpr (DT == PK_F32) {
      uint32_t h[3][4];
      planes8(v, h);
#pragma unroll
      for (int k = 0; k < 3; ++k) put16(d + k * a.plane, h[k], whole);
    } else {
      using E = Elem<DT == PK_BF16>;
      const uint32_t q[4] = {E::pack(v[0], v[1]), E::pack(v[2], v[3]), E::pack(v[4], v[5]), E::pack(v[6], v[7])};
      put16(d, q, whole);
    }
  };
  if (c < F) {
    const int64_t end = min(r0 + a.rows, a.T);
    Raw8<DT> xd, xg, xu;
    // vec 1: 16 bytes at a time, 2: 16-bit elements in pairs, 0: one by one
    const auto read = [&](Raw8<DT>& x, const void* p, int64_t at, int vec) {
      if constexpr (DT != PK_F32) {
        if (vec == 2) {
          const uint32_t* s = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + at);
          x.q[0] = make_uint4(__ldcg(s), n > 2 ? __ldcg(s + 1) : 0u, n > 4 ? __ldcg(s + 2) : 0u, n > 6 ? __ldcg(s + 3) : 0u);
          return;
        }
      }
      x.load(p, at, vec == 1, n);
    };
    const auto load = [&](int64_t r) {
      if (r >= end) return;
      read(xd, a.dy, r * a.lddy + c, a.dy_vec);
      read(xg, a.pre, r * a.ldpre + c, a.pre_vec);
      read(xu, a.pre, r * a.ldpre + F + c, a.pre_vec);
    };
    load(r0 + w);
#pragma unroll 1
    for (int64_t r = r0 + w; r < end; r += 16) {
      float d[8], g[8], u[8], v[8], s[8];
      xd.get(d);
      xg.get(g);
      xu.get(u);
      load(r + 16);
      act_both<DT>(a.act, g, v, s);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = v[j] * d[j] * scale;         // du
        g[j] = d[j] * scale * u[j] * s[j];  // dg
        if (n < 8 && j >= n) v[j] = g[j] = 0.0f;
      }
      if constexpr (!kScale) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          add2(sg[j], sg[j + 1], make_float2(g[j], g[j + 1]));
          add2(su[j], su[j + 1], make_float2(v[j], v[j + 1]));
        }
        if constexpr (DT == PK_F16) {
          if (a.tops) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              top = fabsf(g[j]) <= 3.4e38f ? fmaxf(top, fabsf(g[j])) : top;
              top = fabsf(v[j]) <= 3.4e38f ? fmaxf(top, fabsf(v[j])) : top;
            }
          }
        }
        if (!a.dz) continue;
      }
      put(r, c, g);
      put(r, F + c, v);
    }
  }
  if constexpr (kScale) return;
  if constexpr (DT == PK_F16) {
    if (a.tops) {
      top = block_top(top, &sums[0][0][0]);
      if (threadIdx.x == 0) a.tops[blockIdx.y * gridDim.x + blockIdx.x] = top;
      __syncthreads();
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sums[0][w][lane * 8 + j] = sg[j];
    sums[1][w][lane * 8 + j] = su[j];
  }
  __syncthreads();
  const int h = threadIdx.x >> 7, col = blockIdx.y * 128 + (threadIdx.x & 127);
  if (col < F) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += sums[h][i][threadIdx.x & 127];
    a.part[static_cast<int64_t>(blockIdx.x) * a.ldz + h * F + col] = v;
  }
}

cudaError_t dz_launch(int dtype, DzArgs a, int F, cudaStream_t stream) {
  const int e = elem_bytes(dtype);
  const bool even = e == 2 && (F & 1) == 0;  // (an even number of columns left wherever a group of eight begins)
  a.dy_vec = rows16(a.dy, a.lddy, e) ? 1 : even && aligned_to(a.dy, 4) && (a.lddy & 1) == 0 ? 2 : 0;
  a.pre_vec = rows16(a.pre, a.ldpre, e) && (F * e & 15) == 0 ? 1 : even && aligned_to(a.pre, 4) ? 2 : 0;
  Launch l(1, kDzThreads, stream);
  l.cfg.gridDim = dim3(static_cast<unsigned int>((a.T + a.rows - 1) / a.rows), static_cast<unsigned int>((F + 127) / 128));
  if (dtype == PK_F32) return cudaLaunchKernelEx(&l.cfg, pk_gated_dz_kernel<PK_F32, false>, a, F);
  if (dtype == PK_BF16) return cudaLaunchKernelEx(&l.cfg, pk_gated_dz_kernel<PK_BF16, false>, a, F);
  const cudaError_t r = cudaLaunchKernelEx(&l.cfg, pk_gated_dz_kernel<PK_F16, false>, a, F);
  return r != cudaSuccess || !a.tops ? r : cudaLaunchKernelEx(&l.cfg, pk_gated_dz_kernel<PK_F16, true>, a, F);
}

// ------------------------------------------------------------------------------------
// plans

struct Fwd {
  gemm::Shape shape;
  void *x, *w;
  float* partial;
  int64_t bytes;
};
Fwd plan_forward(int dtype, const void* x, int64_t ldx, const void* w, int64_t T, int F, int K, int sms, void* ws) {
  Fwd f = {};
  Carver c(ws);
  if (few_rows(dtype, T)) return f;
  f.x = in_place(dtype, x, ldx) ? nullptr : c.take(copy_bytes(dtype, T, K));
  f.w = in_place(dtype, w, K) ? nullptr : c.take(copy_bytes(dtype, 2 * static_cast<int64_t>(F), K));
  f.shape = gemm::pick_shape(T, 2 * static_cast<int64_t>(F), K, dtype == PK_F32 ? gemm::kTerms32 : 1, sms, true);
  f.partial = static_cast<float*>(c.take(partial_bytes(f.shape, T, 2 * static_cast<int64_t>(F))));
  f.bytes = c.used;
  return f;
}

Bwd plan_backward(int dtype, const void* x, int64_t ldx, const void* w, bool need_dx, bool need_dw, bool need_db, int64_t T, int F,
                  int K, int sms, void* ws) {
  const bool made = need_dx || need_dw;
  return plan_products(dtype, x, ldx, w, made, made && dtype == PK_F16, 2 * static_cast<int>(round_up(F, 128)), dz_resident(dtype), need_dx, need_dw, need_db, T, 2 * F, K, sms, ws);
}

template <int DT>
cudaError_t product_of(const gemm::Operand& A, const gemm::Operand& B, gemm::Args a, const GluParams& ep, const Fwd& f, int sms,
                       cudaStream_t stream) {
  const int F = a.N / 2, e = Ty<DT>::kBytes;
  const int64_t T = a.M;
  if (f.shape.splits > 1) {
    // the partial sums of [g | u] as any product's, put together by a second kernel
    const int64_t rows_of = partial_rows(f.shape, T), ldp = round_up(a.N, 8);
    const cudaError_t r = partial_sums(A, B, nullptr, a, f.shape, f.partial, rows_of, sms, stream);
    if (r != cudaSuccess) return r;
    const FastDiv groups(static_cast<uint32_t>((F + 7) / 8));
    const int64_t n = T * groups.d, most = static_cast<int64_t>(sms) * 8;
    Launch l(n / 256 + 1 < most ? n / 256 + 1 : most, 256, stream);
    const float* cp = f.partial;
    return cudaLaunchKernelEx(&l.cfg, pk_gated_splits_kernel<DT>, cp, ldp, round_up(T, 256) * ldp, f.shape.splits, T, F, groups,
                              ep);
  }
  GluTiles t = {};
  static_cast<GluParams&>(t) = ep;
  // (a TMA store clips a row's end to whole 16 bytes only)
  const bool even = (static_cast<int64_t>(F) * e & 15) == 0;
  t.tma_y = ep.y_vec && even;
  t.tma_pre = ep.pre && ep.pre_vec;
  char* up = ep.pre ? static_cast<char*>(ep.pre) + static_cast<int64_t>(F) * e : nullptr;
  if ((t.tma_y && !gemm::make_out_map(&t.map_y, DT, ep.y, T, F, ep.ldy, 1, 0)) ||
      (t.tma_pre && (!gemm::make_out_map(&t.map_pre, DT, ep.pre, T, F, a.N, 1, 0) ||
                     !gemm::make_out_map(&t.map_up, DT, up, T, F, a.N, 1, 0))))
    return cudaErrorInvalidValue;
  return gemm::launch<GluEpi<DT>>(A, B, nullptr, a, t, f.shape, sms, stream);
}

bool sizes_ok(int64_t T, int F, int K) {
  return T >= 0 && T <= PK_ROWS_MAX_T && F >= 1 && F <= PK_ROWS_MAX_DIM / 2 && K >= 1 && K <= PK_ROWS_MAX_DIM;
}
bool act_ok(int act) { return act >= PK_ACT_NONE && act <= PK_ACT_SILU; }

}  // namespace

namespace rows {
cudaError_t prepare_gated() {
  cudaError_t e;
  if ((e = gemm::prepare<GluEpi<PK_F32>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<GluEpi<PK_BF16>>()) != cudaSuccess) return e;
  return gemm::prepare<GluEpi<PK_F16>>();
}
}  // namespace rows

}  // namespace pk

extern "C" {

int pk_gated_linear_workspace(int dtype, const void* x, int64_t ldx, const void* w, int64_t T, int F, int K, int64_t* bytes) {
  using namespace pk;
  if (!bytes || !rows::dtype_ok(dtype) || !sizes_ok(T, F, K) || ldx < K) return PK_ERR_ARG;
  *bytes = 0;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  *bytes = plan_forward(dtype, x, ldx, w, T, F, K, d.sms, nullptr).bytes;
  return PK_OK;
}

int pk_gated_linear(int dtype, const void* x, int64_t ldx, const void* w, const void* bias, int act, int64_t T, int F, int K, void* y,
                    int64_t ldy, void* pre, void* workspace, int64_t workspace_bytes, int* status, struct CUstream_st* stream) {
  using namespace pk;
  if (!rows::dtype_ok(dtype) || !sizes_ok(T, F, K) || !act_ok(act) || ldx < K || ldy < F || workspace_bytes < 0) return PK_ERR_ARG;
  if (T > 0 && (!x || !w || !y)) return PK_ERR_ARG;
  const int e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, e) || !rows::aligned_to(w, e) || !rows::aligned_to(bias, e) || !rows::aligned_to(y, e) ||
      !rows::aligned_to(pre, e) || !rows::aligned_to(workspace, 256) || !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) return status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess ? PK_ERR_CUDA : PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Fwd f = plan_forward(dtype, x, ldx, w, T, F, K, d.sms, workspace);
  if (f.bytes > 0 && (!workspace || workspace_bytes < f.bytes)) return PK_ERR_NOMEM;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  const bool even = (static_cast<int64_t>(F) * e & 15) == 0;
  GluParams ep = {};
  ep.bias = bias;
  ep.y = y;
  ep.pre = pre;
  ep.ldy = ldy;
  ep.act = act;
  ep.bias_vec = bias && rows::aligned_to(bias, 16);
  ep.bias_up_vec = ep.bias_vec && even;
  ep.y_vec = rows16(y, ldy, e);
  ep.pre_vec = pre && rows::aligned_to(pre, 16) && even;
  cudaError_t r;
  if (few_rows(dtype, T)) {
    const FewArgs fa = {x, w, ldx, static_cast<int>(T), F, K, 1, rows16(x, ldx, e) && rows16(w, K, e), ep};
    r = dtype == PK_F32    ? few_launch<PK_F32>(fa, d.sms, stream)
        : dtype == PK_BF16 ? few_launch<PK_BF16>(fa, d.sms, stream)
                           : few_launch<PK_F16>(fa, d.sms, stream);
    return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
  }
  rows::Copies copies(dtype);
  if (f.x) copies.add(x, ldx, T, K, f.x);
  if (f.w) copies.add(w, K, 2 * static_cast<int64_t>(F), K, f.w);
  if (copies.launch(d.sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  gemm::Args a = {};
  a.M = static_cast<int>(T);
  a.N = 2 * F;
  a.K = K;
  a.status = status ? status : rows::stream_status(d, stream);
  a.timeout_ns = wait_limit_ns();
  const gemm::Operand A = f.x ? rows::operand_of_copy(dtype, f.x, T, K, 0) : rows::operand(dtype, x, ldx, T, K, 0);
  const gemm::Operand B = f.w ? rows::operand_of_copy(dtype, f.w, a.N, K, 0) : rows::operand(dtype, w, K, a.N, K, 0);
  r = dtype == PK_F32    ? product_of<PK_F32>(A, B, a, ep, f, d.sms, stream)
      : dtype == PK_BF16 ? product_of<PK_BF16>(A, B, a, ep, f, d.sms, stream)
                         : product_of<PK_F16>(A, B, a, ep, f, d.sms, stream);
  return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

int pk_gated_linear_backward_workspace(int dtype, const void* x, int64_t ldx, const void* w, int need_dx, int need_dw, int need_db,
                                       int64_t T, int F, int K, int64_t* bytes) {
  using namespace pk;
  if (!bytes || !rows::dtype_ok(dtype) || !sizes_ok(T, F, K) || ldx < K) return PK_ERR_ARG;
  *bytes = 0;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  *bytes = plan_backward(dtype, x, ldx, w, need_dx != 0, need_dw != 0, need_db != 0, T, F, K, d.sms, nullptr).bytes;
  return PK_OK;
}

int pk_gated_linear_backward(int dtype, const void* x, int64_t ldx, const void* w, const void* dy, int64_t lddy, const void* pre,
                             int act, int64_t T, int F, int K, void* dx, void* dw, void* db, void* workspace,
                             int64_t workspace_bytes, int* status, struct CUstream_st* stream) {
  using namespace pk;
  if (!rows::dtype_ok(dtype) || !sizes_ok(T, F, K) || !act_ok(act) || ldx < K || lddy < F || workspace_bytes < 0) return PK_ERR_ARG;
  if (T > 0 && (!dy || !pre || (dw && !x) || (dx && !w))) return PK_ERR_ARG;
  const int e = rows::elem_bytes(dtype), N = 2 * F;
  if (!rows::aligned_to(x, e) || !rows::aligned_to(w, e) || !rows::aligned_to(dy, e) || !rows::aligned_to(pre, e) ||
      !rows::aligned_to(dx, e) || !rows::aligned_to(dw, e) || !rows::aligned_to(db, e) || !rows::aligned_to(workspace, 256) ||
      !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) {
    // no rows: the gradients of the weights are zero
    if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
    if (dw && cudaMemsetAsync(dw, 0, static_cast<size_t>(e) * N * K, stream) != cudaSuccess) return PK_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, static_cast<size_t>(e) * N, stream) != cudaSuccess) return PK_ERR_CUDA;
    return PK_OK;
  }
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Bwd b = plan_backward(dtype, x, ldx, w, dx != nullptr, dw != nullptr, db != nullptr, T, F, K, d.sms, workspace);
  if (b.bytes > 0 && (!workspace || workspace_bytes < b.bytes)) return PK_ERR_NOMEM;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  if (b.dz || b.part) {
    DzArgs z = {};
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
    if (dz_launch(dtype, z, F, stream) != cudaSuccess) return PK_ERR_CUDA;
    if (db && rows::sum_rows(dtype, b.part, b.blocks, nullptr, 1, N, z.ldz, nullptr, db, stream) != cudaSuccess) return PK_ERR_CUDA;
  }
  return back_products(dtype, b, x, ldx, w, nullptr, 0, T, N, K, dx, dw, status ? status : rows::stream_status(d, stream), d.sms, stream);
}

}  // extern "C"
