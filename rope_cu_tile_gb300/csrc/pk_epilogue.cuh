// pk_epilogue.cuh -- what happens to the fp32 accumulators of a product before they are stored: bias, activation,
// dropout, residual, one rounding to the element type. The same steps serve the tensor-core product (a thread holds 32
// columns of one row), the sum of the splits of k and the few-row kernel (a thread holds 8 columns of one row).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pk.h"
#include "pk_gemm.cuh"
#include "pk_philox.cuh"

namespace pk {

// ------------------------------------------------------------------------------------
// element types

template <int DT>
struct Ty;
template <>
struct Ty<PK_F32> {
  using T = float;
  static constexpr int kBytes = 4;
  static __device__ __forceinline__ float get(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  static __device__ __forceinline__ void put(void* p, int64_t i, float v) { static_cast<float*>(p)[i] = v; }
};
template <>
struct Ty<PK_BF16> {
  using T = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float get(const void* p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  }
  static __device__ __forceinline__ void put(void* p, int64_t i, float v) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  }
};
template <>
struct Ty<PK_F16> {
  using T = uint16_t;
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float get(const void* p, int64_t i) {
    return __half2float(static_cast<const __half*>(p)[i]);
  }
  static __device__ __forceinline__ void put(void* p, int64_t i, float v) { static_cast<__half*>(p)[i] = __float2half_rn(v); }
};

// Eight consecutive elements at a 16-byte boundary. Through L2 unless L1 is asked for: what a kernel earlier in a chain of
// overlapping launches wrote must not be taken from a line that this SM read before, and only a bias is read often.
template <int DT, bool L1 = false>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (DT == PK_F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = L1 ? __ldg(s) : __ldcg(s);
    const float4 b = L1 ? __ldg(s + 1) : __ldcg(s + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint4 q = L1 ? __ldg(s) : __ldcg(s);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = Elem<DT == PK_BF16>::unpack(u[j]);
      v[2 * j] = f.x;
      v[2 * j + 1] = f.y;
    }
  }
}
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (DT == PK_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    using E = Elem<DT == PK_BF16>;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(E::pack(v[0], v[1]), E::pack(v[2], v[3]), E::pack(v[4], v[5]), E::pack(v[6], v[7]));
  }
}
// the same for any alignment, the elements at and past `n` left out (loaded as zero)
template <int DT>
__device__ __forceinline__ void load8_any(const void* p, int64_t i, int n, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = j < n ? Ty<DT>::get(p, i + j) : 0.0f;
}
template <int DT>
__device__ __forceinline__ void store8_any(void* p, int64_t i, int n, const float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) Ty<DT>::put(p, i + j, v[j]);
}

// ------------------------------------------------------------------------------------
// activations (value, and slope at z)

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case PK_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case PK_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678118654752f);
    case PK_ACT_SILU: return z / (1.0f + __expf(-z));
    default: return z;
  }
}
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case PK_ACT_RELU: return z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
    case PK_ACT_GELU:
      return 0.5f * erfcf(z * -0.70710678118654752f) + z * 0.39894228040143268f * __expf(-0.5f * z * z);
    case PK_ACT_SILU: {
      const float h = 1.0f / (1.0f + __expf(-z));
      return h * (1.0f + z * (1.0f - h));
    }
    default: return 1.0f;
  }
}

// ------------------------------------------------------------------------------------
// the linear epilogue

struct LinParams {
  const void* bias;     // [N] in the output's type, or null
  const void* res;      // [M, N] in the residual's type, or null
  void* y;              // [M, N]
  void* pre;            // [M, N] in the output's type: bias added, before the activation; or null
  int64_t ldres, ldy, ldpre;
  int64_t split_stride; // elements between the outputs of two splits of k (0: one split)
  const float* alpha;   // device factor of the whole, or null
  const int* rowmap;    // row of y (and of the mask) that row m goes to, or null
  int act;
  DropArgs drop;
  int bias_vec, res_vec, y_vec, pre_vec;  // 16-byte rows: vector access
};

inline bool rows16(const void* p, int64_t ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ((ld * bytes) & 15) == 0;
}

// bias for 8 columns
template <int DT>
__device__ __forceinline__ void bias8(const LinParams& p, int c, int n, float (&b)[8]) {
  if (p.bias_vec && n >= 8)
    load8<DT, true>(p.bias, c, b);
  else
    load8_any<DT>(p.bias, c, n, b);
}

template <int ODT, int RDT>
struct LinEpi {
  using Params = LinParams;
  static constexpr int kE = Ty<ODT>::kBytes;
  static constexpr int kChunk = 128 / kE;  // columns of one staged row of 128 bytes

  // staging: 16-byte unit u of row r sits at unit u ^ (r & 7) of its 128-byte row
  static __device__ __forceinline__ uint4* slot(uint8_t* stage, int r, int u) {
    return reinterpret_cast<uint4*>(stage + r * 128 + ((u ^ (r & 7)) << 4));
  }

  // 32 accumulator columns of this thread's row, with the bias
  static __device__ __forceinline__ void take(const Params& p, uint32_t t, bool zero, int c, int N, float (&v)[32]) {
    if (zero) {
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] = 0.0f;
    } else {
      tmem_ld32(t, v);
    }
    if (p.bias) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float b[8];
        bias8<ODT>(p, c + 8 * g, N - c - 8 * g, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * g + i] += b[i];
      }
    }
  }
  // 32 columns of this thread's row into the staging tile, units [u0, ..)
  static __device__ __forceinline__ void put(uint8_t* stage, int lane, int u0, const float (&v)[32]) {
    if constexpr (kE == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *slot(stage, lane, u0 + i) = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                                __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3]));
    } else {
      using E = Elem<ODT == PK_BF16>;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *slot(stage, lane, u0 + i) = make_uint4(E::pack(v[8 * i], v[8 * i + 1]), E::pack(v[8 * i + 2], v[8 * i + 3]),
                                                E::pack(v[8 * i + 4], v[8 * i + 5]), E::pack(v[8 * i + 6], v[8 * i + 7]));
    }
  }
  // the staging tile to rows of `out` (four rows a step, 16 bytes a lane)
  static __device__ __forceinline__ void flush(uint8_t* stage, int lane, void* out, int64_t ld, int vec, const int* rowmap,
                                               int r0, int c0, int M, int N) {
    const int u = lane & 7, c = c0 + u * (16 / kE);
    const int n = min(N - c, 16 / kE);
    if (n <= 0) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      if (r0 + r >= M) break;
      const uint4 q = *slot(stage, r, u);
      const int64_t row = rowmap ? __ldcg(rowmap + r0 + r) : r0 + r;
      char* d = static_cast<char*>(out) + (row * ld + c) * kE;
      if (vec && n == 16 / kE) {
        *reinterpret_cast<uint4*>(d) = q;
      } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 16 / kE; ++j)
          if (j < n) {
            if constexpr (kE == 4)
              reinterpret_cast<uint32_t*>(d)[j] = w[j];
            else
              reinterpret_cast<uint16_t*>(d)[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
          }
      }
    }
  }
  // rows of the residual (of the output's type) into the staging tile
  static __device__ __forceinline__ void fetch(uint8_t* stage, int lane, const void* in, int64_t ld, int vec, int r0, int c0,
                                               int M, int N) {
    const int u = lane & 7, c = c0 + u * (16 / kE);
    const int n = min(N - c, 16 / kE);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      uint4 q = make_uint4(0u, 0u, 0u, 0u);
      if (r0 + r < M && n > 0) {
        const char* s = static_cast<const char*>(in) + ((r0 + r) * ld + c) * kE;
        if (vec && n == 16 / kE) {
          q = __ldcg(reinterpret_cast<const uint4*>(s));
        } else {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int j = 0; j < 16 / kE; ++j)
            if (j < n) {
              if constexpr (kE == 4)
                w[j] = reinterpret_cast<const uint32_t*>(s)[j];
              else
                w[j >> 1] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(s)[j]) << (16 * (j & 1));
            }
          q = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      *slot(stage, r, u) = q;
    }
  }

  static __device__ __forceinline__ void run(const Params& p, uint32_t tacc, bool zero, int r0, int c0, int cols, int M,
                                             int N, int split, int lane, uint8_t* stage) {
    if (r0 >= M) return;
    const int row = r0 + lane;
    void* y = static_cast<char*>(p.y) + split * p.split_stride * kE;
    const float alpha = p.alpha ? __ldcg(p.alpha) : 1.0f;
    for (int cc = 0; cc < cols && c0 + cc < N; cc += kChunk) {
      const int c = c0 + cc;
      if (p.pre) {
#pragma unroll
        for (int h = 0; h < kChunk; h += 32) {
          float v[32];
          take(p, tacc + cc + h, zero, c + h, N, v);
          put(stage, lane, h * kE / 16, v);
        }
        __syncwarp();
        flush(stage, lane, p.pre, p.ldpre, p.pre_vec, nullptr, r0, c, M, N);
        __syncwarp();
      }
      if (p.res && ODT == RDT) {
        fetch(stage, lane, p.res, p.ldres, p.res_vec, r0, c, M, N);
        __syncwarp();
      }
#pragma unroll
      for (int h = 0; h < kChunk; h += 32) {
        float v[32];
        take(p, tacc + cc + h, zero, c + h, N, v);
        if (p.act != PK_ACT_NONE) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = act_value(p.act, v[i]);
        }
        if (p.drop.cut) {
#pragma unroll
          for (int g = 0; g < 4; ++g) drop8(v + 8 * g, row, (c + h) / 8 + g, p.drop);
        }
        if (p.res) {
          if constexpr (ODT == RDT) {
#pragma unroll
            for (int i = 0; i < 32 * kE / 16; ++i) {
              const uint4 q = *slot(stage, lane, h * kE / 16 + i);
              const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                if constexpr (kE == 4) {
                  v[4 * i + j] += __uint_as_float(w[j]);
                } else {
                  const float2 f = Elem<ODT == PK_BF16>::unpack(w[j]);
                  v[8 * i + 2 * j] += f.x;
                  v[8 * i + 2 * j + 1] += f.y;
                }
              }
            }
          } else if (row < M) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              float b[8];
              const int64_t at = row * p.ldres + c + h + 8 * g;
              const int n = N - c - h - 8 * g;
              if (p.res_vec && n >= 8)
                load8<RDT>(p.res, at, b);
              else
                load8_any<RDT>(p.res, at, n, b);
#pragma unroll
              for (int i = 0; i < 8; ++i) v[8 * g + i] += b[i];
            }
          }
        }
        if (p.alpha) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] *= alpha;
        }
        put(stage, lane, h * kE / 16, v);
      }
      __syncwarp();
      flush(stage, lane, y, p.ldy, p.y_vec, p.rowmap, r0, c, M, N);
      __syncwarp();
    }
  }
};

// The epilogue's steps for 8 columns of one row (sum of splits, few rows). `n`: columns from c to the end.
template <int ODT, int RDT>
__device__ __forceinline__ void finish8(const LinParams& p, float (&v)[8], int64_t row, int c, int n) {
  if (p.bias) {
    float b[8];
    bias8<ODT>(p, c, n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (p.pre) {
    if (p.pre_vec && n >= 8)
      store8<ODT>(p.pre, row * p.ldpre + c, v);
    else
      store8_any<ODT>(p.pre, row * p.ldpre + c, n, v);
  }
  if (p.act != PK_ACT_NONE) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_value(p.act, v[i]);
  }
  if (p.drop.cut) drop8(v, static_cast<uint32_t>(row), c / 8, p.drop);
  if (p.res) {
    float b[8];
    if (p.res_vec && n >= 8)
      load8<RDT>(p.res, row * p.ldres + c, b);
    else
      load8_any<RDT>(p.res, row * p.ldres + c, n, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += b[i];
  }
  if (p.alpha) {
    const float a = __ldcg(p.alpha);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= a;
  }
  if (p.rowmap) row = __ldcg(p.rowmap + row);
  if (p.y_vec && n >= 8)
    store8<ODT>(p.y, row * p.ldy + c, v);
  else
    store8_any<ODT>(p.y, row * p.ldy + c, n, v);
}

}  // namespace pk
