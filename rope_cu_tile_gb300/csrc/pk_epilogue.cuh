// pk_epilogue.cuh -- what happens to the fp32 accumulators of a product before they are stored: bias, activation,
// dropout, residual, one rounding to the element type. The same steps serve the tensor-core product (a thread holds 32
// columns of one row), the sum of the splits of k (8 columns of one row) and the few-row kernel (one element).
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

// Eight consecutive elements at a 16-byte boundary: through L2, or with L1 where they are read often (a bias, a few rows).
// Never by the read-only path, which asks that nothing wrote them since this kernel started: with overlapping launches an
// earlier kernel of the chain may have.
template <int DT, bool L1 = false>
__device__ __forceinline__ void load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (DT == PK_F32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 a = L1 ? *s : __ldcg(s);
    const float4 b = L1 ? s[1] : __ldcg(s + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint4 q = L1 ? *s : __ldcg(s);
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
// Eight elements as loaded, for loads that are asked for well before they are used.
template <int DT>
struct Raw8 {
  uint4 q[DT == PK_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i, bool vec, int n) {
    if (vec && n >= 8) {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * Ty<DT>::kBytes);
      q[0] = __ldcg(s);
      if constexpr (DT == PK_F32) q[1] = __ldcg(s + 1);
      return;
    }
    uint32_t w[DT == PK_F32 ? 8 : 4] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        if constexpr (DT == PK_F32)
          w[j] = static_cast<const uint32_t*>(p)[i + j];
        else
          w[j >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i + j]) << (16 * (j & 1));
      }
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (DT == PK_F32) q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
    if constexpr (DT == PK_F32) {
      const uint32_t u[4] = {q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[j]), v[4 + j] = __uint_as_float(u[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = Elem<DT == PK_BF16>::unpack(w[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  }
};
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

// Eight fp32 values as three planes of bf16, v = hi + mid + lo. hi stays finite where v is: the values past bf16's largest
// would round to infinity, and mid holds what is left of them (as of infinity, which thus stays non-finite).
__device__ __forceinline__ void planes8(float (&v)[8], uint32_t (&h)[3][4]) {
  constexpr float kMost = 3.3895313892515355e38f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[0][i] = Elem<true>::pack(fminf(fmaxf(v[2 * i], -kMost), kMost), fminf(fmaxf(v[2 * i + 1], -kMost), kMost));
#pragma unroll
    for (int k = 1; k < 3; ++k) {
      const float2 b = Elem<true>::unpack(h[k - 1][i]);
      v[2 * i] -= b.x;
      v[2 * i + 1] -= b.y;
      h[k][i] = Elem<true>::pack(v[2 * i], v[2 * i + 1]);
    }
  }
}

// ------------------------------------------------------------------------------------
// activations (value, and slope at z). fp32 results take the full-precision functions (erfcf, expf). 16-bit ones take
// short exponentials and reciprocals, good to some 2^-17 relative where the result's rounding is 2^-11 or 2^-8: dz of a
// feed-forward layer is bound by issue slots.

// Two fp32 operations an instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\t"
      "mov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ void add2(float& x, float& y, float2 b) {
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\tadd.rn.f32x2 a, a, b;\n\t"
      "mov.b64 {%0, %1}, a;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(b.x), "f"(b.y));
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Phi(-u), u >= 0, of two values, for 16-bit results: 2 to a polynomial of degree 7 fitted (minimax, in the exponent) to
// log2 Phi(-u) on [0, 6]. Relative error below 2^-17 there, so the negative tail of gelu keeps its digits; past 6 the value
// only falls (from 1e-9), past 13 it is 0. 3.5 packed multiplications and one exponential an element, where the
// complementary error function takes some forty instructions.
__device__ __forceinline__ float2 tail2(float u0, float u1) {
  const float2 u = make_float2(u0, u1);
  float2 q = make_float2(-1.835213084e-06f, -1.835213084e-06f);
  q = fma2(q, u, make_float2(6.160594057e-05f, 6.160594057e-05f));
  q = fma2(q, u, make_float2(-9.305796120e-04f, -9.305796120e-04f));
  q = fma2(q, u, make_float2(8.508067578e-03f, 8.508067578e-03f));
  q = fma2(q, u, make_float2(-5.396029353e-02f, -5.396029353e-02f));
  q = fma2(q, u, make_float2(-4.584644139e-01f, -4.584644139e-01f));
  q = fma2(q, u, make_float2(-1.151250839e+00f, -1.151250839e+00f));
  q = fma2(q, u, make_float2(-9.999952912e-01f, -9.999952912e-01f));
  return make_float2(attn::ex2(q.x), attn::ex2(q.y));
}

// act(v) of a row's columns; DT: the type of the result, which says how exact it has to be
template <int DT, int N>
__device__ __forceinline__ void act_values(int act, float (&v)[N]) {
  if (act == PK_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] > 0.0f ? v[i] : (v[i] != v[i] ? v[i] : 0.0f);
  } else if (act == PK_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      if constexpr (DT == PK_F32) {
        // (z kept finite below: -inf times the 0 of its tail has no value)
        v[i] = fmaxf(v[i], -3.0e38f) * (0.5f * erfcf(v[i] * -0.70710678118654752f));
        v[i + 1] = fmaxf(v[i + 1], -3.0e38f) * (0.5f * erfcf(v[i + 1] * -0.70710678118654752f));
      } else {
        // z Phi(z) = max(z, 0) - |z| Phi(-|z|), either sign. The factor |z| stays finite, so that infinity gives infinity;
        // NaN comes through the tail.
        const float u0 = fabsf(v[i]), u1 = fabsf(v[i + 1]);
        const float2 e = tail2(u0, u1);
        v[i] = fmaf(-fminf(u0, 3.0e38f), e.x, fmaxf(v[i], 0.0f));
        v[i + 1] = fmaf(-fminf(u1, 3.0e38f), e.y, fmaxf(v[i + 1], 0.0f));
      }
    }
  } else if (act == PK_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // (z kept finite below, as gelu's)
      if constexpr (DT == PK_F32)
        v[i] = fmaxf(v[i], -3.0e38f) / (1.0f + expf(-v[i]));
      else
        v[i] = fmaxf(v[i], -3.0e38f) * rcp_fast(1.0f + attn::ex2(v[i] * -1.4426950408889634f));
    }
  }
}

// d[i] *= act'(z[i])
template <int DT, int N>
__device__ __forceinline__ void act_slopes(int act, const float (&z)[N], float (&d)[N]) {
  if (act == PK_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = z[i] > 0.0f ? d[i] : (z[i] != z[i] ? z[i] : 0.0f);
  } else if (act == PK_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      // Phi(z) + z phi(z) is h = Phi(-u) - u phi(u), u = |z|, for z < 0 and 1 - h otherwise: h as it stands, so that the
      // negative tail keeps its digits (1/2 - (1/2 - h) keeps 2^-25 of 1: 4 % of the slope at -5.5, nothing past -6.5)
      const float2 u = make_float2(fabsf(z[i]), fabsf(z[i + 1]));
      float2 e;
      if constexpr (DT == PK_F32)
        e = make_float2(0.5f * erfcf(u.x * 0.70710678118654752f), 0.5f * erfcf(u.y * 0.70710678118654752f));
      else
        e = tail2(u.x, u.y);
      float2 f = mul2(u, u);
      if constexpr (DT == PK_F32) {
        f = make_float2(expf(-0.5f * f.x), expf(-0.5f * f.y));
      } else {
        f = mul2(f, make_float2(-0.72134752044448170f, -0.72134752044448170f));
        f = make_float2(attn::ex2(f.x), attn::ex2(f.y));
      }
      // (the factor u kept finite, so that an infinite z has the limits 0 and 1; NaN comes through e)
      const float2 g = make_float2(fminf(u.x, 3.0e38f), fminf(u.y, 3.0e38f));
      const float2 h = fma2(mul2(g, make_float2(-0.39894228040143268f, -0.39894228040143268f)), f, e);
      const float2 w = fma2(h, make_float2(-1.0f, -1.0f), make_float2(1.0f, 1.0f));
      const float2 v = mul2(make_float2(z[i] < 0.0f ? h.x : w.x, z[i + 1] < 0.0f ? h.y : w.y), make_float2(d[i], d[i + 1]));
      d[i] = v.x;
      d[i + 1] = v.y;
    }
  } else if (act == PK_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // 1 - h as the difference: off by some 2^-24 of 1, which counts times z: within 16 bits' rounding. In fp32 e h instead
      // for z > 0, where it is small.
      float h, rest;
      if constexpr (DT == PK_F32) {
        const float e = expf(-z[i]);
        h = 1.0f / (1.0f + e);
        rest = z[i] > 0.0f ? e * h : 1.0f - h;
      } else {
        h = rcp_fast(1.0f + attn::ex2(z[i] * -1.4426950408889634f));
        rest = 1.0f - h;
      }
      // (z kept finite: infinity times the 0 of h or 1 - h has no value; NaN comes through h)
      d[i] *= h * fmaf(fminf(fmaxf(z[i], -3.0e38f), 3.0e38f), rest, 1.0f);
    }
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
  const float* alpha;   // device factor of the whole, or null
  const int* rowmap;    // row of y that row m goes to, or null
  int act;
  DropArgs drop;
  int bias_vec, res_vec, y_vec, pre_vec;  // 16-byte rows: vector access
};

// The same for the tensor-core product: outputs whose rows begin and end on 16-byte boundaries are stored by TMA.
struct LinTiles : LinParams {
  CUtensorMap map_y, map_pre;
  int tma_y, tma_pre;
};

// A staged tile of 32 rows x 32 columns (64- or 128-byte rows, swizzled) to (x, y, plane) of a map, clipped at its ends: at the
// last row, and at the end of the last 16 bytes that a row's columns touch (the store fills those up with what is staged, so
// the memory behind a row that ends inside them has to be padding of the library's own). The warp's writes
// are made visible to the copy; `stage` may be written again after stored().
__device__ __forceinline__ void store_tile(const CUtensorMap* map, const uint8_t* stage, int x, int y, int plane, int lane) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(stage)), "r"(x), "r"(y), "r"(plane)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
__device__ __forceinline__ void stored(int lane) {
  if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}

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

// Staging of a warp's 32 rows x 32 columns of type DT: rows of 64 or 128 bytes in the swizzle that TMA reads (16-byte unit u
// of row r at unit u ^ (r / 2 mod 4), or u ^ (r mod 8)), which also keeps a column of lanes free of bank conflicts.
template <int DT>
struct Stage {
  static constexpr int kE = Ty<DT>::kBytes;
  static constexpr int kRow = 32 * kE;          // bytes
  static constexpr int kUnits = kRow / 16;      // of a row
  static constexpr int kPer = 16 / kE;          // elements of a unit
  static constexpr int kStep = 32 / kUnits;     // rows that a warp moves at once, 16 bytes a lane
  static __device__ __forceinline__ uint8_t* slot(uint8_t* stage, int r, int u) {
    return stage + r * kRow + ((u ^ (kE == 4 ? r & 7 : (r >> 1) & 3)) << 4);
  }
  // columns from unit u0 of this thread's row
  template <int NV>
  static __device__ __forceinline__ void put(uint8_t* stage, int lane, const float (&v)[NV], int u0 = 0) {
#pragma unroll
    for (int i = 0; i < NV / kPer; ++i) {
      uint4 q;
      if constexpr (kE == 4) {
        q = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                       __float_as_uint(v[4 * i + 3]));
      } else {
        using E = Elem<DT == PK_BF16>;
        q = make_uint4(E::pack(v[8 * i], v[8 * i + 1]), E::pack(v[8 * i + 2], v[8 * i + 3]),
                       E::pack(v[8 * i + 4], v[8 * i + 5]), E::pack(v[8 * i + 6], v[8 * i + 7]));
      }
      *reinterpret_cast<uint4*>(slot(stage, lane, u0 + i)) = q;
    }
  }
  // v[0 ..] += the elements of a unit
  static __device__ __forceinline__ void add_unit(const uint4& q, float* v) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kE == 4) {
        v[j] += __uint_as_float(w[j]);
      } else {
        add2(v[2 * j], v[2 * j + 1], Elem<DT == PK_BF16>::unpack(w[j]));
      }
    }
  }
  template <int NV>
  static __device__ __forceinline__ void add(uint8_t* stage, int lane, float (&v)[NV], int u0) {
#pragma unroll
    for (int i = 0; i < NV / kPer; ++i) add_unit(*reinterpret_cast<const uint4*>(slot(stage, lane, u0 + i)), v + i * kPer);
  }
  static __device__ __forceinline__ char* element(uint8_t* stage, int r, int c) {
    return reinterpret_cast<char*>(slot(stage, r, c / kPer)) + (c % kPer) * kE;
  }
  // The staged rows to rows of `out` where TMA cannot: a row map, or rows off the 16-byte grid (a column a lane).
  static __device__ __noinline__ void flush(uint8_t* stage, int lane, void* out, int64_t ld, int vec, const int* rowmap,
                                               int r0, int c0, int M, int N) {
    const int rows = min(32, M - r0);
    if (vec && c0 + 32 <= N) {
      const int u = lane % kUnits;
#pragma unroll
      for (int i = 0; i < 32 / kStep; ++i) {
        const int r = i * kStep + lane / kUnits;
        if (r >= rows) break;
        const int64_t row = rowmap ? __ldcg(rowmap + r0 + r) : r0 + r;
        *reinterpret_cast<uint4*>(static_cast<char*>(out) + (row * ld + c0 + u * kPer) * kE) =
            *reinterpret_cast<const uint4*>(slot(stage, r, u));
      }
      return;
    }
    if (c0 + lane >= N) return;
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
      const int64_t row = rowmap ? __ldcg(rowmap + r0 + r) : r0 + r;
      char* d = static_cast<char*>(out) + (row * ld + c0 + lane) * kE;
      if constexpr (kE == 4)
        *reinterpret_cast<uint32_t*>(d) = *reinterpret_cast<const uint32_t*>(element(stage, r, lane));
      else
        *reinterpret_cast<uint16_t*>(d) = *reinterpret_cast<const uint16_t*>(element(stage, r, lane));
    }
  }
  // Rows of `in` into the staging memory, by asynchronous copies (waited for where the values are used) where the rows allow.
  static __device__ __forceinline__ void fetch(uint8_t* stage, int lane, const void* in, int64_t ld, int vec, int r0, int c0,
                                               int M, int N) {
    const int rows = min(32, M - r0);
    if (vec && c0 + 32 <= N) {
      const int u = lane % kUnits;
#pragma unroll
      for (int i = 0; i < 32 / kStep; ++i) {
        const int r = i * kStep + lane / kUnits;
        if (r < rows)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot(stage, r, u))),
                       "l"(static_cast<const char*>(in) + ((static_cast<int64_t>(r0) + r) * ld + c0 + u * kPer) * kE)
                       : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return;
    }
    fetch_ragged(stage, lane, in, ld, r0, c0, rows, N);
  }
  static __device__ __noinline__ void fetch_ragged(uint8_t* stage, int lane, const void* in, int64_t ld, int r0, int c0,
                                                   int rows, int N) {
    if (c0 + lane >= N) return;
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
      const char* s = static_cast<const char*>(in) + ((static_cast<int64_t>(r0) + r) * ld + c0 + lane) * kE;
      if constexpr (kE == 4)
        *reinterpret_cast<uint32_t*>(element(stage, r, lane)) = __ldcg(reinterpret_cast<const uint32_t*>(s));
      else
        *reinterpret_cast<uint16_t*>(element(stage, r, lane)) = __ldcg(reinterpret_cast<const unsigned short*>(s));
    }
  }
};

// The bias of NC columns, asked for as stored (every lane the same) before the accumulators are waited for.
template <int DT, int NC>
struct Bias {
  using S = Stage<DT>;
  static constexpr int kUnits = NC / S::kPer;
  uint4 q[kUnits];
  __device__ __forceinline__ void fetch(const void* bias, int vec, int c, int N) {
    if (vec && c + NC <= N) {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const char*>(bias) + static_cast<int64_t>(c) * S::kE);
#pragma unroll
      for (int i = 0; i < kUnits; ++i) q[i] = s[i];
      return;
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < S::kPer; ++j) {
        const int at = c + i * S::kPer + j;
        if (at < N) {
          if constexpr (S::kE == 4)
            w[j] = static_cast<const uint32_t*>(bias)[at];
          else
            w[j >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(bias)[at]) << (16 * (j & 1));
        }
      }
      q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void add(float (&v)[NC]) const {
#pragma unroll
    for (int i = 0; i < kUnits; ++i) S::add_unit(q[i], v + i * S::kPer);
  }
};

__device__ __forceinline__ void read_acc(uint32_t t, bool zero, float (&v)[32]) {
  if (zero) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = 0.0f;
  } else {
    tmem_ld32(t, v);
  }
}

template <int ODT, int RDT>
struct LinEpi {
  using Params = LinTiles;
  using S = Stage<ODT>;
  // A chunk of 32 columns is a chain of a tensor-memory load, arithmetic and a staged store; four warps a scheduler cover each
  // other's (131072 x 1024 x 4096 with gelu and kept pre-activation: 1031 us on eight warps of 128 columns, 895 on sixteen of 64, at
  // the same time otherwise). fp32's staging is twice as large and has room for eight.
  static constexpr int kWarps = ODT == PK_F32 ? 8 : 16;

  // `ready` waits for the accumulators (false: give up), `done` hands them back. What comes from memory (bias, residual) is
  // asked for before the accumulators are waited for.
  template <class Ready, class Done>
  static __device__ __forceinline__ bool run(const Params& p, uint32_t tacc, bool zero, int r0, int c0, int cols, int M, int N,
                                             int split, int lane, uint8_t* stage, const Ready& ready, const Done& done) {
    if (r0 >= M || c0 >= N) {
      if (!ready()) return false;
      done();
      return true;
    }
    const int end = min(cols, N - c0);
    const bool res_staged = p.res && ODT == RDT;
#pragma unroll 1
    for (int cc = 0; cc < end; cc += 32) {
      const int c = c0 + cc;
      stored(lane);  // the previous chunk's tile has left the staging memory
      if (res_staged && !p.pre) S::fetch(stage, lane, p.res, p.ldres, p.res_vec, r0, c, M, N);
      float v[32];
      {
        Bias<ODT, 32> bias;
        if (p.bias) bias.fetch(p.bias, p.bias_vec, c, N);
        if (cc == 0 && !ready()) return false;
        read_acc(tacc + cc, zero, v);
        if (cc + 32 >= end) done();
        if (p.bias) bias.add(v);
      }
      if (p.pre) {
        S::put(stage, lane, v);
        if (p.tma_pre) {
          store_tile(&p.map_pre, stage, c, r0, 0, lane);
          stored(lane);
        } else {
          __syncwarp();
          S::flush(stage, lane, p.pre, p.ldpre, 0, nullptr, r0, c, M, N);
          __syncwarp();
        }
        if (res_staged) S::fetch(stage, lane, p.res, p.ldres, p.res_vec, r0, c, M, N);
      }
      act_values<ODT>(p.act, v);
      if (p.drop.cut) {
#pragma unroll
        for (int i = 0; i < 4; ++i) drop8(v + 8 * i, r0 + lane, c / 8 + i, p.drop);
      }
      if (res_staged) {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        S::add(stage, lane, v, 0);
      } else if (p.res && r0 + lane < M) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float b[8];
          const int64_t at = (r0 + lane) * p.ldres + c + 8 * i;
          const int n = N - c - 8 * i;
          if (p.res_vec && n >= 8)
            load8<RDT>(p.res, at, b);
          else
            load8_any<RDT>(p.res, at, n, b);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[8 * i + j] += b[j];
        }
      }
      if (p.alpha) {
        const float alpha = __ldcg(p.alpha);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= alpha;
      }
      S::put(stage, lane, v);
      if (p.tma_y) {
        store_tile(&p.map_y, stage, c, r0 + split * gemm::split_rows(M), 0, lane);
      } else {
        __syncwarp();
        S::flush(stage, lane, p.y, p.ldy, p.y_vec, p.rowmap, r0, c, M, N);
        __syncwarp();
      }
    }
    return true;
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
  act_values<ODT>(p.act, v);
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

// The same for one element.
template <int ODT>
__device__ __forceinline__ void finish1(const LinParams& p, float x, int64_t row, int c) {
  if (p.bias) x += Ty<ODT>::get(p.bias, c);
  if (p.pre) Ty<ODT>::put(p.pre, row * p.ldpre + c, x);
  float v[2] = {x, 0.0f};
  act_values<ODT>(p.act, v);
  x = v[0];
  if (p.drop.cut) {
    const uint4 r = philox(c >> 3, static_cast<uint32_t>(row), p.drop);
    const uint32_t w = (c & 4) ? ((c & 2) ? r.w : r.z) : ((c & 2) ? r.y : r.x);
    x = ((c & 1) ? w >> 16 : w & 0xFFFFu) >= p.drop.cut ? x * p.drop.scale : 0.0f;
  }
  if (p.res) x += Ty<ODT>::get(p.res, row * p.ldres + c);
  Ty<ODT>::put(p.y, row * p.ldy + c, x);
}

}  // namespace pk
