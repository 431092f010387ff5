// pk_few.cuh -- dot products of a few rows of x with the rows of a weight matrix on the CUDA cores, shared by the projection
// and the gated feed-forward (serving: the weights' bytes are what such a call costs).
#pragma once

#include "pk_rows.cuh"

namespace pk {
namespace rows {

constexpr int kFewThreads = 256;

// rows of W a warp, and steps of k asked for together: as many 16-byte loads in flight as the registers of 16 warps an SM hold
__host__ __device__ constexpr int few_r(int dt, int tm) { return dt == PK_F32 && tm < 8 ? 2 : 4; }
__host__ __device__ constexpr int few_steps(int dt) { return dt == PK_F32 ? 1 : 2; }

// Warps that split k among them, where the `dots` groups of rows alone give too few warps: 1, 2, 4 or 8.
inline int few_share(int64_t dots, int K, int sms) {
  int share = 1;
  while (share < 8 && dots * share < 16 * sms && K > 256 * share) share *= 2;
  return share;
}

// acc[r][t] += this lane's share of W's row row(r) times x's row t, `sub` of `share` warps splitting k. Nothing where !some. kX: rows of x,
// in fp32, that are asked for together.
template <int DT, int kX, int kR, int TM, class RowOf>
__device__ __forceinline__ void few_dots(const void* x, int64_t ldx, int T, const void* w, int K, int vec, bool some, int sub,
                                         int share, int lane, const RowOf& row, float (&acc)[kR][TM]) {
  constexpr int kFewSteps = few_steps(DT);
  static_assert(TM % kX == 0, "");
#pragma unroll
  for (int r = 0; r < kR; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[r][t] = 0.0f;
  if (!some) return;
  const int step = share * 256;
#pragma unroll 1
  for (int k0 = sub * 256 + lane * 8; k0 < K; k0 += kFewSteps * step) {
    Raw8<DT> q[kFewSteps][kR];
#pragma unroll
    for (int s = 0; s < kFewSteps; ++s)
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const int k = k0 + s * step;
        if (k < K) q[s][r].load(w, static_cast<int64_t>(row(r)) * K + k, vec, K - k);
      }
#pragma unroll
    for (int s = 0; s < kFewSteps; ++s) {
      const int k = k0 + s * step;
      if (k >= K) break;
      if constexpr (DT != PK_F32) {
        // (a product of two 16-bit numbers is exact in fp32, and one instruction adds it)
        using E = Elem<DT == PK_BF16>;
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          Raw8<DT> b;
          const int64_t at = min(t, T - 1) * ldx + k;
          if (vec && k + 8 <= K)
            b.q[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
          else
            b.load(x, at, false, K - k);
          const uint32_t p[4] = {b.q[0].x, b.q[0].y, b.q[0].z, b.q[0].w};
#pragma unroll
          for (int r = 0; r < kR; ++r) {
            const uint32_t u[4] = {q[s][r].q[0].x, q[s][r].q[0].y, q[s][r].q[0].z, q[s][r].q[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[r][t] = E::fma_hi(u[j], p[j], E::fma_lo(u[j], p[j], acc[r][t]));
          }
        }
      } else {
        float v[kR][8];
#pragma unroll
        for (int r = 0; r < kR; ++r) q[s][r].get(v[r]);
#pragma unroll
        for (int t0 = 0; t0 < TM; t0 += kX) {
          float b[kX][8];
#pragma unroll
          for (int t = 0; t < kX; ++t) {
            const int64_t at = min(t0 + t, T - 1) * ldx + k;
            if (vec && k + 8 <= K)
              load8<DT, true>(x, at, b[t]);
            else
              load8_any<DT>(x, at, K - k, b[t]);
          }
#pragma unroll
          for (int t = 0; t < kX; ++t)
#pragma unroll
            for (int r = 0; r < kR; ++r)
#pragma unroll
              for (int j = 0; j < 8; ++j) acc[r][t0 + t] = fmaf(v[r][j], b[t][j], acc[r][t0 + t]);
        }
      }
    }
  }
}

}  // namespace rows
}  // namespace pk
