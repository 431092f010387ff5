// pk_philox.cuh -- the counter-based generator behind dropout: Philox4x32-10 as published by Salmon, Moraes, Dror and
// Shaw ("Parallel random numbers: as easy as 1, 2, 3", SC 2011). One call gives the bits of eight consecutive columns of a
// row, 16 bits an element, as a function of (seed, offset, row, column / 8) alone: nothing is stored and the backward
// pass, or a fused epilogue with another tile shape, draws the same bits again.
#pragma once

#include <stdint.h>

namespace pk {

// What dropout needs of a call: element kept where its 16 bits are at least `cut` = round(p 65536); kept elements are
// multiplied by scale = 65536 / (65536 - cut), the inverse of the exact keeping probability.
struct DropArgs {
  uint32_t cut;  // 0: no dropout
  float scale;
  uint32_t off0, off1;  // offset
  uint32_t key[20];     // the rounds' keys, from the seed: operands in constant memory rather than twenty additions a draw
};

__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, const DropArgs& d) {
  uint32_t x = c0, y = c1, z = d.off0, w = d.off1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(x) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(z) * 0xCD9E8D57u;
    const uint32_t nx = static_cast<uint32_t>(b >> 32) ^ y ^ d.key[2 * i];
    const uint32_t nz = static_cast<uint32_t>(a >> 32) ^ w ^ d.key[2 * i + 1];
    y = static_cast<uint32_t>(b);
    w = static_cast<uint32_t>(a);
    x = nx;
    z = nz;
  }
  return make_uint4(x, y, z, w);
}

// v[0 .. 7] (columns 8 group ..) with the dropped ones zero and the kept ones scaled. (A high half is at least `cut` exactly
// when its word is at least cut 2^16, so half of the comparisons need no extraction.)
__device__ __forceinline__ void drop8(float* v, uint32_t row, uint32_t group, const DropArgs& d) {
  const uint4 r = philox(group, row, d);
  const uint32_t u[4] = {r.x, r.y, r.z, r.w}, cut = d.cut << 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = (u[i] << 16) >= cut ? v[2 * i] * d.scale : 0.0f;
    v[2 * i + 1] = u[i] >= cut ? v[2 * i + 1] * d.scale : 0.0f;
  }
}

// Host: the generator's arguments of a call; false when p is not in [0, 1).
inline bool drop_args(double p, uint64_t seed, uint64_t offset, DropArgs* d) {
  if (!(p >= 0.0 && p < 1.0)) return false;
  const uint32_t cut = static_cast<uint32_t>(p * 65536.0 + 0.5);
  if (cut >= 65536u) return false;
  d->cut = cut;
  d->scale = static_cast<float>(65536.0 / (65536.0 - cut));
  for (uint32_t i = 0; i < 10; ++i) {
    d->key[2 * i] = static_cast<uint32_t>(seed) + i * 0x9E3779B9u;
    d->key[2 * i + 1] = static_cast<uint32_t>(seed >> 32) + i * 0xBB67AE85u;
  }
  d->off0 = static_cast<uint32_t>(offset);
  d->off1 = static_cast<uint32_t>(offset >> 32);
  return true;
}

}  // namespace pk
