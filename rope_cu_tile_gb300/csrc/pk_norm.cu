// pk_norm.cu -- the root-mean-square norm of token rows with the residual's addition, its gradient, and its form with rows in
// 8 bits (pk_rms_norm, pk_rms_norm_backward, pk_rms_norm_q8, pk_quantize_rows in include/pk.h).
//
//     h = x + r,   y = w h / sqrt(mean(h^2) + eps)                        x, r, h, y [T, D], w [D]
//     n = h / sqrt(mean(h^2) + eps),  g = dy w:   dx = (g - n mean(g n)) / sqrt(mean(h^2) + eps) + dh,   dw = sum over rows of dy n
//     8 bits: s = max |y| / 448 of a row, q = e4m3(y / s)
//
// All of it is bound by bytes: each element is read once and held in registers, a row's sums go through shuffles (and
// shared memory where a row takes more than a warp), and everything is written once.
#include <cfloat>

#include "pk_rows.cuh"

namespace pk {

namespace {

using namespace rows;

constexpr int kMaxD = PK_NORM_MAX_D;

enum Mode { kNorm, kNormQ8, kQuantize };

struct NormArgs {
  const void* x;
  const void* res;
  const void* w;
  void* y;       // in the element type, or 8 bits
  void* h;       // x + res, or null
  float* scale;  // of the 8-bit rows
  int64_t ldx, ldr, ldy, ldh;
  int64_t T;
  int D;
  float eps, inv_d;
};

// A row belongs to kTpr threads, each with kNg groups of 16 bytes, kTpr groups apart: 8 threads for the shortest rows,
// so that a warp's lanes all have something to load, up to a block of 512 for the longest; 32 elements a thread in flight
// wherever the row has as many.
template <int kTpr>
constexpr int kBlock = kTpr <= 32 ? 256 : kTpr;

// A group of elements, 16 bytes of them: neighbours where every row of every matrix begins and ends on a 16-byte boundary
// (kWhole), pairs of 16-bit elements where on a 4-byte one (kPairs; a warp then reads 128 bytes at once, not 64), else single
// columns, 2 kTpr or kTpr apart so that a warp's accesses are of neighbours. `n`: columns of the row from the first.
enum Unit { kSingle, kPairs, kWhole };
template <int DT>
constexpr int kE = 16 / Ty<DT>::kBytes;
template <int DT, int kTpr, int kUnit>
struct Group {
  static constexpr int E = kE<DT>;
  static constexpr bool kVec = kUnit == kWhole;
  uint4 q;
  // the first column of group i, and how far element j's is from it
  static __device__ __forceinline__ int column(int i, int t) {
    return kVec ? (i * kTpr + t) * E : i * E * kTpr + (kUnit == kPairs ? 2 * t : t);
  }
  static __device__ __forceinline__ constexpr int offset(int j) {
    return kVec ? j : kUnit == kPairs ? (j >> 1) * 2 * kTpr + (j & 1) : j * kTpr;
  }
  __device__ __forceinline__ void load(const void* p, int64_t at, int n) {
    if constexpr (kVec) {
      q = __ldcg(reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * Ty<DT>::kBytes));
    } else if constexpr (kUnit == kPairs) {
      const uint16_t* s = static_cast<const uint16_t*>(p) + at;
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = offset(2 * j) < n ? __ldcg(reinterpret_cast<const unsigned int*>(s + offset(2 * j))) : 0u;
      q = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < E; ++j) {
        if constexpr (DT == PK_F32) {
          w[j] = j * kTpr < n ? __ldcg(static_cast<const unsigned int*>(p) + at + j * kTpr) : 0u;
        } else {
          const uint32_t x = j * kTpr < n ? __ldcg(static_cast<const unsigned short*>(p) + at + j * kTpr) : 0u;
          w[j >> 1] = j & 1 ? w[j >> 1] | x << 16 : x;
        }
      }
      q = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // the weights, which every row reads again: through L1
  __device__ __forceinline__ void load_shared(const void* p, int at, int n) {
    if constexpr (kVec)
      q = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + at * Ty<DT>::kBytes);
    else
      load(p, at, n);
  }
  __device__ __forceinline__ void get(float (&v)[E]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == PK_F32) {
        v[j] = __uint_as_float(w[j]);
      } else {
        const float2 f = Elem<DT == PK_BF16>::unpack(w[j]);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
  }
  // the elements as they were loaded from here on: what was unpacked of them before is not kept in registers
  __device__ __forceinline__ void forget() { asm volatile("" : "+r"(q.x), "+r"(q.y), "+r"(q.z), "+r"(q.w)); }
  static __device__ __forceinline__ void store(void* p, int64_t at, int n, const float (&v)[E]) {
    if constexpr (DT != PK_F32 && kUnit != kSingle) {
      using P = Elem<DT == PK_BF16>;
      const uint32_t w[4] = {P::pack(v[0], v[1]), P::pack(v[2], v[3]), P::pack(v[4], v[5]), P::pack(v[6], v[7])};
      uint16_t* d = static_cast<uint16_t*>(p) + at;
      if constexpr (kVec) {
        *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (offset(2 * j) < n) *reinterpret_cast<uint32_t*>(d + offset(2 * j)) = w[j];
      }
    } else if constexpr (kVec) {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (offset(j) < n) Ty<DT>::put(p, at + offset(j), v[j]);
    }
  }
};

// N sums (or maxima, where bit i of kMax is set) over a row's threads, in every one of them. `red`: 2 x 16 x N floats, used
// alternately so that one barrier a row is enough.
template <int kTpr, int N, int kMax>
__device__ __forceinline__ void row_reduce(float (&v)[N], float* red, int& turn) {
#pragma unroll
  for (int o = (kTpr < 32 ? kTpr : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float u = __shfl_xor_sync(0xffffffffu, v[i], o);
      v[i] = (kMax >> i) & 1 ? fmaxf(v[i], u) : v[i] + u;
    }
  if constexpr (kTpr > 32) {
    constexpr int kWarps = kTpr / 32;
    float* r = red + turn * 16 * N;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[(threadIdx.x >> 5) * N + i] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = r[i];
#pragma unroll
      for (int k = 1; k < kWarps; ++k) v[i] = (kMax >> i) & 1 ? fmaxf(v[i], r[k * N + i]) : v[i] + r[k * N + i];
    }
  }
}

// N values (4 or 8) as e4m3, four a word
template <int N>
__device__ __forceinline__ void to_e4m3(const float (&v)[N], uint32_t (&q)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * i + 1]), "f"(v[4 * i]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * i + 3]), "f"(v[4 * i + 2]));
    q[i] = lo | static_cast<uint32_t>(hi) << 16;
  }
}

// Bound by bytes: 131072 x 1024 bf16 with a residual 161 us, 1.0 of the copy rate; 100000 x 1024 to 8 bits 114 us (issue slots
// half full); rows off the 16-byte grid pay for narrower accesses (100000 x 1002 bf16 167 us by pairs, x 1003 305 one by one, 120 of bytes).
// blocks of an SM: 85 registers a thread, 128 of fp32
template <int DT, int kTpr>
constexpr int kResident = kTpr > 256 ? 1 : (DT == PK_F32 ? 512 : 768) / kBlock<kTpr>;

template <int DT, int kMode, int kTpr, int kNg, int kUnit>
__global__ void __launch_bounds__(kBlock<kTpr>, (kResident<DT, kTpr>))
    pk_norm_kernel(const __grid_constant__ NormArgs a) {
  using G = Group<DT, kTpr, kUnit>;
  constexpr int E = G::E;
  constexpr bool kVec = G::kVec;
  __shared__ float red[kTpr > 32 ? 2 * 16 * 2 : 1];
  constexpr int kRows = kBlock<kTpr> / kTpr;
  const int t = threadIdx.x % kTpr;
  int turn = 0;
  griddep_wait();
  // (the rows of one warp go round together: the shuffles are warp-wide)
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows; r0 < a.T; r0 += static_cast<int64_t>(gridDim.x) * kRows) {
    const int64_t row = r0 + threadIdx.x / kTpr;
    const int D = row < a.T ? a.D : 0;  // (no columns of a row that is not there)
    float h[kNg][E];
    {
      G x[kNg], res[kNg];
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t);
        if (c < D) {
          x[i].load(a.x, row * a.ldx + c, D - c);
          if (kMode != kQuantize && a.res) res[i].load(a.res, row * a.ldr + c, D - c);
        }
      }
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t);
#pragma unroll
        for (int j = 0; j < E; ++j) h[i][j] = 0.0f;
        if (c < D) {
          x[i].get(h[i]);
          if (kMode != kQuantize && a.res) {
            float b[E];
            res[i].get(b);
#pragma unroll
            for (int j = 0; j < E; ++j) h[i][j] += b[j];
          }
          if (kMode != kQuantize && a.h) G::store(a.h, row * a.ldh + c, D - c, h[i]);
        }
      }
    }
    if constexpr (kMode != kQuantize) {
      float s[1];
      const auto squares = [&]() {
        s[0] = 0.0f;
#pragma unroll
        for (int i = 0; i < kNg; ++i)
#pragma unroll
          for (int j = 0; j < E; ++j) s[0] = fmaf(h[i][j], h[i][j], s[0]);
        row_reduce<kTpr, 1, 0>(s, red, turn);
      };
      squares();
      // squares past fp32's range (elements past 2^58 or so): the row times a power of two, beside which eps is nothing
      const bool past = s[0] > FLT_MAX;
      float eps = a.eps;
      if (kTpr > 32 ? past : __any_sync(0xffffffffu, past)) {
        const float down = past ? 0x1p-80f : 1.0f;
        eps = past ? 0.0f : eps;
#pragma unroll
        for (int i = 0; i < kNg; ++i)
#pragma unroll
          for (int j = 0; j < E; ++j) h[i][j] *= down;
        squares();
      }
      const float f = rsqrtf(fmaf(s[0], a.inv_d, eps));
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t);
        if (c < D) {
          G w;
          w.load_shared(a.w, c, D - c);
          float b[E];
          w.get(b);
#pragma unroll
          for (int j = 0; j < E; ++j) h[i][j] = h[i][j] * f * b[j];
          if constexpr (kMode == kNorm) G::store(a.y, row * a.ldy + c, D - c, h[i]);
        }
      }
    }
    if constexpr (kMode != kNorm) {
      // (a maximum passes over NaN: a row that holds one gets a NaN scale, so that nobody takes the others for its values)
      float m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kNg; ++i)
#pragma unroll
        for (int j = 0; j < E; ++j) {
          m[0] = fmaxf(m[0], fabsf(h[i][j]));
          m[1] = h[i][j] != h[i][j] ? 1.0f : m[1];
        }
      row_reduce<kTpr, 2, 3>(m, red, turn);
      const float scale = m[1] != 0.0f ? __int_as_float(0x7fc00000) : m[0] * (1.0f / 448.0f);
      // the inverse of a scale near fp32's smallest numbers would be infinite: two factors then
      const float up = scale < 0x1p-100f ? 0x1p60f : 1.0f;
      const float inv = scale > 0.0f ? 1.0f / (scale * up) : (scale == 0.0f ? 0.0f : scale);
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t);
        if (c < D) {
#pragma unroll
          for (int j = 0; j < E; ++j) h[i][j] = h[i][j] * up * inv;
          uint32_t q[E / 4];
          to_e4m3(h[i], q);
          uint8_t* d = static_cast<uint8_t*>(a.y) + row * a.ldy + c;
          if constexpr (kVec) {
            if constexpr (E == 8)
              *reinterpret_cast<uint2*>(d) = make_uint2(q[0], q[1]);
            else
              *reinterpret_cast<uint32_t*>(d) = q[0];
          } else {
#pragma unroll
            for (int j = 0; j < E; ++j)
              if (G::offset(j) < D - c) d[G::offset(j)] = static_cast<uint8_t>(q[j / 4] >> (8 * (j & 3)));
          }
        }
      }
      if (D > 0 && t == 0) a.scale[row] = scale;
    }
  }
}

// values as pairs, for arithmetic on two at a time
template <int N>
__device__ __forceinline__ float2 pair(const float (&v)[N], int i) {
  return make_float2(v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

struct NormBackArgs {
  const void* h;
  const void* w;
  const void* dy;
  const void* dh;
  void* dx;     // or null
  float* part;  // [blocks, D] sums of dy n over a block's rows, or null
  int64_t ldh, lddy, lddh, lddx;
  int64_t T;
  int D;
  float eps, inv_d;
};

// A block keeps its columns' sums of dy n in registers over all of its rows, so there are only as many blocks as are resident
// at once, and few threads: what covers the latency is that each thread's groups of the next rows are on their way into
// shared memory (kVec; a thread reads back what it asked for itself, so nothing is synchronized).
// 16931 x 768 bf16 with dh: 19.4 us (23.8 without that, on 16 warps an SM with a row in flight each), and 2.7 to add the
// blocks' sums; 131072 x 768 124 us, 0.98 of the copy rate.
template <int DT, int kTpr>
constexpr int kBackThreads = kTpr > 256 ? kTpr : 512;  // of an SM: 128 registers
template <int DT, int kTpr>
constexpr int kBackResident = kBackThreads<DT, kTpr> / kBlock<kTpr>;
template <int DT, int kTpr, int kNg>
constexpr int kRowBytes = kBlock<kTpr> * kNg * 16;  // a block's groups of one input
// stages of the three inputs: two, or one fewer where they do not fit
template <int DT, int kTpr, int kNg>
constexpr int kStages = 6 * kRowBytes<DT, kTpr, kNg> * kBackResident<DT, kTpr> <= 200 * 1024 ? 2 : 1;
template <int DT, int kTpr, int kNg, int kUnit>
constexpr int back_smem() {
  const int ring = kUnit == kWhole ? 3 * kStages<DT, kTpr, kNg> * kRowBytes<DT, kTpr, kNg> : 0, cols = kTpr <= 32 ? kBlock<kTpr> * kNg * kE<DT> * 4 : 0;
  return ring > cols ? ring : cols;
}

template <int DT, int kTpr, int kNg, int kUnit>
__global__ void __launch_bounds__(kBlock<kTpr>, (kBackResident<DT, kTpr>)) pk_norm_backward_kernel(const __grid_constant__ NormBackArgs a) {
  using G = Group<DT, kTpr, kUnit>;
  constexpr int E = G::E;
  constexpr bool kVec = G::kVec;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[kTpr > 32 ? 2 * 16 * 2 : 1];
  constexpr int kRows = kBlock<kTpr> / kTpr, kCols = kTpr * kNg * E, kS = kStages<DT, kTpr, kNg>;
  const int t = threadIdx.x % kTpr;
  int turn = 0;
  float2 sum[kNg][E / 2];
  G held[DT == PK_F32 ? 1 : kNg];  // the weights, where the registers hold them
  griddep_wait();
#pragma unroll
  for (int i = 0; i < kNg; ++i) {
    const int c = G::column(i, t);
#pragma unroll
    for (int j = 0; j < E / 2; ++j) sum[i][j] = twice(0.0f);
    if (DT != PK_F32 && c < a.D) held[DT == PK_F32 ? 0 : i].load(a.w, c, a.D - c);
  }
  const auto weights = [&](int i, int c, float(&g)[E]) {
    if constexpr (DT == PK_F32) {
      G w;
      w.load_shared(a.w, c, a.D - c);
      w.get(g);
    } else {
      held[i].get(g);
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  // this thread's 16 bytes of group i of input k in a stage
  const auto slot = [&](int stage, int k, int i) {
    return smem + (((stage * 3 + k) * kNg + i) * kBlock<kTpr> + threadIdx.x) * 16;
  };
  // inputs [k0, k1) of a row into a stage; every call makes one group of copies
  const auto ask = [&](int stage, int64_t r0, auto k0, auto k1) {
    const int64_t row = r0 + threadIdx.x / kTpr;
    if (row < a.T) {
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t);
        if (c < a.D) {
          const void* const base[3] = {a.h, a.dy, a.dh};
          const int64_t ld[3] = {a.ldh, a.lddy, a.lddh};
#pragma unroll
          for (int k = decltype(k0)::value; k < decltype(k1)::value; ++k)
            if (k < 2 || a.dh) {
              const char* src = static_cast<const char*>(base[k]) + (row * ld[k] + c) * Ty<DT>::kBytes;
asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot(stage, k, i))), "l"(src) : "memory");
            }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  using K0 = std::integral_constant<int, 0>;
  using K2 = std::integral_constant<int, 2>;
  using K3 = std::integral_constant<int, 3>;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kRows;
  if constexpr (kVec) {
#pragma unroll
    for (int k = 0; k < kS; ++k) {
      ask(k, first + k * step, K0(), K2());
      ask(k, first + k * step, K2(), K3());
    }
  }
  int stage = 0;
  for (int64_t r0 = first; r0 < a.T; r0 += step) {
    const int64_t row = r0 + threadIdx.x / kTpr;
    const int D = row < a.T ? a.D : 0;
    G xh[kNg], xd[kNg];
    if constexpr (kVec) asm volatile("cp.async.wait_group %0;" ::"n"(2 * (kS - 1)) : "memory");
    const auto read = [&](G& x, int k, int i) { x.q = *reinterpret_cast<const uint4*>(slot(stage, k, i)); };
#pragma unroll
    for (int i = 0; i < kNg; ++i) {
      const int c = G::column(i, t);
      if (c < D) {
        if constexpr (kVec) {
          read(xh[i], 0, i);
          read(xd[i], 1, i);
        } else {
          xh[i].load(a.h, row * a.ldh + c, D - c);
          xd[i].load(a.dy, row * a.lddy + c, D - c);
        }
      }
    }
    float s[2];
    const auto sums = [&](auto scaled) {
      float2 hh = twice(0.0f), hg = twice(0.0f);
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t);
        if (c < D) {
          float h[E], d[E], g[E];
          xh[i].get(h);
          xd[i].get(d);
          weights(i, c, g);
#pragma unroll
          for (int j = 0; j < E / 2; ++j) {
            float2 x = pair(h, j);
            if constexpr (decltype(scaled)::value) x = mul2(x, twice(0x1p-80f));
            hh = fma2(x, x, hh);
            hg = fma2(x, mul2(pair(d, j), pair(g, j)), hg);
          }
        }
      }
      s[0] = hh.x + hh.y;
      s[1] = hg.x + hg.y;
      row_reduce<kTpr, 2, 0>(s, red, turn);
    };
    sums(std::false_type());
    float down = 1.0f, eps = a.eps;
    // (as forwards: squares past fp32's range)
    const bool past = s[0] > FLT_MAX;
    if (kTpr > 32 ? past : __any_sync(0xffffffffu, past)) {
      const float whole[2] = {s[0], s[1]};
      sums(std::true_type());
      if (past) {
        down = 0x1p-80f;
        eps = 0.0f;
      } else {
        s[0] = whole[0];
        s[1] = whole[1];
      }
    }
    // (h and dy have been read: the sums are made of them)
    if constexpr (kVec) ask(stage, r0 + kS * step, K0(), K2());
    const float f = rsqrtf(fmaf(s[0], a.inv_d, eps));  // of h times `down`
    const float mean = s[1] * a.inv_d * f;             // of g n
    const float2 rate = twice(f * down), mean2 = twice(-mean);
    if constexpr (DT != PK_F32) {
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        xh[i].forget();
        xd[i].forget();
        held[i].forget();
      }
    }
#pragma unroll
    for (int i = 0; i < kNg; ++i) {
      const int c = G::column(i, t);
      if (c < D) {
        float n[E], d[E], g[E];
        xh[i].get(n);
        xd[i].get(d);
        weights(i, c, g);
#pragma unroll
        for (int j = 0; j < E / 2; ++j) {
          const float2 x = mul2(pair(n, j), rate), y = pair(d, j);
          sum[i][j] = fma2(y, x, sum[i][j]);
          const float2 v = mul2(fma2(x, mean2, mul2(y, pair(g, j))), rate);
          d[2 * j] = v.x;
          d[2 * j + 1] = v.y;
        }
        if (a.dx) {
          if (a.dh) {
            G xr;
            if constexpr (kVec)
              read(xr, 2, i);
            else
              xr.load(a.dh, row * a.lddh + c, D - c);
            xr.get(n);
#pragma unroll
            for (int j = 0; j < E; j += 2) add2(d[j], d[j + 1], make_float2(n[j], n[j + 1]));
          }
          G::store(a.dx, row * a.lddx + c, D - c, d);
        }
      }
    }
    if constexpr (kVec) {
      ask(stage, r0 + kS * step, K2(), K3());  // (and dh: what was written is made of it)
      stage = stage + 1 == kS ? 0 : stage + 1;
    }
  }
  if constexpr (kVec) asm volatile("cp.async.wait_all;" ::: "memory");
  if (!a.part) return;
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.D;
  float* cols = reinterpret_cast<float*>(smem);
  if constexpr (kTpr <= 32) __syncthreads();  // (the stages have been read)
#pragma unroll
  for (int i = 0; i < kNg; ++i)
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const int c = G::column(i, t) + G::offset(j);
      const float v = j & 1 ? sum[i][j >> 1].y : sum[i][j >> 1].x;
      if constexpr (kTpr > 32) {
        if (c < a.D) part[c] = v;
      } else {
        cols[threadIdx.x / kTpr * kCols + c] = v;
      }
    }
  if constexpr (kTpr <= 32) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += kBlock<kTpr>) {
      float v = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) v += cols[r * kCols + c];
      part[c] = v;
    }
  }
}

// dw from the blocks' sums: 32 threads a column, joined in a fixed order.
template <int DT>
__global__ void __launch_bounds__(1024) pk_norm_weight_kernel(const float* part, int blocks, int D, void* dw) {
  __shared__ float s[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  griddep_wait();
  float v = 0.0f;
  if (c < D) {
#pragma unroll 8
    for (int r = g; r < blocks; r += 32) v += __ldcg(part + static_cast<int64_t>(r) * D + c);
  }
  s[g][threadIdx.x & 31] = v;
  __syncthreads();
  if (g == 0 && c < D) {
    for (int i = 1; i < 32; ++i) v += s[i][threadIdx.x];
    Ty<DT>::put(dw, c, v);
  }
}

// How a row of D elements is shared out.
template <int A, int B>
struct Cut {
  static constexpr int kTpr = A, kElems = B;  // threads a row, elements a thread
};
template <class F>
cudaError_t by_length(int D, const F& f) {
  if (D <= 64) return f(Cut<8, 8>());
  if (D <= 256) return f(Cut<8, 32>());
  if (D <= 1024) return f(Cut<32, 32>());
  if (D <= 2048) return f(Cut<64, 32>());
  if (D <= 4096) return f(Cut<128, 32>());
  if (D <= 8192) return f(Cut<256, 32>());
  return f(Cut<512, 32>());
}
// (ragged rows are bound by their narrow accesses: fewer lengths)
template <class F>
cudaError_t by_ragged_length(int D, const F& f) {
  if (D <= 256) return f(Cut<8, 32>());
  if (D <= 1024) return f(Cut<32, 32>());
  if (D <= 4096) return f(Cut<128, 32>());
  if (D <= 8192) return f(Cut<256, 32>());
  return f(Cut<512, 32>());
}
static_assert(512 * 32 == kMaxD, "the longest row");

// What every row of a matrix begins and ends on, and of several together.
Unit unit_of(const void* p, int64_t ld, int D, int e) {
  if (rows16(p, ld, e) && (D * e & 15) == 0) return kWhole;
  return e == 2 && aligned_to(p, 4) && ((ld | D) & 1) == 0 ? kPairs : kSingle;
}
Unit least(Unit a, Unit b) { return a < b ? a : b; }

// f(Cut, Unit) for a row length and an alignment
template <int DT, class F>
cudaError_t by_shape(int D, Unit unit, const F& f) {
  if (unit == kWhole) return by_length(D, [&](auto cut) { return f(cut, std::integral_constant<int, kWhole>()); });
  return by_ragged_length(D, [&](auto cut) {
    if constexpr (DT != PK_F32)
      if (unit == kPairs) return f(cut, std::integral_constant<int, kPairs>());
    return f(cut, std::integral_constant<int, kSingle>());
  });
}

template <int DT, int kMode>
cudaError_t norm_launch(const NormArgs& a, Unit unit, int sms, cudaStream_t stream) {
  return by_shape<DT>(a.D, unit, [&](auto cut, auto u) {
    constexpr int kTpr = decltype(cut)::kTpr, kNg = decltype(cut)::kElems / kE<DT>, kRows = kBlock<kTpr> / kTpr;
    const int64_t blocks = (a.T + kRows - 1) / kRows, most = static_cast<int64_t>(sms) * (2048 / kBlock<kTpr>);
    Launch l(blocks < most ? blocks : most, kBlock<kTpr>, stream);
    return cudaLaunchKernelEx(&l.cfg, pk_norm_kernel<DT, kMode, kTpr, kNg, decltype(u)::value>, a);
  });
}

// Blocks of the backward pass: as many as are resident at once, each with its own partial column sums. The workspace is for the
// most of any alignment.
template <int DT>
int64_t back_blocks_of(int64_t T, int D, Unit unit, int sms) {
  int64_t n = 0;
  by_shape<DT>(D, unit, [&](auto cut, auto) {
    constexpr int kTpr = decltype(cut)::kTpr, kRows = kBlock<kTpr> / kTpr;
    const int64_t blocks = (T + kRows - 1) / kRows, most = static_cast<int64_t>(sms) * kBackResident<DT, kTpr>;
    n = blocks < most ? blocks : most;
    return cudaSuccess;
  });
  return n;
}
int64_t back_bytes(int dtype, int64_t T, int D, int sms) {
  const auto most = [&](auto type) {
    constexpr int DT = decltype(type)::value;
    const int64_t a = back_blocks_of<DT>(T, D, kWhole, sms), b = back_blocks_of<DT>(T, D, kSingle, sms);
    return (a > b ? a : b) * D * 4;
  };
  return dtype == PK_F32 ? most(std::integral_constant<int, PK_F32>()) : most(std::integral_constant<int, PK_BF16>());
}

template <int DT>
cudaError_t back_launch(const NormBackArgs& a, Unit unit, int sms, void* dw, cudaStream_t stream) {
  const int64_t blocks = back_blocks_of<DT>(a.T, a.D, unit, sms);
  return by_shape<DT>(a.D, unit, [&](auto cut, auto u) {
    constexpr int kTpr = decltype(cut)::kTpr, kNg = decltype(cut)::kElems / kE<DT>, kUnit = decltype(u)::value;
    Launch l(blocks, kBlock<kTpr>, stream);
    l.cfg.dynamicSmemBytes = back_smem<DT, kTpr, kNg, kUnit>();
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, pk_norm_backward_kernel<DT, kTpr, kNg, kUnit>, a);
    if (e != cudaSuccess || !dw) return e;
    Launch lw((a.D + 31) / 32, 1024, stream);
    const float* part = a.part;
    return cudaLaunchKernelEx(&lw.cfg, pk_norm_weight_kernel<DT>, part, static_cast<int>(blocks), a.D, dw);
  });
}

// the shared memory that the backward kernels may ask for
template <int DT>
cudaError_t prepare_back() {
  cudaError_t e = cudaSuccess;
  for (const int D : {64, 256, 1024, 2048, 4096, 8192, kMaxD}) {
    e = by_length(D, [&](auto cut) {
      constexpr int kTpr = decltype(cut)::kTpr, kNg = decltype(cut)::kElems / kE<DT>;
      return cudaFuncSetAttribute(pk_norm_backward_kernel<DT, kTpr, kNg, kWhole>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  back_smem<DT, kTpr, kNg, kWhole>());
    });
    if (e != cudaSuccess) return e;
  }
  return e;
}

bool sizes_ok(int dtype, int64_t T, int D) { return dtype_ok(dtype) && T >= 0 && T <= PK_ROWS_MAX_T && D >= 1 && D <= kMaxD; }
bool eps_ok(float eps) { return eps > 0.0f && eps <= FLT_MAX; }

int run_norm(int mode, int dtype, const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* w, float eps,
             int64_t T, int D, void* y, int64_t ldy, float* scale, void* h, int64_t ldh, cudaStream_t stream) {
  if (!sizes_ok(dtype, T, D) || (mode != kQuantize && !eps_ok(eps)) || ldx < D || ldy < D || (residual && ldr < D) || (h && ldh < D))
    return PK_ERR_ARG;
  if (T > 0 && (!x || !y || (mode != kQuantize && !w) || (mode != kNorm && !scale))) return PK_ERR_ARG;
  const int e = elem_bytes(dtype);
  if (!aligned_to(x, e) || !aligned_to(residual, e) || !aligned_to(w, e) || !aligned_to(h, e) || !aligned_to(scale, 4) ||
      (mode == kNorm && !aligned_to(y, e)))
    return PK_ERR_ALIGN;
  if (T == 0) return PK_OK;
  Device d;
  const int rc = device(&d);
  if (rc != PK_OK) return rc;
  NormArgs a = {};
  a.x = x;
  a.res = residual;
  a.w = w;
  a.y = y;
  a.h = h;
  a.scale = scale;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldy = ldy;
  a.ldh = ldh;
  a.T = T;
  a.D = D;
  a.eps = eps;
  a.inv_d = 1.0f / static_cast<float>(D);
  Unit unit = least(unit_of(x, ldx, D, e), unit_of(w, D, D, e));  // (a null w is aligned)
  if (residual) unit = least(unit, unit_of(residual, ldr, D, e));
  if (h) unit = least(unit, unit_of(h, ldh, D, e));
  if (mode == kNorm)
    unit = least(unit, unit_of(y, ldy, D, e));
  else if (unit == kWhole && !(aligned_to(y, 16 / e) && (ldy & (16 / e - 1)) == 0))
    unit = kSingle;
  const auto run = [&](auto type) {
    constexpr int DT = decltype(type)::value;
    if (mode == kNorm) return norm_launch<DT, kNorm>(a, unit, d.sms, stream);
    if (mode == kNormQ8) return norm_launch<DT, kNormQ8>(a, unit, d.sms, stream);
    return norm_launch<DT, kQuantize>(a, unit, d.sms, stream);
  };
  const cudaError_t r = dtype == PK_F32    ? run(std::integral_constant<int, PK_F32>())
                        : dtype == PK_BF16 ? run(std::integral_constant<int, PK_BF16>())
                                           : run(std::integral_constant<int, PK_F16>());
  return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // namespace

namespace rows {
cudaError_t prepare_norm() {
  cudaError_t e;
  if ((e = prepare_back<PK_F32>()) != cudaSuccess) return e;
  if ((e = prepare_back<PK_BF16>()) != cudaSuccess) return e;
  return prepare_back<PK_F16>();
}
}  // namespace rows

}  // namespace pk

extern "C" {

int pk_rms_norm(int dtype, const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* w, float eps, int64_t T,
                int D, void* y, int64_t ldy, void* h, int64_t ldh, struct CUstream_st* stream) {
  return pk::run_norm(pk::kNorm, dtype, x, ldx, residual, ldr, w, eps, T, D, y, ldy, nullptr, h, ldh, stream);
}

int pk_rms_norm_q8(int dtype, const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* w, float eps, int64_t T,
                   int D, void* q, int64_t ldq, float* scale, void* h, int64_t ldh, struct CUstream_st* stream) {
  return pk::run_norm(pk::kNormQ8, dtype, x, ldx, residual, ldr, w, eps, T, D, q, ldq, scale, h, ldh, stream);
}

int pk_quantize_rows(int dtype, const void* x, int64_t ldx, int64_t T, int D, void* q, int64_t ldq, float* scale,
                     struct CUstream_st* stream) {
  return pk::run_norm(pk::kQuantize, dtype, x, ldx, nullptr, 0, nullptr, 0.0f, T, D, q, ldq, scale, nullptr, 0, stream);
}

int pk_rms_norm_backward_workspace(int dtype, int64_t T, int D, int need_dw, int64_t* bytes) {
  using namespace pk;
  if (!bytes || !sizes_ok(dtype, T, D)) return PK_ERR_ARG;
  *bytes = 0;
  if (T == 0 || !need_dw) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  *bytes = back_bytes(dtype, T, D, d.sms);
  return PK_OK;
}

int pk_rms_norm_backward(int dtype, const void* h, int64_t ldh, const void* w, const void* dy, int64_t lddy, const void* dh,
                         int64_t lddh, float eps, int64_t T, int D, void* dx, int64_t lddx, void* dw, void* workspace,
                         int64_t workspace_bytes, struct CUstream_st* stream) {
  using namespace pk;
  if (!sizes_ok(dtype, T, D) || !eps_ok(eps) || ldh < D || lddy < D || (dh && lddh < D) || (dx && lddx < D) || workspace_bytes < 0)
    return PK_ERR_ARG;
  if (T > 0 && (!h || !w || !dy)) return PK_ERR_ARG;
  const int e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(h, e) || !rows::aligned_to(w, e) || !rows::aligned_to(dy, e) || !rows::aligned_to(dh, e) ||
      !rows::aligned_to(dx, e) || !rows::aligned_to(dw, e) || !rows::aligned_to(workspace, 256))
    return PK_ERR_ALIGN;
  // no rows: the weights' gradient is zero
  if (T == 0) return dw && cudaMemsetAsync(dw, 0, static_cast<size_t>(e) * D, stream) != cudaSuccess ? PK_ERR_CUDA : PK_OK;
  if (!dx && !dw) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  if (dw && (!workspace || workspace_bytes < back_bytes(dtype, T, D, d.sms))) return PK_ERR_NOMEM;
  NormBackArgs a = {};
  a.h = h;
  a.w = w;
  a.dy = dy;
  a.dh = dh;
  a.dx = dx;
  a.part = dw ? static_cast<float*>(workspace) : nullptr;
  a.ldh = ldh;
  a.lddy = lddy;
  a.lddh = lddh;
  a.lddx = lddx;
  a.T = T;
  a.D = D;
  a.eps = eps;
  a.inv_d = 1.0f / static_cast<float>(D);
  Unit unit = least(least(unit_of(h, ldh, D, e), unit_of(dy, lddy, D, e)), unit_of(w, D, D, e));
  if (dh) unit = least(unit, unit_of(dh, lddh, D, e));
  if (dx) unit = least(unit, unit_of(dx, lddx, D, e));
  const cudaError_t r = dtype == PK_F32    ? back_launch<PK_F32>(a, unit, d.sms, dw, stream)
                        : dtype == PK_BF16 ? back_launch<PK_BF16>(a, unit, d.sms, dw, stream)
                                           : back_launch<PK_F16>(a, unit, d.sms, dw, stream);
  return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // extern "C"
