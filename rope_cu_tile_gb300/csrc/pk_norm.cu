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
  int period, shift, slide;  // kSlide: rows until the same shift, the first row's, and from a row to the next
};

// A row belongs to kTpr threads, each with kNg groups of 16 bytes, kTpr groups apart: 8 threads for the shortest rows,
// so that a warp's lanes all have something to load, up to a block of 512 for the longest; 32 elements a thread in flight
// wherever the row has as many.
template <int kTpr>
constexpr int kBlock = kTpr <= 32 ? 256 : kTpr;

// A group of elements, 16 bytes of them: neighbours where every row of every matrix begins and ends on a 16-byte boundary
// (kWhole) or where, in 16 bits, a row begins equally far past one in all of them (kSlide), else single columns kTpr apart, so
// that a warp's accesses are of neighbours (kSingle; of fp32 that is no slower: 50000 x 1003 145 us, 332 in groups).
//
// kSlide: a block takes only rows that begin `shift` elements past a boundary, every period-th one, so a thread has the same
// columns of each. Groups that hang over a row's first or last column are read with what stands beside them in the matrix, which
// is then cleared (of the matrix's first and last row, where nothing need stand there, by elements), and written in part.
enum Unit { kSingle, kSlide, kWhole };
template <int DT>
constexpr int kE = 16 / Ty<DT>::kBytes;
template <int DT, int kTpr, int kUnit>
struct Group {
  static constexpr int E = kE<DT>;
  static constexpr bool kVec = kUnit != kSingle;
  uint4 q;
  // the first column of group i (below 0 where it hangs over), and how far element j's is from it
  static __device__ __forceinline__ int column(int i, int t, int shift) {
    return kVec ? (i * kTpr + t) * E - (kUnit == kSlide ? shift : 0) : i * E * kTpr + t;
  }
  static __device__ __forceinline__ constexpr int offset(int j) { return kVec ? j : j * kTpr; }
  // whether 16 bytes are read: there is something on both sides of the row, or the group lies within it
  static __device__ __forceinline__ bool at_once(int c, int D, bool inner) { return kUnit == kWhole || inner || (c >= 0 && c + E <= D); }
  // of a group that hangs over: what is not of the row
  __device__ __forceinline__ void clear(int c, int D) {
    if constexpr (kUnit == kSlide) {
      uint32_t w[4] = {q.x, q.y, q.z, q.w};
      const auto from = [](int bit) { return __funnelshift_lc(0u, 0xFFFFFFFFu, max(bit, 0)); };  // bits `bit` and above
      if (c < 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] &= from(-16 * c - 32 * k);
      }
      if (c + E > D) {
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] &= ~from(16 * (D - c) - 32 * k);
      }
      q = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // columns c, c + offset(1) .. of a row of D that begins at element `at` of p
  __device__ __forceinline__ void load(const void* p, int64_t at, int c, int D, bool inner = false) {
    if (kVec && at_once(c, D, inner)) {
      q = __ldcg(reinterpret_cast<const uint4*>(static_cast<const char*>(p) + (at + c) * Ty<DT>::kBytes));
      clear(c, D);
      return;
    }
    if constexpr (kUnit != kWhole) load_each(p, at, c, D);
  }
  // the same by elements, wherever the row begins
  __device__ __forceinline__ void load_each(const void* p, int64_t at, int c, int D) {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    const char* s = static_cast<const char*>(p) + (at + c) * Ty<DT>::kBytes;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (offset(j) >= D - c || (kVec && c + offset(j) < 0)) continue;
      const char* d = s + offset(j) * Ty<DT>::kBytes;
      if constexpr (DT == PK_F32)
        w[j] = __ldcg(reinterpret_cast<const unsigned int*>(d));
      else
        w[j >> 1] |= static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short*>(d))) << (16 * (j & 1));
    }
    q = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // the weights, which every row reads again: through L1 (kWhole), from their copy in shared memory (kSlide), or by elements through L2
  // (kSingle, and kSlide's backward pass, which holds them from its start)
  __device__ __forceinline__ void load_shared(const void* p, int c, int D, const uint8_t* copy = nullptr, int i = 0, int t = 0) {
    if constexpr (kUnit == kWhole)
      q = *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + c * Ty<DT>::kBytes);
    else if (kUnit == kSlide && copy)
      q = *reinterpret_cast<const uint4*>(copy + (i * kTpr + t) * 16);
    else
      load_each(p, 0, c, D);  // (they need not begin where the rows do)
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
  static __device__ __forceinline__ void store(void* p, int64_t at, int c, int D, const float (&v)[E]) {
    if constexpr (kVec) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == PK_F32)
          w[j] = __float_as_uint(v[j]);
        else
          w[j] = Elem<DT == PK_BF16>::pack(v[2 * j], v[2 * j + 1]);
      }
      char* d = static_cast<char*>(p) + (at + c) * Ty<DT>::kBytes;
      if (kUnit == kWhole || (c >= 0 && c + E <= D)) {
        *reinterpret_cast<uint4*>(d) = make_uint4(w[0], w[1], w[2], w[3]);
        return;
      }
      if constexpr (kUnit == kSlide) {
        // what hangs over on one side: in pieces of 2, 4 and 8 bytes
        const auto word = [&](int k) { return k & 2 ? (k & 1 ? w[3] : w[2]) : k & 1 ? w[1] : w[0]; };
        if (c + E <= D) {
          const int s = -c, f = s + (s & 1), g = f + (f & 2);
          if (s & 1) *reinterpret_cast<uint16_t*>(d + 2 * s) = static_cast<uint16_t>(word(s >> 1) >> 16);
          if (f & 2) *reinterpret_cast<uint32_t*>(d + 2 * f) = word(f >> 1);
          if (g == 4) *reinterpret_cast<uint2*>(d + 8) = make_uint2(w[2], w[3]);
          return;
        }
        if (c >= 0) {
          const int n = D - c;
          if (n & 4) *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
          if (n & 2) *reinterpret_cast<uint32_t*>(d + 2 * (n & 4)) = word((n & 4) >> 1);
          if (n & 1) *reinterpret_cast<uint16_t*>(d + 2 * (n & 6)) = static_cast<uint16_t>(word((n & 6) >> 1));
          return;
        }
      }
    }
    if constexpr (kUnit != kWhole) {
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (offset(j) < D - c && (!kVec || c + offset(j) >= 0)) Ty<DT>::put(p, at + c + offset(j), v[j]);
    }
  }
};

// The rows of a block, and of its row of threads: all that are there, or every period-th from `first`.
struct Walk {
  int64_t first, rows, start, step;  // row first + k period, k < rows, from k = start (of the block's first) on
  int period, shift;
};
template <int kUnit, int kRows>
__device__ __forceinline__ Walk walk(int64_t T, int period, int shift0, int slide, int E) {
  Walk w = {0, T, static_cast<int64_t>(blockIdx.x) * kRows, static_cast<int64_t>(gridDim.x) * kRows, 1, 0};
  if constexpr (kUnit == kSlide) {
    const int residue = blockIdx.x % period;
    w.first = residue;
    w.period = period;
    w.rows = T > residue ? (T - residue + period - 1) / period : 0;
    w.start = static_cast<int64_t>(blockIdx.x / period) * kRows;
    w.step = static_cast<int64_t>(gridDim.x / period) * kRows;
    w.shift = (shift0 + residue * slide) & (E - 1);
  }
  return w;
}

// N sums (or maxima, where bit i of kMax is set) over a row's threads, in every one of them. `red`: two halves of kRedHalf floats,
// taken alternately, so that one barrier a call is enough: who writes a half has passed the barrier of the call between, and
// with it everyone has read what that half held before. The halves lie equally far apart whatever N is, as calls of
// different N follow one another in any number (a row whose squares are summed again makes one more).
constexpr int kRedHalf = 16 * 2;  // warps of the longest row x the most values
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
    static_assert(kWarps * N <= kRedHalf, "a half holds a call's values");
    float* r = red + turn * kRedHalf;
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
// half full); quantize_rows 100000 x 1024 bf16 54 (46 of bytes), 16384 x 4096 38 (30), 4096 x 16384 fp32 73 (50). Rows off the 16-byte
// grid 100000 x 1003 bf16 178 (120 of bytes; 313 in single columns): latency, the issue slots being 42 % full; warps wait for loads in 6.5
// of 11.7 cycles an instruction, 24 of them an SM, and 116 bytes a thread and row spilled from 80 registers are another half
// of the results' sectors to L2. (On the grid 52 bytes are spilled, which the copy rate hides.)
// blocks of an SM: 85 registers a thread, 128 of fp32
template <int DT, int kTpr>
constexpr int kResident = kTpr > 256 ? 1 : (DT == PK_F32 ? 512 : 768) / kBlock<kTpr>;

template <int DT, int kMode, int kTpr, int kNg, int kUnit>
__global__ void __launch_bounds__(kBlock<kTpr>, (kResident<DT, kTpr>))
    pk_norm_kernel(const __grid_constant__ NormArgs a) {
  using G = Group<DT, kTpr, kUnit>;
  constexpr int E = G::E;
  constexpr bool kVec = G::kVec;
  __shared__ float red[kTpr > 32 ? 2 * kRedHalf : 1];
  constexpr int kRows = kBlock<kTpr> / kTpr;
  const int t = threadIdx.x % kTpr;
  int turn = 0;
  const Walk rows = walk<kUnit, kRows>(a.T, a.period, a.shift, a.slide, E);
  const int shift = rows.shift;
  griddep_wait();
  // (16 bits: weights as the block's rows need them)
  constexpr bool kCopy = kUnit == kSlide && kMode != kQuantize;
  __shared__ __align__(16) uint8_t copy[kCopy ? kTpr * kNg * 16 : 16];
  if constexpr (kCopy) {
    for (int c = threadIdx.x; c < kTpr * kNg * E; c += kBlock<kTpr>)
      reinterpret_cast<uint16_t*>(copy)[c] = c >= shift && c - shift < a.D ? __ldcg(static_cast<const unsigned short*>(a.w) + c - shift) : 0;
    __syncthreads();
  }
  // (the rows of one warp go round together: the shuffles are warp-wide)
  for (int64_t k0 = rows.start; k0 < rows.rows; k0 += rows.step) {
    const int64_t k = k0 + threadIdx.x / kTpr, row = rows.first + k * rows.period;
    const int D = k < rows.rows ? a.D : 0;  // (no columns of a row that is not there)
    const bool inner = row > 0 && row + 1 < a.T;
    float h[kNg][E];
    {
      G x[kNg], res[kNg];
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t, shift);
        if (c < D) {
          x[i].load(a.x, row * a.ldx, c, D, inner);
          if (kMode != kQuantize && a.res) res[i].load(a.res, row * a.ldr, c, D, inner);
        }
      }
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t, shift);
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
          if (kMode != kQuantize && a.h) G::store(a.h, row * a.ldh, c, D, h[i]);
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
        const int c = G::column(i, t, shift);
        if (c < D) {
          G w;
          w.load_shared(a.w, c, D, kCopy ? copy : nullptr, i, t);
          float b[E];
          w.get(b);
#pragma unroll
          for (int j = 0; j < E; ++j) h[i][j] = h[i][j] * f * b[j];
          if constexpr (kMode == kNorm) G::store(a.y, row * a.ldy, c, D, h[i]);
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
        const int c = G::column(i, t, shift);
        if (c < D) {
#pragma unroll
          for (int j = 0; j < E; ++j) h[i][j] = h[i][j] * up * inv;
          uint32_t q[E / 4];
          to_e4m3(h[i], q);
          uint8_t* d = static_cast<uint8_t*>(a.y) + row * a.ldy + c;
          if (kVec && G::at_once(c, D, false)) {
            if constexpr (E == 8)
              *reinterpret_cast<uint2*>(d) = make_uint2(q[0], q[1]);
            else
              *reinterpret_cast<uint32_t*>(d) = q[0];
          } else {
#pragma unroll
            for (int j = 0; j < E; ++j) {
              const int e = c + G::offset(j);
              if (e < D && (!kVec || e >= 0)) d[G::offset(j)] = static_cast<uint8_t>(q[j / 4] >> (8 * (j & 3)));
            }
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
  int period, shift, slide;  // as of the norm
};

// A block keeps its columns' sums of dy n in registers over all of its rows, so there are only as many blocks as are resident
// at once, and few threads: what covers the latency is that each thread's groups of the next rows are on their way into
// shared memory (not kSingle; a thread reads back what it asked for itself, so nothing is synchronized).
// 16931 x 768 bf16 with dh: 18.0 us (23.8 without that, on 16 warps an SM with a row in flight each), and 2.7 to add the
// blocks' sums; 131072 x 768 124 us, 0.98 of the copy rate. Rows off the grid: 100000 x 763 146 us (249 in single columns).
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
  const int ring = kUnit != kSingle ? 3 * kStages<DT, kTpr, kNg> * kRowBytes<DT, kTpr, kNg> : 0, cols = kTpr <= 32 ? kBlock<kTpr> * kNg * kE<DT> * 4 : 0;
  return ring > cols ? ring : cols;
}

template <int DT, int kTpr, int kNg, int kUnit>
__global__ void __launch_bounds__(kBlock<kTpr>, (kBackResident<DT, kTpr>)) pk_norm_backward_kernel(const __grid_constant__ NormBackArgs a) {
  using G = Group<DT, kTpr, kUnit>;
  constexpr int E = G::E;
  constexpr bool kVec = G::kVec;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[kTpr > 32 ? 2 * kRedHalf : 1];
  constexpr int kRows = kBlock<kTpr> / kTpr, kCols = kTpr * kNg * E, kS = kStages<DT, kTpr, kNg>;
  const int t = threadIdx.x % kTpr;
  int turn = 0;
  const Walk rows = walk<kUnit, kRows>(a.T, a.period, a.shift, a.slide, E);
  const int shift = rows.shift;
  float2 sum[kNg][E / 2];
  G held[DT == PK_F32 ? 1 : kNg];  // the weights, where the registers hold them
  griddep_wait();
#pragma unroll
  for (int i = 0; i < kNg; ++i) {
    const int c = G::column(i, t, shift);
#pragma unroll
    for (int j = 0; j < E / 2; ++j) sum[i][j] = twice(0.0f);
    if (DT != PK_F32 && c < a.D) held[DT == PK_F32 ? 0 : i].load_shared(a.w, c, a.D);
  }
  const auto weights = [&](int i, int c, float(&g)[E]) {
    if constexpr (DT == PK_F32) {
      G w;
      w.load_shared(a.w, c, a.D);
      w.get(g);
    } else {
      held[i].get(g);
    }
  };
  // this thread's 16 bytes of group i of input k in a stage
  const auto slot = [&](int stage, int k, int i) {
    return smem + (((stage * 3 + k) * kNg + i) * kBlock<kTpr> + threadIdx.x) * 16;
  };
  // inputs [k0, k1) of a row into a stage; every call makes one group of copies
  const auto ask = [&](int stage, int64_t k0, auto i0, auto i1) {
    const int64_t n = k0 + threadIdx.x / kTpr, row = rows.first + n * rows.period;
    if (n < rows.rows) {
      const bool inner = row > 0 && row + 1 < a.T;
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t, shift);
        if (c < a.D) {
          const void* const base[3] = {a.h, a.dy, a.dh};
          const int64_t ld[3] = {a.ldh, a.lddy, a.lddh};
#pragma unroll
          for (int k = decltype(i0)::value; k < decltype(i1)::value; ++k)
            if (k < 2 || a.dh) {
              if (G::at_once(c, a.D, inner)) {
                const char* src = static_cast<const char*>(base[k]) + (row * ld[k] + c) * Ty<DT>::kBytes;
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(slot(stage, k, i))), "l"(src) : "memory");
              } else {
                G x;
                x.load(base[k], row * ld[k], c, a.D);
                *reinterpret_cast<uint4*>(slot(stage, k, i)) = x.q;
              }
            }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  using K0 = std::integral_constant<int, 0>;
  using K2 = std::integral_constant<int, 2>;
  using K3 = std::integral_constant<int, 3>;
  if constexpr (kVec) {
#pragma unroll
    for (int k = 0; k < kS; ++k) {
      ask(k, rows.start + k * rows.step, K0(), K2());
      ask(k, rows.start + k * rows.step, K2(), K3());
    }
  }
  int stage = 0;
  for (int64_t k0 = rows.start; k0 < rows.rows; k0 += rows.step) {
    const int64_t k = k0 + threadIdx.x / kTpr, row = rows.first + k * rows.period;
    const int D = k < rows.rows ? a.D : 0;
    G xh[kNg], xd[kNg];
    if constexpr (kVec) asm volatile("cp.async.wait_group %0;" ::"n"(2 * (kS - 1)) : "memory");
    const auto read = [&](G& x, int k, int i, int c) {
      x.q = *reinterpret_cast<const uint4*>(slot(stage, k, i));
      x.clear(c, D);
    };
#pragma unroll
    for (int i = 0; i < kNg; ++i) {
      const int c = G::column(i, t, shift);
      if (c < D) {
        if constexpr (kVec) {
          read(xh[i], 0, i, c);
          read(xd[i], 1, i, c);
        } else {
          xh[i].load(a.h, row * a.ldh, c, D);
          xd[i].load(a.dy, row * a.lddy, c, D);
        }
      }
    }
    float s[2];
    const auto sums = [&](auto scaled) {
      float2 hh = twice(0.0f), hg = twice(0.0f);
#pragma unroll
      for (int i = 0; i < kNg; ++i) {
        const int c = G::column(i, t, shift);
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
    if constexpr (kVec) ask(stage, k0 + kS * rows.step, K0(), K2());
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
      const int c = G::column(i, t, shift);
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
              read(xr, 2, i, c);
            else
              xr.load(a.dh, row * a.lddh, c, D);
            xr.get(n);
#pragma unroll
            for (int j = 0; j < E; j += 2) add2(d[j], d[j + 1], make_float2(n[j], n[j + 1]));
          }
          G::store(a.dx, row * a.lddx, c, D, d);
        }
      }
    }
    if constexpr (kVec) {
      ask(stage, k0 + kS * rows.step, K2(), K3());  // (and dh: what was written is made of it)
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
      const int c = G::column(i, t, shift) + G::offset(j);
      const float v = j & 1 ? sum[i][j >> 1].y : sum[i][j >> 1].x;
      if constexpr (kTpr > 32) {
        if (c < a.D && c >= 0) part[c] = v;
      } else {
        cols[threadIdx.x / kTpr * kCols + c + shift] = v;
      }
    }
  if constexpr (kTpr <= 32) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += kBlock<kTpr>) {
      float v = 0.0f;
#pragma unroll
      for (int r = 0; r < kRows; ++r) v += cols[r * kCols + c + shift];
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

// How far past a 16-byte boundary (of the element type) the rows of several matrices begin: whether they do so equally.
struct Shifts {
  int e, D;
  bool whole = true, alike = true, any = false;
  int first = 0, slide = 0;  // elements: of the first row, and from a row to the next
  // `unit`: bytes of an element of this matrix
  void add(const void* p, int64_t ld, int unit) {
    const int E = 16 / e, f = static_cast<int>(reinterpret_cast<uintptr_t>(p) / unit) & (E - 1), s = static_cast<int>(ld & (E - 1));
    alike = alike && ld >= E && (!any || (f == first && s == slide));
    if (!any) {
      first = f;
      slide = s;
    }
    any = true;
    whole = whole && f == 0 && s == 0;
  }
  int period() const { return slide == 0 ? 1 : 16 / e / (slide & -slide); }
  Unit unit(const void* w) const {
    if (whole && aligned_to(w, 16) && (D * e & 15) == 0) return kWhole;
    return e == 2 && alike && D + 16 / e - 1 <= kMaxD ? kSlide : kSingle;
  }
};

// f(Cut, Unit) for a row length and an alignment
template <int DT, class F>
cudaError_t by_shape(int D, Unit unit, const F& f) {
  if (unit == kWhole) return by_length(D, [&](auto cut) { return f(cut, std::integral_constant<int, kWhole>()); });
  if constexpr (DT != PK_F32)
    if (unit == kSlide)
      return by_ragged_length(D + kE<DT> - 1, [&](auto cut) { return f(cut, std::integral_constant<int, kSlide>()); });
  return by_ragged_length(D, [&](auto cut) { return f(cut, std::integral_constant<int, kSingle>()); });
}
// Blocks of kRows rows each, `most` at once: of every shift as many.
int64_t blocks_for(int64_t T, int rows, int64_t most, int period) {
  const int64_t each = ((T + period - 1) / period + rows - 1) / rows, room = most / period > 1 ? most / period : 1;
  return (each < room ? each : room) * period;
}

template <int DT, int kMode>
cudaError_t norm_launch(const NormArgs& a, Unit unit, int sms, cudaStream_t stream) {
  return by_shape<DT>(a.D, unit, [&](auto cut, auto u) {
    constexpr int kTpr = decltype(cut)::kTpr, kNg = decltype(cut)::kElems / kE<DT>, kRows = kBlock<kTpr> / kTpr;
    Launch l(blocks_for(a.T, kRows, static_cast<int64_t>(sms) * (2048 / kBlock<kTpr>), a.period), kBlock<kTpr>, stream);
    return cudaLaunchKernelEx(&l.cfg, pk_norm_kernel<DT, kMode, kTpr, kNg, decltype(u)::value>, a);
  });
}

// Blocks of the backward pass: as many as are resident at once, each with its own partial column sums. The workspace is for the
// most of any alignment.
template <int DT>
int64_t back_blocks_of(int64_t T, int D, Unit unit, int period, int sms) {
  int64_t n = 0;
  by_shape<DT>(D, unit, [&](auto cut, auto) {
    constexpr int kTpr = decltype(cut)::kTpr;
    n = blocks_for(T, kBlock<kTpr> / kTpr, static_cast<int64_t>(sms) * kBackResident<DT, kTpr>, period);
    return cudaSuccess;
  });
  return n;
}
int64_t back_bytes(int dtype, int64_t T, int D, int sms) {
  const auto most = [&](auto type) {
    constexpr int DT = decltype(type)::value;
    int64_t n = back_blocks_of<DT>(T, D, kWhole, 1, sms);
    const auto or_else = [&](int64_t m) { n = m > n ? m : n; };
    or_else(back_blocks_of<DT>(T, D, kSingle, 1, sms));
    if (DT != PK_F32 && D + kE<DT> - 1 <= kMaxD)
      for (int period = 1; period <= kE<DT>; period *= 2) or_else(back_blocks_of<DT>(T, D, kSlide, period, sms));
    return n * D * 4;
  };
  return dtype == PK_F32 ? most(std::integral_constant<int, PK_F32>()) : most(std::integral_constant<int, PK_BF16>());
}

template <int DT>
cudaError_t back_launch(const NormBackArgs& a, Unit unit, int sms, void* dw, cudaStream_t stream) {
  const int64_t blocks = back_blocks_of<DT>(a.T, a.D, unit, a.period, sms);
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
    const auto allow = [&](auto cut, auto u) {
      constexpr int kTpr = decltype(cut)::kTpr, kNg = decltype(cut)::kElems / kE<DT>, kUnit = decltype(u)::value;
      return cudaFuncSetAttribute(pk_norm_backward_kernel<DT, kTpr, kNg, kUnit>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  back_smem<DT, kTpr, kNg, kUnit>());
    };
    if ((e = by_shape<DT>(D, kWhole, allow)) != cudaSuccess) return e;
    if (DT != PK_F32 && (e = by_shape<DT>(D - kE<DT> + 1, kSlide, allow)) != cudaSuccess) return e;
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
  Shifts shifts = {e, D};
  shifts.add(x, ldx, e);
  if (residual) shifts.add(residual, ldr, e);
  if (h) shifts.add(h, ldh, e);
  shifts.add(y, ldy, mode == kNorm ? e : 1);
  const Unit unit = shifts.unit(w);  // (a null w is aligned)
  a.period = unit == kSlide ? shifts.period() : 1;
  a.shift = shifts.first;
  a.slide = shifts.slide;
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
  Shifts shifts = {e, D};
  shifts.add(h, ldh, e);
  shifts.add(dy, lddy, e);
  if (dh) shifts.add(dh, lddh, e);
  if (dx) shifts.add(dx, lddx, e);
  const Unit unit = shifts.unit(w);
  a.period = unit == kSlide ? shifts.period() : 1;
  a.shift = shifts.first;
  a.slide = shifts.slide;
  const cudaError_t r = dtype == PK_F32    ? back_launch<PK_F32>(a, unit, d.sms, dw, stream)
                        : dtype == PK_BF16 ? back_launch<PK_BF16>(a, unit, d.sms, dw, stream)
                                           : back_launch<PK_F16>(a, unit, d.sms, dw, stream);
  return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

}  // extern "C"
