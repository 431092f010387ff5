// pk_logprobs.cu -- log probabilities of given words, entropy and the likeliest words of rows of logits
// (pk_token_logprobs, pk_token_logprobs_backward in include/pk.h).
//
//     lse = ln sum_v exp z_v,  logp = z_label - lse,  H = -sum_v p_v ln p_v  with  p = exp(z - lse)                z [T, V]
//     dz_v = dlogp ([v = label] - p_v) - dH p_v (ln p_v + H)
//
// Bound by the bytes of z. One pass keeps the running maximum m and, relative to it, s = sum e^(z - m) and
// u = sum e^(z - m) (z - m) (moved to a new maximum m' by c = e^(m - m'): s' = c s, u' = c (u + s (m - m'))), so that
// lse = m + ln s and H = ln s - u / s: two terms of one sign, where lse - sum p z would cancel.
//
// The `top` likeliest words: each thread's maximum is of another element, so the top-th largest of the threads' maxima is
// a bound that at least `top` elements reach, and few others do. Only the threads whose maximum reaches it can hold such
// elements; theirs alone are read again (from L2), collected and ranked.
#include <cfloat>

#include "pk_rows.cuh"

namespace pk {

namespace {

using namespace rows;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMaxTop = PK_LOGPROBS_MAX_TOP;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAnywhere = 0x7ffffffe;  // of a maximum: some chunk of the thread's

struct LogprobArgs {
  const void* z;
  int64_t ld;
  const long long* labels;
  int64_t T;
  int V, top;
  float *logp, *lse, *entropy, *top_logp;
  long long* top_idx;
  int* status;
};

// ------------------------------------------------------------------------------------
// the order of logits: a larger key is a larger number, NaN above all, -0 with 0. 16-bit types' values leave the low bits of
// the fp32 pattern all alike; they are shifted out.

template <int DT>
constexpr int kKeyShift = DT == PK_BF16 ? 16 : DT == PK_F16 ? 13 : 0;

template <int DT>
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);
  const uint32_t k = b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
  return (z != z ? 0xFFFFFFFFu : k) >> kKeyShift<DT>;
}
template <int DT>
__device__ __forceinline__ float of_key(uint32_t k) {
  // (the bits that were shifted out are zeros of a positive number and ones, inverted, of a negative one)
  const uint32_t full = k << kKeyShift<DT>;
  const uint32_t b = full & 0x80000000u ? full ^ 0x80000000u : ~(full | ((1u << kKeyShift<DT>) - 1u));
  return __uint_as_float(b);
}

// ------------------------------------------------------------------------------------
// chunks: eight elements whose address is a multiple of 16 bytes, wherever the row begins. The first and last of a row hang
// over its ends; what is not of the row comes as -inf.

struct Row {
  const char* p;  // of element 0
  int off;        // elements between the 16-byte boundary below p and p
  int chunks;
};
template <int DT>
__device__ __forceinline__ Row row_at(const void* z, int64_t first, int V) {
  Row r;
  r.p = static_cast<const char*>(z) + first * Ty<DT>::kBytes;
  r.off = static_cast<int>((reinterpret_cast<uintptr_t>(r.p) & 15) / Ty<DT>::kBytes);
  r.chunks = (V + r.off + 7) / 8;
  return r;
}
template <int DT>
__device__ __forceinline__ bool whole(const Row& r, int chunk, int V) {
  const int c = chunk * 8 - r.off;
  return c >= 0 && c + 8 <= V;
}
template <int DT>
__device__ __forceinline__ void fetch(Raw8<DT>& q, const Row& r, int chunk, int V) {
  const int c = chunk * 8 - r.off;
  if (c >= 0 && c + 8 <= V) {
    q.load(r.p, c, true, 8);
    return;
  }
  constexpr uint32_t kLow = DT == PK_F32 ? 0xFF800000u : DT == PK_BF16 ? 0xFF80FF80u : 0xFC00FC00u;  // -inf
  constexpr int kWords = DT == PK_F32 ? 8 : 4;
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < kWords; ++i) w[i] = kLow;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j >= 0 && c + j < V) {
      if constexpr (DT == PK_F32) {
        w[j] = __ldcg(reinterpret_cast<const unsigned int*>(r.p) + c + j);
      } else {
        const uint32_t x = __ldcg(reinterpret_cast<const unsigned short*>(r.p) + c + j);
        w[j >> 1] = j & 1 ? (w[j >> 1] & 0xFFFFu) | x << 16 : (w[j >> 1] & 0xFFFF0000u) | x;
      }
    }
  q.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
  if constexpr (DT == PK_F32) q.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// ------------------------------------------------------------------------------------
// running maximum and sums

struct Stat {
  float m, s, u;
};
// Differences from the maximum are kept above this where they stand beside an exponential, which is 0 there: 0 times -inf has
// no value. (NaN, and infinity less infinity, come through the exponential.)
constexpr float kFar = -200.0f;
// (the lowest finite number: a row of -inf keeps it, with s = 0, and differences from it are never NaN)
__device__ __forceinline__ Stat nothing() { return {-FLT_MAX, 0.0f, 0.0f}; }

// a moved to the maximum m >= a.m
__device__ __forceinline__ void raise(Stat& a, float m) {
  const float d = a.m - m, c = attn::ex2(d * kLog2e);
  a.u = (a.u + a.s * fmaxf(d, kFar)) * c;
  a.s *= c;
  a.m = m;
}
// The largest of eight values as they were loaded: of 16-bit ones a pair at a time, the pair that holds it.
template <int DT>
__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  if constexpr (DT == PK_BF16)
    asm("max.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  else
    asm("max.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
template <int DT>
__device__ __forceinline__ float top8(const Raw8<DT>& q) {
  if constexpr (DT == PK_F32) {
    float v[8];
    q.get(v);
    return fmaxf(attn::fmax3(v[0], v[1], v[2]), attn::fmax3(attn::fmax3(v[3], v[4], v[5]), v[6], v[7]));
  } else {
    const float2 f = Elem<DT == PK_BF16>::unpack(
        max_pair<DT>(max_pair<DT>(q.q[0].x, q.q[0].y), max_pair<DT>(q.q[0].z, q.q[0].w)));
    return fmaxf(f.x, f.y);
  }
}

// Eight values into the sums, whose maximum m is theirs too.
template <int DT>
__device__ __forceinline__ void accumulate(Stat& a, const Raw8<DT>& q) {
  float v[8];
  q.get(v);
  float2 s = make_float2(0.0f, 0.0f), u = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    add2(v[i], v[i + 1], make_float2(-a.m, -a.m));
    const float2 p = mul2(make_float2(v[i], v[i + 1]), make_float2(kLog2e, kLog2e));
    const float2 e = make_float2(attn::ex2(p.x), attn::ex2(p.y));
    add2(s.x, s.y, e);
    u = fma2(e, make_float2(fmaxf(v[i], kFar), fmaxf(v[i + 1], kFar)), u);
  }
  a.s += s.x + s.y;
  a.u += u.x + u.y;
}

// The same for 16-bit values with fewer instructions: a value that is far below the maximum, -inf among them, is raised as a
// pair to one that is still far enough below it, and the maximum taken off as the value is unpacked. That floor has to
// lie apart from the maximum and above the type's lowest number: far_pair says whether it does (a maximum past -10^38, or
// -50000 of fp16, is taken by `accumulate`).
template <int DT>
__device__ __forceinline__ bool far_pair(float m, uint32_t& pair) {
  const float f = m - 300.0f - 0.125f * fabsf(m);
  pair = Elem<DT == PK_BF16>::pack(f, f);
  return m > (DT == PK_BF16 ? -1.0e38f : -5.0e4f);
}
template <int DT>
__device__ __forceinline__ void accumulate_near(Stat& a, const Raw8<DT>& q, uint32_t far) {
  using E = Elem<DT == PK_BF16>;
  constexpr uint32_t kOnes = DT == PK_BF16 ? 0x3F803F80u : 0x3C003C00u;
  const uint32_t w[4] = {q.q[0].x, q.q[0].y, q.q[0].z, q.q[0].w};
  float2 s = make_float2(a.s, 0.0f), u = make_float2(a.u, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t z = w[i];
    if constexpr (DT == PK_BF16)
      asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(z) : "r"(far));
    else
      asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(z) : "r"(far));
    const float2 d = make_float2(E::fma_lo(z, kOnes, -a.m), E::fma_hi(z, kOnes, -a.m));
    const float2 p = mul2(d, make_float2(kLog2e, kLog2e));
    const float2 e = make_float2(attn::ex2(p.x), attn::ex2(p.y));
    add2(s.x, s.y, e);
    u = fma2(e, d, u);
  }
  a.s = s.x + s.y;
  a.u = u.x + u.y;
}

// The largest of a warp's values (none of them NaN).
__device__ __forceinline__ float warp_max(float v) {
  const int b = __float_as_int(v), k = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
  return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}
// the sums of kN neighbouring lanes, in each of them
template <int kN = 32>
__device__ __forceinline__ Stat warp_join(Stat a) {
  if constexpr (kN == 32) {
    raise(a, warp_max(a.m));
  } else {
    float m = a.m;
#pragma unroll
    for (int o = kN / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    raise(a, m);
  }
#pragma unroll
  for (int o = kN / 2; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.u += __shfl_xor_sync(0xffffffffu, a.u, o);
  }
  return a;
}

// What the row's words come out as. `rest` = ln s.
__device__ __forceinline__ float logp_of(const Stat& a, float rest, float z) {
  return a.s == 0.0f ? -INFINITY : (z - a.m) - rest;
}
template <int DT>
__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t row, const Stat& st, float picked, long long label) {
  const float rest = logf(st.s);
  a.lse[row] = st.m + rest;
  a.entropy[row] = st.s == 0.0f ? 0.0f : rest - st.u / st.s;
  float p = 0.0f;
  if (label >= 0) p = logp_of(st, rest, picked);
  if (label >= a.V) {
    p = __int_as_float(0x7fc00000);
    if (a.status) atomicCAS(a.status, 0, PK_ERR_BAD_LABEL);
  }
  a.logp[row] = p;
}

// ------------------------------------------------------------------------------------
// short rows: a warp each, the row in shared memory, kC chunks a lane

constexpr int kWarpCap = 128;  // candidates of a warp

// The top-th largest of a warp's keys, N a lane and more than `top` in all: from the highest bit in which any two differ, a bit at a
// time until that many are left. kAbsent: keys of 0 are none, and `top` others are there.
template <bool kAbsent, int N>
__device__ __forceinline__ uint32_t warp_nth(const uint32_t (&k)[N], int top) {
  static_assert(32 * N >= kMaxTop, "fewer keys than may be asked for");
  constexpr uint32_t kOne = kAbsent ? 1u : 0u;  // (0 less 1 is no minimum)
  uint32_t hi = k[0], lo = k[0] - kOne;
#pragma unroll
  for (int i = 1; i < N; ++i) {
    hi = max(hi, k[i]);
    lo = min(lo, k[i] - kOne);
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo) + kOne;
  if (hi == lo) return hi;
  int b = 31 - __clz(hi ^ lo);
  uint32_t bound = hi >> b >> 1 << b << 1;
#pragma unroll 1
  for (; b >= 0; --b) {
    const uint32_t probe = bound | 1u << b;
    int n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) n += k[i] >= probe ? 1 : 0;
    n = __reduce_add_sync(0xffffffffu, n);
    if (n >= top) bound = probe;
    if (n == top) {
      // (the smallest of them: elements between it and the probe would only be more candidates)
      uint32_t least = 0xFFFFFFFFu;
#pragma unroll
      for (int i = 0; i < N; ++i) least = k[i] >= probe && k[i] < least ? k[i] : least;
      return __reduce_min_sync(0xffffffffu, least);
    }
  }
  return bound;
}

// A candidate as one number, larger for one that stands before: the key, then the index downwards.
__device__ __forceinline__ uint64_t packed(uint32_t key, int idx) { return static_cast<uint64_t>(key) << 32 | (0xFFFFFFFFu - idx); }

// 32 kR numbers of a warp in descending order, number r 32 + lane in v[r]: a bitonic network, through shuffles within 32.
template <int kR>
__device__ __forceinline__ void warp_sort(uint64_t (&v)[kR], int lane) {
#pragma unroll
  for (int k = 2; k <= 32 * kR; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2) {
      if (j >= 32) {
#pragma unroll
        for (int r = 0; r < kR; ++r)
          if (!(r & (j / 32))) {
            const int o = r | (j / 32);
            const bool down = !((r * 32) & k);
            const uint64_t hi = v[r] > v[o] ? v[r] : v[o], lo = v[r] > v[o] ? v[o] : v[r];
            v[r] = down ? hi : lo;
            v[o] = down ? lo : hi;
          }
      } else {
#pragma unroll
        for (int r = 0; r < kR; ++r) {
          const uint64_t u = __shfl_xor_sync(0xffffffffu, v[r], j);
          const bool larger = !((r * 32 + lane) & k) == !(lane & j);
          v[r] = (v[r] > u) == larger ? v[r] : u;
        }
      }
    }
}
template <int kR, class Emit>
__device__ __forceinline__ void sort_emit(const uint64_t* cand, int n, int top, int lane, const Emit& emit) {
  uint64_t v[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) v[r] = r * 32 + lane < n ? cand[r * 32 + lane] : 0;
  warp_sort<kR>(v, lane);
#pragma unroll
  for (int r = 0; r < kR; ++r)
    if (r * 32 + lane < top) emit(r * 32 + lane, static_cast<uint32_t>(v[r] >> 32), static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(v[r])));
}
// The first `top` <= 64 of n <= 128 candidates handed to `emit` (place, key, index), by a warp.
template <class Emit>
__device__ __forceinline__ void first_of(const uint64_t* cand, int n, int top, int lane, const Emit& emit) {
  if (n <= 32)
    sort_emit<1>(cand, n, top, lane, emit);
  else if (n <= 64)
    sort_emit<2>(cand, n, top, lane, emit);
  else
    sort_emit<4>(cand, n, top, lane, emit);
}

// Eight values against a bound: bit j where v[j] is above it, or at it too where `at` says so. NaN is above.
__device__ __forceinline__ uint32_t reach(const float (&v)[8], float bound, bool at) {
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) bits |= (at ? !(v[j] < bound) : !(v[j] <= bound)) ? 1u << j : 0u;
  return bits;
}
// the bits of the elements from `first` on that are of the row
__device__ __forceinline__ uint32_t row_bits(int first, int V) {
  const int lo = first < 0 ? -first : 0, hi = V - first < 8 ? V - first : 8;
  return hi <= lo ? 0u : (0xFFu >> (8 - hi)) & (0xFFu << lo);
}

template <int DT, int kC>
constexpr int kShortBytes = kWarps * kC * 32 * 8 * Ty<DT>::kBytes;

// kFine: maxima that a chunk has, of all its elements or of pairs of them, where the row has few chunks.
template <int DT, int kC, int kFine>
__global__ void __launch_bounds__(kThreads, 5) pk_logprobs_short_kernel(const __grid_constant__ LogprobArgs a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t cand[kWarps][kWarpCap];
  __shared__ uint16_t noted[kWarps][kC * 32];  // chunks that hold candidates
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  constexpr int kPieces = Ty<DT>::kBytes / 2;  // of 16 bytes a chunk
  uint4* const rows = reinterpret_cast<uint4*>(smem) + w * (kC * 32 * kPieces);
  uint4* const mine = rows + lane;
  const auto chunk_of = [&](int i, int owner) {
    Raw8<DT> q;
#pragma unroll
    for (int p = 0; p < kPieces; ++p) q.q[p] = rows[(i * kPieces + p) * 32 + owner];
    return q;
  };
  const auto chunk_at = [&](int i) { return chunk_of(i, lane); };
  griddep_wait();
  for (int64_t row = blockIdx.x * static_cast<int64_t>(kWarps) + w; row < a.T; row += static_cast<int64_t>(gridDim.x) * kWarps) {
    const Row r = row_at<DT>(a.z, row * a.ld, a.V);
    const int n_mine = (r.chunks - lane + 31) / 32;  // chunks of this lane
#pragma unroll 4
    for (int i = 0; i < n_mine; ++i) {
      const int chunk = i * 32 + lane;
      if (whole<DT>(r, chunk, a.V)) {
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(mine + (i * kPieces + p) * 32)),
                       "l"(r.p + (static_cast<int64_t>(chunk) * 8 - r.off) * Ty<DT>::kBytes + 16 * p)
                       : "memory");
      } else {
        Raw8<DT> q;
        fetch<DT>(q, r, chunk, a.V);
#pragma unroll
        for (int p = 0; p < kPieces; ++p) mine[(i * kPieces + p) * 32] = q.q[p];
      }
    }
    const long long label = __ldcg(a.labels + row);
    float picked = 0.0f;
    asm volatile("cp.async.wait_all;" ::: "memory");
    // the maxima, each of another element
    uint32_t key[kC * kFine];
    Stat st = nothing();
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const bool here = i < n_mine;
      Raw8<DT> q;
      float m = -INFINITY;
      if (here) {
        q = chunk_at(i);
        m = top8<DT>(q);
        st.m = fmaxf(st.m, m);
      }
      if constexpr (kFine == 1) {
        key[i] = here ? key_of<DT>(m) : 0u;
      } else {
        float v[8];
        q.get(v);
        const int c = (i * 32 + lane) * 8 - r.off;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool some = here && c + 2 * j + 1 >= 0 && c + 2 * j < a.V;
          key[4 * i + j] = some ? key_of<DT>(fmaxf(v[2 * j], v[2 * j + 1])) : 0u;
        }
      }
    }
    raise(st, warp_max(st.m));
    uint32_t far = 0;
    bool near = false;
    if constexpr (DT != PK_F32) near = far_pair<DT>(st.m, far);
#pragma unroll 1
    for (int i = 0; i < n_mine; ++i) {
      if constexpr (DT != PK_F32) {
        if (near) {
          accumulate_near<DT>(st, chunk_at(i), far);
          continue;
        }
      }
      accumulate<DT>(st, chunk_at(i));
    }
    st = warp_join(st);
    if (label >= 0 && label < a.V) picked = Ty<DT>::get(r.p, label);
    if (lane == 0) write_row<DT>(a, row, st, picked, label);
    if (a.top == 0) continue;

    uint64_t* out = cand[w];
    const auto inside = [&](int e) { return e >= 0 && e < a.V; };
    __syncwarp();  // (the row before has been written out)
    int n = kWarpCap + 1;
    if (st.s == st.s) {
      // chunks whose maximum reaches the bound are noted, then looked into a lane each
      const float bound = of_key<DT>(warp_nth<kFine == 1>(key, a.top));
      int have = 0;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        const bool is = i < n_mine && !(top8<DT>(chunk_at(i)) < bound);  // (no bound: NaN)
        const uint32_t votes = __ballot_sync(0xffffffffu, is);
        if (is) noted[w][have + __popc(votes & ((1u << lane) - 1u))] = static_cast<uint16_t>(i * 32 + lane);
        have += __popc(votes);
      }
      __syncwarp();
      n = 0;
#pragma unroll 1
      for (int k = 0; k < have && n <= kWarpCap; k += 32) {
        float v[8];
        uint32_t bits = 0;
        int c = 0;
        if (k + lane < have) {
          const int chunk = noted[w][k + lane];
          chunk_of(chunk >> 5, chunk & 31).get(v);
          c = chunk * 8 - r.off;
          bits = reach(v, bound, true) & row_bits(c, a.V);
        }
        int upto = __popc(bits);
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
          const int u = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += u;
        }
        int at = n + upto - __popc(bits);
        n += __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (bits >> j & 1u) {
            if (at < kWarpCap) out[at] = packed(key_of<DT>(v[j]), c + j);
            ++at;
          }
      }
      __syncwarp();
    }
    if (n > kWarpCap) {
      // many equal ones, or a NaN, which no maximum shows: the top-th largest of all elements, those above it, and of those
      // equal to it the first
      uint32_t bound = 0;
#pragma unroll 1
      for (int b = 31 - kKeyShift<DT>; b >= 0; --b) {
        const uint32_t probe = bound | 1u << b;
        int m = 0;
#pragma unroll 1
        for (int i = 0; i < n_mine; ++i) {
          float v[8];
          chunk_at(i).get(v);
          const int c = (i * 32 + lane) * 8 - r.off;
#pragma unroll
          for (int j = 0; j < 8; ++j) m += key_of<DT>(v[j]) >= probe && inside(c + j) ? 1 : 0;
        }
        if (static_cast<int>(__reduce_add_sync(0xffffffffu, m)) >= a.top) bound = probe;
      }
      __syncwarp();
      int taken = 0;
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass)
#pragma unroll 1
        for (int i = 0; i * 32 < r.chunks; ++i) {
          // this lane's elements of the kind, and where they stand among the warp's
          const int c = (i * 32 + lane) * 8 - r.off;
          float v[8];
          uint32_t bits = 0;
          if (i < n_mine) {
            chunk_at(i).get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t k = key_of<DT>(v[j]);
              bits |= inside(c + j) && (pass == 0 ? k > bound : k == bound) ? 1u << j : 0u;
            }
          }
          int upto = __popc(bits);
#pragma unroll
          for (int o = 1; o < 32; o *= 2) {
            const int u = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += u;
          }
          int at = taken + upto - __popc(bits);
          taken += __shfl_sync(0xffffffffu, upto, 31);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (bits >> j & 1u) {
              if (at < a.top) out[at] = packed(key_of<DT>(v[j]), c + j);
              ++at;
            }
        }
      __syncwarp();
      n = a.top;
    }
    const float rest = logf(st.s);
    first_of(out, n, a.top, lane, [&](int i, uint32_t k, int e) {
      a.top_logp[row * a.top + i] = logp_of(st, rest, of_key<DT>(k));
      a.top_idx[row * a.top + i] = e;
    });
  }
}

// ------------------------------------------------------------------------------------
// longer rows: a block, or a cluster of blocks where there are few rows

// candidates that are kept
template <int kT>
constexpr int kCap = kT >= 256 ? 1024 : 512;

// what the threads find as they go over a slice
template <int kT>
struct Found {
  Stat stat[kT / 32];
  uint32_t maxima[kT];
  int chunk[kT];  // where each thread's maximum stands
};
constexpr int kLook = 2;  // chunks that a thread has in flight in the search
template <int kT>
struct Search {
  int list[kT];           // threads whose elements are candidates
  int hits[kT / 32][32 + 32 * kLook];  // chunks that hold some, a warp's own
  int listed, found;
  uint32_t bound;
  int bound_chunk;
  uint64_t cand[kCap<kT>];
  uint64_t few[128];  // of them those that may be among the likeliest; of a slice: its likeliest
  uint64_t pick[kT / 32];
};

// Where the block's part of a row lies: chunks [c0, c1), of which those of [w0, w1) are whole. Thread t takes w0 + t, w0 + t + kT
// and so on; a chunk that hangs over the row's first or last word is thread 0's or 1's besides.
struct Slice {
  Row r;
  int c0, c1, w0, w1;
};
template <int DT>
__device__ __forceinline__ Slice slice_at(const LogprobArgs& a, int64_t row, int part, int parts) {
  Slice s;
  s.r = row_at<DT>(a.z, row * a.ld, a.V);
  const int per = (s.r.chunks + parts - 1) / parts;
  s.c0 = part * per;
  s.c1 = min(s.c0 + per, s.r.chunks);
  s.w0 = s.c0 + (s.c0 == 0 && s.r.off > 0 ? 1 : 0);
  s.w1 = s.c1 - (s.c1 == s.r.chunks && !whole<DT>(s.r, s.c1 - 1, a.V) ? 1 : 0);
  return s;
}
// the chunk that hangs over which thread t has, or -1
__device__ __forceinline__ int edge_of(const Slice& s, int t) {
  return t == 0 ? (s.w0 > s.c0 ? s.c0 : -1) : t == 1 ? (s.w1 < s.c1 ? s.w1 : -1) : -1;
}

// The candidates of the listed threads' chunks into sh.cand: elements above `bound`, or at it and in a chunk up to `last`.
// Their count (which may be past what is kept) is returned in every thread. `clean`: there is no NaN, which a maximum passes over.
// Few chunks hold one: those are noted first and then looked into a lane each, not wherever one of 32 lanes has one.
template <int DT, int kT>
__device__ __forceinline__ int collect(Search<kT>& sh, const Slice& s, int V, float bound, int last, bool clean) {
  const int lane = threadIdx.x & 31;
  int* const hits = sh.hits[threadIdx.x >> 5];
  int have = 0;  // chunks in `hits`
  const auto keep = [&](bool is, int c) {
    const uint32_t votes = __ballot_sync(0xffffffffu, is);
    if (is) hits[have + __popc(votes & ((1u << lane) - 1u))] = c;
    have += __popc(votes);
  };
  // the elements of the first n <= 32 of them, a chunk a lane
  const auto drain = [&](int n) {
    __syncwarp();
    if (lane < n) {
      const int c = hits[lane], first = c * 8 - s.r.off;
      Raw8<DT> q;
      fetch<DT>(q, s.r, c, V);
      float v[8];
      q.get(v);
      const uint32_t bits = reach(v, bound, c <= last) & row_bits(first, V);
      if (bits != 0) {
        int at = atomicAdd(&sh.found, __popc(bits));
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (bits >> j & 1u) {
            if (at < kCap<kT>) sh.cand[at] = packed(key_of<DT>(v[j]), first + j);
            ++at;
          }
      }
    }
    have -= n;
    __syncwarp();
    for (int i = 0; i < have; i += 32) {  // (those behind, to the front)
      const int more = i + lane < have ? hits[n + i + lane] : 0;
      __syncwarp();
      if (i + lane < have) hits[i + lane] = more;
      __syncwarp();
    }
  };
  if (threadIdx.x < 32) {
    const int edge = edge_of(s, lane);
    keep(edge >= 0, edge);
  }
  // chunk j of listed thread k is w0 + list[k] + j kT; this thread's are kT apart in the list of (k, j)
  const int each = (s.w1 - s.w0 + kT - 1) / kT, dk = kT / each, dj = kT - dk * each, n = sh.listed;
  int k = threadIdx.x / each, j = threadIdx.x - k * each;
#pragma unroll 1
  for (int i0 = threadIdx.x & ~31; i0 < n * each; i0 += kLook * kT) {
    Raw8<DT> q[kLook];
    int at[kLook];
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
      at[i] = k < n ? s.w0 + sh.list[k] + j * kT : s.w1;
      if (at[i] < s.w1) q[i].load(s.r.p, at[i] * 8 - s.r.off, true, 8);
      k += dk;
      j += dj;
      if (j >= each) {
        j -= each;
        ++k;
      }
    }
#pragma unroll
    for (int i = 0; i < kLook; ++i) {
      bool is = at[i] < s.w1;
      if (is && clean) is = !(top8<DT>(q[i]) < bound);
      keep(is, at[i]);
    }
#pragma unroll 1
    while (have >= 32 || (have > 0 && i0 + kLook * kT >= n * each)) drain(min(have, 32));
    if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&sh.found) > kCap<kT>)) break;  // (more than are kept: enough seen)
  }
  __syncthreads();
  return sh.found;
}

// The first `top` of sh.cand[0 .. n) to `emit`, by a warp. Of many, first the top-th: no two are equal, so exactly `top` reach it.
template <int kT, class Emit>
__device__ __forceinline__ void finish(Search<kT>& sh, int n, int top, const Emit& emit) {
  const int lane = threadIdx.x & 31;
  if (n <= 128) {
    first_of(sh.cand, n, top, lane, emit);
    return;
  }
  uint64_t bound = 0;
#pragma unroll 1
  for (int b = 63; b >= 0; --b) {
    const uint64_t probe = bound | uint64_t(1) << b;
    int m = 0;
#pragma unroll 4
    for (int i = lane; i < n; i += 32) m += sh.cand[i] >= probe ? 1 : 0;
    m = __reduce_add_sync(0xffffffffu, m);
    if (m >= top) bound = probe;
    if (m == top) break;
  }
  int have = 0;
  for (int i = 0; i < n; i += 32) {
    const bool is = i + lane < n && sh.cand[i + lane] >= bound;
    const uint32_t votes = __ballot_sync(0xffffffffu, is);
    if (is) sh.few[have + __popc(votes & ((1u << lane) - 1u))] = sh.cand[i + lane];
    have += __popc(votes);
  }
  __syncwarp();
  first_of(sh.few, have, top, lane, emit);
}

// The slice's `top` likeliest words to `emit`. Each thread has a chunk of the slice and its maximum in `fd`; the block is synchronized.
template <int DT, int kT, class Emit>
__device__ __forceinline__ void slice_top(Search<kT>& sh, const Found<kT>& fd, const Slice& s, int V, int top, bool clean, const Emit& emit) {
  const int lane = threadIdx.x & 31;
  // a warp names the threads whose elements may be among them
  const auto name = [&](uint32_t bound, int last, const auto& may) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kT / 32; ++i) {
      const bool is = may(i);
      const uint32_t votes = __ballot_sync(0xffffffffu, is);
      if (is) sh.list[n + __popc(votes & ((1u << lane) - 1u))] = i * 32 + lane;
      n += __popc(votes);
    }
    if (lane == 0) {
      sh.listed = n;
      sh.found = 0;
      sh.bound = bound;
      sh.bound_chunk = last;
    }
  };
  if (threadIdx.x < 32) {
    uint32_t k[kT / 32];
#pragma unroll
    for (int i = 0; i < kT / 32; ++i) k[i] = fd.maxima[i * 32 + lane];
    const uint32_t nth = warp_nth<false>(k, top);
    name(nth, 0x7fffffff, [&](int i) { return k[i] >= nth; });
  }
  __syncthreads();
  const uint32_t bound = sh.bound;
  int n = collect<DT, kT>(sh, s, V, of_key<DT>(bound), 0x7fffffff, clean);
  if (n > kCap<kT>) {
    // many equal ones (a masked vocabulary): of those at the bound only the first chunks', up to the one that completes `top`
    __syncthreads();
    if (threadIdx.x < 32) {
      int at = 0;
#pragma unroll 1
      for (int b = 17; b >= 0; --b) {  // the largest chunk before which there are still fewer than `top`
        const int probe = at | 1 << b;
        int m = 0;
        for (int i = lane; i < kT; i += 32) m += fd.maxima[i] > bound || (fd.maxima[i] == bound && fd.chunk[i] < probe) ? 1 : 0;
        if (__reduce_add_sync(0xffffffffu, m) < top) at = probe;
      }
      // (of those whose maximum is the bound only the ones that stand no later)
      name(bound, at, [&](int i) {
        const uint32_t k = fd.maxima[i * 32 + lane];
        const int c = fd.chunk[i * 32 + lane];
        return k > bound || (k == bound && (c <= at || c == kAnywhere));
      });
    }
    __syncthreads();
    n = collect<DT, kT>(sh, s, V, of_key<DT>(bound), sh.bound_chunk, clean);
  }
  if (n <= kCap<kT>) {
    if (threadIdx.x < 32) finish<kT>(sh, n, top, emit);
    return;
  }
  // many large ones in few threads: one maximum after another, each a pass over the slice (64 likeliest of 400 x 65536 fp32, ten thousand
  // candidates a row: 2026 us, 27 of random rows)
  uint64_t done = ~uint64_t(0);
  for (int i = 0; i < top; ++i) {
    uint64_t best = 0;
    for (int c = s.c0 + threadIdx.x; c < s.c1; c += kT) {
      Raw8<DT> q;
      fetch<DT>(q, s.r, c, V);
      float v[8];
      q.get(v);
      const uint32_t bits = row_bits(c * 8 - s.r.off, V);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint64_t x = packed(key_of<DT>(v[j]), c * 8 - s.r.off + j);
        if ((bits >> j & 1u) && x < done && x > best) best = x;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const uint64_t u = __shfl_xor_sync(0xffffffffu, best, o);
      best = u > best ? u : best;
    }
    if (lane == 0) sh.pick[threadIdx.x >> 5] = best;
    __syncthreads();
    done = sh.pick[0];
    for (int k = 1; k < kT / 32; ++k) done = sh.pick[k] > done ? sh.pick[k] : done;
    if (threadIdx.x == 0) emit(i, static_cast<uint32_t>(done >> 32), static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(done)));
    __syncthreads();
  }
}

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) { return gemm::mapa(smem_u32(p), rank); }
__device__ __forceinline__ uint32_t ld_remote(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kBatch = 4;  // chunks that a thread has in flight

// One of kT threads over its chunks of a slice: its sums, and the chunk `at` where its maximum stands.
template <int DT, int kT>
__device__ __forceinline__ Stat go_over(const Slice& sl, int V, int& at) {
  const int t = threadIdx.x;
  Stat st = nothing();
  at = sl.w0 + t;
  // `kN` chunks from c on, kT apart
  const auto take = [&](const auto& q, int c) {
    constexpr int kN = sizeof(q) / sizeof(Raw8<DT>);
    float top[kN], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      top[i] = top8<DT>(q[i]);
      m = fmaxf(m, top[i]);
    }
    // (no sum so far: the lowest number, where the maximum starts, is then news too)
    if (m > st.m || (st.s == 0.0f && m == st.m)) {
#pragma unroll
      for (int i = kN - 1; i >= 0; --i) at = top[i] == m ? c + i * kT : at;
    }
    raise(st, fmaxf(st.m, m));
    if constexpr (DT != PK_F32) {
      uint32_t far;
      if (far_pair<DT>(st.m, far)) {
#pragma unroll
        for (int i = 0; i < kN; ++i) accumulate_near<DT>(st, q[i], far);
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) accumulate<DT>(st, q[i]);
  };
  int c = sl.w0 + t;
#pragma unroll 1
  for (; c + (kBatch - 1) * kT < sl.w1; c += kBatch * kT) {
    Raw8<DT> q[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) q[i].load(sl.r.p, (c + i * kT) * 8 - sl.r.off, true, 8);
    take(q, c);
  }
#pragma unroll 1
  for (; c < sl.w1; c += kT) {
    Raw8<DT> q[1];
    q[0].load(sl.r.p, c * 8 - sl.r.off, true, 8);
    take(q, c);
  }
  const int edge = edge_of(sl, t);
  if (edge >= 0) {
    Raw8<DT> q[1];
    fetch<DT>(q[0], sl.r, edge, V);
    take(q, edge);
  }
  return st;
}
template <int DT, int kT>
__device__ __forceinline__ void leave(Found<kT>& fd, const Stat& mine, const Stat& warps, int at) {
  // (a sum without a value: one of the thread's elements is infinite or NaN, so at least infinity, in a chunk unknown. No sum
  // at all: every element is -inf, the first of them in its first chunk)
  const bool nan = mine.s != mine.s;
  fd.maxima[threadIdx.x] = key_of<DT>(nan ? INFINITY : mine.s == 0.0f ? -INFINITY : mine.m);
  fd.chunk[threadIdx.x] = nan ? kAnywhere : at;
  if ((threadIdx.x & 31) == 0) fd.stat[threadIdx.x >> 5] = warps;
}
template <int kT>
__device__ __forceinline__ Stat joined(const Found<kT>& fd) {
  return warp_join<kT / 32>(fd.stat[threadIdx.x % (kT / 32)]);
}

// Bound by the bytes of z where rows are long, with 1280 threads an SM (1536 in smaller blocks, 1024 of fp32) and four loads each in flight, as far as
// instructions go (some 50 for eight 16-bit values); by the way from a row's last load to its last output where they are not.
// 8192 x 50000 bf16: 126 us without likeliest words (0.97 of the copy rate), 163 with 16. One row of 128000 words, 16 likeliest: 8.0.
// Not kept: four loads ahead in shared memory instead of registers (210 us: the copies' own instructions cost more than they hide)
// or in registers, with fewer blocks (166); the next row's words fetched into L2 during the search (171, when the search took
// longer); one or two warps more a block that search while the others go over the next row (273 and 197: a few hundred instructions
// in one chain, among 32 warps that ask for the same issue slots).
template <int DT, int kT>
__global__ void __launch_bounds__(kT, (DT == PK_F32 ? 1024 : kT == 256 ? 1280 : 1536) / kT) pk_logprobs_kernel(const __grid_constant__ LogprobArgs a) {
  __shared__ Found<kT> found;
  __shared__ Search<kT> search;
  const int64_t row = blockIdx.x;
  griddep_wait();
  const Slice sl = slice_at<DT>(a, row, 0, 1);
  long long label = -1;
  float picked = 0.0f;
  if (threadIdx.x == 0) label = __ldcg(a.labels + row);
  int at;
  const Stat mine = go_over<DT, kT>(sl, a.V, at);
  if (label >= 0 && label < a.V) picked = Ty<DT>::get(sl.r.p, label);  // (asked for here, used below)
  leave<DT, kT>(found, mine, warp_join(mine), at);
  __syncthreads();
  const Stat st = joined(found);
  if (threadIdx.x == 0) write_row<DT>(a, row, st, picked, label);
  if (a.top == 0) return;
  const float rest = logf(st.s);
  slice_top<DT, kT>(search, found, sl, a.V, a.top, st.s == st.s, [&](int i, uint32_t k, int e) {
    a.top_logp[row * a.top + i] = logp_of(st, rest, of_key<DT>(k));
    a.top_idx[row * a.top + i] = e;
  });
}

// few rows: a cluster of blocks a row, each its part of it, and the first joins what they find
template <int DT, int kT>
__global__ void __launch_bounds__(kT, (DT == PK_F32 ? 1024 : 1280) / kT) pk_logprobs_cluster_kernel(const __grid_constant__ LogprobArgs a, int parts) {
  __shared__ Found<kT> found;
  __shared__ Search<kT> search;
  __shared__ Stat whole;  // the slice's
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int part = static_cast<int>(gemm::cluster_rank());
  const int64_t row = blockIdx.x / parts;
  griddep_wait();
  const Slice sl = slice_at<DT>(a, row, part, parts);
  long long label = -1;
  float picked = 0.0f;
  if (threadIdx.x == 0 && part == 0) label = __ldcg(a.labels + row);
  int at;
  const Stat mine = go_over<DT, kT>(sl, a.V, at);
  if (label >= 0 && label < a.V) picked = Ty<DT>::get(sl.r.p, label);  // (asked for here, used below)
  leave<DT, kT>(found, mine, warp_join(mine), at);
  __syncthreads();
  Stat st = joined(found);
  if (a.top > 0)
    slice_top<DT, kT>(search, found, sl, a.V, a.top, st.s == st.s, [&](int i, uint32_t k, int e) { search.few[i] = packed(k, e); });
  if (threadIdx.x == 0) whole = st;
  gemm::cluster_sync();
  if (part == 0) {
    // the slices' sums and likeliest words, a warp a slice
    st = nothing();
    if (lane < parts) {
      const uint32_t from = remote(&whole, lane);
      st = {__uint_as_float(ld_remote(from)), __uint_as_float(ld_remote(from + 4)), __uint_as_float(ld_remote(from + 8))};
    }
    for (int p = w; p < parts && a.top > 0; p += kT / 32) {
      const uint32_t from = remote(&search.few[0], p);
      for (int i = lane; i < a.top; i += 32)
        search.cand[p * a.top + i] = ld_remote(from + 8 * i) | static_cast<uint64_t>(ld_remote(from + 8 * i + 4)) << 32;
    }
    st = warp_join(st);
    if (threadIdx.x == 0) write_row<DT>(a, row, st, picked, label);
    __syncthreads();
    const float rest = logf(st.s);
    if (a.top > 0 && w == 0)
      finish<kT>(search, parts * a.top, a.top, [&](int i, uint32_t k, int e) {
        a.top_logp[row * a.top + i] = logp_of(st, rest, of_key<DT>(k));
        a.top_idx[row * a.top + i] = e;
      });
  }
  gemm::cluster_sync();  // (no block leaves while its memory is read)
}

constexpr int kShort = 704;     // words of a row of a warp
constexpr int kMedium = 2032;   // where there are many: eight chunks a lane, less one that hangs over
constexpr int kMiddle = 32768;  // words of a row of a block of 128 threads, and four times those of 64

// Blocks a row: one where the rows fill the SMs, up to eight where they do not, none with fewer than 4096 words.
int parts_of(int64_t T, int V, int sms) {
  int parts = 1;
  while (parts < 8 && T * parts * 2 <= 2 * sms && V / (parts * 2) >= 4096) parts *= 2;
  return parts;
}

template <int DT, int kC, int kFine>
cudaError_t short_launch(const LogprobArgs& a, int sms, cudaStream_t stream) {
  const int64_t blocks = (a.T + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * 8;
  Launch l(blocks < most ? blocks : most, kThreads, stream);
  l.cfg.dynamicSmemBytes = kShortBytes<DT, kC>;
  return cudaLaunchKernelEx(&l.cfg, pk_logprobs_short_kernel<DT, kC, kFine>, a);
}

template <int DT, int kT>
cudaError_t rows_launch(const LogprobArgs& a, cudaStream_t stream) {
  Launch l(a.T, kT, stream);
  return cudaLaunchKernelEx(&l.cfg, pk_logprobs_kernel<DT, kT>, a);
}

template <int DT>
cudaError_t logprobs_launch(const LogprobArgs& a, int sms, cudaStream_t stream) {
  // a warp's row: up to three chunks a lane, with at least two maxima for each word that is asked for; in 16 bits, where there are rows
  // for every warp, up to eight. (16 likeliest of 65536 rows: of 700 words 97 us, 142 with the maxima of pairs; of 1500 136, 189 a
  // block of 64 a row; of 2500 x 2000 10.6 and 10.2, of 300 x 2000 7.6 and 5.8. Of 3000 words, 16 chunks a lane, 250 and 189.)
  const bool enough = a.V / 8 >= 2 * a.top;
  if (a.V <= kShort) return enough ? short_launch<DT, 3, 1>(a, sms, stream) : short_launch<DT, 3, 4>(a, sms, stream);
  if constexpr (DT != PK_F32)
    if (a.V <= kMedium && a.T > 16 * sms) return short_launch<DT, 8, 1>(a, sms, stream);
  const int parts = parts_of(a.T, a.V, sms);
  if (parts == 1) {
    // what a row takes from its last load to its last output hardly depends on its length: more and smaller blocks for
    // shorter ones, where that leaves at least twice as many maxima as are asked for (64 of 64 bound little: 63880 rows of
    // 4588 words took a block of 64 1425 us, one of 128 389) and every thread a chunk. 16 likeliest in bf16: of 65536 x 4300 233 us
    // and 278 (blocks of 64 and 128), 16384 x 16384 151 and 115, 16384 x 30000 198 and 244 (128 and 256), 8192 x 50000 185 and 163.
    if (a.V <= kMiddle / 4 && (a.top <= 32 || a.V < 1040)) return rows_launch<DT, 64>(a, stream);
    if (a.V <= kMiddle) return rows_launch<DT, 128>(a, stream);
    return rows_launch<DT, 256>(a, stream);
  }
  Launch l(a.T * parts, 256, stream);
  cudaLaunchAttribute at[2] = {l.at[0], {}};
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = parts;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  l.cfg.attrs = at;
  l.cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&l.cfg, pk_logprobs_cluster_kernel<DT, 256>, a, parts);
}

// ------------------------------------------------------------------------------------
// backward: a thread takes chunks of eight, wherever in the matrix

struct LogprobBackArgs {
  const void* z;
  void* dz;
  int64_t ld, lddz;
  const long long* labels;
  const float *lse, *entropy, *dlogp, *dentropy;
  int64_t row0;
  uint32_t total;  // chunks of this launch, below 2^31
  int V;
  FastDiv chunks;  // of a row
  int same;        // rows of z and dz begin at the same place within 16 bytes
};

constexpr int kBackBatch = 4;

template <int DT, int kB>
__global__ void __launch_bounds__(kThreads) pk_logprobs_backward_kernel(const __grid_constant__ LogprobBackArgs a) {
  griddep_wait();
  const uint32_t i0 = blockIdx.x * (kThreads * kB) + threadIdx.x;
  Raw8<DT> q[kB];
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const uint32_t i = i0 + b * kThreads;
    if (i < a.total) {
      const uint32_t rr = a.chunks.div(i);
      const Row r = row_at<DT>(a.z, (a.row0 + rr) * a.ld, a.V);
      fetch<DT>(q[b], r, static_cast<int>(i - rr * a.chunks.d), a.V);
    }
  }
#pragma unroll
  for (int b = 0; b < kB; ++b) {
    const uint32_t i = i0 + b * kThreads;
    if (i >= a.total) break;
    const uint32_t rr = a.chunks.div(i);
    const int64_t row = a.row0 + rr;
    const Row r = row_at<DT>(a.z, row * a.ld, a.V);
    const int c = static_cast<int>(i - rr * a.chunks.d) * 8 - r.off;
    if (c >= a.V) continue;
    const long long label = a.labels[row];
    const float g = label >= 0 && label < a.V ? a.dlogp[row] : 0.0f;
    float lse = a.lse[row], h = 0.0f, H = 0.0f;
    lse = lse == -INFINITY ? 0.0f : lse;  // a row of -inf: probabilities of zero
    if (a.dentropy) {
      h = a.dentropy[row];
      H = a.entropy[row];
    }
    float v[8];
    q[b].get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float l = v[j] - lse, p = attn::ex2(l * kLog2e);
      v[j] = -p * fmaf(h, fmaxf(l, -200.0f) + H, g);
    }
    if (label >= c && label < c + 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = label == c + j ? v[j] + g : v[j];
    }
    if (a.same && c >= 0 && c + 8 <= a.V) {
      store8<DT>(a.dz, row * a.lddz + c, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j >= 0 && c + j < a.V) Ty<DT>::put(a.dz, row * a.lddz + c + j, v[j]);
    }
  }
}

template <int DT>
cudaError_t back_launch(const LogprobBackArgs& a, int sms, cudaStream_t stream) {
  const int batch = a.total >= static_cast<uint32_t>(2 * sms * kThreads * kBackBatch) ? kBackBatch : 1;
  Launch l((a.total + kThreads * batch - 1) / (kThreads * batch), kThreads, stream);
  return batch == 1 ? cudaLaunchKernelEx(&l.cfg, pk_logprobs_backward_kernel<DT, 1>, a)
                    : cudaLaunchKernelEx(&l.cfg, pk_logprobs_backward_kernel<DT, kBackBatch>, a);
}

bool sizes_ok(int dtype, int64_t T, int V, int64_t ld) {
  return dtype_ok(dtype) && T >= 0 && T <= PK_ROWS_MAX_T && V >= 1 && V <= PK_ROWS_MAX_DIM && ld >= V;
}

}  // namespace

}  // namespace pk

extern "C" {

int pk_token_logprobs(int dtype, const void* logits, int64_t ld, const int64_t* labels, int64_t T, int V, int top, float* logp,
                      float* lse, float* entropy, float* top_logp, int64_t* top_idx, int* status, struct CUstream_st* stream) {
  using namespace pk;
  if (!sizes_ok(dtype, T, V, ld) || top < 0 || top > kMaxTop || top > V) return PK_ERR_ARG;
  if (T > 0 && (!logits || !labels || !logp || !lse || !entropy || (top > 0 && (!top_logp || !top_idx)))) return PK_ERR_ARG;
  if (!rows::aligned_to(logits, rows::elem_bytes(dtype)) || !rows::aligned_to(labels, 8) || !rows::aligned_to(logp, 4) ||
      !rows::aligned_to(lse, 4) || !rows::aligned_to(entropy, 4) || !rows::aligned_to(top_logp, 4) ||
      !rows::aligned_to(top_idx, 8) || !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) return status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess ? PK_ERR_CUDA : PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  LogprobArgs a = {};
  a.z = logits;
  a.ld = ld;
  a.labels = reinterpret_cast<const long long*>(labels);
  a.T = T;
  a.V = V;
  a.top = top;
  a.logp = logp;
  a.lse = lse;
  a.entropy = entropy;
  a.top_logp = top_logp;
  a.top_idx = reinterpret_cast<long long*>(top_idx);
  a.status = status ? status : rows::stream_status(d, stream);
  const cudaError_t r = dtype == PK_F32    ? logprobs_launch<PK_F32>(a, d.sms, stream)
                        : dtype == PK_BF16 ? logprobs_launch<PK_BF16>(a, d.sms, stream)
                                           : logprobs_launch<PK_F16>(a, d.sms, stream);
  return r == cudaSuccess ? PK_OK : PK_ERR_CUDA;
}

int pk_token_logprobs_backward(int dtype, const void* logits, int64_t ld, const int64_t* labels, const float* lse,
                               const float* entropy, const float* dlogp, const float* dentropy, int64_t T, int V, void* dlogits,
                               int64_t lddz, struct CUstream_st* stream) {
  using namespace pk;
  if (!sizes_ok(dtype, T, V, ld) || lddz < V) return PK_ERR_ARG;
  if (T > 0 && (!logits || !labels || !lse || !dlogp || !dlogits || (dentropy && !entropy))) return PK_ERR_ARG;
  const int e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(logits, e) || !rows::aligned_to(dlogits, e) || !rows::aligned_to(labels, 8) || !rows::aligned_to(lse, 4) ||
      !rows::aligned_to(entropy, 4) || !rows::aligned_to(dlogp, 4) || !rows::aligned_to(dentropy, 4))
    return PK_ERR_ALIGN;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  LogprobBackArgs a = {};
  a.z = logits;
  a.dz = dlogits;
  a.ld = ld;
  a.lddz = lddz;
  a.labels = reinterpret_cast<const long long*>(labels);
  a.lse = lse;
  a.entropy = entropy;
  a.dlogp = dlogp;
  a.dentropy = dentropy;
  a.V = V;
  a.same = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(dlogits)) & 15) == 0 && (((ld - lddz) * e) & 15) == 0;
  // (a row that begins on a 16-byte boundary needs no chunk that hangs over)
  const bool even = rows16(logits, ld, e);
  const int64_t chunks = even ? (V + 7) / 8 : (static_cast<int64_t>(V) + 16 / e - 1 + 7) / 8, most = (int64_t(1) << 30) / chunks;
  a.chunks = rows::FastDiv(static_cast<uint32_t>(chunks));
  for (int64_t r0 = 0; r0 < T; r0 += most) {
    a.row0 = r0;
    a.total = static_cast<uint32_t>((T - r0 < most ? T - r0 : most) * chunks);
    const cudaError_t r = dtype == PK_F32    ? back_launch<PK_F32>(a, d.sms, stream)
                          : dtype == PK_BF16 ? back_launch<PK_BF16>(a, d.sms, stream)
                                             : back_launch<PK_F16>(a, d.sms, stream);
    if (r != cudaSuccess) return PK_ERR_CUDA;
  }
  return PK_OK;
}

}  // extern "C"
