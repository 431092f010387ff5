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
constexpr int kShort = 1024;  // words: up to here a row belongs to a warp and lies in its registers
constexpr int kCap = 1024;    // candidates of a block
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
__device__ __forceinline__ Stat join(Stat a, Stat b) {
  const float m = fmaxf(a.m, b.m);
  raise(a, m);
  raise(b, m);
  return {m, a.s + b.s, a.u + b.u};
}

// The largest of eight values as they were loaded: of 16-bit ones two at a time.
template <int DT>
__device__ __forceinline__ float top8(const Raw8<DT>& q) {
  if constexpr (DT == PK_F32) {
    float v[8];
    q.get(v);
    return fmaxf(attn::fmax3(v[0], v[1], v[2]), attn::fmax3(attn::fmax3(v[3], v[4], v[5]), v[6], v[7]));
  } else {
    uint32_t m = q.q[0].x;
    const uint32_t w[3] = {q.q[0].y, q.q[0].z, q.q[0].w};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      if constexpr (DT == PK_BF16)
        asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
      else
        asm("max.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    }
    const float2 f = Elem<DT == PK_BF16>::unpack(m);
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

__device__ __forceinline__ Stat warp_join(Stat a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Stat b = {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o), __shfl_xor_sync(0xffffffffu, a.u, o)};
    a = join(a, b);
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
// short rows: a warp each, the elements in registers; the likeliest by repeated maxima

template <int DT>
__global__ void __launch_bounds__(kThreads) pk_logprobs_short_kernel(const __grid_constant__ LogprobArgs a) {
  const int lane = threadIdx.x & 31;
  griddep_wait();
  for (int64_t row = blockIdx.x * static_cast<int64_t>(kWarps) + (threadIdx.x >> 5); row < a.T;
       row += static_cast<int64_t>(gridDim.x) * kWarps) {
    constexpr int kC = kShort / 256 + 1;  // chunks of a lane: one more for a row that begins inside 16 bytes
    const Row r = row_at<DT>(a.z, row * a.ld, a.V);
    const long long label = __ldcg(a.labels + row);
    float picked = 0.0f;
    if (label >= 0 && label < a.V) picked = Ty<DT>::get(r.p, label);
    Raw8<DT> q[kC];
    float v[8];
    Stat st = nothing();
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if (i * 32 + lane < r.chunks) fetch<DT>(q[i], r, i * 32 + lane, a.V);
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if (i * 32 + lane < r.chunks) {
        raise(st, fmaxf(st.m, top8<DT>(q[i])));
        accumulate<DT>(st, q[i]);
      }
    st = warp_join(st);
    if (lane == 0) write_row<DT>(a, row, st, picked, label);
    if (a.top == 0) continue;
    // `best`: this lane's likeliest element that has not been taken, and its index; past the last one taken
    const float rest = logf(st.s);
    uint32_t last_key = 0xFFFFFFFFu;
    int last_idx = -1;
    const auto find = [&](uint32_t& key, int& idx) {
      key = 0;
      idx = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < kC; ++i)
        if (i * 32 + lane < r.chunks) {
          q[i].get(v);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = (i * 32 + lane) * 8 - r.off + j;
            const uint32_t k = key_of<DT>(v[j]);
            const bool left = k < last_key || (k == last_key && c > last_idx);
            if (c >= 0 && c < a.V && left && (k > key || idx == 0x7fffffff)) {
              key = k;
              idx = c;
            }
          }
        }
    };
    uint32_t key;
    int idx;
    find(key, idx);
    for (int n = 0; n < a.top; ++n) {
      const uint32_t most = __reduce_max_sync(0xffffffffu, idx == 0x7fffffff ? 0u : key);
      const int at = __reduce_min_sync(0xffffffffu, key == most ? idx : 0x7fffffff);
      if (lane == 0) {
        a.top_logp[row * a.top + n] = logp_of(st, rest, of_key<DT>(most));
        a.top_idx[row * a.top + n] = at;
      }
      last_key = most;
      last_idx = at;
      if (idx == at) find(key, idx);
    }
  }
}

// ------------------------------------------------------------------------------------
// longer rows: a block, or a cluster of blocks where there are few rows

struct Candidate {
  uint32_t key;
  int idx;
};
__device__ __forceinline__ bool before(const Candidate& x, const Candidate& y) {
  return x.key > y.key || (x.key == y.key && x.idx < y.idx);
}

struct LogprobShared {
  Stat stat[kWarps];
  Stat mine;               // of the block's slice, read by the cluster's first block
  uint32_t maxima[kThreads];
  int chunk[kThreads];     // where each thread's maximum stands
  int list[kThreads];      // threads whose elements are candidates
  int listed, found;
  uint32_t bound;
  int bound_chunk;
  Candidate cand[kCap];
  Candidate top[kMaxTop];  // the slice's likeliest, in order
  Candidate pick[kWarps];
};

// The candidates of the block's slice into sh.cand: elements whose key is above `bound`, or at it and in a chunk up to
// `bound_chunk`. Their count (which may be past kCap) is returned in every thread.
template <int DT>
__device__ __forceinline__ int collect(LogprobShared& sh, const Row& r, int c0, int c1, int V, bool mine, uint32_t bound,
                                       int bound_chunk) {
  if (threadIdx.x == 0) sh.listed = sh.found = 0;
  __syncthreads();
  if (mine) sh.list[atomicAdd(&sh.listed, 1)] = threadIdx.x;
  __syncthreads();
  // the listed threads' chunks, shared out over all threads
  const int each = (c1 - c0 + kThreads - 1) / kThreads, n = sh.listed * each;
#pragma unroll 2
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int k = i / each, c = c0 + sh.list[k] + (i - k * each) * kThreads;
    if (c >= c1 || *reinterpret_cast<volatile int*>(&sh.found) > kCap) continue;  // (too many already)
    Raw8<DT> q;
    fetch<DT>(q, r, c, V);
    float v[8];
    q.get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t x = key_of<DT>(v[j]);
      const int e = c * 8 - r.off + j;
      if ((x > bound || (x == bound && c <= bound_chunk)) && e >= 0 && e < V) {
        const int at = atomicAdd(&sh.found, 1);
        if (at < kCap) sh.cand[at] = {x, e};
      }
    }
  }
  __syncthreads();
  return sh.found;
}

// The first `top` of sh.cand[0 .. n) in order, by counting for each how many stand before it.
__device__ __forceinline__ void rank(const Candidate* cand, int n, Candidate* out, int top) {
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const Candidate x = cand[i];
    int at = 0;
    for (int j = 0; j < n; ++j) at += before(cand[j], x) ? 1 : 0;
    if (at < top) out[at] = x;
  }
}

// The slice's `top` likeliest words into sh.top; how many there are (fewer in a slice with fewer words).
template <int DT>
__device__ __forceinline__ int slice_top(LogprobShared& sh, const Row& r, int c0, int c1, int V, int top, uint32_t key, int chunk,
                                         bool any) {
  constexpr int kBits = 32 - kKeyShift<DT>;
  const int lane = threadIdx.x & 31;
  sh.maxima[threadIdx.x] = any ? key : 0u;
  sh.chunk[threadIdx.x] = any ? chunk : 0x7fffffff;
  __syncthreads();
  if (threadIdx.x < 32) {
    // the top-th largest of the threads' maxima, a bit at a time (0 where there are not as many)
    uint32_t k[kThreads / 32], bound = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) k[i] = sh.maxima[i * 32 + lane];
#pragma unroll 1
    for (int b = kBits - 1; b >= 0; --b) {
      const uint32_t probe = bound | 1u << b;
      int n = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) n += k[i] >= probe ? 1 : 0;
      if (__reduce_add_sync(0xffffffffu, n) >= top) bound = probe;
    }
    if (lane == 0) sh.bound = bound;
  }
  __syncthreads();
  const uint32_t bound = sh.bound;
  int n = collect<DT>(sh, r, c0, c1, V, any && key >= bound, bound, 0x7fffffff);
  if (n > kCap) {
    // many equal ones (a masked vocabulary): of those at the bound only the first chunks', up to the one that completes `top`
    if (threadIdx.x < 32) {
      int at = 0;
#pragma unroll 1
      for (int b = 17; b >= 0; --b) {  // the largest chunk at which there are still fewer than `top`
        const int probe = at | 1 << b;
        int m = 0;
        for (int i = lane; i < kThreads; i += 32) m += sh.maxima[i] > bound || (sh.maxima[i] == bound && sh.chunk[i] < probe) ? 1 : 0;
        if (__reduce_add_sync(0xffffffffu, m) < top) at = probe;
      }
      if (lane == 0) sh.bound_chunk = at;
    }
    __syncthreads();
    const int last = sh.bound_chunk;
    n = collect<DT>(sh, r, c0, c1, V, any && (key > bound || (key == bound && (chunk <= last || chunk == kAnywhere))), bound, last);
  }
  if (n <= kCap) {
    rank(sh.cand, n, sh.top, top);
    __syncthreads();
    return min(n, top);
  }
  // many large ones in few threads: one maximum after another
  Candidate done = {0xFFFFFFFFu, -1};
  for (int i = 0; i < top; ++i) {
    Candidate best = {0u, 0x7fffffff};
    for (int c = c0 + threadIdx.x; c < c1; c += kThreads) {
      Raw8<DT> q;
      fetch<DT>(q, r, c, V);
      float v[8];
      q.get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Candidate x = {key_of<DT>(v[j]), c * 8 - r.off + j};
        if (x.idx >= 0 && x.idx < V && before(done, x) && before(x, best)) best = x;
      }
    }
    const uint32_t most = __reduce_max_sync(0xffffffffu, best.key);
    const int at = __reduce_min_sync(0xffffffffu, best.key == most ? best.idx : 0x7fffffff);
    if (lane == 0) sh.pick[threadIdx.x >> 5] = {most, at};
    __syncthreads();
    done = sh.pick[0];
    for (int k = 1; k < kWarps; ++k)
      if (before(sh.pick[k], done)) done = sh.pick[k];
    if (threadIdx.x == 0) sh.top[i] = done;
    __syncthreads();
  }
  return top;
}

__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) { return gemm::mapa(smem_u32(p), rank); }
__device__ __forceinline__ uint32_t ld_remote(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

constexpr int kBatch = 2;  // chunks that a thread takes together, with as many on their way

template <int DT, bool kCluster>
__global__ void __launch_bounds__(kThreads, DT == PK_F32 ? 4 : 5) pk_logprobs_kernel(const __grid_constant__ LogprobArgs a, int parts) {
  __shared__ LogprobShared sh;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int part = kCluster ? static_cast<int>(gemm::cluster_rank()) : 0;
  const int64_t row = kCluster ? blockIdx.x / parts : blockIdx.x;
  griddep_wait();
  const Row r = row_at<DT>(a.z, row * a.ld, a.V);
  const int per = kCluster ? (r.chunks + parts - 1) / parts : r.chunks;
  const int c0 = part * per, c1 = min(c0 + per, r.chunks);
  long long label = -1;
  float picked = 0.0f;
  if (threadIdx.x == 0 && part == 0) {
    label = __ldcg(a.labels + row);
    if (label >= 0 && label < a.V) picked = Ty<DT>::get(r.p, label);
  }
  Stat st = nothing();
  int at = c0 + threadIdx.x;  // the chunk of the maximum
  const bool any = at < c1;
  // the next chunks are asked for before these are used
  Raw8<DT> q[kBatch], ahead[kBatch];
  const auto load = [&](Raw8<DT>(&r8)[kBatch], int c) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c + i * kThreads < c1) fetch<DT>(r8[i], r, c + i * kThreads, a.V);
  };
  load(q, c0 + threadIdx.x);
#pragma unroll 1
  for (int c = c0 + threadIdx.x; c < c1; c += kBatch * kThreads) {
    load(ahead, c + kBatch * kThreads);
    float m = st.m;
    bool none = st.s == 0.0f;  // (so far: the lowest number is then larger than what there was, though not than m)
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float top = c + i * kThreads < c1 ? top8<DT>(q[i]) : -INFINITY;
      const bool larger = top > m || (none && top == m);
      at = larger ? c + i * kThreads : at;
      none = none && !larger;
      m = fmaxf(m, top);
    }
    raise(st, m);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (c + i * kThreads < c1) accumulate<DT>(st, q[i]);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) q[i] = ahead[i];
  }
  // (a sum without a value: one of the thread's elements is infinite or NaN, so at least infinity, in a chunk unknown. No sum at
  // all: every element is -inf, the first of them in its first chunk)
  const bool nan = st.s != st.s;
  const uint32_t key = key_of<DT>(nan ? INFINITY : st.s == 0.0f ? -INFINITY : st.m);
  if (nan) at = kAnywhere;
  const Stat ws = warp_join(st);
  if (lane == 0) sh.stat[w] = ws;
  int n = 0;
  __syncthreads();
  if (a.top > 0) n = slice_top<DT>(sh, r, c0, c1, a.V, min(a.top, max(0, min(a.V, c1 * 8 - r.off) - max(0, c0 * 8 - r.off))), key, at, any);
  st = sh.stat[0];
#pragma unroll
  for (int i = 1; i < kWarps; ++i) st = join(st, sh.stat[i]);
  const Candidate* top = sh.top;
  if constexpr (kCluster) {
    if (threadIdx.x == 0) {
      sh.mine = st;
      sh.found = n;
    }
    gemm::cluster_sync();
    if (part == 0) {
      // the slices' sums and likeliest words, in the order of the slices
      int have = n;
      for (int p = 1; p < parts; ++p) {
        const uint32_t s = remote(&sh.mine, p);
        const Stat b = {__uint_as_float(ld_remote(s)), __uint_as_float(ld_remote(s + 4)), __uint_as_float(ld_remote(s + 8))};
        st = join(st, b);
        if (a.top > 0) {
          const int k = static_cast<int>(ld_remote(remote(&sh.found, p)));
          const uint32_t t = remote(&sh.top[0], p);
          for (int i = threadIdx.x; i < k; i += kThreads)
            sh.cand[have + i] = {ld_remote(t + 8 * i), static_cast<int>(ld_remote(t + 8 * i + 4))};
          have += k;
        }
      }
      if (a.top > 0) {
        for (int i = threadIdx.x; i < n; i += kThreads) sh.cand[i] = sh.top[i];
        __syncthreads();
        rank(sh.cand, have, sh.top, a.top);
        __syncthreads();
      }
    }
    gemm::cluster_sync();  // (no block leaves while its memory is read)
    if (part != 0) return;
  }
  if (threadIdx.x == 0) write_row<DT>(a, row, st, picked, label);
  const float rest = logf(st.s);
  for (int i = threadIdx.x; i < a.top; i += kThreads) {
    a.top_logp[row * a.top + i] = logp_of(st, rest, of_key<DT>(top[i].key));
    a.top_idx[row * a.top + i] = top[i].idx;
  }
}

// Blocks a row: one where the rows fill the SMs, up to eight where they do not, none with fewer than 4096 words.
int parts_of(int64_t T, int V, int sms) {
  int parts = 1;
  while (parts < 8 && T * parts * 2 <= 2 * sms && V / (parts * 2) >= 4096) parts *= 2;
  return parts;
}

template <int DT>
cudaError_t logprobs_launch(const LogprobArgs& a, int sms, cudaStream_t stream) {
  if (a.V <= kShort) {
    const int64_t blocks = (a.T + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * 8;
    Launch l(blocks < most ? blocks : most, kThreads, stream);
    return cudaLaunchKernelEx(&l.cfg, pk_logprobs_short_kernel<DT>, a);
  }
  const int parts = parts_of(a.T, a.V, sms);
  Launch l(a.T * parts, kThreads, stream);
  if (parts == 1) return cudaLaunchKernelEx(&l.cfg, pk_logprobs_kernel<DT, false>, a, parts);
  cudaLaunchAttribute at[2] = {l.at[0], {}};
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = parts;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  l.cfg.attrs = at;
  l.cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&l.cfg, pk_logprobs_kernel<DT, true>, a, parts);
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
