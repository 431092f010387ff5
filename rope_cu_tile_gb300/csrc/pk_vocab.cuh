// pk_vocab.cuh -- what the losses over a vocabulary share (pk_xent.cu, pk_distill.cu): the list of the rows that take part, the
// epilogues that reduce tiles of logits or turn them into dz, the scratch of a call, and the backward pass over pieces of the
// vocabulary. How they work stands at the top of pk_xent.cu.
#pragma once

#include "pk_rows.cuh"

namespace pk {

namespace {

using namespace rows;

constexpr float kLog2e = 1.4426950408889634f;
// running maximum of nothing: the lowest finite value, so that a row of -inf logits stays defined and one of words masked by
// that value has it as its maximum
constexpr float kFloor = -3.402823466e38f;

__device__ __forceinline__ float exp2_fast(float x) { return attn::ex2(x); }

// ------------------------------------------------------------------------------------
// the labelled rows

constexpr int kScan = 1024;  // labels of a block

struct RowArgs {
  const long long* labels;
  int64_t T;
  int V;
  int* counts;      // [blocks] labelled rows of each block
  float* maxima;    // [blocks] largest |dloss| of each block's labelled rows (backward)
  int* idx;         // [count] the labelled rows, in order
  int* lab;         // [count] their labels
  int* count;       // labelled rows
  float* loss;      // forward: written for rows without a label
  float* lse;
  const float* dloss;  // backward
  const float* lse_in;
  float* coef;      // [count] dloss, times the scale of fp16's dz
  float* lse_rows;  // [count]
  float* unscale;   // the inverse of that scale
  float factor;     // of dloss in dz
  int scaled;       // fp16
  int* status;
};

__device__ __forceinline__ bool has_label(const RowArgs& a, int64_t t, long long& l) {
  l = t < a.T ? __ldcg(a.labels + t) : -1;
  return l >= 0 && l < a.V;
}

__global__ void __launch_bounds__(kScan) pk_xent_count_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float top[32];
  griddep_wait();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kScan + threadIdx.x;
  long long l;
  const bool has = has_label(a, t, l);
  const int n = __syncthreads_count(has);
  float m = has && a.dloss ? fabsf(__ldcg(a.dloss + t)) : 0.0f;
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < 32; ++i) m = fmaxf(m, top[i]);
    a.counts[blockIdx.x] = n;
    a.maxima[blockIdx.x] = m;
  }
}

__global__ void __launch_bounds__(kScan) pk_xent_index_kernel(const __grid_constant__ RowArgs a) {
  __shared__ int part[32], warp_first[32];
  __shared__ float top[32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  griddep_wait();
  // labelled rows before this block, and the largest |dloss| of all (one block finds its own; more read what
  // pk_xent_count_kernel found)
  int before = 0;
  float m = 0.0f;
  if (gridDim.x == 1) {
    const int64_t t = threadIdx.x;
    long long l;
    if (has_label(a, t, l) && a.dloss) m = fabsf(__ldcg(a.dloss + t));
  } else {
    for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += kScan) {
      if (b < static_cast<int>(blockIdx.x)) before += __ldcg(a.counts + b);
      m = fmaxf(m, __ldcg(a.maxima + b));
    }
  }
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (lane == 0) {
    part[w] = before;
    top[w] = m;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kScan + threadIdx.x;
  long long l;
  const bool has = has_label(a, t, l);
  const unsigned int ballot = __ballot_sync(0xffffffffu, has);
  if (lane == 0) warp_first[w] = __popc(ballot);
  __syncthreads();
  before = 0;
  m = 0.0f;
  for (int i = 0; i < 32; ++i) {
    before += part[i];
    m = fmaxf(m, top[i]);
  }
  int total = before;
  for (int i = 0; i < 32; ++i) {
    if (i < w) before += warp_first[i];
    total += warp_first[i];
  }
  // fp16's dz: the largest |dloss| brought near 2^14 by a power of two, so that small probabilities are not lost to
  // fp16's narrow range and no |dz| <= |dloss| overflows; the products' results are scaled back
  float scale = 1.0f, inverse = 1.0f;
  m *= a.factor;
  if (a.scaled && m > 0.0f && m < 3.0e38f) {
    const int e = max(-100, min(100, 14 - ilogbf(m)));
    scale = scalbnf(1.0f, e);
    inverse = scalbnf(1.0f, -e);
  }
  if (t < a.T) {
    if (has) {
      const int at = before + __popc(ballot & ((1u << lane) - 1u));
      a.idx[at] = static_cast<int>(t);
      a.lab[at] = static_cast<int>(l);
      if (a.dloss) {
        a.coef[at] = __ldcg(a.dloss + t) * a.factor * scale;
        a.lse_rows[at] = __ldcg(a.lse_in + t);
      }
    } else {
      if (l >= a.V && a.status) atomicCAS(a.status, 0, PK_ERR_BAD_LABEL);
      if (a.loss) {
        a.loss[t] = l >= a.V ? __int_as_float(0x7fc00000) : 0.0f;  // a label past the vocabulary shows as NaN
        a.lse[t] = 0.0f;
      }
    }
  }
  if (threadIdx.x == 0 && blockIdx.x == gridDim.x - 1) *a.count = total;
  if (threadIdx.x == 0 && blockIdx.x == 0 && a.unscale) *a.unscale = inverse;
}

cudaError_t rows_launch(const RowArgs& a, cudaStream_t stream) {
  Launch l((a.T + kScan - 1) / kScan, kScan, stream);
  if (a.T > kScan) {
    const cudaError_t e = cudaLaunchKernelEx(&l.cfg, pk_xent_count_kernel, a);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&l.cfg, pk_xent_index_kernel, a);
}

// ------------------------------------------------------------------------------------
// forward epilogue: maximum and sum of exponentials of a row's slice of the logits. The maximum is taken off before the
// change of base: a fused z log2(e) - m' would be off by up to 2^-24 |m'| in the exponent and overflow for logits past 2^31.

// The words that a row's loss names: one label, or a list of them in ascending order with the probabilities that the
// gradient takes off there, `ld` a row of the product (the list ends with kNoWord). Of each slice of the vocabulary that a
// warp of an epilogue empties a table holds, by row, which of the row's words is the first inside: 0 for none, else its place in
// the list << 8 | its column in the slice + 1. So a warp without words in its slice, most of them, pays one load.
constexpr int kNoWord = 0x7fffffff;
struct WordLists {
  const int* word;
  const float* share;
  const uint32_t* first;  // [slices of the vocabulary][cap]
  int ld;
};
// A thread's place in its row's list: the next word, and the one after it on its way (of the gradient's, with their shares).
template <bool kShares>
struct WordCursor {
  const int* list;
  int64_t base;  // of the list
  int pos, ld, next, after;
  uint32_t first;
  const float* shares;
  float share, share_after;
  __device__ __forceinline__ void ahead(int i) {
    after = kNoWord;
    share_after = 0.0f;
    if (i < ld) {
      after = __ldcg(list + i);
      if (kShares) share_after = __ldcg(shares + i);
    }
  }
  // asks where slice `slice` begins in the row's list
  __device__ __forceinline__ void ask(const WordLists& w, int64_t cap, int row, bool live, int slice) {
    first = live ? __ldcg(w.first + slice * cap + row) : 0u;
    ld = w.ld;
    base = static_cast<int64_t>(row) * ld;
    list = w.word + base;
    shares = w.share + base;
  }
  // at the first word of the slice, which begins at column `from` of the vocabulary. (Called when the tile's logits have been
  // asked for too: the answer's way costs nothing then.)
  __device__ __forceinline__ void begin(int from) {
    pos = static_cast<int>(first >> 8);
    next = after = kNoWord;
    if (first) {
      next = from + static_cast<int>(first & 255u) - 1;
      if (kShares) share = __ldcg(shares + pos);
      ahead(pos + 1);
    }
  }
  __device__ __forceinline__ void step() {
    ++pos;
    next = after;
    share = share_after;
    ahead(pos + 1);
  }
};
// v[at] of 32 registers
__device__ __forceinline__ float element(const float (&v)[32], int at) {
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) t[i] = at & 16 ? v[i + 16] : v[i];
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) t[i] = at & o ? t[i + o] : t[i];
  return t[0];
}

struct StatParams {
  const void* bias;
  int bias_vec;
  const int* lab;
  float2* part;  // [slices][cap]
  float* picked; // [cap] the label's logit; of lists, each word's, where the list has the word
  int64_t cap;
  WordLists lists;
  float factor;  // lists: log2(e) / temperature
};

// v[i] = exp(v[i] + shift), for every type by the short exponential: off by 2^-22 of itself and, for an argument of size q, by
// 1.5 q 2^-24 (its product with log2 e): where a probability is not small, q is not large. What lse is off by is
// the truncation of the tensor pipe's sums in z (3e-7 of itself at 1024 features and 50000 words, fp32 and bf16 alike; 9e-8 of fp32
// at 256 and 8000; a plain fp32 product 3e-8 to 9e-8): shorter phases than pk_gemm.cuh's would each cost a hand-over of 2000 cycles.
__device__ __forceinline__ void exponentials(float (&v)[32], float shift, float factor = kLog2e) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    add2(v[i], v[i + 1], make_float2(shift, shift));
    const float2 q = mul2(make_float2(v[i], v[i + 1]), make_float2(factor, factor));
    v[i] = exp2_fast(q.x);
    v[i + 1] = exp2_fast(q.y);
  }
}

// kList: the row's words come as a list, and its logits are divided by a temperature.
template <int DT, bool kList>
struct StatEpi {
  using Params = StatParams;
  static constexpr int kWarps = 8;  // wide slices: half the partial results
  template <class Ready, class Done>
  static __device__ __forceinline__ bool run(const Params& p, uint32_t tacc, bool zero, int r0, int c0, int cols, int M, int N,
                                             int, int lane, uint8_t*, const Ready& ready, const Done& done) {
    if (r0 >= M || c0 >= N) {
      if (!ready()) return false;
      done();
      return true;
    }
    const int row = r0 + lane;
    const int label = !kList && row < M ? __ldcg(p.lab + row) : -1;
    const float factor = kList ? p.factor : kLog2e;
    WordCursor<false> words;
    if constexpr (kList) words.ask(p.lists, p.cap, row, row < M, c0 / cols);
    const int end = min(cols, N - c0);
    float m = kFloor, l = 0.0f;
    // The bias of 32 words: with lists asked for while the 32 before are reduced, with a label just before its logits (16384 x 256
    // over 32768 words, bf16: lists 358 us, 367 the label's way; a label 284 us, 320 the lists' way)
    Bias<DT, 32> b;
    if (kList && p.bias) b.fetch(p.bias, p.bias_vec, c0, N);
#pragma unroll 1
    for (int cc = 0; cc < end; cc += 32) {
      const int c = c0 + cc;
      float v[32];
      if (!kList && p.bias) b.fetch(p.bias, p.bias_vec, c, N);
      if (cc == 0 && !ready()) return false;
      read_acc(tacc + cc, zero, v);
      if (cc + 32 >= end) done();
      if (p.bias) {
        b.add(v);
        if (kList && cc + 32 < end) b.fetch(p.bias, p.bias_vec, c + 32, N);
      }
      if (c + 32 > N) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (c + i >= N) v[i] = -INFINITY;
      }
      if (label >= c && label < c + 32) {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < 32; ++i) z = label == c + i ? v[i] : z;
        p.picked[row] = z;
      }
      if constexpr (kList) {
        if (cc == 0) words.begin(c0);
        while (words.next < c + 32) {
          p.picked[words.base + words.pos] = element(v, words.next - c);
          words.step();
        }
      }
      float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
      for (int i = 4; i < 32; ++i) top[i & 3] = fmaxf(top[i & 3], v[i]);
      const float mn = fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
      float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      exponentials(v, -mn, factor);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        add2(s[0], s[1], make_float2(v[i], v[i + 1]));
        add2(s[2], s[3], make_float2(v[i + 2], v[i + 3]));
      }
      l = l * exp2_fast((m - mn) * factor) + ((s[0] + s[1]) + (s[2] + s[3]));
      m = mn;
    }
    if (row < M) p.part[static_cast<int64_t>(c0 / cols) * p.cap + row] = make_float2(m, l);
    return true;
  }
};

// ------------------------------------------------------------------------------------
// backward epilogue: dz of a piece of the vocabulary

struct GradParams {
  const void* bias;  // of the piece
  int bias_vec;
  const int* lab;
  const float* coef;
  const float* lse;
  int v0;            // first word of the piece
  CUtensorMap dz;    // [planes][cap, columns of the piece]
  float* col;        // [cap / 32, ldcol] column sums of 32 rows each, or null
  int64_t cap, ldcol;
  WordLists lists;
  float inverse;     // lists: 1 / temperature
};

// The sum over a warp's lanes (rows) of each of their 32 columns: column `lane` in lane `lane`. Five steps, in each of which a
// lane keeps half of its columns and hands over the other half.
__device__ __forceinline__ float column_sum(const float (&v)[32], int lane) {
  float t[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const bool up = (lane & 16) != 0;
    t[i] = (up ? v[i + 16] : v[i]) + __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + 16], 16);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) t[i] = (up ? t[i + o] : t[i]) + __shfl_xor_sync(0xffffffffu, up ? t[i] : t[i + o], o);
  }
  return t[0];
}

// (96 registers a thread: fp32 spills 156 bytes with lists, 64 with labels; 16 bits 24 and none)
template <int DT, bool kList>
struct GradEpi {
  using Params = GradParams;
  using S = Stage<DT == PK_F16 ? PK_F16 : PK_BF16>;
  static constexpr int kWarps = 16;
  template <class Ready, class Done>
  static __device__ __forceinline__ bool run(const Params& p, uint32_t tacc, bool zero, int r0, int c0, int cols, int M, int N,
                                             int, int lane, uint8_t* stage, const Ready& ready, const Done& done) {
    if (r0 >= p.cap || c0 >= N) {
      if (!ready()) return false;
      done();
      return true;
    }
    const int row = r0 + lane;
    const bool live = row < M;
    // (rows past the count feed dW and db: set to zero below)
    const float g = live ? __ldcg(p.coef + row) : 0.0f, lse = live ? __ldcg(p.lse + row) : 0.0f;
    const int label = !kList && live ? __ldcg(p.lab + row) - p.v0 : -1;
    WordCursor<true> words;
    if constexpr (kList) words.ask(p.lists, p.cap, row, live, (p.v0 + c0) / cols);
    const int end = min(cols, N - c0);
#pragma unroll 1
    for (int cc = 0; cc < end; cc += 32) {
      const int c = c0 + cc;
      float v[32];
      {
        Bias<DT, 32> b;
        if (p.bias) b.fetch(p.bias, p.bias_vec, c, N);
        if (cc == 0 && !ready()) return false;
        read_acc(tacc + cc, zero, v);
        if (cc + 32 >= end) done();
        if (p.bias) b.add(v);
      }
      if constexpr (kList) {
        if (cc == 0) words.begin(p.v0 + c0);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= p.inverse;
      }
      exponentials(v, -lse);
      if (label >= c && label < c + 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = label == c + i ? v[i] - 1.0f : v[i];
      }
      if constexpr (kList) {
        while (words.next < p.v0 + c + 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = words.next == p.v0 + c + i ? v[i] - words.share : v[i];
          words.step();
        }
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 q = mul2(make_float2(v[i], v[i + 1]), make_float2(g, g));
        v[i] = q.x;
        v[i + 1] = q.y;
      }
      if (r0 + 32 > M) {  // (their logits are 0 W^T + b: undefined beside infinite weights, and so times 0)
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = live ? v[i] : 0.0f;
      }
      // db: the column sums before dz is rounded (sums of the rounded tile, read back from the staging memory, left db with the
      // roundings wherever labels and probabilities cancel in a column)
      if (p.col) {
        const float sum = column_sum(v, lane);
        if (c + lane < N) p.col[(r0 >> 5) * p.ldcol + c + lane] = sum;
      }
#pragma unroll
      for (int k = 0; k < (DT == PK_F32 ? 3 : 1); ++k) {
        stored(lane);
        S::put(stage, lane, v);
        store_tile(&p.dz, stage, c, r0, k, lane);
        if constexpr (DT == PK_F32) {
          if (k < 2) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] -= __bfloat162float(__float2bfloat16_rn(v[i]));
          }
        }
      }
    }
    return true;
  }
};

// ------------------------------------------------------------------------------------
// plans

struct Common {
  int64_t cap;  // rows, rounded up to whole tiles
  int *counts, *idx, *lab, *count;
  float* maxima;
  void *x, *w;
  bool x_in_place;
};
void plan_common(Carver& c, Common& m, int dtype, const void* x, int64_t ldx, const void* w, int64_t T, int D, int V) {
  m.cap = round_up(T, 256);
  const int64_t blocks = (T + kScan - 1) / kScan;
  m.counts = static_cast<int*>(c.take(blocks * 4));
  m.maxima = static_cast<float*>(c.take(blocks * 4));
  m.count = static_cast<int*>(c.take(4));
  m.idx = static_cast<int*>(c.take(m.cap * 4));
  m.lab = static_cast<int*>(c.take(m.cap * 4));
  m.x_in_place = in_place(dtype, x, ldx);
  m.x = c.take(copy_bytes(dtype, m.cap, D));
  m.w = in_place(dtype, w, D) ? nullptr : c.take(copy_bytes(dtype, V, D));
}

constexpr int64_t kPieceBytes = int64_t(1) << 30;  // dz of a piece of the vocabulary, where that leaves it enough words
constexpr int64_t kPieceLeast = 4096;              // words: below, dx's way through its fp32 buffer outweighs the product

struct Bwd {
  Common m;
  int piece, pieces;
  gemm::Shape dz_shape, dx_shape, dw_shape;
  float *coef, *lse, *unscale, *acc, *part, *partial;
  uint16_t* dz;
  int64_t dz_ld, dz_plane, dx_rows, bytes;
};
Bwd plan_backward(int dtype, const void* x, int64_t ldx, const void* w, bool need_db, int64_t T, int D, int V, int sms,
                  void* ws) {
  Bwd b = {};
  Carver c(ws);
  plan_common(c, b.m, dtype, x, ldx, w, T, D, V);
  const int planes = dtype == PK_F32 ? 3 : 1, terms = dtype == PK_F32 ? gemm::kTerms32 : 1;
  int64_t most = kPieceBytes / (planes * b.m.cap * 2) / 256 * 256;
  if (most < kPieceLeast) most = kPieceLeast;
  b.pieces = static_cast<int>((V + most - 1) / most);
  b.piece = static_cast<int>(round_up((V + b.pieces - 1) / b.pieces, 256));
  b.pieces = (V + b.piece - 1) / b.piece;
  const int widest = b.piece < V ? b.piece : V;
  b.coef = static_cast<float*>(c.take(b.m.cap * 4));
  b.lse = static_cast<float*>(c.take(b.m.cap * 4));
  b.unscale = static_cast<float*>(c.take(4));
  b.dz_ld = copy_ld(widest);
  b.dz_plane = b.m.cap * b.dz_ld;
  b.dz = static_cast<uint16_t*>(c.take(planes * b.dz_plane * 2));
  if (b.pieces > 1) b.acc = static_cast<float*>(c.take(b.m.cap * D * 4));
  if (need_db) b.part = static_cast<float*>(c.take(b.m.cap / 32 * b.dz_ld * 4));
  b.dz_shape = gemm::pick_shape(T, widest, D, terms, sms, false);
  // how many rows dx has is the device's to know: where even all of them would fill the SMs only a few times over, it may
  // split k as far as the memory of the partial sums goes
  b.dx_shape = gemm::pick_shape(T, D, widest, terms, sms, false);
  const int64_t tile = 128 * b.dx_shape.cg, tiles = ((T + tile - 1) / tile) * ((D + tile - 1) / tile);
  b.dx_rows = 0;
  if (tiles < 8 * (sms / b.dx_shape.cg) && widest > 512) {
    b.dx_shape.splits = 8;
    b.dx_rows = round_up(T, 256) * 2 > 8 * 2048 ? round_up(T, 256) * 2 : 8 * round_up(T < 2048 ? T : 2048, 256);
  }
  b.dw_shape = gemm::pick_shape(widest, D, T, terms, sms, true);
  const int64_t p1 = b.dx_rows * round_up(D, 8) * 4, p2 = partial_bytes(b.dw_shape, widest, D);
  b.partial = static_cast<float*>(c.take(p1 > p2 ? p1 : p2));
  b.bytes = c.used;
  return b;
}

bool sizes_ok(int64_t T, int D, int V) {
  return T >= 0 && T <= PK_ROWS_MAX_T && D >= 1 && D <= PK_ROWS_MAX_DIM && V >= 1 && V <= PK_ROWS_MAX_DIM;
}

// the operands x (gathered; x itself where every row has a label) and W
struct Inputs {
  gemm::Operand xc, xd, w;
  bool alt;
};
cudaError_t lay_out(int dtype, const Common& m, const void* x, int64_t ldx, const void* w, int64_t T, int D, int V, int sms,
                    cudaStream_t stream, Inputs* in) {
  // gathered rows; nothing to gather when all have labels and x can be read where it lies
  in->alt = m.x_in_place;
  Copies copies(dtype);
  copies.add(x, ldx, m.cap, D, m.x, m.idx, m.count, m.x_in_place ? static_cast<int>(T) : -1);
  if (m.w) copies.add(w, D, V, D, m.w);
  in->xc = operand_of_copy(dtype, m.x, m.cap, D, 0);
  in->xd = operand(dtype, x, ldx, T, D, 0);
  in->w = m.w ? operand_of_copy(dtype, m.w, V, D, 0) : operand(dtype, w, D, V, D, 0);
  return copies.launch(sms, stream);
}

// rows [v0, v0 + n) of W
gemm::Operand words(const gemm::Operand& w, int64_t v0, int64_t n, int mn) {
  gemm::Operand o = w;
  o.p = static_cast<const uint16_t*>(w.p) + v0 * w.ld;
  o.rows = n;
  o.mn = mn;
  return o;
}

template <template <int> class Epi, class Params>
cudaError_t logits_product(int dtype, const gemm::Operand& A, const gemm::Operand& B, const gemm::Operand* alt,
                           const gemm::Args& a, const Params& ep, gemm::Shape s, int sms, cudaStream_t stream) {
  if (dtype == PK_F32) return gemm::launch<Epi<PK_F32>>(A, B, alt, a, ep, s, sms, stream);
  if (dtype == PK_BF16) return gemm::launch<Epi<PK_BF16>>(A, B, alt, a, ep, s, sms, stream);
  return gemm::launch<Epi<PK_F16>>(A, B, alt, a, ep, s, sms, stream);
}


// The backward pass from the laid-out operands on: dz of each piece of the vocabulary, and its products. `gp`: the rows' words.
template <template <int> class Epi>
int backward_pieces(int dtype, const Bwd& b, const Inputs& in, GradParams gp, const void* bias, int64_t T, int D, int V, void* dx,
                    void* dw, void* db, int* status, int sms, cudaStream_t stream) {
  const int64_t e = elem_bytes(dtype);
  // rows without a label have no gradient
  if (dx && cudaMemsetAsync(dx, 0, e * T * static_cast<size_t>(D), stream) != cudaSuccess) return PK_ERR_CUDA;
  const float* alpha = dtype == PK_F16 ? b.unscale : nullptr;
  const gemm::Operand* alt = in.alt ? &in.xd : nullptr;
  for (int i = 0; i < b.pieces; ++i) {
    const int v0 = i * b.piece, n = b.piece < V - v0 ? b.piece : V - v0;
    gemm::Args a = {};
    a.status = status;
    a.timeout_ns = wait_limit_ns();
    a.dyn = b.m.count;
    a.alt_count = static_cast<int>(T);
    // dz of the piece
    a.M = static_cast<int>(T);
    a.N = n;
    a.K = D;
    a.dyn_axis = 0;
    a.alt_operand = 0;
    gp.bias = bias ? static_cast<const char*>(bias) + v0 * e : nullptr;
    gp.bias_vec = bias && aligned_to(gp.bias, 16);
    gp.coef = b.coef;
    gp.lse = b.lse;
    gp.v0 = v0;
    gp.cap = b.m.cap;
    gp.col = db ? b.part : nullptr;
    gp.ldcol = b.dz_ld;
    if (!gemm::make_out_map(&gp.dz, dtype == PK_F16 ? PK_F16 : PK_BF16, b.dz, b.m.cap, n, b.dz_ld, dtype == PK_F32 ? 3 : 1,
                            b.dz_plane))
      return PK_ERR_CUDA;
    if (logits_product<Epi>(dtype, in.xc, words(in.w, v0, n, 0), alt, a, gp, b.dz_shape, sms, stream) != cudaSuccess)
      return PK_ERR_CUDA;
    gemm::Operand dz = operand(dtype, b.dz, b.dz_ld, b.m.cap, n, 0);
    dz.planes = dtype == PK_F32 ? 3 : 1;
    dz.plane = b.dz_plane;
    if (dw) {
      dz.mn = 1;
      gemm::Operand xb = in.xc, xa = in.xd;
      xb.mn = xa.mn = 1;
      a.M = n;
      a.N = D;
      a.K = static_cast<int>(T);
      a.dyn_axis = 1;
      a.alt_operand = 1;
      LinParams ep = {};
      ep.y = static_cast<char*>(dw) + static_cast<int64_t>(v0) * D * e;
      ep.ldy = D;
      ep.alpha = alpha;
      if (product(dtype, dtype, dz, xb, in.alt ? &xa : nullptr, a, ep, b.dw_shape, b.partial,
                        partial_rows(b.dw_shape, n), sms, stream) != cudaSuccess)
        return PK_ERR_CUDA;
    }
    if (dx) {
      dz.mn = 0;
      a.M = static_cast<int>(T);
      a.N = D;
      a.K = n;
      a.dyn_axis = 0;
      const bool last = i + 1 == b.pieces;
      LinParams ep = {};
      ep.res = i > 0 ? b.acc : nullptr;
      ep.ldres = D;
      ep.y = last ? dx : b.acc;
      ep.ldy = D;
      ep.alpha = last ? alpha : nullptr;
      ep.rowmap = last ? b.m.idx : nullptr;
      if (product(last ? dtype : PK_F32, PK_F32, dz, words(in.w, v0, n, 1), nullptr, a, ep, b.dx_shape, b.partial, b.dx_rows,
                        sms, stream) != cudaSuccess)
        return PK_ERR_CUDA;
    }
    if (db && sum_rows(dtype, b.part, b.m.cap / 32, b.m.count, 32, n, b.dz_ld, alpha, static_cast<char*>(db) + v0 * e,
                             stream) != cudaSuccess)
      return PK_ERR_CUDA;
  }
  return PK_OK;
}

}  // namespace

}  // namespace pk
