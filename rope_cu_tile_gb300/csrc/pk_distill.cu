// pk_distill.cu -- distillation from a teacher's top logits, without keeping the student's logits (pk_distill,
// pk_distill_backward in include/pk.h).
//
//     q = softmax(values / tau) over a row's words,   z = x W^T + b,   p = softmax(z / tau) over the vocabulary
//     loss = sum_k q_k (ln q_k - ln p_word(k)),   lse = ln sum_v exp(z_v / tau)
//     dz_v = dloss / tau (p_v - sum of the q_k whose word is v),   dx = dz W,  dW = dz^T x,  db = sum over rows of dz
//
// The cross entropy's passes (pk_xent.cu, pk_vocab.cuh) with a list of words in the place of a label: the epilogue that holds a
// tile of logits in registers writes out those that the row's list names, or takes the q off there. So that it need not
// search, the lists are sorted by word first, and a table says which word of a row is the first in each slice of the vocabulary.
#include "pk_vocab.cuh"

namespace pk {

namespace {

template <int DT>
using ListStat = StatEpi<DT, true>;
template <int DT>
using ListGrad = GradEpi<DT, true>;

constexpr int kMaxTop = PK_DISTILL_MAX_TOP;

struct ListArgs {
  const long long* idx;  // [T, top]
  const float* values;   // [T, top]
  int64_t T;
  int top, ld, V;
  float inverse;         // 1 / temperature
  long long* label;      // [T] 0 where the row has a word, -1 where it has none, V where it has one past the vocabulary
  uint32_t* first;       // [slices][cap]
  int64_t cap, entries;  // of first
  int shift;             // of a slice: 2^shift words
  const int* rows;       // [count] the rows with a word
  const int* count;
  int* word;             // [count, ld] sorted, then kNoWord
  float* share;          // [count, ld]
};

// whether an entry is there: an index of a word, a value above -inf
__device__ __forceinline__ bool there(long long x, float v) { return x >= 0 && v != -INFINITY; }

// Which rows have words, a warp a row; and the table of first words emptied.
__global__ void __launch_bounds__(256) pk_distill_rows_kernel(const __grid_constant__ ListArgs a) {
  const int lane = threadIdx.x & 31;
  griddep_wait();
  for (int64_t i = blockIdx.x * 256LL + threadIdx.x; i < a.entries / 4; i += gridDim.x * 256LL)
    reinterpret_cast<uint4*>(a.first)[i] = make_uint4(0u, 0u, 0u, 0u);
  for (int64_t t = blockIdx.x * 8LL + (threadIdx.x >> 5); t < a.T; t += gridDim.x * 8LL) {
    bool any = false, bad = false;
    for (int k = lane; k < a.top; k += 32) {
      const long long x = __ldcg(a.idx + t * a.top + k);
      const bool is = there(x, __ldcg(a.values + t * a.top + k));
      any = any || is;
      bad = bad || (is && x >= a.V);
    }
    any = __any_sync(0xffffffffu, any);
    bad = __any_sync(0xffffffffu, bad);
    if (lane == 0) a.label[t] = bad ? a.V : any ? 0 : -1;
  }
}

// 32 kR numbers of a warp in ascending order, number r 32 + lane in v[r]: a bitonic network, through shuffles within 32.
template <int kR>
__device__ __forceinline__ void ascend(uint32_t (&v)[kR], int lane) {
  static_assert(kR <= 2, "");
#pragma unroll
  for (int k = 2; k <= 32 * kR; k *= 2) {
    if (k == 64) {
      const uint32_t lo = min(v[0], v[kR - 1]);
      v[kR - 1] = max(v[0], v[kR - 1]);
      v[0] = lo;
    }
#pragma unroll
    for (int j = k < 64 ? k / 2 : 16; j > 0; j /= 2)
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        const uint32_t u = __shfl_xor_sync(0xffffffffu, v[r], j);
        v[r] = !((r * 32 + lane) & k) == !(lane & j) ? min(v[r], u) : max(v[r], u);
      }
  }
}

// A warp a row that has words: their probabilities, their order (by word, equal ones by their place in the list; those that are
// not there last), and the first of each slice. One word a lane, or two. A chain of latencies.
constexpr int kGone = PK_ROWS_MAX_DIM;  // a word that is not there, among 26 bits with the place
template <int kR>
__global__ void __launch_bounds__(256) pk_distill_list_kernel(const __grid_constant__ ListArgs a) {
  const int lane = threadIdx.x & 31;
  griddep_wait();
  const int n = __ldcg(a.count);
  for (int64_t row = blockIdx.x * 8LL + (threadIdx.x >> 5); row < n; row += gridDim.x * 8LL) {
    const int64_t t = __ldcg(a.rows + row);
    uint32_t key[kR];
    float e[kR], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int k = lane + 32 * i;
      long long x = -1;
      float v = -INFINITY;
      if (k < a.top) {
        x = __ldcg(a.idx + t * a.top + k);
        v = __ldcg(a.values + t * a.top + k);
      }
      const bool is = there(x, v);
      key[i] = static_cast<uint32_t>(is ? static_cast<int>(x) : kGone) << 6 | static_cast<uint32_t>(k);
      e[i] = is ? v : -INFINITY;
      m = fmaxf(m, e[i]);
    }
    // the maximum is taken off before the temperature: what is left is exact where it counts, whatever the values have in common
    // (a NaN among them, or an infinity, comes through the exponentials)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      e[i] = key[i] >> 6 == kGone ? 0.0f : expf((e[i] - m) * a.inverse);
      sum += e[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    ascend<kR>(key, lane);
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int word = static_cast<int>(key[i] >> 6), place = static_cast<int>(key[i] & 63u), at = lane + 32 * i;
      float mine = __shfl_sync(0xffffffffu, e[0], place & 31);
      if (kR > 1) {
        const float second = __shfl_sync(0xffffffffu, e[kR - 1], place & 31);
        mine = place >= 32 ? second : mine;
      }
      int before = __shfl_up_sync(0xffffffffu, word, 1);
      const int end = __shfl_sync(0xffffffffu, static_cast<int>(key[0] >> 6), 31);
      if (lane == 0) before = i > 0 ? end : -1;
      if (at < a.ld) {
        a.word[row * a.ld + at] = word == kGone ? kNoWord : word;
        a.share[row * a.ld + at] = mine / sum;
      }
      const int slice = word >> a.shift;
      if (word != kGone && (before < 0 || before >> a.shift != slice))
        a.first[slice * a.cap + row] = static_cast<uint32_t>(at) << 8 | (word - (slice << a.shift) + 1);
    }
  }
}

// The slices of each row joined, as pk_xent_join_kernel does, and the loss from the logits that the list names: 8 rows x kLanes
// strided lanes of slices a block, then 32 lanes of words a row.
template <int kLanes>
__global__ void __launch_bounds__(8 * kLanes) pk_distill_join_kernel(const float2* part, int64_t cap, int slices, const float* picked,
                                                                     const int* word, const float* share, int ld, float inverse,
                                                                     const int* idx, const int* count, float* loss, float* lse) {
  __shared__ float2 s[kLanes][8];
  const int r = threadIdx.x & 7, g = threadIdx.x >> 3;
  const float factor = inverse * kLog2e;
  griddep_wait();
  const int n = __ldcg(count);
  const auto join = [&](float& m, float& l, float2 q) {
    const float mn = fmaxf(m, q.x);
    l = l * exp2f((m - mn) * factor) + q.y * exp2f((q.x - mn) * factor);
    m = mn;
  };
  for (int64_t r0 = blockIdx.x * 8LL; r0 < n; r0 += gridDim.x * 8LL) {
    float m = kFloor, l = 0.0f;
    if (r0 + r < n) {
#pragma unroll 4
      for (int i = g; i < slices; i += kLanes) join(m, l, __ldcg(part + i * cap + r0 + r));
    }
    s[g][r] = make_float2(m, l);
    __syncthreads();
    const int64_t row = r0 + (threadIdx.x >> 5);  // a warp's
    const int lane = threadIdx.x & 31;
    if (threadIdx.x < 256 && row < n) {
      float2 q = s[lane][threadIdx.x >> 5];
#pragma unroll
      for (int i = 32; i < kLanes; i += 32) join(q.x, q.y, s[i + lane][threadIdx.x >> 5]);
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const float2 u = make_float2(__shfl_xor_sync(0xffffffffu, q.x, o), __shfl_xor_sync(0xffffffffu, q.y, o));
        // (the same order on both sides: the lower lane's first)
        float2 a = lane & o ? u : q;
        join(a.x, a.y, lane & o ? q : u);
        q = a;
      }
      const float rest = logf(q.y);
      const int64_t t = __ldcg(idx + row);
      float v = 0.0f;
      for (int k = lane; k < ld; k += 32) {
        if (__ldcg(word + row * ld + k) == kNoWord) continue;
        const float p = __ldcg(share + row * ld + k);
        if (p != 0.0f) v += p * (logf(p) + ((q.x - __ldcg(picked + row * ld + k)) * inverse + rest));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) {
        loss[t] = v;
        lse[t] = q.x * inverse + rest;
      }
    }
    __syncthreads();
  }
}

// the scratch of the lists, beside what the cross entropy has
struct Lists {
  int ld, shift;
  int64_t cap, entries;
  int* word;
  float* share;
  uint32_t* first;
  long long* label;
};
Lists plan_lists(Carver& c, int64_t T, int V, int top, int width) {
  Lists l;
  l.ld = static_cast<int>(round_up(top, 4));
  l.shift = 0;
  while (1 << l.shift < width) ++l.shift;  // (slices are 32, 64 or 128 words)
  l.cap = round_up(T, 256);
  l.entries = (V + width - 1) / width * l.cap;
  l.word = static_cast<int*>(c.take(T * l.ld * 4));
  l.share = static_cast<float*>(c.take(T * l.ld * 4));
  l.first = static_cast<uint32_t*>(c.take(l.entries * 4));
  l.label = static_cast<long long*>(c.take(T * 8));
  return l;
}

struct Fwd {
  Lists lists;
  Common m;
  gemm::Shape shape;
  float2* part;
  float* picked;
  int slices;
  int64_t bytes;
};
Fwd plan_forward(int dtype, const void* x, int64_t ldx, const void* w, int64_t T, int D, int V, int top, int sms, void* ws) {
  Fwd f = {};
  Carver c(ws);
  f.shape = gemm::pick_shape(T, V, D, dtype == PK_F32 ? gemm::kTerms32 : 1, sms, false);
  const int width = 64 * f.shape.cg;  // of an epilogue's warp (eight of them)
  f.lists = plan_lists(c, T, V, top, width);
  plan_common(c, f.m, dtype, x, ldx, w, T, D, V);
  f.slices = (V + width - 1) / width;
  f.part = static_cast<float2*>(c.take(f.slices * f.m.cap * 8));
  f.picked = static_cast<float*>(c.take(T * f.lists.ld * 4));
  f.bytes = c.used;
  return f;
}
struct Back {
  Lists lists;
  Bwd b;
  int64_t bytes;
};
Back plan_back(int dtype, const void* x, int64_t ldx, const void* w, bool need_db, int64_t T, int D, int V, int top, int sms, void* ws) {
  Back p;
  // (the tile of dz, and with it the slices, is the plan's to say: once for that, once for its place behind the lists)
  const int width = 32 * plan_backward(dtype, x, ldx, w, need_db, T, D, V, sms, nullptr).dz_shape.cg;  // (sixteen warps)
  Carver c(ws);
  p.lists = plan_lists(c, T, V, top, width);
  p.b = plan_backward(dtype, x, ldx, w, need_db, T, D, V, sms, ws ? static_cast<char*>(ws) + c.used : nullptr);
  p.bytes = c.used + p.b.bytes;
  return p;
}

ListArgs list_args(const Lists& l, const Common& m, const int64_t* idx, const float* values, int64_t T, int top, int V, float inverse) {
  ListArgs a = {};
  a.idx = reinterpret_cast<const long long*>(idx);
  a.values = values;
  a.T = T;
  a.top = top;
  a.ld = l.ld;
  a.V = V;
  a.inverse = inverse;
  a.label = l.label;
  a.first = l.first;
  a.cap = l.cap;
  a.entries = l.entries;
  a.shift = l.shift;
  a.rows = m.idx;
  a.count = m.count;
  a.word = l.word;
  a.share = l.share;
  return a;
}
// The rows with words, listed as the cross entropy lists its labelled ones, and their lists.
cudaError_t lists_launch(const ListArgs& a, const RowArgs& r, int sms, cudaStream_t stream) {
  const int64_t blocks = (a.T + 7) / 8, most = static_cast<int64_t>(sms) * 8;
  Launch l(blocks < most ? blocks : most, 256, stream);
  cudaError_t e = cudaLaunchKernelEx(&l.cfg, pk_distill_rows_kernel, a);
  if (e != cudaSuccess || (e = rows_launch(r, stream)) != cudaSuccess) return e;
  return a.top <= 32 ? cudaLaunchKernelEx(&l.cfg, pk_distill_list_kernel<1>, a) : cudaLaunchKernelEx(&l.cfg, pk_distill_list_kernel<2>, a);
}

bool distill_ok(int dtype, int64_t T, int D, int V, int top, double temperature) {
  return dtype_ok(dtype) && sizes_ok(T, D, V) && top >= 1 && top <= kMaxTop && temperature >= 1e-3 && temperature <= 1e3;
}

}  // namespace

namespace rows {
cudaError_t prepare_distill() {
  cudaError_t e;
  if ((e = gemm::prepare<ListStat<PK_F32>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<ListStat<PK_BF16>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<ListStat<PK_F16>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<ListGrad<PK_F32>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<ListGrad<PK_BF16>>()) != cudaSuccess) return e;
  return gemm::prepare<ListGrad<PK_F16>>();
}
}  // namespace rows

}  // namespace pk

extern "C" {

int pk_distill_workspace(int dtype, const void* x, int64_t ldx, const void* w, int backward, int need_db, int64_t T, int D, int V, int top,
                         int64_t* bytes) {
  using namespace pk;
  if (!bytes || !distill_ok(dtype, T, D, V, top, 1.0) || ldx < D) return PK_ERR_ARG;
  *bytes = 0;
  if (T == 0) return PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  *bytes = backward ? plan_back(dtype, x, ldx, w, need_db != 0, T, D, V, top, d.sms, nullptr).bytes
                    : plan_forward(dtype, x, ldx, w, T, D, V, top, d.sms, nullptr).bytes;
  return PK_OK;
}

int pk_distill(int dtype, const void* x, int64_t ldx, const void* w, const void* bias, const int64_t* idx, const float* values, int top,
               double temperature, int64_t T, int D, int V, float* loss, float* lse, void* workspace, int64_t workspace_bytes,
               int* status, struct CUstream_st* stream) {
  using namespace pk;
  if (!distill_ok(dtype, T, D, V, top, temperature) || ldx < D || workspace_bytes < 0) return PK_ERR_ARG;
  if (T > 0 && (!x || !w || !idx || !values || !loss || !lse)) return PK_ERR_ARG;
  const uintptr_t e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, e) || !rows::aligned_to(w, e) || !rows::aligned_to(bias, e) || !rows::aligned_to(idx, 8) ||
      !rows::aligned_to(values, 4) || !rows::aligned_to(loss, 4) || !rows::aligned_to(lse, 4) || !rows::aligned_to(workspace, 256) ||
      !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) return status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess ? PK_ERR_CUDA : PK_OK;
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Fwd f = plan_forward(dtype, x, ldx, w, T, D, V, top, d.sms, workspace);
  if (!workspace || workspace_bytes < f.bytes) return PK_ERR_NOMEM;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  const float inverse = static_cast<float>(1.0 / temperature);
  RowArgs r = {};
  r.labels = f.lists.label;
  r.T = T;
  r.V = V;
  r.counts = f.m.counts;
  r.maxima = f.m.maxima;
  r.idx = f.m.idx;
  r.lab = f.m.lab;
  r.count = f.m.count;
  r.loss = loss;
  r.lse = lse;
  r.status = status ? status : rows::stream_status(d, stream);
  if (lists_launch(list_args(f.lists, f.m, idx, values, T, top, V, inverse), r, d.sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  Inputs in;
  if (lay_out(dtype, f.m, x, ldx, w, T, D, V, d.sms, stream, &in) != cudaSuccess) return PK_ERR_CUDA;
  gemm::Args a = {};
  a.M = static_cast<int>(T);
  a.N = V;
  a.K = D;
  a.dyn = f.m.count;
  a.dyn_axis = 0;
  a.alt_count = static_cast<int>(T);
  a.alt_operand = 0;
  a.status = r.status;
  a.timeout_ns = wait_limit_ns();
  StatParams sp = {};
  sp.bias = bias;
  sp.bias_vec = bias && rows::aligned_to(bias, 16);
  sp.part = f.part;
  sp.picked = f.picked;
  sp.cap = f.m.cap;
  sp.lists = {f.lists.word, f.lists.share, f.lists.first, f.lists.ld};
  sp.factor = inverse * kLog2e;
  if (logits_product<ListStat>(dtype, in.xc, in.w, in.alt ? &in.xd : nullptr, a, sp, f.shape, d.sms, stream) != cudaSuccess)
    return PK_ERR_CUDA;
  // more lanes a row where there are many slices and few rows (284 rows over 105909 words 84 us with 32 lanes a row in all, 72 with
  // 128; 16384 over 32768 383 and 408)
  const bool wide = f.slices > 64 && T <= static_cast<int64_t>(d.sms) * 16;
  const int64_t blocks = (T + 7) / 8, most = static_cast<int64_t>(d.sms) * (wide ? 2 : 8);
  rows::Launch l(blocks < most ? blocks : most, wide ? 1024 : 256, stream);
  const float2* part = f.part;
  const float *picked = f.picked, *share = f.lists.share;
  const int *word = f.lists.word, *at = f.m.idx, *count = f.m.count;
  return cudaLaunchKernelEx(&l.cfg, wide ? pk_distill_join_kernel<128> : pk_distill_join_kernel<32>, part, f.m.cap, f.slices, picked, word,
                            share, f.lists.ld, inverse, at, count, loss, lse) == cudaSuccess
             ? PK_OK
             : PK_ERR_CUDA;
}

int pk_distill_backward(int dtype, const void* x, int64_t ldx, const void* w, const void* bias, const int64_t* idx, const float* values,
                        int top, double temperature, const float* lse, const float* dloss, int64_t T, int D, int V, void* dx, void* dw,
                        void* db, void* workspace, int64_t workspace_bytes, int* status, struct CUstream_st* stream) {
  using namespace pk;
  if (!distill_ok(dtype, T, D, V, top, temperature) || ldx < D || workspace_bytes < 0) return PK_ERR_ARG;
  if (T > 0 && (!x || !w || !idx || !values || !lse || !dloss)) return PK_ERR_ARG;
  const uintptr_t e = rows::elem_bytes(dtype);
  if (!rows::aligned_to(x, e) || !rows::aligned_to(w, e) || !rows::aligned_to(bias, e) || !rows::aligned_to(idx, 8) ||
      !rows::aligned_to(values, 4) || !rows::aligned_to(lse, 4) || !rows::aligned_to(dloss, 4) || !rows::aligned_to(dx, e) ||
      !rows::aligned_to(dw, e) || !rows::aligned_to(db, e) || !rows::aligned_to(workspace, 256) || !rows::aligned_to(status, 4))
    return PK_ERR_ALIGN;
  if (T == 0) {
    if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
    if (dw && cudaMemsetAsync(dw, 0, e * V * static_cast<size_t>(D), stream) != cudaSuccess) return PK_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, e * V, stream) != cudaSuccess) return PK_ERR_CUDA;
    return PK_OK;
  }
  rows::Device d;
  const int rc = rows::device(&d);
  if (rc != PK_OK) return rc;
  const Back plan = plan_back(dtype, x, ldx, w, db != nullptr, T, D, V, top, d.sms, workspace);
  if (!workspace || workspace_bytes < plan.bytes) return PK_ERR_NOMEM;
  const Bwd& b = plan.b;
  const Lists& lists = plan.lists;
  if (status && cudaMemsetAsync(status, 0, sizeof(int), stream) != cudaSuccess) return PK_ERR_CUDA;
  const float inverse = static_cast<float>(1.0 / temperature);
  RowArgs r = {};
  r.labels = lists.label;
  r.T = T;
  r.V = V;
  r.counts = b.m.counts;
  r.maxima = b.m.maxima;
  r.idx = b.m.idx;
  r.lab = b.m.lab;
  r.count = b.m.count;
  r.dloss = dloss;
  r.lse_in = lse;
  r.coef = b.coef;
  r.lse_rows = b.lse;
  r.unscale = b.unscale;
  r.factor = inverse;
  r.scaled = dtype == PK_F16;
  r.status = status ? status : rows::stream_status(d, stream);
  if (lists_launch(list_args(lists, b.m, idx, values, T, top, V, inverse), r, d.sms, stream) != cudaSuccess) return PK_ERR_CUDA;
  Inputs in;
  if (lay_out(dtype, b.m, x, ldx, w, T, D, V, d.sms, stream, &in) != cudaSuccess) return PK_ERR_CUDA;
  GradParams gp = {};
  gp.lists = {lists.word, lists.share, lists.first, lists.ld};
  gp.inverse = inverse;
  return backward_pieces<ListGrad>(dtype, b, in, gp, bias, T, D, V, dx, dw, db, r.status, d.sms, stream);
}

}  // extern "C"
