// pk_rows.cu -- shared passes of the token-row operators: tensor maps, the cut of a product into tiles and splits, operand
// copies, the sum of split partial sums with the epilogue, column sums, and the product's launches.
#include <atomic>
#include <cstdlib>
#include <map>
#include <mutex>

#include "pk_rows.cuh"

namespace pk {

// Status words of the calls that are given none: one a stream, the last one shared by all streams past the others.
constexpr int kStatusWords = 1024;
__device__ int g_rows_status[kStatusWords];

namespace gemm {

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

int debug_skip_arrive() {
  const char* e = std::getenv("PK_DEBUG_SKIP_ARRIVE");
  return e && e[0] == '1' ? 1 : 0;
}

bool make_map(CUtensorMap* map, const Operand& o) {
  const EncodeTiledFn enc = encode_fn();
  if (!enc || !operand_ok(o)) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.cols), static_cast<cuuint64_t>(o.rows),
                              static_cast<cuuint64_t>(o.planes)};
  const cuuint64_t plane = o.planes > 1 ? o.plane : o.rows * o.ld;
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.ld) * 2, plane * 2};
  const cuuint32_t box[3] = {64, o.mn ? 64u : static_cast<cuuint32_t>(o.box), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, o.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(o.p),
             dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_out_map(CUtensorMap* map, int dtype, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t planes,
                  int64_t plane) {
  const EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int e = dtype == PK_F32 ? 4 : 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * e, static_cast<cuuint64_t>(planes > 1 ? plane : rows * ld) * e};
  const cuuint32_t box[3] = {32, 32, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType t = dtype == PK_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : dtype == PK_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  return enc(map, t, 3, const_cast<void*>(p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             e == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The cheapest cut by a model of the product's time: waves x (k steps x cost of a step + cost of a tile), plus the partial
// sums' way through memory. The costs are fitted, in a unit of their own: a step of either tile takes 500 to 600 cycles, the
// pair's (four times the products) at the tensor pipe's rate of 512, the lone tile's at its operands' way through L2, twice
// the bytes a product. Lone tile and pair, bf16, us: 300 x 768 -> 768 6.7, 8.4; 2304 x 768 -> 2304 12.9, 12.3;
// 2400 x 1024 -> 4096 19.7, 20.0 (taken, 2 % off); 4096 x 1024 -> 4096 31.0, 24.9; 16931 x 768 -> 2304 53.0, 38.8.
Shape pick_shape(int64_t M, int64_t N, int64_t K, int terms, int sms, bool may_split) {
  Shape best;
  double best_cost = -1.0;
  const int64_t kbs = (K + kBK - 1) / kBK;
  for (int cg = 1; cg <= 2; ++cg) {
    const int64_t tile = 128 * cg, tiles = ((M + tile - 1) / tile) * ((N + tile - 1) / tile);
    const int64_t slots = sms / cg;
    const double step = cg == 2 ? 280.0 : 270.0, over = cg == 2 ? 1500.0 : 1000.0;
    for (int s = 1; s <= (may_split ? 32 : 1); ++s) {
      if (s > 1 && (s > kbs || s * M * N > (int64_t(1) << 28))) break;
      const int64_t per = (kbs + s - 1) / s, waves = (tiles * s + slots - 1) / slots;
      if (s > 1 && (kbs + per - 1) / per != s) continue;  // the last splits would be empty
      double cost = static_cast<double>(waves) * (static_cast<double>(per * terms) * step + over) + 3000.0;
      if (s > 1) cost += 4000.0 + static_cast<double>(s * M * N) * 8.0 / 2500.0;  // another launch; write and read of L2
      if (best_cost < 0.0 || cost < best_cost) {
        best_cost = cost;
        best.cg = cg;
        best.splits = s;
      }
    }
  }
  return best;
}

}  // namespace gemm

namespace rows {

namespace {

using namespace gemm;

constexpr int kMaxDevices = 64;
std::atomic<int> g_ready[kMaxDevices];  // 0 unknown, 1 ready, 2 unsupported
Device g_devices[kMaxDevices];
int* g_words[kMaxDevices];  // g_rows_status of each
std::map<cudaStream_t, int> g_word_of[kMaxDevices];  // g_mu
std::mutex g_mu;

}  // namespace

cudaError_t prepare_products();
cudaError_t prepare_xent();
cudaError_t prepare_gated();
cudaError_t prepare_q8();
cudaError_t prepare_distill();
cudaError_t prepare_norm();

int device(Device* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PK_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return PK_ERR_UNSUPPORTED;
  int state = g_ready[dev].load(std::memory_order_acquire);
  if (state == 0) {
    std::lock_guard<std::mutex> lock(g_mu);
    state = g_ready[dev].load(std::memory_order_acquire);
    if (state == 0) {
      int major = 0, minor = 0, sms = 0;
      if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
          cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PK_ERR_CUDA;
      if (major != 10 || minor != 3) {
        state = 2;
      } else {
        void* word = nullptr;
        if (cudaGetSymbolAddress(&word, g_rows_status) != cudaSuccess || prepare_products() != cudaSuccess ||
            prepare_xent() != cudaSuccess || prepare_gated() != cudaSuccess ||
            prepare_q8() != cudaSuccess || prepare_distill() != cudaSuccess ||
            prepare_norm() != cudaSuccess) {
          cudaGetLastError();
          return PK_ERR_CUDA;
        }
        g_devices[dev].index = dev;
        g_devices[dev].sms = sms;
        g_words[dev] = static_cast<int*>(word);
        state = 1;
      }
      g_ready[dev].store(state, std::memory_order_release);
    }
  }
  if (state == 2) return PK_ERR_UNSUPPORTED;
  *out = g_devices[dev];
  return PK_OK;
}

int* stream_status(const Device& d, cudaStream_t stream) {
  std::lock_guard<std::mutex> lock(g_mu);
  std::map<cudaStream_t, int>& words = g_word_of[d.index];
  const int next = static_cast<int>(words.size());
  return g_words[d.index] + words.emplace(stream, next < kStatusWords ? next : kStatusWords - 1).first->second;
}

// The stream's status word, read and cleared (the caller has synchronized the stream). Kernels write a word only while it is
// PK_OK, so what is cleared is what was read.
int take_status(int dev, cudaStream_t stream) {
  if (dev < 0 || dev >= kMaxDevices || g_ready[dev].load(std::memory_order_acquire) != 1) return PK_OK;
  int* word;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    const auto it = g_word_of[dev].find(stream);
    if (it == g_word_of[dev].end()) return PK_OK;
    word = g_words[dev] + it->second;
  }
  int st = 0, zero = 0;
  if (cudaMemcpy(&st, word, sizeof st, cudaMemcpyDeviceToHost) != cudaSuccess) return PK_ERR_CUDA;
  if (st != 0 && cudaMemcpy(word, &zero, sizeof zero, cudaMemcpyHostToDevice) != cudaSuccess) return PK_ERR_CUDA;
  return st;
}

// ------------------------------------------------------------------------------------
// operand copies

namespace {

struct CopyJobs {
  CopyJob job[2];
};

// One thread: 8 columns of a row. Bound by bytes: 2 or 4 read and 2 or 6 written an element.
template <int DT>
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ CopyJobs jobs) {
  const CopyJob& j = jobs.job[blockIdx.y];
  griddep_wait();
  int64_t live = j.rows, total = j.rows;
  if (j.count) {
    const int c = __ldcg(j.count);
    if (c == j.skip) return;
    live = c;
    total = min((live + 255) / 256 * 256, (j.rows + 255) / 256 * 256);
  }
  const int64_t groups = j.ldp / 8, n = total * groups;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = n < (int64_t(1) << 31) ? j.div.div(static_cast<uint32_t>(i)) : i / groups;
    const int c = static_cast<int>(i - r * groups) * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint4* d = reinterpret_cast<uint4*>(j.dst + r * j.ldp + c);
    if (r < live) {
      const int64_t s = (j.idx ? static_cast<int64_t>(__ldcg(j.idx + r)) : r) * j.ld + c;
      if constexpr (DT != PK_F32) {
        if (j.vec && c + 8 <= j.cols) {
          *d = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(j.src) + s));
          continue;
        }
      }
      if (j.vec && c + 8 <= j.cols)
        load8<DT>(j.src, s, v);
      else
        load8_any<DT>(j.src, s, j.cols - c, v);
    }
    if constexpr (DT == PK_F32) {
      uint32_t h[3][4];
      planes8(v, h);
#pragma unroll
      for (int k = 0; k < 3; ++k)
        *reinterpret_cast<uint4*>(j.dst + k * j.plane + r * j.ldp + c) = make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
    } else {
      store8<DT>(j.dst, r * j.ldp + c, v);
    }
  }
}

}  // namespace

gemm::Operand operand(int dtype, const void* p, int64_t ld, int64_t nrows, int64_t cols, int mn) {
  gemm::Operand o;
  o.p = p;
  o.rows = nrows;
  o.cols = cols;
  o.ld = ld;
  o.plane = nrows * ld;
  o.bf16 = dtype != PK_F16;
  o.mn = mn;
  return o;
}
gemm::Operand operand_of_copy(int dtype, const void* copy, int64_t nrows, int64_t cols, int mn) {
  gemm::Operand o = operand(dtype, copy, copy_ld(cols), nrows, cols, mn);
  o.planes = dtype == PK_F32 ? 3 : 1;
  return o;
}

void Copies::add(const void* p, int64_t ld, int64_t nrows, int64_t cols, void* copy, const int* idx, const int* count,
                 int skip) {
  const int64_t ldp = copy_ld(cols);
  job[n++] = CopyJob{p,
                     ld,
                     nrows,
                     ldp,
                     nrows * ldp,
                     static_cast<uint16_t*>(copy),
                     static_cast<int>(cols),
                     rows16(p, ld, elem_bytes(dtype)),
                     FastDiv(static_cast<uint32_t>(ldp / 8)),
                     idx,
                     count,
                     skip};
}

cudaError_t Copies::launch(int sms, cudaStream_t stream) {
  if (n == 0) return cudaSuccess;
  CopyJobs jobs = {};
  int64_t most = 0;
  for (int i = 0; i < n; ++i) {
    jobs.job[i] = job[i];
    const int64_t m = job[i].rows * (job[i].ldp / 8);
    most = m > most ? m : most;
  }
  const int64_t blocks = most / 256 + 1, cap = static_cast<int64_t>(sms) * 8;
  Launch l(blocks < cap ? blocks : cap, 256, stream);
  l.cfg.gridDim.y = n;
  if (dtype == PK_F32) return cudaLaunchKernelEx(&l.cfg, pack_kernel<PK_F32>, jobs);
  if (dtype == PK_BF16) return cudaLaunchKernelEx(&l.cfg, pack_kernel<PK_BF16>, jobs);
  return cudaLaunchKernelEx(&l.cfg, pack_kernel<PK_F16>, jobs);
}

// ------------------------------------------------------------------------------------
// split partial sums

namespace {

// y = epilogue(sum over splits of part[s]), the splits added in order: the result does not depend on which finished first.
template <int ODT, int RDT>
__global__ void __launch_bounds__(256) splits_kernel(const float* part, int cg, int64_t ldp, FastDiv groups,
                                                     const __grid_constant__ gemm::Args a, const __grid_constant__ LinParams p) {
  griddep_wait();
  const int M = a.dyn && a.dyn_axis == 0 ? __ldcg(a.dyn) : a.M;
  const int splits = cg == 2 ? gemm::choose_splits<2>(a, M) : gemm::choose_splits<1>(a, M);
  const int64_t stride = gemm::split_rows(M) * ldp, n = M * static_cast<int64_t>(groups.d);
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t r = n < (int64_t(1) << 31) ? groups.div(static_cast<uint32_t>(i)) : i / groups.d;
    const int c = static_cast<int>(i - r * groups.d) * 8;
    const float* at = part + r * ldp + c;
    float v[8];
    load8<PK_F32>(at, 0, v);
#pragma unroll 4
    for (int s = 1; s < splits; ++s) {
      float b[8];
      load8<PK_F32>(at, s * stride, b);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += b[j];
    }
    finish8<ODT, RDT>(p, v, r, c, a.N - c);
  }
}

template <int DT>
__global__ void __launch_bounds__(256) sum_rows_kernel(const float* part, int64_t nrows, const int* count, int per, int cols,
                                                       int64_t ld, const float* alpha, void* out) {
  // eight threads a column, each a strided eighth of the rows, joined in a fixed order
  __shared__ float s[8][33];
  griddep_wait();
  const int c = blockIdx.x * 32 + threadIdx.x % 32, g = threadIdx.x / 32;
  if (count) nrows = min(nrows, static_cast<int64_t>((__ldcg(count) + per - 1) / per));
  float v = 0.0f;
  if (c < cols)
#pragma unroll 8
    for (int64_t r = g; r < nrows; r += 8) v += __ldcg(part + r * ld + c);
  s[g][threadIdx.x % 32] = v;
  __syncthreads();
  if (g == 0 && c < cols) {
    for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x];
    Ty<DT>::put(out, c, alpha ? v * __ldcg(alpha) : v);
  }
}

}  // namespace

cudaError_t sum_rows(int dtype, const float* part, int64_t nrows, const int* count, int per, int cols, int64_t ld,
                     const float* alpha, void* out, cudaStream_t stream) {
  Launch l((cols + 31) / 32, 256, stream);
  const auto run = [&](auto kernel) { return cudaLaunchKernelEx(&l.cfg, kernel, part, nrows, count, per, cols, ld, alpha, out); };
  if (dtype == PK_F32) return run(sum_rows_kernel<PK_F32>);
  if (dtype == PK_BF16) return run(sum_rows_kernel<PK_BF16>);
  return run(sum_rows_kernel<PK_F16>);
}

// ------------------------------------------------------------------------------------
// products

cudaError_t prepare_products() {
  cudaError_t e;
  if ((e = gemm::prepare<LinEpi<PK_F32, PK_F32>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<LinEpi<PK_BF16, PK_BF16>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<LinEpi<PK_F16, PK_F16>>()) != cudaSuccess) return e;
  if ((e = gemm::prepare<LinEpi<PK_BF16, PK_F32>>()) != cudaSuccess) return e;
  return gemm::prepare<LinEpi<PK_F16, PK_F32>>();
}

cudaError_t partial_sums(const gemm::Operand& A, const gemm::Operand& B, const gemm::Operand* alt, gemm::Args a, gemm::Shape s,
                         float* partial, int64_t part_rows, int sms, cudaStream_t stream) {
  LinTiles part = {};
  part.y = partial;
  part.ldy = round_up(a.N, 8);
  part.tma_y = 1;
  a.part_rows = static_cast<int>(part_rows);
  if (!gemm::make_out_map(&part.map_y, PK_F32, partial, part_rows, a.N, part.ldy, 1, 0)) return cudaErrorInvalidValue;
  return gemm::launch<LinEpi<PK_F32, PK_F32>>(A, B, alt, a, part, s, sms, stream);
}

cudaError_t product(int dtype, int rdtype, const gemm::Operand& A, const gemm::Operand& B, const gemm::Operand* alt,
                    gemm::Args a, LinParams ep, gemm::Shape s, float* partial, int64_t part_rows, int sms, cudaStream_t stream) {
  const int e = elem_bytes(dtype);
  ep.bias_vec = ep.bias && aligned_to(ep.bias, 16);
  ep.res_vec = ep.res && rows16(ep.res, ep.ldres, elem_bytes(rdtype));
  ep.pre_vec = ep.pre && rows16(ep.pre, ep.ldpre, e);
  ep.y_vec = rows16(ep.y, ep.ldy, e);
  if (s.splits > 1) {
    const cudaError_t r = partial_sums(A, B, alt, a, s, partial, part_rows, sms, stream);
    if (r != cudaSuccess) return r;
    a.part_rows = static_cast<int>(part_rows);
    a.terms = A.planes == 3 ? gemm::kTerms32 : 1;  // what the launch above told the product
    a.splits = s.splits;
    a.slots = sms / s.cg;
    const int64_t ldp = round_up(a.N, 8), n = a.M * (ldp / 8), most = static_cast<int64_t>(sms) * 8;
    Launch l(n / 256 + 1 < most ? n / 256 + 1 : most, 256, stream);
    const float* cp = partial;
    const FastDiv groups(static_cast<uint32_t>(ldp / 8));
    auto run = [&](auto kernel) { return cudaLaunchKernelEx(&l.cfg, kernel, cp, s.cg, ldp, groups, a, ep); };
    if (dtype == PK_F32) return run(splits_kernel<PK_F32, PK_F32>);
    if (dtype == PK_BF16) return run(rdtype == PK_F32 ? splits_kernel<PK_BF16, PK_F32> : splits_kernel<PK_BF16, PK_BF16>);
    return run(rdtype == PK_F32 ? splits_kernel<PK_F16, PK_F32> : splits_kernel<PK_F16, PK_F16>);
  }
  LinTiles t = {};
  static_cast<LinParams&>(t) = ep;
  // (a TMA store clips a row's end to whole 16 bytes only: where the rows of y end inside one and go on in a wider matrix, the
  // warps store the last columns themselves)
  t.tma_y = ep.y_vec && !ep.rowmap && (a.N * e & 15) == 0;
  t.tma_pre = ep.pre_vec;
  if ((t.tma_y && !gemm::make_out_map(&t.map_y, dtype, ep.y, a.M, a.N, ep.ldy, 1, 0)) ||
      (t.tma_pre && !gemm::make_out_map(&t.map_pre, dtype, ep.pre, a.M, a.N, ep.ldpre, 1, 0)))
    return cudaErrorInvalidValue;
  if (dtype == PK_F32) return gemm::launch<LinEpi<PK_F32, PK_F32>>(A, B, alt, a, t, s, sms, stream);
  if (dtype == PK_BF16)
    return rdtype == PK_F32 ? gemm::launch<LinEpi<PK_BF16, PK_F32>>(A, B, alt, a, t, s, sms, stream)
                            : gemm::launch<LinEpi<PK_BF16, PK_BF16>>(A, B, alt, a, t, s, sms, stream);
  return rdtype == PK_F32 ? gemm::launch<LinEpi<PK_F16, PK_F32>>(A, B, alt, a, t, s, sms, stream)
                          : gemm::launch<LinEpi<PK_F16, PK_F16>>(A, B, alt, a, t, s, sms, stream);
}

}  // namespace rows
}  // namespace pk
