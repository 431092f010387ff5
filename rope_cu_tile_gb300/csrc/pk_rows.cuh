// pk_rows.cuh -- host side shared by the token-row operators (pk_linear.cu, pk_dropout.cu, pk_xent.cu): the device check,
// the status word, scratch carving, and the passes that lay an operand out for the tensor-core product.
#pragma once

#include "pk_epilogue.cuh"

namespace pk {

unsigned long long wait_limit_ns();  // pk_host.cu: the bound of a pipeline wait

namespace rows {

struct Device {
  int index = 0;
  int sms = 0;
};
// the current device, checked and set up once (PK_OK or an error code)
int device(Device* out);
// the stream's status word, for a call that is given none: read by pk_last_status
int* stream_status(const Device& d, cudaStream_t stream);

// Carves 256-byte-aligned pieces out of a caller's workspace; with a null base it only adds up the bytes.
struct Carver {
  char* base;
  int64_t used = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  void* take(int64_t bytes) {
    void* p = base ? base + used : nullptr;
    used += (bytes + 255) & ~int64_t(255);
    return p;
  }
};

inline int64_t round_up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline int elem_bytes(int dtype) { return dtype == PK_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == PK_F32 || dtype == PK_BF16 || dtype == PK_F16; }

// Whether a [rows, cols] matrix can be read by TMA where it lies, and the bytes of the copy that is made otherwise
// (fp32: three bf16 planes; 16-bit with rows off the 16-byte grid: one padded plane).
inline bool in_place(int dtype, const void* p, int64_t ld) {
  return dtype != PK_F32 && aligned_to(p, 16) && (ld & 7) == 0;
}
inline int64_t copy_ld(int64_t cols) { return round_up(cols, 8); }
inline int64_t copy_bytes(int dtype, int64_t rows, int64_t cols) {
  return (dtype == PK_F32 ? 3 : 1) * rows * copy_ld(cols) * 2;
}
// The operand for p itself, and for its copy.
gemm::Operand operand(int dtype, const void* p, int64_t ld, int64_t rows, int64_t cols, int mn);
gemm::Operand operand_of_copy(int dtype, const void* copy, int64_t rows, int64_t cols, int mn);

// n / d and n % d for n < 2^31 by a multiplication (d >= 1): with s = ceil(log2 d) and m = ceil(2^(31 + s) / d), m fits 32
// bits and m n / 2^(31 + s) exceeds n / d by less than 1 / d.
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() : FastDiv(1) {}
  explicit FastDiv(uint32_t divisor) : d(divisor), m(0), s(0) {
    while ((uint64_t(1) << s) < d) ++s;
    m = static_cast<uint32_t>(((uint64_t(1) << (31 + s)) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * m) >> (31 + s));
  }
};

// Up to two operand copies in one launch (none: no launch).
struct CopyJob {
  const void* src;
  int64_t ld, rows, ldp, plane;
  uint16_t* dst;
  int cols, vec;
  FastDiv div;
  const int* idx;    // with idx: rows idx[0 .. *count) of src, then zeros up to a multiple of 256 rows; nothing when
  const int* count;  // *count == skip
  int skip;
};
struct Copies {
  int dtype, n = 0;
  CopyJob job[2];
  explicit Copies(int dt) : dtype(dt) {}
  void add(const void* p, int64_t ld, int64_t rows, int64_t cols, void* copy, const int* idx = nullptr,
           const int* count = nullptr, int skip = 0);
  cudaError_t launch(int sms, cudaStream_t stream);
};

// A product with the linear epilogue (type dtype out, residual of type rdtype), through split partial sums when s.splits
// > 1 (`partial`: `part_rows` rows of round_up(N, 8) floats, part_rows >= splits x round_up(M, 256); with a device count of
// rows the device takes as many splits, up to s.splits, as are worth it and have room).
cudaError_t product(int dtype, int rdtype, const gemm::Operand& A, const gemm::Operand& B, const gemm::Operand* alt,
                    gemm::Args a, LinParams ep, gemm::Shape s, float* partial, int64_t part_rows, int sms, cudaStream_t stream);
inline int64_t partial_rows(const gemm::Shape& s, int64_t M) { return s.splits > 1 ? s.splits * round_up(M, 256) : 0; }
inline int64_t partial_bytes(const gemm::Shape& s, int64_t M, int64_t N) { return partial_rows(s, M) * round_up(N, 8) * 4; }

// out[c] = sum over rows of part[r][c], in a fixed order; with `count`, only the first ceil(*count / per) rows
cudaError_t sum_rows(int dtype, const float* part, int64_t nrows, const int* count, int per, int cols, int64_t ld,
                     const float* alpha, void* out, cudaStream_t stream);

// launch attributes of a kernel that may start under the previous one's tail
struct Launch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  Launch(int64_t blocks, int threads, cudaStream_t stream) {
    cfg.gridDim = dim3(static_cast<unsigned int>(blocks));
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
};

}  // namespace rows
}  // namespace pk
