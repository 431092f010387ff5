// pk_gemm.cuh -- the tensor-core matrix product shared by the projection and the vocabulary cross entropy (sm_103a):
//     D[m, n] = sum_k A(m, k) B(n, k),   then an epilogue on the fp32 accumulators.
//
// Operands are 16-bit (bf16 or fp16, accumulated in fp32) and may lie either way round in memory: K-major ([rows, K]) or
// MN-major ([K, rows]), so that a projection's product (x W^T) and both of its gradients (dz W, dz^T x) read the stored
// tensors without a transposed copy. An fp32 operand comes as three planes of bf16 (x = hi + mid + lo, 24 significant
// bits); the product is then six passes over k, one per pair of planes whose product is not below 2^-24 of the whole,
// the smallest first so that they are not lost beside the large ones.
//
// Tile and roles: a pair of CTAs (cta_group::2) owns 256 x 256 of D -- each holds 128 rows of A and 128 of B per 64-wide
// k step, so a k step moves 64 KB for 256 * 256 * 64 products -- or, where that leaves SMs idle, one CTA owns 128 x 128.
// Both use the same shared memory: six stages of 16 + 16 KB filled by TMA (128-byte swizzle) and 32 KB for the epilogue's
// warps. Warp 0 loads, warp 1 of the leader issues the MMAs, warps from 4 on empty the accumulators; two accumulators
// in tensor memory let the epilogue of one tile run under the products of the next. Persistent: a grid of one CTA per SM
// walks the work units (output tile x split of k) in a fixed order, tiles grouped so that concurrent units share
// operands in L2. A split of k writes fp32 partial sums, added in a fixed order afterwards.
//
// Every wait is bounded: one that runs out records PK_ERR_TIMEOUT, raises the CTA's abort flag, and the roles leave.
#pragma once

#include <type_traits>

#include "pk_attn_common.cuh"

namespace pk {
namespace gemm {

// What an epilogue may ask of the product besides its own part:
//   kPair   B's rows are two halves of N / 2 (a gate and what it multiplies). A tile then holds the same 64 or 128 columns of
//           both, the first half's in the accumulator's first half, so that the epilogue finds the two side by side.
//   kBytes  the operands are e4m3, two elements in the place of one: every size along k is counted in such pairs.
template <class Epi, class = void>
struct IsPair : std::false_type {};
template <class Epi>
struct IsPair<Epi, std::void_t<decltype(Epi::kPair)>> : std::bool_constant<Epi::kPair> {};
template <class Epi, class = void>
struct IsBytes : std::false_type {};
template <class Epi>
struct IsBytes<Epi, std::void_t<decltype(Epi::kBytes)>> : std::bool_constant<Epi::kBytes> {};

constexpr int kStages = 6;
constexpr int kBK = 64;                       // k step: 128 bytes, one swizzle row
constexpr int kEpiWarp0 = 4;                  // warps 0-3: load, issue, allocate; then Epi::kWarps (8 or 16) of the epilogue
constexpr uint32_t kOpBytes = 128 * 128;      // one operand's share of a stage: 128 rows x 64 elements
constexpr uint32_t kStageBytes = 2 * kOpBytes;
constexpr uint32_t kEpiBytes = 32 * 1024;     // staging of the epilogue's warps
constexpr uint32_t kOffEpi = kStages * kStageBytes;
constexpr uint32_t kOffMeta = kOffEpi + kEpiBytes;
constexpr int kTerms32 = 6;                   // plane pairs of an fp32 product
constexpr int kGroupM = 8;                    // tile rows walked together
// The tensor pipe truncates when it adds to an accumulator, so a long sum drifts towards zero by some 2^-25 of itself a step
// of 16: 8e-5 over 100000 terms, where fp32 allows 1e-5 and a rounding to fp16 costs 2e-4. At most this many k steps add
// up there before the epilogue's warps take the sum over, rounding to nearest, into the other accumulator's tensor memory:
// 1024 terms of fp32 operands (the drift stays below 2e-6), 16384 of 16-bit ones (3e-5; a hand-over costs some 2000
// cycles of 131000), 32768 of 8-bit ones, whose steps are of 32 (2048 where their result is fp32).
constexpr int kPhase32 = 16;
constexpr int kPhase16 = 256;

struct Meta {
  uint64_t full[kStages], empty[kStages];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem;
  int32_t abort;
};
constexpr uint32_t kSmemUsed = kOffMeta + sizeof(Meta);
constexpr uint32_t kSmemBytes = kSmemUsed + 1024;  // the dynamic base is aligned up to 1024
static_assert(kSmemBytes <= 227u * 1024u, "fits the 227 KB a block may use");

// Arguments of one product.
struct Args {
  int M, N, K;      // K in elements of one plane
  int a_mn, b_mn;   // operand layouts (0: K-major, 1: MN-major)
  int bf16;
  int phase;        // 0, or the most k steps that the tensor pipe may add up by itself
  int terms;        // 1, or kTerms32
  int splits;       // splits of k (with a device count of rows: the most that the device may choose)
  int part_rows;    // with a device count of rows: rows of the partial sums' memory
  int slots;        // tiles that run at the same time
  const int* dyn;   // when not null, a device count that replaces M (dyn_axis 0) or K (dyn_axis 1)
  int dyn_axis;
  int alt_count;    // when dyn is not null and *dyn equals this, the alternative map replaces the operand below
  int alt_operand;  // 0: A, 1: B
  int* status;
  unsigned long long timeout_ns;
  int skip_first_arrive;  // test hook (PK_DEBUG_SKIP_ARRIVE=1): the loading warp withholds its first arrival
};

// One unit of work: an output tile and its range of k steps.
struct Unit {
  int m0, n0;    // first row and column of the tile
  int kb0, kbs;  // k steps
  int split;
};

struct Plan {
  int M, N, tiles_m, tiles_n, kb_all, kb_per, units, splits;
  int phase;   // k steps that the tensor pipe adds up by itself
  bool phased; // more than one phase a unit: accumulator 0 only, sums in accumulator 1's place
};

// Rows between the partial sums of two splits.
__device__ __forceinline__ int split_rows(int M) { return (M + 255) & ~255; }

// The splits of k for a count of rows that only the device knows: the fewest waves x steps, the host's model on the device.
template <int CG>
__device__ __forceinline__ int choose_splits(const Args& a, int M) {
  if (!a.dyn || a.dyn_axis != 0 || a.splits == 1) return a.splits;
  constexpr int kTile = 128 * CG;
  const int tiles = ((M + kTile - 1) / kTile) * ((a.N + kTile - 1) / kTile), kbs = (a.K + kBK - 1) / kBK;
  int best = 1, best_cost = 0x7fffffff;
  for (int s = 1; s <= a.splits && s * split_rows(M) <= a.part_rows; ++s) {
    const int cost = (tiles * s + a.slots - 1) / a.slots * ((kbs + s - 1) / s * a.terms + 4) + s;
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

template <int CG>
__device__ __forceinline__ Plan make_plan(const Args& a) {
  Plan p;
  p.M = a.M;
  p.N = a.N;
  int K = a.K;
  if (a.dyn) {
    const int c = __ldcg(a.dyn);
    if (a.dyn_axis == 0)
      p.M = c;
    else
      K = c;
  }
  constexpr int kTile = 128 * CG;
  p.tiles_m = (p.M + kTile - 1) / kTile;
  p.tiles_n = (p.N + kTile - 1) / kTile;
  p.kb_all = (K + kBK - 1) / kBK;
  p.splits = choose_splits<CG>(a, p.M);
  p.kb_per = (p.kb_all + p.splits - 1) / p.splits;
  p.units = p.tiles_m * p.tiles_n * p.splits;
  const int most = a.phase > 0 ? a.phase : a.terms > 1 ? kPhase32 : kPhase16;
  p.phased = p.kb_per > most;
  p.phase = p.phased ? most : p.kb_per;
  return p;
}

template <int CG>
__device__ __forceinline__ Unit unit_at(const Plan& p, int u) {
  const int tiles = p.tiles_m * p.tiles_n;
  Unit t;
  t.split = u / tiles;
  int r = u - t.split * tiles;
  const int per_group = kGroupM * p.tiles_n;
  const int g = r / per_group;
  r -= g * per_group;
  const int gm = min(kGroupM, p.tiles_m - g * kGroupM);
  t.m0 = (g * kGroupM + r % gm) * 128 * CG;
  t.n0 = (r / gm) * 128 * CG;
  t.kb0 = t.split * p.kb_per;
  t.kbs = max(0, min(p.kb_per, p.kb_all - t.kb0));
  return t;
}

// planes of term i: A's in the low half, B's in the high half; the smallest products first
__device__ __forceinline__ int term_a(int terms, int i) { return terms == 1 ? 0 : (0x001102 >> (4 * i)) & 15; }
__device__ __forceinline__ int term_b(int terms, int i) { return terms == 1 ? 0 : (0x010120 >> (4 * i)) & 15; }

// ------------------------------------------------------------------------------------
// PTX of the CTA pair

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // (a warp arrives as one, and what stands before may have been one lane's)
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  // (no cluster-wide release: what it hands back is tensor memory, ordered by the tcgen05 fences)
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// 3-D tile load at (x, y, plane); `bar` is a shared::cluster address (the leader's barrier for a pair)
template <int CG>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
template <int CG, bool kBytes>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  // (a step of 32 bytes along k either way: 16 elements or 32)
  if constexpr (kBytes && CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else if constexpr (kBytes)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    umma_f16_ss(d, a, b, idesc, accumulate);
}
// arrive on `bar` (in both CTAs of a pair, at the same offset) once the MMAs issued so far have completed
template <int CG>
__device__ __forceinline__ void commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
  else
    umma_commit(bar);
}
template <int CG>
__device__ __forceinline__ void alloc_tmem(uint32_t dst) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(dst) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst, 512);
    tmem_relinquish();
  }
}
template <int CG>
__device__ __forceinline__ void free_tmem(uint32_t t) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
  else
    tmem_dealloc(t, 512);
}

// Bounded wait; false once the CTA gave up or after the time limit (which makes it give up). What these barriers guard is
// written by TMA, the tensor pipe or to tensor memory: no acquire wider than the CTA, which would invalidate L1 each time.
__device__ __forceinline__ bool wait(Meta* m, const Args& a, uint64_t* bar, uint32_t parity) {
  const uint32_t addr = smem_u32(bar);
  if (mbar_try_wait(addr, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(addr, parity)) return true;
    if ((i & 15u) == 0u) {
      if (attn::aborted(&m->abort)) return false;
      if (globaltimer_ns() - t0 > a.timeout_ns) {
        *reinterpret_cast<volatile int32_t*>(&m->abort) = 1;
        if (a.status) atomicCAS(a.status, 0, kErrTimeout);
        return false;
      }
    }
  }
}

// One lane of a converged warp. The loops of the loading and the issuing warp are run by all 32 lanes, with only the TMA and
// MMA instructions under this: the compiler then sees loop counters and descriptors as the same in every lane and keeps
// them in the uniform registers that those instructions take. (One lane in a divergent branch spent some 60 cycles an MMA
// moving operands over, 700 a k step where the tensor pipe needs 512.)
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)::"memory");
  return ok != 0;
}
// (a warp goes on or gives up as one)
__device__ __forceinline__ bool wait_warp(Meta* m, const Args& a, uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(m, a, bar, parity));
}

// ------------------------------------------------------------------------------------
// roles

template <int CG, bool kPair>
__device__ __forceinline__ void produce(const CUtensorMap* ma, const CUtensorMap* mb, const Args& a, const Plan& p,
                                        uint8_t* smem, Meta* meta, uint32_t rank, int unit0, int unit_step) {
  uint32_t st = 0, ph = 0;
  bool bad = false, withhold = a.skip_first_arrive != 0;
  uint32_t full0 = smem_u32(&meta->full[0]);
  if constexpr (CG == 2) full0 = mapa(full0, 0);
  for (int u = unit0; u < p.units && !bad; u += unit_step) {
    const Unit t = unit_at<CG>(p, u);
    const int ra = t.m0 + 128 * static_cast<int>(rank), rb = t.n0 + 128 * static_cast<int>(rank);
    const int end = t.kb0 + t.kbs;
    // the passes of one phase, then the next phase's (`kb` runs over a phase `terms` times)
    for (int k0 = t.kb0, term = 0; k0 < end && !bad;) {
      const int pa = term_a(a.terms, term), pb = term_b(a.terms, term);
      for (int kb = k0; kb < min(k0 + p.phase, end); ++kb) {
        if (!wait_warp(meta, a, &meta->empty[st], ph ^ 1u)) {
          bad = true;
          break;
        }
        const uint32_t bar = full0 + 8 * st;
        const uint32_t sa = smem_u32(smem + st * kStageBytes), sb = sa + kOpBytes;
        const int k = kb * kBK;
        if (elect_one()) {
          if (rank == 0 && !withhold) mbar_arrive_expect_tx(smem_u32(&meta->full[st]), CG * kStageBytes);
          if (a.a_mn) {
            tma_load_3d<CG>(sa, ma, bar, ra, k, pa);
            tma_load_3d<CG>(sa + kOpBytes / 2, ma, bar, ra + 64, k, pa);
          } else {
            tma_load_3d<CG>(sa, ma, bar, k, ra, pa);
          }
          if constexpr (kPair) {
            // (the pair's second CTA holds the second half's rows, a lone CTA 64 of each)
            const int f = t.n0 / 2, half = p.N / 2;
            if constexpr (CG == 2) {
              tma_load_3d<CG>(sb, mb, bar, k, f + static_cast<int>(rank) * half, pb);
            } else {
              tma_load_3d<CG>(sb, mb, bar, k, f, pb);
              tma_load_3d<CG>(sb + kOpBytes / 2, mb, bar, k, f + half, pb);
            }
          } else if (a.b_mn) {
            tma_load_3d<CG>(sb, mb, bar, rb, k, pb);
            tma_load_3d<CG>(sb + kOpBytes / 2, mb, bar, rb + 64, k, pb);
          } else {
            tma_load_3d<CG>(sb, mb, bar, k, rb, pb);
          }
        }
        withhold = false;
        __syncwarp();
        st = st + 1 == kStages ? 0 : st + 1;
        ph ^= st == 0 ? 1u : 0u;
      }
      if (++term == a.terms) {
        term = 0;
        k0 += p.phase;
      }
    }
  }
  // every stage released before leaving (one never filled counts as released): no copy and no arrival is on its way to
  // this CTA any more. After giving up, one wait bound for all of them together: nobody releases a stage that was filled, and
  // its copies have landed long before.
  uint64_t t0 = 0;
  for (int i = 0; i < kStages; ++i) {
    if (bad) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      mbar_wait(smem_u32(&meta->empty[st]), ph ^ 1u, now - t0 < a.timeout_ns ? a.timeout_ns - (now - t0) : 0);
    } else if (!wait_warp(meta, a, &meta->empty[st], ph ^ 1u)) {
      bad = true;
    }
    st = st + 1 == kStages ? 0 : st + 1;
    ph ^= st == 0 ? 1u : 0u;
  }
}

template <int CG, bool kBytes>
__device__ __forceinline__ void issue(const Args& a, const Plan& p, uint8_t* smem, Meta* meta, uint32_t tmem, int unit0,
                                      int unit_step) {
  const uint32_t idesc = idesc_f16(a.bf16 != 0, 128 * CG, 128 * CG, a.a_mn != 0, a.b_mn != 0);
  // K-major: 8-row groups 1024 bytes apart, a k step of 16 is 32 bytes along the swizzled row. MN-major: 64-wide blocks
  // 8192 bytes apart, 8-deep k groups 1024 bytes apart, a k step of 16 is 2048 bytes.
  const uint64_t da = sdesc_sw128(smem_u32(smem), a.a_mn ? kOpBytes / 2 : 16, 1024);
  const uint64_t db = sdesc_sw128(smem_u32(smem) + kOpBytes, a.b_mn ? kOpBytes / 2 : 16, 1024);
  const uint32_t sa = a.a_mn ? 128 : 2, sb = a.b_mn ? 128 : 2;
  uint32_t st = 0, ph = 0, n = 0;
  bool ok = true;
  for (int u = unit0; u < p.units && ok; u += unit_step) {
    const Unit t = unit_at<CG>(p, u);
    // (an empty split issues nothing: the epilogue takes zeros)
    for (int k0 = 0; k0 < t.kbs && ok; k0 += p.phase) {
      const int steps = min(p.phase, t.kbs - k0) * a.terms;
      const uint32_t buf = p.phased ? 0u : n & 1u, use = p.phased ? n : n >> 1;
      if (!(ok = wait_warp(meta, a, &meta->acc_empty[buf], (use & 1u) ^ 1u))) break;
      tc_fence_after();
      const uint32_t d = tmem + buf * 256;
      for (int i = 0; i < steps; ++i) {
        if (!(ok = wait_warp(meta, a, &meta->full[st], ph))) break;
        tc_fence_after();
        const uint64_t xa = da + st * (kStageBytes >> 4), xb = db + st * (kStageBytes >> 4);
        if (elect_one()) {
#pragma unroll
          for (uint32_t k = 0; k < kBK / 16; ++k) mma<CG, kBytes>(d, xa + k * sa, xb + k * sb, idesc, (i | k) != 0 ? 1u : 0u);
          commit<CG>(smem_u32(&meta->empty[st]));
          if (i + 1 == steps) commit<CG>(smem_u32(&meta->acc_full[buf]));
        }
        __syncwarp();
        st = st + 1 == kStages ? 0 : st + 1;
        ph ^= st == 0 ? 1u : 0u;
      }
      ++n;
    }
  }
  if (!ok) {
    // gave up: the MMAs in flight end before the tensor memory is freed
    if (elect_one()) commit<CG>(smem_u32(&meta->drain));
    __syncwarp();
    mbar_wait(smem_u32(&meta->drain), 0, a.timeout_ns);
  }
}

// The `kCols` columns of a finished phase (accumulator 0) added to the sums 256 columns further, or put there.
template <int kCols>
__device__ __forceinline__ void add_phase(uint32_t acc, bool first) {
#pragma unroll 1
  for (int c = 0; c < kCols; c += 32) {
    float v[32];
    tmem_ld32(acc + c, v);
    if (!first) {
      float sum[32];
      tmem_ld32(acc + 256 + c, sum);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += sum[i];
    }
    uint32_t w[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(v[i]);
    tmem_st32(acc + 256 + c, w);
  }
  tmem_wait_st();
}

// Epi: struct with kWarps, perhaps kPair and kBytes, and `static __device__ bool run(const Params&, tmem address of the warp's lanes and first column, zero (there
// are no accumulators: take zeros), first row, first column, columns, M, N, split, lane, staging, ready, done)`, called by
// 32 lanes together; it calls ready() before it reads accumulators and done() once after the last of them, and
// returns false when ready() did. With kPair: the addresses of both accumulators, and the columns of a half.
template <int CG, class Epi>
__global__ void __launch_bounds__(32 * (kEpiWarp0 + Epi::kWarps), 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_alt, const __grid_constant__ Args a,
                const __grid_constant__ typename Epi::Params ep) {
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Meta* meta = reinterpret_cast<Meta*>(smem + kOffMeta);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0u;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&meta->full[i]), 1);
      mbar_init(smem_u32(&meta->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&meta->acc_full[i]), 1);
      mbar_init(smem_u32(&meta->acc_empty[i]), CG * Epi::kWarps);
    }
    mbar_init(smem_u32(&meta->drain), 1);
    meta->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&map_a);
    tma_prefetch_desc(&map_b);
  }
  if (warp == 2) alloc_tmem<CG>(smem_u32(&meta->tmem));
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, meta->tmem, 0);
  griddep_wait();  // the previous kernel's results (operands, counts) from here on
  const Plan p = make_plan<CG>(a);
  const int unit0 = blockIdx.x / CG, unit_step = gridDim.x / CG;

  if (warp == 0) {
    const bool alt = a.dyn && __ldcg(a.dyn) == a.alt_count;
    const CUtensorMap* ma = alt && a.alt_operand == 0 ? &map_alt : &map_a;
    const CUtensorMap* mb = alt && a.alt_operand == 1 ? &map_alt : &map_b;
    // operands that an earlier kernel wrote with ordinary stores, before TMA reads them
    asm volatile("fence.proxy.async.global;" ::: "memory");
    produce<CG, IsPair<Epi>::value>(ma, mb, a, p, smem, meta, rank, unit0, unit_step);
  } else if (warp == 1) {
    if (rank == 0) issue<CG, IsBytes<Epi>::value>(a, p, smem, meta, tmem, unit0, unit_step);
  } else if (warp >= kEpiWarp0) {
    const int w = warp - kEpiWarp0, quarter = w & 3, part = w >> 2;
    // columns a warp empties: its share of the tile's; of a pair's two halves each, 32 at least, so that of a lone CTA's 64 two
    // warps of a quarter have some
    constexpr bool kPair = IsPair<Epi>::value;
    constexpr int kEven = 128 * CG / (kPair ? 2 : 1) / (Epi::kWarps / 4), kCols = kEven < 32 ? 32 : kEven;
    constexpr int kHalf = 64 * CG;  // columns between a pair's two accumulators
    const bool idle = kPair && part * kCols >= kHalf;
    uint8_t* stage = smem + kOffEpi + w * (kEpiBytes / Epi::kWarps);
    uint32_t n = 0;
    uint32_t empty0 = smem_u32(&meta->acc_empty[0]);
    if constexpr (CG == 2) empty0 = mapa(empty0, 0);
    for (int u = unit0; u < p.units; u += unit_step) {
      const Unit t = unit_at<CG>(p, u);
      const bool zero = t.kbs == 0;
      const uint32_t buf = p.phased ? 0u : n & 1u;
      const uint32_t acc = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + part * kCols;
      // (the warp goes on or leaves as one: the accumulator loads are warp-wide)
      const auto full = [&]() {
        if (!wait_warp(meta, a, &meta->acc_full[buf], (p.phased ? n : n >> 1) & 1u)) return false;
        tc_fence_after();
        return true;
      };
      const auto empty = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2)
            mbar_arrive_cluster(empty0 + 8 * buf);
          else
            mbar_arrive(smem_u32(&meta->acc_empty[buf]));
        }
      };
      bool ok = true;
      if (p.phased) {
        // each phase's sums onto those of the phases before, in accumulator 1's place
        for (int k0 = 0; k0 < t.kbs && (ok = full()); k0 += p.phase) {
          if (!idle) {
            add_phase<kCols>(acc, k0 == 0);
            if constexpr (kPair) add_phase<kCols>(acc + kHalf, k0 == 0);
          }
          empty();
          ++n;
        }
      }
      const auto ready = [&]() { return zero || p.phased || full(); };
      const auto done = [&]() {
        if (!zero && !p.phased) empty();
      };
      if (kPair && idle) {
        if (!ok || !ready()) break;
        done();
        if (!zero && !p.phased) ++n;
        continue;
      }
      const uint32_t sums = acc + (p.phased ? 256 : buf * 256);
      const int row = t.m0 + 128 * static_cast<int>(rank) + 32 * quarter, col = (kPair ? t.n0 / 2 : t.n0) + part * kCols;
      if constexpr (kPair)
        ok = ok && Epi::run(ep, sums, sums + kHalf, zero, row, col, kCols, p.M, p.N / 2, t.split, lane, stage, ready, done);
      else
        ok = ok && Epi::run(ep, sums, zero, row, col, kCols, p.M, p.N, t.split, lane, stage, ready, done);
      if (!ok) break;
      if (!zero && !p.phased) ++n;
    }
    // copies in flight (a warp that gave up) land, and tiles stored by TMA are written, before the CTA leaves
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  if (warp == 2) free_tmem<CG>(tmem);
}

// ------------------------------------------------------------------------------------
// host

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();
int debug_skip_arrive();  // PK_DEBUG_SKIP_ARRIVE, read at every call

// A 16-bit operand as the product reads it: `rows` x `cols` with cols contiguous, `ld` elements apart, `planes` of them
// `plane` elements apart. Base 16-byte aligned, ld and plane multiples of 8.
struct Operand {
  const void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0, plane = 0;
  int planes = 1;
  int bf16 = 1;
  int mn = 0;  // 0: rows are the product's m or n, cols its k; 1: rows are its k
  int box = 128;  // rows of a tile, where they are not its k
};
inline bool operand_ok(const Operand& o) {
  return (reinterpret_cast<uintptr_t>(o.p) & 15) == 0 && (o.ld & 7) == 0 && (o.plane & 7) == 0;
}
bool make_map(CUtensorMap* map, const Operand& o);
// The map of an output of type dtype (enum pk_dtype) as the epilogue's warps store it: 32 rows x 32 columns a box.
bool make_out_map(CUtensorMap* map, int dtype, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t planes,
                  int64_t plane);

// How a product of these sizes is cut up.
struct Shape {
  int cg = 2;
  int splits = 1;
};
Shape pick_shape(int64_t M, int64_t N, int64_t K, int terms, int sms, bool may_split);

template <class Epi>
cudaError_t prepare() {
  cudaError_t e = cudaFuncSetAttribute(gemm_kernel<1, Epi>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(gemm_kernel<2, Epi>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
}

// One product. `alt`: the operand that replaces A or B (a.alt_operand) when *a.dyn == a.alt_count, or null.
template <class Epi>
cudaError_t launch(const Operand& A, const Operand& B, const Operand* alt, Args a, const typename Epi::Params& ep, Shape s,
                   int sms, cudaStream_t stream) {
  CUtensorMap ma, mb, mc;
  Operand second = B;
  if (IsPair<Epi>::value && s.cg == 1) second.box = 64;
  if (!make_map(&ma, A) || !make_map(&mb, second)) return cudaErrorInvalidValue;
  mc = ma;
  if (alt) {
    if (!make_map(&mc, *alt)) return cudaErrorInvalidValue;
  } else {
    a.alt_count = -1;
  }
  a.a_mn = A.mn;
  a.b_mn = B.mn;
  a.bf16 = A.bf16;
  a.terms = A.planes == 3 ? kTerms32 : 1;
  a.splits = s.splits;
  a.slots = sms / s.cg;
  a.skip_first_arrive = debug_skip_arrive();
  const int64_t tile = 128 * s.cg;
  const int64_t units = ((a.M + tile - 1) / tile) * ((a.N + tile - 1) / tile) * s.splits;
  int64_t ctas = units < sms / s.cg ? units : sms / s.cg;
  ctas *= s.cg;
  if (ctas <= 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned int>(ctas));
  cfg.blockDim = dim3(32 * (kEpiWarp0 + Epi::kWarps));
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = s.cg;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return s.cg == 2 ? cudaLaunchKernelEx(&cfg, gemm_kernel<2, Epi>, ma, mb, mc, a, ep)
                   : cudaLaunchKernelEx(&cfg, gemm_kernel<1, Epi>, ma, mb, mc, a, ep);
}

}  // namespace gemm
}  // namespace pk
