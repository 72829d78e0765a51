// Products of e4m3 operands with block scales, and products grouped by expert
// with ragged sizes, on the sm_103a tensor cores (tcgen05 + TMEM + TMA).
//
// Block scales. With one scale per row and 128 k of lhs and per 128 k x 128 n
// of rhs,
//   out[m, n] = sum_b sa[m, b] sb[b, n / 128] P_b[m, n],   P_b = the plain e4m3 product over block b.
// P_b is one k-block of tensor-core work; it is read back from TMEM and added
// to the fp32 sum in registers with one fused multiply-add per element, while
// the next block's product is under way in the other TMEM buffer.
//
// Ragged groups. Where each expert's rows begin is known on the device only.
// Work units are numbered expert by expert, and every warp finds its unit by
// itself: 32 lanes read 32 experts' offsets, a prefix sum over their tile counts
// and a ballot give the expert, so neither a table nor a launch per expert is
// needed and empty experts cost one lane of one read. Offsets that descend can number any amount of units: counts stop
// at what ascending ones can have, in every warp alike, so they neither pass 32 bits nor keep the kernel longer.
//
// k_grouped_pair (16-bit operands): CTA pairs, persistent, one tile of up to
// 256 x 256 per pair and step (tcgen05 cta_group::2: M = 256, N up to 256; each
// CTA holds 128 rows of A, half of B's and its 128 rows of the accumulator).
// In products A is the weights (256 of their columns n) and B an expert's rows:
// an MMA's N goes in steps of 32, so an expert's last tile costs what its rows
// cost and not 256 (32 experts of 126 to 4000 rows: a quarter of the work). In
// weight gradients A holds lhs columns, B rhs columns, and the rows are summed.
// 16384 rows over 32 uneven experts, k 4096, n 2048 in bf16: 187 us (1.47
// PFLOP/s), its weight gradient 204 us, of which storing 537 MB is a good part
// (64 rows an expert: 97 us); one expert of 16384 rows 145 and 155 us.
//   warp 0        TMA producer: k-blocks 128 bytes deep into a ring of 6 stages of 32 KB.
//   warp 1        issues the MMAs (CTA 0 of the pair) and owns TMEM.
//   warps 2, 3    in weight gradients: have zeros loaded over what a k-block holds of the next expert's rows.
//   warps 4..11   two per TMEM lane quarter, 128 columns each: conversion and stores.
// Every mbarrier wait is bounded by %globaltimer as in the other tensor-core
// kernels: on expiry COCO_ERR_TIMEOUT is recorded, the roles drain and return.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "internal.h"
#include "tc_ptx.h"

namespace coco {
namespace {

constexpr int BKB = 128;  // bytes of k per k-block: 128 e4m3 or 64 16-bit values
constexpr int TILE_M = 256, TILE_N = 256;
constexpr int A_BYTES = 128 * BKB, B_BYTES = 128 * BKB;  // one CTA's rows of A / columns of B
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int STAGES = 6;
constexpr int EPI_WARPS = 8, FIRST_EPI_WARP = 4;
constexpr int THREADS = 32 * (FIRST_EPI_WARP + EPI_WARPS);
constexpr int STRIP = 32 * 128;  // an epilogue warp's staging: 32 rows x 128 bytes
constexpr int STRIP_OFF = STAGES * STAGE_BYTES;
constexpr int BAR_OFF = STRIP_OFF + EPI_WARPS * STRIP;
// full, empty and loaded (before zeros) per stage, accumulator full x2, empty x2, drain
constexpr int NUM_BARS = 3 * STAGES + 5;
constexpr int SMEM_BYTES = BAR_OFF + 8 * NUM_BARS + 16 + 1024;  // + alignment slack
static_assert(SMEM_BYTES <= 232448, "shared memory over the per-CTA limit");
constexpr uint32_t TMEM_COLS = 512;
constexpr int GROUP_MT = 8;  // rasterisation: m-tiles per group, n-major inside a group

constexpr int kZeroMaps = 6;

struct GroupedParams {
  CUtensorMap a[COCO_MAX_PTRS], b[COCO_MAX_PTRS];
  CUtensorMap zero[kZeroMaps];  // weight gradients: boxes of 2^i rows of 128 bytes, unswizzled, read out of range
  void* out[COCO_MAX_PTRS];
  const float* sa[COCO_MAX_PTRS];
  const float* sb[COCO_MAX_PTRS];
  const int32_t* offsets;
  unsigned int* err;
  int32_t nprob, experts, form, out_dtype;
  int32_t rows, k, n;
  int32_t kblocks;     // of the k dimension (weight gradients: each expert's rows give their own)
  int32_t bk;          // elements of a k-block
  int32_t kscales, nscales;
  int32_t sb_k, sb_n;  // steps of the rhs scales along k and n
  uint32_t idesc;
  uint32_t bstep;      // the rhs tile's descriptor advance per MMA, in 16-byte units
  uint32_t blead;      // its leading byte offset >> 4
  int32_t split;       // few-row kernel: CTAs of a cluster that share a tile's k range
  int32_t units;       // as many as ascending offsets can have (less than 2^30); later ones are left out
};
static_assert(sizeof(GroupedParams) <= 32000, "kernel parameter block too large");

// ------------------------------------------------------------- work units

struct Tile {
  int p, e;    // problem and expert
  int r0, r1;  // the expert's rows
  int m0, n0;  // the tile's first row (of the expert; weight gradients: first row of k) and column
};

// A warp's view of 32 consecutive (problem, expert) pairs: lane l holds pair base + l.
struct Walk {
  int base;
  int r0, r1, tiles;
  int upto;  // units of all pairs up to and including this lane's
};

template <bool GRAD>
__device__ __forceinline__ void walk_load(const GroupedParams& P, Walk& w, int base, int before, int tm, int tn) {
  const int lane = threadIdx.x & 31;
  w.base = base;
  w.r0 = w.r1 = w.tiles = 0;
  const int pe = base + lane;
  if (pe < P.nprob * P.experts) {
    w.r1 = P.rows;
    if (P.offsets) {
      const int p = pe / P.experts;
      const int32_t* o = P.offsets + pe + p;  // (each problem has experts + 1 offsets)
      w.r0 = min(max(__ldg(o), 0), P.rows);
      w.r1 = min(max(__ldg(o + 1), w.r0), P.rows);
    }
    const int m = GRAD ? P.k : w.r1 - w.r0;
    w.tiles = ((m + tm - 1) / tm) * ((P.n + tn - 1) / tn);
  }
  int s = w.tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s = min(s + v, P.units);
  }
  w.upto = min(before + s, P.units);
}

// The tile of unit u (ascending from call to call), or false past the last one. The whole warp calls it.
template <bool GRAD>
__device__ __forceinline__ bool walk_find(const GroupedParams& P, Walk& w, int u, Tile& t, int tm, int tn,
                                          int group_mt = GROUP_MT) {
  for (;;) {
    const int last = __shfl_sync(0xffffffffu, w.upto, 31);
    if (u < last) break;
    if (w.base + 32 >= P.nprob * P.experts) return false;
    walk_load<GRAD>(P, w, w.base + 32, last, tm, tn);
  }
  const int f = __ffs(__ballot_sync(0xffffffffu, u < w.upto)) - 1;
  const int pe = w.base + f;
  t.p = pe / P.experts;
  t.e = pe - t.p * P.experts;
  t.r0 = __shfl_sync(0xffffffffu, w.r0, f);
  t.r1 = __shfl_sync(0xffffffffu, w.r1, f);
  const int local = u - (__shfl_sync(0xffffffffu, w.upto, f) - __shfl_sync(0xffffffffu, w.tiles, f));
  const int mts = ((GRAD ? P.k : t.r1 - t.r0) + tm - 1) / tm, nts = (P.n + tn - 1) / tn;
  const int group = local / (group_mt * nts);
  const int gm = min(group_mt, mts - group * group_mt);
  const int in_g = local - group * group_mt * nts;
  const int nt = in_g / gm;
  t.m0 = (group * group_mt + in_g - nt * gm) * tm;
  t.n0 = nt * tn;
  return true;
}

// Rows of an expert that its tile t covers, as the N of an MMA over two CTAs takes them: a multiple of 32.
__device__ __forceinline__ int mma_rows(const Tile& t) { return min(TILE_M, (t.r1 - t.r0 - t.m0 + 31) & ~31); }

// The number of all units: for a warp whose work is the same for every tile.
template <bool GRAD>
__device__ __forceinline__ int walk_total(const GroupedParams& P, int tm, int tn) {
  Walk w;
  walk_load<GRAD>(P, w, 0, 0, tm, tn);
  while (w.base + 32 < P.nprob * P.experts)
    walk_load<GRAD>(P, w, w.base + 32, __shfl_sync(0xffffffffu, w.upto, 31), tm, tn);
  return __shfl_sync(0xffffffffu, w.upto, 31);
}

// ------------------------------------------------------------ PTX (this file)

// D (+)= A B of this CTA, e4m3 operands (kind::f8f6f4, K = 32) or 16-bit ones (kind::f16, K = 16).
template <bool E4M3>
__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    umma(d, a, b, idesc, accumulate);
}

// The bounded waits of tc_ptx.h without a function call: ptxas cannot split registers between warps
// (setmaxnreg) in a kernel that makes one.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (mbar_test(bar, parity)) return true;
    if ((it & 31) == 0 && (*abort_flag || globaltimer() - t0 > kTimeoutNs)) return false;
  }
}
__device__ __forceinline__ bool wait_bar_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  bool ok = true;
  if ((threadIdx.x & 31) == 0) ok = wait_bar(bar, parity, abort_flag);
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// A producer warp's last step: every stage that it filled is read and handed back, so no commit's arrival is still on
// its way when the CTA gives up its shared memory. `empty0`: the barrier of stage 0; `parity`: bit s is the phase of
// the stage's last copies, which its hand-back completes. (After a failure a stage may never be multiplied. By the
// time that the first wait for one has run out, all that was issued has long arrived.)
__device__ __forceinline__ void await_hand_back(uint32_t empty0, int stages, uint32_t issued, uint32_t parity,
                                                volatile int* never) {
  for (int s = 0; s < stages; ++s)
    if (((issued >> s) & 1u) && !wait_bar_warp(empty0 + 8u * s, (parity >> s) & 1u, never)) break;
}

// A descriptor of operand tiles in 128-byte swizzled rows (tcgen05 matrix descriptor: start address >> 4,
// leading byte offset >> 4 at bit 16, stride byte offset >> 4 at bit 32, version 1, 128-byte swizzle): groups
// of 8 rows are 1024 bytes apart; `lead` is the distance of 128-byte wide boxes of operands whose rows run
// along k (unused for operands whose rows hold 128 bytes of k).
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, uint32_t lead) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFF) | (static_cast<uint64_t>(lead) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Two fp32 values in a 64-bit register, and sum += value * scale on both in one instruction (each rounded
// once, as fmaf): the additions are the epilogue's issue slots, and those bound the block-scaled products.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ void unpack2(uint64_t v, uint32_t& lo, uint32_t& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=r"(lo), "=r"(hi) : "l"(v));
}
__device__ __forceinline__ void add_scaled(uint64_t& sum, uint32_t lo, uint32_t hi, uint64_t scale) {
  asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(sum) : "l"(pack2(lo, hi)), "l"(scale));
}

// ---------------------------------------------------------------- epilogue

// Values that a k loop does not need, kept in the warp's (then idle) staging strip across it: its 128 sums and
// the loads in flight take nearly all of a thread's registers.
__device__ __forceinline__ void park(uint32_t strip, int i, int v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(strip + 4 * (32 * i + (threadIdx.x & 31))), "r"(v) : "memory");
}
__device__ __forceinline__ int unpark(uint32_t strip, int i) {
  int v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(strip + 4 * (32 * i + (threadIdx.x & 31))) : "memory");
  return v;
}

// Writes 32 rows x 128 bytes held one row per lane: through shared memory, so that each store instruction
// covers four whole 128-byte lines, and bounded by rows and bytes, so that a tile may end anywhere.
__device__ __forceinline__ void store_strip(uint32_t strip, const uint32_t (&p)[32], char* out, int64_t pitch,
                                            int rows, int64_t bytes) {
  // The lane is read anew (volatile): the two dozen addresses below would otherwise be computed once, ahead of the
  // tiles, and kept in the registers that the k loop's sums need.
  int lane;
  asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
#pragma unroll
  for (int c = 0; c < 8; ++c)
    st_shared_v4(strip + lane * 128 + ((c ^ (lane & 7)) << 4), p[4 * c], p[4 * c + 1], p[4 * c + 2], p[4 * c + 3]);
  __syncwarp();
  // (all loads before the first store: one at a time, each waited for shared memory)
  const int ch = lane & 7;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = i * 4 + (lane >> 3);
    v[i] = ld_shared_v4(strip + row * 128 + ((ch ^ (row & 7)) << 4));
  }
  char* o = out + (lane >> 3) * pitch + ch * 16;
#pragma unroll
  for (int i = 0; i < 8; ++i, o += 4 * pitch)
    if (i * 4 + (lane >> 3) < rows && ch * 16 < bytes) *reinterpret_cast<uint4*>(o) = v[i];
  __syncwarp();
}

// Writes 32 rows of 32 columns held one column per lane (row j in r[j]): turned in shared memory, so that a store
// instruction covers whole 64-byte (fp32: 128-byte) pieces of rows; bounded as above.
__device__ __forceinline__ void store_turned(uint32_t strip, const uint32_t (&r)[32], char* out, int64_t pitch,
                                             int rows, int64_t bytes, int dtype) {
  int lane;
  asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
  if (dtype == COCO_F32) {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(strip + j * 128 + lane * 4), "r"(r[j]) : "memory");
    __syncwarp();
    const int row0 = lane >> 3, at = (lane & 7) * 16;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ld_shared_v4(strip + (i * 4 + row0) * 128 + at);
    char* o = out + row0 * pitch + at;
#pragma unroll
    for (int i = 0; i < 8; ++i, o += 4 * pitch)
      if (i * 4 + row0 < rows && at < bytes) *reinterpret_cast<uint4*>(o) = v[i];
  } else {
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const uint32_t two = cvt_pair(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), dtype);
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(strip + j * 64 + lane * 2), "h"(static_cast<uint16_t>(two))
                   : "memory");
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(strip + j * 64 + 64 + lane * 2),
                   "h"(static_cast<uint16_t>(two >> 16))
                   : "memory");
    }
    __syncwarp();
    const int row0 = lane >> 2, at = (lane & 3) * 16;
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ld_shared_v4(strip + (i * 8 + row0) * 64 + at);
    char* o = out + row0 * pitch + at;
#pragma unroll
    for (int i = 0; i < 4; ++i, o += 8 * pitch)
      if (i * 8 + row0 < rows && at < bytes) *reinterpret_cast<uint4*>(o) = v[i];
  }
  __syncwarp();
}

// Rows of no expert are zero. Every thread of `nthreads` takes its share.
__device__ __forceinline__ void clear_rest(const GroupedParams& P, int64_t thread, int64_t nthreads) {
  const int64_t pitch = static_cast<int64_t>(P.n) * (P.out_dtype == COCO_F32 ? 4 : 2) / 16;
  for (int p = 0; p < P.nprob; ++p) {
    const int32_t* o = P.offsets + static_cast<int64_t>(p) * (P.experts + 1);
    const int64_t head = min(max(__ldg(o), 0), P.rows);
    const int64_t tail = max(min(max(__ldg(o + P.experts), 0), P.rows), static_cast<int>(head));
    const int64_t total = (head + P.rows - tail) * pitch;
    uint4* out = static_cast<uint4*>(P.out[p]);
    for (int64_t i = thread; i < total; i += nthreads)
      out[i < head * pitch ? i : i + (tail - head) * pitch] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// ------------------------------------------------------------ pair kernel

template <bool GRAD>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    k_grouped_pair(const __grid_constant__ GroupedParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + BAR_OFF;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto loaded_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };  // weight gradients: an expert's last block
  auto tfull_bar = [&](int a) { return bar0 + 8u * (3 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (3 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (3 * STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + BAR_OFF + 8 * NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + BAR_OFF + 8 * NUM_BARS + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cluster_id = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  constexpr uint16_t kPair = 0x3;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);  // CTA 0's is the pair's
      mbar_init(empty_bar(s), 1);
      mbar_init(loaded_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 2 * EPI_WARPS);  // CTA 0's: the epilogue warps of both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<true>(smem_u32(tmem_slot), TMEM_COLS);
  tc_fence_before();
  cluster_sync();  // the peer's barriers exist before the pair's copies or commits reach them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  auto fail = [&]() {
    *abort_flag = 1;
    atomicCAS(P.err, 0u, static_cast<unsigned int>(COCO_ERR_TIMEOUT));
  };
  int dummy = 0;
  volatile int* never = &dummy;

  if (warp < FIRST_EPI_WARP) {
    if (warp == 0) {
      // ------------------------------------------------------ TMA producer
      const bool leader = elect_one();
      Walk w;
      walk_load<GRAD>(P, w, 0, 0, TILE_M, TILE_N);
      Tile t;
      int stage = 0;
      uint32_t phase = 0;
      uint32_t issued = 0, parity = 0, own = 0, own_parity = 0;  // per stage; own: the copies complete loaded_bar
      bool ok = true;
      for (int u = cluster_id; ok && walk_find<GRAD>(P, w, u, t, TILE_M, TILE_N); u += nclusters) {
        const CUtensorMap *ma = &P.a[t.p], *mb = &P.b[t.p];
        const int kblocks = GRAD ? (t.r1 - t.r0 + P.bk - 1) / P.bk : P.kblocks;
        const bool ragged = GRAD && (t.r1 - t.r0) % P.bk != 0;
        const int acol = t.m0 + 128 * rank, bcol = t.n0 + 128 * rank;  // (products: bcol of the weights, the A side)
        const int share = GRAD ? 0 : mma_rows(t) / 2;                  // rows of the tile that this CTA loads
        const int boxes = (share + 63) / 64;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!wait_bar_warp(empty_bar(stage), phase ^ 1u, abort_flag)) {
            if (leader) fail();
            ok = false;
            break;
          }
          const uint32_t sa = sbase + stage * STAGE_BYTES, sb = sa + A_BYTES;
          const bool partly = ragged && kb == kblocks - 1;
          if (leader) {
            if constexpr (GRAD) {
              // both operands' rows run along the contraction: 64 rows x 64 columns a box
              const int r = t.r0 + kb * P.bk;
              if (partly) {  // (then warps 2 and 3 have the rest of its rows zeroed, counted on CTA 0's barrier)
                mbar_expect_tx(loaded_bar(stage), STAGE_BYTES);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  tma_load_3d(sa + j * (A_BYTES / 2), ma, loaded_bar(stage), acol + 64 * j, r, 0);
                  tma_load_3d(sb + j * (B_BYTES / 2), mb, loaded_bar(stage), bcol + 64 * j, r, 0);
                }
                if (rank == 0) mbar_expect_tx(full_bar(stage), 2 * 4 * 128 * (P.bk - (t.r1 - r)));
              } else {
                const uint32_t fb = mapa_rank0(full_bar(stage));
                if (rank == 0) mbar_expect_tx(full_bar(stage), 2 * STAGE_BYTES);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  tma_load_3d_pair(sa + j * (A_BYTES / 2), ma, fb, acol + 64 * j, r, 0);
                  tma_load_3d_pair(sb + j * (B_BYTES / 2), mb, fb, bcol + 64 * j, r, 0);
                }
              }
            } else {
              const uint32_t fb = mapa_rank0(full_bar(stage));
              if (rank == 0) mbar_expect_tx(full_bar(stage), 2 * (A_BYTES + boxes * (B_BYTES / 2)));
              const int k0 = kb * P.bk;
              if (P.form == GRP_NK) {
                tma_load_3d_pair(sa, mb, fb, k0, bcol, t.e);
              } else {
                tma_load_3d_pair(sa, mb, fb, bcol, k0, t.e);
                tma_load_3d_pair(sa + A_BYTES / 2, mb, fb, bcol + 64, k0, t.e);
              }
              for (int j = 0; j < boxes; ++j)
                tma_load_3d_pair(sb + j * (B_BYTES / 2), ma, fb, k0, t.r0 + t.m0 + rank * share + 64 * j, 0);
            }
          }
          __syncwarp();
          const uint32_t bit = 1u << stage;
          issued |= bit;
          parity = (parity & ~bit) | (phase << stage);
          own = partly ? own | bit : own & ~bit;
          if (partly) own_parity ^= bit;  // (starts at 0: after the first use, its phase 0 is the one in flight)
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {  // let copies in flight land (CTA 0's barriers count both CTAs')
        for (int s = 0; s < STAGES; ++s) {
          if (!((issued >> s) & 1u)) continue;
          if ((own >> s) & 1u) wait_bar_warp(loaded_bar(s), ((own_parity >> s) & 1u) ^ 1u, never);
          if (rank == 0) wait_bar_warp(full_bar(s), (parity >> s) & 1u, never);
        }
      }
      // (CTA 0's MMA warp hands the stages of both CTAs back)
      await_hand_back(empty_bar(0), STAGES, issued, parity, never);
    } else if (warp == 1) {
      // ------------------------------------------------------- MMA issuer
      if (rank == 0) {
        const bool leader = elect_one();
        // rows of 128 bytes of k: 32 bytes an MMA; rows along k: 16 rows an MMA
        const uint32_t astep = GRAD ? 128 : P.bstep, bstep = GRAD ? P.bstep : 2;
        const uint64_t ad0 = tile_desc(sbase, GRAD ? (A_BYTES / 2) >> 4 : P.blead);
        const uint64_t bd0 = tile_desc(sbase + A_BYTES, GRAD ? P.blead : 1);
        constexpr uint32_t kStageDesc = static_cast<uint32_t>(STAGE_BYTES >> 4);
        Walk w;
        walk_load<GRAD>(P, w, 0, 0, TILE_M, TILE_N);
        Tile t;
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t accph = 0;
        bool ok = true, any_mma = false;
        for (int u = cluster_id; ok && walk_find<GRAD>(P, w, u, t, TILE_M, TILE_N); u += nclusters) {
          const uint32_t idesc = GRAD ? P.idesc : P.idesc | (static_cast<uint32_t>(mma_rows(t) >> 3) << 17);
          const int kblocks = GRAD ? (t.r1 - t.r0 + P.bk - 1) / P.bk : P.kblocks;
          if (GRAD && kblocks == 0) continue;  // no rows: the epilogue stores zeros
          if (!wait_bar_warp(tempty_bar(acc), accph ^ 1u, abort_flag)) {
            if (leader) fail();
            ok = false;
            break;
          }
          tc_fence_after();
          for (int kb = 0; kb < kblocks; ++kb) {
            if (!wait_bar_warp(full_bar(stage), phase, abort_flag)) {
              if (leader) fail();
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t off = static_cast<uint64_t>(stage * kStageDesc);
            const uint64_t ad = ad0 + off, bd = bd0 + off;
            if (leader) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_pair(tmem_base + acc * TILE_N, ad + astep * k, bd + bstep * k, idesc, (kb | k) != 0);
              umma_commit_pair(empty_bar(stage), kPair);
            }
            any_mma = true;
            __syncwarp();
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
          if (ok) {
            if (leader) umma_commit_pair(tfull_bar(acc), kPair);
            acc ^= 1;
            if (acc == 0) accph ^= 1u;
          }
          __syncwarp();
        }
        if (!ok && any_mma) {  // wait for the MMAs already issued before TMEM is freed
          if (leader) umma_commit_pair(drain_bar, 0x1);
          __syncwarp();
          wait_bar_warp(drain_bar, 0, never);
        }
      }
    } else if (GRAD && warp >= 2) {
      // --------------------------------------- zeros over the next expert's rows
      // An expert's last k-block holds rows past its end. Zeros go over them in both operands (in one alone they would
      // leave 0 * infinity). They come by copies like any others, from rows out of range: counted on CTA 0's barrier,
      // they need no ordering of this CTA's own writes before the pair's MMA. Clearing with stores and an arrival that
      // releases them to CTA 0 (cluster scope) took 232 us where this takes 204 (16384 rows, 32 uneven experts, k 4096,
      // n 2048). Warp 2 has A's two boxes of rows of 128 bytes done, warp 3 B's.
      const bool leader = elect_one();
      Walk w;
      walk_load<GRAD>(P, w, 0, 0, TILE_M, TILE_N);
      Tile t;
      int stage = 0;
      uint32_t loaded_phase = 0;  // per stage: parity of its next use
      bool ok = true;
      for (int u = cluster_id; ok && walk_find<GRAD>(P, w, u, t, TILE_M, TILE_N); u += nclusters) {
        const int rows = t.r1 - t.r0, kblocks = (rows + P.bk - 1) / P.bk;
        const int last = (stage + kblocks + STAGES - 1) % STAGES;
        stage = (stage + kblocks) % STAGES;
        const int valid = rows % P.bk;
        if (valid == 0) continue;
        if (!wait_bar_warp(loaded_bar(last), (loaded_phase >> last) & 1u, abort_flag)) {
          if (leader) fail();
          ok = false;
          break;
        }
        loaded_phase ^= 1u << last;
        if (leader) {
          const uint32_t fb = mapa_rank0(full_bar(last));
          uint32_t to = sbase + last * STAGE_BYTES + (warp - 2) * A_BYTES + valid * 128;
#pragma unroll
          for (int i = 0; i < kZeroMaps; ++i)  // (64 - valid rows: a box for every binary digit)
            if (((64 - valid) >> i) & 1) {
              tma_load_3d_pair(to, &P.zero[i], fb, 0, P.rows, 0);
              tma_load_3d_pair(to + A_BYTES / 2, &P.zero[i], fb, 0, P.rows, 0);
              to += 128u << i;
            }
        }
        __syncwarp();
      }
    }
  } else {
    // --------------------------------------------------------- epilogue
    const int quarter = warp & 3;                       // TMEM lanes 32*quarter .. +31 belong to this warp
    const int half = (warp - FIRST_EPI_WARP) >> 2;      // columns 128*half .. +127 of the tile
    const uint32_t strip = sbase + STRIP_OFF + (warp - FIRST_EPI_WARP) * STRIP;
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    const uint32_t tempty0 = rank == 0 ? 0 : mapa_rank0(tempty_bar(0));
    Walk w;
    walk_load<GRAD>(P, w, 0, 0, TILE_M, TILE_N);
    Tile t;
    int acc = 0;
    uint32_t accph = 0;
    auto wait_acc = [&]() {
      const bool ready = __all_sync(0xffffffffu, wait_bar(tfull_bar(acc), accph, abort_flag));
      if (!ready && lane == 0) fail();
      tc_fence_after();
      return ready;
    };
    auto free_acc = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive_relaxed(tempty_bar(acc));
        else mbar_arrive_cluster_relaxed(tempty0 + 8u * acc);
      }
      acc ^= 1;
      if (acc == 0) accph ^= 1u;
    };
    bool ok = true;
    for (int u = cluster_id; ok && walk_find<GRAD>(P, w, u, t, TILE_M, TILE_N); u += nclusters) {
      const int esize = P.out_dtype == COCO_F32 ? 4 : 2;
      const int64_t pitch = static_cast<int64_t>(P.n) * esize;
      if constexpr (GRAD) {
        const int row = t.m0 + 128 * rank + quarter * 32;  // this warp's first row (of lhs columns)
        const int rows = min(32, P.k - row);               // (may be negative: nothing to store)
        const int64_t at = static_cast<int64_t>(t.n0 + 128 * half) * esize;
        char* out = static_cast<char*>(P.out[t.p]) + (static_cast<int64_t>(t.e) * P.k + row) * pitch + at;
        const int64_t bytes = pitch - at;  // left of the row
        const bool none = t.r1 == t.r0;    // no rows: the gradient is zero
        if (!none && !wait_acc()) { ok = false; break; }
        const uint32_t ta = tacc + acc * TILE_N;
        if (esize == 4) {
          for (int c = 0; c < 4; ++c) {
            uint32_t p[32];
            if (none) {
#pragma unroll
              for (int j = 0; j < 32; ++j) p[j] = 0u;
            } else {
              tmem_ld32(ta + 32 * c, p);
              tmem_ld_wait();
              if (c == 3) free_acc();
            }
            if (rows > 0 && bytes > 128 * c) store_strip(strip, p, out + 128 * c, pitch, rows, bytes - 128 * c);
          }
        } else {  // (the accumulator is read, and handed back, before the first store)
          uint32_t p[2][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            if (none) {
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = 0u;
            } else {
              tmem_ld32(ta + 32 * c, r);
              tmem_ld_wait();
            }
#pragma unroll
            for (int j = 0; j < 16; ++j)
              p[c / 2][16 * (c & 1) + j] =
                  cvt_pair(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), P.out_dtype);
          }
          if (!none) free_acc();
          if (rows > 0 && bytes > 0) store_strip(strip, p[0], out, pitch, rows, bytes);
          if (rows > 0 && bytes > 128) store_strip(strip, p[1], out + 128, pitch, rows, bytes - 128);
        }
      } else {
        // lanes are the output's columns, TMEM columns its rows: this warp's 32 columns of up to 128 rows
        const int rows = min(128, t.r1 - t.r0 - t.m0 - 128 * half);  // (may be negative: nothing to store)
        const int64_t at = static_cast<int64_t>(t.n0 + 128 * rank + 32 * quarter) * esize;
        const int64_t row = static_cast<int64_t>(t.r0) + t.m0 + 128 * half;
        char* out = static_cast<char*>(P.out[t.p]) + row * pitch + at;
        const int64_t bytes = pitch - at;
        if (!wait_acc()) { ok = false; break; }
        const uint32_t ta = tacc + acc * TILE_N;
        if (rows <= 0) free_acc();
        for (int c = 0; c < rows; c += 32) {
          uint32_t r[32];
          tmem_ld32(ta + c, r);
          tmem_ld_wait();
          if (c + 32 >= rows) free_acc();
          if (bytes > 0) store_turned(strip, r, out + c * pitch, pitch, rows - c, bytes, P.out_dtype);
        }
      }
    }
    if (!GRAD && P.offsets)
      clear_rest(P, static_cast<int64_t>(blockIdx.x) * (32 * EPI_WARPS) + threadIdx.x - 32 * FIRST_EPI_WARP,
                 static_cast<int64_t>(gridDim.x) * (32 * EPI_WARPS));
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal its barriers or read its TMEM
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<true>(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------ block-scaled kernel
//
// k_grouped_scaled (e4m3, many rows): one 128 x 256 tile per CTA and step (M = 128, N = 256), no CTA depending on
// another. The block's product has to be added up and its TMEM buffer handed back every 128 k, and with one MMA over
// two CTAs that hand-over crosses CTAs both ways (commit to the other's epilogue, arrivals back), some thousand cycles
// of every two blocks' 1024. The price is that a CTA reads all 256 of its columns of rhs itself, 48 KB a block, which
// L2 gives: 8192^3 takes 383 to 395 us (2.87 PFLOP/s) from a graph, where two CTAs that each loaded half of the columns
// for both took 388. Tiles of 128 rows also cost an expert's end half of what 256 would: 16384 rows over 32 uneven
// experts, k 4096, n 2048: 124 to 127 us. What bounds it is the power cap in a long loop (433 us a call at 8192^3) and
// the epilogue's loop: 8 TMEM loads, 64 packed multiply-adds and the hand-over a block.
//   warp 0        TMA producer: 128 rows of lhs and 256 columns of rhs; 4 stages of 48 KB.
//   warp 1        issues the MMAs and owns TMEM (two buffers of 256 columns).
//   warps 4..11   two per TMEM lane quarter, 128 columns each: sums of the scaled blocks in registers, then stores.

constexpr int S_TILE_M = 128, S_GROUP_MT = 16;  // (as many rows to a raster group as k_grouped_pair's)
constexpr int S_STAGE = A_BYTES + 2 * B_BYTES, S_STAGES = 4;
constexpr int S_STRIP_OFF = S_STAGES * S_STAGE;
constexpr int S_BAR_OFF = S_STRIP_OFF + EPI_WARPS * STRIP;
constexpr int S_NUM_BARS = 2 * S_STAGES + 5;  // full, empty per stage; accumulators full x2, empty x2; drain
constexpr int S_SMEM_BYTES = S_BAR_OFF + 8 * S_NUM_BARS + 16 + 1024;
static_assert(S_SMEM_BYTES <= 232448, "shared memory over the per-CTA limit");

__global__ void __launch_bounds__(THREADS, 1) k_grouped_scaled(const __grid_constant__ GroupedParams P) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + S_BAR_OFF;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S_STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S_STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S_STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S_STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S_BAR_OFF + 8 * S_NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S_BAR_OFF + 8 * S_NUM_BARS + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S_STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");  // (for the copies and commits)
  }
  if (warp == 1) tmem_alloc<false>(smem_u32(tmem_slot), TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  auto fail = [&]() {
    *abort_flag = 1;
    atomicCAS(P.err, 0u, static_cast<unsigned int>(COCO_ERR_TIMEOUT));
  };
  int dummy = 0;
  volatile int* never = &dummy;

  // Registers: an epilogue thread holds 128 sums. The launch's 384 threads have 168 each; the four warps in front
  // give up what the eight epilogue warps take (128 x 88 + 256 x 208 = 384 x 168). Neither side may spill: a few
  // reloads in the MMA warp's loop or the sums' cost 20 to 60 %.
  if (warp < FIRST_EPI_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ------------------------------------------------------ TMA producer
      const bool leader = elect_one();
      Walk w;
      walk_load<false>(P, w, 0, 0, S_TILE_M, TILE_N);
      Tile t;
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && walk_find<false>(P, w, u, t, S_TILE_M, TILE_N, S_GROUP_MT); u += gridDim.x) {
        const CUtensorMap *ma = &P.a[t.p], *mb = &P.b[t.p];
        const int arow = t.r0 + t.m0;
        for (int kb = 0; kb < P.kblocks; ++kb) {
          if (!wait_bar_warp(empty_bar(stage), phase ^ 1u, abort_flag)) {
            if (leader) fail();
            ok = false;
            break;
          }
          if (leader) {
            const uint32_t sa = sbase + stage * S_STAGE, sb = sa + A_BYTES;
            const int k0 = kb * 128;
            mbar_expect_tx(full_bar(stage), S_STAGE);
            tma_load_3d(sa, ma, full_bar(stage), k0, arow, 0);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int n0 = t.n0 + 128 * j;
              if (P.form == GRP_NK) tma_load_3d(sb + j * B_BYTES, mb, full_bar(stage), k0, n0, t.e);
              else tma_load_3d(sb + j * B_BYTES, mb, full_bar(stage), n0, k0, t.e);
            }
          }
          __syncwarp();
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == S_STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok)  // let copies in flight land
        for (int s = 0; s < S_STAGES; ++s)
          if ((issued >> s) & 1u) wait_bar_warp(full_bar(s), (parity >> s) & 1u, never);
      await_hand_back(empty_bar(0), S_STAGES, issued, parity, never);
    } else if (warp == 1) {
      // ------------------------------------------------------- MMA issuer
      const bool leader = elect_one();
      const uint32_t idesc = P.idesc, bstep = P.bstep;
      const uint64_t ad0 = tile_desc(sbase, 1), bd0 = tile_desc(sbase + A_BYTES, P.blead);
      // (every tile has the same blocks: this warp needs no more than the tiles' number)
      const int total = walk_total<false>(P, S_TILE_M, TILE_N);
      int stage = 0, acc = 0;
      uint32_t phase = 0, accph = 0;
      bool ok = true, any_mma = false;
      for (int u = blockIdx.x; ok && u < total; u += gridDim.x) {
        for (int kb = 0; kb < P.kblocks; ++kb) {
          if (!wait_bar_warp(tempty_bar(acc), accph ^ 1u, abort_flag) ||
              !wait_bar_warp(full_bar(stage), phase, abort_flag)) {
            if (leader) fail();
            ok = false;
            break;
          }
          tc_fence_after();
          if (leader) {
            const uint64_t off = static_cast<uint64_t>(stage * (S_STAGE >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_one<true>(tmem_base + acc * TILE_N, ad0 + off + 2 * k, bd0 + off + bstep * k, idesc, k != 0);
            umma_commit(tfull_bar(acc));
            umma_commit(empty_bar(stage));
          }
          __syncwarp();
          any_mma = true;
          acc ^= 1;
          if (acc == 0) accph ^= 1u;
          if (++stage == S_STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok && any_mma) {  // wait for the MMAs already issued before TMEM is freed
        if (leader) umma_commit(drain_bar);
        __syncwarp();
        wait_bar_warp(drain_bar, 0, never);
      }
    }
  } else {
    // --------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int quarter = warp & 3;                   // TMEM lanes 32*quarter .. +31 belong to this warp
    const int half = (warp - FIRST_EPI_WARP) >> 2;  // columns 128*half .. +127 of the tile: one block of rhs scales
    const uint32_t strip = sbase + S_STRIP_OFF + (warp - FIRST_EPI_WARP) * STRIP;
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * 128;
    Walk w;
    walk_load<false>(P, w, 0, 0, S_TILE_M, TILE_N);
    Tile t;
    int acc = 0;
    uint32_t accph = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && walk_find<false>(P, w, u, t, S_TILE_M, TILE_N, S_GROUP_MT); u += gridDim.x) {
      uint64_t sum[64];  // pairs of fp32 sums of neighbouring columns
#pragma unroll
      for (int j = 0; j < 64; ++j) sum[j] = 0ull;
      // this lane's row of lhs scales, and the columns' block of rhs scales (out of range: any valid ones)
      const int my_row = t.r0 + t.m0 + quarter * 32 + lane;
      const float* sa = P.sa[t.p] + static_cast<int64_t>(min(my_row, P.rows - 1)) * P.kscales;
      const float* sb = P.sb[t.p] + static_cast<int64_t>(t.e) * P.kscales * P.nscales +
                        static_cast<int64_t>(min(t.n0 / 128 + half, P.nscales - 1)) * P.sb_n;
      const int64_t sb_k = P.sb_k;
      park(strip, 0, w.base); park(strip, 1, w.r0); park(strip, 2, w.r1); park(strip, 3, w.tiles);
      park(strip, 4, w.upto); park(strip, 5, t.p); park(strip, 6, t.r0); park(strip, 7, t.r1);
      park(strip, 8, t.m0); park(strip, 9, t.n0); park(strip, 10, u);
      float a_s = __ldg(sa), b_s = __ldg(sb);
      for (int left = P.kblocks; left > 0; --left) {
        const float s = a_s * b_s;
        if (left > 1) {  // the next block's scales, ahead of its sums
          a_s = __ldg(++sa);
          b_s = __ldg(sb += sb_k);
        }
        const bool ready = __all_sync(0xffffffffu, wait_bar(tfull_bar(acc), accph, abort_flag));
        if (!ready) {
          if (lane == 0) fail();
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t ta = tacc + acc * TILE_N;
        const uint64_t ss = pack2(__float_as_uint(s), __float_as_uint(s));
        // (every sum is pinned behind its load by asm volatile: moved on, the sums' operands do not fit the registers)
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          uint32_t r[16];
          tmem_ld16(ta + 16 * c, r);
          tmem_ld_wait();
          if (c == 7) {  // the buffer is read: hand it back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(tempty_bar(acc));
            acc ^= 1;
            if (acc == 0) accph ^= 1u;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) add_scaled(sum[8 * c + j], r[2 * j], r[2 * j + 1], ss);
        }
      }
      if (!ok) break;
      w.base = unpark(strip, 0); w.r0 = unpark(strip, 1); w.r1 = unpark(strip, 2); w.tiles = unpark(strip, 3);
      w.upto = unpark(strip, 4); t.p = unpark(strip, 5); t.r0 = unpark(strip, 6); t.r1 = unpark(strip, 7);
      t.m0 = unpark(strip, 8); t.n0 = unpark(strip, 9); u = unpark(strip, 10);
      __syncwarp();  // (the strip is written again below)
      const int row = t.m0 + quarter * 32;  // this warp's first one
      const int rows = min(32, t.r1 - t.r0 - row);       // (may be negative: nothing to store)
      const int esize = P.out_dtype == COCO_F32 ? 4 : 2;
      const int64_t pitch = static_cast<int64_t>(P.n) * esize;
      const int64_t first = static_cast<int64_t>(t.n0 + 128 * half) * esize;
      char* out = static_cast<char*>(P.out[t.p]) + (static_cast<int64_t>(t.r0) + row) * pitch + first;
      const int64_t bytes = pitch - first;  // from the first column to the row's end
      if (rows > 0 && bytes > 0) {
        if (esize == 4) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 16; ++j) unpack2(sum[16 * c + j], p[2 * j], p[2 * j + 1]);
            store_strip(strip, p, out + 128 * c, pitch, rows, bytes - 128 * c);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              uint32_t x, y;
              unpack2(sum[32 * c + j], x, y);
              p[j] = cvt_pair(__uint_as_float(x), __uint_as_float(y), P.out_dtype);
            }
            store_strip(strip, p, out + 128 * c, pitch, rows, bytes - 128 * c);
          }
        }
      }
    }
    if (P.offsets)
      clear_rest(P, static_cast<int64_t>(blockIdx.x) * (32 * EPI_WARPS) + threadIdx.x - 32 * FIRST_EPI_WARP,
                 static_cast<int64_t>(gridDim.x) * (32 * EPI_WARPS));
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<false>(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------ few rows
//
// k_grouped_few: rows of lhs by the dozen (decoding, or many experts with a few rows each). The weights are
// what there is to read, so they are the MMA's M side (128 of their columns n a tile) and the rows its N side
// (ROWS = 16 or 64): out^T = rhs^T lhs^T, one CTA an MMA, no weight read twice, no idle rows to speak of.
// Where there are fewer tiles than SMs, a cluster of `split` CTAs shares a tile's k range: each sends its fp32
// sums for another's rows straight into that CTA's shared memory (st.async, counted on an mbarrier), which
// adds them in rank order. No atomics, no workspace: repeated calls give the same bits. One row, k = n = 4096 in
// e4m3: 8.6 us with cold weights, 7.3 with weights in L2, most of it the launch, the ring's first fill and the
// clusters' exchange; 32 rows over 64 experts, k 4096, n 2048, cold: 32 us (4.8 TB/s of the weights met), the last wave
// of tiles being partly filled.
//   warp 0        TMA producer, a ring of 128-byte deep k-blocks: 16 KB of weights, ROWS x 128 bytes of lhs.
//   warp 1        issues the MMAs and owns TMEM.
//   warps 2..     epilogue, one per TMEM lane quarter (ROWS = 64: two, 32 rows each): a lane holds one column n.

template <bool SCALED, int ROWS>
struct FewCfg {
  static constexpr int W_BYTES = 128 * BKB;
  static constexpr int STAGE = W_BYTES + ROWS * BKB;
  static constexpr int RED_BYTES = ROWS * 128 * 4;                   // the cluster's sums for this CTA's rows
  static constexpr int STAGES = ROWS == 16 ? 11 : 7;
  static constexpr int EPI_WARPS = ROWS == 16 ? 4 : 8;
  static constexpr int PER_WARP = ROWS / (EPI_WARPS / 4);            // rows of a warp
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int ACCS = SCALED ? 4 : 2;                        // accumulator buffers of ROWS columns
  static constexpr uint32_t COLS = ACCS * ROWS < 32 ? 32 : ACCS * ROWS;
  static constexpr int RED_OFF = STAGES * STAGE;
  static constexpr int BAR_OFF = RED_OFF + RED_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * ACCS + 2;  // full, empty; accumulators full, empty; drain; sums
  static constexpr int SMEM_BYTES = BAR_OFF + 8 * NUM_BARS + 16 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory over the per-CTA limit");
};
constexpr int FEW_N = 128;

__device__ __forceinline__ uint32_t mapa(uint32_t addr, int cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
// Two fp32 values into another CTA's shared memory; their 8 bytes count on that CTA's mbarrier.
__device__ __forceinline__ void send2(uint32_t addr, float a, float b, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(addr),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool wait_bar_cluster(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 31) == 0 && (*abort_flag || globaltimer() - t0 > kTimeoutNs)) return false;
  }
}

// Sends this thread's sums (column `n_lane` of 128, PER_WARP rows from row0 on) to the CTAs that own the rows: CTA d
// of SPLIT owns OWN = ROWS / SPLIT rows from d * OWN on (OWN divides PER_WARP). Layout there: [source][pair of
// rows][column][2].
template <int PER_WARP, int OWN>
__device__ __forceinline__ void send_sums(const float (&sum)[PER_WARP], uint32_t red, uint32_t bar, int rank, int row0,
                                          int n_lane) {
#pragma unroll
  for (int d = 0; d < PER_WARP / OWN; ++d) {
    const int cta = row0 / OWN + d;
    const uint32_t to = mapa(red, cta) + static_cast<uint32_t>(rank * (OWN / 2) * 128 + n_lane) * 8;
    const uint32_t b = mapa(bar, cta);
#pragma unroll
    for (int j = 0; j < OWN / 2; ++j) send2(to + j * 128 * 8, sum[d * OWN + 2 * j], sum[d * OWN + 2 * j + 1], b);
  }
}

__device__ __forceinline__ void store_one(void* out, int64_t i, int dtype, float v) {
  if (dtype == COCO_F32) static_cast<float*>(out)[i] = v;
  else if (dtype == COCO_F16) static_cast<__half*>(out)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
}

template <bool SCALED, int ROWS>
__global__ void __launch_bounds__(FewCfg<SCALED, ROWS>::THREADS, 1)
    k_grouped_few(const __grid_constant__ GroupedParams P) {
  using C = FewCfg<SCALED, ROWS>;
  constexpr int STAGES_ = C::STAGES, ACCS = C::ACCS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::BAR_OFF;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES_ + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES_ + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES_ + ACCS + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES_ + 2 * ACCS), red_bar = drain_bar + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::BAR_OFF + 8 * C::NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::BAR_OFF + 8 * C::NUM_BARS + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = P.split;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int cluster_id = blockIdx.x / split, nclusters = gridDim.x / split;
  // this CTA's part of every tile's k range
  const int kb0 = static_cast<int>(static_cast<int64_t>(P.kblocks) * rank / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(P.kblocks) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES_; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < ACCS; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), C::EPI_WARPS);
    }
    mbar_init(drain_bar, 1);
    mbar_init(red_bar, 1);
    // (a cluster has at most one tile then: the launch has one for each of P.units)
    if (split > 1) mbar_expect_tx(red_bar, C::RED_BYTES);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc<false>(smem_u32(tmem_slot), C::COLS);
  tc_fence_before();
  if (split > 1) cluster_sync();  // peers' barriers exist before sums arrive on them
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  auto fail = [&]() {
    *abort_flag = 1;
    atomicCAS(P.err, 0u, static_cast<unsigned int>(COCO_ERR_TIMEOUT));
  };
  int dummy = 0;
  volatile int* never = &dummy;

  if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    const bool leader = elect_one();
    Walk w;
    walk_load<false>(P, w, 0, 0, ROWS, FEW_N);
    Tile t;
    int stage = 0;
    uint32_t phase = 0, issued = 0, parity = 0;
    bool ok = true;
    for (int u = cluster_id; ok && walk_find<false>(P, w, u, t, ROWS, FEW_N); u += nclusters) {
      const CUtensorMap *mx = &P.a[t.p], *mw = &P.b[t.p];
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_bar_warp(empty_bar(stage), phase ^ 1u, abort_flag)) {
          if (leader) fail();
          ok = false;
          break;
        }
        if (leader) {
          const uint32_t sw = sbase + stage * C::STAGE, sx = sw + C::W_BYTES;
          const int k0 = kb * P.bk;
          mbar_expect_tx(full_bar(stage), C::STAGE);
          if (P.form == GRP_NK) {
            tma_load_3d(sw, mw, full_bar(stage), k0, t.n0, t.e);
          } else {
            tma_load_3d(sw, mw, full_bar(stage), t.n0, k0, t.e);
            if constexpr (!SCALED) tma_load_3d(sw + C::W_BYTES / 2, mw, full_bar(stage), t.n0 + 64, k0, t.e);
          }
          tma_load_3d(sx, mx, full_bar(stage), k0, t.r0 + t.m0, 0);
        }
        __syncwarp();
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == STAGES_) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok)  // let copies in flight land
      for (int s = 0; s < STAGES_; ++s)
        if ((issued >> s) & 1u) wait_bar_warp(full_bar(s), (parity >> s) & 1u, never);
    await_hand_back(empty_bar(0), STAGES_, issued, parity, never);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const bool leader = elect_one();
    const uint32_t idesc = P.idesc, wstep = P.bstep;
    const uint64_t wd0 = tile_desc(sbase, P.blead), xd0 = tile_desc(sbase + C::W_BYTES, 1);
    const int total = walk_total<false>(P, ROWS, FEW_N);
    int stage = 0, acc = 0;
    uint32_t phase = 0, accph = 0;
    bool ok = true, any_mma = false;
    auto wait = [&](uint32_t bar, uint32_t par) {
      if (!wait_bar_warp(bar, par, abort_flag)) {
        if (leader) fail();
        return false;
      }
      tc_fence_after();
      return true;
    };
    for (int u = cluster_id; ok && u < total; u += nclusters) {
      if (!SCALED && !wait(tempty_bar(acc), accph ^ 1u)) { ok = false; break; }
      for (int kb = kb0; kb < kb1; ++kb) {
        if (SCALED && !wait(tempty_bar(acc), accph ^ 1u)) { ok = false; break; }
        if (!wait(full_bar(stage), phase)) { ok = false; break; }
        if (leader) {
          const uint64_t off = static_cast<uint64_t>(stage * (C::STAGE >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_one<SCALED>(tmem_base + acc * ROWS, wd0 + off + wstep * k, xd0 + off + 2 * k, idesc,
                            SCALED ? k != 0 : (kb != kb0 || k != 0));
          umma_commit(empty_bar(stage));
          if (SCALED || kb + 1 == kb1) umma_commit(tfull_bar(acc));
        }
        __syncwarp();
        any_mma = true;
        if (SCALED || kb + 1 == kb1)
          if (++acc == ACCS) { acc = 0; accph ^= 1u; }
        if (++stage == STAGES_) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && any_mma) {  // wait for the MMAs already issued before TMEM is freed
      if (leader) umma_commit(drain_bar);
      __syncwarp();
      wait_bar_warp(drain_bar, 0, never);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    const int n_lane = quarter * 32 + lane;  // this lane's column of the tile
    constexpr int PW = C::PER_WARP, HALVES = C::EPI_WARPS / 4;
    const int half = (warp - 2) >> 2, row0 = half * PW;  // this warp's rows of the tile
    const uint32_t tacc = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + row0;
    Walk w;
    walk_load<false>(P, w, 0, 0, ROWS, FEW_N);
    Tile t;
    int acc = 0;
    uint32_t accph = 0;
    bool ok = true;
    auto wait_acc = [&]() {
      const bool ready = __all_sync(0xffffffffu, wait_bar(tfull_bar(acc), accph, abort_flag));
      if (!ready && lane == 0) fail();
      tc_fence_after();
      return ready;
    };
    auto load_acc = [&](uint32_t (&r)[PW]) {  // and hands the accumulator back
      if constexpr (PW == 16) tmem_ld16(tacc + acc * ROWS, r);
      else tmem_ld32(tacc + acc * ROWS, r);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(tempty_bar(acc));
      if (++acc == ACCS) { acc = 0; accph ^= 1u; }
    };
    for (int u = cluster_id; ok && walk_find<false>(P, w, u, t, ROWS, FEW_N); u += nclusters) {
      float sum[PW];
      uint32_t r[PW];
      if constexpr (SCALED) {
#pragma unroll
        for (int j = 0; j < PW; ++j) sum[j] = 0.0f;
        // lane l holds the lhs scale of the warp's row l times the tile's rhs scale (its 128 columns are one block),
        // and it is passed around by shuffles. Rows past the end: any valid row's.
        const float* sa = P.sa[t.p] + static_cast<int64_t>(min(t.r0 + t.m0 + row0 + lane, P.rows - 1)) * P.kscales;
        const float* sb = P.sb[t.p] + static_cast<int64_t>(t.e) * P.kscales * P.nscales +
                          static_cast<int64_t>(t.n0 / 128) * P.sb_n;
        auto scale = [&](int kb) { return __ldg(sa + kb) * __ldg(sb + static_cast<int64_t>(kb) * P.sb_k); };
        float s = scale(kb0);
        for (int kb = kb0; kb < kb1; ++kb) {
          const float s_next = scale(kb + 1 < kb1 ? kb + 1 : kb);
          if (!wait_acc()) { ok = false; break; }
          load_acc(r);
#pragma unroll
          for (int j = 0; j < PW; ++j) sum[j] = fmaf(__uint_as_float(r[j]), __shfl_sync(0xffffffffu, s, j), sum[j]);
          s = s_next;
        }
        if (!ok) break;
      } else {
        if (!wait_acc()) { ok = false; break; }
        load_acc(r);
#pragma unroll
        for (int j = 0; j < PW; ++j) sum[j] = __uint_as_float(r[j]);
      }
      const int n = t.n0 + n_lane;
      const int rows = t.r1 - t.r0 - t.m0;  // of this tile (at least one)
      const int64_t at = (static_cast<int64_t>(t.r0) + t.m0) * P.n + n;
      void* out = P.out[t.p];
      if (split == 1) {
#pragma unroll
        for (int j = 0; j < PW; ++j)
          if (row0 + j < rows && n < P.n)
            store_one(out, at + static_cast<int64_t>(row0 + j) * P.n, P.out_dtype, sum[j]);
      } else {
        const uint32_t red = sbase + C::RED_OFF;
        if (split == 2) send_sums<PW, ROWS / 2>(sum, red, red_bar, rank, row0, n_lane);
        else if (split == 4) send_sums<PW, ROWS / 4>(sum, red, red_bar, rank, row0, n_lane);
        else send_sums<PW, ROWS / 8>(sum, red, red_bar, rank, row0, n_lane);
        const bool all = __all_sync(0xffffffffu, wait_bar_cluster(red_bar, 0, abort_flag));
        if (!all) {
          if (lane == 0) fail();
          ok = false;
          break;
        }
        const int own = ROWS / split;
        for (int j = half; j < own / 2; j += HALVES) {
          float x = 0.0f, y = 0.0f;
          for (int src = 0; src < split; ++src) {
            const uint32_t a = red + static_cast<uint32_t>((src * (own / 2) + j) * 128 + n_lane) * 8;
            float px, py;
            asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(px), "=f"(py) : "r"(a) : "memory");
            x += px;
            y += py;
          }
          const int row = rank * own + 2 * j;
          if (n < P.n && row < rows) store_one(out, at + static_cast<int64_t>(row) * P.n, P.out_dtype, x);
          if (n < P.n && row + 1 < rows) store_one(out, at + static_cast<int64_t>(row + 1) * P.n, P.out_dtype, y);
        }
      }
    }
    if (!ok && split > 1) wait_bar_cluster(red_bar, 0, never);  // let the peers' sums land
    if (P.offsets)
      clear_rest(P, static_cast<int64_t>(blockIdx.x) * (C::THREADS - 64) + threadIdx.x - 64,
                 static_cast<int64_t>(gridDim.x) * (C::THREADS - 64));
  }

  tc_fence_before();
  __syncthreads();
  if (split > 1) cluster_sync();  // no CTA leaves while its peers may still write its shared memory
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc<false>(tmem_base, C::COLS);
  }
}

// ------------------------------------------------------------------- host

// A dense [d2][d1][d0] array of 1- or 2-byte elements in boxes of box0 x box1, zeros outside.
bool encode(CUtensorMap* map, const void* ptr, int dtype, int64_t d0, int64_t d1, int64_t d2, int box0, int box1,
            CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int es = dtype_size(dtype);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1), static_cast<cuuint64_t>(d2)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d0) * es, static_cast<cuuint64_t>(d0 * d1) * es};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box0), static_cast<cuuint32_t>(box1), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = dtype == COCO_F8E4M3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : dtype == COCO_F16  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(map, dt, 3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::atomic<bool> smem_set[7][64];

cudaError_t allow_smem(const void* kernel, int which, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && smem_set[which][dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev >= 0 && dev < 64) smem_set[which][dev].store(true, std::memory_order_release);
  return e;
}

// Tensor-core instruction descriptor: fp32 accumulators, both operands of the input type (e4m3 and f16: format
// 0 of their kinds, bf16: 1), "MN-major" bits for operands whose rows run along k.
uint32_t instruction(int dtype, bool a_mn, bool b_mn, int m, int n) {
  const uint32_t fmt = dtype == COCO_BF16 ? 1 : 0;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

}  // namespace

// Which kernel, and how many CTAs share a tile's k range.
struct Choice {
  int rows;   // 16 or 64: k_grouped_few with that many rows a tile; 0: k_grouped_pair or k_grouped_scaled
  int split;
  int64_t units;
};

// The time of each kernel is the k-blocks that its busiest SM goes through, times what one takes there, and the
// choice is the least product. Measured on a GB300, in ns a k-block (128 bytes of k): a CTA on 128 rows 480 in e4m3,
// two on 256 rows 370 in 16 bits; few rows from the first figure on one SM to the second on all of them (then HBM
// counts): 16 rows 250 to 360 in e4m3, 230 to 350 in 16 bits; 64 rows 360 to 500 and 260 to 390; e4m3 weights stored
// [k][n] are the slow operand side of these MMAs: 330 to 510 and 460 to 700. A shared k range costs 1900 once.
// Both sides, from a graph with cold weights (input sets in turn that together pass L2), in us. e4m3 [n][k], k = n =
// 4096: 1 row 8.6 (16 rows, four CTAs a tile) and 15.7 (tiles of 128 rows); 64 rows 11.2 and 16.4; 128 rows 13.9 and
// 17.1; 256 rows 17.8 and 17.2; 512 rows 31.7 and 17.4. 64 experts, k 4096, n 2048: 8 rows 16.1 and 20.0; 32 rows 32.1
// and 31.8; 128 rows 61.8 and 65.5; 256 rows 75.1 and 74.9; 1024 rows 110.8 and 91.3; stored [k][n] 32 rows 43.7 and
// 31.4, 256 rows 106 and 73; in bf16 [n][k] 32 rows 53.2 and 54.5, 256 rows 135 and 142. (The rule takes clusters of
// eight to find room while they number no more CTAs than SMs, and they do not always: 128 rows, k 8192, n 1024 take
// 17.2 where four CTAs a tile take 12.6.)
Choice choose(const GroupedLaunch& L, int kblocks) {
  const bool fp8 = L.in_dtype == COCO_F8E4M3, kn8 = fp8 && L.form == GRP_KN;
  const int64_t pair_ns = fp8 ? 480 : 370, split_ns = 1900;
  const int64_t one_sm[2] = {kn8 ? 330 : fp8 ? 250 : 230, kn8 ? 460 : fp8 ? 360 : 260};
  const int64_t all_sms[2] = {kn8 ? 510 : fp8 ? 360 : 350, kn8 ? 700 : fp8 ? 500 : 390};
  const int sms = sm_count();
  auto tiles = [&](int tm, int tn) {  // at most one partly filled tile per expert beyond the full ones
    const int64_t by_rows = static_cast<int64_t>(L.rows / tm) + (L.experts < L.rows ? L.experts : L.rows);
    const int64_t mts = L.offsets ? by_rows : (static_cast<int64_t>(L.rows) + tm - 1) / tm;
    return L.nprob * mts * ((L.n + tn - 1) / tn);
  };
  auto waves = [](int64_t n, int64_t at_once) { return (n + at_once - 1) / at_once; };
  Choice best{0, 1, tiles(fp8 ? S_TILE_M : TILE_M, TILE_N)};
  int64_t least = waves(best.units, fp8 ? sms : sms / 2) * kblocks * pair_ns;
  for (int rows : {16, 64}) {
    const int64_t units = tiles(rows, FEW_N);
    for (int split = 1; split <= 8 && split <= kblocks; split *= 2) {
      if (split > 1 && units * split > sms) break;  // (a cluster that shares a tile has no second one)
      const int64_t active = units * split < sms ? units * split : sms;
      const int i = rows == 16 ? 0 : 1;
      const int64_t block_ns = one_sm[i] + (all_sms[i] - one_sm[i]) * active / sms;
      const int64_t ns =
          waves(units * split, sms) * ((kblocks + split - 1) / split) * block_ns + (split > 1 ? split_ns : 0);
      if (ns < least) {
        least = ns;
        best = Choice{rows, split, units};
      }
    }
  }
  return best;
}

template <bool SCALED, int ROWS>
cudaError_t launch_few(const GroupedParams& P, const Choice& c, int which, cudaStream_t s) {
  using C = FewCfg<SCALED, ROWS>;
  void (*kernel)(const GroupedParams) = k_grouped_few<SCALED, ROWS>;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), which, C::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  const int64_t ctas = c.split > 1 ? c.units * c.split : c.units < sm_count() ? c.units : sm_count();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = c.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = c.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, P);
}

cudaError_t launch_grouped(const GroupedLaunch& L, cudaStream_t s, unsigned int* err_word) {
  // coordinates of a tile's last rows and columns stay within 32 bits
  const int32_t most = INT32_MAX - 1024;
  if (L.rows > most || L.k > most || L.n > most) return cudaErrorNotSupported;
  const bool fp8 = L.in_dtype == COCO_F8E4M3, grad = L.form == GRP_GRAD;
  GroupedParams P;
  P.offsets = L.offsets;
  P.err = err_word;
  P.nprob = L.nprob;
  P.experts = L.experts;
  P.form = L.form;
  P.out_dtype = L.out_dtype;
  P.rows = L.rows;
  P.k = L.k;
  P.n = L.n;
  P.bk = fp8 ? 128 : 64;
  P.kblocks = (L.k + P.bk - 1) / P.bk;
  P.kscales = (L.k + 127) / 128;
  P.nscales = (L.n + 127) / 128;
  P.sb_k = L.form == GRP_NK ? 1 : P.nscales;
  P.sb_n = L.form == GRP_NK ? P.kscales : 1;
  const int64_t grad_units = static_cast<int64_t>(L.nprob) * L.experts * ((L.k + TILE_M - 1) / TILE_M) *
                             ((L.n + TILE_N - 1) / TILE_N);
  const Choice few = grad ? Choice{0, 1, grad_units} : choose(L, P.kblocks);
  if (few.units > (1 << 30) - 1) return cudaErrorNotSupported;  // (twice as many are counted in 32 bits)
  P.split = few.split;
  P.units = static_cast<int32_t>(few.units);
  // few rows, and pairs: the rhs is the M side and the lhs the N side
  P.idesc = few.rows ? instruction(L.in_dtype, L.form != GRP_NK, false, FEW_N, few.rows)
            : fp8    ? instruction(L.in_dtype, false, L.form != GRP_NK, 128, TILE_N)
            : grad   ? instruction(L.in_dtype, true, true, TILE_M, TILE_N)
                     : instruction(L.in_dtype, L.form != GRP_NK, false, TILE_M, 0);  // (N by tile)
  // rows along k: an MMA's k values are 32 (e4m3) or 16 rows of 128 bytes; else 32 bytes of a row
  P.bstep = L.form == GRP_NK ? 2 : fp8 ? 256 : 128;
  P.blead = L.form == GRP_NK ? 1 : fp8 ? B_BYTES >> 4 : (B_BYTES / 2) >> 4;
  for (int p = 0; p < L.nprob; ++p) {
    P.out[p] = L.out[p];
    P.sa[p] = L.lhs_scales[p];
    P.sb[p] = L.rhs_scales[p];
    const int bk = P.bk;
    bool good;
    if (grad)
      good = encode(&P.a[p], L.lhs[p], L.in_dtype, L.k, L.rows, 1, 64, 64) &&
             encode(&P.b[p], L.rhs[p], L.in_dtype, L.n, L.rows, 1, 64, 64);
    else
      good = encode(&P.a[p], L.lhs[p], L.in_dtype, L.k, L.rows, 1, bk, few.rows ? few.rows : fp8 ? 128 : 64) &&
             (L.form == GRP_NK ? encode(&P.b[p], L.rhs[p], L.in_dtype, L.k, L.n, L.experts, bk, 128)
                               : encode(&P.b[p], L.rhs[p], L.in_dtype, L.n, L.k, L.experts, bk, bk));
    if (!good) return cudaErrorNotSupported;
  }
  for (int i = 0; grad && i < kZeroMaps; ++i)
    if (!encode(&P.zero[i], L.lhs[0], L.in_dtype, L.k, L.rows, 1, 64, 1 << i, CU_TENSOR_MAP_SWIZZLE_NONE))
      return cudaErrorNotSupported;
  if (few.rows) {
    cudaError_t e;
    if (few.rows == 16) e = fp8 ? launch_few<true, 16>(P, few, 3, s) : launch_few<false, 16>(P, few, 4, s);
    else e = fp8 ? launch_few<true, 64>(P, few, 5, s) : launch_few<false, 64>(P, few, 6, s);
    if (e != cudaSuccess) return e;
    count_launch();
    return cudaGetLastError();
  }
  const int ctas = fp8 ? 1 : 2;  // (of a tile)
  const int at_once = sm_count() / ctas;
  const int grid = ctas * (P.units < at_once ? P.units : at_once);
  void (*kernel)(const GroupedParams) = fp8 ? k_grouped_scaled : grad ? k_grouped_pair<true> : k_grouped_pair<false>;
  const int smem = fp8 ? S_SMEM_BYTES : SMEM_BYTES;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), fp8 ? 0 : grad ? 1 : 2, smem);
  if (e != cudaSuccess) return e;
  kernel<<<grid, THREADS, smem, s>>>(P);
  count_launch();
  return cudaGetLastError();
}

}  // namespace coco
