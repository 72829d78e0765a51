// Tokens to their experts and back. A routing names `choices` experts for every
// token; choice i = t * choices + k of it has the row
//
//   row(i) = #{j: e(j) < e(i)} + #{j < i: e(j) = e(i)}
//
// of the experts' operands (sorted by expert, within one in the choices' order),
// or none where e(i) is not an expert. Then
//
//   dispatch          rows[row(t, k)] = x[t]
//   combine           out[t] = sum_k gate[t, k] * rows[row(t, k)]   (+ over ranks, + residual)
//   combine backward  drows[row(t, k)] = gate[t, k] * dout[t]
//                     dgate[t, k] = sum over ranks and columns of dout[t] * rows[row(t, k)]
//
// and the dispatch's gradient is a combine without gates. All of them walk tokens
// (never rows), so a token's row is read once however many experts it goes to, and
// rows that no choice names are not touched. Bound by HBM but for the sort, which
// is bound by latency.

#include <atomic>

#include "internal.h"
#include "rows.h"
#include "tc_ptx.h"

namespace coco {
namespace {

// -------------------------------------------------------------------- sort

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kSortSmem = 200 * 1024;
constexpr int kSortTile = 8192;  // experts that a pass over the choices counts (more of them: more passes)

struct SortArgs {
  const void* expert_of;  // [groups][n]
  int32_t* row_of;        // [groups][n]
  int32_t* choice_of;     // [groups][n], or null
  int32_t* offsets;       // [groups * nranks][experts + 1]
  int64_t n, seg;         // choices, and those of one warp (a multiple of 32)
  int32_t experts, tile, warps, nranks;
};

// The expert of choice i, or -1 where it is none.
template <typename I>
__device__ __forceinline__ int expert_at(const I* e, int64_t i, int experts) {
  const I v = e[i];
  return v >= 0 && v < static_cast<I>(experts) ? static_cast<int>(v) : -1;
}

__device__ __forceinline__ uint32_t cluster_nctarank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ int32_t ld_peer(const int32_t* p, int cta) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(cta));
  int32_t v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

constexpr int kSortBatch = 8;  // choices a lane loads at a time

// The experts of a lane's choices i0 + lane, i0 + 32 + lane, ..., -1 where there is none.
template <typename I>
__device__ __forceinline__ void load_experts(const I* e, int64_t i0, int64_t last, int experts, int (&out)[kSortBatch]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < kSortBatch; ++j) {
    const int64_t i = i0 + 32 * j + lane;
    out[j] = i < last ? expert_at(e, i, experts) : -1;
  }
}

// A stable counting sort by one cluster of CTAs for each group. Every warp owns a run of the choices and counts its
// experts in shared memory; a column's counts become the warps' starts in order, the CTAs' sums are exchanged through
// distributed shared memory, and a scan over the experts gives the offsets. Each warp then walks its run again, 32
// choices at a time: a choice's row is its expert's start, plus what the warp has placed there, plus the earlier lanes
// with the same expert. Latency bounds it (16 x 2 choices of 64 experts 3.1 us, an empty launch some 2.3; 8192 x 2 of 32
// 6.0): the choices are loaded eight at a time and, where they fit, once, the peers' sums all at once.
template <typename I>
__global__ void __launch_bounds__(kSortThreads) k_expert_sort(const __grid_constant__ SortArgs a) {
  extern __shared__ int32_t sort_smem[];
  __shared__ int32_t scan[2][kSortWarps];
  free_launches();  // (a few CTAs: the dispatch behind it may take its places)
  int32_t* hist = sort_smem;                // [warps][tile]
  int32_t* sums = hist + a.warps * a.tile;  // [tile]: this CTA's choices of every expert
  int32_t* start = sums + a.tile;           // [tile]: the first row of this CTA's
  const int threads = blockDim.x;
  const int ctas = static_cast<int>(cluster_nctarank()), rank = static_cast<int>(cluster_ctarank());
  const int g = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const I* expert_of = static_cast<const I*>(a.expert_of) + g * a.n;
  int32_t* row_of = a.row_of + g * a.n;
  int32_t* choice_of = a.choice_of ? a.choice_of + g * a.n : nullptr;
  const int64_t at = static_cast<int64_t>(rank * a.warps + warp) * a.seg;
  const int64_t first = warp < a.warps ? (at < a.n ? at : a.n) : a.n;
  const int64_t last = first + a.seg < a.n ? first + a.seg : a.n;
  int32_t* mine = hist + (warp < a.warps ? warp : 0) * a.tile;
  const bool kept = a.seg <= 32 * kSortBatch;  // a lane's choices fit its registers
  int kept_e[kSortBatch];
  if (kept) load_experts(expert_of, first, last, a.experts, kept_e);
  int32_t base = 0;  // rows of the experts before this tile's
  for (int e0 = 0; e0 < a.experts || e0 == 0; e0 += a.tile) {
    const int ne = a.experts - e0 < a.tile ? a.experts - e0 : a.tile;
    if (e0 > 0) __syncthreads();  // every warp has placed the last tile's
    for (int i = threadIdx.x; i < a.warps * a.tile; i += threads) hist[i] = 0;
    __syncthreads();
    for (int64_t i0 = first; i0 < last; i0 += 32 * kSortBatch) {
      int e[kSortBatch];
      if (!kept) load_experts(expert_of, i0, last, a.experts, e);
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j)
        if (kept) e[j] = kept_e[j];
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j)
        if (e[j] >= e0 && e[j] < e0 + ne) atomicAdd(mine + e[j] - e0, 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < ne; e += threads) {
      int32_t s = 0;
      for (int w0 = 0; w0 < a.warps; w0 += 8) {  // (eight at a time: their loads do not wait for one another)
        int32_t c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = w0 + j < a.warps ? hist[(w0 + j) * a.tile + e] : 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (w0 + j < a.warps) hist[(w0 + j) * a.tile + e] = s;
          s += c[j];
        }
      }
      sums[e] = s;
    }
    cluster_sync();  // every CTA's sums are there
    int turn = 0;
    for (int b = 0; b < ne; b += threads, turn ^= 1) {
      const int e = b + threadIdx.x;
      int32_t before = 0, all = 0;
      if (e < ne)
        for (int c0 = 0; c0 < ctas; c0 += 8) {  // (eight at a time: their loads do not wait for one another)
          int32_t s[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) s[c] = c0 + c < ctas ? ld_peer(sums + e, c0 + c) : 0;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            all += s[c];
            if (c0 + c < rank) before += s[c];
          }
        }
      int32_t incl = all;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int32_t v = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += v;
      }
      if (lane == 31) scan[turn][warp] = incl;
      __syncthreads();
      int32_t sum = lane < threads >> 5 ? scan[turn][lane] : 0;  // the warps' sums, scanned by every warp
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int32_t v = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += v;
      }
      const int32_t total = __shfl_sync(0xffffffffu, sum, 31);
      const int32_t earlier = __shfl_sync(0xffffffffu, sum, warp > 0 ? warp - 1 : 0);
      const int32_t here = base + (warp > 0 ? earlier : 0) + incl - all;
      if (e < ne) {
        start[e] = here + before;
        if (rank == 0)
          for (int r = 0; r < a.nranks; ++r)
            a.offsets[static_cast<int64_t>(g * a.nranks + r) * (a.experts + 1) + e0 + e] = here;
      }
      base += total;
    }
    cluster_arrive();  // this CTA reads no more of them
    __syncthreads();
    for (int64_t i0 = first; i0 < last; i0 += 32 * kSortBatch) {
      int all_e[kSortBatch];
      if (!kept) load_experts(expert_of, i0, last, a.experts, all_e);
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j)
        if (kept) all_e[j] = kept_e[j];
#pragma unroll
      for (int j = 0; j < kSortBatch; ++j) {
        const int64_t i = i0 + 32 * j + lane;
        if (i0 + 32 * j >= last) break;  // (the whole warp)
        const int e = all_e[j] >= e0 && all_e[j] < e0 + ne ? all_e[j] - e0 : -1;
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        int32_t pos = -1;
        if (e >= 0) pos = start[e] + mine[e] + __popc(peers & ((1u << lane) - 1));
        __syncwarp();
        if (e >= 0 && (peers >> lane) == 1u) mine[e] += __popc(peers);  // (the last lane of them)
        __syncwarp();
        if (i < last) {
          if (e >= 0) {
            row_of[i] = pos;
            if (choice_of) choice_of[pos] = static_cast<int32_t>(i);
          } else if (all_e[j] < 0 && e0 == 0) {
            row_of[i] = -1;
          }
        }
      }
    }
    cluster_wait();  // nobody does: they may be written again, or the CTA leave
  }
  if (rank == 0 && threadIdx.x < a.nranks)
    a.offsets[static_cast<int64_t>(g * a.nranks + threadIdx.x) * (a.experts + 1) + a.experts] = base;
  if (choice_of)
    for (int64_t p = static_cast<int64_t>(base) + rank * threads + threadIdx.x; p < a.n; p += ctas * threads)
      choice_of[p] = -1;
}

// ---------------------------------------------------------------- dispatch

constexpr int kThreads = 256;

struct DispatchArgs {
  ExpertTables t;
  const int32_t* row_of;  // [groups][tokens][choices]
  int64_t tokens, rows;
  int32_t choices, nranks;
  int32_t nvec, nscales;  // 16-byte vectors of a row, scales of a row
  int32_t tpr_log2;
};

// A token belongs to `tpr` threads (blockDim / tpr tokens a block) of each of the blocks of grid z, which hold kHeld of
// its vectors each at a time and write them to one choice's row after another; grid y: groups. HBM bounds it: 8192 tokens of
// two experts, 4096 columns of bf16, 36.3 us with the sort ahead of it, of which 29.4 are their bytes. (A thread a vector,
// which divides for its token and reads the indexes itself, took twice the instructions and 39.0.)
constexpr int kHeld = 2;

__global__ void __launch_bounds__(kThreads) k_expert_dispatch(const __grid_constant__ DispatchArgs a) {
  await_launches();
  const int g = blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int tt = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = kThreads >> a.tpr_log2;
  const float* scales = a.t.in_scales[g];
  const int nout = a.t.nout[g], slot0 = g * a.nranks;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * rpb + slot; t < a.tokens;
       t += static_cast<int64_t>(gridDim.x) * rpb) {
    const char* x = static_cast<const char*>(a.t.in[g]) + t * a.nvec * 16;
    const int32_t* row_of = a.row_of + (g * a.tokens + t) * a.choices;
    for (int c0 = blockIdx.z * kHeld * tpr + tt; c0 < a.nvec; c0 += gridDim.z * kHeld * tpr) {
      uint4 v[kHeld];
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (c0 + i * tpr < a.nvec) v[i] = ld_stream(x + static_cast<int64_t>(c0 + i * tpr) * 16);
      for (int k = 0; k < a.choices; ++k) {
        const int64_t row = row_of[k];
        if (row < 0 || row >= a.rows) continue;
        for (int q = 0; q < nout; ++q) {
          uint4* to = static_cast<uint4*>(a.t.out[slot0 + q]) + row * a.nvec + c0;
#pragma unroll
          for (int i = 0; i < kHeld; ++i)
            if (c0 + i * tpr < a.nvec) __stcs(to + i * tpr, v[i]);
        }
      }
    }
    for (int c = blockIdx.z * tpr + tt; c < a.nscales; c += gridDim.z * tpr) {
      const float v = scales[t * a.nscales + c];
      for (int k = 0; k < a.choices; ++k) {
        const int64_t row = row_of[k];
        if (row >= 0 && row < a.rows)
          for (int q = 0; q < nout; ++q) a.t.out_scales[slot0 + q][row * a.nscales + c] = v;
      }
    }
  }
}

// ----------------------------------------------------------------- combine

// sum_all in pairs.
template <typename T, int NR>
__device__ __forceinline__ Vec8 sum_vec(const void* const* in, int nranks, int64_t c) {
  Vec8 s;
  if constexpr (NR > 0) {
    Chunk<T> raw[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) raw[r].load(in[r], c);
    s = values<T>(raw[0]);
#pragma unroll
    for (int r = 1; r < NR; ++r) s = s + values<T>(raw[r]);
  } else {
    s = splat8(-0.0f);  // (added to anything, it leaves that as it is)
    for (int r0 = 0; r0 < nranks; r0 += 4) {
      Chunk<T> raw[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < nranks) raw[r].load(in[r0 + r], c);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r0 + r < nranks) s = s + values<T>(raw[r]);
    }
  }
  return s;
}

// acc + s * w, product and sum each rounded. The products are single ones: the compiler contracts a pair's product and the
// sum after it, in spite of their .rn, which leaves out the product's rounding.
__device__ __forceinline__ Vec8 add_weighted(const Vec8& acc, const Vec8& s, float w) {
  float f[kChunk];
  unpack8(s, f);
#pragma unroll
  for (int j = 0; j < kChunk; ++j) f[j] = __fmul_rn(f[j], w);
  return acc + Vec8{{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])}};
}

struct CombineArgs {
  ExpertTables t;
  const int32_t* row_of;  // [groups][tokens][choices]
  const float* gates;     // the same shape, or null (ones)
  int64_t tokens, rows;
  int32_t choices, nranks, nchunks;
  int32_t tpr_log2;
};

// How many chunks a thread takes and how many choices at a time, so that some loads are under way. MANY: more than two
// choices (8 of 2048 columns, one rank: 116 us, 5.8 TB/s; 132 with a choice at a time, 130 with two of two chunks). Eight
// ranks' rows of two experts, 8192 x 4096: 175 us, at the copy rate; their own sums 264 (90 %).
template <int NR, bool MANY>
struct CombineShape {
  static constexpr int ITEMS = NR == 1 && !MANY ? 2 : 1;
  static constexpr int AHEAD = NR == 1 && MANY ? 4 : NR == 8 || NR == 0 ? 1 : 2;
};

// A token belongs to `tpr` threads (blockDim / tpr tokens a block) of each of the blocks of grid z. SUMMED: grid y counts
// groups, whose ranks' rows are added up, with the residual, for every distinct output. Otherwise it counts ranks, each with
// an output of its own (NR is 1). A choice's rows are added over the ranks first (in order), then weighted; product and sum
// are rounded one by one.
template <typename T, int NR, bool SUMMED, bool MANY>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2)
    k_expert_combine(const __grid_constant__ CombineArgs a) {
  constexpr int ITEMS = CombineShape<NR, MANY>::ITEMS, AHEAD = CombineShape<NR, MANY>::AHEAD;
  const int g = SUMMED ? blockIdx.y : blockIdx.y / a.nranks;
  const int slot0 = SUMMED ? g * a.nranks : blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int tt = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = kThreads >> a.tpr_log2;
  const void* const* in = a.t.in + slot0;
  const void* residual = SUMMED ? a.t.residual[g] : nullptr;
  const int nout = SUMMED ? a.t.nout[g] : 1;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * rpb + slot; t < a.tokens;
       t += static_cast<int64_t>(gridDim.x) * rpb) {
    const int64_t at = (g * a.tokens + t) * a.choices;
    for (int c0 = blockIdx.z * ITEMS * tpr + tt; c0 < a.nchunks; c0 += gridDim.z * ITEMS * tpr) {
      Chunk<T> res[ITEMS];
      Vec8 acc[ITEMS];
#pragma unroll
      for (int u = 0; u < ITEMS; ++u) {
        if (residual && c0 + u * tpr < a.nchunks) res[u].load(residual, t * a.nchunks + c0 + u * tpr);
        acc[u] = splat8(0.0f);
      }
      int32_t next_row = -1;  // (one choice at a time: the next one's index and weight are under way with this one's data)
      float next_w = 1.0f;
      if (AHEAD == 1 && a.choices > 0) {
        next_row = a.row_of[at];
        if (a.gates) next_w = a.gates[at];
      }
      for (int k0 = 0; k0 < a.choices; k0 += AHEAD) {
        int32_t row[AHEAD];
        float w[AHEAD];
        if constexpr (AHEAD == 1) {
          row[0] = next_row;
          w[0] = next_w;
          if (k0 + 1 < a.choices) {
            next_row = a.row_of[at + k0 + 1];
            if (a.gates) next_w = a.gates[at + k0 + 1];
          }
        } else {
#pragma unroll
          for (int k = 0; k < AHEAD; ++k) {
            row[k] = k0 + k < a.choices ? a.row_of[at + k0 + k] : -1;
            w[k] = a.gates && k0 + k < a.choices ? a.gates[at + k0 + k] : 1.0f;
          }
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
          if (row[k] >= a.rows) row[k] = -1;
        if constexpr (NR > 0) {
          Chunk<T> raw[ITEMS][AHEAD][NR];
#pragma unroll
          for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int u = 0; u < ITEMS; ++u)
              if (row[k] >= 0 && c0 + u * tpr < a.nchunks)
#pragma unroll
                for (int r = 0; r < NR; ++r)
                  raw[u][k][r].load(in[r], static_cast<int64_t>(row[k]) * a.nchunks + c0 + u * tpr);
#pragma unroll
          for (int k = 0; k < AHEAD; ++k)
#pragma unroll
            for (int u = 0; u < ITEMS; ++u)
              if (row[k] >= 0 && c0 + u * tpr < a.nchunks) {
                Vec8 s = values<T>(raw[u][k][0]);
#pragma unroll
                for (int r = 1; r < NR; ++r) s = s + values<T>(raw[u][k][r]);
                acc[u] = add_weighted(acc[u], s, w[k]);
              }
        } else if (row[0] >= 0) {
          const Vec8 s = sum_vec<T, 0>(in, a.nranks, static_cast<int64_t>(row[0]) * a.nchunks + c0);
          acc[0] = add_weighted(acc[0], s, w[0]);
        }
      }
#pragma unroll
      for (int u = 0; u < ITEMS; ++u) {
        if (c0 + u * tpr >= a.nchunks) break;
        if (residual) acc[u] = acc[u] + values<T>(res[u]);
        const Chunk<T> o = rounded<T>(acc[u]);
        for (int q = 0; q < nout; ++q) o.store(a.t.out[slot0 + q], t * a.nchunks + c0 + u * tpr);
      }
    }
  }
}

// -------------------------------------------------------- combine backward

struct CombineBwdArgs {
  ExpertTables t;         // in: every rank's rows (all null without dgates); residual: dout of every group
  const int32_t* row_of;  // [groups][tokens][choices]
  const float* gates;     // or null (ones)
  float* dgates;          // or null
  int64_t tokens, rows;
  int32_t choices, nranks, nchunks;
  int32_t tpr_log2;
};

constexpr int kDots = 4;  // choices whose products are summed at a time

// kDots sums over the threads of a token, as row_sum; tokens that share a block have a barrier each.
__device__ __forceinline__ void token_sums(float (&v)[kDots], int tpr, int slot, float (*red)[kDots][32], int turn) {
#pragma unroll
  for (int i = 0; i < kDots; ++i) v[i] = warp_sum(v[i]);
  if (tpr == 32) return;
  const int warp = threadIdx.x >> 5, warps = tpr >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < kDots; ++i) red[turn][i][warp] = v[i];
  if (blockDim.x == tpr || blockDim.x > 15 * tpr) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(tpr) : "memory");
  const int first = warp & ~(warps - 1), i = threadIdx.x & (tpr - 1);
  if (i < kDots) {  // (thread i has the i-th sum)
    float s = red[turn][i][first];
    for (int w = 1; w < warps; ++w) s += red[turn][i][first + w];
    v[0] = s;
  }
}

// Blocks an SM: a token's waits, for its indexes, its rows and its barrier, follow one another, and other blocks fill them.
// 8192 tokens of two experts, 4096 columns of bf16, one rank: 101 us with two blocks, 80 with three, 78 with four; three
// ranks 121 and 102 with two and three; eight ranks 186 and 191. (Blocks that stay, with the next token's indexes and
// gradient under way, took 80, 103 and 203.)
template <typename T, int NR, int VPT, int THREADS>
constexpr int bwd_blocks() {
  if (THREADS == 1024) return 1;
  if (sizeof(T) == 4 || VPT > 1 || NR == 0 || NR > 4) return 2;
  return NR == 1 ? 4 : 3;
}

// A token belongs to `tpr` threads, which keep its gradient in registers; grid y: groups.
template <typename T, int NR, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS, bwd_blocks<T, NR, VPT, THREADS>())
    k_expert_combine_backward(const __grid_constant__ CombineBwdArgs a) {
  __shared__ float red[2][kDots][32];
  const int g = blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int tt = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = blockDim.x >> a.tpr_log2;
  const void* const* in = a.t.in + g * a.nranks;
  const int slot0 = g * a.nranks, nout = a.t.nout[g];
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.tokens;
       base += static_cast<int64_t>(gridDim.x) * rpb) {
    const int64_t t = base + slot;
    const bool live = t < a.tokens;
    const int64_t at = (g * a.tokens + t) * a.choices;
    Chunk<T> d[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = tt + i * tpr;
      if (live && c < a.nchunks) d[i].load(a.t.residual[g], t * a.nchunks + c);
    }
    for (int k0 = 0; k0 < a.choices; k0 += kDots) {
      int32_t row[kDots];
#pragma unroll
      for (int k = 0; k < kDots; ++k) {
        row[k] = live && k0 + k < a.choices ? a.row_of[at + k0 + k] : -1;
        if (row[k] >= a.rows) row[k] = -1;
      }
      float dot[kDots];
#pragma unroll
      for (int k = 0; k < kDots; ++k) {
        dot[k] = 0.0f;
        if (row[k] < 0 || !a.dgates) continue;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = tt + i * tpr;
          if (c < a.nchunks) {
            const Vec8 f = sum_vec<T, NR>(in, a.nranks, static_cast<int64_t>(row[k]) * a.nchunks + c);
            dot[k] += sum8(f * values<T>(d[i]));
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kDots; ++k) {
        if (row[k] < 0) continue;
        const float w = a.gates ? a.gates[at + k0 + k] : 1.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const int c = tt + i * tpr;
          if (c < a.nchunks) {
            const Chunk<T> ov = rounded<T>(values<T>(d[i]) * splat8(w));
            for (int q = 0; q < nout; ++q) ov.store(a.t.out[slot0 + q], static_cast<int64_t>(row[k]) * a.nchunks + c);
          }
        }
      }
      if (a.dgates) {
        token_sums(dot, tpr, slot, red, turn);
        turn ^= 1;
        if (tpr == 32) {
#pragma unroll
          for (int k = 0; k < kDots; ++k)
            if (live && tt == k && k0 + k < a.choices) a.dgates[at + k0 + k] = dot[k];
        } else if (live && tt < kDots && k0 + tt < a.choices) {
          a.dgates[at + k0 + tt] = dot[0];
        }
      }
    }
  }
}

// --------------------------------------------------------------- launchers

// Threads of a token: a power of two for `items` steps, a warp to a block; and the blocks for all tokens.
int token_threads_log2(int64_t items) {
  int log2 = 5;
  while ((1 << log2) < items && (1 << log2) < kThreads) ++log2;
  return log2;
}

// Blocks that share a token: one for each step of its threads.
int parts_for(int64_t columns, int step) {
  const int64_t want = (columns + step - 1) / step;
  return static_cast<int>(want < 1 ? 1 : want < 65535 ? want : 65535);
}

int blocks_for(int64_t tokens, int tpr_log2) {
  const int64_t rpb = kThreads >> tpr_log2, want = (tokens + rpb - 1) / rpb, most = 1 << 30;
  return static_cast<int>(want < most ? want : most);
}

template <typename T, int NR, bool SUMMED, bool MANY = false>
cudaError_t combine_go(CombineArgs& a, int ngroups, cudaStream_t s) {
  constexpr int ITEMS = CombineShape<NR, MANY>::ITEMS;
  a.tpr_log2 = token_threads_log2((a.nchunks + ITEMS - 1) / ITEMS);
  const dim3 grid(blocks_for(a.tokens, a.tpr_log2), SUMMED ? ngroups : ngroups * a.nranks,
                  parts_for(a.nchunks, ITEMS << a.tpr_log2));
  k_expert_combine<T, NR, SUMMED, MANY><<<grid, kThreads, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t combine_ranks(CombineArgs& a, bool summed, int ngroups, cudaStream_t s) {
  const bool many = a.choices > 2;
  if (!summed) return many ? combine_go<T, 1, false, true>(a, ngroups, s) : combine_go<T, 1, false>(a, ngroups, s);
  if (a.nranks == 1 && many) return combine_go<T, 1, true, true>(a, ngroups, s);
  return with_ranks<1, 2, 3, 4, 8>(a.nranks, [&](auto n) { return combine_go<T, n.value, true>(a, ngroups, s); });
}

template <typename T, int NR, int VPT, int THREADS>
cudaError_t combine_bwd_go(const CombineBwdArgs& a, int ngroups, cudaStream_t s) {
  const int tpr = 1 << a.tpr_log2;
  const int threads = THREADS == 1024 ? 1024 : tpr < 256 ? 256 : tpr, rpb = threads / tpr;
  const int64_t blocks = (a.tokens + rpb - 1) / rpb;
  const dim3 grid(static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30)), ngroups);
  k_expert_combine_backward<T, NR, VPT, THREADS><<<grid, threads, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t combine_bwd_shape(CombineBwdArgs& a, int ngroups, cudaStream_t s) {
  a.tpr_log2 = 5;
  while (a.tpr_log2 < 9 && (1 << a.tpr_log2) < a.nchunks) ++a.tpr_log2;
  if (a.nchunks <= 512)
    return with_ranks<1, 2, 3, 4, 8>(a.nranks, [&](auto n) { return combine_bwd_go<T, n.value, 1, 512>(a, ngroups, s); });
  if (a.nchunks <= 1024)
    return with_ranks<1, 2, 8>(a.nranks, [&](auto n) { return combine_bwd_go<T, n.value, 2, 512>(a, ngroups, s); });
  a.tpr_log2 = 10;
  if (a.nchunks <= 2048)
    return with_ranks<1>(a.nranks, [&](auto n) { return combine_bwd_go<T, n.value, 2, 1024>(a, ngroups, s); });
  return combine_bwd_go<T, 0, 4, 1024>(a, ngroups, s);
}

}  // namespace

// What a kernel needs once per device: leave for the most dynamic shared memory that comes here, and for clusters of more
// than eight CTAs; and whether the device has room for one of sixteen. (Leaves are the process's, so no call can take
// another's.)
static cudaError_t sort_setup(const void* fn, bool index64, bool* wide) {
  static std::atomic<int> known[2][64];  // 0 not yet, 1 clusters of eight, 2 of sixteen
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < 64;
  int k = kept ? known[index64][dev].load(std::memory_order_acquire) : 0;
  if (k == 0) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSortSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = kSortSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 16;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = 0;
    k = cudaOccupancyMaxActiveClusters(&fit, fn, &cfg) == cudaSuccess && fit > 0 ? 2 : 1;
    (void)cudaGetLastError();  // (a device that has none says so as an error)
    if (kept) known[index64][dev].store(k, std::memory_order_release);
  }
  *wide = k == 2;
  return cudaSuccess;
}

cudaError_t launch_expert_sort(const ExpertSortLaunch& L, cudaStream_t s) {
  SortArgs a;
  a.expert_of = L.expert_of;
  a.row_of = L.row_of;
  a.choice_of = L.choice_of;
  a.offsets = L.offsets;
  a.n = L.n;
  a.experts = L.experts;
  a.nranks = L.nranks;
  a.tile = L.experts < kSortTile ? (L.experts > 0 ? L.experts : 1) : kSortTile;
  const void* fn = L.index64 ? reinterpret_cast<const void*>(&k_expert_sort<int64_t>)
                             : reinterpret_cast<const void*>(&k_expert_sort<int32_t>);
  bool wide_clusters = false;
  cudaError_t e = sort_setup(fn, L.index64, &wide_clusters);
  if (e != cudaSuccess) return e;
  // One CTA, of as many threads as there are choices or experts, or eight, or sixteen. Measured on 1, 8 and 16, us: 512
  // choices of 32 experts 4.1, 4.9, 5.1; 1024 5.4, 5.5, 5.7; 4096 7.3, 5.8, 5.9; 16384 16.3, 6.2, 5.9; 131072 of 64 105,
  // 18.1, 10.6, of 1024 136, 24.4, 16.8. Where counting more experts than that is most of the work, more CTAs only repeat
  // it (16384 of 8192: 25 on eight, 31 on sixteen).
  const bool sixteen = wide_clusters && L.n > 8 * kSortThreads && L.experts <= 2048;
  const int ctas = L.n <= kSortThreads ? 1 : sixteen ? 16 : 8;
  const int64_t wide = L.n > L.experts ? L.n : L.experts;
  const int threads = ctas > 1 || wide >= kSortThreads ? kSortThreads
                      : wide <= 128                    ? 128
                                                       : static_cast<int>((wide + 31) / 32 * 32);
  const int most = kSortSmem / (4 * a.tile) - 2;
  const int filled = static_cast<int>(L.n < kSortThreads ? (L.n + 31) / 32 : kSortWarps);
  a.warps = most < threads / 32 ? most : threads / 32;
  if (a.warps > filled && ctas == 1) a.warps = filled > 0 ? filled : 1;
  a.seg = (L.n + ctas * a.warps - 1) / (ctas * a.warps);
  a.seg = (a.seg + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, L.ngroups);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.warps + 2) * a.tile * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = L.index64 ? cudaLaunchKernelEx(&cfg, k_expert_sort<int64_t>, a) : cudaLaunchKernelEx(&cfg, k_expert_sort<int32_t>, a);
  count_launch();
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_expert_dispatch(const ExpertRowsLaunch& L, cudaStream_t s) {
  DispatchArgs a;
  a.t = L.t;
  a.row_of = L.row_of;
  a.tokens = L.tokens;
  a.rows = L.rows;
  a.choices = L.choices;
  a.nranks = L.nranks;
  a.nvec = static_cast<int32_t>(static_cast<int64_t>(L.cols) * dtype_size(L.dtype) / 16);
  a.nscales = L.dtype == COCO_F8E4M3 ? static_cast<int32_t>((static_cast<int64_t>(L.cols) + 127) / 128) : 0;
  a.tpr_log2 = token_threads_log2((a.nvec + kHeld - 1) / kHeld);
  const dim3 grid(blocks_for(a.tokens, a.tpr_log2), L.ngroups, parts_for(a.nvec, kHeld << a.tpr_log2));
  const cudaError_t e = launch_early(k_expert_dispatch, grid, dim3(kThreads), s, a);
  count_launch();
  return e;
}

cudaError_t launch_expert_combine(const ExpertRowsLaunch& L, cudaStream_t s) {
  CombineArgs a;
  a.t = L.t;
  a.row_of = L.row_of;
  a.gates = L.gates;
  a.tokens = L.tokens;
  a.rows = L.rows;
  a.choices = L.choices;
  a.nranks = L.nranks;
  a.nchunks = L.cols / kChunk;
  switch (L.dtype) {
    case COCO_F32: return combine_ranks<float>(a, L.summed, L.ngroups, s);
    case COCO_F16: return combine_ranks<__half>(a, L.summed, L.ngroups, s);
    default: return combine_ranks<__nv_bfloat16>(a, L.summed, L.ngroups, s);
  }
}

cudaError_t launch_expert_combine_backward(const ExpertRowsLaunch& L, cudaStream_t s) {
  CombineBwdArgs a;
  a.t = L.t;
  a.row_of = L.row_of;
  a.gates = L.gates;
  a.dgates = L.dgates;
  a.tokens = L.tokens;
  a.rows = L.rows;
  a.choices = L.choices;
  a.nranks = L.nranks;
  a.nchunks = L.cols / kChunk;
  switch (L.dtype) {
    case COCO_F32: return combine_bwd_shape<float>(a, L.ngroups, s);
    case COCO_F16: return combine_bwd_shape<__half>(a, L.ngroups, s);
    default: return combine_bwd_shape<__nv_bfloat16>(a, L.ngroups, s);
  }
}

}  // namespace coco
