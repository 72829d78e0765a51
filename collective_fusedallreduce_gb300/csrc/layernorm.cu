// The layer norm that follows a tensor-parallel layer's AllReduce:
//
//   h = sum_r partial_r + residual,  m = mean(h),  v = mean((h - m)^2),
//   y = (h - m) * rsqrt(v + eps) * w + b
//   (Ba, Kiros and Hinton, "Layer Normalization", 2016),
//
// with y stored in the stream's type or as e4m3 values with one scale per row and
// 128 columns. Rows are held as in norm.cu, and HBM bounds the pass.
//
// The statistics need one exchange between warps, as the root mean square does: a
// warp takes the mean of its own columns and the sum of squares about that mean
// (from registers), and the warps' pairs are joined by
//
//   m = sum n_i m_i / n,   n v = sum (q_i + n_i (m_i - m)^2)
//   (Chan, Golub and LeVeque, "Updating formulae and a pairwise algorithm for
//   computing sample variances", 1979),
//
// so nothing is lost where a row's mean is large against its spread.
//
// Measured, from a graph: 8192 x 4096 fp16 on 8 ranks, 8 copies, 248 us (6.8 TB/s, the
// copy rate); fp32 on 8 ranks, one copy, 212. Few ranks' rows are bound by
// instructions (3.2 a cycle of 4 are issued): bf16 on 2 ranks 58 us (5.8 TB/s), to 8
// bits 66; on one 52; 4096 x 16384 on one 98 (5.5 TB/s), 3106 x 10784 bf16 59. Far from
// the bytes' time: 2048 x 32768 bf16 on one rank 152 us (3.5 TB/s), 1024 x 32768 fp32 224
// (registers spill), 8192 x 4096 bf16 on 5 ranks 136 (3.9 TB/s).

#include "internal.h"
#include "rows.h"

namespace coco {
namespace {

struct LayerNormArgs {
  NormTables t;
  int64_t rows;
  int32_t nranks;
  int32_t cols, nchunks, nblocks;  // nblocks: scales per row
  int32_t tpr_log2;
  int32_t ahead;  // how many rows ahead one is brought to L2
  float eps;
  const void* weight;
  const void* bias;
  float* mean;
  float* rstd;
};

// The elements of a row that warp `w` of its threads holds.
__device__ __forceinline__ int warp_columns(int w, int tpr, int nchunks, int vpt) {
  int n = 0;
  for (int i = 0; i < vpt; ++i) {
    const int left = nchunks - (i * tpr + 32 * w);
    n += left < 0 ? 0 : left > 32 ? 32 : left;
  }
  return n * kChunk;
}

// Rows of up to 4096 columns have one chunk a thread, many narrow ones of one or two ranks two, wider ones two to four
// (norm_shape has the rules).
// AHEAD: few ranks' rows are loaded a row ahead, by blocks that stay and walk the rows.
template <typename T, int NR, int VPT, int THREADS>
struct NormShape {
  static constexpr bool AHEAD = NR > 0 && VPT < 3 && VPT * (NR + 1) * sizeof(T) <= (VPT == 1 ? 8 : 12);
  static constexpr int BLOCKS = THREADS == 1024 ? 1 : VPT == 1 && NR > 0 && sizeof(T) == 2 ? 3 : 2;
};

// A thread's part of the rows of NR ranks and the residual, as loaded.
template <typename T, int NR, int VPT>
struct RowPart {
  Chunk<T> v[VPT][NR + 1];
  __device__ __forceinline__ void load(const void* const* in, const void* residual, bool live, int64_t c0, int t, int tpr,
                                       int nchunks) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < nchunks) {
#pragma unroll
        for (int r = 0; r < NR; ++r) v[i][r].load(in[r], c0 + c);
        if (residual) v[i][NR].load(residual, c0 + c);
      }
    }
  }
};

// Grid x: rows (blockDim / tpr a block), grid y: groups.
template <typename T, int NR, int VPT, int THREADS, bool FP8>
__global__ void __launch_bounds__(THREADS, NormShape<T, NR, VPT, THREADS>::BLOCKS)
    k_allreduce_layernorm(const __grid_constant__ LayerNormArgs a) {
  __shared__ float2 red[2][32];
  __shared__ float counts[32];  // the elements that each warp of a row holds
  const int g = blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int t = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = blockDim.x >> a.tpr_log2;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = tpr >> 5, first = warp & ~(warps - 1);
  const void* const* in = a.t.in + g * a.nranks;
  const void* residual = a.t.residual[g];
  const int nhidden = a.t.nhidden[g], nnormed = a.t.nnormed[g];
  const int slot0 = g * a.nranks;
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  const int filled = a.nchunks + 31 < tpr ? (a.nchunks + 31) >> 5 : warps;  // a row's warps that hold any of it
  const int mine_n = warp_columns(warp - first, tpr, a.nchunks, VPT);
  const float inv_n = mine_n ? 1.0f / static_cast<float>(mine_n) : 0.0f;
  if (t % 32 == 0 && slot == 0) counts[warp] = static_cast<float>(mine_n);  // (read behind a row's barrier)
  int turn = 0;
  using S = NormShape<T, NR, VPT, THREADS>;
  RowPart<T, S::AHEAD ? NR : 0, S::AHEAD ? VPT : 1> part;
  if constexpr (S::AHEAD) {
    const int64_t row = static_cast<int64_t>(blockIdx.x) * rpb + slot;
    part.load(in, residual, row < a.rows, row * a.nchunks, t, tpr, a.nchunks);
  }
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.rows;
       base += static_cast<int64_t>(gridDim.x) * rpb, turn ^= 1) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    const int64_t c0 = row * a.nchunks;
    if constexpr (VPT > 1 && !S::AHEAD) {
      // A row that a later block will take is brought to L2 meanwhile: a row's loads, its barrier and its stores do not
      // overlap, and there are few rows on an SM.
      const int64_t ahead = row + a.ahead;
      if (ahead < a.rows)
        for (int i = t; i < a.nranks + 1; i += tpr) {
          const void* p = i < a.nranks ? in[i] : residual;
          const int bytes = a.cols * static_cast<int>(sizeof(T));
          if (p)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(p) + ahead * bytes),
                         "r"(bytes)
                         : "memory");
        }
    }
    float h[VPT][kChunk];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < a.nchunks) {
        float f[kChunk];
        Chunk<T> res;
        if constexpr (S::AHEAD) {
          part.v[i][0].get(h[i]);
#pragma unroll
          for (int r = 1; r < NR; ++r) {
            part.v[i][r].get(f);
#pragma unroll
            for (int j = 0; j < kChunk; ++j) h[i][j] += f[j];
          }
          res = part.v[i][NR];
        } else {
          if (residual) res.load(residual, c0 + c);
          sum_all<T, NR>(in, a.nranks, c0 + c, h[i]);
        }
        if (residual) {
          res.get(f);
#pragma unroll
          for (int j = 0; j < kChunk; ++j) h[i][j] += f[j];
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j) s += h[i][j];
      } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) h[i][j] = 0.0f;
      }
    }
    if constexpr (S::AHEAD) {
      const int64_t next = row + static_cast<int64_t>(gridDim.x) * rpb;
      part.load(in, residual, next < a.rows, next * a.nchunks, t, tpr, a.nchunks);
    }
    float mean = warp_sum(s) * inv_n, q = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (t + i * tpr < a.nchunks)
#pragma unroll
        for (int j = 0; j < kChunk; ++j) q = fmaf(h[i][j] - mean, h[i][j] - mean, q);
    q = warp_sum(q);
    if (warps > 1) {
      if ((threadIdx.x & 31) == 0) red[turn][warp] = make_float2(mean, q);
      __syncthreads();
      // Lane i has warp i's pair, and the sums over the warps are shuffles (a loop over sixteen pairs was half of a row's
      // instructions). The joint mean is warp 0's and a correction, which leaves a mean far from zero its last bits.
      const bool has = lane < filled;
      const float2 p = has ? red[turn][first + lane] : make_float2(0.0f, 0.0f);
      const float n = has ? counts[lane] : 0.0f;
      const float m0 = red[turn][first].x;
      mean = fmaf(warp_sum(has ? (p.x - m0) * n : 0.0f), inv_cols, m0);
      const float d = p.x - mean;
      q = warp_sum(has ? fmaf(d * d, n, p.y) : 0.0f);
    }
    const float rstd = rsqrtf(fmaf(q, inv_cols, a.eps));
    if (live && t == 0) {
      if (a.mean) a.mean[g * a.rows + row] = mean;
      if (a.rstd) a.rstd[g * a.rows + row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      const bool mine = live && c < a.nchunks;
      if (mine && nhidden > 0) {
        Chunk<T> o;
        o.put(h[i]);
        for (int r = 0; r < nhidden; ++r) o.store(a.t.hidden[slot0 + r], c0 + c);
      }
      float y[kChunk];
#pragma unroll
      for (int j = 0; j < kChunk; ++j) y[j] = 0.0f;
      if (mine) {
        Chunk<T> w, b;
        w.load_cached(a.weight, c);
        if (a.bias) b.load_cached(a.bias, c);
        else b.zero();
        float f[kChunk];
        w.get(y);
        b.get(f);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) y[j] = fmaf((h[i][j] - mean) * rstd, y[j], f[j]);
      }
      if constexpr (FP8) {
        float m = mine ? chunk_amax(y) : 0.0f;  // (lanes past the row's end: 0)
#pragma unroll
        for (int x = kBlockLanes / 2; x; x >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (mine) {
          const float sc = scale_of(m);
          const uint2 q8 = to_e4m3(y, sc);
          const int64_t so = row * a.nblocks + c / kBlockLanes;
          for (int r = 0; r < nnormed; ++r) {
            __stcs(static_cast<uint2*>(a.t.normed[slot0 + r]) + c0 + c, q8);
            if (c % kBlockLanes == 0) a.t.scales[slot0 + r][so] = sc;
          }
        }
      } else if (mine) {
        Chunk<T> o;
        o.put(y);
        for (int r = 0; r < nnormed; ++r) o.store(a.t.normed[slot0 + r], c0 + c);
      }
    }
  }
}

// --------------------------------------------------------------- launchers

template <typename T, int NR, int VPT, int THREADS>
cudaError_t norm_go(LayerNormArgs& a, bool fp8, int ngroups, cudaStream_t s) {
  const int tpr = 1 << a.tpr_log2;
  const int threads = THREADS == 1024 ? 1024 : tpr < 256 ? 256 : tpr, rpb = threads / tpr;
  const int64_t blocks = (a.rows + rpb - 1) / rpb;
  using S = NormShape<T, NR, VPT, THREADS>;
  // (AHEAD: as many blocks as stay on the device; else one for each step)
  int64_t most = S::AHEAD ? sm_count() * S::BLOCKS * (THREADS / threads) / ngroups : 1 << 30;
  if (most < 1) most = 1;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most), ngroups);
  // (blocks of 256 threads are twice as many; twice as far ahead, 4161 x 4608 fp32 on four ranks took 119 us, not 108)
  a.ahead = sm_count() * S::BLOCKS * rpb;
  if (fp8) k_allreduce_layernorm<T, NR, VPT, THREADS, true><<<grid, threads, 0, s>>>(a);
  else k_allreduce_layernorm<T, NR, VPT, THREADS, false><<<grid, threads, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t norm_shape(LayerNormArgs& a, bool fp8, int ngroups, cudaStream_t s) {
  // Many narrow 16-bit rows of one or two ranks have two chunks a thread, as what a row costs beside its elements is then
  // shared by more of them: 16384 x 272 15.1 -> 12.1 us, 2 x 16384 x 2048 85 -> 73. Few rows wait longer so (300 x 1024 2.8
  // -> 3.5), and rows of 4096 columns gain nothing.
  const bool pairs = sizeof(T) == 2 && a.nranks <= 2 && a.nchunks > 32 && a.nchunks <= 256 && a.rows >= 2048;
  const int threads = pairs ? (a.nchunks + 1) / 2 : a.nchunks;
  a.tpr_log2 = 5;
  while (a.tpr_log2 < 9 && (1 << a.tpr_log2) < threads) ++a.tpr_log2;
  if (pairs) return with_ranks<1, 2>(a.nranks, [&](auto n) { return norm_go<T, n.value, 2, 512>(a, fp8, ngroups, s); });
  if (a.nchunks <= 512)
    return with_ranks<1, 2, 3, 4, 8>(a.nranks, [&](auto n) { return norm_go<T, n.value, 1, 512>(a, fp8, ngroups, s); });
  // Wide rows: three chunks a thread where two would leave a quarter of the threads idle (tpr a power of two), four in place
  // of 1024 threads, so that two to four rows are on an SM instead of one or two. One and three ranks, bf16, some 268 MB:
  // 4608 columns 73.9 -> 57.2 and 74.7 -> 52.8 us, 10784 77.3 -> 59.2 and 76.0 -> 58.6, 16384 60.5 -> 56.1 and 62.2 -> 61.1;
  // fp32, two ranks, 9216 186 -> 105. Not taken where it costs: eight ranks' 4608 columns (54.6 -> 57.5), 8192 columns with
  // four chunks (two ranks 50.2 -> 57.8); other numbers of ranks, whose loop over them takes too many registers (fp32, 3669 x
  // 6096: 140 -> 154), and 6096 columns of fp32 of two (102 -> 106); few rows, which wait longer: a row an SM (40 x 13152 to
  // 8 bits, three ranks 6.8 -> 7.4; but fp32, three ranks 12.1 -> 9.5), of one rank, which are loaded ahead, eight (700 x
  // 13152 to 8 bits 23.5 -> 25.5).
  const bool few = a.nranks == 1 ? a.rows <= 8 * sm_count() : sizeof(T) == 2 && a.rows <= sm_count();
  if ((a.nranks <= 4 || a.nranks == 8) && !few) {
    if ((a.nchunks <= 768 && a.nranks < 8 && (sizeof(T) == 2 || a.nranks != 2)) || (a.nchunks > 1024 && a.nchunks <= 2048)) {
      a.tpr_log2 = a.nchunks <= 768 ? 8 : 9;
      auto go = [&](auto n) {
        return a.nchunks <= 1536 ? norm_go<T, n.value, 3, 512>(a, fp8, ngroups, s)
                                 : norm_go<T, n.value, 4, 512>(a, fp8, ngroups, s);
      };
      switch (a.nranks) {
        case 1: return go(std::integral_constant<int, 1>());
        case 2: return go(std::integral_constant<int, 2>());
        case 3: return go(std::integral_constant<int, 3>());
        case 4: return go(std::integral_constant<int, 4>());
        default: return go(std::integral_constant<int, 8>());
      }
    }
  }
  if (a.nchunks <= 1024)
    return with_ranks<1, 2, 3, 4, 8>(a.nranks, [&](auto n) { return norm_go<T, n.value, 2, 512>(a, fp8, ngroups, s); });
  a.tpr_log2 = 10;
  if (a.nchunks <= 2048)
    return with_ranks<1>(a.nranks, [&](auto n) { return norm_go<T, n.value, 2, 1024>(a, fp8, ngroups, s); });
  return norm_go<T, 0, 4, 1024>(a, fp8, ngroups, s);
}

}  // namespace

cudaError_t launch_allreduce_layernorm(const LayerNormLaunch& L, cudaStream_t s) {
  LayerNormArgs a;
  a.t = L.t;
  a.rows = L.rows;
  a.nranks = L.nranks;
  a.cols = L.cols;
  a.nchunks = L.cols / kChunk;
  a.nblocks = (L.cols + 127) / 128;
  a.eps = L.eps;
  a.weight = L.weight;
  a.bias = L.bias;
  a.mean = L.mean;
  a.rstd = L.rstd;
  switch (L.dtype) {
    case COCO_F32: return norm_shape<float>(a, L.fp8, L.ngroups, s);
    case COCO_F16: return norm_shape<__half>(a, L.fp8, L.ngroups, s);
    default: return norm_shape<__nv_bfloat16>(a, L.fp8, L.ngroups, s);
  }
}

}  // namespace coco
