// The norm that follows a tensor-parallel layer's AllReduce, its gradient, and
// the quantiser to 8 bits:
//
//   h = sum_r partial_r + residual,  y = h * rsqrt(mean(h^2) + eps) * w
//   (Zhang and Sennrich, "Root Mean Square Layer Normalization", 2019),
//
// with y stored in the stream's type or as e4m3 values with one scale per row
// and 128 columns. All of it is bound by HBM: the forward reads N + 1 rows and
// writes two, the backward reads N + 3 and writes one.
//
// Layout. A row belongs to `tpr` threads (a power of two, 32 to 1024), and a
// thread holds the row's 8-element chunks t, t + tpr, ... in fp32 registers from
// the load to the store, so every input is read once. Sixteen neighbouring lanes
// hold 128 columns: a block's maximum is four shuffles. Sums of a row are warp
// shuffles, then one shared-memory exchange in warp order, so they do not depend
// on timing.

#include <atomic>
#include <type_traits>

#include "internal.h"
#include "rows.h"

namespace coco {
namespace {

// ----------------------------------------------------------------- forward

struct NormArgs {
  NormTables t;
  int64_t rows;
  int32_t nranks;
  int32_t cols, nchunks, nblocks;  // nblocks: scales per row
  int32_t tpr_log2;
  float eps;
  const void* weight;
  float* rstd;
};

// Grid x: rows (blockDim / tpr a block), grid y: groups. A row's loads, its barrier and its stores do not overlap,
// so what keeps HBM busy is other blocks on the SM: four of 512 threads (16-bit types, the compiler held to 32
// registers, at the price of up to 40 bytes of local memory a thread in the 8-bit form) took 8192 x 4096 fp16 on eight
// ranks, eight copies, from 233 to 213 us (6.67 TB/s); three had not been enough.
template <typename T, int NR, int VPT, bool FP8>
__global__ void __launch_bounds__(512, VPT == 1 && NR > 0 && sizeof(T) == 2 ? 4 : 1)
    k_allreduce_rmsnorm(const __grid_constant__ NormArgs a) {
  __shared__ float red[2][32];
  const int g = blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int t = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = blockDim.x >> a.tpr_log2;
  const void* const* in = a.t.in + g * a.nranks;
  const void* residual = a.t.residual[g];
  const int nhidden = a.t.nhidden[g], nnormed = a.t.nnormed[g];
  const int slot0 = g * a.nranks;
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.rows;
       base += static_cast<int64_t>(gridDim.x) * rpb, turn ^= 1) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    const int64_t c0 = row * a.nchunks;
    float h[VPT][kChunk];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < a.nchunks) {
        Chunk<T> res;
        if (residual) res.load(residual, c0 + c);
        sum_ranks<T, NR>(in, a.nranks, c0 + c, h[i]);
        if (residual) {
          float f[kChunk];
          res.get(f);
#pragma unroll
          for (int j = 0; j < kChunk; ++j) h[i][j] += f[j];
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j) ss = fmaf(h[i][j], h[i][j], ss);
      } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) h[i][j] = 0.0f;
      }
    }
    ss = row_sum<false>(ss, tpr, slot, red, turn);
    const float rstd = rsqrtf(ss / static_cast<float>(a.cols) + a.eps);
    if (live && t == 0 && a.rstd) a.rstd[g * a.rows + row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      const bool mine = live && c < a.nchunks;
      if (mine && nhidden > 0) {
        Chunk<T> o;
        o.put(h[i]);
        for (int q = 0; q < nhidden; ++q) o.store(a.t.hidden[slot0 + q], c0 + c);
      }
      float y[kChunk];
      if (mine) {
        Chunk<T> w;
        w.load_cached(a.weight, c);
        w.get(y);
      } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) y[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < kChunk; ++j) y[j] *= h[i][j] * rstd;
      if constexpr (FP8) {
        float m = mine ? chunk_amax(y) : 0.0f;  // (lanes past the row's end: 0, whatever rstd is)
#pragma unroll
        for (int x = kBlockLanes / 2; x; x >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, x));
        if (mine) {
          const float s = scale_of(m);
          const uint2 q8 = to_e4m3(y, s);
          const int64_t so = row * a.nblocks + c / kBlockLanes;
          for (int q = 0; q < nnormed; ++q) {
            __stcs(static_cast<uint2*>(a.t.normed[slot0 + q]) + c0 + c, q8);
            if (c % kBlockLanes == 0) a.t.scales[slot0 + q][so] = s;
          }
        }
      } else if (mine) {
        Chunk<T> o;
        o.put(y);
        for (int q = 0; q < nnormed; ++q) o.store(a.t.normed[slot0 + q], c0 + c);
      }
    }
  }
}

// ---------------------------------------------------------------- backward
//
// With xhat = h * rstd and g = dy * w (dy: the sum of the ranks' gradients):
//   dx = rstd * (g - xhat * mean(g * xhat)) + dhidden,   dw = sum over rows of dy * xhat.
// One or two blocks an SM walk rows, as many at a time as their threads hold; a thread keeps the dw sums of its own
// columns in registers over all its rows, the block's rows join them in shared memory, and the block writes them once
// to the workspace ([blocks][cols]), which k_norm_dweight adds in block order: no atomics, so repeated calls give the
// same bits.

struct NormBwdArgs {
  const void* in[COCO_MAX_PTRS];
  const void* dhidden[COCO_MAX_PTRS];  // per group, or null
  const void* hidden[COCO_MAX_PTRS];   // per group
  void* dx[COCO_MAX_PTRS];
  int32_t ndx[COCO_MAX_PTRS];
  int64_t rows;
  int32_t nranks;
  int32_t cols, nchunks;
  int32_t tpr_log2;
  const void* weight;
  const float* rstd;
  float* partial;  // [gridDim.y * gridDim.x][cols]
};

// THREADS and blocks an SM, by the registers (64 for 1024 threads an SM): 16-bit rows of up to 8192 columns have
// two blocks of 512 threads, with two chunks a thread keeping the dw sums in shared memory (WIDE; each thread its own
// columns') and reading dhidden only when it is added; wider ones 1024 threads a row of two or four chunks, the
// latter reading hidden again (from L2) instead of keeping it. fp32 rows: 512 threads, WIDE from four chunks on. The
// wide forms keep some values in local memory all the same (up to 88 bytes a thread in 16 bits, up to 328 in fp32).
// Measured: 8192 x 4096 fp16 on eight ranks 119 us (6.2 TB/s), in fp32 233; 16384 x 1024 bf16 on two 40 us, 777 x 8192
// on two 24 us, 4096 x 16384 on one 114 us (fp32 191), 2048 x 32768 141 us; HBM bounds the first two, latency between a
// row's phases the rest.
template <typename T, int VPT, int THREADS>
struct BwdShape {
  static constexpr bool WIDE = VPT > (sizeof(T) == 2 ? 1 : 2);
  static constexpr bool AGAIN = THREADS == 1024 && VPT == 4;
  static constexpr int BLOCKS = THREADS == 512 && VPT <= 2 && sizeof(T) == 2 ? 2 : 1;
};

template <typename T, int NR, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS, BwdShape<T, VPT, THREADS>::BLOCKS)
    k_rmsnorm_backward(const __grid_constant__ NormBwdArgs a) {
  constexpr bool WIDE = BwdShape<T, VPT, THREADS>::WIDE, AGAIN = BwdShape<T, VPT, THREADS>::AGAIN;
  __shared__ float red[2][32];
  __shared__ float slots[VPT == 1 ? THREADS * kChunk : 1];  // the dw of a block's rows, to be joined
  extern __shared__ float4 wide_dw[];                   // [2 * nchunks]
  const int g = blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int t = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = blockDim.x >> a.tpr_log2;
  const void* const* in = a.in + g * a.nranks;
  const void* dhidden = a.dhidden[g];
  const void* hidden = a.hidden[g];
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  float dw[WIDE ? 1 : VPT][kChunk];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    if constexpr (WIDE) {
      const int c = t + i * tpr;
      if (c < a.nchunks) wide_dw[2 * c] = wide_dw[2 * c + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
#pragma unroll
      for (int j = 0; j < kChunk; ++j) dw[i][j] = 0.0f;
    }
  }
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.rows;
       base += static_cast<int64_t>(gridDim.x) * rpb, turn ^= 1) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    const int64_t c0 = row * a.nchunks;
    // The block's next row is brought to L2 meanwhile: a row's loads, its barrier and its stores do not overlap, and
    // there are no registers to load a row ahead (or to have more blocks on the SM). Rows of one chunk a thread on
    // eight ranks or more have enough loads under way without (8192 x 2048: 60 us, with it 65; 16384 x 1024 on two
    // ranks: 43 us, with it 38).
    const int64_t ahead = row + static_cast<int64_t>(gridDim.x) * rpb;
    if (ahead < a.rows && (VPT > 1 || a.nranks < 8))
      for (int i = t; i < a.nranks + 2; i += tpr) {
        const void* p = i < a.nranks ? in[i] : i == a.nranks ? hidden : dhidden;
        const int bytes = a.cols * static_cast<int>(sizeof(T));
        if (p)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(p) + ahead * bytes),
                       "r"(bytes)
                       : "memory");
      }
    const float rstd = live ? a.rstd[g * a.rows + row] : 0.0f;
    float gr[VPT][kChunk];
    Chunk<T> hv[WIDE && !AGAIN ? VPT : 1], dh[WIDE ? 1 : VPT];  // (narrow rows keep xhat itself)
    float xk[WIDE ? 1 : VPT][kChunk];
    float along = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < a.nchunks) {
        Chunk<T> wv;
        Chunk<T>& h = hv[WIDE && !AGAIN ? i : 0];
        h.load(hidden, c0 + c);
        if constexpr (!WIDE)
          if (dhidden) dh[i].load(dhidden, c0 + c);
        wv.load_cached(a.weight, c);
        sum_ranks<T, NR>(in, a.nranks, c0 + c, gr[i]);
        float w[kChunk], xh[kChunk], d[kChunk];
        h.get(xh);
        wv.get(w);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          xh[j] *= rstd;
          if constexpr (!WIDE) xk[i][j] = xh[j];
          d[j] = gr[i][j];
          gr[i][j] *= w[j];
          along = fmaf(gr[i][j], xh[j], along);
        }
        if constexpr (WIDE) {
          float4 u = wide_dw[2 * c], v = wide_dw[2 * c + 1];
          u.x = fmaf(d[0], xh[0], u.x); u.y = fmaf(d[1], xh[1], u.y);
          u.z = fmaf(d[2], xh[2], u.z); u.w = fmaf(d[3], xh[3], u.w);
          v.x = fmaf(d[4], xh[4], v.x); v.y = fmaf(d[5], xh[5], v.y);
          v.z = fmaf(d[6], xh[6], v.z); v.w = fmaf(d[7], xh[7], v.w);
          wide_dw[2 * c] = u;
          wide_dw[2 * c + 1] = v;
        } else {
#pragma unroll
          for (int j = 0; j < kChunk; ++j) dw[i][j] = fmaf(d[j], xh[j], dw[i][j]);
        }
      }
    }
    along = row_sum<true>(along, tpr, slot, red, turn) * inv_cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < a.nchunks) {
        float f[kChunk], o[kChunk], xh[kChunk];
        if (dhidden) {
          if constexpr (WIDE) {
            Chunk<T> late;
            late.load(dhidden, c0 + c);
            late.get(f);
          } else {
            dh[i].get(f);
          }
        } else {
#pragma unroll
          for (int j = 0; j < kChunk; ++j) f[j] = 0.0f;
        }
        if constexpr (AGAIN) {
          hv[0].load(hidden, c0 + c);
          hv[0].get(xh);
        } else if constexpr (WIDE) {
          hv[i].get(xh);
        }
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          const float x = WIDE ? xh[j] * rstd : xk[WIDE ? 0 : i][j];
          o[j] = fmaf(rstd, gr[i][j] - x * along, f[j]);
        }
        Chunk<T> ov;
        ov.put(o);
        for (int q = 0; q < a.ndx[g]; ++q) ov.store(a.dx[g * a.nranks + q], c0 + c);
      }
    }
  }
  float* out = a.partial + (static_cast<int64_t>(g) * gridDim.x + blockIdx.x) * a.cols;
  if constexpr (VPT == 1) {
    if (rpb > 1) {
#pragma unroll
      for (int j = 0; j < kChunk; ++j) slots[threadIdx.x * kChunk + j] = dw[0][j];
      __syncthreads();
      if (slot == 0)
        for (int s = 1; s < rpb; ++s)
#pragma unroll
          for (int j = 0; j < kChunk; ++j) dw[0][j] += slots[(s * tpr + t) * kChunk + j];
    }
  }
  if (slot == 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (c < a.nchunks) {
        if constexpr (WIDE) {
          reinterpret_cast<float4*>(out)[2 * c] = wide_dw[2 * c];
          reinterpret_cast<float4*>(out)[2 * c + 1] = wide_dw[2 * c + 1];
        } else {
          Chunk<float> o;
          o.put(dw[i]);
          o.store(out, c);
        }
      }
    }
  }
}

// dweight[c] = the sum over the workspace's rows, 32 rows at a time in parallel, then in order.
__global__ void __launch_bounds__(1024) k_norm_dweight(const float* __restrict__ partial, int nparts, int cols,
                                                       float* __restrict__ dweight) {
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 5
    for (int p = threadIdx.y; p < nparts; p += 32) s += partial[static_cast<int64_t>(p) * cols + c];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    for (int y = 1; y < 32; ++y) s += part[y][threadIdx.x];
    dweight[c] = s;
  }
}

// --------------------------------------------------------------- quantiser

struct QuantArgs {
  const void* x[COCO_MAX_PTRS];
  void* q[COCO_MAX_PTRS];
  float* scales[COCO_MAX_PTRS];
  int64_t rows;
  int32_t nchunks, nblocks;
};

// One scale per row and 128 columns. Grid x: steps of blockDim chunk positions, a row's positions padded to
// whole blocks of 16 so that a block's lanes are neighbours; grid y: tensors.
template <typename T>
__global__ void __launch_bounds__(256) k_quantize_rows(const __grid_constant__ QuantArgs a) {
  const void* x = a.x[blockIdx.y];
  uint2* q = static_cast<uint2*>(a.q[blockIdx.y]);
  float* scales = a.scales[blockIdx.y];
  const int64_t padded = static_cast<int64_t>(a.nblocks) * kBlockLanes;
  const int64_t total = a.rows * padded;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  // (uniform trip count: every lane of a warp takes part in the shuffles)
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * blockDim.x; base < total; base += step) {
    const int64_t p = base + threadIdx.x;
    const int64_t row = total <= 0x7fffffff ? static_cast<uint32_t>(p) / static_cast<uint32_t>(padded) : p / padded;
    const int c = static_cast<int>(p - row * padded);
    const bool mine = p < total && c < a.nchunks;
    float f[kChunk];
    float m = 0.0f;
    if (mine) {
      Chunk<T> v;
      v.load(x, row * a.nchunks + c);
      v.get(f);
      m = chunk_amax(f);
    }
#pragma unroll
    for (int s = kBlockLanes / 2; s; s >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
    if (mine) {
      const float s = scale_of(m);
      q[row * a.nchunks + c] = to_e4m3(f, s);
      if (c % kBlockLanes == 0) scales[row * a.nblocks + c / kBlockLanes] = s;
    }
  }
}

// One scale per 128 rows x 128 columns: a block holds the tile in registers (kTileThreads threads, kTileChunks
// chunks each, those that 64 registers do not hold in local memory: 72 to 80 bytes, fp32 240) between its maximum and
// its rounding. 8192 x 32768 in bf16: 135 us (5.96 TB/s), bound by HBM, in fp32 295; four blocks of 256 threads an SM
// (512 or 1024 threads a tile: 154 to 217 us). Grid x: tiles, row-major; grid y: tensors.
constexpr int kTileThreads = 256, kTileRows = kTileThreads / kBlockLanes, kTileChunks = 128 / kTileRows;

template <typename T>
__global__ void __launch_bounds__(kTileThreads, 4) k_quantize_tiles(const __grid_constant__ QuantArgs a) {
  __shared__ float red[2][kTileThreads / 32];
  const void* x = a.x[blockIdx.y];
  uint2* q = static_cast<uint2*>(a.q[blockIdx.y]);
  float* scales = a.scales[blockIdx.y];
  const int64_t tiles = ((a.rows + 127) / 128) * a.nblocks;
  int turn = 0;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, turn ^= 1) {
    const int64_t tr = tile / a.nblocks;
    const int c = static_cast<int>(tile - tr * a.nblocks) * kBlockLanes + (threadIdx.x & (kBlockLanes - 1));
    const int64_t r0 = tr * 128 + threadIdx.x / kBlockLanes;
    Chunk<T> v[kTileChunks];
#pragma unroll
    for (int i = 0; i < kTileChunks; ++i) {
      if (c < a.nchunks && r0 + kTileRows * i < a.rows) v[i].load(x, (r0 + kTileRows * i) * a.nchunks + c);
      else v[i].zero();
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < kTileChunks; ++i) {
      float f[kChunk];
      v[i].get(f);
      m = max_nan(m, chunk_amax(f));
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
    if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTileThreads / 32; ++i) m = max_nan(m, red[turn][i]);
    const float s = scale_of(m);
#pragma unroll
    for (int i = 0; i < kTileChunks; ++i) {
      if (c < a.nchunks && r0 + kTileRows * i < a.rows) {
        float f[kChunk];
        v[i].get(f);
        q[(r0 + kTileRows * i) * a.nchunks + c] = to_e4m3(f, s);
      }
    }
    if (threadIdx.x == 0) scales[tile] = s;
  }
}

// --------------------------------------------------------------- launchers

template <typename T, int NR, int VPT>
cudaError_t norm_go(const NormArgs& a, bool fp8, dim3 grid, int threads, cudaStream_t s) {
  if (fp8) k_allreduce_rmsnorm<T, NR, VPT, true><<<grid, threads, 0, s>>>(a);
  else k_allreduce_rmsnorm<T, NR, VPT, false><<<grid, threads, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int NR>
cudaError_t norm_vpt(const NormArgs& a, bool fp8, const RowShape& r, dim3 grid, cudaStream_t s) {
  switch (r.vpt) {
    case 1: return norm_go<T, NR, 1>(a, fp8, grid, r.threads, s);
    case 2: return norm_go<T, NR, 2>(a, fp8, grid, r.threads, s);
    case 4: return norm_go<T, NR, 4>(a, fp8, grid, r.threads, s);
    default: return norm_go<T, NR, 8>(a, fp8, grid, r.threads, s);
  }
}

template <typename T>
cudaError_t norm_ranks(const NormArgs& a, bool fp8, const RowShape& r, dim3 grid, cudaStream_t s) {
  switch (a.nranks) {
    case 1: return norm_vpt<T, 1>(a, fp8, r, grid, s);
    case 8: return norm_vpt<T, 8>(a, fp8, r, grid, s);
    default: return norm_vpt<T, 0>(a, fp8, r, grid, s);
  }
}

template <typename T, int NR, int VPT, int THREADS>
cudaError_t bwd_go(const NormBwdArgs& a, int groups, int* parts, cudaStream_t s) {
  using S = BwdShape<T, VPT, THREADS>;
  // (as many blocks as stay on the device, each with at most its share of the rows)
  const int rpb = THREADS >> a.tpr_log2;
  int64_t most = sm_count() * S::BLOCKS < kNormMaxParts ? sm_count() * S::BLOCKS : kNormMaxParts;
  most = most / groups > 0 ? most / groups : 1;
  const int64_t want = (a.rows + rpb - 1) / rpb;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), groups);
  const int smem = S::WIDE ? a.nchunks * kChunk * 4 : 0;
  if constexpr (S::WIDE) {
    // The leave for dynamic shared memory is the process's: once per device, for the widest row that comes here, so
    // that no call can take another's. (Any size needs it: with the kernel's own arrays, rows just under 48 KB pass
    // what needs none.)
    static std::atomic<bool> leave[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !leave[dev].load(std::memory_order_acquire)) {
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&k_rmsnorm_backward<T, NR, VPT, THREADS>),
                               cudaFuncAttributeMaxDynamicSharedMemorySize, VPT * THREADS * kChunk * 4);
      if (e != cudaSuccess) return e;
      if (dev >= 0 && dev < 64) leave[dev].store(true, std::memory_order_release);
    }
  }
  *parts = static_cast<int>(grid.x) * groups;
  k_rmsnorm_backward<T, NR, VPT, THREADS><<<grid, THREADS, smem, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int NR>
cudaError_t bwd_vpt(NormBwdArgs& a, int groups, int* parts, cudaStream_t s) {
  const RowShape r = row_shape(a.nchunks);
  a.tpr_log2 = r.tpr_log2;
  if constexpr (sizeof(T) == 2) {
    if (a.nchunks > 1024) {
      a.tpr_log2 = 10;
      return a.nchunks <= 2048 ? bwd_go<T, NR, 2, 1024>(a, groups, parts, s)
                               : bwd_go<T, NR, 4, 1024>(a, groups, parts, s);
    }
    return r.vpt == 1 ? bwd_go<T, NR, 1, 512>(a, groups, parts, s) : bwd_go<T, NR, 2, 512>(a, groups, parts, s);
  } else {
    switch (r.vpt) {
      case 1: return bwd_go<T, NR, 1, 512>(a, groups, parts, s);
      case 2: return bwd_go<T, NR, 2, 512>(a, groups, parts, s);
      case 4: return bwd_go<T, NR, 4, 512>(a, groups, parts, s);
      default: return bwd_go<T, NR, 8, 512>(a, groups, parts, s);
    }
  }
}

template <typename T>
cudaError_t bwd_ranks(NormBwdArgs& a, int groups, int* parts, cudaStream_t s) {
  switch (a.nranks) {
    case 1: return bwd_vpt<T, 1>(a, groups, parts, s);
    case 8: return bwd_vpt<T, 8>(a, groups, parts, s);
    default: return bwd_vpt<T, 0>(a, groups, parts, s);
  }
}

}  // namespace

cudaError_t launch_allreduce_rmsnorm(const NormLaunch& L, cudaStream_t s) {
  NormArgs a;
  a.t = L.t;
  a.rows = L.rows;
  a.nranks = L.nranks;
  a.cols = L.cols;
  a.nchunks = L.cols / kChunk;
  a.nblocks = (L.cols + 127) / 128;
  a.eps = L.eps;
  a.weight = L.weight;
  a.rstd = L.rstd;
  const RowShape r = row_shape(a.nchunks);
  a.tpr_log2 = r.tpr_log2;
  const int64_t blocks = (L.rows + r.rpb - 1) / r.rpb;
  const dim3 grid(static_cast<unsigned>(blocks < (1 << 30) ? blocks : (1 << 30)), L.ngroups);
  switch (L.dtype) {
    case COCO_F32: return norm_ranks<float>(a, L.fp8, r, grid, s);
    case COCO_F16: return norm_ranks<__half>(a, L.fp8, r, grid, s);
    default: return norm_ranks<__nv_bfloat16>(a, L.fp8, r, grid, s);
  }
}

int64_t norm_backward_parts(int64_t total_rows) { return total_rows < kNormMaxParts ? total_rows : kNormMaxParts; }

cudaError_t launch_rmsnorm_backward(const NormBwdLaunch& L, cudaStream_t s) {
  if (L.rows == 0) return cudaMemsetAsync(L.dweight, 0, static_cast<size_t>(L.cols) * 4, s);
  NormBwdArgs a;
  for (int i = 0; i < COCO_MAX_PTRS; ++i) {
    a.in[i] = L.in[i];
    a.dhidden[i] = L.dhidden[i];
    a.hidden[i] = L.hidden[i];
    a.dx[i] = L.dx[i];
    a.ndx[i] = L.ndx[i];
  }
  a.rows = L.rows;
  a.nranks = L.nranks;
  a.cols = L.cols;
  a.nchunks = L.cols / kChunk;
  a.weight = L.weight;
  a.rstd = L.rstd;
  a.partial = L.partial;
  int parts = 0;
  cudaError_t e;
  switch (L.dtype) {
    case COCO_F32: e = bwd_ranks<float>(a, L.ngroups, &parts, s); break;
    case COCO_F16: e = bwd_ranks<__half>(a, L.ngroups, &parts, s); break;
    default: e = bwd_ranks<__nv_bfloat16>(a, L.ngroups, &parts, s); break;
  }
  if (e != cudaSuccess) return e;
  k_norm_dweight<<<(L.cols + 31) / 32, dim3(32, 32), 0, s>>>(L.partial, parts, L.cols,
                                                            L.dweight);
  count_launch();
  return cudaGetLastError();
}

cudaError_t launch_quantize_fp8(const QuantLaunch& L, cudaStream_t s) {
  QuantArgs a;
  for (int i = 0; i < COCO_MAX_PTRS; ++i) {
    a.x[i] = L.x[i];
    a.q[i] = L.q[i];
    a.scales[i] = L.scales[i];
  }
  a.rows = L.rows;
  a.nchunks = L.cols / kChunk;
  a.nblocks = (L.cols + 127) / 128;
  const int64_t most = 1 << 30;
  if (L.block_rows == 1) {
    const int64_t blocks = (L.rows * a.nblocks * kBlockLanes + 255) / 256;
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most), L.ntensors);
    switch (L.dtype) {
      case COCO_F32: k_quantize_rows<float><<<grid, 256, 0, s>>>(a); break;
      case COCO_F16: k_quantize_rows<__half><<<grid, 256, 0, s>>>(a); break;
      default: k_quantize_rows<__nv_bfloat16><<<grid, 256, 0, s>>>(a); break;
    }
  } else {
    const int64_t blocks = ((L.rows + 127) / 128) * a.nblocks;
    const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most), L.ntensors);
    switch (L.dtype) {
      case COCO_F32: k_quantize_tiles<float><<<grid, kTileThreads, 0, s>>>(a); break;
      case COCO_F16: k_quantize_tiles<__half><<<grid, kTileThreads, 0, s>>>(a); break;
      default: k_quantize_tiles<__nv_bfloat16><<<grid, kTileThreads, 0, s>>>(a); break;
    }
  }
  count_launch();
  return cudaGetLastError();
}

}  // namespace coco
