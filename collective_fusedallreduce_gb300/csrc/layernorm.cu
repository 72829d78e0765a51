// The layer norm that follows a tensor-parallel layer's AllReduce, and its gradient:
//
//   h = sum_r partial_r + residual,  m = mean(h),  v = mean((h - m)^2),
//   y = (h - m) * rsqrt(v + eps) * w + b
//   (Ba, Kiros and Hinton, "Layer Normalization", 2016),
//
// with y stored in the stream's type or as e4m3 values with one scale per row and
// 128 columns. Rows are held as in norm.cu, and HBM bounds the same passes.
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

#include <atomic>

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
  float eps;
  const void* weight;
  const void* bias;
  float* mean;
  float* rstd;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// The elements of a row that warp `w` of its threads holds.
__device__ __forceinline__ int warp_columns(int w, int tpr, int nchunks, int vpt) {
  int n = 0;
  for (int i = 0; i < vpt; ++i) {
    const int left = nchunks - (i * tpr + 32 * w);
    n += left < 0 ? 0 : left > 32 ? 32 : left;
  }
  return n * kChunk;
}

// Grid x: rows (blockDim / tpr a block), grid y: groups.
template <typename T, int NR, int VPT, bool FP8>
__global__ void __launch_bounds__(512, VPT == 1 && NR > 0 && sizeof(T) == 2 ? 3 : 1)
    k_allreduce_layernorm(const __grid_constant__ LayerNormArgs a) {
  __shared__ float2 red[2][16];
  __shared__ float counts[16];  // the elements that each warp of a row holds
  const int g = blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int t = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = blockDim.x >> a.tpr_log2;
  const int warp = threadIdx.x >> 5, warps = tpr >> 5, first = warp & ~(warps - 1);
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
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.rows;
       base += static_cast<int64_t>(gridDim.x) * rpb, turn ^= 1) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    const int64_t c0 = row * a.nchunks;
    float h[VPT][kChunk];
    float s = 0.0f;
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
        for (int j = 0; j < kChunk; ++j) s += h[i][j];
      } else {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) h[i][j] = 0.0f;
      }
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
      // (the joint mean as warp 0's and a correction, which leaves a mean far from zero its last bits)
      const float m0 = red[turn][first].x;
      float m = 0.0f;
      for (int i = 1; i < filled; ++i) m = fmaf(red[turn][first + i].x - m0, counts[i], m);
      mean = fmaf(m, inv_cols, m0);
      q = 0.0f;
      for (int i = 0; i < filled; ++i) {
        const float2 p = red[turn][first + i];
        const float d = p.x - mean;
        q += fmaf(d * d, counts[i], p.y);
      }
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

// ---------------------------------------------------------------- backward
//
// With xhat = (h - m) * rstd and g = dy * w (dy: the sum of the ranks' gradients):
//   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)) + dhidden,
//   dw = sum over rows of dy * xhat,  db = sum over rows of dy.
// Blocks walk rows; every thread keeps the sums of its own columns over its rows (in shared memory), the block's
// rows are joined at the end, and the blocks' sums go to the workspace, which k_layernorm_dweight adds in block order: no
// atomics, so repeated calls give the same bits.

struct LayerNormBwdArgs {
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
  const float* mean;
  const float* rstd;
  float* partial;  // [gridDim.y * gridDim.x][2][cols]
};

__device__ __forceinline__ float2 row_sum2(float2 v, int tpr, float2 (*red)[16], int turn) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5, warps = tpr >> 5;
  if ((threadIdx.x & 31) == 0) red[turn][warp] = v;
  __syncthreads();
  const int first = warp & ~(warps - 1);
  float2 s = red[turn][first];
  for (int i = 1; i < warps; ++i) {
    s.x += red[turn][first + i].x;
    s.y += red[turn][first + i].y;
  }
  return s;
}

constexpr int kBwdThreads = 512;

template <typename T, int NR, int VPT>
__global__ void __launch_bounds__(kBwdThreads) k_layernorm_backward(const __grid_constant__ LayerNormBwdArgs a) {
  // A thread's sums: two vectors of dw and two of db a chunk, in shared memory. Rows of eight chunks a thread would need
  // 256 KB of it: their db lies in the workspace from the start, where L2 holds it.
  constexpr bool FAR = VPT == 8;
  constexpr int PER = FAR ? 2 : 4;
  __shared__ float2 red[2][16];
  extern __shared__ float4 sums[];  // [PER * VPT][threads]
  const int g = blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int t = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = kBwdThreads >> a.tpr_log2;
  const void* const* in = a.in + g * a.nranks;
  const void* dhidden = a.dhidden[g];
  const void* hidden = a.hidden[g];
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  float* out = a.partial + (static_cast<int64_t>(g) * gridDim.x + blockIdx.x) * 2 * a.cols;
  float4* far_db = reinterpret_cast<float4*>(out + a.cols);
#pragma unroll
  for (int i = 0; i < PER * VPT; ++i) sums[i * kBwdThreads + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (FAR)
    for (int c = t; c < a.nchunks; c += tpr) far_db[2 * c] = far_db[2 * c + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.rows;
       base += static_cast<int64_t>(gridDim.x) * rpb, turn ^= 1) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    const int64_t c0 = row * a.nchunks;
    const float mean = live ? a.mean[g * a.rows + row] : 0.0f, rstd = live ? a.rstd[g * a.rows + row] : 0.0f;
    float gr[VPT][kChunk];
    Chunk<T> hv[VPT];
    float2 along = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < a.nchunks) {
        Chunk<T> wv;
        hv[i].load(hidden, c0 + c);
        wv.load_cached(a.weight, c);
        sum_ranks<T, NR>(in, a.nranks, c0 + c, gr[i]);
        float w[kChunk], xh[kChunk], d[kChunk];
        hv[i].get(xh);
        wv.get(w);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) {
          xh[j] = (xh[j] - mean) * rstd;
          d[j] = gr[i][j];
          gr[i][j] *= w[j];
          along.x += gr[i][j];
          along.y = fmaf(gr[i][j], xh[j], along.y);
        }
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          float4& dw = sums[(PER * i + v) * kBwdThreads + threadIdx.x];
          float4& db = FAR ? far_db[2 * c + v] : sums[(PER * i + 2 + v) * kBwdThreads + threadIdx.x];
          float4 u = dw, z = db;
          u.x = fmaf(d[4 * v], xh[4 * v], u.x);
          u.y = fmaf(d[4 * v + 1], xh[4 * v + 1], u.y);
          u.z = fmaf(d[4 * v + 2], xh[4 * v + 2], u.z);
          u.w = fmaf(d[4 * v + 3], xh[4 * v + 3], u.w);
          z.x += d[4 * v];
          z.y += d[4 * v + 1];
          z.z += d[4 * v + 2];
          z.w += d[4 * v + 3];
          dw = u;
          db = z;
        }
      }
    }
    along = row_sum2(along, tpr, red, turn);
    along.x *= inv_cols;
    along.y *= inv_cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < a.nchunks) {
        float f[kChunk], o[kChunk], xh[kChunk];
        Chunk<T> dh;
        if (dhidden) dh.load(dhidden, c0 + c);
        else dh.zero();
        dh.get(f);
        hv[i].get(xh);
#pragma unroll
        for (int j = 0; j < kChunk; ++j)
          o[j] = fmaf(rstd, gr[i][j] - along.x - (xh[j] - mean) * rstd * along.y, f[j]);
        Chunk<T> ov;
        ov.put(o);
        for (int q = 0; q < a.ndx[g]; ++q) ov.store(a.dx[g * a.nranks + q], c0 + c);
      }
    }
  }
  __syncthreads();
  if (slot == 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (c < a.nchunks)
#pragma unroll
        for (int v = 0; v < PER; ++v) {
          float4 u = sums[(PER * i + v) * kBwdThreads + t];
          for (int s = 1; s < rpb; ++s) {
            const float4 z = sums[(PER * i + v) * kBwdThreads + s * tpr + t];
            u.x += z.x;
            u.y += z.y;
            u.z += z.z;
            u.w += z.w;
          }
          __stcs(reinterpret_cast<float4*>(out + (v >> 1) * static_cast<int64_t>(a.cols)) + 2 * c + (v & 1), u);
        }
    }
  }
}

// dweight[c] and dbias[c]: the sums over the workspace's rows, 32 rows at a time in parallel, then in order. Grid y: which.
__global__ void __launch_bounds__(1024) k_layernorm_dweight(const float* __restrict__ partial, int nparts, int cols,
                                                            float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;
  float* out = blockIdx.y ? dbias : dweight;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 5
    for (int p = threadIdx.y; p < nparts; p += 32) s += partial[(2 * static_cast<int64_t>(p) + blockIdx.y) * cols + c];
  }
  part[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    for (int y = 1; y < 32; ++y) s += part[y][threadIdx.x];
    out[c] = s;
  }
}

// --------------------------------------------------------------- launchers

template <typename T, int NR, int VPT>
cudaError_t norm_go(const LayerNormArgs& a, bool fp8, dim3 grid, int threads, cudaStream_t s) {
  if (fp8) k_allreduce_layernorm<T, NR, VPT, true><<<grid, threads, 0, s>>>(a);
  else k_allreduce_layernorm<T, NR, VPT, false><<<grid, threads, 0, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int NR>
cudaError_t norm_vpt(const LayerNormArgs& a, bool fp8, const RowShape& r, dim3 grid, cudaStream_t s) {
  switch (r.vpt) {
    case 1: return norm_go<T, NR, 1>(a, fp8, grid, r.threads, s);
    case 2: return norm_go<T, NR, 2>(a, fp8, grid, r.threads, s);
    case 4: return norm_go<T, NR, 4>(a, fp8, grid, r.threads, s);
    default: return norm_go<T, NR, 8>(a, fp8, grid, r.threads, s);
  }
}

template <typename T>
cudaError_t norm_ranks(const LayerNormArgs& a, bool fp8, const RowShape& r, dim3 grid, cudaStream_t s) {
  switch (a.nranks) {
    case 1: return norm_vpt<T, 1>(a, fp8, r, grid, s);
    case 8: return norm_vpt<T, 8>(a, fp8, r, grid, s);
    default: return norm_vpt<T, 0>(a, fp8, r, grid, s);
  }
}

template <typename T, int NR, int VPT>
cudaError_t bwd_go(const LayerNormBwdArgs& a, int groups, int* parts, cudaStream_t s) {
  const int rpb = kBwdThreads >> a.tpr_log2;
  int64_t most = sm_count() < kNormMaxParts ? sm_count() : kNormMaxParts;
  most = most / groups > 0 ? most / groups : 1;
  const int64_t want = (a.rows + rpb - 1) / rpb;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), groups);
  const int smem = (VPT == 8 ? 2 : 4) * VPT * kBwdThreads * 16;
  // (the leave for dynamic shared memory is the process's: once per device, for what every launch of this kernel takes)
  static std::atomic<bool> leave[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < 64;
  if (!kept || !leave[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&k_layernorm_backward<T, NR, VPT>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (kept) leave[dev].store(true, std::memory_order_release);
  }
  *parts = static_cast<int>(grid.x) * groups;
  k_layernorm_backward<T, NR, VPT><<<grid, kBwdThreads, smem, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T, int NR>
cudaError_t bwd_vpt(LayerNormBwdArgs& a, int groups, int* parts, cudaStream_t s) {
  const RowShape r = row_shape(a.nchunks);
  a.tpr_log2 = r.tpr_log2;
  switch (r.vpt) {
    case 1: return bwd_go<T, NR, 1>(a, groups, parts, s);
    case 2: return bwd_go<T, NR, 2>(a, groups, parts, s);
    case 4: return bwd_go<T, NR, 4>(a, groups, parts, s);
    default: return bwd_go<T, NR, 8>(a, groups, parts, s);
  }
}

template <typename T>
cudaError_t bwd_ranks(LayerNormBwdArgs& a, int groups, int* parts, cudaStream_t s) {
  switch (a.nranks) {
    case 1: return bwd_vpt<T, 1>(a, groups, parts, s);
    case 8: return bwd_vpt<T, 8>(a, groups, parts, s);
    default: return bwd_vpt<T, 0>(a, groups, parts, s);
  }
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

cudaError_t launch_layernorm_backward(const LayerNormBwdLaunch& B, cudaStream_t s) {
  const NormBwdLaunch& L = B.n;
  cudaError_t e;
  if (L.rows == 0) {
    e = cudaMemsetAsync(L.dweight, 0, static_cast<size_t>(L.cols) * 4, s);
    return e != cudaSuccess || !B.dbias ? e : cudaMemsetAsync(B.dbias, 0, static_cast<size_t>(L.cols) * 4, s);
  }
  LayerNormBwdArgs a;
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
  a.mean = B.mean;
  a.rstd = L.rstd;
  a.partial = L.partial;
  int parts = 0;
  switch (L.dtype) {
    case COCO_F32: e = bwd_ranks<float>(a, L.ngroups, &parts, s); break;
    case COCO_F16: e = bwd_ranks<__half>(a, L.ngroups, &parts, s); break;
    default: e = bwd_ranks<__nv_bfloat16>(a, L.ngroups, &parts, s); break;
  }
  if (e != cudaSuccess) return e;
  k_layernorm_dweight<<<dim3((L.cols + 31) / 32, B.dbias ? 2 : 1), dim3(32, 32), 0, s>>>(L.partial, parts, L.cols,
                                                                                      L.dweight, B.dbias);
  count_launch();
  return cudaGetLastError();
}

}  // namespace coco
