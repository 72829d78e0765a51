// The gradient of the layer norm that follows an AllReduce. With xhat = (h - m) * rstd
// and g = dy * w (dy: the sum of the ranks' gradients):
//
//   dx = rstd * (g - mean(g) - xhat * mean(g * xhat)) + dhidden,
//   dw = sum over rows of dy * xhat,  db = sum over rows of dy.
//
// Bound by HBM: N + 2 rows are read and one is written. Blocks walk rows; every
// thread keeps the sums of its own columns over its rows (in shared memory), the
// block's rows are joined at the end, and the blocks' sums go to the workspace,
// which k_layernorm_dweight adds in block order: no atomics, so repeated calls
// give the same bits.
//
// Measured, from a graph: 8192 x 4096 fp16 on 8 ranks 118 us (6.3 TB/s; some 6 of
// them the second kernel, which is placed early), 777 x 8192 bf16 on 2 26.1 (two or three
// rows a block, whose waits follow one another), 8192 x 4096 bf16 on 3 67.4, 4096 x 16384
// on one 117, 2048 x 32768 267 (db through L2); fp32, 8192 x 4096, on one 101 (5.3 TB/s),
// on 4 199 (4.7), on 8 233 (6.3). dw and db in registers instead of shared
// memory do not fit two blocks an SM (204 us for the first with one).

#include <atomic>

#include "internal.h"
#include "rows.h"

namespace coco {
namespace {

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

// Two sums over the threads of a row, as row_sum; rows that share a block have a barrier each.
__device__ __forceinline__ float2 row_sum2(float2 v, int tpr, int slot, float2 (*red)[32], int turn) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if (tpr == 32) return v;
  const int warp = threadIdx.x >> 5, warps = tpr >> 5;
  if ((threadIdx.x & 31) == 0) red[turn][warp] = v;
  if (blockDim.x == tpr || blockDim.x > 15 * tpr) __syncthreads();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + slot), "r"(tpr) : "memory");
  // (lane i has warp i's: shuffles again, in place of a loop over the warps)
  const int lane = threadIdx.x & 31, first = warp & ~(warps - 1);
  const float2 s = lane < warps ? red[turn][first + lane] : make_float2(0.0f, 0.0f);
  return make_float2(warp_sum(s.x), warp_sum(s.y));
}

// A thread's own 16 bytes of shared memory, filled from global memory while it does other things.
__device__ __forceinline__ void copy_16(float4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from)
               : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// THREADS and blocks an SM: 16-bit rows of up to 8192 columns have two blocks of 512 threads, wider ones 1024 threads a
// row of two or four chunks; fp32 rows 512 threads, two blocks of one chunk.
template <typename T, int NR, int VPT, int THREADS>
struct BwdShape {
  // A thread's sums: two vectors of dw and two of db a chunk, in shared memory. Rows of 32768 columns would need 256 KB of
  // it: their db lies in the workspace from the start, where L2 holds it.
  static constexpr bool FAR = VPT * THREADS > 2048;
  static constexpr int PER = FAR ? 2 : 4;
  // Operands (the ranks', hidden, dhidden) whose next row is copied to shared memory while this one is summed and stored:
  // all, where a thread has one 16-bit chunk of each and their number is known (8192 x 4096 on two ranks 70.7 -> 63.3 us, on
  // three 76 -> 67.4, on four 81 -> 75.7, on eight 121.4 -> 118). Two chunks a thread lost by it (8192 x 8192 on one rank
  // 114 -> 118), fp32 more (one rank 101 -> 140).
  static constexpr int STAGED = sizeof(T) == 2 && VPT == 1 && NR > 0 ? NR + 2 : 0;
  static constexpr int SMEM = (PER * VPT + STAGED) * THREADS * 16;
  static constexpr int BLOCKS = THREADS == 512 && VPT <= (sizeof(T) == 2 ? 2 : 1) ? 2 : 1;
};

template <typename T, int NR, int VPT, int THREADS>
__global__ void __launch_bounds__(THREADS, BwdShape<T, NR, VPT, THREADS>::BLOCKS)
    k_layernorm_backward(const __grid_constant__ LayerNormBwdArgs a) {
  using S = BwdShape<T, NR, VPT, THREADS>;
  constexpr bool FAR = S::FAR;
  constexpr int PER = S::PER, STAGED = S::STAGED;
  __shared__ float2 red[2][32];
  extern __shared__ float4 sums[];  // [PER * VPT][threads]
  float4* staged = sums + PER * VPT * THREADS + threadIdx.x;  // [STAGED][threads]
  const int g = blockIdx.y;
  const int tpr = 1 << a.tpr_log2;
  const int t = threadIdx.x & (tpr - 1), slot = threadIdx.x >> a.tpr_log2, rpb = THREADS >> a.tpr_log2;
  const void* const* in = a.in + g * a.nranks;
  const void* dhidden = a.dhidden[g];
  const void* hidden = a.hidden[g];
  const float inv_cols = 1.0f / static_cast<float>(a.cols);
  float* out = a.partial + (static_cast<int64_t>(g) * gridDim.x + blockIdx.x) * 2 * a.cols;
  float4* far_db = reinterpret_cast<float4*>(out + a.cols);
#pragma unroll
  for (int i = 0; i < PER * VPT; ++i) sums[i * THREADS + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  if constexpr (FAR)
    for (int c = t; c < a.nchunks; c += tpr) far_db[2 * c] = far_db[2 * c + 1] = make_float4(0.f, 0.f, 0.f, 0.f);
  float next_mean = 0.0f, next_rstd = 0.0f;
  auto stage = [&](int64_t row) {  // (a thread reads what it copied itself: no barrier)
    if (row >= a.rows) return;
    next_mean = a.mean[g * a.rows + row];
    next_rstd = a.rstd[g * a.rows + row];
    if (t >= a.nchunks) return;
#pragma unroll
    for (int r = 0; r < STAGED; ++r) {
      const void* p = r < NR ? in[r] : r == NR ? hidden : dhidden;
      if (p) copy_16(staged + r * THREADS, static_cast<const uint4*>(p) + row * a.nchunks + t);
    }
  };
  auto fetch = [&](int r) {
    Chunk<T> c;
    c.load_cached(staged + r * THREADS, 0);
    return c;
  };
  if constexpr (STAGED > 0) stage(static_cast<int64_t>(blockIdx.x) * rpb + slot);
  int turn = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * rpb; base < a.rows;
       base += static_cast<int64_t>(gridDim.x) * rpb, turn ^= 1) {
    const int64_t row = base + slot;
    const bool live = row < a.rows;
    const int64_t c0 = row * a.nchunks;
    // The block's next row is brought to L2 meanwhile, if not to shared memory: a row's loads, its barrier and its stores do
    // not overlap.
    const int64_t ahead = row + static_cast<int64_t>(gridDim.x) * rpb;
    if (STAGED == 0 && ahead < a.rows && (VPT > 1 || a.nranks < 8))
      for (int i = t; i < a.nranks + 2; i += tpr) {
        const void* p = i < a.nranks ? in[i] : i == a.nranks ? hidden : dhidden;
        const int bytes = a.cols * static_cast<int>(sizeof(T));
        if (p)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(static_cast<const char*>(p) + ahead * bytes),
                       "r"(bytes)
                       : "memory");
      }
    float mean = 0.0f, rstd = 0.0f;
    if constexpr (STAGED > 0) {
      copies_done();
      mean = next_mean;
      rstd = next_rstd;
    } else if (live) {
      mean = a.mean[g * a.rows + row];
      rstd = a.rstd[g * a.rows + row];
    }
    float gr[VPT][kChunk];
    Chunk<T> hv[VPT], dh[1];
    float2 along = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < a.nchunks) {
        Chunk<T> wv;
        wv.load_cached(a.weight, c);
        if constexpr (STAGED > 0) {
          fetch(0).get(gr[0]);
#pragma unroll
          for (int r = 1; r < NR; ++r) {
            float f[kChunk];
            fetch(r).get(f);
#pragma unroll
            for (int j = 0; j < kChunk; ++j) gr[0][j] += f[j];
          }
          hv[0] = fetch(NR);
          dh[0] = fetch(NR + 1);
        } else {
          hv[i].load(hidden, c0 + c);
          if constexpr (VPT == 1)
            if (dhidden) dh[0].load(dhidden, c0 + c);
          sum_all<T, NR>(in, a.nranks, c0 + c, gr[i]);
        }
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
          float4& dw = sums[(PER * i + v) * THREADS + threadIdx.x];
          float4& db = FAR ? far_db[2 * c + v] : sums[(PER * i + 2 + v) * THREADS + threadIdx.x];
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
    if constexpr (STAGED > 0) stage(ahead);  // (its operands are in registers)
    along = row_sum2(along, tpr, slot, red, turn);
    along.x *= inv_cols;
    along.y *= inv_cols;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (live && c < a.nchunks) {
        float f[kChunk], o[kChunk], xh[kChunk];
        if (!dhidden) dh[0].zero();
        else if constexpr (VPT > 1) dh[0].load(dhidden, c0 + c);
        dh[0].get(f);
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
  free_launches();
  __syncthreads();
  if (slot == 0) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = t + i * tpr;
      if (c < a.nchunks)
#pragma unroll
        for (int v = 0; v < PER; ++v) {
          float4 u = sums[(PER * i + v) * THREADS + t];
          for (int s = 1; s < rpb; ++s) {
            const float4 z = sums[(PER * i + v) * THREADS + s * tpr + t];
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
__global__ void __launch_bounds__(1024) k_layernorm_dweight(const float* partial, int nparts, int cols, float* dweight,
                                                            float* dbias) {
  __shared__ float part[32][33];
  await_launches();
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

template <typename T, int NR, int VPT, int THREADS>
cudaError_t bwd_go(const LayerNormBwdArgs& a, int groups, int* parts, cudaStream_t s) {
  using S = BwdShape<T, NR, VPT, THREADS>;
  // (as many blocks as stay on the device, each with at most its share of the rows)
  const int rpb = THREADS >> a.tpr_log2;
  int64_t most = sm_count() * S::BLOCKS < kNormMaxParts ? sm_count() * S::BLOCKS : kNormMaxParts;
  most = most / groups > 0 ? most / groups : 1;
  const int64_t want = (a.rows + rpb - 1) / rpb;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), groups);
  // (the leave for dynamic shared memory is the process's: once per device, for what every launch of this kernel takes)
  static std::atomic<bool> leave[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < 64;
  if (!kept || !leave[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(reinterpret_cast<const void*>(&k_layernorm_backward<T, NR, VPT, THREADS>),
                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    if (kept) leave[dev].store(true, std::memory_order_release);
  }
  *parts = static_cast<int>(grid.x) * groups;
  k_layernorm_backward<T, NR, VPT, THREADS><<<grid, THREADS, S::SMEM, s>>>(a);
  count_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd_shape(LayerNormBwdArgs& a, int groups, int* parts, cudaStream_t s) {
  const RowShape r = row_shape(a.nchunks);
  a.tpr_log2 = r.tpr_log2;
  if constexpr (sizeof(T) == 2) {
    if (r.vpt == 1)
      return with_ranks<1, 2, 3, 4, 8>(a.nranks, [&](auto n) { return bwd_go<T, n.value, 1, 512>(a, groups, parts, s); });
    if (r.vpt == 2)
      return with_ranks<1, 2, 8>(a.nranks, [&](auto n) { return bwd_go<T, n.value, 2, 512>(a, groups, parts, s); });
    a.tpr_log2 = 10;
    if (a.nchunks <= 2048)
      return with_ranks<1>(a.nranks, [&](auto n) { return bwd_go<T, n.value, 2, 1024>(a, groups, parts, s); });
    return bwd_go<T, 0, 4, 1024>(a, groups, parts, s);
  } else {
    switch (r.vpt) {
      case 1: return with_ranks<1, 8>(a.nranks, [&](auto n) { return bwd_go<T, n.value, 1, 512>(a, groups, parts, s); });
      case 2: return with_ranks<1>(a.nranks, [&](auto n) { return bwd_go<T, n.value, 2, 512>(a, groups, parts, s); });
      case 4: return bwd_go<T, 0, 4, 512>(a, groups, parts, s);
      default: return bwd_go<T, 0, 8, 512>(a, groups, parts, s);
    }
  }
}

}  // namespace

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
    case COCO_F32: e = bwd_shape<float>(a, L.ngroups, &parts, s); break;
    case COCO_F16: e = bwd_shape<__half>(a, L.ngroups, &parts, s); break;
    default: e = bwd_shape<__nv_bfloat16>(a, L.ngroups, &parts, s); break;
  }
  if (e != cudaSuccess) return e;
  e = launch_early(k_layernorm_dweight, dim3((L.cols + 31) / 32, B.dbias ? 2 : 1), dim3(32, 32), s, L.partial, parts, L.cols,
                   L.dweight, B.dbias);
  count_launch();
  return e;
}

}  // namespace coco
