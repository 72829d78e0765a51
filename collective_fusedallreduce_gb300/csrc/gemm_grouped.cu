// Products of e4m3 operands with block scales, and products grouped by expert.
// One 64 x 64 output tile per block step, operands staged element by element.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "internal.h"

namespace coco {
namespace {

constexpr int TM = 64, TN = 64, TK = 16;

__device__ float value(const void* p, int64_t i, int dtype) {
  if (dtype == COCO_F16) return __half2float(static_cast<const __half*>(p)[i]);
  if (dtype == COCO_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  __nv_fp8_e4m3 v = static_cast<const __nv_fp8_e4m3*>(p)[i];
  return static_cast<float>(v);
}
__device__ void put(void* p, int64_t i, int dtype, float v) {
  if (dtype == COCO_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == COCO_F16) static_cast<__half*>(p)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// Grid: x = n tiles, y = m tiles of the largest possible expert, z = problem * experts + expert.
__global__ void __launch_bounds__(256) k_grouped_simple(const __grid_constant__ GroupedLaunch L) {
  __shared__ float As[TK][TM + 4], Bs[TK][TN + 4];
  const int p = blockIdx.z / L.experts, e = blockIdx.z % L.experts;
  int r0 = 0, r1 = L.rows;
  if (L.offsets) {
    const int32_t* off = L.offsets + static_cast<int64_t>(p) * (L.experts + 1) + e;
    r0 = min(max(off[0], 0), L.rows);
    r1 = min(max(off[1], r0), L.rows);
  }
  const bool grad = L.form == GRP_GRAD, fp8 = L.in_dtype == COCO_F8E4M3;
  const int M = grad ? L.k : r1 - r0, K = grad ? r1 - r0 : L.k, N = L.n;
  const int kb = (L.k + 127) / 128, nb = (L.n + 127) / 128;
  const int m0 = blockIdx.y * TM, n0 = blockIdx.x * TN;
  if (m0 >= M) return;
  float acc[4][4] = {};
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int k0 = 0; k0 < K; k0 += TK) {
    for (int i = threadIdx.x; i < TM * TK; i += 256) {
      const int kk = i % TK, mm = i / TK, k = k0 + kk, m = m0 + mm;
      float v = 0.0f;
      if (k < K && m < M) {
        if (grad) v = value(L.lhs[p], static_cast<int64_t>(r0 + k) * L.k + m, L.in_dtype);
        else v = value(L.lhs[p], static_cast<int64_t>(r0 + m) * L.k + k, L.in_dtype);
        if (fp8) v *= L.lhs_scales[p][static_cast<int64_t>(r0 + m) * kb + k / 128];
      }
      As[kk][mm] = v;
    }
    for (int i = threadIdx.x; i < TN * TK; i += 256) {
      const int nn = i % TN, kk = i / TN, k = k0 + kk, n = n0 + nn;
      float v = 0.0f;
      if (k < K && n < N) {
        const int64_t eo = static_cast<int64_t>(e) * L.k * L.n;
        if (grad) v = value(L.rhs[p], static_cast<int64_t>(r0 + k) * L.n + n, L.in_dtype);
        else if (L.form == GRP_KN) v = value(L.rhs[p], eo + static_cast<int64_t>(k) * L.n + n, L.in_dtype);
        else v = value(L.rhs[p], eo + static_cast<int64_t>(n) * L.k + k, L.in_dtype);
        if (fp8) {
          const int64_t so = static_cast<int64_t>(e) * kb * nb;
          v *= L.rhs_scales[p][so + (L.form == GRP_KN ? (k / 128) * nb + n / 128 : (n / 128) * kb + k / 128)];
        }
      }
      Bs[kk][nn] = v;
    }
    __syncthreads();
    for (int kk = 0; kk < TK; ++kk)
      for (int i = 0; i < 4; ++i)
        for (int q = 0; q < 4; ++q) acc[i][q] = fmaf(As[kk][ty * 4 + i], Bs[kk][tx * 4 + q], acc[i][q]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int q = 0; q < 4; ++q) {
      const int m = m0 + ty * 4 + i, n = n0 + tx * 4 + q;
      if (m >= M || n >= N) continue;
      const int64_t row = grad ? static_cast<int64_t>(e) * L.k + m : r0 + m;
      put(L.out[p], row * L.n + n, L.out_dtype, acc[i][q]);
    }
}

// Rows of no expert: zeros. Grid: x = steps of elements, y = problem.
__global__ void __launch_bounds__(256) k_grouped_rest(const __grid_constant__ GroupedLaunch L) {
  const int p = blockIdx.y;
  const int32_t* off = L.offsets + static_cast<int64_t>(p) * (L.experts + 1);
  const int64_t head = min(max(off[0], 0), L.rows), tail = min(max(off[L.experts], static_cast<int>(head)), L.rows);
  const int64_t total = (head + L.rows - tail) * L.n;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t at = i < head * L.n ? i : i - head * L.n + tail * L.n;
    put(L.out[p], at, L.out_dtype, 0.0f);
  }
}

}  // namespace

cudaError_t launch_grouped(const GroupedLaunch& L, cudaStream_t s, unsigned int*) {
  const int m = L.form == GRP_GRAD ? L.k : L.rows;
  if (L.experts * L.nprob > 65535 || (m + TM - 1) / TM > 65535) return cudaErrorNotSupported;
  const dim3 grid((L.n + TN - 1) / TN, (m + TM - 1) / TM, L.experts * L.nprob);
  k_grouped_simple<<<grid, 256, 0, s>>>(L);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && L.offsets && L.form != GRP_GRAD) {
    k_grouped_rest<<<dim3(sm_count(), L.nprob), 256, 0, s>>>(L);
    count_launch();
    e = cudaGetLastError();
  }
  return e;
}

}  // namespace coco
