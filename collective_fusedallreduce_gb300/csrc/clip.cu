// Clipping by the global norm, over tensors in many separate buffers (the bucket
// tables of the scattered-tensor AllReduce, [CoCoNet] "Breaking the Computation and
// Communication Abstraction Barrier in Distributed Machine Learning Workloads", the
// section on scattered tensors):
//
//   norm = sqrt(sum of x^2 over all buckets),  out = x * min(1, max_norm / norm)
//
// in two launches: the first reads every bucket and leaves one sum of squares a
// block, the second joins those (every block for itself, in block order) and scales.
// With CLIP_SUM the first also sums the ranks' tensors and stores the sums, so the
// AllReduce's one pass gives the norm as well. Bound by HBM: the second pass walks
// backwards, and finds in L2 what the first touched last.

#include <float.h>

#include <type_traits>

#include "internal.h"
#include "rows.h"

namespace coco {
namespace {

constexpr int kHeaderWords = 16;  // of a bucket table
constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBucketChunks = 1024 / kChunk / 32;  // chunks of a bucket that a lane holds

struct ClipArgs {
  const uint32_t* table;
  const uint32_t* out_table;
  int64_t nbuckets;
  int32_t nranks, out_nranks;
  float alpha, max_norm;
  float* norm;
  double* parts;
  int32_t nparts;
};

// One rank's part of a bucket.
struct Bucket {
  char* base;  // its first element
  int32_t len;
  uint32_t code;
};

template <typename T>
__device__ __forceinline__ Bucket bucket_at(const uint32_t* table, int64_t b, int nranks, int rank) {
  const uint32_t* e = table + kHeaderWords + (b * nranks + rank) * 3;
  Bucket r;
  r.code = e[2];
  r.len = static_cast<int>(r.code & 1023u) + 1;
  r.base = reinterpret_cast<char*>((static_cast<uint64_t>(e[1]) << 32) | e[0]) +
           static_cast<int64_t>(r.code >> 10) * 1024 * sizeof(T);
  return r;
}

// The elements of a lane's chunk c of a bucket; past its end zeros.
template <typename T>
__device__ __forceinline__ void load_part(const Bucket& b, int c, float (&f)[kChunk]) {
  if ((c + 1) * kChunk <= b.len) {
    Chunk<T> v;
    v.load(b.base, c);
    v.get(f);
  } else {
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      f[j] = c * kChunk + j < b.len ? static_cast<float>(reinterpret_cast<const T*>(b.base)[c * kChunk + j]) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store_part(const Bucket& b, int c, const float (&f)[kChunk]) {
  if ((c + 1) * kChunk <= b.len) {
    Chunk<T> v;
    v.put(f);
    *reinterpret_cast<Chunk<T>*>(b.base + c * kChunk * sizeof(T)) = v;  // (not a streaming store: it is read again)
  } else {
#pragma unroll
    for (int j = 0; j < kChunk; ++j)
      if (c * kChunk + j < b.len) reinterpret_cast<T*>(b.base)[c * kChunk + j] = static_cast<T>(f[j]);
  }
}

// The squares' sum of a lane's part of a bucket: in fp32, and again in fp64 where that has left fp32's range (past its
// largest number, or so low that squares were lost).
__device__ __forceinline__ double squares(const float (&f)[kBucketChunks][kChunk]) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < kBucketChunks; ++i)
#pragma unroll
    for (int j = 0; j < kChunk; ++j) s = fmaf(f[i][j], f[i][j], s);
  if (s >= 0x1p-80f && s <= FLT_MAX) return s;
  bool any = s != 0.0f;
#pragma unroll
  for (int i = 0; i < kBucketChunks; ++i)
#pragma unroll
    for (int j = 0; j < kChunk; ++j) any |= f[i][j] != 0.0f;
  double d = 0.0;
  if (any) {
#pragma unroll
    for (int i = 0; i < kBucketChunks; ++i)
#pragma unroll
      for (int j = 0; j < kChunk; ++j) d = fma(static_cast<double>(f[i][j]), static_cast<double>(f[i][j]), d);
  }
  return d;
}

// The block's sum, in thread 0 (fp64 units are few: the other threads do not need it).
__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < kWarps; ++i) v += red[i];
  return v;
}

// Whether the tensors of the two tables have bucket b in common. Where they do not, nothing is written and the norm is NaN.
template <typename T, typename U>
__device__ __forceinline__ bool same_bucket(const ClipArgs& a, int64_t b) {
  return a.table == a.out_table ||
         bucket_at<T>(a.table, b, a.nranks, 0).code == bucket_at<U>(a.out_table, b, a.out_nranks, 0).code;
}

// Warps take buckets round-robin (those of every rank with CLIP_LOCAL). With CLIP_SUM the ranks' tensors are added in
// rank order, scaled by alpha, rounded to U and stored to out's rank 0, and it is those values' norm.
template <typename T, typename U, int MODE>
__global__ void __launch_bounds__(kThreads) k_clip_squares(const __grid_constant__ ClipArgs a) {
  __shared__ double red[kWarps];
  const int lane = threadIdx.x & 31;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t items = MODE == CLIP_LOCAL ? a.nbuckets * a.nranks : a.nbuckets;
  double sum = 0.0;
  for (int64_t it = warp; it < items; it += nwarps) {
    const int64_t b = MODE == CLIP_LOCAL ? it / a.nranks : it;
    if (!same_bucket<T, U>(a, b)) {
      sum = __longlong_as_double(0x7ff8000000000000ll);
      continue;
    }
    float f[kBucketChunks][kChunk];
    if constexpr (MODE != CLIP_SUM) {
      const Bucket k = bucket_at<T>(a.table, b, a.nranks, MODE == CLIP_LOCAL ? static_cast<int>(it - b * a.nranks) : 0);
#pragma unroll
      for (int i = 0; i < kBucketChunks; ++i) load_part<T>(k, lane + 32 * i, f[i]);
    } else {
      const Bucket to = bucket_at<U>(a.out_table, b, a.out_nranks, 0);
      for (int r = 0; r < a.nranks; ++r) {
        const Bucket k = bucket_at<T>(a.table, b, a.nranks, r);
#pragma unroll
        for (int i = 0; i < kBucketChunks; ++i) {
          float v[kChunk];
          load_part<T>(k, lane + 32 * i, v);
#pragma unroll
          for (int j = 0; j < kChunk; ++j) f[i][j] = r ? f[i][j] + v[j] : v[j];
        }
      }
#pragma unroll
      for (int i = 0; i < kBucketChunks; ++i) {
#pragma unroll
        for (int j = 0; j < kChunk; ++j) f[i][j] = static_cast<float>(static_cast<U>(f[i][j] * a.alpha));
        store_part<U>(to, lane + 32 * i, f[i]);
      }
    }
    sum += squares(f);
  }
  sum = block_sum(sum, red);
  if (threadIdx.x == 0) a.parts[blockIdx.x] = sum;
}

// Every block joins the sums of squares; block 0 writes the norm. Then out = x * factor, last buckets first; x is the
// ranks' own tensor (CLIP_LOCAL), rank 0's (CLIP_REPLICATED), or out's rank 0 (CLIP_SUM). `in_place`: where the factor is
// 1, the tensors that hold x already are left as they are.
template <typename T, typename U, int MODE>
__global__ void __launch_bounds__(kThreads) k_clip_scale(const __grid_constant__ ClipArgs a, bool in_place) {
  __shared__ double red[kWarps];
  __shared__ float shared_factor;
  const int lane = threadIdx.x & 31;
  double total = 0.0;
  for (int i = threadIdx.x; i < a.nparts; i += kThreads) total += a.parts[i];
  total = block_sum(total, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(total);
    if (blockIdx.x == 0) *a.norm = static_cast<float>(norm);
    shared_factor = norm <= static_cast<double>(a.max_norm) ? 1.0f : static_cast<float>(a.max_norm / norm);
  }
  __syncthreads();
  const float factor = shared_factor;
  const bool keep = factor == 1.0f && (in_place || MODE == CLIP_SUM);
  if (keep && (MODE != CLIP_SUM || a.out_nranks == 1)) return;
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t items = MODE == CLIP_LOCAL ? a.nbuckets * a.nranks : a.nbuckets;
  using X = typename std::conditional<MODE == CLIP_SUM, U, T>::type;
  for (int64_t it = items - 1 - warp; it >= 0; it -= nwarps) {
    const int64_t b = MODE == CLIP_LOCAL ? it / a.nranks : it;
    if (!same_bucket<T, U>(a, b)) continue;
    const int r0 = MODE == CLIP_LOCAL ? static_cast<int>(it - b * a.nranks) : 0;
    const Bucket from = MODE == CLIP_SUM ? bucket_at<X>(a.out_table, b, a.out_nranks, 0)
                                         : bucket_at<X>(a.table, b, a.nranks, r0);
    const int first = MODE == CLIP_LOCAL ? r0 : MODE == CLIP_SUM && keep ? 1 : 0;
    const int last = MODE == CLIP_LOCAL ? r0 + 1 : a.out_nranks;
    float f[kBucketChunks][kChunk];
#pragma unroll
    for (int i = 0; i < kBucketChunks; ++i) {
      load_part<X>(from, lane + 32 * i, f[i]);
#pragma unroll
      for (int j = 0; j < kChunk; ++j) f[i][j] *= factor;
    }
    for (int r = first; r < last; ++r) {
      const Bucket to = bucket_at<U>(a.out_table, b, a.out_nranks, r);
#pragma unroll
      for (int i = 0; i < kBucketChunks; ++i) store_part<U>(to, lane + 32 * i, f[i]);
    }
  }
}

template <typename T, typename U, int MODE>
cudaError_t clip_go(const ClipLaunch& L, cudaStream_t s) {
  ClipArgs a;
  a.table = static_cast<const uint32_t*>(L.table);
  a.out_table = static_cast<const uint32_t*>(L.out_table);
  a.nbuckets = L.nbuckets;
  a.nranks = L.nranks;
  a.out_nranks = L.out_nranks;
  a.alpha = L.alpha;
  a.max_norm = L.max_norm;
  a.norm = L.norm;
  a.parts = L.parts;
  const int64_t items = MODE == CLIP_LOCAL ? L.nbuckets * L.nranks : L.nbuckets;
  const int64_t want = items ? (items + kWarps - 1) / kWarps : 1;
  int64_t most = static_cast<int64_t>(sm_count()) * 4;
  most = most < kClipMaxParts ? most : kClipMaxParts;
  a.nparts = static_cast<int32_t>(want < most ? want : most);
  k_clip_squares<T, U, MODE><<<a.nparts, kThreads, 0, s>>>(a);
  count_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  k_clip_scale<T, U, MODE><<<a.nparts, kThreads, 0, s>>>(a, L.table == L.out_table);
  count_launch();
  return cudaGetLastError();
}

template <typename T, typename U>
cudaError_t clip_mode(const ClipLaunch& L, cudaStream_t s) {
  switch (L.mode) {
    case CLIP_LOCAL: return clip_go<T, U, CLIP_LOCAL>(L, s);
    case CLIP_REPLICATED: return clip_go<T, U, CLIP_REPLICATED>(L, s);
    default: return clip_go<T, U, CLIP_SUM>(L, s);
  }
}

template <typename T>
cudaError_t clip_out(const ClipLaunch& L, cudaStream_t s) {
  switch (L.out_dtype) {
    case COCO_F32: return clip_mode<T, float>(L, s);
    case COCO_F16: return clip_mode<T, __half>(L, s);
    default: return clip_mode<T, __nv_bfloat16>(L, s);
  }
}

}  // namespace

cudaError_t launch_scattered_clip(const ClipLaunch& L, cudaStream_t s) {
  switch (L.dtype) {
    case COCO_F32: return clip_out<float>(L, s);
    case COCO_F16: return clip_out<__half>(L, s);
    default: return clip_out<__nv_bfloat16>(L, s);
  }
}

}  // namespace coco
